// Attention over every visible entry of the FP4 cache and the sliding window,
// under one softmax: l_j = sm_scale q_h . k_j, o_h = sum_j softmax(l)_j k_j,
// lse_h = log sum_j e^l_j (with the sink's e^z_h in the sum).  Every key is its
// own value, so a key is dequantised once and serves both products.
//
// A (row, key) pair costs 131,072 operations and a key 272 or 288 bytes: the
// products bound it even at one query per sequence.  The keys of all rows form
// one list of 128-key tiles that is cut into equal runs, one per SM, whatever
// the lengths; a row that a cut divides leaves partial outputs (fp32) with their
// running maxima and sums in the workspace, which k_dense_merge joins in order.
#include <algorithm>

#include "csa2_dense_common.cuh"

namespace csa2 {

constexpr int DA_MAX_CTAS = 152;                   // runs; sizes the workspace (one per SM of a GB300)
constexpr uint32_t DA_TMEM_COLS = 512;
constexpr uint32_t DA_S_COL = 256;                 // O^T part mt in columns 64 mt .., S^T in 256 ..
constexpr int DA_KEYS = 128;                       // keys per tile: two pages, or the window
constexpr uint32_t DA_KSLAB = DA_KEYS * 128;       // bytes of a 64-dim slab of the tile
constexpr int DA_PARTS = 4;                        // of 128 dims: what the keys are handed over and freed in
static_assert(DA_KEYS == CSA2_SWA_WINDOW && DA_KEYS == 2 * CSA2_PAGE, "a tile");
// eight warps for the keys, eight for the softmax and the output, and a warpgroup
// for the one that issues the products, which leaves the softmax its registers
constexpr int DA_SWARPS = 8, DA_STHREADS = 32 * DA_SWARPS;
constexpr int DA_WARPS = DN_KWARPS + DA_SWARPS + 4, DA_THREADS = 32 * DA_WARPS;
constexpr int DA_REGS = 96, DA_REGS_SOFTMAX = 120, DA_REGS_ISSUE = 48;          // the keys' warps stay at the launch's
static_assert(DN_KWARPS * DA_REGS + DA_SWARPS * DA_REGS_SOFTMAX + 4 * DA_REGS_ISSUE <= DA_WARPS * DA_REGS &&
                  DA_THREADS * DA_REGS <= 65536,
              "the launch's registers");
// The weights of the value product are held between 2^DA_START (the largest, when
// the reference is set) and 2^DA_PASS (when it has to move), inside f16's range.  One
// below 2^-25 adds nothing to the output, while the sum has it: up to 2^-24 of the
// largest for each entry (2^-23 of a window row's, whose scale's mantissa is in its
// weight).  A long rest far below one entry must not go missing like
// that, so when a segment has had DA_FOLD tiles its references go down by up to 8, and a
// later move ends at DA_LATE: n entries lose at most min(n, 16384) 2^-24 + n 2^-32 of the
// largest, 2^-9.7 for a million.  (Without it 2.5 % of the mass were missing behind a first
// entry that stood 17.5 above 1,048,575 others.)  DA_LATE from the start costs moves: 64 x
// 32,768 entries take 449 us, from the 32nd tile on 432, from the 64th 417, from the 128th 408.
constexpr float DA_START = 0.0f, DA_LATE = 8.0f, DA_PASS = 15.5f;
// The sums' terms, 2^(logit - mu), lie between 2^-(Xk + 14) and 2^(16 - Xk) where they
// count; times 2^DA_SUM that is inside fp32's range for every Xk from DN_XZERO to 127,
// a million of them added up.  The factor is a part of the exponent once a segment has
// had a scale above 2^DA_HIGH; otherwise it comes after, for the exponent would be
// rounded at its size.
constexpr float DA_SUM = 25.0f;
constexpr int DA_HIGH = 64;
// The tensor accumulator drops what is below its last place at every step, always
// towards zero: over 1,048,576 entries of one row and values of one sign the output
// came 0.65 % short, more than a step of bf16.  After every DA_FOLD tiles (1,024 steps)
// the output so far is added, rounded to nearest, to the segment's slot in the
// workspace and the accumulator starts again: 0.003 % short, and 152 such rows take
// 24.9 ms instead of 24.5.
constexpr int DA_FOLD = 128;

// A partial result per head: unnormalised output and sum in units of 2^m, m = mu - DA_SUM;
// the output of a segment's earlier tiles until it ends.
struct DenseSlot {
    float o[CSA2_HEADS][CSA2_HEAD_DIM];
    float m[CSA2_HEADS], l[CSA2_HEADS];
};
// Per run: the row whose first part ends it, that part's slot and the number of
// runs that hold the row (row -1: none).  Later parts are in slots 2 c.
struct DenseHead {
    int64_t row;
    int32_t slot, parts;
};

static inline size_t da_align(size_t x) { return (x + 255) & ~(size_t)255; }

static int64_t dense_runs(const csa2_batch &bt)
{
    const int64_t rows = (int64_t)bt.batch * bt.nq;
    const int64_t tiles = rows * ((bt.max_entries + DA_KEYS - 1) / DA_KEYS + 1);
    return std::min<int64_t>(DA_MAX_CTAS, tiles);
}

size_t dense_attn_workspace_bytes(const csa2_batch &bt)
{
    const int64_t g = dense_runs(bt);
    return da_align((size_t)g * sizeof(DenseHead)) + (size_t)g * 2 * sizeof(DenseSlot);
}

struct DaSmem {
    uint8_t k[DN_SLABS * DA_KSLAB];                // key tile [slab][128 keys][128 B]            128 KB
    uint8_t q[DN_QBYTES];                          // query operand [slab][64 heads][128 B]        64 KB
    uint8_t p[DA_KEYS * 128];                      // weights [128 keys][64 heads] f16             16 KB
    float red[4][CSA2_HEADS];                      // per key quarter: maxima, then sums
    float alpha[CSA2_HEADS];                       // factor of the reference's last step; of the output
    float mu[CSA2_HEADS];                          // the reference at a segment's end
    float held[CSA2_HEADS];                        // the reference of what the segment's slot holds
    float back[CSA2_HEADS];                        // 2^(held - mu): its factor
    float qe[2][CSA2_HEADS];                       // the query's 2^e_h (of the tile that brought it)
    float2 kv[2][DA_KEYS];                         // the keys of tile j in j % 2: (Xk, f), Xk = -inf for no key
    int8_t xtop[2][DN_KWARPS];                     // a key warp's largest Xk of the segment up to tile j (at most 127)
    uint32_t moved[2];                             // heads whose reference has just moved
    int64_t sums[DA_WARPS];
    int64_t total, g0;                             // tiles of all rows; the run's first
    int row0, ti0, n;                              // the run's first row, the tile's place in it, the run's tiles
    // phase j
    uint64_t kbar[DA_PARTS];                       // a part of the keys (the first: and a new row's query) is written
    uint64_t sbar;                                 // the logits are done
    uint64_t pbar;                                 // the weights are written
    uint64_t obar[DA_PARTS];                       // the value product of a part is done: its keys are free
    uint64_t dbar;                                 // everything issued is done
    int abort;
    uint32_t tmem;
};

// log(L 2^M): L's own power of two goes to M's, for the two logarithms may cancel.
__device__ __forceinline__ float dense_lse(float M, float L)
{
    const int k = min((int)(__float_as_uint(L) >> 23) - 127, 126);
    return fmaf(M + (float)k, kLn2, logf(L * exp2i(-k)));
}

// Run i of `runs` equal ones takes the tiles from here up to dense_cut(i + 1).
__device__ __forceinline__ int64_t dense_cut(int64_t total, int64_t runs, int64_t i) { return total * i / runs; }

// This run holds the first part of row r, whose last tile is e: the row's parts.
__device__ __forceinline__ void dense_head(DenseHead *heads, int r, int slot, int64_t e, int64_t total)
{
    const int64_t runs = min((int64_t)gridDim.x, total), run = blockIdx.x;
    int64_t c = run;
    while (dense_cut(total, runs, c + 1) <= e) c++;
    heads[run].slot = slot;
    heads[run].parts = (int)(c - run + 1);
    heads[run].row = r;
}

// The output of the last DA_FOLD tiles (the softmax warps) added to the segment's
// slot -- or put there, the first time.
__device__ __forceinline__ void dense_fold(uint32_t tmem, DenseSlot &slot, bool first)
{
    DaSmem &S = dense_smem<DaSmem>();
    const int sw = (threadIdx.x >> 5) - DN_KWARPS, lane = threadIdx.x & 31, quarter = sw & 3;
#pragma unroll 1
    for (int i = 0; i < 8; i++) {                  // as in dense_output: a thread's own elements
        const int mt = 2 * (sw >> 2) + (i >> 2), h0 = 16 * (i & 3);
        float *at = &slot.o[h0][128 * mt + 32 * quarter + lane];
        uint32_t v[16];
        tc::tmem_ld16(tmem + ((uint32_t)(quarter * 32) << 16) + 64u * (uint32_t)mt + (uint32_t)h0, v);
        tc::tmem_ld_wait(v);
#pragma unroll
        for (int j = 0; j < 16; j++) {
            const float x = __uint_as_float(v[j]) * exp2i((int)(DA_SUM - DN_XOFF));
            at[j * CSA2_HEAD_DIM] = first ? x : fmaf(at[j * CSA2_HEAD_DIM], S.back[h0 + j], x);
        }
    }
}

// A finished segment (the softmax warps; the sums per key quarter are in S.red), with
// what its slot holds if it was folded: to its part's slot, unnormalised, or -- `part`
// false: the row is whole -- with the sink in the sum, the RoPE dims turned back, to
// lse and o.
__device__ __forceinline__ void dense_output(uint32_t tmem, DenseSlot &slot, bool part, bool folded, uint16_t *o, float *lse,
                                          const float *sink, bool rope, const int64_t *pos, const RopeTurns &turns)
{
    DaSmem &S = dense_smem<DaSmem>();
    const int sw = (threadIdx.x >> 5) - DN_KWARPS, lane = threadIdx.x & 31, quarter = sw & 3;
    const int h = (int)threadIdx.x - 32 * DN_KWARPS;
    const uint32_t lane_base = (uint32_t)(quarter * 32) << 16;
    if (h < CSA2_HEADS) {
        float L = (S.red[0][h] + S.red[1][h]) + (S.red[2][h] + S.red[3][h]), M = S.mu[h] - DA_SUM;
        if (part) {
            slot.m[h] = L == 0.0f ? -INFINITY : M;
            slot.l[h] = L;
        } else {
            float fct = 1.0f;
            const float z = sink ? sink[h] * kLog2e : -INFINITY;
            if (z != -INFINITY) {
                if (z > M || L == 0.0f) {
                    fct = L == 0.0f ? 0.0f : exp2f(M - z);
                    L = fmaf(L, fct, 1.0f);
                    M = z;
                } else {
                    L += exp2f(z - M);
                }
            }
            S.alpha[h] = L == 0.0f ? 0.0f : fct / L;               // (NaN stays NaN)
            lse[h] = L == 0.0f ? -INFINITY : dense_lse(M, L);
        }
    }
    tc::named_bar_sync(1, DA_STHREADS);
#pragma unroll 1
    for (int i = 0; i < 8; i++) {                  // parts 2 (sw / 4) and the next, 16 heads at a time
        const int mt = 2 * (sw >> 2) + (i >> 2), h0 = 16 * (i & 3);
        const int dim = 128 * mt + 32 * quarter + lane;
        uint32_t v[16];
        tc::tmem_ld16(tmem + lane_base + 64u * (uint32_t)mt + (uint32_t)h0, v);
        tc::tmem_ld_wait(v);
#pragma unroll
        for (int j = 0; j < 16; j++) v[j] = __float_as_uint(__uint_as_float(v[j]) * exp2i((int)(DA_SUM - DN_XOFF)));
        if (__builtin_expect(folded, 0))
#pragma unroll
            for (int j = 0; j < 16; j++) v[j] = __float_as_uint(fmaf(slot.o[h0 + j][dim], S.back[h0 + j], __uint_as_float(v[j])));
        if (part) {
#pragma unroll
            for (int j = 0; j < 16; j++) slot.o[h0 + j][dim] = __uint_as_float(v[j]);
            continue;
        }
#pragma unroll
        for (int j = 0; j < 16; j++) v[j] = __float_as_uint(__uint_as_float(v[j]) * S.alpha[h0 + j]);
        if (rope && mt == 3 && quarter >= 2) {
            // dims 448 + i (quarter 2) pair with 480 + i (quarter 3); the weights are
            // read: their place holds the exchange
            const int qd = quarter - 2;
            float(*xch)[16][32] = reinterpret_cast<float(*)[16][32]>(S.p);
#pragma unroll
            for (int j = 0; j < 16; j++) xch[qd][j][lane] = __uint_as_float(v[j]);
            tc::named_bar_sync(2, 64);
            float sn, cs;
            rope_sincos(*pos, turns.phi[dim & 31], &sn, &cs);
#pragma unroll
            for (int j = 0; j < 16; j++) {
                const float own = __uint_as_float(v[j]), oth = xch[qd ^ 1][j][lane];
                v[j] = __float_as_uint(qd == 0 ? fmaf(own, cs, oth * sn) : fmaf(own, cs, -oth * sn));
            }
            tc::named_bar_sync(2, 64);
        }
        uint16_t *dst = o + h0 * CSA2_HEAD_DIM + dim;
#pragma unroll
        for (int j = 0; j < 16; j++)
            dst[j * CSA2_HEAD_DIM] = __bfloat16_as_ushort(__float2bfloat16_rn(__uint_as_float(v[j])));
    }
    tc::named_bar_sync(1, DA_STHREADS);            // (the exchange is over before the next weights are written)
}

__device__ __forceinline__ void dense_query(const uint16_t *q, int r, int b, int warp, int lane)
{
    DaSmem &S = dense_smem<DaSmem>();
    dense_load_q(S.q, S.qe[b], q, r, warp, DN_KWARPS, lane);
}

// Part mt of a row's window tile (no rows behind the last, or for a row without one).
// xtop: the segment's largest Xk before.
__device__ __forceinline__ void dense_window_part(const csa2_swa &swa, const DenseRow &R, int b, int mt, int key, int lane,
                                                  int xtop)
{
    DaSmem &S = dense_smem<DaSmem>();
    float top = -INFINITY;
#pragma unroll 1
    for (int h = 0; h < 2; h++) {
        const int64_t tok = R.lo + key + 64 * h;
        if (mt == 0) {
            const float2 v = dense_window_scale(swa, R, tok, lane);
            if ((lane & 3) == 0) S.kv[b][key + 64 * h] = v;
            top = fmaxf(top, v.x);
        }
        dense_store_window<DA_KSLAB>(S.k, swa, R, tok, mt, key + 64 * h, lane);
    }
    if (mt == 0) S.xtop[b][key / DN_WKEYS] = (int8_t)max(xtop, __reduce_max_sync(0xffffffffu, (int)fminf(fmaxf(top, DN_XZERO), 127.0f)));
}

// Eight warps load and dequantise, eight take the softmax, one issues the products.
// One tile of 128 keys (128 KB) fits beside the query.  Its four parts of 128 dims go
// round by themselves: a part is refilled when the value product has read it, and the
// logits over a part begin when it is there, so keys, logits and the value product
// of neighbouring tiles run side by side and only the softmax stands alone.
//
// 64 rows of 32,768 entries: 408 us (floor 145), 7,300 cycles a tile and SM.  The
// products are 3,070 of them (32 + 32 instructions of M = 128, N = 64, 6 KB of shared
// memory each at 126 of its 128 B a cycle); the keys' conversion, which the logits
// wait for part by part, takes 2,400, the softmax 1,800, and moves of the reference
// 700 (7,800 cycles each, one in eleven tiles with these logits).  Tiles of 64 keys, two
// in flight, took as long with logits of M = 64 (64 instructions, 32.5 cycles each,
// for as many keys).
//
// The softmax works with y = logit (base 2) + Xk, the exponent of a key's weight
// times its power of two: 2^(y - mu) is the f16 weight of the value product and
// 2^(y - mu - Xk + DA_SUM) the term of the sum (for a key of zeros, whose weight is 0, any Xk
// will do: one that keeps the term finite).  The reference mu of a head is an integer,
// set from the segment's first tile; weights down to 2^-14 of the largest keep
// f16's 11 bits, smaller ones 2^-24 of it (2^-22 and 2^-32 after the first fold), and mu moves (the output then shrinks by
// a power of two) only when a weight would pass 2^15.5, so most tiles need no
// maximum across lanes, only one barrier that says that nothing passed.
template <bool E4M3>
__global__ void __launch_bounds__(DA_THREADS, 1)
    k_dense_attn(const __grid_constant__ csa2_cache c, const __grid_constant__ csa2_batch bt,
                 const int64_t *__restrict__ evicted, const uint16_t *__restrict__ q, float sm_scale,
                 const __grid_constant__ csa2_swa swa, uint16_t *__restrict__ o, float *__restrict__ lse, int64_t rows,
                 DenseHead *__restrict__ heads, DenseSlot *__restrict__ slots, const __grid_constant__ RopeTurns turns,
                 uint32_t polls)
{
    DaSmem &S = dense_smem<DaSmem>();
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    if (tid == 0) {
        for (int i = 0; i < DA_PARTS; i++) {
            tc::mbar_init(&S.kbar[i], DN_KWARPS);
            tc::mbar_init(&S.obar[i], 1);
        }
        tc::mbar_init(&S.sbar, 1);
        tc::mbar_init(&S.pbar, DA_SWARPS);
        tc::mbar_init(&S.dbar, 1);
        tc::fence_mbar_init();
        S.abort = 0;
    }
    if (warp == 0) tc::tmem_alloc(&S.tmem, DA_TMEM_COLS);
    pdl_wait();
    {
        // ---- this CTA's run of the tile list
        const int64_t per = (rows + DA_THREADS - 1) / DA_THREADS;
        const int64_t r_lo = min((int64_t)tid * per, rows), r_hi = min(r_lo + per, rows);
        int64_t mine = 0, total;
        for (int64_t r = r_lo; r < r_hi; r++) mine += dense_row(bt, evicted, swa, r).tiles;
        int64_t at = block_exclusive_sum(mine, S.sums, &total);
        // no run is empty but those at the end, when there are fewer tiles than CTAs
        const int64_t runs = min((int64_t)gridDim.x, total), run = blockIdx.x;
        const int64_t g0 = run < runs ? dense_cut(total, runs, run) : total;
        const int64_t g1 = run < runs ? dense_cut(total, runs, run + 1) : total;
        if (g0 >= at && g0 < at + mine) {
            for (int64_t r = r_lo; r < r_hi; r++) {
                const int n = dense_row(bt, evicted, swa, r).tiles;
                if (g0 < at + n) {
                    S.row0 = (int)r;
                    S.ti0 = (int)(g0 - at);
                    break;
                }
                at += n;
            }
        }
        if (tid == 0) {
            heads[run].row = -1;
            S.total = total;
            S.g0 = g0;
            S.n = (int)(g1 - g0);
        }
    }
    tc::tc_fence_before();
    __syncthreads();
    tc::tc_fence_after();
    const uint32_t tmem = S.tmem;
    const int n = S.n;

    if (n == 0) {
    } else if (warp >= DN_KWARPS + DA_SWARPS) {
        // ================================================ the products
        set_registers_down<DA_REGS_ISSUE>();
        if (warp == DN_KWARPS + DA_SWARPS) {
            const uint64_t kd = dense_desc(S.k, 16), qd = dense_desc(S.q, 16);
            const uint64_t vd = dense_desc(S.k, DA_KSLAB), pd = dense_desc(S.p, 8192);
            const bool leader = elect_one();
            int r = S.row0, ti = S.ti0, tiles = dense_row(bt, evicted, swa, r).tiles;
            bool ok = true;
            for (int j = 0; j < n && ok; j++) {
                const bool fresh = min(j, ti) % DA_FOLD == 0;          // of a segment, or folded just now
#pragma unroll 1
                for (int part = 0; part < DA_PARTS; part++) {
                    // S^T[128 keys x 64 heads] (+)= K Q^T over a part of the dims
                    if (!(ok = dense_wait(&S.kbar[part], j & 1, &S.abort, polls, c.status))) break;
                    tc::tc_fence_after();
                    if (leader) {
                        constexpr uint32_t IDESC = tc::idesc_f16(DA_KEYS, 64, 0, 0, 0, 0);
                        const uint64_t k0 = kd + (uint32_t)part * (2 * DA_KSLAB / 16), q0 = qd + (uint32_t)part * (2 * DN_QSLAB / 16);
#pragma unroll
                        for (int i = 0; i < 8; i++)
                            tc::mma_f16(tmem + DA_S_COL, k0 + (i >> 2) * (DA_KSLAB / 16) + 2u * (i & 3),
                                        q0 + (i >> 2) * (DN_QSLAB / 16) + 2u * (i & 3), IDESC, part > 0 || i > 0);
                        if (part == DA_PARTS - 1) tc::mma_commit(&S.sbar);
                    }
                    __syncwarp();
                }
                if (!ok) break;
                if (__builtin_expect(++ti == tiles && j + 1 < n, 0)) {
                    ti = 0;
                    tiles = dense_row(bt, evicted, swa, ++r).tiles;
                }
                if (!(ok = dense_wait(&S.pbar, j & 1, &S.abort, polls, c.status))) break;
                tc::tc_fence_after();
                if (leader) {
                    // O^T[128 dims x 64 heads] (+)= V^T P of each part, both operands MN-major
                    constexpr uint32_t IDESC = tc::idesc_f16(128, 64, 0, 0, 1, 1);
#pragma unroll 1
                    for (int mt = 0; mt < DA_PARTS; mt++) {
                        const uint64_t v0 = vd + (uint32_t)mt * (2 * DA_KSLAB / 16);
#pragma unroll
                        for (int kk = 0; kk < DA_KEYS / 16; kk++)
                            tc::mma_f16(tmem + 64u * mt, v0 + 128u * kk, pd + 128u * kk, IDESC, !fresh || kk > 0);
                        tc::mma_commit(&S.obar[mt]);
                    }
                }
                __syncwarp();
            }
            // nothing is in flight when the tensor memory goes
            if (leader) tc::mma_commit(&S.dbar);
            __syncwarp();
            tc::mbar_wait(&S.dbar, 0, 1u << 18);
        }
    } else if (warp < DN_KWARPS) {
        // ================================================ the keys
        const int key = DN_WKEYS * warp + (lane >> 2);          // this quad's keys: key and key + 64
        int r = S.row0, ti = S.ti0, xtop = 0;
        DenseRow R = dense_row(bt, evicted, swa, r);
        auto wait = [&](uint64_t *bar, int phase) { return dense_wait(bar, phase & 1, &S.abort, polls, c.status); };
        // The next tile's codes, on their way while this one is in its softmax (loads are
        // not issued before an arrival at a barrier, which would wait for them).
        uint4 code[2][4], raw[2];
        bool there[2];
        auto fetch = [&]() {
#pragma unroll
            for (int h = 0; h < 2; h++) {
                const int64_t e0 = (int64_t)ti * DA_KEYS + h * CSA2_PAGE;
                there[h] = false;
                raw[h] = make_uint4(0, 0, 0, 0);
#pragma unroll
                for (int mt = 0; mt < 4; mt++) code[h][mt] = raw[h];
                if (e0 >= R.vis) continue;
                const int64_t s = dense_page_slot(c, __ldg(c.block_table + (int64_t)R.b * c.max_pages + (e0 >> 6)), warp == 0 ? lane : 1);
                there[h] = s >= 0 && e0 + key < R.vis;
                if (!there[h]) continue;
#pragma unroll
                for (int mt = 0; mt < 4; mt++) code[h][mt] = dense_codes(c, s + key, mt, lane);
                raw[h] = dense_scales<E4M3>(c, s + key, lane);
            }
        };
        fetch();
        for (int j = 0; j < n; j++) {
            const uint32_t b = j & 1;
            const bool entries = (int64_t)ti * DA_KEYS < R.vis;
            if (__builtin_expect(j == 0 || ti == 0, 0)) {
                if (j > 0 && !wait(&S.sbar, j - 1)) break;     // the products have read the query before
                dense_query(q, r, b, warp, lane);
            }
            uint2 sc[2];
            int xk[2];
#pragma unroll
            for (int h = 0; h < 2; h++) {
                sc[h] = dense_pack_scales<E4M3>(raw[h], lane);
                bool zero;
                xk[h] = dense_exponent<E4M3>(code[h], sc[h], &zero);
                if (E4M3) zero = dense_zero_codes(code[h]);
                if (entries && (lane & 3) == 0)
                    S.kv[b][key + 64 * h] = !there[h] ? make_float2(-INFINITY, 0.0f) : zero ? make_float2(DN_XZERO, 0.0f) : make_float2((float)xk[h], 1.0f);
            }
            if (j == 0 || ti == 0) xtop = (int)DN_XZERO;
            if (entries) {
                xtop = max(xtop, E4M3 ? xk[0] : __reduce_max_sync(0xffffffffu, min(max(xk[0], xk[1]), 127)));
                S.xtop[b][warp] = (int8_t)xtop;
            }
            bool ok = true;
#pragma unroll
            for (int mt = 0; mt < DA_PARTS; mt++) {
                // a part's place is free when the value product of the tile before has read it
                if (j > 0 && ok) ok = wait(&S.obar[mt], j - 1);
                if (!ok) break;
                if (__builtin_expect(entries, 1)) {
#pragma unroll
                    for (int h = 0; h < 2; h++)
                        dense_store<E4M3, DA_KSLAB>(S.k, code[h][mt], sc[h], xk[h], there[h], mt, mt, key + 64 * h, lane);
                } else {
                    dense_window_part(swa, R, b, mt, key, lane, xtop);
                }
                tc::fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(&S.kbar[mt]);
            }
            if (!ok) break;
            if (j + 1 < n) {
                if (__builtin_expect(++ti == R.tiles, 0)) {
                    ti = 0;
                    R = dense_row(bt, evicted, swa, ++r);
                }
                fetch();
            }
        }
    } else {
        // ================================================ softmax and output
        set_registers_up<DA_REGS_SOFTMAX>();
        const int sw = warp - DN_KWARPS, quarter = sw & 3;
        const uint32_t lane_base = (uint32_t)(quarter * 32) << 16;              // tensor-memory lane quarter of this warp
        const int h32 = 32 * (sw >> 2);
        const int key = 32 * quarter + (lane >> 2);                             // this thread's keys: key + 8 u (u < 4)
        const int hd = h32 + 2 * (lane & 3);                                    // its heads: hd + 8 i + e (i < 4, e < 2)
        const float scale = sm_scale * kLog2e;
        int r = S.row0, ti = S.ti0, tiles = dense_row(bt, evicted, swa, r).tiles;
        bool owned = ti == 0;                      // this run holds the row's first tile
        bool seen = false;                         // the segment has had a key with a weight
        float a[8], mu[8], l[8];                   // per head: factor of a product, reference, sum
        for (int j = 0; j < n; j++) {
            const uint32_t b = j & 1, ph = j & 1;
            const bool first = j == 0 || ti == 0, last = j == n - 1 || ti == tiles - 1;
            // the keys' part of the arithmetic, while the logits are on their way
            bool ok = dense_wait(&S.kbar[0], ph, &S.abort, polls, c.status);
            if (__builtin_expect(first, 0)) {
                seen = false;
#pragma unroll
                for (int i = 0; i < 8; i++) {
                    a[i] = S.qe[b][hd + 8 * (i >> 1) + (i & 1)] * scale;
                    mu[i] = l[i] = 0.0f;
                }
            }
            // Of each key: its exponent, the factor of its products, and f.
            const int at = min(j, ti);             // the tile's place in its segment
            float kx[4], kf[4], ky[4];
            const uint2 xt = *reinterpret_cast<const uint2 *>(S.xtop[b]);       // eight bytes
            const uint32_t xt4 = __vmaxs4(xt.x, xt.y);
            const bool high = __vcmpgts4(xt4, 0x01010101u * DA_HIGH) != 0;
#pragma unroll
            for (int u = 0; u < 4; u++) {
                const float2 kv = S.kv[b][key + 8 * u];
                const bool none = kv.x == -INFINITY;
                const int xi = none ? 0 : (int)kv.x;
                kx[u] = kv.x;
                ky[u] = kv.y;
                kf[u] = none ? 0.0f : exp2i(xi - (int)DN_XOFF) * kv.y;
            }
            ok = dense_wait(&S.sbar, ph, &S.abort, polls, c.status) && ok;
            tc::tc_fence_after();
            bool pass = !seen;
            float x[32];                           // y - mu: key u of head i at 16 (u / 2) + 4 (i / 2) + 2 (u % 2) + i % 2
#pragma unroll
            for (int w = 0; w < 2; w++) {
                uint32_t v[16];
                tmem_ld_16x32(tmem + DA_S_COL + lane_base + ((uint32_t)(16 * w) << 16) + (uint32_t)h32, v);
                tc::tmem_ld_wait(v);
                float top = -INFINITY;
#pragma unroll
                for (int at = 0; at < 16; at += 2) {
                    const int u = (at >> 1) & 1, i = 2 * (at >> 2), k = 2 * w + u;
                    const float2 y = f32x2_fma(make_float2(__uint_as_float(v[at]), __uint_as_float(v[at + 1])),
                                               f32x2_mul(make_float2(a[i], a[i + 1]), make_float2(kf[k], kf[k])),
                                               f32x2_sub(make_float2(kx[k], kx[k]), make_float2(mu[i], mu[i + 1])));
                    x[16 * w + at] = y.x;
                    x[16 * w + at + 1] = y.y;
                    top = fmaxf(top, fmaxf(y.x, y.y));
                }
                pass = pass || top > DA_PASS;
            }
            if (__builtin_expect(named_bar_or(1, DA_STHREADS, pass || !ok), 0)) {
                // the earlier value products are done before their output shrinks
                if (!first) ok = dense_wait(&S.obar[DA_PARTS - 1], ph ^ 1, &S.abort, polls, c.status) && ok;
                if (named_bar_or(1, DA_STHREADS, !ok)) break;
                tc::tc_fence_after();
                float mx[8];
#pragma unroll
                for (int i = 0; i < 8; i++) {
                    const int at = 4 * (i >> 1) + (i & 1);
                    mx[i] = fmaxf(fmaxf(x[at], x[at + 2]), fmaxf(x[at + 16], x[at + 18]));
#pragma unroll
                    for (int w = 4; w < 32; w <<= 1) mx[i] = fmaxf(mx[i], __shfl_xor_sync(0xffffffffu, mx[i], w));
                    if (lane < 4) S.red[quarter][hd + 8 * (i >> 1) + (i & 1)] = mx[i];
                }
                if (sw == 0 && lane < 2) S.moved[lane] = 0;
                tc::named_bar_sync(1, DA_STHREADS);
#pragma unroll
                for (int i = 0; i < 8; i++) {
                    const int h = hd + 8 * (i >> 1) + (i & 1);
                    const float m = fmaxf(fmaxf(S.red[0][h], S.red[1][h]), fmaxf(S.red[2][h], S.red[3][h]));
                    // (with the head that passed move all that have come near: 9 us less for 64
                    // x 32,768 than with those above 2^7.5 alone, for there are fewer moves to come)
                    const float start = seen && at >= DA_FOLD ? DA_LATE : DA_START;
                    const bool up = seen ? m > start + 1.5f : m > -INFINITY;
                    const float d = up ? ceilf(m) - start : 0.0f;
                    const float f = exp2_approx(fminf(-d, 120.0f));             // (more only for sums of nothing)
                    mx[i] = m;
                    mu[i] += d;
                    // (in two steps: a sum of small scales may be 2^93 where 2^-d is 2^-195)
                    const float d1 = truncf(0.5f * d);
                    if (!first) l[i] = l[i] * exp2_approx(fminf(-d1, 60.0f)) * exp2_approx(fminf(d1 - d, 60.0f));
#pragma unroll
                    for (int u = 0; u < 4; u++) x[16 * (u >> 1) + 4 * (i >> 1) + 2 * (u & 1) + (i & 1)] -= d;
                    if (quarter == 0 && lane < 4) {
                        S.alpha[h] = f;
                        if (d != 0.0f) atomicOr(&S.moved[h >> 5], 1u << (h & 31));
                    }
                }
#pragma unroll
                for (int i = 0; i < 8; i++) seen = seen || mx[i] > -INFINITY;          // (a NaN head's are all -inf)
                if (!first) {
                    tc::named_bar_sync(1, DA_STHREADS);
#pragma unroll 1
                    for (int i = 0; i < 8; i++) {  // parts 2 (sw / 4) and the next, 16 heads at a time
                        if (!((S.moved[(i >> 1) & 1] >> (16 * (i & 1))) & 0xFFFFu)) continue;
                        uint32_t v[16];
                        const uint32_t at = tmem + lane_base + 128u * (uint32_t)(sw >> 2) + 16u * i;
                        tc::tmem_ld16(at, v);
                        tc::tmem_ld_wait(v);
#pragma unroll
                        for (int w = 0; w < 16; w++) v[w] = __float_as_uint(__uint_as_float(v[w]) * S.alpha[16 * (i & 3) + w]);
                        tc::tmem_st16(at, v);
                    }
                    tc::tmem_st_wait();
                    tc::named_bar_sync(1, DA_STHREADS);        // (S.red, S.alpha, S.moved are read)
                }
            }
            // (the last value product has read its weights; if it has not, nothing is
            // written and the next wait ends the loop for all warps together)
            if (j == 0 || dense_wait(&S.obar[DA_PARTS - 1], ph ^ 1, &S.abort, polls, c.status)) {
#pragma unroll
                for (int u = 0; u < 4; u++) {
                    uint8_t *row = S.p + (uint32_t)(key + 8 * u) * 128u + 4u * (lane & 3);
#pragma unroll
                    for (int i = 0; i < 4; i++) {
                        const int at = 16 * (u >> 1) + 4 * i + 2 * (u & 1);
                        // the weights' rounding to f16 (2^-11, an eighth of the output's to bf16; a second
                        // f16 for the rest would be as much value product again, 1,536 cycles a tile, and
                        // 16 KB that are not there); their sum takes fp32 values
                        const float2 wt = f32x2_mul(make_float2(exp2_approx(x[at]), exp2_approx(x[at + 1])), make_float2(ky[u], ky[u]));
                        uint32_t pk;
                        asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(pk) : "f"(wt.y), "f"(wt.x));
                        *reinterpret_cast<uint32_t *>(row + ((((uint32_t)h32 >> 3) + i ^ ((uint32_t)key & 7u)) << 4)) = pk;
                    }
                }
            }
            tc::fence_proxy_async_smem();
            tc::tc_fence_before();
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(&S.pbar);
            // The sums, while the value product runs: 2^(y - mu - Xk) by an exponential of its own,
            // for 2^(y - mu) may be below fp32's range where the term is not.
            const float off = high ? DA_SUM : E4M3 ? DN_XOFF : 0.0f, fct = exp2i((int)(DA_SUM - off));
#pragma unroll
            for (int u = 0; u < 4; u++) {
                const float xk = kx[u] == -INFINITY ? 0.0f : kx[u] - off;
#pragma unroll
                for (int i = 0; i < 8; i += 2) {
                    const int k = 16 * (u >> 1) + 2 * i + 2 * (u & 1);
                    const float2 y = f32x2_sub(make_float2(x[k], x[k + 1]), make_float2(xk, xk));
                    const float2 sum = f32x2_fma(make_float2(exp2_approx(y.x), exp2_approx(y.y)), make_float2(fct, fct), make_float2(l[i], l[i + 1]));
                    l[i] = sum.x;
                    l[i + 1] = sum.y;
                }
            }
            // a segment's slot: a row that a run begins in its middle (or with) is the
            // run's first, any other its second
            DenseSlot &slot = slots[2 * blockIdx.x + (j > ti ? 1 : 0)];
            if (__builtin_expect(last || (at + 1) % DA_FOLD == 0, 0)) {
                ok = dense_wait(&S.obar[DA_PARTS - 1], ph, &S.abort, polls, c.status);
                tc::tc_fence_after();
#pragma unroll
                for (int i = 0; i < 8; i++) {
                    float v = l[i];
#pragma unroll
                    for (int w = 4; w < 32; w <<= 1) v += __shfl_xor_sync(0xffffffffu, v, w);
                    const int h = hd + 8 * (i >> 1) + (i & 1);
                    if (lane < 4) {
                        S.red[quarter][h] = v;
                        if (quarter == 0) {
                            S.back[h] = exp2_approx(fminf(S.held[h] - mu[i], 120.0f));      // (more only for nothing)
                            S.held[h] = S.mu[h] = mu[i];
                        }
                    }
                }
                if (named_bar_or(1, DA_STHREADS, !ok)) break;
            }
            if (__builtin_expect(last, 0)) {
                const bool whole = ti == tiles - 1 && owned;
                if (sw == 0 && lane == 0 && !whole && owned)
                    dense_head(heads, r, (int)(&slot - slots), S.g0 + j - ti + tiles - 1, S.total);
                dense_output(tmem, slot, !whole, at >= DA_FOLD, o + (int64_t)r * CSA2_HEADS * CSA2_HEAD_DIM,
                             lse + (int64_t)r * CSA2_HEADS, swa.sink, swa.rope_base > 0.0f, bt.q_pos + r, turns);
                tc::tc_fence_before();
            } else if (__builtin_expect((at + 1) % DA_FOLD == 0, 0)) {
                dense_fold(tmem, slot, at < DA_FOLD);
                tc::tc_fence_before();
                if (at < DA_FOLD) {
                    // The references go down for the rest, as far as the largest weight so far --
                    // at most 2^Xk of the sum -- stays below 2^13.
                    const int x = max(max((int8_t)xt4, (int8_t)(xt4 >> 8)), max((int8_t)(xt4 >> 16), (int8_t)(xt4 >> 24)));
#pragma unroll
                    for (int i = 0; i < 8; i++) {
                        const int h = hd + 8 * (i >> 1) + (i & 1);
                        const float L = (S.red[0][h] + S.red[1][h]) + (S.red[2][h] + S.red[3][h]);
                        const int top = (int)(__float_as_uint(L) >> 23) - 126 - (int)DA_SUM + x;
                        const int down = L > 0.0f ? min(max(13 - top, 0), (int)(DA_LATE - DA_START)) : 0;
                        mu[i] -= (float)down;
                        l[i] *= exp2i(down);
                    }
                }
            }
            if (__builtin_expect(++ti == tiles && j + 1 < n, 0)) {
                ti = 0;
                tiles = dense_row(bt, evicted, swa, ++r).tiles;
                owned = true;
            }
        }
    }
    pdl_launch_dependents();
    tc::tc_fence_before();
    __syncthreads();
    tc::tc_fence_after();
    if (warp == 0) tc::tmem_dealloc(tmem, DA_TMEM_COLS);
}

// Joins the parts of the rows that the cuts divided: block (run, heads 4 y ..).
constexpr int DM_HEADS = 4, DM_THREADS = 256;

__global__ void __launch_bounds__(DM_THREADS)
    k_dense_merge(const DenseHead *__restrict__ heads, const DenseSlot *__restrict__ slots, csa2_batch bt,
                  const float *__restrict__ sink, uint16_t *__restrict__ o, float *__restrict__ lse, RopeTurns turns,
                  int rope)
{
    __shared__ float wgt[DA_MAX_CTAS][DM_HEADS], sum[DA_MAX_CTAS][DM_HEADS];
    __shared__ float out[DM_HEADS][64];            // the RoPE dims
    pdl_wait();
    const int run = blockIdx.x, h0 = DM_HEADS * blockIdx.y, tid = threadIdx.x;
    const int64_t r = heads[run].row;
    if (r < 0) return;
    const int parts = heads[run].parts, slot0 = heads[run].slot;
    auto slot_of = [&](int i) { return i == 0 ? slot0 : 2 * (run + i); };
    // maxima and sums all at once, then a warp per head (one after the other they were
    // the longest chain of a row of many parts: 40 us for some 58 of them, now 25)
    for (int i = tid; i < parts * DM_HEADS; i += DM_THREADS) {
        const DenseSlot &part = slots[slot_of(i / DM_HEADS)];
        wgt[i / DM_HEADS][i % DM_HEADS] = part.m[h0 + i % DM_HEADS];
        sum[i / DM_HEADS][i % DM_HEADS] = part.l[h0 + i % DM_HEADS];
    }
    __syncthreads();
    if (tid < 32 * DM_HEADS) {
        const int j = tid >> 5, lane = tid & 31, h = h0 + j;
        const float z = sink ? sink[h] * kLog2e : -INFINITY;
        float M = z;
        for (int i = lane; i < parts; i += 32) M = fmaxf(M, wgt[i][j]);
#pragma unroll
        for (int w = 1; w < 32; w <<= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, w));
        const float base = M == -INFINITY ? 0.0f : M;
        float L = 0.0f;
        for (int i = lane; i < parts; i += 32) {
            // (in two steps, as the references move in k_dense_attn)
            const float d = wgt[i][j] - base, d1 = fmaxf(truncf(0.5f * d), -200.0f), w1 = exp2f(d1), w2 = exp2f(d - d1);
            wgt[i][j] = w1 * w2;
            L = fmaf(w1 * sum[i][j], w2, L);
        }
#pragma unroll
        for (int w = 1; w < 32; w <<= 1) L += __shfl_xor_sync(0xffffffffu, L, w);
        if (sink) L += exp2f(z - base);
        const float inv = L == 0.0f ? 0.0f : 1.0f / L;
        for (int i = lane; i < parts; i += 32) wgt[i][j] *= inv;
        if (lane == 0) lse[r * CSA2_HEADS + h] = L == 0.0f ? -INFINITY : dense_lse(M, L);
    }
    __syncthreads();
    // a thread's eight dims of one head
    const int hl = tid >> 6, d0 = 8 * (tid & 63), h = h0 + hl;
    float acc[8];
#pragma unroll
    for (int j = 0; j < 8; j++) acc[j] = 0.0f;
#pragma unroll 8
    for (int i = 0; i < parts; i++) {
        const float w = wgt[i][hl];
        const float4 *src = reinterpret_cast<const float4 *>(&slots[slot_of(i)].o[h][d0]);
        const float4 a = __ldcg(src), b = __ldcg(src + 1);
        const float v[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
        for (int j = 0; j < 8; j++) acc[j] = fmaf(w, v[j], acc[j]);
    }
    if (rope) {
        if (d0 >= 448)
#pragma unroll
            for (int j = 0; j < 8; j++) out[hl][d0 - 448 + j] = acc[j];
        __syncthreads();
        if (d0 >= 448) {
            const int64_t t = bt.q_pos[r];
#pragma unroll
            for (int j = 0; j < 8; j++) {
                const int i = (d0 - 448 + j) & 31;
                float sn, cs;
                rope_sincos(t, turns.phi[i], &sn, &cs);
                const float oth = out[hl][(d0 - 448 + j) ^ 32];
                acc[j] = d0 < 480 ? fmaf(acc[j], cs, oth * sn) : fmaf(acc[j], cs, -oth * sn);
            }
        }
    }
    uint32_t pk[4];
#pragma unroll
    for (int j = 0; j < 4; j++) {
        const __nv_bfloat162 b = __floats2bfloat162_rn(acc[2 * j], acc[2 * j + 1]);
        pk[j] = *reinterpret_cast<const uint32_t *>(&b);
    }
    *reinterpret_cast<uint4 *>(o + (r * CSA2_HEADS + h) * CSA2_HEAD_DIM + d0) = make_uint4(pk[0], pk[1], pk[2], pk[3]);
}

int launch_dense_attn(const csa2_cache &c, const csa2_batch &bt, const int64_t *evicted, const uint16_t *q,
                      float sm_scale, const csa2_swa &swa, uint16_t *o, float *lse, void *ws, cudaStream_t st)
{
    const int64_t rows = (int64_t)bt.batch * bt.nq;
    const int sms = device_sms();
    if (sms <= 0) return CSA2_ERR_CUDA;
    const int64_t runs = std::min<int64_t>(dense_runs(bt), sms);
    DenseHead *heads = static_cast<DenseHead *>(ws);
    DenseSlot *slots = reinterpret_cast<DenseSlot *>(static_cast<char *>(ws) + da_align((size_t)dense_runs(bt) * sizeof(DenseHead)));
    const size_t smem = sizeof(DaSmem) + 1024;
    const RopeTurns turns = rope_turns(swa.rope_base);
    auto kern = c.kv_format == CSA2_KV_FP4_E4M3 ? k_dense_attn<true> : k_dense_attn<false>;
    if (const int s = kernel_smem_limit((const void *)kern, smem, 100)) return s;
    if (const int s = launch_pdl(kern, dim3((unsigned)runs), dim3(DA_THREADS), smem, st, c, bt, evicted, q, sm_scale,
                                 swa, o, lse, rows, heads, slots, turns, wait_polls()))
        return s;
    return launch_pdl(k_dense_merge, dim3((unsigned)runs, CSA2_HEADS / DM_HEADS), dim3(DM_THREADS), 0, st,
                      (const DenseHead *)heads, (const DenseSlot *)slots, bt, swa.sink, o, lse, turns,
                      swa.rope_base > 0.0f ? 1 : 0);
}

}  // namespace csa2
