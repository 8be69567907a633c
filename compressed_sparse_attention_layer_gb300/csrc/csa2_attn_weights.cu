// The attention weight each cache entry received: acc[b][e] += the sum over the
// rows r of sequence b and the 64 heads h of e^(l_rhe - lse_rh), with l and lse
// those of the attention -- over every visible entry, or over the entries that
// each row selected.
//
// One product, the logits: 65,536 operations a (row, key) pair against 272 or
// 288 bytes an entry, so the cache read bounds one query per sequence and the
// products several.  A key is a row of S^T, so its heads are added in a thread or
// four, and an entry's sum is taken over the rows in a fixed order: the result does
// not depend on the schedule.
//
// k_weights_tiles serves one query per sequence and selections, k_weights_rows
// several queries that see a whole sequence: 8 x 131,072 entries, one query each,
// take 126 us with the first (floor 43); 4 x 64 queries over 2,001 to 8,200 entries
// 121 us with the second and 317 with a query brought in for each 64 keys (floor 41).
#include <algorithm>

#include "csa2_dense_common.cuh"

namespace csa2 {

// Weights of several selecting rows of one sequence meet in 64-bit fixed point
// (2^-40): a row gives an entry at most 64, 65,535 rows stay below 2^62, and
// integer sums do not depend on their order.
constexpr float AW_FIX = 1099511627776.0f;         // 2^40

// The two keys' sums of a thread over the heads; its quad of lanes has them all.
__device__ __forceinline__ void weights_sums(const float (&v)[32], const float (&f)[16], const float (&z)[16],
                                             const float (&kf)[2], float (&s)[2])
{
#pragma unroll
    for (int u = 0; u < 2; u++) {
        s[u] = 0.0f;
#pragma unroll
        for (int i = 0; i < 16; i++)               // one rounding at the size of l - lse
            s[u] += exp2_approx(fmaf(v[4 * (i >> 1) + 2 * u + (i & 1)], f[i] * kf[u], -z[i]) * kLog2e);
        s[u] += __shfl_xor_sync(0xffffffffu, s[u], 1);
        s[u] += __shfl_xor_sync(0xffffffffu, s[u], 2);
    }
}

// ---------------------------------------------------------------- one query per sequence, and selections
// A tile is a page, or 64 of a row's selected entries (SELECTED), copied to shared
// memory up to three ahead; the keys go to the products in halves of 256 dims, of which
// three places go round, so that neither waits for the other and the copies have the
// rest of the shared memory.  The loop is as long as the keys' conversion, 2,250
// cycles a tile (the products are 1,030, the page's bytes 800 at an even share of the
// memory); loads into the registers of the warps that convert left it at 3,200.
constexpr int AP_RAW = 3, AP_HALVES = 3, AP_RING = 4;
constexpr uint32_t AP_HALF = DN_KBYTES / 2;
constexpr int AP_SWARPS = 4;
// warps for the copies: one has the pages in hand, selected entries are 16-byte pieces, for four
__host__ __device__ constexpr int ap_cwarps(bool selected) { return selected ? 4 : 1; }
__host__ __device__ constexpr int ap_warps(bool selected) { return DN_KWARPS + AP_SWARPS + ap_cwarps(selected) + 1; }
// The logits of dims 0-255 and 256-511 in columns of their own: the accumulator drops
// the low bits of every step's sum, always towards zero, which the sums over many
// rows and heads do not average out.  Half the steps, smaller sums: half of that.
constexpr uint32_t AP_TMEM_COLS = 2 * 64 * AP_RING;

struct ApProduct {
    int b, row;     // sequence, query row
    int e0;         // the page's first entry
    int lim;        // its keys: the row sees them, and the page is there
    int flags;
};
constexpr int AP_NEW_QUERY = 1, AP_STOP = 2;

struct ApSmem {
    uint8_t k[AP_HALVES][AP_HALF];
    uint8_t q[DN_QBYTES];
    uint8_t raw[AP_RAW][DN_KEYS * 256];
    uint8_t rsc[AP_RAW][DN_KEYS * 32];
    ApProduct prod[AP_RING];
    int32_t entry[AP_RING][DN_KEYS];               // the selected entries, -1: none
    float qe[AP_RING][CSA2_HEADS], lse[AP_RING][CSA2_HEADS];           // the query's 2^e_h and lse, where it is new
    float kf[AP_RING][DN_KEYS];                    // the keys' 2^(Xk - 12)
    uint64_t full[AP_RAW], empty[AP_RAW];          // a page
    uint64_t kready[AP_HALVES], kfree[AP_HALVES];  // a half of the keys
    uint64_t sbar[AP_RING], fbar[AP_RING];         // the product is done; its sums are taken
    uint64_t dbar;
    int64_t sums[ap_warps(true)];
    int64_t b0, tile0;
    int abort;
    uint32_t tmem;
};

struct ApArgs {
    csa2_cache c;
    csa2_batch bt;
    csa2_swa swa;                                  // the attention's window: its flags and start count
    const int64_t *evicted;
    const uint16_t *q;
    const float *lse;
    const int32_t *idx;                            // [rows][k], SELECTED
    int k;
    float sm_scale;
    float *acc;
    int64_t ld;
    unsigned long long *fix;                       // [B][max_entries], or NULL
    uint32_t polls;
};

__device__ __forceinline__ void copy16(void *dst, const void *src)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(tc::smem_u32(dst)), "l"(src) : "memory");
}

// This thread's copies have landed.
__device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// Arrive (one of the count) when this thread's copies so far have landed.
__device__ __forceinline__ void copies_arrive(uint64_t *bar)
{
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(tc::smem_u32(bar)) : "memory");
}

template <bool E4M3, bool SELECTED>
__global__ void __launch_bounds__(32 * ap_warps(SELECTED), 1) k_weights_tiles(const __grid_constant__ ApArgs a)
{
    ApSmem &S = dense_smem<ApSmem>();
    const csa2_cache &c = a.c;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid == 0) {
        for (int i = 0; i < AP_RAW; i++) {
            tc::mbar_init(&S.full[i], SELECTED ? 33 * ap_cwarps(true) : 1);  // (each lane's copies, and a warp's word)
            tc::mbar_init(&S.empty[i], DN_KWARPS);
        }
        for (int i = 0; i < AP_HALVES; i++) {
            tc::mbar_init(&S.kready[i], DN_KWARPS);
            tc::mbar_init(&S.kfree[i], 1);
        }
        for (int i = 0; i < AP_RING; i++) {
            tc::mbar_init(&S.sbar[i], 1);
            tc::mbar_init(&S.fbar[i], AP_SWARPS);
        }
        tc::mbar_init(&S.dbar, 1);
        tc::fence_mbar_init();
        S.abort = 0;
    }
    if (warp == 0) tc::tmem_alloc(&S.tmem, AP_TMEM_COLS);
    pdl_wait();
    // equal runs of the tiles of the rows' selections, or of those that the sequences'
    // rows see, one sequence after the other
    auto seen = [&](int64_t b) { return dense_row(a.bt, a.evicted, a.swa, b).vis; };
    const int kt = SELECTED ? (a.k + DN_KEYS - 1) / DN_KEYS : 1;
    int64_t total = (int64_t)a.bt.batch * a.bt.nq * kt, at = 0, mine = 0;
    const int64_t per = (a.bt.batch + blockDim.x - 1) / blockDim.x;
    const int64_t lo = min((int64_t)tid * per, (int64_t)a.bt.batch), hi = min(lo + per, (int64_t)a.bt.batch);
    if (!SELECTED) {
        for (int64_t b = lo; b < hi; b++) mine += (seen(b) + DN_KEYS - 1) / DN_KEYS;
        at = block_exclusive_sum(mine, S.sums, &total);
    }
    const int64_t g0 = total * blockIdx.x / gridDim.x, g1 = total * (blockIdx.x + 1) / gridDim.x;
    if (!SELECTED && g0 >= at && g0 < at + mine)
        for (int64_t b = lo; b < hi; b++) {
            const int64_t n = (seen(b) + DN_KEYS - 1) / DN_KEYS;
            if (g0 < at + n) {
                S.b0 = b;
                S.tile0 = at;
                break;
            }
            at += n;
        }
    tc::tc_fence_before();
    __syncthreads();
    tc::tc_fence_after();
    const uint32_t tmem = S.tmem;
    auto wait = [&](uint64_t *bar, uint32_t phase) { return dense_wait(bar, phase & 1, &S.abort, a.polls, c.status); };

    if (warp == ap_warps(SELECTED) - 1) {
        // ================================================ the products
        const uint64_t kd = dense_desc(S.k[0], 16), qd = dense_desc(S.q, 16);
        const bool leader = elect_one();
        uint32_t slot = 0, turn = 0;
        for (uint32_t p = 0;; p++) {
            const uint32_t d = p % AP_RING;
            bool ok = true;
#pragma unroll 1
            for (int h = 0; h < 2 && ok; h++) {
                // (the keys follow the pages' warp, which has waited for the sums of product p - 4)
                ok = wait(&S.kready[slot], turn);
                if (!ok) break;
                const bool stop = S.prod[d].flags & AP_STOP;
                tc::tc_fence_after();
                if (leader) {
                    if (!stop) {
                        // S^T[64 keys x 64 heads] = K Q^T over a half of the dims
                        constexpr uint32_t IDESC = tc::idesc_f16(64, 64, 0, 0, 0, 0);
                        uint64_t k0 = kd + slot * (AP_HALF / 16), q0 = qd + (uint32_t)h * (4 * DN_QSLAB / 16);
#pragma unroll 1
                        for (int slab = 0; slab < 4; slab++) {
#pragma unroll
                            for (int kk = 0; kk < 4; kk++)
                                tc::mma_f16(tmem + 128u * d + 64u * h, k0 + 2u * kk, q0 + 2u * kk, IDESC, slab > 0 || kk > 0);
                            k0 += DN_KSLAB / 16;
                            q0 += DN_QSLAB / 16;
                        }
                        tc::mma_commit(&S.kfree[slot]);
                    }
                    if (h == 1 || stop) tc::mma_commit(&S.sbar[d]);
                }
                __syncwarp();
                if (++slot == AP_HALVES) {
                    slot = 0;
                    turn++;
                }
                ok = !stop;
            }
            if (!ok) break;
        }
        // nothing is in flight when the tensor memory goes
        if (leader) tc::mma_commit(&S.dbar);
        __syncwarp();
        tc::mbar_wait(&S.dbar, 0, 1u << 18);
    } else if (warp >= DN_KWARPS + AP_SWARPS) {
        // ================================================ the copies
        constexpr uint32_t SBYTES = E4M3 ? 32 : 16;                    // scales of an entry
        int64_t b = 0, ti = 0, n = 0;
        int32_t page = -1;                         // of the next tile
        const int cw = warp - DN_KWARPS - AP_SWARPS, key = 16 * cw + (lane & 15);
        int32_t e = -1;                            // its selected entry of key, and the slot
        int64_t slot = -1;
        DenseRow R = {};
        int64_t have = -1;                         // the row that R is of
        auto page_of = [&]() { return __ldg(c.block_table + b * c.max_pages + ti); };
        auto find = [&](int64_t g) {
            const int64_t r = g / kt;
            if (r != have) R = dense_row(a.bt, a.evicted, a.swa, r);
            have = r;
            const int j = (int)(g % kt) * DN_KEYS + key;
            e = j < a.k ? __ldg(a.idx + r * a.k + j) : -1;
            slot = -1;
            if (e < 0) return;
            if (e >= R.vis) {                      // beyond the query, or a token of its window
                if (e >= dense_visible(a.bt, a.evicted, R.b, R.t)) flag(c.status, CSA2_DEV_BAD_INDEX);
                return;
            }
            slot = dense_page_slot(c, __ldg(c.block_table + (int64_t)R.b * c.max_pages + (e >> 6)), 0);
            if (slot >= 0) slot += e & 63;
        };
        if (g0 < g1) {
            if (SELECTED) {
                find(g0);
            } else {
                b = S.b0;
                ti = g0 - S.tile0;
                n = seen(b);
                page = page_of();
            }
        }
        bool fresh = true;
        uint32_t p = 0;
        for (int64_t g = g0;; g++, p++) {
            const uint32_t i = p % AP_RAW, d = p % AP_RING;
            if (p >= AP_RAW && !wait(&S.empty[i], p / AP_RAW - 1)) break;
            if (p >= AP_RING && !wait(&S.fbar[d], p / AP_RING - 1)) break;
            if (g >= g1) {
                if (lane == 0) {
                    if (cw == 0) S.prod[d].flags = AP_STOP;
                    tc::mbar_arrive(&S.full[i]);
                }
                if (SELECTED) copies_arrive(&S.full[i]);
                p++;
                break;
            }
            if (SELECTED) {
                if (lane < 16) S.entry[d][key] = slot >= 0 ? e : -1;
                // half a warp an entry (a bulk copy of 256 bytes costs more than its 16 pieces)
#pragma unroll
                for (int j = 0; j < 16; j += 2) {
                    const int64_t s = __shfl_sync(0xffffffffu, slot, j + (lane >> 4));
                    if (s >= 0) copy16(S.raw[i] + (16 * cw + j) * 256 + 16 * lane, c.kv_codes + s * 256 + 16 * (lane & 15));
                }
                if (lane < 16 && slot >= 0)
#pragma unroll
                    for (uint32_t j = 0; j < SBYTES; j += 16) copy16(S.rsc[i] + key * SBYTES + j, c.kv_scales + slot * SBYTES + j);
                copies_arrive(&S.full[i]);
                if (cw == 0 && lane == 0) S.prod[d] = {R.b, (int)have, 0, DN_KEYS, fresh ? AP_NEW_QUERY : 0};
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(&S.full[i]);
                const int64_t r = have;
                if (g + 1 < g1) find(g + 1);
                fresh = have != r;
            } else {
                const int64_t s = dense_page_slot(c, page, lane);
                if (lane == 0) {
                    S.prod[d] = {(int)b, (int)b, (int)(ti * DN_KEYS), s < 0 ? 0 : (int)min(n - ti * DN_KEYS, (int64_t)DN_KEYS), fresh ? AP_NEW_QUERY : 0};
                    tc::mbar_arrive_expect_tx(&S.full[i], s < 0 ? 0 : DN_KEYS * (256 + SBYTES));
                    if (s >= 0) {
                        tc::bulk_load(S.raw[i], c.kv_codes + s * 256, DN_KEYS * 256, &S.full[i]);
                        tc::bulk_load(S.rsc[i], c.kv_scales + s * SBYTES, DN_KEYS * SBYTES, &S.full[i]);
                    }
                }
                __syncwarp();
                fresh = false;
                if (g + 1 < g1) {
                    ti++;
                    while (ti * DN_KEYS >= n) {    // (the run's next tile exists)
                        n = seen(++b);
                        ti = 0;
                        fresh = true;
                    }
                    page = page_of();
                }
            }
        }
        // every copy has landed when the shared memory goes
        if (SELECTED) copies_wait();
        else
            for (uint32_t i = p < AP_RAW ? 0 : p - AP_RAW; i < p; i++) tc::mbar_wait(&S.full[i % AP_RAW], (i / AP_RAW) & 1, 1u << 18);
    } else if (warp < DN_KWARPS) {
        // ================================================ keys and queries
        const int key = DN_WKEYS * warp + (lane >> 2);                 // this quad's key
        auto query = [&](int64_t r, uint32_t d) {
            const float z = tid < CSA2_HEADS ? __ldg(a.lse + r * CSA2_HEADS + tid) : 0.0f;
            dense_load_q(S.q, S.qe[d], a.q, r, warp, DN_KWARPS, lane);
            if (tid < CSA2_HEADS) S.lse[d][tid] = z == -INFINITY ? INFINITY : z;
        };
        uint32_t slot = 0, turn = 0;
        if (g0 < g1) query(SELECTED ? g0 / kt : S.b0, 0);              // the first, while the first tile comes in
        for (uint32_t p = 0;; p++) {
            const uint32_t i = p % AP_RAW, d = p % AP_RING;
            if (!wait(&S.full[i], p / AP_RAW)) break;
            const ApProduct m = S.prod[d];
            if (m.flags & AP_STOP) {
                // As with any half: before its place is free, a slower warp may have yet to
                // arrive for the half that is there, and this arrival would count as its.
                if (turn > 0 && !wait(&S.kfree[slot], turn - 1)) break;
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(&S.kready[slot]);
                break;
            }
            // (odd keys take the two parts of a half in the other order: their codes
            // are in the other half of the banks)
            uint4 code[4], raw;
#pragma unroll
            for (int u = 0; u < 4; u++)
                code[u] = *reinterpret_cast<const uint4 *>(S.raw[i] + key * 256 + 64 * (u ^ (key & 1)) + 16 * (lane & 3));
            if (E4M3) {
                const uint16_t *q16 = reinterpret_cast<const uint16_t *>(S.rsc[i] + key * 32) + (lane & 3);
                raw = make_uint4(q16[0], q16[4], q16[8], q16[12]);
            } else {
                raw = *reinterpret_cast<const uint4 *>(S.rsc[i] + key * 16);
            }
            if (key & 1) raw = make_uint4(raw.y, raw.x, raw.w, raw.z);
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(&S.empty[i]);
            const uint2 sc = dense_pack_scales<E4M3>(raw, lane);
            bool zero;
            const int xk = dense_exponent<E4M3>(code, sc, &zero);
            const bool there = SELECTED ? S.entry[d][key] >= 0 : key < m.lim;
            if ((m.flags & AP_NEW_QUERY) && p > 0) {
                // the products have read the query before
                if (!wait(&S.sbar[(p - 1) % AP_RING], (p - 1) / AP_RING)) break;
                query(m.row, d);
            }
            if ((lane & 3) == 0) S.kf[d][key] = exp2i(xk - (int)DN_XOFF);
            bool ok = true;
#pragma unroll
            for (int h = 0; h < 2; h++) {
                ok = ok && (turn == 0 || wait(&S.kfree[slot], turn - 1));
                if (!ok) break;
#pragma unroll
                for (int u = 2 * h; u < 2 * h + 2; u++)
                    dense_store<E4M3>(S.k[slot], code[u], sc, xk, there, u, (u ^ (key & 1)) - 2 * h, key, lane);
                tc::fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(&S.kready[slot]);
                if (++slot == AP_HALVES) {
                    slot = 0;
                    turn++;
                }
            }
            if (!ok) break;
        }
    } else {
        // ================================================ the sums
        const int sw = warp - DN_KWARPS;
        const int key = 16 * sw + (lane >> 2);     // this thread's keys: key and key + 8
        const uint32_t lane_base = (uint32_t)(32 * sw) << 16;
        float f[16], z[16];                        // heads 8 (i / 2) + 2 (lane % 4) + i % 2: factor, lse
        for (uint32_t p = 0;; p++) {
            const uint32_t d = p % AP_RING;
            if (!wait(&S.sbar[d], p / AP_RING)) break;
            tc::tc_fence_after();
            const ApProduct m = S.prod[d];
            if (m.flags & AP_STOP) break;
            if (m.flags & AP_NEW_QUERY) {
#pragma unroll
                for (int i = 0; i < 16; i++) {
                    const int h = 8 * (i >> 1) + 2 * (lane & 3) + (i & 1);
                    f[i] = S.qe[d][h] * a.sm_scale;
                    z[i] = S.lse[d][h];
                }
            }
            const float kf[2] = {S.kf[d][key], S.kf[d][key + 8]};
            int e[2] = {m.e0 + key, m.e0 + key + 8};
            if (SELECTED) {
                e[0] = S.entry[d][key];
                e[1] = S.entry[d][key + 8];
            }
            float v[32];
#pragma unroll
            for (int g = 0; g < 2; g++) {          // heads 32 g ..
                uint32_t x[16], y[16];
                tmem_ld_16x32(tmem + 128u * d + 32u * g + lane_base, x);
                tmem_ld_16x32(tmem + 128u * d + 64u + 32u * g + lane_base, y);
                tc::tmem_ld_wait(x);
                tc::tmem_ld_wait(y);
#pragma unroll
                for (int i = 0; i < 16; i++) v[16 * g + i] = __uint_as_float(x[i]) + __uint_as_float(y[i]);
            }
            tc::tc_fence_before();
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(&S.fbar[d]);
            float s[2];
            weights_sums(v, f, z, kf, s);
#pragma unroll
            for (int u = 0; u < 2; u++) {
                if (lane & 3) continue;
                if (!SELECTED) {                   // an entry's sum is this CTA's alone
                    if (key + 8 * u < m.lim) a.acc[m.b * a.ld + e[u]] += s[u];
                } else if (e[u] >= 0) {
                    // the same entry twice in a row has the same weight: the order of its sums does not matter
                    // (NaN has no fixed point: it goes to acc, which then stays NaN)
                    if (a.fix && s[u] != s[u]) a.acc[(int64_t)m.b * a.ld + e[u]] = NAN;
                    else if (a.fix) atomicAdd(a.fix + (int64_t)m.b * a.bt.max_entries + e[u], (unsigned long long)(fminf(s[u], 64.0f) * AW_FIX));
                    else atomicAdd(a.acc + (int64_t)m.b * a.ld + e[u], s[u]);
                }
            }
        }
    }
    pdl_launch_dependents();
    tc::tc_fence_before();
    __syncthreads();
    tc::tc_fence_after();
    if (warp == 0) tc::tmem_dealloc(tmem, AP_TMEM_COLS);
}

// ---------------------------------------------------------------- several queries per sequence
// S^T[128 keys x 64 heads] of a key tile and each of its rows in turn: 48 cycles a
// 16-dim step, by the shared memory that the operands are read from, against 2 x 32
// with 64 keys.  The tile stays while the queries pass; a query is converted once,
// by a kernel of its own, to the image that the products read (64 KB, as large as q),
// so that bringing it in is four bulk copies and costs no warp anything.  Few tiles:
// the rows are divided too, and the parts' sums added in order.
constexpr int AM_KEYS = 128;
constexpr uint32_t AM_KSLAB = AM_KEYS * 128;
constexpr int AM_PARTS = 4;                        // of 128 dims: a key part, a query part
constexpr uint32_t AM_STAGE = DN_QBYTES / AM_PARTS;
constexpr int AM_STAGES = 5;                       // query parts in flight
constexpr int AM_RING = 4, AM_KRING = 8;           // products, key tiles whose factors are kept
constexpr int AM_SWARPS = 4, AM_WARPS = DN_KWARPS + AM_SWARPS + 2, AM_THREADS = 32 * AM_WARPS;
constexpr uint32_t AM_TMEM_COLS = 2 * 64 * AM_RING;
constexpr int AM_UNITS = 8 * 152;                  // (tile, rows) units aimed at: eight per SM

struct AmRow {                                     // of a query: l - lse = S f - z
    float f[CSA2_HEADS], z[CSA2_HEADS];
};

// What the queries' warp says of a product; where it begins and ends a tile, its
// tile of 128 keys and the place of its sums.
struct AmProduct {
    int b, chunk, e0;
    int lim;                                       // keys of the tile that the row sees
    int flags;
};
constexpr int AM_NEW_TILE = 1, AM_LAST = 2, AM_SUM = 4, AM_STOP = 8;   // AM_SUM: of its unit the last

struct AmSmem {
    uint8_t k[DN_SLABS * AM_KSLAB];
    uint8_t q[AM_STAGES][AM_STAGE];
    AmRow row[AM_RING];
    AmProduct prod[AM_RING];
    float kf[AM_KRING][AM_KEYS];                   // the keys' 2^(Xk - 12), -1: no key
    uint64_t kready[AM_PARTS], kfree[AM_PARTS];    // part of the tile written; read by its last query
    uint64_t qready[AM_STAGES], qfree[AM_STAGES];
    uint64_t sbar[AM_RING];                        // the product is done
    uint64_t fbar[AM_RING];                        // its sums are taken
    uint64_t dbar;
    int64_t sums[AM_WARPS];
    int64_t b0, tile0;
    int abort;
    uint32_t tmem;
};

struct AmArgs {
    csa2_cache c;
    csa2_batch bt;
    const uint8_t *q;                              // [rows] images
    const AmRow *row;                              // [rows]
    const int32_t *vis;                            // [rows] entries the row sees
    int chunks;                                    // of a sequence's rows
    float *acc;
    int64_t ld;
    float *part;                                   // [chunks][B][tiles][128] if chunks > 1
    int64_t tiles;                                 // of a sequence, at most
    uint32_t polls;
};

__device__ __forceinline__ int64_t am_tiles(const csa2_batch &bt, int64_t b)
{
    const int64_t n = min(bt.n_entries[b], bt.max_entries);
    return n > 0 ? (n + AM_KEYS - 1) / AM_KEYS : 0;
}

// The products of a CTA's units u .. u1 - 1 in order: unit (tile, chunk) of the
// sequences' tiles one after the other, of each the chunk's rows that see the tile.
// A converged warp walks, 32 rows a look.
struct AmWalk {
    int64_t u, u1, t, tiles;
    int b, p, i, i1;
    uint32_t seen;                                 // of rows i - 32 .., those that are still to come
    int vis;                                       // row i - 32 + lane
    int64_t r;                                     // the product's row
    int lim;                                       // and how many entries it sees
    __device__ __forceinline__ void unit(const AmArgs &a)
    {
        i = (int)((int64_t)a.bt.nq * p / a.chunks);
        i1 = (int)((int64_t)a.bt.nq * (p + 1) / a.chunks);
        seen = 0;
    }
    __device__ __forceinline__ void start(const AmArgs &a, int64_t u_lo, int64_t u_hi, int64_t b0, int64_t tile0)
    {
        u = u_lo;
        u1 = u_hi;
        if (u >= u1) return;
        b = (int)b0;
        tiles = am_tiles(a.bt, b);
        t = u / a.chunks - tile0;
        p = (int)(u % a.chunks);
        unit(a);
    }
    __device__ __forceinline__ bool skip(const AmArgs &a, int units)
    {
        u += units;
        p += units;
        if (u >= u1) return false;
        if (p == a.chunks) {
            p = 0;
            t++;
            while (t >= tiles) {
                tiles = am_tiles(a.bt, ++b);
                t = 0;
            }
        }
        unit(a);
        return true;
    }
    __device__ __forceinline__ bool next(const AmArgs &a)
    {
        if (u >= u1) return false;
        do {
            while (!seen && i < i1) {
                const int at = i + (int)(threadIdx.x & 31);
                vis = at < i1 ? a.vis[(int64_t)b * a.bt.nq + at] : 0;
                seen = __ballot_sync(0xffffffffu, vis > t * AM_KEYS);
                i += 32;
            }
            if (seen) {
                const int at = __ffs(seen) - 1;
                seen &= seen - 1;
                r = (int64_t)b * a.bt.nq + i - 32 + at;
                lim = __shfl_sync(0xffffffffu, vis, at);
                return true;
            }
        } while (skip(a, 1));
        return false;
    }
    // the first product of another tile
    __device__ __forceinline__ bool next_tile(const AmArgs &a) { return skip(a, a.chunks - p) && next(a); }
};

// Block r: query r's image and factors, and the entries it sees; all blocks: the
// parts' sums set to zero.
__global__ void __launch_bounds__(256)
    k_weights_queries(const __grid_constant__ csa2_batch bt, const int64_t *evicted, const __grid_constant__ csa2_swa swa,
                      const uint16_t *__restrict__ q, const float *__restrict__ lse, float sm_scale, uint8_t *img, AmRow *row,
                      int32_t *vis, float *part, int64_t parts)
{
    __shared__ float qe[CSA2_HEADS];
    const int tid = threadIdx.x;
    const int64_t r = blockIdx.x;
    pdl_wait();
    dense_load_q(img + r * DN_QBYTES, qe, q, r, tid >> 5, 8, tid & 31);
    if (tid == 0) vis[r] = (int32_t)dense_row(bt, evicted, swa, r).vis;
    for (int64_t i = r * 256 + tid; i < parts; i += (int64_t)gridDim.x * 256) part[i] = 0.0f;
    __syncthreads();
    if (tid < CSA2_HEADS) {
        const float z = __ldg(lse + r * CSA2_HEADS + tid);
        row[r].f[tid] = qe[tid] * sm_scale;
        row[r].z[tid] = z == -INFINITY ? INFINITY : z;
    }
    pdl_launch_dependents();
}

template <bool E4M3>
__global__ void __launch_bounds__(AM_THREADS, 1) k_weights_rows(const __grid_constant__ AmArgs a)
{
    AmSmem &S = dense_smem<AmSmem>();
    const csa2_cache &c = a.c;
    const csa2_batch &bt = a.bt;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid == 0) {
        for (int i = 0; i < AM_PARTS; i++) {
            tc::mbar_init(&S.kready[i], DN_KWARPS);
            tc::mbar_init(&S.kfree[i], 1);
        }
        for (int i = 0; i < AM_STAGES; i++) {
            tc::mbar_init(&S.qready[i], 1);
            tc::mbar_init(&S.qfree[i], 1);
        }
        for (int i = 0; i < AM_RING; i++) {
            tc::mbar_init(&S.sbar[i], 1);
            tc::mbar_init(&S.fbar[i], AM_SWARPS);
        }
        tc::mbar_init(&S.dbar, 1);
        tc::fence_mbar_init();
        S.abort = 0;
    }
    if (warp == 0) tc::tmem_alloc(&S.tmem, AM_TMEM_COLS);
    pdl_wait();
    // the units of the sequences, one after the other, in equal runs
    const int64_t per = (bt.batch + AM_THREADS - 1) / AM_THREADS;
    const int64_t lo = min((int64_t)tid * per, (int64_t)bt.batch), hi = min(lo + per, (int64_t)bt.batch);
    int64_t mine = 0, total;
    for (int64_t b = lo; b < hi; b++) mine += am_tiles(bt, b);
    int64_t at = block_exclusive_sum(mine, S.sums, &total);
    const int64_t units = total * a.chunks;
    const int64_t u0 = units * blockIdx.x / gridDim.x, u1 = units * (blockIdx.x + 1) / gridDim.x;
    const int64_t first = u0 / a.chunks;
    if (first >= at && first < at + mine)
        for (int64_t b = lo; b < hi; b++) {
            const int64_t n = am_tiles(bt, b);
            if (first < at + n) {
                S.b0 = b;
                S.tile0 = at;
                break;
            }
            at += n;
        }
    tc::tc_fence_before();
    __syncthreads();
    tc::tc_fence_after();
    const uint32_t tmem = S.tmem;
    AmWalk w;
    w.start(a, u0, u1, S.b0, S.tile0);

    if (warp == AM_WARPS - 1) {
        // ================================================ the products
        const uint64_t kd = dense_desc(S.k, 16), qd = dense_desc(S.q[0], 16);
        const bool leader = elect_one();
        constexpr uint32_t IDESC = tc::idesc_f16(AM_KEYS, 64, 0, 0, 0, 0);
        uint32_t kt = 0, slot = 0, turn = 0;
        bool ok = true;
        for (uint32_t p = 0; ok; p++) {
            const uint32_t d = p % AM_RING;
            int flags = 0;
#pragma unroll 1
            for (int part = 0; part < AM_PARTS; part++) {
                // (the queries' warp has waited for the sums of product p - 4)
                if (!(ok = dense_wait(&S.qready[slot], turn & 1, &S.abort, a.polls, c.status))) break;
                if (part == 0) flags = S.prod[d].flags;
                if (flags & AM_STOP) {
                    if (leader) tc::mma_commit(&S.sbar[d]);
                    ok = false;
                    break;
                }
                if (flags & AM_NEW_TILE)
                    if (!(ok = dense_wait(&S.kready[part], kt & 1, &S.abort, a.polls, c.status))) break;
                tc::tc_fence_after();
                if (leader) {
                    const uint64_t k0 = kd + (uint32_t)part * (2 * AM_KSLAB / 16), q0 = qd + slot * (AM_STAGE / 16);
#pragma unroll
                    for (int i = 0; i < 8; i++)
                        tc::mma_f16(tmem + 128u * d + 64u * (part >> 1), k0 + (i >> 2) * (AM_KSLAB / 16) + 2u * (i & 3),
                                    q0 + (i >> 2) * (DN_QSLAB / 16) + 2u * (i & 3), IDESC, (part & 1) || i > 0);
                    tc::mma_commit(&S.qfree[slot]);
                    if (flags & AM_LAST) tc::mma_commit(&S.kfree[part]);
                    if (part == AM_PARTS - 1) tc::mma_commit(&S.sbar[d]);
                }
                __syncwarp();
                if (++slot == AM_STAGES) {
                    slot = 0;
                    turn++;
                }
            }
            kt += (flags & AM_LAST) != 0;
        }
        // nothing is in flight when the tensor memory goes
        if (leader) tc::mma_commit(&S.dbar);
        __syncwarp();
        tc::mbar_wait(&S.dbar, 0, 1u << 18);
    } else if (warp == AM_WARPS - 2) {
        // ================================================ the queries
        asm volatile("fence.proxy.async.global;" ::: "memory");        // (written by the kernel before)
        uint32_t p = 0, s = 0;
        bool more = w.next(a), ok = true, fresh = true, stop;
        do {
            const uint32_t d = p % AM_RING;
            AmProduct m = {w.b, w.p, 0, 0, more ? 0 : AM_STOP};
            const int64_t r = w.r;
            if (more) {
                const int64_t u = w.u, t = w.t;
                m.e0 = (int)(t * AM_KEYS);
                m.lim = min(w.lim - m.e0, AM_KEYS);
                more = w.next(a);
                const bool last = !more || w.b != m.b || w.t != t;
                m.flags = (fresh ? AM_NEW_TILE : 0) | (last ? AM_LAST : 0) | (!more || w.u != u ? AM_SUM : 0);
                fresh = last;
            }
            if (p >= AM_RING) ok = dense_wait(&S.fbar[d], (p / AM_RING - 1) & 1, &S.abort, a.polls, c.status);
            for (int part = 0; part < (m.flags & AM_STOP ? 1 : AM_PARTS) && ok; part++) {
                const uint32_t slot = s % AM_STAGES;
                if (s >= AM_STAGES) ok = dense_wait(&S.qfree[slot], (s / AM_STAGES - 1) & 1, &S.abort, a.polls, c.status);
                if (!ok) break;
                if (lane == 0) {
                    if (part == 0) S.prod[d] = m;
                    if (m.flags & AM_STOP) {
                        tc::mbar_arrive(&S.qready[slot]);
                    } else {
                        tc::mbar_arrive_expect_tx(&S.qready[slot], AM_STAGE + (part == 0 ? sizeof(AmRow) : 0));
                        if (part == 0) tc::bulk_load(&S.row[d], a.row + r, sizeof(AmRow), &S.qready[slot]);
                        tc::bulk_load(S.q[slot], a.q + r * DN_QBYTES + part * AM_STAGE, AM_STAGE, &S.qready[slot]);
                    }
                }
                __syncwarp();
                s++;
            }
            p++;
            stop = m.flags & AM_STOP;
        } while (ok && !stop);
        // every copy has landed when the shared memory goes
        for (uint32_t i = s < AM_STAGES ? 0 : s - AM_STAGES; i < s; i++)
            tc::mbar_wait(&S.qready[i % AM_STAGES], (i / AM_STAGES) & 1, 1u << 18);
    } else if (warp < DN_KWARPS) {
        // ================================================ the keys
        const int key = DN_WKEYS * warp + (lane >> 2);                 // this quad's keys: key and key + 64
        uint4 code[2][4], raw[2];
        bool there[2];
        auto fetch = [&]() {
            const int64_t n = min(bt.n_entries[w.b], bt.max_entries);
#pragma unroll
            for (int h = 0; h < 2; h++) {
                const int64_t e0 = w.t * AM_KEYS + h * CSA2_PAGE;
                there[h] = false;
                raw[h] = make_uint4(0, 0, 0, 0);
#pragma unroll
                for (int mt = 0; mt < 4; mt++) code[h][mt] = raw[h];
                if (e0 >= n) continue;
                const int64_t s = dense_page_slot(c, __ldg(c.block_table + (int64_t)w.b * c.max_pages + (e0 >> 6)),
                                                  warp == 0 ? lane : 1);
                there[h] = s >= 0 && e0 + key < n;
                if (!there[h]) continue;
#pragma unroll
                for (int mt = 0; mt < 4; mt++) code[h][mt] = dense_codes(c, s + key, mt, lane);
                raw[h] = dense_scales<E4M3>(c, s + key, lane);
            }
        };
        uint32_t kt = 0;
        bool more = w.next(a);
        if (more) fetch();
        while (more) {
            uint2 sc[2];
            int xk[2];
#pragma unroll
            for (int h = 0; h < 2; h++) {
                sc[h] = dense_pack_scales<E4M3>(raw[h], lane);
                bool zero;
                xk[h] = dense_exponent<E4M3>(code[h], sc[h], &zero);
            }
            bool ok = true;
#pragma unroll
            for (int mt = 0; mt < 4; mt++) {
                if (kt > 0 && ok) ok = dense_wait(&S.kfree[mt], (kt - 1) & 1, &S.abort, a.polls, c.status);
                if (!ok) break;
#pragma unroll
                for (int h = 0; h < 2; h++) {
                    // (the tile before is done with, so the sums of the one seven before are taken)
                    if (mt == 0 && (lane & 3) == 0)
                        S.kf[kt % AM_KRING][key + 64 * h] = there[h] ? exp2i(xk[h] - (int)DN_XOFF) : -1.0f;
                    dense_store<E4M3, AM_KSLAB>(S.k, code[h][mt], sc[h], xk[h], there[h], mt, mt, key + 64 * h, lane);
                }
                tc::fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(&S.kready[mt]);
            }
            if (!ok) break;
            kt++;
            more = w.next_tile(a);
            if (more) fetch();
        }
    } else {
        // ================================================ the sums
        const int key = tid - 32 * DN_KWARPS;                          // tensor-memory lane
        const uint32_t lane_base = (uint32_t)(key & ~31) << 16;
        uint32_t kt = 0;
        float sum = 0.0f, kf = -1.0f;
        for (uint32_t p = 0;; p++) {
            const uint32_t d = p % AM_RING;
            if (!dense_wait(&S.sbar[d], (p / AM_RING) & 1, &S.abort, a.polls, c.status)) break;
            tc::tc_fence_after();
            const AmProduct m = S.prod[d];
            if (m.flags & AM_STOP) break;
            if (m.flags & AM_NEW_TILE) kf = S.kf[kt % AM_KRING][key];
            float s[2] = {0.0f, 0.0f};
#pragma unroll
            for (int h = 0; h < CSA2_HEADS; h += 32) {
                uint32_t v[32], u[32];
                tc::tmem_ld32(tmem + 128u * d + h + lane_base, v);
                tc::tmem_ld32(tmem + 128u * d + 64u + h + lane_base, u);
                tc::tmem_ld_wait(v);
                tc::tmem_ld_wait(u);
                auto at = [&](int i) { return __uint_as_float(v[i]) + __uint_as_float(u[i]); };
#pragma unroll
                for (int i = 0; i < 32; i += 4) {
                    const float4 f = *reinterpret_cast<const float4 *>(&S.row[d].f[h + i]);
                    const float4 z = *reinterpret_cast<const float4 *>(&S.row[d].z[h + i]);
                    // one rounding at the size of l - lse
                    s[0] += exp2_approx(fmaf(at(i), f.x * kf, -z.x) * kLog2e);
                    s[1] += exp2_approx(fmaf(at(i + 1), f.y * kf, -z.y) * kLog2e);
                    s[0] += exp2_approx(fmaf(at(i + 2), f.z * kf, -z.z) * kLog2e);
                    s[1] += exp2_approx(fmaf(at(i + 3), f.w * kf, -z.w) * kLog2e);
                }
            }
            tc::tc_fence_before();
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(&S.fbar[d]);
            if (kf >= 0.0f && key < m.lim) sum += s[0] + s[1];
            if (m.flags & AM_SUM) {
                const int64_t e = m.e0 + key;
                if (a.chunks > 1) a.part[((int64_t)m.chunk * bt.batch + m.b) * a.tiles * AM_KEYS + e] = sum;
                else if (sum != 0.0f) a.acc[m.b * a.ld + e] += sum;    // (a row that saw it, and a page that holds it)
                sum = 0.0f;
            }
            kt += (m.flags & AM_LAST) != 0;
        }
    }
    pdl_launch_dependents();
    tc::tc_fence_before();
    __syncthreads();
    tc::tc_fence_after();
    if (warp == 0) tc::tmem_dealloc(tmem, AM_TMEM_COLS);
}

// The sums of the row chunks added, in order.
__global__ void __launch_bounds__(256) k_weights_join(const __grid_constant__ AmArgs a)
{
    pdl_wait();
    const int64_t n = a.tiles * AM_KEYS, all = a.bt.batch * n;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < all; i += (int64_t)gridDim.x * 256) {
        const int64_t b = i / n, e = i % n;
        float s = 0.0f;
        for (int p = 0; p < a.chunks; p++) s += a.part[p * all + i];
        if (s != 0.0f) a.acc[b * a.ld + e] += s;
    }
}

// Several rows per sequence: [rows] images, factors and entry counts, the chunks' sums.
struct AmSpace {
    int64_t rows, tiles;
    int chunks;
    size_t row_at, vis_at, part_at, bytes;
    explicit AmSpace(const csa2_batch &bt)
    {
        rows = (int64_t)bt.batch * bt.nq;
        tiles = (bt.max_entries + AM_KEYS - 1) / AM_KEYS;
        const int64_t want = tiles > 0 ? (AM_UNITS + bt.batch * tiles - 1) / (bt.batch * tiles) : 1;
        chunks = (int)std::min<int64_t>(want, bt.nq);
        row_at = (size_t)rows * DN_QBYTES;
        vis_at = row_at + (size_t)rows * sizeof(AmRow);
        part_at = (vis_at + (size_t)rows * 4 + 255) & ~(size_t)255;
        bytes = (part_at + (chunks > 1 ? (size_t)chunks * bt.batch * tiles * AM_KEYS * 4 : 0) + 255) & ~(size_t)255;
    }
};

static int launch_weights_rows(const csa2_cache &c, const csa2_batch &bt, const csa2_swa &swa, const int64_t *evicted,
                               const uint16_t *q, float sm_scale, const float *lse, float *acc, int64_t ld, void *ws,
                               int sms, cudaStream_t st)
{
    const AmSpace sp(bt);
    uint8_t *w = static_cast<uint8_t *>(ws);
    AmRow *row = reinterpret_cast<AmRow *>(w + sp.row_at);
    int32_t *vis = reinterpret_cast<int32_t *>(w + sp.vis_at);
    float *part = sp.chunks > 1 ? reinterpret_cast<float *>(w + sp.part_at) : nullptr;
    const int64_t parts = part ? (int64_t)sp.chunks * bt.batch * sp.tiles * AM_KEYS : 0;
    if (const int s = launch_pdl(k_weights_queries, dim3((unsigned)sp.rows), dim3(256), 0, st, bt, evicted, swa, q, lse,
                                 sm_scale, w, row, vis, part, parts))
        return s;
    const AmArgs a = {c, bt, w, row, vis, sp.chunks, acc, ld, part, sp.tiles, wait_polls()};
    auto kern = c.kv_format == CSA2_KV_FP4_E4M3 ? k_weights_rows<true> : k_weights_rows<false>;
    const size_t smem = sizeof(AmSmem) + 1024;
    if (const int s = kernel_smem_limit((const void *)kern, smem, 100)) return s;
    const int64_t units = (int64_t)bt.batch * sp.tiles * sp.chunks;
    if (const int s = launch_pdl(kern, dim3((unsigned)std::min<int64_t>(sms, units)), dim3(AM_THREADS), smem, st, a)) return s;
    if (!part) return CSA2_OK;
    const int64_t blocks = std::min<int64_t>((parts / sp.chunks + 255) / 256, (int64_t)sms * 8);
    return launch_pdl(k_weights_join, dim3((unsigned)blocks), dim3(256), 0, st, a);
}

// The fixed-point sums of a selecting call added to the accumulators.
__global__ void __launch_bounds__(256) k_weights_add(const unsigned long long *__restrict__ fix, int64_t batch, int64_t n,
                                                      float *__restrict__ acc, int64_t ld)
{
    pdl_wait();
    const int64_t all = batch * n;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < all; i += (int64_t)gridDim.x * 256) {
        const unsigned long long v = fix[i];
        if (v) acc[i / n * ld + i % n] += (float)((double)v * 0x1p-40);
    }
}

size_t attn_weights_workspace_bytes(const csa2_batch &bt, int k)
{
    if (bt.nq == 1 || bt.max_entries == 0) return 0;
    return k > 0 ? ((size_t)bt.batch * bt.max_entries * 8 + 255) & ~(size_t)255 : AmSpace(bt).bytes;
}

int launch_attn_weights(const csa2_cache &c, const csa2_batch &bt, const csa2_swa &swa, const int64_t *evicted,
                        const uint16_t *q, float sm_scale, const int32_t *idx, int k, const float *lse, float *acc,
                        int64_t ld, void *ws, cudaStream_t st)
{
    const int sms = device_sms();
    if (sms <= 0) return CSA2_ERR_CUDA;
    if (bt.max_entries == 0) return CSA2_OK;
    if (!idx && bt.nq > 1) return launch_weights_rows(c, bt, swa, evicted, q, sm_scale, lse, acc, ld, ws, sms, st);
    ApArgs a = {c, bt, swa, evicted, q, lse, idx, k, sm_scale, acc, ld, nullptr, wait_polls()};
    const size_t fix_bytes = attn_weights_workspace_bytes(bt, k);
    if (fix_bytes) {
        a.fix = static_cast<unsigned long long *>(ws);
        const cudaError_t e = cudaMemsetAsync(ws, 0, (size_t)bt.batch * bt.max_entries * 8, st);
        if (e != cudaSuccess) {
            set_cuda_error(e);
            return CSA2_ERR_CUDA;
        }
    }
    const bool e4 = c.kv_format == CSA2_KV_FP4_E4M3;
    auto kern = idx ? (e4 ? k_weights_tiles<true, true> : k_weights_tiles<false, true>)
                    : (e4 ? k_weights_tiles<true, false> : k_weights_tiles<false, false>);
    const size_t smem = sizeof(ApSmem) + 1024;
    if (const int s = kernel_smem_limit((const void *)kern, smem, 100)) return s;
    const int64_t tiles = idx ? (int64_t)bt.batch * bt.nq * ((k + DN_KEYS - 1) / DN_KEYS)
                              : (int64_t)bt.batch * ((bt.max_entries + DN_KEYS - 1) / DN_KEYS);
    if (const int s = launch_pdl(kern, dim3((unsigned)std::min<int64_t>(sms, tiles)), dim3(32 * ap_warps(idx != nullptr)), smem, st, a)) return s;
    if (!fix_bytes) return CSA2_OK;
    const int64_t blocks = std::min<int64_t>(((int64_t)bt.batch * bt.max_entries + 255) / 256, (int64_t)sms * 8);
    return launch_pdl(k_weights_add, dim3((unsigned)blocks), dim3(256), 0, st, (const unsigned long long *)a.fix,
                      (int64_t)bt.batch, bt.max_entries, acc, ld);
}

}  // namespace csa2
