// Pieces shared by the operators over the whole FP4 cache (csa2_dense_attn.cu,
// csa2_attn_weights.cu): which entries and window rows a query attends to, the
// loads and exact dequantisation of a page of keys into a 128-byte-swizzled f16
// operand, and the query operand.
//
// The operands are f16 because the hardware turns two FP4 codes into an f16x2 in
// one instruction: a 32-bit word of codes takes 5 issue cycles with its scales, by
// shifts and masks into bf16 21.  f16's range is made enough by powers of two that
// the operands leave out:
//   key    k = K' 2^(Xk - 12) f: for MXFP4 Xk is the largest block exponent of
//          the entry (blocks of zeros aside) and f = 1, so its blocks keep every
//          bit down to 2^-36 of the largest; for the E4M3 scales Xk = 12, f = 1
//          (every product of a code and a scale is an f16); for a window row Xk
//          - 12 and f are the exponent and the mantissa (at most 1) of its scale,
//          K' its codes.  A key of zeros has no exponent: its logit is 0 and it adds
//          nothing to the output, (Xk, f) = (DN_XZERO, 0);
//   query  q_h = Q'_h 2^e_h with the head's largest element in [2^13, 2^14):
//          elements down to 2^-27 of it keep their bf16 value.
#pragma once

#include "csa2_attn_common.cuh"

namespace csa2 {

constexpr int DN_KEYS = CSA2_PAGE;                 // keys per tile (MMA M of the logit product): one page
constexpr int DN_KWARPS = 8, DN_WKEYS = 8;         // the warps that load and dequantise keys, eight each
static_assert(DN_KWARPS * DN_WKEYS == DN_KEYS, "a quad of lanes per key");
constexpr int DN_SLABS = CSA2_HEAD_DIM / 64;       // 64-dim slabs of the operands
constexpr uint32_t DN_KSLAB = DN_KEYS * 128;       // bytes of a slab of the key tile
constexpr uint32_t DN_KBYTES = DN_SLABS * DN_KSLAB, DN_QBYTES = DN_SLABS * CSA2_HEADS * 128;
constexpr uint32_t DN_QSLAB = CSA2_HEADS * 128;    // bytes of a slab of the query operand

constexpr float DN_XOFF = 12.0f;                   // K' is the key times 2^(DN_XOFF - Xk)
// Smallest Xk: the sums of weights divided by 2^Xk stay finite.  (The codes of a block of
// scale 2^-101 are still exact.)
constexpr int DN_XMIN = -66;
constexpr float DN_XZERO = -68.0f;                 // a key of zeros: below the others, which set the reference
constexpr float kLn2 = 0.6931471805599453f, kLog2e = 1.4426950408889634f;

// What query row r attends to.
struct DenseRow {
    int64_t vis;    // entries 0 .. vis - 1 of sequence b
    int64_t lo, t;  // window tokens lo .. t (none if lo > t)
    int b;
    int tiles;      // of 128 keys: ceil(vis / 128), then the window's; at least 1
};

// Entry j of a sequence that has lost `ev` entries to an eviction stands for a
// token group at or before group j + ev, so the causal bound moves down by ev.
__device__ __forceinline__ int64_t dense_visible(const csa2_batch &bt, const int64_t *evicted, int b, int64_t t)
{
    int64_t n = bt.n_entries[b];
    int64_t lim = t < 0 ? 0 : (t + 1) / bt.m - (evicted ? evicted[b] : 0);
    if (lim < n) n = lim;
    if (n > bt.max_entries) n = bt.max_entries;
    return n < 0 ? 0 : n;
}

__device__ __forceinline__ DenseRow dense_row(const csa2_batch &bt, const int64_t *evicted, const csa2_swa &swa,
                                              int64_t r)
{
    DenseRow R;
    R.b = (int)(r / bt.nq);
    R.t = bt.q_pos[r];
    R.vis = dense_visible(bt, evicted, R.b, R.t);
    R.lo = R.t + 1;
    if (swa.codes) {
        const int64_t s0 = swa.start ? swa.start[R.b] : 0;
        R.lo = R.t - (CSA2_SWA_WINDOW - 1);
        R.lo = R.lo < s0 ? s0 : R.lo;
        R.lo = R.lo < 0 ? 0 : R.lo;
        R.lo = R.lo > R.t ? R.t + 1 : R.lo;
        // m = 1: entry j is token j, and the window row stays
        if ((swa.flags & CSA2_ATTN_DEDUP_WINDOW) && bt.m == 1 && R.lo <= R.t && R.vis > R.lo) R.vis = R.lo;
    }
    const int n = (int)((R.vis + 127) / 128) + (int)((R.t - R.lo + 128) / 128);
    R.tiles = n > 0 ? n : 1;
    return R;
}

// The two FP4 codes of byte i of w (low nibble first) -> f16x2, i = 0 .. 3.
__device__ __forceinline__ uint4 e2m1x8_to_f16(uint32_t w)
{
    uint4 o;
    asm("{\n .reg .b8 a, b, c, d;\n mov.b32 {a, b, c, d}, %4;\n"
        " cvt.rn.f16x2.e2m1x2 %0, a;\n cvt.rn.f16x2.e2m1x2 %1, b;\n"
        " cvt.rn.f16x2.e2m1x2 %2, c;\n cvt.rn.f16x2.e2m1x2 %3, d;\n}\n"
        : "=r"(o.x), "=r"(o.y), "=r"(o.z), "=r"(o.w)
        : "r"(w));
    return o;
}

__device__ __forceinline__ uint32_t f16x2_mul(uint32_t a, uint32_t b)
{
    uint32_t r;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// 2^d as an f16 in both halves (0 below 2^-24; d <= 15).
__device__ __forceinline__ uint32_t pow2_f16x2(int d)
{
    const float f = exp2i(d < -100 ? -100 : d);
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %1;" : "=r"(r) : "f"(f));
    return r;
}

// A lane's share of an entry's loads: of the key that its quad of lanes holds,
// the 16 code bytes of dims 128 mt + 32 (lane % 4) .. of part mt, and their block
// scales.  (Four lanes take 64 contiguous bytes of a key and a warp eight
// neighbouring entries of one page, so every sector that is fetched is used.)
__device__ __forceinline__ uint4 dense_codes(const csa2_cache &c, int64_t slot, int mt, int lane)
{
    return __ldg(reinterpret_cast<const uint4 *>(c.kv_codes + slot * 256) + 4 * mt + (lane & 3));
}

// The lane's scales of the four parts, as loaded (nothing waits for them here).
template <bool E4M3>
__device__ __forceinline__ uint4 dense_scales(const csa2_cache &c, int64_t slot, int lane)
{
    if (!E4M3) return __ldg(reinterpret_cast<const uint4 *>(c.kv_scales + slot * 16));
    const uint16_t *sc = reinterpret_cast<const uint16_t *>(c.kv_scales + slot * 32) + (lane & 3);
    return make_uint4(__ldg(sc), __ldg(sc + 4), __ldg(sc + 8), __ldg(sc + 12));
}

// ... and packed: byte mt (E8M0) or half-word mt (E4M3).
template <bool E4M3>
__device__ __forceinline__ uint2 dense_pack_scales(uint4 w, int lane)
{
    if (E4M3) return make_uint2(w.x | w.y << 16, w.z | w.w << 16);
    const int sh = 8 * (lane & 3);
    return make_uint2(((w.x >> sh) & 0xFFu) | ((w.y >> sh) & 0xFFu) << 8 | ((w.z >> sh) & 0xFFu) << 16 | ((w.w >> sh) & 0xFFu) << 24, 0);
}

// First slot of the page that holds entry e of sequence b (which exists), or
// -1 and a flag if its id is outside the cache.
__device__ __forceinline__ int64_t dense_page_slot(const csa2_cache &c, int32_t page, int lane)
{
    if (page >= 0 && ((int64_t)page + 1) * CSA2_PAGE <= c.num_slots) return (int64_t)page * CSA2_PAGE;
    if (lane == 0) flag(c.status, CSA2_DEV_BAD_PAGE);
    return -1;
}

// An entry with E4M3 scales is all zeros, told by its codes.  Called by the whole warp.
__device__ __forceinline__ bool dense_zero_codes(const uint4 (&codes)[4])
{
    uint32_t any = 0;
#pragma unroll
    for (int mt = 0; mt < 4; mt++) any |= codes[mt].x | codes[mt].y | codes[mt].z | codes[mt].w;
    any &= 0x77777777u;
    if (__all_sync(0xffffffffu, any != 0)) return false;
    any |= __shfl_xor_sync(0xffffffffu, any, 1);
    any |= __shfl_xor_sync(0xffffffffu, any, 2);
    return any == 0;
}

// The exponent Xk of a quad's entry, from its four lanes' blocks; *zero: the
// entry is all zeros (MXFP4).
template <bool E4M3>
__device__ __forceinline__ int dense_exponent(const uint4 (&codes)[4], uint2 scales, bool *zero)
{
    *zero = false;
    if (E4M3) return (int)DN_XOFF;
    int x = 0;                                     // the byte: X + 127
#pragma unroll
    for (int mt = 0; mt < 4; mt++) {
        const uint4 c = codes[mt];
        const int b = (int)((scales.x >> (8 * mt)) & 0xFFu);
        if (((c.x | c.y | c.z | c.w) & 0x77777777u) && b > x) x = b;
    }
    x = max(x, __shfl_xor_sync(0xffffffffu, x, 1));
    x = max(x, __shfl_xor_sync(0xffffffffu, x, 2));
    *zero = x == 0;
    return max(x - 127, DN_XMIN);
}

// Write part mt of a key's codes into its row of the f16 key tile (zeros where
// there is no key).  Half of the lanes write their second 16 dims first, so that
// the eight lanes of a store hit eight different 16-byte banks.  SLAB: bytes of a
// slab of the tile.
template <bool E4M3, uint32_t SLAB = DN_KSLAB>
__device__ __forceinline__ void dense_store(uint8_t *ktile, uint4 codes, uint2 scales, int xk, bool exists, int at,
                                            int mt, int key, int lane)
{
    const int ck = lane & 3;
    const bool swap = ck & 2;
    uint8_t *row = ktile + (uint32_t)(2 * mt + (ck >> 1)) * SLAB + (uint32_t)key * 128u;
    const uint32_t c0 = (4u * (ck & 1) + (swap ? 2u : 0u)) ^ ((uint32_t)key & 7u);
    uint32_t fa, fb;
    if (E4M3) {
        const uint32_t b2 = (at < 2 ? scales.x : scales.y) >> (16 * (at & 1));
        const uint32_t v = e4m3x2_to_f16x2((uint16_t)b2);
        const uint32_t lo = __byte_perm(v, v, 0x1010), hi = __byte_perm(v, v, 0x3232);
        fa = swap ? hi : lo;
        fb = swap ? lo : hi;
    } else {
        // (a block of zeros may have a larger exponent than Xk)
        fa = fb = pow2_f16x2(min((int)((scales.x >> (8 * at)) & 0xFFu) - 127 - xk, 0) + (int)DN_XOFF);
    }
    uint32_t w[4] = {swap ? codes.z : codes.x, swap ? codes.w : codes.y, swap ? codes.x : codes.z, swap ? codes.y : codes.w};
    if (!exists) {
        w[0] = w[1] = w[2] = w[3] = 0;
        fa = fb = 0;
    }
#pragma unroll
    for (int j = 0; j < 4; j++) {
        const uint32_t sc = j < 2 ? fa : fb;
        uint4 o = e2m1x8_to_f16(w[j]);
        o.x = f16x2_mul(o.x, sc);
        o.y = f16x2_mul(o.y, sc);
        o.z = f16x2_mul(o.z, sc);
        o.w = f16x2_mul(o.w, sc);
        *reinterpret_cast<uint4 *>(row + ((c0 ^ (uint32_t)j) << 4)) = o;
    }
}

// Part mt of a key of a window tile: the e4m3 codes of token tok.
template <uint32_t SLAB>
__device__ __forceinline__ void dense_store_window(uint8_t *ktile, const csa2_swa &swa, const DenseRow &R, int64_t tok,
                                                   int mt, int key, int lane)
{
    const int ck = lane & 3;
    const bool swap = ck & 2;
    uint4 v0 = make_uint4(0, 0, 0, 0), v1 = v0;
    if (tok <= R.t) {
        const int64_t off = (int64_t)R.b * swa.rows + tok % swa.rows;
        const uint4 *src = reinterpret_cast<const uint4 *>(swa.codes + off * CSA2_HEAD_DIM) + 8 * mt + 2 * ck;
        v0 = __ldg(src + (swap ? 1 : 0));
        v1 = __ldg(src + (swap ? 0 : 1));
    }
    uint8_t *row = ktile + (uint32_t)(2 * mt + (ck >> 1)) * SLAB + (uint32_t)key * 128u;
    const uint32_t c0 = (4u * (ck & 1) + (swap ? 2u : 0u)) ^ ((uint32_t)key & 7u);
    const uint32_t w[8] = {v0.x, v0.y, v0.z, v0.w, v1.x, v1.y, v1.z, v1.w};
#pragma unroll
    for (int j = 0; j < 4; j++)
        *reinterpret_cast<uint4 *>(row + ((c0 ^ (uint32_t)j) << 4)) =
            make_uint4(e4m3x2_to_f16x2((uint16_t)w[2 * j]), e4m3x2_to_f16x2((uint16_t)(w[2 * j] >> 16)),
                       e4m3x2_to_f16x2((uint16_t)w[2 * j + 1]), e4m3x2_to_f16x2((uint16_t)(w[2 * j + 1] >> 16)));
}

// (Xk, f) of the window row that a quad of lanes holds; (-inf, 0) where there is
// no row, (DN_XZERO, 0) for one of zeros.  The quantiser gives a row of zeros the scale 1, which may be far above
// its neighbours': such a row is told by its codes.  Called by the whole warp.
__device__ __forceinline__ float2 dense_window_scale(const csa2_swa &swa, const DenseRow &R, int64_t tok, int lane)
{
    const bool row = tok <= R.t;
    const int64_t off = row ? (int64_t)R.b * swa.rows + tok % swa.rows : 0;
    const float s = row ? __ldg(swa.scales + off) : 0.0f;
    bool zero = s == 0.0f;
    if (__any_sync(0xffffffffu, row && s == 1.0f)) {
        uint32_t any = 0;
        if (row) {
            const uint4 *src = reinterpret_cast<const uint4 *>(swa.codes + off * CSA2_HEAD_DIM) + (lane & 3);
#pragma unroll
            for (int i = 0; i < 8; i++) {
                const uint4 v = __ldg(src + 4 * i);
                any |= (v.x | v.y | v.z | v.w) & 0x7F7F7F7Fu;
            }
        }
        any |= __shfl_xor_sync(0xffffffffu, any, 1);
        any |= __shfl_xor_sync(0xffffffffu, any, 2);
        zero = zero || any == 0;
    }
    if (!row) return make_float2(-INFINITY, 0.0f);
    if (zero) return make_float2(DN_XZERO, 0.0f);
    const int e = max((int)((__float_as_uint(s) >> 23) & 255u) - 126, DN_XMIN - (int)DN_XOFF);    // |f| <= 1
    return make_float2((float)e + DN_XOFF, s * exp2i(-min(e, 126)));
}

// The query operand of a row: 64 heads x 512 dims, K-major slabs of 64 dims, and
// each head's 2^e_h, by `warps` warps (each takes whole heads, two at a time).
__device__ __forceinline__ void dense_load_q(uint8_t *qs, float *qe, const uint16_t *q, int64_t r, int warp, int warps,
                                             int lane)
{
#pragma unroll 1
    for (int h0 = 2 * warp; h0 < CSA2_HEADS; h0 += 2 * warps) {
        const uint4 *src = reinterpret_cast<const uint4 *>(q + (r * CSA2_HEADS + h0) * CSA2_HEAD_DIM);
        uint4 v[2][2];
#pragma unroll
        for (int u = 0; u < 4; u++) v[u >> 1][u & 1] = __ldg(src + 32 * u + lane);
#pragma unroll
        for (int hh = 0; hh < 2; hh++) {
            // bf16 magnitudes order as integers
            uint32_t m = 0;
#pragma unroll
            for (int u = 0; u < 2; u++)
                m = __vmaxu2(m, __vmaxu2(__vmaxu2(v[hh][u].x & 0x7FFF7FFFu, v[hh][u].y & 0x7FFF7FFFu),
                                         __vmaxu2(v[hh][u].z & 0x7FFF7FFFu, v[hh][u].w & 0x7FFF7FFFu)));
            const uint32_t top = __reduce_max_sync(0xffffffffu, max(m & 0xFFFFu, m >> 16));
            const int e = top == 0 ? 0 : max((int)(top >> 7) - 127 - 13, -126);
            const float f = exp2i(-e);
            if (lane == 0) qe[h0 + hh] = exp2i(e);
#pragma unroll
            for (int u = 0; u < 2; u++) {
                const uint32_t in[4] = {v[hh][u].x, v[hh][u].y, v[hh][u].z, v[hh][u].w};
                uint32_t out[4];
#pragma unroll
                for (int j = 0; j < 4; j++) {
                    const float a = __uint_as_float(in[j] << 16) * f, b = __uint_as_float(in[j] & 0xFFFF0000u) * f;
                    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(out[j]) : "f"(b), "f"(a));
                }
                const int ck = 32 * u + lane, h = h0 + hh;
                *reinterpret_cast<uint4 *>(qs + (uint32_t)(ck >> 3) * DN_QSLAB + (uint32_t)h * 128u +
                                           (((uint32_t)(ck & 7) ^ (uint32_t)(h & 7)) << 4)) =
                    make_uint4(out[0], out[1], out[2], out[3]);
            }
        }
    }
}

// Descriptors' lower words: start address and leading offset (16-byte units);
// the products step through an operand by adding to it.
__device__ __forceinline__ uint64_t dense_desc(const void *p, uint32_t lbo) { return tc::smem_desc(tc::smem_u32(p), lbo, 1024, tc::kSwizzle128B); }

// This warp's 16 rows (keys) and 32 columns (heads) of a 64-row accumulator,
// whose row 16 w + i is tensor-memory lane 32 w + i: registers 4 b + e and 4 b + 2
// + e hold rows lane / 4 and lane / 4 + 8, column 8 b + 2 (lane % 4) + e.
__device__ __forceinline__ void tmem_ld_16x32(uint32_t taddr, uint32_t (&r)[16])
{
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
}

// The register share of this warp's warpgroup, out of the launch's: in the branch
// of its role, which all four warps take.
template <int N>
__device__ __forceinline__ void set_registers_up()
{
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void set_registers_down()
{
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// The dynamic shared memory as a T at a 1,024-byte boundary, by an offset (an
// address rounded as an integer loses its state space: generic loads and stores).
template <class T>
__device__ __forceinline__ T &dense_smem()
{
    extern __shared__ uint8_t smem_raw[];
    return *reinterpret_cast<T *>(smem_raw + ((0u - tc::smem_u32(smem_raw)) & 1023u));
}

// One lane of the (converged) warp.
__device__ __forceinline__ bool elect_one()
{
    uint32_t r;
    asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(r));
    return r != 0;
}

// Barrier of `threads` threads; true for all if v holds for any.
__device__ __forceinline__ bool named_bar_or(uint32_t id, uint32_t threads, bool v)
{
    uint32_t r;
    asm volatile("{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n barrier.cta.red.or.pred q, %2, %3, p;\n selp.u32 %0, 1, 0, q;\n}\n"
                 : "=r"(r)
                 : "r"((uint32_t)v), "r"(id), "r"(threads)
                 : "memory");
    return r != 0;
}

// Two fp32 operations in one instruction.
__device__ __forceinline__ float2 f32x2_mul(float2 a, float2 b)
{
    float2 r;
    asm("{\n .reg .b64 a, b, r;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %5};\n mul.rn.f32x2 r, a, b;\n mov.b64 {%0, %1}, r;\n}\n"
        : "=f"(r.x), "=f"(r.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return r;
}
__device__ __forceinline__ float2 f32x2_fma(float2 a, float2 b, float2 c)
{
    float2 r;
    asm("{\n .reg .b64 a, b, c, r;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %5};\n mov.b64 c, {%6, %7};\n"
        " fma.rn.f32x2 r, a, b, c;\n mov.b64 {%0, %1}, r;\n}\n"
        : "=f"(r.x), "=f"(r.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return r;
}
__device__ __forceinline__ float2 f32x2_sub(float2 a, float2 b)
{
    float2 r;
    asm("{\n .reg .b64 a, b, r;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %5};\n sub.rn.f32x2 r, a, b;\n mov.b64 {%0, %1}, r;\n}\n"
        : "=f"(r.x), "=f"(r.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return r;
}

__device__ __forceinline__ float exp2_approx(float x)
{
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// Bounded wait of a whole warp on a phase, cut short by *abort; a timeout is
// flagged and sets *abort.  The same for all lanes, which leave it together (the
// tensor-memory instructions want a converged warp); false: the phase has not
// completed.
__device__ __forceinline__ bool dense_poll(uint64_t *bar, uint32_t parity, volatile int *abort, uint32_t polls, int32_t *status)
{
    bool ok = false;
    for (uint32_t i = 0; !ok && i < polls && !*abort; i++) {
        if (i > 4096) __nanosleep(64);
        ok = tc::mbar_try_wait(bar, parity);
    }
    if (!ok && !*abort) {
        flag(status, CSA2_DEV_TIMEOUT);
        *abort = 1;
    }
    return __all_sync(0xffffffffu, ok);
}

__device__ __forceinline__ bool dense_wait(uint64_t *bar, uint32_t parity, volatile int *abort, uint32_t polls, int32_t *status)
{
    if (__all_sync(0xffffffffu, tc::mbar_test(bar, parity))) return true;
    return dense_poll(bar, parity, abort, polls, status);
}

// Exclusive sum over the block of v (threads in order); *total gets the sum.
__device__ __forceinline__ int64_t block_exclusive_sum(int64_t v, int64_t *warp_sums, int64_t *total)
{
    const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
    int64_t x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    if (lane == 31) warp_sums[wid] = x;
    __syncthreads();
    int64_t base = 0, all = 0;
    for (int i = 0; i < (int)(blockDim.x >> 5); i++) {
        const int64_t s = warp_sums[i];
        if (i < wid) base += s;
        all += s;
    }
    *total = all;
    __syncthreads();
    return base + x - v;
}

}  // namespace csa2
