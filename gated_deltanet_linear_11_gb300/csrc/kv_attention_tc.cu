// kv_attention_tc.cu -- gdn_kv_attention for many new rows (pieces of prompts), on tcgen05:
// bf16 queries, D = 64 or 128.
//
// One CTA takes 256 rows of a kv-head (G query heads x m tokens, token-major) as two tiles
// of 128, and walks the keys in tiles of 128:
//     S = Q K^T       P = 2^(S f - ref)       O += P V
// S, P and O live in TMEM (P over S, as the A operand of P V); K and V are unpacked once per
// CTA into fp16 shared-memory tiles that both row tiles use.
//
// Scores are as exact as fp32 sums allow: a key is minimum + scale * code, and scale * code
// (15 bits) goes in as an fp16 pair hi + lo, the minima as sixteen more columns against the
// sums of q over each group (again a pair), so a 128-deep product becomes 272 deep:
//     q.k = q.(hi + lo) + sum_g (sum of q over g) min_g.
// Where a scale of 16 keys would carry 15 * scale past fp16, that block's scales and minima go
// in at a quarter, and its scores take the factor of four in fp32.
//
// Warps 0-7: softmax, a thread owning one row of a tile; warps 8-15: unpacking, a warp
// taking 16 records of keys, then of values, straight from the cache into registers while
// the ones before are converted; warp 16: products.  The two row tiles take turns: while one
// is in its softmax the tensor pipe works for the other.
//
// A 256 x 128 step has 2 x (1088 + 512) clocks of products at D = 128 (operands at 128 bytes
// a clock), 2048 clocks of base-2 exponentials (16 a clock) and about 2600 instructions a
// scheduler, and takes 5500: the scores of both row tiles, then the unpacking of the next
// keys into the one buffer there is room for, form its chain, and the issue slots are half
// taken.  2048 rows of 32 heads on 8 over 10240 keys take 437 us.  Tried and slower: two
// buffers for hi with lo converted again (462 us where this form took 432), sixteen unpacking
// warps (482), two threads a row (486), a warp of products for each row tile (543, their
// softmaxes fall together).
//
// Fewer bits than fp32: q is scaled by a power of two per row into [2^6, 2^7) and held in
// fp16 (exact down to 2^-21 of the largest); a value is minimum + scale * code rounded once
// to fp16 (2^-11, after the sum, so nothing cancels later); p is rounded to fp16, taken
// against a reference within 8 (in powers of two) of the running maximum and lifted by 2^7,
// so it stays below 2^15 and a weight of 2^-31 of the largest is still held.  Scores, sums
// and outputs are fp32.
#include <algorithm>
#include <atomic>

#include "bulk_ptx.cuh"
#include "kv_format.cuh"

namespace gdn {

constexpr int kTcRows = 256;
constexpr int kTcSoftWarps = 8, kTcUnpackWarps = 8;
constexpr int kTcThreads = 32 * (kTcSoftWarps + kTcUnpackWarps + 1);
constexpr float kTcSlack = 8.f;     // how far (log2) the maximum may pass the reference
constexpr uint32_t kTcTopScale = 0x6c43u;   // fp16 4364: 15 times the next one rounds to infinity
constexpr float kTcLift = 7.f;      // weights are kept at 2^7 times their value (below 2^15)

template <int D> struct TcShape {
    static constexpr int NG = D / 32;
    static constexpr int TILE = 128 * D * 2;     // one 128 x D fp16 tile
    static constexpr int BLK = 16384;            // 64 columns of it
};
struct TcBars {
    uint64_t k_full, k_free, v_full[2], v_free[2];
    uint64_t s_full[2], p_full[2], pv[2];   // per row tile
    uint64_t fin;
};
template <int D> struct TcSmem {
    uint8_t q[2][TcShape<D>::TILE];
    uint8_t hi[TcShape<D>::TILE], lo[TcShape<D>::TILE];   // scale * code of the keys
    uint8_t v[2][TcShape<D>::TILE];
    // group sums of q and minima of the keys: [128][16] fp16 in 8 x 8 blocks of 128 bytes
    uint8_t qx[2][4096], kx[4096];
    uint32_t nan_groups[kTcRows];    // groups of the row's output that a NaN value reached
    uint8_t have[2][8];              // per 16 keys of a tile (even, odd): 1 records present,
                                     // 3 and their scores come at a quarter
    uint32_t tmem;
    int abort;
    TcBars bar;
};

__device__ __forceinline__ void tc_arrive(uint64_t *bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" :: "r"(tc::smem_u32(bar)) : "memory");
}
// Bounded wait by a warp; false once any thread of the CTA has given up.
template <int SLEEP_NS = 0>
__device__ __forceinline__ bool tc_wait(uint64_t *bar, uint32_t parity, volatile int *abort) {
    const bool ok = wait_bounded_poll<SLEEP_NS>(bar, parity, abort);
    if (!ok) *abort = 1;
    return __all_sync(0xffffffffu, ok) != 0;
}

// 32-bit instruction descriptor: fp16 A and B, fp32 D.
__device__ constexpr uint32_t idesc_f16(int M, int N, int b_mn) {
    return (1u << 4) | ((uint32_t)b_mn << 16) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t id, uint32_t add) {
    asm volatile("{\n\t.reg .pred p, e;\n\t"
                 "elect.sync _|e, 0xffffffff;\n\t"
                 "setp.ne.b32 p, %4, 0;\n\t"
                 "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}"
                 :: "r"(d), "r"(a), "l"(b), "r"(id), "r"(add) : "memory");
}
__device__ __forceinline__ void tc_st16(uint32_t taddr, const uint32_t (&r)[16]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
                 "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};"
                 :: "r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]),
                    "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]),
                    "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]) : "memory");
}
__device__ __forceinline__ void tc_st8(uint32_t taddr, const uint32_t (&r)[8]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};"
                 :: "r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]),
                    "r"(r[6]), "r"(r[7]) : "memory");
}
__device__ __forceinline__ float tc_ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ uint32_t h2_bits(__half2 h) { return *reinterpret_cast<const uint32_t *>(&h); }
__device__ __forceinline__ __half2 bits_h2(uint32_t u) { return *reinterpret_cast<const __half2 *>(&u); }

// Descriptor of such a [128][16] operand: K-major without swizzle, 128 bytes between the two
// blocks of a row group, 256 to the next eight rows.
__device__ __forceinline__ uint64_t desc_x(const uint8_t *p) {
    return (uint64_t)((tc::smem_u32(p) >> 4) & 0x3FFFu) | (uint64_t)(128 >> 4) << 16 |
           (uint64_t)(256 >> 4) << 32 | (uint64_t)1u << 46;
}
__device__ __forceinline__ uint32_t at_x(int row, int half) { return (row >> 3) * 256 + half * 128 + (row & 7) * 16; }

// Codes of the nibble pairs (i, i + 4) of a word, i = 0..3, as fp16: 1024 + u, less 1024, or
// 1024 + 16 u, over 16 and less 64 (both exact).
__device__ __forceinline__ void codes_of(uint32_t w, __half2 (&u)[4]) {
    const __half2 k1024 = __floats2half2_rn(1024.f, 1024.f);
    const __half2 k16 = __floats2half2_rn(0.0625f, 0.0625f), k64 = __floats2half2_rn(-64.f, -64.f);
#pragma unroll
    for (int i = 0; i < 4; i += 2) {
        const uint32_t x = w >> (4 * i);
        u[i] = __hsub2(bits_h2((x & 0x000F000Fu) | 0x64006400u), k1024);
        u[i + 1] = __hfma2(bits_h2((x & 0x00F000F0u) | 0x64006400u), k16, k64);
    }
}
__device__ __forceinline__ bool pair_nonfinite(uint32_t w) {
    return (w & 0x7c00u) == 0x7c00u || (w & 0x7c000000u) == 0x7c000000u;
}

template <int D>
__global__ void __launch_bounds__(kTcThreads, 1)
kv_attention_tc_kernel(KvView kv, const bf16 *__restrict__ q, bf16 *__restrict__ o,
                       float *__restrict__ lse, int64_t q_tok, int64_t o_tok, int Hq, int min_rows,
                       int max_kv_len, float scale, int32_t *status) {
    using R = KvRec<D>;
    using T = TcShape<D>;
    constexpr int NG = T::NG, REC = R::BYTES;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    TcSmem<D> &S = *reinterpret_cast<TcSmem<D> *>(smem_raw);
    if (tc::smem_u32(smem_raw) & 1023u) {        // the tiles' swizzle needs it; never seen
        if (threadIdx.x == 0) report(status, GDN_ERR_CUDA);
        return;
    }
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int hkv = blockIdx.y, n = blockIdx.z;
    const int t0 = kv.cu[n], m = kv.cu[n + 1] - t0, len = kv.kv_lens[n];
    const int G = Hq / kv.Hkv, rows = G * m;
    if (Hq * m < min_rows) return;               // the other kernel's
    // the row tiles with the most keys first
    const int tiles = (rows + kTcRows - 1) / kTcRows;
    if ((int)blockIdx.x >= tiles) return;
    const int row0 = (tiles - 1 - (int)blockIdx.x) * kTcRows;
    if (len < 0 || len > max_kv_len || len > kv.capacity()) {
        if (tid == 0) report(status, GDN_ERR_SEQLENS);
        return;
    }
    const int see_last = len - m + (min(row0 + kTcRows, rows) - 1) / G + 1;
    const int steps = see_last > 0 ? (see_last + 127) / 128 : 0;
    volatile int *abort = &S.abort;

    if (warp == 0) {
        tc::tmem_alloc(&S.tmem, 512);
        tc::tmem_relinquish();
    }
    if (tid == 0) {
        S.abort = 0;
        tc::mbar_init(&S.bar.k_full, kTcUnpackWarps);
        tc::mbar_init(&S.bar.k_free, 1);
        for (int x = 0; x < 2; ++x) {
            tc::mbar_init(&S.bar.v_full[x], kTcUnpackWarps);
            tc::mbar_init(&S.bar.v_free[x], 1);
            tc::mbar_init(&S.bar.s_full[x], 1);
            tc::mbar_init(&S.bar.p_full[x], 4);
            tc::mbar_init(&S.bar.pv[x], 1);
        }
        tc::mbar_init(&S.bar.fin, 1);
        tc::mbar_fence_init();
    }
    if (tid < kTcRows) S.nan_groups[tid] = 0;

    // ---- q: a thread converts its row; element order inside eight: 0 4 1 5 2 6 3 7, as the
    // keys' nibble pairs come
    const int rt = warp >> 2;                    // softmax warps: row tile
    const int row = row0 + tid;                  // softmax threads: their row
    float fac = 0.f;
    if (warp < kTcSoftWarps) {
        float mx = 0.f;
        const bf16 *src = q + (int64_t)(t0 + (row < rows ? row / G : 0)) * q_tok +
                          (int64_t)(hkv * G + (row < rows ? row % G : 0)) * D;
#pragma unroll
        for (int c = 0; c < D / 8; ++c) {
            float f[8];
            unpack8(reinterpret_cast<const uint4 *>(src)[c], f);
#pragma unroll
            for (int e = 0; e < 8; ++e) mx = fmaxf(mx, fabsf(f[e]));
        }
        if (row >= rows) mx = 0.f;
        const int ex = mx < INFINITY ? min(6 + 127 - (int)(__float_as_uint(mx) >> 23), 120) : 0;
        const float up = __int_as_float((127 + ex) << 23) * (scale < 0.f ? -1.f : 1.f);
        // never 0, so that a masked score stays -inf
        fac = fmaxf(fabsf(scale) * 1.4426950408889634f * __int_as_float((127 - ex) << 23), 1e-37f);
        __half hi[8] = {}, lo[8] = {};            // sums of q over each group, as pairs
#pragma unroll
        for (int g = 0; g < NG; ++g) {
            float sum = 0.f;
#pragma unroll
            for (int c = 4 * g; c < 4 * g + 4; ++c) {
                float f[8];
                unpack8(row < rows ? reinterpret_cast<const uint4 *>(src)[c] : make_uint4(0, 0, 0, 0), f);
                uint4 u;
                uint32_t *w = &u.x;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const __half2 h = __floats2half2_rn(f[e] * up, f[e + 4] * up);
                    sum += __low2float(h) + __high2float(h);
                    w[e] = h2_bits(h);
                }
                *reinterpret_cast<uint4 *>(S.q[rt] + (c >> 3) * T::BLK + tc::swz(tid & 127, c & 7)) = u;
            }
            hi[g] = __float2half_rn(sum);
            lo[g] = __float2half_rn(sum - __half2float(hi[g]));
        }
        // columns 0..7: hi of the groups, 8..15: lo
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            uint4 u;
            uint32_t *w = &u.x;
#pragma unroll
            for (int e = 0; e < 4; ++e)
                w[e] = half ? h2_bits(__halves2half2(lo[2 * e], lo[2 * e + 1]))
                            : h2_bits(__halves2half2(hi[2 * e], hi[2 * e + 1]));
            *reinterpret_cast<uint4 *>(S.qx[rt] + at_x(tid & 127, half)) = u;
        }
        tc::fence_async_smem();
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = S.tmem;

    if (warp < kTcSoftWarps) {
        const uint32_t tS = tmem + 256 * rt + ((uint32_t)(32 * (warp & 3)) << 16), tO = tS + 128;
        const int see = row < rows ? len - m + row / G + 1 : 0x7fffffff;   // keys this row sees
        // (rows past the end compute on zeros and are not stored)
        const int see_first = min(len - m + min(row0 + 128 * rt, rows - 1) / G + 1, see_last);
        float ref = -INFINITY, l = 0.f;
        bool ok = true;
        for (int t = 0; t < steps; ++t) {
            if (!(ok = tc_wait(&S.bar.s_full[rt], t & 1, abort))) break;
            tc::fence_after_sync();
            const uint2 have = *reinterpret_cast<const uint2 *>(S.have[t & 1]);
            if (128 * (t + 1) > see_first || have.x != 0x01010101u || have.y != 0x01010101u) {
                // keys this row may not use get a score of -inf: those past the ones it sees,
                // and blocks whose records are not there; blocks at a quarter are put right
                const int cnt = min(see, see_last) - 128 * t;
#pragma unroll 1
                for (int c = 0; c < 8; ++c) {
                    const uint32_t hv = (c < 4 ? have.x : have.y) >> (8 * (c & 3));
                    const int stay = (hv & 1u) ? cnt - 16 * c : 0;
                    const float f = (hv & 2u) ? 4.f : 1.f;
                    float v[16];
                    tc::tmem_ld16(tS + 16 * c, v);
                    tc::tmem_wait_ld();
                    uint32_t u[16];
#pragma unroll
                    for (int j = 0; j < 16; ++j) u[j] = j < stay ? __float_as_uint(f * v[j]) : 0xff800000u;
                    tc_st16(tS + 16 * c, u);
                }
                tc::tmem_wait_st();
            }
            // two passes over the scores, each load issued one chunk of 16 ahead
            float s[2][16];
            tc::tmem_ld16(tS, s[0]);
            float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
            for (int c = 0; c < 8; ++c) {
                tc::tmem_wait_ld();
                tc::tmem_ld16(tS + 16 * ((c + 1) & 7), s[(c + 1) & 1]);
#pragma unroll
                for (int j = 0; j < 16; ++j) m4[j & 3] = fmaxf(m4[j & 3], s[c & 1][j]);
            }
            const float mx = fac * fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]));
            const bool move = mx > ref + kTcSlack;
            if (__any_sync(0xffffffffu, move)) {
                const float keep = move ? tc_ex2(ref - mx) : 1.f;
                if (move) ref = mx;
                l *= keep;
                if (t > 0) {
                    tc::tmem_wait_ld();
#pragma unroll 1
                    for (int c = 0; c < D / 16; ++c) {
                        float v[16];
                        tc::tmem_ld16(tO + 16 * c, v);
                        tc::tmem_wait_ld();
                        uint32_t u[16];
#pragma unroll
                        for (int j = 0; j < 16; ++j) u[j] = __float_as_uint(v[j] * keep);
                        tc_st16(tO + 16 * c, u);
                    }
                    tc::tmem_wait_st();
                }
            }
            const float sub = ref == -INFINITY ? 0.f : kTcLift - ref;
            const float2 fac2 = make_float2(fac, fac), sub2 = make_float2(sub, sub);
            float2 ls[2] = {};
#pragma unroll
            for (int c = 0; c < 8; ++c) {
                tc::tmem_wait_ld();
                if (c < 7) tc::tmem_ld16(tS + 16 * (c + 1), s[(c + 1) & 1]);
                float *x = s[c & 1];
                uint32_t p[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    float2 e = fma_f32x2(make_float2(x[2 * j], x[2 * j + 1]), fac2, sub2);
                    e = make_float2(tc_ex2(e.x), tc_ex2(e.y));
                    p[j] = h2_bits(__floats2half2_rn(e.x, e.y));
                    ls[j & 1] = add_f32x2(ls[j & 1], e);
                }
                tc_st8(tS + 8 * c, p);         // over scores that this thread has read
            }
            l += (ls[0].x + ls[0].y) + (ls[1].x + ls[1].y);
            tc::tmem_wait_st();
            tc::fence_before_sync();
            __syncwarp();
            if (lane == 0) tc_arrive(&S.bar.p_full[rt]);
        }
        // ---- output: columns 8 W + 2 i + h hold d = 64 (W / 8) + 32 h + 4 (W % 8) + i
        if (steps > 0) ok = ok && tc_wait(&S.bar.pv[rt], (steps - 1) & 1, abort);
        if (ok) {
            tc::fence_after_sync();
            const float inv = l == 0.f ? 0.f : 1.f / l;
            const uint32_t nan = S.nan_groups[tid];
            const int64_t t = t0 + (row < rows ? row / G : 0);
            const int hq = hkv * G + (row < rows ? row % G : 0);
            bf16 *dst = o + t * o_tok + (int64_t)hq * D;
#pragma unroll
            for (int c = 0; c < D / 16; ++c) {
                float v[16];
                if (steps > 0) {
                    tc::tmem_ld16(tO + 16 * c, v);
                    tc::tmem_wait_ld();
                } else {
#pragma unroll
                    for (int j = 0; j < 16; ++j) v[j] = 0.f;
                }
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int d = 64 * (c >> 2) + 32 * h + 8 * (c & 3);
                    uint4 u;
                    uint32_t *w = &u.x;
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        // elements d + 2 e, d + 2 e + 1: word e / 2 of the two, nibbles 2 (e % 2) ..
                        const int at = 8 * (e >> 1) + 4 * (e & 1) + h;
                        w[e] = pack_bf2(v[at] * inv, v[at + 2] * inv);
                    }
                    if (((nan >> (d >> 5)) & 1u) || l != l) u = make_uint4(0x7fff7fffu, 0x7fff7fffu, 0x7fff7fffu, 0x7fff7fffu);
                    if (row < rows) *reinterpret_cast<uint4 *>(dst + d) = u;
                }
            }
            if (lse && row < rows)
                lse[t * Hq + hq] = l == 0.f ? -INFINITY : (ref - kTcLift + log2f(l)) * 0.6931471805599453f;
        }
    } else if (warp < kTcSoftWarps + kTcUnpackWarps) {
        // ---- unpacking: this warp has keys 16 w .. +15 of each tile, then their values; lane
        // (r, x) takes a quarter of the codes of records r and r + 8
        const int w = warp - kTcSoftWarps, x = lane & 3;
        // Eight lanes store 16 bytes each at a time, two rows of a swizzled tile.  A row's four
        // chunks of keys fill half of the banks, and rows r and r + 4 opposite halves; its chunks
        // of values (D = 128, with words exchanged in pairs for x >= 2) meet those of r + 2 nowhere.
        const int rk = 4 * ((lane >> 2) & 1) + (lane >> 3);
        const int rv = D == 128 ? 2 * ((lane >> 2) & 1) + ((lane >> 3) & 1) + 4 * (lane >> 4) : lane >> 2;
        constexpr int NW = D / 32;               // words of codes a lane takes
        const int32_t *table = kv.table + (int64_t)n * kv.table_width;
        const int64_t page_bytes = (int64_t)(2 * kv.Hkv * REC) << kv.page_log2;
        const uint8_t *base = kv.block(0, 0, hkv, REC);
        const int64_t to_v = kv.block(0, 1, hkv, REC) - base;
        const int slot_mask = (1 << kv.page_log2) - 1;
        uint32_t code[2][2][NW], par[2][2][NG];  // [keys / values][r, r + 8]
        auto lookup = [&](int t) {
            const int j = 128 * t + 16 * w;
            return j < see_last ? table[j >> kv.page_log2] : -1;
        };
        // keys (u = 0) or values (1) of tile t; records that are not there, or past the last key
        // the tile's rows see, read as zeros
        auto fetch = [&](int t, int u, int pg) {
            const int j = 128 * t + 16 * w;
            const bool want = pg >= 0 && pg < kv.pages;
            if (!want && j < see_last && u == 0 && lane == 0) report(status, GDN_ERR_INDEX);
            const uint8_t *rec = base + (int64_t)pg * page_bytes + (u ? to_v : 0) + ((j & slot_mask) + (u ? rv : rk)) * REC;
#pragma unroll
            for (int y = 0; y < 2; ++y) {
                const uint8_t *p = rec + 8 * y * REC;
                const bool in = want && j + (u ? rv : rk) + 8 * y < see_last;
                if constexpr (D == 128) {
                    const uint4 a = in ? *reinterpret_cast<const uint4 *>(p + 16 * x) : make_uint4(0, 0, 0, 0);
                    const uint4 b = in ? *reinterpret_cast<const uint4 *>(p + R::CODES) : make_uint4(0, 0, 0, 0);
                    code[u][y][0] = a.x; code[u][y][1] = a.y; code[u][y][2] = a.z; code[u][y][3] = a.w;
                    par[u][y][0] = b.x; par[u][y][1] = b.y; par[u][y][2] = b.z; par[u][y][3] = b.w;
                } else {
                    const uint2 a = in ? *reinterpret_cast<const uint2 *>(p + 8 * x) : make_uint2(0, 0);
                    const uint2 b = in ? *reinterpret_cast<const uint2 *>(p + R::CODES) : make_uint2(0, 0);
                    code[u][y][0] = a.x; code[u][y][1] = a.y;
                    par[u][y][0] = b.x; par[u][y][1] = b.y;
                }
            }
        };
        int page = steps > 0 ? lookup(0) : -1;
        if (steps > 0) {
            fetch(0, 0, page);
            fetch(0, 1, page);
        }
        const int first_row_sees = len - m + row0 / G + 1;
        for (int t = 0; t < steps; ++t) {
            const int s = t & 1;
            const int page_next = lookup(t + 1);
            uint32_t any = 0u;
#pragma unroll
            for (int g = 0; g < NG; ++g) any |= par[0][0][g] | par[0][1][g];
            bool quarter = false;
            if (__any_sync(0xffffffffu, any & 0x4000u)) {        // some scale of 2 or more
                uint32_t most = 0u;          // as fp16 bits, which order like the numbers
#pragma unroll
                for (int g = 0; g < NG; ++g) most = max(most, max(par[0][0][g] & 0x7fffu, par[0][1][g] & 0x7fffu));
                quarter = __any_sync(0xffffffffu, most > kTcTopScale);
            }
            if (quarter) {
                const __half2 q4 = __floats2half2_rn(0.25f, 0.25f);
#pragma unroll
                for (int y = 0; y < 2; ++y)
#pragma unroll
                    for (int g = 0; g < NG; ++g) par[0][y][g] = h2_bits(__hmul2(bits_h2(par[0][y][g]), q4));
            }
            if (t >= 1 && !tc_wait<100>(&S.bar.k_free, (t - 1) & 1, abort)) break;
#pragma unroll
            for (int y = 0; y < 2; ++y) {
                // word x NG + g is elements 32 g + 8 x ..: 16-byte chunk 4 g + x
                const int key = 16 * w + rk + 8 * y;
#pragma unroll
                for (int g = 0; g < NG; ++g) {
                    const __half2 sc = __low2half2(bits_h2(par[0][y][g]));
                    __half2 c[4];
                    codes_of(code[0][y][g], c);
                    uint32_t hi[4], lo[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const __half2 h = __hmul2(c[i], sc);
                        hi[i] = h2_bits(h);
                        lo[i] = h2_bits(__hfma2(c[i], sc, __hneg2(h)));
                    }
                    const uint32_t at = ((4 * g + x) >> 3) * T::BLK + tc::swz(key, (4 * g + x) & 7);
                    *reinterpret_cast<uint4 *>(S.hi + at) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                    *reinterpret_cast<uint4 *>(S.lo + at) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
                }
                if (x < 2) {                 // the minima, against the sums' hi and lo
                    uint4 v = make_uint4(__byte_perm(par[0][y][0], par[0][y][1], 0x7632), 0u, 0u, 0u);
                    if (NG == 4) v.y = __byte_perm(par[0][y][NG - 2], par[0][y][NG - 1], 0x7632);
                    *reinterpret_cast<uint4 *>(S.kx + at_x(key, x)) = v;
                }
            }
            if (lane == 0) S.have[s][w] = page >= 0 && page < kv.pages ? (quarter ? 3 : 1) : 0;
            if (t + 1 < steps) fetch(t + 1, 0, page_next);
            tc::fence_async_smem();
            __syncwarp();
            if (lane == 0) tc_arrive(&S.bar.k_full);
            if (t >= 2 && !tc_wait<100>(&S.bar.v_free[s], ((t >> 1) & 1) ^ 1, abort)) break;
            if (128 * (t + 1) > first_row_sees) {
                // some row does not see some key of this tile: a non-finite value pair would
                // reach it through its zero weight, so such a group is zeroed here and made
                // NaN in just the rows that see the key
#pragma unroll
                for (int y = 0; y < 2; ++y)
#pragma unroll
                    for (int g = 0; g < NG; ++g) {
                        if (!pair_nonfinite(par[1][y][g])) continue;
                        const int j = 128 * t + 16 * w + rv + 8 * y;
                        if (x == 0)
                            for (int i = 0; i < kTcRows && row0 + i < rows; ++i)
                                if (j < len - m + (row0 + i) / G + 1) atomicOr(S.nan_groups + i, 1u << g);
                        par[1][y][g] = 0u;
                    }
            }
#pragma unroll
            for (int y = 0; y < 2; ++y) {
                // word W is chunk W; its low nibbles are of group 2 (W / 8), its high of the next
                const int key = 16 * w + rv + 8 * y;
                const uint32_t a = NG == 4 && x >= 2 ? par[1][y][NG - 2] : par[1][y][0];
                const uint32_t b = NG == 4 && x >= 2 ? par[1][y][NG - 1] : par[1][y][1];
                const __half2 sc = bits_h2(__byte_perm(a, b, 0x5410)), mn = bits_h2(__byte_perm(a, b, 0x7632));
                const __half2 top = __floats2half2_rn(65504.f, 65504.f);
#pragma unroll
                for (int e = 0; e < NW; ++e) {
                    const int W = NW * x + (D == 128 && x >= 2 ? e ^ 1 : e);
                    __half2 c[4];
                    codes_of(D == 128 && x >= 2 ? code[1][y][e ^ 1] : code[1][y][e], c);
                    uint32_t v[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) v[i] = h2_bits(__hmin2_nan(__hfma2(c[i], sc, mn), top));
                    *reinterpret_cast<uint4 *>(S.v[s] + (W >> 3) * T::BLK + tc::swz(key, W & 7)) =
                        make_uint4(v[0], v[1], v[2], v[3]);
                }
            }
            if (t + 1 < steps) fetch(t + 1, 1, page_next);
            tc::fence_async_smem();
            __syncwarp();
            if (lane == 0) tc_arrive(&S.bar.v_full[s]);
            page = page_next;
        }
    } else {
        // ---- products.  P V of a tile completes before the next scores overwrite P.
        constexpr uint32_t idS = idesc_f16(128, 128, 0), idO = idesc_f16(128, D, 1);
        auto scores = [&](int i) {
            const uint32_t a = tc::smem_u32(S.q[i]), h = tc::smem_u32(S.hi), l = tc::smem_u32(S.lo);
            tc::mma_bf16_warp(tmem + 256 * i, desc_x(S.qx[i]), desc_x(S.kx), idS, 0);
#pragma unroll
            for (int ks = 0; ks < D / 16; ++ks) {
                const uint32_t off = (ks >> 2) * T::BLK + (ks & 3) * 32;
                const uint64_t da = tc::sdesc(a + off, 16, 1024);
                tc::mma_bf16_warp(tmem + 256 * i, da, tc::sdesc(h + off, 16, 1024), idS, 1);
                tc::mma_bf16_warp(tmem + 256 * i, da, tc::sdesc(l + off, 16, 1024), idS, 1);
            }
            tc::mma_commit_warp(&S.bar.s_full[i]);
            if (i == 1) tc::mma_commit_warp(&S.bar.k_free);
        };
        bool ok = steps > 0 && tc_wait(&S.bar.k_full, 0, abort);
        if (ok) {
            tc::fence_after_sync();
#pragma unroll 1
            for (int i = 0; i < 2; ++i) scores(i);
        }
        for (int t = 0; t < steps && ok; ++t) {
            if (!(ok = tc_wait(&S.bar.v_full[t & 1], (t >> 1) & 1, abort))) break;
#pragma unroll 1
            for (int i = 0; i < 2 && ok; ++i) {
                if (!(ok = tc_wait(&S.bar.p_full[i], t & 1, abort))) break;
                tc::fence_after_sync();
                const uint32_t b = tc::smem_u32(S.v[t & 1]);
#pragma unroll
                for (int ks = 0; ks < 8; ++ks)
                    mma_ts(tmem + 256 * i + 128, tmem + 256 * i + 8 * ks, tc::sdesc(b + ks * 2048, T::BLK, 1024), idO,
                           t > 0 || ks > 0);
                tc::mma_commit_warp(&S.bar.pv[i]);
                if (i == 1) tc::mma_commit_warp(&S.bar.v_free[t & 1]);
                if (t + 1 < steps) {
                    if (i == 0 && !(ok = tc_wait(&S.bar.k_full, (t + 1) & 1, abort))) break;
                    if (!(ok = tc_wait(&S.bar.pv[i], t & 1, abort))) break;
                    tc::fence_after_sync();
                    scores(i);
                }
            }
        }
        // everything issued has completed before the TMEM is freed
        tc::mma_commit_warp(&S.bar.fin);
        wait_copy(&S.bar.fin, 0);
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    if (warp == 0) tc::tmem_dealloc(tmem, 512);
    if (tid == 0 && *abort) report(status, GDN_ERR_TIMEOUT);
}

}  // namespace gdn

namespace gdn_host {

namespace {

template <int D>
gdn_status_t tc_launch(const KvArgs &a, int min_rows, cudaStream_t st) {
    auto kern = gdn::kv_attention_tc_kernel<D>;
    constexpr int smem = sizeof(gdn::TcSmem<D>);
    static_assert(smem <= 227 * 1024, "one CTA fits on an SM");
    static std::atomic<uint64_t> ready{0};   // one bit per device (beyond 63: set every time)
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return GDN_ERR_CUDA;
    if (dev > 63 || !((ready.load() >> dev) & 1u)) {
        if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
            return GDN_ERR_CUDA;
        if (dev <= 63) ready.fetch_or(1ull << dev);
    }
    const int64_t rows = (int64_t)(a.Hq / a.kv.Hkv) * a.max_q_len;
    const dim3 grid((unsigned)((rows + gdn::kTcRows - 1) / gdn::kTcRows), a.kv.Hkv, a.kv.N);
    kern<<<grid, gdn::kTcThreads, smem, st>>>(a.kv, (const gdn::bf16 *)a.q, (gdn::bf16 *)a.q_out, a.lse,
                                              a.q_tok, a.o_tok, a.Hq, min_rows, a.max_kv_len, a.scale,
                                              a.status);
    return cudaGetLastError() == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

}  // namespace

bool kv_attention_tc_supported(int32_t D) { return D == 64 || D == 128; }

gdn_status_t launch_kv_attention_tc(const KvArgs &a, int min_rows, cudaStream_t st) {
    return a.D == 64 ? tc_launch<64>(a, min_rows, st) : tc_launch<128>(a, min_rows, st);
}

}  // namespace gdn_host
