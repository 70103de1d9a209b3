// linear_tc.cu -- linear attention with a decay for each head over packed prompts, on the
// tensor cores (tcgen05, TMEM, TMA): bf16 activations, D = 128.
//
// A sequence is cut into chunks of 128 tokens.  With G_i the chunk's inclusive sums of the
// log decays, T their total and S the fp32 state at the chunk's start,
//     O = scale (e^{G_i} q_i S + sum_{j <= i} e^{G_i - G_j} (q_i.k_j) v_j)
//     S <- e^T S + sum_j e^{T - G_j} k_j v_j^T
// which is four 128 x 128 x 128 products a chunk, two of them over the weighted keys, which
// go in as a bf16 pair hi + lo so that the state keeps fp32-level accuracy:
//     Q K^T,   Q S,   P V,   (hi + lo)^T V
// e^{T - G_j} comes from sums taken from the chunk's end and e^{G_i - G_j} inside a 32 x 32
// block from its exponent, elsewhere as a product of two factors at most 1, so nothing
// overflows however strong the decay.
//
// Roundings below fp32, all to bf16 and all in operands whose products only reach the bf16
// output: P, and S where it multiplies Q.  The state itself never goes through them.
//
// linear_out_kernel: one CTA per (sequence range, v-head) walks its chunks with the state
// in registers (32 floats a thread).  Warps 0-7 do the elementwise work, a thread holding
// one TMEM lane and half the columns: weighted keys (A), P (B), state (C), output (D);
// warp 8 issues the products, warp 9 the tile loads, warp 10 the sums of the gates.  Seven
// 32 KB tiles (Q, K, V, hi, lo, S, P) leave room for one buffer each; the order A B C D
// lets every load and product run behind another phase, and the chain of a chunk is what
// bounds the kernel (about 1.5 us; its products are 1.35 us of tensor time).
//
// A long sequence over few heads would leave SMs idle, so it is cut into ranges that run
// side by side: linear_range_kernel gives every range's own state (hi + lo products added
// up in TMEM with decays to the range's end), linear_start_kernel folds them in order into
// start states, and linear_out_kernel runs the ranges from those.  The cut depends on the
// sequence's own length, the head count and the SM count only, so a sequence's bits do not
// depend on its batch.
#include <cuda.h>
#include <cudaTypedefs.h>

#include <algorithm>
#include <atomic>

#include "bulk_ptx.cuh"
#include "linear.cuh"
#include "tmap.cuh"

namespace gdn {

constexpr int kLinC = 128;                 // tokens per chunk
constexpr uint32_t kTile = 32768;          // one 128 x 128 bf16 tile: two 64-column blocks
constexpr uint32_t kBlk = 16384;
constexpr int kLinWarps = 16;              // warps that do elementwise work
constexpr int kLinThreads = 32 * (kLinWarps + 3);
constexpr int kMinSplitChunks = 12;        // shorter sequences are one range
constexpr int kMinRangeChunks = 4;
constexpr int kMinRangeTokens = kMinRangeChunks * kLinC;

struct LinMaps {
    CUtensorMap q, k, v;
};

struct LinParams {
    const float *g;
    int64_t g_tok;
    const int32_t *cu;
    const float *h0;
    float *hT;
    bf16 *o;
    int64_t o_tok;
    float *ranges;        // [slots][Hv][128][128]: slot r + 1 of a sequence takes range r's own
                          // state, then the start of range r + 1
    float *range_decay;   // [slots][Hv]: slot r + 1: range r's total log decay
    int Hk, Hv;
    int max_par;          // ranges of one sequence that fill the device
    int slots_per_seq;    // > 0: sequence n's slots start at n * this; 0: at cu[n] / 512 + n
    int in_place;         // hT is h0: slot 0 takes a copy of h0, which the last range of a
                          // sequence may overwrite before its first range has read it
    float scale;
    int32_t *status;
};

// Chunks per range of a sequence of nch chunks.  Under 12 chunks the second pass and its
// launches cost more than they save (12 chunks of 1.5 us against 4 + 4 of 0.6 and 6 us).
__host__ __device__ __forceinline__ int range_chunks_of(int nch, int max_par) {
    if (nch < kMinSplitChunks || max_par <= 1) return nch > 0 ? nch : 1;
    const int rc = (nch + max_par - 1) / max_par;
    return rc > kMinRangeChunks ? rc : kMinRangeChunks;
}
// A sequence of len tokens has at most len / 512 ranges after its first, and cu[n] / 512
// grows by at least that much from one sequence to the next.
__device__ __forceinline__ int64_t range_slot0(const LinParams &p, int n, int t0) {
    return p.slots_per_seq ? (int64_t)n * p.slots_per_seq : t0 / kMinRangeTokens + n;
}

// ------------------------------------------------------------------------ shared memory

struct LinBars {
    uint64_t q, k[3], v[2];              // tiles loaded
    uint64_t qk, qs, kv[2], pv;          // products done
    uint64_t gates;                      // this chunk's gate arrays are written
    uint64_t r_kt[2], r_p, r_s, r_o, r_arr;   // every elementwise warp: operands written, arrays read
    uint64_t fin;
};
struct LinSmem {
    uint8_t tile[7][kTile];
    float g2[kLinC];     // G log2 e
    float eg[kLinC];     // scale e^G
    float w[kLinC];      // e^{T - G}
    float b[kLinC];      // e^{G(end of the token's block of 32) - G}
    float ref[4];        // G log2 e at the end of each block
    float decay;         // e^T
    float total;         // T
    uint32_t tmem;
    int abort;
    LinBars bar;
};
static_assert(sizeof(LinSmem) <= 227 * 1024, "one CTA fits on an SM");

constexpr float kLog2E = 1.4426950408889634f;

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ void mbar_arrive(uint64_t *bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" :: "r"(tc::smem_u32(bar)) : "memory");
}

// Two fp32 operations in one instruction, rounded like the single ones.
__device__ __forceinline__ float2 mul_f32x2(float2 a, float2 b) {
    float2 d;
    asm("mul.rn.f32x2 %0, %1, %2;"
        : "=l"(*reinterpret_cast<unsigned long long *>(&d))
        : "l"(*reinterpret_cast<const unsigned long long *>(&a)),
          "l"(*reinterpret_cast<const unsigned long long *>(&b)));
    return d;
}
__device__ __forceinline__ float2 fma_f32x2(float2 a, float2 b, float2 c) {
    float2 d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;"
        : "=l"(*reinterpret_cast<unsigned long long *>(&d))
        : "l"(*reinterpret_cast<const unsigned long long *>(&a)),
          "l"(*reinterpret_cast<const unsigned long long *>(&b)),
          "l"(*reinterpret_cast<const unsigned long long *>(&c)));
    return d;
}

// Bounded wait on an mbarrier phase.  Gives up when the bound has passed or another thread
// of the CTA has given up; every role then leaves its loop.
__device__ __forceinline__ bool lin_wait(LinSmem &S, uint64_t *bar, uint32_t parity) {
    if (tc::mbar_try_wait(bar, parity)) return true;
    uint64_t t0, t;
    asm volatile("mov.u64 %0, %globaltimer;" : "=l"(t0));
    volatile int *abort = &S.abort;
    for (;;) {
        if (tc::mbar_try_wait(bar, parity)) return true;
        if (*abort) return false;
        asm volatile("mov.u64 %0, %globaltimer;" : "=l"(t));
        if (t - t0 > kCopyWaitNs) {
            *abort = 1;
            return false;
        }
    }
}

// The same by a whole warp, which stays together whatever its lanes saw.
__device__ __forceinline__ bool warp_wait(LinSmem &S, uint64_t *bar, uint32_t parity) {
    return __all_sync(0xffffffffu, lin_wait(S, bar, parity)) != 0;
}

// The writes of this warp (shared memory for the async proxy, TMEM reads done) happen
// before the arrival.
__device__ __forceinline__ void warp_arrive(uint64_t *bar) {
    tc::fence_async_smem();
    tc::fence_before_sync();
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
}

__device__ __forceinline__ void load_tile(uint8_t *dst, const CUtensorMap *map, uint64_t *bar,
                                          int head, int t) {
    tc::mbar_expect_tx(bar, kTile);
    tc::tma_load_3d(dst, map, bar, 0, head, t);
    tc::tma_load_3d(dst + kBlk, map, bar, 64, head, t);
}

// D[128 x 128] (+)= A B over a depth of 128.  K-major operands step 32 bytes inside a
// 64-column block; MN-major ones step 16 rows.
template <int A_MN, int B_MN>
__device__ __forceinline__ void product(uint32_t d, const uint8_t *a, const uint8_t *b, bool add) {
    constexpr uint32_t id = tc::idesc_bf16(128, 128, A_MN, B_MN);
    const uint32_t a0 = tc::smem_u32(a), b0 = tc::smem_u32(b);
#pragma unroll
    for (int ks = 0; ks < 8; ++ks) {
        const uint32_t km = (ks >> 2) * kBlk + (ks & 3) * 32, mn = ks * 2048;
        const uint64_t da = A_MN ? tc::sdesc(a0 + mn, kBlk, 1024) : tc::sdesc(a0 + km, 16, 1024);
        const uint64_t db = B_MN ? tc::sdesc(b0 + mn, kBlk, 1024) : tc::sdesc(b0 + km, 16, 1024);
        tc::mma_bf16_warp(d, da, db, id, add || ks > 0);
    }
}

// ------------------------------------------------------------------------- gates (warp)
// Lane l has tokens 4 l .. 4 l + 3 of the chunk at t (L of them; past the end the log
// decay is 0).  -inf (and anything below -110, where e^g is 0 in fp32) becomes -110 so that
// the sums stay finite; a NaN stays.
__device__ __forceinline__ void load_gates(const LinParams &p, int hv, int t, int L, float (&x)[4]) {
    const int l = threadIdx.x & 31;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const int i = 4 * l + e;
        const float g = i < L ? p.g[(int64_t)(t + i) * p.g_tok + hv] : 0.f;
        x[e] = g < -110.f ? -110.f : g;
    }
}
// Exclusive sums over the lanes below and above.
__device__ __forceinline__ float lanes_below(float x) {
    const int l = threadIdx.x & 31;
    float s = x;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const float y = __shfl_up_sync(0xffffffffu, s, off);
        if (l >= off) s += y;
    }
    const float y = __shfl_up_sync(0xffffffffu, s, 1);
    return l > 0 ? y : 0.f;
}
__device__ __forceinline__ float lanes_above(float x) {
    const int l = threadIdx.x & 31;
    float s = x;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const float y = __shfl_down_sync(0xffffffffu, s, off);
        if (l + off < 32) s += y;
    }
    const float y = __shfl_down_sync(0xffffffffu, s, 1);
    return l < 31 ? y : 0.f;
}

// --------------------------------------------------------------- weighted keys (phase A)
// hi, lo <- bf16 pair of w_j k_j for rows j < L, zero rows after (hi may be k).  A quarter
// warp takes the eight 16-byte chunks of a row.
__device__ __forceinline__ void weigh_keys(const uint8_t *k, uint8_t *hi, uint8_t *lo, const float *w,
                                           int L) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, ch = lane & 7;
#pragma unroll
    for (int it = 0; it < 128 / (4 * kLinWarps); ++it) {
        const int row = 4 * kLinWarps * it + 4 * warp + (lane >> 3);
        const float wj = w[row];
        const float2 w2 = make_float2(wj, wj), m1 = make_float2(-1.f, -1.f);
#pragma unroll
        for (int kb = 0; kb < 2; ++kb) {
            const uint32_t at = kb * kBlk + tc::swz(row, ch);
            const uint4 u = *reinterpret_cast<const uint4 *>(k + at);
            const uint32_t uw[4] = {u.x, u.y, u.z, u.w};
            uint32_t h[4], r[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float2 x = mul_f32x2(
                    make_float2(__uint_as_float(uw[e] << 16), __uint_as_float(uw[e] & 0xffff0000u)), w2);
                h[e] = pack_bf2(x.x, x.y);
                const float2 d = fma_f32x2(
                    make_float2(__uint_as_float(h[e] << 16), __uint_as_float(h[e] & 0xffff0000u)), m1, x);
                r[e] = pack_bf2(d.x, d.y);
            }
            if (L < kLinC && row >= L) {
#pragma unroll
                for (int e = 0; e < 4; ++e) h[e] = r[e] = 0u;
            }
            *reinterpret_cast<uint4 *>(hi + at) = make_uint4(h[0], h[1], h[2], h[3]);
            *reinterpret_cast<uint4 *>(lo + at) = make_uint4(r[0], r[1], r[2], r[3]);
        }
    }
}
// Rows past the end hold another sequence's values: zero them (a NaN there would survive
// the zero weights).
__device__ __forceinline__ void clear_rows(uint8_t *tile, int L) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, ch = lane & 7;
#pragma unroll
    for (int it = 0; it < 128 / (4 * kLinWarps); ++it) {
        const int row = 4 * kLinWarps * it + 4 * warp + (lane >> 3);
        if (row < L) continue;
#pragma unroll
        for (int kb = 0; kb < 2; ++kb)
            *reinterpret_cast<uint4 *>(tile + kb * kBlk + tc::swz(row, ch)) = make_uint4(0, 0, 0, 0);
    }
}
// 32 floats of one row as bf16 into columns 32 quarter .. of a tile.
__device__ __forceinline__ void store_row(uint8_t *tile, int quarter, int row, const float (&v)[32]) {
    const int blk = quarter >> 1, n0 = 32 * (quarter & 1);
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        uint4 u;
        u.x = pack_bf2(v[8 * c], v[8 * c + 1]);
        u.y = pack_bf2(v[8 * c + 2], v[8 * c + 3]);
        u.z = pack_bf2(v[8 * c + 4], v[8 * c + 5]);
        u.w = pack_bf2(v[8 * c + 6], v[8 * c + 7]);
        *reinterpret_cast<uint4 *>(tile + blk * kBlk + tc::swz(row, n0 / 8 + c)) = u;
    }
}

// ------------------------------------------------------------------------- output pass

__global__ void __launch_bounds__(kLinThreads, 1)
linear_out_kernel(const __grid_constant__ LinMaps maps, const LinParams p) {
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    LinSmem &S = *reinterpret_cast<LinSmem *>(smem_raw);
    if (tc::smem_u32(smem_raw) & 1023u) {        // the tiles' swizzle needs it; never seen
        if (threadIdx.x == 0) report(p.status, GDN_ERR_CUDA);
        return;
    }
    uint8_t *sQ = S.tile[0], *sK = S.tile[1], *sV = S.tile[2], *sHi = S.tile[3], *sLo = S.tile[4],
            *sS = S.tile[5], *sP = S.tile[6];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int range = blockIdx.x, hv = blockIdx.y, n = blockIdx.z, hk = hv / (p.Hv / p.Hk);
    const int t0 = p.cu[n], len = p.cu[n + 1] - t0;
    const int nch = (len + kLinC - 1) / kLinC;
    const int rc = range_chunks_of(nch, p.max_par);
    const int c_first = range * rc, c_last = min(nch, c_first + rc);
    if (range > 0 && c_first >= nch) return;
    const int count = c_last - c_first;          // 0 for an empty sequence
    const bool last = c_last >= nch;
    const uint32_t colSc = 0, colOi = 128, colOa = 256, colD = 384;

    if (warp == 0) {
        tc::tmem_alloc(&S.tmem, 512);
        tc::tmem_relinquish();
    }
    if (tid == 0) {
        S.abort = 0;
        LinBars &b = S.bar;
        for (uint64_t *x : {&b.q, &b.k[0], &b.v[0], &b.qk, &b.qs, &b.kv[0], &b.pv, &b.gates, &b.fin})
            tc::mbar_init(x, 1);
        for (uint64_t *x : {&b.r_kt[0], &b.r_p, &b.r_s, &b.r_o, &b.r_arr}) tc::mbar_init(x, kLinWarps);
        tc::mbar_fence_init();
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = S.tmem;

    if (warp < kLinWarps) {
        const int lq = warp & 3, jb = warp >> 2;    // rows 32 lq .., columns 32 jb ..
        const int row = 32 * lq + lane;
        const uint32_t tm = tmem + ((uint32_t)(32 * lq) << 16) + 32 * jb;
        const int64_t st_off = (int64_t)row * 128 + 32 * jb;
        float st[32];
        const float *src = nullptr;
        if (range > 0 || (p.in_place && rc < nch)) {
            grid_dependency_wait();
            src = p.ranges + ((range_slot0(p, n, t0) + range) * p.Hv + hv) * 16384;
        } else if (p.h0) {
            src = p.h0 + ((int64_t)n * p.Hv + hv) * 16384;
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float4 x = src ? reinterpret_cast<const float4 *>(src + st_off)[e]
                                 : make_float4(0.f, 0.f, 0.f, 0.f);
            st[4 * e] = x.x; st[4 * e + 1] = x.y; st[4 * e + 2] = x.z; st[4 * e + 3] = x.w;
        }
        if (count > 0) {
            store_row(sS, jb, row, st);
            warp_arrive(&S.bar.r_s);
        }
        for (int i = 0; i < count; ++i) {
            const uint32_t ph = i & 1;
            const int t = t0 + (c_first + i) * kLinC;
            const int L = min(kLinC, t0 + len - t);
            // ---- A: weighted keys
            if (!warp_wait(S, &S.bar.gates, ph) || !warp_wait(S, &S.bar.k[0], ph)) break;
            weigh_keys(sK, sHi, sLo, S.w, L);
            if (L < kLinC) {
                if (!warp_wait(S, &S.bar.v[0], ph)) break;
                clear_rows(sV, L);
            }
            warp_arrive(&S.bar.r_kt[0]);
            // ---- B: P = decay-weighted lower triangle of Q K^T
            if (!warp_wait(S, &S.bar.qk, ph)) break;
            tc::fence_after_sync();
            const float eg = S.eg[row], decay = S.decay;
            float v[32];
            if (jb <= lq) {
                const float gi = S.g2[row];
                tc::tmem_ld32(tm + colSc, v);
                if (jb < lq) {
                    const float f = p.scale * ex2(gi - S.ref[jb]);
                    float4 b4[8];
#pragma unroll
                    for (int j = 0; j < 8; ++j) b4[j] = reinterpret_cast<const float4 *>(S.b)[8 * jb + j];
                    tc::tmem_wait_ld();
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        v[4 * j] *= f * b4[j].x;
                        v[4 * j + 1] *= f * b4[j].y;
                        v[4 * j + 2] *= f * b4[j].z;
                        v[4 * j + 3] *= f * b4[j].w;
                    }
                } else {
                    float w[32];
#pragma unroll
                    for (int j = 0; j < 32; ++j) w[j] = p.scale * ex2(gi - S.g2[32 * jb + j]);
                    tc::tmem_wait_ld();
#pragma unroll
                    for (int j = 0; j < 32; ++j) v[j] = j <= lane ? v[j] * w[j] : 0.f;
                }
            } else {
#pragma unroll
                for (int j = 0; j < 32; ++j) v[j] = 0.f;
            }
            store_row(sP, jb, row, v);
            warp_arrive(&S.bar.r_p);
            if (lane == 0) mbar_arrive(&S.bar.r_arr);
            // ---- C: state
            if (!warp_wait(S, &S.bar.kv[0], ph)) break;
            tc::fence_after_sync();
            tc::tmem_ld32(tm + colD, v);
            tc::tmem_wait_ld();
#pragma unroll
            for (int j = 0; j < 32; ++j) st[j] = fmaf(decay, st[j], v[j]);
            if (!warp_wait(S, &S.bar.qs, ph)) break;
            store_row(sS, jb, row, st);
            warp_arrive(&S.bar.r_s);
            // ---- D: output, through this warp's own part of the P tile (PV has read it), so
            // that a row's 64 bytes leave as full sectors
            if (!warp_wait(S, &S.bar.pv, ph)) break;
            tc::fence_after_sync();
            float a[32];
            tc::tmem_ld32(tm + colOi, a);
            tc::tmem_ld32(tm + colOa, v);
            tc::tmem_wait_ld();
            tc::fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(&S.bar.r_o);
#pragma unroll
            for (int j = 0; j < 32; ++j) v[j] = fmaf(eg, a[j], v[j]);
            store_row(sP, jb, row, v);
            __syncwarp();
            bf16 *dst = p.o + (int64_t)(t + 32 * lq) * p.o_tok + (int64_t)hv * 128 + 32 * jb;
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                const int rr = 8 * x + (lane >> 2), cc = lane & 3;
                const uint4 u = *reinterpret_cast<const uint4 *>(
                    sP + (jb >> 1) * kBlk + tc::swz(32 * lq + rr, 4 * (jb & 1) + cc));
                if (32 * lq + rr < L) reinterpret_cast<uint4 *>(dst + rr * p.o_tok)[cc] = u;
            }
            __syncwarp();
        }
        if (last && p.hT && !*(volatile int *)&S.abort) {
            float4 *out = reinterpret_cast<float4 *>(p.hT + ((int64_t)n * p.Hv + hv) * 16384 + st_off);
#pragma unroll
            for (int e = 0; e < 8; ++e)
                out[e] = make_float4(st[4 * e], st[4 * e + 1], st[4 * e + 2], st[4 * e + 3]);
        }
    } else if (warp == kLinWarps) {
        // ---- products
        for (int i = 0; i < count; ++i) {
            const uint32_t ph = i & 1;
            if (!warp_wait(S, &S.bar.q, ph) || !warp_wait(S, &S.bar.k[0], ph)) break;
            tc::fence_after_sync();
            product<0, 0>(tmem + colSc, sQ, sK, false);
            tc::mma_commit_warp(&S.bar.qk);
            if (!warp_wait(S, &S.bar.r_s, ph)) break;
            if (i > 0 && !warp_wait(S, &S.bar.r_o, ph ^ 1)) break;
            tc::fence_after_sync();
            product<0, 1>(tmem + colOi, sQ, sS, false);
            tc::mma_commit_warp(&S.bar.qs);
            if (!warp_wait(S, &S.bar.r_kt[0], ph) || !warp_wait(S, &S.bar.v[0], ph)) break;
            tc::fence_after_sync();
            product<1, 1>(tmem + colD, sHi, sV, false);
            product<1, 1>(tmem + colD, sLo, sV, true);
            tc::mma_commit_warp(&S.bar.kv[0]);
            if (!warp_wait(S, &S.bar.r_p, ph)) break;
            tc::fence_after_sync();
            product<0, 1>(tmem + colOa, sP, sV, false);
            tc::mma_commit_warp(&S.bar.pv);
        }
        // everything issued has completed before the TMEM is freed
        tc::mma_commit_warp(&S.bar.fin);
        wait_copy(&S.bar.fin, 0);
    } else if (warp == kLinWarps + 1) {
        // ---- tile loads
        int loads = 0;
        if (lane == 0) {
            tc::prefetch_tmap(&maps.q);
            tc::prefetch_tmap(&maps.k);
            tc::prefetch_tmap(&maps.v);
            for (int i = 0; i < count; ++i) {
                const uint32_t pp = (i & 1) ^ 1;
                const int t = t0 + (c_first + i) * kLinC;
                if (i > 0 && (!lin_wait(S, &S.bar.qk, pp) || !lin_wait(S, &S.bar.r_kt[0], pp))) break;
                load_tile(sK, &maps.k, &S.bar.k[0], hk, t);
                if (i > 0 && !lin_wait(S, &S.bar.qs, pp)) {
                    wait_copy(&S.bar.k[0], i & 1);
                    break;
                }
                load_tile(sQ, &maps.q, &S.bar.q, hk, t);
                if (i > 0 && (!lin_wait(S, &S.bar.kv[0], pp) || !lin_wait(S, &S.bar.pv, pp))) {
                    wait_copy(&S.bar.k[0], i & 1);
                    wait_copy(&S.bar.q, i & 1);
                    break;
                }
                load_tile(sV, &maps.v, &S.bar.v[0], hv, t);
                ++loads;
            }
            if (loads > 0) {
                // (bounded) everything loaded has landed
                wait_copy(&S.bar.k[0], (loads - 1) & 1);
                wait_copy(&S.bar.q, (loads - 1) & 1);
                wait_copy(&S.bar.v[0], (loads - 1) & 1);
            }
        }
    } else {
        // ---- gates
        float x[4];
        if (count > 0) load_gates(p, hv, t0 + c_first * kLinC, min(kLinC, len - c_first * kLinC), x);
        for (int i = 0; i < count; ++i) {
            float pre[4], suf[4];
            pre[0] = x[0];
#pragma unroll
            for (int e = 1; e < 4; ++e) pre[e] = pre[e - 1] + x[e];
            suf[3] = 0.f;
#pragma unroll
            for (int e = 2; e >= 0; --e) suf[e] = suf[e + 1] + x[e + 1];
            const float below = lanes_below(pre[3]), above = lanes_above(pre[3]);
            float y[4];
            const int t = t0 + (c_first + i + 1) * kLinC;
            if (i + 1 < count) load_gates(p, hv, t, min(kLinC, t0 + len - t), y);
            if (i > 0 && !warp_wait(S, &S.bar.r_arr, (i & 1) ^ 1)) break;
            const float end = below + pre[3];
            const float ref = __shfl_sync(0xffffffffu, end, lane | 7) * kLog2E;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int j = 4 * lane + e;
                const float G = below + pre[e];
                S.g2[j] = G * kLog2E;
                S.eg[j] = p.scale * expf(G);
                S.w[j] = expf(above + suf[e]);
                S.b[j] = ex2(ref - G * kLog2E);
            }
            if ((lane & 7) == 7) S.ref[lane >> 3] = ref;
            if (lane == 31) S.decay = expf(end);
            __syncwarp();
            if (lane == 0) mbar_arrive(&S.bar.gates);
#pragma unroll
            for (int e = 0; e < 4; ++e) x[e] = y[e];
        }
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    if (warp == 0) tc::tmem_dealloc(tmem, 512);
    if (tid == 0 && S.abort) report(p.status, GDN_ERR_TIMEOUT);
}

// -------------------------------------------------------------------------- range states
// State that one range adds, from zero, with decays to the range's end: its chunks in
// reverse, each chunk's weights carrying the sum of the later ones, all added up in TMEM.
// Tiles: K x 3 (hi replaces K in place), lo x 2, V x 2; the products bound it.
__global__ void __launch_bounds__(kLinThreads, 1)
linear_range_kernel(const __grid_constant__ LinMaps maps, const LinParams p) {
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    LinSmem &S = *reinterpret_cast<LinSmem *>(smem_raw);
    if (tc::smem_u32(smem_raw) & 1023u) {        // the tiles' swizzle needs it; never seen
        if (threadIdx.x == 0) report(p.status, GDN_ERR_CUDA);
        return;
    }
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int range = blockIdx.x, hv = blockIdx.y, n = blockIdx.z, hk = hv / (p.Hv / p.Hk);
    const int t0 = p.cu[n], len = p.cu[n + 1] - t0;
    const int nch = (len + kLinC - 1) / kLinC;
    const int rc = range_chunks_of(nch, p.max_par);
    const int c_first = range * rc, count = rc;
    if (c_first + rc >= nch) return;             // a last range: nothing reads its state
    const int64_t slot = (range_slot0(p, n, t0) + range + 1) * p.Hv + hv;

    if (warp == 0) {
        tc::tmem_alloc(&S.tmem, 128);
        tc::tmem_relinquish();
    }
    if (tid == 0) {
        S.abort = 0;
        LinBars &b = S.bar;
        for (uint64_t *x : {&b.k[0], &b.k[1], &b.k[2], &b.v[0], &b.v[1], &b.kv[0], &b.kv[1], &b.gates, &b.fin})
            tc::mbar_init(x, 1);
        for (uint64_t *x : {&b.r_kt[0], &b.r_kt[1], &b.r_arr}) tc::mbar_init(x, kLinWarps);
        tc::mbar_fence_init();
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = S.tmem;
    // step i takes chunk c_first + count - 1 - i; its use of a buffer among two is that
    // buffer's (i >> 1)-th, among three its (i / 3)-th
    if (warp < kLinWarps) {
        bool ok = true;
        for (int i = 0; i < count && ok; ++i) {
            const int bf = i & 1, kb = i % 3;
            if (!(ok = warp_wait(S, &S.bar.gates, i & 1) && warp_wait(S, &S.bar.k[kb], (i / 3) & 1))) break;
            if (i >= 2 && !(ok = warp_wait(S, &S.bar.kv[bf], ((i >> 1) & 1) ^ 1))) break;
            weigh_keys(S.tile[kb], S.tile[kb], S.tile[3 + bf], S.w, kLinC);
            warp_arrive(&S.bar.r_kt[bf]);
            if (lane == 0) mbar_arrive(&S.bar.r_arr);
        }
        const int e = count - 1;
        if (ok && warp_wait(S, &S.bar.kv[e & 1], (e >> 1) & 1)) {
            tc::fence_after_sync();
            const int lq = warp & 3, jb = warp >> 2;
            float4 *out = reinterpret_cast<float4 *>(p.ranges + slot * 16384 + (32 * lq + lane) * 128 + 32 * jb);
            float v[32];
            tc::tmem_ld32(tmem + ((uint32_t)(32 * lq) << 16) + 32 * jb, v);
            tc::tmem_wait_ld();
#pragma unroll
            for (int x = 0; x < 8; ++x)
                out[x] = make_float4(v[4 * x], v[4 * x + 1], v[4 * x + 2], v[4 * x + 3]);
        }
    } else if (warp == kLinWarps) {
        for (int i = 0; i < count; ++i) {
            const int bf = i & 1;
            if (!warp_wait(S, &S.bar.r_kt[bf], (i >> 1) & 1) || !warp_wait(S, &S.bar.v[bf], (i >> 1) & 1)) break;
            tc::fence_after_sync();
            product<1, 1>(tmem, S.tile[i % 3], S.tile[5 + bf], i > 0);
            product<1, 1>(tmem, S.tile[3 + bf], S.tile[5 + bf], true);
            tc::mma_commit_warp(&S.bar.kv[bf]);
        }
        tc::mma_commit_warp(&S.bar.fin);
        wait_copy(&S.bar.fin, 0);
    } else if (warp == kLinWarps + 1) {
        if (lane == 0) {
            // K of step i goes where step i - 3 was, V where step i - 2 was; K is asked for
            // a step ahead of V
            int ks = 0, vs = 0;
            auto load_k = [&](int i) {
                if (i >= 3 && !lin_wait(S, &S.bar.kv[(i - 3) & 1], ((i - 3) >> 1) & 1)) return false;
                load_tile(S.tile[i % 3], &maps.k, &S.bar.k[i % 3], hk, t0 + (c_first + count - 1 - i) * kLinC);
                ++ks;
                return true;
            };
            bool ok = load_k(0);
            for (int i = 0; i < count && ok; ++i) {
                if (i + 1 < count && !(ok = load_k(i + 1))) break;
                if (i >= 2 && !(ok = lin_wait(S, &S.bar.kv[i & 1], ((i >> 1) & 1) ^ 1))) break;
                load_tile(S.tile[5 + (i & 1)], &maps.v, &S.bar.v[i & 1], hv,
                          t0 + (c_first + count - 1 - i) * kLinC);
                ++vs;
            }
            for (int x = max(0, ks - 3); x < ks; ++x) wait_copy(&S.bar.k[x % 3], (x / 3) & 1);
            for (int x = max(0, vs - 2); x < vs; ++x) wait_copy(&S.bar.v[x & 1], (x >> 1) & 1);
        }
    } else {
        float x[4], carry = 0.f;
        load_gates(p, hv, t0 + (c_first + count - 1) * kLinC, kLinC, x);
        for (int i = 0; i < count; ++i) {
            const float sum = x[0] + x[1] + x[2] + x[3];
            float suf[4];
            suf[3] = 0.f;
#pragma unroll
            for (int e = 2; e >= 0; --e) suf[e] = suf[e + 1] + x[e + 1];
            const float above = lanes_above(sum);
            const float all = __shfl_sync(0xffffffffu, above + sum, 0);
            float y[4];
            if (i + 1 < count) load_gates(p, hv, t0 + (c_first + count - 2 - i) * kLinC, kLinC, y);
            if (i > 0 && !warp_wait(S, &S.bar.r_arr, (i & 1) ^ 1)) break;
#pragma unroll
            for (int e = 0; e < 4; ++e) S.w[4 * lane + e] = expf(carry + (above + suf[e]));
            __syncwarp();
            if (lane == 0) mbar_arrive(&S.bar.gates);
            carry += all;
#pragma unroll
            for (int e = 0; e < 4; ++e) x[e] = y[e];
        }
        if (lane == 0) p.range_decay[slot] = carry;
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    if (warp == 0) tc::tmem_dealloc(tmem, 128);
    if (tid == 0 && S.abort) report(p.status, GDN_ERR_TIMEOUT);
}

// Start states of a sequence's ranges, in order, over the ranges' own states (the slot of
// range r receives the start of range r + 1): S <- e^{decay_r} S + R_r, four columns a
// thread.  Bound by memory; the loads of later ranges do not wait for the chain.
constexpr int kStartThreads = 256;
__global__ void __launch_bounds__(kStartThreads)
linear_start_kernel(const LinParams p) {
    const int hv = blockIdx.y, n = blockIdx.z;
    const int t0 = p.cu[n], len = p.cu[n + 1] - t0;
    const int nch = (len + kLinC - 1) / kLinC;
    const int rc = range_chunks_of(nch, p.max_par);
    const int ranges = (nch + rc - 1) / rc;
    if (ranges <= 1) return;
    const int at = blockIdx.x * kStartThreads + threadIdx.x;     // float4 of the 128 x 128
    const int64_t step = (int64_t)p.Hv * 4096;
    float4 *R = reinterpret_cast<float4 *>(p.ranges) + (range_slot0(p, n, t0) * p.Hv + hv) * 4096 + at;
    const float *dec = p.range_decay + (range_slot0(p, n, t0) + 1) * p.Hv + hv;
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
    if (p.h0) s = reinterpret_cast<const float4 *>(p.h0 + ((int64_t)n * p.Hv + hv) * 16384)[at];
    grid_dependency_wait();
    if (p.in_place) R[0] = s;
    R += step;
    for (int r = 0; r < ranges - 1; r += 4) {
        float4 x[4];
        float a[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            if (r + e < ranges - 1) {
                x[e] = R[(r + e) * step];
                a[e] = expf(dec[(int64_t)(r + e) * p.Hv]);
            }
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            if (r + e < ranges - 1) {
                s.x = fmaf(a[e], s.x, x[e].x);
                s.y = fmaf(a[e], s.y, x[e].y);
                s.z = fmaf(a[e], s.z, x[e].z);
                s.w = fmaf(a[e], s.w, x[e].w);
                R[(r + e) * step] = s;
            }
        }
    }
}

}  // namespace gdn

namespace gdn_host {

namespace {

constexpr int kMaxDev = 64;

int device_sms() {
    static std::atomic<int> cached[kMaxDev];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDev) return 0;
    int v = cached[dev].load(std::memory_order_relaxed);
    if (v == 0) {
        if (cudaDeviceGetAttribute(&v, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
        cached[dev].store(v, std::memory_order_relaxed);
    }
    return v;
}

// [T, H, 128] bf16 token-major view -> map (d, head, token), boxes of 64 x 1 x 128.
bool tile_map(CUtensorMap *m, const void *ptr, int64_t T, int H, int64_t tok) {
    auto fn = tensor_map_encoder();
    if (!fn) return false;
    cuuint64_t dims[3] = {128, (cuuint64_t)H, (cuuint64_t)T};
    cuuint64_t strides[2] = {256, (cuuint64_t)tok * 2};
    cuuint32_t box[3] = {64, 1, gdn::kLinC}, unit[3] = {1, 1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(ptr), dims, strides, box,
              unit, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

struct Plan {
    int max_par, max_ranges, slots_per_seq;
    int64_t slots;
};
Plan plan_ranges(const int32_t *cu, int N, int64_t T, int Hv) {
    Plan pl = {1, 1, 0, 0};
    const int sms = device_sms();
    pl.max_par = std::max(1, sms / std::max(1, Hv));
    for (int n = 0; n < N; ++n) {
        const int nch = (cu[n + 1] - cu[n] + gdn::kLinC - 1) / gdn::kLinC;
        const int rc = gdn::range_chunks_of(nch, pl.max_par);
        pl.max_ranges = std::max(pl.max_ranges, (nch + rc - 1) / rc);
    }
    if (pl.max_ranges <= 1) return pl;
    const int64_t by_seq = (int64_t)N * pl.max_ranges, by_tok = T / gdn::kMinRangeTokens + N;
    pl.slots = std::min(by_seq, by_tok);
    pl.slots_per_seq = by_seq <= by_tok ? pl.max_ranges : 0;
    return pl;
}
size_t range_bytes(int64_t slots, int Hv) { return (size_t)slots * Hv * 65536; }

}  // namespace

bool linear_tc_supported(int64_t D, int in_f32, uint32_t flags) {
    return D == 128 && !in_f32 && !(flags & GDN_PREFILL_SIMT);
}

size_t linear_tc_workspace(const int32_t *cu, int32_t N, int64_t T, int32_t Hv) {
    const Plan pl = plan_ranges(cu, N, T, Hv);
    return pl.slots ? range_bytes(pl.slots, Hv) + ((size_t)pl.slots * Hv * 4 + 255) / 256 * 256 : 0;
}

gdn_status_t launch_linear_tc(const LinearArgs &a, cudaStream_t st) {
    const Plan pl = plan_ranges(a.cu_host, a.N, a.T, a.Hv);
    gdn::LinMaps maps;
    if (!tile_map(&maps.q, a.q, a.T, a.Hk, a.q_tok) || !tile_map(&maps.k, a.k, a.T, a.Hk, a.k_tok) ||
        !tile_map(&maps.v, a.v, a.T, a.Hv, a.v_tok))
        return GDN_ERR_CUDA;
    gdn::LinParams p = {};
    p.g = a.g;
    p.g_tok = a.g_tok;
    p.cu = a.cu;
    p.h0 = a.h0;
    p.hT = a.hT;
    p.o = (gdn::bf16 *)a.o;
    p.o_tok = a.o_tok;
    p.ranges = (float *)a.ws;
    p.range_decay = (float *)((uint8_t *)a.ws + range_bytes(pl.slots, a.Hv));
    p.Hk = a.Hk;
    p.Hv = a.Hv;
    p.max_par = pl.max_par;
    p.in_place = a.h0 && a.h0 == a.hT;
    p.slots_per_seq = pl.slots_per_seq;
    p.scale = a.scale;
    p.status = a.status;
    static std::atomic<uint64_t> ready{0};   // one bit per device
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return GDN_ERR_CUDA;
    if (dev >= kMaxDev || !((ready.load() >> dev) & 1u)) {
        if (cudaFuncSetAttribute(gdn::linear_out_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 (int)sizeof(gdn::LinSmem)) != cudaSuccess ||
            cudaFuncSetAttribute(gdn::linear_range_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 (int)sizeof(gdn::LinSmem)) != cudaSuccess)
            return GDN_ERR_CUDA;
        if (dev < kMaxDev) ready.fetch_or(1ull << dev);
    }
    const dim3 block(gdn::kLinThreads), grid(pl.max_ranges, a.Hv, a.N);
    if (pl.max_ranges <= 1) {
        gdn::linear_out_kernel<<<grid, block, sizeof(gdn::LinSmem), st>>>(maps, p);
        return cudaGetLastError() == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
    }
    gdn::linear_range_kernel<<<dim3(pl.max_ranges - 1, a.Hv, a.N), block, sizeof(gdn::LinSmem), st>>>(maps, p);
    if (cudaGetLastError() != cudaSuccess) return GDN_ERR_CUDA;
    if (launch_dependent(gdn::linear_start_kernel, dim3(4096 / gdn::kStartThreads, a.Hv, a.N),
                         dim3(gdn::kStartThreads), 0, st, p) != cudaSuccess ||
        launch_dependent(gdn::linear_out_kernel, grid, block, sizeof(gdn::LinSmem), st, maps, p) != cudaSuccess)
        return GDN_ERR_CUDA;
    return GDN_OK;
}

}  // namespace gdn_host
