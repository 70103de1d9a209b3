// linear_tc.cu -- linear attention with a decay for each head over packed prompts, on the
// tensor cores (tcgen05, TMEM, TMA): bf16 activations, D = 128.
//
// A sequence is cut into chunks of 128 tokens.  With G_i the chunk's inclusive sums of the
// log decays, T their total and S the fp32 state at the chunk's start,
//     O = scale (e^{G_i} q_i S + sum_{j <= i} e^{G_i - G_j} (q_i.k_j) v_j)
//     S <- e^T S + sum_j e^{T - G_j} k_j v_j^T
// which is four 128 x 128 x 128 products a chunk, the last of them over the weighted keys,
// which go in as three bf16 terms, 24 bits together, so that the state keeps fp32 accuracy
// (a pair left it off by 3e-6 of its norm, three terms by 3e-7 to 6e-7; 62 -> 71 us on 4096
// tokens of 48 heads):
//     Q K^T,   Q S,   P V,   (hi + lo + rest)^T V
// e^{T - G_j} comes from sums taken from the chunk's end and e^{G_i - G_j} inside a 32 x 32
// block as a product of two factors where the block decays by less than 2^60, else (or with a
// NaN in it) from its exponent, and elsewhere as a product of two factors at most 1: nothing
// overflows however strong the decay.
//
// Roundings below fp32, all to bf16 and all in operands whose products only reach the bf16
// output: P, and S where it multiplies Q.  The state itself never goes through them.
//
// linear_out_kernel: one CTA per (sequence range, v-head) walks its chunks with the state
// in registers (32 floats a thread).  Warps 0-15 do the elementwise work, a thread holding
// one TMEM lane and a quarter of the columns: weighted keys (A), P (B), state (C), output
// (D); warp 16 issues the products, warp 17 the tile loads, warp 18 the sums of the gates.
//
// A value that is not finite would reach the chunk's earlier tokens through its weights of zero.
// It leaves its column of the state so to the end, which costs nothing to see; a CTA that sees it
// runs once more, and this time warp 18 takes such values out before the products and their
// columns become NaN from their tokens on, in the outputs and in the state.  (4096 tokens of 48
// heads 70 us, 68.5 without all this, 81 where every call looks at every chunk's values.)
//
// An SM's shared memory passes 128 bytes a clock, which a 128 x 128 product with both
// operands there uses up: with P and the weighted keys in shared memory a chunk moved 5100
// clocks' worth (measured 8700 a chunk).  They are TMEM operands instead: P over the scores
// it came from, the keys (transposed on the way by ldmatrix) over the output accumulator
// that is not in use yet, their third term over the half of the scores that P leaves.  That
// leaves 3328 clocks of traffic and room for two buffers of each of Q, K and V.  TMEM (512
// columns): scores / P and rest, Q S, P V / weighted keys, state.
//
// 4096 tokens of 16 k-heads and 48 v-heads take 70 us, 8 packed prompts of 27598 tokens 405:
// 2.0 and 2.4 TB/s of what has to be moved, 183 and 214 TFLOP/s.  A chunk takes about 5700
// clocks, A 1500 (packing on the ALU pipe), B 1300, C 750, D 900 and the waits for products
// between them; one CTA fills an SM's TMEM and shared memory, so nothing else hides them.
//
// A long sequence over few heads would leave SMs idle, so it is cut into ranges that run
// side by side: linear_range_kernel gives every range's own state (the products added
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

constexpr int kOrdered = 64;

struct LinMaps {
    CUtensorMap q, k, v, o;
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
    // Sequences from the longest to the shortest, where there are at most kOrdered of them: a
    // long one started last would leave the device to itself (eight packed prompts of 951 to
    // 8192 tokens: 407 us as they come, 399 so; with more of them each is a small part).
    int ordered;
    uint8_t order[kOrdered];
    __device__ __forceinline__ int sequence(int z) const { return ordered ? order[z] : z; }
};

// Chunks per range of a sequence of nch chunks.  Under 12 chunks the other passes cost more
// than they save wherever the device is busy (alone, split against whole: 8 chunks 37 us
// against 33, 10 chunks 35 against 39 with 8 heads and 40 against 39 with 48; a batch of
// eight ragged sequences of 48 heads, split from 10 on: 434 against 419).
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
    uint64_t q[2], k[3], v[4];           // tiles loaded
    uint64_t qk[2], qs[2], kv[2], pv[2]; // products done (two: by the buffers they read)
    uint64_t gates;                      // this chunk's gate arrays are written
    uint64_t vs[2];                      // the values have been looked at
    uint64_t r_kt[2], r_p, r_s, r_o, r_arr;   // every elementwise warp: operands written, arrays read
    uint64_t out[2];                     // an output tile is written (over its chunk's Q)
    uint64_t kf[3], vf[4];               // range pass: tiles free
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
    uint32_t tmem;
    int abort;
    // by chunk mod 3: whether some value is not finite, and each column's first such token
    int bad[3];
    int again;           // the first pass saw a state that is not finite
    uint32_t first_bad[3][kLinC / 4];    // four columns a word; 255: none
    LinBars bar[2];      // one set for each pass
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

// Bounded wait on an mbarrier phase.  Gives up when the bound has passed or another thread
// of the CTA has given up; every role then leaves its loop.
template <int SLEEP_NS = 0>
__device__ __forceinline__ bool lin_wait(LinSmem &S, uint64_t *bar, uint32_t parity) {
    volatile int *abort = &S.abort;
    const bool ok = wait_bounded_poll<SLEEP_NS>(bar, parity, abort);
    if (!ok) *abort = 1;
    return ok;
}

// The same by a whole warp, which stays together whatever its lanes saw.
template <int SLEEP_NS = 0>
__device__ __forceinline__ bool warp_wait(LinSmem &S, uint64_t *bar, uint32_t parity) {
    return __all_sync(0xffffffffu, lin_wait<SLEEP_NS>(S, bar, parity)) != 0;
}

// The TMEM accesses of this warp (waited for) happen before the arrival.
__device__ __forceinline__ void warp_arrive_tmem(uint64_t *bar) {
    tc::fence_before_sync();
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
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

// The same with A in TMEM: 128 lanes, two of the depth's elements a word, 32 elements in the
// first 16 of each PITCH columns; B MN-major.
template <int PITCH>
__device__ __forceinline__ void product_ts(uint32_t d, uint32_t a, const uint8_t *b, bool add) {
    constexpr uint32_t id = tc::idesc_bf16(128, 128, 0, 1);
    const uint32_t b0 = tc::smem_u32(b);
#pragma unroll
    for (int ks = 0; ks < 8; ++ks) {
        const uint64_t db = tc::sdesc(b0 + ks * 2048, kBlk, 1024);
        asm volatile("{\n\t.reg .pred p, e;\n\t"
                     "elect.sync _|e, 0xffffffff;\n\t"
                     "setp.ne.b32 p, %4, 0;\n\t"
                     "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}"
                     :: "r"(d), "r"(a + PITCH * (ks >> 1) + 8 * (ks & 1)), "l"(db), "r"(id), "r"((uint32_t)(add || ks > 0)) : "memory");
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

__device__ __forceinline__ void ldmatrix_x4_trans(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
// 16 lanes x 16 words: register 2 x + y of lane l is lane l / 4 + 8 y, word 4 x + l % 4.
__device__ __forceinline__ void tmem_st_16x128b_x4(uint32_t taddr, const uint32_t (&r)[8]) {
    asm volatile("tcgen05.st.sync.aligned.16x128b.x4.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};"
                 :: "r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]),
                    "r"(r[6]), "r"(r[7]) : "memory");
}
// 32 lanes x 16 words, a lane's words in its thread.
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
                 "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};"
                 :: "r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]),
                    "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]),
                    "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]) : "memory");
}

// w_j k_j as three bf16 terms hi, lo, rest, transposed: TMEM lane d; of each PITCH columns, 16
// words of hi for 32 tokens, then 16 of lo; zero for tokens j >= L.  This warp takes d = 32 lq
// .. and j = 32 jb .., so it writes only columns that it alone has read before; ldmatrix hands
// it 8 x 8 blocks transposed, in the layout the 16-lane store wants.  rest is handed back, for
// store_rest() to place.
__device__ __forceinline__ void store_rest(uint32_t tmem, int lq, const uint32_t (&rest)[2][8]) {
#pragma unroll
    for (int th = 0; th < 2; ++th) tmem_st_16x128b_x4(tmem + ((uint32_t)(32 * lq + 16 * th) << 16), rest[th]);
}
template <bool TAIL, int PITCH>
__device__ __forceinline__ void weigh_keys(const uint8_t *k, uint32_t tmem, int lq, int jb, const float *w,
                                           int L, uint32_t (&rest)[2][8]) {
    const int lane = threadIdx.x & 31;
    float2 w2[4];
#pragma unroll
    for (int tg = 0; tg < 4; ++tg)
        w2[tg] = *reinterpret_cast<const float2 *>(w + 32 * jb + 8 * tg + 2 * (lane & 3));
    const float2 m1 = make_float2(-1.f, -1.f);
    const uint32_t base = tc::smem_u32(k) + (lq >> 1) * kBlk;
#pragma unroll
    for (int th = 0; th < 2; ++th) {
        uint32_t hi[8], lo[8];
#pragma unroll
        for (int tp = 0; tp < 2; ++tp) {
            // matrix lane / 8: tokens of group 2 tp + (matrix / 2), columns of group 2 th + matrix % 2
            const int mat = lane >> 3, tok = 32 * jb + 8 * (2 * tp + (mat >> 1)) + (lane & 7);
            uint32_t x[4];
            ldmatrix_x4_trans(x, base + tc::swz(tok, 4 * (lq & 1) + 2 * th + (mat & 1)));
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int tg = 2 * tp + (e >> 1);
                const float2 v = mul_f32x2(
                    make_float2(__uint_as_float(x[e] << 16), __uint_as_float(x[e] & 0xffff0000u)), w2[tg]);
                uint32_t h = pack_bf2(v.x, v.y);
                const float2 d = fma_f32x2(
                    make_float2(__uint_as_float(h << 16), __uint_as_float(h & 0xffff0000u)), m1, v);
                uint32_t r = pack_bf2(d.x, d.y);
                const float2 dd = fma_f32x2(
                    make_float2(__uint_as_float(r << 16), __uint_as_float(r & 0xffff0000u)), m1, d);
                uint32_t rr = pack_bf2(dd.x, dd.y);
                if (TAIL) {
                    const int j = 32 * jb + 8 * tg + 2 * (lane & 3);
                    const uint32_t keep = j + 1 < L ? 0xffffffffu : j < L ? 0x0000ffffu : 0u;
                    h &= keep;
                    r &= keep;
                    rr &= keep;
                }
                hi[4 * tp + e] = h;
                lo[4 * tp + e] = r;
                rest[th][4 * tp + e] = rr;
            }
        }
        const uint32_t at = tmem + ((uint32_t)(32 * lq + 16 * th) << 16) + PITCH * jb;
        tmem_st_16x128b_x4(at, hi);
        tmem_st_16x128b_x4(at + 16, lo);
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
// Whether some value of the first L tokens is not finite (one warp): 0 times it is NaN.
__device__ __forceinline__ bool any_nonfinite(const uint8_t *tile, int L) {
    const int lane = threadIdx.x & 31;
    const __nv_bfloat162 zero = __floats2bfloat162_rn(0.f, 0.f);
    __nv_bfloat162 acc[4] = {zero, zero, zero, zero};
#pragma unroll 4
    for (int r0 = 0; r0 < L; r0 += 4) {
        const int row = r0 + (lane >> 3);
#pragma unroll
        for (int kb = 0; kb < 2; ++kb) {
            uint4 x = make_uint4(0, 0, 0, 0);
            if (row < L) x = *reinterpret_cast<const uint4 *>(tile + kb * kBlk + tc::swz(row, lane & 7));
            const __nv_bfloat162 *p = reinterpret_cast<const __nv_bfloat162 *>(&x);
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[e] = __hfma2(p[e], zero, acc[e]);
        }
    }
    uint32_t any = 0u;
#pragma unroll
    for (int e = 0; e < 4; ++e) any |= *reinterpret_cast<const uint32_t *>(&acc[e]);
    return __any_sync(0xffffffffu, (any & 0x7f807f80u) != 0u) != 0;
}
// Zeroes them and notes each column's first token with one.
__device__ __noinline__ void take_out_nonfinite(uint8_t *tile, int L, uint8_t *first_bad) {
    for (int c = threadIdx.x & 31; c < 128; c += 32) {
        int first = 255;
        for (int row = L - 1; row >= 0; --row) {
            uint16_t *x = reinterpret_cast<uint16_t *>(tile + (c >> 6) * kBlk + tc::swz(row, (c & 63) >> 3)) + (c & 7);
            if ((*x & 0x7f80u) != 0x7f80u) continue;
            first = row;
            *x = 0;
        }
        first_bad[c] = (uint8_t)first;
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

// A range's pass over its chunks.  CAREFUL: values that are not finite are taken out; otherwise
// true where they have to be, and no final state is written then.
template <bool CAREFUL>
__device__ __forceinline__ bool linear_out_pass(const LinMaps &maps, const LinParams &p, LinSmem &S) {
    LinBars &B = S.bar[CAREFUL];
    uint8_t *sS = S.tile[6];      // Q, K, V of chunk i: tiles 0, 2, 4 + (i & 1)
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int range = blockIdx.x, hv = blockIdx.y, n = p.sequence(blockIdx.z), hk = hv / (p.Hv / p.Hk);
    const int t0 = p.cu[n], len = p.cu[n + 1] - t0;
    const int nch = (len + kLinC - 1) / kLinC;
    const int rc = range_chunks_of(nch, p.max_par);
    const int c_first = range * rc, c_last = min(nch, c_first + rc);
    const int count = c_last - c_first;          // 0 for an empty sequence
    const bool last = c_last >= nch;
    const uint32_t colSc = 0, colOi = 128, colOa = 256, colD = 384;   // P over Sc, keys over Oa

    if (tid == 0) {
        LinBars &b = B;
        for (uint64_t *x : {&b.q[0], &b.q[1], &b.k[0], &b.k[1], &b.v[0], &b.v[1], &b.qk[0], &b.qk[1], &b.qs[0], &b.qs[1],
                            &b.kv[0], &b.kv[1], &b.pv[0], &b.pv[1], &b.gates, &b.vs[0], &b.vs[1], &b.fin})
            tc::mbar_init(x, 1);
        for (uint64_t *x : {&b.r_kt[0], &b.r_kt[1], &b.r_p, &b.r_s, &b.r_o, &b.r_arr, &b.out[0], &b.out[1]})
            tc::mbar_init(x, kLinWarps);
        tc::mbar_fence_init();
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = S.tmem;

    const int lq = warp & 3, jb = warp >> 2;        // rows 32 lq .., columns 32 jb ..
    const int row = 32 * lq + lane;
    const int64_t st_off = (int64_t)row * 128 + 32 * jb;
    float st[32];                                   // (the elementwise warps')
    if (warp < kLinWarps) {
        const uint32_t tm = tmem + ((uint32_t)(32 * lq) << 16) + 32 * jb;
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
            warp_arrive(&B.r_s);
        }
        for (int i = 0; i < count; ++i) {
            // a buffer of two serves every other chunk
            const uint32_t ph = i & 1, ph2 = (i >> 1) & 1;
            const int t = t0 + (c_first + i) * kLinC;
            const int L = min(kLinC, t0 + len - t);
            // ---- A: weighted keys, over the P V that this warp has read (the gates' warp has
            // seen the keys' tile arrive)
            if (!warp_wait(S, &B.gates, ph)) break;
            uint32_t rest[2][8];
            if (L == kLinC) {
                weigh_keys<false, 32>(S.tile[2 + ph], tmem + colOa, lq, jb, S.w, L, rest);
            } else {
                weigh_keys<true, 32>(S.tile[2 + ph], tmem + colOa, lq, jb, S.w, L, rest);
                if (!warp_wait(S, &B.v[ph], ph2)) break;
                clear_rows(S.tile[4 + ph], L);
                tc::fence_async_smem();
            }
            tc::tmem_wait_st();
            warp_arrive_tmem(&B.r_kt[ph]);
            // ---- B: P = decay-weighted lower triangle of Q K^T
            if (!warp_wait(S, &B.qk[ph], ph2)) break;
            tc::fence_after_sync();
            const float eg = S.eg[row], decay = S.decay;
            uint32_t pk[16];
            if (jb <= lq) {
                const float gi = S.g2[row];
                // (a NaN among the block's gates makes its end NaN, but not the rows before it)
                const bool slow = jb == lq && !(S.g2[32 * jb] - S.ref[jb] < 60.f);
                const float f = p.scale * ex2(gi - S.ref[jb]);
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    float v[16];
                    tc::tmem_ld16(tm + colSc + 16 * c, v);
                    if (!slow) {
                        float4 b4[4];
#pragma unroll
                        for (int j = 0; j < 4; ++j) b4[j] = reinterpret_cast<const float4 *>(S.b)[8 * jb + 4 * c + j];
                        tc::tmem_wait_ld();
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            v[4 * j] *= f * b4[j].x;
                            v[4 * j + 1] *= f * b4[j].y;
                            v[4 * j + 2] *= f * b4[j].z;
                            v[4 * j + 3] *= f * b4[j].w;
                        }
                        if (jb == lq) {
#pragma unroll
                            for (int j = 0; j < 16; ++j) v[j] = 16 * c + j <= lane ? v[j] : 0.f;
                        }
                    } else {
                        tc::tmem_wait_ld();
#pragma unroll
                        for (int j = 0; j < 16; ++j)
                            v[j] = 16 * c + j <= lane ? v[j] * (p.scale * ex2(gi - S.g2[32 * jb + 16 * c + j])) : 0.f;
                    }
#pragma unroll
                    for (int j = 0; j < 8; ++j) pk[8 * c + j] = pack_bf2(v[2 * j], v[2 * j + 1]);
                }
            } else {
#pragma unroll
                for (int j = 0; j < 16; ++j) pk[j] = 0u;
            }
            // P and the keys' rest over the scores that this warp has read
            tmem_st16(tm + colSc, pk);
            store_rest(tmem + colSc + 32 * jb + 16, lq, rest);
            tc::tmem_wait_st();
            warp_arrive_tmem(&B.r_p);
            // (the values two chunks on are looked at after this arrival only)
            if (CAREFUL && !warp_wait(S, &B.vs[ph], ph2)) break;
            if (lane == 0) mbar_arrive(&B.r_arr);
            // ---- C: state
            if (!warp_wait(S, &B.kv[1], ph)) break;
            tc::fence_after_sync();
            float v[32];
            tc::tmem_ld32(tm + colD, v);
            tc::tmem_wait_ld();
#pragma unroll
            for (int j = 0; j < 32; ++j) st[j] = fmaf(decay, st[j], v[j]);
            const bool bad = CAREFUL && S.bad[i % 3] != 0;
            const uint32_t *first_bad = S.first_bad[i % 3] + 8 * jb;
            if (bad) {
#pragma unroll
                for (int j = 0; j < 32; ++j)
                    if (((first_bad[j >> 2] >> (8 * (j & 3))) & 255u) != 255u) st[j] = __int_as_float(0x7fffffff);
            }
            store_row(sS, jb, row, st);      // Q S came before the keys' product: it is done

            warp_arrive(&B.r_s);
            // ---- D: output; a full chunk goes over its Q tile (Q K and Q S are done) and leaves
            // by tensor store, a last, partial one straight from the threads
            if (!warp_wait(S, &B.pv[ph], ph2)) break;
            tc::fence_after_sync();
            uint32_t u[16];
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                float a[16];
                tc::tmem_ld16(tm + colOi + 16 * c, a);
                tc::tmem_ld16(tm + colOa + 16 * c, v);
                tc::tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    u[8 * c + e] = pack_bf2(fmaf(eg, a[2 * e], v[2 * e]), fmaf(eg, a[2 * e + 1], v[2 * e + 1]));
            }
            warp_arrive_tmem(&B.r_o);
            if (bad) {
#pragma unroll
                for (int j = 0; j < 32; ++j)
                    if (((first_bad[j >> 2] >> (8 * (j & 3))) & 255u) <= (uint32_t)row) u[j >> 1] |= 0x7fffu << (16 * (j & 1));
            }
            if (L == kLinC) {
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    *reinterpret_cast<uint4 *>(S.tile[ph] + (jb >> 1) * kBlk + tc::swz(row, 4 * (jb & 1) + c)) =
                        make_uint4(u[4 * c], u[4 * c + 1], u[4 * c + 2], u[4 * c + 3]);
                warp_arrive(&B.out[ph]);
            } else if (row < L) {
                uint4 *dst = reinterpret_cast<uint4 *>(p.o + (int64_t)(t + row) * p.o_tok + (int64_t)hv * 128 + 32 * jb);
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    dst[c] = make_uint4(u[4 * c], u[4 * c + 1], u[4 * c + 2], u[4 * c + 3]);
            }
        }
        if (!CAREFUL && count > 0) {
            float zero = 0.f;                       // or NaN
#pragma unroll
            for (int j = 0; j < 32; ++j) zero = fmaf(st[j], 0.f, zero);
            if (__any_sync(0xffffffffu, zero != zero) && lane == 0) S.again = 1;
        }
    } else if (warp == kLinWarps) {
        // ---- products
        for (int i = 0; i < count; ++i) {
            const uint32_t ph = i & 1, ph2 = (i >> 1) & 1;
            const uint8_t *sQ = S.tile[ph], *sK = S.tile[2 + ph], *sV = S.tile[4 + ph];
            if (!warp_wait(S, &B.q[ph], ph2) || !warp_wait(S, &B.k[ph], ph2)) break;
            if (i > 0 && !warp_wait(S, &B.pv[ph ^ 1], ((i - 1) >> 1) & 1)) break;      // P is read: the scores' turn
            tc::fence_after_sync();
            product<0, 0>(tmem + colSc, sQ, sK, false);
            tc::mma_commit_warp(&B.qk[ph]);
            if (!warp_wait(S, &B.r_s, ph)) break;
            if (i > 0 && !warp_wait(S, &B.r_o, ph ^ 1)) break;
            tc::fence_after_sync();
            product<0, 1>(tmem + colOi, sQ, sS, false);
            tc::mma_commit_warp(&B.qs[ph]);
            if (!warp_wait(S, &B.r_kt[ph], ph2) || !warp_wait(S, &B.v[ph], ph2)) break;
            if (CAREFUL && !warp_wait(S, &B.vs[ph], ph2)) break;
            tc::fence_after_sync();
            product_ts<32>(tmem + colD, tmem + colOa, sV, false);
            product_ts<32>(tmem + colD, tmem + colOa + 16, sV, true);
            tc::mma_commit_warp(&B.kv[0]);
            if (!warp_wait(S, &B.r_p, ph)) break;
            tc::fence_after_sync();
            product_ts<32>(tmem + colD, tmem + colSc + 16, sV, true);
            tc::mma_commit_warp(&B.kv[1]);
            // the keys' columns take P V next
            if (!warp_wait(S, &B.kv[0], ph)) break;
            tc::fence_after_sync();
            product_ts<32>(tmem + colOa, tmem + colSc, sV, false);
            tc::mma_commit_warp(&B.pv[ph]);
        }
        // everything issued has completed before the TMEM is freed
        tc::mma_commit_warp(&B.fin);
        wait_copy(&B.fin, 0);
    } else if (warp == kLinWarps + 1) {
        // ---- tile loads: buffers of two, each refilled when its last reader is done
        if (lane == 0) {
            tc::prefetch_tmap(&maps.q);
            tc::prefetch_tmap(&maps.k);
            tc::prefetch_tmap(&maps.v);
            int nk = 0, nq = 0, nv = 0;
            const int full = last && len % kLinC ? count - 1 : count;     // chunks of 128 tokens
            // the output of chunk i, when it is written over Q
            auto put = [&](int i) {
                if (!lin_wait<100>(S, &B.out[i & 1], (i >> 1) & 1)) return false;
                const int t = t0 + (c_first + i) * kLinC;
                tc::tma_store_3d(&maps.o, S.tile[i & 1], 0, hv, t);
                tc::tma_store_3d(&maps.o, S.tile[i & 1] + kBlk, 64, hv, t);
                tc::bulk_commit();
                return true;
            };
            bool ok = true;
            for (int i = 0; i < count && ok; ++i) {
                const uint32_t b = i & 1, was = ((i >> 1) & 1) ^ 1;   // chunk i - 2's use of the buffer
                const int t = t0 + (c_first + i) * kLinC;
                if (i >= 2 && !(ok = lin_wait<100>(S, &B.qk[b], was) && lin_wait<100>(S, &B.r_kt[b], was))) break;
                load_tile(S.tile[2 + b], &maps.k, &B.k[b], hk, t);
                ++nk;
                if (i >= 2) {
                    if (!(ok = put(i - 2))) break;
                    tc::bulk_wait_read<0>();
                }
                load_tile(S.tile[b], &maps.q, &B.q[b], hk, t);
                ++nq;
                if (i >= 2 && !(ok = lin_wait<100>(S, &B.pv[b], was))) break;
                load_tile(S.tile[4 + b], &maps.v, &B.v[b], hv, t);
                ++nv;
            }
            for (int i = max(0, count - 2); i < full && ok; ++i) ok = put(i);
            tc::bulk_wait_all();
            // (bounded) everything loaded has landed
            for (int x = max(0, nk - 2); x < nk; ++x) wait_copy(&B.k[x & 1], (x >> 1) & 1);
            for (int x = max(0, nq - 2); x < nq; ++x) wait_copy(&B.q[x & 1], (x >> 1) & 1);
            for (int x = max(0, nv - 2); x < nv; ++x) wait_copy(&B.v[x & 1], (x >> 1) & 1);
        }
    } else {
        // ---- gates; carefully, a look at the next chunk's values too
        auto look = [&](int i) {
            if (!warp_wait<100>(S, &B.v[i & 1], (i >> 1) & 1)) return false;
            const int L = min(kLinC, len - (c_first + i) * kLinC);
            uint8_t *tile = S.tile[4 + (i & 1)];
            const bool bad = any_nonfinite(tile, L);
            if (bad) {
                take_out_nonfinite(tile, L, reinterpret_cast<uint8_t *>(S.first_bad[i % 3]));
                tc::fence_async_smem();
            }
            if (lane == 0) S.bad[i % 3] = bad;
            __syncwarp();
            if (lane == 0) mbar_arrive(&B.vs[i & 1]);
            return true;
        };
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
            if (i > 0 && !warp_wait<100>(S, &B.r_arr, (i & 1) ^ 1)) break;
            if (!warp_wait<100>(S, &B.k[i & 1], (i >> 1) & 1)) break;
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
            if (lane == 0) mbar_arrive(&B.gates);
            // (chunk i + 1 has the words of chunk i - 2, which every warp has left)
            if (CAREFUL && i == 0 && !look(0)) break;
            if (CAREFUL && i + 1 < count && !look(i + 1)) break;
#pragma unroll
            for (int e = 0; e < 4; ++e) x[e] = y[e];
        }
    }
    // everything that was issued has completed
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    if (!CAREFUL && S.again && !S.abort) return true;
    if (warp < kLinWarps && last && p.hT && !S.abort) {
        float4 *out = reinterpret_cast<float4 *>(p.hT + ((int64_t)n * p.Hv + hv) * 16384 + st_off);
#pragma unroll
        for (int e = 0; e < 8; ++e)
            out[e] = make_float4(st[4 * e], st[4 * e + 1], st[4 * e + 2], st[4 * e + 3]);
    }
    return false;
}
// (a function of its own, so that the first pass is compiled without it)
__device__ __noinline__ void linear_out_careful(const LinMaps &maps, const LinParams &p, LinSmem &S) {
    linear_out_pass<true>(maps, p, S);
}

__global__ void __launch_bounds__(kLinThreads, 1)
linear_out_kernel(const __grid_constant__ LinMaps maps, const __grid_constant__ LinParams p) {
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    LinSmem &S = *reinterpret_cast<LinSmem *>(smem_raw);
    if (tc::smem_u32(smem_raw) & 1023u) {        // the tiles' swizzle needs it; never seen
        if (threadIdx.x == 0) report(p.status, GDN_ERR_CUDA);
        return;
    }
    const int n = p.sequence(blockIdx.z), len = p.cu[n + 1] - p.cu[n];
    const int nch = (len + kLinC - 1) / kLinC;
    if (blockIdx.x > 0 && (int)blockIdx.x * range_chunks_of(nch, p.max_par) >= nch) return;
    const int warp = threadIdx.x >> 5;
    if (warp == 0) {
        tc::tmem_alloc(&S.tmem, 512);
        tc::tmem_relinquish();
    }
    if (threadIdx.x == 0) S.abort = S.again = 0;
    if (linear_out_pass<false>(maps, p, S)) linear_out_careful(maps, p, S);
    __syncthreads();
    if (warp == 0) tc::tmem_dealloc(S.tmem, 512);
    if (threadIdx.x == 0 && S.abort) report(p.status, GDN_ERR_TIMEOUT);
}


// -------------------------------------------------------------------------- range states
// State that one range adds, from zero, with decays to the range's end: its chunks in
// reverse, each chunk's weights carrying the sum of the later ones, all added up in TMEM.
// Tiles: K x 3, V x 4; the weighted keys alternate between two TMEM places.
__global__ void __launch_bounds__(kLinThreads, 1)
linear_range_kernel(const __grid_constant__ LinMaps maps, const LinParams p) {
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    LinSmem &S = *reinterpret_cast<LinSmem *>(smem_raw);
    if (tc::smem_u32(smem_raw) & 1023u) {        // the tiles' swizzle needs it; never seen
        if (threadIdx.x == 0) report(p.status, GDN_ERR_CUDA);
        return;
    }
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    LinBars &B = S.bar[0];
    const int range = blockIdx.x, hv = blockIdx.y, n = p.sequence(blockIdx.z), hk = hv / (p.Hv / p.Hk);
    const int t0 = p.cu[n], len = p.cu[n + 1] - t0;
    const int nch = (len + kLinC - 1) / kLinC;
    const int rc = range_chunks_of(nch, p.max_par);
    const int c_first = range * rc, count = rc;
    if (c_first + rc >= nch) return;             // a last range: nothing reads its state
    const int64_t slot = (range_slot0(p, n, t0) + range + 1) * p.Hv + hv;

    if (warp == 0) {
        tc::tmem_alloc(&S.tmem, 512);
        tc::tmem_relinquish();
    }
    if (tid == 0) {
        S.abort = 0;
        LinBars &b = B;
        for (uint64_t *x : {&b.k[0], &b.k[1], &b.k[2], &b.v[0], &b.v[1], &b.v[2], &b.v[3], &b.kv[0],
                            &b.kv[1], &b.vf[0], &b.vf[1], &b.vf[2], &b.vf[3], &b.gates, &b.fin})
            tc::mbar_init(x, 1);
        for (uint64_t *x : {&b.r_kt[0], &b.r_kt[1], &b.kf[0], &b.kf[1], &b.kf[2], &b.r_arr})
            tc::mbar_init(x, kLinWarps);
        tc::mbar_fence_init();
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = S.tmem;
    // step i takes chunk c_first + count - 1 - i; its use of a buffer among x is that
    // buffer's (i / x)-th.  TMEM: the state at 0, weighted keys at 128 and 320.
    if (warp < kLinWarps) {
        bool ok = true;
        for (int i = 0; i < count && ok; ++i) {
            const int bf = i & 1, kb = i % 3;
            if (!(ok = warp_wait(S, &B.gates, i & 1) && warp_wait(S, &B.k[kb], (i / 3) & 1))) break;
            if (i >= 2 && !(ok = warp_wait(S, &B.kv[bf], ((i >> 1) & 1) ^ 1))) break;
            tc::fence_after_sync();
            uint32_t rest[2][8];
            weigh_keys<false, 48>(S.tile[kb], tmem + 128 + 192 * bf, warp & 3, warp >> 2, S.w, kLinC, rest);
            store_rest(tmem + 128 + 192 * bf + 48 * (warp >> 2) + 32, warp & 3, rest);
            tc::tmem_wait_st();
            warp_arrive_tmem(&B.r_kt[bf]);
            if (lane == 0) mbar_arrive(&B.kf[kb]);
            if (lane == 0) mbar_arrive(&B.r_arr);
        }
        const int e = count - 1;
        if (ok && warp_wait(S, &B.kv[e & 1], (e >> 1) & 1)) {
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
            const int bf = i & 1, vb = i & 3;
            if (!warp_wait(S, &B.r_kt[bf], (i >> 1) & 1) || !warp_wait(S, &B.v[vb], (i >> 2) & 1)) break;
            tc::fence_after_sync();
            product_ts<48>(tmem, tmem + 128 + 192 * bf, S.tile[3 + vb], i > 0);
            product_ts<48>(tmem, tmem + 144 + 192 * bf, S.tile[3 + vb], true);
            product_ts<48>(tmem, tmem + 160 + 192 * bf, S.tile[3 + vb], true);
            tc::mma_commit_warp(&B.kv[bf]);
            tc::mma_commit_warp(&B.vf[vb]);
        }
        tc::mma_commit_warp(&B.fin);
        wait_copy(&B.fin, 0);
    } else if (warp == kLinWarps + 1) {
        if (lane == 0) {
            int nk = 0, nv = 0;
            for (int i = 0; i < count; ++i) {
                const int kb = i % 3, vb = i & 3, t = t0 + (c_first + count - 1 - i) * kLinC;
                if (i >= 3 && !lin_wait<100>(S, &B.kf[kb], ((i / 3) & 1) ^ 1)) break;
                load_tile(S.tile[kb], &maps.k, &B.k[kb], hk, t);
                ++nk;
                if (i >= 4 && !lin_wait<100>(S, &B.vf[vb], ((i >> 2) & 1) ^ 1)) break;
                load_tile(S.tile[3 + vb], &maps.v, &B.v[vb], hv, t);
                ++nv;
            }
            for (int x = max(0, nk - 3); x < nk; ++x) wait_copy(&B.k[x % 3], (x / 3) & 1);
            for (int x = max(0, nv - 4); x < nv; ++x) wait_copy(&B.v[x & 3], (x >> 2) & 1);
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
            if (i > 0 && !warp_wait<100>(S, &B.r_arr, (i & 1) ^ 1)) break;
#pragma unroll
            for (int e = 0; e < 4; ++e) S.w[4 * lane + e] = expf(carry + (above + suf[e]));
            __syncwarp();
            if (lane == 0) mbar_arrive(&B.gates);
            carry += all;
#pragma unroll
            for (int e = 0; e < 4; ++e) x[e] = y[e];
        }
        if (lane == 0) p.range_decay[slot] = carry;
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    if (warp == 0) tc::tmem_dealloc(tmem, 512);
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
        !tile_map(&maps.v, a.v, a.T, a.Hv, a.v_tok) || !tile_map(&maps.o, a.o, a.T, a.Hv, a.o_tok))
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
    p.ordered = a.N > 1 && a.N <= gdn::kOrdered;
    if (p.ordered) {
        for (int n = 0; n < a.N; ++n) p.order[n] = (uint8_t)n;
        const int32_t *cu = a.cu_host;
        std::sort(p.order, p.order + a.N, [cu](int x, int y) {
            const int lx = cu[x + 1] - cu[x], ly = cu[y + 1] - cu[y];
            return lx != ly ? lx > ly : x < y;
        });
    }
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
