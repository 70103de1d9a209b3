// kv_attention.cu -- attention of new tokens over a paged 4-bit key/value cache.
//
//     o = sum_j p_j v_j / sum_j p_j,   p_j = exp(scale q.k_j),   j <= kv_len - m + i
// for token i of the m new tokens of a sequence with kv_len tokens (the new ones
// included, already in the cache).  A row that sees no key (kv_len < m - i) gives zeros,
// and a log-sum-exp of -inf.
#include <algorithm>
#include <atomic>

#include "bulk_ptx.cuh"
#include "kv_format.cuh"

namespace gdn {

// ------------------------------------------------------------------ general form
// Any activation type: one CTA per (token, query head).  A thread takes one key of a tile
// for the scores and D / 128 elements (or half the keys, for D = 64) for the values.
// Everything is fp32.
constexpr int kKvSimtThreads = 128;

template <typename T, int D>
__global__ void __launch_bounds__(kKvSimtThreads)
kv_attention_simt_kernel(KvView kv, const T *__restrict__ q, T *__restrict__ o, float *lse,
                         int64_t q_tok, int64_t o_tok, int Hq, int max_kv_len, float scale,
                         int32_t *status) {
    using R = KvRec<D>;
    constexpr int NT = kKvSimtThreads;
    constexpr int EL = D / NT < 1 ? 1 : D / NT;       // elements per thread
    constexpr int SPLIT = D / NT < 1 ? NT / D : 1;    // threads that share an element
    __shared__ float sq[D];
    __shared__ float sp[NT];
    __shared__ int64_t srec[NT];
    __shared__ float sred[NT / 32];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int64_t t = blockIdx.x;
    const int hq = blockIdx.y, hkv = hq / (Hq / kv.Hkv);
    const int n = kv.cu ? sequence_of(kv.cu, kv.N, (int)t) : (int)t;
    const int len = kv.kv_lens[n];
    if (len < 0 || len > max_kv_len || len > kv.capacity()) {
        if (tid == 0) report(status, GDN_ERR_SEQLENS);
        return;
    }
    const int keys = len - (kv.cu ? kv.cu[n + 1] - (int)t : 1) + 1;   // keys this row sees
    for (int d = tid; d < D; d += NT) sq[d] = to_f32(q[t * q_tok + (int64_t)hq * D + d]);
    __syncthreads();

    float m = -INFINITY, l = 0.f, acc[EL] = {};
    for (int base = 0; base < keys; base += NT) {
        const int j = base + tid;
        float s = -INFINITY;
        int64_t vrec = -1;
        if (j < keys) {
            const int page = kv.table[(int64_t)n * kv.table_width + (j >> kv.page_log2)];
            if (page >= 0 && page < kv.pages) {
                const int64_t at = (int64_t)(j & ((1 << kv.page_log2) - 1)) * R::BYTES;
                const uint8_t *rec = kv.block(page, 0, hkv, R::BYTES) + at;
                vrec = kv.block(page, 1, hkv, R::BYTES) + at - kv.data;
                s = 0.f;
#pragma unroll 1
                for (int g = 0; g < R::NG; ++g) {
                    float dot = 0.f, sum = 0.f;
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        const uint32_t w = reinterpret_cast<const uint32_t *>(rec)[c * R::NG + g];
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            const float qe = sq[32 * g + 8 * c + e];
                            dot = fmaf(qe, (float)((w >> (4 * e)) & 15u), dot);
                            sum += qe;
                        }
                    }
                    const float2 sm = __half22float2(reinterpret_cast<const __half2 *>(rec + R::CODES)[g]);
                    s = fmaf(sm.x, dot, fmaf(sm.y, sum, s));
                }
                s *= scale;
            } else {
                report(status, GDN_ERR_INDEX);
            }
        }
        // the tile's maximum, then the running one
        float mt = s;
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, off));
        if (lane == 0) sred[warp] = mt;
        __syncthreads();
        mt = fmaxf(fmaxf(sred[0], sred[1]), fmaxf(sred[2], sred[3]));
        const float mnew = fmaxf(m, mt);
        const float msafe = mnew == -INFINITY ? 0.f : mnew;
        const float keep = expf(m - msafe);
        const float p = vrec < 0 ? 0.f : expf(s - msafe);
        m = mnew;
        sp[tid] = p;
        srec[tid] = vrec;
        l = fmaf(l, keep, p);      // this thread's keys only; summed at the end
#pragma unroll
        for (int x = 0; x < EL; ++x) acc[x] *= keep;
        __syncthreads();
        const int cnt = min(NT, keys - base);
#pragma unroll
        for (int x = 0; x < EL; ++x) {
            const int d = SPLIT > 1 ? tid % D : tid + NT * x;
            const int word = 8 * (d / 64) + (d % 32) / 4, sh = 16 * ((d / 32) & 1) + 4 * (d & 3);
            for (int i = SPLIT > 1 ? tid / D : 0; i < cnt; i += SPLIT) {
                if (srec[i] < 0) continue;
                const uint8_t *rec = kv.data + srec[i];
                const uint32_t w = reinterpret_cast<const uint32_t *>(rec)[word];
                const float2 sm = __half22float2(reinterpret_cast<const __half2 *>(rec + R::CODES)[d / 32]);
                acc[x] = fmaf(sp[i], fmaf(sm.x, (float)((w >> sh) & 15u), sm.y), acc[x]);
            }
        }
        __syncthreads();
    }
    // sum of the threads' l, and of the threads that share an element
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) l += __shfl_xor_sync(0xffffffffu, l, off);
    if (lane == 0) sred[warp] = l;
    sp[tid] = acc[0];
    __syncthreads();
    l = sred[0] + sred[1] + sred[2] + sred[3];
    const float inv = l > 0.f ? 1.f / l : (l == l ? 0.f : l);
    if (SPLIT > 1) {
        if (tid < D) {
            float s = 0.f;
            for (int x = 0; x < SPLIT; ++x) s += sp[tid + D * x];
            o[t * o_tok + (int64_t)hq * D + tid] = from_f32<T>(s * inv);
        }
    } else {
#pragma unroll
        for (int x = 0; x < EL; ++x)
            o[t * o_tok + (int64_t)hq * D + tid + NT * x] = from_f32<T>(acc[x] * inv);
    }
    if (lse && tid == 0) lse[t * Hq + hq] = l == 0.f ? -INFINITY : m + logf(l);
}

// ------------------------------------------------------------------ tensor-core form
// bf16 activations.  The rows of one kv-head (G query heads x m tokens, token-major) are
// cut into tiles of 8 NT; one CTA takes one row tile and one split of the keys, its four
// warps taking every fourth block of 32 keys with a softmax state of their own, joined at
// the end (wide rows: blocks of 64 keys between the four of them, below).  All products run as m16n8k16 on fp16 with keys (then elements) as the 16 rows
// and query rows as the 8 columns, so that few rows waste little of an instruction and
// each stored code is unpacked once per warp however many rows use it:
//     S^T = K Q^T      O^T = V^T P^T
//
// A code u enters as the fp16 bit pattern u or u << 4, i.e. the subnormal u 2^-24 or
// u 2^-20: one AND per pair of codes, no conversion, and exact.  Scale and minimum stay
// outside: with q', p' the rows as the fragments hold them and g the groups of 32,
//     q.k = sum_g scale_kg (q'.u)_g + sum_g min_kg (sum of q' over g)
//     o_d = sum_k (p_k scale_kg) u_kd + sum_k p_k min_kg
// the first scales applied to the fp32 products, the second to p in fp16, and both terms
// in the minima as one small product more (the sums of q' as an fp16 pair hi + lo).
//
// Fewer bits than fp32: q is scaled by a power of two per row so that its largest element
// lies in [2^11, 2^12), where fp16 holds a bf16 exactly (down to 2^-26 of the largest);
// p is rounded to fp16 (2^-11); it is taken against a reference within 2 (in powers of two)
// of the running maximum and lifted by 2^8, so it stays below 2^10 and a weight of 2^-32 of
// the largest is still held.  p scale goes in as an fp16 pair (product and what its rounding
// left out): scale * code and minimum cancel to a value several times smaller than either, so
// one fp16 product would show where few keys carry a row.  (Without the lift, values of 2^-11
// their usual size left outputs 30 times their bound off, and a key that outweighs each of
// 12000 others by 2^18 four times.)  Scores, sums, maxima and outputs are fp32.
//
// Scales from 64 on (groups of values that span 960) may carry p scale past fp16.  Then sums
// are not finite, and a CTA that ends with one takes its keys once more, with a lift that
// follows the scales.  (64 sequences of up to 16384 keys 180 us, 178.5 without lift and end
// check, 183 where every pass looks at its scales.)
//
// Keys come in blocks of 16 records of a page (pages hold a multiple of 16) by bulk copies
// into a ring that each warp runs for itself: no barrier of the CTA inside the loop, but
// where warps share the blocks.
//
// 64 sequences of up to 16384 keys, 32 query heads over 8 of 128, take 180 us: 640 MB, 52% of
// the HBM rate, bound by issue (59%): a block of 32 keys costs a warp 880 instructions, start
// and join of eight such blocks included.  24 rows of 256 elements over 131072 keys of 4 heads
// take 102 us, 24% of the HBM rate, bound by latency at twelve warps an SM.
constexpr int kAttnWarps = 4;
constexpr int kAttnThreads = 32 * kAttnWarps;

// NT tiles of eight rows; VS: warps that share a slice of the keys (four where the output
// accumulators, D NT / 4 registers a thread, would not fit otherwise).  Each of the four takes
// the scores of a quarter of a block's keys and, with the others' weights, a quarter of the
// values' elements (24 rows of 256 over 131072 keys 98 us, with two warps a slice 107; 16
// sequences of 4096 to 8192 keys 87 and 124; before the centring below).
template <int D, int NT> struct AttnShape {
    using R = KvRec<D>;
    static constexpr int ROWS = 8 * NT;
    static constexpr int VS = D * NT > 256 ? 4 : 1;
    static constexpr int SLICES = kAttnWarps / VS;
    static constexpr int KSUB = VS > 1 ? 4 : 2;                 // a block: parts of 16 keys
    static constexpr int BLOCK = 16 * KSUB;
    static constexpr int PART = 16 * R::BYTES;
    static constexpr int KEYS = BLOCK / VS * R::BYTES;          // a block's keys of one warp
    static constexpr int VALUES = BLOCK * R::BYTES;             // and its values
    // two blocks of each: keys for every warp, values for every slice
    static constexpr int RING = 2 * (kAttnWarps * KEYS + SLICES * VALUES);
    static constexpr int JOIN = SLICES * ROWS * D * 4;          // reuses the ring
    static constexpr int BUF = RING > JOIN ? RING : JOIN;
    static constexpr int QF = NT * R::NG * 32 * 16;             // q fragments
    static constexpr int QM = NT * 32 * 8;                      // group sums of q
    static constexpr int SWAP = VS > 1 ? kAttnWarps * (NT * 256 + ROWS * 4 + 16) : 0;   // weights, maxima, flag
    static constexpr int TAIL = SWAP + ROWS * (4 + 4) + kAttnWarps * ROWS * 8 + 2 * 8 * 4 * kAttnWarps + 4 * 4 * kAttnWarps;
    static constexpr int SMEM = BUF + QF + QM + TAIL;
    // CTAs per SM: latency is what more of them hide, until registers spill (64 sequences of
    // up to 16384 keys, D NT = 128: 173 us with four, 192 with three, 191 with five)
    static constexpr int CTAS = D * NT <= 128 ? 4 : VS > 1 ? 3 : 2;
};

// Keys per split of a context of len keys.  A warp's start and join cost about as much as 40
// keys, so long splits serve a full device and short ones a lone sequence: 128 keys up to
// 512, 256 up to 2048, 1024 above (8 kv-heads of 128, 64 sequences of 4096 to 8192 keys: 140
// us with 1024, 161 with 512, 206 with 256; one sequence of 8192: 21, 16.5 and 14.5), 512
// where four warps share them (24 rows of 256 elements over 4 kv-heads: 64 sequences 326 us
// with 512, 297 with 1024; one 37 and 55); and so long that one sequence's CTAs, row tiles
// times kv-heads times splits, all fit on the device at once (131072 keys, two CTAs an SM
// then: 116 us with 1728, 131 with 2048, 144 with 1024, 204 with 3456).  From 256 new rows on
// nothing is split.  All of it depends on the sequence's own lengths and heads only.
constexpr int kSplitMaxRows = 256;
// CTAs on the device at once that splits are made for (tiles of 256 elements: two an SM for
// eight rows, three for more), and the most of them.
__host__ __device__ __forceinline__ int split_ctas(int rows, int D) { return (D == 256 && rows > 8 ? 3 : 2) * 152; }
constexpr int kSplitMaxCtas = 3 * 152;
// Most tiles of eight rows a CTA takes.  What more would save in reading and unpacking keys is
// lost again in registers: 16 sequences of 4096 to 8192 keys, 32 rows of 128 elements, 131 us
// with two tiles, 155 with four; 72 rows of 256, 223 us with three, 303 with one, and from 96
// rows on four lose a little to three.
__host__ __device__ constexpr int attn_max_nt(int D) { return D == 256 ? 3 : D == 128 ? 2 : 4; }
__host__ __device__ __forceinline__ int kv_split_base(int len, bool shared) { return len <= 512 ? 128 : len <= 2048 ? 256 : shared ? 512 : 1024; }
// Splits that one sequence of m new rows has room for among `fit` CTAs.
__host__ __device__ __forceinline__ int kv_split_room(int m, int G, int Hkv, int D, int fit) {
    const int rows = 8 * attn_max_nt(D);
    const int64_t ctas = (int64_t)Hkv * ((G * m + rows - 1) / rows);
    return m >= kSplitMaxRows || 2 * ctas > fit ? 1 : (int)(fit / (ctas > 0 ? ctas : 1));
}
// (room for single tokens comes with the launch: a division less on the way to the first load)
__device__ __forceinline__ int kv_split_len(int len, int m, int G, int Hkv, int D, int room_one) {
    const int room = m == 1 ? room_one : kv_split_room(m, G, Hkv, D, split_ctas(G * m, D)), base = kv_split_base(len, D == 256 && G * m > 8);
    if (room <= 1) return 0x40000000;
    if ((int64_t)room * base >= len) return base;
    return ((len + room - 1) / room + 63) / 64 * 64;
}
// Splits of len keys (0 where there are none).
__device__ __forceinline__ int splits_of(int len, int split_len) {
    return len > 0 ? (int)(((uint32_t)len + (uint32_t)split_len - 1) / (uint32_t)split_len) : 0;
}

// d = a b + c on 16 x 8 x 16, fp16 in, fp32 out.
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, "
        "{%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma16816_first(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                               uint32_t a3, uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, "
        "{%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}
__device__ __forceinline__ uint32_t mul_half2(uint32_t a, uint32_t b) {
    const __half2 h = __hmul2(*reinterpret_cast<const __half2 *>(&a), *reinterpret_cast<const __half2 *>(&b));
    return *reinterpret_cast<const uint32_t *>(&h);
}
// What rounding the product ab = a b left out.
__device__ __forceinline__ uint32_t mul_rest(uint32_t a, uint32_t b, uint32_t ab) {
    const __half2 h = __hfma2(*reinterpret_cast<const __half2 *>(&a), *reinterpret_cast<const __half2 *>(&b),
                              __hneg2(*reinterpret_cast<const __half2 *>(&ab)));
    return *reinterpret_cast<const uint32_t *>(&h);
}
__device__ __forceinline__ float exp2_approx(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// 4 x K contiguous 32-bit words, as wide loads.
template <int K>
__device__ __forceinline__ void load_words(const uint8_t *p, uint32_t (&w)[K]) {
    if constexpr (K == 2) {
        const uint2 t = *reinterpret_cast<const uint2 *>(p);
        w[0] = t.x; w[1] = t.y;
    } else {
#pragma unroll
        for (int i = 0; i < K / 4; ++i) {
            const uint4 t = reinterpret_cast<const uint4 *>(p)[i];
            w[4 * i] = t.x; w[4 * i + 1] = t.y; w[4 * i + 2] = t.z; w[4 * i + 3] = t.w;
        }
    }
}
__device__ __forceinline__ bool half_pair_nonfinite(uint32_t w) {
    return (w & 0x7c00u) == 0x7c00u || (w & 0x7c000000u) == 0x7c000000u;
}

// Weights are held at 2^lift times their size, below 2^(lift + 2) with the reference's slack.
// With a lift of 13 - k the scales may be up to 1.984 * 2^k; k is 5 where no pass has to be careful.
constexpr int kLeastK = 5;
constexpr uint32_t kTopScale = 0x3ff0u, kHalfExp = 0x0400u;     // fp16 bits
// Keys of a warp after which sums of long runs are stowed.
constexpr int kStowKeys = 2048;

constexpr uint32_t kNib0 = 0x000F000Fu, kNib1 = 0x00F000F0u;

struct AttnParams {
    KvView kv;
    const bf16 *q;
    bf16 *o;
    float *lse, *part_o;
    float2 *part_ml;
    int64_t q_tok, o_tok, slab;
    int Hq, row_tiles, tc_rows, room_one, max_kv_len;
    float scale;
    int32_t *status;
};

// A CTA's pass over its keys.  CAREFUL: every block's scales are looked at before its products,
// and the lift fits them; otherwise true where some sum is not finite, with nothing written.
template <int D, int NT, bool LONG, bool CAREFUL>
__device__ __forceinline__ bool attention_pass(const AttnParams &a) {
    const KvView &kv = a.kv;
    const bf16 *__restrict__ q = a.q;
    bf16 *__restrict__ o = a.o;
    float *__restrict__ lse = a.lse, *__restrict__ part_o = a.part_o;
    float2 *__restrict__ part_ml = a.part_ml;
    const int64_t q_tok = a.q_tok, o_tok = a.o_tok, slab = a.slab;
    const int Hq = a.Hq, row_tiles = a.row_tiles, tc_rows = a.tc_rows, room_one = a.room_one, max_kv_len = a.max_kv_len;
    const float scale = a.scale;
    int32_t *status = a.status;
    using R = KvRec<D>;
    using A = AttnShape<D, NT>;
    constexpr int NG = R::NG, NP = D / 64, REC = R::BYTES;
    extern __shared__ __align__(128) uint8_t smem[];
    uint8_t *ring = smem;
    uint4 *qf = reinterpret_cast<uint4 *>(smem + A::BUF);
    uint2 *qm = reinterpret_cast<uint2 *>(smem + A::BUF + A::QF);
    uint8_t *swap = smem + A::BUF + A::QF + A::QM;
    float *sfac = reinterpret_cast<float *>(swap + A::SWAP);
    uint32_t *snan = reinterpret_cast<uint32_t *>(sfac + A::ROWS);
    float2 *sml = reinterpret_cast<float2 *>(snan + A::ROWS);
    uint64_t *bars = reinterpret_cast<uint64_t *>(sml + kAttnWarps * A::ROWS);   // a set for each pass
    uint32_t *spages = reinterpret_cast<uint32_t *>(bars + 8 * kAttnWarps);
    if (CAREFUL) bars += 4 * kAttnWarps;

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, r = lane >> 2, c = lane & 3;
    const int split = blockIdx.x / row_tiles, rt = blockIdx.x % row_tiles;
    const int hkv = blockIdx.y, n = blockIdx.z;
    const int t0 = kv.cu ? kv.cu[n] : n, m = kv.cu ? kv.cu[n + 1] - t0 : 1;
    const int len = kv.kv_lens[n];
    const int G = Hq / kv.Hkv, rows = G * m, row0 = rt * A::ROWS;
    if (row0 >= rows || Hq * m >= tc_rows) return false;   // (tc_rows: the other kernel's sequences)
    if (len < 0 || len > max_kv_len || len > kv.capacity()) {
        if (tid == 0) report(status, GDN_ERR_SEQLENS);
        return false;
    }
    // keys seen by the tile's first and last row
    const int see_first = len - m + row0 / G + 1;
    const int see_last = len - m + (min(row0 + A::ROWS, rows) - 1) / G + 1;
    const int split_len = kv_split_len(len, m, G, kv.Hkv, D, room_one);
    const int splits = splits_of(see_last, split_len);   // 0: no key at all
    if (split > 0 && split >= splits) return false;      // (the grid is made for the most)
    const int k0 = split * split_len, k1 = see_last - k0 > split_len ? k0 + split_len : see_last;

    // ---- the warp's rings of keys and of values: block b holds keys k0 + 32 (slice + SLICES b) ..
    const int slice = warp / A::VS, dh = warp % A::VS;
    constexpr int STEP = A::BLOCK * A::SLICES, KSUB = A::KSUB;
    uint64_t *bar_k = bars + 4 * warp, *bar_v = (A::VS > 1 ? bars : bar_k) + 2;
    uint32_t *pg = spages + 4 * warp;          // per block (mod 4): which parts are there
    uint8_t *ring_k = ring + warp * 2 * A::KEYS, *ring_v = ring + 2 * (kAttnWarps * A::KEYS + slice * A::VALUES);
    const int first = k0 + A::BLOCK * slice;
    const int blocks = k1 > first ? (k1 - first + STEP - 1) / STEP : 0;
    // A lane each looks up the pages of a block's parts, for its keys and then for its values,
    // and copies them (warps that share a slice: each its own part); a page outside the cache
    // is left out and marked.  Keys run two blocks ahead, values one; the page of a lane's next
    // copy is looked up one copy ahead.
    const int sub_l = lane % KSUB, which = (lane / KSUB) & 1;
    const bool copies = A::VS == 1 || sub_l == dh;
    const uint32_t all_parts = (1u << KSUB) - 1, my_parts = A::VS > 1 ? 1u << dh : all_parts;
    const int32_t *table = kv.table + (int64_t)n * kv.table_width;
    const int64_t page_bytes = (int64_t)(2 * kv.Hkv * REC) << kv.page_log2;
    const uint8_t *base = kv.block(0, which, hkv, REC);
    const int slot_mask = (1 << kv.page_log2) - 1;
    int jf = lane < 2 * KSUB ? first + 16 * sub_l : 0x40000000;   // the next copy's first key
    int page_next = jf < k1 ? table[jf >> kv.page_log2] : -1;
    auto fetch = [&](int bk, int bv) {         // block bk of the keys, bv of the values; -1: none
        const bool mine = lane < 2 * KSUB && (which ? bv : bk) >= 0;
        const int j = jf, page = page_next;
        if (mine) {
            jf += STEP;
            page_next = jf < k1 ? table[jf >> kv.page_log2] : -1;
        }
        const bool want = mine && page >= 0 && page < kv.pages;
        if (mine && !want && j < k1) report(status, GDN_ERR_INDEX);
        const uint32_t ok = __ballot_sync(0xffffffffu, want);
        if (lane == 0 && bk >= 0) {
            pg[bk & 3] = ok & all_parts;
            tc::mbar_expect_tx(bar_k + (bk & 1), __popc(ok & my_parts) * A::PART);
        }
        if (lane == 0 && bv >= 0) tc::mbar_expect_tx(bar_v + (bv & 1), __popc((ok >> KSUB) & my_parts) * A::PART);
        __syncwarp();
        if (want && copies) {
            uint8_t *dst = which ? ring_v + (bv & 1) * A::VALUES + sub_l * A::PART
                                 : ring_k + (bk & 1) * A::KEYS + (A::VS > 1 ? 0 : sub_l * A::PART);
            bulk_load(dst, base + page * page_bytes + (j & slot_mask) * REC, A::PART,
                      which ? bar_v + (bv & 1) : bar_k + (bk & 1));
        }
    };
    if (lane == 0) {
        for (int x = 0; x < 4; ++x) tc::mbar_init(bar_k + x, x < 2 ? 1 : A::VS);
        tc::mbar_fence_init();
    }
    if (A::VS > 1) __syncthreads();            // the values' barriers are everyone's
    __syncwarp();
    if (blocks > 0) fetch(0, 0);
    if (blocks > 1) fetch(1, -1);

    // ---- q as fragments: lane (r, c) of a tile's warp holds elements 32 g + 8 c .. +7 of
    // row r, scaled; odd elements also by 1/16 (their codes come as u << 4)
    for (int nt = warp; nt < NT && !CAREFUL; nt += kAttnWarps) {
        const int row = row0 + 8 * nt + r;
        float x[NG][8];
        float mx = 0.f;
        const bf16 *src = q + (int64_t)(t0 + (row < rows ? row / G : 0)) * q_tok +
                          (int64_t)(hkv * G + (row < rows ? row % G : 0)) * D + 8 * c;
#pragma unroll
        for (int g = 0; g < NG; ++g) {
            if (row < rows) {
                unpack8(*reinterpret_cast<const uint4 *>(src + 32 * g), x[g]);
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e) x[g][e] = 0.f;
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) mx = fmaxf(mx, fabsf(x[g][e]));
        }
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
        // 2^ex brings the largest element into [2^11, 2^12) (rows below 2^-109 stay smaller)
        const int ex = mx < INFINITY ? min(11 + 127 - (int)(__float_as_uint(mx) >> 23), 120) : 0;
        // (the scale's sign goes to q, so that larger products mean larger scores)
        const float up = __int_as_float((127 + ex) << 23) * (scale < 0.f ? -1.f : 1.f);
        const float down = __int_as_float((127 - ex) << 23);
        float sums[NG];
#pragma unroll
        for (int g = 0; g < NG; ++g) {
            float sum = 0.f;
            __half h[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                h[e] = __float2half_rn(x[g][e] * up);
                sum += __half2float(h[e]);
            }
            sum += __shfl_xor_sync(0xffffffffu, sum, 1);
            sum += __shfl_xor_sync(0xffffffffu, sum, 2);
            sums[g] = sum;
            const __half2 sixteenth = __floats2half2_rn(0.0625f, 0.0625f);
            const __half2 f0 = __halves2half2(h[0], h[4]), f1 = __hmul2(__halves2half2(h[1], h[5]), sixteenth);
            const __half2 f2 = __halves2half2(h[2], h[6]), f3 = __hmul2(__halves2half2(h[3], h[7]), sixteenth);
            qf[(nt * NG + g) * 32 + lane] =
                make_uint4(*reinterpret_cast<const uint32_t *>(&f0), *reinterpret_cast<const uint32_t *>(&f1),
                           *reinterpret_cast<const uint32_t *>(&f2), *reinterpret_cast<const uint32_t *>(&f3));
        }
        // group sums times 2^-12 as hi + lo: lane c has group c (and c + 4)
        uint32_t mw[2] = {0u, 0u};
#pragma unroll
        for (int g = 0; g < NG; ++g) {
            const float v = sums[g] * 0.000244140625f;
            const float hi = __half2float(__float2half_rn(v));
            if ((g & 3) == c) mw[g >> 2] = pack_half2(hi, v - hi);
        }
        qm[nt * 32 + lane] = make_uint2(mw[0], mw[1]);
        // a score is (sum of products) 2^24 2^-ex scale; its log2 weight times log2 e
        if (c == 0) {
            sfac[8 * nt + r] = fmaxf(fabsf(scale) * (1.4426950408889634f * 16777216.f) * down, 1e-37f);   // not 0
            snan[8 * nt + r] = 0;
        }
    }
    __syncthreads();

    constexpr int NGV = NG / A::VS, NPV = NP / A::VS;      // this warp's groups, words of the values
    float O[NT][2 * NGV][4], Om[NT][4], off[NT][2], mrun[NT][2], lrun[NT][2], fac[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int x = 0; x < 2 * NGV; ++x)
#pragma unroll
            for (int e = 0; e < 4; ++e) O[nt][x][e] = 0.f;
#pragma unroll
        for (int e = 0; e < 4; ++e) Om[nt][e] = 0.f;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            off[nt][e] = 0.f;
            mrun[nt][e] = -INFINITY;
            lrun[nt][e] = 0.f;
            fac[nt][e] = sfac[8 * nt + 2 * c + e];
        }
    }

    // products of the block's keys with q, in units of 2^-24 of q's scale
    constexpr int SUBS = KSUB / A::VS;     // 16-key parts of a block that this warp scores
    auto scores = [&](const uint8_t *st, float (&S)[SUBS][NT][4]) {
#pragma unroll
        for (int sub = 0; sub < SUBS; ++sub) {
            const uint8_t *rec0 = st + (16 * sub + r) * REC, *rec1 = rec0 + 8 * REC;
            // minima: k slots (2c, 2c+1) take group c against the pair (hi, lo)
            // (with two groups, lanes 2 and 3 repeat them against zeros)
            uint32_t am[4] = {0u, 0u, 0u, 0u};
            am[0] = __byte_perm(reinterpret_cast<const uint32_t *>(rec0 + R::CODES)[c % NG], 0u, 0x3232);
            am[1] = __byte_perm(reinterpret_cast<const uint32_t *>(rec1 + R::CODES)[c % NG], 0u, 0x3232);
            if (NG == 8) {
                am[2] = __byte_perm(reinterpret_cast<const uint32_t *>(rec0 + R::CODES)[c + 4], 0u, 0x3232);
                am[3] = __byte_perm(reinterpret_cast<const uint32_t *>(rec1 + R::CODES)[c + 4], 0u, 0x3232);
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                float t[4];
                const uint2 bm = qm[nt * 32 + lane];
                mma16816_first(t, am[0], am[1], am[2], am[3], bm.x, bm.y);
#pragma unroll
                for (int e = 0; e < 4; ++e) S[sub][nt][e] = t[e] * 0.000244140625f;
            }
            constexpr int GL = NG < 4 ? NG : 4;      // groups per load
#pragma unroll
            for (int gl = 0; gl < NG; gl += GL) {
                uint32_t w0[GL], w1[GL], s0[GL], s1[GL];
                load_words<GL>(rec0 + c * 4 * NG + 4 * gl, w0);
                load_words<GL>(rec1 + c * 4 * NG + 4 * gl, w1);
                load_words<GL>(rec0 + R::CODES + 4 * gl, s0);
                load_words<GL>(rec1 + R::CODES + 4 * gl, s1);
#pragma unroll
                for (int g = 0; g < GL; ++g) {
                    const float f0 = __low2float(*reinterpret_cast<const __half2 *>(&s0[g]));
                    const float f1 = __low2float(*reinterpret_cast<const __half2 *>(&s1[g]));
                    const uint32_t h0 = w0[g] >> 8, h1 = w1[g] >> 8;
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        const uint4 bq = qf[(nt * NG + gl + g) * 32 + lane];
                        float t[4];
                        mma16816_first(t, w0[g] & kNib0, w1[g] & kNib0, w0[g] & kNib1, w1[g] & kNib1, bq.x, bq.y);
                        mma16816(t, h0 & kNib0, h1 & kNib0, h0 & kNib1, h1 & kNib1, bq.z, bq.w);
                        S[sub][nt][0] = fmaf(f0, t[0], S[sub][nt][0]);
                        S[sub][nt][1] = fmaf(f0, t[1], S[sub][nt][1]);
                        S[sub][nt][2] = fmaf(f1, t[2], S[sub][nt][2]);
                        S[sub][nt][3] = fmaf(f1, t[3], S[sub][nt][3]);
                    }
                }
            }
        }
    };
    // every key of the block is in the cache and seen by every row
    auto is_full = [&](int b) {
        return pg[b & 3] == all_parts && first + b * STEP + A::BLOCK <= min(k1, see_first);
    };
    uint32_t P[SUBS][NT][2];   // this warp's weights of the last block, as fragments of the second operand
    // The block's maxima, before scaling: columns 2c, 2c+1 of each tile; keys r, r+8 of each
    // part of block b.  Warps that share a slice leave theirs for one another.
    float *smax = reinterpret_cast<float *>(swap + kAttnWarps * NT * 256);
    int *sok = reinterpret_cast<int *>(smax + kAttnWarps * A::ROWS);
    uint2 *sp = reinterpret_cast<uint2 *>(swap);
    auto maxima = [&](int b, float (&S)[SUBS][NT][4], float (&bm)[NT][2]) {
        if (!is_full(b)) {
            const int j0 = first + b * STEP;
            const uint32_t have = pg[b & 3];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int row = min(row0 + 8 * nt + 2 * c + e, rows - 1);
                    const int stop = min(k1, len - m + row / G + 1) - j0;
#pragma unroll
                    for (int x = 0; x < 2 * SUBS; ++x) {
                        const int kk = 8 * x + r + (A::VS > 1 ? 16 * dh : 0);
                        if (kk >= stop || !((have >> (kk >> 4)) & 1u)) S[x >> 1][nt][2 * (x & 1) + e] = -INFINITY;
                    }
                }
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float x = fmaxf(S[0][nt][e], S[0][nt][2 + e]);
                if (SUBS > 1) x = fmaxf(x, fmaxf(S[SUBS - 1][nt][e], S[SUBS - 1][nt][2 + e]));
                x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
                x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
                bm[nt][e] = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
            }
            if (A::VS > 1 && r == 0)
                reinterpret_cast<float2 *>(smax + warp * A::ROWS + 8 * nt)[c] = make_float2(bm[nt][0], bm[nt][1]);
        }
    };
    volatile float held[LONG ? NT : 1][2 * NGV][4], held_at[LONG ? NT : 1][2];     // see stow(); local memory
    bool stowed = false;
    float lift = 13.f - kLeastK;
    uint32_t top_scale = kTopScale + kLeastK * kHalfExp;
    uint32_t fresh = 0u;         // not 0: what a change of lift asks of the block's shared weights
    // The warps of a slice at one point (they take the same steps); false where one of them has
    // given up on a copy.
    auto meet = [&]() { asm volatile("bar.sync 1, %0;" ::"n"(kAttnThreads) : "memory"); };
    auto agree = [&](bool ok) {
        if (A::VS > 1) {
            if (lane == 0) sok[warp] = ok;
            meet();
            ok = sok[0] && sok[1] && sok[2] && sok[3];
        }
        return ok;
    };
    // Softmax step.  The reference moves only when a score passes it by 2 (powers of two), so
    // p < 4 before the lift.
    auto weigh = [&](float (&S)[SUBS][NT][4], float (&bm)[NT][2]) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            bool move[2];
            if (A::VS > 1) {
#pragma unroll
                for (int w = 1; w < A::VS; ++w) {
                    const float2 x = reinterpret_cast<const float2 *>(smax + (warp ^ w) * A::ROWS + 8 * nt)[c];
                    bm[nt][0] = fmaxf(bm[nt][0], x.x);
                    bm[nt][1] = fmaxf(bm[nt][1], x.y);
                }
            }
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                bm[nt][e] *= fac[nt][e];
                move[e] = bm[nt][e] > mrun[nt][e] + 2.f;
            }
            if (__any_sync(0xffffffffu, move[0] || move[1])) {
                float keep[2];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    keep[e] = move[e] ? exp2_approx(mrun[nt][e] - bm[nt][e]) : 1.f;
                    mrun[nt][e] = move[e] ? bm[nt][e] : mrun[nt][e];
                    lrun[nt][e] *= keep[e];
                }
#pragma unroll
                for (int x = 0; x < 2 * NGV; ++x)
#pragma unroll
                    for (int e = 0; e < 4; ++e) O[nt][x][e] *= keep[e & 1];
#pragma unroll
                for (int e = 0; e < 4; ++e) Om[nt][e] *= keep[e & 1];
                off[nt][0] *= keep[0];
                off[nt][1] *= keep[1];
            }
            float msub[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) msub[e] = mrun[nt][e] == -INFINITY ? 0.f : lift - mrun[nt][e];
#pragma unroll
            for (int sub = 0; sub < SUBS; ++sub) {
                float p[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    p[e] = exp2_approx(fmaf(S[sub][nt][e], fac[nt][e & 1], msub[e & 1]));
                    lrun[nt][e & 1] += p[e];
                }
                P[sub][nt][0] = transpose8x8(pack_half2(p[0], p[1]));
                P[sub][nt][1] = transpose8x8(pack_half2(p[2], p[3]));
                if (A::VS > 1) sp[(warp * NT + nt) * 32 + lane] = make_uint2(P[0][nt][0], P[0][nt][1]);
            }
        }
        if (A::VS > 1) meet();
    };
    // O += V^T P over the block's values: k slots 2c, 2c+1, 2c+8, 2c+9 are the keys of the
    // same number
    auto values = [&](const uint8_t *st) {
#pragma unroll
        for (int sub = 0; sub < KSUB; ++sub) {
            uint32_t Pv[NT][2];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                if (A::VS > 1) {
                    const uint2 x = sp[(sub * NT + nt) * 32 + lane];
                    Pv[nt][0] = x.x; Pv[nt][1] = x.y;
                    if (fresh != 0u) {
                        Pv[nt][0] = mul_half2(Pv[nt][0], fresh);
                        Pv[nt][1] = mul_half2(Pv[nt][1], fresh);
                    }
                } else {
                    Pv[nt][0] = P[sub % SUBS][nt][0]; Pv[nt][1] = P[sub % SUBS][nt][1];
                }
            }
            const uint8_t *v0 = st + (16 * sub + 2 * c) * REC;
            const uint8_t *vk[4] = {v0, v0 + REC, v0 + 8 * REC, v0 + 9 * REC};
            uint32_t pr[4][NGV], mr[4];
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                load_words<NGV>(vk[x] + R::CODES + 4 * NGV * dh, pr[x]);
                mr[x] = reinterpret_cast<const uint32_t *>(vk[x] + R::CODES)[r % NG];   // rows past NG are not read
            }
            // rows 0..7: sums of p times the groups' minima, 8..15: times their scales
            const uint32_t a0 = __byte_perm(mr[0], mr[1], 0x7632), a2 = __byte_perm(mr[2], mr[3], 0x7632);
            const uint32_t a1 = __byte_perm(mr[0], mr[1], 0x5410), a3 = __byte_perm(mr[2], mr[3], 0x5410);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) mma16816(Om[nt], a0, a1, a2, a3, Pv[nt][0], Pv[nt][1]);
#pragma unroll
            for (int p = 0; p < NPV; ++p) {
                uint32_t w[4];
#pragma unroll
                for (int x = 0; x < 4; ++x) w[x] = reinterpret_cast<const uint32_t *>(vk[x])[8 * (NPV * dh + p) + r];
#pragma unroll
                for (int hgrp = 0; hgrp < 2; ++hgrp) {
                    const int g = 2 * p + hgrp;
                    const uint32_t sel = hgrp ? 0x7632 : 0x5410;
                    const uint32_t x1 = __byte_perm(w[0], w[1], sel), x2 = __byte_perm(w[2], w[3], sel);
                    const uint32_t y1 = x1 >> 8, y2 = x2 >> 8;
                    const uint32_t sc1 = __byte_perm(pr[0][g], pr[1][g], 0x5410);
                    const uint32_t sc2 = __byte_perm(pr[2][g], pr[3][g], 0x5410);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        const uint32_t b0 = mul_half2(Pv[nt][0], sc1);
                        const uint32_t b1 = mul_half2(Pv[nt][1], sc2);
                        const uint32_t e0 = mul_rest(Pv[nt][0], sc1, b0);
                        const uint32_t e1 = mul_rest(Pv[nt][1], sc2, b1);
                        mma16816(O[nt][2 * g], x1 & kNib0, x1 & kNib1, x2 & kNib0, x2 & kNib1, b0, b1);
                        mma16816(O[nt][2 * g + 1], y1 & kNib0, y1 & kNib1, y2 & kNib0, y2 & kNib1, b0, b1);
                        mma16816(O[nt][2 * g], x1 & kNib0, x1 & kNib1, x2 & kNib0, x2 & kNib1, e0, e1);
                        mma16816(O[nt][2 * g + 1], y1 & kNib0, y1 & kNib1, y2 & kNib0, y2 & kNib1, e0, e1);
                    }
                }
            }
        }
    };
    // Codes are sums of positive numbers, which the minima take back at the end, and the matrix
    // instructions cut their sums off towards zero: over a long run of keys the error would
    // grow with its length (1152 keys: outputs 0.23% off, as much as their own rounding).  So
    // every 256 keys the mean code, 7.5 times the scales, is moved from the sums to `off`, in
    // fp32 rounded to nearest, together with the minima that nearly cancel it (98 -> 101 us on
    // those keys, 175 -> 179 for the 64 sequences).
    auto center = [&]() {
        const float mean = 7.5f;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int g = 0; g < NGV; ++g) {
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float b = mean * __shfl_sync(0xffffffffu, Om[nt][2 + e], 4 * (NGV * dh + g) + c);
#pragma unroll
                    for (int y = 2 * g; y < 2 * g + 2; ++y) {
                        O[nt][y][e] = fmaf(-0x1p-24f, b, O[nt][y][e]);
                        O[nt][y][2 + e] = fmaf(-0x1p-20f, b, O[nt][y][2 + e]);
                    }
                }
            }
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                off[nt][e] += fmaf(mean, Om[nt][2 + e], Om[nt][e]);
                Om[nt][e] = Om[nt][2 + e] = 0.f;
            }
        }
    };
    constexpr int EVERY = 256 / A::BLOCK;
    // What centring leaves is small where many keys carry a row, but not where one does: its code
    // stays in the sums, and each smaller product that joins it is cut off (one key that weighs
    // 2^21 times as much as each of 12000 others left outputs of 256 elements 1.2 times their
    // bound off).  So every kStowKeys keys of a warp the sums move to fp32 words in local memory
    // and start again from zero.  LONG is for calls whose runs can be that long, which splits
    // are not: without it 64 sequences of up to 16384 keys take 180 us, with it 193.
    auto stow = [&](bool again) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            float f[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const float at = held_at[LONG ? nt : 0][e], now = mrun[nt][e] - lift;
                f[e] = stowed && at != -INFINITY ? exp2_approx(at - now) : 0.f;
                held_at[LONG ? nt : 0][e] = now;
            }
#pragma unroll
            for (int x = 0; x < 2 * NGV; ++x)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    if (stowed) O[nt][x][e] = fmaf(held[LONG ? nt : 0][x][e], f[e & 1], O[nt][x][e]);
                    if (again) {
                        held[LONG ? nt : 0][x][e] = O[nt][x][e];
                        O[nt][x][e] = 0.f;
                    }
                }
        }
        stowed = true;
    };
    constexpr int STOW = kStowKeys / A::BLOCK;
    // Values of a block that some row does not see in full: records no row of this tile sees
    // are taken as zero; so are non-finite pairs, whose group becomes NaN in just the rows
    // that see the key (through a zero weight it would reach the others too).
    auto clean = [&](int b, uint8_t *st) {
        const int at = A::VS > 1 ? 16 * dh + (lane & 15) : lane, j = first + b * STEP + at;
        const bool in = j < k1 && ((pg[b & 3] >> (at >> 4)) & 1u);
        uint32_t *par = reinterpret_cast<uint32_t *>(st + at * REC + R::CODES);
#pragma unroll 1
        for (int g = 0; g < NG && (A::VS == 1 || lane < 16); ++g) {
            const bool bad = in && half_pair_nonfinite(par[g]);
            if (bad)
                for (int y = 0; y < A::ROWS && row0 + y < rows; ++y)
                    if (j < len - m + (row0 + y) / G + 1) atomicOr(snan + y, 1u << g);
            if (bad || !in) par[g] = 0u;
        }
        // the next copy into this buffer is the async proxy's, and comes after these writes
        tc::fence_async_smem();
        __syncwarp();
    };

    // Scales of a block's values (one key a lane, or two) that the lift leaves no room for: it
    // is lowered, and with it the weights of the block and all sums so far.  Warps that share a
    // slice see the same scales and keep the same lift.
    auto fit_scales = [&](const uint8_t *st) {
        __half2 m = __floats2half2_rn(0.f, 0.f);
#pragma unroll
        for (int x = 0; x < A::BLOCK / 32; ++x) {
            uint32_t w[NG];
            load_words<NG>(st + (lane + 32 * x) * REC + R::CODES, w);
#pragma unroll
            for (int g = 0; g < NG; ++g) m = __hmax2(m, *reinterpret_cast<const __half2 *>(&w[g]));
        }
        const uint32_t h = __half_as_ushort(__low2half(m));
        if (__any_sync(0xffffffffu, h > top_scale)) {
            const uint32_t most = min(__reduce_max_sync(0xffffffffu, h), 0x7000u);     // 2^13 and more: k = 13
            const uint32_t k = min((most >> 10) - 14u, 13u);
            const float was = lift;
            lift = 13.f - (float)k;
            top_scale = k == 13u ? 0x7fffu : kTopScale + k * kHalfExp;
            const float f = __int_as_float((127 + (int)(lift - was)) << 23);
            fresh = pack_half2(f, f);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
                for (int x = 0; x < 2 * NGV; ++x)
#pragma unroll
                    for (int e = 0; e < 4; ++e) O[nt][x][e] *= f;
#pragma unroll
                for (int e = 0; e < 4; ++e) Om[nt][e] *= f;
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    off[nt][e] *= f;
                    lrun[nt][e] *= f;
                }
#pragma unroll
                for (int x = 0; x < SUBS; ++x)
#pragma unroll
                    for (int e = 0; e < 2; ++e) P[x][nt][e] = mul_half2(P[x][nt][e], fresh);
            }
        }
    };

    // The scores of block b + 1 come before the values of block b: independent products that
    // hide each other's latency.
    bool ok = true;
    if (blocks > 0) {
        float S[SUBS][NT][4], bm[NT][2];
        ok = __all_sync(0xffffffffu, wait_copy(bar_k, 0));
        if (ok) {
            scores(ring_k, S);
            maxima(0, S, bm);
        }
        if ((ok = agree(ok))) weigh(S, bm);
    }
    int b = 0;
    auto walk = [&](int stop) {
        for (; b < stop && ok; ++b) {
            const bool more = b + 1 < blocks;
            if (more) fetch(b + 2 < blocks ? b + 2 : -1, b + 1);
            uint8_t *sv = ring_v + (b & 1) * A::VALUES;
            ok = __all_sync(0xffffffffu, wait_copy(bar_v + (b & 1), (b >> 1) & 1));
            if (!is_full(b)) {
                if (ok) clean(b, sv);
                if (A::VS > 1) meet();               // each has cleaned its part (alike for all of them)
            }
            if (CAREFUL && ok) fit_scales(sv);
            if (ok && more) ok = __all_sync(0xffffffffu, wait_copy(bar_k + ((b + 1) & 1), ((b + 1) >> 1) & 1));
            float S[SUBS][NT][4], bm[NT][2];
            if (ok) {
                if (more) scores(ring_k + ((b + 1) & 1) * A::KEYS, S);
                if (more && A::VS > 1) maxima(b + 1, S, bm);
                values(sv);
                fresh = 0u;
                if (more && (b & (EVERY - 1)) == EVERY - 1) center();
                if (more && A::VS == 1) maxima(b + 1, S, bm);
                __syncwarp();          // the tiles read here are free for the next fetch
            }
            if (more && (ok = agree(ok))) weigh(S, bm);
            if (!ok) break;
        }
    };
    if (LONG) {
#pragma unroll 1
        while (b < blocks && ok) {
            walk(min(blocks, b + STOW));
            if (b < blocks && ok) stow(true);
        }
    } else {
        walk(blocks);
    }
    if (!ok) {
        // a copy never signalled: report, and let what is in flight land (bounded too)
        if (lane == 0) report(status, GDN_ERR_TIMEOUT);
        for (int x = b; x < blocks && x < b + 3; ++x) wait_copy(bar_k + (x & 1), (x >> 1) & 1);
        for (int x = b; x < blocks && x < b + 2; ++x) wait_copy(bar_v + (x & 1), (x >> 1) & 1);
    }

    center();
    if (LONG && stowed) stow(false);
    bool again = false;
    if (!CAREFUL) {
        float zero = 0.f;                       // or NaN
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int x = 0; x < 2 * NGV; ++x)
#pragma unroll
                for (int e = 0; e < 4; ++e) zero = fmaf(O[nt][x][e], 0.f, zero);
        again = zero != zero;
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) mrun[nt][e] -= lift;      // sums are in units of 2^mrun from here on
    // ---- join the warps: maxima and sums, then outputs through shared memory
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            float l = lrun[nt][e];
            l += __shfl_xor_sync(0xffffffffu, l, 4);
            l += __shfl_xor_sync(0xffffffffu, l, 8);
            l += __shfl_xor_sync(0xffffffffu, l, 16);
            lrun[nt][e] = l;
            if (r == 0) sml[warp * A::ROWS + 8 * nt + 2 * c + e] = make_float2(mrun[nt][e], l);
        }
    // every warp is done with its ring
    if (CAREFUL) __syncthreads();
    else if (__syncthreads_or(again) && __syncthreads_and(ok)) return true;
    float *join = reinterpret_cast<float *>(smem);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        float wgt[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            float mall = -INFINITY;
#pragma unroll
            for (int w = 0; w < kAttnWarps; w += A::VS) mall = fmaxf(mall, sml[w * A::ROWS + 8 * nt + 2 * c + e].x);
            wgt[e] = mrun[nt][e] == -INFINITY ? 0.f : exp2_approx(mrun[nt][e] - mall);
        }
#pragma unroll
        for (int g = 0; g < NGV; ++g) {
            const int gd = NGV * dh + g;
            const float m0 = __shfl_sync(0xffffffffu, off[nt][0], 4 * gd + c);
            const float m1 = __shfl_sync(0xffffffffu, off[nt][1], 4 * gd + c);
            const float up = 16777216.f, up16 = 1048576.f;   // 2^24; 2^20 where u came as u << 4
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const float mm = e ? m1 : m0;
                float4 v;
                v.x = wgt[e] * fmaf(O[nt][2 * g][e], up, mm);
                v.y = wgt[e] * fmaf(O[nt][2 * g][2 + e], up16, mm);
                v.z = wgt[e] * fmaf(O[nt][2 * g + 1][e], up, mm);
                v.w = wgt[e] * fmaf(O[nt][2 * g + 1][2 + e], up16, mm);
                reinterpret_cast<float4 *>(join + (size_t)(slice * A::ROWS + 8 * nt + 2 * c + e) * D)[8 * gd + r] = v;
            }
        }
    }
    __syncthreads();
    for (int i = tid; i < A::ROWS * (D / 4); i += kAttnThreads) {
        const int y = i / (D / 4), d4 = i % (D / 4), row = row0 + y;
        if (row >= rows) continue;
        float mall = -INFINITY, l = 0.f;
#pragma unroll
        for (int w = 0; w < kAttnWarps; w += A::VS) mall = fmaxf(mall, sml[w * A::ROWS + y].x);
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < kAttnWarps; ++w) {
            const float2 ml = sml[w * A::ROWS + y];
            if (ml.x != -INFINITY || ml.y != ml.y) l += ml.y * (ml.x == -INFINITY ? 1.f : exp2_approx(ml.x - mall));
            if (w % A::VS) continue;
            const float4 t = reinterpret_cast<const float4 *>(join + (size_t)(w / A::VS * A::ROWS + y) * D)[d4];
            v.x += t.x; v.y += t.y; v.z += t.z; v.w += t.w;
        }
        if ((snan[y] >> (d4 >> 3)) & 1u) v.x = v.y = v.z = v.w = __int_as_float(0x7fffffff);
        const int64_t t = t0 + row / G;
        const int hq = hkv * G + row % G;
        if (splits > 1) {
            const int64_t at = n * slab + ((t - t0) * Hq + hq) * splits_of(len, split_len) + split;
            reinterpret_cast<float4 *>(part_o + at * D)[d4] = v;
            if (d4 == 0) part_ml[at] = make_float2(mall, l);
        } else {
            const float inv = l == 0.f ? 0.f : 1.f / l;
            uint2 u;
            u.x = pack_bf2(v.x * inv, v.y * inv);
            u.y = pack_bf2(v.z * inv, v.w * inv);
            if (l != l) u.x = u.y = 0x7fff7fffu;
            reinterpret_cast<uint2 *>(o + t * o_tok + (int64_t)hq * D)[d4] = u;
            if (lse && d4 == 0) lse[t * Hq + hq] = l == 0.f ? -INFINITY : (mall + log2f(l)) * 0.6931471805599453f;
        }
    }
    return false;
}
// (a function of its own, so that the first pass is compiled without it)
template <int D, int NT>
__device__ __noinline__ void attention_careful(const AttnParams &a) {
    attention_pass<D, NT, true, true>(a);
}
template <int D, int NT, bool LONG>
__global__ void __launch_bounds__(kAttnThreads, AttnShape<D, NT>::CTAS)
kv_attention_mma_kernel(const __grid_constant__ AttnParams a) {
    if (attention_pass<D, NT, LONG, false>(a)) attention_careful<D, NT>(a);
}

// Joins the splits of a row: one CTA per row, warp w taking splits w, w + 4, ..., with
// weights 2^(m_s - max); then the warps in order.  Rows of one split were written by the
// kernel above.
template <int D>
__global__ void __launch_bounds__(128)
kv_attention_join_kernel(KvView kv, bf16 *__restrict__ o, float *__restrict__ lse,
                         const float *__restrict__ part_o, const float2 *__restrict__ part_ml,
                         int64_t o_tok, int Hq, int tile_rows, int64_t slab, int tc_rows,
                         int room_one, int max_kv_len) {
    __shared__ __align__(16) float sacc[4][D];
    __shared__ float sl[4];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t t = blockIdx.x;
    const int hq = blockIdx.y;
    const int n = kv.cu ? sequence_of(kv.cu, kv.N, (int)t) : (int)t;
    const int t0 = kv.cu ? kv.cu[n] : n, m = kv.cu ? kv.cu[n + 1] - t0 : 1;
    const int len = kv.kv_lens[n];
    const bool ours = len >= 0 && len <= max_kv_len && len <= kv.capacity() && Hq * m < tc_rows;
    const int G = Hq / kv.Hkv, rows = G * m, row = (int)(t - t0) * G + hq % G;
    const int last = min((row / tile_rows + 1) * tile_rows, rows) - 1;
    const int see_last = len - m + last / G + 1;
    const int split_len = ours ? kv_split_len(len, m, G, kv.Hkv, D, room_one) : 0;
    const int splits = ours ? splits_of(see_last, split_len) : 0;
    if (splits <= 1) {
        // a grid that has nothing to join must not end before the kernel whose rows are final
        // already: what comes next in the stream waits for this one only
        grid_dependency_wait();
        return;
    }
    const int64_t at = n * slab + ((t - t0) * Hq + hq) * splits_of(len, split_len);
    const float2 *ml = part_ml + at;
    grid_dependency_wait();
    float mall = -INFINITY;
    for (int s = lane; s < splits; s += 32) mall = fmaxf(mall, ml[s].x);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) mall = fmaxf(mall, __shfl_xor_sync(0xffffffffu, mall, off));
    constexpr int E = D / 32;
    float acc[E] = {}, l = 0.f;
    const float *po = part_o + at * D + E * lane;
    for (int s0 = warp; s0 < splits; s0 += 4 * 32) {
        // lane i holds the weight of split s0 + 4 i; a lane past the end holds zero
        const int mine = s0 + 4 * lane;
        float w = 0.f;
        if (mine < splits) {
            const float2 x = ml[mine];
            w = x.x == -INFINITY ? (x.y == x.y ? 0.f : x.y) : exp2_approx(x.x - mall);
            l = fmaf(w, x.y, l);
        }
        const int cnt = min(32, (splits - s0 + 3) / 4);
#pragma unroll 8
        for (int i = 0; i < cnt; ++i) {
            const float wi = __shfl_sync(0xffffffffu, w, i);
            float v[E];
            if constexpr (E == 2) {
                *reinterpret_cast<float2 *>(v) = *reinterpret_cast<const float2 *>(po + (int64_t)(s0 + 4 * i) * D);
            } else {
#pragma unroll
                for (int e = 0; e < E / 4; ++e)
                    reinterpret_cast<float4 *>(v)[e] =
                        reinterpret_cast<const float4 *>(po + (int64_t)(s0 + 4 * i) * D)[e];
            }
#pragma unroll
            for (int e = 0; e < E; ++e) acc[e] = fmaf(wi, v[e], acc[e]);
        }
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) l += __shfl_xor_sync(0xffffffffu, l, off);
    if (lane == 0) sl[warp] = l;
#pragma unroll
    for (int e = 0; e < E; ++e) sacc[warp][E * lane + e] = acc[e];
    __syncthreads();
    l = sl[0] + sl[1] + sl[2] + sl[3];
    const float inv = l == 0.f ? 0.f : 1.f / l;
    for (int d = 2 * tid; d < D; d += 256) {
        const float a = sacc[0][d] + sacc[1][d] + sacc[2][d] + sacc[3][d];
        const float b = sacc[0][d + 1] + sacc[1][d + 1] + sacc[2][d + 1] + sacc[3][d + 1];
        *reinterpret_cast<uint32_t *>(o + t * o_tok + (int64_t)hq * D + d) = pack_bf2(a * inv, b * inv);
    }
    if (lse && tid == 0) lse[t * Hq + hq] = l == 0.f ? -INFINITY : (mall + log2f(l)) * 0.6931471805599453f;
}

}  // namespace gdn

namespace gdn_host {

namespace {

template <typename T, int D>
gdn_status_t simt_launch(const KvArgs &a, cudaStream_t st) {
    if (a.T > 0x7fffffff || a.Hq > 65535) return GDN_ERR_SHAPE;
    gdn::kv_attention_simt_kernel<T, D>
        <<<dim3((unsigned)a.T, a.Hq), gdn::kKvSimtThreads, 0, st>>>(
            a.kv, (const T *)a.q, (T *)a.q_out, a.lse, a.q_tok, a.o_tok, a.Hq, a.max_kv_len,
            a.scale, a.status);
    return cudaGetLastError() == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

}  // namespace

gdn_status_t launch_kv_attention_simt(const KvArgs &a, cudaStream_t st) {
    switch (a.D) {
    case 64: return a.in_f32 ? simt_launch<float, 64>(a, st) : simt_launch<gdn::bf16, 64>(a, st);
    case 128: return a.in_f32 ? simt_launch<float, 128>(a, st) : simt_launch<gdn::bf16, 128>(a, st);
    case 256: return a.in_f32 ? simt_launch<float, 256>(a, st) : simt_launch<gdn::bf16, 256>(a, st);
    }
    return GDN_ERR_UNSUPPORTED;
}

namespace {

// Query heads times new tokens from which a sequence takes the tcgen05 kernel: 20 of its
// CTAs (256 rows each).  Below that too few SMs would be at work on it (8192 keys; this kernel
// against that one, us, at 4096 and at 5120: D = 128 over 8 kv-heads 138, 186 and 240, 187;
// over 2 138, 185 and 238, 185; D = 64 over 2 125, 133 and 149, 133).
constexpr int kTcMinRows = 20 * 256;

// Tiles of eight rows per CTA: as few CTAs as can take every row of a kv-head, alike.
int attn_nt(int64_t rows, int D) {
    const int64_t most = 8 * gdn::attn_max_nt(D), tiles = std::max<int64_t>(1, (rows + most - 1) / most);
    return (int)std::max<int64_t>(1, (rows + 8 * tiles - 1) / (8 * tiles));
}

// The most splits that a context of at most max_len keys with m new rows can have: by the
// least length of a split, and by what has room.  It does not grow with m.
int attn_max_splits(int max_len, int m, int G, int Hkv, int D) {
    const int s = gdn::kv_split_base(max_len, D == 256), most = max_len <= 512 ? 1 : max_len <= 2048 ? 4 : 8;
    return std::min(std::max(most, max_len / s + (max_len % s != 0)),
                    gdn::kv_split_room(std::max(m, 1), G, Hkv, D, gdn::split_ctas(9, D)));
}

// The most keys in one piece for a sequence of m new rows.
int attn_longest(int max_len, int m, int G, int Hkv, int D) {
    const int room = gdn::kv_split_room(m, G, Hkv, D, gdn::split_ctas(G * m, D));
    if (room <= 1) return max_len;
    return std::max(gdn::kv_split_base(max_len, D == 256 && G * m > 8), (max_len + room - 1) / room + 63);
}

// Partial results of one sequence, in rows: Hq m rows of S(m) splits.  S(m) is at most the
// CTAs at once (456) over Hkv times the tiles of at most 32 of the G m rows, so Hq m S(m) <=
// 32 * 456 where anything is split.
int64_t attn_slab(int Hq, int Hkv, int64_t T, int N, int max_q_len, int max_len, int D) {
    const int G = Hq / Hkv, one = attn_max_splits(max_len, 1, G, Hkv, D);
    if (one <= 1) return 0;
    if (N == 1) {
        const int s = attn_max_splits(max_len, (int)std::min<int64_t>(T, gdn::kSplitMaxRows), G, Hkv, D);
        return s > 1 ? T * Hq * s : 0;
    }
    const int64_t m = std::min(max_q_len, gdn::kSplitMaxRows);
    return std::min<int64_t>(Hq * m * one, 32 * gdn::kSplitMaxCtas);
}

size_t part_ml_bytes(int64_t rows) { return ((size_t)rows * 8 + 255) / 256 * 256; }

template <int D, int NT>
gdn_status_t mma_launch(const KvArgs &a, int row_tiles, int splits, int tc_rows, int longest, cudaStream_t st) {
    using A = gdn::AttnShape<D, NT>;
    const bool is_long = longest > gdn::kStowKeys * A::SLICES;      // keys of one warp
    auto kern = is_long ? gdn::kv_attention_mma_kernel<D, NT, true> : gdn::kv_attention_mma_kernel<D, NT, false>;
    static std::atomic<uint64_t> readies[2];   // one bit per device (beyond 63: set every time)
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return GDN_ERR_CUDA;
    std::atomic<uint64_t> &ready = readies[is_long];
    if (dev > 63 || !((ready.load() >> dev) & 1u)) {
        if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, A::SMEM) != cudaSuccess)
            return GDN_ERR_CUDA;
        if (dev <= 63) ready.fetch_or(1ull << dev);
    }
    const int64_t slab = attn_slab(a.Hq, a.kv.Hkv, a.T, a.kv.N, a.max_q_len, a.max_kv_len, D);
    const int room = gdn::kv_split_room(1, a.Hq / a.kv.Hkv, a.kv.Hkv, D, gdn::split_ctas(a.Hq / a.kv.Hkv, D));
    float2 *ml = (float2 *)a.ws;
    float *po = slab ? (float *)((uint8_t *)a.ws + part_ml_bytes(slab * a.kv.N)) : nullptr;
    const gdn::AttnParams p = {a.kv, (const gdn::bf16 *)a.q, (gdn::bf16 *)a.q_out, a.lse, po, ml, a.q_tok, a.o_tok,
                               slab, a.Hq, row_tiles, tc_rows, room, a.max_kv_len, a.scale, a.status};
    kern<<<dim3((unsigned)((int64_t)splits * row_tiles), a.kv.Hkv, a.kv.N), gdn::kAttnThreads, A::SMEM, st>>>(p);
    if (cudaGetLastError() != cudaSuccess) return GDN_ERR_CUDA;
    if (splits > 1 &&
        launch_dependent(gdn::kv_attention_join_kernel<D>, dim3((unsigned)a.T, a.Hq), dim3(128), 0, st, a.kv,
                         (gdn::bf16 *)a.q_out, a.lse, po, ml, a.o_tok, a.Hq, 8 * NT, slab, tc_rows,
                         room, a.max_kv_len) != cudaSuccess)
        return GDN_ERR_CUDA;
    return GDN_OK;
}

}  // namespace

size_t kv_attention_workspace(int32_t D, int32_t Hq, int32_t Hkv, int64_t T, int32_t N,
                              int32_t max_q_len, int32_t max_kv_len, int in_f32, uint32_t flags) {
    if (in_f32 || (flags & GDN_PREFILL_SIMT) || T <= 0 || Hq <= 0 || Hkv <= 0 || Hq % Hkv) return 0;
    const int64_t slab = attn_slab(Hq, Hkv, T, N, max_q_len, max_kv_len, D);
    return slab ? part_ml_bytes(slab * N) + (size_t)slab * N * D * sizeof(float) : 0;
}

gdn_status_t launch_kv_attention(const KvArgs &a, cudaStream_t st) {
    if (a.in_f32 || (a.flags & GDN_PREFILL_SIMT)) return launch_kv_attention_simt(a, st);
    // sequences of many rows go to the tcgen05 kernel, the others to this one
    const bool tc = a.kv.cu && kv_attention_tc_supported(a.D);
    const int tc_rows = tc ? kTcMinRows : 0x7fffffff;
    int64_t m_most = a.max_q_len;
    if (tc && a.Hq * m_most >= tc_rows) {
        const gdn_status_t s = launch_kv_attention_tc(a, tc_rows, st);
        if (s != GDN_OK || (int64_t)a.Hq * a.min_q_len >= tc_rows) return s;
        m_most = (tc_rows - 1) / a.Hq;
    }
    const int64_t rows = (int64_t)(a.Hq / a.kv.Hkv) * m_most;
    const int nt = attn_nt(rows, a.D);
    const int64_t tiles = (rows + 8 * nt - 1) / (8 * nt);
    const int splits = attn_max_splits(a.max_kv_len, a.min_q_len, a.Hq / a.kv.Hkv, a.kv.Hkv, a.D);
    if (tiles * splits > 0x7fffffff || a.kv.N > 65535) return GDN_ERR_SHAPE;
    // the longest run of keys: of the most new rows that are there for this kernel, or the least
    // (room falls as m grows, but for the step in split_ctas)
    const int G = a.Hq / a.kv.Hkv;
    int m_there = a.min_q_len;
    for (int n = 0; a.kv.cu && n < a.kv.N; ++n) {
        const int m = a.cu_host[n + 1] - a.cu_host[n];
        if ((int64_t)a.Hq * m < tc_rows) m_there = std::max(m_there, m);
    }
    const int longest = std::max(attn_longest(a.max_kv_len, a.min_q_len, G, a.kv.Hkv, a.D),
                                 attn_longest(a.max_kv_len, m_there, G, a.kv.Hkv, a.D));
    switch (a.D * 10 + nt) {
    case 641: return mma_launch<64, 1>(a, (int)tiles, splits, tc_rows, longest, st);
    case 642: return mma_launch<64, 2>(a, (int)tiles, splits, tc_rows, longest, st);
    case 643: return mma_launch<64, 3>(a, (int)tiles, splits, tc_rows, longest, st);
    case 644: return mma_launch<64, 4>(a, (int)tiles, splits, tc_rows, longest, st);
    case 1281: return mma_launch<128, 1>(a, (int)tiles, splits, tc_rows, longest, st);
    case 1282: return mma_launch<128, 2>(a, (int)tiles, splits, tc_rows, longest, st);
    case 2561: return mma_launch<256, 1>(a, (int)tiles, splits, tc_rows, longest, st);
    case 2562: return mma_launch<256, 2>(a, (int)tiles, splits, tc_rows, longest, st);
    case 2563: return mma_launch<256, 3>(a, (int)tiles, splits, tc_rows, longest, st);
    }
    return GDN_ERR_UNSUPPORTED;
}

}  // namespace gdn_host
