// kvcache.cu -- writing a paged 4-bit key/value cache, with the position rotation of q
// and k on the way, and reading rows of it back as values.
//
// Token i of the m new tokens of a sequence with kv_len tokens (the new ones included) has
// position kv_len - m + i, which is slot position mod page of page
// block_table[n][position div page].  Rotation of the first `rot` elements by the angle
// tables' row `position` (half = rot / 2; pairs (e, e + half), or (2e, 2e + 1) interleaved):
//     a' = a cos_e - b sin_e,   b' = b cos_e + a sin_e
// in fp32, each product and sum rounded by itself (no fused multiply-add), so that the
// codes are a fixed function of the inputs.
//
// A warp takes one token and walks its rows, 32 / (D / 8) at a time: a lane has eight adjacent
// elements (a 16-byte load of bf16), four lanes share a group.  The token's place and its
// angles are found once for all its heads, and rows of q skip the quantisation; with one row
// per lane group and everything per row the kernel was bound by instruction issue (362 a
// warp, 83 us for 8314 tokens of 32 + 2 x 8 heads of 128; 47 us now, 185 MB at 58% of the HBM
// rate, issue slots 59% taken).  Reading the same rows back as fp32 moves 79 MB in 22 us, 53%
// of the HBM rate, bound by the latency of its loads.
#include <algorithm>

#include "kv_format.cuh"

namespace gdn {

constexpr int kKvThreads = 256;

__device__ __forceinline__ void load8(const bf16 *p, float (&f)[8]) {
    unpack8(*reinterpret_cast<const uint4 *>(p), f);
}
__device__ __forceinline__ void load8(const float *p, float (&f)[8]) {
    const float4 a = reinterpret_cast<const float4 *>(p)[0], b = reinterpret_cast<const float4 *>(p)[1];
    f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
    f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
}
__device__ __forceinline__ void store8(bf16 *p, const float (&f)[8]) {
    *reinterpret_cast<uint4 *>(p) = pack8(f);
}
__device__ __forceinline__ void store8(float *p, const float (&f)[8]) {
    reinterpret_cast<float4 *>(p)[0] = make_float4(f[0], f[1], f[2], f[3]);
    reinterpret_cast<float4 *>(p)[1] = make_float4(f[4], f[5], f[6], f[7]);
}

// A token's sequence, position and page; false (reported) when it has no place.
struct KvPlace {
    int n, pos, page, slot;
};
__device__ __forceinline__ bool place_of(const KvView &kv, int t, int tab_rows, KvPlace &pl) {
    pl.n = kv.cu ? sequence_of(kv.cu, kv.N, t) : t;
    pl.pos = kv.kv_lens[pl.n] - (kv.cu ? kv.cu[pl.n + 1] - t : 1);
    // the position must be inside the block table, and inside the angle tables
    if (pl.pos < 0 || pl.pos >= kv.capacity() || pl.pos >= tab_rows) return false;
    pl.page = kv.table[(int64_t)pl.n * kv.table_width + (pl.pos >> kv.page_log2)];
    pl.slot = pl.pos & ((1 << kv.page_log2) - 1);
    return pl.page >= 0 && pl.page < kv.pages;
}

// The angles of a lane's eight elements d0 .. (the row of the tables for the position), the
// place of their partners, and whether they turn at all.  Half-split: cos and (signed) sin of
// the elements; interleaved: of four pairs.
struct KvAngles {
    float c[8], s[8];
    int mate;
    bool turn;
};
template <bool INTER>
__device__ __forceinline__ KvAngles load_angles(const float *cosr, const float *sinr, int d0, int rot) {
    KvAngles a;
    a.turn = d0 < rot;
    a.mate = d0;
#pragma unroll
    for (int e = 0; e < 8; ++e) a.c[e] = a.s[e] = 0.f;
    if (!a.turn) return a;
    if (INTER) {
        const float4 c = *reinterpret_cast<const float4 *>(cosr + d0 / 2);
        const float4 s = *reinterpret_cast<const float4 *>(sinr + d0 / 2);
        a.c[0] = c.x; a.c[1] = c.y; a.c[2] = c.z; a.c[3] = c.w;
        a.s[0] = s.x; a.s[1] = s.y; a.s[2] = s.z; a.s[3] = s.w;
    } else {
        const bool first = d0 < rot / 2;
        a.mate = first ? d0 + rot / 2 : d0 - rot / 2;
        load8(cosr + min(d0, a.mate), a.c);
        load8(sinr + min(d0, a.mate), a.s);
        // the second of a pair adds where the first subtracts: a sign on the sine, exact
#pragma unroll
        for (int e = 0; e < 8; ++e) a.s[e] = first ? -a.s[e] : a.s[e];
    }
    return a;
}
// Elements d0 .. d0+7 of a row, rotated (no branches, so that loads of several rows overlap).
template <bool INTER, typename T>
__device__ __forceinline__ void load_rotated(const T *row, int d0, const KvAngles &a, float (&x)[8]) {
    load8(row + d0, x);
    if (INTER) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float p = x[2 * e], q = x[2 * e + 1];
            const float u = __fsub_rn(__fmul_rn(p, a.c[e]), __fmul_rn(q, a.s[e]));
            const float w = __fadd_rn(__fmul_rn(q, a.c[e]), __fmul_rn(p, a.s[e]));
            x[2 * e] = a.turn ? u : p;
            x[2 * e + 1] = a.turn ? w : q;
        }
    } else {
        float y[8];
        load8(row + a.mate, y);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float u = __fadd_rn(__fmul_rn(x[e], a.c[e]), __fmul_rn(y[e], a.s[e]));
            x[e] = a.turn ? u : x[e];
        }
    }
}

// Blocks of kKvThreads / 32 tokens, one a warp; gridDim.y parts share a token's rows.  Rows:
// the keys and values of Hkv heads, then Hq rows of q (0 when q is not rotated here).
template <typename T, int D, bool INTER>
__global__ void __launch_bounds__(kKvThreads, 4)
kv_append_kernel(KvView kv, const T *__restrict__ k, const T *__restrict__ v,
                 const T *__restrict__ q, T *__restrict__ q_out, int64_t k_tok, int64_t v_tok,
                 int64_t q_tok, int64_t qo_tok, int Hq, int T_new,
                 const float *__restrict__ cos_tab, const float *__restrict__ sin_tab,
                 int tab_rows, int rot, int32_t *status) {
    using R = KvRec<D>;
    constexpr int LANES = D / 8, RPW = 32 / LANES;      // lanes per row, rows at a time
    const int t = blockIdx.x * (kKvThreads / 32) + (threadIdx.x >> 5);
    if (t >= T_new) return;
    const int lane = threadIdx.x & 31, l = lane % LANES, sub = lane / LANES, d0 = 8 * l;
    KvPlace pl;
    if (!place_of(kv, t, cos_tab ? tab_rows : 0x7fffffff, pl)) {
        if (lane == 0) report(status, GDN_ERR_INDEX);
        return;
    }
    if (!cos_tab) rot = 0;
    const KvAngles ang = load_angles<INTER>(cos_tab + (int64_t)pl.pos * (rot >> 1),
                                            sin_tab + (int64_t)pl.pos * (rot >> 1), d0, rot);
    const int g = l >> 2, c = l & 3;
    const int kv_rows = 2 * kv.Hkv, kv_its = (kv_rows + RPW - 1) / RPW, q_its = (Hq + RPW - 1) / RPW;
    int it = blockIdx.y;
#pragma unroll 1
    for (; it < kv_its; it += gridDim.y) {
        const int r = it * RPW + sub;
        const bool live = r < kv_rows, is_k = r < kv.Hkv;
        const int head = is_k ? r : r - kv.Hkv;
        float x[8] = {};
        if (live) {
            if (is_k) load_rotated<INTER>(k + (int64_t)t * k_tok + head * D, d0, ang, x);
            else load8(v + (int64_t)t * v_tok + head * D + d0, x);
        }
        // minimum, maximum (clamped to the fp16 range) and NaN flag of the group: this lane's
        // eight elements, then its four lanes (every lane takes part in the shuffles).  A NaN
        // counts as -65504 in what is stored beside the flag.
        float mn = INFINITY, mx = -INFINITY;
        bool nan = false;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const bool no = x[e] != x[e];
            nan |= no;
            x[e] = no ? -65504.f : x[e];
            mn = fminf(mn, x[e]);
            mx = fmaxf(mx, x[e]);
        }
#pragma unroll
        for (int off = 1; off < 4; off <<= 1) {
            mn = fminf(mn, __shfl_xor_sync(0xffffffffu, mn, off));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
        }
        const uint32_t bad = __ballot_sync(0xffffffffu, nan) >> (lane & ~3) & 15u;
        if (!live) continue;
        mn = fminf(fmaxf(mn, -65504.f), 65504.f);
        mx = fminf(fmaxf(mx, -65504.f), 65504.f);
        const __half mh = __float2half_rn(mn);
        const float mf = __half2float(mh);
        const __half sh = __float2half_rn(__fmul_rn(__fsub_rn(mx, mf), 1.0f / 15.0f));
        const float sf = __half2float(sh);
        const float inv = sf > 0.f ? __frcp_rn(sf) : 0.f;
        // Round to the nearest integer, ties to even, by adding 1.5 * 2^23: a code ends up in
        // the low bits.  Values past the clamped ends (infinities too) land on 0 or 15.
        uint32_t code = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float u = fminf(fmaxf(__fmul_rn(__fsub_rn(x[e], mf), inv), 0.f), 15.f);
            code |= (__float_as_uint(__fadd_rn(u, 12582912.f)) & 15u) << (4 * e);
        }
        uint8_t *rec = kv.block(pl.page, is_k ? 0 : 1, head, R::BYTES) + pl.slot * R::BYTES;
        if (is_k) {
            reinterpret_cast<uint32_t *>(rec)[c * R::NG + g] = code;
        } else {
            uint16_t *w = reinterpret_cast<uint16_t *>(rec) + 2 * (8 * (g >> 1) + 2 * c) + (g & 1);
            w[0] = (uint16_t)code;
            w[2] = (uint16_t)(code >> 16);
        }
        if (c == 0) {
            __half2 sm = __halves2half2(sh, mh);
            if (bad) sm = __halves2half2(__ushort_as_half(0), __ushort_as_half(0x7fff));
            reinterpret_cast<__half2 *>(rec + R::CODES)[g] = sm;
        }
    }
    q += (int64_t)t * q_tok;
    q_out += (int64_t)t * qo_tok;
#pragma unroll 4
    for (it -= kv_its; it < q_its; it += gridDim.y) {
        const int h = it * RPW + sub;
        float x[8];
        load_rotated<INTER>(q + min(h, Hq - 1) * D, d0, ang, x);
        if (h < Hq) store8(q_out + h * D + d0, x);
    }
}

// The same tokens' rows as values: k_out, v_out [T, Hkv, D].
template <typename T, int D>
__global__ void __launch_bounds__(kKvThreads)
kv_read_kernel(KvView kv, T *__restrict__ k_out, T *__restrict__ v_out, int64_t k_tok,
               int64_t v_tok, int T_new, int32_t *status) {
    using R = KvRec<D>;
    constexpr int LANES = D / 8, RPW = 32 / LANES;
    const int t = blockIdx.x * (kKvThreads / 32) + (threadIdx.x >> 5);
    if (t >= T_new) return;
    const int lane = threadIdx.x & 31, l = lane % LANES, sub = lane / LANES;
    KvPlace pl;
    if (!place_of(kv, t, 0x7fffffff, pl)) {
        if (lane == 0) report(status, GDN_ERR_INDEX);
        return;
    }
    const int g = l >> 2, c = l & 3;
#pragma unroll 4
    for (int r = blockIdx.y * RPW + sub; r < 2 * kv.Hkv; r += gridDim.y * RPW) {
        const bool is_k = r < kv.Hkv;
        const int head = is_k ? r : r - kv.Hkv;
        const uint8_t *rec = kv.block(pl.page, is_k ? 0 : 1, head, R::BYTES) + pl.slot * R::BYTES;
        uint32_t code;
        if (is_k) {
            code = reinterpret_cast<const uint32_t *>(rec)[c * R::NG + g];
        } else {
            const uint16_t *w = reinterpret_cast<const uint16_t *>(rec) + 2 * (8 * (g >> 1) + 2 * c) + (g & 1);
            code = (uint32_t)w[0] | (uint32_t)w[2] << 16;
        }
        const float2 sm = __half22float2(reinterpret_cast<const __half2 *>(rec + R::CODES)[g]);
        float x[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = fmaf(sm.x, (float)((code >> (4 * e)) & 15u), sm.y);
        store8((is_k ? k_out + (int64_t)t * k_tok : v_out + (int64_t)t * v_tok) + head * D + 8 * l, x);
    }
}

}  // namespace gdn

namespace gdn_host {

namespace {

// Parts a token's rows are cut into, so that a few tokens fill the device and many leave no
// long last round: enough for 16000 warps in all (three rounds of what fits), at most one part
// per row step.  Every part looks the place and the angles up again (8314 tokens written and
// read back, from HBM: one part 73.5 us, two 69.2, four 69, six 82).
int kv_parts(int64_t tokens, int steps) {
    const int64_t want = (16000 + tokens - 1) / tokens;
    return (int)std::max<int64_t>(1, std::min<int64_t>(std::min<int64_t>(want, steps), 65535));
}

template <typename T, int D>
gdn_status_t append_launch(const KvArgs &a, cudaStream_t st) {
    constexpr int rpw = 256 / D;
    const int steps = (2 * a.kv.Hkv + rpw - 1) / rpw + (a.Hq + rpw - 1) / rpw;
    const dim3 grid((unsigned)((a.T * 32 + gdn::kKvThreads - 1) / gdn::kKvThreads), kv_parts(a.T, steps));
    auto kern = a.interleaved ? gdn::kv_append_kernel<T, D, true> : gdn::kv_append_kernel<T, D, false>;
    kern<<<grid, gdn::kKvThreads, 0, st>>>(
        a.kv, (const T *)a.k, (const T *)a.v, (const T *)a.q, (T *)a.q_out, a.k_tok, a.v_tok,
        a.q_tok, a.o_tok, a.Hq, (int)a.T, a.cos_tab, a.sin_tab, a.tab_rows, a.rot, a.status);
    return cudaGetLastError() == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

template <typename T, int D>
gdn_status_t read_launch(const KvArgs &a, cudaStream_t st) {
    constexpr int rpw = 256 / D;
    const dim3 grid((unsigned)((a.T * 32 + gdn::kKvThreads - 1) / gdn::kKvThreads),
                    kv_parts(a.T, (2 * a.kv.Hkv + rpw - 1) / rpw));
    gdn::kv_read_kernel<T, D><<<grid, gdn::kKvThreads, 0, st>>>(
        a.kv, (T *)const_cast<void *>(a.k), (T *)const_cast<void *>(a.v), a.k_tok, a.v_tok, (int)a.T,
        a.status);
    return cudaGetLastError() == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

}  // namespace

#define GDN_KV_DISPATCH(fn, a, st)                                                     \
    switch ((a).D) {                                                                   \
    case 64: return (a).in_f32 ? fn<float, 64>(a, st) : fn<gdn::bf16, 64>(a, st);      \
    case 128: return (a).in_f32 ? fn<float, 128>(a, st) : fn<gdn::bf16, 128>(a, st);   \
    case 256: return (a).in_f32 ? fn<float, 256>(a, st) : fn<gdn::bf16, 256>(a, st);   \
    }                                                                                  \
    return GDN_ERR_UNSUPPORTED

gdn_status_t launch_kv_append(const KvArgs &a, cudaStream_t st) {
    GDN_KV_DISPATCH(append_launch, a, st);
}
gdn_status_t launch_kv_read(const KvArgs &a, cudaStream_t st) {
    GDN_KV_DISPATCH(read_launch, a, st);
}

}  // namespace gdn_host
