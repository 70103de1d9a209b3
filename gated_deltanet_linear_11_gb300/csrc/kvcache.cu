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
// Both kernels are bound by memory traffic: a lane takes eight adjacent elements (a
// 16-byte load of bf16), a row takes D / 8 adjacent lanes, four of which share a group.
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

// Elements d0 .. d0+7 of a row, rotated.
template <typename T>
__device__ __forceinline__ void load_rotated(const T *row, int d0, const float *cosr,
                                             const float *sinr, int rot, int interleaved,
                                             float (&x)[8]) {
    load8(row + d0, x);
    if (d0 >= rot) return;
    const int half = rot >> 1;
    if (interleaved) {
        const float4 c = *reinterpret_cast<const float4 *>(cosr + d0 / 2);
        const float4 s = *reinterpret_cast<const float4 *>(sinr + d0 / 2);
        const float cc[4] = {c.x, c.y, c.z, c.w}, ss[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float a = x[2 * e], b = x[2 * e + 1];
            x[2 * e] = __fsub_rn(__fmul_rn(a, cc[e]), __fmul_rn(b, ss[e]));
            x[2 * e + 1] = __fadd_rn(__fmul_rn(b, cc[e]), __fmul_rn(a, ss[e]));
        }
    } else {
        const bool first = d0 < half;
        float y[8], c[8], s[8];
        load8(row + (first ? d0 + half : d0 - half), y);
        load8(cosr + (first ? d0 : d0 - half), c);
        load8(sinr + (first ? d0 : d0 - half), s);
#pragma unroll
        for (int e = 0; e < 8; ++e)
            x[e] = first ? __fsub_rn(__fmul_rn(x[e], c[e]), __fmul_rn(y[e], s[e]))
                         : __fadd_rn(__fmul_rn(x[e], c[e]), __fmul_rn(y[e], s[e]));
    }
}

// One row per D / 8 lanes: rows 0 .. Hkv-1 of a token are its keys, then its values, then
// its queries (Hq of them; 0 when q is not rotated here).
template <typename T, int D>
__global__ void __launch_bounds__(kKvThreads)
kv_append_kernel(KvView kv, const T *__restrict__ k, const T *__restrict__ v,
                 const T *__restrict__ q, T *__restrict__ q_out, int64_t k_tok, int64_t v_tok,
                 int64_t q_tok, int64_t qo_tok, int Hq, int64_t T_new,
                 const float *__restrict__ cos_tab, const float *__restrict__ sin_tab,
                 int tab_rows, int rot, int interleaved, int32_t *status) {
    using R = KvRec<D>;
    constexpr int LANES = D / 8;
    const int64_t row = ((int64_t)blockIdx.x * kKvThreads + threadIdx.x) / LANES;
    const int l = threadIdx.x % LANES, d0 = 8 * l;
    const int per = 2 * kv.Hkv + Hq;
    const bool live = row < T_new * per;
    const int64_t t = live ? row / per : 0;
    const int r = live ? (int)(row - t * per) : 0;
    const int n = kv.cu ? sequence_of(kv.cu, kv.N, (int)t) : (int)t;
    const int pos = kv.kv_lens[n] - (kv.cu ? kv.cu[n + 1] - (int)t : 1);
    const bool is_k = r < kv.Hkv, is_q = r >= 2 * kv.Hkv;
    const int head = is_k ? r : is_q ? r - 2 * kv.Hkv : r - kv.Hkv;
    // the position must be inside the block table, and inside the angle tables
    bool ok = live && pos >= 0 && pos < kv.capacity() && (!cos_tab || pos < tab_rows);
    int page = 0;
    if (ok) {
        page = kv.table[(int64_t)n * kv.table_width + (pos >> kv.page_log2)];
        ok = page >= 0 && page < kv.pages;
    }
    if (live && !ok && l == 0) report(status, GDN_ERR_INDEX);

    float x[8] = {};
    if (ok) {
        const float *cosr = cos_tab + (int64_t)pos * (rot >> 1);
        const float *sinr = sin_tab + (int64_t)pos * (rot >> 1);
        const int rr = cos_tab ? rot : 0;
        if (is_q) {
            load_rotated(q + t * q_tok + (int64_t)head * D, d0, cosr, sinr, rr, interleaved, x);
            store8(q_out + t * qo_tok + (int64_t)head * D + d0, x);
        } else if (is_k) {
            load_rotated(k + t * k_tok + (int64_t)head * D, d0, cosr, sinr, rr, interleaved, x);
        } else {
            load8(v + t * v_tok + (int64_t)head * D + d0, x);
        }
    }
    // minimum, maximum and NaN flag of the group: this lane's eight elements, then the
    // four lanes of the group (every lane of the warp takes part in the shuffles)
    float mn = 65504.f, mx = -65504.f;
    bool nan = false;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        nan |= isnan(x[e]);
        x[e] = fminf(fmaxf(x[e], -65504.f), 65504.f);
        mn = fminf(mn, x[e]);
        mx = fmaxf(mx, x[e]);
    }
    int bad = nan;
#pragma unroll
    for (int off = 1; off < 4; off <<= 1) {
        mn = fminf(mn, __shfl_xor_sync(0xffffffffu, mn, off));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
        bad |= __shfl_xor_sync(0xffffffffu, bad, off);
    }
    if (!ok || is_q) return;
    const __half mh = __float2half_rn(mn);
    const float mf = __half2float(mh);
    const __half sh = __float2half_rn(__fmul_rn(__fsub_rn(mx, mf), 1.0f / 15.0f));
    const float sf = __half2float(sh);
    const float inv = sf > 0.f ? __frcp_rn(sf) : 0.f;
    uint32_t code = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const float u = fminf(fmaxf(rintf(__fmul_rn(__fsub_rn(x[e], mf), inv)), 0.f), 15.f);
        code |= (uint32_t)u << (4 * e);
    }
    const int slot = pos & ((1 << kv.page_log2) - 1);
    uint8_t *rec = kv.block(page, is_k ? 0 : 1, head, R::BYTES) + (int64_t)slot * R::BYTES;
    const int g = l >> 2, c = l & 3;
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

// The same tokens' rows as values: k_out, v_out [T, Hkv, D].
template <typename T, int D>
__global__ void __launch_bounds__(kKvThreads)
kv_read_kernel(KvView kv, T *__restrict__ k_out, T *__restrict__ v_out, int64_t k_tok,
               int64_t v_tok, int64_t T_new, int32_t *status) {
    using R = KvRec<D>;
    constexpr int LANES = D / 8;
    const int64_t row = ((int64_t)blockIdx.x * kKvThreads + threadIdx.x) / LANES;
    const int l = threadIdx.x % LANES;
    const int per = 2 * kv.Hkv;
    if (row >= T_new * per) return;
    const int64_t t = row / per;
    const int r = (int)(row - t * per);
    const int n = kv.cu ? sequence_of(kv.cu, kv.N, (int)t) : (int)t;
    const int pos = kv.kv_lens[n] - (kv.cu ? kv.cu[n + 1] - (int)t : 1);
    const bool is_k = r < kv.Hkv;
    const int head = is_k ? r : r - kv.Hkv;
    int page = -1;
    if (pos >= 0 && pos < kv.capacity())
        page = kv.table[(int64_t)n * kv.table_width + (pos >> kv.page_log2)];
    if (page < 0 || page >= kv.pages) {
        if (l == 0) report(status, GDN_ERR_INDEX);
        return;
    }
    const int slot = pos & ((1 << kv.page_log2) - 1);
    const uint8_t *rec = kv.block(page, is_k ? 0 : 1, head, R::BYTES) + (int64_t)slot * R::BYTES;
    const int g = l >> 2, c = l & 3;
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
    store8((is_k ? k_out + t * k_tok : v_out + t * v_tok) + (int64_t)head * D + 8 * l, x);
}

}  // namespace gdn

namespace gdn_host {

namespace {

template <typename T, int D>
gdn_status_t append_launch(const KvArgs &a, cudaStream_t st) {
    const int64_t rows = a.T * (2 * a.kv.Hkv + a.Hq);
    const int64_t blocks = (rows * (D / 8) + gdn::kKvThreads - 1) / gdn::kKvThreads;
    if (blocks > 0x7fffffff) return GDN_ERR_SHAPE;
    gdn::kv_append_kernel<T, D><<<(unsigned)blocks, gdn::kKvThreads, 0, st>>>(
        a.kv, (const T *)a.k, (const T *)a.v, (const T *)a.q, (T *)a.q_out, a.k_tok, a.v_tok,
        a.q_tok, a.o_tok, a.Hq, a.T, a.cos_tab, a.sin_tab, a.tab_rows, a.rot, a.interleaved,
        a.status);
    return cudaGetLastError() == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

template <typename T, int D>
gdn_status_t read_launch(const KvArgs &a, cudaStream_t st) {
    const int64_t rows = a.T * 2 * a.kv.Hkv;
    const int64_t blocks = (rows * (D / 8) + gdn::kKvThreads - 1) / gdn::kKvThreads;
    if (blocks > 0x7fffffff) return GDN_ERR_SHAPE;
    gdn::kv_read_kernel<T, D><<<(unsigned)blocks, gdn::kKvThreads, 0, st>>>(
        a.kv, (T *)const_cast<void *>(a.k), (T *)const_cast<void *>(a.v), a.k_tok, a.v_tok, a.T,
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
