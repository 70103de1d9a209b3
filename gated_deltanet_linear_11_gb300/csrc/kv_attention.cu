// kv_attention.cu -- attention of new tokens over a paged 4-bit key/value cache.
//
//     o = sum_j p_j v_j / sum_j p_j,   p_j = exp(scale q.k_j),   j <= kv_len - m + i
// for token i of the m new tokens of a sequence with kv_len tokens (the new ones
// included, already in the cache).  A row that sees no key (kv_len < m - i) gives zeros,
// and a log-sum-exp of -inf.
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

size_t kv_attention_workspace(int32_t D, int32_t Hq, int32_t Hkv, int64_t T, int32_t N,
                              int32_t max_q_len, int32_t max_kv_len, int in_f32, uint32_t flags) {
    return 0;
}

gdn_status_t launch_kv_attention(const KvArgs &a, cudaStream_t st) {
    return launch_kv_attention_simt(a, st);
}

}  // namespace gdn_host
