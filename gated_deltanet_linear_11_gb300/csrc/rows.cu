// rows.cu -- operators on the rows between the mixers: 8 bits with a scale for each row, the
// root-mean-square norm with the residual's addition, and the Gated DeltaNet layer's output
// norm.
//
//   quantize:   y = x
//   add norm:   h = x + residual;  y = h (offset + w) / sqrt(mean h^2 + eps)
//   gated norm: y = x w / sqrt(mean_head x^2 + eps) * z / (1 + e^-z)
//   8 bits:     scale = max|y| / 127, code = y / scale to the nearest integer
//
// All three read a row once and write it once, so HBM bounds them.  A row stays in the
// registers of one warp (up to 1024 elements) or of one CTA, 8 consecutive elements at a time
// per thread; sums and maxima go over the row with shuffles and one pass through shared
// memory.  The split of a row depends on its length alone, so a row's results are the same in
// any batch.
#include "rows.cuh"

namespace gdn {

namespace {

constexpr float kTinyScale = 1.17549435e-38f;   // 2^-126: the scale of a row of zeros
constexpr uint32_t kInfBits = 0x7f800000u;

// n <= 8 elements from p on, the rest zero; vec: all 8, 16-byte aligned.
template <typename T>
__device__ __forceinline__ void load8(const T *p, int n, bool vec, float (&f)[8]) {
    if (vec) {
        if constexpr (sizeof(T) == 2) {
            unpack8(*reinterpret_cast<const uint4 *>(p), f);
        } else {
            const float4 a = reinterpret_cast<const float4 *>(p)[0];
            const float4 b = reinterpret_cast<const float4 *>(p)[1];
            f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
            f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
        }
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] = j < n ? to_f32(p[j]) : 0.f;
    }
}

template <typename T>
__device__ __forceinline__ void store8(T *p, int n, bool vec, const float (&f)[8]) {
    if (vec) {
        if constexpr (sizeof(T) == 2) {
            *reinterpret_cast<uint4 *>(p) = pack8(f);
        } else {
            reinterpret_cast<float4 *>(p)[0] = make_float4(f[0], f[1], f[2], f[3]);
            reinterpret_cast<float4 *>(p)[1] = make_float4(f[4], f[5], f[6], f[7]);
        }
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (j < n) p[j] = from_f32<T>(f[j]);
    }
}

__device__ __forceinline__ void store_codes(int8_t *p, int n, bool vec, const int (&c)[8]) {
    if (vec) {
        uint2 u;
        u.x = (c[0] & 255) | (c[1] & 255) << 8 | (c[2] & 255) << 16 | (uint32_t)c[3] << 24;
        u.y = (c[4] & 255) | (c[5] & 255) << 8 | (c[6] & 255) << 16 | (uint32_t)c[7] << 24;
        *reinterpret_cast<uint2 *>(p) = u;
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (j < n) p[j] = (int8_t)c[j];
    }
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int s = 16; s > 0; s >>= 1) v += __shfl_xor_sync(0xffffffffu, v, s);
    return v;
}

// Sum of `v` and maximum of `m` over the row's threads.  Magnitudes are compared as bits, so
// that a NaN is above everything.  slot: 64 words of shared memory used by no other call.
template <bool WARP_ROW>
__device__ __forceinline__ void reduce_row(float &v, uint32_t &m, uint32_t *slot) {
    v = warp_sum(v);
    m = __reduce_max_sync(0xffffffffu, m);
    if constexpr (!WARP_ROW) {
        const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
        if (lane == 0) {
            slot[warp] = __float_as_uint(v);
            slot[32 + warp] = m;
        }
        __syncthreads();
        v = warp_sum(lane < warps ? __uint_as_float(slot[lane]) : 0.f);
        m = __reduce_max_sync(0xffffffffu, lane < warps ? slot[32 + lane] : 0u);
    }
}

__device__ __forceinline__ uint32_t magnitude(float x) { return __float_as_uint(x) & 0x7fffffffu; }

template <typename T> __device__ __forceinline__ float gate(float z);
template <> __device__ __forceinline__ float gate<float>(float z) { return z / (1.0f + expf(-z)); }
template <> __device__ __forceinline__ float gate<bf16>(float z) { return silu(z); }

}  // namespace

// One row per warp (WARP_ROW) or per CTA; a thread holds NV times 8 consecutive elements.
template <typename T, int MODE, bool OUT8, int NV, bool WARP_ROW>
__global__ void __launch_bounds__(WARP_ROW ? 128 : 1024)
rows_kernel(const RowParams p) {
    __shared__ uint32_t slots[2][64];
    grid_dependency_wait();
    const int G = WARP_ROW ? 32 : blockDim.x, t = WARP_ROW ? threadIdx.x & 31 : threadIdx.x;
    const int64_t row = WARP_ROW ? (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5) : blockIdx.x;
    if (row >= p.T) return;                         // a whole warp, which then meets no barrier
    const bool vec = p.vec;
    const int D = p.D;
    const T *x = (const T *)p.x + row * p.x_st;

    float v[NV][8], g[MODE == kRowGatedNorm ? NV : 1][8];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int e = (i * G + t) * 8, n = D - e;
        if (n > 0) {
            load8(x + e, n, vec, v[i]);
            if constexpr (MODE == kRowGatedNorm)
                load8((const T *)p.z + row * p.z_st + e, n, vec, g[i]);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                v[i][j] = 0.f;
                if constexpr (MODE == kRowGatedNorm) g[i][j] = 0.f;
            }
        }
    }

    float r = 1.f;                                  // what the elements of v still lack
    uint32_t m = 0;                                 // largest |v|, as bits
    if constexpr (MODE == kRowQuantize) {
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) m = max(m, magnitude(v[i][j]));
        float none = 0.f;
        reduce_row<WARP_ROW>(none, m, slots[0]);
    } else if constexpr (MODE == kRowAddNorm) {
        if (p.res) {
            const T *res = (const T *)p.res + row * p.res_st;
            T *res_out = (T *)p.res_out + row * p.res_out_st;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int e = (i * G + t) * 8, n = D - e;
                if (n <= 0) continue;
                float u[8];
                load8(res + e, n, vec, u);
#pragma unroll
                for (int j = 0; j < 8; ++j) v[i][j] += u[j];
                store8(res_out + e, n, vec, v[i]);
            }
        }
        // The largest |h (offset + w)| is found together with the sum of squares: the common
        // factor r does not move the place of the maximum, so one reduction serves both.
        float ss = 0.f;
        float hw[NV][8];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int e = (i * G + t) * 8, n = D - e;
            float w[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) w[j] = 0.f;
            if (n > 0) {
                if (p.w_f32) load8((const float *)p.w + e, n, vec, w);
                else load8((const bf16 *)p.w + e, n, vec, w);
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                ss = fmaf(v[i][j], v[i][j], ss);
                hw[i][j] = v[i][j] * (p.offset + w[j]);
                m = max(m, magnitude(hw[i][j]));
            }
        }
        reduce_row<WARP_ROW>(ss, m, slots[0]);
        float shrink = 1.f;
        if (!(ss < __uint_as_float(kInfBits)) || m >= kInfBits) {
            // Squares or products past fp32: once more with h / 2^80.  A row that holds an
            // infinity or a NaN stays without a finite sum.
            shrink = 8.271806125530277e-25f;
            ss = 0.f;
            m = 0;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int e = (i * G + t) * 8, n = D - e;
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    if (j >= n) continue;
                    const float h = v[i][j] * shrink;
                    const float w = p.w_f32 ? ((const float *)p.w)[e + j] : to_f32(((const bf16 *)p.w)[e + j]);
                    ss = fmaf(h, h, ss);
                    hw[i][j] = h * (p.offset + w);
                    m = max(m, magnitude(hw[i][j]));
                }
            }
            reduce_row<WARP_ROW>(ss, m, slots[1]);
        }
        r = 1.f / sqrtf(ss / (float)D + p.eps * shrink * shrink);
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) v[i][j] = hw[i][j];
    } else {
        const int lanes = p.head >> 3;              // threads of a head: a power of two up to 32
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int e = (i * G + t) * 8, n = D - e;
            float ss = 0.f, shrink = 1.f;
#pragma unroll
            for (int j = 0; j < 8; ++j) ss = fmaf(v[i][j], v[i][j], ss);
            for (int s = lanes >> 1; s > 0; s >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, s);
            const bool big = !(ss < __uint_as_float(kInfBits));
            if (__any_sync(0xffffffffu, big)) {     // as above, for the heads that need it
                float s2 = 0.f;
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float h = v[i][j] * 8.271806125530277e-25f;
                    s2 = fmaf(h, h, s2);
                }
                for (int s = lanes >> 1; s > 0; s >>= 1) s2 += __shfl_xor_sync(0xffffffffu, s2, s);
                if (big) {
                    ss = s2;
                    shrink = 8.271806125530277e-25f;
                }
            }
            const float rh = 1.f / sqrtf(ss / (float)p.head + p.eps * shrink * shrink);
            float w[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) w[j] = 0.f;
            if (n > 0) {
                const int o = e & (p.head - 1);
                if (p.w_f32) load8((const float *)p.w + o, 8, vec, w);
                else load8((const bf16 *)p.w + o, 8, vec, w);
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                v[i][j] = v[i][j] * shrink * rh * w[j] * gate<T>(g[i][j]);
                m = max(m, magnitude(v[i][j]));
            }
        }
        if constexpr (OUT8) {
            float none = 0.f;
            reduce_row<WARP_ROW>(none, m, slots[0]);
        }
    }

    if constexpr (OUT8) {
        // r max|v|, at least 127 * 2^-126: then neither the scale nor its inverse overflows.
        const float largest = fmaxf(r * __uint_as_float(m), 127.f * kTinyScale);
        const bool bad = m >= kInfBits || !(largest < __uint_as_float(kInfBits));
        const float inv = bad ? 0.f : 127.f / largest;
        if (t == 0) p.scale[row] = bad ? __uint_as_float(0x7fc00000u) : largest / 127.f;
        int8_t *y = (int8_t *)p.y + row * p.y_st;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int e = (i * G + t) * 8, n = D - e;
            if (n <= 0) continue;
            int c[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                float q = v[i][j] * r * inv;
                // bf16 rows meet ties exactly (an element of half the largest stands at 63.5).
                // With significands X and A of 8 bits, 127 X / (A 2^s) is a tie or at least
                // 2^-16 of itself away from one, so rounding it to 18 bits brings ties back
                // and moves nothing else across.
                if (MODE == kRowQuantize && sizeof(T) == 2)
                    q = __int_as_float((__float_as_int(q) + 32) & ~63);
                c[j] = bad ? 0 : __float2int_rn(q);
            }
            store_codes(y + e, n, vec, c);
        }
    } else {
        T *y = (T *)p.y + row * p.y_st;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int e = (i * G + t) * 8, n = D - e;
            if (n <= 0) continue;
#pragma unroll
            for (int j = 0; j < 8; ++j) v[i][j] *= r;
            store8(y + e, n, vec, v[i]);
        }
    }
}

}  // namespace gdn

namespace gdn_host {

using namespace gdn;

template <typename T, int MODE, bool OUT8>
static gdn_status_t launch_rows_t(const RowParams &p, cudaStream_t st) {
    const int chunks = (p.D + 7) / 8;               // 8-element pieces of a row
    cudaError_t e;
    if (chunks <= 128) {                            // a warp per row
        const dim3 grid((unsigned)((p.T + 3) / 4));
        e = chunks <= 32 ? launch_dependent(rows_kernel<T, MODE, OUT8, 1, true>, grid, dim3(128), 0, st, p)
                         : launch_dependent(rows_kernel<T, MODE, OUT8, 4, true>, grid, dim3(128), 0, st, p);
    } else {
        const int nv = chunks <= 2048 ? 2 : 4, threads = ((chunks + nv - 1) / nv + 31) / 32 * 32;
        const dim3 grid((unsigned)p.T);
        e = nv == 2 ? launch_dependent(rows_kernel<T, MODE, OUT8, 2, false>, grid, dim3(threads), 0, st, p)
                    : launch_dependent(rows_kernel<T, MODE, OUT8, 4, false>, grid, dim3(threads), 0, st, p);
    }
    return e == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

template <typename T>
static gdn_status_t launch_rows_m(const RowParams &p, int mode, bool eight_bit, cudaStream_t st) {
    if (mode == kRowQuantize) return launch_rows_t<T, kRowQuantize, true>(p, st);
    if (mode == kRowAddNorm)
        return eight_bit ? launch_rows_t<T, kRowAddNorm, true>(p, st) : launch_rows_t<T, kRowAddNorm, false>(p, st);
    return eight_bit ? launch_rows_t<T, kRowGatedNorm, true>(p, st) : launch_rows_t<T, kRowGatedNorm, false>(p, st);
}

gdn_status_t launch_rows(const RowParams &p, int mode, bool in_f32, bool eight_bit, cudaStream_t st) {
    return in_f32 ? launch_rows_m<float>(p, mode, eight_bit, st) : launch_rows_m<bf16>(p, mode, eight_bit, st);
}

}  // namespace gdn_host
