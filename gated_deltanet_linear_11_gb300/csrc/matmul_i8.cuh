// matmul_i8.cuh -- arguments of the product of 8-bit integers.
#pragma once

#include "common.cuh"

namespace gdn {

// The sum of K products of codes stays within an int32 up to here: K * 128^2 < 2^31.
constexpr int64_t kMatmulMaxK = 131071;

struct MatmulParams {
    const int8_t *a, *w;            // [M, K], [N, K], rows a_st and w_st bytes apart
    const float *a_scale, *w_scale; // [M], [N]
    const void *bias;               // [N] or null
    void *out;                      // [M, N], rows out_st elements apart
    int64_t a_st, w_st, out_st;
    int64_t M, N;
    int32_t K;
    int32_t bias_f32, out_f32;
    int32_t *status;
};

// sum * a_scale * w_scale + bias, each step rounded to fp32 (sum: the integer, rounded once).
__device__ __forceinline__ float matmul_value(float sum, float as, float ws, float bias) {
    return __fadd_rn(__fmul_rn(__fmul_rn(sum, as), ws), bias);
}

__device__ __forceinline__ float matmul_bias(const MatmulParams &p, int64_t n) {
    if (!p.bias) return -0.f;       // leaves every value as it is
    return p.bias_f32 ? ((const float *)p.bias)[n] : to_f32(((const bf16 *)p.bias)[n]);
}

}  // namespace gdn

namespace gdn_host {
size_t matmul_i8_workspace(int64_t M, int64_t N, int64_t K, uint32_t flags);
gdn_status_t launch_matmul_i8(const gdn::MatmulParams &p, uint32_t flags, void *ws, size_t ws_bytes,
                              cudaStream_t st);
// the tensor-core kernels: rows of both operands on 16 bytes
bool matmul_i8_tc_supported(const gdn::MatmulParams &p, uint32_t flags);
size_t matmul_i8_tc_workspace(int64_t M, int64_t K);
gdn_status_t launch_matmul_i8_tc(const gdn::MatmulParams &p, void *ws, cudaStream_t st);
}  // namespace gdn_host
