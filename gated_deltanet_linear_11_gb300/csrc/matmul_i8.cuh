// matmul_i8.cuh -- arguments of the product of 8-bit integers.
#pragma once

#include <cuda_fp16.h>

#include "common.cuh"
#include "tc_ptx.cuh"
#include "tmap.cuh"

namespace gdn {

struct I8Maps {
    CUtensorMap w, a;
};

struct MatmulParams {
    const int8_t *a, *w;            // [M, K], [N, K], rows a_st and w_st bytes apart
    const float *a_scale, *w_scale; // [M], [N]
    const void *bias;               // [N] or null
    void *out;                      // [M, N], rows out_st elements apart
    int64_t a_st, w_st, out_st;
    int64_t M, N;
    int32_t K;
    int32_t bias_f32, out_f32;
    int32_t out_vec;                // rows of out start on 16 bytes
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

__device__ __forceinline__ void matmul_store(const MatmulParams &p, int64_t m, int64_t n, float v) {
    if (p.out_f32) ((float *)p.out)[m * p.out_st + n] = v;
    else ((bf16 *)p.out)[m * p.out_st + n] = from_f32<bf16>(v);
}

__device__ __forceinline__ void load_2d(void *dst, const CUtensorMap *map, uint64_t *bar, int x, int y) {
    asm volatile("cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
                 " [%0], [%1, {%2, %3}], [%4];"
                 :: "r"(tc::smem_u32(dst)), "l"(map), "r"(x), "r"(y), "r"(tc::smem_u32(bar)) : "memory");
}
__device__ __forceinline__ void prefetch_2d(const CUtensorMap *map, int x, int y) {
    asm volatile("cp.async.bulk.prefetch.tensor.2d.L2.global.tile [%0, {%1, %2}];"
                 :: "l"(map), "r"(x), "r"(y) : "memory");
}

// Four codes as fp16 pairs (elements 0 and 1, 2 and 3): x ^ 0x80 is x + 128 in 0..255; as the
// low byte of 0x6400 that is the fp16 number 1024 + 128 + x, less 1152 (exact).
__device__ __forceinline__ void i8_halves(uint32_t w, uint32_t &lo, uint32_t &hi) {
    const uint32_t u = w ^ 0x80808080u;
    const __half2 less = __floats2half2_rn(1152.f, 1152.f);
    uint32_t a = __byte_perm(u, 0x64646464u, 0x4140), b = __byte_perm(u, 0x64646464u, 0x4342);
    const __half2 x = __hsub2(*reinterpret_cast<__half2 *>(&a), less);
    const __half2 y = __hsub2(*reinterpret_cast<__half2 *>(&b), less);
    lo = *reinterpret_cast<const uint32_t *>(&x);
    hi = *reinterpret_cast<const uint32_t *>(&y);
}

}  // namespace gdn

namespace gdn_host {
// Boxes of 128 bytes of `box_rows` rows of codes, or of fp16; a row's end and the rows' end
// read as zeros.
bool row_map(CUtensorMap *m, const void *ptr, bool half, int64_t rows, int64_t K, int64_t stride, int box_rows,
             bool swizzle);
int matmul_sm_count(int dev);           // 0 on an error
size_t matmul_i8_workspace(const gdn::MatmulParams &p, uint32_t flags);
gdn_status_t launch_matmul_i8(const gdn::MatmulParams &p, uint32_t flags, void *ws, cudaStream_t st);
// rows of w (and of a, unless by pairs) on 16 bytes
bool matmul_i8_pairs(int64_t M, int64_t N, int64_t K);
gdn_status_t launch_matmul_i8_few(const gdn::MatmulParams &p, cudaStream_t st);
size_t matmul_i8_pair_workspace(int64_t M, int64_t N, int64_t K);
gdn_status_t launch_matmul_i8_pair(const gdn::MatmulParams &p, void *ws, cudaStream_t st);
}  // namespace gdn_host
