// matmul_i8.cu -- product of 8-bit integers with a scale for each token and channel,
//
//   out[m][n] = a_scale[m] w_scale[n] sum_k a[m][k] w[n][k] + bias[n],
//
// the sum exact in int32: any order and split of it gives the same bits.  This file holds the
// CUDA-core kernel, for every size, stride and alignment.
#include "matmul_i8.cuh"

namespace gdn {

// A CTA of 256 threads makes a tile of 64 x 64 outputs, a thread 4 x 4 of them, from 64
// products at a time of both operands' rows in shared memory (dp4a: four products).
constexpr int kSimtTile = 64, kSimtK = 64, kSimtPad = kSimtK / 4 + 1;

__global__ void __launch_bounds__(256) matmul_i8_simt_kernel(const MatmulParams p) {
    __shared__ int32_t As[kSimtTile][kSimtPad], Ws[kSimtTile][kSimtPad];
    grid_dependency_wait();
    const int64_t tiles_m = (p.M + kSimtTile - 1) / kSimtTile;
    const int64_t m0 = (blockIdx.x % tiles_m) * kSimtTile, n0 = (blockIdx.x / tiles_m) * kSimtTile;
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    int32_t acc[4][4] = {};
    for (int k0 = 0; k0 < p.K; k0 += kSimtK) {
        for (int i = threadIdx.x; i < kSimtTile * kSimtK; i += 256) {
            const int r = i / kSimtK, c = i % kSimtK, k = k0 + c;
            const int64_t m = m0 + r, n = n0 + r;
            reinterpret_cast<int8_t *>(As[r])[c] = m < p.M && k < p.K ? p.a[m * p.a_st + k] : 0;
            reinterpret_cast<int8_t *>(Ws[r])[c] = n < p.N && k < p.K ? p.w[n * p.w_st + k] : 0;
        }
        __syncthreads();
#pragma unroll
        for (int c = 0; c < kSimtK / 4; ++c) {
            int32_t x[4], y[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                x[i] = As[ty + 16 * i][c];
                y[i] = Ws[tx + 16 * i][c];
            }
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[i][j] = __dp4a(x[i], y[j], acc[i][j]);
        }
        __syncthreads();
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int64_t n = n0 + tx + 16 * j;
        if (n >= p.N) continue;
        const float ws = p.w_scale[n], bias = matmul_bias(p, n);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int64_t m = m0 + ty + 16 * i;
            if (m >= p.M) continue;
            const float v = matmul_value((float)acc[i][j], p.a_scale[m], ws, bias);
            if (p.out_f32) ((float *)p.out)[m * p.out_st + n] = v;
            else ((bf16 *)p.out)[m * p.out_st + n] = from_f32<bf16>(v);
        }
    }
}

}  // namespace gdn

namespace gdn_host {

using namespace gdn;

size_t matmul_i8_workspace(int64_t M, int64_t N, int64_t K, uint32_t flags) {
    (void)N;
    return flags & GDN_PREFILL_SIMT ? 0 : matmul_i8_tc_workspace(M, K);
}

gdn_status_t launch_matmul_i8(const MatmulParams &p, uint32_t flags, void *ws, size_t ws_bytes,
                              cudaStream_t st) {
    (void)ws_bytes;
    if (matmul_i8_tc_supported(p, flags)) return launch_matmul_i8_tc(p, ws, st);
    const int64_t tiles = ((p.M + kSimtTile - 1) / kSimtTile) * ((p.N + kSimtTile - 1) / kSimtTile);
    if (tiles > 0x7fffffff) return GDN_ERR_SHAPE;
    return launch_dependent(matmul_i8_simt_kernel, dim3((unsigned)tiles), dim3(256), 0, st, p) == cudaSuccess
               ? GDN_OK : GDN_ERR_CUDA;
}

}  // namespace gdn_host
