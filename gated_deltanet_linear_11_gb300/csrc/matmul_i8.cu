// matmul_i8.cu -- product of 8-bit integers with a scale for each token and channel,
//
//   out[m][n] = a_scale[m] w_scale[n] sum_k a[m][k] w[n][k] + bias[n],
//
// the sum exact in int32: any order and split of it gives the same bits.  This file holds the
// kernel for few tokens, which streams the channels' codes, and the CUDA-core kernel.
#include <atomic>

#include "bulk_ptx.cuh"
#include "matmul_i8.cuh"

namespace gdn {

// ------------------------------------------------------------------ few tokens
//
// HBM bounds a product with few tokens: every code of w is read once.  A warp takes 32 channels
// and every eighth step of 128 codes; a step's codes of w and of MT tokens come by TMA into a
// ring that is the warp's own.  A lane has one channel, so the tokens' codes are the same for
// all lanes (one read of shared memory for the warp) and nothing is added across lanes; dp4a
// makes four products an instruction, 64 lanes a clock: 512 clocks for 16 KB of w and 8 tokens,
// where HBM takes 700.  The eight warps of a CTA add up their int32 sums in shared memory.
// Measured: one token of 16480 channels of 5120 15.2 us (5.6 TB/s, 82% of a copy's rate), four
// 16.2; of 5120 channels of 6144 9.1 us, 31 MB whose first and last bytes take half of the time.
constexpr int kStreamWarps = 8, kStreamRows = 32, kStreamStep = 128;

template <int MT> struct StreamSmem {
    static constexpr int STAGES = MT <= 4 ? 3 : 2;
    uint8_t w[kStreamWarps][STAGES][kStreamRows * kStreamStep];
    uint8_t a[kStreamWarps][STAGES][MT * kStreamStep];
    int32_t sums[2][MT][kStreamRows];            // of a tile (even, odd)
    uint64_t full[kStreamWarps][STAGES];
    int abort;
};

template <int MT>
__global__ void __launch_bounds__(32 * kStreamWarps, 2)
matmul_i8_stream_kernel(const __grid_constant__ I8Maps maps, const __grid_constant__ MatmulParams p, int tiles) {
    using Sm = StreamSmem<MT>;
    constexpr int STAGES = Sm::STAGES;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    Sm &S = *reinterpret_cast<Sm *>(smem_raw);
    if (tc::smem_u32(smem_raw) & 1023u) {        // the swizzle needs it; never seen
        if (threadIdx.x == 0) report(p.status, GDN_ERR_CUDA);
        return;
    }
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int steps = (p.K + kStreamStep - 1) / kStreamStep;
    const int mine = (steps - warp + kStreamWarps - 1) / kStreamWarps;       // of a tile
    volatile int *abort = &S.abort;
    grid_dependents_launch();
    if (lane == 0) {
        for (int i = 0; i < STAGES; ++i) tc::mbar_init(&S.full[warp][i], 1);
        tc::mbar_fence_init();
    }
    if (tid == 0) S.abort = 0;
    for (int i = tid; i < 2 * MT * kStreamRows; i += 32 * kStreamWarps) (&S.sums[0][0][0])[i] = 0;
    // the copies: tile and step of the next one
    int next_tile = blockIdx.x, next_s = 0, issued = 0;
    // codes of w on their way to L2 while the kernel before this one ends
    if (lane == 0) {
        tc::prefetch_tmap(&maps.w);
        tc::prefetch_tmap(&maps.a);
        for (int i = 0; i < min(mine, STAGES); ++i)
            prefetch_2d(&maps.w, kStreamStep * (warp + kStreamWarps * i), next_tile * kStreamRows);
    }
    __syncthreads();
    grid_dependency_wait();
    auto copy = [&]() {                          // lane 0
        if (mine == 0 || next_tile >= tiles) return;
        const int slot = issued % STAGES, k = kStreamStep * (warp + kStreamWarps * next_s);
        tc::mbar_expect_tx(&S.full[warp][slot], kStreamRows * kStreamStep + MT * kStreamStep);
        load_2d(S.w[warp][slot], &maps.w, &S.full[warp][slot], k, next_tile * kStreamRows);
        load_2d(S.a[warp][slot], &maps.a, &S.full[warp][slot], k, 0);
        ++issued;
        if (++next_s == mine) next_s = 0, next_tile += gridDim.x;
    };
    if (lane == 0)
        for (int i = 0; i < STAGES; ++i) copy();

    int used = 0;
    bool ok = true;
    for (int tile = blockIdx.x, turn = 0; tile < tiles; tile += gridDim.x, turn ^= 1) {
        int32_t acc[MT];
#pragma unroll
        for (int j = 0; j < MT; ++j) acc[j] = 0;
        for (int s = 0; s < mine && ok; ++s, ++used) {
            const int slot = used % STAGES;
            ok = wait_bounded_poll<0>(&S.full[warp][slot], (used / STAGES) & 1, abort);
            if (!ok) *abort = 1;
            if (!(ok = __all_sync(0xffffffffu, ok))) break;
            const uint8_t *w = S.w[warp][slot], *a = S.a[warp][slot];
#pragma unroll
            for (int c = 0; c < kStreamStep / 16; ++c) {
                const uint4 x = *reinterpret_cast<const uint4 *>(w + tc::swz(lane, c));
#pragma unroll
                for (int j = 0; j < MT; ++j) {
                    const uint4 y = *reinterpret_cast<const uint4 *>(a + j * kStreamStep + 16 * c);
                    acc[j] = __dp4a((int)x.x, (int)y.x, acc[j]);
                    acc[j] = __dp4a((int)x.y, (int)y.y, acc[j]);
                    acc[j] = __dp4a((int)x.z, (int)y.z, acc[j]);
                    acc[j] = __dp4a((int)x.w, (int)y.w, acc[j]);
                }
            }
            __syncwarp();                        // all have read the stage
            if (lane == 0) copy();
        }
        if (mine > 0)
#pragma unroll
            for (int j = 0; j < MT; ++j) atomicAdd(&S.sums[turn][j][lane], acc[j]);
        __syncthreads();
        // the other tile's sums are added to meanwhile
        for (int i = tid; i < MT * kStreamRows; i += 32 * kStreamWarps) {
            const int m = i / kStreamRows;
            const int64_t n = (int64_t)tile * kStreamRows + i % kStreamRows;
            int32_t *sum = &S.sums[turn][m][i % kStreamRows];
            if (n < p.N && m < p.M)
                matmul_store(p, m, n, matmul_value((float)*sum, p.a_scale[m], p.w_scale[n], matmul_bias(p, n)));
            *sum = 0;
        }
    }
    // nothing may land after the CTA has left
    if (lane == 0)
        for (; used < issued; ++used)
            wait_bounded_poll<0>(&S.full[warp][used % STAGES], (used / STAGES) & 1, nullptr);
    __syncthreads();
    if (tid == 0 && *abort) report(p.status, GDN_ERR_TIMEOUT);
}

// Rows of codes that do not start on 16 bytes, of one operand or both, copied to rows that do
// (st bytes apart, zeros from K on).  A thread makes 16 bytes of the aligned words that hold any
// of them.
struct AlignRows {
    const int8_t *src;
    int8_t *dst;
    int64_t src_st, rows;                        // rows 0: nothing to copy
};
__global__ void __launch_bounds__(256) matmul_i8_align_kernel(const __grid_constant__ AlignRows a,
                                                              const __grid_constant__ AlignRows b, int64_t st, int32_t K) {
    grid_dependents_launch();
    grid_dependency_wait();
    const int64_t per = st / 16, first = a.rows * per, total = first + b.rows * per;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
        const AlignRows &m = i < first ? a : b;
        const int64_t piece = i < first ? i : i - first, row = piece / per;
        const int k = (int)(piece - row * per) * 16, n = min(K - k, 16);
        const uintptr_t at = (uintptr_t)(m.src + row * m.src_st + k);
        const uint32_t *word = (const uint32_t *)(at & ~(uintptr_t)3);
        const int off = (int)(at & 3u), words = (off + n + 3) / 4;
        uint32_t w[5], out[4];
#pragma unroll
        for (int j = 0; j < 5; ++j) w[j] = j < words ? word[j] : 0u;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            out[j] = __funnelshift_r(w[j], w[j + 1], 8 * off);
            const int left = n - 4 * j;          // bytes of this word that are in the row
            if (left < 4) out[j] = left > 0 ? out[j] & ((1u << (8 * left)) - 1u) : 0u;
        }
        *reinterpret_cast<uint4 *>(m.dst + row * st + k) = make_uint4(out[0], out[1], out[2], out[3]);
    }
}

// ------------------------------------------------------------------ CUDA cores
//
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

bool row_map(CUtensorMap *m, const void *ptr, bool half, int64_t rows, int64_t K, int64_t stride, int box_rows,
             bool swizzle) {
    auto fn = tensor_map_encoder();
    if (!fn) return false;
    const int size = half ? 2 : 1;
    cuuint64_t dims[2] = {(cuuint64_t)K, (cuuint64_t)rows};
    cuuint64_t strides[1] = {(cuuint64_t)(rows > 1 ? stride * size : (K * size + 15) / 16 * 16)};
    cuuint32_t box[2] = {(cuuint32_t)(128 / size), (cuuint32_t)box_rows}, unit[2] = {1, 1};
    return fn(m, half ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_UINT8, 2,
              const_cast<void *>(ptr), dims, strides, box, unit, CU_TENSOR_MAP_INTERLEAVE_NONE,
              swizzle ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

int matmul_sm_count(int dev) {
    static std::atomic<int> known[64];
    if (dev < 64) {
        const int n = known[dev].load();
        if (n > 0) return n;
    }
    int n = 0;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0) return 0;
    if (dev < 64) known[dev].store(n);
    return n;
}

namespace {

bool on_16_bytes(const int8_t *ptr, int64_t rows, int64_t st) {
    return ((uintptr_t)ptr & 15u) == 0 && (rows == 1 || st % 16 == 0);
}
size_t up256(size_t n) { return (n + 255) / 256 * 256; }

// Bytes of the aligned copies of a and of w (0: none needed).
void align_sizes(const MatmulParams &p, size_t &a, size_t &w) {
    const size_t st = ((size_t)p.K + 15) / 16 * 16;
    a = matmul_i8_pairs(p.M, p.N, p.K) || on_16_bytes(p.a, p.M, p.a_st) ? 0 : up256((size_t)p.M * st);
    w = on_16_bytes(p.w, p.N, p.w_st) ? 0 : up256((size_t)p.N * st);
}

// Copies the operands that need it to `to` and points p at the copies.
gdn_status_t launch_align(MatmulParams &p, size_t a_bytes, size_t w_bytes, uint8_t *to, cudaStream_t st) {
    const int64_t row = ((int64_t)p.K + 15) / 16 * 16;
    const AlignRows a = {p.a, (int8_t *)to, p.a_st, a_bytes ? p.M : 0};
    const AlignRows w = {p.w, (int8_t *)to + a_bytes, p.w_st, w_bytes ? p.N : 0};
    const int64_t blocks = ((a.rows + w.rows) * (row / 16) + 255) / 256;
    if (launch_dependent(matmul_i8_align_kernel, dim3((unsigned)(blocks < 4096 ? blocks : 4096)), dim3(256), 0, st, a, w,
                         row, p.K) != cudaSuccess)
        return GDN_ERR_CUDA;
    if (a_bytes) { p.a = a.dst; p.a_st = row; }
    if (w_bytes) { p.w = w.dst; p.w_st = row; }
    return GDN_OK;
}

template <int MT>
gdn_status_t launch_stream(const MatmulParams &p, cudaStream_t st) {
    auto kern = matmul_i8_stream_kernel<MT>;
    constexpr int smem = sizeof(StreamSmem<MT>);
    static_assert(2 * (smem + 1024) <= 228 * 1024, "two CTAs fit on an SM");
    static std::atomic<uint64_t> ready{0};   // one bit per device (beyond 63: set every time)
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return GDN_ERR_CUDA;
    if (dev > 63 || !((ready.load() >> dev) & 1u)) {
        if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
            return GDN_ERR_CUDA;
        if (dev <= 63) ready.fetch_or(1ull << dev);
    }
    const int sms = matmul_sm_count(dev);
    if (sms <= 0) return GDN_ERR_CUDA;
    I8Maps maps;
    if (!row_map(&maps.w, p.w, false, p.N, p.K, p.w_st, kStreamRows, true) ||
        !row_map(&maps.a, p.a, false, p.M, p.K, p.a_st, MT, false))
        return GDN_ERR_CUDA;
    const int64_t tiles = (p.N + kStreamRows - 1) / kStreamRows;
    return launch_dependent(kern, dim3((unsigned)(tiles < 2 * sms ? tiles : 2 * sms)), dim3(32 * kStreamWarps), smem,
                            st, maps, p, (int)tiles) == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

}  // namespace

size_t matmul_i8_workspace(const MatmulParams &p, uint32_t flags) {
    if (flags & GDN_PREFILL_SIMT) return 0;
    size_t a, w;
    align_sizes(p, a, w);
    return a + w + (matmul_i8_pairs(p.M, p.N, p.K) ? matmul_i8_pair_workspace(p.M, p.N, p.K) : 0);
}

gdn_status_t launch_matmul_i8(const MatmulParams &given, uint32_t flags, void *ws, cudaStream_t st) {
    MatmulParams p = given;
    if (flags & GDN_PREFILL_SIMT) {
        const int64_t tiles = ((p.M + kSimtTile - 1) / kSimtTile) * ((p.N + kSimtTile - 1) / kSimtTile);
        if (tiles > 0x7fffffff) return GDN_ERR_SHAPE;
        return launch_dependent(matmul_i8_simt_kernel, dim3((unsigned)tiles), dim3(256), 0, st, p) == cudaSuccess
                   ? GDN_OK : GDN_ERR_CUDA;
    }
    uint8_t *at = (uint8_t *)ws;
    size_t a, w;
    align_sizes(p, a, w);
    if (a + w > 0) {
        const gdn_status_t s = launch_align(p, a, w, at, st);
        if (s != GDN_OK) return s;
        at += a + w;
    }
    if (p.M == 1) return launch_stream<1>(p, st);
    if (p.M == 2) return launch_stream<2>(p, st);
    if (p.M <= 4) return launch_stream<4>(p, st);
    if (p.M <= 8) return launch_stream<8>(p, st);
    if (matmul_i8_pairs(p.M, p.N, p.K)) return launch_matmul_i8_pair(p, at, st);
    return launch_matmul_i8_few(p, st);
}

}  // namespace gdn_host
