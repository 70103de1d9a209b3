// linear.cu -- linear attention with a decay for each head, on the CUDA cores: the
// recurrence over packed sequences (any D in {16, 32, 64, 128}, fp32 or bf16), and the
// one-token step on a pool of states.
//
//     S_t = e^{g_t} S_{t-1} + k_t v_t^T      (S: D x D, fp32)
//     o_t = scale * S_t^T q_t
//
// It is the gated delta rule without its correction term, so the state's columns do not
// interact: column j of S needs v_j only.
#include <algorithm>

#include "linear.cuh"

namespace gdn {

// ------------------------------------------------------------------ prompts, CUDA cores
// The decay factor as a sum hi + lo of two floats.  A slow decay multiplies the state
// hundreds of times, so e^g rounded to 24 bits would leave a relative error of that many
// half-ulps; for g above -1/2, 1 + expm1(g) keeps it to about |g| 2^-23 a step.  Below, expm1
// near -1 has no finer step than 2^-24, which is much of a small factor (2.6% at g = -15) and
// all of it from -17.4 on; there e^g itself is good to 2^-22 and its error counts for the few
// steps that such a decay leaves anything of.
__device__ __forceinline__ float2 decay_pair(float g) {
    if (g < -0.5f) return make_float2(expf(g), 0.f);
    const float e = expm1f(g), hi = 1.f + e;
    return make_float2(hi, e - (hi - 1.f));
}

// Ranges of one sequence that run side by side, where a walk over all its tokens would leave
// SMs idle: linear_scan_kernel first gives each range's own state from zero (STATE_ONLY), then
// linear_fold_kernel the ranges' start states, then linear_scan_kernel runs the ranges from
// those.  A token costs a walk 118 ns (D = 64), all of it latency, so ranges are short: 64
// tokens or more, from 256 tokens on (fp32, D = 64, 8 v-heads: 4096 tokens 438 us whole, 64 in
// ranges; 256 tokens 33 and 21; ranges of 32, 64 and 128 tokens, two sequences of 800: 39, 37
// and 42; 64 sequences of 384, which fill the device by themselves, 204 whole and 273 so).
// The cut depends on the sequence's own length, the heads and the column tiles only.
constexpr int kScanMinTokens = 256;      // shorter sequences are one range
constexpr int kScanMinRange = 64;
constexpr int kScanCtas = 4 * 152;       // CTAs that ranges are made for
__host__ __device__ __forceinline__ int scan_range_tokens(int len, int ctas) {   // ctas: of one range
    if (len < kScanMinTokens) return len > 0 ? len : 1;
    const int par = kScanCtas / ctas > 1 ? kScanCtas / ctas : 1;
    const int rt = ((len + par - 1) / par + 15) / 16 * 16;
    return rt > kScanMinRange ? rt : kScanMinRange;
}
// A sequence's first slot in the workspace (a state and a decay for each v-head); it has one
// slot more than ranges after its first, at most len / 64.
__device__ __forceinline__ int64_t scan_slot0(int n, int t0) { return t0 / kScanMinRange + n; }

// One CTA per (sequence, range, v-head, tile of columns), walking the tokens.  A lane holds two
// columns of D / RG rows: lanes with equal column pairs split the rows in groups of four
// (rows 4 rg + 4 RG x ..+3), so a float4 of k or q is read by all lanes of a warp without
// bank conflicts, and o is summed over the RG lanes by shuffles in a fixed order.
template <int D> struct LinShape {
    static constexpr int RG = D / 4 < 8 ? D / 4 : 8;     // lanes that split the rows
    static constexpr int CW = (32 / RG) * 2;             // columns per warp
    static constexpr int WARPS = D / CW < 4 ? D / CW : 4;
    static constexpr int COLS = CW * WARPS;              // columns per CTA
    static constexpr int RX = D / (4 * RG);              // groups of four rows per lane
    static constexpr int TB = 16;                        // tokens staged at a time
    static constexpr int FIX = 8;                        // tokens per correction of the decay
};

template <typename T, int D, bool STATE_ONLY>
__global__ void __launch_bounds__(LinShape<D>::WARPS * 32)
linear_scan_kernel(const T *__restrict__ q, const T *__restrict__ k, const T *__restrict__ v,
                   T *__restrict__ o, int64_t q_tok, int64_t k_tok, int64_t v_tok,
                   int64_t o_tok, const float *__restrict__ g, int64_t g_tok,
                   const int32_t *__restrict__ cu, const float *h0, float *hT,
                   float *ranges, float *range_decay, int in_place, int Hk, int Hv, float scale) {
    using L = LinShape<D>;
    constexpr int TILES = D / L::COLS;
    constexpr int THREADS = L::WARPS * 32;
    constexpr int NQ = L::TB * D / THREADS, NV = L::TB * L::COLS / THREADS;   // staged per thread
    __shared__ float4 sq[2][L::TB][D / 4], sk[2][L::TB][D / 4];
    __shared__ float2 sv[2][L::TB][L::COLS / 2];
    __shared__ float sa[2][L::TB], slo[2][L::TB];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int rg = lane % L::RG, cp = warp * (L::CW / 2) + lane / L::RG;
    const int j0 = blockIdx.x % TILES * L::COLS, range = blockIdx.x / TILES, hv = blockIdx.y, n = blockIdx.z;
    const int hk = hv / (Hv / Hk);
    const int seq0 = cu[n], seq_len = cu[n + 1] - seq0;
    const int rt = scan_range_tokens(seq_len, Hv * TILES);
    const bool last = (range + 1) * rt >= seq_len;
    if (range > 0 && range * rt >= seq_len || STATE_ONLY && last) return;
    const int t0 = seq0 + range * rt, len = min(rt, seq_len - range * rt);
    const size_t col0 = j0 + 2 * cp;
    const size_t slot = ((size_t)(scan_slot0(n, seq0) + range) * Hv + hv) * D * D;
    // where the range starts from: the caller's state, or its slot (which has a copy of the
    // caller's where that may be overwritten by the last range)
    const float *from = nullptr;
    if (!STATE_ONLY) {
        if (range > 0 || in_place && !last) {
            grid_dependency_wait();
            from = ranges + slot;
        } else if (h0) from = h0 + ((size_t)n * Hv + hv) * D * D;
    }

    float2 S[L::RX][4];
#pragma unroll
    for (int x = 0; x < L::RX; ++x)
#pragma unroll
        for (int e = 0; e < 4; ++e)
            S[x][e] = from ? *reinterpret_cast<const float2 *>(
                                 from + col0 + (size_t)(4 * rg + 4 * L::RG * x + e) * D)
                           : make_float2(0.f, 0.f);

    // The next block of tokens is on its way to registers while this one is worked on; rows
    // past the end read as zeros.
    T rq[NQ], rk[NQ], rv[NV];
    float rgate = 0.f;
    double gates = 0.;           // STATE_ONLY: sum of this thread's
    auto load = [&](int b) {
#pragma unroll
        for (int x = 0; x < NQ; ++x) {
            const int i = tid + THREADS * x, t = b + i / D, d = i % D;
            const bool in = t < len;
            const int64_t row = t0 + (in ? t : 0);
            if (!STATE_ONLY) rq[x] = in ? q[row * q_tok + (int64_t)hk * D + d] : from_f32<T>(0.f);
            rk[x] = in ? k[row * k_tok + (int64_t)hk * D + d] : from_f32<T>(0.f);
        }
#pragma unroll
        for (int x = 0; x < NV; ++x) {
            const int i = tid + THREADS * x, t = b + i / L::COLS, j = i % L::COLS;
            rv[x] = t < len ? v[(t0 + t) * v_tok + (int64_t)hv * D + j0 + j] : from_f32<T>(0.f);
        }
        if (tid < L::TB) rgate = b + tid < len ? g[(t0 + b + tid) * g_tok + hv] : 0.f;
    };
    auto stage = [&](int u) {
#pragma unroll
        for (int x = 0; x < NQ; ++x) {
            const int i = tid + THREADS * x;
            if (!STATE_ONLY) reinterpret_cast<float *>(sq[u][i / D])[i % D] = to_f32(rq[x]);
            reinterpret_cast<float *>(sk[u][i / D])[i % D] = to_f32(rk[x]);
        }
#pragma unroll
        for (int x = 0; x < NV; ++x) {
            const int i = tid + THREADS * x;
            reinterpret_cast<float *>(sv[u][i / L::COLS])[i % L::COLS] = to_f32(rv[x]);
        }
        if (tid < L::TB) {
            if (STATE_ONLY) gates += rgate;
            const float2 a = decay_pair(rgate);
            sa[u][tid] = a.x;
            slo[u][tid] = a.x > 0.f ? a.y / a.x : 0.f;
        }
    };
    T *out = o + t0 * o_tok + (int64_t)hv * D + j0 + 2 * cp;
    if (len > 0) {
        load(0);
        stage(0);
    }
    for (int b = 0; b < len; b += L::TB) {
        const int u = (b / L::TB) & 1;
        __syncthreads();
        const bool more = b + L::TB < len;
        if (more) load(b + L::TB);
        // eight tokens in one stretch, so that their loads and the shuffles of o overlap;
        // tokens past the end have k = v = q = 0 and no decay, and only their o is left out
#pragma unroll 1
        for (int f = 0; f < L::TB && b + f < len; f += L::FIX) {
            float fix = 0.f;
            float2 acc[L::FIX];
#pragma unroll
            for (int e = 0; e < L::FIX; ++e) {
                const int t = f + e;
                const float a = sa[u][t];
                const float2 vv = sv[u][t][cp];
                fix += slo[u][t];
                acc[e] = make_float2(0.f, 0.f);
#pragma unroll
                for (int x = 0; x < L::RX; ++x) {
                    const float4 k4 = sk[u][t][rg + L::RG * x];
                    const float4 q4 = STATE_ONLY ? make_float4(0.f, 0.f, 0.f, 0.f) : sq[u][t][rg + L::RG * x];
                    const float kk[4] = {k4.x, k4.y, k4.z, k4.w}, qq[4] = {q4.x, q4.y, q4.z, q4.w};
#pragma unroll
                    for (int y = 0; y < 4; ++y) {
                        S[x][y].x = fmaf(S[x][y].x, a, kk[y] * vv.x);
                        S[x][y].y = fmaf(S[x][y].y, a, kk[y] * vv.y);
                        if (!STATE_ONLY) {
                            acc[e].x = fmaf(qq[y], S[x][y].x, acc[e].x);
                            acc[e].y = fmaf(qq[y], S[x][y].y, acc[e].y);
                        }
                    }
                }
            }
            // sum over the RG lanes, halving the tokens a lane keeps at each step: lane rg ends
            // with tokens rg FIX / RG ..
            int keep = L::FIX;
#pragma unroll
            for (int off = STATE_ONLY ? 0 : L::RG / 2; off > 0; off >>= 1) {
                keep >>= 1;
                const bool up = rg & off;
#pragma unroll
                for (int e = 0; e < keep; ++e) {
                    const float2 mine = up ? acc[keep + e] : acc[e], theirs = up ? acc[e] : acc[keep + e];
                    acc[e].x = mine.x + __shfl_xor_sync(0xffffffffu, theirs.x, off);
                    acc[e].y = mine.y + __shfl_xor_sync(0xffffffffu, theirs.y, off);
                }
            }
#pragma unroll
            for (int e = 0; e < (STATE_ONLY ? 0 : L::FIX / L::RG); ++e) {
                const int64_t t = b + f + rg * (L::FIX / L::RG) + e;
                if (t < len) {
                    out[t * o_tok] = from_f32<T>(scale * acc[e].x);
                    out[t * o_tok + 1] = from_f32<T>(scale * acc[e].y);
                }
            }
            // the low parts of these decays at once (the sum is at most about 2^-21)
#pragma unroll
            for (int x = 0; x < L::RX; ++x)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    S[x][e].x = fmaf(S[x][e].x, fix, S[x][e].x);
                    S[x][e].y = fmaf(S[x][e].y, fix, S[x][e].y);
                }
        }
        if (more) stage(u ^ 1);
    }
    float *to = STATE_ONLY ? ranges + slot + (size_t)Hv * D * D
                           : last && hT ? hT + ((size_t)n * Hv + hv) * D * D : nullptr;
    if (to) {
#pragma unroll
        for (int x = 0; x < L::RX; ++x)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                *reinterpret_cast<float2 *>(to + col0 + (size_t)(4 * rg + 4 * L::RG * x + e) * D) =
                    S[x][e];
    }
    if (STATE_ONLY && warp == 0) {
#pragma unroll
        for (int off = 8; off > 0; off >>= 1) gates += __shfl_xor_sync(0xffffffffu, gates, off);
        if (tid == 0 && j0 == 0) range_decay[slot / (D * D) + Hv] = (float)gates;
    }
}

// Start states of a sequence's ranges, in order, over the ranges' own states: the slot of range
// r has the state that range r - 1 adds, and receives the start of range r,
// S <- e^{decay of r - 1} S + it.  Four elements a thread; bound by memory.
template <int D> struct LinFold {
    static constexpr int THREADS = D * D / 4 < 256 ? D * D / 4 : 256;
};
template <int D>
__global__ void __launch_bounds__(LinFold<D>::THREADS)
linear_fold_kernel(const int32_t *__restrict__ cu, const float *__restrict__ h0, float *ranges,
                   const float *__restrict__ range_decay, int in_place, int ctas, int Hv) {
    const int hv = blockIdx.y, n = blockIdx.z;
    const int t0 = cu[n], len = cu[n + 1] - t0;
    const int rt = scan_range_tokens(len, ctas), count = (len + rt - 1) / rt;
    if (count <= 1) return;
    const int at = blockIdx.x * LinFold<D>::THREADS + threadIdx.x;
    const int64_t row = scan_slot0(n, t0) * Hv + hv;
    float4 *R = reinterpret_cast<float4 *>(ranges + row * D * D) + at;
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
    grid_dependency_wait();
    if (h0) s = reinterpret_cast<const float4 *>(h0 + ((int64_t)n * Hv + hv) * D * D)[at];
    if (in_place) *R = s;
    constexpr int AHEAD = 8;         // loads that do not wait for the chain
    const int64_t step = (int64_t)Hv * (D * D / 4);
    for (int r0 = 1; r0 < count; r0 += AHEAD) {
        float4 x[AHEAD];
        float a[AHEAD];
#pragma unroll
        for (int e = 0; e < AHEAD; ++e) {
            if (r0 + e < count) {
                x[e] = R[(r0 + e) * step];
                a[e] = expf(range_decay[row + (int64_t)(r0 + e) * Hv]);
            }
        }
#pragma unroll
        for (int e = 0; e < AHEAD; ++e) {
            if (r0 + e < count) {
                s.x = fmaf(a[e], s.x, x[e].x);
                s.y = fmaf(a[e], s.y, x[e].y);
                s.z = fmaf(a[e], s.z, x[e].z);
                s.w = fmaf(a[e], s.w, x[e].w);
                R[(r0 + e) * step] = s;
            }
        }
    }
}

// --------------------------------------------------------------------- one-token step
// One CTA per (sequence, v-head): the state tile goes through registers once, as float4
// of four columns, so a warp's load is a contiguous 512 bytes; o is summed over the row
// groups in shared memory in a fixed order.  Bound by HBM: 256 sequences of 48 heads of 128,
// 1.62 GB, 235 us, 6.9 TB/s (101% of the copy rate).
template <int D> struct LinDecShape {
    static constexpr int THREADS = D * D / 4 < 256 ? D * D / 4 : 256;
    static constexpr int RG = THREADS / (D / 4);   // row groups
    static constexpr int ROWS = D / RG;            // rows per thread
};

template <typename T, int D>
__global__ void __launch_bounds__(LinDecShape<D>::THREADS)
linear_decode_kernel(const T *__restrict__ q, const T *__restrict__ k, const T *__restrict__ v,
                     T *__restrict__ o, int64_t q_tok, int64_t k_tok, int64_t v_tok,
                     int64_t o_tok, const float *__restrict__ g, int64_t g_tok,
                     float *__restrict__ state, int P, const int32_t *__restrict__ idx, int Hk,
                     int Hv, float scale, int32_t *status) {
    using L = LinDecShape<D>;
    __shared__ float sq[D], sk[D];
    __shared__ __align__(16) float red[L::RG][D];
    const int hv = blockIdx.x, n = blockIdx.y, tid = threadIdx.x;
    const int slot = idx ? idx[n] : n;
    if (slot < 0 || slot >= P) {
        if (tid == 0) report(status, GDN_ERR_INDEX);
        return;
    }
    const int hk = hv / (Hv / Hk);
    const int c4 = tid % (D / 4), rg = tid / (D / 4);
    float4 *tile = reinterpret_cast<float4 *>(state + ((size_t)slot * Hv + hv) * D * D);
    float4 H[L::ROWS];
#pragma unroll
    for (int r = 0; r < L::ROWS; ++r) H[r] = tile[(size_t)(rg + L::RG * r) * (D / 4) + c4];
    const float2 a = decay_pair(g[n * g_tok + hv]);
    const T *vr = v + n * v_tok + (int64_t)hv * D + 4 * c4;
    const float4 vv = make_float4(to_f32(vr[0]), to_f32(vr[1]), to_f32(vr[2]), to_f32(vr[3]));
    for (int i = tid; i < D; i += L::THREADS) {
        sq[i] = to_f32(q[n * q_tok + (int64_t)hk * D + i]);
        sk[i] = to_f32(k[n * k_tok + (int64_t)hk * D + i]);
    }
    __syncthreads();
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int r = 0; r < L::ROWS; ++r) {
        const int i = rg + L::RG * r;
        const float ki = sk[i], qi = sq[i];
        float4 h = H[r];
        h.x = fmaf(a.x, h.x, fmaf(a.y, h.x, ki * vv.x)); acc.x = fmaf(qi, h.x, acc.x);
        h.y = fmaf(a.x, h.y, fmaf(a.y, h.y, ki * vv.y)); acc.y = fmaf(qi, h.y, acc.y);
        h.z = fmaf(a.x, h.z, fmaf(a.y, h.z, ki * vv.z)); acc.z = fmaf(qi, h.z, acc.z);
        h.w = fmaf(a.x, h.w, fmaf(a.y, h.w, ki * vv.w)); acc.w = fmaf(qi, h.w, acc.w);
        tile[(size_t)i * (D / 4) + c4] = h;
    }
    reinterpret_cast<float4 *>(red[rg])[c4] = acc;
    __syncthreads();
    for (int j = tid; j < D; j += L::THREADS) {
        float s = 0.f;
#pragma unroll
        for (int r = 0; r < L::RG; ++r) s += red[r][j];
        o[n * o_tok + (int64_t)hv * D + j] = from_f32<T>(scale * s);
    }
}

}  // namespace gdn

namespace gdn_host {

namespace {

template <int D> constexpr int scan_tiles() { return D / gdn::LinShape<D>::COLS; }
int scan_tiles_of(int64_t D) { return D == 16 ? scan_tiles<16>() : D == 32 ? scan_tiles<32>() : D == 64 ? scan_tiles<64>() : scan_tiles<128>(); }

// Most ranges that a sequence of the batch has, and slots of the workspace (0: none needed).
struct ScanPlan {
    int ranges;
    int64_t slots;
};
ScanPlan plan_scan(const int32_t *cu, int32_t N, int64_t T, int ctas) {
    int most = 1;
    for (int32_t n = 0; n < N; ++n) {
        const int len = cu[n + 1] - cu[n], rt = gdn::scan_range_tokens(len, ctas);
        most = std::max(most, (len + rt - 1) / rt);
    }
    return {most, most > 1 ? T / gdn::kScanMinRange + N : 0};
}
size_t scan_state_bytes(int64_t slots, int32_t Hv, int64_t D) { return (size_t)slots * Hv * D * D * sizeof(float); }

template <typename T, int D>
gdn_status_t scan_launch(const LinearArgs &a, cudaStream_t st) {
    using L = gdn::LinShape<D>;
    constexpr int tiles = scan_tiles<D>();
    const ScanPlan pl = plan_scan(a.cu_host, a.N, a.T, a.Hv * tiles);
    float *ranges = (float *)a.ws;
    float *decay = (float *)((uint8_t *)a.ws + scan_state_bytes(pl.slots, a.Hv, D));
    const int in_place = a.h0 && a.h0 == a.hT;
    const dim3 block(L::WARPS * 32), grid(pl.ranges * tiles, a.Hv, a.N);
    const T *q = (const T *)a.q, *k = (const T *)a.k, *v = (const T *)a.v;
    if (pl.ranges <= 1) {
        gdn::linear_scan_kernel<T, D, false><<<grid, block, 0, st>>>(
            q, k, v, (T *)a.o, a.q_tok, a.k_tok, a.v_tok, a.o_tok, a.g, a.g_tok, a.cu, a.h0, a.hT,
            ranges, decay, in_place, a.Hk, a.Hv, a.scale);
        return cudaGetLastError() == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
    }
    gdn::linear_scan_kernel<T, D, true><<<dim3((pl.ranges - 1) * tiles, a.Hv, a.N), block, 0, st>>>(
        q, k, v, (T *)a.o, a.q_tok, a.k_tok, a.v_tok, a.o_tok, a.g, a.g_tok, a.cu, a.h0, a.hT,
        ranges, decay, in_place, a.Hk, a.Hv, a.scale);
    if (cudaGetLastError() != cudaSuccess) return GDN_ERR_CUDA;
    constexpr int threads = gdn::LinFold<D>::THREADS;
    if (launch_dependent(gdn::linear_fold_kernel<D>, dim3(D * D / 4 / threads, a.Hv, a.N), dim3(threads), 0, st,
                         a.cu, a.h0, ranges, decay, in_place, a.Hv * tiles, a.Hv) != cudaSuccess ||
        launch_dependent(gdn::linear_scan_kernel<T, D, false>, grid, block, 0, st, q, k, v, (T *)a.o, a.q_tok,
                         a.k_tok, a.v_tok, a.o_tok, a.g, a.g_tok, a.cu, a.h0, a.hT, ranges, decay, in_place,
                         a.Hk, a.Hv, a.scale) != cudaSuccess)
        return GDN_ERR_CUDA;
    return GDN_OK;
}

template <typename T, int D>
gdn_status_t decode_launch(const LinearArgs &a, cudaStream_t st) {
    gdn::linear_decode_kernel<T, D>
        <<<dim3(a.Hv, a.N), gdn::LinDecShape<D>::THREADS, 0, st>>>(
            (const T *)a.q, (const T *)a.k, (const T *)a.v, (T *)a.o, a.q_tok, a.k_tok,
            a.v_tok, a.o_tok, a.g, a.g_tok, a.state, a.P, a.idx, a.Hk, a.Hv, a.scale,
            a.status);
    return cudaGetLastError() == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

}  // namespace

#define GDN_LIN_DISPATCH(fn, a, st)                                          \
    switch ((a).D) {                                                         \
    case 16: return (a).in_f32 ? fn<float, 16>(a, st) : fn<gdn::bf16, 16>(a, st);    \
    case 32: return (a).in_f32 ? fn<float, 32>(a, st) : fn<gdn::bf16, 32>(a, st);    \
    case 64: return (a).in_f32 ? fn<float, 64>(a, st) : fn<gdn::bf16, 64>(a, st);    \
    case 128: return (a).in_f32 ? fn<float, 128>(a, st) : fn<gdn::bf16, 128>(a, st); \
    }                                                                        \
    return GDN_ERR_UNSUPPORTED

bool linear_supported(int64_t D) { return D == 16 || D == 32 || D == 64 || D == 128; }

size_t linear_scan_workspace(const int32_t *cu, int32_t N, int64_t T, int32_t Hv, int64_t D) {
    const int64_t slots = plan_scan(cu, N, T, Hv * scan_tiles_of(D)).slots;
    return slots ? scan_state_bytes(slots, Hv, D) + (size_t)slots * Hv * sizeof(float) : 0;
}

gdn_status_t launch_linear_scan(const LinearArgs &a, cudaStream_t st) {
    GDN_LIN_DISPATCH(scan_launch, a, st);
}

gdn_status_t launch_linear_decode(const LinearArgs &a, cudaStream_t st) {
    GDN_LIN_DISPATCH(decode_launch, a, st);
}

}  // namespace gdn_host
