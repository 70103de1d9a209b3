// rows.cu -- operators on the rows between the mixers: 8 bits with a scale for each row, the
// root-mean-square norm with the residual's addition, and the Gated DeltaNet layer's output
// norm.
//
//   quantize:   y = x
//   add norm:   h = x + residual;  y = h (offset + w) / sqrt(mean h^2 + eps)
//   gated norm: y = x w / sqrt(mean_head x^2 + eps) * z / (1 + e^-z)
//   8 bits:     scale = max|y| / 127, code = y / scale to the nearest integer
//
// All of them read a row once and write it once, so HBM bounds them.  A row stays in the
// registers of one warp (up to 512 elements, 1024 to be put in 8 bits) or of one CTA, 8
// consecutive elements at a time per thread; sums and maxima go over the row with shuffles and
// one pass through shared memory.  The split of a row depends on its length alone, so a row's
// results are the same in any batch.
//
// Measured, 4096 bf16 rows: norm with residual of 5120 29.8 us (5.6 TB/s, 83% of a copy's rate),
// to 8 bits 24.9 (87%); gated norm of 48 x 128 25.5 (87%), to 8 bits 29.1 (64%: gates and codes
// together are 22% more instructions than the gates alone, which fill 73% of the issue slots);
// 10240 rows of 5120 to 8 bits 29 to 30 (78%), from fp32 43 (90%).  fp32: 4096 norms of 5120 57.5
// (86%), to 8 bits 44 (91%); 4096 gated norms of 48 x 128 52 (85%), to 8 bits 44 (76%).  64 rows and
// fewer take 1.5 to 3 us, a launch and the row's way through the SM.  Rows too long for the ring
// (1000 fp32 norms of 16384: 77 us, 50%) and rows off 16 bytes go element by element.
#include <atomic>

#include "bulk_ptx.cuh"
#include "matmul_i8.cuh"
#include "rows.cuh"

namespace gdn {

namespace {

constexpr float kTinyScale = 1.17549435e-38f;   // 2^-126: the scale of a row of zeros
constexpr uint32_t kInfBits = 0x7f800000u;
constexpr float kShrink = 8.271806125530277e-25f;   // 2^-80
constexpr uint32_t kSmallBits = 0x0d800000u;        // 2^-100: what is 2^-26 of it is a normal number still

// Eight elements from a 16-byte boundary on (weights, shared memory).
template <typename T>
__device__ __forceinline__ void load8(const T *p, float (&f)[8]) {
    if constexpr (sizeof(T) == 2) {
        unpack8(*reinterpret_cast<const uint4 *>(p), f);
    } else {
        const float4 a = reinterpret_cast<const float4 *>(p)[0];
        const float4 b = reinterpret_cast<const float4 *>(p)[1];
        f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
        f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
    }
}
// n <= 8 elements from p on, the rest zero.
template <typename T>
__device__ __forceinline__ void load_some(const T *p, int n, float (&f)[8]) {
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] = j < n ? to_f32(p[j]) : 0.f;
}

template <typename T>
__device__ __forceinline__ void store8(T *p, const float (&f)[8]) {
    if constexpr (sizeof(T) == 2) {
        *reinterpret_cast<uint4 *>(p) = pack8(f);
    } else {
        reinterpret_cast<float4 *>(p)[0] = make_float4(f[0], f[1], f[2], f[3]);
        reinterpret_cast<float4 *>(p)[1] = make_float4(f[4], f[5], f[6], f[7]);
    }
}
// Codes in the low bytes of c.
__device__ __forceinline__ void store8(int8_t *p, const int (&c)[8]) {
    uint2 u;
    u.x = __byte_perm(__byte_perm(c[0], c[1], 0x0040), __byte_perm(c[2], c[3], 0x0040), 0x5410);
    u.y = __byte_perm(__byte_perm(c[4], c[5], 0x0040), __byte_perm(c[6], c[7], 0x0040), 0x5410);
    *reinterpret_cast<uint2 *>(p) = u;
}

// Rows off the boundaries go by way of 1 KB of shared memory per warp: its 256 consecutive
// elements are moved to and from memory by neighbouring lanes, one element each.  n: elements
// of the warp that are in the row (all lanes; at most 0 for none).
template <typename T>
__device__ __forceinline__ void warp_load(const T *p, int n, float *mid, float (&f)[8]) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int j = 0; j < 8; ++j) mid[32 * j + lane] = 32 * j + lane < n ? to_f32(p[32 * j + lane]) : 0.f;
    __syncwarp();
    load8(mid + 8 * lane, f);
    __syncwarp();
}
template <typename T>
__device__ __forceinline__ void warp_store(T *p, int n, float *mid, const float (&f)[8]) {
    const int lane = threadIdx.x & 31;
    store8(mid + 8 * lane, f);
    __syncwarp();
#pragma unroll
    for (int j = 0; j < 8; ++j)
        if (32 * j + lane < n) p[32 * j + lane] = from_f32<T>(mid[32 * j + lane]);
    __syncwarp();
}
__device__ __forceinline__ void warp_store(int8_t *p, int n, float *mid, const int (&c)[8]) {
    const int lane = threadIdx.x & 31;
    store8(reinterpret_cast<int8_t *>(mid) + 8 * lane, c);
    __syncwarp();
#pragma unroll
    for (int j = 0; j < 8; ++j)
        if (32 * j + lane < n) p[32 * j + lane] = reinterpret_cast<const int8_t *>(mid)[32 * j + lane];
    __syncwarp();
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int s = 16; s > 0; s >>= 1) v += __shfl_xor_sync(0xffffffffu, v, s);
    return v;
}

// Sum of `v` (where SUM) and maximum of `m` over the row's threads.  Magnitudes are compared as
// bits, so that a NaN is above everything.  slot: 64 words of shared memory used by no other
// call.
template <bool WARP_ROW, bool SUM>
__device__ __forceinline__ void reduce_row(float &v, uint32_t &m, uint32_t *slot) {
    if (SUM) v = warp_sum(v);
    m = __reduce_max_sync(0xffffffffu, m);
    if constexpr (!WARP_ROW) {
        const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
        if (lane == 0) {
            if (SUM) slot[warp] = __float_as_uint(v);
            slot[32 + warp] = m;
        }
        __syncthreads();
        if (SUM) v = warp_sum(lane < warps ? __uint_as_float(slot[lane]) : 0.f);
        m = __reduce_max_sync(0xffffffffu, lane < warps ? slot[32 + lane] : 0u);
    }
}

// f op g and f op c, two elements an instruction (the kernel is short of issue slots).
__device__ __forceinline__ void add8(float (&f)[8], const float (&g)[8]) {
#pragma unroll
    for (int j = 0; j < 8; j += 2) {
        const float2 t = add_f32x2(make_float2(f[j], f[j + 1]), make_float2(g[j], g[j + 1]));
        f[j] = t.x;
        f[j + 1] = t.y;
    }
}
__device__ __forceinline__ void mul8(float (&f)[8], const float (&g)[8]) {
#pragma unroll
    for (int j = 0; j < 8; j += 2) {
        const float2 t = mul_f32x2(make_float2(f[j], f[j + 1]), make_float2(g[j], g[j + 1]));
        f[j] = t.x;
        f[j + 1] = t.y;
    }
}
__device__ __forceinline__ void mul8(float (&f)[8], float c) {
#pragma unroll
    for (int j = 0; j < 8; j += 2) {
        const float2 t = mul_f32x2(make_float2(f[j], f[j + 1]), make_float2(c, c));
        f[j] = t.x;
        f[j + 1] = t.y;
    }
}
// sum += f^2, of even and of odd elements.
__device__ __forceinline__ void squares8(float2 &sum, const float (&f)[8]) {
#pragma unroll
    for (int j = 0; j < 8; j += 2) {
        const float2 t = make_float2(f[j], f[j + 1]);
        sum = fma_f32x2(t, t, sum);
    }
}
// The same of f / 2^80.
__device__ __forceinline__ void shrunk_squares8(float2 &sum, const float (&f)[8]) {
#pragma unroll
    for (int j = 0; j < 8; j += 2) {
        const float2 t = mul_f32x2(make_float2(f[j], f[j + 1]), make_float2(kShrink, kShrink));
        sum = fma_f32x2(t, t, sum);
    }
}
__device__ __forceinline__ uint32_t magnitude(float x) { return __float_as_uint(x) & 0x7fffffffu; }
__device__ __forceinline__ void largest8(uint32_t &m, const float (&f)[8]) {
#pragma unroll
    for (int j = 0; j < 8; j += 2) m = max(m, max(magnitude(f[j]), magnitude(f[j + 1])));
}

// |q| <= 127 added to 1.5 * 2^23 leaves the nearest integer, ties to even, in the low bits of the
// sum (a conversion to integers runs at an eighth of the rate).
constexpr float kToInteger = 12582912.f;

// v silu(z).  For bf16, 1 / (1 + e^-z) from the hardware's base-2 exponential and reciprocal
// (about 2^-22 each, and the exponent's rounding): far under bf16's half step of 2^-9, and for codes
// up to 127 under 2^-13 of a step, where 2^-10 is allowed.  200 x 64 tokens of 48 x 128 had 43 codes
// of 79 million beside the nearest, all within 2^-15 of a border; with an exact exponential and
// division 41.  e^-z past 2^126 gives a zero.
template <typename T>
__device__ __forceinline__ void gate8(float (&v)[8], const float (&z)[8]) {
#pragma unroll
    for (int j = 0; j < 8; j += 2) {
        float2 s;
        if constexpr (sizeof(T) == 2) {
            s = mul_f32x2(make_float2(z[j], z[j + 1]), make_float2(-1.4426950408889634f, -1.4426950408889634f));
            asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(s.x));
            asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(s.y));
            s = add_f32x2(s, make_float2(1.f, 1.f));
            asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(s.x));
            asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(s.y));
            s = mul_f32x2(s, make_float2(z[j], z[j + 1]));
        } else {
            s = make_float2(z[j] / (1.0f + expf(-z[j])), z[j + 1] / (1.0f + expf(-z[j + 1])));
        }
        s = mul_f32x2(s, make_float2(v[j], v[j + 1]));
        v[j] = s.x;
        v[j + 1] = s.y;
    }
}

}  // namespace

// Asynchronous copy of 8 elements to shared memory (16-byte aligned).
template <typename T>
__device__ __forceinline__ void copy8(uint8_t *dst, const T *src) {
    const uint32_t to = (uint32_t)__cvta_generic_to_shared(dst);
#pragma unroll
    for (int b = 0; b < 8 * (int)sizeof(T); b += 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;"
                     :: "r"(to + b), "l"(reinterpret_cast<const uint8_t *>(src) + b) : "memory");
}

// Registers of a thread, by which the launch counts the CTAs of an SM.  56 for the gated norm: a
// third CTA of 384 threads fits beside two, which its barrier needs most (see below).
constexpr int row_registers(int mode, int nv, bool warp_row, bool vec) {
    if (warp_row && !vec) return 96;             // their number is not counted
    if (!warp_row && nv == 2 && mode == kRowGatedNorm) return 56;
    return nv == 1 || (nv == 2 && mode == kRowQuantize) ? 48 : 64;
}

// One row per warp (WARP_ROW) or per CTA; a thread holds NV times 8 consecutive elements.
// Rows go round the grid.  VEC (rows on 16 bytes): a thread copies its elements of the next two
// rows into a place of its own in shared memory while it works on this one, so that the loads
// never pause; the weights stay in registers.
template <typename T, int MODE, bool OUT8, int NV, bool WARP_ROW, bool VEC>
__global__ void __maxnreg__(row_registers(MODE, NV, WARP_ROW, VEC))
rows_kernel(const __grid_constant__ RowParams p) {
    constexpr int INPUTS = MODE == kRowQuantize ? 1 : 2, PIECE = 8 * (int)sizeof(T);
    constexpr bool HELD = MODE == kRowGatedNorm || (MODE == kRowAddNorm && NV <= 2);   // weights in registers
    extern __shared__ __align__(16) uint8_t ring[];     // [slot][input][NV][thread]
    __shared__ uint32_t slots[2][3][64];
    const int G = WARP_ROW ? 32 : blockDim.x, t = WARP_ROW ? threadIdx.x & 31 : threadIdx.x;
    const int64_t step = WARP_ROW ? (int64_t)gridDim.x * 4 : gridDim.x;
    const int64_t begin = WARP_ROW ? (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5) : blockIdx.x;
    const int D = p.D;
    const T *second = (const T *)(MODE == kRowGatedNorm ? p.z : p.res);      // may be null
    const int64_t second_st = MODE == kRowGatedNorm ? p.z_st : p.res_st;
    grid_dependents_launch();
    grid_dependency_wait();
    if (begin >= p.T) return;                           // a whole warp, which then meets no barrier

    // A head's length divides 256, so all vectors of a thread have the same weights of a head.
    constexpr int KEPT = HELD && MODE == kRowAddNorm ? NV : 1;
    float w[KEPT][8];
    // the weights of vector i: zero past the row's end
    auto weights = [&](int i, float (&f)[8]) {
        const int e = (i * G + t) * 8, n = D - e;
        const int at = MODE == kRowGatedNorm ? e & (p.head - 1) : e;
        if (VEC && n > 0) {
            if (p.w_f32) load8((const float *)p.w + at, f);
            else load8((const bf16 *)p.w + at, f);
        } else {
            if (p.w_f32) load_some((const float *)p.w + at, n, f);
            else load_some((const bf16 *)p.w + at, n, f);
        }
        if (MODE == kRowAddNorm)
#pragma unroll
            for (int j = 0; j < 8; ++j) f[j] = j < n ? p.offset + f[j] : 0.f;
    };
    float *mid = reinterpret_cast<float *>(ring) + (threadIdx.x >> 5) * 256;     // not VEC
    // vector i of an input: its 8 elements, zero past the row's end
    auto input = [&](const T *row, const uint8_t *here, int i, float (&f)[8]) {
        const int e = (i * G + t) * 8;
        if constexpr (!VEC) {
            const int first = e - 8 * (t & 31);
            warp_load(row + first, D - first, mid, f);
        } else if (e < D) {
            load8(reinterpret_cast<const T *>(here), f);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) f[j] = 0.f;
        }
    };
    auto output = [&](auto *row, int i, const auto &f) {
        const int e = (i * G + t) * 8;
        if constexpr (!VEC) warp_store(row + (e - 8 * (t & 31)), D - (e - 8 * (t & 31)), mid, f);
        else if (e < D) store8(row + e, f);
    };
    auto place = [&](int slot, int input, int i) {
        return ring + (((slot * INPUTS + input) * NV + i) * (int)blockDim.x + (int)threadIdx.x) * PIECE;
    };
    auto fetch = [&](int64_t row, int slot) {
        if (row < p.T) {
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int e = (i * G + t) * 8;
                if (e >= D) continue;
                copy8(place(slot, 0, i), (const T *)p.x + row * p.x_st + e);
                if (INPUTS == 2 && second) copy8(place(slot, 1, i), second + row * second_st + e);
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    if constexpr (VEC) {
        fetch(begin, 0);
        fetch(begin + step, 1);
    }
    if constexpr (HELD)
#pragma unroll
        for (int i = 0; i < KEPT; ++i) weights(i, w[i]);

    int slot = 0;
    for (int64_t row = begin; row < p.T; row += step, slot ^= 1) {
        float v[NV][8];
        const T *x = (const T *)p.x + row * p.x_st, *y = second + row * second_st;
        if constexpr (VEC) asm volatile("cp.async.wait_group 1;" ::: "memory");
        uint32_t pairs = 0;                             // largest magnitudes of bf16 elements, two by two
        if constexpr (MODE != kRowGatedNorm) {
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                if constexpr (MODE == kRowQuantize && sizeof(T) == 2 && VEC) {
                    const uint4 u = (i * G + t) * 8 < D ? *reinterpret_cast<const uint4 *>(place(slot, 0, i))
                                                        : make_uint4(0, 0, 0, 0);
                    pairs = __vmaxu2(__vmaxu2(pairs, u.x & 0x7fff7fffu), u.y & 0x7fff7fffu);
                    pairs = __vmaxu2(__vmaxu2(pairs, u.z & 0x7fff7fffu), u.w & 0x7fff7fffu);
                    unpack8(u, v[i]);
                    continue;
                }
                input(x, place(slot, 0, i), i, v[i]);
                if (MODE == kRowAddNorm && second) {
                    float u[8];
                    input(y, place(slot, 1, i), i, u);
                    add8(v[i], u);
                }
            }
            if constexpr (VEC) fetch(row + 2 * step, slot);     // over what this thread has read
            if (MODE == kRowAddNorm && second)
#pragma unroll
                for (int i = 0; i < NV; ++i) output((T *)p.res_out + row * p.res_out_st, i, v[i]);
        }

        float r = 1.f;                                  // what the elements still lack
        uint32_t m = 0;                                 // largest of them, as bits
        if constexpr (MODE == kRowQuantize) {
            if constexpr (sizeof(T) == 2 && VEC) {
                m = max(pairs & 0xffff0000u, pairs << 16);
            } else {
#pragma unroll
                for (int i = 0; i < NV; ++i) largest8(m, v[i]);
            }
            float none = 0.f;
            reduce_row<WARP_ROW, false>(none, m, slots[slot][0]);
        } else if constexpr (MODE == kRowAddNorm) {
            // For 8 bits the largest |h (offset + w)| is found together with the sum of squares: the
            // common factor r does not move the place of the maximum, so one reduction serves both.
            float ss = 0.f;
            auto times_weights = [&](int i, float (&f)[8]) {        // f w
                if constexpr (HELD) {
                    mul8(f, w[i]);
                } else {
                    float u[8];
                    weights(i, u);
                    mul8(f, u);
                }
            };
            auto largest = [&]() {
                m = 0;
#pragma unroll
                for (int i = 0; i < NV; ++i) {
                    float f[8];
#pragma unroll
                    for (int j = 0; j < 8; ++j) f[j] = v[i][j];
                    times_weights(i, f);
                    largest8(m, f);
                }
            };
            auto measure = [&]() {
                float2 sum = make_float2(0.f, 0.f);
#pragma unroll
                for (int i = 0; i < NV; ++i) squares8(sum, v[i]);
                ss = sum.x + sum.y;
                if constexpr (OUT8) largest();
            };
            measure();
            reduce_row<WARP_ROW, true>(ss, m, slots[slot][0]);
            float shrink = 1.f;
            if (!(ss < __uint_as_float(kInfBits))) {
                // Squares past fp32: once more with h / 2^80.  A row that holds an infinity or a NaN
                // stays without a finite sum.
                shrink = kShrink;
                if constexpr (OUT8) {
#pragma unroll
                    for (int i = 0; i < NV; ++i) mul8(v[i], shrink);
                    measure();
                } else {
                    float2 sum = make_float2(0.f, 0.f);
#pragma unroll
                    for (int i = 0; i < NV; ++i) shrunk_squares8(sum, v[i]);
                    ss = sum.x + sum.y;
                }
                reduce_row<WARP_ROW, true>(ss, m, slots[slot][1]);
            }
            r = rsqrtf(__fadd_rn(ss * p.per_mean, p.eps * shrink * shrink));
            if (!OUT8 && shrink != 1.f) {       // r first: the row's small elements stay normal numbers
#pragma unroll
                for (int i = 0; i < NV; ++i) mul8(v[i], r);
                r = shrink;
            }
            // Products past fp32 or among its smallest numbers, though h r w may be neither: h r, at
            // most sqrt(D), comes first then, as it does in rows of floating-point type.  (Not where
            // all are zero, as in rows of padding, and r is up to 2^22: with products of at most
            // 2^-150 the row's codes are zeros.)
            if (!OUT8 || (m - kSmallBits >= kInfBits - kSmallBits && (m != 0 || r > 4194304.f))) {
#pragma unroll
                for (int i = 0; i < NV; ++i) mul8(v[i], r);
                if constexpr (OUT8) {
                    r = 1.f;
                    largest();
                    float none = 0.f;
                    reduce_row<WARP_ROW, false>(none, m, slots[slot][2]);
                }
            }
#pragma unroll
            for (int i = 0; i < NV; ++i) times_weights(i, v[i]);
        } else {
            const int lanes = p.head >> 3;              // threads of a head: a power of two up to 32
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                float g[8], f[8];
                input(x, place(slot, 0, i), i, v[i]);
                input(y, place(slot, INPUTS - 1, i), i, g);
                float2 sum = make_float2(0.f, 0.f);
                squares8(sum, v[i]);
                float ss = sum.x + sum.y;
                for (int s = lanes >> 1; s > 0; s >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, s);
                float rh = rsqrtf(__fadd_rn(ss * p.per_mean, p.eps));
                const bool big = !(ss < __uint_as_float(kInfBits));
                if (__any_sync(0xffffffffu, big)) {     // as above, for the heads that need it
                    sum = make_float2(0.f, 0.f);
                    shrunk_squares8(sum, v[i]);
                    ss = sum.x + sum.y;
                    for (int s = lanes >> 1; s > 0; s >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, s);
                    if (big) {
                        mul8(v[i], rsqrtf(__fadd_rn(ss * p.per_mean, p.eps * kShrink * kShrink)));
                        rh = kShrink;
                    }
                }
                mul8(v[i], rh);
                if constexpr (HELD) {
                    mul8(v[i], w[0]);
                } else {
                    weights(i, f);
                    mul8(v[i], f);
                }
                gate8<T>(v[i], g);
                if constexpr (OUT8) largest8(m, v[i]);
            }
            if constexpr (VEC) fetch(row + 2 * step, slot);
            if constexpr (OUT8) {
                float none = 0.f;
                reduce_row<WARP_ROW, false>(none, m, slots[slot][0]);
            }
        }

        if constexpr (OUT8) {
            // r max|v|, at least 127 * 2^-126: then neither the scale nor its inverse overflows.
            const float largest = fmaxf(r * __uint_as_float(m), 127.f * kTinyScale);
            const bool bad = m >= kInfBits || !(largest < __uint_as_float(kInfBits));
            const float inv = bad ? 0.f : 127.f / largest;
            if (t == 0) p.scale[row] = bad ? __uint_as_float(0x7fc00000u) : largest / 127.f;
            float to_code = r * inv;
            if (!(to_code < __uint_as_float(kInfBits))) {       // a row near the smallest numbers
                to_code = inv;
#pragma unroll
                for (int i = 0; i < NV; ++i) mul8(v[i], r);
            }
            if (bad) {
                to_code = 0.f;
#pragma unroll
                for (int i = 0; i < NV; ++i)
#pragma unroll
                    for (int j = 0; j < 8; ++j) v[i][j] = 0.f;
            }
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                int c[8];
                if constexpr (MODE == kRowQuantize && sizeof(T) == 2) {
                    // bf16 rows meet ties exactly (an element of half the largest stands at 63.5).
                    // With significands X and A of 8 bits, 127 X / (A 2^s) is a tie or at least
                    // 2^-16 of itself away from one, so rounding it to 18 bits brings ties back
                    // and moves nothing else across.
                    mul8(v[i], to_code);
#pragma unroll
                    for (int j = 0; j < 8; j += 2) {
                        const float2 q = add_f32x2(
                            make_float2(__int_as_float((__float_as_int(v[i][j]) + 32) & ~63),
                                        __int_as_float((__float_as_int(v[i][j + 1]) + 32) & ~63)),
                            make_float2(kToInteger, kToInteger));
                        c[j] = __float_as_int(q.x);
                        c[j + 1] = __float_as_int(q.y);
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < 8; j += 2) {        // rounded once
                        const float2 q = fma_f32x2(make_float2(v[i][j], v[i][j + 1]), make_float2(to_code, to_code),
                                                   make_float2(kToInteger, kToInteger));
                        c[j] = __float_as_int(q.x);
                        c[j + 1] = __float_as_int(q.y);
                    }
                }
                output((int8_t *)p.y + row * p.y_st, i, c);
            }
        } else {
#pragma unroll
            for (int i = 0; i < NV; ++i) output((T *)p.y + row * p.y_st, i, v[i]);
        }
    }
}

}  // namespace gdn

namespace gdn_host {

using namespace gdn;

constexpr int kRowSmem = 220 * 1024;

template <typename T, int MODE, bool OUT8, int NV, bool WARP_ROW, bool VEC>
static gdn_status_t launch_rows_k(const RowParams &p, int threads, cudaStream_t st) {
    auto kern = rows_kernel<T, MODE, OUT8, NV, WARP_ROW, VEC>;
    const int smem = VEC ? 2 * (MODE == kRowQuantize ? 1 : 2) * NV * threads * 8 * (int)sizeof(T) : 32 * threads;
    static std::atomic<uint64_t> ready{0};   // one bit per device (beyond 63: set every time)
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return GDN_ERR_CUDA;
    if (VEC && (dev > 63 || !((ready.load() >> dev) & 1u))) {
        if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kRowSmem) != cudaSuccess)
            return GDN_ERR_CUDA;
        if (dev <= 63) ready.fetch_or(1ull << dev);
    }
    const int sms = matmul_sm_count(dev);
    if (sms <= 0) return GDN_ERR_CUDA;
    // as many CTAs as the SMs take at once, by registers and by shared memory
    int per = 65536 / (threads * row_registers(MODE, NV, WARP_ROW, VEC));
    if (per > 220 * 1024 / (smem + 2048)) per = 220 * 1024 / (smem + 2048);
    if (per < 1) per = 1;
    const int64_t rows = WARP_ROW ? (p.T + 3) / 4 : p.T, most = VEC ? (int64_t)sms * per : rows;
    return launch_dependent(kern, dim3((unsigned)(rows < most ? rows : most)), dim3(threads), smem, st, p) == cudaSuccess
               ? GDN_OK : GDN_ERR_CUDA;
}

template <typename T, int MODE, bool OUT8>
static gdn_status_t launch_rows_t(const RowParams &p, cudaStream_t st) {
    const int chunks = (p.D + 7) / 8;               // 8-element pieces of a row
    // two rows of every input have to fit, padded to whole warps (norms: 27136 elements of bf16)
    constexpr int fits = kRowSmem / (2 * (MODE == kRowQuantize ? 1 : 2) * (int)sizeof(T)) - 1024;
    const bool vec = p.vec && p.D <= fits;
    if (chunks <= 32)
        return vec ? launch_rows_k<T, MODE, OUT8, 1, true, true>(p, 128, st)
                   : launch_rows_k<T, MODE, OUT8, 1, true, false>(p, 128, st);
    if (chunks <= 64)
        return vec ? launch_rows_k<T, MODE, OUT8, 2, true, true>(p, 128, st)
                   : launch_rows_k<T, MODE, OUT8, 2, true, false>(p, 128, st);
    if constexpr (MODE == kRowQuantize)
        if (chunks <= 128)                          // little to hold: 4096 x 1000 in 4.5 us, by CTAs 6.1
            return vec ? launch_rows_k<T, MODE, OUT8, 4, true, true>(p, 128, st)
                       : launch_rows_k<T, MODE, OUT8, 4, true, false>(p, 128, st);
    if (chunks <= 128)
        return vec ? launch_rows_k<T, MODE, OUT8, 1, false, true>(p, (chunks + 31) / 32 * 32, st)
                   : launch_rows_k<T, MODE, OUT8, 1, false, false>(p, (chunks + 31) / 32 * 32, st);
    const int nv = chunks <= 2048 ? 2 : 4, threads = ((chunks + nv - 1) / nv + 31) / 32 * 32;
    if (nv == 2)
        return vec ? launch_rows_k<T, MODE, OUT8, 2, false, true>(p, threads, st)
                   : launch_rows_k<T, MODE, OUT8, 2, false, false>(p, threads, st);
    if constexpr (fits > 2048 * 8)
        if (vec) return launch_rows_k<T, MODE, OUT8, 4, false, true>(p, threads, st);
    return launch_rows_k<T, MODE, OUT8, 4, false, false>(p, threads, st);
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
