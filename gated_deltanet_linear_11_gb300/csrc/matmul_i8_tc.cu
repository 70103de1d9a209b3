// matmul_i8_tc.cu -- gdn_matmul_i8 for many tokens, on tcgen05.
//
// sm_103a has no 8-bit integer form of tcgen05.mma, and its legacy integer path is a small
// part of the fp16 rate.  An int8 is exact in fp16, a product of two is exact in fp32, and so
// is every sum of them that stays within 2^24 (1024 products of any codes): the products run
// as kind::f16 with fp32 sums in TMEM, and sums move to registers before they could pass 2^24.
// The result is the exact integer for any input, whatever the split.
//
// Channels are the rows of the product (M = 256, half in either CTA of a pair): their codes go
// from shared memory through registers into TMEM as fp16, where the tensor core takes them as
// operand A.  Tokens are its columns, operand B.
#include <atomic>

#include "bulk_ptx.cuh"
#include "matmul_i8.cuh"
#include "tmap.cuh"

namespace gdn {

constexpr int kI8Channels = 128;    // channels of a tile
constexpr int kI8Step = 128;        // codes of a row per step
constexpr int kI8Exact = 7;         // steps whose sums, on top of kI8Near, fp32 holds exactly
constexpr float kI8Near = 2097152.f;    // 2^21: 7 * 128 * 2^14 + 2^21 = 2^24
constexpr int kI8ConvWarps = 8;
constexpr int kI8Threads = 32 * (kI8ConvWarps + 2);

template <int NT> struct I8Shape {
    static constexpr int RAW_W = kI8Channels * kI8Step, RAW_A = NT * kI8Step;
    static constexpr int STAGES = NT <= 32 ? 4 : 3;
    static constexpr int CONV = NT * kI8Step * 2;
    static constexpr int CTAS = 2;                       // that fit on an SM
    // TMEM columns: two accumulators of NT, two steps of 64 columns of operand A
    static constexpr int COL_A = 2 * NT, COLS = 256;
    static_assert(COL_A + 128 <= COLS, "the columns fit");
};
template <int NT> struct I8Smem {
    uint8_t raw_w[I8Shape<NT>::STAGES][I8Shape<NT>::RAW_W];
    uint8_t raw_a[I8Shape<NT>::STAGES][I8Shape<NT>::RAW_A];
    uint8_t conv[2][I8Shape<NT>::CONV];      // [step][64-code block][token][128 bytes]
    uint64_t raw_full[I8Shape<NT>::STAGES], raw_free[I8Shape<NT>::STAGES];
    uint64_t ab_full[2], ab_free[2], d_full[2], d_free[2];
    uint64_t sums_full;
    alignas(16) float scale[NT];             // of the tokens
    uint32_t tmem;
    int abort;
};

__device__ __forceinline__ void i8_arrive(uint64_t *bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" :: "r"(tc::smem_u32(bar)) : "memory");
}
// Bounded wait by a warp; false once any thread of the CTA has given up.
template <int SLEEP_NS = 0>
__device__ __forceinline__ bool i8_wait(uint64_t *bar, uint32_t parity, volatile int *abort) {
    const bool ok = wait_bounded_poll<SLEEP_NS>(bar, parity, abort);
    if (!ok) *abort = 1;
    return __all_sync(0xffffffffu, ok) != 0;
}

// 32-bit instruction descriptor: fp16 A and B, both K-major, fp32 D.
__device__ constexpr uint32_t i8_idesc(int M, int N) {
    return (1u << 4) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}
__device__ __forceinline__ void i8_mma(uint32_t d, uint32_t a, uint64_t b, uint32_t id, uint32_t add) {
    asm volatile("{\n\t.reg .pred p, e;\n\t"
                 "elect.sync _|e, 0xffffffff;\n\t"
                 "setp.ne.b32 p, %4, 0;\n\t"
                 "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}"
                 :: "r"(d), "r"(a), "l"(b), "r"(id), "r"(add) : "memory");
}
__device__ __forceinline__ void i8_st16(uint32_t taddr, const uint32_t (&r)[16]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
                 "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};"
                 :: "r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]),
                    "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]),
                    "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]) : "memory");
}
// 16 codes: eight words of fp16 pairs.
__device__ __forceinline__ void i8_halves16(const uint4 &v, uint32_t *r) {
    i8_halves(v.x, r[0], r[1]);
    i8_halves(v.y, r[2], r[3]);
    i8_halves(v.z, r[4], r[5]);
    i8_halves(v.w, r[6], r[7]);
}

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
    uint32_t r;
    asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t cluster_addr(const void *p, uint32_t rank) {
    uint32_t remote;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(tc::smem_u32(p)), "r"(rank));
    return remote;
}
// The halves of a cluster's barrier that order no memory.
__device__ __forceinline__ void cluster_arrive_relaxed() {
    asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// 16 bytes to a CTA of the cluster, counted by its barrier when they are there.
__device__ __forceinline__ void cluster_put(uint32_t to, uint32_t bar, uint4 v) {
    asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.v4.b32 [%0], {%1, %2, %3, %4}, [%5];"
                 :: "r"(to), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w), "r"(bar) : "memory");
}

// A lane's four tokens of one channel, the first n of them, to rows st apart; neighbouring lanes
// have neighbouring channels.  vec (bf16, all lanes, rows on 16 bytes): four lanes trade, and each
// stores four channels of one token (by stores of two bytes 64 tokens took 0.6 us longer).
template <typename T>
__device__ __forceinline__ void i8_put4(T *to, int64_t st, int n, const float (&v)[4], bool vec) {
    if constexpr (sizeof(T) == 2) {
        if (vec) {
            const bool odd = threadIdx.x & 1, up = threadIdx.x & 2;
            const uint32_t lo = pack_bf2(v[0], v[1]), hi = pack_bf2(v[2], v[3]);
            uint32_t got = __shfl_xor_sync(0xffffffffu, odd ? lo : hi, 1);
            const uint32_t left = odd ? got : lo, right = odd ? hi : got;       // two tokens' channels
            const uint32_t first = __byte_perm(left, right, 0x5410), second = __byte_perm(left, right, 0x7632);
            got = __shfl_xor_sync(0xffffffffu, up ? first : second, 2);
            const int i = 2 * odd + up;
            if (i < n)
                *reinterpret_cast<uint2 *>(to + i * st - (threadIdx.x & 3)) =
                    up ? make_uint2(got, second) : make_uint2(first, got);
            return;
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (i < n) to[i * st] = from_f32<T>(v[i]);
}

// Sums of a thread's outputs over the chunks: fp32 while they stay within kI8Near, so that the
// next chunk's addition is exact, which ordinary codes never leave.  A warp in which one does
// moves its sums to int32 words in local memory (a conversion to integers runs at an eighth of
// the rate of an addition, and as many registers again are not to be had).
template <int N> struct ExactSums {
    float s[N];
    float big;                                   // largest |s| since the last look
    volatile int32_t far[N];
    bool moved;

    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int i = 0; i < N; ++i) s[i] = 0.f;
        big = 0.f;
        moved = false;
    }
    // adds W whole numbers, sums of a chunk, to the elements from `at` on
    template <int W> __device__ __forceinline__ void add(int at, const float (&v)[W]) {
#pragma unroll
        for (int j = 0; j < W; j += 2) {
            const float2 t = add_f32x2(make_float2(s[at + j], s[at + j + 1]), make_float2(v[j], v[j + 1]));
            s[at + j] = t.x;
            s[at + j + 1] = t.y;
            big = fmaxf(big, fmaxf(fabsf(t.x), fabsf(t.y)));
        }
    }
    // after every chunk
    __device__ __forceinline__ void settle() {
        if (__any_sync(0xffffffffu, big > kI8Near)) {
#pragma unroll
            for (int i = 0; i < N; ++i) {
                far[i] = (moved ? far[i] : 0) + __float2int_rn(s[i]);
                s[i] = 0.f;
            }
            moved = true;
        }
        big = 0.f;
    }
    // s + kRaised (mod 2^32): |s| <= 2^21 after a chunk, so added to 1.5 * 2^23 it is the low bits
    // of the sum
    static constexpr uint32_t kRaised = 0x4b400000;
    __device__ __forceinline__ uint32_t raised(int i) const { return __float_as_uint(__fadd_rn(s[i], 12582912.f)); }
    __device__ __forceinline__ int32_t whole(int i) const {
        return (int32_t)((moved ? (uint32_t)far[i] : 0u) + raised(i) - kRaised);
    }
    // makes s the sums, rounded once, or where they have moved leaves all of them in `far`
    __device__ __forceinline__ void finish(bool stay = false) {
        if (!__any_sync(0xffffffffu, moved)) return;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            if (stay) far[i] = whole(i);
            else s[i] = (float)whole(i);
        }
    }
};

// ------------------------------------------------------------------ up to 64 tokens
//
// A CTA makes 128 channels x NT tokens over a range of K; the CTAs of a cluster share a tile
// by ranges of K.  Each sends its int32 sums to the CTA that adds them up, one of its share of
// the channels (reading the others' memory between two barriers took 2 us longer at 64 tokens).
// Tokens are converted into fp16 tiles in shared memory.
// Measured, 16480 channels of 5120: 16 tokens 18.3 us, 64 tokens 23.9 us, where HBM takes 12.5:
// each step's chain (copy, codes out of shared memory, conversion, TMEM, products) is waited for
// with two CTAs an SM; issue slots are 54% busy, the tensor pipe 16%.  5120 channels of 6144 make
// 160 CTAs, mostly one an SM, with 12 steps each: 16 tokens 11.7 us, 64 tokens 16.1 (HBM: 4.7).
// More converting warps shorten no chain and take the registers (16 of 56 registers took 3.6 us
// longer at 64 tokens, 16480 channels).
template <int NT>
__global__ void __launch_bounds__(kI8Threads, I8Shape<NT>::CTAS)
matmul_i8_tc_kernel(const __grid_constant__ I8Maps maps, const __grid_constant__ MatmulParams p, int tiles_m) {
    using Sh = I8Shape<NT>;
    constexpr int HALF = NT / 2;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    I8Smem<NT> &S = *reinterpret_cast<I8Smem<NT> *>(smem_raw);
    if (tc::smem_u32(smem_raw) & 1023u) {        // the tiles' swizzle needs it; never seen
        if (threadIdx.x == 0) report(p.status, GDN_ERR_CUDA);
        return;
    }
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t rank = cluster_rank(), parts = cluster_size();
    const int tile = blockIdx.x / parts;
    const int m0 = (tile % tiles_m) * NT, n0 = (tile / tiles_m) * kI8Channels;
    const int all = (p.K + kI8Step - 1) / kI8Step;
    const int first = (int)((int64_t)all * rank / parts), n = (int)((int64_t)all * (rank + 1) / parts) - first;
    const int chunks = (n + kI8Exact - 1) / kI8Exact;
    volatile int *abort = &S.abort;

    if (warp == 0) {
        tc::tmem_alloc(&S.tmem, Sh::COLS);
        tc::tmem_relinquish();
    }
    if (tid == 0) {
        S.abort = 0;
        for (int i = 0; i < Sh::STAGES; ++i) {
            tc::mbar_init(&S.raw_full[i], 1);
            tc::mbar_init(&S.raw_free[i], kI8ConvWarps);
        }
        for (int i = 0; i < 2; ++i) {
            tc::mbar_init(&S.ab_full[i], kI8ConvWarps);
            tc::mbar_init(&S.ab_free[i], 1);
            tc::mbar_init(&S.d_full[i], 1);
            tc::mbar_init(&S.d_free[i], kI8ConvWarps);
        }
        tc::mbar_init(&S.sums_full, 1);
        tc::mbar_fence_init();
        if (parts > 1) tc::mbar_expect_tx(&S.sums_full, NT * kI8Channels * 4);
        tc::prefetch_tmap(&maps.w);
        tc::prefetch_tmap(&maps.a);
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = S.tmem;
    grid_dependents_launch();
    // codes of w on their way to L2 while the kernel before this one ends
    if (tid < Sh::STAGES && tid < n) prefetch_2d(&maps.w, (first + tid) * kI8Step, n0);
    __syncwarp();
    grid_dependency_wait();

    // scales for the end: those of the channel that this thread then stores, and the tokens'
    const int share = kI8Channels / parts, share_log = __ffs(share) - 1;
    const int64_t own = n0 + rank * share + (tid & (share - 1));
    const float ws = own < p.N ? p.w_scale[own] : 0.f, bias = own < p.N ? matmul_bias(p, own) : 0.f;
    for (int i = tid; i < NT; i += kI8Threads) S.scale[i] = p.a_scale[min((int64_t)m0 + i, p.M - 1)];
    ExactSums<HALF> sums;                        // this thread's channel, half of the tokens
    sums.clear();
    const int row = 32 * (warp & 3) + lane, half = warp >> 2;

    if (warp < kI8ConvWarps) {
        const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
        // sums of the products of chunk c, which are whole numbers up to 2^24
        auto drain = [&](int c) {
            if (!i8_wait(&S.d_full[c & 1], (c >> 1) & 1, abort)) return;
            tc::fence_after_sync();
            const uint32_t at = tmem + lanes + (c & 1) * NT + half * HALF;
            constexpr int W = HALF < 16 ? 8 : 16;
#pragma unroll
            for (int i = 0; i < HALF; i += W) {
                float v[W];
                if constexpr (W == 8) tc::tmem_ld8(at + i, v);
                else tc::tmem_ld16(at + i, v);
                tc::tmem_wait_ld();
                sums.add(i, v);
            }
            tc::fence_before_sync();
            __syncwarp();
            if (lane == 0) i8_arrive(&S.d_free[c & 1]);
            sums.settle();
        };
        int drained = 0;
        bool ok = true;
        for (int s = 0; s < n; ++s) {
            const int slot = s % Sh::STAGES, buf = s & 1;
            if (!(ok = i8_wait(&S.raw_full[slot], (s / Sh::STAGES) & 1, abort))) break;
            if (s >= 2 && !(ok = i8_wait(&S.ab_free[buf], ((s >> 1) - 1) & 1, abort))) break;
            tc::fence_after_sync();
            // channels: half a step of this thread's row
#pragma unroll
            for (int c = 0; c < 4; c += 2) {
                uint32_t r[16];
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    i8_halves16(*reinterpret_cast<const uint4 *>(S.raw_w[slot] + tc::swz(row, 4 * half + c + i)),
                                r + 8 * i);
                i8_st16(tmem + lanes + Sh::COL_A + 64 * buf + 32 * half + 8 * c, r);
            }
            // Tokens: a warp takes eight rows of one 64-code block.  Eight lanes take four chunks
            // of rows r and r ^ 5, whose swizzled places differ both where they are read
            // (chunks 0-3 or 4-7) and where they are written (even or odd chunks).
#pragma unroll
            for (int u = warp; u < NT / 4; u += kI8ConvWarps) {
                const int blk = u & 1, t = 8 * (u >> 1) + ((lane >> 3) ^ (lane & 4 ? 5 : 0)), c = lane & 3;
                uint32_t r[8];
                i8_halves16(*reinterpret_cast<const uint4 *>(S.raw_a[slot] + tc::swz(t, 4 * blk + c)), r);
                uint8_t *dst = S.conv[buf] + blk * NT * 128;
                *reinterpret_cast<uint4 *>(dst + tc::swz(t, 2 * c)) = make_uint4(r[0], r[1], r[2], r[3]);
                *reinterpret_cast<uint4 *>(dst + tc::swz(t, 2 * c + 1)) = make_uint4(r[4], r[5], r[6], r[7]);
            }
            tc::fence_async_smem();
            tc::tmem_wait_st();
            tc::fence_before_sync();
            __syncwarp();
            if (lane == 0) {
                i8_arrive(&S.raw_free[slot]);
                i8_arrive(&S.ab_full[buf]);
            }
            // a chunk is fetched while the next one's first steps run
            if (s % kI8Exact == 1 && s > kI8Exact) drain(drained++);
        }
        __syncwarp();
        cluster_arrive_relaxed();                // of this warp's copied codes all are used
        while (ok && drained < chunks) drain(drained++);
    } else if (warp == kI8ConvWarps) {
        int issued = 0;
        for (int s = 0; s < n; ++s) {
            const int slot = s % Sh::STAGES;
            if (s >= Sh::STAGES && !i8_wait(&S.raw_free[slot], ((s / Sh::STAGES) - 1) & 1, abort)) break;
            if (lane == 0) {
                tc::mbar_expect_tx(&S.raw_full[slot], Sh::RAW_W + Sh::RAW_A);
                load_2d(S.raw_w[slot], &maps.w, &S.raw_full[slot], (first + s) * kI8Step, n0);
                load_2d(S.raw_a[slot], &maps.a, &S.raw_full[slot], (first + s) * kI8Step, m0);
            }
            __syncwarp();
            issued = s + 1;
        }
        // nothing may land after the CTA has left
        for (int s = max(0, issued - Sh::STAGES); s < issued; ++s)
            wait_bounded_poll<0>(&S.raw_full[s % Sh::STAGES], (s / Sh::STAGES) & 1, nullptr);
        __syncwarp();
        cluster_arrive_relaxed();
    } else {
        const uint32_t id = i8_idesc(kI8Channels, NT);
        for (int s = 0; s < n; ++s) {
            const int buf = s & 1, c = s / kI8Exact;
            if (s % kI8Exact == 0 && c >= 2 && !i8_wait(&S.d_free[c & 1], ((c >> 1) - 1) & 1, abort)) break;
            if (!i8_wait(&S.ab_full[buf], (s >> 1) & 1, abort)) break;
            tc::fence_after_sync();
#pragma unroll
            for (int k = 0; k < kI8Step / 16; ++k)
                i8_mma(tmem + (c & 1) * NT, tmem + Sh::COL_A + 64 * buf + 8 * k,
                       tc::sdesc(tc::smem_u32(S.conv[buf] + (k >> 2) * NT * 128 + (k & 3) * 32), 0, 1024), id,
                       s % kI8Exact != 0 || k > 0);
            tc::mma_commit_warp(&S.ab_free[buf]);
            if (s % kI8Exact == kI8Exact - 1 || s == n - 1) tc::mma_commit_warp(&S.d_full[c & 1]);
        }
        __syncwarp();
        cluster_arrive_relaxed();
    }
    __syncwarp();
    cluster_wait();                              // no CTA's ring is in use

    static_assert(kI8ConvWarps == 8, "thread i of the converting warps has channel i mod 128 both ways");
    __syncthreads();                             // the scales are there
    const int rows = (int)min((int64_t)NT, p.M - m0);
    const bool vec = p.out_vec && n0 + kI8Channels <= p.N;
    auto put4 = [&](int t, const float (&v)[4]) {
        const int n = own < p.N ? rows - t : 0;
        const int64_t at = ((int64_t)m0 + t) * p.out_st + own;
        if (p.out_f32) i8_put4((float *)p.out + at, p.out_st, n, v, vec);
        else i8_put4((bf16 *)p.out + at, p.out_st, n, v, vec);
    };
    if (parts == 1) {
        sums.finish();
        if (warp < kI8ConvWarps)
#pragma unroll
            for (int i = 0; i < HALF; i += 4) {
                float v[4];
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    v[j] = matmul_value(sums.s[i + j], S.scale[half * HALF + i + j], ws, bias);
                put4(half * HALF + i, v);
            }
    } else {
        // Over the codes that have all been used: sums, raised, as [CTA][four tokens][channel of the
        // share].
        // They are sent whatever went wrong before, so that none is on its way to a CTA that left.
        uint4 *in = reinterpret_cast<uint4 *>(S.raw_w);
        static_assert(NT * kI8Channels * 4 <= sizeof(S.raw_w), "the sums fit");
        if (warp < kI8ConvWarps) {
            const uint32_t to = row >> share_log, bar = cluster_addr(&S.sums_full, to);
            const uint32_t at = cluster_addr(in + ((rank * (NT / 4) + half * (HALF / 4)) << share_log) +
                                             (row & (share - 1)), to);
            if (sums.moved)
#pragma unroll
                for (int i = 0; i < HALF; ++i) sums.far[i] = (int32_t)((uint32_t)sums.far[i] + sums.raised(i));
#pragma unroll
            for (int i = 0; i < HALF; i += 4) {
                uint4 v = make_uint4(sums.raised(i), sums.raised(i + 1), sums.raised(i + 2), sums.raised(i + 3));
                if (sums.moved) v = make_uint4(sums.far[i], sums.far[i + 1], sums.far[i + 2], sums.far[i + 3]);
                cluster_put(at + (i * 4 << share_log), bar, v);
            }
        }
        __syncwarp();
        cluster_arrive_relaxed();
        if (warp < kI8ConvWarps) {
            if (!wait_bounded_poll<0>(&S.sums_full, 0, nullptr)) *abort = 1;
            // (a warp's threads all or none: their number is a multiple of 32)
#pragma unroll 1
            for (int g = tid >> share_log; g < NT / 4; g += 32 * kI8ConvWarps >> share_log) {
                const uint4 *at = in + (g << share_log) + (tid & (share - 1));
                uint32_t sum[4] = {};
#pragma unroll 2
                for (int r = 0; r < parts; ++r, at += NT / 4 << share_log) {
                    const uint4 u = *at;
                    sum[0] += u.x - sums.kRaised;
                    sum[1] += u.y - sums.kRaised;
                    sum[2] += u.z - sums.kRaised;
                    sum[3] += u.w - sums.kRaised;
                }
                float v[4];
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    v[j] = matmul_value((float)(int32_t)sum[j], S.scale[4 * g + j], ws, bias);
                put4(4 * g, v);
            }
        }
        __syncwarp();
        cluster_wait();                          // every CTA has sent
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    if (warp == 0) tc::tmem_dealloc(tmem, Sh::COLS);
    if (tid == 0 && *abort) report(p.status, GDN_ERR_TIMEOUT);
}

// ------------------------------------------------------------------ pairs of CTAs
//
// Many tokens: two CTAs of a cluster make 256 channels x NT tokens (NT = 128 or 256) with one
// cta_group::2 product.  Each converts its own 128 channels into its TMEM and holds half of
// the tokens in shared memory, as fp16 that a kernel before this one wrote: converting tokens
// here as well would take 512 clocks of shared memory for 64 codes (128 bytes a clock: codes
// and fp16 in, fp16 out to the tensor core), as many as their products take; without it they
// take 320.  A product of 16 codes takes 128 clocks for 256 tokens and no less for fewer
// (operand A leaves TMEM at 32 bytes a clock), so a tile has as many tokens as there are.
//
// 256 columns of sums and four steps of operand A fill TMEM, so moving sums every 896 products
// would leave the tensor core waiting a fifth of the time.  Most tiles need no move: with
// |a|^2 and |w|^2 the sums of squares of a token's and a channel's codes, every partial sum is
// at most |a||w| (Cauchy and Schwarz), and where that is at most 2^24 fp32 sums are exact to
// the end.  |a|^2 comes with the fp16 tokens, |w|^2 from the converting warps when a tile is
// done.  Units that turn out otherwise are made again with moves, after all others; those whose
// tokens alone are above kPairCareful are made so at once.  Which it is changes no result.
//
// Persistent: a pair takes units in turn.  A unit is a tile; those tiles that are left when
// every pair has had the same number are cut along K into PairShape::parts units each, whose
// int32 sums go to the workspace and are added up by a kernel after this one.  Warps 0-7 move
// sums (a thread: one channel, half of the tokens), 8-11 convert, 12 copies, 13 issues products
// (in the first CTA of a pair).
// Measured, 16480 channels of 5120: 4096 tokens 344 us (2000 TFLOP/s) for a few calls and 371 to
// 379 in a long run of them, where power limits the clock (1850; a library bf16 product's rate is
// 1905), 1024 tokens 97 us (1770; the tensor pipe is 78% busy), 256 tokens 33 us, of which some 11
// are the tokens' kernel, the first copies and the sums' way out.  Where the tiles are fewer than
// the pairs and no cut pays, pairs stay idle: 500 tokens of 5120 channels of 6144, 37 us, are 40
// tiles for 76 pairs.
constexpr int kPairSumWarps = 8, kPairConvWarps = 4, kPairMaxStages = 4;
constexpr int kPairThreads = 32 * (kPairSumWarps + kPairConvWarps + 4);  // two warps idle
constexpr int kPairTokens = 256;                 // most tokens of a tile
constexpr int kPairCareful = 15000000;           // |a|^2: with a like |w|^2, near 2^24 squared
constexpr int kPairMarks = 1024;                 // units of a pair with marks of their own

struct PairShape {                               // of a launch
    int NT, stages;                              // TMEM: 256 columns of sums, 64 a stage
    uint32_t stage_bytes;                        // codes, then two 64-code blocks of tokens
    int tiles_m, steps;                          // tiles along the tokens; steps of K
    int full, parts, units;                      // whole tiles; units of each other tile; all units
    const int32_t *squares;                      // |a|^2 of the tokens
    int32_t *sums;                               // [unit - full][64 fours of tokens][256 channels][4]
};
struct PairUnit {
    int tile, first, last;                       // steps of K
    bool whole;
};
__device__ __forceinline__ PairUnit pair_unit(const PairShape &sh, int unit) {
    if (unit < sh.full) return {unit, 0, sh.steps, true};
    const int j = unit - sh.full, part = j % sh.parts;
    return {sh.full + j / sh.parts, sh.steps * part / sh.parts, sh.steps * (part + 1) / sh.parts, false};
}
struct PairBars {
    uint64_t full[kPairMaxStages], conv[kPairMaxStages], free[kPairMaxStages], d_full[2], d_free[2];
    uint32_t again[kPairMarks / 32];             // units to make again (the last mark: any after it too)
    uint32_t any;                                // whether there are any
    uint32_t tmem;
    int abort;
};
constexpr uint32_t kPairRaw = kI8Channels * kI8Step;
constexpr uint32_t kPairRing = 192 * 1024;
// Of a sums' warp, on the way out: 16 tokens of 32 channels as bf16 pairs of tokens (12 words a
// channel, 8 more after every eighth, so that neither the channels' rows nor a pair of eight
// channels meet in a bank), and the tokens' scales.
struct PairOut {
    uint32_t pairs[32 * 12 + 3 * 8];
    float tokens[8][16];                         // of the warp's groups
};
constexpr int kPairSmem = (int)(kPairRing + kPairSumWarps * sizeof(PairOut) + sizeof(PairBars));

// Largest |a|^2 of the tile's tokens (a warp).  The kernel before this one writes them while this
// one is already there, so the loads are not of the read-only kind.
__device__ __forceinline__ int32_t pair_squares(const PairShape &sh, int64_t M, int tile) {
    const int64_t m0 = (int64_t)(tile % sh.tiles_m) * sh.NT;
    int32_t most = 0;
#pragma unroll
    for (int i = 0; i < kPairTokens / 32; ++i) {
        const int64_t m = m0 + 32 * i + (threadIdx.x & 31);
        if (32 * i < sh.NT && m < M) most = max(most, sh.squares[m]);
    }
    return __reduce_max_sync(0xffffffffu, most);
}
// Marks the pair's unit `turn` in both CTAs' lists, or looks it up in this one's.
__device__ __forceinline__ void pair_mark(PairBars &S, int turn) {
    turn = min(turn, kPairMarks - 1);
#pragma unroll
    for (uint32_t r = 0; r < 2; ++r) {
        uint32_t at, any;
        asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(tc::smem_u32(&S.again[turn >> 5])), "r"(r));
        asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(any) : "r"(tc::smem_u32(&S.any)), "r"(r));
        asm volatile("red.shared::cluster.or.b32 [%0], %1;" :: "r"(at), "r"(1u << (turn & 31)) : "memory");
        asm volatile("red.shared::cluster.or.b32 [%0], 1;" :: "r"(any) : "memory");
    }
}
__device__ __forceinline__ bool pair_marked(const PairBars &S, int turn) {
    turn = min(turn, kPairMarks - 1);
    return (*(volatile const uint32_t *)&S.again[turn >> 5] >> (turn & 31)) & 1;
}

__device__ __forceinline__ void pair_mma(uint32_t d, uint32_t a, uint64_t b, uint32_t id, uint32_t add) {
    asm volatile("{\n\t.reg .pred p, e;\n\t"
                 "elect.sync _|e, 0xffffffff;\n\t"
                 "setp.ne.b32 p, %4, 0;\n\t"
                 "@e tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n\t}"
                 :: "r"(d), "r"(a), "l"(b), "r"(id), "r"(add) : "memory");
}
// Arrives on the barrier of both CTAs when the products issued so far are done.
__device__ __forceinline__ void pair_commit(uint64_t *bar) {
    asm volatile("{\n\t.reg .pred e;\n\t.reg .b16 m;\n\t"
                 "mov.b16 m, 3;\n\t"
                 "elect.sync _|e, 0xffffffff;\n\t"
                 "@e tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], m;\n\t}"
                 :: "r"(tc::smem_u32(bar)) : "memory");
}
// Arrives on the first CTA's barrier.  What it announces is ordered by tcgen05's own waits and
// fences; with release.cluster the arrival alone would take 1300 clocks.
__device__ __forceinline__ void pair_arrive(uint64_t *bar) {
    uint32_t first;
    asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(first) : "r"(tc::smem_u32(bar)));
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" :: "r"(first) : "memory");
}

template <int N> __device__ __forceinline__ void regs_up() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" :: "n"(N));
}
template <int N> __device__ __forceinline__ void regs_down() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" :: "n"(N));
}
// Registers a thread at launch, and then of the sums' warps, the converting ones and the rest;
// a raise waits until the other warps' cuts cover it.  The ring leaves hardly any L1, so a value
// that goes to local memory comes back from L2: with 176, 96 and 64, 42 of the sums' warps' did,
// and 256 tokens of 16480 channels of 5120 took 38 us (34).
constexpr int kPairRegs = 128, kPairSumRegs = 200, kPairConvRegs = 72, kPairRestRegs = 40;
static_assert(2 * kPairSumRegs + kPairConvRegs + kPairRestRegs <= 4 * kPairRegs, "a raise waits forever");

// Group i of a thread's sums: a choice of one in eight by halves.
template <int LO, int N>
__device__ __forceinline__ void pair_take(float (&v)[16], const float (&s)[128], int i) {
    if constexpr (N == 1) {
#pragma unroll
        for (int j = 0; j < 16; ++j) v[j] = s[16 * LO + j];
    } else if (i < LO + N / 2) {
        pair_take<LO, N / 2>(v, s, i);
    } else {
        pair_take<LO + N / 2, N / 2>(v, s, i);
    }
}

// Stores the results of 16 tokens and this lane's channel; m, n: the first token, the channel.
// As bf16 in rows on 16 bytes a lane takes eight channels of two tokens, by way of shared memory
// in pairs (as sums, four bytes each, 500 tokens of 10240 channels of 5120 took 0.5 us longer).
__device__ __forceinline__ void pair_store(const MatmulParams &p, PairOut &o, int64_t m, int64_t n, const float (&v)[16]) {
    const int lane = threadIdx.x & 31, rows = (int)min(p.M - m, (int64_t)16);
    if (p.out_f32 || !p.out_vec || n - lane + 32 > p.N) {
        if (n < p.N)
#pragma unroll
            for (int i = 0; i < 16; ++i)
                if (i < rows) matmul_store(p, m + i, n, v[i]);
        return;
    }
    uint4 *to = reinterpret_cast<uint4 *>(o.pairs + lane * 12 + (lane >> 3) * 8);
    to[0] = make_uint4(pack_bf2(v[0], v[1]), pack_bf2(v[2], v[3]), pack_bf2(v[4], v[5]), pack_bf2(v[6], v[7]));
    to[1] = make_uint4(pack_bf2(v[8], v[9]), pack_bf2(v[10], v[11]), pack_bf2(v[12], v[13]), pack_bf2(v[14], v[15]));
    __syncwarp();
    const int c = 8 * (lane & 3), j = lane >> 2;
    const uint32_t *from = o.pairs + c * 12 + c + j;
    uint32_t w[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) w[e] = from[12 * e];
    bf16 *out = (bf16 *)p.out + (m + 2 * j) * p.out_st + (n - lane) + c;
#pragma unroll
    for (int x = 0; x < 2; ++x) {
        const uint32_t half = x ? 0x7632 : 0x5410;
        if (2 * j + x < rows)
            *reinterpret_cast<uint4 *>(out + x * p.out_st) =
                make_uint4(__byte_perm(w[0], w[1], half), __byte_perm(w[2], w[3], half),
                           __byte_perm(w[4], w[5], half), __byte_perm(w[6], w[7], half));
    }
    __syncwarp();
}

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kPairThreads, 1)
matmul_i8_pair_kernel(const __grid_constant__ I8Maps maps, const __grid_constant__ MatmulParams p,
                      const __grid_constant__ PairShape sh) {
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    PairBars &S = *reinterpret_cast<PairBars *>(smem_raw + (kPairSmem - sizeof(PairBars)));
    if (tc::smem_u32(smem_raw) & 1023u) {        // the tiles' swizzle needs it; never seen
        if (threadIdx.x == 0) report(p.status, GDN_ERR_CUDA);
        return;
    }
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int rank = (int)cluster_rank(), pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
    const int NT = sh.NT, stages = sh.stages;
    const int buffers = NT <= 128 ? 2 : 1;       // of sums
    volatile int *abort = &S.abort;

    if (warp == 0) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;"
                     :: "r"(tc::smem_u32(&S.tmem)) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
    if (tid == 0) {
        S.abort = 0;
        for (int i = 0; i < kPairMaxStages; ++i) {
            tc::mbar_init(&S.full[i], 1);
            tc::mbar_init(&S.conv[i], 2 * kPairConvWarps);
            tc::mbar_init(&S.free[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            tc::mbar_init(&S.d_full[i], 1);
            tc::mbar_init(&S.d_free[i], 2 * kPairSumWarps);
        }
        for (int i = 0; i < kPairMarks / 32; ++i) S.again[i] = 0;
        S.any = 0;
        tc::mbar_fence_init();
        tc::prefetch_tmap(&maps.w);
        tc::prefetch_tmap(&maps.a);
    }
    tc::fence_before_sync();
    __syncthreads();
    cluster_sync();
    tc::fence_after_sync();
    const uint32_t tmem = S.tmem;
    grid_dependents_launch();
    // codes of w on their way to L2 while the kernel before this one ends
    if (tid < stages) {
        const PairUnit u = pair_unit(sh, pair);
        if (u.first + tid < u.last)
            prefetch_2d(&maps.w, (u.first + tid) * kI8Step, u.tile / sh.tiles_m * 256 + 128 * rank);
    }
    __syncwarp();

    // Every role goes over the pair's units twice; the second time over those marked by then.
    if (warp < kPairSumWarps) {
        regs_up<kPairSumRegs>();
        grid_dependency_wait();
        // groups of 16 columns: this warp has q, q + 2, ..
        const int q = warp >> 2, row = 32 * (warp & 3) + lane, groups = NT / 16;
        const uint32_t at = tmem + ((uint32_t)(32 * (warp & 3)) << 16) + 16 * q;
        uint32_t c = 0;                          // chunks so far
        bool ok = true;
        ExactSums<128> sums;
        PairOut &out = reinterpret_cast<PairOut *>(smem_raw + kPairRing)[warp];
        for (int pass = 0; pass < 2; ++pass) {
            for (int unit = pair, turn = 0; unit < sh.units && ok; unit += pairs, ++turn) {
                if (pass && !pair_marked(S, turn)) continue;
                const PairUnit u = pair_unit(sh, unit);
                const int steps = u.last - u.first;
                const int64_t n = (int64_t)(u.tile / sh.tiles_m) * 256 + 128 * rank + row;
                const int64_t m0 = (int64_t)(u.tile % sh.tiles_m) * NT;
                const int chunk = pass || pair_squares(sh, p.M, u.tile) > kPairCareful ? kI8Exact : steps;
                float ws = 0.f, bias = 0.f;
                if (u.whole) {
                    if (n < p.N) ws = p.w_scale[n], bias = matmul_bias(p, n);
#pragma unroll
                    for (int i = lane >> 4; i < 8; i += 2)
                        out.tokens[i][lane & 15] = p.a_scale[min(m0 + 16 * (q + 2 * i) + (lane & 15), p.M - 1)];
                }
                sums.clear();
                for (int s = 0; s < steps && ok; s += chunk) {
                    const int buf = c & (buffers - 1);
                    if (!(ok = i8_wait<20>(&S.d_full[buf], (c / buffers) & 1, abort))) break;
                    ++c;
                    tc::fence_after_sync();
                    if (chunk >= steps) {            // all there is
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            if (q + 2 * i < groups) tc::tmem_ld16(at + buf * 128 + 32 * i, sums.s + 16 * i);
                        tc::tmem_wait_ld();
                    } else {
                        float v[2][16];
                        tc::tmem_ld16(at + buf * 128, v[0]);
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            if (q + 2 * i >= groups) continue;
                            tc::tmem_wait_ld();
                            if (i < 7 && q + 2 * i + 2 < groups)
                                tc::tmem_ld16(at + buf * 128 + 32 * (i + 1), v[(i + 1) & 1]);
                            sums.add(16 * i, v[i & 1]);
                        }
                    }
                    tc::fence_before_sync();
                    __syncwarp();
                    if (lane == 0) pair_arrive(&S.d_free[buf]);
                    if (chunk < steps) sums.settle();
                }
                if (!ok) break;
                if (chunk < steps) sums.finish(!u.whole);
                int4 *to = reinterpret_cast<int4 *>(sh.sums) + ((int64_t)(unit - sh.full) << 14) + 128 * rank + row;
                if (!u.whole && sums.moved) {
                    for (int i = 0; i < 32; ++i) {
                        const int tok = 16 * (q + 2 * (i >> 2)) + 4 * (i & 3);
                        if (tok < NT && m0 + tok < p.M)
                            to[tok / 4 * 256] = make_int4(sums.far[4 * i], sums.far[4 * i + 1], sums.far[4 * i + 2],
                                                          sums.far[4 * i + 3]);
                    }
                } else if (!u.whole) {
#pragma unroll
                    for (int i = 0; i < 32; ++i) {
                        const int tok = 16 * (q + 2 * (i >> 2)) + 4 * (i & 3);
                        if (tok < NT && m0 + tok < p.M)
                            to[tok / 4 * 256] =
                                make_int4(__float2int_rn(sums.s[4 * i]), __float2int_rn(sums.s[4 * i + 1]),
                                          __float2int_rn(sums.s[4 * i + 2]), __float2int_rn(sums.s[4 * i + 3]));
                    }
                } else {
#pragma unroll 1
                    for (int i = 0; i < 8; ++i) {
                        const int tok = 16 * (q + 2 * i);
                        if (tok >= NT || m0 + tok >= p.M) break;
                        float v[16];
                        pair_take<0, 8>(v, sums.s, i);
#pragma unroll
                        for (int j = 0; j < 16; ++j) v[j] = matmul_value(v[j], out.tokens[i][j], ws, bias);
                        pair_store(p, out, m0 + tok, n, v);
                    }
                }
                __syncwarp();
            }
            __syncwarp();
            tc::fence_before_sync();
            cluster_arrive_relaxed();            // no other warp reads what this one stored
            cluster_wait();
            if (*(volatile uint32_t *)&S.any == 0) break;
        }
    } else if (warp < kPairSumWarps + kPairConvWarps) {
        regs_down<kPairConvRegs>();
        grid_dependency_wait();
        const int row = 32 * (warp & 3) + lane;
        const uint32_t at = tmem + ((uint32_t)(32 * (warp & 3)) << 16) + 256;
        int slot = 0;
        uint32_t round = 0;
        bool ok = true;
        for (int pass = 0; pass < 2; ++pass) {
            for (int unit = pair, turn = 0; unit < sh.units && ok; unit += pairs, ++turn) {
                if (pass && !pair_marked(S, turn)) continue;
                const PairUnit u = pair_unit(sh, unit);
                const int32_t tokens = pass ? 0 : pair_squares(sh, p.M, u.tile);
                int32_t squares = 0;             // of this thread's channel
                for (int s = u.first; s < u.last; ++s) {
                    if (!(ok = i8_wait(&S.full[slot], round & 1, abort))) break;
                    tc::fence_after_sync();
                    const uint8_t *raw = smem_raw + slot * sh.stage_bytes;
                    uint4 codes[8];
#pragma unroll
                    for (int c = 0; c < 8; ++c) codes[c] = *reinterpret_cast<const uint4 *>(raw + tc::swz(row, c));
#pragma unroll
                    for (int c = 0; c < 8; c += 2) {
                        uint32_t r[16];
                        i8_halves16(codes[c], r);
                        i8_halves16(codes[c + 1], r + 8);
                        i8_st16(at + 64 * slot + 8 * c, r);
                    }
#pragma unroll
                    for (int c = 0; c < 8; ++c) {
                        squares = __dp4a((int)codes[c].x, (int)codes[c].x, squares);
                        squares = __dp4a((int)codes[c].y, (int)codes[c].y, squares);
                        squares = __dp4a((int)codes[c].z, (int)codes[c].z, squares);
                        squares = __dp4a((int)codes[c].w, (int)codes[c].w, squares);
                    }
                    tc::tmem_wait_st();
                    tc::fence_before_sync();
                    __syncwarp();
                    if (lane == 0) pair_arrive(&S.conv[slot]);
                    if (++slot == stages) slot = 0, ++round;
                }
                // 2^48 less what the product's rounding could hide
                const bool far = (float)squares * (float)tokens > 2.8147e14f;
                if (tokens <= kPairCareful && __any_sync(0xffffffffu, far) && lane == 0) pair_mark(S, turn);
            }
            __syncwarp();
            tc::fence_before_sync();
            cluster_sync();                      // the other CTA's products and arrivals are done
            if (*(volatile uint32_t *)&S.any == 0) break;
        }
    } else {
        regs_down<kPairRestRegs>();
        grid_dependency_wait();
        const bool copies = warp == kPairSumWarps + kPairConvWarps;
        const bool products = warp == kPairSumWarps + kPairConvWarps + 1 && rank == 0;
        const uint32_t bytes = kPairRaw + NT * 128, block = NT * 64, id = i8_idesc(256, NT);
        int slot = 0, issued = 0;
        uint32_t round = 0, c = 0;
        bool ok = true;
        for (int pass = 0; pass < 2; ++pass) {
            for (int unit = pair, turn = 0; (copies || products) && unit < sh.units && ok; unit += pairs, ++turn) {
                if (pass && !pair_marked(S, turn)) continue;
                const PairUnit u = pair_unit(sh, unit);
                if (copies) {
                    const int n0 = u.tile / sh.tiles_m * 256 + 128 * rank;
                    const int m0 = u.tile % sh.tiles_m * NT + NT / 2 * rank;
                    for (int s = u.first; s < u.last; ++s) {
                        if (round > 0 && !(ok = i8_wait(&S.free[slot], (round - 1) & 1, abort))) break;
                        if (lane == 0) {
                            uint8_t *to = smem_raw + slot * sh.stage_bytes;
                            tc::mbar_expect_tx(&S.full[slot], bytes);
                            load_2d(to, &maps.w, &S.full[slot], s * kI8Step, n0);
                            load_2d(to + kPairRaw, &maps.a, &S.full[slot], s * kI8Step, m0);
                            load_2d(to + kPairRaw + block, &maps.a, &S.full[slot], s * kI8Step + 64, m0);
                        }
                        __syncwarp();
                        if (issued < stages) ++issued;
                        if (++slot == stages) slot = 0, ++round;
                    }
                } else {
                    const int steps = u.last - u.first;
                    const int chunk = pass || pair_squares(sh, p.M, u.tile) > kPairCareful ? kI8Exact : steps;
                    for (int s = 0, left = 0; s < steps; ++s) {
                        const int buf = c & (buffers - 1);
                        const bool fresh = left == 0;
                        if (fresh) {
                            left = min(chunk, steps - s);
                            if (c >= (uint32_t)buffers && !(ok = i8_wait(&S.d_free[buf], (c / buffers - 1) & 1, abort))) break;
                        }
                        if (!(ok = i8_wait(&S.conv[slot], round & 1, abort))) break;
                        tc::fence_after_sync();
                        const uint32_t tok = tc::smem_u32(smem_raw + slot * sh.stage_bytes + kPairRaw);
#pragma unroll
                        for (int k = 0; k < kI8Step / 16; ++k)
                            pair_mma(tmem + buf * 128, tmem + 256 + 64 * slot + 8 * k,
                                     tc::sdesc(tok + (k >> 2) * block + (k & 3) * 32, 0, 1024), id, !fresh || k > 0);
                        pair_commit(&S.free[slot]);
                        if (--left == 0) {
                            pair_commit(&S.d_full[buf]);
                            ++c;
                        }
                        if (++slot == stages) slot = 0, ++round;
                    }
                }
            }
            if (products)                        // the other CTA's sums' warps have arrived
                for (uint32_t k = c < (uint32_t)buffers ? 0 : c - buffers; k < c && ok; ++k)
                    ok = i8_wait(&S.d_free[k & (buffers - 1)], (k / buffers) & 1, abort);
            __syncwarp();
            tc::fence_before_sync();
            cluster_sync();                      // the other CTA's products and arrivals are done
            if (*(volatile uint32_t *)&S.any == 0) break;
        }
        // nothing may land after the CTA has left
        for (int i = 0; i < issued; ++i) {
            if (--slot < 0) slot = stages - 1, --round;
            wait_bounded_poll<0>(&S.full[slot], round & 1, nullptr);
        }
    }
    tc::fence_after_sync();
    if (warp == 0)
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" :: "r"(tmem) : "memory");
    if (tid == 0 && *abort) report(p.status, GDN_ERR_TIMEOUT);
}

// The units' sums of tiles in parts, added up and scaled: a CTA takes four tokens of a tile, a
// thread a channel.
__global__ void __launch_bounds__(256) matmul_i8_join_kernel(const __grid_constant__ MatmulParams p,
                                                             const __grid_constant__ PairShape sh) {
    grid_dependents_launch();
    const int tile = sh.full + blockIdx.y;
    const int64_t n = (int64_t)(tile / sh.tiles_m) * 256 + threadIdx.x, m0 = (int64_t)(tile % sh.tiles_m) * sh.NT;
    grid_dependency_wait();
    if (n >= p.N) return;
    const float ws = p.w_scale[n], bias = matmul_bias(p, n);
    const int4 *from = reinterpret_cast<const int4 *>(sh.sums) + ((int64_t)blockIdx.y * sh.parts << 14) +
                       blockIdx.x * 256 + threadIdx.x;
    const int tok = blockIdx.x * 4;
    if (m0 + tok >= p.M) return;
    int32_t sum[4] = {0, 0, 0, 0};
#pragma unroll 4
    for (int j = 0; j < sh.parts; ++j) {
        const int4 v = from[(int64_t)j << 14];
        sum[0] += v.x;
        sum[1] += v.y;
        sum[2] += v.z;
        sum[3] += v.w;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (m0 + tok + i < p.M)
            matmul_store(p, m0 + tok + i, n, matmul_value((float)sum[i], p.a_scale[m0 + tok + i], ws, bias));
}

// Tokens' codes as fp16, rows `st` elements apart (a multiple of 8; what lies between K and st
// is not read), and the sums of their squares: a CTA per token, a thread takes eight codes, all
// at once for K up to 8192.  Latency bounds it (1024 tokens of 5120: 7 us alone, some of it
// beside the kernels before and after); a warp per token took 12 us longer at 500 tokens.
__global__ void __launch_bounds__(1024) matmul_i8_tokens_kernel(const int8_t *a, int64_t a_st, __half *out, int64_t st,
                                                               int32_t *squares, int32_t K, int vec) {
    __shared__ int32_t part[32];
    grid_dependents_launch();
    grid_dependency_wait();
    const int64_t m = blockIdx.x;
    int32_t sum = 0;
    for (int k = threadIdx.x * 8; k < K; k += blockDim.x * 8) {
        const int8_t *src = a + m * a_st + k;
        uint2 w = make_uint2(0, 0);
        if (vec && k + 8 <= K) {
            w = *reinterpret_cast<const uint2 *>(src);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (k + j < K) (j < 4 ? w.x : w.y) |= (uint32_t)(uint8_t)src[j] << (8 * (j & 3));
        }
        sum = __dp4a((int)w.x, (int)w.x, __dp4a((int)w.y, (int)w.y, sum));
        uint4 h;
        i8_halves(w.x, h.x, h.y);
        i8_halves(w.y, h.z, h.w);
        *reinterpret_cast<uint4 *>(out + m * st + k) = h;
    }
    sum = __reduce_add_sync(0xffffffffu, sum);
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = sum;
    __syncthreads();
    if (threadIdx.x < 32) {
        sum = __reduce_add_sync(0xffffffffu, threadIdx.x < blockDim.x >> 5 ? part[threadIdx.x] : 0);
        if (threadIdx.x == 0) squares[m] = sum;
    }
}

}  // namespace gdn

namespace gdn_host {

using namespace gdn;

namespace {

size_t up256(size_t n) { return (n + 255) / 256 * 256; }

int pair_tokens(int64_t M) { return M <= 128 ? 128 : 256; }

// Tiles, those made whole, and the units of each other one.  The parts along K are as many as
// make the last turns shortest; a turn's fill and its sums' way out cost about six steps and
// the join five (128 tokens of 5120 channels of 6144: whole 29 us, three parts 21; 500 tokens of
// the same: whole 40, three parts in two turns 48; all four are 2 to 4 us less since).
constexpr int kPairMaxParts = 12, kPairUnitCost = 6, kPairJoinCost = 5;
struct PairPlan {
    int64_t tiles, full;
    int parts;
};
PairPlan pair_plan(int64_t M, int64_t N, int64_t K, int pairs) {
    const int NT = pair_tokens(M);
    const int64_t steps = (K + kI8Step - 1) / kI8Step;
    PairPlan plan;
    plan.tiles = (M + NT - 1) / NT * ((N + 255) / 256);
    plan.full = plan.tiles;
    plan.parts = 1;
    if (pairs <= 0 || plan.tiles % pairs == 0) return plan;
    const int64_t left = plan.tiles % pairs;
    int64_t best = steps;
    for (int parts = 2; parts <= kPairMaxParts && parts * 2 <= steps; ++parts) {
        const int64_t turns = (left * parts + pairs - 1) / pairs,
                      cost = turns * ((steps + parts - 1) / parts + kPairUnitCost) + kPairJoinCost;
        if (cost < best) {
            best = cost;
            plan.parts = parts;
            plan.full = plan.tiles - left;
        }
    }
    return plan;
}

// Ranges of K of a tile of the cluster kernel: a power of two, up to eight, while all CTAs fit at
// once and the ranges have two steps each (one of them may have a single one); clusters of such
// sizes fit the device best (40 tiles: 13.7 us in fours, 17.1 in sevens).
int64_t few_parts(int64_t tiles, int64_t steps, int64_t ctas) {
    int64_t parts = 1;
    while (parts < 8 && 2 * parts * tiles <= ctas && 4 * parts <= steps + 1) parts *= 2;
    return parts;
}

template <int NT>
gdn_status_t launch_tc(const MatmulParams &p, cudaStream_t st) {
    using Sh = I8Shape<NT>;
    auto kern = matmul_i8_tc_kernel<NT>;
    constexpr int smem = sizeof(I8Smem<NT>);
    static_assert(Sh::CTAS * (smem + 1024) <= 228 * 1024, "the CTAs of an SM fit");
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
    if (!row_map(&maps.w, p.w, false, p.N, p.K, p.w_st, kI8Channels, true) ||
        !row_map(&maps.a, p.a, false, p.M, p.K, p.a_st, NT, true))
        return GDN_ERR_CUDA;
    const int64_t tiles_m = (p.M + NT - 1) / NT, tiles = tiles_m * ((p.N + kI8Channels - 1) / kI8Channels);
    const int64_t parts = few_parts(tiles, (p.K + kI8Step - 1) / kI8Step, (int64_t)sms * Sh::CTAS);
    if (tiles * parts > 0x7fffffff) return GDN_ERR_SHAPE;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(tiles * parts));
    cfg.blockDim = dim3(kI8Threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)parts;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kern, maps, p, (int)tiles_m) == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}
}  // namespace

gdn_status_t launch_matmul_i8_pair(const MatmulParams &p, void *ws, cudaStream_t st) {
    auto kern = matmul_i8_pair_kernel;
    constexpr int smem = kPairSmem;
    static_assert(smem <= 227 * 1024, "one CTA fits on an SM");
    static std::atomic<uint64_t> ready{0};   // one bit per device (beyond 63: set every time)
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return GDN_ERR_CUDA;
    if (dev > 63 || !((ready.load() >> dev) & 1u)) {
        cudaFuncAttributes built;
        if (cudaFuncGetAttributes(&built, kern) != cudaSuccess) return GDN_ERR_CUDA;
        if (built.numRegs != kPairRegs) return GDN_ERR_UNSUPPORTED;     // the raise would wait forever
        if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
            return GDN_ERR_CUDA;
        if (dev <= 63) ready.fetch_or(1ull << dev);
    }
    const int sms = matmul_sm_count(dev);
    if (sms <= 1) return GDN_ERR_CUDA;
    const int pairs = sms / 2, NT = pair_tokens(p.M);
    const PairPlan plan = pair_plan(p.M, p.N, p.K, pairs);
    if (plan.tiles > 0x3fffffff / kPairMaxParts) return GDN_ERR_SHAPE;
    gdn::PairShape sh;
    sh.NT = NT;
    sh.stage_bytes = gdn::kPairRaw + NT * 128;
    sh.stages = (int)(gdn::kPairRing / sh.stage_bytes);
    if (sh.stages > 4) sh.stages = 4;           // 64 of TMEM's columns each
    sh.tiles_m = (int)((p.M + NT - 1) / NT);
    sh.steps = (int)((p.K + kI8Step - 1) / kI8Step);
    sh.full = (int)plan.full;
    sh.parts = plan.parts;
    sh.units = (int)(plan.full + (plan.tiles - plan.full) * plan.parts);
    const int64_t half_st = ((int64_t)p.K + 7) / 8 * 8;
    int32_t *squares = (int32_t *)((uint8_t *)ws + up256((size_t)p.M * half_st * 2));
    sh.squares = squares;
    sh.sums = (int32_t *)((uint8_t *)squares + up256((size_t)p.M * 4));
    I8Maps maps;
    if (!row_map(&maps.w, p.w, false, p.N, p.K, p.w_st, kI8Channels, true) ||
        !row_map(&maps.a, ws, true, p.M, p.K, half_st, NT / 2, true))
        return GDN_ERR_CUDA;
    const int64_t eights = (half_st / 8 + 31) / 32 * 32, threads = eights < 1024 ? eights : 1024;
    const bool vec = ((uintptr_t)p.a & 7u) == 0 && (p.M == 1 || p.a_st % 8 == 0);
    if (launch_dependent(matmul_i8_tokens_kernel, dim3((unsigned)p.M), dim3((unsigned)threads), 0, st, p.a, p.a_st, (__half *)ws,
                         half_st, squares, p.K, (int)vec) != cudaSuccess)
        return GDN_ERR_CUDA;
    const unsigned grid = (unsigned)(2 * (sh.units < pairs ? sh.units : pairs));
    if (launch_dependent(kern, dim3(grid), dim3(kPairThreads), smem, st, maps, p, sh) != cudaSuccess)
        return GDN_ERR_CUDA;
    if (sh.parts > 1 &&
        launch_dependent(matmul_i8_join_kernel, dim3(NT / 4, (unsigned)(plan.tiles - plan.full)), dim3(256), 0, st, p,
                         sh) != cudaSuccess)
        return GDN_ERR_CUDA;
    return GDN_OK;
}

gdn_status_t launch_matmul_i8_few(const MatmulParams &p, cudaStream_t st) {
    if (p.M <= 16) return launch_tc<16>(p, st);
    if (p.M <= 32) return launch_tc<32>(p, st);
    return launch_tc<64>(p, st);
}

// Which kernel takes a product of more than eight tokens.
bool matmul_i8_pairs(int64_t M, int64_t N, int64_t K) {
    if (M <= 64) return false;
    int dev = 0;
    const int sms = cudaGetDevice(&dev) == cudaSuccess ? matmul_sm_count(dev) : 0;
    if (sms <= 1) return true;
    const int64_t pairs = sms / 2, steps = (K + kI8Step - 1) / kI8Step;
    const PairPlan plan = pair_plan(M, N, K, (int)pairs);
    const int64_t left = plan.tiles - plan.full;
    const double turns = (double)((plan.full + pairs - 1) / pairs * steps) +
                         (double)((left * plan.parts + pairs - 1) / pairs * ((steps + plan.parts - 1) / plan.parts));
    const int64_t tiles = (M + 63) / 64 * ((N + kI8Channels - 1) / kI8Channels), ctas = sms * I8Shape<64>::CTAS;
    const int64_t parts = few_parts(tiles, steps, ctas);
    const double few = (double)((tiles * parts + ctas - 1) / ctas * ((steps + parts - 1) / parts));
    // in us: 333 tokens of 515 channels of 1008 take 7 here and 16 by pairs, 2000 of 1024 of 1024
    // 11.5 and 14.5, 100 of 5120 of 6144 26.5 and 18
    return 10.5 + 0.54 * turns + (plan.parts > 1 ? 1.5 : 0.) < 6 + 0.75 * few;
}

size_t matmul_i8_pair_workspace(int64_t M, int64_t N, int64_t K) {
    int dev = 0;
    const int sms = cudaGetDevice(&dev) == cudaSuccess ? matmul_sm_count(dev) : 0;
    const PairPlan plan = pair_plan(M, N, K, sms / 2);
    const size_t sums = plan.parts > 1 ? (size_t)((plan.tiles - plan.full) * plan.parts) << 18 : 0;
    return up256((size_t)M * (size_t)((K + 7) / 8 * 8) * 2) + up256((size_t)M * 4) + sums;
}

}  // namespace gdn_host
