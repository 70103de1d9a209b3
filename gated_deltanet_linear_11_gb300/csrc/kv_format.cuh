// kv_format.cuh -- the paged 4-bit key/value cache.
//
// data: uint8 [pages, 2 (keys, values), Hkv, page, record].  A record is one token of one
// head: D/2 bytes of 4-bit codes, then for each group of 32 consecutive elements an fp16
// pair (scale, minimum).  Element d of group d / 32 stands for minimum + scale * code.
// Per group of x (clamped to +-65504, the fp16 range):
//     minimum = fp16(min x),  scale = fp16((max x - minimum) / 15),
//     code    = round((x - minimum) * (1 / scale)) in 0..15, ties to even; 0 if scale <= 0
//               (a minimum that rounded above a nearly constant group's maximum).
// A group that holds a NaN gets minimum = NaN: all of it reads as NaN.
//
// The codes are stored in the order in which the attention's matrix fragments take them:
// 32-bit word W of a record (eight nibbles i, low first) holds
//     keys:    d = 32 (W mod D/32) + 8 (W div D/32) + i
//     values:  d = 64 (W div 8) + 32 (i div 4) + 4 (W mod 8) + (i mod 4)
// In a key record the D/32 words of one quarter-group lane are contiguous (one wide load
// gives a lane eight elements of every group); in a value record a word holds four
// elements of each of two adjacent groups.
//
// Fewer bits than the inputs': the codes are the format's purpose; scale and minimum are
// fp16 because their 2^-11 rounding is small against the 1/30 of a group's range that a
// code can be off, and the codes are taken against the rounded pair, so the rounding adds
// no error of its own except for clamped extremes.
#pragma once

#include <cuda_fp16.h>

#include "common.cuh"

namespace gdn {

constexpr int kKvGroup = 32;

template <int D> struct KvRec {
    static constexpr int NG = D / kKvGroup;            // groups
    static constexpr int CODES = D / 2;                // bytes of codes
    static constexpr int BYTES = CODES + 4 * NG;       // 40, 80 or 160
};

// What the kernels need of a gdn_kv_cache_t.
struct KvView {
    uint8_t *data;
    const int32_t *table;     // [N, table_width]
    const int32_t *kv_lens;   // [N]
    const int32_t *cu;        // [N + 1] offsets of the new tokens, or null: one each
    int pages, page_log2, Hkv, table_width, N;

    __device__ __forceinline__ int64_t block_bytes(int rec) const {
        return ((int64_t)rec) << page_log2;
    }
    // first byte of the (page, which, head) block
    __device__ __forceinline__ uint8_t *block(int page, int which, int head, int rec) const {
        return data + (((int64_t)page * 2 + which) * Hkv + head) * block_bytes(rec);
    }
    __device__ __forceinline__ int capacity() const {   // positions the table can hold
        const int64_t c = (int64_t)table_width << page_log2;
        return c > 0x7fffffff ? 0x7fffffff : (int)c;
    }
};

// Sequence of packed token t: the n with cu[n] <= t < cu[n + 1].
__device__ __forceinline__ int sequence_of(const int32_t *cu, int N, int t) {
    int lo = 0, hi = N - 1;
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (cu[mid + 1] <= t) lo = mid + 1;
        else hi = mid;
    }
    return lo;
}

}  // namespace gdn

namespace gdn_host {
// One call on a paged cache.  append: k, v in, q rotated to q_out; read: k, v out;
// attention: q in, q_out is o.
struct KvArgs {
    gdn::KvView kv;
    const void *k, *v, *q;
    void *q_out;
    int64_t k_tok, v_tok, q_tok, o_tok;
    const float *cos_tab, *sin_tab;
    int32_t tab_rows, rot, interleaved;
    float *lse;
    int64_t T;
    const int32_t *cu_host;   // the host copy of kv.cu
    int32_t D, Hq, max_q_len, min_q_len, max_kv_len;   // min_q_len: over sequences with rows
    float scale;
    uint32_t flags;
    int in_f32;
    int32_t *status;
    void *ws;
    size_t ws_bytes;
};
gdn_status_t launch_kv_append(const KvArgs &a, cudaStream_t st);
gdn_status_t launch_kv_read(const KvArgs &a, cudaStream_t st);
gdn_status_t launch_kv_attention(const KvArgs &a, cudaStream_t st);
// Sequences with Hq m >= min_rows only, m new tokens each (kv.cu set).
bool kv_attention_tc_supported(int32_t D);
gdn_status_t launch_kv_attention_tc(const KvArgs &a, int min_rows, cudaStream_t st);
size_t kv_attention_workspace(int32_t D, int32_t Hq, int32_t Hkv, int64_t T, int32_t N,
                              int32_t max_q_len, int32_t max_kv_len, int in_f32,
                              uint32_t flags);
}  // namespace gdn_host
