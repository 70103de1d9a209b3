// linear.cuh -- host side of the linear-attention kernels.
#pragma once

#include "common.cuh"

namespace gdn_host {
// Linear attention with a decay for each head (prompts: cu, h0, hT; one token: state, P,
// idx).  g_tok: Hv for gates per token, 0 for one gate per head.
struct LinearArgs {
    const void *q, *k, *v;
    void *o;
    int64_t q_tok, k_tok, v_tok, o_tok;
    const float *g;
    int64_t g_tok;
    const int32_t *cu;
    const int32_t *cu_host;
    const float *h0;
    float *hT;
    float *state;
    const int32_t *idx;
    int64_t T;
    int32_t N, P, Hk, Hv, D, max_len;
    float scale;
    uint32_t flags;
    int in_f32;
    int32_t *status;
    void *ws;
    size_t ws_bytes;
};
bool linear_supported(int64_t D);
bool linear_tc_supported(int64_t D, int in_f32, uint32_t flags);
size_t linear_tc_workspace(const int32_t *cu_host, int32_t N, int64_t T, int32_t Hv);
gdn_status_t launch_linear_tc(const LinearArgs &a, cudaStream_t st);
size_t linear_scan_workspace(const int32_t *cu_host, int32_t N, int64_t T, int32_t Hv, int64_t D);
gdn_status_t launch_linear_scan(const LinearArgs &a, cudaStream_t st);
gdn_status_t launch_linear_decode(const LinearArgs &a, cudaStream_t st);
}  // namespace gdn_host
