// rows.cuh -- arguments of the row operators: root-mean-square norms and 8-bit rows.
#pragma once

#include "common.cuh"

namespace gdn {

enum RowMode { kRowQuantize = 0, kRowAddNorm = 1, kRowGatedNorm = 2 };

struct RowParams {
    const void *x, *res, *z;                // res: residual or null; z: gate (gated norm)
    void *res_out;                          // null without a residual
    const void *w;
    void *y;                                // type of x, or int8 with scale
    float *scale;                           // [T] of the 8-bit rows
    int64_t x_st, res_st, res_out_st, z_st, y_st;   // row strides in elements
    int64_t T;
    int32_t D;                              // row length
    int32_t head;                           // gated norm: elements of a head
    int32_t w_f32;
    int32_t vec;                            // every row starts on 16 bytes (8 of an 8-bit one)
                                            // and D is a multiple of 8
    float offset, eps;
    float per_mean;                         // 1 / the elements that a mean is over
};

}  // namespace gdn

namespace gdn_host {
gdn_status_t launch_rows(const gdn::RowParams &p, int mode, bool in_f32, bool eight_bit, cudaStream_t st);
}  // namespace gdn_host
