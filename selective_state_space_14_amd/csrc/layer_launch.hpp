// layer_launch.hpp -- host-side argument blocks and launchers of the operators around a gated linear recurrence: its scan and
// step, the norm with the residual's addition and 8-bit output, the 8-bit projection.
#pragma once

#include "ssd_launch.hpp"

namespace ssd {

// The norm with the residual's addition and 8-bit output.
struct AddNormArgs {
    int64_t R;
    int W, x_dtype, s_dtype, dtype, rms;   // s_dtype: residual's and sum's, x's without a residual
    int vec;
    float eps;
    const void* x; int64_t x_stride;
    const void* residual; int64_t residual_stride;     // or null
    const float* w; const float* b;        // [W] or null
    const void* z; int64_t z_stride;       // dtype, or null
    void* sum; int64_t sum_stride;         // s_dtype, or null
    void* y; int64_t y_stride;             // dtype, or null
    uint8_t* q; int64_t q_stride;          // e4m3, or null
    float* scale; int64_t scale_stride;    // [R][ceil(W / 128)], with q
};
// The backward: ssd_norm_bwd's with the gradient that reaches the norm's input past it.
struct AddNormBwdArgs : NormArgs {
    const void* gs; int64_t gs_stride;     // x_dtype, added to dx, or null
};

// Gated linear recurrence: forward (gy = null), one token (final_state in place) and backward.
struct GlrArgs {
    int B, L, D, dtype;
    int pair;                              // even widths and strides, bases on pairs: two channels a load
    int vec;                               // the step: 16-byte rows and D % 8 == 0
    int tiles;                             // set by the launchers
    const void* x; int64_t x_stride;       // [B][L][D] (dtype)
    const void* r; int64_t r_stride;
    const void* i; int64_t i_stride;
    const float* A;                        // [D]
    const float* r_bias; const float* i_bias;      // [D] or null
    const int32_t* doc; const int32_t* lengths;
    const float* init_state; float* final_state;   // [B][D]
    float* states;                         // [B][chunks of 64][D]: the states entering them, or null
    void* y; int64_t y_stride;             // null in the backward's own forward pass
    // backward
    const void* gy; int64_t gy_stride;
    const float* g_final;                  // [B][D] or null
    void* dx; int64_t dx_stride;
    void* dr; int64_t dr_stride;
    void* di; int64_t di_stride;
    float* dA; float* dr_bias; float* di_bias;     // [D]; the biases' or null
    float* g_init;                         // [B][D] or null
};

// The 8-bit projection: y [M][N] from a [M][K] and w [N][K], a scale for every 128 columns of K (and rows of w).
struct ProjArgs {
    int M, N, K, dtype;
    int wide;                              // y's base and rows on four elements
    const uint8_t* a; int64_t a_stride;
    const float* a_scale; int64_t a_scale_stride;      // [M][ceil(K / 128)]
    const uint8_t* w; int64_t w_stride;
    const float* w_scale; int64_t w_scale_stride;      // [ceil(N / 128)][ceil(K / 128)]
    void* y; int64_t y_stride;             // dtype
};

hipError_t launch_add_norm(const AddNormArgs& a, hipStream_t stream);
hipError_t launch_add_norm_bwd(const AddNormBwdArgs& a, hipStream_t stream);
hipError_t launch_proj(const ProjArgs& a, hipStream_t stream);
int proj_tile_rows(int M, int N, int K, int dtype);    // rows of y of a workgroup of the kernel for these sizes
size_t glr_fwd_workspace_bytes(int B, int L, int D, int dtype);
hipError_t launch_glr_fwd(const GlrArgs& a, void* ws, hipStream_t stream);
size_t glr_bwd_workspace_bytes(int B, int L, int D, int dtype);
hipError_t launch_glr_bwd(const GlrArgs& a, void* ws, hipStream_t stream);
hipError_t launch_glr_step(const GlrArgs& a, hipStream_t stream);
// n floats from `from` (null: zeros)
hipError_t launch_glr_copy(const float* from, float* to, int64_t n, hipStream_t stream);

}  // namespace ssd
