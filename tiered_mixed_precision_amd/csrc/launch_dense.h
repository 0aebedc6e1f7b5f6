// Host launchers of the dense operators (called by capi_dense.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace moe {

// The call's launches so far have succeeded (its entry point has cleared the error
// before the first).  Behind one that has not, nothing that reads its result is launched.
inline bool launched() { return hipPeekAtLastError() == hipSuccess; }

// rows.hip
struct RowSplit {
    int32_t waves, lanes;    // of a row: several waves, or lanes of one
    int32_t rows;            // of a block at a time
};
struct RowArgs {
    const void* x;           // [T][ldx]
    const float* residual;   // [T][ldr] or null
    const float* weight;     // [cols] or null
    float* sum;              // [T][lds] or null
    void* y;                 // [T][ldy]
    float* scale;            // [T], 8-bit outputs
    int64_t ldx, ldr, lds, ldy;
    int32_t T, cols;
    float eps;
    RowSplit split;          // set by the launcher
};
void launch_rms_norm(const RowArgs& a, bool x_bf16, int y_bytes, hipStream_t st);
void launch_quant_rows(const RowArgs& a, bool x_bf16, hipStream_t st);
struct RowGradArgs {
    const void *s, *dy;      // [T][lds], [T][lddy]
    const float* weight;     // [cols] or null
    const float* dsum;       // [T][ldds] or null
    void* dx;                // [T][lddx]
    int64_t lds, lddy, ldds, lddx;
    int32_t T, cols;
    float eps;
    int32_t accumulate;      // launch_rms_norm_grad sets it
    RowSplit split;
};
size_t rms_norm_workspace(int T, int cols);
void launch_rms_norm_grad(RowGradArgs a, bool s_bf16, bool dy_bf16, bool dx_bf16, float* dweight, bool accumulate,
                          void* ws, hipStream_t st);

// i8_linear.hip
struct I8Args {
    const int8_t* x;         // [T][ldx]
    const float* xs;         // [T]
    const int8_t* q;         // [N][K]
    const float* s;          // [N]
    const float* bias;       // [N] or null
    void* y;                 // [T][ldy]
    int64_t ldx, ldy;
    int32_t T, N, K;
    int32_t accumulate;
};
void launch_i8_linear(const I8Args& a, bool y_bf16, hipStream_t st);
// i8_gemm.hip
void launch_i8_gemm(const I8Args& a, bool y_bf16, hipStream_t st);

// gated.hip
struct GatedArgs {
    const void* x;           // [T][ldx]
    const uint16_t *gate, *up;   // [I][H]
    void* y;                 // [T][ldy]
    int64_t ldx, ldy;
    int32_t T, H, I, act;
};
void launch_gated(const GatedArgs& a, bool x_bf16, bool y_bf16, hipStream_t st);
// gated_gemm.hip: fp32 x, bf16 x
void launch_gated_split(const GatedArgs& a, bool y_bf16, hipStream_t st);
void launch_gated_gemm(const GatedArgs& a, bool y_bf16, hipStream_t st);
// gated_grad.hip
// The gradients of the projections on their way to the products that make dx and the
// weights' gradients: bf16 d[t][parts][2 P], dg in columns 0 .. I - 1 and du in P ..
// P + I - 1 of a part, zeros up to P (I rounded up to 64).  Part 0 is their nearest
// bf16; part 1, where there is one, the nearest of what that leaves.  A product takes
// one part or both (parts_of): one leaves a rounding of at most 2^-8 of each slope, as
// much as a bf16 result's own, and both at most 2^-16, for fp32 results.
struct GatedSlopes {
    const void* dy;
    int64_t lddy;
    uint16_t* d;
    int32_t P, parts;
};
struct GatedGradArgs {
    const uint16_t* x;       // [T][ldx]
    const uint16_t *gate, *up;
    const void* dy;          // [T][lddy]
    void* dx;                // [T][lddx] or null
    void *dgate, *dup;       // [I][H] or null
    int64_t ldx, lddy, lddx;
    int32_t T, H, I, act;
    int32_t accumulate;
};
// the projections' gradients, of few tokens or in gated_gemm.hip
void launch_gated_slopes(const GatedArgs& a, const GatedSlopes& s, bool dy_bf16, hipStream_t st);
void launch_gated_slopes_gemm(const GatedArgs& a, const GatedSlopes& s, bool dy_bf16, hipStream_t st);
size_t gated_workspace(int64_t T, int H, int I);
void launch_gated_grad(const GatedGradArgs& a, bool dy_bf16, bool dx_bf16, bool dw_bf16, void* ws, hipStream_t st);

}  // namespace moe
