// Host-side launchers of the gated norm (arguments already validated).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace gdr {

constexpr int kActNone = 0, kActSilu = 1, kActSigmoid = 2;
constexpr int kNormMaxDim = 16384;

struct NormArgs {
    const void *x, *gate, *residual;      // [rows, dim]; gate, residual or null
    const float *weight, *next_weight;    // [dim] or null: no norm of x / of y
    float scale, eps, inv_dim;
    int act, dim;
    int64_t rows;
    void *y, *y_norm;                     // forward
    const void *dy, *dn;                  // gradient: either may be null
    void *dx, *dgate, *dresidual;
    float *dweight, *dnext_weight;
    float *part, *part2;                  // [blocks, dim] each
};

int norm_gate_blocks(int64_t rows, int dim);
cudaError_t launch_norm_gate(const NormArgs &p, bool bf16, cudaStream_t stream);
cudaError_t launch_norm_gate_backward(const NormArgs &p, bool bf16, cudaStream_t stream);

}  // namespace gdr
