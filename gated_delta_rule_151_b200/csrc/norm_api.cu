// C ABI of the gated norm: argument checks and launches.
#include <cmath>

#include "api_common.h"
#include "norm_gate.h"

namespace {

using gdr::api::apart;
using gdr::api::given16;
using gdr::api::io_type;
using gdr::api::maybe16;
using gdr::api::Range;

bool ok_shape(int64_t rows, int32_t dim) {
    return rows >= 0 && dim >= 8 && dim <= gdr::kNormMaxDim && dim % 8 == 0 &&
           rows <= ((int64_t)1 << 40) / dim && rows <= (int64_t)INT32_MAX;
}

bool ok_scalars(float scale, float eps, gdr_activation_t act) {
    return std::isfinite(scale) && std::isfinite(eps) && eps > 0.f &&
           (act == GDR_ACT_NONE || act == GDR_ACT_SILU || act == GDR_ACT_SIGMOID);
}

gdr::NormArgs base_args(const void *x, const float *weight, const void *gate, const void *residual,
                        const float *next_weight, int64_t rows, int32_t dim, float scale, float eps,
                        gdr_activation_t act) {
    gdr::NormArgs p = {};
    p.x = x;
    p.gate = gate;
    p.residual = residual;
    p.weight = weight;
    p.next_weight = next_weight;
    p.scale = scale;
    p.eps = eps;
    p.inv_dim = 1.0f / (float)dim;
    p.act = act;
    p.dim = dim;
    p.rows = rows;
    return p;
}

gdr_status_t status_of(cudaError_t e) { return e == cudaSuccess ? GDR_OK : GDR_ERR_CUDA; }

}  // namespace

extern "C" {

gdr_status_t gdr_norm_gate(const void *x, const float *weight, const void *gate,
                           const void *residual, const float *next_weight, int64_t rows,
                           int32_t dim, float scale, float eps, gdr_activation_t activation,
                           gdr_dtype_t io_dtype, void *y, void *y_norm, void *stream) {
    if (!ok_shape(rows, dim) || !io_type(io_dtype) || !ok_scalars(scale, eps, activation))
        return GDR_ERR_INVALID_ARG;
    if (rows == 0) return GDR_OK;
    if (!given16(x) || !given16(y) || !maybe16(weight) || !maybe16(gate) || !maybe16(residual) ||
        !maybe16(next_weight) || !maybe16(y_norm) || (next_weight == nullptr) != (y_norm == nullptr))
        return GDR_ERR_INVALID_ARG;
    const size_t n = (size_t)rows * dim * (io_dtype == GDR_BF16 ? 2 : 4), w = (size_t)dim * 4;
    const Range in[] = {{x, n}, {weight, w}, {gate, n}, {residual == y ? nullptr : residual, n}, {next_weight, w}};
    const Range out[] = {{y, n}, {y_norm, n}};
    if (!apart(in, out)) return GDR_ERR_INVALID_ARG;
    gdr::NormArgs p = base_args(x, weight, gate, residual, next_weight, rows, dim, scale, eps, activation);
    p.y = y;
    p.y_norm = y_norm;
    return status_of(gdr::launch_norm_gate(p, io_dtype == GDR_BF16, static_cast<cudaStream_t>(stream)));
}

gdr_status_t gdr_norm_gate_workspace_size(int64_t rows, int32_t dim, size_t *bytes) {
    if (bytes == nullptr || !ok_shape(rows, dim)) return GDR_ERR_INVALID_ARG;
    *bytes = rows == 0 ? 0 : 2 * (size_t)gdr::norm_gate_blocks(rows, dim) * dim * 4;
    return GDR_OK;
}

gdr_status_t gdr_norm_gate_backward(const void *x, const float *weight, const void *gate,
                                    const void *residual, const float *next_weight, int64_t rows,
                                    int32_t dim, float scale, float eps,
                                    gdr_activation_t activation, gdr_dtype_t io_dtype,
                                    const void *dy, const void *dn, void *dx, float *dweight,
                                    void *dgate, void *dresidual, float *dnext_weight,
                                    void *workspace, size_t workspace_bytes, void *stream) {
    if (!ok_shape(rows, dim) || !io_type(io_dtype) || !ok_scalars(scale, eps, activation))
        return GDR_ERR_INVALID_ARG;
    if (!maybe16(weight) || !maybe16(next_weight) || !maybe16(dweight) || !maybe16(dnext_weight))
        return GDR_ERR_INVALID_ARG;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (rows == 0) {   // sums over no rows (the tensors with rows have no address then)
        if (dweight != nullptr && cudaMemsetAsync(dweight, 0, (size_t)dim * 4, s) != cudaSuccess) return GDR_ERR_CUDA;
        if (dnext_weight != nullptr && cudaMemsetAsync(dnext_weight, 0, (size_t)dim * 4, s) != cudaSuccess)
            return GDR_ERR_CUDA;
        return GDR_OK;
    }
    // each gradient goes with its input; without dn nothing reaches next_weight
    if ((weight == nullptr) != (dweight == nullptr) || (gate == nullptr) != (dgate == nullptr) ||
        (dresidual != nullptr && residual == nullptr) || (dn != nullptr) != (dnext_weight != nullptr) ||
        (dn != nullptr && next_weight == nullptr))
        return GDR_ERR_INVALID_ARG;
    if (!given16(x) || !given16(dx) || !maybe16(gate) || !maybe16(residual) || !maybe16(dy) || !maybe16(dn) ||
        !maybe16(dgate) || !maybe16(dresidual) || (dy == nullptr && dn == nullptr))
        return GDR_ERR_INVALID_ARG;
    const size_t part = (size_t)gdr::norm_gate_blocks(rows, dim) * dim;
    const bool sums = dweight != nullptr || dnext_weight != nullptr;
    if (sums && (!given16(workspace) || workspace_bytes < 2 * part * 4)) return GDR_ERR_WORKSPACE;
    const size_t n = (size_t)rows * dim * (io_dtype == GDR_BF16 ? 2 : 4), w = (size_t)dim * 4;
    const Range in[] = {{x, n}, {weight, w}, {gate, n}, {residual, n}, {next_weight, w}, {dy, n}, {dn, n}};
    const Range out[] = {{dx, n}, {dweight, w}, {dgate, n}, {dresidual, n}, {dnext_weight, w},
                         {sums ? workspace : nullptr, 2 * part * 4}};
    if (!apart(in, out)) return GDR_ERR_INVALID_ARG;
    gdr::NormArgs p = base_args(x, weight, gate, residual, next_weight, rows, dim, scale, eps, activation);
    p.dy = dy;
    p.dn = dn;
    p.dx = dx;
    p.dgate = dgate;
    p.dresidual = dresidual;
    p.dweight = dweight;
    p.dnext_weight = dnext_weight;
    p.part = static_cast<float *>(workspace);
    p.part2 = p.part + part;
    return status_of(gdr::launch_norm_gate_backward(p, io_dtype == GDR_BF16, s));
}

}  // extern "C"
