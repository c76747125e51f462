// Norm of a block's output, its gate, the scaled residual and the next block's
// norm in one pass over the rows, and the gradient in another.
//
//     u = act(z) * x / sqrt(mean x^2 + eps) * w,   y = residual + scale * u,
//     n = y / sqrt(mean y^2 + eps) * w2
//
// Every tensor is read and written once, 16 bytes a load, and HBM bounds both.
// A row belongs to TPR threads, eight neighbouring channels (a vector) per
// thread and step of TPR vectors; it stays in registers between its norms, so
// the second norm costs no second read.  Sums are fp32: over a thread's
// channels, then over the row's threads by a butterfly (and, beyond a warp, in
// the order of the warps).  n is taken from y before y is rounded.
//
// The gradient, with xh and yh the normalised rows, r = 1 / sqrt(mean x^2 + eps)
// and r2 the same of y:
//
//     g   = dy + r2 (dn w2 - yh mean(dn w2 yh))          (= d residual)
//     dz  = scale g xh w act'(z),   dw = sum scale g act(z) xh,   dw2 = sum dn yh
//     dx  = r (t - xh mean(t xh)),  t = scale g act(z) w
//
// x, z and residual are read again and xh, yh recomputed from them in fp32.  The
// weights' gradients are sums over all rows: a block keeps its rows' sums in
// registers over a grid-stride loop, adds them up over its row groups in a fixed
// order and writes one partial row; a second kernel adds the partial rows.  No
// atomics: the same inputs give the same bits.
#include "norm_gate.h"

#include <algorithm>

#include "common.cuh"

namespace gdr {
namespace {

constexpr int kSMs = 148;

__device__ __forceinline__ void load8(const float *p, float (&f)[8]) {
    const float4 a = *reinterpret_cast<const float4 *>(p), b = *reinterpret_cast<const float4 *>(p + 4);
    f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
    f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
}
__device__ __forceinline__ void load8(const __nv_bfloat16 *p, float (&f)[8]) {
    const uint4 a = *reinterpret_cast<const uint4 *>(p);
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = __uint_as_float(w[i] << 16);
        f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}
__device__ __forceinline__ void store8(float *p, const float (&f)[8]) {
    *reinterpret_cast<float4 *>(p) = make_float4(f[0], f[1], f[2], f[3]);
    *reinterpret_cast<float4 *>(p + 4) = make_float4(f[4], f[5], f[6], f[7]);
}
__device__ __forceinline__ void store8(__nv_bfloat16 *p, const float (&f)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 x = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t *>(&x);
    }
    *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ float sigmoid(float z) { return 1.0f / (1.0f + expf(-z)); }

// act(z) and, for the gradient, act'(z).
__device__ __forceinline__ float act_of(int act, float z) {
    return act == kActSilu ? z * sigmoid(z) : act == kActSigmoid ? sigmoid(z) : z;
}
__device__ __forceinline__ void act_both(int act, float z, float &a, float &da) {
    if (act == kActNone) {
        a = z;
        da = 1.f;
        return;
    }
    const float s = sigmoid(z);
    a = act == kActSilu ? z * s : s;
    da = act == kActSilu ? s * (1.f + z * (1.f - s)) : s * (1.f - s);
}

// Sum over the TPR threads of a row; every thread of the block takes part.
// scratch: one float per warp and value, `turn` alternates its halves.
template <int TPR, int NV>
__device__ __forceinline__ void row_sum(float (&x)[NV], float *scratch, int &turn) {
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
        for (int off = (TPR < 32 ? TPR : 32) / 2; off > 0; off >>= 1)
            x[v] += __shfl_xor_sync(0xffffffffu, x[v], off);
    if constexpr (TPR > 32) {
        constexpr int WPR = TPR / 32;
        const int warp = threadIdx.x >> 5;
        float *s = scratch + turn * 32;      // NV * 16 warps at most
        turn ^= 1;
        if ((threadIdx.x & 31) == 0) {
#pragma unroll
            for (int v = 0; v < NV; ++v) s[v * 16 + warp] = x[v];
        }
        __syncthreads();
        const int w0 = warp / WPR * WPR;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            float sum = 0.f;
#pragma unroll
            for (int w = 0; w < WPR; ++w) sum += s[v * 16 + w0 + w];
            x[v] = sum;
        }
    }
}

template <typename T, int TPR, int VPT>
struct Shape {
    static constexpr int NT = TPR > 256 ? TPR : 256;
    static constexpr int ROWS = NT / TPR;      // rows of a block at a time
};

template <typename T, int TPR, int VPT>
__global__ void __launch_bounds__(Shape<T, TPR, VPT>::NT)
norm_gate_kernel(const NormArgs p) {
    using Sh = Shape<T, TPR, VPT>;
    __shared__ float scratch[64];
    int turn = 0;
    const int lane = threadIdx.x % TPR;
    const int64_t row = (int64_t)blockIdx.x * Sh::ROWS + threadIdx.x / TPR;
    const int vecs = p.dim / 8;
    const bool live = row < p.rows;
    const int64_t at = row * p.dim;
    const T *x_ = static_cast<const T *>(p.x), *z_ = static_cast<const T *>(p.gate);
    const T *res_ = static_cast<const T *>(p.residual);

    float y[VPT][8], z[VPT][8], res[VPT][8];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int c = lane + i * TPR;
        const bool in = live && c < vecs;
#pragma unroll
        for (int e = 0; e < 8; ++e) { y[i][e] = 0.f; z[i][e] = 1.f; res[i][e] = 0.f; }
        if (in) {
            load8(x_ + at + c * 8, y[i]);
            if (z_ != nullptr) load8(z_ + at + c * 8, z[i]);
            if (res_ != nullptr) load8(res_ + at + c * 8, res[i]);
        }
    }
    float r = 1.f;
    if (p.weight != nullptr) {
        float s[1] = {0.f};
#pragma unroll
        for (int i = 0; i < VPT; ++i)
#pragma unroll
            for (int e = 0; e < 8; ++e) s[0] = fmaf(y[i][e], y[i][e], s[0]);
        row_sum<TPR>(s, scratch, turn);
        r = rsqrtf(s[0] * p.inv_dim + p.eps);
    }
    float s2[1] = {0.f};
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int c = lane + i * TPR;
        const bool in = live && c < vecs;
        float w[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) w[e] = 1.f;
        if (in && p.weight != nullptr) load8(p.weight + c * 8, w);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            float u = y[i][e] * r * w[e];
            if (z_ != nullptr) u *= act_of(p.act, z[i][e]);
            y[i][e] = res_ != nullptr ? fmaf(p.scale, u, res[i][e]) : p.scale * u;
            s2[0] = fmaf(y[i][e], y[i][e], s2[0]);
        }
        if (in) store8(static_cast<T *>(p.y) + at + c * 8, y[i]);
    }
    if (p.next_weight == nullptr) return;
    row_sum<TPR>(s2, scratch, turn);
    const float r2 = rsqrtf(s2[0] * p.inv_dim + p.eps);
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int c = lane + i * TPR;
        if (live && c < vecs) {
            float w[8];
            load8(p.next_weight + c * 8, w);
#pragma unroll
            for (int e = 0; e < 8; ++e) w[e] *= y[i][e] * r2;
            store8(static_cast<T *>(p.y_norm) + at + c * 8, w);
        }
    }
}

template <typename T, int TPR, int VPT>
__global__ void __launch_bounds__(Shape<T, TPR, VPT>::NT)
norm_gate_backward_kernel(const NormArgs p) {
    using Sh = Shape<T, TPR, VPT>;
    __shared__ float scratch[64];
    __shared__ float sums[Sh::ROWS > 1 ? Sh::NT * 8 : 1];
    int turn = 0;
    const int lane = threadIdx.x % TPR, group = threadIdx.x / TPR;
    const int vecs = p.dim / 8;
    const T *x_ = static_cast<const T *>(p.x), *z_ = static_cast<const T *>(p.gate);
    const T *res_ = static_cast<const T *>(p.residual);
    const T *dy_ = static_cast<const T *>(p.dy), *dn_ = static_cast<const T *>(p.dn);

    float dw[VPT][8], dw2[VPT][8];
#pragma unroll
    for (int i = 0; i < VPT; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) dw[i][e] = dw2[i][e] = 0.f;

    for (int64_t r0 = (int64_t)blockIdx.x * Sh::ROWS; r0 < p.rows; r0 += (int64_t)gridDim.x * Sh::ROWS) {
        const int64_t row = r0 + group;
        const bool live = row < p.rows;
        const int64_t at = row * p.dim;
        float x[VPT][8], z[VPT][8], g[VPT][8], y[VPT][8], t[VPT][8];
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int c = lane + i * TPR;
            const bool in = live && c < vecs;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                x[i][e] = 0.f; z[i][e] = 0.f; g[i][e] = 0.f; y[i][e] = 0.f; t[i][e] = 0.f;
            }
            if (in) {
                load8(x_ + at + c * 8, x[i]);
                if (z_ != nullptr) load8(z_ + at + c * 8, z[i]);
                if (dy_ != nullptr) load8(dy_ + at + c * 8, g[i]);
                if (dn_ != nullptr) {
                    load8(dn_ + at + c * 8, t[i]);
                    if (res_ != nullptr) load8(res_ + at + c * 8, y[i]);
                }
            }
        }
        float r = 1.f;
        if (p.weight != nullptr) {
            float s[1] = {0.f};
#pragma unroll
            for (int i = 0; i < VPT; ++i)
#pragma unroll
                for (int e = 0; e < 8; ++e) s[0] = fmaf(x[i][e], x[i][e], s[0]);
            row_sum<TPR>(s, scratch, turn);
            r = rsqrtf(s[0] * p.inv_dim + p.eps);
        }
        if (dn_ != nullptr) {
            // y again, and the two sums of the second norm
            float s[2] = {0.f, 0.f};
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                const int c = lane + i * TPR;
                const bool in = live && c < vecs;
                float w[8], w2[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) w[e] = w2[e] = 1.f;
                if (in && p.weight != nullptr) load8(p.weight + c * 8, w);
                if (in) load8(p.next_weight + c * 8, w2);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    float u = x[i][e] * r * w[e];
                    if (z_ != nullptr) u *= act_of(p.act, z[i][e]);
                    y[i][e] = fmaf(p.scale, u, y[i][e]);
                    s[0] = fmaf(y[i][e], y[i][e], s[0]);
                    s[1] = fmaf(t[i][e] * w2[e], y[i][e], s[1]);
                }
            }
            row_sum<TPR>(s, scratch, turn);
            const float r2 = rsqrtf(s[0] * p.inv_dim + p.eps);
            const float m = s[1] * r2 * p.inv_dim;       // mean(dn w2 yh)
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                const int c = lane + i * TPR;
                float w2[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) w2[e] = 0.f;
                if (live && c < vecs) load8(p.next_weight + c * 8, w2);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float yh = y[i][e] * r2;
                    dw2[i][e] = fmaf(t[i][e], yh, dw2[i][e]);
                    g[i][e] = fmaf(r2, fmaf(-yh, m, t[i][e] * w2[e]), g[i][e]);
                }
            }
        }
        float s[1] = {0.f};
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int c = lane + i * TPR;
            const bool in = live && c < vecs;
            if (in && p.dresidual != nullptr) store8(static_cast<T *>(p.dresidual) + at + c * 8, g[i]);
            float w[8], dz[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) w[e] = 1.f;
            if (in && p.weight != nullptr) load8(p.weight + c * 8, w);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float du = p.scale * g[i][e], xh = x[i][e] * r;
                float a = 1.f, da = 0.f;
                if (z_ != nullptr) act_both(p.act, z[i][e], a, da);
                dz[e] = du * xh * w[e] * da;
                const float dua = du * a;
                dw[i][e] = fmaf(dua, xh, dw[i][e]);
                g[i][e] = dua * w[e];
                s[0] = fmaf(g[i][e], xh, s[0]);
                x[i][e] = xh;
            }
            if (in && z_ != nullptr) store8(static_cast<T *>(p.dgate) + at + c * 8, dz);
        }
        if (p.weight != nullptr) row_sum<TPR>(s, scratch, turn);
        const float m = p.weight != nullptr ? s[0] * p.inv_dim : 0.f;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int c = lane + i * TPR;
            if (live && c < vecs) {
#pragma unroll
                for (int e = 0; e < 8; ++e) x[i][e] = r * fmaf(-x[i][e], m, g[i][e]);
                store8(static_cast<T *>(p.dx) + at + c * 8, x[i]);
            }
        }
    }

    // the block's sums: over its row groups in their order, then one partial row
    auto put = [&](float (&v)[VPT][8], float *part) {
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int c = lane + i * TPR;
            if constexpr (Sh::ROWS > 1) {
                __syncthreads();
#pragma unroll
                for (int e = 0; e < 8; ++e) sums[e * Sh::NT + threadIdx.x] = v[i][e];
                __syncthreads();
                if (group == 0) {
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        for (int q = 1; q < Sh::ROWS; ++q) v[i][e] += sums[e * Sh::NT + q * TPR + lane];
                }
            }
            if (group == 0 && c < vecs) store8(part + (int64_t)blockIdx.x * p.dim + c * 8, v[i]);
        }
    };
    if (p.weight != nullptr) put(dw, p.part);
    if (dn_ != nullptr) put(dw2, p.part2);
}

// Partial rows -> the weights' gradients: 32 columns a block, eight runs of
// partial rows added up side by side, then the runs in their order.
__global__ void __launch_bounds__(256)
norm_sums_kernel(const float *part, float *dw, const float *part2, float *dw2, int blocks, int dim) {
    __shared__ float s[8][33];
    const float *src = blockIdx.y == 0 ? part : part2;
    float *dst = blockIdx.y == 0 ? dw : dw2;
    if (dst == nullptr) return;
    const int col = blockIdx.x * 32 + (threadIdx.x & 31), run = threadIdx.x >> 5;
    float sum = 0.f;
    if (col < dim) {
        const int per = (blocks + 7) / 8;
        const int b1 = min(blocks, (run + 1) * per);
#pragma unroll 8
        for (int b = run * per; b < b1; ++b) sum += src[(int64_t)b * dim + col];
    }
    s[run][threadIdx.x & 31] = sum;
    __syncthreads();
    if (run == 0 && col < dim) {
#pragma unroll
        for (int q = 1; q < 8; ++q) sum += s[q][threadIdx.x];
        dst[col] = sum;
    }
}

template <typename T, int TPR, int VPT>
cudaError_t launch_forward(const NormArgs &p, cudaStream_t s) {
    using Sh = Shape<T, TPR, VPT>;
    const int64_t blocks = (p.rows + Sh::ROWS - 1) / Sh::ROWS;
    norm_gate_kernel<T, TPR, VPT><<<(unsigned)blocks, Sh::NT, 0, s>>>(p);
    return cudaGetLastError();
}

template <typename T, int TPR, int VPT>
cudaError_t launch_backward_rows(const NormArgs &p, cudaStream_t s) {
    using Sh = Shape<T, TPR, VPT>;
    const unsigned blocks = (unsigned)norm_gate_blocks(p.rows, p.dim);
    norm_gate_backward_kernel<T, TPR, VPT><<<blocks, Sh::NT, 0, s>>>(p);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || (p.dweight == nullptr && p.dnext_weight == nullptr)) return e;
    norm_sums_kernel<<<dim3((p.dim + 31) / 32, p.dnext_weight != nullptr ? 2 : 1), 256, 0, s>>>(
        p.part, p.dweight, p.part2, p.dnext_weight, (int)blocks, p.dim);
    return cudaGetLastError();
}

// Threads of a row: the power of two that gives each one vector, as far as 512
// threads reach; then several vectors a thread.
int threads_of(int dim) {
    int t = 1;
    while (t < 512 && t * 8 < dim) t *= 2;
    return t;
}

template <typename T, bool BACK, int TPR, int VPT>
cudaError_t launch_as(const NormArgs &p, cudaStream_t s) {
    if constexpr (BACK) return launch_backward_rows<T, TPR, VPT>(p, s);
    else return launch_forward<T, TPR, VPT>(p, s);
}

template <typename T, bool BACK>
cudaError_t launch_any(const NormArgs &p, cudaStream_t s) {
    switch (threads_of(p.dim)) {
        case 1: return launch_as<T, BACK, 1, 1>(p, s);
        case 2: return launch_as<T, BACK, 2, 1>(p, s);
        case 4: return launch_as<T, BACK, 4, 1>(p, s);
        case 8: return launch_as<T, BACK, 8, 1>(p, s);
        case 16: return launch_as<T, BACK, 16, 1>(p, s);
        case 32: return launch_as<T, BACK, 32, 1>(p, s);
        case 64: return launch_as<T, BACK, 64, 1>(p, s);
        case 128: return launch_as<T, BACK, 128, 1>(p, s);
        case 256: return launch_as<T, BACK, 256, 1>(p, s);
    }
    if (p.dim <= 4096) return launch_as<T, BACK, 512, 1>(p, s);
    if (p.dim <= 8192) return launch_as<T, BACK, 512, 2>(p, s);
    return launch_as<T, BACK, 512, 4>(p, s);
}

}  // namespace

// Blocks of the gradient's grid-stride loop: as many as the GPU holds at once.
int norm_gate_blocks(int64_t rows, int dim) {
    const int t = threads_of(dim), per = t > 256 ? 1 : 256 / t;
    const int64_t all = (rows + per - 1) / per;
    return (int)std::max<int64_t>(1, std::min<int64_t>(all, t > 256 ? kSMs * 2 : kSMs * 4));
}

cudaError_t launch_norm_gate(const NormArgs &p, bool bf16, cudaStream_t stream) {
    return bf16 ? launch_any<__nv_bfloat16, false>(p, stream) : launch_any<float, false>(p, stream);
}

cudaError_t launch_norm_gate_backward(const NormArgs &p, bool bf16, cudaStream_t stream) {
    return bf16 ? launch_any<__nv_bfloat16, true>(p, stream) : launch_any<float, true>(p, stream);
}

}  // namespace gdr
