// Norm of a block's output, its gate, the scaled residual and the next block's
// norm in one pass over the rows, and the gradient in another.
//
//     u = act(z) * x / sqrt(mean x^2 + eps) * w,   y = residual + scale * u,
//     n = y / sqrt(mean y^2 + eps) * w2
//
// Every tensor is read and written once, 16 bytes a load, and HBM bounds both.
// A row belongs to TPR threads, 16-byte pieces of it to a thread; it stays in
// registers between its norms, so the second norm costs no second read, while the
// next row is on its way to shared memory.  Sums are fp32: over a thread's
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
#include <atomic>

#include "launch.cuh"

namespace gdr {
namespace {

constexpr int kSMs = 148;

// A piece is 16 bytes of a row: E channels, 8 in bf16 and 4 in fp32.
template <int E>
__device__ __forceinline__ void load_weights(const float *p, float (&f)[E]) {
#pragma unroll
    for (int e = 0; e < E; e += 4) {
        const float4 a = *reinterpret_cast<const float4 *>(p + e);
        f[e] = a.x; f[e + 1] = a.y; f[e + 2] = a.z; f[e + 3] = a.w;
    }
}
template <int E>
__device__ __forceinline__ void store_floats(float *p, const float (&f)[E]) {
#pragma unroll
    for (int e = 0; e < E; e += 4) *reinterpret_cast<float4 *>(p + e) = make_float4(f[e], f[e + 1], f[e + 2], f[e + 3]);
}
__device__ __forceinline__ void store_piece(float *p, const float (&f)[4]) { store_floats(p, f); }
__device__ __forceinline__ void store_piece(__nv_bfloat16 *p, const float (&f)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 x = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t *>(&x);
    }
    *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}

// Two channels at a time: the arithmetic took half of the issue slots and more (131,072 x
// 128 bf16: 17.7 -> 17.1 us, its gradient 34.4 -> 32.4; 4096 x 8192: gradient 214 -> 178).
__device__ __forceinline__ float2 two(const float *f) { return make_float2(f[0], f[1]); }
__device__ __forceinline__ float2 two(float f) { return make_float2(f, f); }
__device__ __forceinline__ void put2(float *f, float2 x) { f[0] = x.x; f[1] = x.y; }
__device__ __forceinline__ float2 mul2(float2 a, float2 b) { return __fmul2_rn(a, b); }
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) { return __ffma2_rn(a, b, c); }

// e^-z, and with it the sigmoid 1 / (1 + e^-z).  For bf16 tensors the single-instruction
// exponential, within 2^-20 (1 + |z| / 8) of the value, where the result's rounding is 2^-8;
// the full-precision one takes the heads' forward pass from 23 to 35 us.  fp32 tensors get it.
template <int E>
__device__ __forceinline__ float exp_minus(float z) { return E == 8 ? ex2_approx(-kLog2e * z) : expf(-z); }

// act(z) in place of z and, for the gradient, act'(z), of a piece.  The choice stands
// outside the channels' loops, whose exponentials then overlap.
template <int E>
__device__ __forceinline__ void act_of(int act, float (&z)[E]) {
    if (act == kActNone) return;
    const bool silu = act == kActSilu;
#pragma unroll
    for (int e = 0; e < E; ++e) {
        const float s = rcp_approx(1.f + exp_minus<E>(z[e]));
        z[e] = s * (silu ? z[e] : 1.f);
    }
}
template <int E>
__device__ __forceinline__ void act_both(int act, float (&z)[E], float (&da)[E]) {
    if (act == kActNone) {
#pragma unroll
        for (int e = 0; e < E; ++e) da[e] = 1.f;
        return;
    }
    const bool silu = act == kActSilu;
#pragma unroll
    for (int e = 0; e < E; ++e) {
        // what the sigmoid leaves to 1, as a product: the difference has no bits left beyond
        // z = 15 (and is 1 % off at 10 in bf16).  Where e^-z overflows s is 0.
        const float x = exp_minus<E>(z[e]), s = rcp_approx(1.f + x), rest = s * fminf(x, 0x1p127f);
        da[e] = s * (silu ? fmaf(z[e], rest, 1.f) : rest);
        z[e] = s * (silu ? z[e] : 1.f);
    }
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

constexpr int kMostRing = 200 * 1024;

template <typename T, int TPR, int VPT>
struct Shape {
    static constexpr int NT = TPR > 256 ? TPR : 256;
    static constexpr int ROWS = NT / TPR;                  // rows of a block at a time
    static constexpr int E = 16 / sizeof(T);
    // Row groups a block holds, one at work and the others on their way.  A third helps
    // the gradient (8191 x 2048 fp32: 97 -> 86 us of GPU time; a fourth nothing) and costs the forward
    // pass resident blocks (131,072 x 128 bf16: 18.7 -> 20.0 before the packed arithmetic).
    static constexpr int stages(bool back, int tensors) {
        return back && 3 * tensors * VPT * NT * 16 <= kMostRing ? 3 : 2;
    }
};

// A thread's pieces of the next row groups, copied to shared memory without
// registers while it works on this one.  Each thread reads only what it copied
// itself: no barriers.  `Tensors` rows side by side.  Two stages fit for rows of 16 KB with
// any number of tensors and of 32 KB with up to three (all forward passes, gradients without
// the second norm); wider ones are read from memory where they are used.
template <typename T, int TPR, int VPT, int Tensors, int Stages>
struct Ring {
    using Sh = Shape<T, TPR, VPT>;
    static constexpr int WANTED = Stages * Tensors * VPT * Sh::NT * 16;
    static constexpr bool STAGED = WANTED <= kMostRing;
    static constexpr int BYTES = STAGED ? WANTED : 0;
    uint32_t base;

    __device__ __forceinline__ uint32_t place(int stage, int tensor, int i) const {
        return base + (((stage * Tensors + tensor) * VPT + i) * Sh::NT) * 16;
    }
    __device__ __forceinline__ void copy(int stage, int tensor, int i, const T *src) const {
        if (STAGED)
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(place(stage, tensor, i)), "l"(src) : "memory");
    }
    __device__ __forceinline__ void read(int stage, int tensor, int i, const T *src, float (&f)[Sh::E]) const {
        uint32_t w[4];
        if (STAGED) {
            asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                         : "r"(place(stage, tensor, i))
                         : "memory");
        } else {
            const uint4 x = *reinterpret_cast<const uint4 *>(src);
            w[0] = x.x; w[1] = x.y; w[2] = x.z; w[3] = x.w;
        }
#pragma unroll
        for (int e = 0; e < Sh::E; ++e) {
            if (sizeof(T) == 4) f[e] = __uint_as_float(w[e & 3]);
            else f[e] = __uint_as_float(e & 1 ? w[e / 2] & 0xffff0000u : w[e / 2] << 16);
        }
    }
    static __device__ __forceinline__ void commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
    static __device__ __forceinline__ void wait() { asm volatile("cp.async.wait_group %0;" ::"n"(Stages - 1) : "memory"); }
};

// GATE: a gate is given; NEXT: next_weight is.
template <typename T, int TPR, int VPT, bool GATE, bool NEXT>
__global__ void __launch_bounds__(Shape<T, TPR, VPT>::NT)
norm_gate_kernel(const NormArgs p) {
    using Sh = Shape<T, TPR, VPT>;
    constexpr int kStages = Sh::stages(false, 2 + GATE);
    constexpr int E = Sh::E;
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ float scratch[64];
    const Ring<T, TPR, VPT, 2 + GATE, kStages> ring{static_cast<uint32_t>(__cvta_generic_to_shared(smem)) + threadIdx.x * 16};
    int turn = 0;
    const int lane = threadIdx.x % TPR, group = threadIdx.x / TPR;
    const int pieces = p.dim / E;
    const T *x_ = static_cast<const T *>(p.x), *z_ = static_cast<const T *>(p.gate);
    const T *res_ = static_cast<const T *>(p.residual);
    const int64_t stride = (int64_t)gridDim.x * Sh::ROWS, first = (int64_t)blockIdx.x * Sh::ROWS + group;

    auto fetch = [&](int64_t row, int stage) {
        if (row < p.rows) {
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                const int c = lane + i * TPR;
                if (c >= pieces) continue;
                const int64_t at = row * p.dim + c * E;
                ring.copy(stage, 0, i, x_ + at);
                if (res_ != nullptr) ring.copy(stage, 1, i, res_ + at);
                if (GATE) ring.copy(stage, 1 + GATE, i, z_ + at);
            }
        }
        ring.commit();
    };
    float w[VPT][E], w2[VPT][E];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int c = lane + i * TPR;
#pragma unroll
        for (int e = 0; e < E; ++e) { w[i][e] = 1.f; w2[i][e] = 0.f; }
        if (c < pieces && p.weight != nullptr) load_weights(p.weight + c * E, w[i]);
        if (c < pieces && NEXT) load_weights(p.next_weight + c * E, w2[i]);
    }
#pragma unroll
    for (int s = 0; s < kStages - 1; ++s) fetch(first + s * stride, s);
    int stage = 0;
    for (int64_t row = first; row - group < p.rows; row += stride) {
        fetch(row + (kStages - 1) * stride, stage == 0 ? kStages - 1 : stage - 1);
        ring.wait();
        const bool live = row < p.rows;
        float y[VPT][E];
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
#pragma unroll
            for (int e = 0; e < E; ++e) y[i][e] = 0.f;
            if (live && lane + i * TPR < pieces) ring.read(stage, 0, i, x_ + row * p.dim + (lane + i * TPR) * E, y[i]);
        }
        float r = 1.f;
        if (p.weight != nullptr) {
            float2 ss = two(0.f);
#pragma unroll
            for (int i = 0; i < VPT; ++i)
#pragma unroll
                for (int e = 0; e < E; e += 2) ss = fma2(two(&y[i][e]), two(&y[i][e]), ss);
            float s[1] = {ss.x + ss.y};
            row_sum<TPR>(s, scratch, turn);
            r = rsqrtf(s[0] * p.inv_dim + p.eps);
        }
        float2 sy = two(0.f);
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int c = lane + i * TPR;
            if (live && c < pieces) {
                float z[E], res[E];
                const int64_t at = row * p.dim + c * E;
                if (GATE) {
                    ring.read(stage, 1 + GATE, i, z_ + at, z);
                    act_of(p.act, z);
                }
#pragma unroll
                for (int e = 0; e < E; ++e) res[e] = 0.f;
                if (res_ != nullptr) ring.read(stage, 1, i, res_ + at, res);
#pragma unroll
                for (int e = 0; e < E; e += 2) {
                    float2 u = mul2(mul2(two(&y[i][e]), two(r)), two(&w[i][e]));
                    if (GATE) u = mul2(u, two(&z[e]));
                    const float2 yy = fma2(two(p.scale), u, two(&res[e]));
                    put2(&y[i][e], yy);
                    if (NEXT) sy = fma2(yy, yy, sy);
                }
                store_piece(static_cast<T *>(p.y) + row * p.dim + c * E, y[i]);
            }
        }
        if (NEXT) {
            float s2[1] = {sy.x + sy.y};
            row_sum<TPR>(s2, scratch, turn);
            const float r2 = rsqrtf(s2[0] * p.inv_dim + p.eps);
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                const int c = lane + i * TPR;
                if (live && c < pieces) {
#pragma unroll
                    for (int e = 0; e < E; e += 2) put2(&y[i][e], mul2(two(&y[i][e]), mul2(two(r2), two(&w2[i][e]))));
                    store_piece(static_cast<T *>(p.y_norm) + row * p.dim + c * E, y[i]);
                }
            }
        }
        stage = stage + 1 == kStages ? 0 : stage + 1;
    }
}

// Blocks an SM has to have room for: 80 registers a thread hold a piece's gradient without
// the second norm (131,072 x 128 bf16: 39 -> 37 us against 128), with it they spill (8192 x
// 2048: 59 -> 79).  Two fp32 pieces with it fill the ring of the only block.
constexpr int backward_blocks(int threads_per_row, int pieces, bool next) {
    return threads_per_row > 256 || pieces > 2 || (pieces > 1 && next) ? 1 : pieces > 1 || next ? 2 : 3;
}

// GATE: a gate is given; NEXT: dn is (and next_weight).
template <typename T, int TPR, int VPT, bool GATE, bool NEXT>
__global__ void __launch_bounds__(Shape<T, TPR, VPT>::NT, backward_blocks(TPR, VPT, NEXT))
norm_gate_backward_kernel(const NormArgs p) {
    using Sh = Shape<T, TPR, VPT>;
    constexpr int kStages = Sh::stages(true, 2 + GATE + 2 * NEXT);
    constexpr int E = Sh::E;
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ float scratch[64];
    const Ring<T, TPR, VPT, 2 + GATE + 2 * NEXT, kStages> ring{static_cast<uint32_t>(__cvta_generic_to_shared(smem)) + threadIdx.x * 16};
    int turn = 0;
    const int lane = threadIdx.x % TPR, group = threadIdx.x / TPR;
    const int pieces = p.dim / E;
    const T *x_ = static_cast<const T *>(p.x), *z_ = static_cast<const T *>(p.gate);
    const T *res_ = static_cast<const T *>(p.residual);
    const T *dy_ = static_cast<const T *>(p.dy), *dn_ = static_cast<const T *>(p.dn);
    const int64_t stride = (int64_t)gridDim.x * Sh::ROWS, first = (int64_t)blockIdx.x * Sh::ROWS + group;

    auto fetch = [&](int64_t row, int stage) {
        if (row < p.rows) {
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                const int c = lane + i * TPR;
                if (c >= pieces) continue;
                const int64_t at = row * p.dim + c * E;
                ring.copy(stage, 0, i, x_ + at);
                if (dy_ != nullptr) ring.copy(stage, 1, i, dy_ + at);
                if (GATE) ring.copy(stage, 2, i, z_ + at);
                if (NEXT) ring.copy(stage, 2 + GATE, i, dn_ + at);
                if (NEXT && res_ != nullptr) ring.copy(stage, 3 + GATE, i, res_ + at);
            }
        }
        ring.commit();
    };
    // the weights stay in registers as far as there is room beside their gradients; wider
    // rows read them again from the caches where they are used
    constexpr bool KEPT = VPT * E <= 8;
    auto load_w = [&](int i, float (&f)[E]) {
        const int c = lane + i * TPR;
#pragma unroll
        for (int e = 0; e < E; ++e) f[e] = 1.f;
        if (c < pieces && p.weight != nullptr) load_weights(p.weight + c * E, f);
    };
    auto load_w2 = [&](int i, float (&f)[E]) {
        const int c = lane + i * TPR;
#pragma unroll
        for (int e = 0; e < E; ++e) f[e] = 0.f;
        if (c < pieces && NEXT) load_weights(p.next_weight + c * E, f);
    };
    float dw[VPT][E], dw2[VPT][E], kept_w[VPT][E], kept_w2[VPT][E];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
#pragma unroll
        for (int e = 0; e < E; ++e) dw[i][e] = dw2[i][e] = 0.f;
        load_w(i, kept_w[i]);
        load_w2(i, kept_w2[i]);
    }
    auto weights = [&](int i, float (&f)[E]) {
        if (!KEPT) return load_w(i, f);
#pragma unroll
        for (int e = 0; e < E; ++e) f[e] = kept_w[i][e];
    };
    auto next_weights = [&](int i, float (&f)[E]) {
        if (!KEPT) return load_w2(i, f);
#pragma unroll
        for (int e = 0; e < E; ++e) f[e] = kept_w2[i][e];
    };
#pragma unroll
    for (int s = 0; s < kStages - 1; ++s) fetch(first + s * stride, s);
    int stage = 0;
    for (int64_t row = first; row - group < p.rows; row += stride) {
        fetch(row + (kStages - 1) * stride, stage == 0 ? kStages - 1 : stage - 1);
        ring.wait();
        const bool live = row < p.rows;
        const int64_t at = row * p.dim;
        float x[VPT][E], g[VPT][E];
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
#pragma unroll
            for (int e = 0; e < E; ++e) { x[i][e] = 0.f; g[i][e] = 0.f; }
            if (live && lane + i * TPR < pieces) {
                const int64_t here = at + (lane + i * TPR) * E;
                ring.read(stage, 0, i, x_ + here, x[i]);
                if (dy_ != nullptr) ring.read(stage, 1, i, dy_ + here, g[i]);
            }
        }
        float r = 1.f;
        if (p.weight != nullptr) {
            float2 ss = two(0.f);
#pragma unroll
            for (int i = 0; i < VPT; ++i)
#pragma unroll
                for (int e = 0; e < E; e += 2) ss = fma2(two(&x[i][e]), two(&x[i][e]), ss);
            float s[1] = {ss.x + ss.y};
            row_sum<TPR>(s, scratch, turn);
            r = rsqrtf(s[0] * p.inv_dim + p.eps);
        }
        float a[VPT][E], da[VPT][E];           // act(z) and act'(z)
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
#pragma unroll
            for (int e = 0; e < E; ++e) {
                a[i][e] = GATE ? 0.f : 1.f;
                da[i][e] = 0.f;
            }
            if (GATE && live && lane + i * TPR < pieces) {
                ring.read(stage, 2, i, z_ + at + (lane + i * TPR) * E, a[i]);
                act_both(p.act, a[i], da[i]);
            }
#pragma unroll
            for (int e = 0; e < E; e += 2) put2(&x[i][e], mul2(two(&x[i][e]), two(r)));          // xh
        }
        if (NEXT) {
            // y again, and the two sums of the second norm
            float y[VPT][E], t[VPT][E];
            float2 sy = two(0.f), st = sy;
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                const bool in = live && lane + i * TPR < pieces;
#pragma unroll
                for (int e = 0; e < E; ++e) { y[i][e] = 0.f; t[i][e] = 0.f; }
                const int64_t here = at + (lane + i * TPR) * E;
                if (in) ring.read(stage, 2 + GATE, i, dn_ + here, t[i]);
                if (in && res_ != nullptr) ring.read(stage, 3 + GATE, i, res_ + here, y[i]);
                float w[E], w2[E];
                weights(i, w);
                next_weights(i, w2);
#pragma unroll
                for (int e = 0; e < E; e += 2) {
                    float2 u = mul2(two(&x[i][e]), two(&w[e]));
                    if (GATE) u = mul2(u, two(&a[i][e]));
                    const float2 yy = fma2(two(p.scale), u, two(&y[i][e]));
                    put2(&y[i][e], yy);
                    sy = fma2(yy, yy, sy);
                    st = fma2(mul2(two(&t[i][e]), two(&w2[e])), yy, st);
                }
            }
            float s[2] = {sy.x + sy.y, st.x + st.y};
            row_sum<TPR>(s, scratch, turn);
            const float r2 = rsqrtf(s[0] * p.inv_dim + p.eps);
            const float m = s[1] * r2 * p.inv_dim;       // mean(dn w2 yh)
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                float w2[E];
                next_weights(i, w2);
#pragma unroll
                for (int e = 0; e < E; e += 2) {
                    const float2 yh = mul2(two(&y[i][e]), two(r2)), tt = two(&t[i][e]);
                    put2(&dw2[i][e], fma2(tt, yh, two(&dw2[i][e])));
                    put2(&g[i][e], fma2(two(r2), fma2(yh, two(-m), mul2(tt, two(&w2[e]))), two(&g[i][e])));
                }
            }
        }
        float2 sg = two(0.f);
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int c = lane + i * TPR;
            const bool in = live && c < pieces;
            if (in && p.dresidual != nullptr) store_piece(static_cast<T *>(p.dresidual) + at + c * E, g[i]);
            float dz[E], w[E];
            weights(i, w);
#pragma unroll
            for (int e = 0; e < E; e += 2) {
                const float2 xh = two(&x[i][e]), ww = two(&w[e]);
                const float2 du = mul2(two(p.scale), two(&g[i][e])), dua = GATE ? mul2(du, two(&a[i][e])) : du;
                if (GATE) put2(&dz[e], mul2(mul2(mul2(du, xh), ww), two(&da[i][e])));
                put2(&dw[i][e], fma2(dua, xh, two(&dw[i][e])));
                const float2 t = mul2(dua, ww);
                put2(&g[i][e], t);
                sg = fma2(t, xh, sg);
            }
            if (GATE && in) store_piece(static_cast<T *>(p.dgate) + at + c * E, dz);
        }
        float s[1] = {sg.x + sg.y};
        if (p.weight != nullptr) row_sum<TPR>(s, scratch, turn);
        const float m = p.weight != nullptr ? s[0] * p.inv_dim : 0.f;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int c = lane + i * TPR;
            if (live && c < pieces) {
#pragma unroll
                for (int e = 0; e < E; e += 2) put2(&x[i][e], mul2(two(r), fma2(two(&x[i][e]), two(-m), two(&g[i][e]))));
                store_piece(static_cast<T *>(p.dx) + at + c * E, x[i]);
            }
        }
        stage = stage + 1 == kStages ? 0 : stage + 1;
    }
    __shared__ float sums[Sh::ROWS > 1 ? Sh::NT * E : 1];

    launch_dependents();
    // the block's sums: over its row groups in their order, then one partial row
    auto put = [&](float (&v)[VPT][E], float *part) {
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int c = lane + i * TPR;
            if constexpr (Sh::ROWS > 1) {
                __syncthreads();
#pragma unroll
                for (int e = 0; e < E; ++e) sums[e * Sh::NT + threadIdx.x] = v[i][e];
                __syncthreads();
                if (group == 0) {
#pragma unroll
                    for (int e = 0; e < E; ++e)
                        for (int q = 1; q < Sh::ROWS; ++q) v[i][e] += sums[e * Sh::NT + q * TPR + lane];
                }
            }
            if (group == 0 && c < pieces) store_floats(part + (int64_t)blockIdx.x * p.dim + c * E, v[i]);
        }
    };
    if (p.weight != nullptr) put(dw, p.part);
    if (NEXT) put(dw2, p.part2);
}

// Partial rows -> the weights' gradients: 8 columns a block, 32 runs of partial rows
// added up side by side, then the runs in their order.
__global__ void __launch_bounds__(256)
norm_sums_kernel(const float *part, float *dw, const float *part2, float *dw2, int blocks, int dim) {
    __shared__ float s[32][9];
    const float *src = blockIdx.y == 0 ? part : part2;
    float *dst = blockIdx.y == 0 ? dw : dw2;
    wait_for_previous();
    if (dst == nullptr) return;
    const int x = threadIdx.x & 7, run = threadIdx.x >> 3, col = blockIdx.x * 8 + x;
    const int per = (blocks + 31) / 32, end = min(blocks, (run + 1) * per);
    float sum = 0.f;
#pragma unroll 8
    for (int b = run * per; b < end; ++b) sum += src[(int64_t)b * dim + col];
    s[run][x] = sum;
    __syncthreads();
    if (run == 0) {
#pragma unroll
        for (int q = 1; q < 32; ++q) sum += s[q][x];
        dst[col] = sum;
    }
}

// Threads of a row: the power of two that gives each one vector, as far as 512
// threads reach; then several vectors a thread (two and four a thread at smaller
// widths took the heads' passes from 23 and 58 us to 28 and 83: what hides the
// memory's latency is threads).
int threads_of(int dim) {
    int t = 1;
    while (t < 512 && t * 8 < dim) t *= 2;
    return t;
}

// Blocks of the grid-stride loops: those that the GPU holds at once (a part of a
// second round would leave most of it idle), and at most this many an SM, which
// bounds the gradient's partial rows.
int most_per_sm(int dim) { return threads_of(dim) > 256 ? 2 : 4; }

template <typename Kernel>
int64_t blocks_of(Kernel kernel, std::atomic<int> &resident, int threads, int rows_at_once, int bytes, const NormArgs &p) {
    int per_sm = resident.load(std::memory_order_relaxed);
    if (per_sm == 0) {
        if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kernel, threads, bytes) != cudaSuccess || per_sm < 1)
            per_sm = 1;
        resident.store(per_sm, std::memory_order_relaxed);
    }
    const int64_t groups = (p.rows + rows_at_once - 1) / rows_at_once;
    return std::min<int64_t>(groups, (int64_t)std::min(per_sm, most_per_sm(p.dim)) * kSMs);
}

template <typename T, bool BACK, int TPR, int VPT, bool GATE, bool NEXT>
cudaError_t launch_as(const NormArgs &p, cudaStream_t s) {
    using Sh = Shape<T, TPR, VPT>;
    auto kernel = BACK ? norm_gate_backward_kernel<T, TPR, VPT, GATE, NEXT> : norm_gate_kernel<T, TPR, VPT, GATE, NEXT>;
    constexpr int tensors = BACK ? 2 + GATE + 2 * NEXT : 2 + GATE;
    constexpr int bytes = Ring<T, TPR, VPT, tensors, Sh::stages(BACK, tensors)>::BYTES;
    static std::atomic<int> resident{0};
    cudaError_t e = ensure_dynamic_smem(reinterpret_cast<const void *>(kernel), bytes);
    if (e != cudaSuccess) return e;
    const int64_t blocks = blocks_of(kernel, resident, Sh::NT, Sh::ROWS, bytes, p);
    kernel<<<(unsigned)blocks, Sh::NT, bytes, s>>>(p);
    e = cudaGetLastError();
    if (!BACK || e != cudaSuccess || (p.dweight == nullptr && p.dnext_weight == nullptr)) return e;
    return launch_kernel(true, norm_sums_kernel, dim3(p.dim / 8, p.dnext_weight != nullptr ? 2 : 1), 256, 0, s, p.part,
                         p.dweight, p.part2, p.dnext_weight, (int)blocks, p.dim);
}

template <typename T, bool BACK, int TPR, int VPT>
cudaError_t launch_flags(const NormArgs &p, cudaStream_t s) {
    const bool gate = p.gate != nullptr, next = BACK ? p.dn != nullptr : p.next_weight != nullptr;
    if (gate) return next ? launch_as<T, BACK, TPR, VPT, true, true>(p, s) : launch_as<T, BACK, TPR, VPT, true, false>(p, s);
    return next ? launch_as<T, BACK, TPR, VPT, false, true>(p, s) : launch_as<T, BACK, TPR, VPT, false, false>(p, s);
}

template <typename T, bool BACK>
cudaError_t launch_any(const NormArgs &p, cudaStream_t s) {
    constexpr int V = sizeof(T) / 2;     // pieces of a vector
    switch (threads_of(p.dim)) {
        case 1: return launch_flags<T, BACK, 1, V>(p, s);
        case 2: return launch_flags<T, BACK, 2, V>(p, s);
        case 4: return launch_flags<T, BACK, 4, V>(p, s);
        case 8: return launch_flags<T, BACK, 8, V>(p, s);
        case 16: return launch_flags<T, BACK, 16, V>(p, s);
        case 32: return launch_flags<T, BACK, 32, V>(p, s);
        case 64: return launch_flags<T, BACK, 64, V>(p, s);
        case 128: return launch_flags<T, BACK, 128, V>(p, s);
        case 256: return launch_flags<T, BACK, 256, V>(p, s);
    }
    if (p.dim <= 4096) return launch_flags<T, BACK, 512, V>(p, s);
    if (p.dim <= 8192) return launch_flags<T, BACK, 512, 2 * V>(p, s);
    return launch_flags<T, BACK, 512, 4 * V>(p, s);
}

}  // namespace

// At most this many blocks of the gradient's pass, each with a partial row of either
// weight's gradient.
int norm_gate_blocks(int64_t rows, int dim) {
    const int t = threads_of(dim), per = t > 256 ? 1 : 256 / t;
    return (int)std::max<int64_t>(1, std::min<int64_t>((rows + per - 1) / per, most_per_sm(dim) * kSMs));
}

cudaError_t launch_norm_gate(const NormArgs &p, bool bf16, cudaStream_t stream) {
    return bf16 ? launch_any<__nv_bfloat16, false>(p, stream) : launch_any<float, false>(p, stream);
}

cudaError_t launch_norm_gate_backward(const NormArgs &p, bool bf16, cudaStream_t stream) {
    return bf16 ? launch_any<__nv_bfloat16, true>(p, stream) : launch_any<float, true>(p, stream);
}

}  // namespace gdr
