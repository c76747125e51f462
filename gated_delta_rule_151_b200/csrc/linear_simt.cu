// Linear attention with a decay for each head on the CUDA cores (fp32 or bf16
// inputs, any served d), the passes between segments, and the decode step.
//
// The scan of linear_common.cuh runs token by token with one state row per
// thread, in registers: S_r <- x S_r + v_r b, o_r = S_r . a (reverse: the decay
// comes after the output instead of before the update).  A row needs no other
// row, so there is no reduction across threads, and at d = 128 the 3 d_b
// operations per row and token are about what the blocked form costs without
// tensor cores.  a, b and v of eight tokens at a time are staged in shared
// memory as fp32 (every thread reads the same a and b: broadcasts); the next
// eight are fetched meanwhile.  The arithmetic is fp32 throughout.
#include "linear_common.cuh"

namespace gdr {
namespace {

constexpr int kTok = 8;   // tokens per stage

__device__ __forceinline__ float4 load4f(const float *p) { return *reinterpret_cast<const float4 *>(p); }
__device__ __forceinline__ float4 load4f(const __nv_bfloat16 *p) {
    const uint2 x = *reinterpret_cast<const uint2 *>(p);
    return make_float4(__uint_as_float(x.x << 16), __uint_as_float(x.x & 0xffff0000u),
                       __uint_as_float(x.y << 16), __uint_as_float(x.y & 0xffff0000u));
}

template <int DB, int DV, bool OUT, bool REV, typename In, typename Out>
__global__ void __launch_bounds__(DV < 32 ? 32 : DV)
scan_simt_kernel(const ScanArgs p) {
    constexpr int NT = DV < 32 ? 32 : DV;
    constexpr int ROWS = OUT ? 2 * DB + DV : DB + DV;      // floats per staged token: b, v, a
    constexpr int VECS = kTok * ROWS / 4;                  // float4 per stage
    constexpr int PER = (VECS + NT - 1) / NT;
    __shared__ __align__(16) float tile[2][kTok * ROWS];
    __shared__ int scratch[34];
    const int tid = threadIdx.x;
    const int slot = blockIdx.x / p.H, h = blockIdx.x % p.H;
    launch_dependents();
    wait_for_previous();
    if (OUT && blockIdx.x == 0 && tid == 0) *p.header = p.status_words;
    const Segment seg = find_segment(p, slot, !OUT, REV, scratch, NT);
    if (seg.n < 0) return;
    const bool last = seg.index == seg.count - 1;
    const int ha = h / (p.H / p.HA), hb = h / (p.H / p.HB), hv = h / (p.H / p.HV);
    const float decay = expf(clamp_log_gate(p.decay[h]));
    const float2 x2 = make_float2(decay, decay);
    const bool row = tid < DV;
    const size_t state_at = ((size_t)seg.n * p.H + h) * (DV * DB);

    float2 S[DB / 2];
#pragma unroll
    for (int i = 0; i < DB / 2; ++i) S[i] = make_float2(0.f, 0.f);
    if (row) {
        if (OUT && seg.index > 0) {
            const float4 *src = reinterpret_cast<const float4 *>(
                p.seg + ((size_t)(seg.state - 1) * p.H + h) * (DV * DB)) + tid;
#pragma unroll
            for (int i = 0; i < DB / 4; ++i) {
                const float4 x = src[i * DV];
                S[2 * i] = make_float2(x.x, x.y);
                S[2 * i + 1] = make_float2(x.z, x.w);
            }
        } else if (seg.index == 0 && p.s_in != nullptr && p.turned) {
            const float *src = p.s_in + state_at + tid;
#pragma unroll
            for (int i = 0; i < DB / 2; ++i) S[i] = make_float2(src[2 * i * DV], src[(2 * i + 1) * DV]);
        } else if (seg.index == 0 && p.s_in != nullptr) {
            const float4 *src = reinterpret_cast<const float4 *>(p.s_in + state_at + (size_t)tid * DB);
#pragma unroll
            for (int i = 0; i < DB / 4; ++i) {
                const float4 x = src[i];
                S[2 * i] = make_float2(x.x, x.y);
                S[2 * i + 1] = make_float2(x.z, x.w);
            }
        }
    }

    // token u of the scan, and element e (a multiple of 4) of its staged row
    auto token = [&](int u) { return (size_t)(seg.t0 + (REV ? seg.len - 1 - u : u)); };
    auto fetch = [&](int u, int e) {
        const size_t t = token(u);
        if (e < DB) return load4f(static_cast<const In *>(p.b) + (t * p.HB + hb) * DB + e);
        if (e < DB + DV) return load4f(static_cast<const In *>(p.v) + (t * p.HV + hv) * DV + (e - DB));
        return load4f(static_cast<const In *>(p.a) + (t * p.HA + ha) * DB + (e - DB - DV));
    };
    float4 next[PER];
    auto fetch_all = [&](int u0) {
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int at = (i * NT + tid) * 4, u = u0 + at / ROWS;
            next[i] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (at < kTok * ROWS && u < seg.len) next[i] = fetch(u, at % ROWS);
        }
    };
    if (seg.len > 0) fetch_all(0);
    for (int u0 = 0, buf = 0; u0 < seg.len; u0 += kTok, buf ^= 1) {
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int at = (i * NT + tid) * 4;
            if (at < kTok * ROWS) *reinterpret_cast<float4 *>(&tile[buf][at]) = next[i];
        }
        __syncthreads();
        if (u0 + kTok < seg.len) fetch_all(u0 + kTok);
        const int n = min(kTok, seg.len - u0);
        if (row) {
            for (int u = 0; u < n; ++u) {
                const float *t = &tile[buf][u * ROWS];
                const float4 *b4 = reinterpret_cast<const float4 *>(t);
                const float4 *a4 = reinterpret_cast<const float4 *>(t + DB + DV);
                const float v = t[DB + tid];
                const float2 v2 = make_float2(v, v);
                float2 o0 = make_float2(0.f, 0.f), o1 = o0;
#pragma unroll
                for (int i = 0; i < DB / 4; ++i) {
                    const float4 b = b4[i];
                    float2 s0 = S[2 * i], s1 = S[2 * i + 1];
                    if (!REV) {
                        s0 = __fmul2_rn(s0, x2);
                        s1 = __fmul2_rn(s1, x2);
                    }
                    s0 = __ffma2_rn(v2, make_float2(b.x, b.y), s0);
                    s1 = __ffma2_rn(v2, make_float2(b.z, b.w), s1);
                    if (OUT) {
                        const float4 a = a4[i];
                        o0 = __ffma2_rn(s0, make_float2(a.x, a.y), o0);
                        o1 = __ffma2_rn(s1, make_float2(a.z, a.w), o1);
                    }
                    if (REV) {
                        s0 = __fmul2_rn(s0, x2);
                        s1 = __fmul2_rn(s1, x2);
                    }
                    S[2 * i] = s0;
                    S[2 * i + 1] = s1;
                }
                if (OUT)
                    store_io(static_cast<Out *>(p.out) + (token(u0 + u) * p.H + h) * DV + tid,
                             (o0.x + o0.y) + (o1.x + o1.y));
            }
        }
    }
    if (row && !OUT) {
        float4 *dst = reinterpret_cast<float4 *>(p.seg + ((size_t)seg.state * p.H + h) * (DV * DB)) + tid;
#pragma unroll
        for (int i = 0; i < DB / 4; ++i)
            dst[i * DV] = make_float4(S[2 * i].x, S[2 * i].y, S[2 * i + 1].x, S[2 * i + 1].y);
    }
    if (row && OUT && last && p.s_out != nullptr) {
        float4 *dst = reinterpret_cast<float4 *>(p.s_out + state_at + (size_t)tid * DB);
#pragma unroll
        for (int i = 0; i < DB / 4; ++i)
            dst[i] = make_float4(S[2 * i].x, S[2 * i].y, S[2 * i + 1].x, S[2 * i + 1].y);
    }
}

template <int DB, int DV, typename In, typename Out>
cudaError_t launch_shape(const ScanArgs &p, bool reverse, bool states, bool after, cudaStream_t s) {
    constexpr int NT = DV < 32 ? 32 : DV;
    const unsigned grid = (unsigned)(states ? p.inner : p.slots) * p.H;
    if (states)
        return reverse ? launch_kernel(after, scan_simt_kernel<DB, DV, false, true, In, In>, grid, NT, 0, s, p)
                       : launch_kernel(after, scan_simt_kernel<DB, DV, false, false, In, In>, grid, NT, 0, s, p);
    return reverse ? launch_kernel(after, scan_simt_kernel<DB, DV, true, true, In, Out>, grid, NT, 0, s, p)
                   : launch_kernel(after, scan_simt_kernel<DB, DV, true, false, In, Out>, grid, NT, 0, s, p);
}

template <typename In, typename Out>
cudaError_t launch_dims(const ScanArgs &p, int d_b, int d_v, bool reverse, bool states, bool after,
                        cudaStream_t s) {
    switch (d_b * 1000 + d_v) {
        case 16016: return launch_shape<16, 16, In, Out>(p, reverse, states, after, s);
        case 16032: return launch_shape<16, 32, In, Out>(p, reverse, states, after, s);
        case 16064: return launch_shape<16, 64, In, Out>(p, reverse, states, after, s);
        case 16128: return launch_shape<16, 128, In, Out>(p, reverse, states, after, s);
        case 32016: return launch_shape<32, 16, In, Out>(p, reverse, states, after, s);
        case 32032: return launch_shape<32, 32, In, Out>(p, reverse, states, after, s);
        case 32064: return launch_shape<32, 64, In, Out>(p, reverse, states, after, s);
        case 32128: return launch_shape<32, 128, In, Out>(p, reverse, states, after, s);
        case 64016: return launch_shape<64, 16, In, Out>(p, reverse, states, after, s);
        case 64032: return launch_shape<64, 32, In, Out>(p, reverse, states, after, s);
        case 64064: return launch_shape<64, 64, In, Out>(p, reverse, states, after, s);
        case 64128: return launch_shape<64, 128, In, Out>(p, reverse, states, after, s);
        case 128016: return launch_shape<128, 16, In, Out>(p, reverse, states, after, s);
        case 128032: return launch_shape<128, 32, In, Out>(p, reverse, states, after, s);
        case 128064: return launch_shape<128, 64, In, Out>(p, reverse, states, after, s);
        case 128128: return launch_shape<128, 128, In, Out>(p, reverse, states, after, s);
    }
    return cudaErrorInvalidValue;
}

// ------------------------------------------------ states between segments ----

// X_0 = the first segment's state, X_s = x^{tokens of s} X_{s-1} + (state of s):
// every block takes 1024 elements along one sequence's segments.  All of them
// but the first in scan order are full (the last one's state is not needed).
constexpr int kJoinThreads = 256;

__global__ void __launch_bounds__(kJoinThreads)
scan_join_kernel(const ScanArgs p, int elements, bool reverse) {
    __shared__ int scratch[34];
    const int h = blockIdx.x % p.H;
    int slot = blockIdx.x / p.H;
    launch_dependents();
    wait_for_previous();
    // equal lengths: a block for each sequence, else for each state, of which the first goes on
    if (p.cu == nullptr) slot *= p.inner / p.N;
    const Segment seg = find_segment(p, slot, true, reverse, scratch, kJoinThreads);
    if (seg.n < 0 || seg.index != 0 || seg.count < 3) return;
    const int e = (blockIdx.y * kJoinThreads + threadIdx.x) * 4;
    if (e >= elements) return;
    const float w = expf(clamp_log_gate(p.decay[h]) * (float)p.seg_tokens);
    const size_t step = (size_t)p.H * elements / 4;
    float4 *at = reinterpret_cast<float4 *>(p.seg + ((size_t)seg.state * p.H + h) * elements + e);
    const int end = min(seg.count - 1, p.inner - seg.state);
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int s = 0; s < end; s += 8) {   // eight loads in flight
        float4 y[8];
#pragma unroll
        for (int u = 0; u < 8; ++u)
            if (s + u < end) y[u] = at[(size_t)(s + u) * step];
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            if (s + u >= end) break;
            x = make_float4(fmaf(w, x.x, y[u].x), fmaf(w, x.y, y[u].y), fmaf(w, x.z, y[u].z),
                            fmaf(w, x.w, y[u].w));
            if (s + u > 0) at[(size_t)(s + u) * step] = x;
        }
    }
}

// ------------------------------------------------------------- group sums ----

constexpr int kSumThreads = 256;

template <typename Out>
__global__ void __launch_bounds__(kSumThreads)
group_sum_kernel(const float *__restrict__ part, int64_t vecs, int group, int d4, Out *__restrict__ out) {
    launch_dependents();
    wait_for_previous();
    for (int64_t i = (int64_t)blockIdx.x * kSumThreads + threadIdx.x; i < vecs;
         i += (int64_t)gridDim.x * kSumThreads) {
        const int64_t head = i / d4;
        const float4 *src = reinterpret_cast<const float4 *>(part) + head * group * d4 + i % d4;
        float4 x = __ldcs(src);
        for (int g = 1; g < group; ++g) {
            const float4 y = __ldcs(src + (int64_t)g * d4);
            x = make_float4(x.x + y.x, x.y + y.y, x.z + y.z, x.w + y.w);
        }
        store_io(out + 4 * i, x.x);
        store_io(out + 4 * i + 1, x.y);
        store_io(out + 4 * i + 2, x.z);
        store_io(out + 4 * i + 3, x.w);
    }
}

// ------------------------------------------------------------ decode step ----

// S <- x S + v k^T, o = S q for one token per sequence: one read and one write
// of the fp32 state, which bounds it.  DK / 16 lanes share a row; every load of
// the state is issued before any arithmetic.  PASSES x (256 / lanes) rows per
// block: a whole head where there are enough heads to fill the GPU, else one
// pass, so that few heads still spread over the SMs.
constexpr int kStepThreads = 256;

template <int DK, int PASSES, typename IoT>
__global__ void __launch_bounds__(kStepThreads)
linear_step_kernel(const IoT *__restrict__ q, const IoT *__restrict__ k, const IoT *__restrict__ v,
                   const float *__restrict__ decay, float *__restrict__ state, int Hqk, int H,
                   int DV, IoT *__restrict__ o) {
    constexpr int LPR = DK / 16;
    constexpr int RP = kStepThreads / LPR;
    const size_t nh = blockIdx.x;
    const int h = (int)(nh % H);
    const size_t qh = (nh / H) * Hqk + h / (H / Hqk);
    const int lane = threadIdx.x % LPR;
    const int r0 = blockIdx.y * (PASSES * RP) + threadIdx.x / LPR;
    float4 *S = reinterpret_cast<float4 *>(state + nh * (size_t)DV * DK) + lane;

    float4 s[PASSES][4];
#pragma unroll
    for (int pp = 0; pp < PASSES; ++pp)
#pragma unroll
        for (int m = 0; m < 4; ++m) {
            const int r = r0 + pp * RP;
            s[pp][m] = r < DV ? __ldcs(S + (size_t)r * (DK / 4) + LPR * m) : make_float4(0.f, 0.f, 0.f, 0.f);
        }
    float4 kf[4], qf[4];
#pragma unroll
    for (int m = 0; m < 4; ++m) {
        kf[m] = load4f(k + qh * DK + 4 * (lane + LPR * m));
        qf[m] = load4f(q + qh * DK + 4 * (lane + LPR * m));
    }
    const float x = expf(clamp_log_gate(decay[h]));
#pragma unroll
    for (int pp = 0; pp < PASSES; ++pp) {
        const int r = r0 + pp * RP;
        const float vr = r < DV ? to_f32(v[nh * DV + r]) : 0.f;
        float out = 0.f;
#pragma unroll
        for (int m = 0; m < 4; ++m) {
            float4 &y = s[pp][m];
            y = make_float4(fmaf(x, y.x, vr * kf[m].x), fmaf(x, y.y, vr * kf[m].y),
                            fmaf(x, y.z, vr * kf[m].z), fmaf(x, y.w, vr * kf[m].w));
            out = fmaf(y.x, qf[m].x, fmaf(y.y, qf[m].y, fmaf(y.z, qf[m].z, fmaf(y.w, qf[m].w, out))));
            if (r < DV) __stcs(S + (size_t)r * (DK / 4) + LPR * m, y);
        }
#pragma unroll
        for (int off = LPR / 2; off > 0; off >>= 1) out += __shfl_xor_sync(0xffffffffu, out, off);
        if (r < DV && lane == 0) store_io(o + nh * DV + r, out);
    }
}

template <int DK, typename IoT>
cudaError_t launch_step(const void *q, const void *k, const void *v, const float *decay,
                        float *state, int N, int Hqk, int H, int DV, void *o, cudaStream_t s) {
    constexpr int RP = kStepThreads * 16 / DK;
    constexpr int ALL = RP >= 128 ? 1 : 128 / RP;
    const size_t heads = (size_t)N * H;
    const IoT *qq = static_cast<const IoT *>(q), *kk = static_cast<const IoT *>(k);
    const IoT *vv = static_cast<const IoT *>(v);
    IoT *oo = static_cast<IoT *>(o);
    if (ALL > 1 && heads < 296 && DV > RP)
        linear_step_kernel<DK, 1, IoT><<<dim3((unsigned)heads, (DV + RP - 1) / RP), kStepThreads, 0, s>>>(
            qq, kk, vv, decay, state, Hqk, H, DV, oo);
    else
        linear_step_kernel<DK, ALL, IoT><<<(unsigned)heads, kStepThreads, 0, s>>>(
            qq, kk, vv, decay, state, Hqk, H, DV, oo);
    return cudaGetLastError();
}

template <typename IoT>
cudaError_t launch_step_dk(const void *q, const void *k, const void *v, const float *decay,
                           float *state, int N, int Hqk, int H, int DK, int DV, void *o,
                           cudaStream_t s) {
    switch (DK) {
        case 16: return launch_step<16, IoT>(q, k, v, decay, state, N, Hqk, H, DV, o, s);
        case 32: return launch_step<32, IoT>(q, k, v, decay, state, N, Hqk, H, DV, o, s);
        case 64: return launch_step<64, IoT>(q, k, v, decay, state, N, Hqk, H, DV, o, s);
        default: return launch_step<128, IoT>(q, k, v, decay, state, N, Hqk, H, DV, o, s);
    }
}

}  // namespace

cudaError_t launch_scan_simt(const ScanArgs &p, int d_b, int d_v, bool reverse, bool states,
                             bool bf16, bool out_f32, bool after, cudaStream_t stream) {
    if (!bf16) return launch_dims<float, float>(p, d_b, d_v, reverse, states, after, stream);
    if (out_f32) return launch_dims<__nv_bfloat16, float>(p, d_b, d_v, reverse, states, after, stream);
    return launch_dims<__nv_bfloat16, __nv_bfloat16>(p, d_b, d_v, reverse, states, after, stream);
}

cudaError_t launch_scan_join(const ScanArgs &p, int elements, bool reverse, cudaStream_t stream) {
    const dim3 grid((unsigned)(p.cu == nullptr ? p.N : p.inner) * p.H, (elements / 4 + kJoinThreads - 1) / kJoinThreads);
    return launch_kernel(true, scan_join_kernel, grid, kJoinThreads, 0, stream, p, elements, reverse);
}

cudaError_t launch_group_sum(const float *part, int64_t T, int H_qk, int group, int d, bool bf16,
                             void *out, cudaStream_t stream) {
    const int64_t vecs = T * H_qk * (d / 4);
    const unsigned grid = (unsigned)std::min<int64_t>((vecs + kSumThreads - 1) / kSumThreads, 148 * 16);
    if (bf16)
        return launch_kernel(true, group_sum_kernel<__nv_bfloat16>, dim3(grid), kSumThreads, 0, stream, part, vecs,
                             group, d / 4, static_cast<__nv_bfloat16 *>(out));
    return launch_kernel(true, group_sum_kernel<float>, dim3(grid), kSumThreads, 0, stream, part, vecs, group, d / 4,
                         static_cast<float *>(out));
}

cudaError_t launch_linear_decode(const void *q, const void *k, const void *v, const float *decay,
                                 float *state, int N, int Hqk, int H, int DK, int DV, bool bf16,
                                 void *o, cudaStream_t stream) {
    return bf16 ? launch_step_dk<__nv_bfloat16>(q, k, v, decay, state, N, Hqk, H, DK, DV, o, stream)
                : launch_step_dk<float>(q, k, v, decay, state, N, Hqk, H, DK, DV, o, stream);
}

}  // namespace gdr
