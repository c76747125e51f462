// Linear attention with a decay for each head on the CUDA cores (fp32 or bf16
// inputs, any served d), the passes between segments, and the decode step.
//
// The scan of linear_common.cuh in tiles of eight tokens, all in fp32.  With u and
// j the places of a tile of n tokens in scan order and x = e^g,
//
//     o_u = x^{u+1-r} S a_u + sum_{j<=u} x^{u-j} (a_u . b_j) v_j
//     S  <- x^n S + sum_j x^{n-1+r-j} v_j b_j^T
//
// The state stays in registers: a thread has 32 columns (every SPL-th group of
// four) of two rows, so that each 16 bytes of a or b read from shared memory
// meet four packed products, and eight outputs run side by side.  The 36 dots
// a_u . b_j of a tile are made one tile ahead by a few of the threads; a, b and v
// of the tile after that are on their way in registers.  One barrier a tile.
// Against a loop over single tokens this takes two products a state element and
// token instead of three, and rounds the state once a tile.
#include "linear_common.cuh"

namespace gdr {
namespace {

constexpr int kTok = 8;   // tokens of a tile

__device__ __forceinline__ float4 load4f(const float *p) { return *reinterpret_cast<const float4 *>(p); }
__device__ __forceinline__ float4 load4f(const __nv_bfloat16 *p) {
    const uint2 x = *reinterpret_cast<const uint2 *>(p);
    return make_float4(__uint_as_float(x.x << 16), __uint_as_float(x.x & 0xffff0000u),
                       __uint_as_float(x.y << 16), __uint_as_float(x.y & 0xffff0000u));
}

template <int DB, int DV>
struct Tiling {
    static constexpr int COLS = DB < 32 ? DB : 32;    // columns of a thread
    static constexpr int SPL = DB / COLS;             // threads of a row
    static constexpr int RT = DV / 2;                 // its rows: r and r + RT
    static constexpr int USED = RT * SPL;
    static constexpr int NT = USED < 32 ? 32 : USED;
    static constexpr int LD = DB + 4;                 // row stride of a and b: eight rows cover all banks
};

template <int DB, int DV, bool OUT, bool REV, typename In, typename Out>
__global__ void __launch_bounds__(Tiling<DB, DV>::NT)
scan_simt_kernel(const ScanArgs p) {
    using Ti = Tiling<DB, DV>;
    constexpr int NT = Ti::NT, SPL = Ti::SPL, RT = Ti::RT, LD = Ti::LD, M = Ti::COLS / 4;
    constexpr int ROW = DB + DV + (OUT ? DB : 0);          // floats of a token: b, v, a
    constexpr int PER = (kTok * ROW / 4 + NT - 1) / NT;    // of their groups of four, for each thread
    __shared__ __align__(16) float sb[3][kTok][LD], sa[OUT ? 3 : 1][OUT ? kTok : 1][LD], sv[3][kTok][DV];
    __shared__ __align__(16) float dots[2][kTok][kTok];
    __shared__ float pw[kTok + 2];
    __shared__ int scratch[34];
    const int tid = threadIdx.x;
    const int slot = blockIdx.x / p.H, h = blockIdx.x % p.H;
    launch_dependents();
    if (!OUT || !p.late) wait_for_previous();
    if (OUT && blockIdx.x == 0 && tid == 0) *p.header = p.status_words;
    const Segment seg = find_segment(p, slot, !OUT, REV, scratch, NT);
    if (seg.n < 0) return;
    // a late pass runs beside the one before, but not where it reads the states between segments
    const bool beside = OUT && p.late && seg.index == 0;
    if (OUT && p.late && !beside) wait_for_previous();
    const bool last = seg.index == seg.count - 1;
    const int ha = h / (p.H / p.HA), hb = h / (p.H / p.HB), hv = h / (p.H / p.HV);
    if (tid <= kTok) pw[tid] = expf(clamp_log_gate(p.decay[h]) * (float)tid);
    const bool used = tid < Ti::USED;
    const int split = tid % SPL, r0 = used ? tid / SPL : 0, r1 = r0 + RT;
    const size_t state_at = ((size_t)seg.n * p.H + h) * (DV * DB);

    float2 S[2][2 * M];
#pragma unroll
    for (int i = 0; i < 2 * M; ++i) S[0][i] = S[1][i] = make_float2(0.f, 0.f);
    // a row's float4 number m of this thread is number split + SPL m of the row
    auto each = [&](auto f) {
#pragma unroll
        for (int q = 0; q < 2; ++q)
#pragma unroll
            for (int m = 0; m < M; ++m) f(q, m, q == 0 ? r0 : r1, split + SPL * m);
    };
    // the state that enters: between segments, the caller's, or zero
    const float *from = OUT && seg.index > 0 ? p.seg + ((size_t)(seg.state - 1) * p.H + h) * (DV * DB)
                        : seg.index > 0 || p.s_in == nullptr ? nullptr : p.s_in + state_at;
    if (used && from != nullptr) {
        const bool turned = seg.index > 0 ? p.seg_turned : p.turned;
        each([&](int q, int m, int r, int c) {
            float4 x;
            if (turned) x = make_float4(from[(4 * c) * DV + r], from[(4 * c + 1) * DV + r], from[(4 * c + 2) * DV + r], from[(4 * c + 3) * DV + r]);
            else x = reinterpret_cast<const float4 *>(from)[r * (DB / 4) + c];
            S[q][2 * m] = make_float2(x.x, x.y);
            S[q][2 * m + 1] = make_float2(x.z, x.w);
        });
    }

    // the token at place u of the scan
    auto token = [&](int u) { return (size_t)(seg.t0 + (REV ? seg.len - 1 - u : u)); };
    // what this thread fetches of a tile: where its groups lie in the first one, and how
    // far the next tile's are
    float4 next[PER];
    const In *src[PER];
    int64_t step[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int at = (i * NT + tid) * 4, u = at / ROW, e = at % ROW;
        const int64_t t = seg.t0 + (REV ? seg.len - 1 - u : u);
        const int64_t heads = e < DB ? (int64_t)p.HB * DB : e < DB + DV ? (int64_t)p.HV * DV : (int64_t)p.HA * DB;
        const In *from = e < DB ? static_cast<const In *>(p.b) + hb * DB + e
                       : e < DB + DV ? static_cast<const In *>(p.v) + hv * DV + (e - DB)
                                     : static_cast<const In *>(p.a) + ha * DB + (e - DB - DV);
        src[i] = from + t * heads;
        step[i] = (REV ? -kTok : kTok) * heads;
    }
    auto fetch = [&](int u0) {
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int at = (i * NT + tid) * 4;
            next[i] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (at < kTok * ROW && u0 + at / ROW < seg.len) next[i] = load4f(src[i]);
            src[i] += step[i];
        }
    };
    auto put = [&](int buf) {
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int at = (i * NT + tid) * 4, u = at / ROW, e = at % ROW;
            if (at >= kTok * ROW) continue;
            float *dst = e < DB ? &sb[buf][u][e] : e < DB + DV ? &sv[buf][u][e - DB] : &sa[OUT ? buf : 0][OUT ? u : 0][e - DB - DV];
            *reinterpret_cast<float4 *>(dst) = next[i];
        }
    };
    auto make_dots = [&](int buf, int to) {
        for (int i = tid; i < kTok * kTok; i += NT) {
            const int u = i / kTok, j = i % kTok;
            if (j > u) continue;
            float2 s0 = make_float2(0.f, 0.f), s1 = s0;
#pragma unroll 8
            for (int c = 0; c < DB; c += 4) {
                const float4 a = *reinterpret_cast<const float4 *>(&sa[OUT ? buf : 0][OUT ? u : 0][c]);
                const float4 b = *reinterpret_cast<const float4 *>(&sb[buf][j][c]);
                s0 = __ffma2_rn(make_float2(a.x, a.y), make_float2(b.x, b.y), s0);
                s1 = __ffma2_rn(make_float2(a.z, a.w), make_float2(b.z, b.w), s1);
            }
            dots[to][u][j] = ((s0.x + s0.y) + (s1.x + s1.y)) * pw[u - j];
        }
    };
    const int tiles = (seg.len + kTok - 1) / kTok;
    if (tiles > 0) {
        fetch(0);
        put(0);
        fetch(kTok);
        __syncthreads();
        if (OUT) make_dots(0, 0);
    }
    for (int k = 0, buf = 0; k < tiles; ++k) {
        const int after = buf == 2 ? 0 : buf + 1, n = min(kTok, seg.len - k * kTok);
        put(after);
        __syncthreads();
        if (k + 1 < tiles) {
            fetch((k + 2) * kTok);
            if (OUT) make_dots(after, (k + 1) & 1);
        }
        float v[2][kTok];
#pragma unroll
        for (int j = 0; j < kTok; ++j) {
            v[0][j] = sv[buf][j][r0];
            v[1][j] = sv[buf][j][r1];
        }
        if (OUT) {
            float2 acc[2][kTok];
#pragma unroll
            for (int u = 0; u < kTok; ++u) acc[0][u] = acc[1][u] = make_float2(0.f, 0.f);
#pragma unroll
            for (int m = 0; m < M; ++m)
#pragma unroll
                for (int u = 0; u < kTok; ++u) {
                    const float4 a = *reinterpret_cast<const float4 *>(&sa[OUT ? buf : 0][OUT ? u : 0][4 * (split + SPL * m)]);
#pragma unroll
                    for (int q = 0; q < 2; ++q)
                        acc[q][u] = __ffma2_rn(S[q][2 * m + 1], make_float2(a.z, a.w),
                                               __ffma2_rn(S[q][2 * m], make_float2(a.x, a.y), acc[q][u]));
                }
            // the row's threads add up; each stores every SPL-th token
            Out *dst = static_cast<Out *>(p.out) + (token(k * kTok) * p.H + h) * DV;
            const int64_t row = REV ? -(int64_t)p.H * DV : (int64_t)p.H * DV;
#pragma unroll
            for (int u = 0; u < kTok; ++u) {
                float o[2];
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    o[q] = acc[q][u].x + acc[q][u].y;
#pragma unroll
                    for (int off = SPL / 2; off > 0; off >>= 1) o[q] += __shfl_xor_sync(0xffffffffu, o[q], off);
                    o[q] *= pw[REV ? u : u + 1];
                }
#pragma unroll
                for (int j = 0; j <= u; j += 4) {
                    const float4 w = *reinterpret_cast<const float4 *>(&dots[k & 1][u][j]);
                    const float ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (j + e <= u) {
                            o[0] = fmaf(ws[e], v[0][j + e], o[0]);
                            o[1] = fmaf(ws[e], v[1][j + e], o[1]);
                        }
                }
                if (used && u % SPL == split && u < n) {
                    store_io(dst + u * row + r0, o[0]);
                    store_io(dst + u * row + r1, o[1]);
                }
            }
        }
#pragma unroll
        for (int j = 0; j < kTok; ++j) {
            const float w = pw[max(n - 1 - j, 0) + (REV ? 1 : 0)];      // (the tokens behind n are zeros)
            v[0][j] *= w;
            v[1][j] *= w;
        }
        const float2 xn = make_float2(pw[n], pw[n]);
#pragma unroll
        for (int m = 0; m < M; ++m) {
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                S[q][2 * m] = __fmul2_rn(S[q][2 * m], xn);
                S[q][2 * m + 1] = __fmul2_rn(S[q][2 * m + 1], xn);
            }
#pragma unroll
            for (int j = 0; j < kTok; ++j) {
                const float4 b = *reinterpret_cast<const float4 *>(&sb[buf][j][4 * (split + SPL * m)]);
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    const float2 w = make_float2(v[q][j], v[q][j]);
                    S[q][2 * m] = __ffma2_rn(w, make_float2(b.x, b.y), S[q][2 * m]);
                    S[q][2 * m + 1] = __ffma2_rn(w, make_float2(b.z, b.w), S[q][2 * m + 1]);
                }
            }
        }
        buf = after;
    }
    if (beside) wait_for_previous();
    float *out_state = OUT ? (last ? p.s_out : nullptr) : p.seg;
    if (used && out_state != nullptr) {
        float4 *dst = reinterpret_cast<float4 *>(out_state + (OUT ? state_at : ((size_t)seg.state * p.H + h) * (DV * DB)));
        each([&](int q, int m, int r, int c) {
            dst[r * (DB / 4) + c] = make_float4(S[q][2 * m].x, S[q][2 * m].y, S[q][2 * m + 1].x, S[q][2 * m + 1].y);
        });
    }
}

template <int DB, int DV, typename In, typename Out>
cudaError_t launch_shape(const ScanArgs &p, bool reverse, bool states, bool after, cudaStream_t s) {
    constexpr int NT = Tiling<DB, DV>::NT;
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
// every block takes some of the elements along one sequence's segments.  All of them
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
    const float w = expf(clamp_log_gate(p.decay[h]) * (float)p.seg_tokens);
    const size_t step = (size_t)p.H * elements / 4;
    const int end = min(seg.count - 1, p.inner - seg.state);
    for (int e = (blockIdx.y * kJoinThreads + threadIdx.x) * 4; e < elements; e += gridDim.y * kJoinThreads * 4) {
        float4 *at = reinterpret_cast<float4 *>(p.seg + ((size_t)seg.state * p.H + h) * elements + e);
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
}

// ------------------------------------------------------------- group sums ----

constexpr int kSumThreads = 256;

// (Tokens behind the last packed sequence have no parts: they stay as they are.)
template <typename Out>
__global__ void __launch_bounds__(kSumThreads)
group_sum_kernel(const float *__restrict__ part0, const float *__restrict__ part1, const int32_t *__restrict__ cu,
                 int N, int64_t T, int H_qk, int group, int d4, Out *__restrict__ out0, Out *__restrict__ out1) {
    const float *part = blockIdx.y == 0 ? part0 : part1;
    Out *out = blockIdx.y == 0 ? out0 : out1;
    wait_for_previous();
    int64_t first = 0, end = T * H_qk * d4;
    if (cu != nullptr) {
        first = min(max((int64_t)cu[0], (int64_t)0), T) * H_qk * d4;
        end = min(max((int64_t)cu[N], (int64_t)0), T) * H_qk * d4;
    }
    for (int64_t i = first + (int64_t)blockIdx.x * kSumThreads + threadIdx.x; i < end;
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
    // packed lengths: most blocks only find that they have nothing to do, so there are fewer
    const int all = (elements / 4 + kJoinThreads - 1) / kJoinThreads;
    const dim3 grid((unsigned)(p.cu == nullptr ? p.N : p.inner) * p.H, p.cu == nullptr ? all : std::min(all, 4));
    return launch_kernel(true, scan_join_kernel, grid, kJoinThreads, 0, stream, p, elements, reverse);
}

cudaError_t launch_group_sum(const float *const (&part)[2], const int32_t *cu, int N, int64_t T, int H_qk,
                             int group, int d, bool bf16, void *const (&out)[2], cudaStream_t stream) {
    const int64_t groups = (T * H_qk * (d / 4) + kSumThreads - 1) / kSumThreads;
    const dim3 grid((unsigned)std::min<int64_t>(groups, 148 * 8), 2);
    if (bf16)
        return launch_kernel(true, group_sum_kernel<__nv_bfloat16>, grid, kSumThreads, 0, stream, part[0], part[1], cu, N,
                             T, H_qk, group, d / 4, static_cast<__nv_bfloat16 *>(out[0]),
                             static_cast<__nv_bfloat16 *>(out[1]));
    return launch_kernel(true, group_sum_kernel<float>, grid, kSumThreads, 0, stream, part[0], part[1], cu, N, T, H_qk,
                         group, d / 4, static_cast<float *>(out[0]), static_cast<float *>(out[1]));
}

cudaError_t launch_linear_decode(const void *q, const void *k, const void *v, const float *decay,
                                 float *state, int N, int Hqk, int H, int DK, int DV, bool bf16,
                                 void *o, cudaStream_t stream) {
    return bf16 ? launch_step_dk<__nv_bfloat16>(q, k, v, decay, state, N, Hqk, H, DK, DV, o, stream)
                : launch_step_dk<float>(q, k, v, decay, state, N, Hqk, H, DK, DV, o, stream);
}

}  // namespace gdr
