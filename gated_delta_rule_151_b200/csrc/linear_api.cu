// C ABI of linear attention with a decay for each head: argument checks, the
// plan (how sequences are cut into segments), workspace layout and launches.
#include <algorithm>
#include <cmath>
#include <cstdint>

#include "api_common.h"
#include "common.cuh"
#include "linear_common.cuh"

namespace gdr {
namespace {

using api::apart;
using api::given16;
using api::head_dim;
using api::io_type;
using api::maybe16;
using api::Range;

constexpr size_t kHeader = 256;
constexpr int kSMs = 148;

size_t up256(size_t x) { return (x + 255) & ~size_t(255); }

struct Plan {
    int seg_tokens, slots, inner;
};

// Measured costs, in microseconds, of a 64-token block of one head in the output and
// in the state pass: alone on an SM, and the SM's time for it among others.  The
// tensor-core CTAs have an SM to themselves; several of the others share one.
struct Costs {
    bool exclusive;
    double out_alone, out_shared, state_alone, state_shared;
    double cta, join;   // beside: a CTA's start and end; the pass between segments
};

bool tensor_cores(int d_k, int d_v, bool bf16) { return bf16 && d_k == 128 && d_v == 128; }

Costs costs_of(int d_k, int d_v, bool bf16) {
    if (tensor_cores(d_k, d_v, bf16)) return Costs{true, 2.1, 2.1, 0.9, 0.9, 4.0, 5.0};
    const double x = (double)d_k * d_v / 16384;
    return Costs{false, 9 + 28 * x, 29 * x, 4 + 10 * x, 12 * x, 3.0, 4.0};
}

// A pass over `items` segments of at most `blocks` blocks, `work` blocks in all.
double pass_time(const Costs &c, double items, double blocks, double work, double alone, double shared, bool even) {
    const double one = blocks * alone + c.cta;
    if (c.exclusive && even) return std::ceil(items / kSMs) * one;
    if (items <= kSMs) return one;
    const double tail = even ? 0 : 0.5 * one;    // unequal segments end at different times
    return std::max(one, (work * shared + (c.exclusive ? items * c.cta : 0)) / kSMs + tail);
}

// The segment length whose passes end first by these costs.  Packed lengths are not
// known here: they are taken to lie around their mean, up to twice of it, so that
// with a segment below that some sequences are cut.
Plan make_plan(int N, int total_T, int H, int d_k, int d_v, bool bf16, bool equal) {
    const Costs c = costs_of(d_k, d_v, bf16);
    const double state_bytes = (double)H * d_k * d_v * 4, most_bytes = 128e6;
    const int len = total_T / N;
    const int64_t total = std::max<int64_t>(1, ((int64_t)total_T + kScanBlock - 1) / kScanBlock);
    const int64_t own = std::max(1, (len + kScanBlock - 1) / kScanBlock);         // blocks of an equal sequence
    const int64_t longest = equal ? own : std::min<int64_t>(total, 2 * ((total + N - 1) / N));
    const double work = (double)(equal ? own * N : total) * H;
    auto segments = [&](int64_t per) -> double {
        return equal ? (double)N * ((own + per - 1) / per) : per >= longest ? N : (double)total / per + 0.5 * N;
    };
    int64_t best = longest;
    double least = pass_time(c, (double)N * H, (double)longest, work, c.out_alone, c.out_shared, equal);
    for (int64_t per = 1; per < longest; per += per < 64 ? 1 : per / 32) {
        const double all = segments(per), inner = std::max(0.0, all - N);
        if (inner * state_bytes > most_bytes) continue;
        const double t = pass_time(c, inner * H, (double)per, inner * H * per, c.state_alone, c.state_shared, equal) +
                         pass_time(c, all * H, (double)per, work, c.out_alone, c.out_shared, equal) + c.join +
                         inner * state_bytes / 1.5e6;    // the join reads and writes them: 3 TB/s
        if (t < least) {
            least = t;
            best = per;
        }
    }
    if (!equal) {
        // a sequence far beyond the assumed lengths is cut all the same, as finely as the
        // states fit
        if (best == longest) best = std::max<int64_t>(2 * longest, 16);
        best = std::max<int64_t>(best, (int64_t)std::ceil((double)total * state_bytes / most_bytes));
    }
    Plan p;
    p.seg_tokens = (int)std::min<int64_t>(best, INT32_MAX / kScanBlock) * kScanBlock;
    if (equal) {
        const int n = segments_of(len, p.seg_tokens);
        p.slots = N * n;
        p.inner = N * (n - 1);
    } else {
        p.inner = total_T / p.seg_tokens;
        p.slots = N + p.inner;
    }
    return p;
}

// Workspace of one call: header, status words of every pass, a copy of the
// incoming state, the states between segments (forward scan, reverse scan), fp32
// partial gradients.
struct Layout {
    size_t status, copy, seg[2], part[2], total;
    uint32_t words;
};

Layout make_layout(const Plan &p, int N, int total_T, int H_qk, int H, int d_k, int d_v,
                   bool backward) {
    Layout l;
    const size_t state = (size_t)H * d_k * d_v * 4;
    l.words = (uint32_t)((size_t)(backward ? 3 * p.slots + 2 * p.inner : p.slots + p.inner) * H);
    l.status = kHeader;
    l.copy = l.status + up256((size_t)l.words * 4);
    l.seg[0] = l.copy + (p.inner > 0 && !backward ? up256(N * state) : 0);
    l.seg[1] = l.seg[0] + up256(p.inner * state);
    const size_t part = backward && H != H_qk ? up256((size_t)total_T * H * d_k * 4) : 0;
    l.part[0] = l.seg[1] + (backward ? up256(p.inner * state) : 0);
    l.part[1] = l.part[0] + part;
    l.total = l.part[1] + part;
    return l;
}

size_t workspace_bytes(int N, int total_T, int H_qk, int H, int d_k, int d_v, bool bf16,
                       bool backward) {
    if (N == 0 || total_T == 0) return 0;
    size_t most = 0;
    for (int equal = 0; equal < 2; ++equal) {
        if (equal && total_T % N != 0) continue;
        const Plan p = make_plan(N, total_T, H, d_k, d_v, bf16, equal != 0);
        most = std::max(most, make_layout(p, N, total_T, H_qk, H, d_k, d_v, backward).total);
    }
    return most;
}

struct Call {
    const int32_t *cu;
    const float *decay;
    int N, total_T, H;
    Plan plan;
    Layout lay;
    uint8_t *ws;
    bool bf16;
    cudaStream_t stream;
    uint32_t used;   // status words handed out
    bool launched;   // a kernel of this call went before
    cudaError_t error;
    struct {
        const void *base;
        int heads;
        CUtensorMap map;
    } maps[4];       // of the call's bf16 tensors: each is made once
    int map_count;

    void begin(const int32_t *cu_, const float *decay_, int N_, int T_, int H_, const Plan &plan_, const Layout &lay_,
               void *ws_, bool bf16_, cudaStream_t stream_) {
        cu = cu_; decay = decay_; N = N_; total_T = T_; H = H_; plan = plan_; lay = lay_;
        ws = static_cast<uint8_t *>(ws_);
        bf16 = bf16_; stream = stream_;
        used = 0; launched = false; error = cudaSuccess; map_count = 0;
    }

    const CUtensorMap *map_of(const void *base, int heads) {
        for (int i = 0; i < map_count; ++i)
            if (maps[i].base == base && maps[i].heads == heads) return &maps[i].map;
        if (map_count == 4 || !scan_tile_map(&maps[map_count].map, base, total_T, heads)) return nullptr;
        maps[map_count].base = base;
        maps[map_count].heads = heads;
        return &maps[map_count++].map;
    }

    // A scan's arguments; `buffer`: which states between segments it goes by.
    ScanArgs args(const void *a, int HA, const void *b, int HB, const void *v, int HV, const float *s_in,
                  bool turned, float *s_out, void *out, int buffer, bool seg_turned) const {
        ScanArgs p;
        p.a = a; p.b = b; p.v = v;
        p.out = out;
        p.decay = decay;
        p.s_in = s_in;
        p.s_out = s_out;
        p.seg = reinterpret_cast<float *>(ws + lay.seg[buffer]);
        p.header = reinterpret_cast<uint32_t *>(ws);
        p.status = nullptr;
        p.status_words = 0;
        p.cu = cu;
        p.N = N; p.total_T = total_T; p.H = H;
        p.HA = HA; p.HB = HB; p.HV = HV;
        p.seg_tokens = plan.seg_tokens;
        p.slots = plan.slots;
        p.inner = plan.inner;
        p.turned = turned;
        p.seg_turned = seg_turned;
        p.late = 0;
        return p;
    }

    // One pass, and the pass between segments; nothing after an error.
    void pass(ScanArgs p, int d_b, int d_v, bool reverse, bool states, bool out_f32, bool late = false) {
        if (error != cudaSuccess || (states && plan.inner == 0)) return;
        const bool tc = tensor_cores(d_b, d_v, bf16);
        p.status = reinterpret_cast<uint32_t *>(ws + lay.status) + used;
        p.status_words = tc ? lay.words : 0;
        p.late = late;
        used += (uint32_t)(states ? plan.inner : plan.slots) * H;
        if (tc) {
            const CUtensorMap *a = map_of(p.a, p.HA), *b = map_of(p.b, p.HB), *v = map_of(p.v, p.HV);
            error = a == nullptr || b == nullptr || v == nullptr
                        ? cudaErrorInvalidValue
                        : launch_scan_tc(*a, *b, *v, p, reverse, states, out_f32, launched, stream);
        } else {
            error = launch_scan_simt(p, d_b, d_v, reverse, states, bf16, out_f32, launched, stream);
        }
        launched = true;
    }
    void join(const ScanArgs &p, int d_b, int d_v, bool reverse) {
        // (of two segments the first one's own state is what the second starts from)
        if (error != cudaSuccess || plan.inner == 0 || (cu == nullptr && plan.inner == N)) return;
        error = launch_scan_join(p, d_b * d_v, reverse, stream);
    }
};

// Shapes both directions share; GDR_OK with *todo = false when nothing is to be run.
gdr_status_t check_shape(int32_t num_seqs, int32_t total_T, int32_t H_qk, int32_t H, int32_t d_k,
                         int32_t d_v, gdr_dtype_t io_dtype, bool equal) {
    if (num_seqs < 0 || total_T < 0 || H < 1 || H_qk < 1 || H % H_qk != 0) return GDR_ERR_INVALID_ARG;
    if (!head_dim(d_k) || !head_dim(d_v) || !io_type(io_dtype)) return GDR_ERR_INVALID_ARG;
    if (num_seqs == 0 && total_T != 0) return GDR_ERR_INVALID_ARG;
    if (equal && num_seqs > 0 && total_T % num_seqs != 0) return GDR_ERR_INVALID_ARG;
    // token, grid and status indices are 32-bit
    if ((int64_t)total_T * H > INT32_MAX || (int64_t)num_seqs * H > INT32_MAX / 8)
        return GDR_ERR_INVALID_ARG;
    return GDR_OK;
}

cudaError_t pass_state(float *dst, const float *src, size_t bytes, cudaStream_t s) {
    if (dst == nullptr || dst == src || bytes == 0) return cudaSuccess;
    if (src == nullptr) return cudaMemsetAsync(dst, 0, bytes, s);
    return cudaMemcpyAsync(dst, src, bytes, cudaMemcpyDeviceToDevice, s);
}

gdr_status_t status_of(cudaError_t e) { return e == cudaSuccess ? GDR_OK : GDR_ERR_CUDA; }

}  // namespace
}  // namespace gdr

using namespace gdr;

extern "C" {

gdr_status_t gdr_linear_workspace_size(int32_t num_seqs, int32_t total_T, int32_t H_qk, int32_t H,
                                       int32_t d_k, int32_t d_v, gdr_dtype_t io_dtype,
                                       int32_t backward, size_t *bytes) {
    if (bytes == nullptr) return GDR_ERR_INVALID_ARG;
    const gdr_status_t st = check_shape(num_seqs, total_T, H_qk, H, d_k, d_v, io_dtype, false);
    if (st != GDR_OK) return st;
    *bytes = workspace_bytes(num_seqs, total_T, H_qk, H, d_k, d_v, io_dtype == GDR_BF16,
                             backward != 0);
    return GDR_OK;
}

gdr_status_t gdr_linear_prefill(const void *q, const void *k, const void *v, const float *decay,
                                const float *initial_state, const int32_t *cu_seqlens,
                                int32_t num_seqs, int32_t total_T, int32_t H_qk, int32_t H,
                                int32_t d_k, int32_t d_v, gdr_dtype_t io_dtype, void *o,
                                float *final_state, void *workspace, size_t workspace_bytes,
                                void *stream) {
    const bool equal = cu_seqlens == nullptr;
    gdr_status_t st = check_shape(num_seqs, total_T, H_qk, H, d_k, d_v, io_dtype, equal);
    if (st != GDR_OK) return st;
    if (!maybe16(initial_state) || !maybe16(final_state) || !api::aligned(cu_seqlens, 4))
        return GDR_ERR_INVALID_ARG;
    if (num_seqs == 0) return GDR_OK;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const size_t state = (size_t)num_seqs * H * d_k * d_v * 4;
    const size_t e = io_dtype == GDR_BF16 ? 2 : 4, T = (size_t)total_T;
    if (total_T > 0 && (!given16(q) || !given16(k) || !given16(v) || !given16(o) || decay == nullptr ||
                        !api::aligned(decay, 4)))
        return GDR_ERR_INVALID_ARG;
    const Plan plan = total_T > 0 ? make_plan(num_seqs, total_T, H, d_k, d_v, io_dtype == GDR_BF16, equal) : Plan{kScanBlock, 0, 0};
    const Layout lay = make_layout(plan, num_seqs, total_T, H_qk, H, d_k, d_v, false);
    const size_t need = total_T > 0 ? lay.total : 0;
    if (need > 0 && (!given16(workspace) || workspace_bytes < need)) return GDR_ERR_WORKSPACE;
    const Range in[] = {{q, T * H_qk * d_k * e}, {k, T * H_qk * d_k * e}, {v, T * H * d_v * e},
                        {decay, (size_t)H * 4},
                        {initial_state == final_state ? nullptr : initial_state, state},
                        {cu_seqlens, equal ? 0 : ((size_t)num_seqs + 1) * 4}};
    const Range out[] = {{o, T * H * d_v * e}, {final_state, state}, {workspace, need}};
    if (!apart(in, out)) return GDR_ERR_INVALID_ARG;
    if (total_T == 0) return status_of(pass_state(final_state, initial_state, state, s));

    Call c;
    c.begin(cu_seqlens, decay, num_seqs, total_T, H, plan, lay, workspace, io_dtype == GDR_BF16, s);
    // in place and in segments: the last segment of a sequence may end before its
    // first one has read the incoming state, which therefore moves aside
    if (initial_state != nullptr && initial_state == final_state && plan.inner > 0) {
        float *copy = reinterpret_cast<float *>(c.ws + lay.copy);
        if (pass_state(copy, initial_state, state, s) != cudaSuccess) return GDR_ERR_CUDA;
        initial_state = copy;
    }
    const ScanArgs p = c.args(q, H_qk, k, H_qk, v, H, initial_state, false, final_state, o, 0, false);
    c.pass(p, d_k, d_v, false, true, false);
    c.join(p, d_k, d_v, false);
    c.pass(p, d_k, d_v, false, false, false);
    return status_of(c.error);
}

gdr_status_t gdr_linear_check_workspace(const void *workspace, size_t workspace_bytes, void *stream) {
    if (!given16(workspace) || workspace_bytes < kHeader) return GDR_ERR_WORKSPACE;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const uint8_t *ws = static_cast<const uint8_t *>(workspace);
    uint32_t words = 0;
    if (cudaMemcpyAsync(&words, ws, 4, cudaMemcpyDeviceToHost, s) != cudaSuccess ||
        cudaStreamSynchronize(s) != cudaSuccess)
        return GDR_ERR_CUDA;
    if ((size_t)words > (workspace_bytes - kHeader) / 4) return GDR_ERR_WORKSPACE;
    uint32_t any = 0, part[1024];
    for (size_t at = 0; at < words; at += 1024) {
        const size_t n = std::min<size_t>(1024, words - at);
        if (cudaMemcpyAsync(part, ws + kHeader + at * 4, n * 4, cudaMemcpyDeviceToHost, s) != cudaSuccess ||
            cudaStreamSynchronize(s) != cudaSuccess)
            return GDR_ERR_CUDA;
        for (size_t i = 0; i < n; ++i) any |= part[i];
    }
    return any == 0 ? GDR_OK : GDR_ERR_DEVICE_TIMEOUT;
}

gdr_status_t gdr_linear_decode(const void *q, const void *k, const void *v, const float *decay,
                               float *state, int32_t N, int32_t H_qk, int32_t H, int32_t d_k,
                               int32_t d_v, gdr_dtype_t io_dtype, void *o, void *stream) {
    if (N < 0 || H < 1 || H_qk < 1 || H % H_qk != 0) return GDR_ERR_INVALID_ARG;
    if (!head_dim(d_k) || !head_dim(d_v) || !io_type(io_dtype)) return GDR_ERR_INVALID_ARG;
    if ((int64_t)N * H > INT32_MAX) return GDR_ERR_INVALID_ARG;
    if (N == 0) return GDR_OK;
    if (!given16(q) || !given16(k) || !given16(v) || !given16(state) || !given16(o) ||
        decay == nullptr || !api::aligned(decay, 4))
        return GDR_ERR_INVALID_ARG;
    const size_t e = io_dtype == GDR_BF16 ? 2 : 4, n = (size_t)N;
    const Range in[] = {{q, n * H_qk * d_k * e}, {k, n * H_qk * d_k * e}, {v, n * H * d_v * e},
                        {decay, (size_t)H * 4}};
    const Range out[] = {{o, n * H * d_v * e}, {state, n * H * d_k * d_v * 4}};
    if (!apart(in, out)) return GDR_ERR_INVALID_ARG;
    return status_of(launch_linear_decode(q, k, v, decay, state, N, H_qk, H, d_k, d_v,
                                          io_dtype == GDR_BF16, o, static_cast<cudaStream_t>(stream)));
}

gdr_status_t gdr_linear_backward(const void *q, const void *k, const void *v, const float *decay,
                                 const float *initial_state, const int32_t *cu_seqlens,
                                 int32_t num_seqs, int32_t total_T, int32_t H_qk, int32_t H,
                                 int32_t d_k, int32_t d_v, gdr_dtype_t io_dtype, const void *d_o,
                                 const float *d_final_state, void *dq, void *dk, void *dv,
                                 float *d_initial_state, void *workspace, size_t workspace_bytes,
                                 void *stream) {
    const bool equal = cu_seqlens == nullptr;
    gdr_status_t st = check_shape(num_seqs, total_T, H_qk, H, d_k, d_v, io_dtype, equal);
    if (st != GDR_OK) return st;
    if (!maybe16(initial_state) || !maybe16(d_final_state) || !maybe16(d_initial_state) ||
        !api::aligned(cu_seqlens, 4))
        return GDR_ERR_INVALID_ARG;
    if (num_seqs == 0) return GDR_OK;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const size_t state = (size_t)num_seqs * H * d_k * d_v * 4;
    const size_t e = io_dtype == GDR_BF16 ? 2 : 4, T = (size_t)total_T;
    if (total_T > 0 && (!given16(q) || !given16(k) || !given16(v) || !given16(d_o) || !given16(dq) ||
                        !given16(dk) || !given16(dv) || decay == nullptr || !api::aligned(decay, 4)))
        return GDR_ERR_INVALID_ARG;
    const Plan plan = total_T > 0 ? make_plan(num_seqs, total_T, H, d_k, d_v, io_dtype == GDR_BF16, equal) : Plan{kScanBlock, 0, 0};
    const Layout lay = make_layout(plan, num_seqs, total_T, H_qk, H, d_k, d_v, true);
    const size_t need = total_T > 0 ? lay.total : 0;
    if (need > 0 && (!given16(workspace) || workspace_bytes < need)) return GDR_ERR_WORKSPACE;
    const size_t nq = T * H_qk * d_k * e, nv = T * H * d_v * e;
    const Range in[] = {{q, nq}, {k, nq}, {v, nv}, {decay, (size_t)H * 4}, {initial_state, state},
                        {d_o, nv}, {d_final_state, state},
                        {cu_seqlens, equal ? 0 : ((size_t)num_seqs + 1) * 4}};
    const Range out[] = {{dq, nq}, {dk, nq}, {dv, nv}, {d_initial_state, state}, {workspace, need}};
    if (!apart(in, out)) return GDR_ERR_INVALID_ARG;
    if (total_T == 0) return status_of(pass_state(d_initial_state, d_final_state, state, s));

    Call c;
    c.begin(cu_seqlens, decay, num_seqs, total_T, H, plan, lay, workspace, io_dtype == GDR_BF16, s);
    // heads that share a query/key head: each one's dq and dk in fp32, then their sums.
    // A pass follows one that it does not need, so that the segments that enter with the
    // caller's state need not wait for the other's end.
    const bool group = H != H_qk;
    float *part[2] = {reinterpret_cast<float *>(c.ws + lay.part[0]), reinterpret_cast<float *>(c.ws + lay.part[1])};
    const ScanArgs pq = c.args(d_o, H, v, H, k, H_qk, initial_state, true, nullptr, group ? part[0] : dq, 0, false);
    const ScanArgs pv = c.args(k, H_qk, q, H_qk, d_o, H, d_final_state, false, d_initial_state, dv, 1, false);
    const ScanArgs pk = c.args(v, H, d_o, H, q, H_qk, d_final_state, true, nullptr, group ? part[1] : dk, 1, true);
    c.pass(pq, d_v, d_k, false, true, false);
    c.pass(pv, d_k, d_v, true, true, false);
    c.join(pq, d_v, d_k, false);
    c.join(pv, d_k, d_v, true);
    c.pass(pq, d_v, d_k, false, false, group);
    c.pass(pv, d_k, d_v, true, false, false, true);
    c.pass(pk, d_v, d_k, true, false, group, true);
    if (c.error == cudaSuccess && group) {
        const float *const parts[2] = {part[0], part[1]};
        void *const sums[2] = {dq, dk};
        c.error = launch_group_sum(parts, cu_seqlens, num_seqs, total_T, H_qk, H / H_qk, d_k, c.bf16, sums, s);
    }
    return status_of(c.error);
}

}  // extern "C"
