// Shared by the kernels of linear attention with a decay for each head
//
//     S_t = e^g S_{t-1} + v_t k_t^T,    o_t = S_t q_t          (g <= 0, one per head)
//
// Forward pass and all three gradients are one scan with its inputs exchanged.
// For the positions p = 0 .. L-1 of a sequence, taken first to last or last to
// first (r = 1), and x = e^g:
//
//     o_p   = x^{p + 1 - r} S_in a_p + sum_{j <= p} x^{p - j} (a_p . b_j) v_j
//     S_out = x^L S_in + sum_j x^{L - 1 + r - j} v_j b_j^T
//
//     forward  a = q,   b = k,   v = v            S_in = initial state
//     dq       a = d_o, b = v,   v = k            S_in = initial state, transposed
//     dk       a = v,   b = d_o, v = q,   r = 1   S_in = d_final_state, transposed
//     dv       a = k,   b = q,   v = d_o, r = 1   S_in = d_final_state; S_out = d_initial_state
//
// (The gradient with respect to S_t is G_t = x G_{t+1} + d_o_t q_t^T; it reaches
// the last token undecayed, which is why r shifts the exponents by one.)
//
// Long sequences are cut into segments of a fixed number of tokens.  One pass
// over b and v gives every segment's own state, a pass over those states alone
// turns them into the states that enter the segments, and the output pass then
// runs all segments at once.  A slot is one segment of one sequence, and each
// sequence has at least one; the states in between are numbered without each
// sequence's last segment, so there are at most total_T / seg_tokens of them
// however many sequences there are.  dk and dv need the same states, one turned.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "launch.cuh"

namespace gdr {

constexpr int kScanBlock = 64;   // tokens: the unit of segment lengths

struct ScanArgs {
    const void *a, *b, *v;           // [total_T, HA, d_b], [total_T, HB, d_b], [total_T, HV, d_v]
    void *out;                       // [total_T, H, d_v]
    const float *decay;              // [H]
    const float *s_in;               // [N, H, d_v, d_b] ([N, H, d_b, d_v] if turned) or null
    float *s_out;                    // [N, H, d_v, d_b] or null
    float *seg;                      // [inner, H, d_v * d_b] states between segments
    uint32_t *header;                // word 0: how many status words the call has
    uint32_t *status;                // one word for each block of this pass, 0 unless a wait gave up
    uint32_t status_words;
    const int32_t *cu;
    int N, total_T, H, HA, HB, HV;
    int seg_tokens;                  // multiple of kScanBlock
    int slots, inner;                // segments, and those that are not their sequence's last
    int turned, seg_turned;          // s_in, the states between segments are stored [d_b, d_v]
    int late;                        // output pass behind another one: needs none of its results, but the states from before it
};

struct Segment {
    int n;          // sequence (-1: this slot is behind the last one)
    int index;      // place in the sequence's chain of segments, in scan order
    int count;      // segments of the sequence
    int state;      // number of the state behind this segment
    int t0, len;    // its tokens
    int seq_len;
};

__host__ __device__ inline int segments_of(int len, int seg_tokens) {
    return len <= seg_tokens ? 1 : 1 + (len - 1) / seg_tokens;
}

// The segment of a slot, or with `inner` of a state between segments.  Called
// by all `threads` (a multiple of 32, at most 1024) of a block; scratch: 34
// ints of shared memory.  With cu_seqlens every thread counts the segments of a
// run of sequences, a scan over the block's counts finds the run that holds the
// slot, and its thread walks it.
__device__ inline Segment find_segment(const ScanArgs &p, int slot, bool inner, bool reverse,
                                       int *scratch, int threads) {
    Segment s;
    s.n = -1; s.index = 0; s.count = 1; s.state = 0; s.t0 = 0; s.len = 0; s.seq_len = 0;
    if (p.cu == nullptr) {
        const int per = segments_of(p.total_T / p.N, p.seg_tokens) - (inner ? 1 : 0);
        if (per == 0 || slot >= p.N * per) return s;
        s.n = slot / per;
        s.index = slot % per;
    } else {
        const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
        const int run = (p.N + threads - 1) / threads;
        const int64_t first = (int64_t)tid * run;
        auto count = [&](int64_t n) {
            int t0, len;
            sequence_range(p.cu, (int)n, p.N, p.total_T, t0, len);
            return segments_of(len, p.seg_tokens) - (inner ? 1 : 0);
        };
        int mine = 0;
        for (int64_t n = first; n < first + run && n < p.N; ++n) mine += count(n);
        int upto = mine;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int x = __shfl_up_sync(0xffffffffu, upto, off);
            if (lane >= off) upto += x;
        }
        if (tid == 0) scratch[32] = -1;
        if (lane == 31) scratch[warp] = upto;
        __syncthreads();
        int at = upto - mine;
        for (int w = 0; w < warp; ++w) at += scratch[w];
        if (slot >= at && slot < at + mine) {
            for (int64_t n = first; n < first + run && n < p.N; ++n) {
                const int c = count(n);
                if (slot < at + c) {
                    scratch[32] = (int)n;
                    scratch[33] = slot - at;
                    break;
                }
                at += c;
            }
        }
        __syncthreads();
        s.n = scratch[32];
        s.index = scratch[33];
        if (s.n < 0) return s;
    }
    int t0, len;
    sequence_range(p.cu, s.n, p.N, p.total_T, t0, len);
    s.seq_len = len;
    s.count = segments_of(len, p.seg_tokens);
    s.state = inner ? slot : slot - s.n;
    // a cu_seqlens that is no partition may count more segments than there is room for,
    // or than an int holds
    if ((unsigned)s.index >= (unsigned)s.count || s.state > p.inner || (!inner && s.state < s.index)) {
        s.n = -1;
        return s;
    }
    const int place = reverse ? s.count - 1 - s.index : s.index;
    s.t0 = t0 + place * p.seg_tokens;
    s.len = min(p.seg_tokens, len - place * p.seg_tokens);
    return s;
}

// Launchers.  `states`: the pass that writes the segments' own states (all but
// each sequence's last segment in scan order); otherwise the output pass.
// (tensor cores: bf16, d_b = d_v = 128, with the tensors' tile maps)
bool scan_tile_map(CUtensorMap *map, const void *base, int total_T, int H);
cudaError_t launch_scan_tc(const CUtensorMap &a, const CUtensorMap &b, const CUtensorMap &v, const ScanArgs &p,
                           bool reverse, bool states, bool out_f32, bool after, cudaStream_t stream);
cudaError_t launch_scan_simt(const ScanArgs &p, int d_b, int d_v, bool reverse, bool states,
                             bool bf16, bool out_f32, bool after, cudaStream_t stream);
// Segments' own states -> states behind each segment, in place (after the states' pass).
cudaError_t launch_scan_join(const ScanArgs &p, int elements, bool reverse, cudaStream_t stream);
// [T, H, d] fp32 partial gradients (dq's and dk's) summed over each group of H / H_qk heads (after a pass).
cudaError_t launch_group_sum(const float *const (&part)[2], const int32_t *cu, int N, int64_t T, int H_qk,
                             int group, int d, bool bf16, void *const (&out)[2], cudaStream_t stream);
cudaError_t launch_linear_decode(const void *q, const void *k, const void *v, const float *decay,
                                 float *state, int N, int Hqk, int H, int DK, int DV, bool bf16,
                                 void *o, cudaStream_t stream);

}  // namespace gdr
