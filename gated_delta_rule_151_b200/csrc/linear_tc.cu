// Linear attention with a decay for each head on the tensor cores: bf16
// inputs, d = 128, blocks of 64 tokens (the scan of linear_common.cuh).
//
// One CTA runs one segment of one (sequence, head) block after block.  With
// x = e^g, i and j the rows of a block of n tokens and S the state entering it,
//
//     P   = (A B^T) .* M,            M_ij = x^|i-j| on the causal side, else 0
//     O^T = (S A^T) diag(x^lead) + V^T P^T
//     S  <- x^n S + (diag(w) V)^T B
//     forward: lead = i + 1,     w_j = x^{n-1-j};   reverse: lead = n - 1 - i,  w_j = x^{j+1}
//
// Every exponent is >= 0 times g <= 0: nothing overflows however fast a head
// decays.  All four products are tcgen05.mma with M = 128: O^T and S carry the
// value channels on the TMEM lanes, so neither wastes half of the unit on 64
// tokens, and S can be its own A operand from TMEM.
//
// Rounding.  A, B, V are exact bf16 operands.  P and the copy of S that meets A enter
// their products as two bf16 terms each (16 significant bits), so that a result has the
// one rounding of its own type: with one term each it was 1.4 output roundings off, and
// more where a few tokens hang on one score.  (The second terms take 15 %: 1 x 8192
// tokens, 16 heads 52 -> 60 us of GPU time, the gradient 177 -> 217; half of it the
// packing of S, a tenth the products.)  The state itself is never rounded: it stays
// in fp32 registers, and diag(w) V enters its product as three bf16 terms (24 significant
// bits), so S is as exact as fp32 sums make it over any number of blocks.
//
// 16 warps: 0-1 turn the scores into P (one row a thread); 2 issues the products
// of a block's tokens alone (scores, (diag(w) V)^T B), 3 starts the TMA loads into
// a ring of tiles (each takes its issuer 300 cycles) and issues the products that
// wait for S and P; 4-7 write O; 8-15 hold S, 64 columns of one row a thread, and
// split the weighted V.  The pass that only wants the state uses 2, 3 and 8-15.
#include <cstddef>
#include <type_traits>

#include "chunk_common.cuh"
#include "linear_common.cuh"

namespace gdr {
namespace {

constexpr int kThreads = 512;
constexpr int kSThreads = 256, kOThreads = 128, kPThreads = 64;

constexpr uint32_t TILE = 16384;            // 64 tokens x 128 channels bf16, two 64-channel halves

template <bool OUT>
struct Shape {
    static constexpr int NS = OUT ? 3 : 4;                   // tiles in the ring
    static constexpr int NB = OUT ? 1 : 2;                   // buffers of the split V and of its product
    static constexpr uint32_t STAGE = (OUT ? 3 : 2) * TILE;
    static constexpr uint32_t B_OFF = OUT ? TILE : 0;        // A, B, V in a stage
    static constexpr uint32_t V_OFF = B_OFF + TILE;
    static constexpr uint32_t P_OFF = NS * STAGE;            // two buffers of 64 x 64 bf16, high and low part
    static constexpr uint32_t O_OFF = P_OFF + (OUT ? 2 * 16384 : 0);  // a tile of O on its way out
    static constexpr uint32_t W_OFF = O_OFF + (OUT ? TILE : 0);      // the low part of diag(w) V, laid out as V
    static constexpr uint32_t MISC = W_OFF + (OUT ? TILE : 0);
    // TMEM columns.  Beside the two copies of S there is no room for the low part of the split V.
    static constexpr uint32_t W_COLS = OUT ? 64 : 96;
    static constexpr uint32_t T_KV = 0;                      // NB of 128: (diag(w) V)^T B
    static constexpr uint32_t T_W = NB * 128;                // NB of W_COLS: (diag(w) V)^T, its high, middle (low) part
};

struct Misc {
    uint64_t full[4];                   // a stage's tiles have arrived
    uint64_t w_full[4];                 // half of the split V is written
    uint64_t kv_full[4], kv_free[2];    // its product is done (and its buffer free), and read
    uint64_t sc_full[2], p_full[2];     // scores are done; P is written
    uint64_t s_full, s_free;            // S in bf16 is written; S A^T is done
    uint64_t done[3], o_free[2];        // V^T P^T is done too; they are read
    uint64_t end[2];
    uint32_t tmem;
    int abort;
    int scratch[34];
    float pw[kScanBlock + 1];                // x^k
    alignas(16) float lead[kScanBlock];      // of S A^T in a full block
    alignas(16) float weight[kScanBlock];    // of V in a full block
    // Of four blocks in turn: the last one whose V had infinities or NaN, in any of its
    // channels and in 16 of them each, and its first (reverse: last) such token per channel.
    int bad[4], bad_part[4][8], bad_token[4][128];
};

static_assert(Shape<true>::NS == 3 && Shape<false>::NS == 4, "copies of done and kv_full");
template <bool OUT>
constexpr int smem_bytes() { return (int)(Shape<OUT>::MISC + sizeof(Misc)); }
static_assert(smem_bytes<true>() <= 232448 && smem_bytes<false>() <= 232448, "shared memory");

constexpr uint32_t T_SL = 192;      // what S in bf16 leaves, in bf16
constexpr uint32_t T_X = 256;       // two buffers of 64: a block's scores, then its V^T P^T
constexpr uint32_t T_OI = 384;      // S A^T
constexpr uint32_t T_SB = 448;      // S in bf16
constexpr uint32_t T_COLS = 512;

constexpr uint32_t ID_N64 = make_idesc(1, 128, 64);
constexpr uint32_t ID_PV = ID_N64 | kIdescAMN;
constexpr uint32_t ID_KV = make_idesc(1, 128, 128) | kIdescBMN;
static_assert(Shape<true>::T_W + Shape<true>::W_COLS <= T_SL && T_SL + 64 <= T_X, "TMEM columns");

enum : uint32_t { E_ALIGN = 1, E_TMA = 2, E_MMA = 4, E_HANDOFF = 8 };

// Parity cannot tell a barrier's phase from the one two later, so a barrier whose
// owner can run ahead of a waiter has several copies, one block after another:
// enough that a copy's next phase needs that waiter to have gone on.  Commits are
// few (each holds the issuer up by 200 cycles): one barrier can have many waiters.

__device__ __forceinline__ bool try_wait(uint32_t bar, uint32_t phase) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(phase)
        : "memory");
    return ok != 0;
}

__device__ __forceinline__ void arrive(uint32_t bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}

// The rest of a wait whose first look found its phase unfinished: polls, a
// bounded number of times, until the phase completes or some role has given up
// (at `abort`).  Called by whole warps; kept out of line, as every wait has one.
__device__ __noinline__ bool wait_on(uint32_t bar, uint32_t phase, uint32_t abort) {
    for (uint32_t it = 0; it < (1u << 18); ++it) {
        const bool ok = try_wait(bar, phase);
        if (__all_sync(0xffffffffu, ok)) return true;
        uint32_t stop;
        asm volatile("ld.volatile.shared.u32 %0, [%1];" : "=r"(stop) : "r"(abort) : "memory");
        if (__any_sync(0xffffffffu, stop != 0)) return false;
    }
    return false;
}

// Whether any thread of a group of whole warps says stop; all of them come here.
__device__ __forceinline__ bool group_stop(int id, int threads, bool stop) {
    uint32_t any;
    asm volatile(
        "{\n\t.reg .pred pc, pr;\n\t"
        "setp.ne.u32 pc, %1, 0;\n\t"
        "barrier.red.or.pred pr, %2, %3, pc;\n\t"
        "selp.u32 %0, 1, 0, pr;\n\t}"
        : "=r"(any)
        : "r"((uint32_t)stop), "r"(id), "r"(threads)
        : "memory");
    return any != 0;
}

__device__ __forceinline__ void load_tile(void *dst, const CUtensorMap *map, uint64_t *bar, int t0, int head) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(0), "r"(t0), "r"(0), "r"(head)
        : "memory");
}

// 32 TMEM columns of 16 lanes: registers 4 k to 4 k + 3 hold columns 8 k + 2 (lane % 4)
// and the next one of TMEM lane lane / 4, then of lane / 4 + 8.
__device__ __forceinline__ void tmem_ld_frag(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x4.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]),
          "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
}

// The same fragment of 16 lanes by 16 columns of 32 bits to TMEM: registers 2 k and 2 k + 1
// go to column 4 k + lane % 4 of TMEM lanes lane / 4 and lane / 4 + 8.
__device__ __forceinline__ void tmem_st_frag(uint32_t taddr, const uint32_t (&r)[8]) {
    asm volatile("tcgen05.st.sync.aligned.16x128b.x4.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr),
                 "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
}

__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\tselp.u32 %0, 1, 0, q;\n\t}" : "=r"(p));
    return p != 0;
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    __nv_bfloat162 x = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<uint32_t *>(&x);
}
__device__ __forceinline__ float bf16_lo(uint32_t x) { return __uint_as_float(x << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t x) { return __uint_as_float(x & 0xffff0000u); }
// What a pair's bf16 values leave of it, in bf16.
__device__ __forceinline__ uint32_t rest_bf16(float2 f, uint32_t x) {
    const float2 r = __ffma2_rn(make_float2(bf16_lo(x), bf16_hi(x)), make_float2(-1.f, -1.f), f);
    return pack_bf16(r.x, r.y);
}

// Infinities and NaN of V, which the zeros of P would carry to tokens on the other side of
// the mask: they leave the tile, and the tokens that they do reach get NaN where O is
// written (the split V has them, and so has S).  A warp looks through its 16 channels of the
// block's tokens.  Both are rare, and kept out of line.
template <bool REV>
__device__ __noinline__ void take_out(uint32_t v, int n, int b, Misc *m) {
    const int lane = threadIdx.x & 31, part = (threadIdx.x >> 5) & 7;
    const int c = (part & 3) * 32 + (part >> 2) * 16 + (lane & 15);
    int found = REV ? -1 : C;
    for (int j = lane >> 4; j < n; j += 2) {
        const uint32_t at = v + (c >> 6) * 8192 + sw128_offset(j, (c >> 3) & 7) + (c & 7) * 2;
        uint16_t x;
        asm volatile("ld.shared.u16 %0, [%1];" : "=h"(x) : "r"(at) : "memory");
        if ((x & 0x7f80) != 0x7f80) continue;
        asm volatile("st.shared.u16 [%0], %1;" ::"r"(at), "h"((uint16_t)0) : "memory");
        found = REV ? j : min(found, j);
    }
    const int other = __shfl_xor_sync(0xffffffffu, found, 16);
    m->bad_token[b & 3][c] = REV ? max(found, other) : min(found, other);
    m->bad_part[b & 3][part] = b;
    m->bad[b & 3] = b;
    fence_proxy_async();
}

// NaN to the tokens of channel c that it reaches: `put` of each.
template <bool REV, typename Put>
__device__ __noinline__ void put_back(int c, int n, int b, const Misc *m, Put put) {
    if (m->bad_part[b & 3][(c >> 5) + ((c >> 4) & 1) * 4] != b) return;
    const int token = m->bad_token[b & 3][c];
    for (int i = REV ? 0 : token; i < (REV ? token + 1 : n); ++i) put(i);
}

template <bool OUT, bool REV, typename OutT>
__global__ void __launch_bounds__(kThreads, 1)
scan_tc_kernel(const __grid_constant__ CUtensorMap ma, const __grid_constant__ CUtensorMap mb,
               const __grid_constant__ CUtensorMap mv, const ScanArgs p) {
    using Sh = Shape<OUT>;
    extern __shared__ __align__(1024) uint8_t sm[];
    const uint32_t sbase = smem_u32(sm);
    Misc *m = reinterpret_cast<Misc *>(sm + Sh::MISC);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int slot = blockIdx.x / p.H, h = blockIdx.x % p.H;
    uint32_t *status = p.status + blockIdx.x;
    if (tid == 0) *status = 0;
    if (OUT && blockIdx.x == 0 && tid == 0) *p.header = p.status_words;

    const Segment seg = find_segment(p, slot, !OUT, REV, m->scratch, kThreads);
    if (seg.n < 0) return;
    const bool last = seg.index == seg.count - 1;
    const int blocks = (seg.len + C - 1) / C;
    const size_t state_at = ((size_t)seg.n * p.H + h) * (D * D);
    float *seg_out = OUT ? nullptr : p.seg + ((size_t)seg.state * p.H + h) * (D * D);
    // the state behind this segment: for the caller, for the join, or for nobody
    const bool want_state = OUT ? (last && p.s_out != nullptr) : true;
    if ((sbase & 1023u) != 0) {
        if (tid == 0) atomicOr(status, E_ALIGN);
        return;
    }

    const uint32_t mbase = sbase + Sh::MISC;
#define BAR(name, i) (mbase + (uint32_t)offsetof(Misc, name) + 8 * (i))
    // block b in scan order: its first token and its tokens
    auto block_t0 = [&](int b) { return seg.t0 + (REV ? blocks - 1 - b : b) * C; };
    auto block_n = [&](int b) { return min(C, seg.len - (REV ? blocks - 1 - b : b) * C); };
    auto load = [&](int b) {
        if (elect_one()) {
            const int ha = h / (p.H / p.HA), hb = h / (p.H / p.HB), hv = h / (p.H / p.HV);
            uint64_t *bar = &m->full[b % Sh::NS];
            uint8_t *st = sm + (b % Sh::NS) * Sh::STAGE;
            const int t0 = block_t0(b);
            mbar_arrive_expect_tx(bar, Sh::STAGE);
            if (OUT) load_tile(st, &ma, bar, t0, ha);
            load_tile(st + Sh::B_OFF, &mb, bar, t0, hb);
            load_tile(st + Sh::V_OFF, &mv, bar, t0, hv);
        }
        __syncwarp();
    };
    // never leave a copy in flight into this CTA's shared memory
    auto drain = [&](int issued) {
        for (int b = issued > Sh::NS ? issued - Sh::NS : 0; b < issued; ++b)
            (void)mbar_wait_sleep(&m->full[b % Sh::NS], (b / Sh::NS) & 1);
    };

    // the loader's first block is on its way before anything else is ready
    int issued = 0;
    if (warp == 3) {
        if (elect_one()) {
            for (int s = 0; s < 4; ++s) {
                mbar_init(&m->full[s], 1);
                mbar_init(&m->kv_full[s], 1);
            }
            for (int s = 0; s < 3; ++s) mbar_init(&m->done[s], 1);
            for (int b = 0; b < 2; ++b) {
                mbar_init(&m->w_full[b], kSThreads);
                mbar_init(&m->w_full[2 + b], kSThreads);
                mbar_init(&m->kv_free[b], kSThreads);
                mbar_init(&m->sc_full[b], 1);
                mbar_init(&m->p_full[b], kPThreads);
                mbar_init(&m->o_free[b], kOThreads);
            }
            mbar_init(&m->s_full, kSThreads);
            mbar_init(&m->s_free, 1);
            mbar_init(&m->end[0], 1);
            mbar_init(&m->end[1], 1);
            m->abort = 0;
            fence_barrier_init();
            fence_proxy_async();
        }
        __syncwarp();
        if (blocks > 0) load(issued++);
    }
    launch_dependents();
    // A pass whose inputs are all the caller's runs beside the one before; the states
    // between segments are not.
    const bool beside = !OUT || (p.late && seg.index == 0);
    auto wait_here = [&]() {
        if (!beside) wait_for_previous();
    };
    const float g = clamp_log_gate(p.decay[h]);
    if (tid <= C) m->pw[tid] = expf(g * (float)tid);
    if (tid < C) {
        m->lead[tid] = expf(g * (float)(REV ? C - 1 - tid : tid + 1));
        m->weight[tid] = expf(g * (float)(REV ? tid + 1 : C - 1 - tid));
    }
    if (OUT && tid < 32) {
        m->bad[tid & 3] = -1;
        m->bad_part[tid >> 3][tid & 7] = -1;
    }
    if (warp == 0) {
        tmem_alloc(&m->tmem, T_COLS);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = m->tmem;
    // Bounded wait of a whole warp; false, and everyone told, when it or another role
    // gave up.  A phase that is complete already costs one look.
    auto warp_wait = [&](uint32_t bar, uint32_t phase, uint32_t code) {
        if (__all_sync(0xffffffffu, try_wait(bar, phase & 1))) return true;
        if (wait_on(bar, phase & 1, BAR(abort, 0))) return true;
        if (lane == 0) {
            *reinterpret_cast<volatile int *>(&m->abort) = 1;
            atomicOr(status, code);
        }
        return false;
    };
    const uint64_t kmajor = sw128_kmajor_desc(sbase), mnmajor = sw128_mnmajor_desc(sbase, 8192, 1024);
    if (warp >= 8) {
        // ------------------------------------------------ S: row r, 64 columns ----
        const int t = tid - kSThreads;
        const int r = (warp & 3) * 32 + lane, half = (warp - 8) >> 2;
        const uint32_t lanes = (uint32_t)(warp & 3) << 21;
        float2 S[32];
        wait_here();
        // the state that enters: between segments, the caller's, or zero
        const float *from = OUT && seg.index > 0 ? p.seg + ((size_t)(seg.state - 1) * p.H + h) * (D * D)
                            : seg.index > 0 || p.s_in == nullptr ? nullptr : p.s_in + state_at;
        if (from == nullptr) {
#pragma unroll
            for (int i = 0; i < 32; ++i) S[i] = make_float2(0.f, 0.f);
        } else if (seg.index > 0 ? p.seg_turned : p.turned) {
            const float *src = from + (size_t)half * 64 * D + r;
#pragma unroll
            for (int i = 0; i < 32; ++i) S[i] = make_float2(src[2 * i * D], src[(2 * i + 1) * D]);
        } else {
            const float4 *src = reinterpret_cast<const float4 *>(from + r * D + half * 64);
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const float4 x = src[i];
                S[2 * i] = make_float2(x.x, x.y);
                S[2 * i + 1] = make_float2(x.z, x.w);
            }
        }
        bool ok = true;
        // where a lane's row of eight channels lies, in V's tile: 16 tokens from 32 h2 + 16 k
        auto v_at = [&](int ch, int h2, int k) {
            const int j = h2 * 32 + k * 16 + (lane & 7) + ((lane >> 4) << 3);
            return (uint32_t)((ch >> 6) * 8192) + sw128_offset(j, (ch >> 3) & 7);
        };
        // (diag(w) V)^T of block b in three bf16 parts to TMEM, the product's other operand:
        // 32 tokens, then the other 32, whose split the first ones' product hides.  A warp
        // takes 16 channels (half of its lanes) by the 32 tokens.  ldmatrix hands a thread
        // tokens 8 m + 2 (lane % 4) and the next one of channels lane / 4 + {0, 8}, the
        // fragment that tcgen05.st writes; through shared memory the parts cost 96 KB of its
        // 336 KB of traffic a block, which was the bound.  The output pass leaves the low part
        // there, as its TMEM holds the second copy of S.
        auto split_v = [&](int b) {
            const int s = b % Sh::NS, n = block_n(b);
            if (!(ok = warp_wait(BAR(full, s), b / Sh::NS, E_TMA))) return;
            const uint32_t stage = sbase + s * Sh::STAGE;
            // rows behind the segment's last token hold another sequence's tokens (or
            // anything): they leave B and V, since 0 * inf is not 0
            if (n < C) {
                for (int e = t; e < 2 * (C - n) * 8; e += kSThreads) {
                    const uint32_t at = (e & 1) * 8192 + (n + (e >> 4)) * 128 + ((e >> 1) & 7) * 16;
                    st_shared_v4(stage + Sh::B_OFF + at, 0, 0, 0, 0);
                    st_shared_v4(stage + Sh::V_OFF + at, 0, 0, 0, 0);
                }
                fence_proxy_async();
            }
            // (the product that last read this buffer was waited for by its update of S)
            tc_fence_after();
            __nv_bfloat162 any = __float2bfloat162_rn(0.f);
            // (rolled, as the instructions of all roles together are what the cache holds:
            // unrolled, packed prompts took 170 us in place of 158)
#pragma unroll 1
            for (int h2 = 0; h2 < 2; ++h2) {
                const bool kv = b + 1 < blocks || want_state;
                if (OUT || kv) {
                    const int ch = (warp & 3) * 32 + half * 16 + (lane & 8), j0 = h2 * 32 + 2 * (lane & 3);
                    uint32_t hi[8], mid[8], lo[8];
#pragma unroll
                    for (int k = 0; k < 2; ++k) {      // 16 tokens
                        asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                                     : "=r"(hi[4 * k]), "=r"(hi[4 * k + 1]), "=r"(hi[4 * k + 2]), "=r"(hi[4 * k + 3])
                                     : "r"(stage + Sh::V_OFF + v_at(ch, h2, k))
                                     : "memory");
                    }
                    if (n < C) {
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            const int j = j0 + 8 * (e >> 1);
                            hi[e] = j + 1 < n ? hi[e] : j < n ? hi[e] & 0xffffu : 0u;
                        }
                    }
                    if (OUT) {
#pragma unroll
                        for (int e = 0; e < 8; ++e)      // NaN if one of them is not finite, else 0
                            any = __hfma2(*reinterpret_cast<const __nv_bfloat162 *>(&hi[e]), __float2bfloat162_rn(0.f), any);
                    }
                    if (kv) {
                        float2 weight[4];
#pragma unroll
                        for (int k = 0; k < 4; ++k) weight[k] = *reinterpret_cast<const float2 *>(m->weight + j0 + 8 * k);
                        if (!REV && n < C) {
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                const int j = j0 + 8 * k;
                                weight[k] = make_float2(m->pw[max(n - 1 - j, 0)], m->pw[max(n - 2 - j, 0)]);
                            }
                        }
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            const float2 minus = make_float2(-1.f, -1.f);
                            float2 f = __fmul2_rn(make_float2(bf16_lo(hi[e]), bf16_hi(hi[e])), weight[e >> 1]);
                            hi[e] = pack_bf16(f.x, f.y);
                            f = __ffma2_rn(make_float2(bf16_lo(hi[e]), bf16_hi(hi[e])), minus, f);
                            mid[e] = pack_bf16(f.x, f.y);
                            f = __ffma2_rn(make_float2(bf16_lo(mid[e]), bf16_hi(mid[e])), minus, f);
                            lo[e] = pack_bf16(f.x, f.y);
                        }
                        const uint32_t to = tmem + lanes + ((uint32_t)half << 20) + Sh::T_W + (b % Sh::NB) * Sh::W_COLS + h2 * 16;
                        tmem_st_frag(to, hi);
                        tmem_st_frag(to + 32, mid);
                        if (OUT) {
#pragma unroll
                            for (int k = 0; k < 2; ++k)
                                asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::
                                                 "r"(sbase + Sh::W_OFF + v_at(ch, h2, k)),
                                             "r"(lo[4 * k]), "r"(lo[4 * k + 1]), "r"(lo[4 * k + 2]), "r"(lo[4 * k + 3])
                                             : "memory");
                            if (h2 == 1) fence_proxy_async();
                        } else {
                            tmem_st_frag(to + 64, lo);
                        }
                        tmem_wait_st();
                        tc_fence_before();
                    }
                }
                arrive(BAR(w_full, (b % Sh::NB) * 2 + h2));
            }
            if (OUT && __any_sync(0xffffffffu, (*reinterpret_cast<const uint32_t *>(&any) & 0x7fff7fffu) != 0))
                take_out<REV>(stage + Sh::V_OFF, n, b, m);
        };
        if (blocks > 0) split_v(0);
        for (int b = 0; b < blocks && ok; ++b) {
            if (OUT) {
                if (b > 0 && !(ok = warp_wait(BAR(s_free, 0), b - 1, E_MMA))) break;
                tc_fence_after();
                uint32_t x[32];
#pragma unroll
                for (int i = 0; i < 32; ++i) x[i] = pack_bf16(S[i].x, S[i].y);
                tmem_st32(tmem + lanes + T_SB + half * 32, x);
#pragma unroll
                for (int i = 0; i < 32; ++i) x[i] = rest_bf16(S[i], x[i]);
                tmem_st32(tmem + lanes + T_SL + half * 32, x);
                tmem_wait_st();
                tc_fence_before();
                arrive(BAR(s_full, 0));
            }
            if (!OUT && b + 1 < blocks) {       // two buffers: the next split goes ahead of this update
                split_v(b + 1);
                if (!ok) break;
            }
            if (b + 1 == blocks && !want_state) break;
            if (!(ok = warp_wait(BAR(kv_full, b & 3), b >> 2, E_MMA))) break;
            tc_fence_after();
            const float gn = REV || b + 1 == blocks ? m->pw[block_n(b)] : m->pw[C];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                uint32_t x[16];
                tmem_ld16(tmem + lanes + Sh::T_KV + (b % Sh::NB) * D + half * 64 + q * 16, x);
                tmem_wait_ld();
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    S[q * 8 + i] = __ffma2_rn(make_float2(gn, gn), S[q * 8 + i],
                                              make_float2(__uint_as_float(x[2 * i]), __uint_as_float(x[2 * i + 1])));
            }
            tc_fence_before();
            arrive(BAR(kv_free, b % Sh::NB));
            if (OUT && b + 1 < blocks) split_v(b + 1);
        }
        // an earlier pass of this call may still read the states, or run beside this one
        if (beside) wait_for_previous();
        if (want_state) {
            float4 *dst = reinterpret_cast<float4 *>((OUT ? p.s_out + state_at : seg_out) + r * D + half * 64);
#pragma unroll
            for (int i = 0; i < 16; ++i)
                dst[i] = make_float4(S[2 * i].x, S[2 * i].y, S[2 * i + 1].x, S[2 * i + 1].y);
        }
    } else if (warp >= 4) {
        // ------------------------------------------ O: 32 channels a warp, all tokens ----
        // TMEM comes in as fragments: a thread has the tokens 8 k + 2 (lane % 4) and the next
        // one of the channels lane / 4 + {0, 8} of each 16, which stmatrix turns into rows of
        // the tile [token][channel] (16-byte pieces swapped by token % 8 against conflicts).
        const int t = tid - 128;
        const uint32_t lanes = (uint32_t)(warp & 3) << 21;
        const size_t row = (size_t)p.H * D;
        float2 lead[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) lead[k] = *reinterpret_cast<const float2 *>(m->lead + 8 * k + 2 * (lane & 3));
        wait_here();
        for (int b = 0; OUT && b < blocks; ++b) {
            const bool ok = warp_wait(BAR(done, b % 3), b / 3, E_MMA);
            if (group_stop(1, kOThreads, !ok)) break;   // (and the last tile has left)
            tc_fence_after();
            const int n = block_n(b);
            OutT *dst = static_cast<OutT *>(p.out) + ((size_t)block_t0(b) * p.H + h) * D;
            if (REV && (n < C || b == 1)) {             // lead counts from the block's last token
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const int i = 8 * k + 2 * (lane & 3);
                    lead[k] = make_float2(m->pw[max(n - 1 - i, 0)], m->pw[max(n - 2 - i, 0)]);
                }
            }
#pragma unroll
            for (int c = 0; c < 2; ++c) {               // channels 32 (warp % 4) + 16 c ..
#pragma unroll
                for (int half = 0; half < 2; ++half) {  // tokens 32 half ..
                    uint32_t xi[16], xa[16];
                    const uint32_t from = tmem + lanes + ((uint32_t)c << 20) + half * 32;
                    tmem_ld_frag(from + T_OI, xi);
                    tmem_ld_frag(from + T_X + (b & 1) * 64, xa);
                    tmem_wait_ld();
                    if (c == 1 && half == 1) {
                        tc_fence_before();
                        arrive(BAR(o_free, b & 1));
                    }
                    const int ch = 32 * (warp & 3) + 16 * c;
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const float2 w = lead[half * 4 + k];
                        const float2 top = __ffma2_rn(w, make_float2(__uint_as_float(xi[4 * k]), __uint_as_float(xi[4 * k + 1])),
                                                      make_float2(__uint_as_float(xa[4 * k]), __uint_as_float(xa[4 * k + 1])));
                        const float2 low = __ffma2_rn(w, make_float2(__uint_as_float(xi[4 * k + 2]), __uint_as_float(xi[4 * k + 3])),
                                                      make_float2(__uint_as_float(xa[4 * k + 2]), __uint_as_float(xa[4 * k + 3])));
                        const int i = half * 32 + 8 * k;
                        if constexpr (sizeof(OutT) == 2) {
                            // matrices: channels ch + {0, 8}; lane l gives the place of token i + l % 8
                            const uint32_t at = sbase + Sh::O_OFF + (i + (lane & 7)) * 256 +
                                                ((((ch >> 3) + ((lane >> 3) & 1)) ^ (lane & 7)) << 4);
                            asm volatile("stmatrix.sync.aligned.m8n8.x2.trans.shared.b16 [%0], {%1, %2};" ::"r"(at),
                                         "r"(pack_bf16(top.x, top.y)), "r"(pack_bf16(low.x, low.y))
                                         : "memory");
                        } else {
                            const int i0 = i + 2 * (lane & 3), c0 = ch + (lane >> 2);
                            if (i0 < n) {
                                store_io(dst + i0 * row + c0, top.x);
                                store_io(dst + i0 * row + c0 + 8, low.x);
                            }
                            if (i0 + 1 < n) {
                                store_io(dst + (i0 + 1) * row + c0, top.y);
                                store_io(dst + (i0 + 1) * row + c0 + 8, low.y);
                            }
                        }
                    }
                }
            }
            const bool bad = m->bad[b & 3] == b;
            if constexpr (sizeof(OutT) == 2) {
                if (group_stop(1, kOThreads, false)) break;
                if (bad) {
                    put_back<REV>(t, n, b, m, [=](int i) {
                        const uint32_t at = sbase + Sh::O_OFF + i * 256 + (((t >> 3) ^ (i & 7)) << 4) + (t & 7) * 2;
                        asm volatile("st.shared.u16 [%0], %1;" ::"r"(at), "h"((uint16_t)0x7fff) : "memory");
                    });
                    if (group_stop(1, kOThreads, false)) break;
                }
#pragma unroll
                for (int u = 0; u < 8; ++u) {
                    const int e = u * kOThreads + t, i = e >> 4, piece = e & 15;
                    const uint4 x = *reinterpret_cast<const uint4 *>(sm + Sh::O_OFF + i * 256 + ((piece ^ (i & 7)) << 4));
                    if (i < n) *reinterpret_cast<uint4 *>(dst + i * row + piece * 8) = x;
                }
            } else if (bad) {
                if (group_stop(1, kOThreads, false)) break;     // (the tile is written)
                put_back<REV>(t, n, b, m, [=](int i) { store_io(dst + i * row + t, __uint_as_float(0x7fffffffu)); });
            }
        }
    } else if (warp == 2) {
        // ---------------------------------- issuer: scores and the state's update ----
        // An issuing warp stays together and one elected lane issues, so that
        // descriptors are uniform values: a base, plus a constant for each step.
        bool ok = true;
        auto scores = [&](int b) {
            const int s = b % Sh::NS;
            if (!(ok = warp_wait(BAR(full, s), b / Sh::NS, E_TMA))) return;
            if (block_n(b) < C && !(ok = warp_wait(BAR(w_full, (b % Sh::NB) * 2), b / Sh::NB, E_HANDOFF))) return;
            // the buffer last held block b - 2's V^T P^T
            if (b >= 2 && !(ok = warp_wait(BAR(o_free, b & 1), (b - 2) >> 1, E_HANDOFF))) return;
            tc_fence_after();
            // rows 64 to 127 of A are what follows the tile: their scores are not read
            const uint64_t at = kmajor + ((s * Sh::STAGE) >> 4);
            if (elect_one()) {
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const uint32_t step = ((k >> 2) * 8192 + (k & 3) * 32) >> 4;
                    mma_f16_ss(tmem + T_X + (b & 1) * 64, at + step, at + (Sh::B_OFF >> 4) + step, ID_N64, k != 0);
                }
                mma_commit(&m->sc_full[b & 1]);
            }
            __syncwarp();
        };
        // (here and below: the polls that follow do not count that time; those of a first block
        // that is not full wait for the split of V, and with it for the states)
        if (block_n(0) < C) wait_here();
        if (OUT && blocks > 0) scores(0);
        wait_here();
        for (int b = 0; b < blocks && ok; ++b) {
            const int w = b % Sh::NB;
            const bool kv = b + 1 < blocks || want_state;
            if (kv && b >= Sh::NB && !(ok = warp_wait(BAR(kv_free, w), b / Sh::NB - 1, E_HANDOFF))) break;
            const uint64_t bd = mnmajor + (((b % Sh::NS) * Sh::STAGE + Sh::B_OFF) >> 4);
            const uint64_t lo = mnmajor + (Sh::W_OFF >> 4);
            const uint32_t d = tmem + Sh::T_KV + w * D, a = tmem + Sh::T_W + w * Sh::W_COLS;
#pragma unroll
            for (int h2 = 0; h2 < 2; ++h2) {
                if (ok) ok = warp_wait(BAR(w_full, w * 2 + h2), b / Sh::NB, E_HANDOFF);
                tc_fence_after();
                if (ok && kv && elect_one()) {
#pragma unroll
                    for (int part = OUT ? 1 : 2; part >= 0; --part)     // the small terms first
#pragma unroll
                        for (int k = 2 * h2; k < 2 * h2 + 2; ++k)
                            mma_f16_ts(d, a + part * 32 + k * 8, bd + ((k * 2048) >> 4), ID_KV, part != (OUT ? 1 : 2) || k != 0);
                    if (OUT && h2 == 1) {     // (the low part is complete with the second half)
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            mma_f16_ss(d, lo + ((k * 2048) >> 4), bd + ((k * 2048) >> 4), ID_KV | kIdescAMN, 1);
                    }
                    if (h2 == 1) mma_commit(&m->kv_full[b & 3]);
                }
                __syncwarp();
            }
            if (!ok) break;
            if (OUT && b + 1 < blocks) scores(b + 1);
        }
        // every MMA issued here is complete before TMEM is freed
        if (elect_one()) mma_commit(&m->end[0]);
        __syncwarp();
        (void)mbar_wait_sleep(&m->end[0], 0);
    } else if (warp == 3 && OUT) {
        // ------------------------------------------- issuer: S A^T and V^T P^T ----
        for (; issued < min(Sh::NS - 1, blocks); ++issued) load(issued);
        wait_here();
        for (int b = 0; b < blocks; ++b) {
            // block b - 1 is done, and its state product, which the other issuer committed:
            // its stage takes block b + 2 while S is on its way
            if (b > 0 && !warp_wait(BAR(done, (b - 1) % 3), (b - 1) / 3, E_MMA)) break;
            if (issued < blocks) {
                if (b > 0 && !warp_wait(BAR(kv_full, (b - 1) & 3), (b - 1) >> 2, E_MMA)) break;
                load(issued);
                ++issued;
            }
            if (!warp_wait(BAR(full, b % Sh::NS), b / Sh::NS, E_TMA)) break;
            if (!warp_wait(BAR(s_full, 0), b, E_HANDOFF)) break;
            if (b > 0 && !warp_wait(BAR(o_free, (b - 1) & 1), (b - 1) >> 1, E_HANDOFF)) break;
            tc_fence_after();
            const uint32_t st = ((b % Sh::NS) * Sh::STAGE) >> 4;
            const uint64_t ad = kmajor + st, vd = mnmajor + (st + (Sh::V_OFF >> 4));
            const uint64_t pd = kmajor + ((Sh::P_OFF + (b & 1) * 16384) >> 4);
            if (elect_one()) {
#pragma unroll
                for (int part = 1; part >= 0; --part)
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        mma_f16_ts(tmem + T_OI, tmem + (part ? T_SL : T_SB) + k * 8,
                                   ad + (((k >> 2) * 8192 + (k & 3) * 32) >> 4), ID_N64, part != 1 || k != 0);
                mma_commit(&m->s_free);
            }
            __syncwarp();
            if (!warp_wait(BAR(p_full, b & 1), b >> 1, E_HANDOFF)) break;
            tc_fence_after();
            if (elect_one()) {
#pragma unroll
                for (int part = 1; part >= 0; --part)
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        mma_f16_ss(tmem + T_X + (b & 1) * 64, vd + ((k * 2048) >> 4),
                                   pd + ((part * 8192 + k * 32) >> 4), ID_PV, part != 1 || k != 0);
                mma_commit(&m->done[b % 3]);
            }
            __syncwarp();
        }
        if (elect_one()) mma_commit(&m->end[1]);
        __syncwarp();
        (void)mbar_wait_sleep(&m->end[1], 0);
        drain(issued);
    } else if (warp == 3) {
        // ---------------------------------------- loader of the state's pass ----
        for (; issued < blocks; ++issued) {
            // a stage is free when the product that reads it is done
            const int f = issued - Sh::NS;
            if (f >= 0 && !warp_wait(BAR(kv_full, f & 3), f >> 2, E_MMA)) break;
            load(issued);
        }
        drain(issued);
    } else if (OUT) {
        // ------------------------------------------- P = scores .* decay, row i ----
        const int i = tid;
        const uint32_t lanes = (uint32_t)warp << 21;
        // Row i of M in halves of 32 columns: one lies on the diagonal, the other one on the
        // causal side of all of this warp's rows or on the other side of them all.
        float2 near[16], far[16];
#pragma unroll
        for (int e = 0; e < 32; e += 2) {
            const int a0 = REV ? e - lane : lane - e, a1 = REV ? a0 + 1 : a0 - 1;
            near[e / 2] = make_float2(m->pw[max(a0, 0)], m->pw[max(a1, 0)]);
            far[e / 2] = make_float2(m->pw[32 + a0], m->pw[32 + a1]);
        }
        const bool both = warp == (REV ? 0 : 1);
        if (!both)                       // zeros that stay
            for (int q = 0; q < 16; ++q)
                st_shared_v4(sbase + Sh::P_OFF + (q >> 2) * 8192 + sw128_offset(i, (1 - warp) * 4 + (q & 3)), 0, 0, 0, 0);
        for (int b = 0; b < blocks; ++b) {
            if (b == (block_n(0) == C)) wait_here();
            if (!warp_wait(BAR(sc_full, b & 1), b >> 1, E_MMA)) break;
            if (b >= 2 && !warp_wait(BAR(done, (b - 2) % 3), (b - 2) / 3, E_MMA)) break;
            tc_fence_after();
            const uint32_t dst = sbase + Sh::P_OFF + (b & 1) * 16384, from = tmem + lanes + T_X + (b & 1) * 64;
            auto columns = [&](auto on_diagonal, const float2 (&decay)[16], int half) {
                uint32_t x[32];
                tmem_ld32(from + half * 32, x);
                tmem_wait_ld();
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    uint32_t hi[4], lo[4];
#pragma unroll
                    for (int u = 0; u < 4; ++u) {
                        const int e = q * 8 + u * 2;
                        float2 s = __fmul2_rn(make_float2(__uint_as_float(x[e]), __uint_as_float(x[e + 1])), decay[e / 2]);
                        if (decltype(on_diagonal)::value) {    // by selection: a score may be anything there
                            s.x = (REV ? e >= lane : e <= lane) ? s.x : 0.f;
                            s.y = (REV ? e + 1 >= lane : e + 1 <= lane) ? s.y : 0.f;
                        }
                        hi[u] = pack_bf16(s.x, s.y);
                        lo[u] = rest_bf16(s, hi[u]);
                    }
                    const uint32_t to = dst + sw128_offset(i, half * 4 + q);
                    st_shared_v4(to, hi[0], hi[1], hi[2], hi[3]);
                    st_shared_v4(to + 8192, lo[0], lo[1], lo[2], lo[3]);
                }
            };
            // (behind a reversed segment's last token the scores are zeros, as B's rows are)
            columns(std::true_type{}, near, warp);
            if (both) columns(std::false_type{}, far, 1 - warp);
            tc_fence_before();
            fence_proxy_async();
            arrive(BAR(p_full, b & 1));
        }
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 0) {
        tc_fence_after();
        tmem_dealloc(tmem, T_COLS);
    }
}

template <bool OUT, bool REV, typename OutT>
cudaError_t launch(const CUtensorMap &ma, const CUtensorMap &mb, const CUtensorMap &mv,
                   const ScanArgs &p, bool after, cudaStream_t stream) {
    auto fn = scan_tc_kernel<OUT, REV, OutT>;
    cudaError_t e = ensure_dynamic_smem(reinterpret_cast<const void *>(fn), smem_bytes<OUT>());
    if (e != cudaSuccess) return e;
    return launch_kernel(after, fn, dim3((unsigned)(OUT ? p.slots : p.inner) * p.H), kThreads, smem_bytes<OUT>(),
                         stream, ma, mb, mv, p);
}

}  // namespace

// [T, H, 128] bf16 seen as {64 channels, T, 2 halves, H}: one box is a tile of 64
// tokens by 128 channels of one head, its halves one after the other.
bool scan_tile_map(CUtensorMap *map, const void *base, int total_T, int H) {
    cuuint64_t dims[4] = {64, (cuuint64_t)total_T, 2, (cuuint64_t)H};
    cuuint64_t strides[3] = {(cuuint64_t)H * D * 2, 128, (cuuint64_t)D * 2};
    cuuint32_t box[4] = {64, C, 2, 1};
    cuuint32_t estr[4] = {1, 1, 1, 1};
    return encode_map(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void *>(base), dims, strides, box, estr,
                      CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                      CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
}

cudaError_t launch_scan_tc(const CUtensorMap &ma, const CUtensorMap &mb, const CUtensorMap &mv, const ScanArgs &p,
                           bool reverse, bool states, bool out_f32, bool after, cudaStream_t stream) {
    if (states)
        return reverse ? launch<false, true, float>(ma, mb, mv, p, after, stream)
                       : launch<false, false, float>(ma, mb, mv, p, after, stream);
    if (out_f32)
        return reverse ? launch<true, true, float>(ma, mb, mv, p, after, stream)
                       : launch<true, false, float>(ma, mb, mv, p, after, stream);
    return reverse ? launch<true, true, __nv_bfloat16>(ma, mb, mv, p, after, stream)
                   : launch<true, false, __nv_bfloat16>(ma, mb, mv, p, after, stream);
}

}  // namespace gdr
