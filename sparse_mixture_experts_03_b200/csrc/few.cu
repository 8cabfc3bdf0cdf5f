// The whole layer for a few tokens (T <= 16) in two launches.
//
// With a few tokens the layer is a stream of weights: every byte of the
// touched experts is read once (T = 1 at d 2048, inter 1536, 6 + 4 experts:
// 189 MB in bf16) and each is used for at most T multiply-adds, so what counts
// is that the reads never pause.  The five launches of moe_forward pause them
// at each boundary (routing, permutation, the two GEMMs, the sum); here
//
//   few_logits_kernel  the router logits (one CTA per expert, fp32 sums in a
//                      fixed order) and the reset of the counters below
//   few_layer_kernel   everything else, one persistent CTA per SM:
//     - its producer warp streams weights into a ring of shared-memory stages
//       (one bulk copy per weight row piece of up to 2 KB) and takes its work
//       from one ticket counter: first units of 8 gate + 8 up rows, shared
//       experts before routed ones, then units of down rows.  The shared
//       experts need no routing, so their weights stream while the logits are
//       still being made, and nothing that the second half waits for holds
//       back its weights: the ring is full again when h is ready.
//     - its 8 consumer warps split the reduction of each unit (every 8th block
//       of 128) and multiply on mma.sync m16n8k16: the weights are the 16 rows
//       of A, read from the stage as 16 bytes per lane, the tokens the 8
//       columns of B.  The tensor work is a few percent of what the SM can do;
//       tcgen05 tiles of 128 rows would only make the units coarser.
//     - every consumer warp in turn adds the 8 partial sums of a unit in warp
//       order; gate and up rows of a feature meet in one lane, h = silu(g) u is
//       rounded once to bf16 (the operand type of the down product).  Down
//       sums go, times the gate weight, into fp32 slots [token][S + k][d]; the
//       last unit of a 16-column piece of y adds the slots, shared experts
//       first, then the token's choices in top-k order, and rounds once.
//
// Results do not depend on which CTA took which ticket: every unit is summed
// the same way wherever it runs, and the slots are added in order.
//
// Waits between CTAs (down units wait for the h of their expert) cannot
// deadlock whatever else runs on the GPU: tickets are handed out in order, so
// all that a ticket waits for is in the hands of CTAs that already run and
// that never wait for a later ticket.  All waits are bounded.
//
// 8-bit weights (e4m3, one fp32 scale per 128 x 128 block) take half the
// bytes: a stage row of 2 KB holds 2048 of them, the codes become bf16 (exact)
// on the way to the same products, and each 128-block's sum is scaled in fp32
// before it is added; the scales travel with the stage.
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <limits.h>

#include <algorithm>

#include "moe_device.cuh"
#include "moe_internal.h"
#include "route_select.cuh"

namespace moe {
namespace {

constexpr int kFewMaxT = 16;
constexpr int kWarps = 8;                       // consumer warps
constexpr int kFewThreads = 32 * (kWarps + 1);  // + the producer warp
constexpr int kRowBytes = 2048;                 // bytes of one weight row in a stage
// Row pitch: 64 bytes more than a multiple of 128, so that the 8 lanes of a
// quarter warp (2 rows x 64 bytes) read 8 different 16-byte bank groups.
constexpr int kRowPitch = kRowBytes + 64;
constexpr int kStageBytes = 16 * kRowPitch;
constexpr int kMaxStages = 6;
constexpr int kMaxShared = 64;                  // shared experts
constexpr int kMaxEntries = kMaxShared + kFewMaxT * kMaxK;
constexpr int kSmemMax = 227 * 1024;
constexpr int kLogitThreads = 256;

// Control words (reset by few_logits_kernel): the ticket counter, finished
// gate/up units per entry, finished entries per 16 columns of y.
constexpr int kCtrlTicket = 0;
constexpr int kCtrlH = 32;
constexpr int kCtrlY = kCtrlH + kMaxEntries;

struct FewArgs {
    const __nv_bfloat16* x;
    const void* w_gate_up;  // [E, 2 I, d]
    const void* w_down;     // [E, d, I]
    const void* w_shared;   // [2 S I, d], then [d, S I]
    const float* s_gate_up; // 8-bit weights: scales [E, 2 I / 128, d / 128]
    const float* s_down;    // [E, d / 128, I / 128]
    const float* s_shared;  // [2 S I / 128, d / 128], then [d / 128, S I / 128]
    const float* logits;    // [T, E]
    const float* bias;
    int T, d, E, k, G, TG, gate, I, S, out_f32;
    int stages;
    int tile_rows;          // 16-row pieces of a down ticket
    void* y;
    int32_t* idx_out;
    float* w_out;
    int* status;
    int* ctrl;
    __nv_bfloat16* h;       // [entries][T][I]
    float* slots;           // [T][S + k][d]
    unsigned long long wait_limit_ns;
};

// One CTA per expert: logits[t][e] = x[t] . W_router[e]; a warp per token.
__global__ void __launch_bounds__(kLogitThreads) few_logits_kernel(
    const __nv_bfloat16* __restrict__ x, const __nv_bfloat16* __restrict__ Wr, int T, int d,
    int E, float* __restrict__ logits, int* status, int* ctrl, int n_ctrl) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int e = blockIdx.x;
    pdl_wait();
    // the layer kernel may be scheduled: it waits for this one where it needs it
    pdl_trigger();
    for (int i = e * kLogitThreads + tid; i < n_ctrl; i += gridDim.x * kLogitThreads) ctrl[i] = 0;
    if (e == 0 && tid < 16) status[tid] = 0;
    const uint4* wr = reinterpret_cast<const uint4*>(Wr + (size_t)e * d);
    for (int t = warp; t < T; t += kLogitThreads / 32) {
        const uint4* xr = reinterpret_cast<const uint4*>(x + (size_t)t * d);
        float a0 = 0.f, a1 = 0.f;  // even and odd columns
#pragma unroll 4
        for (int i = lane; i < d / 8; i += 32) {
            const uint4 a = __ldg(xr + i), b = __ldg(wr + i);
            const uint32_t aw[4] = {a.x, a.y, a.z, a.w}, bw[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                a0 = fmaf(__uint_as_float(aw[q] << 16), __uint_as_float(bw[q] << 16), a0);
                a1 = fmaf(__uint_as_float(aw[q] & 0xffff0000u),
                          __uint_as_float(bw[q] & 0xffff0000u), a1);
            }
        }
        float v = a0 + a1;
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
        if (lane == 0) logits[(size_t)t * E + e] = (v != v) ? -INFINITY : v;
    }
}

// ---------------------------------------------------------------- copies
__device__ __forceinline__ void bulk_copy(void* dst, const void* src, uint32_t bytes,
                                          uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
        ::"r"(smem_u32(dst)), "l"(src), "r"(bytes), "r"(smem_u32(bar))
        : "memory");
}
__device__ __forceinline__ void prefetch_l2(const void* src, uint32_t bytes) {
    asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void copy_scale(float* dst, const float* src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(dst)), "l"(src)
                 : "memory");
}
// one arrival on `bar` when this lane's cp.async copies have landed
__device__ __forceinline__ void copies_arrive(uint64_t* bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar))
                 : "memory");
}
__device__ __forceinline__ void consumers_sync() {
    asm volatile("bar.sync 1, %0;" ::"n"(32 * kWarps) : "memory");
}

__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, "
        "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// four e4m3 codes as two bf16 pairs (exact: 4 significant bits; NaN stays NaN)
__device__ __forceinline__ void widen(uint32_t codes, uint32_t& lo, uint32_t& hi) {
    const __half2_raw h0 = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(codes & 0xffffu),
                                                      __NV_E4M3);
    const __half2_raw h1 = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(codes >> 16),
                                                      __NV_E4M3);
    const float2 f0 = __half22float2(__half2(h0)), f1 = __half22float2(__half2(h1));
    lo = pack_bf16x2(f0.x, f0.y);
    hi = pack_bf16x2(f1.x, f1.y);
}

// ---------------------------------------------------------------- work
// A unit is 16 weight rows over their whole reduction.  up: gate/up rows
// (8 gate + the 8 matching up rows) of feature 8 * tile; else down rows
// [16 * tile, 16 * tile + 16).
struct Unit {
    int up;     // 1 gate/up, 0 down, -1 no more work
    int entry;  // 0 .. S-1 shared experts, then the routed experts that have tokens
    int tile;
};

struct Smem {
    uint8_t* ring;
    uint4* b;        // operand B: x (gate/up units), then the h of one entry
    float4* red;     // [2][kWarps][NT][32]
    float* scales;   // [stages][32]
    int4* info;      // [stages]
    uint64_t* full;
    uint64_t* empty;
    uint64_t* routed;  // the entry list is there
    uint64_t* meet;    // the consumer warps, once or twice per unit
    int* s_idx;      // [T][k]
    float* s_w;
    uint32_t* s_mask;  // [E] tokens of each expert
    int* list;         // [entries]: expert of a routed entry
    int* n_entries;
    int* abort;
};

template <int NT>
__host__ __device__ constexpr int red_bytes() {
    return 2 * kWarps * NT * 32 * 16;  // also holds the logits: T * E * 4 <= 8 NT * 256 * 4
}
constexpr int kSmallBytes = kMaxStages * (32 * 4 + 16 + 16) + 64 + kFewMaxT * kMaxK * 8 +
                            kMaxE * 4 + kMaxEntries * 4 + 64;

template <int NT>
__host__ __device__ inline int b_bytes(int d, int I) {
    return 8 * NT * 2 * (d > I ? d : I);
}

template <int NT>
__device__ __forceinline__ Smem carve(uint8_t* p, int stages, int d, int I) {
    Smem s;
    s.ring = p;
    p += stages * kStageBytes;
    s.b = reinterpret_cast<uint4*>(p);
    p += b_bytes<NT>(d, I);
    s.red = reinterpret_cast<float4*>(p);
    p += red_bytes<NT>();
    s.info = reinterpret_cast<int4*>(p);
    p += kMaxStages * 16;
    s.full = reinterpret_cast<uint64_t*>(p);
    p += kMaxStages * 8;
    s.empty = reinterpret_cast<uint64_t*>(p);
    p += kMaxStages * 8;
    s.routed = reinterpret_cast<uint64_t*>(p);
    s.meet = s.routed + 1;
    p += 16;
    s.scales = reinterpret_cast<float*>(p);
    p += kMaxStages * 32 * 4;
    s.s_idx = reinterpret_cast<int*>(p);
    p += kFewMaxT * kMaxK * 4;
    s.s_w = reinterpret_cast<float*>(p);
    p += kFewMaxT * kMaxK * 4;
    s.s_mask = reinterpret_cast<uint32_t*>(p);
    p += kMaxE * 4;
    s.list = reinterpret_cast<int*>(p);
    p += kMaxEntries * 4;
    s.n_entries = reinterpret_cast<int*>(p);
    s.abort = s.n_entries + 1;
    return s;
}

// Pieces of a reduction of K elements: n of len elements (a multiple of 128)
// whose rows fit a stage; the last may be shorter.
struct Pieces {
    int n, len;
};
__device__ __forceinline__ Pieces pieces(int K, int esz) {
    Pieces p;
    p.n = (K * esz + kRowBytes - 1) / kRowBytes;
    p.len = ((K + p.n - 1) / p.n + 127) / 128 * 128;
    p.n = (K + p.len - 1) / p.len;
    return p;
}

// Wait until *p (written by other CTAs) is at least `want`; bounded.
__device__ __forceinline__ bool wait_count(const int* p, int want, volatile int* abort,
                                           int* status, int site, unsigned long long limit_ns) {
    const long long t0 = clock64();
    for (;;) {
        int v;
        asm volatile("ld.acquire.gpu.global.s32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
        if (v >= want) return true;
        if (*abort) return false;
        if ((unsigned long long)(clock64() - t0) > 2 * limit_ns) {
            *abort = 1;
            set_status(status, MOE_ERR_TIMEOUT, site);
            return false;
        }
        __nanosleep(40);
    }
}

// ---------------------------------------------------------------- producer
template <bool FP8>
__device__ __forceinline__ void producer(const FewArgs& a, const Smem& s, int lane) {
    constexpr int esz = FP8 ? 1 : 2;
    const int d = a.d, I = a.I, S = a.S;
    const int up_tiles = I / 8, down_tickets = d / 16 / a.tile_rows;
    const int shared_units = S * up_tiles;
    const Pieces pu = pieces(d, esz), pd = pieces(I, esz);
    const char* wgu = static_cast<const char*>(a.w_gate_up);
    const char* wdn = static_cast<const char*>(a.w_down);
    const char* wsh = static_cast<const char*>(a.w_shared);
    const size_t SI = (size_t)S * I;
    // The first tickets are shared gate/up units: this CTA's part of them goes
    // to L2 now, while the logits are being made.  (Which CTA takes a ticket is
    // open, but together they take these.)
    if (lane < 16) {
        for (int u = blockIdx.x; u < shared_units && u < 2 * (int)gridDim.x; u += gridDim.x) {
            const size_t row = (size_t)u * 8 + (lane & 7) + (lane >= 8 ? SI : 0);
            prefetch_l2(wsh + row * d * esz, (uint32_t)(d * esz));
        }
    }
    pdl_wait();  // the control words are reset
    int slot = 0, phase = 0;
    int n_entries = -1;  // unknown until the routing is there
    int ticket = 0, next = 0;
    if (lane == 0) ticket = atomicAdd(a.ctrl + kCtrlTicket, 1);
    for (;;) {
        ticket = __shfl_sync(0xffffffffu, ticket, 0);
        if (ticket >= shared_units && n_entries < 0) {
            bool ok = mbar_wait_bounded(s.routed, 0, s.abort, a.status, SITE_GEMM_PRODUCER,
                                        a.wait_limit_ns);
            if (!__all_sync(0xffffffffu, ok)) break;
            n_entries = *s.n_entries;
        }
        const bool is_up = ticket < shared_units || ticket < n_entries * up_tiles;
        const int rest = ticket - (is_up ? 0 : n_entries * up_tiles);
        if (!is_up && rest >= n_entries * down_tickets) break;
        if (lane == 0) next = atomicAdd(a.ctrl + kCtrlTicket, 1);  // used one ticket later
        const int entry = rest / (is_up ? up_tiles : down_tickets);
        const int within = rest - entry * (is_up ? up_tiles : down_tickets);
        const int expert = entry < S ? -1 : s.list[entry];
        const Pieces p = is_up ? pu : pd;
        const int K = is_up ? d : I;
        const int n_tiles = is_up ? 1 : a.tile_rows;
        bool ok = true;
        for (int i = 0; i < n_tiles && ok; ++i) {
            const int tile = is_up ? within : within * a.tile_rows + i;
            // this lane's weight row and (8-bit) its row of scales
            const char* row;
            const float* sc = nullptr;
            const int r = lane & 15;
            if (is_up) {
                const size_t f = (size_t)tile * 8 + (r & 7);
                const size_t F = expert < 0 ? SI : (size_t)I;
                const size_t in = f + (expert < 0 ? (size_t)entry * I : 0);
                const size_t g = (expert < 0 ? 0 : (size_t)expert * 2 * I) + in + (r >= 8 ? F : 0);
                row = (expert < 0 ? wsh : wgu) + g * d * esz;
                if (FP8) {
                    // lanes 0..15: the gate rows' scales, 16..31: the up rows'
                    const size_t first = (expert < 0 ? 0 : (size_t)expert * 2 * I) +
                                         (size_t)tile * 8 +
                                         (expert < 0 ? (size_t)entry * I : 0) +
                                         (lane >= 16 ? F : 0);
                    sc = (expert < 0 ? a.s_shared : a.s_gate_up) + first / 128 * (d / 128);
                }
            } else {
                const size_t o = (size_t)tile * 16 + r;
                row = expert < 0 ? wsh + (2 * SI * d + o * SI + (size_t)entry * I) * esz
                                 : wdn + ((size_t)expert * d + o) * I * esz;
                if (FP8) {
                    const size_t ob = (size_t)tile * 16 / 128;
                    sc = expert < 0 ? a.s_shared + 2 * SI / 128 * (d / 128) + ob * (SI / 128) +
                                          (size_t)entry * I / 128
                                    : a.s_down + ((size_t)expert * (d / 128) + ob) * (I / 128);
                }
            }
            for (int c = 0; c < p.n; ++c) {
                ok = mbar_wait_bounded(s.empty + slot, phase ^ 1, s.abort, a.status,
                                       SITE_GEMM_PRODUCER, a.wait_limit_ns);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                const int k0 = c * p.len, len = min(p.len, K - k0);
                if (lane == 0) {
                    s.info[slot] = make_int4(is_up ? 1 : 0, entry, tile, c);
                    mbar_arrive_expect_tx(s.full + slot, (uint32_t)(16 * len * esz));
                }
                __syncwarp();
                if (lane < 16)
                    bulk_copy(s.ring + slot * kStageBytes + lane * kRowPitch,
                              row + (size_t)k0 * esz, (uint32_t)(len * esz), s.full + slot);
                if (FP8) {
                    if ((lane & 15) < len / 128 && (is_up || lane < 16))
                        copy_scale(s.scales + slot * 32 + lane, sc + k0 / 128 + (lane & 15));
                    copies_arrive(s.full + slot);
                }
                if (++slot == a.stages) {
                    slot = 0;
                    phase ^= 1;
                }
            }
        }
        if (!ok) break;
        ticket = next;
    }
    // the end of the work, or of a CTA that gave up: a stage without data
    bool ok = mbar_wait_bounded(s.empty + slot, phase ^ 1, s.abort, a.status, SITE_GEMM_PRODUCER,
                                a.wait_limit_ns);
    if (__all_sync(0xffffffffu, ok)) {
        if (lane == 0) {
            s.info[slot] = make_int4(-1, 0, 0, 0);
            mbar_arrive(s.full + slot);
        }
        if (FP8) copies_arrive(s.full + slot);
    } else {
        // gave up: wait for this CTA's own copies before its memory goes away
        // (the stages before `slot`, newest first; those never filled time out)
        int q = slot, ph = phase;
        for (int i = 0; i < a.stages; ++i) {
            if (--q < 0) {
                q = a.stages - 1;
                ph ^= 1;
            }
            mbar_wait_bounded(s.full + q, ph, nullptr, nullptr, SITE_GEMM_DRAIN, 1000000ull);
        }
    }
}

// ---------------------------------------------------------------- consumers
// Rows [T][K] of bf16 into operand B: the 8 tokens of a column group as the
// lanes (token, quarter) hold them.  A group of reduction elements (64 bytes
// of a weight row: 32 bf16, 64 e4m3) is split into quarters of consecutive
// elements, the same for A and B, which permutes the reduction inside the
// group and nothing else.  Piece j (8 elements, 16 bytes) of a quarter of group
// i of token t is b[((i * PPQ + j) * NT + t / 8) * 32 + (t % 8) * 4 + quarter],
// PPQ = pieces per quarter (1 or 2).
template <int NT, bool FP8>
__device__ __forceinline__ void fill_b(uint4* b, const __nv_bfloat16* src, size_t ld, int K,
                                       uint32_t mask, int n_tok, bool zero_rest, int tid) {
    constexpr int PPQ = FP8 ? 2 : 1;
    const int per_tok = K / 8;
    for (int i = tid; i < n_tok * per_tok; i += 32 * kWarps) {
        const int t = i / per_tok, p = i - t * per_tok;
        const bool have = (mask >> t) & 1u;
        if (!have && !zero_rest) continue;
        uint4 v = make_uint4(0, 0, 0, 0);
        if (have) v = __ldcg(reinterpret_cast<const uint4*>(src + (size_t)t * ld) + p);
        const int grp = p / (4 * PPQ), in = p - grp * 4 * PPQ;
        const int quarter = in / PPQ, j = in - quarter * PPQ;
        b[((grp * PPQ + j) * NT + (t >> 3)) * 32 + (t & 7) * 4 + quarter] = v;
    }
}

// This warp's part of one stage: blocks of 128 whose number (counted over the
// whole reduction) is the warp's modulo 8.
template <int NT, bool FP8>
__device__ __forceinline__ void stage_mma(const uint8_t* st, const uint4* b, const float* scales,
                                          int k0, int len, bool up, int warp, int lane,
                                          float (&acc)[NT][4]) {
    const uint8_t* r0 = st + (lane >> 2) * kRowPitch + (lane & 3) * 16;
    const uint8_t* r1 = r0 + 8 * kRowPitch;
    const int first = k0 / 128;
    for (int j = (warp - first) & 7; j < len / 128; j += kWarps) {
        if constexpr (!FP8) {
#pragma unroll
            for (int g = 0; g < 4; ++g) {  // 32 elements each
                const uint4 lo = *reinterpret_cast<const uint4*>(r0 + j * 256 + g * 64);
                const uint4 hi = *reinterpret_cast<const uint4*>(r1 + j * 256 + g * 64);
                const uint4* bp = b + ((first + j) * 4 + g) * NT * 32 + lane;
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    const uint4 v = bp[n * 32];
                    mma16816(acc[n], lo.x, hi.x, lo.y, hi.y, v.x, v.y);
                    mma16816(acc[n], lo.z, hi.z, lo.w, hi.w, v.z, v.w);
                }
            }
        } else {
            float part[NT][4];
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int q = 0; q < 4; ++q) part[n][q] = 0.f;
#pragma unroll
            for (int g = 0; g < 2; ++g) {  // 64 elements each
                const uint4 lo = *reinterpret_cast<const uint4*>(r0 + j * 128 + g * 64);
                const uint4 hi = *reinterpret_cast<const uint4*>(r1 + j * 128 + g * 64);
                const uint32_t l4[4] = {lo.x, lo.y, lo.z, lo.w}, h4[4] = {hi.x, hi.y, hi.z, hi.w};
                const uint4* bp = b + ((first + j) * 2 + g) * 2 * NT * 32 + lane;
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    uint32_t a0, a1, a2, a3;
                    widen(l4[q], a0, a2);
                    widen(h4[q], a1, a3);
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        const uint2 v = reinterpret_cast<const uint2*>(
                            bp + ((q >> 1) * NT + n) * 32)[q & 1];
                        mma16816(part[n], a0, a1, a2, a3, v.x, v.y);
                    }
                }
            }
            const float s0 = scales[j], s1 = up ? scales[16 + j] : s0;
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                acc[n][0] = fmaf(part[n][0], s0, acc[n][0]);
                acc[n][1] = fmaf(part[n][1], s0, acc[n][1]);
                acc[n][2] = fmaf(part[n][2], s1, acc[n][2]);
                acc[n][3] = fmaf(part[n][3], s1, acc[n][3]);
            }
        }
    }
}

// All consumer warps meet (bounded, unlike bar.sync: a warp that gave up does
// not come).
__device__ __forceinline__ bool warps_meet(const FewArgs& a, const Smem& s, int lane,
                                           int& parity) {
    __syncwarp();
    if (lane == 0) mbar_arrive(s.meet);
    const bool ok = mbar_wait_bounded(s.meet, parity, s.abort, a.status, SITE_GEMM_EPILOGUE,
                                      a.wait_limit_ns);
    parity ^= 1;
    return __all_sync(0xffffffffu, ok);
}

template <int NT, bool FP8>
__device__ __forceinline__ void consumer(const FewArgs& a, const Smem& s, int warp, int lane) {
    constexpr int esz = FP8 ? 1 : 2;
    const int tid = warp * 32 + lane;
    const int T = a.T, d = a.d, E = a.E, k = a.k, I = a.I, S = a.S;
    const uint32_t all = T >= 32 ? 0xffffffffu : (1u << T) - 1u;
    // ---- x as operand B
    fill_b<NT, FP8>(s.b, a.x, d, d, all, 8 * NT, true, tid);
    for (int e = tid; e < E; e += 32 * kWarps) s.s_mask[e] = 0;
    // ---- routing: every CTA chooses for itself, CTA 0 writes it out
    pdl_wait();
    float* lg = reinterpret_cast<float*>(s.red);
    for (int i = tid; i < T * E; i += 32 * kWarps) lg[i] = __ldcg(a.logits + i);
    consumers_sync();
    for (int t = warp; t < T; t += kWarps) {
        warp_topk<kMaxE / 32>(lg + t * E, lane, E, k, a.G, a.TG, a.gate, a.bias, s.s_idx + t * k,
                              s.s_w + t * k);
        __syncwarp();
        if (lane < k) {
            atomicOr(s.s_mask + s.s_idx[t * k + lane], 1u << t);
            if (blockIdx.x == 0) {
                if (a.idx_out != nullptr) a.idx_out[t * k + lane] = s.s_idx[t * k + lane];
                if (a.w_out != nullptr) a.w_out[t * k + lane] = s.s_w[t * k + lane];
            }
        }
    }
    consumers_sync();
    if (warp == 0) {
        int n = S;
        for (int e0 = 0; e0 < E; e0 += 32) {
            const int e = e0 + lane;
            const bool on = e < E && s.s_mask[e] != 0;
            const uint32_t vote = __ballot_sync(0xffffffffu, on);
            if (on) s.list[n + __popc(vote & ((1u << lane) - 1u))] = e;
            n += __popc(vote);
        }
        if (lane == 0) *s.n_entries = n;
        __syncwarp();
        if (lane == 0) mbar_arrive(s.routed);
    }
    consumers_sync();
    const int n_entries = *s.n_entries;

    // ---- units
    const Pieces pu = pieces(d, esz), pd = pieces(I, esz);
    float acc[NT][4];
    int slot = 0, phase = 0;
    int unit = 0;          // finished units: whose turn it is, and which buffer
    int have = -1;         // entry whose h is operand B
    int parity = 0;
    for (;;) {
        const bool filled = mbar_wait_bounded(s.full + slot, phase, s.abort, a.status,
                                              SITE_GEMM_MMA, a.wait_limit_ns);
        if (!__all_sync(0xffffffffu, filled)) return;
        const int4 info = s.info[slot];
        if (info.x < 0) return;
        const bool up = info.x == 1;
        const int entry = info.y, tile = info.z, c = info.w;
        const Pieces p = up ? pu : pd;
        const int K = up ? d : I;
        const uint32_t mask = entry < S ? all : s.s_mask[s.list[entry]];
        if (!up && have != entry) {
            // every warp is past the last unit's products (they met after it)
            bool ok = wait_count(a.ctrl + kCtrlH + entry, I / 8, s.abort, a.status,
                                 SITE_GEMM_BOUNDS, a.wait_limit_ns);
            if (!__all_sync(0xffffffffu, ok)) return;
            fill_b<NT, FP8>(s.b, a.h + (size_t)entry * T * I, I, I, mask, T, false, tid);
            have = entry;
            if (!warps_meet(a, s, lane, parity)) return;
        }
        if (c == 0) {
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int q = 0; q < 4; ++q) acc[n][q] = 0.f;
        }
        const int k0 = c * p.len;
        stage_mma<NT, FP8>(s.ring + slot * kStageBytes, s.b, s.scales + slot * 32, k0,
                           min(p.len, K - k0), up, warp, lane, acc);
        __syncwarp();
        if (lane == 0) mbar_arrive(s.empty + slot);
        if (++slot == a.stages) {
            slot = 0;
            phase ^= 1;
        }
        if (c + 1 < p.n) continue;
        // ---- the unit's sums
        float4* red = s.red + (unit & 1) * kWarps * NT * 32;
#pragma unroll
        for (int n = 0; n < NT; ++n)
            red[(warp * NT + n) * 32 + lane] =
                make_float4(acc[n][0], acc[n][1], acc[n][2], acc[n][3]);
        if (!warps_meet(a, s, lane, parity)) return;
        const bool mine = (unit & 7) == warp;
        ++unit;
        if (!mine) continue;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            float4 v = red[n * 32 + lane];
#pragma unroll
            for (int w = 1; w < kWarps; ++w) {
                const float4 o = red[(w * NT + n) * 32 + lane];
                v.x += o.x;
                v.y += o.y;
                v.z += o.z;
                v.w += o.w;
            }
            const int g = lane >> 2;
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                const int t = 8 * n + 2 * (lane & 3) + q;
                if (t >= T || !((mask >> t) & 1u)) continue;
                const float s0 = q ? v.y : v.x, s1 = q ? v.w : v.z;  // rows g and g + 8
                if (up) {
                    const float h = s0 / (1.f + expf(-s0)) * s1;
                    a.h[((size_t)entry * T + t) * I + tile * 8 + g] = __float2bfloat16_rn(h);
                } else {
                    int j = entry;
                    float wt = 1.f;
                    if (entry >= S) {
                        const int e = s.list[entry];
                        for (int i = 0; i < k; ++i)
                            if (s.s_idx[t * k + i] == e) {
                                j = S + i;
                                wt = s.s_w[t * k + i];
                            }
                    }
                    float* o = a.slots + ((size_t)t * (S + k) + j) * d + tile * 16 + g;
                    __stcg(o, wt * s0);
                    __stcg(o + 8, wt * s1);
                }
            }
        }
        __syncwarp();
        int last = 0;
        if (lane == 0) {
            __threadfence();
            if (up)
                atomicAdd(a.ctrl + kCtrlH + entry, 1);
            else
                last = atomicAdd(a.ctrl + kCtrlY + tile, 1) == n_entries - 1;
            __threadfence();
        }
        last = __shfl_sync(0xffffffffu, last, 0);
        __syncwarp();  // lane 0's fence comes before the other lanes' reads
        if (!last) continue;
        // ---- y of these 16 columns: the slots of each token in order
        for (int i = lane; i < T * 4; i += 32) {
            const int t = i >> 2, col = tile * 16 + (i & 3) * 4;
            const float* src = a.slots + (size_t)t * (S + k) * d + col;
            float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
            for (int j = 0; j < S + k; ++j) {
                const float4 o = __ldcg(reinterpret_cast<const float4*>(src + (size_t)j * d));
                v.x += o.x;
                v.y += o.y;
                v.z += o.z;
                v.w += o.w;
            }
            if (a.out_f32)
                *reinterpret_cast<float4*>(static_cast<float*>(a.y) + (size_t)t * d + col) = v;
            else
                *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.y) + (size_t)t * d + col) =
                    make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
        }
    }
}

template <int NT, bool FP8>
__global__ void __launch_bounds__(kFewThreads, 1) few_layer_kernel(const FewArgs a) {
    extern __shared__ __align__(1024) uint8_t few_smem[];
    const Smem s = carve<NT>(few_smem, a.stages, a.d, a.I);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int i = 0; i < a.stages; ++i) {
            mbar_init(s.full + i, FP8 ? 33 : 1);  // the copies' bytes; 8-bit: + 32 lanes' scales
            mbar_init(s.empty + i, kWarps);
        }
        mbar_init(s.routed, 1);
        mbar_init(s.meet, kWarps);
        *s.abort = 0;
        fence_barrier_init();
    }
    __syncthreads();
    if (warp == kWarps)
        producer<FP8>(a, s, lane);
    else
        consumer<NT, FP8>(a, s, warp, lane);
    __syncthreads();
    pdl_trigger();
}

// ---------------------------------------------------------------- host
enum FewRegion : int { FW_STATUS, FW_CTRL, FW_LOGITS, FW_H, FW_SLOTS, FW_TOTAL };

int few_stages(int T, int d, int I) {
    const int nt = T > 8 ? 2 : 1;
    const long long fixed = (long long)8 * nt * 2 * (d > I ? d : I) +
                            (nt == 1 ? red_bytes<1>() : red_bytes<2>()) + kSmallBytes;
    const long long n = (kSmemMax - fixed) / kStageBytes;
    return n < 2 ? 0 : (int)std::min<long long>(n, kMaxStages);
}

int few_check(int T, int d, int E, int k, int inter, int n_shared) {
    if (T < 0 || d <= 0 || E < 1 || E > kMaxE || k < 1 || k > kMaxK || k > E || inter <= 0 ||
        n_shared < 0)
        return MOE_ERR_INVALID_ARG;
    if (d % 256 != 0 || inter % 128 != 0 || n_shared > kMaxShared || T > kFewMaxT ||
        (long long)n_shared * inter > INT_MAX / 2 || few_stages(T, d, inter) == 0)
        return MOE_ERR_UNSUPPORTED;
    return MOE_OK;
}

bool few_layout(int T, int d, int E, int k, int inter, int n_shared, size_t (&off)[FW_TOTAL + 1]) {
    if (few_check(T, d, E, k, inter, n_shared) != MOE_OK) return false;
    const size_t entries = (size_t)n_shared + std::min(E, T * k);
    const size_t sizes[FW_TOTAL] = {sizeof(int) * kStatusWords, sizeof(int) * (kCtrlY + d / 16),
                                    sizeof(float) * T * E, 2 * entries * T * inter,
                                    sizeof(float) * T * (n_shared + k) * (size_t)d};
    size_t o = 0;
    for (int i = 0; i < FW_TOTAL; ++i) {
        off[i] = o;
        o = (o + sizes[i] + 255) / 256 * 256;
    }
    off[FW_TOTAL] = o;
    return true;
}

template <int NT, bool FP8>
cudaError_t launch_layer(const FewArgs& a, cudaStream_t s) {
    auto kern = few_layer_kernel<NT, FP8>;
    const int smem = a.stages * kStageBytes + b_bytes<NT>(a.d, a.I) + red_bytes<NT>() + kSmallBytes;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    return launch_pdl(kern, dim3((unsigned)num_sms()), dim3(kFewThreads), (size_t)smem, s, 1, a);
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

MOE_API int moe_few_max_tokens(int d, int E, int k, int inter, int n_shared) {
    for (int T = kFewMaxT; T > 0; T = T > 8 ? 8 : 0)
        if (few_check(T, d, E, k, inter, n_shared) == MOE_OK) return T;
    return 0;
}

MOE_API size_t moe_few_workspace_bytes(int T, int d, int E, int k, int inter, int n_shared) {
    size_t off[FW_TOTAL + 1];
    return few_layout(T, d, E, k, inter, n_shared, off) ? off[FW_TOTAL] : 0;
}

MOE_API int moe_forward_few(const void* x, const void* W_router, const void* W_gate_up,
                            const void* W_down, const void* W_shared, const float* s_gate_up,
                            const float* s_down, const float* s_shared, int T, int d, int E,
                            int k, int n_group, int topk_group, int inter, int n_shared,
                            int in_dt, int out_dt, int gate, const float* expert_bias, void* y,
                            int32_t* topk_idx_out, float* topk_w_out, void* workspace,
                            size_t workspace_bytes, void* stream) {
    if (in_dt != MOE_F32 && in_dt != MOE_BF16) return MOE_ERR_INVALID_ARG;
    if (in_dt != MOE_BF16) return MOE_ERR_UNSUPPORTED;
    int st = few_check(T, d, E, k, inter, n_shared);
    if (st != MOE_OK) return st;
    st = check_routing(E, k, n_group, topk_group);
    if (st != MOE_OK) return st;
    if (out_dt != MOE_F32 && out_dt != MOE_BF16) return MOE_ERR_INVALID_ARG;
    if ((n_shared > 0) != (W_shared != nullptr)) return MOE_ERR_INVALID_ARG;
    const bool fp8 = s_gate_up != nullptr;
    if ((s_down != nullptr) != fp8 || (s_shared != nullptr) != (fp8 && n_shared > 0))
        return MOE_ERR_INVALID_ARG;
    size_t off[FW_TOTAL + 1];
    few_layout(T, d, E, k, inter, n_shared, off);
    if (workspace == nullptr || workspace_bytes < off[FW_TOTAL]) return MOE_ERR_WORKSPACE;
    st = check_gating(gate, expert_bias, nullptr);
    if (st != MOE_OK) return st;
    if (T == 0) return MOE_OK;
    const void* p16[] = {x, W_router, W_gate_up, W_down, y, workspace};
    for (const void* p : p16)
        if (!is_device_ptr(p) || !aligned(p, 16)) return MOE_ERR_INVALID_ARG;
    if (n_shared > 0 && (!is_device_ptr(W_shared) || !aligned(W_shared, 16)))
        return MOE_ERR_INVALID_ARG;
    if (!aligned(workspace, 256)) return MOE_ERR_INVALID_ARG;
    const void* p4[] = {s_gate_up, s_down, s_shared, topk_idx_out, topk_w_out};
    for (const void* p : p4)
        if (p != nullptr && (!is_device_ptr(p) || !aligned(p, 4))) return MOE_ERR_INVALID_ARG;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    char* ws = static_cast<char*>(workspace);
    FewArgs a{};
    a.x = static_cast<const __nv_bfloat16*>(x);
    a.w_gate_up = W_gate_up;
    a.w_down = W_down;
    a.w_shared = W_shared;
    a.s_gate_up = s_gate_up;
    a.s_down = s_down;
    a.s_shared = s_shared;
    a.logits = reinterpret_cast<float*>(ws + off[FW_LOGITS]);
    a.bias = expert_bias;
    a.T = T;
    a.d = d;
    a.E = E;
    a.k = k;
    a.G = n_group;
    a.TG = topk_group;
    a.gate = gate;
    a.I = inter;
    a.S = n_shared;
    a.out_f32 = out_dt == MOE_F32;
    a.stages = few_stages(T, d, inter);
    a.tile_rows = 2;
    a.y = y;
    a.idx_out = topk_idx_out;
    a.w_out = topk_w_out;
    a.status = reinterpret_cast<int*>(ws + off[FW_STATUS]);
    a.ctrl = reinterpret_cast<int*>(ws + off[FW_CTRL]);
    a.h = reinterpret_cast<__nv_bfloat16*>(ws + off[FW_H]);
    a.slots = reinterpret_cast<float*>(ws + off[FW_SLOTS]);
    a.wait_limit_ns = kWaitLimitNs;
    cudaError_t e = launch_pdl(few_logits_kernel, dim3((unsigned)E), dim3(kLogitThreads), 0, s, 1,
                               a.x, static_cast<const __nv_bfloat16*>(W_router), T, d, E,
                               reinterpret_cast<float*>(ws + off[FW_LOGITS]), a.status, a.ctrl,
                               kCtrlY + d / 16);
    if (e != cudaSuccess) return MOE_ERR_CUDA;
    if (fp8) return ret(T > 8 ? launch_layer<2, true>(a, s) : launch_layer<1, true>(a, s));
    return ret(T > 8 ? launch_layer<2, false>(a, s) : launch_layer<1, false>(a, s));
}

}  // extern "C"
