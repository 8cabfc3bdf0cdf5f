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
//     - its producer warp streams weights into a ring of shared-memory stages of
//       up to 32 KB, unit after unit of 16 rows: 8 gate + 8 up rows of the shared
//       experts, then of the routed ones, then down rows.  A stage is one TMA
//       box (the rows as 128-byte swizzled atoms): row by row with
//       cp.async.bulk each copy took about 65 ns whatever its size, 4 TB/s
//       in all.  The shared experts need no routing, so their weights
//       stream while the logits are still being made, and nothing that the
//       down rows wait for holds back their weights: the ring is full again
//       when h is ready.
//     - its 8 product warps split the reduction of each unit (every 8th block
//       of 128) and multiply on mma.sync m16n8k16: the weights are the 16 rows
//       of A, read from the stage as 16 bytes per lane, the tokens the 8
//       columns of B.  The tensor work is a few percent of what the SM can do;
//       tcgen05 tiles of 128 rows would only make the units coarser.
//     - 4 sum warps take the units in turn and add their partial sums in warp
//       order; gate and up rows of a feature meet in one lane, h = silu(g) u is
//       rounded once to bf16 (the operand type of the down product).  Down
//       sums go, times the gate weight, into fp32 slots [token][S + k][d]; y adds
//       a token's slots, shared experts first, then its choices in top-k
//       order, and rounds once.
//       What other CTAs wait for (h, the slots) is told once per run of units:
//       a fence behind the stores and a counter take a microsecond or two, more
//       than streaming a unit.  (Told per unit, by the product warps, it made
//       T = 1 take 83 us and T = 16 432 us; per unit but by the sum warps 65
//       and 322.)
//   The units of each part (shared up, routed up, down, y) are cut into gridDim.x
//   runs of neighbours.  CTA b claims run b of each part (ahead of time, so that
//   nothing waits for the answer) and, at its end, any run that a CTA which is
//   not on the GPU yet has left.  Its first run's loads do not wait for the claim
//   or the logits: were the run another's by then, it would store the same h
//   again and not count it.
//
// Results do not depend on which CTA took which run: every unit is summed
// the same way wherever it runs, and the slots are added in order.
//
// Waits between CTAs (down units wait for the h of their expert) cannot
// deadlock whatever else runs on the GPU: a CTA goes to the next part when all
// runs of this one are claimed, so all that a run waits for is in the hands of
// CTAs that already run, and they do it before they wait for anything later.
// All waits are bounded.
//
// 8-bit weights (e4m3, one fp32 scale per 128 x 128 block) take half the
// bytes: a stage row of 2 KB holds 2048 of them, and each 128-block's sum is
// scaled in fp32 before it is added; the scales travel with the stage.  The
// codes become fp16, one instruction for two of them (exact; bf16 takes four
// or five, as much time as the stream), so the tokens are fp16 too: each row
// times a power of two that brings its largest magnitude to [2^14, 2^15).
// bf16's 8 bits fit fp16's 11 down to 2^-28 of the largest magnitude, and what
// lies below is off by at most 2^-39 of it, far less than the fp32 sums are.
// What bounds the 8-bit layer is not one of these steps: at T = 5 it takes 72 us,
// without the products 69, without the conversions 71, without both and the
// reads of the stage 61; a unit is one stage, and a product warp's way through it
// (wait, reads, conversions, products, hand-over) is a chain as long as the
// stage takes to arrive.  Not faster: shifts and masks instead of conversions
// (90 us where this took 80), half and half (87), 16 product warps (82), and
// m16n8k32 on the codes with the tokens as two e4m3 terms (86).
//
// Measured (d 2048, inter 1536, 64 experts of which 6, 4 shared; GPU time): T = 1
// 44.3 us for 189 MB (4.3 TB/s; the floor at the copy rate is 28.9), T = 16
// 184 us for about 1.03 GB (5.6 TB/s; 158), T = 5 on 8-bit weights 71.2 us for
// 273 MB (41.7).  While weights stream they come at 6.4 TB/s; the rest is the
// logits launch and the first loads (5 us), the wait for h between the two
// halves (2 to 4 us) and y (2 us).
#include <cuda_fp16.h>
#include <limits.h>

#include <algorithm>

#include "moe_device.cuh"
#include "moe_internal.h"

namespace moe {
namespace {

constexpr int kFewMaxT = 16;
constexpr int kWarps = 8;                       // product warps
constexpr int kSumWarps = 4;
constexpr int kSumBufs = 2;                     // partial sums in flight (a sum warp frees its
                                                // buffer before it stores and tells)
constexpr int kFewThreads = 32 * (kWarps + kSumWarps + 1);  // + the producer warp
constexpr int kAtomBytes = 16 * 128;            // 16 rows x 128 bytes
// Atoms of a stage.  Half as many made 16 tokens 20% slower (1 KB of a row at a
// time instead of 2).
constexpr int kStageAtoms = 16;
constexpr int kStageBytes = kStageAtoms * kAtomBytes;
constexpr int kMaxStages = 6;
constexpr int kMinRing = 64 * 1024;
constexpr int kMaxGrid = 256;
constexpr int kMaxShared = 64;                  // shared experts
constexpr int kMaxEntries = kMaxShared + kFewMaxT * kMaxK;
constexpr int kSmemMax = 227 * 1024;
constexpr int kLogitThreads = 256;

// The parts of the work, and what a stage or a unit is.
enum Part : int { PART_SHARED_UP, PART_ROUTED_UP, PART_DOWN, PART_Y, kParts };
enum What : int {
    WHAT_END = -1,
    WHAT_DOWN = 0,  // 16 down rows of an entry
    WHAT_UP = 1,    // 8 gate and the 8 matching up rows
    WHAT_TOLD = 2,  // the end of a run: tell the other CTAs
    WHAT_Y = 3,     // 16 columns of y
};
// Control words (reset by few_logits_kernel): the claims of each part's runs,
// the sum warps that finished a down run, finished gate/up units per entry.
constexpr int kCtrlClaim = 0;  // + kMaxGrid * part
constexpr int kCtrlDown = kMaxGrid * kParts;
constexpr int kCtrlH = kCtrlDown + 8;
constexpr int kCtrlWords = kCtrlH + kMaxEntries;

struct FewArgs {
    // Boxes of 16 rows x the atoms of a piece: up [part] {128 bytes, rows, gate |
    // up, atoms}, down [part] {128 bytes, rows, atoms}; 0 shared, 1 routed experts.
    CUtensorMap up_map[2], down_map[2];
    const __nv_bfloat16* x;
    const float* s_gate_up; // 8-bit weights: scales [E, 2 I / 128, d / 128]
    const float* s_down;    // [E, d / 128, I / 128]
    const float* s_shared;  // [2 S I / 128, d / 128], then [d / 128, S I / 128]
    const float* logits;    // [T, E]
    const float* bias;
    int T, d, E, k, G, TG, gate, I, S, out_f32;
    int stages;
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

// ---------------------------------------------------------------- routing
// fp32 as an unsigned number of the same order (NaN and -0 as -inf and +0)
__device__ __forceinline__ uint32_t ordered(float v) {
    if (v != v) v = -INFINITY;
    const uint32_t u = __float_as_uint(v + 0.f);
    return (u >> 31) ? ~u : (u | 0x80000000u);
}

// The k experts of one token and their weights, by one warp: the rules of the
// router kernels (largest keys inside the topk_group groups of largest maximum,
// ties to the lower index).  Lane l holds experts l EJ ..; a round is a warp
// maximum and a vote.  The code runs once per launch and its instructions come
// from L2, so the loops over choices stay loops.  key [E] is scratch.
template <int EJ>
__device__ __forceinline__ void choose(const float* logit, uint32_t* key, int lane, int E, int k,
                                       int G, int TG, int gate, const float* bias, int* idx,
                                       float* w) {
    const int gsz = E / G;
    float mine[EJ];
    uint32_t mk[EJ];
#pragma unroll
    for (int j = 0; j < EJ; ++j) {
        const int e = lane * EJ + j;
        mine[j] = e < E ? __ldcg(logit + e) : 0.f;
    }
#pragma unroll
    for (int j = 0; j < EJ; ++j) {
        const int e = lane * EJ + j;
        mk[j] = 0;  // ordered() never gives 0: it marks what is out
        if (e < E) {
            // the gate score is monotone in the logit: without a bias the logit is the key
            float g = mine[j];
            if (bias != nullptr)
                g = (gate == MOE_GATE_SIGMOID ? 1.f / (1.f + expf(-g)) : g) + bias[e];
            mk[j] = ordered(g);
            key[e] = mk[j];
        }
    }
    __syncwarp();
    uint32_t best = 0;
    if (lane < G) {
#pragma unroll 4
        for (int i = 0; i < gsz; ++i) best = max(best, key[lane * gsz + i]);
    }
    uint32_t kept = 0;
#pragma unroll 1
    for (int r = 0; r < TG; ++r) {
        const uint32_t top = __reduce_max_sync(0xffffffffu, best);
        const int g = __ffs(__ballot_sync(0xffffffffu, best == top)) - 1;
        kept |= 1u << g;
        if (lane == g) best = 0;
    }
#pragma unroll
    for (int j = 0; j < EJ; ++j)
        if (!((kept >> ((unsigned)min(lane * EJ + j, E - 1) / (unsigned)gsz)) & 1u)) mk[j] = 0;
    float l = 0.f;  // lane r: the r-th choice's logit
#pragma unroll 1
    for (int r = 0; r < k; ++r) {
        uint32_t b = mk[0];
        int bj = 0;
        float bl = mine[0];
#pragma unroll
        for (int j = 1; j < EJ; ++j)
            if (mk[j] > b) {
                b = mk[j];
                bj = j;
                bl = mine[j];
            }
        const uint32_t top = __reduce_max_sync(0xffffffffu, b);
        const int src = __ffs(__ballot_sync(0xffffffffu, b == top)) - 1;
        const int e = src * EJ + __shfl_sync(0xffffffffu, bj, src);
        const float v = __shfl_sync(0xffffffffu, bl, src);
        if (lane == r) {
            l = v;
            idx[r] = e;
        }
        if (lane == src) {
#pragma unroll
            for (int j = 0; j < EJ; ++j)
                if (j == bj) mk[j] = 0;
        }
    }
    // weights in the router kernels' order of operations
    float sc;
    if (gate == MOE_GATE_SIGMOID) {
        sc = 1.f / (1.f + expf(-l));
    } else {
        float m = __shfl_sync(0xffffffffu, l, 0);
        for (int r = 1; r < k; ++r) m = fmaxf(m, __shfl_sync(0xffffffffu, l, r));
        sc = expf(l - m);
    }
    float sum = 0.f;
    for (int r = 0; r < k; ++r) sum += __shfl_sync(0xffffffffu, sc, r);
    if (lane < k) w[lane] = sc / sum;
}

// ---------------------------------------------------------------- copies
__device__ __forceinline__ void box_3d(void* dst, const CUtensorMap* map, uint64_t* bar, int row,
                                       int atom) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(0), "r"(row), "r"(atom)
        : "memory");
}
__device__ __forceinline__ void box_4d(void* dst, const CUtensorMap* map, uint64_t* bar, int row,
                                       int atom) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %3, %5}], [%2];" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(0), "r"(row), "r"(atom)
        : "memory");
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
__device__ __forceinline__ void products_sync() {
    asm volatile("bar.sync 1, %0;" ::"n"(32 * kWarps) : "memory");
}
__device__ __forceinline__ void sums_sync() {
    asm volatile("bar.sync 2, %0;" ::"n"(32 * kSumWarps) : "memory");
}

__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, "
        "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma16816_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                             uint32_t a3, uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, "
        "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// four e4m3 codes as two fp16 pairs (exact; NaN stays NaN)
__device__ __forceinline__ void widen(uint32_t codes, uint32_t& lo, uint32_t& hi) {
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(codes));
}

// ---------------------------------------------------------------- work
// A unit is 16 weight rows over their whole reduction: gate/up rows (8 gate + the
// 8 matching up rows) of features 8 * tile .., or down rows 16 * tile ...  It
// belongs to an entry: 0 .. S-1 the shared experts, then the routed experts that
// have tokens, in order.  Stages and units carry (what, entry, tile, piece).
struct Smem {
    uint8_t* ring;
    uint4* b;        // operand B: x (gate/up units), then the h of one entry
    float4* red;     // [kSumBufs][product warps][NT][32]
    float* scales;   // [stages][32]
    int4* info;      // [stages]
    uint64_t* full;
    uint64_t* empty;
    uint64_t* routed;  // the entry list is there
    uint32_t* keys;    // [kSumWarps][E] selection keys
    uint64_t* claimed; // the claims of this CTA's first runs are answered:
    int* first_mine;   // 1: the first shared run is its own
    int* ahead;        // 0: so is the routed one
    uint64_t* meet;    // the product warps, around a new operand B
    uint64_t* sum_full;   // [kSumWarps]: a unit's partial sums are there
    uint64_t* sum_empty;  // [kSumBufs]
    int4* unit;        // [kSumWarps]: the unit
    float* unscale;    // [kFewMaxT] 8-bit weights: 1 / the power of two of operand B's row
    int* s_idx;      // [T][k]
    float* s_w;
    uint32_t* s_mask;  // [E] tokens of each expert
    int* list;         // [entries]: expert of a routed entry
    int* n_entries;
    int* abort;
};

template <int NT>
__host__ __device__ constexpr int red_bytes() {
    return kSumBufs * kWarps * NT * 32 * 16;
}
// everything else in shared memory (1024: the ring's alignment)
constexpr int kSmallBytes = 1024 + kMaxStages * (32 * 4 + 16 + 16) + 64 + kSumWarps * 24 +
                            kSumBufs * 8 + kFewMaxT * 4 + kFewMaxT * kMaxK * 8 + kMaxE * 4 +
                            kMaxEntries * 4 + kSumWarps * kMaxE * 4 + 64;

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
    s.unit = reinterpret_cast<int4*>(p);
    p += kSumWarps * 16;
    s.sum_full = reinterpret_cast<uint64_t*>(p);
    p += kSumWarps * 8;
    s.sum_empty = reinterpret_cast<uint64_t*>(p);
    p += kSumBufs * 8;
    s.unscale = reinterpret_cast<float*>(p);
    p += kFewMaxT * 4;
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
    s.first_mine = s.n_entries + 2;
    s.ahead = s.n_entries + 3;
    p += 16;
    s.claimed = reinterpret_cast<uint64_t*>(p);
    p += 16;
    s.keys = reinterpret_cast<uint32_t*>(p);
    return s;
}

// Pieces of a reduction of K elements: n of len elements (a multiple of 128)
// whose rows fit a stage; the last may be shorter (its box reads on into what
// follows, or zeros, and that is not used).
struct Pieces {
    int n, len;
};
__host__ __device__ __forceinline__ Pieces pieces(int K, int esz) {
    Pieces p;
    const int row_bytes = kStageAtoms * 128;
    p.n = (K * esz + row_bytes - 1) / row_bytes;
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
    const int up_tiles = I / 8, down_tiles = d / 16;
    const int shared_units = S * up_tiles;
    const Pieces pu = pieces(d, esz), pd = pieces(I, esz);
    const size_t SI = (size_t)S * I;
    const int atoms_u = pu.len * esz / 128, atoms_d = pd.len * esz / 128;
    const int grid = (int)gridDim.x;
    auto cut = [&](int run, int units) { return (int)((long long)run * units / grid); };
    int slot = 0, phase = 0;
    int part = 0, run = blockIdx.x;
    bool ok = true, mine = true;
    int ahead = 0;        // the claim of this CTA's own run of the next part: 0 if it got it
    auto next_stage = [&]() {
        if (++slot == a.stages) {
            slot = 0;
            phase ^= 1;
        }
    };
    auto wait_slot = [&]() {
        const bool free = mbar_wait_bounded(s.empty + slot, phase ^ 1, s.abort, a.status,
                                            SITE_GEMM_PRODUCER, a.wait_limit_ns);
        ok = __all_sync(0xffffffffu, free);
        return ok;
    };
    // a stage that carries no weights
    auto put_word = [&](int what, int tile) {
        if (!wait_slot()) return;
        if (lane == 0) {
            s.info[slot] = make_int4(what, part, tile, 0);
            mbar_arrive(s.full + slot);
        }
        if (FP8) copies_arrive(s.full + slot);
        next_stage();
    };
    while (part < kParts) {
        const int routed_units = part == 0 ? 0 : (*s.n_entries - S) * up_tiles;
        // units [first, last) of the run: shared and routed gate/up runs of one
        // number differ by at most one unit together
        int first, last;
        if (part == PART_SHARED_UP) {
            first = cut(run, shared_units);
            last = cut(run + 1, shared_units);
        } else if (part == PART_ROUTED_UP && routed_units >= grid) {
            const int all_units = shared_units + routed_units;
            first = cut(run, all_units) - cut(run, shared_units);
            last = cut(run + 1, all_units) - cut(run + 1, shared_units);
        } else {
            const int units = part == PART_ROUTED_UP ? routed_units
                              : part == PART_DOWN    ? *s.n_entries * down_tiles
                                                     : down_tiles;
            first = cut(run, units);
            last = cut(run + 1, units);
        }
        if (!mine) last = first;
        const bool is_up = part < PART_DOWN;
        const Pieces p = is_up ? pu : pd;
        const int K = is_up ? d : I;
        const int tiles = is_up ? up_tiles : down_tiles;
        for (int u = first; u < last && ok; ++u) {
            if (part == PART_Y) {
                put_word(WHAT_Y, u);
                continue;
            }
            const int entry = u / tiles + (part == PART_ROUTED_UP ? S : 0);
            const int tile = u % tiles;
            const int expert = entry < S ? -1 : s.list[entry];
            // the unit's first weight row (of the gate rows, or the down rows)
            const int row = is_up ? (expert < 0 ? entry * I : expert * 2 * I) + tile * 8
                                  : (expert < 0 ? 0 : expert * d) + tile * 16;
            const CUtensorMap* map = (is_up ? a.up_map : a.down_map) + (expert < 0 ? 0 : 1);
            const int atom0 = !is_up && expert < 0 ? entry * (I * esz / 128) : 0;
            const int atoms = is_up ? atoms_u : atoms_d;
            const float* sc = nullptr;  // 8-bit: this lane's row of scales
            if (FP8) {
                if (is_up) {
                    // lanes 0..15: the gate rows' scales, 16..31: the up rows'
                    const size_t F = expert < 0 ? SI : (size_t)I;
                    const size_t row0 = (expert < 0 ? (size_t)entry * I : (size_t)expert * 2 * I) +
                                        (size_t)tile * 8 + (lane >= 16 ? F : 0);
                    sc = (expert < 0 ? a.s_shared : a.s_gate_up) + row0 / 128 * (d / 128);
                } else {
                    const size_t ob = (size_t)tile * 16 / 128;
                    sc = expert < 0 ? a.s_shared + 2 * SI / 128 * (d / 128) + ob * (SI / 128) +
                                          (size_t)entry * I / 128
                                    : a.s_down + ((size_t)expert * (d / 128) + ob) * (I / 128);
                }
            }
            for (int c = 0; c < p.n; ++c) {
                if (!wait_slot()) break;
                const int k0 = c * p.len, len = min(p.len, K - k0);
                if (lane == 0) {
                    s.info[slot] = make_int4(is_up ? WHAT_UP : WHAT_DOWN, entry, tile, c);
                    mbar_arrive_expect_tx(s.full + slot, (uint32_t)(atoms * kAtomBytes));
                    uint8_t* dst = s.ring + slot * kStageBytes;
                    if (is_up)
                        box_4d(dst, map, s.full + slot, row, atom0 + c * atoms);
                    else
                        box_3d(dst, map, s.full + slot, row, atom0 + c * atoms);
                }
                __syncwarp();
                if (FP8) {
                    if ((lane & 15) < len / 128 && (is_up || lane < 16))
                        copy_scale(s.scales + slot * 32 + lane, sc + k0 / 128 + (lane & 15));
                    copies_arrive(s.full + slot);
                }
                next_stage();
            }
        }
        if (ok && part != PART_Y && mine) put_word(WHAT_TOLD, 0);
        if (!ok) break;
        // the sum warps have claimed this CTA's first runs by now
        if (part == 0) {
            const bool known = mbar_wait_bounded(s.claimed, 0, s.abort, a.status,
                                                 SITE_GEMM_PRODUCER, a.wait_limit_ns);
            ok = __all_sync(0xffffffffu, known);
            if (!ok) break;
            ahead = *s.ahead;
        }
        // a run of this part that no CTA has claimed?
        mine = false;
        int claims[kMaxGrid / 32];
#pragma unroll
        for (int i = 0; i < kMaxGrid / 32; ++i) {
            claims[i] = 1;
            if (32 * i + lane < grid)
                asm volatile("ld.relaxed.gpu.global.s32 %0, [%1];"
                             : "=r"(claims[i])
                             : "l"(a.ctrl + kCtrlClaim + kMaxGrid * part + 32 * i + lane)
                             : "memory");
        }
#pragma unroll
        for (int i = 0; i < kMaxGrid / 32; ++i) {
            for (uint32_t vote = __ballot_sync(0xffffffffu, claims[i] == 0); vote != 0 && !mine;
                 vote &= vote - 1) {
                run = 32 * i + __ffs(vote) - 1;
                int got = 0;
                if (lane == 0)
                    got = atomicExch(a.ctrl + kCtrlClaim + kMaxGrid * part + run, 1) == 0;
                mine = __shfl_sync(0xffffffffu, got, 0);
            }
        }
        if (mine) continue;
        // the next part, from this CTA's own run on
        ++part;
        run = blockIdx.x;
        if (part == PART_ROUTED_UP) {
            const bool there = mbar_wait_bounded(s.routed, 0, s.abort, a.status,
                                                 SITE_GEMM_PRODUCER, a.wait_limit_ns);
            ok = __all_sync(0xffffffffu, there);
            if (!ok) break;
        }
        mine = __shfl_sync(0xffffffffu, ahead, 0) == 0;
        if (lane == 0 && part + 1 < kParts)
            ahead = atomicExch(a.ctrl + kCtrlClaim + kMaxGrid * (part + 1) + run, 1);
    }
    if (ok) put_word(WHAT_END, 0);
    if (!ok) {
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

// ---------------------------------------------------------------- products
// Rows [T][K] of bf16 into operand B: the 8 tokens of a column group as the
// lanes (token, quarter) hold them.  An atom (128 bytes of a weight row: 64
// bf16, 128 e4m3) is 8 chunks of 16 bytes; lane quarter c takes chunks 2c and
// 2c + 1 as its part of two groups of products, the same for A and B, which
// permutes the reduction inside the atom and nothing else.  (With chunks c and
// c + 4 the two rows that a quarter warp reads would swizzle to the same banks.)
// Piece j (8 elements, 16 bytes of operand B) of the chunk of group g (atom
// g / 2) of token t is b[((g * PPQ + j) * NT + t / 8) * 32 + (t % 8) * 4 + c],
// PPQ = pieces per chunk (1 or 2).  A warp per token; 8-bit weights: as fp16
// times a power of two (1 / it goes to unscale).
template <int NT, bool FP8>
__device__ __forceinline__ void fill_b(const Smem& s, const __nv_bfloat16* src, size_t ld, int K,
                                       uint32_t mask, int n_tok, bool zero_rest, int warp,
                                       int lane) {
    constexpr int PPQ = FP8 ? 2 : 1;
    for (int t = warp; t < n_tok; t += kWarps) {
        const bool have = (mask >> t) & 1u;
        if (!have && !zero_rest) continue;
        const uint4* row = reinterpret_cast<const uint4*>(src + (size_t)t * ld);
        const int n = K / 8;
        // up to 2048 elements are read once, kPass pieces per lane
        constexpr int kPass = 8;
        uint4 v[kPass];
        auto read = [&](int p0) {
#pragma unroll
            for (int i = 0; i < kPass; ++i) {
                const int p = p0 + 32 * i + lane;
                v[i] = make_uint4(0, 0, 0, 0);
                if (have && p < n) v[i] = __ldcg(row + p);
            }
        };
        read(0);
        float scale = 1.f;
        if (FP8 && have) {
            uint32_t m = 0;
            for (int p0 = 0;;) {
#pragma unroll
                for (int i = 0; i < kPass; ++i) {
                    const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        m = max(m, max(w[q] & 0x7fffu, (w[q] >> 16) & 0x7fffu));
                }
                p0 += 32 * kPass;
                if (p0 >= n) break;
                read(p0);
            }
            if (n > 32 * kPass) read(0);
            // exponent field of the largest magnitude (bf16); infinities and
            // NaN, whose results are not numbers anyway, keep a scale of 1
            const int e = (int)(__reduce_max_sync(0xffffffffu, m) >> 7);
            const int up = e == 255 ? 0 : 14 - (max(e, 27) - 127);
            scale = __uint_as_float((uint32_t)(127 + up) << 23);
            if (lane == 0) s.unscale[t] = __uint_as_float((uint32_t)(127 - up) << 23);
        }
        for (int p0 = 0;;) {
#pragma unroll
            for (int i = 0; i < kPass; ++i) {
                const int p = p0 + 32 * i + lane;
                if (p >= n) continue;
                uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
                if (FP8) {
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const __half2 h =
                            __floats2half2_rn(__uint_as_float(w[q] << 16) * scale,
                                              __uint_as_float(w[q] & 0xffff0000u) * scale);
                        w[q] = *reinterpret_cast<const uint32_t*>(&h);
                    }
                }
                const int chunk = p / PPQ, j = p % PPQ;
                const int grp = (chunk >> 3) * 2 + (chunk & 1), c = (chunk >> 1) & 3;
                s.b[((grp * PPQ + j) * NT + (t >> 3)) * 32 + (t & 7) * 4 + c] =
                    make_uint4(w[0], w[1], w[2], w[3]);
            }
            p0 += 32 * kPass;
            if (p0 >= n) break;
            read(p0);
        }
    }
}

// This warp's part of one stage: the blocks of 128 whose number (counted over the
// whole reduction) is the warp's modulo 8, at most one of bf16 and two of 8-bit
// weights.  Operand A: 16 bytes of row lane / 4 and of row lane / 4 + 8 for each
// group of products (bf16: 4 of 32 elements, 8-bit: 2 of 64).
struct StageView {
    const uint8_t* r0;
    int pos[2];  // this lane's chunk of group 0 and 1 of an atom, swizzled
    __device__ __forceinline__ StageView(const uint8_t* st, int lane) {
        const int row = lane >> 2;
        r0 = st + row * 128;
        pos[0] = ((2 * (lane & 3)) ^ row) << 4;
        pos[1] = ((2 * (lane & 3) + 1) ^ row) << 4;
    }
    __device__ __forceinline__ void read(int atom, int g, uint4& lo, uint4& hi) const {
        const uint8_t* p = r0 + atom * kAtomBytes + pos[g];
        lo = *reinterpret_cast<const uint4*>(p);
        hi = *reinterpret_cast<const uint4*>(p + 8 * 128);
    }
};

// bf16: the stage is free as soon as the warp's block is in registers, before
// the products (16 tokens 188.7 -> 184.4 us, 1 token 45.2 -> 44.9).
struct Block16 {
    uint4 lo[4], hi[4];
};
__device__ __forceinline__ void read_16bit(const StageView& st, int j, Block16& o) {
#pragma unroll
    for (int g = 0; g < 4; ++g) st.read(2 * j + (g >> 1), g & 1, o.lo[g], o.hi[g]);
}
template <int NT>
__device__ __forceinline__ void multiply_16bit(const Block16& o, const uint4* b, int block,
                                               int lane, float (&acc)[NT][4]) {
#pragma unroll
    for (int g = 0; g < 4; ++g) {
        const uint4 lo = o.lo[g], hi = o.hi[g];
        const uint4* bp = b + (block * 4 + g) * NT * 32 + lane;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const uint4 v = bp[n * 32];
            mma16816(acc[n], lo.x, hi.x, lo.y, hi.y, v.x, v.y);
            mma16816(acc[n], lo.z, hi.z, lo.w, hi.w, v.z, v.w);
        }
    }
}

// 8-bit: one block after the other, straight from the stage (both first, or the
// stage freed first: 71.5 and 74.4 us at 5 tokens where this takes 71.7).
template <int NT>
__device__ __forceinline__ void block_8bit(const StageView& st, const uint4* b,
                                           const float* scales, int j, int block, bool up,
                                           int lane, float (&acc)[NT][4]) {
    float part[2][NT][4];  // two chains of products
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int q = 0; q < 4; ++q) part[0][n][q] = part[1][n][q] = 0.f;
#pragma unroll
    for (int g = 0; g < 2; ++g) {
        uint4 lo, hi;
        st.read(j, g, lo, hi);
        const uint32_t l4[4] = {lo.x, lo.y, lo.z, lo.w}, h4[4] = {hi.x, hi.y, hi.z, hi.w};
        const uint4* bp = b + (block * 2 + g) * 2 * NT * 32 + lane;
#pragma unroll
        for (int q = 0; q < 4; q += 2) {
            uint32_t a[8];
            widen(l4[q], a[0], a[2]);
            widen(h4[q], a[1], a[3]);
            widen(l4[q + 1], a[4], a[6]);
            widen(h4[q + 1], a[5], a[7]);
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const uint4 v = bp[((q >> 1) * NT + n) * 32];
                mma16816_f16(part[0][n], a[0], a[1], a[2], a[3], v.x, v.y);
                mma16816_f16(part[1][n], a[4], a[5], a[6], a[7], v.z, v.w);
            }
        }
    }
    const float s0 = scales[j], s1 = up ? scales[16 + j] : s0;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        acc[n][0] = fmaf(part[0][n][0] + part[1][n][0], s0, acc[n][0]);
        acc[n][1] = fmaf(part[0][n][1] + part[1][n][1], s0, acc[n][1]);
        acc[n][2] = fmaf(part[0][n][2] + part[1][n][2], s1, acc[n][2]);
        acc[n][3] = fmaf(part[0][n][3] + part[1][n][3], s1, acc[n][3]);
    }
}

// All product warps meet (bounded, unlike bar.sync: a warp that gave up does
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
__device__ __forceinline__ void products(const FewArgs& a, const Smem& s, int warp, int lane) {
    constexpr int esz = FP8 ? 1 : 2;
    const int tid = warp * 32 + lane;
    const int T = a.T, d = a.d, I = a.I, S = a.S;
    const uint32_t all = (1u << T) - 1u;
    // ---- x as operand B
    fill_b<NT, FP8>(s, a.x, d, d, all, 8 * NT, true, warp, lane);
    products_sync();

    // ---- units
    const Pieces pu = pieces(d, esz), pd = pieces(I, esz);
    float acc[NT][4];
    int slot = 0, phase = 0;
    int unit = 0;          // units so far
    int have = -1;         // entry whose h is operand B
    int parity = 0;
    float un[NT][2];       // 8-bit weights: unscale of this lane's two tokens per column group
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int q = 0; q < 2; ++q)
            un[n][q] = FP8 && 8 * n + 2 * (lane & 3) + q < T
                           ? s.unscale[8 * n + 2 * (lane & 3) + q] : 1.f;
    // the unit and this warp's partial sums, to the sum warp whose turn it is
    auto hand_over = [&](const int4& info, bool data) {
        const int buf = unit % kSumBufs, who = unit % kSumWarps;
        const bool ok = mbar_wait_bounded(s.sum_empty + buf, ((unit / kSumBufs) & 1) ^ 1, s.abort,
                                          a.status, SITE_GEMM_EPILOGUE, a.wait_limit_ns);
        if (!__all_sync(0xffffffffu, ok)) return false;
        if (data) {
            float4* red = s.red + buf * kWarps * NT * 32;
#pragma unroll
            for (int n = 0; n < NT; ++n)
                red[(warp * NT + n) * 32 + lane] =
                    make_float4(acc[n][0] * un[n][0], acc[n][1] * un[n][1], acc[n][2] * un[n][0],
                                acc[n][3] * un[n][1]);
        }
        if (tid == 0) s.unit[who] = info;
        __syncwarp();
        if (lane == 0) mbar_arrive(s.sum_full + who);
        ++unit;
        return true;
    };
    for (;;) {
        const bool filled = mbar_wait_bounded(s.full + slot, phase, s.abort, a.status,
                                              SITE_GEMM_MMA, a.wait_limit_ns);
        if (!__all_sync(0xffffffffu, filled)) return;
        const int4 info = s.info[slot];
        if (info.x == WHAT_END || info.x == WHAT_TOLD || info.x == WHAT_Y) {
            __syncwarp();
            if (lane == 0) mbar_arrive(s.empty + slot);
            if (++slot == a.stages) {
                slot = 0;
                phase ^= 1;
            }
            // y goes to one sum warp, the others concern them all
            for (int i = 0; i < (info.x == WHAT_Y ? 1 : kSumWarps); ++i)
                if (!hand_over(info, false)) return;
            if (info.x == WHAT_END) return;
            continue;
        }
        const bool up = info.x == WHAT_UP;
        const int entry = info.y, c = info.w;
        const Pieces p = up ? pu : pd;
        const int K = up ? d : I;
        if (!up && have != entry) {
            // the last products with the old operand are done, and h is there
            if (!warps_meet(a, s, lane, parity)) return;
            bool ok = mbar_wait_bounded(s.routed, 0, s.abort, a.status, SITE_GEMM_EPILOGUE,
                                        a.wait_limit_ns);  // the entry list: long there
            ok = ok && wait_count(a.ctrl + kCtrlH + entry, I / 8, s.abort, a.status,
                                  SITE_GEMM_BOUNDS, a.wait_limit_ns);
            if (!__all_sync(0xffffffffu, ok)) return;
            const uint32_t mask = entry < S ? all : s.s_mask[s.list[entry]];
            fill_b<NT, FP8>(s, a.h + (size_t)entry * T * I, I, I, mask, T, false, warp, lane);
            have = entry;
            if (!warps_meet(a, s, lane, parity)) return;
            if (FP8) {
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int q = 0; q < 2; ++q)
                        if (8 * n + 2 * (lane & 3) + q < T)
                            un[n][q] = s.unscale[8 * n + 2 * (lane & 3) + q];
            }
        }
        if (c == 0) {
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int q = 0; q < 4; ++q) acc[n][q] = 0.f;
        }
        const int k0 = c * p.len;
        const StageView st(s.ring + slot * kStageBytes, lane);
        const int first = k0 / 128, n_blocks = min(p.len, K - k0) / 128;
        const int j = (warp - first) & (kWarps - 1);
        Block16 o;
        if constexpr (FP8) {
            for (int i = j; i < n_blocks; i += kWarps)
                block_8bit<NT>(st, s.b, s.scales + slot * 32, i, first + i, up, lane, acc);
        } else {
            if (j < n_blocks) read_16bit(st, j, o);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(s.empty + slot);
        if (++slot == a.stages) {
            slot = 0;
            phase ^= 1;
        }
        if (!FP8 && j < n_blocks) multiply_16bit<NT>(o, s.b, first + j, lane, acc);
        if (c + 1 < p.n) continue;
        if (!hand_over(info, true)) return;
    }
}

// ---------------------------------------------------------------- sums
template <int NT>
__device__ __forceinline__ void sums(const FewArgs& a, const Smem& s, int who, int lane) {
    const int T = a.T, d = a.d, E = a.E, k = a.k, I = a.I, S = a.S;
    const uint32_t all = (1u << T) - 1u;
    // ---- routing: every CTA chooses for itself, CTA 0 writes it out
    const int tid = who * 32 + lane;
    for (int e = tid; e < E; e += 32 * kSumWarps) s.s_mask[e] = 0;
    pdl_wait();  // the control words are reset, the logits there
    if (tid == 0) {
        int* claim = a.ctrl + kCtrlClaim + blockIdx.x;
        *s.first_mine = atomicExch(claim, 1) == 0;
        *s.ahead = atomicExch(claim + kMaxGrid, 1);
        mbar_arrive(s.claimed);
    }
    sums_sync();
    for (int t = who; t < T; t += kSumWarps) {
        uint32_t* key = s.keys + who * E;
        int* idx = s.s_idx + t * k;
        float* w = s.s_w + t * k;
        const float* lg = a.logits + (size_t)t * E;
        if (E <= 64)
            choose<2>(lg, key, lane, E, k, a.G, a.TG, a.gate, a.bias, idx, w);
        else
            choose<kMaxE / 32>(lg, key, lane, E, k, a.G, a.TG, a.gate, a.bias, idx, w);
        __syncwarp();
        if (lane < k) {
            atomicOr(s.s_mask + s.s_idx[t * k + lane], 1u << t);
            if (blockIdx.x == 0) {
                if (a.idx_out != nullptr) a.idx_out[t * k + lane] = s.s_idx[t * k + lane];
                if (a.w_out != nullptr) a.w_out[t * k + lane] = s.s_w[t * k + lane];
            }
        }
    }
    sums_sync();
    if (who == 0) {
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
    sums_sync();

    // ---- units
    bool first_lost = false;
    int told_entry = 0, untold = 0;  // gate/up units stored and not told yet
    bool checked = false;
    auto tell = [&]() {
        __syncwarp();
        if (!checked) {
            // the first run's units count if the run is this CTA's
            checked = true;
            const bool known = mbar_wait_bounded(s.claimed, 0, s.abort, a.status,
                                                 SITE_GEMM_EPILOGUE, a.wait_limit_ns);
            if (!known || !*s.first_mine) first_lost = true;
        }
        if (lane == 0 && untold > 0 && !first_lost) {
            __threadfence();
            atomicAdd(a.ctrl + kCtrlH + told_entry, untold);
        }
        untold = 0;
    };
    for (int unit = who;; unit += kSumWarps) {
        const bool filled = mbar_wait_bounded(s.sum_full + who, (unit / kSumWarps) & 1, s.abort,
                                              a.status, SITE_GEMM_EPILOGUE, a.wait_limit_ns);
        if (!__all_sync(0xffffffffu, filled)) return;
        const int4 info = s.unit[who];
        const int buf = unit % kSumBufs;
        const float4* red = s.red + buf * kWarps * NT * 32 + lane;
        float4 sum[NT];
        if (info.x == WHAT_UP || info.x == WHAT_DOWN) {
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                float4 v = red[n * 32];
#pragma unroll
                for (int w = 1; w < kWarps; ++w) {
                    const float4 o = red[(w * NT + n) * 32];
                    v.x += o.x;
                    v.y += o.y;
                    v.z += o.z;
                    v.w += o.w;
                }
                sum[n] = v;
            }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(s.sum_empty + buf);
        if (info.x == WHAT_END) return;
        if (info.x == WHAT_TOLD) {
            tell();
            first_lost = false;  // the first run is over
            if (info.y == PART_DOWN && lane == 0) {
                __threadfence();
                atomicAdd(a.ctrl + kCtrlDown, 1);
            }
            continue;
        }
        const int entry = info.y, tile = info.z;
        if (info.x == WHAT_Y) {
            // ---- 16 columns of y: the slots of each token in order, once every
            // sum warp of every down run has told
            const bool ok = wait_count(a.ctrl + kCtrlDown, kSumWarps * (int)gridDim.x, s.abort,
                                       a.status, SITE_GEMM_BOUNDS, a.wait_limit_ns);
            if (!__all_sync(0xffffffffu, ok)) return;
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
                    *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.y) + (size_t)t * d +
                                              col) =
                        make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
            }
            continue;
        }
        const bool up = info.x == WHAT_UP;
        const int expert = entry < S ? -1 : s.list[entry];
        const uint32_t mask = expert < 0 ? all : s.s_mask[expert];
        if (up) {
            if (entry != told_entry) tell();
            told_entry = entry;
            ++untold;
        }
        const int g = lane >> 2;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                const int t = 8 * n + 2 * (lane & 3) + q;
                if (!((mask >> t) & 1u)) continue;
                // rows g and g + 8 of the unit
                const float s0 = q ? sum[n].y : sum[n].x, s1 = q ? sum[n].w : sum[n].z;
                if (up) {
                    const float h = s0 / (1.f + expf(-s0)) * s1;
                    a.h[((size_t)entry * T + t) * I + tile * 8 + g] = __float2bfloat16_rn(h);
                } else {
                    int j = entry;
                    float wt = 1.f;
                    if (expert >= 0)
                        for (int i = 0; i < k; ++i)
                            if (s.s_idx[t * k + i] == expert) {
                                j = S + i;
                                wt = s.s_w[t * k + i];
                            }
                    float* o = a.slots + ((size_t)t * (S + k) + j) * d + tile * 16 + g;
                    __stcg(o, wt * s0);
                    __stcg(o + 8, wt * s1);
                }
            }
        }
    }
}

template <int NT, bool FP8>
__global__ void __launch_bounds__(kFewThreads, 1) few_layer_kernel(const __grid_constant__ FewArgs a) {
    extern __shared__ uint8_t few_smem[];
    // swizzled stages start at multiples of 1024 bytes
    uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(few_smem) + 1023) &
                                               ~(uintptr_t)1023);
    const Smem s = carve<NT>(base, a.stages, a.d, a.I);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int i = 0; i < a.stages; ++i) {
            mbar_init(s.full + i, FP8 ? 33 : 1);  // the copies' bytes; 8-bit: + 32 lanes' scales
            mbar_init(s.empty + i, kWarps);
        }
        mbar_init(s.routed, 1);
        mbar_init(s.claimed, 1);
        mbar_init(s.meet, kWarps);
        for (int i = 0; i < kSumWarps; ++i) mbar_init(s.sum_full + i, kWarps);
        for (int i = 0; i < kSumBufs; ++i) mbar_init(s.sum_empty + i, 1);
        *s.abort = 0;
        fence_barrier_init();
    }
    __syncthreads();
    pdl_trigger();  // the next kernel waits for this one's end by itself
    if (warp < kWarps)
        products<NT, FP8>(a, s, warp, lane);
    else if (warp < kWarps + kSumWarps)
        sums<NT>(a, s, warp - kWarps, lane);
    else
        producer<FP8>(a, s, lane);
}

// ---------------------------------------------------------------- host
enum FewRegion : int { FW_STATUS, FW_CTRL, FW_LOGITS, FW_H, FW_SLOTS, FW_TOTAL };

// stages of the ring (0: operand B leaves too little room for one)
int few_stages(int T, int d, int I) {
    const int nt = T > 8 ? 2 : 1;
    const long long fixed = (long long)8 * nt * 2 * (d > I ? d : I) +
                            nt * red_bytes<1>() + kSmallBytes;
    const long long ring = kSmemMax - fixed;
    if (ring < kMinRing) return 0;
    return (int)std::min<long long>(ring / kStageBytes, kMaxStages);
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
    const size_t sizes[FW_TOTAL] = {sizeof(int) * kStatusWords, sizeof(int) * kCtrlWords,
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
    return launch_pdl(kern, dim3((unsigned)std::min(num_sms(), kMaxGrid)), dim3(kFewThreads), (size_t)smem, s, 1, a);
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
    const int esz = fp8 ? 1 : 2;
    const Pieces pu = pieces(d, esz), pd = pieces(inter, esz);
    const uint64_t SI = (uint64_t)n_shared * inter;
    const uint32_t au = (uint32_t)(pu.len * esz / 128), ad = (uint32_t)(pd.len * esz / 128);
    const char* sh = static_cast<const char*>(W_shared);
    if (!make_map_atoms16(&a.up_map[1], W_gate_up, (uint64_t)E * 2 * inter, (uint64_t)d * esz,
                          inter, au) ||
        !make_map_atoms16(&a.down_map[1], W_down, (uint64_t)E * d, (uint64_t)inter * esz, 0, ad) ||
        (n_shared > 0 &&
         (!make_map_atoms16(&a.up_map[0], sh, 2 * SI, (uint64_t)d * esz, SI, au) ||
          !make_map_atoms16(&a.down_map[0], sh + 2 * SI * d * esz, (uint64_t)d, SI * esz, 0, ad))))
        return MOE_ERR_CUDA;
    a.x = static_cast<const __nv_bfloat16*>(x);
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
    a.y = y;
    a.idx_out = topk_idx_out;
    a.w_out = topk_w_out;
    a.status = reinterpret_cast<int*>(ws + off[FW_STATUS]);
    a.ctrl = reinterpret_cast<int*>(ws + off[FW_CTRL]);
    a.h = reinterpret_cast<__nv_bfloat16*>(ws + off[FW_H]);
    a.slots = reinterpret_cast<float*>(ws + off[FW_SLOTS]);
    a.wait_limit_ns = kWaitLimitNs;
    // the layer kernel needs all of an SM's shared memory: an SM that runs the
    // logits kernel with another split could not take it before that ends
    cudaError_t e = cudaFuncSetAttribute(few_logits_kernel,
                                         cudaFuncAttributePreferredSharedMemoryCarveout,
                                         cudaSharedmemCarveoutMaxShared);
    if (e != cudaSuccess) return MOE_ERR_CUDA;
    e = launch_pdl(few_logits_kernel, dim3((unsigned)E), dim3(kLogitThreads), 0, s, 1,
                               a.x, static_cast<const __nv_bfloat16*>(W_router), T, d, E,
                               reinterpret_cast<float*>(ws + off[FW_LOGITS]), a.status, a.ctrl,
                               kCtrlWords);
    if (e != cudaSuccess) return MOE_ERR_CUDA;
    if (fp8) return ret(T > 8 ? launch_layer<2, true>(a, s) : launch_layer<1, true>(a, s));
    return ret(T > 8 ? launch_layer<2, false>(a, s) : launch_layer<1, false>(a, s));
}

}  // extern "C"
