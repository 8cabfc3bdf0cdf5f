// 8-bit product of rows and weights by groups of rows (experts):
//
//   y[r, n] = sum_j sa[j, r] sb[g, n / 128, j] P_j[r, n],
//   P_j[r, n] = sum_{k in block j} a[r, k] b[g, n, k]      (e4m3 operands)
//
// P_j is a tcgen05 product (kind::f8f6f4, fp32 accumulator in TMEM) of one
// 128-deep block.  The scales are arbitrary fp32 numbers, so they cannot ride
// in the tensor core's own block scaling: the epilogue warps take P_j out of
// TMEM and add it, scaled, to fp32 sums in registers, block by block, while
// the tensor core makes the next block in the other half of TMEM.  The rows
// are the M side of the product: a thread owns one row of the tile, so its
// scale is one register, and b's scale is one number for 128 columns.
//
// CTA (one per SM, persistent): 128 rows x BN columns.  Warp 0 loads the
// operands by TMA (128-byte swizzle) into a ring of stages, warp 1 issues the
// products, warp 2 decodes tiles ahead of them (a search and two divisions, 1 us
// per tile in the adding warps), warps 4..11 add (two warps per SM
// sub-partition: TMEM lanes 32 (w % 4).., columns half (w - 4) / 4).  128 sums a
// thread need more registers than an even split leaves: warps 0..3 hand some of
// theirs over (of the launch's 384 x 168, 128 x 120 + 256 x 192; with 128 x 56 the
// issuing warps spilled and the kernel took a quarter longer).  At 256 columns 24
// bytes a thread still spill (48 bytes of stores, 176 of loads in the code), at
// the other widths none.
//
// Many rows (24576 rows in 64 uneven groups, n 2048, k 1536: 128 us, 1.2
// PFLOP/s, in bursts of up to 40 ms; in a longer loop, under the power cap at
// 1.57 GHz, 155 us): the time goes with what the tiles read from L2, 1.05 GB a
// launch, 8 TB/s, where the bf16 CTA-pair GEMM reads 9.7.  A pair of CTAs on one 256-row tile
// reads two thirds of that, but its accumulators are released across the two
// SMs, and with the two that TMEM holds it waited for that: 139 us.  Few
// rows (384 rows in 64 groups: 41 us): the weights, at 6.4 TB/s once the first
// tile has arrived; 4 tiles for some CTAs and 3 for others.
#include <cudaTypedefs.h>
#include <limits.h>

#include <algorithm>

#include "moe_device.cuh"
#include "moe_internal.h"

namespace moe {
namespace {

constexpr int kM8 = 128;          // rows of a tile
constexpr int kK8 = 128;          // depth of a block
constexpr int kEpiWarps8 = 8;
constexpr int kThreads8 = 32 * (4 + kEpiWarps8);
constexpr int kABytes8 = kM8 * kK8;
constexpr uint64_t kDrainNs8 = 1000000;
constexpr int kTileRing = 4;

struct Fp8Args {
    const float* sa;        // [kb][R]
    const float* sb;        // [G][nb][kb]
    const int32_t* counts;  // nullptr: one group of R rows
    int R, G, n, k;
    int out_f32;
    int split;      // CTAs per tile (split launches)
    int wide_rows;  // rows of y are 32-byte aligned
    void* y;
    int* status;
    unsigned long long wait_limit_ns;
};
// Rows of a are loaded in boxes of 32, 64 or 128: a tile of a few rows (an
// expert's at decode) does not bring its neighbours' rows along.  What the stage
// holds behind them is multiplied too, into sums that nobody reads.
constexpr int kRowBoxes = 3;
struct Fp8Maps {
    CUtensorMap a[kRowBoxes], b;
};

template <int BN>
struct Shape8 {
    static constexpr int kStageBytes = kABytes8 + BN * kK8;
    static constexpr int kStages = BN == 256 ? 4 : BN == 128 ? 6 : 8;
    static constexpr int kTmemCols = 2 * BN;
};

template <int STAGES>
struct __align__(16) Tail8 {
    uint4 out[kEpiWarps8][128];  // per adding warp: 32 rows x 64 bytes on their way out
    uint64_t full[STAGES];
    uint64_t empty[STAGES];
    uint64_t tfull[2];
    uint64_t tempty[2];
    uint64_t drain;
    uint64_t tile_full[kTileRing];   // a decoded tile is there
    uint64_t tile_empty[kTileRing];  // the loading lane and the adding warps have it
    int4 tile[kTileRing];
    uint32_t tmem_base;
    int abort;
    int row_off[kMaxE + 1];   // first row of each group
    int tile_off[kMaxE + 1];  // first row tile of each group
};

template <int BN>
constexpr size_t smem_bytes8() {
    return 1024 + (size_t)Shape8<BN>::kStages * Shape8<BN>::kStageBytes +
           sizeof(Tail8<Shape8<BN>::kStages>);
}

__device__ __forceinline__ void tma_load_2d(void* dst, const CUtensorMap* map, uint64_t* bar,
                                            int c0, int c1) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4}], [%2];" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(c0), "r"(c1)
        : "memory");
}
__device__ __forceinline__ void tma_load_3d(void* dst, const CUtensorMap* map, uint64_t* bar,
                                            int c0, int c1, int c2) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(c0), "r"(c1), "r"(c2)
        : "memory");
}
// the four 32-deep products of one block; the first starts the accumulator anew
__device__ __forceinline__ void mma_block8(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.b32 p, %3, %3;\n\t"
        "setp.eq.b32 q, %3, %3;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %4, %5, %3, q;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %6, %7, %3, q;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %8, %9, %3, q;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "l"(a + 2), "l"(b + 2), "l"(a + 4), "l"(b + 4), "l"(a + 6),
        "l"(b + 6)
        : "memory");
}
__device__ __forceinline__ void commit8(uint64_t* bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
                     smem_u32(bar))
                 : "memory");
}
__device__ __forceinline__ uint64_t fma_pair(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t pair2(float a, float b) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float2 unpair(uint64_t v) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
    return r;
}

// Instruction descriptor for kind::f8f6f4: fp32 accumulator (D format 1 in
// [4,6)), A and B e4m3 (0 in [7,10) and [10,13)), both K-major, N >> 3 in
// [17,23), M >> 4 in [24,29).
constexpr uint32_t idesc_e4m3_f32(int M, int N) {
    return (1u << 4) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

// One tile of the launch.
struct Tile8 {
    int g, row0, rows, nt;
};
// The nth tile of this CTA, as warp 2 decoded it.
template <class TAIL>
__device__ __forceinline__ bool take_tile(TAIL* tail, int nth, Tile8& t, volatile int* abort,
                                          int* status, int site, uint64_t limit) {
    const int slot = nth % kTileRing;
    if (!mbar_wait_bounded(&tail->tile_full[slot], (nth / kTileRing) & 1, abort, status, site,
                           limit))
        return false;
    const int4 v = tail->tile[slot];
    t = Tile8{v.x, v.y, v.z, v.w};
    return true;
}
template <class TAIL>
__device__ __forceinline__ Tile8 decode8(const TAIL* t, int G, int n_tiles, int tile) {
    // row tiles of a group are neighbours: a weight tile is read from memory once
    int lo = 0, hi = G - 1;
    while (lo < hi) {  // the last group that starts at or before this tile
        const int mid = (lo + hi + 1) >> 1;
        if ((long long)t->tile_off[mid] * n_tiles <= tile)
            lo = mid;
        else
            hi = mid - 1;
    }
    const int m_tiles = t->tile_off[lo + 1] - t->tile_off[lo];
    const int local = tile - t->tile_off[lo] * n_tiles;
    const int mt = local % m_tiles;
    Tile8 r;
    r.g = lo;
    r.nt = local / m_tiles;
    r.row0 = t->row_off[lo] + mt * kM8;
    r.rows = min(kM8, t->row_off[lo + 1] - r.row0);
    return r;
}

// Four columns of a row.
__device__ __forceinline__ void store4(const Fp8Args& a, size_t row, int col, const float4& v) {
    const size_t at = row * (size_t)a.n + col;
    const float f[4] = {v.x, v.y, v.z, v.w};
    if (a.n % 4 == 0) {
        if (col >= a.n) return;
        if (a.out_f32)
            *reinterpret_cast<float4*>(static_cast<float*>(a.y) + at) = v;
        else
            *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.y) + at) =
                make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
        return;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (col + i >= a.n) return;
        if (a.out_f32)
            static_cast<float*>(a.y)[at + i] = f[i];
        else
            static_cast<__nv_bfloat16*>(a.y)[at + i] = __float2bfloat16_rn(f[i]);
    }
}

// Columns col .. col + 2 W - 1 of the warp's 32 rows (lane = row; `rows` of them
// exist) from sums in registers.  A lane's 64 bytes at a time go through the
// warp's staging rows (16-byte chunk q of row r at q ^ (r / 2 % 4): both sides
// without bank conflicts), so that each store instruction writes 8 whole
// 64-byte row pieces; straight from the lanes, 16 bytes of 32 rows, the stores
// of a tile took about 4 us.  Rows of y that are not 16-byte aligned are
// written from the lanes.
template <int W>
__device__ __forceinline__ void store_rows(const Fp8Args& a, uint4* stage, size_t row0, int rows,
                                           int col, int lane, const uint64_t (&acc)[W]) {
    const int per16 = a.out_f32 ? 4 : 8;  // columns in 16 bytes
    if (a.n % per16 != 0) {
        if (lane >= rows) return;
        const size_t base = (row0 + lane) * (size_t)a.n + col;
#pragma unroll
        for (int i = 0; i < W; ++i) {
            const float2 u = unpair(acc[i]);
            if (a.out_f32) {
                float* y = static_cast<float*>(a.y) + base;
                if (col + 2 * i < a.n) y[2 * i] = u.x;
                if (col + 2 * i + 1 < a.n) y[2 * i + 1] = u.y;
            } else {
                __nv_bfloat16* y = static_cast<__nv_bfloat16*>(a.y) + base;
                if (col + 2 * i < a.n) y[2 * i] = __float2bfloat16_rn(u.x);
                if (col + 2 * i + 1 < a.n) y[2 * i + 1] = __float2bfloat16_rn(u.y);
            }
        }
        return;
    }
    if (!a.out_f32 && a.wide_rows) {
        // 32 bytes per lane and instruction: whole sectors
        if (lane >= rows) return;
        __nv_bfloat16* y = static_cast<__nv_bfloat16*>(a.y) + (row0 + lane) * (size_t)a.n + col;
#pragma unroll
        for (int i = 0; i < W; i += 8) {
            if (col + 2 * i >= a.n) return;
            uint32_t w[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const float2 u = unpair(acc[i + k]);
                w[k] = pack_bf16x2(u.x, u.y);
            }
            asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(y + 2 * i),
                         "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]),
                         "r"(w[6]), "r"(w[7])
                         : "memory");
        }
        return;
    }
    const int sw = (lane >> 1) & 3;
    const int q = lane & 3;  // chunk of the row pieces this lane stores
    // 64 bytes: 8 pairs of fp32, 16 pairs of bf16
    auto flush = [&](int first_col) {
        __syncwarp();
#pragma unroll
        for (int it = 0; it < 4; ++it) {
            const int r = it * 8 + (lane >> 2);
            const int c = first_col + q * per16;
            const uint4 v = stage[r * 4 + (q ^ ((r >> 1) & 3))];
            if (r < rows && c < a.n) {
                const size_t at = (row0 + r) * (size_t)a.n + c;
                if (a.out_f32)
                    *reinterpret_cast<uint4*>(static_cast<float*>(a.y) + at) = v;
                else
                    *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.y) + at) = v;
            }
        }
        __syncwarp();
    };
    if (a.out_f32) {
#pragma unroll
        for (int i = 0; i < W; i += 8) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float2 u = unpair(acc[i + 2 * j]), v = unpair(acc[i + 2 * j + 1]);
                stage[lane * 4 + (j ^ sw)] =
                    make_uint4(__float_as_uint(u.x), __float_as_uint(u.y), __float_as_uint(v.x),
                               __float_as_uint(v.y));
            }
            flush(col + 2 * i);
        }
    } else {
#pragma unroll
        for (int i = 0; i < W; i += 16) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                uint32_t w[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const float2 u = unpair(acc[i + 4 * j + k]);
                    w[k] = pack_bf16x2(u.x, u.y);
                }
                stage[lane * 4 + (j ^ sw)] = make_uint4(w[0], w[1], w[2], w[3]);
            }
            flush(col + 2 * i);
        }
    }
}

// Split launches (few row tiles and a long reduction): a cluster of S CTAs takes
// one tile, each a part of the blocks, and they add their fp32 sums over
// distributed shared memory, in rank order.
constexpr int kMaxSplit = 8;
__device__ __forceinline__ void cluster_meet() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;"
                 ::: "memory");
}
__device__ __forceinline__ float4 ld_rank(uint32_t addr, uint32_t rank) {
    float4 v;
    asm volatile(
        "{\n\t.reg .u32 p;\n\tmapa.shared::cluster.u32 p, %4, %5;\n\t"
        "ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [p];\n\t}"
        : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
        : "r"(addr), "r"(rank)
        : "memory");
    return v;
}

template <int BN, bool SPLIT>
__global__ void __launch_bounds__(kThreads8, 1) fp8_gemm_kernel(
    const __grid_constant__ Fp8Maps maps, const __grid_constant__ Fp8Args a) {
    using SH = Shape8<BN>;
    constexpr int kStages = SH::kStages;
    constexpr int kPartRow = BN / 4 + 1;  // float4 per row of sums: no bank conflicts
    extern __shared__ uint8_t raw8[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw8) + 1023) &
                                               ~(uintptr_t)1023);
    auto* tail = reinterpret_cast<Tail8<kStages>*>(smem + (size_t)kStages * SH::kStageBytes);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    volatile int* abort_flag = &tail->abort;
    int* status = a.status;
    const uint64_t limit = a.wait_limit_ns;

    if (threadIdx.x == 0) {
        for (int i = 0; i < kStages; ++i) {
            mbar_init(&tail->full[i], 1);
            mbar_init(&tail->empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&tail->tfull[i], 1);
            mbar_init(&tail->tempty[i], kEpiWarps8);
        }
        mbar_init(&tail->drain, 1);
        for (int i = 0; i < kTileRing; ++i) {
            mbar_init(&tail->tile_full[i], 1);
            mbar_init(&tail->tile_empty[i], 1 + kEpiWarps8);
        }
        tail->abort = 0;
        fence_barrier_init();
    }
    pdl_wait();
    pdl_trigger();  // the next kernel waits for this one's end by itself
    if (warp == 0) {
        // rows and row tiles of each group (exclusive prefix sums), cut at R rows
        int rows = 0, tiles = 0;
        for (int g0 = 0; g0 < a.G; g0 += 32) {
            const int g = g0 + lane;
            // summed as given (64 bits hold 256 of them): a single count beyond R is
            // seen too; the offsets are cut at R below
            const int c = g < a.G ? (a.counts != nullptr ? max(a.counts[g], 0) : a.R) : 0;
            long long ir = c;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const long long v = __shfl_up_sync(0xffffffffu, ir, o);
                if (lane >= o) ir += v;
            }
            const long long all = __shfl_sync(0xffffffffu, ir, 31);
            const int first = (int)min((long long)rows + ir - c, (long long)a.R);
            const int last = (int)min((long long)rows + ir, (long long)a.R);
            const int tl = (last - first + kM8 - 1) / kM8;
            int it = tl;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int v = __shfl_up_sync(0xffffffffu, it, o);
                if (lane >= o) it += v;
            }
            if (g < a.G) {
                tail->row_off[g] = first;
                tail->tile_off[g] = tiles + it - tl;
            }
            if (blockIdx.x == 0 && lane == 0 && (long long)rows + all > a.R)
                set_status(status, MOE_ERR_DEVICE, SITE_GEMM_BOUNDS, a.R);
            rows = (int)min((long long)rows + all, (long long)a.R);
            tiles += __shfl_sync(0xffffffffu, it, 31);
        }
        if (lane == 0) {
            tail->row_off[a.G] = rows;
            tail->tile_off[a.G] = tiles;
        }
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                         smem_u32(&tail->tmem_base)),
                     "n"(SH::kTmemCols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tail->tmem_base;
    const int n_tiles = (a.n + BN - 1) / BN;
    const int total = tail->tile_off[a.G] * n_tiles;
    const int kb_n = (a.k + kK8 - 1) / kK8;
    // tiles first_tile, first_tile + step, .. of this CTA, blocks [kb0, kb1) of each
    const int S = SPLIT ? a.split : 1;
    const int rank = SPLIT ? (int)blockIdx.x % S : 0;
    const int first_tile = SPLIT ? (int)blockIdx.x / S : (int)blockIdx.x;
    const int step = SPLIT ? 1 << 30 : (int)gridDim.x;  // split: one tile
    const int kb0 = rank * kb_n / S, kb1 = (rank + 1) * kb_n / S;

    if (warp < 4) {
      asm volatile("setmaxnreg.dec.sync.aligned.u32 120;");
      if (warp == 0) {
        // ------------------------------------------------ loads
        if (lane == 0) {
            int s = 0;
            uint32_t ph = 0, issued = 0, issued_ph = 0;
            bool ok = true;
            int nth = 0;
            for (int tile = first_tile; tile < total && ok; tile += step, ++nth) {
                Tile8 t;
                ok = take_tile(tail, nth, t, abort_flag, status, SITE_GEMM_PRODUCER, limit);
                if (!ok) break;
                mbar_arrive(&tail->tile_empty[nth % kTileRing]);
                const int box = t.rows <= 32 ? 0 : t.rows <= 64 ? 1 : 2;
                const uint32_t bytes = (uint32_t)((32 << box) * kK8 + BN * kK8);
                for (int kb = kb0; kb < kb1; ++kb) {
                    ok = mbar_wait_bounded(&tail->empty[s], ph ^ 1u, abort_flag, status,
                                           SITE_GEMM_PRODUCER, limit);
                    if (!ok) break;
                    uint8_t* st = smem + (size_t)s * SH::kStageBytes;
                    mbar_arrive_expect_tx(&tail->full[s], bytes);
                    tma_load_2d(st, &maps.a[box], &tail->full[s], kb * kK8, t.row0);
                    tma_load_3d(st + kABytes8, &maps.b, &tail->full[s], kb * kK8, t.nt * BN, t.g);
                    issued |= 1u << s;
                    issued_ph = (issued_ph & ~(1u << s)) | (ph << s);
                    if (++s == kStages) {
                        s = 0;
                        ph ^= 1u;
                    }
                }
            }
            if (!ok)  // no copy of this CTA may land after it has gone
                for (int i = 0; i < kStages; ++i)
                    if (issued & (1u << i))
                        mbar_wait_bounded(&tail->full[i], (issued_ph >> i) & 1u, nullptr, status,
                                          SITE_GEMM_DRAIN, kDrainNs8);
        }
      } else if (warp == 1) {
        // ------------------------------------------------ products
        if (lane == 0) {
            int s = 0, blk = 0;
            uint32_t ph = 0;
            bool ok = true;
            const uint64_t ad0 = sw128_kmajor_desc(smem_u32(smem));
            const uint64_t bd0 = sw128_kmajor_desc(smem_u32(smem) + kABytes8);
            constexpr uint32_t idesc = idesc_e4m3_f32(kM8, BN);
            for (int tile = first_tile; tile < total && ok; tile += step) {
                for (int kb = kb0; kb < kb1; ++kb, ++blk) {
                    const int buf = blk & 1;
                    ok = mbar_wait_bounded(&tail->tempty[buf], ((blk >> 1) & 1) ^ 1u, abort_flag,
                                           status, SITE_GEMM_MMA, limit) &&
                         mbar_wait_bounded(&tail->full[s], ph, abort_flag, status, SITE_GEMM_MMA,
                                           limit);
                    if (!ok) break;
                    tc_fence_after();
                    const uint64_t off = (uint64_t)s * (SH::kStageBytes >> 4);
                    mma_block8(tmem + (uint32_t)(buf * BN), ad0 + off, bd0 + off, idesc);
                    commit8(&tail->empty[s]);
                    commit8(&tail->tfull[buf]);
                    if (++s == kStages) {
                        s = 0;
                        ph ^= 1u;
                    }
                }
            }
            if (!ok) *abort_flag = 1;
            commit8(&tail->drain);
            mbar_wait_bounded(&tail->drain, 0u, nullptr, status, SITE_GEMM_DRAIN, limit);
        }
      } else if (warp == 2) {
        // ------------------------------------------------ tiles, decoded
        if (lane == 0) {
            int nth = 0;
            for (int tile = first_tile; tile < total; tile += step, ++nth) {
                const Tile8 t = decode8(tail, a.G, n_tiles, tile);
                const int slot = nth % kTileRing;
                if (!mbar_wait_bounded(&tail->tile_empty[slot], ((nth / kTileRing) & 1) ^ 1u,
                                       abort_flag, status, SITE_GEMM_PRODUCER, limit))
                    break;
                tail->tile[slot] = make_int4(t.g, t.row0, t.rows, t.nt);
                mbar_arrive(&tail->tile_full[slot]);
            }
        }
      }
    } else {
        // ------------------------------------------------ sums
        asm volatile("setmaxnreg.inc.sync.aligned.u32 192;");
        constexpr int kCols = BN / 2;  // columns of this warp
        const int wq = warp & 3, half = (warp - 4) >> 2;
        const int nb = (a.n + 127) / 128;
        const int r = wq * 32 + lane;
        uint4* stage = tail->out[warp - 4];
        int blk = 0;
        bool ok = true;
        // a tile's scales: of this lane's row and of the columns' block (columns
        // behind n belong to no block of b: any scale will do)
        Tile8 t{};
        const float *sa = nullptr, *sb = nullptr;
        float sa_next = 0.f, sb_next = 0.f;
        bool live = false;
        auto open = [&](int nth) {
            const bool there =
                take_tile(tail, nth, t, abort_flag, status, SITE_GEMM_EPILOGUE, limit);
            ok = __all_sync(0xffffffffu, there);
            if (!ok) return;
            if (lane == 0) mbar_arrive(&tail->tile_empty[nth % kTileRing]);
            live = r < t.rows;
            sa = a.sa + t.row0 + r;
            sb = a.sb +
                 ((size_t)t.g * nb + min((t.nt * BN + half * kCols) / 128, nb - 1)) * kb_n;
            sa_next = live ? __ldg(sa + (size_t)kb0 * a.R) : 0.f;
            sb_next = __ldg(sb + kb0);
        };
        int nth = 0;
        if (first_tile < total) open(nth);
        for (int tile = first_tile; tile < total && ok; tile += step) {
            uint64_t acc[kCols / 2];
#pragma unroll
            for (int i = 0; i < kCols / 2; ++i) acc[i] = 0;
            for (int kb = kb0; kb < kb1; ++kb, ++blk) {
                const float sc = sa_next * sb_next;
                const uint64_t s2 = pair2(sc, sc);
                if (kb + 1 < kb1) {
                    sa_next = live ? __ldg(sa + (size_t)(kb + 1) * a.R) : 0.f;
                    sb_next = __ldg(sb + kb + 1);
                }
                const int buf = blk & 1;
                ok = mbar_wait_bounded(&tail->tfull[buf], (blk >> 1) & 1, abort_flag, status,
                                       SITE_GEMM_EPILOGUE, limit);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                tc_fence_after();
                const uint32_t ta = tmem + (uint32_t)(buf * BN + half * kCols) +
                                    ((uint32_t)(wq * 32) << 16);
                if (wq * 32 < t.rows) {  // else none of the warp's rows exist
                    // the next 32 columns are on their way while these are added
                    uint32_t v[2][32];
                    tmem_ld32(ta, v[0]);
#pragma unroll
                    for (int c = 0; c < kCols / 32; ++c) {
                        tmem_ld_wait();
                        if (c + 1 < kCols / 32) tmem_ld32(ta + 32 * (c + 1), v[(c + 1) & 1]);
#pragma unroll
                        for (int i = 0; i < 16; ++i)
                            acc[16 * c + i] = fma_pair(pair2(__uint_as_float(v[c & 1][2 * i]),
                                                             __uint_as_float(v[c & 1][2 * i + 1])),
                                                       s2, acc[16 * c + i]);
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&tail->tempty[buf]);
            }
            if (!ok) break;
            if (SPLIT) {
                // all of this CTA's products are done: the ring is free for its sums
                float4* part = reinterpret_cast<float4*>(smem) + r * kPartRow + half * (kCols / 4);
                if (live) {
#pragma unroll
                    for (int i = 0; i < kCols / 4; ++i) {
                        const float2 u = unpair(acc[2 * i]), v = unpair(acc[2 * i + 1]);
                        part[i] = make_float4(u.x, u.y, v.x, v.y);
                    }
                }
                break;
            }
            // the next tile's scales are on their way while this one is stored
            const size_t row0 = (size_t)t.row0 + wq * 32;
            const int rows = t.rows - wq * 32, col0 = t.nt * BN + half * kCols;
            if (tile + step < total) open(++nth);
            store_rows(a, stage, row0, rows, col0, lane, acc);
        }
    }
    if (SPLIT) {
        __syncthreads();
        cluster_meet();
        // this CTA's share of the tile's rows, 4 columns per thread
        if (first_tile < total && !*abort_flag) {
            const int m_tiles = tail->tile_off[1];
            const int row0 = first_tile % m_tiles * kM8, col0 = first_tile / m_tiles * BN;
            const int rows = min(kM8, a.R - row0);
            const int r0 = rank * rows / S, r1 = (rank + 1) * rows / S;
            for (int i = threadIdx.x; i < (r1 - r0) * (BN / 4); i += kThreads8) {
                const int r = r0 + i / (BN / 4), c = i % (BN / 4);
                const uint32_t at = smem_u32(smem) + (uint32_t)(r * kPartRow + c) * 16;
                float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
                for (int q = 0; q < S; ++q) {
                    const float4 o = ld_rank(at, (uint32_t)q);
                    v.x += o.x;
                    v.y += o.y;
                    v.z += o.z;
                    v.w += o.w;
                }
                store4(a, (size_t)(row0 + r), col0 + 4 * c, v);
            }
        }
        cluster_meet();  // no CTA leaves while another reads its sums
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem),
                     "n"(SH::kTmemCols)
                     : "memory");
}

// split == 1: persistent, one CTA per SM; else clusters of split CTAs, one per tile
template <int BN, bool SPLIT = false>
cudaError_t launch_fp8(const void* a8, const void* b8, const Fp8Args& a, cudaStream_t s,
                       int tiles = 0) {
    Fp8Maps m;
    for (int i = 0; i < kRowBoxes; ++i)
        if (!make_map_e4m3(&m.a[i], a8, (uint64_t)a.k, (uint64_t)a.R, 1, 32u << i, false))
            return cudaErrorInvalidValue;
    if (!make_map_e4m3(&m.b, b8, (uint64_t)a.k, (uint64_t)a.n, (uint64_t)a.G, BN, true))
        return cudaErrorInvalidValue;
    auto kern = fp8_gemm_kernel<BN, SPLIT>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)smem_bytes8<BN>());
    if (e != cudaSuccess) return e;
    const unsigned grid = SPLIT ? (unsigned)(tiles * a.split) : (unsigned)num_sms();
    return launch_pdl(kern, dim3(grid), dim3(kThreads8), smem_bytes8<BN>(), s, a.split, m, a);
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

MOE_API int moe_matmul_fp8(const void* a, const float* a_scales, const void* b,
                           const float* b_scales, const int32_t* counts, int R, int G, int n,
                           int k, int out_dt, void* y, void* status_ws, void* stream) {
    if (R < 0 || G < 1 || G > kMaxE || n <= 0 || k <= 0) return MOE_ERR_INVALID_ARG;
    if (out_dt != MOE_F32 && out_dt != MOE_BF16) return MOE_ERR_INVALID_ARG;
    if (counts == nullptr && G != 1) return MOE_ERR_INVALID_ARG;
    // tiles are numbered in 32 bits, with room for a step behind the last
    const long long m_tiles = ((long long)R + kM8 - 1) / kM8 + G;
    // rows and depth are rounded up to blocks of 128, columns to 256, in 32 bits
    if (R > INT_MAX - 127 || k > INT_MAX - 127 || n > INT_MAX - 255) return MOE_ERR_UNSUPPORTED;
    if (k % 16 != 0 || m_tiles * (((long long)n + 63) / 64) > (1LL << 30))
        return MOE_ERR_UNSUPPORTED;
    if (R == 0) return MOE_OK;
    const void* p16[] = {a, b, y};
    for (const void* p : p16)
        if (!is_device_ptr(p) || !aligned(p, 16)) return MOE_ERR_INVALID_ARG;
    const void* p4[] = {a_scales, b_scales};
    for (const void* p : p4)
        if (!is_device_ptr(p) || !aligned(p, 4)) return MOE_ERR_INVALID_ARG;
    if (counts != nullptr && (!is_device_ptr(counts) || !aligned(counts, 4)))
        return MOE_ERR_INVALID_ARG;
    if (status_ws != nullptr && (!is_device_ptr(status_ws) || !aligned(status_ws, 256)))
        return MOE_ERR_INVALID_ARG;
    Fp8Args f{};
    f.sa = a_scales;
    f.sb = b_scales;
    f.counts = counts;
    f.R = R;
    f.G = G;
    f.n = n;
    f.k = k;
    f.out_f32 = out_dt == MOE_F32 ? 1 : 0;
    f.y = y;
    f.split = 1;
    f.wide_rows = n % 16 == 0 && aligned(y, 32);
    f.status = static_cast<int*>(status_ws);
    f.wait_limit_ns = kWaitLimitNs;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    // The tile width whose rounds over the SMs take least, by what a block of 128
    // and a tile's start and end take (us, measured at d 2048, inter 1536: a
    // block 0.73 of 256 columns, 0.40 of 128, 0.42 of 64; a tile 2).  64 rows, n
    // 12288, k 2048: 96 tiles of 128 columns take 11.5 us, 192 of 64 columns 16.8;
    // 1024 rows, n 2048, k 6144: 28 and 44; 384 rows in 64 groups, n 2048, k 1536:
    // 256 columns 41, 128 columns 46, 64 columns 76.  How many row tiles the groups make is on the device: one each, or R / 128.
    const long long row_tiles =
        std::max((long long)std::min(G, R), ((long long)R + kM8 - 1) / kM8);
    const int kb_n = (k + kK8 - 1) / kK8, sms = num_sms();
    auto cost = [&](int bn, double block) {
        const long long tiles = row_tiles * (((long long)n + bn - 1) / bn);
        return (double)((tiles + sms - 1) / sms) * (kb_n * block + 2.0);
    };
    // One group with few tiles and a long reduction: several CTAs per tile, at
    // least 4 blocks each (64 rows, n 2048, k 6144: 10.5 us by 4 CTAs per tile, 22.5
    // by one).
    const long long tiles = row_tiles * (((long long)n + 63) / 64);
    while (counts == nullptr && f.split < kMaxSplit && 2 * f.split * tiles <= sms &&
           kb_n >= 8 * f.split)
        f.split *= 2;
    if (f.split > 1) return ret(launch_fp8<64, true>(a, b, f, s, (int)tiles));
    const double c256 = cost(256, 0.73), c128 = cost(128, 0.40), c64 = cost(64, 0.42);
    if (c256 <= c128 && c256 <= c64) return ret(launch_fp8<256>(a, b, f, s));
    if (c128 <= c64) return ret(launch_fp8<128>(a, b, f, s));
    return ret(launch_fp8<64>(a, b, f, s));
}

}  // extern "C"
