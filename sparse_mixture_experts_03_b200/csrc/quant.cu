// 8-bit rows and weights with one fp32 scale per block of 128.
//
// A block's scale is s = A / 448 with A = max(max |x|, 2^-100) over the block
// (448: the largest e4m3 value), its codes are q = the e4m3 value nearest to
// x / s, ties to even, with the quotient 448 x / A taken exactly: a code never
// depends on how a reciprocal was rounded.  2^-100 keeps blocks of zeros (and
// of values too small for an fp32 scale) at codes of 0 without a special case;
// a block with an infinity or a NaN gets a NaN scale and NaN codes.
//
//   moe_quantize_rows          blocks of 1 x 128 along each row (activations)
//   moe_swiglu_quantize_rows   the same of h = silu(gate) * up, in fp32
//   moe_quantize_weight        blocks of 128 x 128 (weights)
//
// The exact quotient.  t = x448 * r (r = 1 / A rounded) is a few ulp off;
// rem = x448 - t A by one fma and t' = t + rem r correct it.  For bf16 input
// x448 = 448 x is exact in fp32, and a border between two codes is b with 5
// significant bits: either the quotient equals b, then rem = (b - t) A is
// exact (a few ulp times 8 bits) and t' = b; or the two differ by at least
// 2^-14 relative (integers of at most 13 bits), far more than t' is off.  So
// rounding t' gives the code of the exact quotient.  fp32 input carries 24
// bits: the few quotients within 4 ulp of a border, or below the smallest
// normal code, are redone in fp64, where 448 x and b A are exact again.
//
// The kernels read and write each value once.  What bounds them is the number
// of instructions they issue, then the memory: rows of d 2048 (24576 of them)
// 30 us, 5.1 TB/s; SwiGLU rows (24581 of inter 1536) 36 us, 5.3 TB/s; weights
// (64 x 2048 x 1536) 96.8 us, 6.2 TB/s, of 6.55 that a copy reaches.  Loading one
// batch ahead, deeper or shallower batches, and 16 rows per CTA made no
// difference or were slower.
#include <cuda_fp8.h>
#include <limits.h>

#include <algorithm>

#include "moe_device.cuh"
#include "moe_internal.h"

namespace moe {
namespace {

constexpr int kQuantThreads = 256;
constexpr int kQuantRows = 8;         // rows per CTA: 8 scales of a block column are one 32-byte piece
constexpr float kE4m3Max = 448.f;
constexpr uint32_t kAmaxFloorBits = 27u << 23;  // 2^-100

// How one block is quantised: t = x * mul * r, corrected with A = den.
struct BlockScale {
    float scale;  // A / 448 (NaN for a block with an infinity or a NaN)
    float mul;    // 448, or 448 * 2^-20 where 448 A would overflow
    float den;    // A times the same power of two
    float rcp;    // 1 / den, to an ulp or two
};

// amax_bits: the bits of max |x| as an fp32 value; infinities and NaN are at
// or above 0x7f800000, so an integer maximum keeps them
__device__ __forceinline__ BlockScale block_scale(uint32_t amax_bits) {
    BlockScale b;
    amax_bits = amax_bits >= 0x7f800000u ? 0x7fffffffu : max(amax_bits, kAmaxFloorBits);
    const float A = __uint_as_float(amax_bits);
    const float pre = A > 1.2676506e30f ? 9.5367431640625e-07f : 1.f;  // above 2^100: 2^-20
    // A / 448, rounded once: a product with 1 / 448 and its correction (all
    // lanes of a block do this: a division would be a tenth of the kernel)
    const float t = A * (1.f / kE4m3Max);
    b.scale = fmaf(fmaf(-t, kE4m3Max, A), 1.f / kE4m3Max, t);
    b.mul = kE4m3Max * pre;
    b.den = A * pre;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(b.rcp) : "f"(b.den));  // 2^-108 <= 1 / den <= 2^100
    return b;
}

// Pairs of fp32 values: one instruction for two of them (the kernels are bound
// by the instructions they issue).
__device__ __forceinline__ uint64_t pair_of(float a, float b) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ uint64_t mul_pair(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t fma_pair(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}

// The quotients of two values: t = n rcp, corrected by (n - t den) rcp.
__device__ __forceinline__ float2 quotients(float x, float y, const BlockScale& b) {
    const uint64_t r = pair_of(b.rcp, b.rcp);
    const uint64_t n = mul_pair(pair_of(x, y), pair_of(b.mul, b.mul));
    const uint64_t t = mul_pair(n, r);
    const uint64_t q = fma_pair(fma_pair(t, pair_of(-b.den, -b.den), n), r, t);
    float2 f;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(f.x), "=f"(f.y) : "l"(q));
    return f;
}

// The fp32 input's quotient, on the right side of every border (see above).
__device__ __forceinline__ float settle_f32(float x, float t, const BlockScale& b) {
    const uint32_t u = __float_as_uint(t) & 0x7fffffffu;
    const uint32_t off = (u & 0xfffffu) - 0x7fffcu;  // low 20 bits within 4 of 0x80000: 0..8
    if (__builtin_expect(u >= 0x3c800000u && off > 8u, 1)) return t;  // 0x3c800000: 2^-6
    const double den = (double)b.den, n = (double)x * (double)b.mul;
    const double r = 1.0 / den;
    double d = n * r;
    d = fma(fma(-d, den, n), r, d);
    // round to odd on the way to fp32, so that the one rounding to e4m3 is right
    float f = __double2float_rz(d);
    if ((double)f != d) f = __uint_as_float(__float_as_uint(f) | 1u);
    return f;
}

__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
    return lo | (hi << 16);
}

__device__ __forceinline__ uint32_t amax_bits8(const float (&f)[8]) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(f[i]) & 0x7fffffffu);
    return m;
}

// Eight consecutive values of a row, as one lane holds them.
struct Bf16x8 {
    uint4 v;
    static constexpr bool kExact = false;
    __device__ __forceinline__ void zero() { v = make_uint4(0, 0, 0, 0); }
    __device__ __forceinline__ void load(const void* p, size_t i) {
        v = __ldcs(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + i));
    }
    // the bits of the largest magnitude, as fp32
    __device__ __forceinline__ uint32_t amax() const {
        uint32_t m;
        asm("{\n\t.reg .b32 a, b, c, d;\n\t"
            "abs.bf16x2 a, %1;\n\tabs.bf16x2 b, %2;\n\tabs.bf16x2 c, %3;\n\t"
            "abs.bf16x2 d, %4;\n\tmax.NaN.bf16x2 a, a, b;\n\tmax.NaN.bf16x2 c, c, d;\n\t"
            "max.NaN.bf16x2 %0, a, c;\n\t}"
            : "=r"(m)
            : "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w));
        return max(m & 0xffff0000u, m << 16);
    }
    __device__ __forceinline__ void get(float (&f)[8]) const {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[2 * i] = __uint_as_float(w[i] << 16);
            f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
};
struct F32x8 {
    uint4 v[2];
    static constexpr bool kExact = true;
    __device__ __forceinline__ void zero() { v[0] = v[1] = make_uint4(0, 0, 0, 0); }
    __device__ __forceinline__ void load(const void* p, size_t i) {
        const uint4* q = reinterpret_cast<const uint4*>(static_cast<const float*>(p) + i);
        v[0] = __ldcs(q);
        v[1] = __ldcs(q + 1);
    }
    __device__ __forceinline__ uint32_t amax() const {
        float f[8];
        get(f);
        return amax_bits8(f);
    }
    __device__ __forceinline__ void get(float (&f)[8]) const {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            f[4 * i] = __uint_as_float(v[i].x);
            f[4 * i + 1] = __uint_as_float(v[i].y);
            f[4 * i + 2] = __uint_as_float(v[i].z);
            f[4 * i + 3] = __uint_as_float(v[i].w);
        }
    }
};

template <bool EXACT>
__device__ __forceinline__ uint2 codes8(const float (&f)[8], const BlockScale& b) {
    float t[8];
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
        const float2 q = quotients(f[i], f[i + 1], b);
        t[i] = EXACT ? settle_f32(f[i], q.x, b) : q.x;
        t[i + 1] = EXACT ? settle_f32(f[i + 1], q.y, b) : q.y;
    }
    return make_uint2(e4m3x4(t[0], t[1], t[2], t[3]), e4m3x4(t[4], t[5], t[6], t[7]));
}

// Rows.  CTA: 8 rows; its 8 warps take the rows' 256-column chunks in order, 16
// lanes per block of 128, 8 columns per lane, kUnroll chunks in flight each.
// The scales [block][row] leave through shared memory, 32 bytes (8 rows) at a
// time.  SRC::fetch starts a chunk's loads, loaded makes its values, amax and
// get give them.
template <typename V>
struct PlainSrc {
    static constexpr bool kExact = V::kExact;
    V v;
    __device__ __forceinline__ void fetch(const void* x, size_t row, int d, int col, bool ok) {
        v.zero();
        if (ok) v.load(x, row * (size_t)d + col);
    }
    __device__ __forceinline__ void loaded() {}
    __device__ __forceinline__ uint32_t amax() const { return v.amax(); }
    __device__ __forceinline__ void get(float (&f)[8]) const { v.get(f); }
};
struct SwigluSrc {
    static constexpr bool kExact = false;  // h itself is an fp32 result
    Bf16x8 g, u;
    float h[8];
    __device__ __forceinline__ void fetch(const void* x, size_t row, int d, int col, bool ok) {
        g.zero();
        u.zero();
        if (ok) {
            g.load(x, row * 2 * (size_t)d + col);
            u.load(x, row * 2 * (size_t)d + d + col);
        }
    }
    // silu(g) u with the hardware exponential and reciprocal.  The argument of the
    // exponential is rounded once, so h is off by at most 2^-22 (4 + |g|) of itself:
    // as much as the exponential for |g| up to 16, 2e-5 at -88, a thousandth of a
    // step of e4m3.  (Of 37.8 million codes of normal gates 72 are not those of 64
    // bits; with fp32's own exponential and division 66, at half as much time again.)
    // The denominator is scaled by 2^-8: 1 / (1 + exp(-g)) lies below
    // the smallest normal number from -87.4 on and would be flushed to zero, where
    // a large up value makes h an ordinary number (fp32's exponential itself ends
    // at -88.7: zero from there).  The scaled sum is one instruction for a pair where
    // two additions were, and undoing the scale one more: 35.7 us at 24581 rows of
    // 1536 with and without the scale.
    __device__ __forceinline__ void loaded() {
        const uint64_t small = pair_of(0.00390625f, 0.00390625f);  // 2^-8
        float a[8], b[8];
        g.get(a);
        u.get(b);
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
            const uint64_t gg = pair_of(a[i], a[i + 1]);
            float2 e;  // exp(-g) = 2^(-g log2(e)), then 2^8 / (1 + it)
            asm("mov.b64 {%0, %1}, %2;" : "=f"(e.x), "=f"(e.y)
                : "l"(mul_pair(gg, pair_of(-1.4426950408889634f, -1.4426950408889634f))));
            asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(e.x));
            asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(e.y));
            asm("mov.b64 {%0, %1}, %2;" : "=f"(e.x), "=f"(e.y)
                : "l"(fma_pair(pair_of(e.x, e.y), small, small)));
            asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(e.x));
            asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(e.y));
            asm("mov.b64 {%0, %1}, %2;" : "=f"(h[i]), "=f"(h[i + 1])
                : "l"(mul_pair(mul_pair(mul_pair(gg, small), pair_of(e.x, e.y)),
                               pair_of(b[i], b[i + 1]))));
        }
    }
    __device__ __forceinline__ uint32_t amax() const { return amax_bits8(h); }
    __device__ __forceinline__ void get(float (&f)[8]) const {
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = h[i];
    }
};

template <typename SRC, int UNROLL>
__global__ void __launch_bounds__(kQuantThreads) quantize_rows_kernel(
    const void* __restrict__ x, const float* __restrict__ w, int R, int d, int n_blocks, int cut,
    uint8_t* __restrict__ q, float* __restrict__ scales) {
    extern __shared__ float s_scale[];  // [n_blocks][8]
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int r0 = blockIdx.x * kQuantRows;
    const int rows = min(kQuantRows, R - r0);
    // this CTA's 256-column chunks of the rows (few rows are cut across CTAs)
    const int ch0 = (int)blockIdx.y * cut;
    const int chunks = min(cut, (d + 255) / 256 - ch0);
    pdl_wait();
    pdl_trigger();  // the next kernel waits for this one's end by itself
    // the next chunk of this warp, 8 further on each time (no division per chunk)
    const int step_row = 8 / chunks, step_ch = 8 - step_row * chunks;
    int row_n = warp / chunks, ch_n = warp - row_n * chunks;
    while (row_n < rows) {
        SRC src[UNROLL];
        int rows_i[UNROLL], cols_i[UNROLL];
#pragma unroll
        for (int i = 0; i < UNROLL; ++i) {
            rows_i[i] = row_n;
            cols_i[i] = row_n < rows ? (ch0 + ch_n) * 256 + lane * 8 : d;  // d: nothing there
            row_n += step_row;
            ch_n += step_ch;
            if (ch_n >= chunks) {
                ch_n -= chunks;
                ++row_n;
            }
            src[i].fetch(x, (size_t)(r0 + rows_i[i]), d, cols_i[i], cols_i[i] < d);
        }
        // the blocks' maxima side by side: 16 lanes each
        uint32_t m[UNROLL];
#pragma unroll
        for (int i = 0; i < UNROLL; ++i) {
            src[i].loaded();
            m[i] = src[i].amax();
        }
#pragma unroll
        for (int off = 8; off > 0; off >>= 1)
#pragma unroll
            for (int i = 0; i < UNROLL; ++i)
                m[i] = max(m[i], __shfl_xor_sync(0xffffffffu, m[i], off));
#pragma unroll
        for (int i = 0; i < UNROLL; ++i) {
            const int row = rows_i[i], col = cols_i[i];
            float f[8];
            src[i].get(f);
            const BlockScale b = block_scale(m[i]);
            if (col < d) {
                *reinterpret_cast<uint2*>(q + (size_t)(r0 + row) * d + col) =
                    codes8<SRC::kExact>(f, b);
                if ((lane & 15) == 0)
                    s_scale[((col >> 7) - 2 * ch0) * kQuantRows + row] =
                        w != nullptr ? b.scale * w[r0 + row] : b.scale;
            }
        }
    }
    __syncthreads();
    const int blk0 = 2 * ch0, blks = min(n_blocks - blk0, 2 * chunks);
    for (int i = tid; i < blks * kQuantRows; i += kQuantThreads) {
        const int row = i % kQuantRows;
        if (row < rows) scales[(size_t)(blk0 + i / kQuantRows) * R + r0 + row] = s_scale[i];
    }
}

// Weights.  CTA: one 128 x 128 block held in registers (8 columns x 8 rows per
// thread): one read, the maximum over the CTA, one write.
template <typename V>
__global__ void __launch_bounds__(kQuantThreads) quantize_weight_kernel(
    const void* __restrict__ W, int n, int k, int nb, int kb, uint8_t* __restrict__ q,
    float* __restrict__ scales) {
    __shared__ uint32_t s_max[kQuantThreads / 32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const size_t blk = blockIdx.x;  // (matrix, row block, column block)
    const int bk = (int)(blk % kb), bn = (int)(blk / kb % nb);
    const size_t g = blk / ((size_t)kb * nb);
    const int col = bk * 128 + (tid & 15) * 8, row0 = bn * 128 + (tid >> 4);
    pdl_wait();
    pdl_trigger();  // the next kernel waits for this one's end by itself
    V v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        v[i].zero();
        const int row = row0 + 16 * i;
        if (row < n && col < k) v[i].load(W, (g * n + row) * (size_t)k + col);
    }
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, v[i].amax());
    m = __reduce_max_sync(0xffffffffu, m);
    if (lane == 0) s_max[warp] = m;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kQuantThreads / 32; ++i) m = max(m, s_max[i]);
    const BlockScale b = block_scale(m);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int row = row0 + 16 * i;
        if (row < n && col < k) {
            float f[8];
            v[i].get(f);
            *reinterpret_cast<uint2*>(q + (g * n + row) * (size_t)k + col) =
                codes8<V::kExact>(f, b);
        }
    }
    if (tid == 0) scales[blk] = b.scale;
}

// One row's scales have to fit the kernel's default shared memory.
constexpr int kMaxRowBlocks = 48 * 1024 / (int)(sizeof(float) * kQuantRows);

template <typename SRC, int UNROLL>
cudaError_t launch_rows(const void* x, const float* w, int R, int d, void* q, float* scales,
                        cudaStream_t s) {
    const int nb = (d + 127) / 128;
    const long long groups = ((long long)R + kQuantRows - 1) / kQuantRows;
    // Few rows are cut along their columns until there are two CTAs per SM or a
    // CTA's warps have one chunk each (64 rows of inter 6144: 15 us by 8 CTAs, 2.9
    // cut).
    const long long chunks = (d + 255) / 256, per_cta = 8 / std::min(R, kQuantRows);
    const long long most = std::max(1LL, chunks / std::max(1LL, per_cta));
    const long long cuts = std::min(most, std::max(1LL, 2LL * num_sms() / groups));
    const int cut = (int)((chunks + cuts - 1) / cuts);  // chunks of a CTA
    return launch_pdl(quantize_rows_kernel<SRC, UNROLL>,
                      dim3((unsigned)groups, (unsigned)((chunks + cut - 1) / cut)),
                      dim3(kQuantThreads), sizeof(float) * kQuantRows * 2 * cut, s, 1, x, w, R, d,
                      nb, cut, static_cast<uint8_t*>(q), scales);
}

int check_rows(int R, int d) {
    if (R < 0 || d <= 0) return MOE_ERR_INVALID_ARG;
    if (d % 16 != 0 || (d + 127) / 128 > kMaxRowBlocks) return MOE_ERR_UNSUPPORTED;
    return MOE_OK;
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

MOE_API int moe_quantize_rows(const void* x, int R, int d, int in_dt, void* q, float* scales,
                              void* stream) {
    if (in_dt != MOE_F32 && in_dt != MOE_BF16) return MOE_ERR_INVALID_ARG;
    const int st = check_rows(R, d);
    if (st != MOE_OK) return st;
    if (R == 0) return MOE_OK;
    if (!is_device_ptr(x) || !aligned(x, 16) || !is_device_ptr(q) || !aligned(q, 16) ||
        !is_device_ptr(scales) || !aligned(scales, 4))
        return MOE_ERR_INVALID_ARG;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    return ret(in_dt == MOE_BF16
                   ? launch_rows<PlainSrc<Bf16x8>, 4>(x, nullptr, R, d, q, scales, s)
                   : launch_rows<PlainSrc<F32x8>, 4>(x, nullptr, R, d, q, scales, s));
}

MOE_API int moe_swiglu_quantize_rows(const void* gate_up, const float* w, int R, int inter,
                                     int in_dt, void* q, float* scales, void* stream) {
    if (in_dt != MOE_F32 && in_dt != MOE_BF16) return MOE_ERR_INVALID_ARG;
    const int st = check_rows(R, inter);
    if (st != MOE_OK) return st;
    if (in_dt != MOE_BF16 || inter > INT_MAX / 2) return MOE_ERR_UNSUPPORTED;
    if (R == 0) return MOE_OK;
    if (!is_device_ptr(gate_up) || !aligned(gate_up, 16) || !is_device_ptr(q) ||
        !aligned(q, 16) || !is_device_ptr(scales) || !aligned(scales, 4))
        return MOE_ERR_INVALID_ARG;
    if (w != nullptr && (!is_device_ptr(w) || !aligned(w, 4))) return MOE_ERR_INVALID_ARG;
    return ret(launch_rows<SwigluSrc, 2>(gate_up, w, R, inter, q, scales,
                                         static_cast<cudaStream_t>(stream)));
}

MOE_API int moe_quantize_weight(const void* W, int G, int n, int k, int in_dt, void* q,
                                float* scales, void* stream) {
    if (in_dt != MOE_F32 && in_dt != MOE_BF16) return MOE_ERR_INVALID_ARG;
    if (G < 0 || n <= 0 || k <= 0) return MOE_ERR_INVALID_ARG;
    if (k % 16 != 0) return MOE_ERR_UNSUPPORTED;
    const long long nb = ((long long)n + 127) / 128, kb = ((long long)k + 127) / 128;
    if (nb * kb > INT_MAX || (long long)G * nb * kb > INT_MAX) return MOE_ERR_UNSUPPORTED;
    if (G == 0) return MOE_OK;
    if (!is_device_ptr(W) || !aligned(W, 16) || !is_device_ptr(q) || !aligned(q, 16) ||
        !is_device_ptr(scales) || !aligned(scales, 4))
        return MOE_ERR_INVALID_ARG;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const dim3 grid((unsigned)(G * nb * kb));
    uint8_t* q8 = static_cast<uint8_t*>(q);
    if (in_dt == MOE_BF16)
        return ret(launch_pdl(quantize_weight_kernel<Bf16x8>, grid, dim3(kQuantThreads), 0, s, 1,
                              W, n, k, (int)nb, (int)kb, q8, scales));
    return ret(launch_pdl(quantize_weight_kernel<F32x8>, grid, dim3(kQuantThreads), 0, s, 1, W, n,
                          k, (int)nb, (int)kb, q8, scales));
}

}  // extern "C"
