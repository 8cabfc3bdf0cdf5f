// Group-limited top-k of one token's fp32 logits and the gate weights of the
// chosen experts (device code shared by the router kernels and the layer's
// form for a few tokens).
#pragma once

#include <limits.h>

#include "moe_device.cuh"
#include "moe_internal.h"

namespace moe {

// Selection key of expert e from its fp32 logit l.
__device__ __forceinline__ float sel_key(float l, int e, int gate, const float* bias) {
    if (bias == nullptr) return l;  // monotone in the gate score for both gates
    const float g = gate == MOE_GATE_SIGMOID ? 1.f / (1.f + expf(-l)) : l;
    return g + bias[e];
}

// Weights of the k chosen experts from their logits (one thread).
__device__ __forceinline__ void gate_weights(const float (&l)[kMaxK], int k, int gate,
                                             float (&w)[kMaxK]) {
    float sum = 0.f;
    if (gate == MOE_GATE_SIGMOID) {
#pragma unroll
        for (int r = 0; r < kMaxK; ++r) {
            if (r >= k) break;
            w[r] = 1.f / (1.f + expf(-l[r]));
            sum += w[r];
        }
    } else {
        float m = l[0];
#pragma unroll
        for (int r = 1; r < kMaxK; ++r)
            if (r < k) m = fmaxf(m, l[r]);
#pragma unroll
        for (int r = 0; r < kMaxK; ++r) {
            if (r >= k) break;
            w[r] = expf(l[r] - m);
            sum += w[r];
        }
    }
#pragma unroll
    for (int r = 0; r < kMaxK; ++r)
        if (r < k) w[r] /= sum;
}

// (v, i) beats (bv, bi): larger value, ties to the lower index; bi == INT_MAX
// marks "nothing yet".
__device__ __forceinline__ bool beats(float v, int i, float bv, int bi) {
    return bi == INT_MAX || v > bv || (v == bv && i < bi);
}

__device__ __forceinline__ void warp_argmax(float& v, int& i) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
        float ov = __shfl_xor_sync(0xffffffffu, v, off);
        int oi = __shfl_xor_sync(0xffffffffu, i, off);
        if (oi != INT_MAX && beats(ov, oi, v, i)) {
            v = ov;
            i = oi;
        }
    }
}

// Argmax over each aligned segment of 8 lanes (same tie rule as warp_argmax).
__device__ __forceinline__ void seg8_argmax(float& v, int& i) {
#pragma unroll
    for (int off = 4; off > 0; off >>= 1) {
        float ov = __shfl_xor_sync(0xffffffffu, v, off);
        int oi = __shfl_xor_sync(0xffffffffu, i, off);
        if (oi != INT_MAX && beats(ov, oi, v, i)) {
            v = ov;
            i = oi;
        }
    }
}

// Group-limited top-k of one token from its fp32 logits L[0..E) (shared
// memory), by one warp.  Writes k expert ids (descending, ties to the lower
// index) and the normalised sigmoid weights.
template <int EJ>
__device__ __forceinline__ void warp_topk(const float* L, int lane, int E, int k, int G, int TG,
                                          int gate, const float* __restrict__ bias,
                                          int32_t* __restrict__ idx_out,
                                          float* __restrict__ w_out) {
    const int gsz = E / G;
    // group scores: max key of each group (lane g < G owns group g)
    float gval = -INFINITY;
    if (lane < G)
        for (int e = lane * gsz; e < (lane + 1) * gsz; ++e)
            gval = fmaxf(gval, sel_key(L[e], e, gate, bias));
    uint32_t kept = 0;
    for (int r = 0; r < TG; ++r) {
        float v = -INFINITY;
        int i = INT_MAX;
        if (lane < G && !((kept >> lane) & 1u)) {
            v = gval;
            i = lane;
        }
        warp_argmax(v, i);
        kept |= 1u << i;
    }
    // candidates: experts lane + 32 j inside kept groups
    float cv[EJ];
    bool cand[EJ];
#pragma unroll
    for (int j = 0; j < EJ; ++j) {
        int e = lane + 32 * j;
        cand[j] = e < E && ((kept >> (e / gsz)) & 1u);
        cv[j] = cand[j] ? sel_key(L[e], e, gate, bias) : -INFINITY;
    }
    int sel_e[kMaxK];
    float sel_l[kMaxK];
#pragma unroll
    for (int r = 0; r < kMaxK; ++r) {
        if (r >= k) break;
        float bv = -INFINITY;
        int bi = INT_MAX;
#pragma unroll
        for (int j = 0; j < EJ; ++j) {
            int e = lane + 32 * j;
            if (cand[j] && beats(cv[j], e, bv, bi)) {
                bv = cv[j];
                bi = e;
            }
        }
        warp_argmax(bv, bi);
#pragma unroll
        for (int j = 0; j < EJ; ++j)
            if (lane + 32 * j == bi) cand[j] = false;
        sel_e[r] = bi;
    }
    if (lane == 0) {
#pragma unroll
        for (int r = 0; r < kMaxK; ++r)
            if (r < k) sel_l[r] = L[sel_e[r]];
        float wv[kMaxK];
        gate_weights(sel_l, k, gate, wv);
#pragma unroll
        for (int r = 0; r < kMaxK; ++r) {
            if (r >= k) break;
            idx_out[r] = sel_e[r];
            w_out[r] = wv[r];
        }
    }
}

}  // namespace moe
