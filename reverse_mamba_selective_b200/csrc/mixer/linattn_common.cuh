// linattn_common.cuh -- what the kernels of linear attention share: one "pass" of the operator, its
// decay factors and its addressing.
//
// A pass computes, for every sequence and head and in scan order (forward or reverse),
//   S_t = gamma S_(t-1) + s_in k_t v_t^T,   y_t = q_t . S_t       (shift = 0), or
//   A_t = R_t + s_in k_t v_t^T,  y_t = q_t . A_t,  R_(t+1) = gamma A_t   (shift = 1)
// with y scaled by s_out.  shift = 1 is the adjoint's form: the decay stands behind the token, not before it.
// The forward operator is the pass (q, k, v); its gradients are three more passes of the same kind:
//   dq = (dy, v, k)  forward, state transposed     dv = (k, q, dy) against the scan order, shift 1
//   dk = (v, dy, q)  against the scan order, shift 1, state transposed
#pragma once

#include "../common.cuh"

namespace r2l {

constexpr int kLaTok = 64;        // tokens per chunk

struct LaPass {
    const void *q, *k, *v;
    void* y;
    long long q_tok, k_tok, v_tok, y_tok;  // elements from token to token
    int nseq, seq_len, heads;              // a sequence: a batch row, or a block of one
    int q_div, k_div, v_div;               // head h reads q head h / q_div, ...
    int dk, dv;
    int reverse, shift;
    int y_f32;                             // y is fp32 whatever the inputs' type
    const float* log_decay;
    const int* lens;                       // [nseq] or NULL
    const float* h0;                       // [nseq][heads] states or NULL
    float* h_last;
    int h_t;                               // states are stored [dv][dk] instead of [dk][dv]
    float s_in, s_out;
};

// A decay of -inf would turn e^(0 * g) into NaN; e^-10000 is zero and its zeroth power one.
__device__ __forceinline__ float la_clamp_decay(float g) { return g < -1e4f ? -1e4f : g; }

// e^(g n) in fp32 from the exact product g n (the product's rounding error is put back to first order).
__device__ __forceinline__ float la_decay_pow_of(float g, float n) {
    const float x = g * n;
    const float e = expf(x);
    return fmaf(e, fmaf(g, n, -x), e);
}
// Not inlined: for tables that are built once a head.
__device__ __noinline__ float la_decay_pow(float g, float n) { return la_decay_pow_of(g, n); }

// e as the sum of two fp32 numbers, neither negative, the second not zero: an infinite state times both stays what it is
// (times zero, or with the signs apart, it would become NaN).
__device__ __forceinline__ float2 la_two_parts(double e) {
    const float hi = __double2float_rz(e), lo = (float)(e - (double)hi);
    return make_float2(hi, hi > 0.f ? fmaxf(lo, __uint_as_float(1u)) : lo);
}
// e^(g n) in two parts: a state that is multiplied by it thousands of times keeps fp32 precision (one fp32 factor is
// up to 2^-24 off, the same way each time: 4.9e-4 after 8192 tokens).
__device__ __forceinline__ float2 la_decay_pair_of(float g, float n) { return la_two_parts(exp((double)g * (double)n)); }
__device__ __noinline__ float2 la_decay_pair_call(float g, float n) { return la_decay_pair_of(g, n); }
__device__ __forceinline__ void la_decay_pair(float g, float n, float& hi, float& lo) {
    const float2 e = la_decay_pair_call(g, n);
    hi = e.x;
    lo = e.y;
}

// Two fp32 values rounded to bf16, infinities to the largest number: the first part of a split leaves an infinity to the
// second, where plain rounding would leave it inf - inf.
__device__ __forceinline__ uint32_t la_pack_sat(float lo, float hi) {
    uint32_t d;
    asm("cvt.rn.satfinite.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
    return d;
}

__device__ __forceinline__ int la_len(const LaPass& p, int seq) {
    if (!p.lens) return p.seq_len;
    const int n = p.lens[seq];
    return n < 0 ? 0 : (n > p.seq_len ? p.seq_len : n);
}

// Up to three passes in one launch (the gradients): blockIdx.z says which.  nseg > 1: sequences are divided into segments of
// seg_tok tokens, first their states alone (states), then, from those before each, the outputs.
struct LaPasses {
    LaPass p[3];
    float* seg[3];  // [item][nseg] states after the segments but the last, then h0's copy
    int nseg, seg_tok, states;
};

// States before the segments: seg[s] = gamma^tokens(s) seg[s - 1] + seg[s], in place (seg[0] is complete: its run
// began with h0); and h0's copy, as it is stored, in the last place.
__global__ void __launch_bounds__(256) linattn_segments_kernel(const __grid_constant__ LaPasses passes) {
    const LaPass& p = passes.p[blockIdx.z];
    const int nseg = passes.nseg, seg_chunks = passes.seg_tok / kLaTok;
    pdl_trigger();
    pdl_wait();
    const int dd = p.dk * p.dv;
    const int e = blockIdx.x * 256 + threadIdx.x;
    const int item = blockIdx.y;
    if (e >= dd) return;
    const int seq = item / p.heads, h = item - seq * p.heads;
    const int len = la_len(p, seq), nch = (len + kLaTok - 1) / kLaTok;
    const int missing = nch * kLaTok - len;  // tokens that the ragged chunk lacks
    const int ragged = p.reverse ? 0 : nch - 1;
    const float g = la_clamp_decay(p.log_decay[h]);
    float* a = passes.seg[blockIdx.z] + (size_t)item * nseg * dd + e;
    if (p.h0) a[(size_t)(nseg - 1) * dd] = p.h0[(size_t)item * dd + e];
    // whole segments share a decay; eight states are on their way at once
    const float2 whole = la_decay_pair_of(g, (float)(seg_chunks * kLaTok));
    float s = a[0];
    for (int i0 = 1; i0 < nseg - 1; i0 += 8) {
        float x[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) x[u] = i0 + u < nseg - 1 ? a[(size_t)(i0 + u) * dd] : 0.f;
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            const int i = i0 + u;
            if (i >= nseg - 1) break;
            const int c0 = min(i * seg_chunks, nch), c1 = min(c0 + seg_chunks, nch);
            const int tok = (c1 - c0) * kLaTok - (ragged >= c0 && ragged < c1 ? missing : 0);
            float2 e = whole;
            if (tok != seg_chunks * kLaTok) la_decay_pair(g, (float)tok, e.x, e.y);
            s = fmaf(s, e.x, fmaf(s, e.y, x[u]));
            a[(size_t)i * dd] = s;
        }
    }
}

}  // namespace r2l
