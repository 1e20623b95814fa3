// linattn_rec.cuh -- linear attention token by token, the state in registers: runs of fp32 inputs, and single tokens of
// either type (the serving step).
//
// One CTA of 256 threads owns 4 TPR value columns of one (sequence, head): the state slice lies in registers,
// a thread holding four neighbouring columns of every (256 / TPR)-th row.  Per token and state element: t = k v,
// t += S gamma_lo, S = S gamma_hi + t, and one FMA for q.S; the partial outputs of a warp's rows are
// joined by a reduce-scatter of shuffles, those of the 8 warps in shared memory, kRecTok tokens at a time (two
// barriers), while the next tokens are on their way into registers.
//
// Where (sequence, head) pairs fill the GPU, a run in fp32 takes a third of the FMA rate (4 operations an element and
// token, paired): 64 pairs of 1000 tokens, 128 x 128, 372 us (418 unpaired), two CTAs an SM by their registers (128,
// with 32 bytes of spills).  Else it is bound by the latency of a token; then the columns are spread over more CTAs, the
// instructions of four tokens run into each other, and long sequences are divided.  Gradients of 2 x 8 sequences and heads of 200 tokens, 64 x 48: 39 us after
// another kernel, 0.2 us a token of one pass (61 us a token at a time); 63 to 66 us right after each other, when a launch's
// CTAs have been placed beside those of the one before it.  The step is bound by memory: 2048 states of 128 x 128, 44 us in
// and out, 6.1 TB/s.
#pragma once

#include <algorithm>
#include <cstring>
#include <type_traits>

#include "linattn_common.cuh"
#include "pairs.cuh"

namespace r2l {

constexpr int kRecThreads = 256;
constexpr int kRecTok = 8;       // tokens staged at once: one a warp
constexpr int kRecMaxD = 128;

__device__ __forceinline__ float4 rec_fma(float4 a, float b, float4 c) {
    const float2 x = fma2(make_float2(a.x, a.y), make_float2(b, b), make_float2(c.x, c.y));
    const float2 y = fma2(make_float2(a.z, a.w), make_float2(b, b), make_float2(c.z, c.w));
    return make_float4(x.x, x.y, y.x, y.y);
}
__device__ __forceinline__ float4 rec_mul(float4 a, float b) {
    const float2 x = mul2(make_float2(a.x, a.y), make_float2(b, b)), y = mul2(make_float2(a.z, a.w), make_float2(b, b));
    return make_float4(x.x, x.y, y.x, y.y);
}

// DK: 64 or 128, the passes' key channels at most.
template <int TPR, int DK>
__global__ void __launch_bounds__(kRecThreads) linattn_rec_kernel(const __grid_constant__ LaPasses passes) {
    constexpr int COLS = 4 * TPR, ROWS = kRecThreads / TPR, M = DK / ROWS, W = 32 / TPR;  // W: rows a warp holds at once
    constexpr int J = DK / 32, JV = (COLS + 31) / 32;
    constexpr int U = M <= 2 ? 4 : 1;  // tokens in flight: a token of few rows is all latency
    __shared__ float2 sqk[kRecTok][DK];
    __shared__ __align__(16) float sv[kRecTok][COLS];
    __shared__ __align__(16) float part[kRecTok][kRecThreads / 32][COLS];
    const LaPass& p = passes.p[blockIdx.z];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int rr = tid / TPR, cq = (tid % TPR) * 4;  // first row, first column (in the slice)
    const int c0 = blockIdx.y * COLS;
    if (c0 >= p.dv) return;  // a pass with fewer slices than another
    const int ncol = min(COLS, p.dv - c0);           // a multiple of 4
    const bool col_ok = cq < ncol;
    pdl_trigger();
    pdl_wait();

    const bool quiet = passes.states != 0;
    const int runs = passes.nseg - (quiet ? 1 : 0);
    const long long item = blockIdx.x / (unsigned)runs;
    const int sg = (int)(blockIdx.x - (unsigned)item * (unsigned)runs);
    const int seq = (int)(item / p.heads), h = (int)(item - (long long)seq * p.heads);
    // this segment's tokens: `len` from the scan position `first` of the row's `all`
    const int all = la_len(p, seq), first = (int)min((long long)sg * passes.seg_tok, (long long)all), len = min(all - first, passes.seg_tok);
    const int t0 = p.reverse ? all - 1 - first : first, dt = p.reverse ? -1 : 1;
    const size_t tok0 = (size_t)seq * p.seq_len;
    const float* q = static_cast<const float*>(p.q) + tok0 * p.q_tok + (size_t)(h / p.q_div) * p.dk;
    const float* k = static_cast<const float*>(p.k) + tok0 * p.k_tok + (size_t)(h / p.k_div) * p.dk;
    const float* v = static_cast<const float*>(p.v) + tok0 * p.v_tok + (size_t)(h / p.v_div) * p.dv + c0;
    float* y = static_cast<float*>(p.y) + tok0 * p.y_tok + (size_t)h * p.dv + c0;

    const size_t dd = (size_t)p.dk * p.dv, sbase = (size_t)item * dd;
    float* const segs = passes.seg[blockIdx.z] + (size_t)item * passes.nseg * dd;
    const float* in = nullptr;
    float* out = nullptr;
    bool in_t = p.h_t != 0, out_t = in_t;
    if (sg == 0) {
        // a divided sequence starts from the copy: its last segment may write h_last over h0 at any time
        if (p.h0) in = passes.nseg > 1 && !quiet ? segs + (size_t)(passes.nseg - 1) * dd : p.h0 + sbase;
    } else if (!quiet) {
        in = segs + (size_t)(sg - 1) * dd;
        in_t = false;
    }
    if (quiet) {
        out = segs + (size_t)sg * dd;
        out_t = false;
    } else if (sg == passes.nseg - 1 && p.h_last) {
        out = p.h_last + sbase;
    }
    float4 s[M];
#pragma unroll
    for (int m = 0; m < M; ++m) {
        const int r = rr + m * ROWS;
        s[m] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (in && col_ok && r < p.dk) {
            if (!in_t) {
                s[m] = *reinterpret_cast<const float4*>(in + (size_t)r * p.dv + c0 + cq);
            } else {
                const float* a = in + (size_t)(c0 + cq) * p.dk + r;
                s[m] = make_float4(a[0], a[p.dk], a[2 * p.dk], a[3 * p.dk]);
            }
        }
    }
    // the values of this warp's token of the group that begins at n0 (zeros past the end)
    float fq[J], fk[J], fv[JV];
    auto fetch = [&](int n0) {
        const int n = n0 + warp, t = t0 + dt * n;
        const bool live = n < len;
#pragma unroll
        for (int j = 0; j < J; ++j) {
            const int r = lane + 32 * j;
            fq[j] = live && r < p.dk ? q[(size_t)t * p.q_tok + r] : 0.f;
            fk[j] = live && r < p.dk ? k[(size_t)t * p.k_tok + r] : 0.f;
        }
#pragma unroll
        for (int j = 0; j < JV; ++j) {
            const int c = lane + 32 * j;
            fv[j] = live && c < ncol ? v[(size_t)t * p.v_tok + c] : 0.f;
        }
    };
    fetch(0);
    float ghi, glo;
    la_decay_pair(la_clamp_decay(p.log_decay[h]), 1.f, ghi, glo);

    for (int n0 = 0; n0 < len; n0 += kRecTok) {
        const int nt = min(kRecTok, len - n0);
#pragma unroll
        for (int j = 0; j < J; ++j) sqk[warp][lane + 32 * j] = make_float2(fq[j], fk[j] * p.s_in);
#pragma unroll
        for (int j = 0; j < JV; ++j)
            if (lane + 32 * j < COLS) sv[warp][lane + 32 * j] = fv[j];
        __syncthreads();
        fetch(n0 + kRecTok);
        auto tokens = [&](auto shift, auto silent) {
            constexpr bool SHIFT = decltype(shift)::value, QUIET = decltype(silent)::value;
#pragma unroll U
            for (int tt = 0; tt < nt; ++tt) {
                const float4 vv = *reinterpret_cast<const float4*>(&sv[tt][cq]);
                float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                for (int m = 0; m < M; ++m) {
                    const float2 qk = sqk[tt][rr + m * ROWS];
                    float4 a = s[m];
                    if constexpr (SHIFT)
                        a = rec_fma(vv, qk.y, a);
                    else
                        a = rec_fma(a, ghi, rec_fma(a, glo, rec_mul(vv, qk.y)));
                    if constexpr (!QUIET) o = rec_fma(a, qk.x, o);
                    if constexpr (SHIFT) a = rec_fma(a, ghi, rec_mul(a, glo));
                    s[m] = a;
                }
                // the warp's W rows: each step halves what a lane sums, down to one column a lane
                if constexpr (QUIET) {
                } else if constexpr (W == 1) {
                    *reinterpret_cast<float4*>(&part[tt][warp][cq]) = o;
                } else {
                    const bool hi = lane & TPR;
                    const float sx = hi ? o.x : o.z, sy = hi ? o.y : o.w;
                    float2 u = hi ? make_float2(o.z, o.w) : make_float2(o.x, o.y);
                    u.x += __shfl_xor_sync(0xffffffffu, sx, TPR);
                    u.y += __shfl_xor_sync(0xffffffffu, sy, TPR);
                    if constexpr (W == 2) {
                        *reinterpret_cast<float2*>(&part[tt][warp][cq + (hi ? 2 : 0)]) = u;
                    } else {
                        const bool hi2 = lane & (2 * TPR);
                        float w = hi2 ? u.y : u.x;
                        w += __shfl_xor_sync(0xffffffffu, hi2 ? u.x : u.y, 2 * TPR);
                        if constexpr (W == 8) w += __shfl_xor_sync(0xffffffffu, w, 4 * TPR);
                        if (W == 4 || lane < 4 * TPR) part[tt][warp][cq + (hi ? 2 : 0) + (hi2 ? 1 : 0)] = w;
                    }
                }
            }
        };
        if (quiet) {
            if (p.shift)
                tokens(std::true_type(), std::true_type());
            else
                tokens(std::false_type(), std::true_type());
        } else if (p.shift) {
            tokens(std::true_type(), std::false_type());
        } else {
            tokens(std::false_type(), std::false_type());
        }
        __syncthreads();
        if (quiet) continue;
        for (int i = tid; i < nt * COLS; i += kRecThreads) {
            const int tt = i / COLS, c = i % COLS;
            if (c < ncol) {
                float o = 0.f;
#pragma unroll
                for (int g = 0; g < kRecThreads / 32; ++g) o += part[tt][g][c];
                const int t = t0 + dt * (n0 + tt);
                y[(size_t)t * p.y_tok + c] = o * p.s_out;
            }
        }
        // the staging of the next group writes sqk and sv, last read before the barrier above; `part` is written
        // again only behind the next group's first barrier
    }
    if (tid < ncol && sg == 0 && !quiet)
        for (int t = all; t < p.seq_len; ++t) y[(size_t)t * p.y_tok + tid] = 0.f;
    if (out && col_ok) {
#pragma unroll
        for (int m = 0; m < M; ++m) {
            const int r = rr + m * ROWS;
            if (r < p.dk) {
                if (!out_t) {
                    *reinterpret_cast<float4*>(out + (size_t)r * p.dv + c0 + cq) = s[m];
                } else {
                    float* a = out + (size_t)(c0 + cq) * p.dk + r;
                    a[0] = s[m].x;
                    a[p.dk] = s[m].y;
                    a[2 * p.dk] = s[m].z;
                    a[3 * p.dk] = s[m].w;
                }
            }
        }
    }
}

// One token of every sequence (no shift, no lengths): a stream over the states.  The layout is the kernel's above; the
// rows are taken kStepRows at a time, all of their loads in flight at once, and written back as they are updated.
constexpr int kStepRows = 4;

template <typename T>
__global__ void __launch_bounds__(kRecThreads, 4) linattn_step_kernel(const __grid_constant__ LaPass p, int cols) {
    __shared__ float sq[kRecMaxD], sk[kRecMaxD];
    __shared__ __align__(16) float part[kRecThreads * 4];  // [row group][cols]
    const int tid = threadIdx.x;
    const int tpr = cols >> 2, rows_par = kRecThreads / tpr;
    const int rr = tid / tpr, cq = (tid - rr * tpr) * 4;
    const int c0 = blockIdx.y * cols, ncol = min(cols, p.dv - c0);
    const bool col_ok = tid < tpr * rows_par && cq < ncol;
    pdl_trigger();
    pdl_wait();

    const long long item = blockIdx.x;
    const int seq = (int)(item / p.heads), h = (int)(item - (long long)seq * p.heads);
    const float* in = p.h0 + (size_t)item * p.dk * p.dv + c0 + cq;
    float* out = p.h_last + (size_t)item * p.dk * p.dv + c0 + cq;
    float4 s[kStepRows];
    auto load = [&](int m0) {
#pragma unroll
        for (int m = 0; m < kStepRows; ++m) {
            const int r = rr + (m0 + m) * rows_par;
            if (col_ok && r < p.dk) s[m] = *reinterpret_cast<const float4*>(in + (size_t)r * p.dv);
        }
    };
    load(0);
    const T* q = static_cast<const T*>(p.q) + (size_t)seq * p.q_tok + (size_t)(h / p.q_div) * p.dk;
    const T* k = static_cast<const T*>(p.k) + (size_t)seq * p.k_tok + (size_t)(h / p.k_div) * p.dk;
    const T* v = static_cast<const T*>(p.v) + (size_t)seq * p.v_tok + (size_t)(h / p.v_div) * p.dv + c0 + cq;
    for (int i = tid; i < p.dk; i += kRecThreads) {
        sq[i] = to_f32(q[i]);
        sk[i] = to_f32(k[i]) * p.s_in;
    }
    float4 vv = make_float4(0.f, 0.f, 0.f, 0.f);
    if (col_ok) vv = make_float4(to_f32(v[0]), to_f32(v[1]), to_f32(v[2]), to_f32(v[3]));
    // gamma while the loads are on their way
    const float2 gamma = la_decay_pair_of(la_clamp_decay(p.log_decay[h]), 1.f);
    const float ghi = gamma.x, glo = gamma.y;
    __syncthreads();
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int m0 = 0; rr + m0 * rows_par < p.dk; m0 += kStepRows) {
        if (m0 > 0) load(m0);
#pragma unroll
        for (int m = 0; m < kStepRows; ++m) {
            const int r = rr + (m0 + m) * rows_par;
            if (col_ok && r < p.dk) {
                const float kr = sk[r], qr = sq[r];
                float4 a = s[m];
                a.x = fmaf(a.x, ghi, fmaf(a.x, glo, kr * vv.x));
                a.y = fmaf(a.y, ghi, fmaf(a.y, glo, kr * vv.y));
                a.z = fmaf(a.z, ghi, fmaf(a.z, glo, kr * vv.z));
                a.w = fmaf(a.w, ghi, fmaf(a.w, glo, kr * vv.w));
                *reinterpret_cast<float4*>(out + (size_t)r * p.dv) = a;
                o.x = fmaf(qr, a.x, o.x);
                o.y = fmaf(qr, a.y, o.y);
                o.z = fmaf(qr, a.z, o.z);
                o.w = fmaf(qr, a.w, o.w);
            }
        }
    }
    if (col_ok) *reinterpret_cast<float4*>(&part[rr * cols + cq]) = o;
    __syncthreads();
    if (tid < ncol) {
        float y = 0.f;
        for (int g = 0; g < rows_par; ++g) y += part[g * cols + tid];
        static_cast<T*>(p.y)[(size_t)seq * p.y_tok + (size_t)h * p.dv + c0 + tid] = from_f32<T>(y * p.s_out);
    }
}

// ------------------------------------------------------------------------------------ host

// Segments of a sequence and tokens in each, for n passes of at most `width` value channels.  A token's latency (0.15 to 0.2 us)
// bounds a run until some 2.5 CTAs of 32 columns an SM share the time; up to there sequences are divided, as finely as 14
// CTAs an SM and 64 tokens a segment allow: the states' part of every token runs twice, but all segments at once.  Five
// segments are the least that pay: gradients of 8 pairs, 64 x 64, 256 tokens in four 43 us, 40 undivided, 300 tokens in five
// 45 and 48; 4000 tokens 182 and 599 (forward 73 and 599).  32 pairs, 128 x 128, 1024 tokens: 303 us and 200 in 16.
inline void rec_segments(int nseq, int heads, int seq_len, int n, int width, int nsm, int& nseg, int& seg_tok) {
    const long long ctas = (long long)nseq * heads * n * ((width + 31) / 32);
    nseg = 1;
    if (ctas > 0 && 2 * ctas < 5LL * nsm)
        nseg = (int)std::min<long long>(std::min<long long>(14LL * nsm / ctas, 128), (seq_len + kLaTok - 1) / kLaTok);
    if (nseg < 5) nseg = 1;
    seg_tok = nseg > 1 ? (int)(((long long)seq_len + kLaTok * nseg - 1) / (kLaTok * nseg) * kLaTok) : seq_len;
    if (nseg > 1) nseg = (int)(((long long)seq_len + seg_tok - 1) / seg_tok);
}

inline size_t rec_segment_bytes(int nseq, int heads, int seq_len, int n, int dk, int dv, int nsm) {
    int nseg, seg_tok;
    rec_segments(nseq, heads, seq_len, n, n > 1 ? std::max(dk, dv) : dv, nsm, nseg, seg_tok);
    return nseg > 1 ? (size_t)n * nseq * heads * nseg * dk * dv * sizeof(float) : 0;
}

// One launch of the passes.  Columns per CTA: as many as the widest pass has when the (sequence, head, segment) triples fill
// the GPU, fewer (down to 16) when few have to spread over the SMs.
inline cudaError_t linattn_rec_go(const LaPasses& all, int n, int dk, int dv, int nsm, cudaStream_t stream) {
    const long long items = (long long)all.p[0].nseq * all.p[0].heads * (all.nseg - (all.states ? 1 : 0));
    int tpr = 32;
    while (tpr > 4 && (4 * tpr >= 2 * dv || items * n * ((dv + 4 * tpr - 1) / (4 * tpr)) < 2LL * nsm)) tpr >>= 1;
    const dim3 grid((unsigned)items, (unsigned)((dv + 4 * tpr - 1) / (4 * tpr)), (unsigned)n);
    auto go = [&](auto kernel) { return launch_pdl(kernel, grid, dim3(kRecThreads), 0, stream, all); };
    if (dk <= 64) {
        switch (tpr) {
            case 32: return go(linattn_rec_kernel<32, 64>);
            case 16: return go(linattn_rec_kernel<16, 64>);
            case 8: return go(linattn_rec_kernel<8, 64>);
            default: return go(linattn_rec_kernel<4, 64>);
        }
    }
    switch (tpr) {
        case 32: return go(linattn_rec_kernel<32, 128>);
        case 16: return go(linattn_rec_kernel<16, 128>);
        case 8: return go(linattn_rec_kernel<8, 128>);
        default: return go(linattn_rec_kernel<4, 128>);
    }
}

// `n` passes over the same sequences and heads; seg: rec_segment_bytes bytes, or NULL when that is 0.
inline cudaError_t linattn_rec_launch(const LaPass* p, int n, float* seg, int nsm, cudaStream_t stream) {
    LaPasses all;
    std::memset(&all, 0, sizeof(all));
    int dk = 0, dv = 0;
    for (int i = 0; i < n; ++i) {
        all.p[i] = p[i];
        dk = std::max(dk, p[i].dk);
        dv = std::max(dv, p[i].dv);
    }
    rec_segments(p->nseq, p->heads, p->seq_len, n, dv, nsm, all.nseg, all.seg_tok);
    if (all.nseg > 1) {
        const size_t items = (size_t)p->nseq * p->heads, dd = (size_t)p->dk * p->dv;  // dd is the same for all passes
        for (int i = 0; i < n; ++i) all.seg[i] = seg + i * items * all.nseg * dd;
        all.states = 1;
        cudaError_t e = linattn_rec_go(all, n, dk, dv, nsm, stream);
        if (e != cudaSuccess) return e;
        all.states = 0;
        LaPasses scan = all;
        for (int i = 0; i < n; ++i) scan.p[i].reverse = 0;  // segments are counted from where the scan begins
        e = launch_pdl(linattn_segments_kernel, dim3((unsigned)((dd + 255) / 256), (unsigned)items, (unsigned)n), dim3(256), 0, stream, scan);
        if (e != cudaSuccess) return e;
    }
    return linattn_rec_go(all, n, dk, dv, nsm, stream);
}

// The serving step: h0 and h_last given, one token.
template <typename T>
inline cudaError_t linattn_step_launch(const LaPass& p, int nsm, cudaStream_t stream) {
    const long long items = (long long)p.nseq * p.heads;
    int cols = p.dv;
    while (cols > 32 && items * ((p.dv + cols - 1) / cols) < 2LL * nsm) cols = (cols / 2 + 3) & ~3;
    const dim3 grid((unsigned)items, (unsigned)((p.dv + cols - 1) / cols));
    return launch_pdl(linattn_step_kernel<T>, grid, dim3(kRecThreads), 0, stream, p, cols);
}

// h_last = h0 (or zero) where there is no token at all.
__global__ void __launch_bounds__(256) linattn_copy_state_kernel(const float* h0, float* h_last, size_t n) {
    pdl_trigger();
    pdl_wait();
    for (size_t i = (size_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (size_t)gridDim.x * 256)
        h_last[i] = h0 ? h0[i] : 0.f;
}

// Gradients of shared heads: out[token][g][d] = sum over the `div` heads of group g of part[token][head][d].
template <typename T>
__global__ void __launch_bounds__(256)
    linattn_sum_heads_kernel(const float* __restrict__ part, T* __restrict__ out, size_t n, int groups, int div, int d) {
    pdl_trigger();
    pdl_wait();
    for (size_t i = (size_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (size_t)gridDim.x * 256) {
        const size_t c = i % d, tg = i / d, g = tg % groups, t = tg / groups;
        const float* a = part + ((t * groups + g) * div) * d + c;
        float s = 0.f;
        for (int j = 0; j < div; ++j) s += a[(size_t)j * d];
        out[i] = from_f32<T>(s);
    }
}

}  // namespace r2l
