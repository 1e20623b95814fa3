// linattn_rec.cuh -- linear attention token by token, the state in registers: fp32 inputs, single tokens
// (the serving step) and runs of a few tokens.
//
// One CTA of 256 threads owns `cols` value columns of one (sequence, head): the state slice
// [dk][cols] lies in registers, a thread holding four neighbouring columns of every rows_par-th row.
// Per token and state element: t = k v, t += S gamma_lo, S = S gamma_hi + t, and one FMA for q.S.
// A group of kRecTok tokens is staged in shared memory, their row-partial outputs are summed there.
//
// A single token is bound by the state's read and write (2 x 4 bytes an element, all of a thread's loads in
// flight at once); runs in fp32 by the FMA pipe (4 operations an element and token).
#pragma once

#include "linattn_common.cuh"

namespace r2l {

constexpr int kRecThreads = 256;
constexpr int kRecTok = 8;       // tokens staged at once
constexpr int kRecMaxD = 128;

template <typename T>
__device__ __forceinline__ void la_store(T* p, float v) {
    *p = from_f32<T>(v);
}

// MAXM: rows a thread holds (ceil(dk / rows_par) <= MAXM).
template <typename T, typename TY, int MAXM, bool SHIFT>
__global__ void __launch_bounds__(kRecThreads) linattn_rec_kernel(LaPass p, int cols) {
    __shared__ float sq[kRecTok][kRecMaxD], sk[kRecTok][kRecMaxD];
    __shared__ float sv[kRecTok][kRecMaxD];
    __shared__ __align__(16) float part[kRecTok][kRecThreads * 4];  // [token][row group][cols]
    const int tid = threadIdx.x;
    const int tpr = cols >> 2, rows_par = kRecThreads / tpr;
    const bool act = tid < tpr * rows_par;
    const int rr = tid / tpr, cq = (tid - rr * tpr) * 4;  // first row, first column (in the slice)
    const int c0 = blockIdx.y * cols;
    const int ncol = min(cols, p.dv - c0);                // dv and cols are multiples of 4
    const bool col_ok = act && cq < ncol;
    pdl_trigger();
    pdl_wait();

    const long long item = blockIdx.x;
    const int seq = (int)(item / p.heads), h = (int)(item - (long long)seq * p.heads);
    const int len = la_len(p, seq);
    const size_t tok0 = (size_t)seq * p.seq_len;
    const T* q = static_cast<const T*>(p.q) + tok0 * p.q_tok + (size_t)(h / p.q_div) * p.dk;
    const T* k = static_cast<const T*>(p.k) + tok0 * p.k_tok + (size_t)(h / p.k_div) * p.dk;
    const T* v = static_cast<const T*>(p.v) + tok0 * p.v_tok + (size_t)(h / p.v_div) * p.dv + c0;
    TY* y = static_cast<TY*>(p.y) + tok0 * p.y_tok + (size_t)h * p.dv + c0;

    const size_t sbase = (size_t)item * p.dk * p.dv;
    float4 s[MAXM];
#pragma unroll
    for (int m = 0; m < MAXM; ++m) {
        const int r = rr + m * rows_par;
        s[m] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (p.h0 && col_ok && r < p.dk) {
            if (!p.h_t) {
                s[m] = *reinterpret_cast<const float4*>(p.h0 + sbase + (size_t)r * p.dv + c0 + cq);
            } else {
                const float* a = p.h0 + sbase + (size_t)(c0 + cq) * p.dk + r;
                s[m] = make_float4(a[0], a[p.dk], a[2 * p.dk], a[3 * p.dk]);
            }
        }
    }
    float ghi, glo;
    la_decay_pair(la_clamp_decay(p.log_decay[h]), 1.f, ghi, glo);

    for (int n0 = 0; n0 < len; n0 += kRecTok) {
        const int nt = min(kRecTok, len - n0);
        // stage the group's rows (scan order)
        for (int i = tid; i < nt * p.dk; i += kRecThreads) {
            const int tt = i / p.dk, r = i - tt * p.dk;
            const int t = p.reverse ? len - 1 - (n0 + tt) : n0 + tt;
            sq[tt][r] = to_f32(q[(size_t)t * p.q_tok + r]);
            sk[tt][r] = to_f32(k[(size_t)t * p.k_tok + r]) * p.s_in;
        }
        for (int i = tid; i < nt * ncol; i += kRecThreads) {
            const int tt = i / ncol, c = i - tt * ncol;
            const int t = p.reverse ? len - 1 - (n0 + tt) : n0 + tt;
            sv[tt][c] = to_f32(v[(size_t)t * p.v_tok + c]);
        }
        __syncthreads();
        if (col_ok) {
            for (int tt = 0; tt < nt; ++tt) {
                const float4 vv = *reinterpret_cast<const float4*>(&sv[tt][cq]);
                float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                for (int m = 0; m < MAXM; ++m) {
                    const int r = rr + m * rows_par;
                    if (r < p.dk) {
                        const float kr = sk[tt][r], qr = sq[tt][r];
                        float4 a = s[m];
                        if (SHIFT) {
                            a = make_float4(fmaf(kr, vv.x, a.x), fmaf(kr, vv.y, a.y), fmaf(kr, vv.z, a.z), fmaf(kr, vv.w, a.w));
                        } else {
                            a.x = fmaf(a.x, ghi, fmaf(a.x, glo, kr * vv.x));
                            a.y = fmaf(a.y, ghi, fmaf(a.y, glo, kr * vv.y));
                            a.z = fmaf(a.z, ghi, fmaf(a.z, glo, kr * vv.z));
                            a.w = fmaf(a.w, ghi, fmaf(a.w, glo, kr * vv.w));
                        }
                        o.x = fmaf(qr, a.x, o.x);
                        o.y = fmaf(qr, a.y, o.y);
                        o.z = fmaf(qr, a.z, o.z);
                        o.w = fmaf(qr, a.w, o.w);
                        if (SHIFT) {
                            a.x = fmaf(a.x, ghi, a.x * glo);
                            a.y = fmaf(a.y, ghi, a.y * glo);
                            a.z = fmaf(a.z, ghi, a.z * glo);
                            a.w = fmaf(a.w, ghi, a.w * glo);
                        }
                        s[m] = a;
                    }
                }
                *reinterpret_cast<float4*>(&part[tt][rr * cols + cq]) = o;
            }
        }
        __syncthreads();
        for (int i = tid; i < nt * ncol; i += kRecThreads) {
            const int tt = i / ncol, c = i - tt * ncol;
            float o = 0.f;
            for (int g = 0; g < rows_par; ++g) o += part[tt][g * cols + c];
            const int t = p.reverse ? len - 1 - (n0 + tt) : n0 + tt;
            la_store(y + (size_t)t * p.y_tok + c, o * p.s_out);
        }
        // the next group's staging writes sq, sk and sv, last read before the barrier above; `part` is
        // written again only behind the next group's first barrier
    }
    if (tid < ncol)
        for (int t = len; t < p.seq_len; ++t) la_store(y + (size_t)t * p.y_tok + tid, 0.f);
    if (p.h_last && col_ok) {
#pragma unroll
        for (int m = 0; m < MAXM; ++m) {
            const int r = rr + m * rows_par;
            if (r < p.dk) {
                if (!p.h_t) {
                    *reinterpret_cast<float4*>(p.h_last + sbase + (size_t)r * p.dv + c0 + cq) = s[m];
                } else {
                    float* a = p.h_last + sbase + (size_t)(c0 + cq) * p.dk + r;
                    a[0] = s[m].x;
                    a[p.dk] = s[m].y;
                    a[2 * p.dk] = s[m].z;
                    a[3 * p.dk] = s[m].w;
                }
            }
        }
    }
}

// ------------------------------------------------------------------------------------ host

template <typename T, typename TY, int MAXM>
inline cudaError_t linattn_rec_launch_m(const LaPass& p, int cols, cudaStream_t stream) {
    const dim3 grid((unsigned)((long long)p.nseq * p.heads), (unsigned)((p.dv + cols - 1) / cols));
    if (p.shift) return launch_pdl(linattn_rec_kernel<T, TY, MAXM, true>, grid, dim3(kRecThreads), 0, stream, p, cols);
    return launch_pdl(linattn_rec_kernel<T, TY, MAXM, false>, grid, dim3(kRecThreads), 0, stream, p, cols);
}

// Columns per CTA: all of them when the (sequence, head) pairs fill the GPU, else half or a quarter, so
// that a few heads still spread over the SMs.
template <typename T, typename TY>
inline cudaError_t linattn_rec_launch(const LaPass& p, int nsm, cudaStream_t stream) {
    const long long items = (long long)p.nseq * p.heads;
    int cols = p.dv;
    while (cols > 32 && items * ((p.dv + cols - 1) / cols) < 2LL * nsm) cols = (cols / 2 + 3) & ~3;
    const int rows_par = kRecThreads / (cols / 4);
    const int m = (p.dk + rows_par - 1) / rows_par;
    if (m <= 4) return linattn_rec_launch_m<T, TY, 4>(p, cols, stream);
    if (m <= 8) return linattn_rec_launch_m<T, TY, 8>(p, cols, stream);
    return linattn_rec_launch_m<T, TY, 16>(p, cols, stream);
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
