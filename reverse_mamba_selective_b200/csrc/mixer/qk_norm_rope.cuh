// qk_norm_rope.cuh -- per-head RMS norm of queries and keys with the rotary position embedding, and its
// gradients.
//
// Bound by memory: every head is read once and written once (16-byte pieces).  A group of G lanes owns a
// head; lane s holds the two pieces that rotate together (channels s V .. and rot / 2 + s V ..), so the
// rotation needs no exchange and the norm one shuffle tree over the group.  The angles of a token are
// shared by all its heads: a CTA forms them once for its tokens, in fp64 up to the fraction of a turn
// (position 100000 x frequency 1 leaves fp32 half a degree), while the first heads are on their way.
#pragma once

#include "../common.cuh"

namespace r2l {

constexpr int kRopeThreads = 256;
constexpr int kRopeTok = 4;       // tokens per CTA step (1 for few tokens)
constexpr int kRopeMaxDim = 256;

struct RopeParams {
    const void *x[2], *dy[2];   // queries, keys
    void* out[2];
    long long x_tok[2], out_tok[2], dy_tok[2];
    int heads[2];
    const float* weight[2];
    float* part;                // [2][gridDim.x][head_dim] partial weight gradients, or NULL
    const void* positions;
    const float* inv_freq;
    int tokens, dim, rot, interleaved, pos64, tok_step;
    float eps, inv_dim;
};

// V neighbouring values at p (16 bytes for V > 1), as fp32.
template <typename T, int V>
__device__ __forceinline__ void rope_load(const T* p, float (&v)[V]) {
    if constexpr (V == 1) {
        v[0] = to_f32(*p);
    } else if constexpr (sizeof(T) == 4) {
        const float4 a = *reinterpret_cast<const float4*>(p);
        v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
    } else {
        const uint4 a = *reinterpret_cast<const uint4*>(p);
        const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = __uint_as_float(w[i] << 16);
            v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        }
    }
}

template <typename T, int V>
__device__ __forceinline__ void rope_store(T* p, const float (&v)[V]) {
    if constexpr (V == 1) {
        *p = from_f32<T>(v[0]);
    } else if constexpr (sizeof(T) == 4) {
        *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
    } else {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t*>(&b);
        }
        *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    }
}

// The pieces (of V channels) of slot s: a and b, b < 0 where there is none.
template <int V>
__device__ __forceinline__ void rope_slot(int s, int dim, int rot, bool inter, int& a, int& b) {
    const int np = dim / V, rp = inter ? 0 : rot / 2 / V;
    if (s < rp) {
        a = s;
        b = s + rp;
    } else {
        a = 2 * rp + 2 * (s - rp);
        b = a + 1;
    }
    if (a >= np) a = -1;
    if (b >= np) b = -1;
}

// Rotates the slot's channels; sign -1 takes the rotation back.  cs: (cos, sin) of the token's pairs.
template <int V>
__device__ __forceinline__ void rope_rotate(float (&xa)[V], float (&xb)[V], int a, int b, int rot, bool inter, float sign,
                                            const float2* cs) {
    if (!inter) {
        if (a >= 0 && a < rot / 2 / V) {
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const float2 t = cs[a * V + i];
                const float sn = sign * t.y, u = xa[i], w = xb[i];
                xa[i] = u * t.x - w * sn;
                xb[i] = w * t.x + u * sn;
            }
        }
    } else if constexpr (V == 1) {
        if (a >= 0 && a < rot) {
            const float2 t = cs[a >> 1];
            const float sn = sign * t.y, u = xa[0], w = xb[0];
            xa[0] = u * t.x - w * sn;
            xb[0] = w * t.x + u * sn;
        }
    } else {
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            float(&x)[V] = half ? xb : xa;
            const int piece = half ? b : a;
            if (piece >= 0 && piece * V < rot) {
#pragma unroll
                for (int i = 0; i < V; i += 2) {
                    const float2 t = cs[(piece * V + i) >> 1];
                    const float sn = sign * t.y, u = x[i], w = x[i + 1];
                    x[i] = u * t.x - w * sn;
                    x[i + 1] = w * t.x + u * sn;
                }
            }
        }
    }
}

// (cos, sin) of the angles of tokens t0 .. t0 + nt - 1 into cs[token][rot / 2].
__device__ __forceinline__ void rope_angles(const RopeParams& p, int t0, int nt, float2* cs) {
    const int half = p.rot >> 1;
    for (int i = threadIdx.x; i < nt * half; i += kRopeThreads) {
        const int tt = i / half, f = i - tt * half;
        const double pos = p.pos64 ? (double)static_cast<const long long*>(p.positions)[t0 + tt]
                                   : (double)static_cast<const int*>(p.positions)[t0 + tt];
        const double turns = pos * (double)p.inv_freq[f] * 0.15915494309189535;  // 1 / (2 pi)
        float sn, cn;
        sincospif((float)(2.0 * (turns - rint(turns))), &sn, &cn);
        cs[i] = make_float2(cn, sn);
    }
}

// The weights of both operands into shared memory (ones where there are none).
__device__ __forceinline__ void rope_weights(const RopeParams& p, float (*sw)[kRopeMaxDim]) {
    for (int i = threadIdx.x; i < 2 * p.dim; i += kRopeThreads) {
        const int w = i >= p.dim, c = w ? i - p.dim : i;
        sw[w][c] = p.weight[w] ? p.weight[w][c] : 1.f;
    }
}

template <int V>
__device__ __forceinline__ void rope_weight(const float* sw, float (&v)[V]) {
    if constexpr (V == 1) {
        v[0] = *sw;
    } else {
#pragma unroll
        for (int i = 0; i < V; i += 4) {
            const float4 a = *reinterpret_cast<const float4*>(sw + i);
            v[i] = a.x, v[i + 1] = a.y, v[i + 2] = a.z, v[i + 3] = a.w;
        }
    }
}

template <int G>
__device__ __forceinline__ float rope_group_sum(float v) {
#pragma unroll
    for (int o = G / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// G lanes per head, SL slots per lane (SL > 1 only for single channels, V = 1).
template <typename T, int V, int G, int SL>
__global__ void __launch_bounds__(kRopeThreads) qk_norm_rope_kernel(const __grid_constant__ RopeParams p) {
    __shared__ __align__(16) float2 cs[kRopeTok][kRopeMaxDim / 2];
    __shared__ __align__(16) float sw[2][kRopeMaxDim];
    constexpr int kGroups = kRopeThreads / G;
    const int g = threadIdx.x / G, s0 = threadIdx.x % G;
    const int t0 = blockIdx.x * p.tok_step, nt = min(p.tok_step, p.tokens - t0);
    const int ht = p.heads[0] + p.heads[1], nvec = nt * ht;
    const bool inter = p.interleaved != 0;
    int pa[SL], pb[SL];
#pragma unroll
    for (int j = 0; j < SL; ++j) rope_slot<V>(s0 + j * G, p.dim, p.rot, inter, pa[j], pb[j]);
    pdl_trigger();
    pdl_wait();

    float xa[SL][V], xb[SL][V];
    auto fetch = [&](int vec) {
        const int tt = vec / ht, hh = vec - tt * ht, w = hh >= p.heads[0];
        const T* x = static_cast<const T*>(p.x[w]) + (size_t)(t0 + tt) * p.x_tok[w] + (size_t)(w ? hh - p.heads[0] : hh) * p.dim;
#pragma unroll
        for (int j = 0; j < SL; ++j) {
#pragma unroll
            for (int i = 0; i < V; ++i) xa[j][i] = xb[j][i] = 0.f;
            if (vec < nvec && pa[j] >= 0) rope_load<T, V>(x + pa[j] * V, xa[j]);
            if (vec < nvec && pb[j] >= 0) rope_load<T, V>(x + pb[j] * V, xb[j]);
        }
    };
    fetch(g);
    rope_weights(p, sw);
    rope_angles(p, t0, nt, &cs[0][0]);
    __syncthreads();
    const int half = p.rot >> 1;
    for (int v0 = 0; v0 < nvec; v0 += kGroups) {  // uniform over the CTA: the shuffles need whole warps
        const int vec = v0 + g;
        float ya[SL][V], yb[SL][V], ss = 0.f;
#pragma unroll
        for (int j = 0; j < SL; ++j)
#pragma unroll
            for (int i = 0; i < V; ++i) {
                ya[j][i] = xa[j][i];
                yb[j][i] = xb[j][i];
                ss = fmaf(xa[j][i], xa[j][i], ss);
                ss = fmaf(xb[j][i], xb[j][i], ss);
            }
        if (v0 + kGroups < nvec) fetch(vec + kGroups);
        const float inv = rsqrtf(fmaf(rope_group_sum<G>(ss), p.inv_dim, p.eps));
        if (vec >= nvec) continue;
        const int tt = vec / ht, hh = vec - tt * ht, w = hh >= p.heads[0];
        T* out = static_cast<T*>(p.out[w]) + (size_t)(t0 + tt) * p.out_tok[w] + (size_t)(w ? hh - p.heads[0] : hh) * p.dim;
        const float2* tcs = &cs[0][0] + tt * half;
#pragma unroll
        for (int j = 0; j < SL; ++j) {
            float wa[V], wb[V];
            rope_weight<V>(&sw[w][pa[j] >= 0 ? pa[j] * V : 0], wa);
            rope_weight<V>(&sw[w][pb[j] >= 0 ? pb[j] * V : 0], wb);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                ya[j][i] *= inv * wa[i];
                yb[j][i] *= inv * wb[i];
            }
            rope_rotate<V>(ya[j], yb[j], pa[j], pb[j], p.rot, inter, 1.f, tcs);
            if (pa[j] >= 0) rope_store<T, V>(out + pa[j] * V, ya[j]);
            if (pb[j] >= 0) rope_store<T, V>(out + pb[j] * V, yb[j]);
        }
    }
}

// Gradients of the queries (blockIdx.y 0) or keys (1).  With z = x / rms and u = the rotation taken back
// from dy: dx = (u w - z mean(u w z)) / rms, dw = sum of u z over tokens and heads.  A lane keeps its channels'
// share of dw in registers over all its heads; a CTA's groups add theirs in a fixed order at the end.
template <typename T, int V, int G, int SL>
__global__ void __launch_bounds__(kRopeThreads) qk_norm_rope_bwd_kernel(const __grid_constant__ RopeParams p) {
    __shared__ __align__(16) float2 cs[kRopeTok][kRopeMaxDim / 2];
    __shared__ float red[kRopeThreads / G][kRopeMaxDim < 2 * V * G * SL ? kRopeMaxDim : 2 * V * G * SL];
    constexpr int kGroups = kRopeThreads / G;
    const int g = threadIdx.x / G, s0 = threadIdx.x % G;
    const int w = blockIdx.y, heads = p.heads[w];
    const bool inter = p.interleaved != 0;
    const int half = p.rot >> 1;
    int pa[SL], pb[SL];
    float wa[SL][V], wb[SL][V], da[SL][V], db[SL][V];
    pdl_trigger();
    pdl_wait();
    __shared__ __align__(16) float sw[2][kRopeMaxDim];
    rope_weights(p, sw);
    __syncthreads();
#pragma unroll
    for (int j = 0; j < SL; ++j) {
        rope_slot<V>(s0 + j * G, p.dim, p.rot, inter, pa[j], pb[j]);
        rope_weight<V>(&sw[w][pa[j] >= 0 ? pa[j] * V : 0], wa[j]);
        rope_weight<V>(&sw[w][pb[j] >= 0 ? pb[j] * V : 0], wb[j]);
#pragma unroll
        for (int i = 0; i < V; ++i) da[j][i] = db[j][i] = 0.f;
    }
    const int steps = (p.tokens + p.tok_step - 1) / p.tok_step;
    for (int st = blockIdx.x; st < steps && heads > 0; st += gridDim.x) {
        const int t0 = st * p.tok_step, nt = min(p.tok_step, p.tokens - t0), nvec = nt * heads;
        __syncthreads();  // the previous step's angles have been read
        rope_angles(p, t0, nt, &cs[0][0]);
        __syncthreads();
        for (int v0 = 0; v0 < nvec; v0 += kGroups) {
            const int vec = v0 + g;
            const bool live = vec < nvec;
            const int tt = live ? vec / heads : 0, hh = live ? vec - tt * heads : 0;
            const T* x = static_cast<const T*>(p.x[w]) + (size_t)(t0 + tt) * p.x_tok[w] + (size_t)hh * p.dim;
            const T* dy = static_cast<const T*>(p.dy[w]) + (size_t)(t0 + tt) * p.dy_tok[w] + (size_t)hh * p.dim;
            float xa[SL][V], xb[SL][V], ua[SL][V], ub[SL][V];
            float ss = 0.f, dot = 0.f;
#pragma unroll
            for (int j = 0; j < SL; ++j) {
#pragma unroll
                for (int i = 0; i < V; ++i) xa[j][i] = xb[j][i] = ua[j][i] = ub[j][i] = 0.f;
                if (live && pa[j] >= 0) {
                    rope_load<T, V>(x + pa[j] * V, xa[j]);
                    rope_load<T, V>(dy + pa[j] * V, ua[j]);
                }
                if (live && pb[j] >= 0) {
                    rope_load<T, V>(x + pb[j] * V, xb[j]);
                    rope_load<T, V>(dy + pb[j] * V, ub[j]);
                }
            }
#pragma unroll
            for (int j = 0; j < SL; ++j) {
                if (live) rope_rotate<V>(ua[j], ub[j], pa[j], pb[j], p.rot, inter, -1.f, &cs[0][0] + tt * half);
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    ss = fmaf(xa[j][i], xa[j][i], ss);
                    ss = fmaf(xb[j][i], xb[j][i], ss);
                    dot = fmaf(ua[j][i] * wa[j][i], xa[j][i], dot);
                    dot = fmaf(ub[j][i] * wb[j][i], xb[j][i], dot);
                }
            }
            const float inv = rsqrtf(fmaf(rope_group_sum<G>(ss), p.inv_dim, p.eps));
            const float m = rope_group_sum<G>(dot) * p.inv_dim * inv * inv;  // mean(u w z) / rms
            if (!live) continue;
            T* out = static_cast<T*>(p.out[w]) + (size_t)(t0 + tt) * p.out_tok[w] + (size_t)hh * p.dim;
#pragma unroll
            for (int j = 0; j < SL; ++j) {
                float oa[V], ob[V];
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    da[j][i] = fmaf(ua[j][i], xa[j][i] * inv, da[j][i]);
                    db[j][i] = fmaf(ub[j][i], xb[j][i] * inv, db[j][i]);
                    oa[i] = inv * (ua[j][i] * wa[j][i] - xa[j][i] * m);
                    ob[i] = inv * (ub[j][i] * wb[j][i] - xb[j][i] * m);
                }
                if (pa[j] >= 0) rope_store<T, V>(out + pa[j] * V, oa);
                if (pb[j] >= 0) rope_store<T, V>(out + pb[j] * V, ob);
            }
        }
    }
    if (!p.part) return;
#pragma unroll
    for (int j = 0; j < SL; ++j)
#pragma unroll
        for (int i = 0; i < V; ++i) {
            if (pa[j] >= 0) red[g][pa[j] * V + i] = da[j][i];
            if (pb[j] >= 0) red[g][pb[j] * V + i] = db[j][i];
        }
    __syncthreads();
    float* part = p.part + ((size_t)w * gridDim.x + blockIdx.x) * p.dim;
    for (int c = threadIdx.x; c < p.dim; c += kRopeThreads) {
        float s = 0.f;
        for (int q = 0; q < kGroups; ++q) s += red[q][c];
        part[c] = s;
    }
}

// dw[c] = sum over the `n` CTAs' partials, 8 warps a CTA, each a fixed share, 32 channels a CTA.
__global__ void __launch_bounds__(256)
    qk_norm_rope_dw_kernel(const float* __restrict__ part, int n, int dim, float* dq_weight, float* dk_weight) {
    __shared__ float red[8][32];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int c = blockIdx.x * 32 + lane, w = blockIdx.y;
    pdl_trigger();
    pdl_wait();
    float s = 0.f;
    if (c < dim)
        for (int i = warp; i < n; i += 8) s += part[((size_t)w * n + i) * dim + c];
    red[warp][lane] = s;
    __syncthreads();
    float* out = w ? dk_weight : dq_weight;
    if (warp == 0 && c < dim && out) {
        for (int i = 1; i < 8; ++i) s += red[i][lane];
        out[c] = s;
    }
}

// ------------------------------------------------------------------------------------ host

inline bool rope_piece_aligned(const void* p, long long stride, int es) {
    return (reinterpret_cast<uintptr_t>(p) & 15u) == 0 && (stride * es) % 16 == 0;
}

// Whether every head is made of 16-byte pieces that rotate together; others take the single-channel path.
inline bool rope_wide(const RopeParams& p, int es, bool bwd) {
    const int v = 16 / es;
    if (p.dim % v != 0 || p.dim > 2 * v * 32) return false;
    if (p.interleaved ? p.rot % v != 0 : (p.rot / 2) % v != 0) return false;
    for (int w = 0; w < 2; ++w) {
        if (p.heads[w] == 0) continue;
        if (!rope_piece_aligned(p.x[w], p.x_tok[w], es) || !rope_piece_aligned(p.out[w], p.out_tok[w], es)) return false;
        if (bwd && !rope_piece_aligned(p.dy[w], p.dy_tok[w], es)) return false;
    }
    return true;
}

template <bool BWD, typename T, int V, int G, int SL>
inline cudaError_t rope_go(const RopeParams& p, dim3 grid, cudaStream_t stream) {
    if constexpr (BWD) return launch_pdl(qk_norm_rope_bwd_kernel<T, V, G, SL>, grid, dim3(kRopeThreads), 0, stream, p);
    return launch_pdl(qk_norm_rope_kernel<T, V, G, SL>, grid, dim3(kRopeThreads), 0, stream, p);
}

template <bool BWD, typename T>
inline cudaError_t rope_launch(const RopeParams& p, dim3 grid, cudaStream_t stream) {
    constexpr int V = 16 / (int)sizeof(T);
    if (!rope_wide(p, (int)sizeof(T), BWD)) return rope_go<BWD, T, 1, 32, 4>(p, grid, stream);
    const int slots = (p.dim / V + 1) / 2;
    if (slots <= 4) return rope_go<BWD, T, V, 4, 1>(p, grid, stream);
    if (slots <= 8) return rope_go<BWD, T, V, 8, 1>(p, grid, stream);
    if (slots <= 16) return rope_go<BWD, T, V, 16, 1>(p, grid, stream);
    return rope_go<BWD, T, V, 32, 1>(p, grid, stream);
}

// CTAs per operand of the gradient kernel: a few per SM, each walking over many tokens, so that the weight
// gradients leave few partial sums.  Depends on the sizes only.
inline int rope_bwd_ctas(int tokens) {
    const int steps = (tokens + kRopeTok - 1) / kRopeTok;
    return steps < 148 * 4 ? steps : 148 * 4;
}

}  // namespace r2l
