// qk_norm_rope.cuh -- per-head RMS norm of queries and keys with the rotary position embedding, and its
// gradients.
//
// Bound by memory: every head is read once and written once (16-byte pieces).  A group of G lanes owns a token
// (or, for few tokens, a share of its heads) and walks over its heads.  Lane s holds the two pieces that rotate together
// (channels s V .. and rot / 2 + s V ..), the same ones in every head: the rotation needs no exchange, the norm one
// shuffle tree, and the token's angles and the weights stay in registers.  (Angles and weights in shared memory, read
// anew for every head, bound the kernel at 3.9 TB/s by bank conflicts.)  The heads ahead are on their way into a ring of
// shared memory that every lane has to itself, with no barrier: registers for them left too few bytes in flight
// (4.1 TB/s).  What was left was bound by what it issued (74 % of the slots): paired fp32 operations and addresses
// formed once a token took 32768 tokens of 24 heads of 128 from 81 to 72 us (5.6 TB/s), and the gradients of 16384 tokens
// from 66 to 64 us; there the ring runs on across tokens, three heads ahead: 61 us (4.9 TB/s, two CTAs an SM).
// The same bytes in fp32: 16384 tokens 70 us (5.8 TB/s), gradients of 8192 56 us (5.4 TB/s).  64 tokens take 4 us, a launch
// and one trip through memory.  Angles are formed in fp64 up to the fraction of a turn: position 100000 x frequency 1 leaves
// fp32 half a degree.
#pragma once

#include <algorithm>

#include "../common.cuh"
#include "pairs.cuh"

namespace r2l {

constexpr int kRopeThreads = 256;
constexpr int kRopeMaxDim = 256;
constexpr int kRopeAhead = 4;     // heads that a group has in flight, forward
constexpr int kRopeAheadBwd = 3;  // and in the gradients (two operands)

struct RopeParams {
    const void *x[2], *dy[2];   // queries, keys
    void* out[2];
    long long x_tok[2], out_tok[2], dy_tok[2];
    int heads[2];
    const float* weight[2];
    float* part;                // [2][gridDim.x][head_dim] partial weight gradients, or NULL
    const void* positions;
    const float* inv_freq;
    int tokens, dim, rot, interleaved, pos64;
    int split;                  // groups that share a token's heads (forward)
    float eps, inv_dim;
};

// A lane's values on their way from memory: N heads ahead, each of P pieces of V neighbouring channels (16 bytes for
// V > 1).  For V > 1 a ring in shared memory, filled by asynchronous copies; single channels are loaded when they are asked for.
template <typename T, int V, int N, int P>
struct RopeRing {
    uint4* mine;  // [N][P][kRopeThreads], this lane's column
    __device__ __forceinline__ RopeRing(uint4* ring) : mine(ring + threadIdx.x) {}
    // zeros unless `in`, and then src is not read
    __device__ __forceinline__ void fetch(int slot, int piece, const T* src, bool in) {
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_addr(mine + (slot * P + piece) * kRopeThreads)),
                     "l"(src), "r"(in ? 16 : 0)
                     : "memory");
    }
    __device__ __forceinline__ void commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
    // until at most N - 1 heads are on their way
    __device__ __forceinline__ void wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N - 1) : "memory"); }
    __device__ __forceinline__ void get(int slot, int piece, const T*, bool, float (&f)[V]) {
        const uint4 v = *(mine + (slot * P + piece) * kRopeThreads);
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (sizeof(T) == 4) {
                f[i] = __uint_as_float(w[i]);
            } else {
                f[2 * i] = __uint_as_float(w[i] << 16);
                f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
            }
        }
    }
};
template <typename T, int N, int P>
struct RopeRing<T, 1, N, P> {
    __device__ __forceinline__ RopeRing(uint4*) {}
    __device__ __forceinline__ void fetch(int, int, const T*, bool) {}
    __device__ __forceinline__ void commit() {}
    __device__ __forceinline__ void wait() {}
    __device__ __forceinline__ void get(int, int, const T* src, bool in, float (&f)[1]) { f[0] = in ? to_f32(*src) : 0.f; }
};
template <int V>
constexpr int rope_ring_bytes(int n, int p) {
    return V > 1 ? n * p * kRopeThreads * 16 : 0;
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

// The slot's angles: cos and sin (times sign) for the pair i of its channels, 1 and 0 where it does not rotate.
template <int V>
__device__ __forceinline__ void rope_angles(const RopeParams& p, int token, int a, int b, float sign, float (&co)[V], float (&si)[V]) {
    const bool inter = p.interleaved != 0;
    const double pos = p.rot == 0 ? 0.0
                       : p.pos64  ? (double)static_cast<const long long*>(p.positions)[token]
                                  : (double)static_cast<const int*>(p.positions)[token];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        int f;  // the pair's frequency
        if (!inter)
            f = a < p.rot / 2 / V ? a * V + i : -1;
        else if constexpr (V == 1)
            f = a < p.rot ? a >> 1 : -1;
        else if (i < V / 2)
            f = a * V < p.rot ? a * V / 2 + i : -1;
        else
            f = b * V < p.rot ? b * V / 2 + i - V / 2 : -1;
        co[i] = 1.f, si[i] = 0.f;
        if (a >= 0 && f >= 0) {
            const double turns = pos * (double)__ldg(p.inv_freq + f) * 0.15915494309189535;  // 1 / (2 pi)
            sincospif((float)(2.0 * (turns - rint(turns))), &si[i], &co[i]);
            si[i] *= sign;
        }
    }
}

template <int V>
__device__ __forceinline__ float2 rope_pair(const float (&x)[V], int i) {
    return make_float2(x[i], x[i + 1]);
}

// Rotates the slot's channels.
template <int V>
__device__ __forceinline__ void rope_rotate(float (&xa)[V], float (&xb)[V], int a, int b, int rot, bool inter, const float (&co)[V],
                                            const float (&si)[V]) {
    if constexpr (V == 1) {
        if (a >= 0 && (inter ? a < rot : a < rot / 2)) {
            const float u = xa[0], w = xb[0];
            xa[0] = u * co[0] - w * si[0];
            xb[0] = w * co[0] + u * si[0];
        }
    } else if (!inter) {
        if (a >= 0 && a < rot / 2 / V) {
#pragma unroll
            for (int i = 0; i < V; i += 2) {
                const float2 u = rope_pair(xa, i), w = rope_pair(xb, i), c = rope_pair(co, i), s = rope_pair(si, i);
                const float2 x = fma2(u, c, mul2(w, make_float2(-s.x, -s.y))), y = fma2(w, c, mul2(u, s));
                xa[i] = x.x, xa[i + 1] = x.y;
                xb[i] = y.x, xb[i + 1] = y.y;
            }
        }
    } else {
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            float(&x)[V] = half ? xb : xa;
            const int piece = half ? b : a;
            if (piece >= 0 && piece * V < rot) {
#pragma unroll
                for (int i = 0; i < V; i += 2) {
                    const float c = co[half * (V / 2) + i / 2], sn = si[half * (V / 2) + i / 2], u = x[i], w = x[i + 1];
                    x[i] = u * c - w * sn;
                    x[i + 1] = w * c + u * sn;
                }
            }
        }
    }
}

// s += the sum of a b, in two halves where V allows.
template <int V>
__device__ __forceinline__ void rope_dot(float2& s, const float (&a)[V], const float (&b)[V]) {
    if constexpr (V == 1) {
        s.x = fmaf(a[0], b[0], s.x);
    } else {
#pragma unroll
        for (int i = 0; i < V; i += 2) s = fma2(rope_pair(a, i), rope_pair(b, i), s);
    }
}

// y = a b
template <int V>
__device__ __forceinline__ void rope_times(float (&y)[V], const float (&a)[V], const float (&b)[V]) {
    if constexpr (V == 1) {
        y[0] = a[0] * b[0];
    } else {
#pragma unroll
        for (int i = 0; i < V; i += 2) {
            const float2 t = mul2(rope_pair(a, i), rope_pair(b, i));
            y[i] = t.x, y[i + 1] = t.y;
        }
    }
}

// y = (s a) b
template <int V>
__device__ __forceinline__ void rope_mul(float (&y)[V], float s, const float (&a)[V], const float (&b)[V]) {
    if constexpr (V == 1) {
        y[0] = s * a[0] * b[0];
    } else {
#pragma unroll
        for (int i = 0; i < V; i += 2) {
            const float2 t = mul2(mul2(make_float2(s, s), rope_pair(a, i)), rope_pair(b, i));
            y[i] = t.x, y[i + 1] = t.y;
        }
    }
}

// y += s a
template <int V>
__device__ __forceinline__ void rope_axpy(float (&y)[V], float s, const float (&a)[V]) {
    if constexpr (V == 1) {
        y[0] = fmaf(s, a[0], y[0]);
    } else {
#pragma unroll
        for (int i = 0; i < V; i += 2) {
            const float2 t = fma2(make_float2(s, s), rope_pair(a, i), rope_pair(y, i));
            y[i] = t.x, y[i + 1] = t.y;
        }
    }
}

// y += (s a) b
template <int V>
__device__ __forceinline__ void rope_fma(float (&y)[V], float s, const float (&a)[V], const float (&b)[V]) {
    if constexpr (V == 1) {
        y[0] = fmaf(s * a[0], b[0], y[0]);
    } else {
#pragma unroll
        for (int i = 0; i < V; i += 2) {
            const float2 t = fma2(mul2(make_float2(s, s), rope_pair(a, i)), rope_pair(b, i), rope_pair(y, i));
            y[i] = t.x, y[i + 1] = t.y;
        }
    }
}

// The slot's weights of operand w (ones where there are none).
template <int V>
__device__ __forceinline__ void rope_weight(const RopeParams& p, int w, int piece, float (&v)[V]) {
    const float* wt = p.weight[w];
    if (V >= 4 && piece >= 0 && wt && (reinterpret_cast<uintptr_t>(wt) & 15u) == 0) {
#pragma unroll
        for (int i = 0; i + 3 < V; i += 4) {
            const float4 a = __ldg(reinterpret_cast<const float4*>(wt + piece * V + i));
            v[i] = a.x, v[i + 1] = a.y, v[i + 2] = a.z, v[i + 3] = a.w;
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = wt && piece >= 0 ? __ldg(wt + piece * V + i) : 1.f;
}

template <int G>
__device__ __forceinline__ float rope_group_sum(float v) {
#pragma unroll
    for (int o = G / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// G lanes per head, SL slots per lane (SL > 1 only for single channels, V = 1).
template <typename T, int V, int G, int SL>
__global__ void __launch_bounds__(kRopeThreads, 3) qk_norm_rope_kernel(const __grid_constant__ RopeParams p) {
    constexpr int kGroups = kRopeThreads / G, U = kRopeAhead;
    const int s0 = threadIdx.x % G;
    const long long item = (long long)blockIdx.x * kGroups + threadIdx.x / G;
    const int ht = p.heads[0] + p.heads[1], per = (ht + p.split - 1) / p.split;
    const bool live = item < (long long)p.tokens * p.split;
    int token = live ? (int)item : 0, h0 = 0;
    if (p.split > 1 && live) {  // then tokens * split is small
        token = (int)item / p.split;
        h0 = ((int)item - token * p.split) * per;
    }
    const int hn = live ? min(per, ht - h0) : 0;  // this group's heads: h0 .. h0 + hn - 1 (queries first)
    const bool inter = p.interleaved != 0;
    int pa[SL], pb[SL];
#pragma unroll
    for (int j = 0; j < SL; ++j) rope_slot<V>(s0 + j * G, p.dim, p.rot, inter, pa[j], pb[j]);
    pdl_trigger();
    pdl_wait();

    extern __shared__ __align__(16) uint4 rope_ring[];
    RopeRing<T, V, U, 2> ring(rope_ring);
    // a token's heads, numbered through: queries, then keys (whose pointers count from the first query on)
    const T* xs[2];
    T* outs[2];
#pragma unroll
    for (int w = 0; w < 2; ++w) {
        const long long from = w ? -(long long)p.heads[0] * p.dim : 0;
        xs[w] = static_cast<const T*>(p.x[w]) + ((long long)token * p.x_tok[w] + from);
        outs[w] = static_cast<T*>(p.out[w]) + ((long long)token * p.out_tok[w] + from);
    }
    // head i of the group; behind the last one the token's first, which is not read there
    auto source = [&](int i) -> const T* {
        const int hh = i < hn ? h0 + i : 0;
        return (hh >= p.heads[0] ? xs[1] : xs[0]) + (long long)hh * p.dim;
    };
    auto fetch = [&](int slot, int i) {
        const T* x = source(i);
        ring.fetch(slot, 0, x + max(pa[0], 0) * V, i < hn && pa[0] >= 0);
        ring.fetch(slot, 1, x + max(pb[0], 0) * V, i < hn && pb[0] >= 0);
        ring.commit();
    };
#pragma unroll
    for (int u = 0; u < U; ++u) fetch(u, u);
    float co[SL][V], si[SL][V];
#pragma unroll
    for (int j = 0; j < SL; ++j) rope_angles<V>(p, token, pa[j], pb[j], 1.f, co[j], si[j]);
    float wa[SL][V], wb[SL][V];
    int wcur = -1;
    // the same count in the whole warp: the shuffles need all lanes
    int slot = 0;
    for (int i = 0; i < per; ++i) {
        const int hh = h0 + i, w = hh >= p.heads[0];
        float ya[SL][V], yb[SL][V];
        float2 ss = make_float2(0.f, 0.f);
        ring.wait();
        const T* x = V > 1 ? nullptr : source(i);
#pragma unroll
        for (int j = 0; j < SL; ++j) {
            ring.get(slot, 0, x + pa[j] * V, i < hn && pa[j] >= 0, ya[j]);
            ring.get(slot, 1, x + pb[j] * V, i < hn && pb[j] >= 0, yb[j]);
            rope_dot<V>(ss, ya[j], ya[j]);
            rope_dot<V>(ss, yb[j], yb[j]);
        }
        const float inv = rsqrtf(fmaf(rope_group_sum<G>(ss.x + ss.y), p.inv_dim, p.eps));
        fetch(slot, i + U);
        slot = slot + 1 == U ? 0 : slot + 1;
        if (i >= hn) continue;
        if (w != wcur) {
            wcur = w;
#pragma unroll
            for (int j = 0; j < SL; ++j) {
                rope_weight<V>(p, w, pa[j], wa[j]);
                rope_weight<V>(p, w, pb[j], wb[j]);
            }
        }
        T* out = (w ? outs[1] : outs[0]) + (long long)hh * p.dim;
#pragma unroll
        for (int j = 0; j < SL; ++j) {
            rope_mul<V>(ya[j], inv, wa[j], ya[j]);
            rope_mul<V>(yb[j], inv, wb[j], yb[j]);
            rope_rotate<V>(ya[j], yb[j], pa[j], pb[j], p.rot, inter, co[j], si[j]);
            if (pa[j] >= 0) rope_store<T, V>(out + pa[j] * V, ya[j]);
            if (pb[j] >= 0) rope_store<T, V>(out + pb[j] * V, yb[j]);
        }
    }
}

// Gradients of the queries (blockIdx.y 0) or keys (1).  With z = x / rms and u = the rotation taken back
// from dy: dx = (u w - z mean(u w z)) / rms, dw = sum of u z over tokens and heads.  A lane keeps its channels'
// share of dw in registers over all its heads; a CTA's groups add theirs in a fixed order at the end.
template <typename T, int V, int G, int SL>
__global__ void __launch_bounds__(kRopeThreads, 2) qk_norm_rope_bwd_kernel(const __grid_constant__ RopeParams p) {
    constexpr int kGroups = kRopeThreads / G;
    const int g = threadIdx.x / G, s0 = threadIdx.x % G;
    const int w = blockIdx.y, heads = p.heads[w];
    const bool inter = p.interleaved != 0;
    int pa[SL], pb[SL];
    float wa[SL][V], wb[SL][V], da[SL][V], db[SL][V];
    pdl_trigger();
    pdl_wait();
#pragma unroll
    for (int j = 0; j < SL; ++j) {
        rope_slot<V>(s0 + j * G, p.dim, p.rot, inter, pa[j], pb[j]);
        rope_weight<V>(p, w, pa[j], wa[j]);
        rope_weight<V>(p, w, pb[j], wb[j]);
#pragma unroll
        for (int i = 0; i < V; ++i) da[j][i] = db[j][i] = 0.f;
    }
    extern __shared__ __align__(16) uint4 rope_ring[];
    constexpr int U = kRopeAheadBwd;
    RopeRing<T, V, U, 4> ring(rope_ring);
    // A group walks over whole tokens, kGroups * gridDim.x apart (the same count in the whole CTA); the ring runs on from a
    // token's last head to the next one's first.
    const long long step = (long long)gridDim.x * kGroups;
    long long ft = (long long)blockIdx.x * kGroups + g;  // what is fetched next
    int fh = 0;
    auto fetch = [&](int slot) {
        const bool in = ft < p.tokens;
        const long long at = (long long)fh * p.dim, t = in ? ft : 0;
        const T* x = static_cast<const T*>(p.x[w]) + (in ? t * p.x_tok[w] + at : 0);
        const T* dy = static_cast<const T*>(p.dy[w]) + (in ? t * p.dy_tok[w] + at : 0);
        ring.fetch(slot, 0, x + max(pa[0], 0) * V, in && pa[0] >= 0);
        ring.fetch(slot, 1, x + max(pb[0], 0) * V, in && pb[0] >= 0);
        ring.fetch(slot, 2, dy + max(pa[0], 0) * V, in && pa[0] >= 0);
        ring.fetch(slot, 3, dy + max(pb[0], 0) * V, in && pb[0] >= 0);
        ring.commit();
        if (++fh == heads) fh = 0, ft += step;
    };
    if (heads > 0) {
#pragma unroll
        for (int u = 0; u < U; ++u) fetch(u);
    }
    int slot = 0;
    for (long long t0 = (long long)blockIdx.x * kGroups; t0 < p.tokens && heads > 0; t0 += step) {
        const bool live = t0 + g < p.tokens;
        const int token = live ? (int)(t0 + g) : 0;
        const T* x = static_cast<const T*>(p.x[w]) + (size_t)token * p.x_tok[w];
        const T* dy = static_cast<const T*>(p.dy[w]) + (size_t)token * p.dy_tok[w];
        T* out = static_cast<T*>(p.out[w]) + (size_t)token * p.out_tok[w];
        float co[SL][V], si[SL][V];
#pragma unroll
        for (int j = 0; j < SL; ++j) rope_angles<V>(p, token, pa[j], pb[j], -1.f, co[j], si[j]);
        for (int h = 0; h < heads; ++h) {
            float xa[SL][V], xb[SL][V], ua[SL][V], ub[SL][V];
            float2 ss = make_float2(0.f, 0.f), dot = ss;
            ring.wait();
            const long long at = (long long)h * p.dim;
#pragma unroll
            for (int j = 0; j < SL; ++j) {
                ring.get(slot, 0, x + at + pa[j] * V, live && pa[j] >= 0, xa[j]);
                ring.get(slot, 1, x + at + pb[j] * V, live && pb[j] >= 0, xb[j]);
                ring.get(slot, 2, dy + at + pa[j] * V, live && pa[j] >= 0, ua[j]);
                ring.get(slot, 3, dy + at + pb[j] * V, live && pb[j] >= 0, ub[j]);
                rope_rotate<V>(ua[j], ub[j], pa[j], pb[j], p.rot, inter, co[j], si[j]);
                rope_dot<V>(ss, xa[j], xa[j]);
                rope_dot<V>(ss, xb[j], xb[j]);
                float t[V];
                rope_times<V>(t, ua[j], wa[j]);
                rope_dot<V>(dot, t, xa[j]);
                rope_times<V>(t, ub[j], wb[j]);
                rope_dot<V>(dot, t, xb[j]);
            }
            const float inv = rsqrtf(fmaf(rope_group_sum<G>(ss.x + ss.y), p.inv_dim, p.eps));
            const float m = rope_group_sum<G>(dot.x + dot.y) * p.inv_dim * inv * inv;  // mean(u w z) / rms
            fetch(slot);
            slot = slot + 1 == U ? 0 : slot + 1;
            if (!live) continue;
#pragma unroll
            for (int j = 0; j < SL; ++j) {
                float oa[V], ob[V];
                rope_fma<V>(da[j], inv, xa[j], ua[j]);
                rope_fma<V>(db[j], inv, xb[j], ub[j]);
                // inv (u w - x m)
                rope_mul<V>(oa, inv, ua[j], wa[j]);
                rope_axpy<V>(oa, -inv * m, xa[j]);
                rope_mul<V>(ob, inv, ub[j], wb[j]);
                rope_axpy<V>(ob, -inv * m, xb[j]);
                if (pa[j] >= 0) rope_store<T, V>(out + (size_t)h * p.dim + pa[j] * V, oa);
                if (pb[j] >= 0) rope_store<T, V>(out + (size_t)h * p.dim + pb[j] * V, ob);
            }
        }
    }
    if (!p.part) return;
    // the groups' sums, where the ring was
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncthreads();
    float* red = reinterpret_cast<float*>(rope_ring);
#pragma unroll
    for (int j = 0; j < SL; ++j)
#pragma unroll
        for (int i = 0; i < V; ++i) {
            if (pa[j] >= 0) red[g * p.dim + pa[j] * V + i] = da[j][i];
            if (pb[j] >= 0) red[g * p.dim + pb[j] * V + i] = db[j][i];
        }
    __syncthreads();
    float* part = p.part + ((size_t)w * gridDim.x + blockIdx.x) * p.dim;
    for (int c = threadIdx.x; c < p.dim; c += kRopeThreads) {
        float s = 0.f;
        for (int q = 0; q < kGroups; ++q) s += red[q * p.dim + c];
        part[c] = s;
    }
}

// dw[c] = sum over the `n` CTAs' partials, 32 warps a CTA, each a fixed share, 32 channels a CTA.
constexpr int kRopeDwThreads = 1024;
__global__ void __launch_bounds__(kRopeDwThreads)
    qk_norm_rope_dw_kernel(const float* __restrict__ part, int n, int dim, float* dq_weight, float* dk_weight) {
    __shared__ float red[32][32];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int c = blockIdx.x * 32 + lane, w = blockIdx.y;
    pdl_trigger();
    pdl_wait();
    float s = 0.f;
    if (c < dim)
#pragma unroll 5
        for (int i = warp; i < n; i += 32) s += part[((size_t)w * n + i) * dim + c];
    red[warp][lane] = s;
    __syncthreads();
    float* out = w ? dk_weight : dq_weight;
    if (warp == 0 && c < dim && out) {
        for (int i = 1; i < 32; ++i) s += red[i][lane];
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

// Groups of a CTA for heads of these parameters: as rope_launch chooses them.
inline int rope_lanes(const RopeParams& p, int es, bool bwd) {
    if (!rope_wide(p, es, bwd)) return 32;
    const int v = 16 / es, slots = (p.dim / v + 1) / 2;
    return slots <= 4 ? 4 : slots <= 8 ? 8 : slots <= 16 ? 16 : 32;
}

// Groups per token in the forward kernel: one, which forms the token's angles once, when the tokens alone fill the SMs
// (768 threads each) twice; for fewer tokens the heads are shared out, up to a group each, and each forms the angles.
inline int rope_split(int tokens, int heads, int lanes, int nsm) {
    const long long threads = (long long)tokens * lanes, want = 2LL * nsm * 768;
    const long long split = threads >= want ? 1 : (want + threads - 1) / threads;
    return (int)(split < heads ? split : heads);
}

// CTAs per operand of the gradient kernel: at most two per SM (a wave of both operands), each walking over many
// tokens, so that the weight gradients leave few partial sums.  Depends on the sizes only.
inline int rope_bwd_ctas(int tokens, int lanes) {
    const long long ctas = ((long long)tokens * lanes + kRopeThreads - 1) / kRopeThreads;
    return (int)(ctas < 148 * 2 ? ctas : 148 * 2);
}

template <bool BWD, typename T, int V, int G, int SL>
inline cudaError_t rope_go(const RopeParams& p, int ctas, cudaStream_t stream) {
    if constexpr (BWD) {
        const int sums = kRopeThreads / G * p.dim * (int)sizeof(float), smem = std::max(rope_ring_bytes<V>(kRopeAheadBwd, 4), sums);
        auto kernel = qk_norm_rope_bwd_kernel<T, V, G, SL>;
        if (prepare_kernel_smem(reinterpret_cast<const void*>(kernel), smem) != 0) return cudaErrorInvalidValue;
        return launch_pdl(kernel, dim3((unsigned)ctas, 2), dim3(kRopeThreads), (size_t)smem, stream, p);
    } else {
        const long long n = ((long long)p.tokens * p.split * G + kRopeThreads - 1) / kRopeThreads;
        return launch_pdl(qk_norm_rope_kernel<T, V, G, SL>, dim3((unsigned)n), dim3(kRopeThreads),
                          (size_t)rope_ring_bytes<V>(kRopeAhead, 2), stream, p);
    }
}

// ctas: of the gradient kernel, per operand.
template <bool BWD, typename T>
inline cudaError_t rope_launch(const RopeParams& p, int ctas, cudaStream_t stream) {
    constexpr int V = 16 / (int)sizeof(T);
    if (!rope_wide(p, (int)sizeof(T), BWD)) return rope_go<BWD, T, 1, 32, 4>(p, ctas, stream);
    switch (rope_lanes(p, (int)sizeof(T), BWD)) {
        case 4: return rope_go<BWD, T, V, 4, 1>(p, ctas, stream);
        case 8: return rope_go<BWD, T, V, 8, 1>(p, ctas, stream);
        case 16: return rope_go<BWD, T, V, 16, 1>(p, ctas, stream);
        default: return rope_go<BWD, T, V, 32, 1>(p, ctas, stream);
    }
}

}  // namespace r2l
