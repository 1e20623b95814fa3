// linattn_block.cuh -- linear attention over blocks of at most 64 tokens (bf16), without and with a state: the
// right-to-left pass over the active block of parallel decoding, a block resumed from the cached state of its prefix, and
// their gradients.
//
// Without a state the operator is  y_i = s sum over j not behind i of gamma^|i - j| (q_i . k_j) v_j,  one small tile per
// (block, head).  It is bound by memory: 16 tokens of d = 128 move 16 KB and take 0.4 MFLOP.  What counts is bytes in
// flight and no serial chain, so a warp owns 16 query rows, its CTA's whole tiles are fetched at once (48 KB for
// d = 128, four CTAs an SM) and the products are warp-level MMAs: the tcgen05 kernel, one tile at a time through
// its pipeline of roles, takes 2.8 us a tile and SM, 79 us for 4096 blocks of 16 tokens; this one 18.7 us (3.6 TB/s).
//
// With a state (64 KB in and out for d = 128, against 16 KB of tokens) it is a stream over the states, with products in
// between.  Persistent CTAs, a warp per 16 value channels: S^T lies in registers as the accumulator of an MMA, a layout
// that is also the B operand's of the next product, so that S meets Q (in two bf16 parts) and takes up V^T K~ (K~ in
// three, split once a CTA) without being moved.  The next state is fetched into shared memory meanwhile.  1024 states
// of 128 x 128 and 16 tokens each: 36 us (4.2 TB/s; 65 us in the tcgen05 kernel, whose CTAs load, compute and store in
// turn), and 17 us for every 16 tokens more, bound by the instructions of the splits and the legacy MMA's rate
// (measured: one m16n8k16 in 8.6 cycles a quarter of an SM).  For heads of 128 x 64 it spills 56 bytes at 168 registers.
//
// P is split into two bf16 parts, as in the chunk kernel.  A masked key is a zero weight, and zero times an infinity
// is NaN: outputs that come out not finite are summed again with zeros in place of V's non-finite values (the same sums,
// to the bit, where those were masked), and one by one over the unmasked keys where they were not.
#pragma once

#include "linattn_common.cuh"
#include "linattn_rec.cuh"

namespace r2l {

constexpr int kBlkMaxTok = 64;  // without a state
constexpr int kBlkThreads = 128;

__device__ __forceinline__ void blk_mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void blk_ldm(uint32_t saddr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(saddr)
                 : "memory");
}
__device__ __forceinline__ void blk_ldm_trans(uint32_t saddr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(saddr)
                 : "memory");
}
__device__ __forceinline__ uint32_t blk_pack(float lo, float hi) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ float blk_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float blk_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// Byte offset of the 16-byte piece c of a token's row of D channels: pieces permuted within 128 bytes by the row, so that
// eight rows of one piece lie in different banks.
template <int D>
__device__ __forceinline__ uint32_t blk_off(int row, int c) {
    return (uint32_t)(row * (D * 2) + ((c & ~7) | ((c ^ row) & 7)) * 16);
}

// One output that came out not finite: the sum over the unmasked keys alone, from the tiles.  Not inlined: it is rare.
template <int D>
__device__ __noinline__ float blk_redo(const unsigned char* tiles, int bytes, const float* wtab, int i, int ch, int j0, int j1) {
    float acc = 0.f;
#pragma unroll 1
    for (int j = j0; j < j1; ++j) {
        float s = 0.f;
#pragma unroll 1
        for (int c = 0; c < D / 2; ++c) {
            const uint32_t a = *reinterpret_cast<const uint32_t*>(tiles + blk_off<D>(i, c >> 2) + (c & 3) * 4);
            const uint32_t b = *reinterpret_cast<const uint32_t*>(tiles + bytes + blk_off<D>(j, c >> 2) + (c & 3) * 4);
            s = fmaf(blk_lo(a), blk_lo(b), fmaf(blk_hi(a), blk_hi(b), s));
        }
        const float v = __bfloat162float(
            *reinterpret_cast<const __nv_bfloat16*>(tiles + 2 * bytes + blk_off<D>(j, ch >> 3) + (ch & 7) * 2));
        acc = fmaf(s * wtab[i > j ? i - j : j - i], v, acc);
    }
    return acc;
}

// Weighted, masked scores of rows r0 .. and keys k0 .. (16 each), in two bf16 parts, as A fragments over the keys.
template <int D>
__device__ __forceinline__ void blk_scores(uint32_t qs, uint32_t ks, const float* wtab, int r0, int k0, int reverse,
                                           uint32_t (&hi)[4], uint32_t (&lo)[4]) {
    const int lane = threadIdx.x & 31, fr = lane >> 2, fc = (lane & 3) * 2;
    float sc[2][4] = {};
#pragma unroll
    for (int k = 0; k < D / 16; ++k) {
        uint32_t a[4], b[4];
        blk_ldm(qs + blk_off<D>(r0 + (lane & 15), 2 * k + (lane >> 4)), a);
        blk_ldm(ks + blk_off<D>(k0 + (lane & 7) + ((lane >> 4) << 3), 2 * k + ((lane >> 3) & 1)), b);
        blk_mma(sc[0], a, b[0], b[1]);
        blk_mma(sc[1], a, b[2], b[3]);
    }
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int e = 0; e < 4; e += 2) {
            float x[2];
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                const int i = r0 + fr + (e ? 8 : 0), j = k0 + t * 8 + fc + b, d = reverse ? j - i : i - j;
                x[b] = d >= 0 ? sc[t][e + b] * wtab[d & 63] : 0.f;
            }
            const uint32_t u = blk_pack(x[0], x[1]);
            hi[t * 2 + e / 2] = u;
            lo[t * 2 + e / 2] = blk_pack(x[0] - blk_lo(u), x[1] - blk_hi(u));
        }
}

__device__ __forceinline__ bool blk_finite(float x) { return x * 0.f == 0.f; }

// One step of P V with V's non-finite values (fragments b) taken as zeros; cnt: how many of them a row does not mask.
__device__ __forceinline__ void blk_clean_step(float (&o)[2][4], float (&cnt)[2][4], const uint32_t (&hi)[4], const uint32_t (&lo)[4],
                                               const uint32_t (&b)[4], int r0, int k0, int reverse) {
    const int lane = threadIdx.x & 31, fr = lane >> 2, fc = (lane & 3) * 2;
    uint32_t m[4], v[4], f[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const int i = r0 + fr + (e & 1) * 8, j = k0 + (e >> 1) * 8 + fc;
        const int d = reverse ? j - i : i - j, d1 = reverse ? d + 1 : d - 1;
        m[e] = (d >= 0 ? 0x3F80u : 0u) | (d1 >= 0 ? 0x3F800000u : 0u);
        const bool x = (b[e] & 0x7F80u) == 0x7F80u, y = (b[e] & 0x7F800000u) == 0x7F800000u;
        v[e] = b[e] & ((x ? 0u : 0xFFFFu) | (y ? 0u : 0xFFFF0000u));
        f[e] = (x ? 0x3F80u : 0u) | (y ? 0x3F800000u : 0u);
    }
    blk_mma(o[0], hi, v[0], v[1]);
    blk_mma(o[1], hi, v[2], v[3]);
    blk_mma(o[0], lo, v[0], v[1]);
    blk_mma(o[1], lo, v[2], v[3]);
    blk_mma(cnt[0], m, f[0], f[1]);
    blk_mma(cnt[1], m, f[2], f[3]);
}

// Fetches rows 0 .. lp - 1 of a tile (D channels a row, zeros past `len` rows and d channels) into shared memory.
template <int D>
__device__ __forceinline__ void blk_fetch(uint32_t dst, const __nv_bfloat16* src, long long tok, int lp, int len, int d,
                                          int threads = kBlkThreads) {
    for (int i = threadIdx.x; i < lp * (D / 8); i += threads) {
        const int row = i / (D / 8), c = i % (D / 8);
        const bool in = row < len && c * 8 < d;
        const __nv_bfloat16* a = in ? src + (size_t)row * tok + c * 8 : src;
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst + blk_off<D>(row, c)), "l"(a), "r"(in ? 16 : 0)
                     : "memory");
    }
}

// The 16 x 16 outputs of rows r0 .. and channels c0 .., where not all are finite (z: those of the two fragments).
template <int D>
__device__ __noinline__ void blk_redo_tile(const unsigned char* tiles, int bytes, const float* wtab, int r0, int c0, int kb0, int kb1,
                                           int len, int reverse, float (&z)[8]) {
    const int lane = threadIdx.x & 31, fr = lane >> 2, fc = (lane & 3) * 2;
    const uint32_t qs = smem_addr(tiles), ks = qs + bytes, vs = ks + bytes;
    float o[2][4] = {}, cnt[2][4] = {};
#pragma unroll 1
    for (int kb = kb0; kb < kb1; ++kb) {
        uint32_t hi[4], lo[4], b[4];
        blk_scores<D>(qs, ks, wtab, r0, kb * 16, reverse, hi, lo);
        blk_ldm_trans(vs + blk_off<D>(kb * 16 + (lane & 15), c0 / 8 + (lane >> 4)), b);
        blk_clean_step(o, cnt, hi, lo, b, r0, kb * 16, reverse);
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const int i = r0 + fr + ((e >> 1) & 1) * 8;
        const float x = o[e >> 2][e & 3];
        if (i >= len)
            z[e] = 0.f;
        else if (!blk_finite(z[e]))
            z[e] = cnt[e >> 2][e & 3] == 0.f && blk_finite(x)
                       ? x
                       : blk_redo<D>(tiles, bytes, wtab, i, c0 + (e >> 2) * 8 + fc + (e & 1), reverse ? i : 0, reverse ? len : i + 1);
    }
}

// Rows r0 .. of an item, some of whose outputs came out not finite, done again and stored.  Out of line as a whole: the
// usual path's registers are all taken.
template <int D>
__device__ __noinline__ void blk_redo_rows(const LaPass& p, const unsigned char* tiles, int bytes, const float* wtab, int seq, int h, int r0,
                                           int kb0, int kb1, int len) {
    const int lane = threadIdx.x & 31, fr = lane >> 2, fc = (lane & 3) * 2;
    const size_t y0 = ((size_t)seq * p.seq_len + r0) * p.y_tok + (size_t)h * p.dv;
#pragma unroll 1
    for (int c0 = 0; c0 < p.dv; c0 += 16) {
        float z[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) z[e] = __int_as_float(0x7FC00000);  // all of them
        blk_redo_tile<D>(tiles, bytes, wtab, r0, c0, kb0, kb1, len, p.reverse, z);
#pragma unroll
        for (int e = 0; e < 8; e += 2) {
            const int i = fr + ((e >> 1) & 1) * 8, c = c0 + (e >> 2) * 8 + fc;
            if (r0 + i >= p.seq_len || c >= p.dv) continue;
            const size_t at = y0 + (size_t)i * p.y_tok + c;
            if (p.y_f32)
                *reinterpret_cast<float2*>(static_cast<float*>(p.y) + at) = make_float2(z[e], z[e + 1]);
            else
                *reinterpret_cast<uint32_t*>(static_cast<__nv_bfloat16*>(p.y) + at) = blk_pack(z[e], z[e + 1]);
        }
    }
}

// wpi: warps (of 16 rows) per item; per_cta: items per CTA.
template <int D>
__global__ void __launch_bounds__(kBlkThreads, 4) linattn_block_kernel(const __grid_constant__ LaPasses passes, int wpi, int per_cta) {
    extern __shared__ __align__(128) unsigned char blk_smem[];
    __shared__ float wtab[kBlkThreads / 32][kBlkMaxTok];
    const LaPass& p = passes.p[blockIdx.z];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int lp = wpi * 16, bytes = lp * D * 2;  // of one of an item's three tiles: q, k, v
    const long long nitems = (long long)p.nseq * p.heads, item0 = (long long)blockIdx.x * per_cta;
    pdl_trigger();
    pdl_wait();

    for (int s = 0; s < per_cta && item0 + s < nitems; ++s) {
        const int seq = (int)((item0 + s) / p.heads), h = (int)((item0 + s) - (long long)seq * p.heads);
        const int len = la_len(p, seq);
        const size_t tok0 = (size_t)seq * p.seq_len;
        const uint32_t dst = smem_addr(blk_smem) + (uint32_t)s * 3 * bytes;
        blk_fetch<D>(dst, static_cast<const __nv_bfloat16*>(p.q) + tok0 * p.q_tok + (size_t)(h / p.q_div) * p.dk, p.q_tok, lp, len, p.dk);
        blk_fetch<D>(dst + bytes, static_cast<const __nv_bfloat16*>(p.k) + tok0 * p.k_tok + (size_t)(h / p.k_div) * p.dk, p.k_tok, lp,
                     len, p.dk);
        blk_fetch<D>(dst + 2 * bytes, static_cast<const __nv_bfloat16*>(p.v) + tok0 * p.v_tok + (size_t)(h / p.v_div) * p.dv, p.v_tok,
                     lp, len, p.dv);
        // s_in s_out gamma^d
        if (tid < kBlkMaxTok) wtab[s][tid] = p.s_in * p.s_out * la_decay_pow(la_clamp_decay(p.log_decay[h]), (float)tid);
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncthreads();

    const int s = warp / wpi, w = warp - s * wpi, r0 = w * 16;
    if (s >= per_cta || item0 + s >= nitems) return;
    const int seq = (int)((item0 + s) / p.heads), h = (int)((item0 + s) - (long long)seq * p.heads);
    const int len = la_len(p, seq);
    unsigned char* tiles = blk_smem + (size_t)s * 3 * bytes;
    const uint32_t qs = smem_addr(tiles), ks = qs + bytes, vs = ks + bytes;
    const int fr = lane >> 2, fc = (lane & 3) * 2;
    float o[D / 8][4];
#pragma unroll
    for (int n = 0; n < D / 8; ++n) o[n][0] = o[n][1] = o[n][2] = o[n][3] = 0.f;
    const int kb0 = p.reverse ? w : 0, kb1 = p.reverse ? wpi : w + 1;
    for (int kb = kb0; kb < kb1; ++kb) {
        uint32_t hi[4], lo[4];
        blk_scores<D>(qs, ks, wtab[s], r0, kb * 16, p.reverse, hi, lo);
#pragma unroll
        for (int n = 0; n < D / 16; ++n) {
            uint32_t b[4];
            blk_ldm_trans(vs + blk_off<D>(kb * 16 + (lane & 15), 2 * n + (lane >> 4)), b);
            blk_mma(o[2 * n], hi, b[0], b[1]);
            blk_mma(o[2 * n + 1], hi, b[2], b[3]);
            blk_mma(o[2 * n], lo, b[0], b[1]);
            blk_mma(o[2 * n + 1], lo, b[2], b[3]);
        }
    }
    float any = 0.f;
#pragma unroll
    for (int n = 0; n < D / 8; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) any = fmaf(o[n][e], 0.f, any);  // NaN once anything is not finite
    if (__any_sync(0xffffffffu, any != 0.f)) {
        blk_redo_rows<D>(p, tiles, bytes, wtab[s], seq, h, r0, kb0, kb1, len);
        return;
    }
    const size_t y0 = ((size_t)seq * p.seq_len + r0) * p.y_tok + (size_t)h * p.dv;
    if (p.y_f32) {
        float* y = static_cast<float*>(p.y) + y0;
#pragma unroll
        for (int n = 0; n < D / 8; ++n)
#pragma unroll
            for (int e = 0; e < 4; e += 2) {
                const int i = fr + (e ? 8 : 0), c = n * 8 + fc;
                if (r0 + i < p.seq_len && c < p.dv) *reinterpret_cast<float2*>(y + (size_t)i * p.y_tok + c) = make_float2(o[n][e], o[n][e + 1]);
            }
        return;
    }
    // through the warp's own query rows, which nobody else reads, to 16-byte stores of whole rows
    __syncwarp();
#pragma unroll
    for (int n = 0; n < D / 8; ++n)
#pragma unroll
        for (int e = 0; e < 4; e += 2)
            *reinterpret_cast<uint32_t*>(tiles + blk_off<D>(r0 + fr + (e ? 8 : 0), n) + fc * 2) = blk_pack(o[n][e], o[n][e + 1]);
    __syncwarp();
    __nv_bfloat16* y = static_cast<__nv_bfloat16*>(p.y) + y0;
#pragma unroll
    for (int i = lane; i < 16 * (D / 8); i += 32) {
        const int row = i / (D / 8), c = i % (D / 8);
        if (r0 + row < p.seq_len && c * 8 < p.dv)
            *reinterpret_cast<uint4*>(y + (size_t)row * p.y_tok + c * 8) = *reinterpret_cast<const uint4*>(tiles + blk_off<D>(r0 + row, c));
    }
}

// A block with a state before it, or one wanted behind it, 16 tokens at a time.
template <int DK, int DV>
struct ResumeCfg {
    static constexpr int D = DK > DV ? DK : DV;         // channels of a tile's rows
    static constexpr int Tile = 16 * D * 2;             // q, k, v of an item; a part of K~
    static constexpr int Tokens = DK * DV * 4;          // two sets of (q, k, v) behind the state
    static constexpr int Keys = Tokens + 6 * Tile;      // K~ in three parts
    static constexpr int P = Keys + 3 * Tile;           // P in two
    static constexpr int Bytes = P + 2 * 16 * 32;
    static constexpr int Threads = 2 * DV;              // a warp per 16 value channels
    static constexpr int Fit = 224 * 1024 / (Bytes + 2048), Ctas = Fit < 256 / DV ? Fit : 256 / DV;  // of an SM
};

template <int DK, int DV>
__global__ void __launch_bounds__(2 * DV, ResumeCfg<DK, DV>::Ctas) linattn_resume_kernel(const __grid_constant__ LaPass p) {
    using Cfg = ResumeCfg<DK, DV>;
    constexpr int D = Cfg::D, KT = DK / 8;  // this warp's S^T: 16 value channels x KT tiles of 8 key channels
    extern __shared__ __align__(128) unsigned char blk_smem[];
    __shared__ float wtabs[2][16], gtabs[2][17];  // s_in s_out gamma^d, gamma^d
    __shared__ float2 gns[2];                     // gamma^n
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int fr = lane >> 2, fc = (lane & 3) * 2, c0 = warp * 16, ch = c0 + 2 * fr;
    const int nitems = p.nseq * p.heads, nrow = (p.seq_len + 15) >> 4;
    const uint32_t smem = smem_addr(blk_smem), kts = smem + Cfg::Keys, ps = smem + Cfg::P;
    pdl_trigger();
    pdl_wait();

    // the tokens of 16 rows, the c-th in scan order; an item's state
    auto fetch = [&](int item, int c, int buf) {
        const int seq = item / p.heads, h = item - seq * p.heads, r0 = 16 * (p.reverse ? nrow - 1 - c : c);
        const int n = min(max(la_len(p, seq) - r0, 0), 16);
        const size_t tok0 = (size_t)seq * p.seq_len + r0;
        const uint32_t dst = smem + Cfg::Tokens + buf * 3 * Cfg::Tile;
        blk_fetch<D>(dst, static_cast<const __nv_bfloat16*>(p.q) + tok0 * p.q_tok + (size_t)(h / p.q_div) * p.dk, p.q_tok, 16, n, p.dk,
                     Cfg::Threads);
        blk_fetch<D>(dst + Cfg::Tile, static_cast<const __nv_bfloat16*>(p.k) + tok0 * p.k_tok + (size_t)(h / p.k_div) * p.dk, p.k_tok,
                     16, n, p.dk, Cfg::Threads);
        blk_fetch<D>(dst + 2 * Cfg::Tile, static_cast<const __nv_bfloat16*>(p.v) + tok0 * p.v_tok + (size_t)(h / p.v_div) * p.dv,
                     p.v_tok, 16, n, p.dv, Cfg::Threads);
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    auto fetch_state = [&](int item) {
        if (p.h0) {  // rows of 16-byte pieces, permuted so that rows 0, 2, 4, 6 of a piece lie in different banks
            const float* a = p.h0 + (size_t)item * p.dk * p.dv;
#pragma unroll
            for (int m = 0; m < DK / 8; ++m) {
                const int i = tid + m * Cfg::Threads, k = i / (DV / 4), c = i % (DV / 4);
                const bool in = k < p.dk && c * 4 < p.dv;
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem + k * DV * 4 + (c ^ (k & 6)) * 16),
                             "l"(in ? a + k * p.dv + c * 4 : a), "r"(in ? 16 : 0)
                             : "memory");
            }
        }
    };
    if ((int)blockIdx.x < nitems) {
        fetch_state(blockIdx.x);
        fetch(blockIdx.x, 0, 0);
    }

    // S[t]: value channels ch (0, 1) and ch + 1 (2, 3), key channels 8 t + fc and the next
    float S[KT][4];
    int buf = 0, c = 0;
    for (int item = blockIdx.x; item < nitems; buf ^= 1) {
        const int seq = item / p.heads, h = item - seq * p.heads, r0 = 16 * (p.reverse ? nrow - 1 - c : c);
        const int len = min(max(la_len(p, seq) - r0, 0), 16);  // of these rows
        const bool first = c == 0, last = c == nrow - 1;
        unsigned char* const tiles = blk_smem + Cfg::Tokens + buf * 3 * Cfg::Tile;
        const uint32_t qs = smem_addr(tiles), ks = qs + Cfg::Tile, vs = ks + Cfg::Tile;
        float *wtab = wtabs[buf], *gtab = gtabs[buf];
        const float g = la_clamp_decay(p.log_decay[h]);
        if (tid < 17) {
            const float w = la_decay_pow_of(g, (float)tid);
            gtab[tid] = w;
            if (tid < 16) wtab[tid] = p.s_in * p.s_out * w;
        } else if (tid == 32) {
            gns[buf] = la_decay_pair_of(g, (float)len);
        }
        if (first)
            asm volatile("cp.async.wait_all;" ::: "memory");
        else
            asm volatile("cp.async.wait_group 1;" ::: "memory");  // the next item's state may still be on its way
        __syncthreads();
        if (first)
#pragma unroll
            for (int t = 0; t < KT; ++t) {
                const unsigned char* a = blk_smem + (8 * t + fc) * DV * 4 + ((ch >> 2) ^ (fc & 6)) * 16 + (fr & 1) * 8;
                float2 x = make_float2(0.f, 0.f), y = x;
                if (p.h0) {
                    x = *reinterpret_cast<const float2*>(a);
                    y = *reinterpret_cast<const float2*>(a + DV * 4);
                }
                S[t][0] = x.x, S[t][1] = y.x, S[t][2] = x.y, S[t][3] = y.y;
            }
        // what all warps share: P (one warp), V and K~
        if (warp == DV / 16 - 1) {
            uint32_t hi[4], lo[4];
            blk_scores<D>(qs, ks, wtab, 0, 0, p.reverse, hi, lo);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const uint32_t at = ps + (fr + (e & 1) * 8) * 32 + (e >> 1) * 16 + fc * 2;
                asm volatile("st.shared.b32 [%0], %1;" ::"r"(at), "r"(hi[e]) : "memory");
                asm volatile("st.shared.b32 [%0], %1;" ::"r"(at + 512), "r"(lo[e]) : "memory");
            }
        } else if (tid < DV) {
            // of every 16 value channels the even ones first: a thread's two rows of S^T are then neighbouring channels
            const int row = tid / (DV / 16), c = 2 * (tid % (DV / 16));
            uint4 *x = reinterpret_cast<uint4*>(tiles + 2 * Cfg::Tile + blk_off<D>(row, c)),
                  *y = reinterpret_cast<uint4*>(tiles + 2 * Cfg::Tile + blk_off<D>(row, c + 1));
            const uint4 a = *x, b = *y;
            *x = make_uint4(__byte_perm(a.x, a.y, 0x5410), __byte_perm(a.z, a.w, 0x5410), __byte_perm(b.x, b.y, 0x5410),
                            __byte_perm(b.z, b.w, 0x5410));
            *y = make_uint4(__byte_perm(a.x, a.y, 0x7632), __byte_perm(a.z, a.w, 0x7632), __byte_perm(b.x, b.y, 0x7632),
                            __byte_perm(b.z, b.w, 0x7632));
        }
        const bool update = p.h_last || !last;
        if (update) {
            for (int i = tid; i < 16 * (DK / 8); i += Cfg::Threads) {
                const int j = i / (DK / 8), off = blk_off<D>(j, i % (DK / 8));
                const float w = j < len ? p.s_in * gtab[p.reverse ? j : len - 1 - j] : 0.f;
                const uint4 a = *reinterpret_cast<const uint4*>(tiles + Cfg::Tile + off);
                const uint32_t u[4] = {a.x, a.y, a.z, a.w};
                float x[8];
#pragma unroll
                for (int e = 0; e < 4; ++e) x[2 * e] = blk_lo(u[e]) * w, x[2 * e + 1] = blk_hi(u[e]) * w;
#pragma unroll
                for (int part = 0; part < 3; ++part) {
                    uint32_t o[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        o[e] = blk_pack(x[2 * e], x[2 * e + 1]);
                        x[2 * e] -= blk_lo(o[e]);
                        x[2 * e + 1] -= blk_hi(o[e]);
                    }
                    *reinterpret_cast<uint4*>(blk_smem + Cfg::Keys + part * Cfg::Tile + off) = make_uint4(o[0], o[1], o[2], o[3]);
                }
            }
        }
        __syncthreads();
        if (!last)
            fetch(item, c + 1, buf ^ 1);
        else if (item + (int)gridDim.x < nitems)
            fetch(item + gridDim.x, 0, buf ^ 1);
        if (first && item + (int)gridDim.x < nitems) fetch_state(item + gridDim.x);
        asm volatile("cp.async.commit_group;" ::: "memory");

        float o[2][4] = {}, a2[2][4] = {};
        if (p.h0 || !first) {
#pragma unroll
            for (int k = 0; k < DK / 16; ++k) {
                uint32_t a[4];
                blk_ldm(qs + blk_off<D>(lane & 15, 2 * k + (lane >> 4)), a);
#pragma unroll
                for (int n = 0; n < 2; ++n) {
                    const float *x = &S[2 * k][n * 2], *y = &S[2 * k + 1][n * 2];
                    const uint32_t b0 = la_pack_sat(x[0], x[1]), b1 = la_pack_sat(y[0], y[1]);
                    blk_mma(o[n], a, b0, b1);
                    blk_mma(a2[n], a, blk_pack(x[0] - blk_lo(b0), x[1] - blk_hi(b0)), blk_pack(y[0] - blk_lo(b1), y[1] - blk_hi(b1)));
                }
            }
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const int i = fr + 8 * u;
                const float f = i < len ? p.s_out * gtab[(p.reverse ? len - 1 - i : i) + 1] : 0.f;
#pragma unroll
                for (int n = 0; n < 2; ++n)
#pragma unroll
                    for (int e = 2 * u; e < 2 * u + 2; ++e) o[n][e] = f * (o[n][e] + a2[n][e]), a2[n][e] = 0.f;
            }
        }
        {
            uint32_t hi[4], lo[4], b[4];
            blk_ldm(ps + (lane & 15) * 32 + (lane >> 4) * 16, hi);
            blk_ldm(ps + 512 + (lane & 15) * 32 + (lane >> 4) * 16, lo);
            blk_ldm_trans(vs + blk_off<D>(lane & 15, c0 / 8 + (lane >> 4)), b);
            blk_mma(a2[0], hi, b[0], b[1]);
            blk_mma(a2[1], hi, b[2], b[3]);
            blk_mma(a2[0], lo, b[0], b[1]);
            blk_mma(a2[1], lo, b[2], b[3]);
            float any = 0.f;
#pragma unroll
            for (int n = 0; n < 2; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) any = fmaf(a2[n][e], 0.f, any);
            if (__any_sync(0xffffffffu, any != 0.f)) {
                float z[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) z[e] = a2[e >> 2][e & 3];
                blk_redo_tile<D>(tiles, Cfg::Tile, wtab, 0, c0, 0, 1, len, p.reverse, z);
#pragma unroll
                for (int e = 0; e < 8; ++e) a2[e >> 2][e & 3] = z[e];
            }
        }
        // four neighbouring channels a thread
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const int row = fr + 8 * u, cv = c0 + 2 * fc;
            float x[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
                x[e] = row < len ? o[e & 1][2 * u + (e >> 1)] + a2[e & 1][2 * u + (e >> 1)] : 0.f;
            if (r0 + row < p.seq_len && cv < p.dv)
                *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.y) + ((size_t)seq * p.seq_len + r0 + row) * p.y_tok +
                                          (size_t)h * p.dv + cv) = make_uint2(blk_pack(x[0], x[1]), blk_pack(x[2], x[3]));
        }
        if (update && len > 0) {
            // S^T = gamma^n S^T + V^T K~
            const float2 gn = gns[buf];
            uint32_t a[4];
            blk_ldm_trans(vs + blk_off<D>((lane & 7) + ((lane >> 4) << 3), c0 / 8 + ((lane >> 3) & 1)), a);
#pragma unroll
            for (int t = 0; t < KT; t += 2) {
#pragma unroll
                for (int u = t; u < t + 2; ++u)
#pragma unroll
                    for (int e = 0; e < 4; ++e) S[u][e] = fmaf(S[u][e], gn.x, S[u][e] * gn.y);
#pragma unroll
                for (int part = 0; part < 3; ++part) {
                    uint32_t b[4];  // 16 tokens of the key channels of tiles t (0, 1) and t + 1 (2, 3)
                    blk_ldm_trans(kts + part * Cfg::Tile + blk_off<D>(lane & 15, t + (lane >> 4)), b);
                    blk_mma(S[t], a, b[0], b[1]);
                    blk_mma(S[t + 1], a, b[2], b[3]);
                }
            }
        }
        if (last && p.h_last) {
            float* out = p.h_last + ((size_t)item * p.dk + fc) * p.dv + ch;
#pragma unroll
            for (int t = 0; t < KT; ++t, out += 8 * p.dv)
                if (8 * t < p.dk && ch < p.dv) {
                    *reinterpret_cast<float2*>(out) = make_float2(S[t][0], S[t][2]);
                    *reinterpret_cast<float2*>(out + p.dv) = make_float2(S[t][1], S[t][3]);
                }
        }
        if (last)
            item += gridDim.x, c = 0;
        else
            ++c;
    }
}

// ------------------------------------------------------------------------------------ host

template <int D>
inline cudaError_t linattn_block_go(const LaPasses& all, int n, cudaStream_t stream) {
    const LaPass& p = all.p[0];
    const int wpi = (p.seq_len + 15) / 16;
    const long long items = (long long)p.nseq * p.heads;
    // an item a CTA while that leaves SMs idle (latency), then as many as its warps take
    const int per_cta = (int)std::max(1LL, std::min<long long>(kBlkThreads / 32 / wpi, items * n / (2 * 148)));
    const size_t smem = (size_t)per_cta * wpi * 16 * D * 2 * 3;
    auto kernel = linattn_block_kernel<D>;
    // with room for the static part: together they may pass the default limit where the dynamic part alone does not
    if (prepare_kernel_smem(reinterpret_cast<const void*>(kernel), (int)smem + 4096) != 0) return cudaErrorInvalidValue;
    return launch_pdl(kernel, dim3((unsigned)((items + per_cta - 1) / per_cta), 1, (unsigned)n), dim3(kBlkThreads), smem, stream, all, wpi,
                      per_cta);
}

template <int DK, int DV>
inline cudaError_t linattn_resume_go(const LaPass& p, int nsm, cudaStream_t stream) {
    using Cfg = ResumeCfg<DK, DV>;
    auto kernel = linattn_resume_kernel<DK, DV>;
    if (prepare_kernel_smem(reinterpret_cast<const void*>(kernel), Cfg::Bytes + 4096) != 0) return cudaErrorInvalidValue;
    const unsigned grid = (unsigned)std::min<long long>((long long)p.nseq * p.heads, Cfg::Ctas * nsm);
    return launch_pdl(kernel, dim3(grid), dim3(Cfg::Threads), (size_t)Cfg::Bytes, stream, p);
}

// Tokens up to which a block with a state is not worth the chunk kernel: 1024 states of 128 x 128 and 32 tokens 52 us
// here and 67 there, 48 tokens 69 and 71, 64 tokens 87 and 73; of 64 x 64 and 64 tokens 29 and 39.  64 x 128 goes as 128 x 128:
// 32 tokens 33 and 35, 48 tokens 45 and 41.  128 x 64 would gain beyond 32 (48 tokens 47 and 61, 64 tokens 58 and 64).
inline int linattn_resume_max(const LaPass& p) { return p.dk <= 64 && p.dv <= 64 ? 64 : 32; }

// One pass in scan order over sequences of at most linattn_resume_max tokens, with states.
inline cudaError_t linattn_resume_launch(const LaPass& p, int nsm, cudaStream_t stream) {
    if (p.dk <= 64) return p.dv <= 64 ? linattn_resume_go<64, 64>(p, nsm, stream) : linattn_resume_go<64, 128>(p, nsm, stream);
    return p.dv <= 64 ? linattn_resume_go<128, 64>(p, nsm, stream) : linattn_resume_go<128, 128>(p, nsm, stream);
}

// `n` passes without states over the same sequences of at most kBlkMaxTok tokens and heads in one launch.
inline cudaError_t linattn_block_launch(const LaPass* p, int n, cudaStream_t stream) {
    LaPasses all;
    std::memset(&all, 0, sizeof(all));
    bool narrow = true;
    for (int i = 0; i < n; ++i) {
        all.p[i] = p[i];
        narrow = narrow && p[i].dk <= 64 && p[i].dv <= 64;
    }
    return narrow ? linattn_block_go<64>(all, n, stream) : linattn_block_go<128>(all, n, stream);
}

}  // namespace r2l
