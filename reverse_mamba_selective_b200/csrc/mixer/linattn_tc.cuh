// linattn_tc.cuh -- linear attention with a decay per head on the 5th-generation tensor cores (tcgen05), in
// chunks of 64 tokens, bf16 operands.
//
// With gamma = e^g, positions p = 0 .. n-1 of a chunk's tokens in scan order and S the state before it,
//   y_i = s_out [ gamma^(p_i + 1) q_i . S + s_in sum over p_j <= p_i of gamma^(p_i - p_j) (q_i . k_j) v_j ]
//   S'  = gamma^n S + s_in sum_j gamma^(n - 1 - p_j) k_j v_j^T
// (one power of gamma less before, one more behind, for shift = 1).  Everything that depends on the values is a
// product of matrices; all of them run with 128 rows by taking the value channels as rows:
//   QK  [tok i][tok j]  = Q K^T              (64 rows used)
//   OA^T[dv][tok i]     = V^T P^T            P = masked, decayed scores
//   OI^T[dv][tok i]     = S^T Q^T            S^T an operand in tensor memory
//   KV^T[dv][dk]        = V^T K~             K~ = decayed keys
// The state itself is fp32 in registers (a thread holds half a row of S^T): S = gamma^n S + KV.  The computed factors
// P, S and K~ are split into two bf16 parts each (the product runs once a part): one part would leave 2^-9 of
// each term, as much as the rounding of the output and more where an output is small beside its terms; two leave
// 2^-17.  K~ gets a third part (2^-25) when the caller takes the final state, which is an fp32 result.
//
// One CTA per SM walks over its (sequence, head) items; 16 warps with fixed roles:
//   0-7   state: K~ from the K tile; S's operand copy; the update of S
//   8-11  epilogue: y from the two accumulators, straight to global memory (a warp writes 32 neighbouring
//         channels of a token)
//   12-13 scores: QK -> P
//   14    TMA producer (ring of chunk tiles), 15 MMA issuer
// Bound by memory for heads of 64 to 128: a chunk moves 64 KB (d = 128), 1.5 us of an SM's share of the
// bandwidth, against 0.7 us of tensor time.
//
// Masked places never reach an output: scores are selected, not multiplied, rows past a sequence's length are
// zeroed where they would meet a zero weight, and a chunk whose P V product is not finite is summed again from
// shared memory over its unmasked pairs (a zero weight times a later token's infinity is NaN).
//
// Every wait is bounded; one that runs out sets the device status word and the CTA stops.
#pragma once

#include "../tc_common.cuh"
#include "../tmap.cuh"
#include "linattn_common.cuh"

namespace r2l {

constexpr int kLaTok = 64;        // tokens per chunk
constexpr int kLaThreads = 512;
constexpr int kLaBlock = 8192;    // 64 tokens x 64 channels of bf16

struct TcLaunch {
    CUtensorMap tq, tk, tv;       // [seq][token][head][channel], boxes of box_rows tokens x 64 channels
    LaPass p;
    float* seg;                   // [item][nseg] states after the segments but the last, then h0's copy; or NULL
    int nseg, seg_chunks;         // segments of a sequence, chunks in each
    int nwork, box_rows, n16;     // n16: box_rows rounded up to 16
    int nsplit;                   // parts of K~
};

template <int DK, int DV, bool Y>
struct LaCfg {
    static constexpr int KB = DK / 64, VB = DV / 64;
    static constexpr int QBytes = Y ? KB * kLaBlock : 0, KBytes = KB * kLaBlock, VBytes = VB * kLaBlock;
    static constexpr int StageBytes = QBytes + KBytes + VBytes;
    static constexpr int KtBytes = 3 * KBytes;
    static constexpr int PBytes = Y ? 2 * kLaBlock : 0;  // two parts
    static constexpr int Free = 232448 - 1024 /*align*/ - 8192 /*static*/ - 512 /*barriers*/ - KtBytes - PBytes;
    static constexpr int Stages = Free / StageBytes > 6 ? 6 : Free / StageBytes;
    static constexpr int SmemBytes = 1024 + Stages * StageBytes + KtBytes + PBytes + 512;
    // tensor memory columns
    static constexpr int QK = 0, OI = 128, OA = 192, KV = 256, SB = 384, Cols = 512;  // SB: two parts of DK / 2
    static_assert(Stages >= 2, "ring depth");
};

// MN-major tile with 128-byte swizzle: 64 channels (128 bytes) per token row, 8 tokens 1024 bytes apart (stride
// byte offset), the next 64 channels one block on (leading byte offset).
__device__ __forceinline__ uint64_t la_mn_desc(uint32_t saddr) {
    uint64_t d = 0;
    d |= (uint64_t)((saddr >> 4) & 0x3FFFu);
    d |= (uint64_t)(kLaBlock >> 4) << 16;
    d |= (uint64_t)(1024u >> 4) << 32;
    d |= (uint64_t)1u << 46;
    d |= (uint64_t)2u << 61;
    return d;
}

// MMA with A in tensor memory (two bf16 of K per column, a row per lane).
__device__ __forceinline__ void tc_mma_ts(uint32_t tmem_d, uint32_t tmem_a, uint64_t db, uint32_t idesc, uint32_t accum) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}\n" ::"r"(tmem_d),
        "r"(tmem_a), "l"(db), "r"(idesc), "r"(accum)
        : "memory");
}

__device__ __forceinline__ void tc_st16(uint32_t taddr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15};" ::"r"(r[0]),
        "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
        "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(taddr)
        : "memory");
}
__device__ __forceinline__ void tc_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ void tma_load_4d(void* dst, const CUtensorMap* map, int x, int y, int z, int w, uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(
            smem_addr(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(smem_addr(bar))
        : "memory");
}

__device__ __forceinline__ bool la_wait(uint64_t* bar, uint32_t parity) {
    return __all_sync(0xffffffffu, mbar_wait(bar, parity));
}

// One (sequence, head, segment): chunks a .. b - 1 in scan order of the nch chunks of its sequence.
struct LaItem {
    int seq, h, len, nch, a, b;
    const float* in;   // state before chunk a, or NULL
    float* out;        // state after chunk b - 1, or NULL
    bool in_t, out_t;
    float g;
};

template <bool Y>
__device__ __forceinline__ LaItem la_item(const TcLaunch& L, int work) {
    const LaPass& p = L.p;
    const int runs = Y ? L.nseg : L.nseg - 1;  // the last segment's state is nobody's start
    LaItem it;
    it.h = work % p.heads;
    const int rest = work / p.heads, seg = rest % runs;
    it.seq = rest / runs;
    it.len = la_len(p, it.seq);
    it.nch = (it.len + kLaTok - 1) / kLaTok;
    it.a = min(seg * L.seg_chunks, it.nch);
    it.b = min(it.a + L.seg_chunks, it.nch);
    const size_t dd = (size_t)p.dk * p.dv, i = (size_t)it.seq * p.heads + it.h;
    float* segs = L.seg + i * L.nseg * dd;
    it.in = nullptr;
    it.in_t = false;
    if (seg == 0) {
        // a divided sequence starts from the copy: its last segment may write h_last over h0 at any time
        if (p.h0) it.in = Y && L.nseg > 1 ? segs + (size_t)(L.nseg - 1) * dd : p.h0 + i * dd;
        it.in_t = p.h_t != 0;
    } else if (Y) {
        it.in = segs + (size_t)(seg - 1) * dd;
    }
    it.out = nullptr;
    it.out_t = false;
    if (!Y) {
        it.out = segs + (size_t)seg * dd;
    } else if (seg == L.nseg - 1 && p.h_last) {
        it.out = p.h_last + i * dd;
        it.out_t = p.h_t != 0;
    }
    it.g = la_clamp_decay(p.log_decay[it.h]);
    return it;
}

// Tokens of the c-th chunk in scan order: first row (in the sequence) and number.
__device__ __forceinline__ void la_chunk(const LaPass& p, const LaItem& it, int c, int& row0, int& n) {
    const int ci = p.reverse ? it.nch - 1 - c : c;
    row0 = ci * kLaTok;
    n = min(kLaTok, it.len - row0);
}

__device__ __forceinline__ float la_bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float la_bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// Rows n .. of a chunk's V tile become zero (they stand behind the sequence's length: whatever they hold must
// not meet a zero weight).
__device__ __forceinline__ void la_zero_rows(unsigned char* v, int vb, int n, int tid, int nthreads) {
    const int per = (kLaTok - n) * 8;
    for (int u = tid; u < vb * per; u += nthreads) {
        const int b = u / per, r = u - b * per;
        *reinterpret_cast<uint4*>(v + b * kLaBlock + n * 128 + r * 16) = make_uint4(0, 0, 0, 0);
    }
}

template <int DK, int DV, bool Y>
__global__ void __launch_bounds__(kLaThreads, 1) linattn_tc_kernel(const __grid_constant__ TcLaunch L) {
    using Cfg = LaCfg<DK, DV, Y>;
    constexpr int NST = Cfg::Stages;
    extern __shared__ __align__(16) unsigned char smem_raw[];
    __shared__ uint32_t s_tmem;
    __shared__ int s_abort;
    // decay tables of the item that a warp is at; each warp has its own, as the warps are at different items
    __shared__ float tab[14][2 * kLaTok];
    unsigned char* smem =
        reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    unsigned char* kt = smem + NST * Cfg::StageBytes;
    unsigned char* pbuf = kt + Cfg::KtBytes;
    uint64_t* full = reinterpret_cast<uint64_t*>(pbuf + Cfg::PBytes);
    uint64_t* empty = full + NST;
    uint64_t* qk_full = empty + NST;   // [2]
    uint64_t* qk_empty = qk_full + 2;  // [2]
    uint64_t* p_full = qk_empty + 2;
    uint64_t* p_empty = p_full + 1;
    uint64_t* kt_go = p_empty + 1;
    uint64_t* kt_full = kt_go + 1;
    uint64_t* kv_full = kt_full + 1;
    uint64_t* s_full = kv_full + 1;
    uint64_t* qs_done = s_full + 1;
    uint64_t* o_full = qs_done + 1;
    uint64_t* o_empty = o_full + 1;

    const LaPass& p = L.p;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    float* wtab = tab[min(warp, 13)];
    if (tid == 0) {
        for (int i = 0; i < NST; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], Y ? 5 : 1);  // the last MMA, and the four epilogue warps
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&qk_full[i], 1);
            mbar_init(&qk_empty[i], 64);
        }
        mbar_init(p_full, 64);
        mbar_init(p_empty, 4);
        mbar_init(kt_go, 1);
        mbar_init(kt_full, 256);
        mbar_init(kv_full, 1);
        mbar_init(s_full, 256);
        mbar_init(qs_done, 1);
        mbar_init(o_full, 1);
        mbar_init(o_empty, 128);
        fence_mbar_init();
        s_abort = 0;
    }
    if (L.box_rows < kLaTok)  // rows that no load writes
        for (int i = tid; i < NST * Cfg::StageBytes / 16; i += kLaThreads)
            reinterpret_cast<uint4*>(smem)[i] = make_uint4(0, 0, 0, 0);
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    if (warp == 15) tmem_alloc(&s_tmem, Cfg::Cols);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = s_tmem;
    pdl_trigger();
    pdl_wait();

    bool ok = true;
    uint32_t issued = 0;  // chunks whose loads were issued (producer)

    if (warp == 14) {
        // ------------------------------------------------------------------ producer
        const uint32_t tx = (uint32_t)(Cfg::StageBytes / kLaBlock) * (uint32_t)L.box_rows * 128u;
        uint32_t pos = 0;
        for (int work = blockIdx.x; work < L.nwork && ok; work += gridDim.x) {
            const LaItem it = la_item<Y>(L, work);
            const int hq = it.h / p.q_div, hk = it.h / p.k_div, hv = it.h / p.v_div;
            for (int c = it.a; c < it.b; ++c, ++pos) {
                const int st = pos % NST;
                if (!(ok = la_wait(&empty[st], ((pos / NST) & 1u) ^ 1u))) break;
                int row0, n;
                la_chunk(p, it, c, row0, n);
                if (elect_one()) {
                    unsigned char* s = smem + st * Cfg::StageBytes;
                    mbar_arrive_expect_tx(&full[st], tx);
                    if (Y)
                        for (int b = 0; b < Cfg::KB; ++b) tma_load_4d(s + b * kLaBlock, &L.tq, 64 * b, hq, row0, it.seq, &full[st]);
                    for (int b = 0; b < Cfg::KB; ++b)
                        tma_load_4d(s + Cfg::QBytes + b * kLaBlock, &L.tk, 64 * b, hk, row0, it.seq, &full[st]);
                    for (int b = 0; b < Cfg::VB; ++b)
                        tma_load_4d(s + Cfg::QBytes + Cfg::KBytes + b * kLaBlock, &L.tv, 64 * b, hv, row0, it.seq, &full[st]);
                }
                __syncwarp();
                issued = pos + 1;
            }
        }
    } else if (warp == 15) {
        // ------------------------------------------------------------------ MMA issuer
        constexpr uint32_t kDesc = (1u << 4) | (1u << 7) | (1u << 10) | ((128u >> 4) << 24);  // fp32 += bf16 bf16, M 128
        constexpr uint32_t kMnA = 1u << 15, kMnB = 1u << 16;
        const uint32_t n_tok = (uint32_t)(L.n16 >> 3) << 17, n_dk = (uint32_t)(DK >> 3) << 17;
        const int kd_steps = (p.dk + 15) >> 4, tok_steps = L.n16 >> 4;
        const uint64_t dq = sw128_kmajor_desc(smem_addr(smem)), dk = sw128_kmajor_desc(smem_addr(smem + Cfg::QBytes));
        const uint64_t dv = la_mn_desc(smem_addr(smem + Cfg::QBytes + Cfg::KBytes));
        const uint64_t dkt = la_mn_desc(smem_addr(kt)), dp = sw128_kmajor_desc(smem_addr(pbuf));
        uint32_t total = 0;
        for (int work = blockIdx.x; work < L.nwork; work += gridDim.x) {
            const LaItem it = la_item<Y>(L, work);
            total += (uint32_t)(it.b - it.a);
        }
        auto stage_off = [&](uint32_t pos) { return (uint64_t)((uint32_t)((pos % NST) * Cfg::StageBytes) >> 4); };
        // scores of the chunk at `pos`, whose tiles have landed
        auto scores = [&](uint32_t pos) -> bool {
            if (!la_wait(&qk_empty[pos & 1], ((pos >> 1) & 1u) ^ 1u)) return false;
            tc_fence_after();
            if (elect_one()) {
                const uint64_t so = stage_off(pos);
                for (int kk = 0; kk < kd_steps; ++kk) {
                    const uint64_t o = so + (uint64_t)(((kk >> 2) * kLaBlock + (kk & 3) * 32) >> 4);
                    tc_mma(tmem + Cfg::QK + (pos & 1) * 64, dq + o, dk + o, kDesc | n_tok, kk > 0);
                }
                tc_commit(&qk_full[pos & 1]);
            }
            __syncwarp();
            return true;
        };
        uint32_t pos = 0, nkv = 0, nqs = 0, nqk = 0;
        for (int work = blockIdx.x; work < L.nwork && ok; work += gridDim.x) {
            const LaItem it = la_item<Y>(L, work);
            for (int c = it.a; c < it.b && ok; ++c, ++pos) {
                const bool has = it.in || c > it.a, need = c < it.b - 1 || it.out;
                const int st = pos % NST;
                const uint64_t so = stage_off(pos);
                if (!(ok = la_wait(&full[st], (pos / NST) & 1u))) break;
                if (need && lane == 0) mbar_arrive(kt_go);
                if (Y && nqk == pos) {
                    if (!(ok = scores(pos))) break;
                    nqk = pos + 1;
                }
                if (need) {
                    if (!(ok = la_wait(kt_full, nkv & 1u))) break;
                    tc_fence_after();
                    if (elect_one()) {
                        for (int part = 0; part < L.nsplit; ++part)
                            for (int kk = 0; kk < tok_steps; ++kk)
                                tc_mma(tmem + Cfg::KV, dv + so + (uint64_t)(kk * 2048 >> 4),
                                       dkt + (uint64_t)((part * Cfg::KBytes + kk * 2048) >> 4), kDesc | kMnA | kMnB | n_dk,
                                       part > 0 || kk > 0);
                        tc_commit(kv_full);
                        if (!Y) tc_commit(&empty[st]);
                    }
                    __syncwarp();
                    ++nkv;
                }
                if (Y) {
                    // the next chunk's scores early, if its tiles are there
                    if (pos + 1 < total &&
                        __all_sync(0xffffffffu, mbar_try_wait(&full[(pos + 1) % NST], ((pos + 1) / NST) & 1u))) {
                        if (!(ok = scores(pos + 1))) break;
                        nqk = pos + 2;
                    }
                    if (!(ok = la_wait(o_empty, (pos & 1u) ^ 1u))) break;
                    if (has) {
                        if (!(ok = la_wait(s_full, nqs & 1u))) break;
                        tc_fence_after();
                        if (elect_one()) {
                            for (int part = 0; part < 2; ++part)
                                for (int kk = 0; kk < kd_steps; ++kk)
                                    tc_mma_ts(tmem + Cfg::OI, tmem + Cfg::SB + part * (DK / 2) + kk * 8,
                                              dq + so + (uint64_t)(((kk >> 2) * kLaBlock + (kk & 3) * 32) >> 4), kDesc | n_tok,
                                              part > 0 || kk > 0);
                            tc_commit(qs_done);
                        }
                        __syncwarp();
                        ++nqs;
                    }
                    if (!(ok = la_wait(p_full, pos & 1u))) break;
                    tc_fence_after();
                    if (elect_one()) {
                        for (int part = 0; part < 2; ++part)
                            for (int kk = 0; kk < tok_steps; ++kk)
                                tc_mma(tmem + Cfg::OA, dv + so + (uint64_t)(kk * 2048 >> 4),
                                       dp + (uint64_t)((part * kLaBlock + kk * 32) >> 4), kDesc | kMnA | n_tok, part > 0 || kk > 0);
                        tc_commit(o_full);
                        tc_commit(&empty[st]);
                    }
                    __syncwarp();
                }
            }
        }
    } else if (warp < 8) {
        // ------------------------------------------------------------------ state
        constexpr int H = DK / 2;                   // state columns of a thread
        const int quarter = warp & 3, half = warp >> 2;
        const int row = quarter * 32 + lane;        // value channel
        const int k0 = half * H;                    // first key channel
        const bool rows_used = quarter * 32 < DV;   // warp-uniform
        const bool live = row < p.dv;
        const uint32_t lane_off = (uint32_t)(quarter * 32) << 16;
        float S[H];
        uint32_t pos = 0, nkv = 0, nqs = 0;
        for (int work = blockIdx.x; work < L.nwork && ok; work += gridDim.x) {
            const LaItem it = la_item<Y>(L, work);
            const bool carries = it.in || it.out || it.b - it.a > 1;
            if (!carries) {
                pos += (uint32_t)(it.b - it.a);
                continue;
            }
#pragma unroll
            for (int i = 0; i < H; ++i) S[i] = 0.f;
            if (it.in && live) {
                if (it.in_t) {
                    const float* a = it.in + (size_t)row * p.dk + k0;
#pragma unroll
                    for (int i = 0; i < H; i += 4)
                        if (k0 + i < p.dk) {
                            const float4 x = *reinterpret_cast<const float4*>(a + i);
                            S[i] = x.x, S[i + 1] = x.y, S[i + 2] = x.z, S[i + 3] = x.w;
                        }
                } else {
                    const float* a = it.in + (size_t)k0 * p.dv + row;
#pragma unroll
                    for (int i = 0; i < H; ++i)
                        if (k0 + i < p.dk) S[i] = a[(size_t)i * p.dv];
                }
            }
            __syncwarp();
            for (int i = lane; i <= kLaTok; i += 32) wtab[i] = p.s_in * la_decay_pow(it.g, (float)i);  // s_in gamma^i
            __syncwarp();
            float ghi, glo;
            la_decay_pair(it.g, (float)kLaTok, ghi, glo);
            for (int c = it.a; c < it.b; ++c, ++pos) {
                const bool has = it.in || c > it.a, need = c < it.b - 1 || it.out;
                int row0, n;
                la_chunk(p, it, c, row0, n);
                if (need) {
                    const int st = pos % NST;
                    if (!(ok = la_wait(kt_go, nkv & 1u) && la_wait(&full[st], (pos / NST) & 1u))) break;
                    unsigned char* s = smem + st * Cfg::StageBytes;
                    // K~: the swizzle only permutes 16-byte pieces within a token's row
#pragma unroll
                    for (int m = 0; m < Cfg::KB * 2; ++m) {
                        const int u = tid + m * 256, j = (u >> 3) & 63;
                        if (j >= L.n16) continue;
                        uint32_t hi[4] = {0, 0, 0, 0}, mid[4] = {0, 0, 0, 0}, lo[4] = {0, 0, 0, 0};
                        if (j < n) {
                            const uint4 x = *reinterpret_cast<const uint4*>(s + Cfg::QBytes + u * 16);
                            const float w = wtab[(p.reverse ? j : n - 1 - j) + p.shift];
                            const uint32_t xs[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                float a = la_bf16_lo(xs[e]) * w, b = la_bf16_hi(xs[e]) * w;
                                hi[e] = pack_bf16x2(a, b);
                                a -= la_bf16_lo(hi[e]);
                                b -= la_bf16_hi(hi[e]);
                                mid[e] = pack_bf16x2(a, b);
                                if (L.nsplit > 2) lo[e] = pack_bf16x2(a - la_bf16_lo(mid[e]), b - la_bf16_hi(mid[e]));
                            }
                        }
                        unsigned char* o = kt + u * 16;
                        *reinterpret_cast<uint4*>(o) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                        *reinterpret_cast<uint4*>(o + Cfg::KBytes) = make_uint4(mid[0], mid[1], mid[2], mid[3]);
                        if (L.nsplit > 2)
                            *reinterpret_cast<uint4*>(o + 2 * Cfg::KBytes) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
                    }
                    if (n < kLaTok && row0 + n < p.seq_len) la_zero_rows(s + Cfg::QBytes + Cfg::KBytes, Cfg::VB, n, tid, 256);
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                    mbar_arrive(kt_full);
                }
                if (Y && has) {
                    // the operand copy of S, once the previous chunk's product has read the last one
                    if (!(ok = la_wait(qs_done, (nqs & 1u) ^ 1u))) break;
                    tc_fence_after();
                    if (rows_used) {
#pragma unroll
                        for (int q = 0; q < H / 32; ++q) {
                            uint32_t w[16];
                            const uint32_t to = tmem + lane_off + Cfg::SB + half * (H / 2) + q * 16;
#pragma unroll
                            for (int e = 0; e < 16; ++e) w[e] = pack_bf16x2(S[q * 32 + 2 * e], S[q * 32 + 2 * e + 1]);
                            tc_st16(to, w);
#pragma unroll
                            for (int e = 0; e < 16; ++e)
                                w[e] = pack_bf16x2(S[q * 32 + 2 * e] - la_bf16_lo(w[e]), S[q * 32 + 2 * e + 1] - la_bf16_hi(w[e]));
                            tc_st16(to + DK / 2, w);
                        }
                        tc_wait_st();
                    }
                    tc_fence_before();
                    mbar_arrive(s_full);
                    ++nqs;
                }
                if (need) {
                    float dhi = ghi, dlo = glo;
                    if (n != kLaTok) la_decay_pair(it.g, (float)n, dhi, dlo);
                    if (!(ok = la_wait(kv_full, nkv & 1u))) break;
                    ++nkv;
                    tc_fence_after();
                    if (rows_used) {
#pragma unroll
                        for (int q = 0; q < H / 32; ++q) {
                            uint32_t r[32];
                            tc_ld32_issue(tmem + lane_off + Cfg::KV + k0 + q * 32, r);
                            tc_wait_ld32(r);
#pragma unroll
                            for (int e = 0; e < 32; ++e) {
                                const float x = S[q * 32 + e];
                                S[q * 32 + e] = fmaf(x, dhi, fmaf(x, dlo, __uint_as_float(r[e])));
                            }
                        }
                    }
                    tc_fence_before();
                }
            }
            if (it.out && live && ok) {
                if (it.out_t) {
                    float* a = it.out + (size_t)row * p.dk + k0;
#pragma unroll
                    for (int i = 0; i < H; i += 4)
                        if (k0 + i < p.dk) *reinterpret_cast<float4*>(a + i) = make_float4(S[i], S[i + 1], S[i + 2], S[i + 3]);
                } else {
                    float* a = it.out + (size_t)k0 * p.dv + row;
#pragma unroll
                    for (int i = 0; i < H; ++i)
                        if (k0 + i < p.dk) a[(size_t)i * p.dv] = S[i];
                }
            }
        }
    } else if (Y && warp < 12) {
        // ------------------------------------------------------------------ epilogue
        const int quarter = warp & 3, row = quarter * 32 + lane;
        const uint32_t lane_off = (uint32_t)(quarter * 32) << 16;
        const bool rows_used = quarter * 32 < DV, live = row < p.dv;
        uint32_t pos = 0;
        for (int work = blockIdx.x; work < L.nwork && ok; work += gridDim.x) {
            const LaItem it = la_item<Y>(L, work);
            __syncwarp();
            for (int i = lane; i <= kLaTok; i += 32) wtab[i] = p.s_out * la_decay_pow(it.g, (float)i);  // s_out gamma^i
            __syncwarp();
            const size_t base = (size_t)it.seq * p.seq_len * p.y_tok + (size_t)it.h * p.dv + row;
            float* yf = static_cast<float*>(p.y) + base;
            __nv_bfloat16* yb = static_cast<__nv_bfloat16*>(p.y) + base;
            for (int c = it.a; c < it.b; ++c, ++pos) {
                const bool has = it.in || c > it.a;
                const int st = pos % NST;
                int row0, n;
                la_chunk(p, it, c, row0, n);
                if (!(ok = la_wait(o_full, pos & 1u))) break;
                tc_fence_after();
                float o[kLaTok];
                bool finite = true;
                if (rows_used) {
                    float any = 0.f;
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        uint32_t r[32];
                        tc_ld32_issue(tmem + lane_off + Cfg::OA + q * 32, r);
                        tc_wait_ld32(r);
#pragma unroll
                        for (int e = 0; e < 32; ++e) {
                            o[q * 32 + e] = __uint_as_float(r[e]);
                            if (q * 32 + e < n) any = fmaf(o[q * 32 + e], 0.f, any);  // NaN once anything is not finite
                        }
                    }
                    finite = __all_sync(0xffffffffu, any == 0.f);
                    if (!finite) {
                        // a masked token may have met a zero weight: the same sums over the unmasked pairs alone
                        la_wait(p_full, pos & 1u);
                        la_wait(&full[st], (pos / NST) & 1u);
                        const unsigned char* v = smem + st * Cfg::StageBytes + Cfg::QBytes + Cfg::KBytes + (row >> 6) * kLaBlock;
                        const int ch = row & 63;
#pragma unroll
                        for (int i = 0; i < kLaTok; ++i) {
                            if (i >= n) continue;
                            const int j0 = p.reverse ? i : 0, j1 = p.reverse ? n : i + 1;
                            float acc = 0.f;
                            for (int j = j0; j < j1; ++j) {
                                const unsigned char* pa = pbuf + i * 128 + (((j >> 3) ^ (i & 7)) << 4) + (j & 7) * 2;
                                const float pw = __bfloat162float(*reinterpret_cast<const __nv_bfloat16*>(pa)) +
                                                 __bfloat162float(*reinterpret_cast<const __nv_bfloat16*>(pa + kLaBlock));
                                const float vv = __bfloat162float(*reinterpret_cast<const __nv_bfloat16*>(
                                    v + j * 128 + (((ch >> 3) ^ (j & 7)) << 4) + (ch & 7) * 2));
                                acc = fmaf(pw, vv, acc);
                            }
                            o[i] = acc;
                        }
                    }
                    if (has) {
#pragma unroll
                        for (int q = 0; q < 2; ++q) {
                            uint32_t r[32];
                            tc_ld32_issue(tmem + lane_off + Cfg::OI + q * 32, r);
                            tc_wait_ld32(r);
                            // gamma^(position + 1 - shift)
                            const float* f = p.reverse ? wtab + (n - p.shift) : wtab + (1 - p.shift);
#pragma unroll
                            for (int e = 0; e < 32; ++e) {
                                const int i = q * 32 + e;
                                const float w = p.reverse ? (i < n ? f[-i] : 0.f) : f[i];
                                o[i] = fmaf(w, __uint_as_float(r[e]), o[i]);
                            }
                        }
                    }
                }
                tc_fence_before();
                mbar_arrive(o_empty);
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(p_empty);
                    mbar_arrive(&empty[st]);
                }
                if (live) {
                    if (p.y_f32) {
                        float* y = yf + (size_t)row0 * p.y_tok;
#pragma unroll
                        for (int i = 0; i < kLaTok; ++i)
                            if (i < n) y[(size_t)i * p.y_tok] = o[i];
                    } else {
                        __nv_bfloat16* y = yb + (size_t)row0 * p.y_tok;
#pragma unroll
                        for (int i = 0; i < kLaTok; ++i)
                            if (i < n) y[(size_t)i * p.y_tok] = __float2bfloat16_rn(o[i]);
                    }
                }
            }
            if (it.a == 0 && live && ok) {  // the first segment's CTA also writes the zeros behind the row's tokens
                for (int t = it.len; t < p.seq_len; ++t) {
                    if (p.y_f32)
                        yf[(size_t)t * p.y_tok] = 0.f;
                    else
                        yb[(size_t)t * p.y_tok] = __float2bfloat16_rn(0.f);
                }
            }
        }
    } else if (Y && warp < 14) {
        // ------------------------------------------------------------------ scores
        const int i = tid - 384;  // the row (token) of this thread
        const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
        uint32_t pos = 0;
        for (int work = blockIdx.x; work < L.nwork && ok; work += gridDim.x) {
            const LaItem it = la_item<Y>(L, work);
            const float s = p.s_in * p.s_out;
            __syncwarp();
            for (int d = lane - 63; d <= 63; d += 32) {  // s_in s_out gamma^|d| at 63 + d, zero where masked
                const float w = s * la_decay_pow(it.g, (float)abs(d));
                wtab[63 + d] = (p.reverse ? d <= 0 : d >= 0) ? w : 0.f;
            }
            __syncwarp();
            for (int c = it.a; c < it.b; ++c, ++pos) {
                int row0, n;
                la_chunk(p, it, c, row0, n);
                if (!(ok = la_wait(&qk_full[pos & 1], (pos >> 1) & 1u))) break;
                tc_fence_after();
                uint32_t r0[32], r1[32];
                tc_ld32_issue(tmem + lane_off + Cfg::QK + (pos & 1) * 64, r0);
                tc_ld32_issue(tmem + lane_off + Cfg::QK + (pos & 1) * 64 + 32, r1);
                tc_wait_ld32(r0);
                tc_wait_ld32(r1);
                tc_fence_before();
                mbar_arrive(&qk_empty[pos & 1]);
                if (!(ok = la_wait(p_empty, (pos & 1u) ^ 1u))) break;
                unsigned char* pb = pbuf + i * 128;
                const float* t = wtab + 63 + i;
#pragma unroll
                for (int q = 0; q < 8; ++q) {
                    uint32_t w[4], u[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        float v[2];
#pragma unroll
                        for (int b = 0; b < 2; ++b) {
                            const int j = q * 8 + e * 2 + b;
                            const float x = __uint_as_float(j < 32 ? r0[j & 31] : r1[j & 31]);
                            const float d = t[-j];
                            v[b] = (d != 0.f && j < n) ? x * d : 0.f;
                        }
                        w[e] = pack_bf16x2(v[0], v[1]);
                        u[e] = pack_bf16x2(v[0] - la_bf16_lo(w[e]), v[1] - la_bf16_hi(w[e]));
                    }
                    *reinterpret_cast<uint4*>(pb + ((q ^ (i & 7)) << 4)) = make_uint4(w[0], w[1], w[2], w[3]);
                    *reinterpret_cast<uint4*>(pb + kLaBlock + ((q ^ (i & 7)) << 4)) = make_uint4(u[0], u[1], u[2], u[3]);
                }
                if (n < kLaTok && row0 + n < p.seq_len) {
                    const int st = pos % NST;
                    if (!(ok = la_wait(&full[st], (pos / NST) & 1u))) break;
                    la_zero_rows(smem + st * Cfg::StageBytes + Cfg::QBytes + Cfg::KBytes, Cfg::VB, n, i, 64);
                }
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                mbar_arrive(p_full);
            }
        }
    }

    if (!ok) {
        atomicExch(&s_abort, 1);
        if (lane == 0) atomicOr(&g_status_word, kStatusTimeoutGemm);
    }
    tc_fence_before();
    __syncthreads();
    if (s_abort && warp == 14) {
        // the loads in flight still write this CTA's shared memory: wait for them before it is given back
        for (uint32_t q = issued > (uint32_t)NST ? issued - NST : 0; q < issued; ++q)
            if (!mbar_wait_bounded(&full[q % NST], (q / NST) & 1u) && lane == 0) atomicOr(&g_status_word, kStatusDrainTimeout);
    }
    __syncthreads();
    if (warp == 15) {
        tc_fence_after();
        tmem_dealloc(tmem, Cfg::Cols);
    }
}

// States before the segments: seg[s] = gamma^tokens(s) seg[s - 1] + seg[s], in place (seg[0] is complete: its run
// began with h0); and h0's copy, as it is stored, in the last place.
__global__ void __launch_bounds__(256) linattn_segments_kernel(LaPass p, float* seg, int nseg, int seg_chunks) {
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
    float* a = seg + (size_t)item * nseg * dd + e;
    if (p.h0) a[(size_t)(nseg - 1) * dd] = p.h0[(size_t)item * dd + e];
    float s = a[0];
    for (int i = 1; i < nseg - 1; ++i) {
        const int c0 = min(i * seg_chunks, nch), c1 = min(c0 + seg_chunks, nch);
        const int tok = (c1 - c0) * kLaTok - (ragged >= c0 && ragged < c1 ? missing : 0);
        float hi, lo;
        la_decay_pair(g, (float)tok, hi, lo);
        s = fmaf(s, hi, fmaf(s, lo, a[(size_t)i * dd]));
        a[(size_t)i * dd] = s;
    }
}

// ------------------------------------------------------------------------------------ host

// [seq][token][head][channel] with the given element strides, boxes of box_rows tokens x 64 channels of a head.
inline bool la_encode(CUtensorMap* out, const void* base, int d, int heads, int seq_len, int nseq, long long tok, int box_rows) {
    auto enc = tensor_map_encoder();
    if (!enc) {
        snprintf(last_error_buffer(), 256, "cuTensorMapEncodeTiled: driver entry point unavailable");
        return false;
    }
    cuuint64_t dims[4] = {(cuuint64_t)d, (cuuint64_t)heads, (cuuint64_t)seq_len, (cuuint64_t)nseq};
    cuuint64_t strides[3] = {(cuuint64_t)d * 2, (cuuint64_t)tok * 2, (cuuint64_t)tok * 2 * (cuuint64_t)seq_len};
    cuuint32_t box[4] = {64, 1, (cuuint32_t)box_rows, 1};
    cuuint32_t estr[4] = {1, 1, 1, 1};
    const CUresult r = enc(out, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(base), dims, strides, box, estr,
                           CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                           CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r == CUDA_SUCCESS) return true;
    snprintf(last_error_buffer(), 256, "cuTensorMapEncodeTiled failed (CUresult %d)", (int)r);
    return false;
}

// How a pass is divided: segments per sequence and chunks in each.  Sequences are divided when there are fewer
// (sequence, head) pairs than half the SMs, into as many segments as fill them, of four chunks at least: dividing
// reads k and v a second time.
inline void la_segments(int nseq, int heads, int seq_len, int nsm, int& nseg, int& seg_chunks) {
    const long long items = (long long)nseq * heads;
    const int nch = (seq_len + kLaTok - 1) / kLaTok;
    nseg = 1;
    if (items > 0 && 2 * items <= nsm) nseg = (int)std::min<long long>(nsm / items, nch / 4);
    if (nseg < 2) nseg = 1;
    seg_chunks = (nch + nseg - 1) / nseg;
    nseg = seg_chunks > 0 ? (nch + seg_chunks - 1) / seg_chunks : 1;
}

inline size_t la_segment_bytes(int nseq, int heads, int seq_len, int dk, int dv, int nsm) {
    int nseg, seg_chunks;
    la_segments(nseq, heads, seq_len, nsm, nseg, seg_chunks);
    return nseg > 1 ? (size_t)nseq * heads * nseg * dk * dv * sizeof(float) : 0;
}

template <int DK, int DV, bool Y>
inline bool la_tc_go(const TcLaunch& L, int nsm, cudaStream_t stream) {
    using Cfg = LaCfg<DK, DV, Y>;
    auto kernel = linattn_tc_kernel<DK, DV, Y>;
    if (prepare_kernel_smem(reinterpret_cast<const void*>(kernel), Cfg::SmemBytes) != 0) return false;
    return cuda_ok(launch_pdl(kernel, dim3((unsigned)std::min(L.nwork, nsm)), dim3(kLaThreads), (size_t)Cfg::SmemBytes, stream, L),
                   "linear attention chunk kernel launch");
}

template <bool Y>
inline bool la_tc_pick(const TcLaunch& L, int nsm, cudaStream_t stream) {
    if (L.p.dk <= 64) return L.p.dv <= 64 ? la_tc_go<64, 64, Y>(L, nsm, stream) : la_tc_go<64, 128, Y>(L, nsm, stream);
    return L.p.dv <= 64 ? la_tc_go<128, 64, Y>(L, nsm, stream) : la_tc_go<128, 128, Y>(L, nsm, stream);
}

// One pass; seg: la_segment_bytes bytes, or NULL when that is 0.
inline bool linattn_tc_launch(const LaPass& p, float* seg, int nsm, cudaStream_t stream) {
    TcLaunch L;
    std::memset(&L, 0, sizeof(L));
    L.p = p;
    L.seg = seg;
    la_segments(p.nseq, p.heads, p.seq_len, nsm, L.nseg, L.seg_chunks);
    L.box_rows = std::min(kLaTok, (p.seq_len + 7) & ~7);
    L.n16 = (L.box_rows + 15) & ~15;
    L.nsplit = p.h_last ? 3 : 2;
    if (!la_encode(&L.tq, p.q, p.dk, p.heads / p.q_div, p.seq_len, p.nseq, p.q_tok, L.box_rows) ||
        !la_encode(&L.tk, p.k, p.dk, p.heads / p.k_div, p.seq_len, p.nseq, p.k_tok, L.box_rows) ||
        !la_encode(&L.tv, p.v, p.dv, p.heads / p.v_div, p.seq_len, p.nseq, p.v_tok, L.box_rows))
        return false;
    if (L.nseg > 1) {
        L.nwork = p.nseq * p.heads * (L.nseg - 1);
        if (!la_tc_pick<false>(L, nsm, stream)) return false;
        const dim3 grid((unsigned)((p.dk * p.dv + 255) / 256), (unsigned)(p.nseq * p.heads));
        if (!cuda_ok(launch_pdl(linattn_segments_kernel, grid, dim3(256), 0, stream, p, seg, L.nseg, L.seg_chunks),
                     "linear attention segment kernel launch"))
            return false;
    }
    L.nwork = p.nseq * p.heads * L.nseg;
    return la_tc_pick<true>(L, nsm, stream);
}

}  // namespace r2l
