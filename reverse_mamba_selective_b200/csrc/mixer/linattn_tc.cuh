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
// P, S and K~ are split into two bf16 parts each (the product runs once a part): one part would leave up to 2^-8 of
// each term, as much as the rounding of the output and more where an output is small beside its terms; two leave
// 2^-16.  K~ gets a third part (2^-24) when the caller takes the final state, which is an fp32 result; else the states,
// those between a divided sequence's segments too, only form outputs that are rounded to bf16 themselves.  (Three parts
// in every pass: gradients of 8 x 4096 tokens, 16 heads of 128, 533 us against 492.)
//
// One CTA per SM walks over its (sequence, head) items; 16 warps with fixed roles:
//   0-7   state: K~ from the K tile; S's operand copy; the update of S
//   8-11  epilogue: y from the two accumulators, 32 channels a warp, transposed by stmatrix into the chunk's dead
//         Q (and K) tile and stored from there by TMA
//   12-13 scores: QK -> P, 32 tokens a warp, in blocks of 32 x 32: one on the diagonal, one full, one zero
//   14    TMA producer (ring of chunk tiles), 15 MMA issuer
// A chunk moves 64 KB (d = 128), 1.5 us of an SM's share of the bandwidth, against 0.7 us of tensor time.  What
// bounds it is the chain through the state, 3.5 thousand cycles a chunk: K~ (1100, and 260 until the MMA may read it), the
// split copy of S (800), KV's product and its way back (700), the rest waits; under a long run the 1000 W limit
// lowers the clock as well.  128 heads and sequences of 4096 tokens: 151 us at 1.9 GHz (3.6 TB/s), 175 to 181 us back to
// back at the limit.  At its cap of 128 registers a thread the outputs' kernel spills 108 bytes of stores and 200 of loads
// (68 and 148 for d_k up to 64).  Measured and not kept: V~ instead of K~ through tensor memory (224 us against 173), two
// issuing warps (205), 30 warps of 64 registers (155 against 148), the next K~ held in registers (more spills: 293), spinning
// waits (161 against 149), a truncating split (172 against 169).
//
// The pass over the states of a divided sequence (Y false) has room for two K~ and two KV: the next chunk's K~ is
// made before this one's KV is waited for (one sequence of 32768 tokens of 16 heads: 248 -> 226 us in all, now 222).
//
// Masked places never reach an output: rows of V past a sequence's length are zeroed, keys past it are not read into
// K~, and where an output comes out not finite (a masked weight is a zero factor, and zero times an infinity is
// NaN) the chunk's scores and values, still in shared memory, are summed again over the unmasked pairs alone, in fp32
// and one after another: such an output may differ in its last bit from one that met no masked value.
//
// Every wait is bounded; one that runs out sets the device status word and the CTA stops.
#pragma once

#include "../tc_common.cuh"
#include "../tmap.cuh"
#include "linattn_common.cuh"
#include "pairs.cuh"

namespace r2l {

constexpr int kLaThreads = 512;
constexpr int kLaBlock = 8192;    // 64 tokens x 64 channels of bf16

struct TcLaunch {
    CUtensorMap tq, tk, tv;       // [seq][token][head][channel], boxes of box_rows tokens x 64 channels
    CUtensorMap ty;               // y the same way, boxes of box_rows x 32 (bf16 outputs)
    LaPass p;
    float* seg;                   // [item][nseg] states after the segments but the last, then h0's copy; or NULL
    int nseg, seg_chunks;         // segments of a sequence, chunks in each
    int nwork, box_rows;
    int nsplit;                   // parts of K~
};

template <int DK, int DV, bool Y>
struct LaCfg {
    static constexpr int KB = DK / 64, VB = DV / 64;
    static constexpr int QBytes = Y ? KB * kLaBlock : 0, KBytes = KB * kLaBlock, VBytes = VB * kLaBlock;
    static constexpr int StageBytes = QBytes + KBytes + VBytes;
    static constexpr int KtBuf = 3 * KBytes, KtBytes = Y ? KtBuf : 2 * KtBuf;
    static constexpr int PPart = kLaBlock, PBytes = Y ? 2 * 2 * PPart : 0;  // two buffers of two parts
    static constexpr int TabBytes = 6 * kLaTok * 4, BarBytes = 256;
    static constexpr int Fixed = 1024 /*alignment*/ + KtBytes + PBytes + TabBytes + BarBytes;
    static constexpr int Free = 232448 - 64 /*static*/ - Fixed;
    static constexpr int Stages = Free / StageBytes > 6 ? 6 : Free / StageBytes;
    static constexpr int SmemBytes = Fixed + Stages * StageBytes;
    static_assert((3 * Stages + 13) * 8 <= BarBytes, "barriers");
    // tensor memory columns
    static constexpr int QK = 0, OI = 128, OA = 192, KV = 256, SB = 384, Cols = 512;  // SB: two parts of DK / 2, or a second KV
    static_assert(Stages >= 2, "ring depth");
};

// Shared-memory descriptors of the MMAs, by their low words (address / 16 and leading byte offset / 16): the high word is
// the same for all.  Both kinds have 128-byte swizzle and 8 rows 1024 bytes apart (stride byte offset):
// K-major, a token's (or score row's) 128 bytes along K, as sw128_kmajor_desc; MN-major, 64 channels of a token in
// a row, the rows along K, the next 64 channels one block on (leading byte offset).
constexpr uint32_t kLaDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ uint32_t la_k_desc(uint32_t saddr) { return (saddr >> 4) | (1u << 16); }
__device__ __forceinline__ uint32_t la_mn_desc(uint32_t saddr) { return (saddr >> 4) | ((uint32_t)(kLaBlock >> 4) << 16); }

__device__ __forceinline__ void la_mma(uint32_t tmem_d, uint32_t da, uint32_t db, uint32_t idesc, bool accum) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "mov.b64 a, {%1, %5};\n\tmov.b64 b, {%2, %5};\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, p;\n\t}\n" ::"r"(tmem_d),
        "r"(da), "r"(db), "r"(idesc), "r"((uint32_t)accum), "n"(kLaDescHi)
        : "memory");
}

// The same with A in tensor memory (two bf16 of K per column, a row per lane).
__device__ __forceinline__ void la_mma_ts(uint32_t tmem_d, uint32_t tmem_a, uint32_t db, uint32_t idesc, bool accum) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 b;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "mov.b64 b, {%2, %5};\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %3, p;\n\t}\n" ::"r"(tmem_d),
        "r"(tmem_a), "r"(db), "r"(idesc), "r"((uint32_t)accum), "n"(kLaDescHi)
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
// 64 fp32 columns of 16 lanes as 8 x 8 fragments: r[4 k + 2 a + b] is lane t / 4 + 8 a, column 8 k + 2 (t % 4) + b for
// thread t of the warp; issued without waiting (tc_wait_ld32 completes it).
__device__ __forceinline__ void tc_ld_frag_issue(uint32_t taddr, uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
          "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
          "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr));
}

// Two 8 x 8 matrices of 16-bit values, stored transposed; lane l gives the address of row l % 8 of matrix l / 8.
__device__ __forceinline__ void st_matrix2_trans(uint32_t saddr, uint32_t a, uint32_t b) {
    asm volatile("stmatrix.sync.aligned.m8n8.x2.trans.shared.b16 [%0], {%1, %2};" ::"r"(saddr), "r"(a), "r"(b) : "memory");
}

__device__ __forceinline__ void tma_store_4d(const CUtensorMap* map, const void* src, int x, int y, int z, int w) {
    asm volatile("cp.async.bulk.tensor.4d.global.shared::cta.bulk_group [%0, {%1, %2, %3, %4}], [%5];" ::"l"(
                     reinterpret_cast<uint64_t>(map)),
                 "r"(x), "r"(y), "r"(z), "r"(w), "r"(smem_addr(src))
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

// Waits for the phase with the given parity, at most kWaitLimitNs; the same answer for the whole warp.  The clock is
// read every 32 polls only: the busy warps need the issue slots.
__device__ __noinline__ bool la_wait_long(uint64_t* bar, uint32_t parity) {
    const uint64_t t0 = globaltimer_ns();
    bool ok = false;
    do {
#pragma unroll 1
        for (int i = 0; i < 32 && !ok; ++i) ok = mbar_try_wait(bar, parity);
    } while (!ok && globaltimer_ns() - t0 <= kWaitLimitNs);
    return __all_sync(0xffffffffu, ok);
}
__device__ __forceinline__ bool la_wait(uint64_t* bar, uint32_t parity) {
    return __all_sync(0xffffffffu, mbar_try_wait(bar, parity)) || la_wait_long(bar, parity);
}

// One arrival for the whole warp, behind all of its lanes' work (an arrival a lane costs a turn in the barrier unit each).
__device__ __forceinline__ void la_arrive(uint64_t* bar) {
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
}

// Whether the phase with the given parity has completed; never suspends the warp (try_wait may, for microseconds).
__device__ __forceinline__ bool la_test(uint64_t* bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.b32 %0, 1, 0, p;\n\t}\n"
        : "=r"(ok)
        : "r"(smem_addr(bar)), "r"(parity)
        : "memory");
    return __all_sync(0xffffffffu, ok != 0);
}

// One (sequence, head, segment): chunks a .. b - 1 in scan order of the nch chunks of its sequence.
struct LaItem {
    int seq, h, len, nch, a, b;
    const float* in;   // state before chunk a, or NULL
    float* out;        // state after chunk b - 1, or NULL
    bool in_t, out_t;
};

// This CTA's share of the work: [begin, end).
__device__ __forceinline__ int la_share(int nwork, unsigned i) { return (int)((unsigned long long)nwork * i / gridDim.x); }

template <bool Y>
__device__ __forceinline__ LaItem la_item(const TcLaunch& L, int work) {
    const LaPass& p = L.p;
    const int runs = Y ? L.nseg : L.nseg - 1;  // the last segment's state is nobody's start
    LaItem it;
    // heads slowest: a CTA's items mostly share their head, and with it the decay's tables
    const int per_head = p.nseq * runs;
    it.h = work / per_head;
    const int rest = work - it.h * per_head, seg = rest % runs;
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

// x rounded to two bf16; x becomes what the rounding left (exact).  SAT: an infinity is left as one.
template <bool SAT = false>
__device__ __forceinline__ uint32_t la_split(float2& x) {
    const uint32_t w = SAT ? la_pack_sat(x.x, x.y) : pack_bf16x2(x.x, x.y);
    x = fma2(make_float2(la_bf16_lo(w), la_bf16_hi(w)), make_float2(-1.f, -1.f), x);
    return w;
}

// max(|m|, |w|) of the bf16 halves but for the sign, NaN if either is.
__device__ __forceinline__ uint32_t la_absmax_bf16x2(uint32_t m, uint32_t w) {
    uint32_t d;
    asm("max.NaN.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(m), "r"(w));
    return d;
}
__device__ __forceinline__ bool la_not_finite(uint32_t m) { return (m & 0x7F80u) == 0x7F80u || (m & 0x7F800000u) == 0x7F800000u; }

// Rows n .. of a chunk's V tile become zero (they stand behind the sequence's length: whatever they hold must
// not meet a zero weight).
__device__ __noinline__ void la_zero_rows(unsigned char* v, int vb, int n, int tid, int nthreads) {
    const int per = (kLaTok - n) * 8;
    for (int u = tid; u < vb * per; u += nthreads) {
        const int b = u / per, r = u - b * per;
        *reinterpret_cast<uint4*>(v + b * kLaBlock + n * 128 + r * 16) = make_uint4(0, 0, 0, 0);
    }
}

// Rows t0 .. of a sequence's outputs become zeros, by 128 threads: 16-byte pieces (dv is a multiple of 8, 32 pieces a row at
// most).  Rows and pieces are counted apart: their product may pass 2^31.
__device__ __noinline__ void la_zero_tail(const LaPass& p, int seq, int h, int t0, int tid) {
    const int es = p.y_f32 ? 4 : 2, per_row = p.dv * es / 16, rows = p.seq_len - t0, rows_par = 128 / per_row;
    const int first = tid / per_row, piece = tid - first * per_row;
    if (first >= rows_par) return;
    unsigned char* y = static_cast<unsigned char*>(p.y) +
                       (((size_t)seq * p.seq_len + t0) * p.y_tok + (size_t)h * p.dv) * es + piece * 16;
    for (int t = first; t < rows; t += rows_par) *reinterpret_cast<uint4*>(y + (size_t)t * p.y_tok * es) = make_uint4(0, 0, 0, 0);
}

// r += fac * s2 on fragments: a column pair's factors are those of its tokens.
__device__ __forceinline__ void la_add_inter(uint32_t (&r)[32], const uint32_t (&s2)[32], const float2 (&fac)[8]) {
#pragma unroll
    for (int k = 0; k < 16; ++k) {
        const float2 y = fma2(fac[k >> 1], make_float2(__uint_as_float(s2[2 * k]), __uint_as_float(s2[2 * k + 1])),
                                 make_float2(__uint_as_float(r[2 * k]), __uint_as_float(r[2 * k + 1])));
        r[2 * k] = __float_as_uint(y.x);
        r[2 * k + 1] = __float_as_uint(y.y);
    }
}

// Not inlined, as all code off the usual path: the roles' loops together have to stay in the instruction cache.
// What an epilogue warp does out of the ordinary for its 16 channels (from ch0 of the head), on a thread's fragment `out`:
//  - outputs that came out not finite (redo): a masked token may have met a zero weight.  The sum over the unmasked pairs
//    alone, from the swizzled tiles of P (two parts) and V, plus the state's part (oi: its accumulator, 0 where there is none;
//    fac: the tokens' factors);
//  - rows past the length become zeros;
//  - fp32 outputs are stored.
__device__ __noinline__ void la_finish(uint32_t* out, bool redo, const unsigned char* pt, const unsigned char* vt, uint32_t oi,
                                       const float* fac, int ch0, int n, const LaPass& p, int seq, int h, int row0) {
    const int lane = threadIdx.x & 31, fr = lane >> 2, fc = (lane & 3) * 2;
    if (redo) {
        uint32_t s2[32] = {};
        if (oi) {
            tc_ld_frag_issue(oi, s2);
            tc_wait_ld32(s2);
        }
#pragma unroll 1
        for (int e = 0; e < 32; ++e) {
            if ((out[e] & 0x7F800000u) != 0x7F800000u) continue;
            const int i = 8 * (e >> 2) + fc + (e & 1), ch = (ch0 & 63) + fr + 8 * ((e >> 1) & 1);
            const int j0 = p.reverse ? i : 0, j1 = i >= n ? 0 : p.reverse ? n : i + 1;
            float acc = 0.f;
#pragma unroll 1
            for (int j = j0; j < j1; ++j) {
                const unsigned char* pa = pt + i * 128 + (((j >> 3) ^ (i & 7)) << 4) + (j & 7) * 2;
                const float pw = __bfloat162float(*reinterpret_cast<const __nv_bfloat16*>(pa)) +
                                 __bfloat162float(*reinterpret_cast<const __nv_bfloat16*>(pa + kLaBlock));
                const float vv = __bfloat162float(
                    *reinterpret_cast<const __nv_bfloat16*>(vt + j * 128 + (((ch >> 3) ^ (j & 7)) << 4) + (ch & 7) * 2));
                acc = fmaf(pw, vv, acc);
            }
            out[e] = __float_as_uint(oi ? fmaf(fac[i], __uint_as_float(s2[e]), acc) : acc);
        }
    }
    float* y = static_cast<float*>(p.y) + ((size_t)seq * p.seq_len + row0) * p.y_tok + (size_t)h * p.dv + ch0 + fr;
#pragma unroll 1
    for (int e = 0; e < 32; ++e) {
        const int i = 8 * (e >> 2) + fc + (e & 1), ch = 8 * ((e >> 1) & 1);
        if (i >= n) out[e] = 0u;
        if (p.y_f32 && row0 + i < p.seq_len && ch0 + fr + ch < p.dv) y[(size_t)i * p.y_tok + ch] = __uint_as_float(out[e]);
    }
}

template <int DK, int DV, bool Y>
__global__ void __launch_bounds__(kLaThreads, 1) linattn_tc_kernel(const __grid_constant__ TcLaunch L) {
    using Cfg = LaCfg<DK, DV, Y>;
    constexpr int NST = Cfg::Stages;
    extern __shared__ __align__(16) unsigned char smem_raw[];
    __shared__ uint32_t s_tmem;
    __shared__ int s_abort;
    unsigned char* smem =
        reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    unsigned char* kt = smem + NST * Cfg::StageBytes;
    unsigned char* pbuf = kt + Cfg::KtBytes;
    float* tab = reinterpret_cast<float*>(pbuf + Cfg::PBytes);
    uint64_t* full = reinterpret_cast<uint64_t*>(reinterpret_cast<unsigned char*>(tab) + Cfg::TabBytes);
    uint64_t* empty = full + NST;
    uint64_t* qk_full = empty + NST;   // [2]
    uint64_t* qk_empty = qk_full + 2;  // [2]
    uint64_t* p_full = qk_empty + 2;   // [2]
    uint64_t* p_empty = p_full + 2;    // [2]
    uint64_t* kt_full = p_empty + 2;   // [NST]: one phase per chunk, whether or not its keys are needed
    uint64_t* kv_full = kt_full + NST;
    uint64_t* s_full = kv_full + 1;
    uint64_t* qs_done = s_full + 1;
    uint64_t* o_full = qs_done + 1;
    uint64_t* o_empty = o_full + 1;

    const LaPass& p = L.p;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    // decay tables of the epilogue's and the scores' warps, one each: the warps are at different items
    float* wtab = tab + (warp >= 8 && warp < 14 ? warp - 8 : 0) * kLaTok;
    if (tid == 0) {
        for (int i = 0; i < NST; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], Y ? 5 : 1);  // the last MMA, and the four epilogue warps
            mbar_init(&kt_full[i], 8);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&qk_full[i], 1);
            mbar_init(&qk_empty[i], 2);
            mbar_init(&p_full[i], 2);
            mbar_init(&p_empty[i], 4);
        }
        mbar_init(kv_full, 1);
        mbar_init(s_full, 8);
        mbar_init(qs_done, 1);
        mbar_init(o_full, 1);
        mbar_init(o_empty, 4);
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

    const int work0 = la_share(L.nwork, blockIdx.x), work1 = la_share(L.nwork, blockIdx.x + 1);
    bool ok = true;
    uint32_t issued = 0;  // chunks whose loads were issued (producer)

    if (warp == 14) {
        // ------------------------------------------------------------------ producer
        const uint32_t tx = (uint32_t)(Cfg::StageBytes / kLaBlock) * (uint32_t)L.box_rows * 128u;
        uint32_t pos = 0;
        for (int work = work0; work < work1 && ok; ++work) {
            const LaItem it = la_item<Y>(L, work);
            if (work + 1 < work1 && elect_one()) {
                // the next item's initial state into L2: its load stands at the head of that item's chain
                const float* in = la_item<Y>(L, work + 1).in;
                if (in)
                    asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(in), "r"(p.dk * p.dv * 4) : "memory");
            }
            __syncwarp();
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
        constexpr uint32_t n_tok = (uint32_t)(kLaTok >> 3) << 17, n_dk = (uint32_t)(DK >> 3) << 17;
        const uint32_t dq = la_k_desc(smem_addr(smem)), dk = la_k_desc(smem_addr(smem + Cfg::QBytes));
        const uint32_t dv = la_mn_desc(smem_addr(smem + Cfg::QBytes + Cfg::KBytes));
        const uint32_t dkt = la_mn_desc(smem_addr(kt)), dp = la_k_desc(smem_addr(pbuf));
        auto stage_off = [&](uint32_t pos) { return (pos % NST) * (uint32_t)(Cfg::StageBytes >> 4); };
        // scores of the chunk at `pos`, whose tiles have landed
        auto scores = [&](uint32_t pos) -> bool {
            if (!la_wait(&qk_empty[pos & 1], ((pos >> 1) & 1u) ^ 1u)) return false;
            tc_fence_after();
            if (elect_one()) {
                const uint32_t so = stage_off(pos), a = dq + so, b = dk + so, d = tmem + Cfg::QK + (pos & 1) * 64;
#pragma unroll
                for (int kk = 0; kk < DK / 16; ++kk) {
                    const uint32_t o = ((kk >> 2) * kLaBlock + (kk & 3) * 32) >> 4;
                    la_mma(d, a + o, b + o, kDesc | n_tok, kk > 0);
                }
                tc_commit(&qk_full[pos & 1]);
            }
            __syncwarp();
            return true;
        };
        uint32_t pos = 0, nqs = 0, nqk = 0;
        for (int work = work0; work < work1 && ok; ++work) {
            const LaItem it = la_item<Y>(L, work);
            for (int c = it.a; c < it.b && ok; ++c, ++pos) {
                const bool has = it.in || c > it.a, need = c < it.b - 1 || it.out;
                const int st = pos % NST;
                const uint32_t so = stage_off(pos);
                if (!(ok = la_wait(&full[st], (pos / NST) & 1u))) break;
                if (Y && nqk == pos) {
                    if (!(ok = scores(pos))) break;
                    nqk = pos + 1;
                }
                if (!(ok = la_wait(&kt_full[st], (pos / NST) & 1u))) break;
                if (need) {
                    tc_fence_after();
                    if (elect_one()) {
                        const uint32_t b = Y ? 0 : pos & 1;  // the state pass has two of K~ and of KV
#pragma unroll
                        for (int part = 0; part < 3; ++part)
                            if (part < 2 || L.nsplit > 2)
#pragma unroll
                                for (int kk = 0; kk < 4; ++kk)
                                    la_mma(tmem + Cfg::KV + b * 128, dv + so + (kk * 2048 >> 4),
                                           dkt + b * (Cfg::KtBuf >> 4) + ((part * Cfg::KBytes + kk * 2048) >> 4),
                                           kDesc | kMnA | kMnB | n_dk, part > 0 || kk > 0);
                        tc_commit(Y ? kv_full : &qk_full[b]);
                        if (!Y) tc_commit(&empty[st]);
                    }
                    __syncwarp();
                }
                if (Y) {
                    // the next chunk's scores early, if its tiles are there (behind the last chunk they never are)
                    if (la_test(&full[(pos + 1) % NST], ((pos + 1) / NST) & 1u)) {
                        if (!(ok = scores(pos + 1))) break;
                        nqk = pos + 2;
                    }
                    if (!(ok = la_wait(o_empty, (pos & 1u) ^ 1u))) break;
                    if (has) {
                        if (!(ok = la_wait(s_full, nqs & 1u))) break;
                        tc_fence_after();
                        if (elect_one()) {
#pragma unroll
                            for (int part = 0; part < 2; ++part)
#pragma unroll
                                for (int kk = 0; kk < DK / 16; ++kk)
                                    la_mma_ts(tmem + Cfg::OI, tmem + Cfg::SB + part * (DK / 2) + kk * 8,
                                              dq + so + (((kk >> 2) * kLaBlock + (kk & 3) * 32) >> 4), kDesc | n_tok,
                                              part > 0 || kk > 0);
                            tc_commit(qs_done);
                        }
                        __syncwarp();
                        ++nqs;
                    }
                    if (!(ok = la_wait(&p_full[pos & 1], (pos >> 1) & 1u))) break;
                    tc_fence_after();
                    if (elect_one()) {
#pragma unroll
                        for (int part = 0; part < 2; ++part)
#pragma unroll
                            for (int kk = 0; kk < 4; ++kk)
                                la_mma(tmem + Cfg::OA, dv + so + (kk * 2048 >> 4),
                                       dp + (pos & 1) * (Cfg::PPart * 2 >> 4) + ((part * Cfg::PPart + kk * 32) >> 4),
                                       kDesc | kMnA | n_tok, part > 0 || kk > 0);
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
        float2 S[H / 2];
        // of the head and chunk length at hand: the chunk's decay, and the weights of the two tokens whose keys this
        // thread scales
        float dhi = 0.f, dlo = 0.f, kw[2] = {0.f, 0.f};
        int head = -1, kw_n = -1, d_n = -1;
        float g = 0.f;
        uint32_t pos = 0, nkv = 0, nqs = 0;
        for (int work = work0; work < work1 && ok; ++work) {
            const LaItem it = la_item<Y>(L, work);
#pragma unroll
            for (int i = 0; i < H / 2; ++i) S[i] = make_float2(0.f, 0.f);
            if (it.in && live) {
                if (it.in_t) {
                    const float* a = it.in + (size_t)row * p.dk + k0;
#pragma unroll
                    for (int i = 0; i < H; i += 4)
                        if (k0 + i < p.dk) {
                            const float4 x = *reinterpret_cast<const float4*>(a + i);
                            S[i / 2] = make_float2(x.x, x.y);
                            S[i / 2 + 1] = make_float2(x.z, x.w);
                        }
                } else {
                    const float* a = it.in + (size_t)k0 * p.dv + row;
#pragma unroll
                    for (int i = 0; i < H; i += 2)  // dk is a multiple of 8
                        if (k0 + i < p.dk) S[i / 2] = make_float2(a[(size_t)i * p.dv], a[(size_t)(i + 1) * p.dv]);
                }
            }
            if (it.h != head) {
                head = it.h;
                g = la_clamp_decay(p.log_decay[head]);
                kw_n = d_n = -1;
            }
            // K~ of the chunk c, the at-th of this CTA
            auto keys = [&](int c, uint32_t at) -> bool {
                int row0, n;
                la_chunk(p, it, c, row0, n);
                const int st = at % NST;
                if (!la_wait(&full[st], (at / NST) & 1u)) return false;
                if (c < it.b - 1 || it.out) {
                    unsigned char* s = smem + st * Cfg::StageBytes;
                    if (n != kw_n) {
                        kw_n = n;
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const int j = (tid >> 3) + 32 * e;
                            kw[e] = j < n ? p.s_in * la_decay_pow(g, (float)((p.reverse ? j : n - 1 - j) + p.shift)) : 0.f;
                        }
                    }
                    // K~: the swizzle only permutes 16-byte pieces within a token's row.  Piece tid + 256 m belongs to token
                    // tid / 8 + 32 (m % 2); all pieces are fetched before the first is written
                    uint4 x[Cfg::KB * 2];
#pragma unroll
                    for (int m = 0; m < Cfg::KB * 2; ++m) {
                        x[m] = make_uint4(0, 0, 0, 0);
                        if ((tid >> 3) + 32 * (m & 1) < n) x[m] = *reinterpret_cast<const uint4*>(s + Cfg::QBytes + (tid + m * 256) * 16);
                    }
#pragma unroll
                    for (int m = 0; m < Cfg::KB * 2; ++m) {
                        const float2 w = make_float2(kw[m & 1], kw[m & 1]);
                        const uint32_t xs[4] = {x[m].x, x[m].y, x[m].z, x[m].w};
                        float2 a[4];
                        uint32_t t[4];
                        unsigned char* o = kt + (Y ? 0 : (at & 1) * Cfg::KtBuf) + (tid + m * 256) * 16;
#pragma unroll
                        for (int e = 0; e < 4; ++e) a[e] = mul2(make_float2(la_bf16_lo(xs[e]), la_bf16_hi(xs[e])), w);
#pragma unroll
                        for (int part = 0; part < 3; ++part) {
                            if (part == 2 && L.nsplit < 3) break;
#pragma unroll
                            for (int e = 0; e < 4; ++e) t[e] = part < 2 ? la_split(a[e]) : pack_bf16x2(a[e].x, a[e].y);
                            *reinterpret_cast<uint4*>(o + part * Cfg::KBytes) = make_uint4(t[0], t[1], t[2], t[3]);
                        }
                    }
                    if (n < kLaTok && row0 + n < p.seq_len) la_zero_rows(s + Cfg::QBytes + Cfg::KBytes, Cfg::VB, n, tid, 256);
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                }
                la_arrive(&kt_full[st]);
                return true;
            };
            // the state pass, which has room for two, prepares the next chunk's before it waits for this one's product
            if (!Y && it.a < it.b && !(ok = keys(it.a, pos))) break;
            for (int c = it.a; c < it.b; ++c, ++pos) {
                const bool has = it.in || c > it.a, need = c < it.b - 1 || it.out;
                int row0, n;
                la_chunk(p, it, c, row0, n);
                if (Y ? !(ok = keys(c, pos)) : c + 1 < it.b && !(ok = keys(c + 1, pos + 1))) break;
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
                            for (int e = 0; e < 16; ++e) w[e] = la_pack_sat(S[q * 16 + e].x, S[q * 16 + e].y);
                            tc_st16(to, w);
#pragma unroll
                            for (int e = 0; e < 16; ++e) {
                                float2 x = S[q * 16 + e];
                                la_split<true>(x);
                                w[e] = pack_bf16x2(x.x, x.y);
                            }
                            tc_st16(to + DK / 2, w);
                        }
                        tc_wait_st();
                    }
                    tc_fence_before();
                    la_arrive(s_full);
                    ++nqs;
                }
                if (need) {
                    if (!(ok = Y ? la_wait(kv_full, nkv & 1u) : la_wait(&qk_full[pos & 1], (pos >> 1) & 1u))) break;
                    ++nkv;
                    tc_fence_after();
                    if (n != d_n) {
                        d_n = n;
                        la_decay_pair(g, (float)n, dhi, dlo);
                    }
                    if (rows_used) {
#pragma unroll
                        for (int q = 0; q < H / 32; ++q) {
                            uint32_t r[32];
                            tc_ld32_issue(tmem + lane_off + Cfg::KV + (Y ? 0 : (pos & 1) * 128) + k0 + q * 32, r);
                            tc_wait_ld32(r);
#pragma unroll
                            for (int e = 0; e < 16; ++e) {
                                const float2 x = S[q * 16 + e];
                                const float2 kv = make_float2(__uint_as_float(r[2 * e]), __uint_as_float(r[2 * e + 1]));
                                S[q * 16 + e] = fma2(x, make_float2(dhi, dhi), fma2(x, make_float2(dlo, dlo), kv));
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
                        if (k0 + i < p.dk) *reinterpret_cast<float4*>(a + i) = make_float4(S[i / 2].x, S[i / 2].y, S[i / 2 + 1].x, S[i / 2 + 1].y);
                } else {
                    float* a = it.out + (size_t)k0 * p.dv + row;
#pragma unroll
                    for (int i = 0; i < H; ++i)
                        if (k0 + i < p.dk) a[(size_t)i * p.dv] = i & 1 ? S[i / 2].y : S[i / 2].x;
                }
            }
        }
    } else if (Y && warp < 12) {
        // ------------------------------------------------------------------ epilogue
        const int quarter = warp & 3, c0 = quarter * 32;  // this warp's channels c0 .. c0 + 31
        const uint32_t lane_off = (uint32_t)c0 << 16;
        const bool used = c0 < p.dv;                      // warp-uniform
        const int fc = (lane & 3) * 2;                    // this thread's column of an 8 x 8 fragment
        float2 fac[8];  // s_out gamma^(position + 1 - shift) of tokens 8 k + fc, 8 k + fc + 1, for the head and chunk length
        int head = -1, fac_n = -1;
        float g = 0.f;
        uint32_t pos = 0;
        for (int work = work0; work < work1 && ok; ++work) {
            const LaItem it = la_item<Y>(L, work);
            if (it.h != head) {
                head = it.h;
                g = la_clamp_decay(p.log_decay[head]);
                fac_n = -1;
            }
            for (int c = it.a; c < it.b; ++c, ++pos) {
                const bool has = it.in || c > it.a;
                const int st = pos % NST;
                int row0, n;
                la_chunk(p, it, c, row0, n);
                if (has && n != fac_n) {
                    fac_n = n;
                    __syncwarp();
#pragma unroll
                    for (int i = lane; i < kLaTok; i += 32)
                        wtab[i] = i < n ? p.s_out * la_decay_pow(g, (float)((p.reverse ? n - 1 - i : i) + 1 - p.shift)) : 0.f;
                    __syncwarp();
#pragma unroll
                    for (int k = 0; k < 8; ++k) fac[k] = *reinterpret_cast<const float2*>(wtab + 8 * k + fc);
                }
                if (!(ok = la_wait(o_full, pos & 1u))) break;
                tc_fence_after();
                unsigned char* tile = smem + st * Cfg::StageBytes + quarter * (kLaBlock / 2);
                // channels c0 + 16 half ..; bf16 results wait in w until the accumulators are given back
                uint32_t w[2][16];
                if (used) {
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        uint32_t r[32], s2[32];
                        const uint32_t ta = tmem + lane_off + ((uint32_t)(half * 16) << 16);
                        tc_ld_frag_issue(ta + Cfg::OA, r);
                        if (has) tc_ld_frag_issue(ta + Cfg::OI, s2);
                        tc_wait_ld32(r);
                        if (has) {
                            tc_wait_ld32(s2);
                            la_add_inter(r, s2, fac);
                        }
                        uint32_t big = 0;
#pragma unroll
                        for (int k = 0; k < 16; ++k) {
                            w[half][k] = pack_bf16x2(__uint_as_float(r[2 * k]), __uint_as_float(r[2 * k + 1]));
                            big = la_absmax_bf16x2(big, w[half][k]);
                        }
                        const bool redo = __any_sync(0xffffffffu, la_not_finite(big));
                        if (redo || row0 + n < min(row0 + kLaTok, p.seq_len) || p.y_f32) {
                            if (redo) {
                                la_wait(&p_full[pos & 1], (pos >> 1) & 1u);
                                la_wait(&full[st], (pos / NST) & 1u);
                            }
                            uint32_t out[32];
#pragma unroll
                            for (int e = 0; e < 32; ++e) out[e] = r[e];
                            la_finish(out, redo, pbuf + (pos & 1) * 2 * Cfg::PPart,
                                      smem + st * Cfg::StageBytes + Cfg::QBytes + Cfg::KBytes + (c0 >> 6) * kLaBlock,
                                      has ? ta + Cfg::OI : 0u, wtab, c0 + half * 16, n, p, it.seq, it.h, row0);
#pragma unroll
                            for (int k = 0; k < 16; ++k)
                                w[half][k] = pack_bf16x2(__uint_as_float(out[2 * k]), __uint_as_float(out[2 * k + 1]));
                        }
                    }
                }
                // both accumulators, P and V have been read
                tc_fence_before();
                la_arrive(o_empty);
                __syncwarp();
                if (lane == 0) mbar_arrive(&p_empty[pos & 1]);
                if (used && !p.y_f32) {
                    // [token][32 channels], 64-byte rows, 16-byte pieces swizzled by the row pair
                    const uint32_t ts = smem_addr(tile);
                    const int tr = lane & 7;
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        const int m = half * 2 + ((lane >> 3) & 1);
#pragma unroll
                        for (int k = 0; k < 8; ++k) {
                            const int i = 8 * k + tr;
                            st_matrix2_trans(ts + i * 64 + ((m ^ ((i >> 1) & 3)) << 4), w[half][2 * k], w[half][2 * k + 1]);
                        }
                    }
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                    __syncwarp();
                    if (lane == 0) {
                        tma_store_4d(&L.ty, tile, c0, it.h, row0, it.seq);
                        asm volatile("cp.async.bulk.commit_group;" ::: "memory");
                        asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
                    }
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&empty[st]);
            }
            // chunks that lie wholly behind the row's tokens: zeros
            if (it.a == 0 && ok && it.nch * kLaTok < p.seq_len) la_zero_tail(p, it.seq, it.h, it.nch * kLaTok, tid - 256);
        }
        if (lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
    } else if (Y && warp < 14) {
        // ------------------------------------------------------------------ scores
        const int w = warp - 12, i = 32 * w + lane;  // the row (token) of this thread
        const uint32_t lane_off = (uint32_t)(32 * w) << 16;
        unsigned char* const prow = pbuf + i * 128;
        // of the two blocks off the diagonal one is all masked: it stays zero
        const bool full_block = p.reverse ? w == 0 : w == 1;
#pragma unroll
        for (int q = 0; q < 8; ++q)
#pragma unroll
            for (int part = 0; part < 4; ++part)
                *reinterpret_cast<uint4*>(prow + part * Cfg::PPart + q * 16) = make_uint4(0, 0, 0, 0);
        __syncwarp();
        const float s = p.s_in * p.s_out;
        // weights of this row, for the head at hand: on the diagonal block, and on the full one (its columns are farther)
        float2 wd[16], wo[16];
        int head = -1;
        float g = 0.f;
        uint32_t pos = 0;
        for (int work = work0; work < work1 && ok; ++work) {
            const LaItem it = la_item<Y>(L, work);
            if (it.b > it.a && it.h != head) {
                head = it.h;
                g = la_clamp_decay(p.log_decay[head]);
                __syncwarp();
                wtab[lane] = s * la_decay_pow(g, (float)lane);
                wtab[lane + 32] = s * la_decay_pow(g, (float)(lane + 32));
                __syncwarp();
#pragma unroll
                for (int j = 0; j < 32; j += 2) {
                    auto diag = [&](int c) { return (p.reverse ? c >= lane : c <= lane) ? wtab[abs(lane - c)] : 0.f; };
                    wd[j / 2] = make_float2(diag(j), diag(j + 1));
                    wo[j / 2] = p.reverse ? make_float2(wtab[32 + j - lane], wtab[33 + j - lane])
                                          : make_float2(wtab[32 + lane - j], wtab[31 + lane - j]);
                }
            }
            for (int c = it.a; c < it.b; ++c, ++pos) {
                int row0, n;
                la_chunk(p, it, c, row0, n);
                if (!(ok = la_wait(&qk_full[pos & 1], (pos >> 1) & 1u))) break;
                tc_fence_after();
                const uint32_t ta = tmem + lane_off + Cfg::QK + (pos & 1) * 64;
                unsigned char* pb = prow + (pos & 1) * 2 * Cfg::PPart;
                uint32_t r[32];
                // 32 scores of this row, weighted, in two bf16 parts, to columns c0 .. c0 + 31 of P
                auto put = [&](int col0, const float2 (&wt)[16]) {
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        uint32_t a[4], b[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            float2 x = mul2(make_float2(__uint_as_float(r[q * 8 + 2 * e]), __uint_as_float(r[q * 8 + 2 * e + 1])),
                                               wt[q * 4 + e]);
                            a[e] = la_split<true>(x);
                            b[e] = pack_bf16x2(x.x, x.y);
                        }
                        unsigned char* o = pb + ((((col0 >> 3) + q) ^ (i & 7)) << 4);
                        *reinterpret_cast<uint4*>(o) = make_uint4(a[0], a[1], a[2], a[3]);
                        *reinterpret_cast<uint4*>(o + kLaBlock) = make_uint4(b[0], b[1], b[2], b[3]);
                    }
                };
                tc_ld32_issue(ta + 32 * w, r);
                tc_wait_ld32(r);
                // masked scores are zeros, not scores times zero: a key there may be infinite
                const int left = n - 32 * w;  // columns inside the length
                const uint32_t keep = (p.reverse ? ~0u << lane : 2u * (1u << lane) - 1u) & (left >= 32 ? ~0u : left <= 0 ? 0u : (1u << left) - 1u);
#pragma unroll
                for (int j = 0; j < 32; ++j) r[j] = keep >> j & 1u ? r[j] : 0u;
                if (!(ok = la_wait(&p_empty[pos & 1], ((pos >> 1) & 1u) ^ 1u))) break;
                put(32 * w, wd);
                if (full_block && n > 32) {
                    tc_ld32_issue(ta + 32 * (1 - w), r);
                    tc_wait_ld32(r);
                    if (p.reverse && n < kLaTok)
#pragma unroll
                        for (int j = 0; j < 32; ++j) r[j] = 32 + j < n ? r[j] : 0u;
                    put(32 * (1 - w), wo);
                }
                tc_fence_before();
                la_arrive(&qk_empty[pos & 1]);
                if (n < kLaTok && row0 + n < p.seq_len) {
                    const int st = pos % NST;
                    if (!(ok = la_wait(&full[st], (pos / NST) & 1u))) break;
                    la_zero_rows(smem + st * Cfg::StageBytes + Cfg::QBytes + Cfg::KBytes, Cfg::VB, n, i, 64);
                }
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                la_arrive(&p_full[pos & 1]);
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

// ------------------------------------------------------------------------------------ host

// [seq][token][head][channel] with the given element strides, boxes of box_rows tokens x box_cols (64 or 32) channels
// of a head.
inline bool la_encode(CUtensorMap* out, const void* base, int d, int heads, int seq_len, int nseq, long long tok, int box_rows,
                      int box_cols = 64) {
    auto enc = tensor_map_encoder();
    if (!enc) {
        snprintf(last_error_buffer(), 256, "cuTensorMapEncodeTiled: driver entry point unavailable");
        return false;
    }
    cuuint64_t dims[4] = {(cuuint64_t)d, (cuuint64_t)heads, (cuuint64_t)seq_len, (cuuint64_t)nseq};
    cuuint64_t strides[3] = {(cuuint64_t)d * 2, (cuuint64_t)tok * 2, (cuuint64_t)tok * 2 * (cuuint64_t)seq_len};
    cuuint32_t box[4] = {(cuuint32_t)box_cols, 1, (cuuint32_t)box_rows, 1};
    cuuint32_t estr[4] = {1, 1, 1, 1};
    const CUresult r = enc(out, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(base), dims, strides, box, estr,
                           CU_TENSOR_MAP_INTERLEAVE_NONE,
                           box_cols == 64 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                           CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r == CUDA_SUCCESS) return true;
    snprintf(last_error_buffer(), 256, "cuTensorMapEncodeTiled failed (CUresult %d)", (int)r);
    return false;
}

// How a pass is divided: segments per sequence and chunks in each.  Few (sequence, head) pairs are divided into as many
// segments as fill the SMs, of four chunks at least.  Dividing runs the state part of a chunk (half its time) twice and
// adds two launches and the segments' states, 14 us and 0.2 a pair: n segments pay where (1 - 1.55 / n) nch chunk times
// (2 us) exceed that.  Heads of 128, undivided and divided: 64 pairs, n = 2: 32 chunks 73 and 87 us, 47 chunks 102 and 112,
// 64 chunks 135 and 140; 32 pairs, n = 4, 16 chunks 38 and 39; 8 pairs, n = 4, 16 chunks 38 and 32; 16 pairs, n = 9, 512 chunks
// 1030 and 222 us.  The rule is fitted to those.  Heads of 64 have shorter chunks (1.5 us), cheaper states and much the same
// borders: 64 pairs: 32 chunks 53 and 53, 47 chunks 75 and 71, 64 chunks 99 and 91; 32 pairs, 16 chunks 29 and 26; 8 pairs, 10
// chunks 20 and 24, 16 chunks 28 and 22.  (One launch in which the second part's CTA forms the state before it itself gained
// nothing: the state is what takes the time.)
inline void la_segments(int nseq, int heads, int seq_len, int nsm, int& nseg, int& seg_chunks) {
    const long long items = (long long)nseq * heads;
    const int nch = (seq_len + kLaTok - 1) / kLaTok;
    nseg = items > 0 ? (int)std::min<long long>(nsm / items, nch / 4) : 1;
    if (nseg < 2 || (20 * nseg - 31LL) * nch < (140 + 2 * items) * nseg) nseg = 1;
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
    L.nsplit = p.h_last ? 3 : 2;
    if (!la_encode(&L.tq, p.q, p.dk, p.heads / p.q_div, p.seq_len, p.nseq, p.q_tok, L.box_rows) ||
        !la_encode(&L.tk, p.k, p.dk, p.heads / p.k_div, p.seq_len, p.nseq, p.k_tok, L.box_rows) ||
        !la_encode(&L.tv, p.v, p.dv, p.heads / p.v_div, p.seq_len, p.nseq, p.v_tok, L.box_rows))
        return false;
    if (!p.y_f32 && !la_encode(&L.ty, p.y, p.dv, p.heads, p.seq_len, p.nseq, p.y_tok, L.box_rows, 32)) return false;
    if (L.nseg > 1) {
        L.nwork = p.nseq * p.heads * (L.nseg - 1);
        if (!la_tc_pick<false>(L, nsm, stream)) return false;
        const dim3 grid((unsigned)((p.dk * p.dv + 255) / 256), (unsigned)(p.nseq * p.heads));
        LaPasses one;
        std::memset(&one, 0, sizeof(one));
        one.p[0] = p;
        one.seg[0] = seg;
        one.nseg = L.nseg;
        one.seg_tok = L.seg_chunks * kLaTok;
        if (!cuda_ok(launch_pdl(linattn_segments_kernel, grid, dim3(256), 0, stream, one),
                     "linear attention segment kernel launch"))
            return false;
    }
    L.nwork = p.nseq * p.heads * L.nseg;
    return la_tc_pick<true>(L, nsm, stream);
}

}  // namespace r2l
