// mixer.cu -- host side of libr2l_mixer: argument validation, kernel choice and the extern "C" entry points
// declared in include/r2l_mixer.h.  Single translation unit, as libr2l.
#include <algorithm>
#include <atomic>
#include <climits>
#include <cstdint>
#include <cstring>

#include "r2l_mixer.h"
#include "../common.cuh"
#include "linattn_block.cuh"
#include "linattn_common.cuh"
#include "linattn_rec.cuh"
#include "linattn_tc.cuh"
#include "qk_norm_rope.cuh"

namespace r2l {
namespace {

constexpr int kMixerAbiVersion = 100;

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline bool aligned256(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 255u) == 0; }
inline int esize(r2l_dtype t) { return t == R2L_BF16 ? 2 : 4; }
inline bool valid_dtype(r2l_dtype t) { return t == R2L_F32 || t == R2L_BF16; }
inline size_t align256(size_t v) { return (v + 255) & ~size_t(255); }

// SMs of the current device (asked once per device).
int sm_count() {
    static std::atomic<int> known[64];
    int dev = 0, v = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return 148;
    if (dev >= 0 && dev < 64 && (v = known[dev].load(std::memory_order_relaxed)) > 0) return v;
    if (cudaDeviceGetAttribute(&v, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || v <= 0) return 148;
    if (dev >= 0 && dev < 64) known[dev].store(v, std::memory_order_relaxed);
    return v;
}

// ---------------------------------------------------------------------------- linear attention

bool la_empty(const r2l_linattn_args* a) { return a->batch == 0 || a->n_heads == 0 || a->d_v == 0 || a->d_k == 0; }

// Checks everything but the outputs.
r2l_status check_linattn(const r2l_linattn_args* a) {
    if (!a) return R2L_ERR_INVALID_ARG;
    if (a->batch < 0 || a->seqlen < 0 || a->n_heads < 0 || a->d_k < 0 || a->d_v < 0) return R2L_ERR_INVALID_ARG;
    if (!valid_dtype(a->dtype)) return R2L_ERR_INVALID_ARG;
    const int vec = 16 / esize(a->dtype);
    if (a->d_k > kRecMaxD || a->d_v > kRecMaxD) return R2L_ERR_UNSUPPORTED;
    if (a->d_k % vec != 0 || a->d_v % vec != 0) return R2L_ERR_INVALID_ARG;
    if (a->reverse && a->seqlen > 0 && (a->block_len <= 0 || a->seqlen % a->block_len != 0)) return R2L_ERR_INVALID_ARG;
    if (a->seq_lens && a->reverse && a->block_len != a->seqlen) return R2L_ERR_INVALID_ARG;
    if (reinterpret_cast<uintptr_t>(a->seq_lens) & 3u) return R2L_ERR_INVALID_ARG;
    if (a->n_heads > 0)
        for (int n : {a->q_heads, a->k_heads, a->v_heads})
            if (n <= 0 || a->n_heads % n != 0) return R2L_ERR_INVALID_ARG;
    const long long strides[3] = {a->q_stride, a->k_stride, a->v_stride};
    const long long dense[3] = {(long long)a->q_heads * a->d_k, (long long)a->k_heads * a->d_k, (long long)a->v_heads * a->d_v};
    for (int i = 0; i < 3; ++i)
        if (strides[i] != 0 && (strides[i] < dense[i] || strides[i] % vec != 0 || strides[i] > (1LL << 38)))
            return R2L_ERR_INVALID_ARG;
    if (la_empty(a)) return R2L_OK;
    // the kernels' token counters run a few chunks past the last token
    if ((long long)a->batch * a->seqlen > INT_MAX - 256 || (long long)a->batch * a->n_heads > INT_MAX) return R2L_ERR_UNSUPPORTED;
    const long long nblk = a->reverse && a->seqlen > 0 ? a->seqlen / a->block_len : 1;
    if (a->batch * nblk * a->n_heads > INT_MAX) return R2L_ERR_UNSUPPORTED;
    if (!a->log_decay || (reinterpret_cast<uintptr_t>(a->log_decay) & 3u)) return R2L_ERR_INVALID_ARG;
    if (a->seqlen == 0) return R2L_OK;
    if (!a->q || !a->k || !a->v || !aligned16(a->q) || !aligned16(a->k) || !aligned16(a->v)) return R2L_ERR_INVALID_ARG;
    return R2L_OK;
}

// States are carried across one sequence per row: forward, or a reverse run without inner blocks.
bool carries_state(const r2l_linattn_args* a) { return !a->reverse || a->block_len == a->seqlen; }

LaPass forward_pass(const r2l_linattn_args* a, const float* h0, float* h_last, void* y) {
    LaPass p;
    std::memset(&p, 0, sizeof(p));
    const int nblk = a->reverse ? a->seqlen / a->block_len : 1;
    p.nseq = a->batch * nblk;
    p.seq_len = a->seqlen / nblk;
    p.heads = a->n_heads;
    p.q = a->q, p.k = a->k, p.v = a->v, p.y = y;
    p.q_tok = a->q_stride ? a->q_stride : (long long)a->q_heads * a->d_k;
    p.k_tok = a->k_stride ? a->k_stride : (long long)a->k_heads * a->d_k;
    p.v_tok = a->v_stride ? a->v_stride : (long long)a->v_heads * a->d_v;
    p.y_tok = (long long)a->n_heads * a->d_v;
    p.q_div = a->n_heads / a->q_heads;
    p.k_div = a->n_heads / a->k_heads;
    p.v_div = a->n_heads / a->v_heads;
    p.dk = a->d_k;
    p.dv = a->d_v;
    p.reverse = a->reverse ? 1 : 0;
    p.log_decay = a->log_decay;
    p.lens = a->seq_lens;
    p.h0 = h0;
    p.h_last = h_last;
    p.s_in = 1.f;
    p.s_out = a->scale;
    return p;
}

// Workspace of n passes (the states between a divided sequence's segments): one after another in bf16, at once in fp32.
size_t pass_bytes(const r2l_linattn_args* a, int n) {
    const int nblk = a->reverse ? a->seqlen / a->block_len : 1, len = a->seqlen / nblk;
    return align256(a->dtype == R2L_BF16 ? la_segment_bytes(a->batch * nblk, a->n_heads, len, a->d_k, a->d_v, sm_count())
                                         : rec_segment_bytes(a->batch * nblk, a->n_heads, len, n, a->d_k, a->d_v, sm_count()));
}

// `n` passes over the same sequences and heads; seg: pass_bytes bytes.  fp32 runs token by
// token; bf16 in chunks, short blocks by the kernels for them (the gradients of a block with a state transpose it,
// which the resuming kernel does not).
bool run_passes(const LaPass* p, int n, r2l_dtype dtype, void* seg, cudaStream_t stream) {
    const int nsm = sm_count();
    if (dtype == R2L_F32) return cuda_ok(linattn_rec_launch(p, n, static_cast<float*>(seg), nsm, stream), "linear attention kernel launch");
    bool state = false;
    for (int i = 0; i < n; ++i) state = state || p[i].h0 || p[i].h_last;
    if (!state && p->seq_len <= kBlkMaxTok)
        return cuda_ok(linattn_block_launch(p, n, stream), "linear attention block kernel launch");
    if (n == 1 && p->seq_len <= linattn_resume_max(*p))
        return cuda_ok(linattn_resume_launch(*p, nsm, stream), "linear attention block kernel launch");
    for (int i = 0; i < n; ++i)
        if (!linattn_tc_launch(p[i], static_cast<float*>(seg), nsm, stream)) return false;
    return true;
}

r2l_status copy_state(const float* h0, float* h_last, size_t n, cudaStream_t stream) {
    if (!h_last || h_last == h0 || n == 0) return R2L_OK;
    const unsigned blocks = (unsigned)std::min<size_t>((n + 255) / 256, 148 * 8);
    return cuda_ok(launch_pdl(linattn_copy_state_kernel, dim3(blocks), dim3(256), 0, stream, h0, h_last, n),
                   "linear attention state copy launch")
               ? R2L_OK
               : R2L_ERR_CUDA;
}

// An output [batch][seqlen][heads][d] whose sums have no terms (no heads, or no channels to sum over): zeros.
r2l_status zero_output(const r2l_linattn_args* a, void* out, int heads, int d, cudaStream_t stream) {
    if (!out || heads <= 0 || d == 0) return R2L_OK;
    // d is a multiple of 16 bytes
    return copy_state(nullptr, static_cast<float*>(out), (size_t)a->batch * a->seqlen * heads * (d * esize(a->dtype) / 4), stream);
}

// Workspace of the backward call: per-head fp32 gradients of those of q, k, v whose heads are shared.
struct BwdParts {
    size_t off[3], total;
};
BwdParts bwd_parts(const r2l_linattn_args* a) {
    const size_t rows = (size_t)a->batch * a->seqlen * a->n_heads;
    const int groups[3] = {a->q_heads, a->k_heads, a->v_heads}, d[3] = {a->d_k, a->d_k, a->d_v};
    BwdParts w;
    w.total = 0;
    for (int i = 0; i < 3; ++i) {
        w.off[i] = w.total;
        if (groups[i] != a->n_heads) w.total += align256(rows * d[i] * sizeof(float));
    }
    return w;
}

bool bad_workspace(const void* ws, size_t have, size_t need) { return need > 0 && (!ws || !aligned256(ws) || have < need); }

}  // namespace
}  // namespace r2l

using namespace r2l;

extern "C" {

size_t r2l_linattn_workspace_size(const r2l_linattn_args* a) {
    if (check_linattn(a) != R2L_OK || la_empty(a) || a->seqlen == 0) return 0;
    return pass_bytes(a, 1);
}

r2l_status r2l_linattn(const r2l_linattn_args* a, const float* h0, float* h_last, void* y, void* workspace,
                       size_t workspace_bytes, cudaStream_t stream) {
    r2l_status st = check_linattn(a);
    if (st != R2L_OK) return st;
    if ((h0 || h_last) && !carries_state(a)) return R2L_ERR_INVALID_ARG;
    if (!aligned16(h0) || !aligned16(h_last)) return R2L_ERR_INVALID_ARG;
    if (la_empty(a)) return aligned16(y) ? zero_output(a, y, a->n_heads, a->d_v, stream) : R2L_ERR_INVALID_ARG;
    if (a->seqlen == 0) return copy_state(h0, h_last, (size_t)a->batch * a->n_heads * a->d_k * a->d_v, stream);
    if (!y || !aligned16(y)) return R2L_ERR_INVALID_ARG;
    if (bad_workspace(workspace, workspace_bytes, r2l_linattn_workspace_size(a))) return R2L_ERR_INVALID_ARG;
    const LaPass p = forward_pass(a, h0, h_last, y);
    return run_passes(&p, 1, a->dtype, workspace, stream) ? R2L_OK : R2L_ERR_CUDA;
}

r2l_status r2l_linattn_step(const r2l_linattn_args* a, const float* h, float* h_out, void* y, cudaStream_t stream) {
    r2l_status st = check_linattn(a);
    if (st != R2L_OK) return st;
    if (a->seqlen != 1 || a->reverse || a->seq_lens) return R2L_ERR_INVALID_ARG;
    if (la_empty(a)) return aligned16(y) ? zero_output(a, y, a->n_heads, a->d_v, stream) : R2L_ERR_INVALID_ARG;
    if (!h || !h_out || !y || !aligned16(h) || !aligned16(h_out) || !aligned16(y)) return R2L_ERR_INVALID_ARG;
    const LaPass p = forward_pass(a, h, h_out, y);
    const cudaError_t e = a->dtype == R2L_F32 ? linattn_step_launch<float>(p, sm_count(), stream)
                                              : linattn_step_launch<__nv_bfloat16>(p, sm_count(), stream);
    return cuda_ok(e, "linear attention step launch") ? R2L_OK : R2L_ERR_CUDA;
}

size_t r2l_linattn_bwd_workspace_size(const r2l_linattn_args* a) {
    if (check_linattn(a) != R2L_OK || la_empty(a) || a->seqlen == 0) return 0;
    return bwd_parts(a).total + pass_bytes(a, 3);
}

r2l_status r2l_linattn_bwd(const r2l_linattn_args* a, const void* dy, const float* h0, const float* dh_last, void* dq,
                           void* dk, void* dv, float* dh0, void* workspace, size_t workspace_bytes, cudaStream_t stream) {
    r2l_status st = check_linattn(a);
    if (st != R2L_OK) return st;
    if ((h0 || dh_last || dh0) && !carries_state(a)) return R2L_ERR_INVALID_ARG;
    if (!aligned16(h0) || !aligned16(dh_last) || !aligned16(dh0)) return R2L_ERR_INVALID_ARG;
    if (dh0 && (dh0 == dh_last || dh0 == h0)) return R2L_ERR_INVALID_ARG;
    if (la_empty(a)) {
        if (!aligned16(dq) || !aligned16(dk) || !aligned16(dv)) return R2L_ERR_INVALID_ARG;
        if ((st = zero_output(a, dq, a->q_heads, a->d_k, stream)) != R2L_OK) return st;
        if ((st = zero_output(a, dk, a->k_heads, a->d_k, stream)) != R2L_OK) return st;
        return zero_output(a, dv, a->v_heads, a->d_v, stream);
    }
    if (a->seqlen == 0) return copy_state(dh_last, dh0, (size_t)a->batch * a->n_heads * a->d_k * a->d_v, stream);
    for (const void* q : {dy, (const void*)dq, (const void*)dk, (const void*)dv})
        if (!q || !aligned16(q)) return R2L_ERR_INVALID_ARG;
    if (bad_workspace(workspace, workspace_bytes, r2l_linattn_bwd_workspace_size(a))) return R2L_ERR_INVALID_ARG;

    const LaPass f = forward_pass(a, h0, nullptr, nullptr);
    const long long rows = (long long)a->batch * a->seqlen, dy_tok = (long long)a->n_heads * a->d_v;
    const BwdParts parts = bwd_parts(a);
    unsigned char* ws = static_cast<unsigned char*>(workspace);
    LaPass p[3] = {f, f, f};
    // dq = (dy, v, k) in scan order from h0 transposed
    p[0].q = dy, p[0].q_tok = dy_tok, p[0].q_div = 1;
    p[0].k = f.v, p[0].k_tok = f.v_tok, p[0].k_div = f.v_div;
    p[0].v = f.k, p[0].v_tok = f.k_tok, p[0].v_div = f.k_div;
    p[0].dk = a->d_v, p[0].dv = a->d_k;
    p[0].h_t = 1;
    // dk = (v, dy, q) against the scan order, the adjoint state transposed
    p[1].q = f.v, p[1].q_tok = f.v_tok, p[1].q_div = f.v_div;
    p[1].k = dy, p[1].k_tok = dy_tok, p[1].k_div = 1;
    p[1].v = f.q, p[1].v_tok = f.q_tok, p[1].v_div = f.q_div;
    p[1].dk = a->d_v, p[1].dv = a->d_k;
    p[1].h_t = 1;
    // dv = (k, q, dy) against the scan order; its final state is dh0
    p[2].q = f.k, p[2].q_tok = f.k_tok, p[2].q_div = f.k_div;
    p[2].k = f.q, p[2].k_tok = f.q_tok, p[2].k_div = f.q_div;
    p[2].v = dy, p[2].v_tok = dy_tok, p[2].v_div = 1;
    for (int i = 1; i < 3; ++i) {
        p[i].reverse = !f.reverse;
        p[i].shift = 1;
        p[i].s_in = a->scale, p[i].s_out = 1.f;
        p[i].h0 = dh_last;
    }
    p[2].h_last = dh0;
    // each into the gradient itself, or (shared heads) per head into the workspace and summed from there
    void* outs[3] = {dq, dk, dv};
    const int groups[3] = {a->q_heads, a->k_heads, a->v_heads};
    for (int i = 0; i < 3; ++i) {
        const bool shared = groups[i] != a->n_heads;
        p[i].y = shared ? static_cast<void*>(ws + parts.off[i]) : outs[i];
        p[i].y_f32 = shared;
        p[i].y_tok = (long long)a->n_heads * p[i].dv;
    }
    if (!run_passes(p, 3, a->dtype, ws + parts.total, stream)) return R2L_ERR_CUDA;
    for (int i = 0; i < 3; ++i) {
        if (!p[i].y_f32) continue;
        const int div = a->n_heads / groups[i], d = p[i].dv;
        const size_t n = (size_t)rows * groups[i] * d;
        const unsigned blocks = (unsigned)std::min<size_t>((n + 255) / 256, 148 * 16);
        const float* part = static_cast<const float*>(p[i].y);
        const cudaError_t e = a->dtype == R2L_BF16
                                  ? launch_pdl(linattn_sum_heads_kernel<__nv_bfloat16>, dim3(blocks), dim3(256), 0, stream, part,
                                               static_cast<__nv_bfloat16*>(outs[i]), n, groups[i], div, d)
                                  : launch_pdl(linattn_sum_heads_kernel<float>, dim3(blocks), dim3(256), 0, stream, part,
                                               static_cast<float*>(outs[i]), n, groups[i], div, d);
        if (!cuda_ok(e, "linear attention head sum launch")) return R2L_ERR_CUDA;
    }
    return R2L_OK;
}

}  // extern "C"

namespace r2l {
namespace {

// ---------------------------------------------------------------------------- norm and rotation

r2l_status check_rope(const r2l_qk_norm_rope_args* a) {
    if (!a) return R2L_ERR_INVALID_ARG;
    if (a->tokens < 0 || a->q_heads < 0 || a->k_heads < 0 || a->head_dim < 0 || a->rot_dim < 0) return R2L_ERR_INVALID_ARG;
    if (!valid_dtype(a->dtype)) return R2L_ERR_INVALID_ARG;
    if (a->head_dim > kRopeMaxDim) return R2L_ERR_UNSUPPORTED;
    if (a->head_dim % 2 != 0 || a->rot_dim % 2 != 0 || a->rot_dim > a->head_dim) return R2L_ERR_INVALID_ARG;
    if (!(a->eps >= 0.f)) return R2L_ERR_INVALID_ARG;
    if ((long long)a->q_heads + a->k_heads > INT_MAX / 8) return R2L_ERR_UNSUPPORTED;
    if ((a->q_stride != 0 && a->q_stride < (long long)a->q_heads * a->head_dim) ||
        (a->k_stride != 0 && a->k_stride < (long long)a->k_heads * a->head_dim))
        return R2L_ERR_INVALID_ARG;
    if (a->tokens == 0 || a->head_dim == 0 || a->q_heads + a->k_heads == 0) return R2L_OK;
    const uintptr_t em = esize(a->dtype) - 1;
    if (a->q_heads > 0 && (!a->q || (reinterpret_cast<uintptr_t>(a->q) & em))) return R2L_ERR_INVALID_ARG;
    if (a->k_heads > 0 && (!a->k || (reinterpret_cast<uintptr_t>(a->k) & em))) return R2L_ERR_INVALID_ARG;
    if ((reinterpret_cast<uintptr_t>(a->q_weight) | reinterpret_cast<uintptr_t>(a->k_weight) |
         reinterpret_cast<uintptr_t>(a->inv_freq)) & 3u)
        return R2L_ERR_INVALID_ARG;
    if (a->rot_dim > 0 && (!a->positions || !a->inv_freq)) return R2L_ERR_INVALID_ARG;
    if (reinterpret_cast<uintptr_t>(a->positions) & (a->position_64 ? 7u : 3u)) return R2L_ERR_INVALID_ARG;
    return R2L_OK;
}

bool rope_empty(const r2l_qk_norm_rope_args* a) { return a->tokens == 0 || a->head_dim == 0 || a->q_heads + a->k_heads == 0; }

RopeParams rope_params(const r2l_qk_norm_rope_args* a) {
    RopeParams p;
    std::memset(&p, 0, sizeof(p));
    p.x[0] = a->q, p.x[1] = a->k;
    p.heads[0] = a->q_heads, p.heads[1] = a->k_heads;
    const long long st[2] = {a->q_stride, a->k_stride};
    for (int w = 0; w < 2; ++w) p.x_tok[w] = st[w] ? st[w] : (long long)p.heads[w] * a->head_dim;
    p.weight[0] = a->q_weight, p.weight[1] = a->k_weight;
    p.positions = a->positions;
    p.inv_freq = a->inv_freq;
    p.tokens = a->tokens;
    p.dim = a->head_dim;
    p.rot = a->rot_dim;
    p.interleaved = a->interleaved ? 1 : 0;
    p.pos64 = a->position_64 ? 1 : 0;
    p.eps = a->eps;
    p.inv_dim = 1.f / (float)a->head_dim;
    return p;
}

// For the narrowest groups, which need the most CTAs: the alignment of the outputs, not known here, may choose others.
size_t rope_part_bytes(const r2l_qk_norm_rope_args* a) {
    return align256((size_t)2 * rope_bwd_ctas(a->tokens, 32) * a->head_dim * sizeof(float));
}

}  // namespace
}  // namespace r2l

extern "C" {

r2l_status r2l_qk_norm_rope(const r2l_qk_norm_rope_args* a, void* q_out, long long q_out_stride, void* k_out,
                            long long k_out_stride, cudaStream_t stream) {
    r2l_status st = check_rope(a);
    if (st != R2L_OK) return st;
    if (rope_empty(a)) return R2L_OK;
    RopeParams p = rope_params(a);
    void* outs[2] = {q_out, k_out};
    const long long strides[2] = {q_out_stride, k_out_stride};
    for (int w = 0; w < 2; ++w) {
        const long long dense = (long long)p.heads[w] * p.dim;
        if (strides[w] != 0 && strides[w] < dense) return R2L_ERR_INVALID_ARG;
        if (p.heads[w] > 0 && (!outs[w] || (reinterpret_cast<uintptr_t>(outs[w]) & (esize(a->dtype) - 1))))
            return R2L_ERR_INVALID_ARG;
        p.out[w] = outs[w];
        p.out_tok[w] = strides[w] ? strides[w] : dense;
    }
    const int heads = a->q_heads + a->k_heads, es = esize(a->dtype);
    p.split = rope_split(a->tokens, heads, rope_lanes(p, es, false), sm_count());
    const cudaError_t e = a->dtype == R2L_BF16 ? rope_launch<false, __nv_bfloat16>(p, 0, stream)
                                               : rope_launch<false, float>(p, 0, stream);
    return cuda_ok(e, "norm and rotation kernel launch") ? R2L_OK : R2L_ERR_CUDA;
}

size_t r2l_qk_norm_rope_bwd_workspace_size(const r2l_qk_norm_rope_args* a) {
    if (check_rope(a) != R2L_OK || rope_empty(a)) return 0;
    return rope_part_bytes(a);
}

r2l_status r2l_qk_norm_rope_bwd(const r2l_qk_norm_rope_args* a, const void* dq_out, const void* dk_out, void* dq, void* dk,
                                float* dq_weight, float* dk_weight, void* workspace, size_t workspace_bytes,
                                cudaStream_t stream) {
    r2l_status st = check_rope(a);
    if (st != R2L_OK) return st;
    if ((reinterpret_cast<uintptr_t>(dq_weight) | reinterpret_cast<uintptr_t>(dk_weight)) & 3u) return R2L_ERR_INVALID_ARG;
    const bool empty = rope_empty(a);
    if (a->head_dim == 0) return R2L_OK;
    RopeParams p = rope_params(a);
    const bool want_w = dq_weight || dk_weight;
    int n = 0;
    if (!empty) {
        const void* dys[2] = {dq_out, dk_out};
        void* outs[2] = {dq, dk};
        const uintptr_t em = esize(a->dtype) - 1;
        for (int w = 0; w < 2; ++w) {
            if (p.heads[w] > 0 && (!dys[w] || !outs[w] || ((reinterpret_cast<uintptr_t>(dys[w]) | reinterpret_cast<uintptr_t>(outs[w])) & em)))
                return R2L_ERR_INVALID_ARG;
            p.dy[w] = dys[w];
            p.out[w] = outs[w];
            p.dy_tok[w] = p.out_tok[w] = (long long)p.heads[w] * p.dim;
        }
        if (want_w && bad_workspace(workspace, workspace_bytes, rope_part_bytes(a))) return R2L_ERR_INVALID_ARG;
        p.part = want_w ? static_cast<float*>(workspace) : nullptr;
        n = rope_bwd_ctas(a->tokens, rope_lanes(p, esize(a->dtype), true));
        const cudaError_t e = a->dtype == R2L_BF16 ? rope_launch<true, __nv_bfloat16>(p, n, stream)
                                                   : rope_launch<true, float>(p, n, stream);
        if (!cuda_ok(e, "norm and rotation gradient launch")) return R2L_ERR_CUDA;
    }
    if (!want_w) return R2L_OK;
    // sums over nothing are zero: n is 0 then and the partials are not read
    return cuda_ok(launch_pdl(qk_norm_rope_dw_kernel, dim3((a->head_dim + 31) / 32, 2), dim3(kRopeDwThreads), 0, stream,
                              static_cast<const float*>(workspace), n, a->head_dim, dq_weight, dk_weight),
                   "weight gradient sum launch")
               ? R2L_OK
               : R2L_ERR_CUDA;
}

r2l_status r2l_mixer_device_status(cudaStream_t stream) {
    if (!cuda_ok(cudaStreamSynchronize(stream), "cudaStreamSynchronize")) return R2L_ERR_CUDA;
    unsigned int word = 0, zero = 0;
    if (!cuda_ok(cudaMemcpyFromSymbol(&word, g_status_word, sizeof(word)), "read device status word")) return R2L_ERR_CUDA;
    if (word != 0 && !cuda_ok(cudaMemcpyToSymbol(g_status_word, &zero, sizeof(zero)), "clear device status word"))
        return R2L_ERR_CUDA;
    return word ? R2L_ERR_TIMEOUT : R2L_OK;
}

const char* r2l_mixer_last_error(void) { return last_error_buffer(); }

int r2l_mixer_abi_version(void) { return kMixerAbiVersion; }

}  // extern "C"
