// gdn_decay_api.cu -- the extern "C" entry points of the decayed linear
// attention and of the block norms: argument checks, path selection and
// stream-ordered launches.
#include <cmath>

#include "gdn_block_norm.cuh"
#include "gdn_decay.cuh"

using namespace gdn;

namespace {

// The checks common to the prefill and the backward.
gdn_status_t check_decay_shape(const gdn_shape_t *s, const int32_t *cu_seqlens, bool layout_known) {
    const gdn_status_t st = check_shape(s);
    if (st != GDN_OK) return st;
    if (s->flags & ~GDN_FLAG_FORCE_SIMT)
        return fail(GDN_ERR_UNSUPPORTED, "the decayed linear attention takes no flags but GDN_FLAG_FORCE_SIMT (got 0x%x)",
                    s->flags);
    if (s->chunk_size != kDecayChunk)
        return fail(GDN_ERR_UNSUPPORTED, "the decayed linear attention uses chunks of %d tokens (got %d)", kDecayChunk,
                    s->chunk_size);
    if (s->num_v_heads > 65535) return fail(GDN_ERR_UNSUPPORTED, "more than 65535 value heads");
    if (int64_t(s->batch) * s->seq_len > kDecayMaxTokens)
        return fail(GDN_ERR_UNSUPPORTED, "more than %d tokens", kDecayMaxTokens);
    if (s->num_seqs > (1 << 24)) return fail(GDN_ERR_UNSUPPORTED, "more than 2^24 sequences");
    if (layout_known) {
        if (cu_seqlens) {
            if (s->batch != 1) return fail(GDN_ERR_INVALID_ARGUMENT, "batch must be 1 with cu_seqlens");
        } else if (s->num_seqs != s->batch) {
            return fail(GDN_ERR_INVALID_ARGUMENT, "num_seqs (%d) must equal batch (%d) without cu_seqlens",
                        s->num_seqs, s->batch);
        }
        if (s->num_seqs == 0 && int64_t(s->batch) * s->seq_len > 0)
            return fail(GDN_ERR_INVALID_ARGUMENT, "tokens without sequences");
    }
    return GDN_OK;
}

gdn_status_t check_aligned(const void *const *ptrs, const char *const *names, int n) {
    for (int i = 0; i < n; ++i)
        if (ptrs[i] && !aligned16(ptrs[i])) return fail(GDN_ERR_MISALIGNED, "%s is not 16-byte aligned", names[i]);
    return GDN_OK;
}

gdn_status_t check_workspace(const void *ws, size_t bytes, size_t need) {
    if (!ws) return fail(GDN_ERR_INVALID_ARGUMENT, "workspace is NULL");
    if (bytes < need) return fail(GDN_ERR_WORKSPACE_TOO_SMALL, "workspace has %zu bytes, needs %zu", bytes, need);
    if ((reinterpret_cast<uintptr_t>(ws) & 255u) != 0)
        return fail(GDN_ERR_MISALIGNED, "workspace is not 256-byte aligned");
    return GDN_OK;
}

gdn_status_t check_gate_layout(int32_t g_layout) {
    if (g_layout != GDN_DECAY_PER_TOKEN && g_layout != GDN_DECAY_PER_HEAD)
        return fail(GDN_ERR_INVALID_ARGUMENT, "decay layout %d is not GDN_DECAY_PER_TOKEN or GDN_DECAY_PER_HEAD",
                    g_layout);
    return GDN_OK;
}

cudaError_t run_pass(const DecayPass &p, const gdn_shape_t &s, int64_t max_units, cudaStream_t stream,
                     const DecayPass *also = nullptr) {
    int major = 0;
    device_sm_count(&major);
    // the tensor-core form where it applies (bf16, head sizes multiples of 8)
    if (major == 10 && decay_tc_supported(s)) {
        const cudaError_t e = launch_decay_pass_tc(p, max_units, stream);
        return e == cudaSuccess && also ? launch_decay_pass_tc(*also, max_units, stream) : e;
    }
    return launch_decay_pass_simt(p, also, s.dtype, max_units, stream);
}

DecayPass pass_of(const gdn_shape_t &s, const DecaySched &sc, const float *g, int32_t g_layout) {
    DecayPass p = {};
    p.hv = s.num_v_heads;
    p.tokens = s.batch * s.seq_len;
    p.g = g;
    p.g_const = g_layout == GDN_DECAY_PER_HEAD;
    p.sched = sc;
    return p;
}

}  // namespace

extern "C" {

gdn_status_t gdn_decay_forward_workspace_size(const gdn_shape_t *s, size_t *bytes) {
    clear_error();
    if (!bytes) return fail(GDN_ERR_INVALID_ARGUMENT, "bytes is NULL");
    const gdn_status_t st = check_decay_shape(s, nullptr, false);
    if (st != GDN_OK) return st;
    *bytes = decay_layout(*s, false).total;
    return GDN_OK;
}

gdn_status_t gdn_decay_forward(const gdn_shape_t *s, const void *q, const void *k, const void *v, const float *g,
                               int32_t g_layout, const float *initial_state, const int32_t *cu_seqlens,
                               const gdn_output_side_t *out_side, void *o, float *final_state, void *workspace,
                               size_t workspace_bytes, void *stream_) {
    clear_error();
    gdn_status_t st = check_decay_shape(s, cu_seqlens, true);
    if (st != GDN_OK) return st;
    st = check_gate_layout(g_layout);
    if (st != GDN_OK) return st;
    OutSide out;
    st = check_output_side(out_side, &out);
    if (st != GDN_OK) return st;
    const int64_t tokens = int64_t(s->batch) * s->seq_len;
    if (tokens > 0 && (!q || !k || !v || !g || !o))
        return fail(GDN_ERR_INVALID_ARGUMENT, "q, k, v, g and o must be non-NULL");
    const DecayLayout L = decay_layout(*s, false);
    st = check_workspace(workspace, workspace_bytes, L.total);
    if (st != GDN_OK) return st;
    const void *ptrs[] = {q, k, v, g, initial_state, cu_seqlens, o, final_state};
    const char *names[] = {"q", "k", "v", "g", "initial_state", "cu_seqlens", "o", "final_state"};
    st = check_aligned(ptrs, names, 8);
    if (st != GDN_OK) return st;
    if (device_sm_count(nullptr) <= 0) return fail(GDN_ERR_CUDA, "no usable CUDA device");
    cudaStream_t stream = static_cast<cudaStream_t>(stream_);
    char *ws = static_cast<char *>(workspace);
    const DecaySched sc = decay_sched(ws, L);
    cudaError_t e = launch_decay_schedule(*s, cu_seqlens, ws, L, stream);
    if (e != cudaSuccess) return cuda_fail(e, "schedule kernel launch");

    DecayPass p = pass_of(*s, sc, g, g_layout);
    p.x = q; p.y = k; p.z = v;
    p.hx = p.hy = s->num_qk_heads;
    p.hz = s->num_v_heads;
    p.dy = s->head_dim_k;
    p.dz = s->head_dim_v;
    p.s_in = initial_state;
    float *states = reinterpret_cast<float *>(ws + L.state_off[0]);
    float *dec = reinterpret_cast<float *>(ws + L.segdec_off[0]);
    if (L.max_slots > 0) {
        DecayPass w = p;
        w.state_only = 1;
        w.seg_local = states;
        w.seg_dec = dec;
        e = run_pass(w, *s, L.max_slots * s->num_v_heads, stream);
        if (e != cudaSuccess) return cuda_fail(e, "segment state launch");
        e = launch_decay_combine(*s, L, sc, states, dec, initial_state, false, p.dz, p.dy, false, stream);
        if (e != cudaSuccess) return cuda_fail(e, "segment state launch");
    }
    p.seg_state = states;
    p.s_out = final_state;
    p.out = o;
    e = run_pass(p, *s, L.max_segs * s->num_v_heads, stream);
    if (e != cudaSuccess) return cuda_fail(e, "prefill launch");
    if (out.flags && tokens > 0) {
        e = launch_output_side(o, int32_t(tokens), s->num_v_heads, s->head_dim_v, s->dtype, out, stream, &sc.hdr->status);
        if (e != cudaSuccess) return cuda_fail(e, "output-side launch");
    }
    return GDN_OK;
}

gdn_status_t gdn_decay_decode_step(int32_t n, int32_t hk, int32_t hv, int32_t dk, int32_t dv, int32_t dtype,
                                   const void *q, const void *k, const void *v, const float *g, int32_t g_layout,
                                   float *state, const gdn_output_side_t *out_side, void *o, void *stream_) {
    clear_error();
    OutSide out;
    gdn_status_t st = check_output_side(out_side, &out);
    if (st != GDN_OK) return st;
    st = check_gate_layout(g_layout);
    if (st != GDN_OK) return st;
    if (n < 0 || hk <= 0 || hv <= 0 || dk <= 0 || dv <= 0) return fail(GDN_ERR_INVALID_ARGUMENT, "bad decode shape");
    if (hv % hk != 0) return fail(GDN_ERR_INVALID_ARGUMENT, "num_v_heads must be a multiple of num_qk_heads");
    if (dtype != GDN_DTYPE_F32 && dtype != GDN_DTYPE_BF16)
        return fail(GDN_ERR_INVALID_ARGUMENT, "dtype %d is not GDN_DTYPE_F32 or GDN_DTYPE_BF16", dtype);
    if (dk > 256) return fail(GDN_ERR_UNSUPPORTED, "decode supports d_k <= 256 (got %d)", dk);
    if (dv > (1 << 20)) return fail(GDN_ERR_UNSUPPORTED, "decode supports d_v <= 2^20 (got %d)", dv);
    if (out.flags && dv > 128)
        return fail(GDN_ERR_UNSUPPORTED, "decode with an output side supports d_v <= 128 (got %d)", dv);
    if (n == 0) return GDN_OK;
    const void *ptrs[] = {q, k, v, g, state, o};
    const char *names[] = {"q", "k", "v", "g", "state", "o"};
    for (int i = 0; i < 6; ++i)
        if (!ptrs[i]) return fail(GDN_ERR_INVALID_ARGUMENT, "%s is NULL", names[i]);
    st = check_aligned(ptrs, names, 6);
    if (st != GDN_OK) return st;
    if (int64_t(n) * hv > INT32_MAX || double(n) * hv * dv * dk > double(int64_t(1) << 40))
        return fail(GDN_ERR_UNSUPPORTED, "state too large");
    cudaStream_t stream = static_cast<cudaStream_t>(stream_);
    cudaError_t e = launch_decay_decode(n, hk, hv, dk, dv, dtype, q, k, v, g, g_layout == GDN_DECAY_PER_HEAD, state, o,
                                        stream);
    if (e == cudaSuccess && out.flags) e = launch_output_side(o, n, hv, dv, dtype, out, stream);
    if (e != cudaSuccess) return cuda_fail(e, "decode launch");
    return GDN_OK;
}

gdn_status_t gdn_decay_backward_workspace_size(const gdn_shape_t *s, size_t *bytes) {
    clear_error();
    if (!bytes) return fail(GDN_ERR_INVALID_ARGUMENT, "bytes is NULL");
    const gdn_status_t st = check_decay_shape(s, nullptr, false);
    if (st != GDN_OK) return st;
    *bytes = decay_layout(*s, true).total;
    return GDN_OK;
}

gdn_status_t gdn_decay_backward(const gdn_shape_t *s, const void *q, const void *k, const void *v, const float *g,
                                int32_t g_layout, const float *initial_state, const int32_t *cu_seqlens,
                                const void *d_o, const float *d_final_state, void *dq, void *dk, void *dv, float *dg,
                                float *d_initial_state, void *workspace, size_t workspace_bytes, void *stream_) {
    clear_error();
    gdn_status_t st = check_decay_shape(s, cu_seqlens, true);
    if (st != GDN_OK) return st;
    st = check_gate_layout(g_layout);
    if (st != GDN_OK) return st;
    const int64_t tokens = int64_t(s->batch) * s->seq_len;
    if (tokens > 0 && (!q || !k || !v || !g || !d_o || !dq || !dk || !dv))
        return fail(GDN_ERR_INVALID_ARGUMENT, "inputs, d_o, dq, dk and dv must be non-NULL");
    const DecayLayout L = decay_layout(*s, true);
    st = check_workspace(workspace, workspace_bytes, L.total);
    if (st != GDN_OK) return st;
    const void *ptrs[] = {q, k, v, g, initial_state, cu_seqlens, d_o, d_final_state, dq, dk, dv, dg, d_initial_state};
    const char *names[] = {"q", "k", "v", "g", "initial_state", "cu_seqlens", "d_o", "d_final_state",
                           "dq", "dk", "dv", "dg", "d_initial_state"};
    st = check_aligned(ptrs, names, 13);
    if (st != GDN_OK) return st;
    if (device_sm_count(nullptr) <= 0) return fail(GDN_ERR_CUDA, "no usable CUDA device");
    cudaStream_t stream = static_cast<cudaStream_t>(stream_);
    char *ws = static_cast<char *>(workspace);
    const DecaySched sc = decay_sched(ws, L);
    const int hk = s->num_qk_heads, hv = s->num_v_heads, d_k = s->head_dim_k, d_v = s->head_dim_v;
    cudaError_t e = launch_decay_schedule(*s, cu_seqlens, ws, L, stream);
    if (e != cudaSuccess) return cuda_fail(e, "schedule kernel launch");
    auto at = [&](size_t off) { return reinterpret_cast<float *>(ws + off); };
    const bool grouped = hv != hk;
    const DecayPass base = pass_of(*s, sc, g, g_layout);

    // dq: out_t = S_t^T do_t, forward in time over the transposed state
    DecayPass pq = base;
    pq.x = d_o; pq.hx = hv;
    pq.y = v; pq.hy = hv;
    pq.z = k; pq.hz = hk;
    pq.dy = d_v;
    pq.dz = d_k;
    pq.s_in = initial_state;
    pq.s_trans = 1;
    // dk: out_t = dS_t^T v_t, backward in time
    DecayPass pk = base;
    pk.reverse = 1;
    pk.x = v; pk.hx = hv;
    pk.y = d_o; pk.hy = hv;
    pk.z = q; pk.hz = hk;
    pk.dy = d_v;
    pk.dz = d_k;
    pk.s_in = d_final_state;
    pk.s_trans = 1;
    if (L.max_slots > 0) {
        DecayPass w[2] = {pq, pk};
        for (int i = 0; i < 2; ++i) {
            w[i].state_only = 1;
            w[i].seg_local = at(L.state_off[i]);
            w[i].seg_dec = at(L.segdec_off[i]);
        }
        e = run_pass(w[0], *s, L.max_slots * hv, stream, &w[1]);
        for (int i = 0; i < 2 && e == cudaSuccess; ++i)
            e = launch_decay_combine(*s, L, sc, w[i].seg_local, w[i].seg_dec, w[i].s_in, true, d_k, d_v, i == 1, stream);
        if (e != cudaSuccess) return cuda_fail(e, "segment state launch");
    }
    const int64_t units = L.max_segs * hv;
    pq.seg_state = at(L.state_off[0]);
    pq.out = grouped ? static_cast<void *>(at(L.part_off[0])) : dq;
    pq.out_f32 = grouped;
    pk.seg_state = at(L.state_off[1]);
    pk.out = grouped ? static_cast<void *>(at(L.part_off[1])) : dk;
    pk.out_f32 = grouped;
    pk.s_out = d_initial_state;
    if (dg) {
        pq.aux = q; pq.haux = hk; pq.dot = at(L.dot_off[0]);
        pq.starts = at(L.start_off);
        pk.s_first = initial_state;
        pk.aux = k; pk.haux = hk; pk.dot = at(L.dot_off[1]);
        pk.starts = at(L.start_off);
        pk.span = at(L.span_off);
    }
    // dv: out_t = dS_t k_t, backward in time
    DecayPass pv = base;
    pv.reverse = 1;
    pv.x = k; pv.hx = hk;
    pv.y = q; pv.hy = hk;
    pv.z = d_o; pv.hz = hv;
    pv.dy = d_k;
    pv.dz = d_v;
    pv.s_in = d_final_state;
    pv.seg_state = at(L.state_off[1]);
    pv.seg_trans = 1;
    pv.out = dv;
    // (dk's pass reads the start states that dq's pass writes)
    if ((e = run_pass(pq, *s, units, stream, &pv)) != cudaSuccess || (e = run_pass(pk, *s, units, stream)) != cudaSuccess)
        return cuda_fail(e, "backward launch");
    if (tokens == 0) {  // (a rejected cu_seqlens leaves dg as it was: the kernel looks at the status)
        e = dg && base.g_const ? launch_decay_dg(*s, cu_seqlens, L, sc, nullptr, nullptr, nullptr, nullptr, g, true,
                                                 at(L.dgtok_off), dg, stream)
                               : cudaSuccess;
        return e == cudaSuccess ? GDN_OK : cuda_fail(e, "decay gradient launch");
    }
    if (dg) {
        e = decay_tc_supported(*s)
                ? launch_decay_intra(*s, cu_seqlens, L, sc, q, k, v, d_o, g, base.g_const, at(L.intra_off), stream)
                : launch_decay_intra_simt(*s, cu_seqlens, L, sc, q, k, v, d_o, g, base.g_const, at(L.intra_off), stream);
        if (e == cudaSuccess)
            e = launch_decay_dg(*s, cu_seqlens, L, sc, pq.dot, pk.dot, at(L.intra_off), pk.span, g, base.g_const,
                                at(L.dgtok_off), dg, stream);
        if (e != cudaSuccess) return cuda_fail(e, "decay gradient launch");
    }
    if (grouped) {
        e = launch_decay_group_sum(sc.hdr, at(L.part_off[0]), dq, tokens, hk, hv, d_k, s->dtype, stream);
        if (e == cudaSuccess)
            e = launch_decay_group_sum(sc.hdr, at(L.part_off[1]), dk, tokens, hk, hv, d_k, s->dtype, stream);
        if (e != cudaSuccess) return cuda_fail(e, "group sum launch");
    }
    return GDN_OK;
}

}  // extern "C"

// ---------------------------------------------------------------------------
// Block norms
// ---------------------------------------------------------------------------
namespace {

gdn_status_t check_block_norm(int64_t rows, int32_t width, int32_t dtype, int32_t residual_dtype, const void *x,
                              const void *residual, const void *gate, const gdn_block_norm_t *norm,
                              BlockNormArgs *a) {
    if (!norm) return fail(GDN_ERR_INVALID_ARGUMENT, "norm is NULL");
    if (rows < 0 || width <= 0) return fail(GDN_ERR_INVALID_ARGUMENT, "bad block-norm shape");
    if (dtype != GDN_DTYPE_F32 && dtype != GDN_DTYPE_BF16)
        return fail(GDN_ERR_INVALID_ARGUMENT, "dtype %d is not GDN_DTYPE_F32 or GDN_DTYPE_BF16", dtype);
    if (residual_dtype != GDN_DTYPE_F32 && residual_dtype != dtype)
        return fail(GDN_ERR_UNSUPPORTED, "the residual stream must be GDN_DTYPE_F32 or of x's type");
    if (width > kBlockNormMaxWidth)
        return fail(GDN_ERR_UNSUPPORTED, "width %d above %d", width, kBlockNormMaxWidth);
    const uint32_t gates = GDN_BLOCK_GATE_SILU | GDN_BLOCK_GATE_SIGMOID;
    if (norm->flags & ~(gates | GDN_BLOCK_POST_NORM | GDN_BLOCK_PRE_NORM | GDN_BLOCK_ZERO_CENTRED))
        return fail(GDN_ERR_INVALID_ARGUMENT, "unknown block-norm flag bits 0x%x", norm->flags);
    const uint32_t got = norm->flags & gates;
    // (an empty tensor's pointer may be NULL)
    if (rows > 0 && (gate ? (got != GDN_BLOCK_GATE_SILU && got != GDN_BLOCK_GATE_SIGMOID) : got != 0))
        return fail(GDN_ERR_INVALID_ARGUMENT, "a gate needs exactly one of GDN_BLOCK_GATE_SILU, GDN_BLOCK_GATE_SIGMOID, "
                                              "and neither may be set without one");
    if (norm->post_weight && !(norm->flags & GDN_BLOCK_POST_NORM))
        return fail(GDN_ERR_INVALID_ARGUMENT, "post_weight without GDN_BLOCK_POST_NORM");
    if (norm->pre_weight && !(norm->flags & GDN_BLOCK_PRE_NORM))
        return fail(GDN_ERR_INVALID_ARGUMENT, "pre_weight without GDN_BLOCK_PRE_NORM");
    if (!(norm->eps > 0.f) || !(norm->eps < 3.0e38f))
        return fail(GDN_ERR_INVALID_ARGUMENT, "eps must be finite and > 0");
    if (!std::isfinite(norm->residual_scale) || !std::isfinite(norm->branch_scale))
        return fail(GDN_ERR_INVALID_ARGUMENT, "residual_scale and branch_scale must be finite");
    if (rows > 0 && !x) return fail(GDN_ERR_INVALID_ARGUMENT, "x is NULL");
    if (double(rows) * width > double(int64_t(1) << 40) || rows > INT32_MAX)
        return fail(GDN_ERR_UNSUPPORTED, "problem too large");
    const void *ptrs[] = {x, residual, gate, norm->post_weight, norm->scale, norm->pre_weight};
    const char *names[] = {"x", "residual", "gate", "post_weight", "scale", "pre_weight"};
    const gdn_status_t st = check_aligned(ptrs, names, 6);
    if (st != GDN_OK) return st;
    *a = BlockNormArgs{};
    a->rows = rows;
    a->width = width;
    a->flags = norm->flags;
    a->x = x;
    a->residual = residual;
    a->gate = gate;
    a->post_weight = norm->post_weight;
    a->scale = norm->scale;
    a->pre_weight = norm->pre_weight;
    a->eps = norm->eps;
    a->residual_scale = norm->residual_scale;
    a->branch_scale = norm->branch_scale;
    return GDN_OK;
}

}  // namespace

extern "C" {

gdn_status_t gdn_block_norm_forward(int64_t rows, int32_t width, int32_t dtype, int32_t residual_dtype, const void *x,
                                    const void *residual, const void *gate, const gdn_block_norm_t *norm, void *h,
                                    void *y, void *stream_) {
    clear_error();
    BlockNormArgs a;
    gdn_status_t st = check_block_norm(rows, width, dtype, residual_dtype, x, residual, gate, norm, &a);
    if (st != GDN_OK) return st;
    const bool pre = norm->flags & GDN_BLOCK_PRE_NORM;
    if (pre != (y != nullptr) && rows > 0)
        return fail(GDN_ERR_INVALID_ARGUMENT, "y goes with GDN_BLOCK_PRE_NORM and only with it");
    if (h && h == y) return fail(GDN_ERR_INVALID_ARGUMENT, "h and y are the same buffer");
    if (!h && !y && rows > 0) return fail(GDN_ERR_INVALID_ARGUMENT, "neither h nor y is wanted");
    const void *ptrs[] = {h, y};
    const char *names[] = {"h", "y"};
    st = check_aligned(ptrs, names, 2);
    if (st != GDN_OK) return st;
    if (rows == 0) return GDN_OK;
    if (device_sm_count(nullptr) <= 0) return fail(GDN_ERR_CUDA, "no usable CUDA device");
    a.h = h;
    a.y = y;
    const cudaError_t e = launch_block_norm_forward(a, dtype, residual_dtype, static_cast<cudaStream_t>(stream_));
    return e == cudaSuccess ? GDN_OK : cuda_fail(e, "block norm launch");
}

gdn_status_t gdn_block_norm_backward_workspace_size(int64_t rows, int32_t width, size_t *bytes) {
    clear_error();
    if (!bytes) return fail(GDN_ERR_INVALID_ARGUMENT, "bytes is NULL");
    if (rows < 0 || width <= 0) return fail(GDN_ERR_INVALID_ARGUMENT, "bad block-norm shape");
    if (width > kBlockNormMaxWidth)
        return fail(GDN_ERR_UNSUPPORTED, "width %d above %d", width, kBlockNormMaxWidth);
    *bytes = align256(size_t(block_norm_lines(rows, width)) * 3 * size_t(width) * sizeof(float));
    return GDN_OK;
}

gdn_status_t gdn_block_norm_backward(int64_t rows, int32_t width, int32_t dtype, int32_t residual_dtype, const void *x,
                                     const void *residual, const void *gate, const gdn_block_norm_t *norm,
                                     const void *d_h, const void *d_y, void *dx, void *d_residual, void *d_gate,
                                     float *d_post_weight, float *d_scale, float *d_pre_weight, void *workspace,
                                     size_t workspace_bytes, void *stream_) {
    clear_error();
    BlockNormArgs a;
    gdn_status_t st = check_block_norm(rows, width, dtype, residual_dtype, x, residual, gate, norm, &a);
    if (st != GDN_OK) return st;
    if (d_y && !(norm->flags & GDN_BLOCK_PRE_NORM))
        return fail(GDN_ERR_INVALID_ARGUMENT, "d_y without GDN_BLOCK_PRE_NORM");
    if (rows > 0 && !d_y && !d_h) return fail(GDN_ERR_INVALID_ARGUMENT, "neither d_h nor d_y is given");
    if (d_residual && !residual && rows > 0) return fail(GDN_ERR_INVALID_ARGUMENT, "d_residual without a residual");
    if (d_gate && !gate && rows > 0) return fail(GDN_ERR_INVALID_ARGUMENT, "d_gate without a gate");
    if (d_post_weight && !(norm->flags & GDN_BLOCK_POST_NORM))
        return fail(GDN_ERR_INVALID_ARGUMENT, "d_post_weight without GDN_BLOCK_POST_NORM");
    if (d_pre_weight && !(norm->flags & GDN_BLOCK_PRE_NORM))
        return fail(GDN_ERR_INVALID_ARGUMENT, "d_pre_weight without GDN_BLOCK_PRE_NORM");
    size_t need = 0;
    gdn_block_norm_backward_workspace_size(rows, width, &need);
    st = check_workspace(workspace, workspace_bytes, need);
    if (st != GDN_OK) return st;
    const void *ptrs[] = {d_h, d_y, dx, d_residual, d_gate, d_post_weight, d_scale, d_pre_weight};
    const char *names[] = {"d_h", "d_y", "dx", "d_residual", "d_gate", "d_post_weight", "d_scale", "d_pre_weight"};
    st = check_aligned(ptrs, names, 8);
    if (st != GDN_OK) return st;
    if (device_sm_count(nullptr) <= 0) return fail(GDN_ERR_CUDA, "no usable CUDA device");
    cudaStream_t stream = static_cast<cudaStream_t>(stream_);
    a.d_h = d_h;
    a.d_y = d_y;
    a.dx = dx;
    a.d_residual = d_residual;
    a.d_gate = d_gate;
    a.d_post_weight = d_post_weight;
    a.d_scale = d_scale;
    a.d_pre_weight = d_pre_weight;
    a.partial = static_cast<float *>(workspace);
    // without rows the kernel still writes its (zero) column sums
    const cudaError_t e = launch_block_norm_backward(a, dtype, residual_dtype, stream);
    return e == cudaSuccess ? GDN_OK : cuda_fail(e, "block norm backward launch");
}

}  // extern "C"
