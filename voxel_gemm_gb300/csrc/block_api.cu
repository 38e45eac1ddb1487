// extern "C" entry points of the attention-block operators declared in
// include/vg.h: argument checks and workspace layout.  No memory is allocated here.
#include <cmath>

#include "attn.cuh"

namespace vg {

namespace {

bool misaligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) != 0; }
bool known_dtype(int dt) { return dt == VG_F32 || dt == VG_F16 || dt == VG_BF16; }

// A [rows][heads][d] operand: 16-byte vectors everywhere; `write`: no element twice.
int check_heads(const vg_heads* h, int64_t rows, int heads, int d, int dtype, bool write) {
    if (rows == 0 || heads == 0) return VG_OK;
    if (!h || !h->data || misaligned(h->data, 16)) return VG_ERR_INVALID_ARG;
    const int64_t vec = dtype == VG_F32 ? 4 : 8;
    const int64_t rs = h->row_stride, hs = h->head_stride;
    if (rows > 1 && (rs < d || rs % vec)) return VG_ERR_INVALID_ARG;
    if (heads > 1 && (hs < d || hs % vec)) return VG_ERR_INVALID_ARG;
    // element offsets stay within 2^47, far from any overflow
    if ((rows > 1 && rs > (int64_t(1) << 46) / rows) || (heads > 1 && hs > (int64_t(1) << 46) / heads))
        return VG_ERR_INVALID_ARG;
    if (write && rows > 1 && heads > 1 && rs < (heads - 1) * hs + d && hs < (rows - 1) * rs + d)
        return VG_ERR_INVALID_ARG;
    return VG_OK;
}

int check_rope(int64_t N, int hq, int hk, int d, int dtype, const vg_heads* q, const vg_heads* k, const void* qw,
               const void* kw, const int32_t* coords, const float* freqs, const int* pairs, double eps,
               unsigned flags, bool bwd) {
    if (N < 0 || N >= (int64_t(1) << 31) || hq < 0 || hk < 0 || hq > 4096 || hk > 4096 || hq + hk == 0 || d <= 0 ||
        !known_dtype(dtype))
        return VG_ERR_INVALID_ARG;
    if (flags & ~(VG_ROPE_HALVES | VG_QK_NO_NORM | VG_QK_SHARED_WEIGHT)) return VG_ERR_UNSUPPORTED;
    if (d % 8 || d > 256 || hq + hk > 4096) return VG_ERR_UNSUPPORTED;
    const bool norm = !(flags & VG_QK_NO_NORM);
    if (!norm && (qw || kw)) return VG_ERR_INVALID_ARG;
    if (N > 0 && !norm && !coords) return VG_ERR_INVALID_ARG;  // nothing to do
    if (norm && !(eps >= 0.0 && eps < INFINITY)) return VG_ERR_INVALID_ARG;
    if ((qw && misaligned(qw, 16)) || (kw && misaligned(kw, 16))) return VG_ERR_INVALID_ARG;
    if (N > 0 && !coords && freqs) return VG_ERR_INVALID_ARG;
    if (coords) {
        if (!pairs || misaligned(coords, 4) || misaligned(freqs, 4)) return VG_ERR_INVALID_ARG;
        int64_t sum = 0;
        for (int i = 0; i < 3; ++i) {
            if (pairs[i] < 0) return VG_ERR_INVALID_ARG;
            sum += pairs[i];
        }
        if (sum > d / 2 || (sum > 0 && !freqs)) return VG_ERR_INVALID_ARG;
    }
    if (bwd && !norm) return VG_OK;  // the rotation's gradient does not read its input
    int st = check_heads(q, N, hq, d, dtype, false);
    return st != VG_OK ? st : check_heads(k, N, hk, d, dtype, false);
}

QkRope rope_call(int64_t N, int hq, int hk, int d, int dtype, const vg_heads* q, const vg_heads* k, const void* qw,
                 const void* kw, const int32_t* coords, const float* freqs, const int* pairs, double eps,
                 unsigned flags) {
    QkRope c{};
    c.n = N;
    c.heads_q = hq;
    c.heads_k = hk;
    c.head_dim = d;
    c.dtype = dtype;
    c.q = q;
    c.k = k;
    c.q_weight = qw;
    c.k_weight = kw;
    c.coords = coords;
    c.freqs = freqs;
    for (int i = 0; i < 3; ++i) c.axis_pairs[i] = coords ? pairs[i] : 0;
    c.eps = eps;
    c.flags = flags;
    c.sms = plan_sms(0);
    return c;
}

int attn_shape(const vg_attn* a, bool backward, AttnPlan* p) {
    if (!a) return VG_ERR_INVALID_ARG;
    return attn_plan(AttnShape{a->n_q, a->n_k, a->batch, a->heads_q, a->heads_k, a->head_dim, a->dtype, backward}, p);
}

int check_attn(const vg_attn* a, const vg_heads* q, const vg_heads* k, const vg_heads* v, const vg_heads* out,
               bool backward, const void* ws, size_t ws_bytes, AttnPlan* p) {
    int st = attn_shape(a, backward, p);
    if (st != VG_OK) return st;
    if (!(a->scale > 0.f && a->scale < INFINITY)) return VG_ERR_INVALID_ARG;
    if (!a->q_offsets || !a->k_offsets || misaligned(a->q_offsets, 4) || misaligned(a->k_offsets, 4) ||
        misaligned(a->k_lens, 4))
        return VG_ERR_INVALID_ARG;
    if (!ws || misaligned(ws, 256)) return VG_ERR_INVALID_ARG;
    if (ws_bytes < p->total) return VG_ERR_WORKSPACE_TOO_SMALL;
    const int d = a->head_dim, dt = a->dtype;
    if ((st = check_heads(q, a->n_q, a->heads_q, d, dt, false)) != VG_OK) return st;
    if ((st = check_heads(k, a->n_k, a->heads_k, d, dt, false)) != VG_OK) return st;
    if ((st = check_heads(v, a->n_k, a->heads_k, d, dt, false)) != VG_OK) return st;
    return check_heads(out, a->n_q, a->heads_q, d, dt, !backward);
}

AttnArgs attn_args(const vg_attn* c, const vg_heads* q, const vg_heads* k, const vg_heads* v, const vg_heads* out) {
    AttnArgs a{};
    a.n_q = c->n_q;
    a.n_k = c->n_k;
    a.batch = c->batch;
    a.hq = c->heads_q;
    a.hk = c->heads_k;
    a.d = c->head_dim;
    a.q_off = c->q_offsets;
    a.k_off = c->k_offsets;
    a.k_len = c->k_lens;
    a.scale = c->scale;
    a.scale_log2 = (float)((double)c->scale * 1.4426950408889634);
    const vg_heads none{};
    a.q = q ? *q : none;
    a.k = k ? *k : none;
    a.v = v ? *v : none;
    a.o = out ? *out : none;
    return a;
}

}  // namespace

}  // namespace vg

using namespace vg;

extern "C" {

int vg_qk_norm_rope_fwd(int64_t N, int heads_q, int heads_k, int head_dim, int dtype, const vg_heads* q,
                        const vg_heads* k, const void* q_weight, const void* k_weight, const int32_t* coords,
                        const float* freqs, const int axis_pairs[3], double eps, unsigned flags,
                        const vg_heads* q_out, const vg_heads* k_out, void* stream) {
    int st = check_rope(N, heads_q, heads_k, head_dim, dtype, q, k, q_weight, k_weight, coords, freqs, axis_pairs, eps,
                        flags, false);
    if (st != VG_OK) return st;
    if ((st = check_heads(q_out, N, heads_q, head_dim, dtype, true)) != VG_OK) return st;
    if ((st = check_heads(k_out, N, heads_k, head_dim, dtype, true)) != VG_OK) return st;
    if (N == 0) return VG_OK;
    cudaGetLastError();
    QkRope c = rope_call(N, heads_q, heads_k, head_dim, dtype, q, k, q_weight, k_weight, coords, freqs, axis_pairs, eps,
                         flags);
    c.q_out = q_out;
    c.k_out = k_out;
    return qk_norm_rope(c, false, static_cast<cudaStream_t>(stream));
}

size_t vg_qk_norm_rope_workspace_bytes(int64_t N, int heads_q, int heads_k, int head_dim) {
    const int st = check_rope(N, heads_q, heads_k, head_dim, VG_F32, nullptr, nullptr, nullptr, nullptr,
                              reinterpret_cast<const int32_t*>(16), reinterpret_cast<const float*>(16),
                              (const int[3]){0, 0, 0}, 0.0, VG_QK_NO_NORM, true);
    return st == VG_OK ? rope_workspace_bytes(N, heads_q, heads_k, head_dim, plan_sms(0)) : 0;
}

int vg_qk_norm_rope_bwd(int64_t N, int heads_q, int heads_k, int head_dim, int dtype, const vg_heads* q,
                        const vg_heads* k, const void* q_weight, const void* k_weight, const int32_t* coords,
                        const float* freqs, const int axis_pairs[3], double eps, unsigned flags,
                        const vg_heads* grad_q_out, const vg_heads* grad_k_out, const vg_heads* grad_q,
                        const vg_heads* grad_k, void* grad_q_weight, void* grad_k_weight, void* ws, size_t ws_bytes,
                        void* stream) {
    int st = check_rope(N, heads_q, heads_k, head_dim, dtype, q, k, q_weight, k_weight, coords, freqs, axis_pairs, eps,
                        flags, true);
    if (st != VG_OK) return st;
    if ((st = check_heads(grad_q_out, N, heads_q, head_dim, dtype, false)) != VG_OK) return st;
    if ((st = check_heads(grad_k_out, N, heads_k, head_dim, dtype, false)) != VG_OK) return st;
    if ((st = check_heads(grad_q, N, heads_q, head_dim, dtype, true)) != VG_OK) return st;
    if ((st = check_heads(grad_k, N, heads_k, head_dim, dtype, true)) != VG_OK) return st;
    if (grad_q_weight || grad_k_weight) {
        if (flags & VG_QK_NO_NORM) return VG_ERR_INVALID_ARG;
        if ((grad_q_weight && heads_q == 0) || (grad_k_weight && heads_k == 0)) return VG_ERR_INVALID_ARG;
        if (misaligned(grad_q_weight, 16) || misaligned(grad_k_weight, 16)) return VG_ERR_INVALID_ARG;
        if (!ws || misaligned(ws, 256)) return VG_ERR_INVALID_ARG;
        if (ws_bytes < rope_workspace_bytes(N, heads_q, heads_k, head_dim, plan_sms(0)))
            return VG_ERR_WORKSPACE_TOO_SMALL;
    }
    if (N == 0 && !grad_q_weight && !grad_k_weight) return VG_OK;
    cudaGetLastError();
    QkRope c = rope_call(N, heads_q, heads_k, head_dim, dtype, q, k, q_weight, k_weight, coords, freqs, axis_pairs, eps,
                         flags);
    c.q_out = grad_q;
    c.k_out = grad_k;
    c.grad_q = grad_q_out;
    c.grad_k = grad_k_out;
    c.grad_q_weight = grad_q_weight;
    c.grad_k_weight = grad_k_weight;
    c.partial = static_cast<float*>(ws);
    return qk_norm_rope(c, true, static_cast<cudaStream_t>(stream));
}

size_t vg_cross_attn_workspace_bytes(const vg_attn* a, int backward) {
    AttnPlan p;
    return attn_shape(a, backward != 0, &p) == VG_OK ? p.total : 0;
}

int vg_cross_attn_fwd(const vg_attn* a, const vg_heads* q, const vg_heads* k, const vg_heads* v, const vg_heads* out,
                      float* lse, void* ws, size_t ws_bytes, void* stream) {
    AttnPlan p;
    const int st = check_attn(a, q, k, v, out, false, ws, ws_bytes, &p);
    if (st != VG_OK) return st;
    if (misaligned(lse, 4)) return VG_ERR_INVALID_ARG;
    cudaGetLastError();
    AttnArgs args = attn_args(a, q, k, v, out);
    args.lse = lse;
    return attn_fwd(args, p, a->dtype, static_cast<char*>(ws), static_cast<cudaStream_t>(stream));
}

int vg_cross_attn_bwd(const vg_attn* a, const vg_heads* q, const vg_heads* k, const vg_heads* v, const vg_heads* out,
                      const float* lse, const vg_heads* grad_out, const vg_heads* grad_q, const vg_heads* grad_k,
                      const vg_heads* grad_v, void* ws, size_t ws_bytes, void* stream) {
    AttnPlan p;
    int st = check_attn(a, q, k, v, out, true, ws, ws_bytes, &p);
    if (st != VG_OK) return st;
    const int d = a->head_dim, dt = a->dtype;
    if ((st = check_heads(grad_out, a->n_q, a->heads_q, d, dt, false)) != VG_OK) return st;
    if ((st = check_heads(grad_q, a->n_q, a->heads_q, d, dt, true)) != VG_OK) return st;
    if ((st = check_heads(grad_k, a->n_k, a->heads_k, d, dt, true)) != VG_OK) return st;
    if ((st = check_heads(grad_v, a->n_k, a->heads_k, d, dt, true)) != VG_OK) return st;
    if (a->n_q > 0 && (!lse || misaligned(lse, 4))) return VG_ERR_INVALID_ARG;
    cudaGetLastError();
    AttnArgs args = attn_args(a, q, k, v, out);
    args.lse = const_cast<float*>(lse);
    const vg_heads none{};
    args.go = grad_out ? *grad_out : none;
    args.gq = grad_q ? *grad_q : none;
    args.gk = grad_k ? *grad_k : none;
    args.gv = grad_v ? *grad_v : none;
    return attn_bwd(args, p, dt, static_cast<char*>(ws), static_cast<cudaStream_t>(stream));
}

int vg_cross_attn_status(void* ws, void* stream) {
    if (!ws) return VG_ERR_INVALID_ARG;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    uint32_t h = 0;
    if (cudaMemcpyAsync(&h, ws, sizeof(h), cudaMemcpyDeviceToHost, s) != cudaSuccess) return VG_ERR_CUDA;
    if (cudaStreamSynchronize(s) != cudaSuccess) return VG_ERR_CUDA;
    if (cudaMemsetAsync(ws, 0, sizeof(h), s) != cudaSuccess) return VG_ERR_CUDA;
    if (cudaStreamSynchronize(s) != cudaSuccess) return VG_ERR_CUDA;
    if (h & kErrRange) return VG_ERR_INVALID_ARG;
    return (h & kErrTimeout) ? VG_ERR_DEVICE_TIMEOUT : VG_OK;
}

int vg_adamw_step(const vg_adamw_tensor* tensors, int count, int state_bits, int64_t step, double lr, double beta1,
                  double beta2, double eps, double grad_scale, void* stream) {
    if (count < 0 || (count > 0 && !tensors) || step < 1) return VG_ERR_INVALID_ARG;
    if (state_bits != 8 && state_bits != 32) return VG_ERR_UNSUPPORTED;
    if (!(lr >= 0.0 && lr < INFINITY) || !(beta1 >= 0.0 && beta1 < 1.0) || !(beta2 >= 0.0 && beta2 < 1.0) ||
        !(eps >= 0.0 && eps < INFINITY) || !std::isfinite(grad_scale))
        return VG_ERR_INVALID_ARG;
    for (int i = 0; i < count; ++i) {
        const vg_adamw_tensor& t = tensors[i];
        if (t.n < 0 || !known_dtype(t.dtype) || !(t.weight_decay >= 0.0 && t.weight_decay < INFINITY))
            return VG_ERR_INVALID_ARG;
        if (t.n == 0) continue;
        const size_t es = t.dtype == VG_F32 ? 4 : 2;
        if (!t.param || !t.grad || !t.m || !t.v || misaligned(t.param, es) || misaligned(t.grad, es) ||
            misaligned(t.master, 4))
            return VG_ERR_INVALID_ARG;
        if (state_bits == 32 && (misaligned(t.m, 4) || misaligned(t.v, 4))) return VG_ERR_INVALID_ARG;
        if (state_bits == 8 &&
            (!t.m_scale || !t.v_scale || misaligned(t.m_scale, 4) || misaligned(t.v_scale, 4)))
            return VG_ERR_INVALID_ARG;
        if (t.n >= (int64_t(1) << 40)) return VG_ERR_UNSUPPORTED;
    }
    cudaGetLastError();
    return adamw_step(tensors, count, state_bits, step, lr, beta1, beta2, eps, grad_scale,
                      static_cast<cudaStream_t>(stream));
}

int vg_adamw_decode(const uint8_t* codes, const float* scales, int64_t n, int second, float* out, void* stream) {
    if (n < 0 || (second != 0 && second != 1)) return VG_ERR_INVALID_ARG;
    if (n > 0 && (!codes || !scales || !out || misaligned(scales, 4) || misaligned(out, 4))) return VG_ERR_INVALID_ARG;
    cudaGetLastError();
    return adamw_decode(codes, scales, n, second, out, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
