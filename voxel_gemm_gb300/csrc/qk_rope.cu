// Per-head RMS norm of queries and keys and their rotation by several position
// axes, in one pass over the rows; forward and backward.
//
//   r = 1 / sqrt(mean_d x_d^2 + eps);  n_d = x_d r w_d
//   pair p of axis a, angle t = fp32(pos_a) * freq_p (one fp32 rounding):
//   (y0, y1) = (n0 cos t - n1 sin t, n0 sin t + n1 cos t)
// backward: g = the pair gradients turned by -t, then
//   dw_d = sum over tokens of g_d x_d r,   dx_d = r w_d g_d - x_d r^3 mean_e(x_e w_e g_e)
//
// Bound by memory (each element is read and written once).  A group of 1..32
// lanes holds one head's vector, 8 elements a lane (4 pairs, whichever of the
// two pair layouts), so the row statistics are shuffles inside the group and the
// rotation needs no exchange.  A 256-thread block takes all heads of a few
// tokens: the tokens' cosines and sines are computed once per block into shared
// memory and used by every head, each lane keeps its head's weights (and, in the
// backward pass, its weight-gradient sums) in registers over all tokens that the
// block visits, and each lane has the loads of several tokens in flight.  The
// weight gradients leave as one fp32 row per block, added in a fixed order by a
// second kernel, so they do not change from run to run.
#include "common.cuh"
#include "internal.h"

namespace vg {

namespace {

constexpr int kThreads = 256;
constexpr int kUnroll = 4;     // tokens of a lane in flight
constexpr int kReduceRows = 8;  // row lanes of the weight-gradient reduce

struct View {
    const void* p;
    int64_t row, head;  // strides in elements
};

struct RopeArgs {
    int64_t n;
    int hq, ht, d;              // query heads, all heads, head width
    int lanes;                  // lanes of a vector: power of two >= d / 8
    int chunk;                  // heads of a block (grid.y chunks cover ht)
    int per;                    // tokens a block holds side by side
    View q, k;                  // x
    View qo, ko;                // y (forward), dx (backward)
    View gq, gk;                // dy
    const void* wq;             // weights or null
    const void* wk;
    int64_t w_head;             // stride between two heads' weights (0: shared)
    const int32_t* coords;      // [n][4] or null
    const float* freqs;
    int pairs[3];
    float eps;
    float inv_d;
    int norm;
    float* partial;             // [grid.x][ht][d] weight-gradient rows
};

template <typename T>
__device__ __forceinline__ void load_vec(const T* p, int lane, int d, bool halves, float (&x)[8]) {
    const T* a = halves ? p + 4 * lane : p + 8 * lane;
    const T* b = halves ? p + d / 2 + 4 * lane : a + 4;
    if constexpr (sizeof(T) == 4) {
        const float4 u = *reinterpret_cast<const float4*>(a), v = *reinterpret_cast<const float4*>(b);
        x[0] = u.x; x[1] = u.y; x[2] = u.z; x[3] = u.w;
        x[4] = v.x; x[5] = v.y; x[6] = v.z; x[7] = v.w;
    } else {
        uint2 u, v;
        if (halves) {
            u = *reinterpret_cast<const uint2*>(a);
            v = *reinterpret_cast<const uint2*>(b);
        } else {
            const uint4 w = *reinterpret_cast<const uint4*>(a);
            u = make_uint2(w.x, w.y);
            v = make_uint2(w.z, w.w);
        }
        const T* e = reinterpret_cast<const T*>(&u);
        const T* f = reinterpret_cast<const T*>(&v);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            x[j] = to_f32<T>(e[j]);
            x[4 + j] = to_f32<T>(f[j]);
        }
    }
}
template <typename T>
__device__ __forceinline__ void store_vec(T* p, int lane, int d, bool halves, const float (&x)[8]) {
    T* a = halves ? p + 4 * lane : p + 8 * lane;
    T* b = halves ? p + d / 2 + 4 * lane : a + 4;
    if constexpr (sizeof(T) == 4) {
        *reinterpret_cast<float4*>(a) = make_float4(x[0], x[1], x[2], x[3]);
        *reinterpret_cast<float4*>(b) = make_float4(x[4], x[5], x[6], x[7]);
    } else {
        uint2 u, v;
        T* e = reinterpret_cast<T*>(&u);
        T* f = reinterpret_cast<T*>(&v);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            e[j] = from_f32<T>(x[j]);
            f[j] = from_f32<T>(x[4 + j]);
        }
        if (halves) {
            *reinterpret_cast<uint2*>(a) = u;
            *reinterpret_cast<uint2*>(b) = v;
        } else {
            *reinterpret_cast<uint4*>(a) = make_uint4(u.x, u.y, v.x, v.y);
        }
    }
}

// Indexes of pair j's members among a lane's 8 elements.
template <bool HALVES> __device__ __forceinline__ constexpr int first_of(int j) { return HALVES ? j : 2 * j; }
template <bool HALVES> __device__ __forceinline__ constexpr int second_of(int j) { return HALVES ? 4 + j : 2 * j + 1; }

__device__ __forceinline__ float group_sum(float x, int lanes) {
    for (int o = 1; o < lanes; o <<= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

template <typename T, bool HALVES, bool BWD>
__global__ void __launch_bounds__(kThreads) k_qk_norm_rope(const RopeArgs a) {
    extern __shared__ float2 s_turn[];  // [tile tokens][d / 2] cosine and sine
    const int lane = threadIdx.x & (a.lanes - 1);
    const int group = threadIdx.x / a.lanes;
    const int h0 = blockIdx.y * a.chunk;
    const int heads = min(a.chunk, a.ht - h0);
    const int sub = group / a.chunk;                       // which of the block's tokens
    const int hl = group - sub * a.chunk;
    const int h = h0 + hl;                                 // this group's head
    const bool mine = sub < a.per && hl < heads && lane * 8 < a.d;
    const bool is_q = h < a.hq;
    const int hh = is_q ? h : h - a.hq;
    const int half_d = a.d / 2;
    const int tile = a.per * kUnroll;                      // tokens of a tile
    const bool turn = a.coords != nullptr;

    float w[8], gw[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) w[j] = 1.f, gw[j] = 0.f;
    const void* wp = is_q ? a.wq : a.wk;
    if (mine && wp) load_vec<T>(static_cast<const T*>(wp) + hh * a.w_head, lane, a.d, HALVES, w);
    const View xv = is_q ? a.q : a.k, yv = is_q ? a.qo : a.ko, gv = is_q ? a.gq : a.gk;
    const T* xp = static_cast<const T*>(xv.p) + hh * xv.head;
    T* yp = static_cast<T*>(const_cast<void*>(yv.p)) + hh * yv.head;
    const T* gp = BWD ? static_cast<const T*>(gv.p) + hh * gv.head : nullptr;

    for (int64_t t0 = (int64_t)blockIdx.x * tile; t0 < a.n; t0 += (int64_t)gridDim.x * tile) {
        float x[kUnroll][8], g[kUnroll][8];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int64_t t = t0 + u * a.per + sub;
            if (mine && t < a.n) {
                if (!BWD || a.norm) load_vec<T>(xp + t * xv.row, lane, a.d, HALVES, x[u]);
                if constexpr (BWD) load_vec<T>(gp + t * gv.row, lane, a.d, HALVES, g[u]);
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) x[u][j] = g[u][j] = 0.f;
            }
        }
        if (turn) {
            __syncthreads();  // the previous tile's angles have been used
            for (int e = threadIdx.x; e < tile * half_d; e += kThreads) {
                const int tt = e / half_d, p = e - tt * half_d;
                float c = 1.f, s = 0.f;
                if (p < a.pairs[0] + a.pairs[1] + a.pairs[2] && t0 + tt < a.n) {
                    const int axis = p < a.pairs[0] ? 0 : (p < a.pairs[0] + a.pairs[1] ? 1 : 2);
                    sincosf(__fmul_rn((float)a.coords[(t0 + tt) * 4 + 1 + axis], a.freqs[p]), &s, &c);
                }
                s_turn[e] = make_float2(c, s);
            }
            __syncthreads();
        }
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int64_t t = t0 + u * a.per + sub;
            float2 cs[4];
#pragma unroll
            for (int j = 0; j < 4; ++j)
                cs[j] = turn && mine ? s_turn[(u * a.per + sub) * half_d + 4 * lane + j] : make_float2(1.f, 0.f);
            float r = 1.f;
            if constexpr (!BWD) {
                if (a.norm) {
                    float ss = 0.f;
#pragma unroll
                    for (int j = 0; j < 8; ++j) ss += x[u][j] * x[u][j];
                    r = rsqrtf(group_sum(ss, a.lanes) * a.inv_d + a.eps);
                }
                float y[8];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    constexpr bool H = HALVES;
                    const float n0 = x[u][first_of<H>(j)] * r * w[first_of<H>(j)];
                    const float n1 = x[u][second_of<H>(j)] * r * w[second_of<H>(j)];
                    y[first_of<H>(j)] = n0 * cs[j].x - n1 * cs[j].y;
                    y[second_of<H>(j)] = n0 * cs[j].y + n1 * cs[j].x;
                }
                if (mine && t < a.n) store_vec<T>(yp + t * yv.row, lane, a.d, HALVES, y);
            } else {
                float gn[8];  // the gradient of the normed, unturned vector
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    constexpr bool H = HALVES;
                    const float g0 = g[u][first_of<H>(j)], g1 = g[u][second_of<H>(j)];
                    gn[first_of<H>(j)] = g0 * cs[j].x + g1 * cs[j].y;
                    gn[second_of<H>(j)] = g1 * cs[j].x - g0 * cs[j].y;
                }
                float dx[8];
                if (a.norm) {
                    float ss = 0.f, dot = 0.f;
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        ss += x[u][j] * x[u][j];
                        dot += x[u][j] * w[j] * gn[j];
                    }
                    r = rsqrtf(group_sum(ss, a.lanes) * a.inv_d + a.eps);
                    const float back = group_sum(dot, a.lanes) * a.inv_d * r * r;
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        gw[j] += gn[j] * (x[u][j] * r);
                        dx[j] = r * (w[j] * gn[j] - x[u][j] * back);
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < 8; ++j) dx[j] = gn[j];
                }
                if (mine && t < a.n) store_vec<T>(yp + t * yv.row, lane, a.d, HALVES, dx);
            }
        }
    }
    if constexpr (BWD) {
        if (a.partial) {
            // one row per block: the tokens held side by side are added in order
            __syncthreads();
            float* s_gw = reinterpret_cast<float*>(s_turn);  // [per][chunk][d]
            if (mine) {
                float* dst = s_gw + ((size_t)sub * a.chunk + hl) * a.d;
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    dst[HALVES ? (j < 4 ? 4 * lane + j : half_d + 4 * lane + j - 4) : 8 * lane + j] = gw[j];
            }
            __syncthreads();
            for (int e = threadIdx.x; e < heads * a.d; e += kThreads) {
                float sum = 0.f;
                for (int s = 0; s < a.per; ++s) sum += s_gw[(size_t)s * a.chunk * a.d + e];
                a.partial[((size_t)blockIdx.x * a.ht + h0) * a.d + e] = sum;
            }
        }
    }
}

// dw[head][d] = sum over the rows (and, for shared weights, over the heads too) of
// the blocks' partial rows, in a fixed order: kReduceRows running sums, then those.
template <typename T>
__global__ void __launch_bounds__(32 * kReduceRows) k_rope_weight_reduce(const float* __restrict__ partial, int rows,
                                                                         int ht, int hq, int d, bool shared, T* gwq,
                                                                         T* gwk) {
    __shared__ float s[kReduceRows][33];
    const int cols_q = shared ? d : hq * d;
    const int cols = cols_q + (shared ? d : (ht - hq) * d);
    const int c = blockIdx.x * 32 + (threadIdx.x & 31);
    const int rl = threadIdx.x >> 5;
    float sum = 0.f;
    if (c < cols) {
        const bool is_q = c < cols_q;
        const int cc = is_q ? c : c - cols_q;
        const int head0 = is_q ? 0 : hq, nh = shared ? (is_q ? hq : ht - hq) : 1;
        const float* src = partial + (size_t)head0 * d + cc;
        const int64_t total = (int64_t)rows * nh;
        for (int64_t i = rl; i < total; i += kReduceRows) {
            const int64_t row = i / nh, hh = i - row * nh;
            sum += src[(row * ht + hh) * d];
        }
    }
    s[rl][threadIdx.x & 31] = sum;
    __syncthreads();
    if (rl == 0 && c < cols) {
        float tot = 0.f;
#pragma unroll
        for (int i = 0; i < kReduceRows; ++i) tot += s[i][threadIdx.x & 31];
        if (c < cols_q) {
            if (gwq) gwq[c] = from_f32<T>(tot);
        } else if (gwk) {
            gwk[c - cols_q] = from_f32<T>(tot);
        }
    }
}

// Lanes of a vector, heads of a block and tokens side by side: as many heads as
// the block's lane groups hold, in equal chunks, then as many tokens as fit.
void shape(int ht, int d, int* lanes, int* chunk, int* per) {
    int l = 1;
    while (l * 8 < d) l <<= 1;
    const int groups = kThreads / l;
    const int chunks = (ht + groups - 1) / groups;
    *lanes = l;
    *chunk = (ht + chunks - 1) / chunks;
    *per = groups / *chunk;
}

int grid_x(int64_t n, int per, int chunks, int sms) {
    const int64_t tiles = (n + (int64_t)per * kUnroll - 1) / ((int64_t)per * kUnroll);
    const int64_t cap = std::max<int64_t>(1, (int64_t)sms * 4 / chunks);
    return (int)std::max<int64_t>(1, std::min(tiles, cap));
}

template <typename T>
int launch(const RopeArgs& a, bool halves, bool bwd, int gx, int chunks, size_t smem, cudaStream_t s) {
    const dim3 grid(gx, chunks);
    if (bwd) {
        if (halves) k_qk_norm_rope<T, true, true><<<grid, kThreads, smem, s>>>(a);
        else k_qk_norm_rope<T, false, true><<<grid, kThreads, smem, s>>>(a);
    } else {
        if (halves) k_qk_norm_rope<T, true, false><<<grid, kThreads, smem, s>>>(a);
        else k_qk_norm_rope<T, false, false><<<grid, kThreads, smem, s>>>(a);
    }
    return cudaPeekAtLastError() == cudaSuccess ? VG_OK : VG_ERR_CUDA;
}

}  // namespace

size_t rope_workspace_bytes(int64_t n, int hq, int hk, int d, int sms) {
    int lanes, chunk, per;
    const int ht = hq + hk;
    shape(ht, d, &lanes, &chunk, &per);
    const int chunks = (ht + chunk - 1) / chunk;
    return align_up((size_t)grid_x(n, per, chunks, sms) * ht * d * 4, 256);
}

int qk_norm_rope(const QkRope& c, bool bwd, cudaStream_t s) {
    RopeArgs a{};
    a.n = c.n;
    a.hq = c.heads_q;
    a.ht = c.heads_q + c.heads_k;
    a.d = c.head_dim;
    shape(a.ht, a.d, &a.lanes, &a.chunk, &a.per);
    const int chunks = (a.ht + a.chunk - 1) / a.chunk;
    const auto view = [](const vg_heads* h) { return h ? View{h->data, h->row_stride, h->head_stride} : View{}; };
    a.q = view(c.q);
    a.k = view(c.k);
    a.qo = view(c.q_out);
    a.ko = view(c.k_out);
    a.gq = view(c.grad_q);
    a.gk = view(c.grad_k);
    a.norm = !(c.flags & VG_QK_NO_NORM);
    a.wq = c.q_weight;
    a.wk = c.k_weight;
    a.w_head = c.flags & VG_QK_SHARED_WEIGHT ? 0 : a.d;
    a.coords = c.coords;
    a.freqs = c.freqs;
    for (int i = 0; i < 3; ++i) a.pairs[i] = c.coords ? c.axis_pairs[i] : 0;
    a.eps = (float)c.eps;
    a.inv_d = 1.f / (float)a.d;
    const bool gw = bwd && a.norm && (c.grad_q_weight || c.grad_k_weight);
    a.partial = gw ? c.partial : nullptr;
    const int gx = grid_x(c.n, a.per, chunks, c.sms);
    const size_t smem = std::max((size_t)a.per * kUnroll * (a.d / 2) * sizeof(float2),
                                 bwd ? (size_t)a.per * a.chunk * a.d * sizeof(float) : 0);
    const bool halves = (c.flags & VG_ROPE_HALVES) != 0;
    int st = c.dtype == VG_F32   ? launch<float>(a, halves, bwd, gx, chunks, smem, s)
             : c.dtype == VG_F16 ? launch<__half>(a, halves, bwd, gx, chunks, smem, s)
                                 : launch<__nv_bfloat16>(a, halves, bwd, gx, chunks, smem, s);
    if (st != VG_OK || !gw) return st;
    const bool shared = (c.flags & VG_QK_SHARED_WEIGHT) != 0;
    const int cols = shared ? 2 * a.d : a.ht * a.d;
    const dim3 grid((cols + 31) / 32);
    if (c.dtype == VG_F32)
        k_rope_weight_reduce<float><<<grid, 32 * kReduceRows, 0, s>>>(c.partial, gx, a.ht, a.hq, a.d, shared,
                                                                      (float*)c.grad_q_weight, (float*)c.grad_k_weight);
    else if (c.dtype == VG_F16)
        k_rope_weight_reduce<__half><<<grid, 32 * kReduceRows, 0, s>>>(
            c.partial, gx, a.ht, a.hq, a.d, shared, (__half*)c.grad_q_weight, (__half*)c.grad_k_weight);
    else
        k_rope_weight_reduce<__nv_bfloat16><<<grid, 32 * kReduceRows, 0, s>>>(
            c.partial, gx, a.ht, a.hq, a.d, shared, (__nv_bfloat16*)c.grad_q_weight, (__nv_bfloat16*)c.grad_k_weight);
    return cudaPeekAtLastError() == cudaSuccess ? VG_OK : VG_ERR_CUDA;
}

}  // namespace vg
