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
// rotation needs no exchange.  A 256-thread block takes all heads of one or a few
// tokens at a time and runs along a range of tokens; each lane keeps its head's
// weights (and, in the backward pass, its weight-gradient sums) in registers all along.
// Every lane copies the vectors of its next tokens into its own places of a ring in shared
// memory (asynchronously, without a barrier: no lane reads another's), so that the
// loads in flight cost no registers.  The cosines and sines of the tokens that
// follow are computed into shared memory once for all heads, while the
// present ones are used.  The weight gradients leave as one fp32 row per block, added
// in a fixed order by a second kernel, so they do not change from run to run.
// 319,057 tokens of 16 + 16 heads of 64 in bf16: forward 423 us (6.2 TB/s), backward
// 673 us (5.8 TB/s).  With the vectors of four tokens in registers and angles computed
// between two barriers it was 771 and 2614 us (165 registers, one block per SM).
#include "common.cuh"
#include "internal.h"
#include "tc_ptx.cuh"

namespace vg {

namespace {

using namespace ptx;

constexpr int kThreads = 256;
constexpr int per_sm(bool bwd) { return bwd ? 3 : 4; }  // blocks per SM (80, 64 registers a thread)
constexpr int kStages = 4;       // ring places of a lane
constexpr int kReduceRows = 32;  // row lanes of the weight-gradient reduce

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
    int64_t range;              // tokens of a block
    int turns;                  // steps that share a table of angles
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
    float* partial;             // [blocks][heads_w][d] weight-gradient rows
    int shared;                 // heads_w: 2 (queries', keys'), else ht
};

// Copy a lane's 8 elements to its ring place, 16-byte pieces kThreads apart.
template <typename T, bool HALVES>
__device__ __forceinline__ void fetch(uint32_t to, const T* p, int lane, int d) {
    const T* a = HALVES ? p + 4 * lane : p + 8 * lane;
    const T* b = HALVES ? p + d / 2 + 4 * lane : a + 4;
    if constexpr (sizeof(T) == 4) {
        cp_async16(to, a, 16);
        cp_async16(to + 16 * kThreads, b, 16);
    } else if constexpr (HALVES) {
        cp_async8(to, a);
        cp_async8(to + 8, b);
    } else {
        cp_async16(to, a, 16);
    }
}
// The 8 elements at a ring place, zeros if there are none.
template <typename T>
__device__ __forceinline__ void read(const uint4* from, bool have, float (&x)[8]) {
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i) {
        const uint4 v = have ? from[i * kThreads] : make_uint4(0, 0, 0, 0);
        const T* e = reinterpret_cast<const T*>(&v);
#pragma unroll
        for (int j = 0; j < 16 / (int)sizeof(T); ++j) x[i * 4 + j] = to_f32<T>(e[j]);
    }
}
template <typename T, bool HALVES>
__device__ __forceinline__ void load_vec(const T* p, int lane, int d, float (&x)[8]) {
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] = to_f32<T>(p[HALVES ? 4 * lane + (j < 4 ? j : d / 2 + j - 4) : 8 * lane + j]);
}
template <typename T, bool HALVES>
__device__ __forceinline__ void store_vec(T* p, int lane, int d, const float (&x)[8]) {
    T* a = HALVES ? p + 4 * lane : p + 8 * lane;
    T* b = HALVES ? p + d / 2 + 4 * lane : a + 4;
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
        if constexpr (HALVES) {
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
__global__ void __launch_bounds__(kThreads, per_sm(BWD)) k_qk_norm_rope(const RopeArgs a) {
    extern __shared__ uint4 s_ring[];  // [kStages][x, dy][sizeof(T) / 2][kThreads], then two tables of angles
    constexpr int kPieces = (int)sizeof(T) / 2, kPlace = kPieces * (BWD ? 2 : 1) * kThreads;
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
    const int tile = a.per * a.turns;                      // tokens that share a table of angles
    const bool turn = a.coords != nullptr;

    float w[8], gw[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) w[j] = 1.f, gw[j] = 0.f;
    const T* wp = static_cast<const T*>(is_q ? a.wq : a.wk);
    if (mine && wp) load_vec<T, HALVES>(wp + hh * a.w_head, lane, a.d, w);

    // the block's tokens [t0, t1); this group's are t0 + sub, + per, ..
    const int64_t t0 = (int64_t)blockIdx.x * a.range, t1 = min(t0 + a.range, a.n);
    int ahead = mine ? (int)((t1 - t0 - sub + a.per - 1) / a.per) : 0;  // vectors still to fetch, to work on
    int todo = ahead;
    const View xv = is_q ? a.q : a.k, yv = is_q ? a.qo : a.ko, gv = is_q ? a.gq : a.gk;
    const T* xp = static_cast<const T*>(xv.p) + hh * xv.head + (t0 + sub) * xv.row;
    T* yp = static_cast<T*>(const_cast<void*>(yv.p)) + hh * yv.head + (t0 + sub) * yv.row;
    const T* gp = BWD ? static_cast<const T*>(gv.p) + hh * gv.head + (t0 + sub) * gv.row : nullptr;
    const int64_t xstep = xv.row * a.per, ystep = yv.row * a.per, gstep = gv.row * a.per;
    const uint32_t ring = smem_u32(s_ring + threadIdx.x);
    auto fetch_next = [&](int place) {
        if (ahead > 0) {
            const uint32_t to = ring + place * kPlace * 16;
            if (!BWD || a.norm) fetch<T, HALVES>(to, xp, lane, a.d);
            if constexpr (BWD) fetch<T, HALVES>(to + kPieces * kThreads * 16, gp, lane, a.d);
            xp += xstep;
            if constexpr (BWD) gp += gstep;
            --ahead;
        }
        cp_async_commit();
    };
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) fetch_next(i);

    float2* now = reinterpret_cast<float2*>(s_ring + kStages * kPlace);  // [tile][d / 2] cosine and sine
    float2* then = now + tile * half_d;
    auto angles = [&](int64_t t, float2* to) {
        for (int e = threadIdx.x; e < tile * half_d; e += kThreads) {
            const int tt = e / half_d, p = e - tt * half_d;
            float c = 1.f, s = 0.f;
            if (p < a.pairs[0] + a.pairs[1] + a.pairs[2] && t + tt < t1) {
                const int axis = p < a.pairs[0] ? 0 : (p < a.pairs[0] + a.pairs[1] ? 1 : 2);
                sincosf(__fmul_rn((float)a.coords[(t + tt) * 4 + 1 + axis], a.freqs[p]), &s, &c);
            }
            to[e] = make_float2(c, s);
        }
    };
    if (turn) {
        angles(t0, now);
        __syncthreads();
    }
    int place = 0;
    for (int64_t tt = t0; tt < t1; tt += tile) {
        if (turn && tt + tile < t1) angles(tt + tile, then);
        for (int k = 0; k < a.turns; ++k) {
            cp_async_wait<kStages - 2>();
            const bool have = todo-- > 0;
            float x[8];
            const uint4* from = s_ring + place * kPlace + threadIdx.x;
            read<T>(from, have && (!BWD || a.norm), x);
            // the place before this one has been read and used
            const int free = place == 0 ? kStages - 1 : place - 1;
            place = place == kStages - 1 ? 0 : place + 1;
            fetch_next(free);
            float4 cs[2] = {make_float4(1.f, 0.f, 1.f, 0.f), make_float4(1.f, 0.f, 1.f, 0.f)};
            if (turn && have) {
                const float4* c = reinterpret_cast<const float4*>(now + (k * a.per + sub) * half_d + 4 * lane);
                cs[0] = c[0];
                cs[1] = c[1];
            }
            float y[8];
            if constexpr (!BWD) {
                float r = 1.f;
                if (a.norm) {
                    float ss = 0.f;
#pragma unroll
                    for (int j = 0; j < 8; ++j) ss += x[j] * x[j];
                    r = rsqrtf(group_sum(ss, a.lanes) * a.inv_d + a.eps);
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    constexpr bool H = HALVES;
                    const float c = j & 1 ? cs[j >> 1].z : cs[j >> 1].x, sn = j & 1 ? cs[j >> 1].w : cs[j >> 1].y;
                    const float n0 = x[first_of<H>(j)] * r * w[first_of<H>(j)];
                    const float n1 = x[second_of<H>(j)] * r * w[second_of<H>(j)];
                    y[first_of<H>(j)] = n0 * c - n1 * sn;
                    y[second_of<H>(j)] = n0 * sn + n1 * c;
                }
            } else {
                float g[8];
                read<T>(from + kPieces * kThreads, have, g);
#pragma unroll
                for (int j = 0; j < 4; ++j) {  // y: the gradient of the normed, unturned vector
                    constexpr bool H = HALVES;
                    const float c = j & 1 ? cs[j >> 1].z : cs[j >> 1].x, sn = j & 1 ? cs[j >> 1].w : cs[j >> 1].y;
                    const float g0 = g[first_of<H>(j)], g1 = g[second_of<H>(j)];
                    y[first_of<H>(j)] = g0 * c + g1 * sn;
                    y[second_of<H>(j)] = g1 * c - g0 * sn;
                }
                if (a.norm) {
                    float ss = 0.f, dot = 0.f;
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        ss += x[j] * x[j];
                        g[j] = w[j] * y[j];
                        dot += x[j] * g[j];
                    }
                    const float r = rsqrtf(group_sum(ss, a.lanes) * a.inv_d + a.eps);
                    const float back = group_sum(dot, a.lanes) * a.inv_d * r * r;
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        gw[j] += y[j] * (x[j] * r);
                        y[j] = r * (g[j] - x[j] * back);
                    }
                }
            }
            if (have) store_vec<T, HALVES>(yp, lane, a.d, y);
            yp += ystep;
        }
        if (turn) {
            __syncthreads();  // the next angles are there, these have been used
            float2* t = now;
            now = then;
            then = t;
        }
    }
    cp_async_wait_all();
    if constexpr (BWD) {
        if (a.partial) {
            // one row per block: the tokens held side by side are added in order
            __syncthreads();
            float* s_gw = reinterpret_cast<float*>(s_ring);  // [per][chunk][d]
            if (mine) {
                float* dst = s_gw + ((size_t)sub * a.chunk + hl) * a.d;
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    dst[HALVES ? (j < 4 ? 4 * lane + j : half_d + 4 * lane + j - 4) : 8 * lane + j] = gw[j];
            }
            __syncthreads();
            float* row = a.partial + (size_t)blockIdx.x * a.ht * a.d;
            if (a.shared) {  // a row for each block of the token's blocks: its query heads' sum, its key heads' sum
                row = a.partial + ((size_t)blockIdx.x * gridDim.y + blockIdx.y) * 2 * a.d;
                const int split = max(0, min(heads, a.hq - h0));
                for (int e = threadIdx.x; e < 2 * a.d; e += kThreads) {
                    const int col = e < a.d ? e : e - a.d;
                    float sum = 0.f;
                    for (int s = 0; s < a.per; ++s)
                        for (int i = e < a.d ? 0 : split; i < (e < a.d ? split : heads); ++i)
                            sum += s_gw[((size_t)s * a.chunk + i) * a.d + col];
                    row[e] = sum;
                }
            } else {
                for (int e = threadIdx.x; e < heads * a.d; e += kThreads) {
                    float sum = 0.f;
                    for (int s = 0; s < a.per; ++s) sum += s_gw[(size_t)s * a.chunk * a.d + e];
                    row[h0 * a.d + e] = sum;
                }
            }
        }
    }
}

// Column sums of the blocks' weight-gradient rows, in a fixed order: kReduceRows running
// sums, then those.  The first cols_a columns are the first output's.
template <typename T>
__global__ void __launch_bounds__(32 * kReduceRows) k_weight_reduce(const float* __restrict__ partial, int rows,
                                                                    int cols, int cols_a, T* ga, T* gb) {
    __shared__ float s[kReduceRows][33];
    const int c = blockIdx.x * 32 + (threadIdx.x & 31);
    const int rl = threadIdx.x >> 5;
    float sum = 0.f;
    wait_for_previous();
    if (c < cols) {
#pragma unroll 8
        for (int row = rl; row < rows; row += kReduceRows) sum += partial[(size_t)row * cols + c];
    }
    s[rl][threadIdx.x & 31] = sum;
    __syncthreads();
    if (rl == 0 && c < cols) {
        float tot = 0.f;
#pragma unroll
        for (int i = 0; i < kReduceRows; ++i) tot += s[i][threadIdx.x & 31];
        if (c < cols_a) {
            if (ga) ga[c] = from_f32<T>(tot);
        } else if (gb) {
            gb[c - cols_a] = from_f32<T>(tot);
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

// Blocks along the tokens: one round of them.
int grid_x(int64_t n, int per, int chunks, int sms, bool bwd) {
    const int64_t cap = std::max<int64_t>(1, (int64_t)sms * per_sm(bwd) / chunks);
    return (int)std::max<int64_t>(1, std::min((n + per - 1) / per, cap));
}

template <typename T>
int launch(const RopeArgs& a, bool halves, bool bwd, int gx, int chunks, size_t smem, cudaStream_t s) {
    auto kernel = bwd ? (halves ? k_qk_norm_rope<T, true, true> : k_qk_norm_rope<T, false, true>)
                      : (halves ? k_qk_norm_rope<T, true, false> : k_qk_norm_rope<T, false, false>);
    if (smem > 48 * 1024 &&
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess)
        return VG_ERR_CUDA;
    kernel<<<dim3(gx, chunks), kThreads, smem, s>>>(a);
    return cudaPeekAtLastError() == cudaSuccess ? VG_OK : VG_ERR_CUDA;
}

}  // namespace

size_t rope_workspace_bytes(int64_t n, int hq, int hk, int d, int sms) {
    int lanes, chunk, per;
    const int ht = hq + hk;
    shape(ht, d, &lanes, &chunk, &per);
    const int chunks = (ht + chunk - 1) / chunk;
    // shared weights: chunks rows of two heads in place of one of ht
    return align_up((size_t)grid_x(n, per, chunks, sms, true) * std::max(ht, 2 * chunks) * d * 4, 256);
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
    a.shared = (c.flags & VG_QK_SHARED_WEIGHT) != 0;
    const int gx = grid_x(c.n, a.per, chunks, c.sms, bwd);
    a.range = (c.n + gx - 1) / gx;
    // a table of angles has one for every thread, if the block's tokens are that many
    const int steps = (int)std::min<int64_t>((a.range + a.per - 1) / a.per, kThreads);
    a.turns = std::max(1, std::min(steps, kThreads / (a.per * (a.d / 2))));
    const size_t ring = (size_t)kStages * kThreads * 8 * (c.dtype == VG_F32 ? 4 : 2) * (bwd ? 2 : 1);
    const size_t smem = std::max(ring + (size_t)2 * a.per * a.turns * (a.d / 2) * sizeof(float2),
                                 bwd ? (size_t)a.per * a.chunk * a.d * sizeof(float) : 0);
    const bool halves = (c.flags & VG_ROPE_HALVES) != 0;
    int st = c.dtype == VG_F32   ? launch<float>(a, halves, bwd, gx, chunks, smem, s)
             : c.dtype == VG_F16 ? launch<__half>(a, halves, bwd, gx, chunks, smem, s)
                                 : launch<__nv_bfloat16>(a, halves, bwd, gx, chunks, smem, s);
    if (st != VG_OK || !gw) return st;
    return reduce_rows(a.partial, a.shared ? gx * chunks : gx, (a.shared ? 2 : a.ht) * a.d, (a.shared ? 1 : a.hq) * a.d,
                       c.dtype, c.grad_q_weight, c.grad_k_weight, false, s);
}

template <typename T>
static int reduce_rows(const float* partial, int rows, int cols, int cols_a, void* a, void* b, bool overlap,
                       cudaStream_t s) {
    const unsigned grid = (cols + 31) / 32, threads = 32 * kReduceRows;
    T *ta = static_cast<T*>(a), *tb = static_cast<T*>(b);
    if (overlap)
        return launch_after(k_weight_reduce<T>, grid, threads, 0, s, partial, rows, cols, cols_a, ta, tb) == cudaSuccess
                   ? VG_OK : VG_ERR_CUDA;
    k_weight_reduce<T><<<grid, threads, 0, s>>>(partial, rows, cols, cols_a, ta, tb);
    return cudaPeekAtLastError() == cudaSuccess ? VG_OK : VG_ERR_CUDA;
}
int reduce_rows(const float* partial, int rows, int cols, int cols_a, int dtype, void* a, void* b, bool overlap,
                cudaStream_t s) {
    return dtype == VG_F32   ? reduce_rows<float>(partial, rows, cols, cols_a, a, b, overlap, s)
           : dtype == VG_F16 ? reduce_rows<__half>(partial, rows, cols, cols_a, a, b, overlap, s)
                             : reduce_rows<__nv_bfloat16>(partial, rows, cols, cols_a, a, b, overlap, s);
}

}  // namespace vg
