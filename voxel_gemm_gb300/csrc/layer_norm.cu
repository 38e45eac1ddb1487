// Layer norm of rows of channels, forward and backward, one pass over the rows each.
//
//   z = (x - mean) rstd,  y = z w + b
// backward, g = dy w:  dx = rstd (g - mean(g) - z mean(g z)) (+ the skipped gradient),
//   dw = sum over rows of dy z,  db = sum of dy
//
// Bound by memory (every element is read and written once).  A group of lanes holds a row, some
// 16-byte vectors a lane, so the row's sums are shuffles, and beyond 32 lanes one exchange in
// shared memory: the squares are taken from the mean of the warp's own elements and moved to
// the row's mean afterwards, M2 = sum over warps (M2_w + n_w (mean_w - mean)^2), so there is no
// difference of large numbers and no second exchange.  A block of 256 threads runs along a range
// of rows.  Every lane copies its vectors of the next rows into its own places of a ring in shared
// memory (asynchronously, without a barrier: no lane reads another's), so that the loads in flight
// cost no registers; the weights, and in the backward pass the sums of dw and db, stay in
// registers.  Those sums leave as one fp32 row per block, added in a fixed order by a second
// kernel, so they do not change from run to run.
#include "common.cuh"
#include "internal.h"
#include "tc_ptx.cuh"

namespace vg {

namespace {

using namespace ptx;

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxSmem = 227 * 1024;

// Ring places of a lane, by its vectors of a row.
constexpr int stages(int nv, bool bwd) { return nv == 1 ? (bwd ? 4 : 6) : nv == 2 ? (bwd ? 3 : 4) : nv <= 4 ? 3 : 2; }

struct Rows {
    const void* p;
    int64_t stride;
};

struct LnArgs {
    int64_t n;
    int c;
    int lanes;      // lanes of a row: a power of two, at most kThreads
    int64_t range;  // rows of a block
    Rows x, y;      // y: dx in the backward pass
    Rows gy, skip;
    const void* w;
    const void* b;
    float* stats;   // [n][2]
    float eps, inv_c;
    float* partial; // [blocks][2][c]: dw, db
};

__device__ __forceinline__ float lanes_sum(float x, int lanes) {
    for (int o = 1; o < lanes; o <<= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

template <typename T>
__device__ __forceinline__ void unpack(uint4 v, float (&x)[16 / sizeof(T)]) {
    const T* e = reinterpret_cast<const T*>(&v);
#pragma unroll
    for (int j = 0; j < 16 / (int)sizeof(T); ++j) x[j] = to_f32<T>(e[j]);
}
template <typename T>
__device__ __forceinline__ uint4 pack(const float (&x)[16 / sizeof(T)]) {
    uint4 v;
    T* e = reinterpret_cast<T*>(&v);
#pragma unroll
    for (int j = 0; j < 16 / (int)sizeof(T); ++j) e[j] = from_f32<T>(x[j]);
    return v;
}

template <typename T, int NV, bool BWD>
__global__ void __launch_bounds__(kThreads, NV == 1 ? 4 : NV == 2 ? 3 : 2) k_layer_norm(const LnArgs a) {
    extern __shared__ uint4 s_ring[];  // [stages][x, dy, skip][NV][kThreads]
    __shared__ float2 s_sum[2][kWarps];
    __shared__ float s_count[kWarps];
    constexpr int V = 16 / (int)sizeof(T), kStages = stages(NV, BWD);
    const int parts = BWD ? (a.skip.p ? 3 : 2) : 1;
    const int lane = threadIdx.x & (a.lanes - 1), sub = threadIdx.x / a.lanes;
    const int per = kThreads / a.lanes, warp = threadIdx.x >> 5;
    const int width = min(a.lanes, 32);
    const int warps = a.lanes > 32 ? a.lanes / 32 : 1;  // of a row
    const int vectors = a.c / V;
    int mine = 0;  // vectors of this lane: lane, lane + lanes, ..
    for (int i = 0; i < NV; ++i) mine += i * a.lanes + lane < vectors;

    // how many of the row's elements each of its warps holds
    if (warps > 1) {
        const float count = lanes_sum((float)(mine * V), 32);
        if ((threadIdx.x & 31) == 0) s_count[warp] = count;
        __syncthreads();
    }
    const float warp_count = warps > 1 ? s_count[warp] : (float)a.c;
    const float inv_count = warp_count > 0.f ? 1.f / warp_count : 0.f;

    uint4 w[NV], b[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        float ones[V], zeros[V];
#pragma unroll
        for (int j = 0; j < V; ++j) ones[j] = 1.f, zeros[j] = 0.f;
        w[i] = pack<T>(ones);
        b[i] = pack<T>(zeros);
        if (i < mine) {
            if (a.w) w[i] = static_cast<const uint4*>(a.w)[i * a.lanes + lane];
            if (!BWD && a.b) b[i] = static_cast<const uint4*>(a.b)[i * a.lanes + lane];
        }
    }
    constexpr int kAcc = BWD ? NV * V : 1;
    float gw[kAcc], gb[kAcc];
#pragma unroll
    for (int j = 0; j < kAcc; ++j) gw[j] = gb[j] = 0.f;

    // the block's rows [r0, r1); this group's are r0 + sub, + per, ..; all groups take as many turns
    const int64_t r0 = (int64_t)blockIdx.x * a.range, r1 = min(r0 + a.range, a.n);
    const int turns = r1 > r0 ? (int)((r1 - r0 + per - 1) / per) : 0;
    const uint32_t ring = smem_u32(s_ring + threadIdx.x);
    const int place_size = parts * NV * kThreads;
    int fetched = 0;
    auto fetch_next = [&](int place) {
        const int64_t r = r0 + sub + (int64_t)fetched * per;
        if (r < r1) {
            const uint32_t to = ring + place * place_size * 16;
            const T* xp = static_cast<const T*>(a.x.p) + r * a.x.stride + lane * V;
            const T* gp = BWD ? static_cast<const T*>(a.gy.p) + r * a.gy.stride + lane * V : nullptr;
            const T* sp = BWD && parts == 3 ? static_cast<const T*>(a.skip.p) + r * a.skip.stride + lane * V : nullptr;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                if (i < mine) {
                    cp_async16(to + i * kThreads * 16, xp + i * a.lanes * V, 16);
                    if constexpr (BWD) {
                        cp_async16(to + (NV + i) * kThreads * 16, gp + i * a.lanes * V, 16);
                        if (parts == 3) cp_async16(to + (2 * NV + i) * kThreads * 16, sp + i * a.lanes * V, 16);
                    }
                }
            }
        }
        ++fetched;
        cp_async_commit();
    };
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) fetch_next(i);

    int place = 0;
    for (int t = 0; t < turns; ++t) {
        const int64_t r = r0 + sub + (int64_t)t * per;
        const bool have = r < r1;
        cp_async_wait<kStages - 2>();
        fetch_next(place == 0 ? kStages - 1 : place - 1);  // the place before this one has been read and used
        const uint4* from = s_ring + place * place_size + threadIdx.x;
        float x[NV][V];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            unpack<T>(have && i < mine ? from[i * kThreads] : make_uint4(0, 0, 0, 0), x[i]);
        }
        if constexpr (!BWD) {
            float sum = 0.f;
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
                for (int j = 0; j < V; ++j) sum += x[i][j];
            sum = lanes_sum(sum, width);
            float mean = sum * inv_count, m2 = 0.f;
#pragma unroll
            for (int i = 0; i < NV; ++i)
                if (i < mine) {
#pragma unroll
                    for (int j = 0; j < V; ++j) m2 += (x[i][j] - mean) * (x[i][j] - mean);
                }
            m2 = lanes_sum(m2, width);
            if (warps > 1) {
                float2* buf = s_sum[t & 1];
                if ((threadIdx.x & 31) == 0) buf[warp] = make_float2(sum, m2);
                __syncthreads();
                const int w0 = warp & ~(warps - 1);
                sum = 0.f;
                for (int k = 0; k < warps; ++k) sum += buf[w0 + k].x;
                mean = sum * a.inv_c;
                m2 = 0.f;
                for (int k = 0; k < warps; ++k) {
                    const float cnt = s_count[w0 + k];
                    const float off = cnt > 0.f ? buf[w0 + k].x / cnt - mean : 0.f;
                    m2 += buf[w0 + k].y + cnt * off * off;
                }
            }
            const float rstd = rsqrtf(m2 * a.inv_c + a.eps);
            if (have) {
                if (a.stats && lane == 0) *reinterpret_cast<float2*>(a.stats + 2 * r) = make_float2(mean, rstd);
                T* yp = static_cast<T*>(const_cast<void*>(a.y.p)) + r * a.y.stride + lane * V;
#pragma unroll
                for (int i = 0; i < NV; ++i)
                    if (i < mine) {
                        float wf[V], bf[V], y[V];
                        unpack<T>(w[i], wf);
                        unpack<T>(b[i], bf);
#pragma unroll
                        for (int j = 0; j < V; ++j) y[j] = (x[i][j] - mean) * rstd * wf[j] + bf[j];
                        *reinterpret_cast<uint4*>(yp + i * a.lanes * V) = pack<T>(y);
                    }
            }
        } else {
            float2 st = make_float2(0.f, 0.f);
            if (have) st = *reinterpret_cast<const float2*>(a.stats + 2 * r);
            const float mean = st.x, rstd = st.y;
            float s1 = 0.f, s2 = 0.f;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                float g[V], wf[V];
                unpack<T>(have && i < mine ? from[(NV + i) * kThreads] : make_uint4(0, 0, 0, 0), g);
                unpack<T>(w[i], wf);
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    const float z = (x[i][j] - mean) * rstd;
                    gw[i * V + j] += g[j] * z;
                    gb[i * V + j] += g[j];
                    const float gz = g[j] * wf[j];
                    s1 += gz;
                    s2 += gz * z;
                }
            }
            s1 = lanes_sum(s1, width);
            s2 = lanes_sum(s2, width);
            if (warps > 1) {
                float2* buf = s_sum[t & 1];
                if ((threadIdx.x & 31) == 0) buf[warp] = make_float2(s1, s2);
                __syncthreads();
                const int w0 = warp & ~(warps - 1);
                s1 = s2 = 0.f;
                for (int k = 0; k < warps; ++k) {
                    s1 += buf[w0 + k].x;
                    s2 += buf[w0 + k].y;
                }
            }
            s1 *= a.inv_c;
            s2 *= a.inv_c;
            if (have) {
                T* yp = static_cast<T*>(const_cast<void*>(a.y.p)) + r * a.y.stride + lane * V;
#pragma unroll
                for (int i = 0; i < NV; ++i)
                    if (i < mine) {
                        float g[V], wf[V], y[V];
                        unpack<T>(from[(NV + i) * kThreads], g);
                        unpack<T>(w[i], wf);
#pragma unroll
                        for (int j = 0; j < V; ++j) {
                            const float z = (x[i][j] - mean) * rstd;
                            y[j] = (g[j] * wf[j] - s1 - z * s2) * rstd;
                        }
                        if (parts == 3) {
                            float k[V];
                            unpack<T>(from[(2 * NV + i) * kThreads], k);
#pragma unroll
                            for (int j = 0; j < V; ++j) y[j] += k[j];
                        }
                        *reinterpret_cast<uint4*>(yp + i * a.lanes * V) = pack<T>(y);
                    }
            }
        }
        place = place == kStages - 1 ? 0 : place + 1;
    }
    cp_async_wait_all();
    if constexpr (BWD) {
        if (a.partial) {
            // one row of dw and one of db per block: the rows held side by side are added in order
            __syncthreads();
            float* s_acc = reinterpret_cast<float*>(s_ring);  // [per][2][c]
#pragma unroll
            for (int i = 0; i < NV; ++i)
                if (i < mine) {
                    float* to = s_acc + (size_t)sub * 2 * a.c + (i * a.lanes + lane) * V;
#pragma unroll
                    for (int j = 0; j < V; ++j) {
                        to[j] = gw[i * V + j];
                        to[a.c + j] = gb[i * V + j];
                    }
                }
            __syncthreads();
            float* row = a.partial + (size_t)blockIdx.x * 2 * a.c;
            for (int e = threadIdx.x; e < 2 * a.c; e += kThreads) {
                float sum = 0.f;
                for (int k = 0; k < per; ++k) sum += s_acc[(size_t)k * 2 * a.c + e];
                row[e] = sum;
            }
        }
    }
}

// Lanes of a row and vectors of a lane: the fewest idle places with at most `most` vectors a lane
// (twice, then four times as many for the widest rows); among equals the most lanes of one warp.
void shape(int vectors, int most, int* lanes, int* nv) {
    while ((vectors + kThreads - 1) / kThreads > most) most *= 2;
    int best = 1 << 30;
    for (int l = 1; l <= kThreads; l <<= 1) {
        const int k = (vectors + l - 1) / l;
        if (k > most) continue;
        const int used = k <= 4 ? k : 8;  // compiled: 1, 2, 3, 4, 8
        if (l * used < best || (l * used == best && l <= 32)) {
            best = l * used;
            *lanes = l;
            *nv = used;
        }
        if (l >= vectors) break;
    }
}

struct Launch {
    int lanes, nv, per_sm, grid;
    int64_t range;
    size_t smem;
};

Launch plan(int64_t n, int c, int es, int parts, bool bwd, int sms) {
    Launch l{};
    shape(c * es / 16, bwd ? 2 : 4, &l.lanes, &l.nv);
    const int per = kThreads / l.lanes;
    l.smem = (size_t)stages(l.nv, bwd) * parts * l.nv * kThreads * 16;
    if (bwd) l.smem = std::max(l.smem, (size_t)per * 2 * c * 4);
    l.per_sm = std::max(1, std::min<int>(l.nv == 1 ? 4 : l.nv == 2 ? 3 : 2, kMaxSmem / (int)(l.smem + 1536)));
    const int64_t turns = std::max<int64_t>(1, (n + per - 1) / per);
    const int64_t cap = (int64_t)sms * l.per_sm;
    l.range = (turns + std::min(turns, cap) - 1) / std::min(turns, cap) * per;
    l.grid = (int)std::max<int64_t>(1, (n + l.range - 1) / l.range);
    return l;
}

template <typename T, int NV>
int launch(const LnArgs& a, const Launch& l, bool bwd, cudaStream_t s) {
    auto kernel = bwd ? k_layer_norm<T, NV, true> : k_layer_norm<T, NV, false>;
    if (l.smem > 40 * 1024 &&  // with the static part, above what every block may have
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)l.smem) != cudaSuccess)
        return VG_ERR_CUDA;
    kernel<<<l.grid, kThreads, l.smem, s>>>(a);
    return cudaPeekAtLastError() == cudaSuccess ? VG_OK : VG_ERR_CUDA;
}
template <typename T>
int launch(const LnArgs& a, const Launch& l, bool bwd, cudaStream_t s) {
    switch (l.nv) {
        case 1: return launch<T, 1>(a, l, bwd, s);
        case 2: return launch<T, 2>(a, l, bwd, s);
        case 3: return launch<T, 3>(a, l, bwd, s);
        case 4: return launch<T, 4>(a, l, bwd, s);
    }
    if constexpr (sizeof(T) == 4) return launch<T, 8>(a, l, bwd, s);  // more than 4096 channels in fp32
    return VG_ERR_UNSUPPORTED;
}

}  // namespace

size_t layer_norm_workspace_bytes(int64_t n, int c, int sms) {
    // the widest grid of any element type and operand count
    int grid = 1;
    for (int es = 2; es <= 4; es += 2)
        for (int parts = 2; parts <= 3; ++parts) grid = std::max(grid, plan(n, c, es, parts, true, sms).grid);
    return align_up((size_t)grid * 2 * c * 4, 256);
}

int layer_norm(const LayerNorm& q, bool bwd, cudaStream_t s) {
    const auto rows = [](const vg_rows* r) { return r ? Rows{r->data, r->row_stride} : Rows{}; };
    LnArgs a{};
    a.n = q.n;
    a.c = q.c;
    a.x = rows(q.x);
    a.y = rows(q.y);
    a.gy = rows(q.grad_y);
    a.skip = rows(q.grad_skip);
    a.w = q.weight;
    a.b = q.bias;
    a.stats = q.stats;
    a.eps = q.eps;
    a.inv_c = 1.f / (float)q.c;
    const bool sums = bwd && (q.grad_weight || q.grad_bias);
    a.partial = sums ? q.partial : nullptr;
    const Launch l = plan(q.n, q.c, q.dtype == VG_F32 ? 4 : 2, bwd ? (q.grad_skip ? 3 : 2) : 1, bwd, q.sms);
    a.lanes = l.lanes;
    a.range = l.range;
    const int st = q.dtype == VG_F32   ? launch<float>(a, l, bwd, s)
                   : q.dtype == VG_F16 ? launch<__half>(a, l, bwd, s)
                                       : launch<__nv_bfloat16>(a, l, bwd, s);
    if (st != VG_OK || !sums) return st;
    return reduce_rows(a.partial, l.grid, 2 * q.c, q.c, q.dtype, q.grad_weight, q.grad_bias, s);
}

}  // namespace vg
