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
// difference of large numbers and no second exchange.  Blocks of 256 threads go through the rows side
// by side.  Every lane copies its vectors of the next rows into its own places of a ring in shared
// memory (asynchronously, without a barrier: no lane reads another's), so that the loads in flight
// cost no registers; the weights, and in the backward pass the sums of dw and db, stay in
// registers.  Those sums leave as one fp32 row per block, added in a fixed order by a second
// kernel, so they do not change from run to run.
//
// GB300, bf16: 602,492 rows of 1024 forward 362 us (6.8 TB/s), backward 535 and 5 (6.9 TB/s; fp16, where four vectors a lane
// spill, 576); 319,057 rows of 128 forward 33 us, backward with a skipped gradient 53 in all (72 us of memory
// traffic).
#include "common.cuh"
#include "internal.h"
#include "tc_ptx.cuh"

namespace vg {

namespace {

using namespace ptx;

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxSmem = 227 * 1024;

// Ring places of a lane, by its vectors of a row: one or two rows on their way.  (More make memory
// slower: with two in place of one, 602k rows of 1024 took 413 us forward, so 368.)
constexpr int stages(int nv) { return nv == 1 ? 3 : 2; }

// Blocks per SM, by their registers (64, 80, 128 a thread).
constexpr int per_sm(int nv) { return nv == 1 ? 4 : nv == 2 ? 3 : 2; }

struct Rows {
    const void* p;
    uint32_t stride;  // in bytes
};
__device__ __forceinline__ const char* at(const Rows& r, uint32_t row, int byte) {
    return static_cast<const char*>(r.p) + (uint64_t)row * r.stride + byte;
}

struct LnArgs {
    int64_t n;
    int c;
    int lanes;      // lanes of a row: a power of two, at most kThreads
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

// 16 bytes as pairs of fp32, which the paired instructions work on.
template <typename T> struct Vec {
    static constexpr int H = 8 / (int)sizeof(T);  // pairs
    float2 v[H];
};
template <typename T> __device__ __forceinline__ Vec<T> unpack(uint4 q) {
    Vec<T> r;
    if constexpr (sizeof(T) == 4) {
        r.v[0] = make_float2(__uint_as_float(q.x), __uint_as_float(q.y));
        r.v[1] = make_float2(__uint_as_float(q.z), __uint_as_float(q.w));
    } else {
        r.v[0] = Pair<T>::unpack(q.x);
        r.v[1] = Pair<T>::unpack(q.y);
        r.v[2] = Pair<T>::unpack(q.z);
        r.v[3] = Pair<T>::unpack(q.w);
    }
    return r;
}
template <typename T> __device__ __forceinline__ uint4 pack(const Vec<T>& r) {
    if constexpr (sizeof(T) == 4)
        return make_uint4(__float_as_uint(r.v[0].x), __float_as_uint(r.v[0].y), __float_as_uint(r.v[1].x),
                          __float_as_uint(r.v[1].y));
    else
        return make_uint4(Pair<T>::pack(r.v[0]), Pair<T>::pack(r.v[1]), Pair<T>::pack(r.v[2]), Pair<T>::pack(r.v[3]));
}
template <typename T> __device__ __forceinline__ Vec<T> filled(float x) {
    Vec<T> r;
#pragma unroll
    for (int j = 0; j < Vec<T>::H; ++j) r.v[j] = make_float2(x, x);
    return r;
}
// A vector kept for the whole run: unpacked while there are few.
template <typename T, bool OPEN> struct Kept {
    Vec<T> r;
    __device__ __forceinline__ void set(uint4 q) { r = unpack<T>(q); }
    __device__ __forceinline__ Vec<T> get() const { return r; }
};
template <typename T> struct Kept<T, false> {
    uint4 q;
    __device__ __forceinline__ void set(uint4 x) { q = x; }
    __device__ __forceinline__ Vec<T> get() const { return unpack<T>(q); }
};

// PARTS operands: 1 forward, 2 backward, 3 with a skipped gradient.
template <typename T, int NV, int PARTS>
__global__ void __launch_bounds__(kThreads, per_sm(NV)) k_layer_norm(const LnArgs a) {
    constexpr bool BWD = PARTS > 1;
    extern __shared__ uint4 s_ring[];  // [stages][x, dy, skip][NV][kThreads]
    __shared__ float2 s_sum[2][kWarps];
    __shared__ float s_count[kWarps];
    using W = Vec<T>;
    constexpr int V = 16 / (int)sizeof(T), H = W::H, kStages = stages(NV);
    constexpr bool kOpen = NV <= (BWD ? 1 : 2);
    constexpr int kPlace = PARTS * NV * kThreads;
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

    Kept<T, kOpen> w[NV], b[BWD ? 1 : NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        w[i].set(a.w && i < mine ? static_cast<const uint4*>(a.w)[i * a.lanes + lane] : pack<T>(filled<T>(1.f)));
        if constexpr (!BWD)
            b[i].set(a.b && i < mine ? static_cast<const uint4*>(a.b)[i * a.lanes + lane] : make_uint4(0, 0, 0, 0));
    }
    constexpr int kAcc = BWD ? NV : 1;
    W gw[kAcc], gb[kAcc];
#pragma unroll
    for (int i = 0; i < kAcc; ++i) gw[i] = gb[i] = filled<T>(0.f);

    // this group's rows are blockIdx.x * per + sub, + the whole grid's, ..; all groups of a block take
    // as many turns.  (Rows that are far apart in time lie far apart: with a range of rows to each block
    // 602k rows of 1024 took 1021 us for both passes, so 968.)
    const uint32_t r0 = blockIdx.x * per, r1 = (uint32_t)a.n, hop = gridDim.x * per;
    const int turns = r1 > r0 ? (int)((r1 - r0 + hop - 1) / hop) : 0;
    const uint32_t ring = smem_u32(s_ring + threadIdx.x);
    const int byte = lane * 16, step = a.lanes * 16;  // of the lane's first vector, and to the next
    uint32_t row = r0 + sub, ahead = row;             // this turn's, and the next to be sent for (32 bits leave 2^31 behind the last row)
    auto fetch_next = [&](int place) {
        if (ahead < r1) {
            const uint32_t to = ring + place * kPlace * 16;
#pragma unroll
            for (int p = 0; p < PARTS; ++p) {
                const char* from = at(p == 0 ? a.x : p == 1 ? a.gy : a.skip, ahead, byte);
#pragma unroll
                for (int i = 0; i < NV; ++i)
                    if (i < mine) cp_async16(to + (p * NV + i) * kThreads * 16, from + i * step, 16);
            }
        }
        ahead += hop;
        cp_async_commit();
    };
    for (int k = 0; k < kStages * PARTS; ++k)  // places that no row fills: zeros
        for (int i = mine; i < NV; ++i) s_ring[(k * NV + i) * kThreads + threadIdx.x] = make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) fetch_next(i);

    int place = 0;
    float2 st = make_float2(0.f, 0.f);
    const float2* const stats = reinterpret_cast<const float2*>(a.stats);
    if (BWD && row < r1) st = stats[row];
#pragma unroll 1
    for (int t = 0; t < turns; ++t, row += hop) {
        const bool have = row < r1;
        cp_async_wait<kStages - 2>();
        fetch_next(place == 0 ? kStages - 1 : place - 1);  // the place before this one has been read and used
        const uint4* from = s_ring + place * kPlace + threadIdx.x;
        // (Without a row: whatever was there.  It enters the sums of this group's lanes alone, which then
        // go nowhere.)
        const auto vec = [&](int part, int i) { return unpack<T>(from[(part * NV + i) * kThreads]); };
        if constexpr (!BWD) {
            W x[NV];
            float2 sum2 = make_float2(0.f, 0.f);
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                x[i] = vec(0, i);
#pragma unroll
                for (int j = 0; j < H; ++j) sum2 = add2(sum2, x[i].v[j]);
            }
            float sum = lanes_sum(sum2.x + sum2.y, width);
            float mean = sum * inv_count;
            float2 m22 = make_float2(0.f, 0.f);
            const float2 off2 = make_float2(-mean, -mean);
#pragma unroll
            for (int i = 0; i < NV; ++i)
                if (i < mine) {
#pragma unroll
                    for (int j = 0; j < H; ++j) {
                        const float2 d = add2(x[i].v[j], off2);
                        m22 = fma2(d, d, m22);
                    }
                }
            float m2 = lanes_sum(m22.x + m22.y, width);
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
                if (stats && lane == 0) reinterpret_cast<float2*>(a.stats)[row] = make_float2(mean, rstd);
                char* const y = const_cast<char*>(at(a.y, row, byte));
                const float2 r2 = make_float2(rstd, rstd), n2 = make_float2(-mean, -mean);
#pragma unroll
                for (int i = 0; i < NV; ++i)
                    if (i < mine) {
                        const W wf = w[i].get(), bf = b[i].get();
                        W o;
#pragma unroll
                        for (int j = 0; j < H; ++j)
                            o.v[j] = fma2(mul2(add2(x[i].v[j], n2), r2), wf.v[j], bf.v[j]);
                        *reinterpret_cast<uint4*>(y + i * step) = pack<T>(o);
                    }
            }
        } else {
            const float rstd = st.y;
            const float2 r2 = make_float2(rstd, rstd), n2 = make_float2(-st.x, -st.x);
            if (row + hop < r1) st = stats[row + hop];
            float2 s1 = make_float2(0.f, 0.f), s2 = s1;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const W x = vec(0, i), g = vec(1, i), wf = w[i].get();
#pragma unroll
                for (int j = 0; j < H; ++j) {
                    const float2 z = mul2(add2(x.v[j], n2), r2);  // as forward: mean rstd would be rounded too
                    if (have) {
                        gw[i].v[j] = fma2(g.v[j], z, gw[i].v[j]);
                        gb[i].v[j] = add2(gb[i].v[j], g.v[j]);
                    }
                    const float2 gz = mul2(g.v[j], wf.v[j]);
                    s1 = add2(s1, gz);
                    s2 = fma2(gz, z, s2);
                }
            }
            float a1 = lanes_sum(s1.x + s1.y, width), a2 = lanes_sum(s2.x + s2.y, width);
            if (warps > 1) {
                float2* buf = s_sum[t & 1];
                if ((threadIdx.x & 31) == 0) buf[warp] = make_float2(a1, a2);
                __syncthreads();
                const int w0 = warp & ~(warps - 1);
                a1 = a2 = 0.f;
                for (int k = 0; k < warps; ++k) {
                    a1 += buf[w0 + k].x;
                    a2 += buf[w0 + k].y;
                }
            }
            a1 *= -a.inv_c;
            a2 *= -a.inv_c * rstd;
            if (have) {  // dx = rstd (g - mean(g) - (x - mean) (mean(g z) rstd)), from the ring once more
                const float2 c1 = make_float2(a1, a1), c2 = make_float2(a2, a2);
                char* const y = const_cast<char*>(at(a.y, row, byte));
                int place_again = 0;
                asm volatile("" : "+r"(place_again));  // read again: what is kept since the sums would spill
                const auto vec = [&](int part, int i) {
                    return unpack<T>(from[place_again + (part * NV + i) * kThreads]);
                };
#pragma unroll
                for (int i = 0; i < NV; ++i)
                    if (i < mine) {
                        const W x = vec(0, i), g = vec(1, i), wf = w[i].get();
                        W o;
#pragma unroll
                        for (int j = 0; j < H; ++j)
                            o.v[j] = fma2(add2(x.v[j], n2), c2, fma2(g.v[j], wf.v[j], c1));
                        if constexpr (PARTS == 3) {
                            const W k = vec(2, i);
#pragma unroll
                            for (int j = 0; j < H; ++j) o.v[j] = fma2(o.v[j], r2, k.v[j]);
                        } else {
#pragma unroll
                            for (int j = 0; j < H; ++j) o.v[j] = mul2(o.v[j], r2);
                        }
                        *reinterpret_cast<uint4*>(y + i * step) = pack<T>(o);
                    }
            }
        }
        place = place == kStages - 1 ? 0 : place + 1;
    }
    cp_async_wait_all();
    if constexpr (BWD) {
        dependents_may_start();  // now, not before: the sums' blocks would take the place of these
        if (a.partial) {
            // one row of dw and one of db per block: the rows held side by side are added in order
            __syncthreads();
            float* s_acc = reinterpret_cast<float*>(s_ring);  // [per][2][c]
#pragma unroll
            for (int i = 0; i < NV; ++i)
                if (i < mine) {
                    float2* to = reinterpret_cast<float2*>(s_acc + (size_t)sub * 2 * a.c + (i * a.lanes + lane) * V);
#pragma unroll
                    for (int j = 0; j < H; ++j) {
                        to[j] = gw[i].v[j];
                        to[a.c / 2 + j] = gb[i].v[j];
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

// Lanes of a row and vectors of a lane, up to 4, or 2 in the backward pass where several warps hold a
// row (twice that for the widest): the fewest idle places; among equals the fewest lanes from 8 (128 bytes) on,
// which leaves fewer exchanges a row.  (bf16, both passes: 319k rows of 256 161 us with 8 lanes, 166 with
// 32.  602k rows of 1024: 1026 with 4 vectors in one warp, 1115 with 2 in two, 1183 with 1 in four.  150k rows of
// 4096: backward pass 736 with 2 in eight warps, 1030 with 4 in four; forward 431 with 4 in four, 638 with 2 in eight.)
void shape(int vectors, bool bwd, int* lanes, int* nv) {
    int most = bwd && vectors > 4 * 32 ? 2 : 4;
    while ((vectors + kThreads - 1) / kThreads > most) most *= 2;
    int best = 1 << 30;
    for (int l = 1; l <= kThreads; l <<= 1) {
        const int k = (vectors + l - 1) / l;
        if (k > most) continue;
        const int used = k <= 4 ? k : 8;  // compiled: 1, 2, 3, 4, 8
        if (l * used < best || (l * used == best && l <= 8)) {
            best = l * used;
            *lanes = l;
            *nv = used;
        }
        if (l >= vectors) break;
    }
}

struct Launch {
    int lanes, nv, grid;
    size_t smem;
};

Launch plan(int64_t n, int c, int es, int parts, bool bwd, int sms) {
    Launch l{};
    shape(c * es / 16, bwd, &l.lanes, &l.nv);
    const int per = kThreads / l.lanes;
    l.smem = (size_t)stages(l.nv) * parts * l.nv * kThreads * 16;
    if (bwd) l.smem = std::max(l.smem, (size_t)per * 2 * c * 4);
    const int blocks = std::max(1, std::min<int>(per_sm(l.nv), kMaxSmem / (int)(l.smem + 1536)));
    l.grid = (int)std::max<int64_t>(1, std::min((n + per - 1) / per, (int64_t)sms * blocks));
    return l;
}

template <typename T, int NV>
int launch(const LnArgs& a, const Launch& l, int parts, cudaStream_t s) {
    const auto kernel = parts == 1 ? k_layer_norm<T, NV, 1> : parts == 2 ? k_layer_norm<T, NV, 2> : k_layer_norm<T, NV, 3>;
    if (l.smem > 40 * 1024 &&  // with the static part, above what every block may have
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)l.smem) != cudaSuccess)
        return VG_ERR_CUDA;
    kernel<<<l.grid, kThreads, l.smem, s>>>(a);
    return cudaPeekAtLastError() == cudaSuccess ? VG_OK : VG_ERR_CUDA;
}
template <typename T>
int launch(const LnArgs& a, const Launch& l, int parts, cudaStream_t s) {
    switch (l.nv) {
        case 1: return launch<T, 1>(a, l, parts, s);
        case 2: return launch<T, 2>(a, l, parts, s);
        case 3: return launch<T, 3>(a, l, parts, s);
        case 4: return launch<T, 4>(a, l, parts, s);
    }
    if constexpr (sizeof(T) == 4) return launch<T, 8>(a, l, parts, s);  // more than 4096 channels in fp32
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
    const int es = q.dtype == VG_F32 ? 4 : 2, parts = bwd ? (q.grad_skip ? 3 : 2) : 1;
    const auto rows = [&](const vg_rows* r) {
        return r ? Rows{r->data, q.n > 1 ? (uint32_t)(r->row_stride * es) : 0u} : Rows{};
    };
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
    const Launch l = plan(q.n, q.c, es, parts, bwd, q.sms);
    a.lanes = l.lanes;
    const int st = q.dtype == VG_F32   ? launch<float>(a, l, parts, s)
                   : q.dtype == VG_F16 ? launch<__half>(a, l, parts, s)
                                       : launch<__nv_bfloat16>(a, l, parts, s);
    if (st != VG_OK || !sums) return st;
    return reduce_rows(a.partial, l.grid, 2 * q.c, q.c, q.dtype, q.grad_weight, q.grad_bias, true, s);
}

}  // namespace vg
