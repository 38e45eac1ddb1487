// Cross attention on the CUDA cores, exact fp32: forward, query gradient, and key
// and value gradient.
//
//   S = scale q k^T over a sample's valid keys, P = softmax(S), O = P V
//   dP = dO V^T, dS = P (dP - delta), delta = sum_d dO O
//   dQ = scale dS K,  dK = scale dS^T Q,  dV = P^T dO
//
// One block of 256 threads per 64 queries (forward, dQ) or 64 keys (dK, dV) of a
// sample and head, running along the other axis in tiles of 64 with the running
// maximum and sum of the softmax; scores are recomputed from the saved log-sum in
// the backward pass, so nothing of size queries x keys is stored.  Each thread
// holds 4 x 4 of a 64 x 64 product, so every float4 read from shared memory feeds
// 8 multiply-adds, issued two to an instruction; row pitches of d + 4 and 68 floats keep
// those reads free of bank conflicts.  Bound by the reads of shared memory and, at two
// blocks per SM, their latency: 20,000 queries over 2 x 2,000 keys, 8 heads of 64, take
// 2.6 ms forward (32 TFLOP/s), 3.6 for dQ and 6.2 for dK and dV.  8 x 4 per thread with half
// the threads takes fewer reads but was slower (3.3, 5.2, 8.6 ms): too few warps.
#include "attn.cuh"
#include "tc_ptx.cuh"

namespace vg {

namespace {

constexpr int kT = 64;             // rows and columns of a tile
constexpr int kThreads = 256;
constexpr int kPP = kT + 4;        // pitch of a score tile
constexpr float kLn2 = 0.69314718055994530942f;

// 64 rows from `row` on of one head into shared memory; rows from `rows` on are zero.
__device__ __forceinline__ void load_tile(float* dst, const vg_heads& h, int64_t row, int head, int rows, int d) {
    const int q4 = d / 4;
    for (int e = threadIdx.x; e < kT * q4; e += kThreads) {
        const int r = e / q4, c = (e - r * q4) * 4;
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        if (r < rows) v = *reinterpret_cast<const float4*>(head_row<const float>(h, row + r, head) + c);
        *reinterpret_cast<float4*>(dst + r * (d + 4) + c) = v;
    }
}

// acc[a][b] = sum_d A[ty + 16 a][d] B[tx + 16 b][d]; even and odd channels have sums of their own
__device__ __forceinline__ void product_nt(const float* A, const float* B, int d, int ty, int tx, float (&acc)[4][4]) {
    const int p = d + 4;
    float2 sum[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) sum[i][j] = make_float2(0.f, 0.f);
#pragma unroll 2
    for (int c = 0; c < d; c += 4) {
        float4 x[4], y[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = *reinterpret_cast<const float4*>(A + (ty + 16 * i) * p + c);
#pragma unroll
        for (int j = 0; j < 4; ++j) y[j] = *reinterpret_cast<const float4*>(B + (tx + 16 * j) * p + c);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                sum[i][j] = ptx::fma2(make_float2(x[i].x, x[i].y), make_float2(y[j].x, y[j].y), sum[i][j]);
                sum[i][j] = ptx::fma2(make_float2(x[i].z, x[i].w), make_float2(y[j].z, y[j].w), sum[i][j]);
            }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = sum[i][j].x + sum[i][j].y;
}

// acc[a][c] (columns 4 tx + 64 c ..) += sum_j W[ty + 16 a][j] B[j][columns]
template <int NC>
__device__ __forceinline__ void product_nn(const float* W, const float* B, int d, int ty, int tx,
                                           float4 (&acc)[4][NC]) {
    const int p = d + 4;
#pragma unroll 2
    for (int j = 0; j < kT; j += 4) {
        float4 w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = *reinterpret_cast<const float4*>(W + (ty + 16 * i) * kPP + j);
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            const int col = tx * 4 + 64 * c;
            if (col >= d) continue;
#pragma unroll
            for (int jj = 0; jj < 4; ++jj) {
                const float4 v = *reinterpret_cast<const float4*>(B + (j + jj) * p + col);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float s = jj == 0 ? w[i].x : jj == 1 ? w[i].y : jj == 2 ? w[i].z : w[i].w;
                    const float2 s2 = make_float2(s, s);
                    float4& o = acc[i][c];
                    const float2 lo = ptx::fma2(s2, make_float2(v.x, v.y), make_float2(o.x, o.y));
                    const float2 hi = ptx::fma2(s2, make_float2(v.z, v.w), make_float2(o.z, o.w));
                    o = make_float4(lo.x, lo.y, hi.x, hi.y);
                }
            }
        }
    }
}

template <int NC>
__device__ __forceinline__ void zero(float4 (&acc)[4][NC]) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int c = 0; c < NC; ++c) acc[i][c] = make_float4(0.f, 0.f, 0.f, 0.f);
}

__device__ __forceinline__ void put4(float* p, float4 v) { *reinterpret_cast<float4*>(p) = v; }
__device__ __forceinline__ float4 times(float4 v, float s) { return make_float4(v.x * s, v.y * s, v.z * s, v.w * s); }

// ---------------------------------------------------------------- forward
template <int NC>
__global__ void __launch_bounds__(kThreads, 2) k_attn_fwd(const AttnArgs a) {
    extern __shared__ float sm[];
    const int p = a.d + 4;
    float *sQ = sm, *sK = sQ + kT * p, *sV = sK + kT * p, *sP = sV + kT * p;
    if (!attn_offsets_ok(a)) return;
    const AttnTile t = attn_find_tile<false>(a, kT, blockIdx.x);
    if (t.b < 0) return;
    const int h = blockIdx.y, hk = h / (a.hq / a.hk);
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    load_tile(sQ, a.q, t.q0 + t.first, h, t.lq - t.first, a.d);
    float m[4], l[4];
    float4 acc[4][NC];
#pragma unroll
    for (int i = 0; i < 4; ++i) m[i] = -INFINITY, l[i] = 0.f;
    zero<NC>(acc);
    int lo, hi;
    attn_split(a, t.lk, t.part, &lo, &hi);
    for (int kt = lo; kt < hi; ++kt) {
        const int left = t.lk - kt * kT;  // valid keys of the tile
        __syncthreads();
        load_tile(sK, a.k, t.k0 + kt * kT, hk, left, a.d);
        load_tile(sV, a.v, t.k0 + kt * kT, hk, left, a.d);
        __syncthreads();
        float s[4][4];
        product_nt(sQ, sK, a.d, ty, tx, s);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float top = m[i];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                s[i][j] = tx + 16 * j < left ? s[i][j] * a.scale_log2 : -INFINITY;
                top = fmaxf(top, s[i][j]);
            }
#pragma unroll
            for (int o = 1; o < 16; o <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
            const float base = top == -INFINITY ? 0.f : top;  // a row of scores -inf so far
            const float shrink = exp2f(m[i] - base);
            float sum = 0.f;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                s[i][j] = exp2f(s[i][j] - base);
                sum += s[i][j];
                sP[(ty + 16 * i) * kPP + tx + 16 * j] = s[i][j];
            }
#pragma unroll
            for (int o = 1; o < 16; o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
            l[i] = l[i] * shrink + sum;
            m[i] = top;
#pragma unroll
            for (int c = 0; c < NC; ++c) acc[i][c] = times(acc[i][c], shrink);
        }
        __syncthreads();
        product_nn<NC>(sP, sV, a.d, ty, tx, acc);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = t.first + ty + 16 * i;
        if (r >= t.lq) continue;
        const int64_t row = t.q0 + r;
        // no keys: zero; only keys of weight zero: NaN (a part of them has no sum to be normalised by)
        const float inv = hi <= lo ? 0.f : a.splits > 1 && l[i] == 0.f ? 1.f : 1.f / l[i];
        const float lse = hi > lo ? (m[i] + log2f(l[i])) * kLn2 : -INFINITY;
        if (tx == 0) {
            float* dst = a.splits > 1 ? a.part_lse + (size_t)t.part * a.hq * a.n_q : a.lse;
            if (dst) dst[(int64_t)h * a.n_q + row] = lse;
        }
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            const int col = tx * 4 + 64 * c;
            if (col >= a.d) continue;
            const float4 v = times(acc[i][c], inv);
            if (a.splits > 1)
                put4(a.part + (((size_t)t.part * a.n_q + row) * a.hq + h) * a.d + col, v);
            else
                put4(head_row<float>(a.o, row, h) + col, v);
        }
    }
}

// ---------------------------------------------------------------- query gradient
template <int NC>
__global__ void __launch_bounds__(kThreads, NC == 1 ? 2 : 1) k_attn_dq(const AttnArgs a) {
    extern __shared__ float sm[];
    const int p = a.d + 4;
    float *sQ = sm, *sG = sQ + kT * p, *sK = sG + kT * p, *sV = sK + kT * p, *sS = sV + kT * p;
    if (!attn_offsets_ok(a)) return;
    const AttnTile t = attn_find_tile<false>(a, kT, blockIdx.x);
    if (t.b < 0) return;
    const int h = blockIdx.y, hk = h / (a.hq / a.hk);
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    load_tile(sQ, a.q, t.q0 + t.first, h, t.lq - t.first, a.d);
    load_tile(sG, a.go, t.q0 + t.first, h, t.lq - t.first, a.d);
    float2 st[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = t.first + ty + 16 * i;
        st[i] = r < t.lq ? attn_stats(a, (int64_t)h * a.n_q + t.q0 + r) : make_float2(0.f, 0.f);
    }
    float4 acc[4][NC];
    zero<NC>(acc);
    int lo, hi;
    attn_split(a, t.lk, t.part, &lo, &hi);
    for (int kt = lo; kt < hi; ++kt) {
        const int left = t.lk - kt * kT;
        __syncthreads();
        load_tile(sK, a.k, t.k0 + kt * kT, hk, left, a.d);
        load_tile(sV, a.v, t.k0 + kt * kT, hk, left, a.d);
        __syncthreads();
        float s[4][4], dp[4][4];
        product_nt(sQ, sK, a.d, ty, tx, s);
        product_nt(sG, sV, a.d, ty, tx, dp);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float pr = exp2f(s[i][j] * a.scale_log2 + st[i].x);
                sS[(ty + 16 * i) * kPP + tx + 16 * j] = tx + 16 * j < left ? pr * (dp[i][j] + st[i].y) : 0.f;
            }
        __syncthreads();
        product_nn<NC>(sS, sK, a.d, ty, tx, acc);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = t.first + ty + 16 * i;
        if (r >= t.lq) continue;
        const int64_t row = t.q0 + r;
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            const int col = tx * 4 + 64 * c;
            if (col >= a.d) continue;
            const float4 v = times(acc[i][c], a.scale);
            if (a.splits > 1)
                put4(a.part + (((size_t)t.part * a.n_q + row) * a.hq + h) * a.d + col, v);
            else
                put4(head_row<float>(a.gq, row, h) + col, v);
        }
    }
}

// ---------------------------------------------------------------- key and value gradient
// The block's 64 keys run along the sample's queries of every head that reads
// them, in head order: gradients of shared heads are sums in one accumulator.
template <int NC>
__global__ void __launch_bounds__(kThreads, NC == 1 ? 2 : 1) k_attn_dkv(const AttnArgs a, float* part_dv) {
    extern __shared__ float sm[];
    const int p = a.d + 4;
    float *sQ = sm, *sG = sQ + kT * p, *sK = sG + kT * p, *sV = sK + kT * p;
    float *sP = sV + kT * p, *sS = sP + kT * kPP;
    if (!attn_offsets_ok(a)) return;
    const AttnTile t = attn_find_tile<true>(a, kT, blockIdx.x);
    if (t.b < 0) return;
    const int hk = blockIdx.y, group = a.hq / a.hk;
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    load_tile(sK, a.k, t.k0 + t.first, hk, t.lk - t.first, a.d);
    load_tile(sV, a.v, t.k0 + t.first, hk, t.lk - t.first, a.d);
    float4 dk[4][NC], dv[4][NC];
    zero<NC>(dk);
    zero<NC>(dv);
    int lo, hi;
    attn_split(a, t.lq, t.part, &lo, &hi);
    if (t.first >= t.lk) hi = lo;  // no valid key in the tile
    for (int g = 0; g < group; ++g) {
        const int h = hk * group + g;
        for (int qt = lo; qt < hi; ++qt) {
            const int left = t.lq - qt * kT;
            __syncthreads();
            load_tile(sQ, a.q, t.q0 + qt * kT, h, left, a.d);
            load_tile(sG, a.go, t.q0 + qt * kT, h, left, a.d);
            __syncthreads();
            float s[4][4], dp[4][4];
            product_nt(sK, sQ, a.d, ty, tx, s);
            product_nt(sV, sG, a.d, ty, tx, dp);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int c = tx + 16 * j;
                const int64_t at = (int64_t)h * a.n_q + t.q0 + qt * kT + c;
                const float2 st = c < left ? attn_stats(a, at) : make_float2(0.f, 0.f);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const bool in = c < left && t.first + ty + 16 * i < t.lk;
                    const float pr = in ? exp2f(s[i][j] * a.scale_log2 + st.x) : 0.f;
                    sP[(ty + 16 * i) * kPP + c] = pr;
                    sS[(ty + 16 * i) * kPP + c] = in ? pr * (dp[i][j] + st.y) : 0.f;
                }
            }
            __syncthreads();
            product_nn<NC>(sP, sG, a.d, ty, tx, dv);
            product_nn<NC>(sS, sQ, a.d, ty, tx, dk);
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = t.first + ty + 16 * i;
        if (r >= t.krows) continue;  // rows past the valid keys get zeros
        const int64_t row = t.k0 + r;
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            const int col = tx * 4 + 64 * c;
            if (col >= a.d) continue;
            const float4 vk = times(dk[i][c], a.scale), vv = dv[i][c];
            if (a.splits > 1) {
                const size_t at = (((size_t)t.part * a.n_k + row) * a.hk + hk) * a.d + col;
                put4(a.part + at, vk);
                put4(part_dv + at, vv);
            } else {
                put4(head_row<float>(a.gk, row, hk) + col, vk);
                put4(head_row<float>(a.gv, row, hk) + col, vv);
            }
        }
    }
}

size_t smem_bytes(int d, int tiles, int scores) {
    return ((size_t)tiles * kT * (d + 4) + (size_t)scores * kT * kPP) * sizeof(float);
}

template <typename K>
bool allow_smem(K kernel, size_t bytes) {
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes) == cudaSuccess;
}

template <int NC>
int fwd(const AttnArgs& a, cudaStream_t s) {
    const size_t smem = smem_bytes(a.d, 3, 1);
    if (!allow_smem(k_attn_fwd<NC>, smem)) return VG_ERR_CUDA;
    const dim3 grid((unsigned)(attn_max_tiles(a.n_q, a.batch, 1, kT) * a.splits), a.hq);
    k_attn_fwd<NC><<<grid, kThreads, smem, s>>>(a);
    return cudaPeekAtLastError() == cudaSuccess ? VG_OK : VG_ERR_CUDA;
}
template <int NC>
int dq(const AttnArgs& a, cudaStream_t s) {
    const size_t smem = smem_bytes(a.d, 4, 1);
    if (!allow_smem(k_attn_dq<NC>, smem)) return VG_ERR_CUDA;
    const dim3 grid((unsigned)(attn_max_tiles(a.n_q, a.batch, 1, kT) * a.splits), a.hq);
    k_attn_dq<NC><<<grid, kThreads, smem, s>>>(a);
    return cudaPeekAtLastError() == cudaSuccess ? VG_OK : VG_ERR_CUDA;
}
template <int NC>
int dkv(const AttnArgs& a, float* part_dv, cudaStream_t s) {
    const size_t smem = smem_bytes(a.d, 4, 2);
    if (!allow_smem(k_attn_dkv<NC>, smem)) return VG_ERR_CUDA;
    const dim3 grid((unsigned)(attn_max_tiles(a.n_k, a.batch, 1, kT) * a.splits), a.hk);
    k_attn_dkv<NC><<<grid, kThreads, smem, s>>>(a, part_dv);
    return cudaPeekAtLastError() == cudaSuccess ? VG_OK : VG_ERR_CUDA;
}

}  // namespace

int attn_simt_fwd(const AttnArgs& a, cudaStream_t s) { return a.d <= 64 ? fwd<1>(a, s) : fwd<2>(a, s); }
int attn_simt_dq(const AttnArgs& a, cudaStream_t s) { return a.d <= 64 ? dq<1>(a, s) : dq<2>(a, s); }
int attn_simt_dkv(const AttnArgs& a, float* part_dv, cudaStream_t s) {
    return a.d <= 64 ? dkv<1>(a, part_dv, s) : dkv<2>(a, part_dv, s);
}

}  // namespace vg
