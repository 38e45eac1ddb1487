// Cross attention: the plan of a call (how rows are packed, how long axes are cut,
// where the scratch lies), the row sums that the backward pass starts from, and the
// joins of split work.
#include <type_traits>

#include "attn.cuh"

namespace vg {

namespace {

constexpr int kThreads = 256;

// 8 consecutive elements of a head's row, 16-byte aligned.
template <typename T>
__device__ __forceinline__ void load8(const T* p, float (&x)[8]) {
    if constexpr (sizeof(T) == 4) {
        const float4 u = *reinterpret_cast<const float4*>(p), v = *reinterpret_cast<const float4*>(p + 4);
        x[0] = u.x; x[1] = u.y; x[2] = u.z; x[3] = u.w;
        x[4] = v.x; x[5] = v.y; x[6] = v.z; x[7] = v.w;
    } else {
        const uint4 u = *reinterpret_cast<const uint4*>(p);
        const T* e = reinterpret_cast<const T*>(&u);
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = to_f32<T>(e[j]);
    }
}

// The sample that holds row j.
__device__ __forceinline__ int sample_of(const AttnArgs& a, const int32_t* off, int64_t j) {
    int lo = 0, hi = a.batch;  // the last sample that does not start past j
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (off[mid] <= j) lo = mid;
        else hi = mid;
    }
    return lo;
}

// Rows of the other axis that the results of query row (kKeys: key row) j are sums over: its sample's valid keys
// (kKeys: its packed query rows).
template <bool kKeys>
__device__ __forceinline__ int64_t summed_rows(const AttnArgs& a, int64_t j) {
    const int b = sample_of(a, kKeys ? a.k_off : a.q_off, j);
    if (kKeys) return (int64_t)(a.q_off[b + 1] - a.q_off[b]) * a.gp;
    return a.k_len ? a.k_len[b] : a.k_off[b + 1] - a.k_off[b];
}

// The largest norm of each sample's rows into dst[2 * sample], as the bits of an fp32 value (of values that are not
// negative the bits have the same order, so the result does not depend on the order of arrival).  A group of lanes
// gives its rows in rising order; rows that are not finite, or not valid, do not count.
struct SampleMax {
    uint32_t* dst;
    const int32_t* off;
    const int32_t* len;  // valid rows of each sample, or null
    int b = 0;
    int64_t end = 0, live = 0;  // of sample b: the row past its last one, past its last valid one
    float big = 0.f;            // squared

    __device__ __forceinline__ void add(const AttnArgs& a, int64_t i, bool writes, float sq) {
        if (i >= end) {
            if (writes) flush();
            big = 0.f;
            b = sample_of(a, off, i);
            end = off[b + 1];
            live = len ? off[b] + len[b] : end;
        }
        if (sq < INFINITY && i < live) big = fmaxf(big, sq);
    }
    __device__ __forceinline__ void flush() const {
        if (big > 0.f) atomicMax(dst + 2 * b, __float_as_uint(sqrtf(big)));
    }
    // By the whole block, at its end: one atomic for all of it if it saw one sample last.
    __device__ __forceinline__ void finish(bool writes) const {
        __shared__ uint32_t s_max[kThreads / 32];
        __shared__ int s_b[kThreads / 32];
        int same;
        __match_all_sync(0xffffffffu, b, &same);
        if (!same && writes) flush();
        const uint32_t v = __reduce_max_sync(0xffffffffu, same ? __float_as_uint(sqrtf(big)) : 0u);
        if ((threadIdx.x & 31) == 0) s_max[threadIdx.x >> 5] = v, s_b[threadIdx.x >> 5] = b;
        __syncthreads();
        if (threadIdx.x > 0) return;
        for (int i = 0; i < kThreads / 32; ++i) {
            uint32_t m = s_max[i];
            while (i + 1 < kThreads / 32 && s_b[i + 1] == s_b[i]) m = max(m, s_max[++i]);
            if (m > 0) atomicMax(dst + 2 * s_b[i], m);
        }
    }
};

// fp16: the largest norm of each sample's valid rows of V, which with that of dO's rows bounds dP.  Rows [first, end)
// of (key, head).
template <typename T>
__device__ __forceinline__ void value_bounds(const AttnArgs& a, int lanes, int64_t first, int64_t end) {
    const int lane = threadIdx.x & (lanes - 1), groups = kThreads / lanes;
    SampleMax most{a.bound + 1, a.k_off, a.k_len};
    for (int64_t r0 = first; r0 < end; r0 += groups) {  // the same trips for the whole block
        const int64_t r = r0 + threadIdx.x / lanes, j = r / a.hk;
        float sq = 0.f;
        if (r < end && lane * 8 < a.d) {
            float v[8];
            load8<T>(head_row<const T>(a.v, j, (int)(r - j * a.hk)) + lane * 8, v);
#pragma unroll
            for (int i = 0; i < 8; ++i) sq = fmaf(v[i], v[i], sq);
        }
        for (int o = 1; o < lanes; o <<= 1) sq += __shfl_xor_sync(0xffffffffu, sq, o);
        if (r < end) most.add(a, j, lane == 0, sq);
    }
    most.finish(lane == 0);
}

// Blocks of a kernel over rows, each of which takes `per` rows in a row.
struct Rows {
    int blocks = 0;
    int64_t per = 0;
};

// stats[packed row] = -lse * log2 e (+ 15 in fp16: the weights' exponent), -sum_d dO O: a group
// of 1..16 lanes per row, 16-byte loads; reads O and dO once, bound by memory.  fp16: also |dO row|,
// and the largest norms of a sample's rows of dO and of its valid rows of V (the blocks behind the first).
template <typename T>
__global__ void __launch_bounds__(kThreads) k_attn_stats(const AttnArgs a, int lanes, Rows queries, Rows values) {
    constexpr bool kHalf = sizeof(T) == 2 && !std::is_same<T, __nv_bfloat16>::value;
    if constexpr (kHalf) {
        if ((int)blockIdx.x >= queries.blocks) {
            const int64_t first = (int64_t)(blockIdx.x - queries.blocks) * values.per;
            value_bounds<T>(a, lanes, first, min(first + values.per, a.n_k * a.hk));
            return;
        }
    }
    const int lane = threadIdx.x & (lanes - 1), groups = kThreads / lanes;
    const int64_t rows = a.n_q * a.hq;
    const int64_t first = (int64_t)blockIdx.x * queries.per, end = min(first + queries.per, rows);
    SampleMax most{a.bound, a.q_off, nullptr};
    // row r = (i, h), carried along without a division
    int64_t r = first + threadIdx.x / lanes, i = r / a.hq;
    int h = (int)(r - i * a.hq);
    const int di = groups / a.hq, dh = groups - di * a.hq;
    for (int64_t r0 = first; r0 < end; r0 += groups, r += groups) {  // the same trips for the whole block
        float sum = 0.f, sq = 0.f;
        if (r < end && lane * 8 < a.d) {
            float o[8], g[8];
            load8<T>(head_row<const T>(a.o, i, h) + lane * 8, o);
            load8<T>(head_row<const T>(a.go, i, h) + lane * 8, g);
#pragma unroll
            for (int j = 0; j < 8; ++j) sum = fmaf(o[j], g[j], sum), sq = fmaf(g[j], g[j], sq);
        }
        for (int o = 1; o < lanes; o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        if constexpr (kHalf) {
            for (int o = 1; o < lanes; o <<= 1) sq += __shfl_xor_sync(0xffffffffu, sq, o);
            if (r < end) most.add(a, i, lane == 0, sq);
        }
        if (r < end && lane == 0) {
            float* st = a.stats + (((int64_t)(h >> a.gp_log2) * a.n_q + i) << a.gp_log2) + (h & (a.gp - 1));
            st[0] = fmaf(a.lse[(int64_t)h * a.n_q + i], -1.4426950408889634f, kHalf ? kHalfLift : 0.f);
            st[rows] = -sum;
            if (kHalf) st[2 * rows] = sqrtf(sq);
        }
        i += di;
        if ((h += dh) >= a.hq) h -= a.hq, ++i;
    }
    if constexpr (kHalf) most.finish(lane == 0);
}

// Four consecutive elements, 8 or 16 bytes.
template <typename T>
__device__ __forceinline__ void put4(T* p, float4 v) {
    if constexpr (sizeof(T) == 4) {
        *reinterpret_cast<float4*>(p) = v;
    } else {
        T e[4] = {from_f32<T>(v.x), from_f32<T>(v.y), from_f32<T>(v.z), from_f32<T>(v.w)};
        *reinterpret_cast<uint2*>(p) = *reinterpret_cast<const uint2*>(e);
    }
}

// The parts' outputs, each normalised by its own sum, weighed by exp(lse_s - max lse).  Every part counts, with a
// weight of zero too: 0 x its output is 0, or NaN where it holds something that is not finite, as in a call that is not
// cut.  (A part whose scores are all -inf has no sum to be normalised by and comes as it is.)  The maximum leaves NaN
// out, so a sum that is NaN says that something is.  A thread has four columns of a row, and with LANES > 1 every
// LANES-th part: a few rows over many parts (one token's) would otherwise be a long chain of loads in few threads (32
// rows, 64 parts: 14 us with one lane, 5 us with eight).
template <typename T, int LANES>
__global__ void __launch_bounds__(kThreads) k_attn_join_out(const AttnArgs a) {
    constexpr int kItems = kThreads / LANES;  // pieces of rows of a block
    __shared__ float s_top[LANES][kItems], s_sum[LANES][kItems];
    __shared__ float4 s_acc[LANES][kItems];
    if (!attn_offsets_ok(a)) return;
    const int q4 = a.d / 4, item = threadIdx.x % kItems, lane = threadIdx.x / kItems;
    const int64_t e = (int64_t)blockIdx.x * kItems + item;
    const bool mine = e < a.n_q * a.hq * q4;
    const int64_t r = mine ? e / q4 : 0;
    const int c = mine ? (int)(e - r * q4) * 4 : 0;
    const int64_t i = r / a.hq;
    const int h = (int)(r - i * a.hq);
    const float* lse = a.part_lse + (int64_t)h * a.n_q + i;
    const int64_t lstep = (int64_t)a.hq * a.n_q;
    const int64_t keys = mine ? summed_rows<false>(a, i) : 0;
    const int parts = mine ? attn_parts(a, keys) : 0;
    float top = -INFINITY;
#pragma unroll 4
    for (int s = lane; s < parts; s += LANES) top = fmaxf(top, lse[s * lstep]);
    const float base = top == -INFINITY ? 0.f : top;
    const float* src = a.part + r * a.d + c;
    const int64_t step = a.n_q * a.hq * a.d;
    float sum = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int s = lane; s < parts; s += LANES) {
        const float w = expf(lse[s * lstep] - base);
        const float4 v = *reinterpret_cast<const float4*>(src + s * step);
        sum += w;
        acc.x = fmaf(w, v.x, acc.x); acc.y = fmaf(w, v.y, acc.y);
        acc.z = fmaf(w, v.z, acc.z); acc.w = fmaf(w, v.w, acc.w);
    }
    if constexpr (LANES > 1) {  // the lanes' sums likewise, in their order
        s_top[lane][item] = top;
        s_sum[lane][item] = sum;
        s_acc[lane][item] = acc;
        __syncthreads();
        if (lane > 0) return;
        for (int l = 1; l < LANES; ++l) top = fmaxf(top, s_top[l][item]);
        sum = 0.f;
        acc = make_float4(0.f, 0.f, 0.f, 0.f);
        const float all = top == -INFINITY ? 0.f : top;
        for (int l = 0; l < LANES; ++l) {
            const float w = expf(s_top[l][item] - all);
            const float4 v = s_acc[l][item];
            sum = fmaf(w, s_sum[l][item], sum);
            acc.x = fmaf(w, v.x, acc.x); acc.y = fmaf(w, v.y, acc.y);
            acc.z = fmaf(w, v.z, acc.z); acc.w = fmaf(w, v.w, acc.w);
        }
    }
    if (!mine) return;
    const float inv = keys > 0 ? 1.f / sum : 0.f;  // no keys: zero; only keys of weight zero: NaN
    put4(head_row<T>(a.o, i, h) + c, make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv));
    if (c == 0 && a.lse) a.lse[(int64_t)h * a.n_q + i] = (top == -INFINITY ? 0.f : top) + logf(sum);
}

// The parts' gradients, added in their order; blockIdx.y: which of two tensors of one shape.
struct Join { const float* part; vg_heads dst; };
template <typename T, bool kKeys>
__global__ void __launch_bounds__(kThreads) k_attn_join_sum(const AttnArgs a, Join one, Join two, int lanes_log2) {
    if (!attn_offsets_ok(a)) return;
    const Join& j = blockIdx.y == 0 ? one : two;
    const int c = (threadIdx.x & ((1 << lanes_log2) - 1)) * 4;  // 2^lanes_log2 threads to a row
    const int64_t rows = kKeys ? a.n_k : a.n_q;
    const int heads = kKeys ? a.hk : a.hq;
    const int64_t r = (int64_t)blockIdx.x * (kThreads >> lanes_log2) + (threadIdx.x >> lanes_log2);
    if (r >= rows * heads || c >= a.d) return;
    const int64_t i = r < (int64_t(1) << 31) ? (uint32_t)r / (uint32_t)heads : r / heads;
    const int parts = attn_parts(a, summed_rows<kKeys>(a, i));
    const float* src = j.part + r * a.d + c;
    const int64_t step = rows * heads * a.d;
    float4 acc = *reinterpret_cast<const float4*>(src);
#pragma unroll 4
    for (int s = 1; s < parts; ++s) {
        const float4 v = *reinterpret_cast<const float4*>(src + s * step);
        acc.x += v.x; acc.y += v.y; acc.z += v.z; acc.w += v.w;
    }
    put4(head_row<T>(j.dst, i, (int)(r - i * heads)) + c, acc);
}

int launched() { return cudaPeekAtLastError() == cudaSuccess ? VG_OK : VG_ERR_CUDA; }

// At most 16 blocks an SM, `step` rows or a multiple of them for each.
Rows rows_of(int64_t rows, int step, int sms) {
    if (rows == 0) return {};
    const int64_t steps = (rows + step - 1) / step, most = std::min<int64_t>(steps, (int64_t)sms * 16);
    const int64_t per = (steps + most - 1) / most * step;
    return {(int)((rows + per - 1) / per), per};
}
template <typename T>
int stats(const AttnArgs& a, int sms, cudaStream_t s) {
    int lanes = 1;
    while (lanes * 8 < a.d) lanes <<= 1;
    const Rows queries = rows_of(a.n_q * a.hq, kThreads / lanes, sms);
    const Rows values = std::is_same<T, __half>::value ? rows_of(a.n_k * a.hk, kThreads / lanes, sms) : Rows{};
    k_attn_stats<T><<<queries.blocks + values.blocks, kThreads, 0, s>>>(a, lanes, queries, values);
    return launched();
}
template <typename T>
int join_out(const AttnArgs& a, cudaStream_t s) {
    const int64_t n = a.n_q * a.hq * (a.d / 4);
    if (a.splits > 8) k_attn_join_out<T, 8><<<(unsigned)((n + kThreads / 8 - 1) / (kThreads / 8)), kThreads, 0, s>>>(a);
    else k_attn_join_out<T, 1><<<(unsigned)((n + kThreads - 1) / kThreads), kThreads, 0, s>>>(a);
    return launched();
}
template <typename T, bool kKeys>
int join_rows(const AttnArgs& a, const Join& one, const Join& two, int count, cudaStream_t s) {
    int log2 = 0;
    while ((4 << log2) < a.d) ++log2;
    const int64_t rows = kKeys ? a.n_k * a.hk : a.n_q * a.hq, per = kThreads >> log2;
    const dim3 grid((unsigned)((rows + per - 1) / per), count);
    k_attn_join_sum<T, kKeys><<<grid, kThreads, 0, s>>>(a, one, two, log2);
    return launched();
}
template <typename T>
int join_queries(const AttnArgs& a, cudaStream_t s) {
    const Join q{a.part, a.gq};
    return join_rows<T, false>(a, q, q, 1, s);
}
template <typename T>
int join_keys(const AttnArgs& a, const float* part_dv, cudaStream_t s) {
    return join_rows<T, true>(a, Join{a.part, a.gk}, Join{part_dv, a.gv}, 2, s);
}

#define VG_BY_TYPE(f, ...)                                \
    (dtype == VG_F32 ? f<float>(__VA_ARGS__)              \
     : dtype == VG_F16 ? f<__half>(__VA_ARGS__) : f<__nv_bfloat16>(__VA_ARGS__))

// How to cut an axis of `tiles` tiles in all (every sample's together) when there are
// `units` independent tiles of work along the other one, in `batch` samples, and `slots` run at a time.
// Parts have one size for all samples, so that a call with one long sample and short ones is even
// too; a part has at least `least` tiles.  Not cut when the units fill the slots.  With `fill` it is cut then too where
// that evens out the last wave by more than the parts' fp32 results and their join cost (some 20 us): in calls of 256
// tiles (over 100 us) and more per slot.  dK and dV of 5,000 queries over 2,740 keys, 16 heads: 75 us uncut, 82 + 19 in
// parts; of 25,179 over 5,001 keys: 290 and 241 + 21; of 100,003 over 2,740: 1280 and 1087 + 21.
struct Cut { int parts, per; };
Cut cut_axis(int64_t units, int64_t tiles, int batch, int slots, int least, bool fill) {
    if (units <= 0 || tiles <= 0) return {1, 0};
    int64_t want = slots / units;
    if (fill && units * ((tiles + batch - 1) / batch) >= 256 * (int64_t)slots) {
        double best = 0.0;
        for (int64_t s = std::max<int64_t>(1, want), end = std::max<int64_t>(8, s); s <= end; ++s) {
            const int64_t n = units * s, waves = (n + slots - 1) / slots;
            const double full = (double)n / (double)(waves * slots);
            if (full > best + 0.03) want = s, best = full;
            if (best > 0.93) break;
        }
    }
    if (want <= 1) return {1, 0};
    // `want` parts of a sample of average length; a sample that holds all rows has batch times as many, of
    // which the scratch takes up to four times the average
    const int64_t most = std::min<int64_t>(want * std::min(batch, 4), 1024);
    const int64_t even = (tiles + want * batch - 1) / (want * batch);
    const int64_t per = std::max<int64_t>({least, even, (tiles + most - 1) / most});
    const int64_t parts = (tiles + per - 1) / per;
    return parts <= 1 ? Cut{1, 0} : Cut{(int)parts, (int)per};
}

}  // namespace

int attn_plan(const AttnShape& c, AttnPlan* P) {
    if (c.n_q < 0 || c.n_k < 0 || c.n_q >= (int64_t(1) << 31) || c.n_k >= (int64_t(1) << 31)) return VG_ERR_INVALID_ARG;
    if (c.batch <= 0 || c.hq <= 0 || c.hk <= 0 || c.hq % c.hk || c.d <= 0) return VG_ERR_INVALID_ARG;
    if (c.dtype != VG_F32 && c.dtype != VG_F16 && c.dtype != VG_BF16) return VG_ERR_INVALID_ARG;
    if (c.d % 8 || c.d > 128 || c.hq > 65535) return VG_ERR_UNSUPPORTED;
    AttnPlan p;
    p.sms = plan_sms(0);
    p.tc = c.dtype != VG_F32;
    const int group = c.hq / c.hk;
    if (p.tc && group <= 16 && !(group & (group - 1)) && c.n_q * group < (int64_t(1) << 31)) p.gp = group;
    const auto tiles = [](int64_t rows, int tile) { return (rows + tile - 1) / tile; };
    const int64_t qt = attn_max_tiles(c.n_q, c.batch, 1, 64), kt = attn_max_tiles(c.n_k, c.batch, 1, 64);
    Cut f, q, k;
    if (p.tc) {
        const int sets = c.hq / p.gp;
        // Forward, two row tiles a block against one, where that leaves no SM without a block.  d = 64, 16 heads over
        // 2,740 keys: 30.7 us against 31.2 with 2,500 queries, 46.0 and 47.5 with 5,000, 71.6 and 75.5 with 10,000,
        // 132 and 142 with 25,179 over 5,001 keys, 571 and 635 with 100,003.  d = 128, where one tile leaves room for
        // one block all the same: 40.0 against 51.7 with 2,500, 60.8 and 80.6 with 5,000.  Below, with 2 queries over
        // 319,057 keys (d = 64), 135 and 97.
        p.nq = attn_max_tiles(c.n_q, c.batch, p.gp, 256) * sets >= p.sms ? 2 : 1;
        const int64_t units = attn_max_tiles(c.n_q, c.batch, p.gp, 128 * p.nq) * sets;
        const int slots = p.nq == 1 && c.d <= 64 ? 2 * p.sms : p.sms;
        f = cut_axis(units, tiles(c.n_k, 128), c.batch, slots, 4, false);
        q = cut_axis(attn_max_tiles(c.n_q, c.batch, p.gp, 128) * sets, tiles(c.n_k, 128), c.batch, p.sms, 4, false);
        k = cut_axis(attn_max_tiles(c.n_k, c.batch, 1, 128) * c.hk, tiles(c.n_q * p.gp, 64), c.batch, p.sms, 4, true);
    } else {
        // four parts per SM, down to two tiles: 2,013 queries over 1,001 keys took 129 us in dK, dV and 50 forward
        // with parts of four tiles, 67 and 42 with two
        f = q = cut_axis(qt * c.hq, tiles(c.n_k, 64), c.batch, 4 * p.sms, 2, false);
        k = cut_axis(kt * c.hk, tiles(c.n_q, 64), c.batch, 4 * p.sms, 2, false);
    }
    p.s_fwd = f.parts;
    p.per_fwd = f.per;
    p.s_dq = q.parts;
    p.per_dq = q.per;
    p.s_dkv = k.parts;
    p.per_dkv = k.per;
    const size_t vq = (size_t)c.n_q * c.hq, vk = (size_t)c.n_k * c.hk;
    size_t fwd = 0, bwd = 0;
    if (p.s_fwd > 1) {
        fwd = align_up(p.s_fwd * vq * c.d * 4, 256);
        p.off_lse = 256 + fwd;
        fwd += align_up(p.s_fwd * vq * 4, 256);
    }
    if (c.backward) {
        size_t o = align_up(vq * sizeof(float) * (c.dtype == VG_F16 ? 3 : 2), 256);
        p.off_bound = 256 + o;
        if (c.dtype == VG_F16) o += align_up((size_t)c.batch * 8, 256);
        p.off_dq = 256 + o;
        if (p.s_dq > 1) o += align_up(p.s_dq * vq * c.d * 4, 256);
        p.off_dk = 256 + o;
        if (p.s_dkv > 1) o += align_up(p.s_dkv * vk * c.d * 4, 256);
        p.off_dv = 256 + o;
        if (p.s_dkv > 1) o += align_up(p.s_dkv * vk * c.d * 4, 256);
        bwd = o;
    }
    p.total = 256 + std::max(fwd, bwd);
    *P = p;
    return VG_OK;
}

int attn_fwd(AttnArgs a, const AttnPlan& p, int dtype, char* ws, cudaStream_t s) {
    if (a.n_q == 0) return VG_OK;
    a.gp = p.gp;
    a.gp_log2 = __builtin_ctz((unsigned)p.gp);
    a.err = reinterpret_cast<uint32_t*>(ws);
    a.splits = p.s_fwd;
    a.per_part = p.per_fwd;
    a.tile = p.tc ? 128 : 64;
    a.part = reinterpret_cast<float*>(ws + 256);
    a.part_lse = reinterpret_cast<float*>(ws + p.off_lse);
    const int st = p.tc ? attn_tc_fwd(a, dtype, p.nq, p.sms, s) : attn_simt_fwd(a, s);
    if (st != VG_OK || a.splits == 1) return st;
    return VG_BY_TYPE(join_out, a, s);
}

int attn_bwd(AttnArgs a, const AttnPlan& p, int dtype, char* ws, cudaStream_t s) {
    a.gp = p.gp;
    a.gp_log2 = __builtin_ctz((unsigned)p.gp);
    a.err = reinterpret_cast<uint32_t*>(ws);
    a.stats = reinterpret_cast<float*>(ws + 256);
    int st;
    a.bound = reinterpret_cast<uint32_t*>(ws + p.off_bound);
    if (dtype == VG_F16 && cudaMemsetAsync(a.bound, 0, (size_t)a.batch * 8, s) != cudaSuccess) return VG_ERR_CUDA;
    if (a.n_q > 0) {
        if ((st = VG_BY_TYPE(stats, a, p.sms, s)) != VG_OK) return st;
        a.splits = p.s_dq;
        a.per_part = p.per_dq;
        a.tile = p.tc ? 128 : 64;
        a.part = reinterpret_cast<float*>(ws + p.off_dq);
        st = p.tc ? attn_tc_dq(a, dtype, p.sms, s) : attn_simt_dq(a, s);
        if (st != VG_OK) return st;
        if (a.splits > 1 && (st = VG_BY_TYPE(join_queries, a, s)) != VG_OK) return st;
    }
    if (a.n_k > 0) {
        a.splits = p.s_dkv;
        a.per_part = p.per_dkv;
        a.tile = 64;
        a.part = reinterpret_cast<float*>(ws + p.off_dk);
        float* part_dv = reinterpret_cast<float*>(ws + p.off_dv);
        st = p.tc ? attn_tc_dkv(a, part_dv, dtype, p.sms, s) : attn_simt_dkv(a, part_dv, s);
        if (st != VG_OK) return st;
        if (a.splits > 1 && (st = VG_BY_TYPE(join_keys, a, part_dv, s)) != VG_OK) return st;
    }
    return VG_OK;
}

}  // namespace vg
