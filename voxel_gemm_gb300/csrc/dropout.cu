// Dropout into the residual stream: out = residual + (keep ? x / (1 - p) : 0), and its gradient
// (the same without a residual).  The mask is w >= round(p 2^32) for the words w of a
// counter-based generator, Philox 4x32 with ten rounds, from Salmon, Moraes, Dror and Shaw,
// "Parallel random numbers: as easy as 1, 2, 3" (SC 2011): a word depends on the element's index
// and the call's key alone, so nothing is stored and the backward pass computes it again.
//
// A dropped element is zero whatever x holds (a selection, not a product).  One group of four
// words serves four consecutive elements; a thread takes 16-byte vectors, two groups for 16-bit
// types.  Two thirds of the work are the generator's 32-bit products, so what all groups of
// a call have in common is done once: the keys, and half of the first two rounds, which see only the
// call and the step.
//
// 308 M elements in bf16 (GB300): 270 us with a residual (6.8 TB/s), 225 without (5.5 TB/s; the
// generator's products take as long as memory would).  A grid of 64 blocks per SM, a few turns each, was
// best: 8 blocks 564 us for both, one block for every two vectors 552 (keys made anew each time), 64 495.
#include <cmath>

#include "common.cuh"
#include "internal.h"
#include "tc_ptx.cuh"

namespace vg {

namespace {

using namespace ptx;

constexpr int kThreads = 256;
constexpr int kUnroll = 2;  // vectors of a thread in flight
constexpr int kBlocksPerSm = 64;
constexpr int kRounds = 10;
constexpr uint32_t kM0 = 0xD2511F53u, kM1 = 0xCD9E8D57u;

struct DropArgs {
    const void* x;
    const void* residual;  // or null
    void* out;
    const uint64_t* rng;   // [2] seed, step (device)
    int64_t n;
    uint32_t call, threshold;
    float scale;
};

// Words of elements 4 g .. 4 g + 3, for groups g below 2^32.
struct Philox {
    uint32_t k0[kRounds], k1[kRounds];
    // Of the counters (g, 0, step, call) the first round's second product, and of that the second round's
    // first, are the same for every g.
    uint32_t c1, c3, p_hi, p_lo;

    __device__ __forceinline__ Philox(uint64_t seed, uint32_t step, uint32_t call) {
#pragma unroll
        for (int i = 0; i < kRounds; ++i) {
            k0[i] = (uint32_t)seed + i * 0x9E3779B9u;
            k1[i] = (uint32_t)(seed >> 32) + i * 0xBB67AE85u;
        }
        const uint64_t q = (uint64_t)kM1 * step;
        const uint64_t p = (uint64_t)kM0 * ((uint32_t)(q >> 32) ^ k0[0]);  // the groups' high words are 0
        c1 = (uint32_t)q ^ k0[1];
        c3 = call ^ k1[0];
        p_hi = (uint32_t)(p >> 32) ^ k1[1];
        p_lo = (uint32_t)p;
    }
    __device__ __forceinline__ uint4 words(uint32_t g) const {
        const uint64_t p1 = (uint64_t)kM0 * g;
        const uint64_t q2 = (uint64_t)kM1 * ((uint32_t)(p1 >> 32) ^ c3);
        uint32_t a = (uint32_t)(q2 >> 32) ^ c1, b = (uint32_t)q2, c = p_hi ^ (uint32_t)p1, d = p_lo;
#pragma unroll
        for (int i = 2; i < kRounds; ++i) {
            const uint64_t p = (uint64_t)kM0 * a, q = (uint64_t)kM1 * c;
            a = (uint32_t)(q >> 32) ^ b ^ k0[i];
            b = (uint32_t)q;
            c = (uint32_t)(p >> 32) ^ d ^ k1[i];
            d = (uint32_t)p;
        }
        return make_uint4(a, b, c, d);
    }
};
// The same for any group, round by round.
__device__ __forceinline__ uint4 philox(uint64_t g, uint32_t step, uint32_t call, uint64_t seed) {
    uint32_t a = (uint32_t)g, b = (uint32_t)(g >> 32), c = step, d = call;
    uint32_t k0 = (uint32_t)seed, k1 = (uint32_t)(seed >> 32);
#pragma unroll
    for (int i = 0; i < kRounds; ++i) {
        const uint64_t p = (uint64_t)kM0 * a, q = (uint64_t)kM1 * c;
        a = (uint32_t)(q >> 32) ^ b ^ k0;
        b = (uint32_t)q;
        c = (uint32_t)(p >> 32) ^ d ^ k1;
        d = (uint32_t)p;
        k0 += 0x9E3779B9u;
        k1 += 0xBB67AE85u;
    }
    return make_uint4(a, b, c, d);
}

// One element: its sum with the residual is rounded once to fp32, and once to T.
template <typename T, bool RES>
__device__ __forceinline__ void one(const DropArgs& a, int64_t i, uint32_t w) {
    const float x = w >= a.threshold ? to_f32<T>(static_cast<const T*>(a.x)[i]) : 0.f;
    const float y = RES ? fmaf(x, a.scale, to_f32<T>(static_cast<const T*>(a.residual)[i])) : x * a.scale;
    static_cast<T*>(a.out)[i] = from_f32<T>(y);
}

// A pair of elements.
template <bool RES>
__device__ __forceinline__ float2 both(const DropArgs& a, float2 x, float2 r, uint32_t w0, uint32_t w1) {
    x = make_float2(w0 >= a.threshold ? x.x : 0.f, w1 >= a.threshold ? x.y : 0.f);
    const float2 s = make_float2(a.scale, a.scale);
    if constexpr (RES) return fma2(x, s, r);
    return mul2(x, s);
}
template <typename T, bool RES>
__device__ __forceinline__ uint4 vector(const DropArgs& a, const Philox& gen, uint32_t v, uint4 x, uint4 r) {
    if constexpr (sizeof(T) == 4) {
        const uint4 w = gen.words(v);
        const auto f = [](uint32_t lo, uint32_t hi) { return make_float2(__uint_as_float(lo), __uint_as_float(hi)); };
        const float2 y = both<RES>(a, f(x.x, x.y), f(r.x, r.y), w.x, w.y);
        const float2 z = both<RES>(a, f(x.z, x.w), f(r.z, r.w), w.z, w.w);
        return make_uint4(__float_as_uint(y.x), __float_as_uint(y.y), __float_as_uint(z.x), __float_as_uint(z.y));
    } else {
        const uint4 w = gen.words(2 * v), u = gen.words(2 * v + 1);
        using P = Pair<T>;
        return make_uint4(P::pack(both<RES>(a, P::unpack(x.x), P::unpack(r.x), w.x, w.y)),
                          P::pack(both<RES>(a, P::unpack(x.y), P::unpack(r.y), w.z, w.w)),
                          P::pack(both<RES>(a, P::unpack(x.z), P::unpack(r.z), u.x, u.y)),
                          P::pack(both<RES>(a, P::unpack(x.w), P::unpack(r.w), u.z, u.w)));
    }
}

// Aligned pointers, fewer than 2^34 elements.
template <typename T, bool RES>
__global__ void __launch_bounds__(kThreads) k_dropout_vec(const DropArgs a) {
    constexpr int W = 16 / (int)sizeof(T);
    const Philox gen(a.rng[0], (uint32_t)a.rng[1], a.call);
    const uint4* x = static_cast<const uint4*>(a.x);
    const uint4* r = static_cast<const uint4*>(a.residual);
    uint4* out = static_cast<uint4*>(a.out);
    const int64_t vectors = a.n / W, stride = (int64_t)gridDim.x * kThreads * kUnroll;
    for (int64_t v0 = ((int64_t)blockIdx.x * kUnroll) * kThreads + threadIdx.x; v0 < vectors; v0 += stride) {
        uint4 xv[kUnroll], rv[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int64_t v = v0 + u * kThreads;
            if (v < vectors) {
                xv[u] = x[v];
                rv[u] = RES ? r[v] : make_uint4(0, 0, 0, 0);
            }
        }
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int64_t v = v0 + u * kThreads;
            if (v < vectors) out[v] = vector<T, RES>(a, gen, (uint32_t)v, xv[u], rv[u]);
        }
    }
    // the elements behind the last whole vector: one thread each
    const int64_t i = vectors * W + threadIdx.x;
    if (blockIdx.x == 0 && i < a.n) {
        const uint4 w = gen.words((uint32_t)(i / 4));
        const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
        one<T, RES>(a, i, ws[i & 3]);
    }
}

// Other calls: a thread takes a group of four elements.
template <typename T, bool RES>
__global__ void __launch_bounds__(kThreads) k_dropout_any(const DropArgs a) {
    const uint64_t seed = a.rng[0];
    const uint32_t step = (uint32_t)a.rng[1];
    const int64_t groups = (a.n + 3) / 4;
    for (int64_t g = (int64_t)blockIdx.x * kThreads + threadIdx.x; g < groups; g += (int64_t)gridDim.x * kThreads) {
        const uint4 w = philox((uint64_t)g, step, a.call, seed);
        const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (4 * g + j < a.n) one<T, RES>(a, 4 * g + j, ws[j]);
    }
}

template <typename T>
int launch(const DropArgs& a, int sms, cudaStream_t s) {
    const uintptr_t bits = reinterpret_cast<uintptr_t>(a.x) | reinterpret_cast<uintptr_t>(a.residual) |
                           reinterpret_cast<uintptr_t>(a.out);
    const bool wide = (bits & 15) == 0 && a.n < (int64_t(1) << 34);
    const int64_t per = wide ? (int64_t)kThreads * kUnroll * (16 / (int)sizeof(T)) : (int64_t)kThreads * 4;
    const int grid = (int)std::max<int64_t>(1, std::min<int64_t>((a.n + per - 1) / per, (int64_t)sms * kBlocksPerSm));
    if (wide)
        a.residual ? k_dropout_vec<T, true><<<grid, kThreads, 0, s>>>(a)
                   : k_dropout_vec<T, false><<<grid, kThreads, 0, s>>>(a);
    else
        a.residual ? k_dropout_any<T, true><<<grid, kThreads, 0, s>>>(a)
                   : k_dropout_any<T, false><<<grid, kThreads, 0, s>>>(a);
    return cudaPeekAtLastError() == cudaSuccess ? VG_OK : VG_ERR_CUDA;
}

}  // namespace

int dropout_add(int64_t n, int dtype, const void* x, const void* residual, double p, const uint64_t* rng,
                uint32_t call, void* out, int sms, cudaStream_t s) {
    DropArgs a{};
    a.x = x;
    a.residual = residual;
    a.out = out;
    a.rng = rng;
    a.n = n;
    a.call = call;
    a.threshold = (uint32_t)std::nearbyint(p * 4294967296.0);
    a.scale = (float)(1.0 / (1.0 - p));
    return dtype == VG_F32 ? launch<float>(a, sms, s)
           : dtype == VG_F16 ? launch<__half>(a, sms, s)
                             : launch<__nv_bfloat16>(a, sms, s);
}

}  // namespace vg
