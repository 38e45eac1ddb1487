// Dropout into the residual stream: out = residual + (keep ? x / (1 - p) : 0), and its gradient
// (the same without a residual).  The mask is w >= round(p 2^32) for the words w of a
// counter-based generator, Philox 4x32 with ten rounds, from Salmon, Moraes, Dror and Shaw,
// "Parallel random numbers: as easy as 1, 2, 3" (SC 2011): a word depends on the element's index
// and the call's key alone, so nothing is stored and the backward pass computes it again.
//
// A dropped element is zero whatever x holds (a selection, not a product).  One group of four
// words serves four consecutive elements; a thread takes 16-byte vectors, two groups for 16-bit
// types.
#include <cmath>

#include "common.cuh"
#include "internal.h"

namespace vg {

namespace {

constexpr int kThreads = 256;
constexpr int kUnroll = 4;  // vectors of a thread in flight

struct DropArgs {
    const void* x;
    const void* residual;  // or null
    void* out;
    const uint64_t* rng;   // [2] seed, step (device)
    int64_t n;
    uint32_t call, threshold;
    float scale;
};

// Words of elements 4 g .. 4 g + 3.
__device__ __forceinline__ uint4 philox(uint64_t g, uint32_t step, uint32_t call, uint32_t k0, uint32_t k1) {
    uint32_t c0 = (uint32_t)g, c1 = (uint32_t)(g >> 32), c2 = step, c3 = call;
#pragma unroll
    for (int i = 0; i < 10; ++i) {
        const uint64_t p = (uint64_t)0xD2511F53u * c0, q = (uint64_t)0xCD9E8D57u * c2;
        c0 = (uint32_t)(q >> 32) ^ c1 ^ k0;
        c1 = (uint32_t)q;
        c2 = (uint32_t)(p >> 32) ^ c3 ^ k1;
        c3 = (uint32_t)p;
        k0 += 0x9E3779B9u;
        k1 += 0xBB67AE85u;
    }
    return make_uint4(c0, c1, c2, c3);
}

__device__ __forceinline__ float dropped(uint32_t w, const DropArgs& a, float x) {
    return w >= a.threshold ? x * a.scale : 0.f;
}

template <typename T, bool RES>
__global__ void __launch_bounds__(kThreads) k_dropout_vec(const DropArgs a) {
    constexpr int W = 16 / (int)sizeof(T);
    const uint64_t seed = a.rng[0];
    const uint32_t step = (uint32_t)a.rng[1], k0 = (uint32_t)seed, k1 = (uint32_t)(seed >> 32);
    const uint4* x = static_cast<const uint4*>(a.x);
    const uint4* r = static_cast<const uint4*>(a.residual);
    uint4* out = static_cast<uint4*>(a.out);
    const int64_t vectors = a.n / W;
    const int64_t stride = (int64_t)gridDim.x * kThreads * kUnroll;
    for (int64_t v0 = ((int64_t)blockIdx.x * kUnroll) * kThreads + threadIdx.x; v0 < vectors; v0 += stride) {
        uint4 xv[kUnroll], rv[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int64_t v = v0 + u * kThreads;
            if (v < vectors) {
                xv[u] = x[v];
                if constexpr (RES) rv[u] = r[v];
            }
        }
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int64_t v = v0 + u * kThreads;
            if (v >= vectors) break;
            uint4 o;
            const T* xe = reinterpret_cast<const T*>(&xv[u]);
            const T* re = reinterpret_cast<const T*>(&rv[u]);
            T* oe = reinterpret_cast<T*>(&o);
#pragma unroll
            for (int h = 0; h < W / 4; ++h) {
                const uint4 w = philox((uint64_t)v * (W / 4) + h, step, a.call, k0, k1);
                const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    float y = dropped(ws[j], a, to_f32<T>(xe[4 * h + j]));
                    if constexpr (RES) y += to_f32<T>(re[4 * h + j]);
                    oe[4 * h + j] = from_f32<T>(y);
                }
            }
            out[v] = o;
        }
    }
    // the elements behind the last whole vector: one thread each
    const int64_t i = vectors * W + threadIdx.x;
    if (blockIdx.x == 0 && i < a.n) {
        const uint4 w = philox((uint64_t)i / 4, step, a.call, k0, k1);
        const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
        float y = dropped(ws[i & 3], a, to_f32<T>(static_cast<const T*>(a.x)[i]));
        if constexpr (RES) y += to_f32<T>(static_cast<const T*>(a.residual)[i]);
        static_cast<T*>(a.out)[i] = from_f32<T>(y);
    }
}

// Pointers that are not aligned to 16 bytes: a thread takes a group of four elements.
template <typename T, bool RES>
__global__ void __launch_bounds__(kThreads) k_dropout_any(const DropArgs a) {
    const uint64_t seed = a.rng[0];
    const uint32_t step = (uint32_t)a.rng[1], k0 = (uint32_t)seed, k1 = (uint32_t)(seed >> 32);
    const int64_t groups = (a.n + 3) / 4;
    for (int64_t g = (int64_t)blockIdx.x * kThreads + threadIdx.x; g < groups; g += (int64_t)gridDim.x * kThreads) {
        const uint4 w = philox((uint64_t)g, step, a.call, k0, k1);
        const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int64_t i = 4 * g + j;
            if (i >= a.n) break;
            float y = dropped(ws[j], a, to_f32<T>(static_cast<const T*>(a.x)[i]));
            if constexpr (RES) y += to_f32<T>(static_cast<const T*>(a.residual)[i]);
            static_cast<T*>(a.out)[i] = from_f32<T>(y);
        }
    }
}

template <typename T>
int launch(const DropArgs& a, int sms, cudaStream_t s) {
    const uintptr_t bits = reinterpret_cast<uintptr_t>(a.x) | reinterpret_cast<uintptr_t>(a.residual) |
                           reinterpret_cast<uintptr_t>(a.out);
    const bool wide = (bits & 15) == 0;
    const int64_t per = wide ? (int64_t)kThreads * kUnroll * (16 / (int)sizeof(T)) : (int64_t)kThreads * 4;
    const int grid = (int)std::max<int64_t>(1, std::min<int64_t>((a.n + per - 1) / per, (int64_t)sms * 6));
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
