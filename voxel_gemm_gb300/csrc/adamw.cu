// AdamW over many tensors in one launch, first and second moments in 32 or 8 bits.
//
//   g = grad * grad_scale;  m = m * b1 + g * (1 - b1);  v = v * b2 + (g * g) * (1 - b2)
//   p = p * (1 - lr wd) - (m / (sqrt(v) * (1 / sqrt(1 - b2^t)) + eps)) * (lr / (1 - b1^t))
//
// The factors that do not depend on the element are computed on the host in 64 bits and
// rounded once.  Every product, sum, root and quotient of the kernel is rounded once in fp32,
// in the order written (no contraction into fused multiply-adds), so the results do not
// depend on how the compiler schedules it.  (So no f32x2 instructions either: their products
// and sums came out fused.)
//
// 8-bit moments come in blocks of 256 elements that share one power-of-two scale,
// so that scaling and unscaling are exact:
//   m       sign, 4 exponent and 3 mantissa bits (a value k / 512 below 2^-6), the
//           block's largest in [2^7, 2^8): relative error 1/16 over a range of 2^13;
//   sqrt(v) unsigned, 4 exponent and 4 mantissa bits, the block's largest in
//           [2^14, 2^15), code 0 for zero alone: a small positive value becomes the
//           smallest one and not zero, since the step divides by it.  The root has
//           half of v's range in logarithms, so 4 exponent bits reach 2^-28 of the
//           block's largest v.
// A moment that is not finite is held as NaN and does not count for the scale.
//
// One pass: each 256-thread block takes a chunk of one tensor (found by bisection in
// the launch's parameter table, no device-side table and no upload), 8 elements a
// thread with 16-byte accesses; a warp holds exactly one 256-element block, so the
// 8-bit scales are warp reductions.  bf16 weights with fp32 masters (which are read in the
// weights' place): 65.0 M with fp32 moments 262 us (28 bytes each, 6.9 TB/s, bound by
// memory); 32.5 M with 8-bit moments 107 us (16 bytes each, 4.9 TB/s, bound by the rounded
// roots and quotients more than by memory).  The conversion instructions for m's codes and a
// maximum that looks for infinities only when it finds one brought the latter from 132 us.
#include "common.cuh"
#include "internal.h"

namespace vg {

namespace {

constexpr int kThreads = 256;
constexpr int kPer = 8;                      // elements of a thread
constexpr int kChunk = kThreads * kPer;      // elements of a block
constexpr int kStateBlock = VG_ADAMW_BLOCK;  // elements of a scale
static_assert(kStateBlock == 32 * kPer, "one scale per warp");

struct TensorArgs {
    void* param;
    const void* grad;
    float* master;
    void* m;
    void* v;
    float* m_scale;
    float* v_scale;
    int64_t n;
    float decay;     // 1 - lr * weight_decay
    int32_t flags;   // dtype | kVec
};
constexpr int kVec = 16;  // every pointer allows 16-byte accesses (8-byte for codes)

// The table travels in the launch's parameters: a short one for the common few
// tensors, a long one (30 KB of parameters) above.
template <int CAP>
struct Table {
    TensorArgs t[CAP];
    int32_t first[CAP + 1];  // first block of each tensor
    int32_t count;
};

struct Hyper {
    float b1, omb1, b2, omb2, step_size, inv_sqrt_bc2, eps, grad_scale;
};

template <typename T>
__device__ __forceinline__ void load8(const T* p, int64_t i, int64_t n, bool vec, float (&x)[kPer]) {
    if (vec && i + kPer <= n) {
        if constexpr (sizeof(T) == 4) {
            const float4 a = *reinterpret_cast<const float4*>(p + i), b = *reinterpret_cast<const float4*>(p + i + 4);
            x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
            x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
        } else {
            const uint4 a = *reinterpret_cast<const uint4*>(p + i);
            const T* h = reinterpret_cast<const T*>(&a);
#pragma unroll
            for (int j = 0; j < kPer; ++j) x[j] = to_f32<T>(h[j]);
        }
    } else {
#pragma unroll
        for (int j = 0; j < kPer; ++j) x[j] = i + j < n ? to_f32<T>(p[i + j]) : 0.f;
    }
}

template <typename T>
__device__ __forceinline__ void store8(T* p, int64_t i, int64_t n, bool vec, const float (&x)[kPer]) {
    if (vec && i + kPer <= n) {
        if constexpr (sizeof(T) == 4) {
            *reinterpret_cast<float4*>(p + i) = make_float4(x[0], x[1], x[2], x[3]);
            *reinterpret_cast<float4*>(p + i + 4) = make_float4(x[4], x[5], x[6], x[7]);
        } else {
            uint4 a;
            T* h = reinterpret_cast<T*>(&a);
#pragma unroll
            for (int j = 0; j < kPer; ++j) h[j] = from_f32<T>(x[j]);
            *reinterpret_cast<uint4*>(p + i) = a;
        }
    } else {
#pragma unroll
        for (int j = 0; j < kPer; ++j)
            if (i + j < n) p[i + j] = from_f32<T>(x[j]);
    }
}

// Eight codes, element j in byte j of (x, y).
__device__ __forceinline__ uint2 load_codes(const uint8_t* p, int64_t i, int64_t n, bool vec) {
    if (vec && i + kPer <= n) return *reinterpret_cast<const uint2*>(p + i);
    uint32_t w[2] = {0, 0};
#pragma unroll
    for (int j = 0; j < kPer; ++j)
        if (i + j < n) w[j >> 2] |= (uint32_t)p[i + j] << 8 * (j & 3);
    return make_uint2(w[0], w[1]);
}
__device__ __forceinline__ void store_codes(uint8_t* p, int64_t i, int64_t n, bool vec, uint2 c) {
    if (vec && i + kPer <= n) {
        *reinterpret_cast<uint2*>(p + i) = c;
    } else {
#pragma unroll
        for (int j = 0; j < kPer; ++j)
            if (i + j < n) p[i + j] = (uint8_t)((j < 4 ? c.x : c.y) >> 8 * (j & 3));
    }
}

// First moment, four codes at a time: the format is the one that the conversion instructions know as e4m3.
__device__ __forceinline__ void decode_m4(uint32_t c, float* x) {
    uint32_t h[2];
    asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, lo;\n\tcvt.rn.f16x2.e4m3x2 %1, hi;\n\t}"
        : "=r"(h[0]), "=r"(h[1])
        : "r"(c));
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h[i]));
        x[2 * i] = f.x;
        x[2 * i + 1] = f.y;
    }
}
__device__ __forceinline__ uint32_t encode_m4(const float* x, float inv) {
    float y[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) y[i] = fmaf(x[i], 0.f, __fmul_rn(x[i], inv));  // 0 x: infinities become NaN as well
    uint32_t c;
    asm("{\n\t.reg .b16 lo, hi;\n\tcvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\n\t"
        "cvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\n\tmov.b32 %0, {lo, hi};\n\t}"
        : "=r"(c)
        : "f"(y[0]), "f"(y[1]), "f"(y[2]), "f"(y[3]));
    return c;
}
// Root of the second moment.
__device__ __forceinline__ float decode_u(uint32_t c) {
    float x = __uint_as_float((c << 19) + ((127u << 23) - (1u << 19)));
    if (c == 0u) x = 0.f;
    if (c == 255u) x = __uint_as_float(0x7fc00000u);
    return x;
}
__device__ __forceinline__ void decode_u4(uint32_t c, float* x) {
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = decode_u((c >> 8 * i) & 255u);
}
__device__ __forceinline__ uint32_t encode_u(float u, float inv) {
    const float y = __fmul_rn(u, inv);
    const uint32_t b = __float_as_uint(fmaxf(y, 1.f)) - ((127u << 23) - (1u << 19));
    uint32_t t = (b + 0x3FFFFu + ((b >> 19 & 1u) ^ 1u)) >> 19;  // to nearest, ties to even (the code's lowest bit is
    if (!(y > 0.f)) t = 0u;                                     // the mantissa's plus one)
    if (!(u < INFINITY)) t = 255u;
    return t;
}
__device__ __forceinline__ uint32_t encode_u4(const float* u, float inv) {
    const uint32_t lo = __byte_perm(encode_u(u[0], inv), encode_u(u[1], inv), 0x0040);
    const uint32_t hi = __byte_perm(encode_u(u[2], inv), encode_u(u[3], inv), 0x0040);
    return __byte_perm(lo, hi, 0x5410);
}

// Scale exponent of a block: its largest finite |x| goes to [2^top, 2^(top + 1)).
__device__ __forceinline__ int block_exponent(const float (&x)[kPer], int top) {
    float most = 0.f;  // (a NaN is no maximum)
#pragma unroll
    for (int j = 0; j < kPer; ++j) most = fmaxf(most, fabsf(x[j]));
    uint32_t big = __reduce_max_sync(0xffffffffu, __float_as_uint(most));
    if (big == 0x7f800000u) {  // infinities do not count
        most = 0.f;
#pragma unroll
        for (int j = 0; j < kPer; ++j)
            if (fabsf(x[j]) < INFINITY) most = fmaxf(most, fabsf(x[j]));
        big = __reduce_max_sync(0xffffffffu, __float_as_uint(most));
    }
    if (big == 0u) return 0;  // scale 1
    return min(max((int)(big >> 23) - 127 - top, -100), 120);
}
__device__ __forceinline__ float pow2(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

template <typename T, int BITS>
__device__ __forceinline__ void step_chunk(const TensorArgs& a, const Hyper& h, int64_t i) {
    const bool vec = (a.flags & kVec) != 0;
    const int64_t n = a.n;
    float p[kPer], g[kPer], m[kPer], v[kPer], u[kPer];
    uint2 cm, cv;
    float ms = 0.f, vs = 0.f;
    if constexpr (BITS == 8) {
        cm = load_codes(static_cast<const uint8_t*>(a.m), i, n, vec);
        cv = load_codes(static_cast<const uint8_t*>(a.v), i, n, vec);
        if (i < n) {
            ms = a.m_scale[i / kStateBlock];
            vs = a.v_scale[i / kStateBlock];
        }
    } else {
        load8(static_cast<const float*>(a.m), i, n, vec, m);
        load8(static_cast<const float*>(a.v), i, n, vec, v);
    }
    load8(static_cast<const T*>(a.grad), i, n, vec, g);
    if (a.master) load8(a.master, i, n, vec, p);
    else load8(static_cast<const T*>(a.param), i, n, vec, p);
    if constexpr (BITS == 8) {
        decode_m4(cm.x, m);
        decode_m4(cm.y, m + 4);
        decode_u4(cv.x, v);
        decode_u4(cv.y, v + 4);
    }
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
        if constexpr (BITS == 8) {
            m[j] = __fmul_rn(m[j], ms);
            v[j] = __fmul_rn(v[j], vs);
            v[j] = __fmul_rn(v[j], v[j]);
        }
        const float gj = __fmul_rn(g[j], h.grad_scale);
        m[j] = __fadd_rn(__fmul_rn(m[j], h.b1), __fmul_rn(gj, h.omb1));
        v[j] = __fadd_rn(__fmul_rn(v[j], h.b2), __fmul_rn(__fmul_rn(gj, gj), h.omb2));
        u[j] = __fsqrt_rn(v[j]);
        const float den = __fadd_rn(__fmul_rn(u[j], h.inv_sqrt_bc2), h.eps);
        p[j] = __fsub_rn(__fmul_rn(p[j], a.decay), __fmul_rn(__fdiv_rn(m[j], den), h.step_size));
    }
    store8(static_cast<T*>(a.param), i, n, vec, p);
    if (a.master) store8(a.master, i, n, vec, p);
    if constexpr (BITS == 8) {
        if (i >= n) {  // elements past the tensor's end weigh nothing in the block's scale
#pragma unroll
            for (int j = 0; j < kPer; ++j) m[j] = u[j] = 0.f;
        } else if (i + kPer > n) {
#pragma unroll
            for (int j = 0; j < kPer; ++j)
                if (i + j >= n) m[j] = u[j] = 0.f;
        }
        const int em = block_exponent(m, 7), eu = block_exponent(u, 14);
        const float im = pow2(-em), iu = pow2(-eu);
        cm = make_uint2(encode_m4(m, im), encode_m4(m + 4, im));
        cv = make_uint2(encode_u4(u, iu), encode_u4(u + 4, iu));
        store_codes(static_cast<uint8_t*>(a.m), i, n, vec, cm);
        store_codes(static_cast<uint8_t*>(a.v), i, n, vec, cv);
        if ((threadIdx.x & 31) == 0 && i < n) {
            a.m_scale[i / kStateBlock] = pow2(em);
            a.v_scale[i / kStateBlock] = pow2(eu);
        }
    } else {
        store8(static_cast<float*>(a.m), i, n, vec, m);
        store8(static_cast<float*>(a.v), i, n, vec, v);
    }
}

template <int CAP, int BITS>
__global__ void __launch_bounds__(kThreads, BITS == 8 ? 6 : 5) k_adamw(const __grid_constant__ Table<CAP> tab, const Hyper h) {
    int lo = 0, hi = tab.count;  // the last tensor whose first block is not past this one
    const int blk = blockIdx.x;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (tab.first[mid] <= blk) lo = mid;
        else hi = mid;
    }
    const TensorArgs& a = tab.t[lo];
    const int64_t i = (int64_t)(blk - tab.first[lo]) * kChunk + threadIdx.x * kPer;
    switch (a.flags & 3) {
        case VG_F32: step_chunk<float, BITS>(a, h, i); break;
        case VG_F16: step_chunk<__half, BITS>(a, h, i); break;
        default: step_chunk<__nv_bfloat16, BITS>(a, h, i); break;
    }
}

// Four elements a thread and access, so that a warp's stores are whole lines.
template <bool SECOND>
__global__ void __launch_bounds__(kThreads) k_adamw_decode(const uint8_t* __restrict__ codes,
                                                           const float* __restrict__ scales, int64_t n, bool vec,
                                                           float* __restrict__ out) {
    const int64_t first = (int64_t)blockIdx.x * kChunk + threadIdx.x * 4;
    uint32_t c[kPer / 4];
    float s[kPer / 4];
#pragma unroll
    for (int k = 0; k < kPer / 4; ++k) {
        const int64_t i = first + k * 4 * kThreads;
        c[k] = 0;
        s[k] = i < n ? scales[i / kStateBlock] : 0.f;
        if (vec && i + 4 <= n) {
            c[k] = *reinterpret_cast<const uint32_t*>(codes + i);
        } else {
            for (int j = 0; j < 4; ++j)
                if (i + j < n) c[k] |= (uint32_t)codes[i + j] << 8 * j;
        }
    }
#pragma unroll
    for (int k = 0; k < kPer / 4; ++k) {
        const int64_t i = first + k * 4 * kThreads;
        float x[4];
        if constexpr (SECOND) decode_u4(c[k], x);
        else decode_m4(c[k], x);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            x[j] = __fmul_rn(x[j], s[k]);
            if (SECOND) x[j] = __fmul_rn(x[j], x[j]);
        }
        if (vec && i + 4 <= n) {
            *reinterpret_cast<float4*>(out + i) = make_float4(x[0], x[1], x[2], x[3]);
        } else {
            for (int j = 0; j < 4; ++j)
                if (i + j < n) out[i + j] = x[j];
        }
    }
}

template <int CAP>
int launch_group(const vg_adamw_tensor* ts, int count, int bits, double lr, const Hyper& h, cudaStream_t s) {
    Table<CAP> tab;
    int64_t blocks = 0;
    tab.count = 0;
    for (int i = 0; i < count; ++i) {
        const vg_adamw_tensor& t = ts[i];
        if (t.n == 0) continue;
        TensorArgs& a = tab.t[tab.count];
        a = TensorArgs{t.param, t.grad, t.master, t.m, t.v, t.m_scale, t.v_scale, t.n,
                       (float)(1.0 - lr * t.weight_decay), t.dtype};
        const uintptr_t wide = reinterpret_cast<uintptr_t>(t.param) | reinterpret_cast<uintptr_t>(t.grad) |
                               reinterpret_cast<uintptr_t>(t.master);
        const uintptr_t state = reinterpret_cast<uintptr_t>(t.m) | reinterpret_cast<uintptr_t>(t.v);
        if (!(wide & 15) && !(state & (bits == 8 ? 7 : 15))) a.flags |= kVec;
        tab.first[tab.count++] = (int32_t)blocks;
        blocks += (t.n + kChunk - 1) / kChunk;
    }
    if (blocks == 0) return VG_OK;
    if (blocks >= (int64_t(1) << 31)) return VG_ERR_UNSUPPORTED;
    tab.first[tab.count] = (int32_t)blocks;
    if (bits == 8) k_adamw<CAP, 8><<<(unsigned)blocks, kThreads, 0, s>>>(tab, h);
    else k_adamw<CAP, 32><<<(unsigned)blocks, kThreads, 0, s>>>(tab, h);
    return cudaPeekAtLastError() == cudaSuccess ? VG_OK : VG_ERR_CUDA;
}

constexpr int kShort = 32, kLong = 384;
static_assert(sizeof(Table<kShort>) + sizeof(Hyper) <= 4000 && sizeof(Table<kLong>) + sizeof(Hyper) <= 32764,
              "launch parameters");

}  // namespace

int adamw_step(const vg_adamw_tensor* ts, int count, int bits, int64_t step, double lr, double beta1, double beta2,
               double eps, double grad_scale, cudaStream_t s) {
    const double bc1 = 1.0 - pow(beta1, (double)step), bc2 = 1.0 - pow(beta2, (double)step);
    const Hyper h{(float)beta1, (float)(1.0 - beta1), (float)beta2, (float)(1.0 - beta2),
                  (float)(lr / bc1), (float)(1.0 / sqrt(bc2)), (float)eps, (float)grad_scale};
    for (int i = 0; i < count;) {
        const int left = count - i;
        const int take = left <= kShort ? left : std::min(left, kLong);
        const int st = take <= kShort ? launch_group<kShort>(ts + i, take, bits, lr, h, s)
                                      : launch_group<kLong>(ts + i, take, bits, lr, h, s);
        if (st != VG_OK) return st;
        i += take;
    }
    return VG_OK;
}

int adamw_decode(const uint8_t* codes, const float* scales, int64_t n, int second, float* out, cudaStream_t s) {
    if (n == 0) return VG_OK;
    const bool vec = !(reinterpret_cast<uintptr_t>(codes) & 7) && !(reinterpret_cast<uintptr_t>(out) & 15);
    const int64_t blocks = (n + kChunk - 1) / kChunk;
    if (blocks >= (int64_t(1) << 31)) return VG_ERR_UNSUPPORTED;
    if (second) k_adamw_decode<true><<<(unsigned)blocks, kThreads, 0, s>>>(codes, scales, n, vec, out);
    else k_adamw_decode<false><<<(unsigned)blocks, kThreads, 0, s>>>(codes, scales, n, vec, out);
    return cudaPeekAtLastError() == cudaSuccess ? VG_OK : VG_ERR_CUDA;
}

}  // namespace vg
