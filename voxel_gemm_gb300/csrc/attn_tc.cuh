// Cross attention on the tensor cores: what the 16-bit forward and backward kernels
// share.
//
// Every operand tile is a box of a [rows][heads][d] tensor, copied by the TMA engine
// into rows of 128 bytes (64 channels) in the 128-byte swizzle; d > 64 takes two such
// blocks.  Channels past d and rows past the tensor read as zero.  The same tile
// serves as a K-major operand (contraction over channels) and as an MN-major one
// (contraction over rows), so nothing is transposed.  Boxes of query rows hold gp
// heads of 128/gp queries: the packed rows of attn.cuh, in order.
#pragma once
#include <cuda.h>

#include <type_traits>

#include "attn.cuh"
#include "attn_waits.h"
#include "tc_ptx.cuh"

namespace vg {

struct AttnMaps {
    CUtensorMap q, k, v, go;
};

// Tensor map over a [rows][heads][d] operand with boxes of 64 channels x `box_heads`
// heads x `box_rows` rows.  VG_OK, VG_ERR_UNSUPPORTED (strides beyond what the engine
// takes) or VG_ERR_CUDA.
int attn_make_map(CUtensorMap* map, const vg_heads& h, int64_t rows, int heads, int d, int dtype, int box_heads,
                  int box_rows);

namespace attn_tc {

using namespace ptx;

constexpr float kLn2 = 0.69314718055994530942f;

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

template <bool BF16>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    uint32_t r;
    if constexpr (BF16) asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    else asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

__device__ __forceinline__ float2 two(const uint32_t* r) {
    return make_float2(__uint_as_float(r[0]), __uint_as_float(r[1]));
}

// ---- products, issued by an elected lane.  A short product leaves it a few dozen cycles, so
// the steps are unrolled and a step's descriptors are its tile's plus a constant.

// D (+)= A B^T over `steps` (<= STEPS) K = 16 steps, both K-major in shared memory; ABLK, BBLK: bytes
// between the operands' 64-channel blocks.
template <int STEPS, int ABLK, int BBLK>
__device__ __forceinline__ void mma_channels(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                             int steps) {
#pragma unroll
    for (int j = 0; j < STEPS; ++j) {
        if (j >= steps) break;
        const uint32_t ao = ((j >> 2) * ABLK + (j & 3) * 32) >> 4, bo = ((j >> 2) * BBLK + (j & 3) * 32) >> 4;
        mma_f16(d, a + ao, b + bo, idesc, j > 0);
    }
}
// D (+)= A B over `steps` (<= STEPS) K = 16 steps of rows, A in TMEM, B MN-major in shared memory.
template <int STEPS>
__device__ __forceinline__ void mma_rows(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, int steps,
                                         uint32_t acc) {
#pragma unroll
    for (int j = 0; j < STEPS; ++j) {
        if (j >= steps) break;
        if (j == 0) mma_f16_ta(d, a, b, idesc, acc);
        else mma_f16_ta(d, a + 8 * j, b + j * (2048 >> 4), idesc, 1);
    }
}

// Zero rows [from, to) of a tile of `blocks` 64-channel blocks, `block_bytes` apart, by one warp.
__device__ __forceinline__ void zero_rows(uint32_t tile, int from, int to, int blocks, int block_bytes) {
    const int per = (to - from) * 8;  // 16-byte pieces of a block
    for (int e = threadIdx.x & 31; e < per * blocks; e += 32) {
        const int b = e / per, i = e - b * per;
        asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(tile + b * block_bytes + from * 128 + i * 16),
                     "r"(0)
                     : "memory");
    }
}

// Write 32 fp32 columns of a row as 16-bit values; `n` of them exist (a multiple of 8).
template <bool BF16>
__device__ __forceinline__ void store_cols32(void* dst, const uint32_t (&acc)[32], float mul, int n) {
    uint4* d4 = static_cast<uint4*>(dst);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (8 * i >= n) break;
        uint32_t w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint32_t* two = acc + 8 * i + 2 * j;
            w[j] = pack2<BF16>(__uint_as_float(two[0]) * mul, __uint_as_float(two[1]) * mul);
        }
        d4[i] = make_uint4(w[0], w[1], w[2], w[3]);
    }
}
__device__ __forceinline__ void store_cols32_f32(float* dst, const uint32_t (&acc)[32], float mul, int n) {
    float4* d4 = reinterpret_cast<float4*>(dst);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        if (4 * i >= n) break;
        d4[i] = make_float4(__uint_as_float(acc[4 * i]) * mul, __uint_as_float(acc[4 * i + 1]) * mul,
                            __uint_as_float(acc[4 * i + 2]) * mul, __uint_as_float(acc[4 * i + 3]) * mul);
    }
}

// Whether whole 32-byte pieces of an output's rows can be stored.
__device__ __forceinline__ bool lines_ok(const vg_heads& h) {
    return ((reinterpret_cast<uintptr_t>(h.data) | (uintptr_t)(h.row_stride * 2) | (uintptr_t)(h.head_stride * 2)) &
            31u) == 0;
}

// A thread's row of an accumulator of DP columns at `t` (lanes of its warp), times `mul`: to `dst` in 16 bits, or to
// `part` in fp32 when the axis is cut.  have: the accumulator holds something (else zeros); store: the thread
// has a row; live: the row is not zeros by definition; of, ofs: this warp does every ofs-th piece from `of` on.  By
// the whole warp.
template <bool BF16, int DP>
__device__ __forceinline__ void store_row(const AttnArgs& a, bool have, uint32_t t, float mul, bool store,
                                          uint16_t* dst, float* part, int lane, bool v8ok, bool live = true,
                                          int of = 0, int ofs = 1) {
    __syncwarp();
    auto columns = [&](int col, uint32_t (&o)[32]) {
        if (have) {
            tmem_ld32(t + col, o);
            tmem_ld_wait();
            tmem_ld_done(o);
        }
        if (!have || !live) {
#pragma unroll
            for (int j = 0; j < 32; ++j) o[j] = 0u;
        }
        __syncwarp();
    };
    if (a.splits == 1 && a.d == DP) {  // whole 128-byte lines of 64 columns
#pragma unroll 1
        for (int line = of; line < DP / 64; line += ofs) {
            uint32_t z[32];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                uint32_t o[32];
                columns(line * 64 + 32 * i, o);
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    const float2 v = two(o + 2 * j);
                    z[16 * i + j] = pack2<BF16>(v.x * mul, v.y * mul);
                }
            }
            store_lines_quad(store ? reinterpret_cast<uint8_t*>(dst + line * 64) : nullptr, z, lane, v8ok);
        }
    } else {
#pragma unroll 1
        for (int col = 32 * of; col < a.d; col += 32 * ofs) {
            uint32_t o[32];
            columns(col, o);
            if (store) {
                if (a.splits > 1) store_cols32_f32(part + col, o, mul, a.d - col);
                else store_cols32<BF16>(dst + col, o, mul, a.d - col);
            }
            __syncwarp();
        }
    }
}

// Bounded waits of a whole warp, which goes on or gives up together; a wait that gives
// up (after kWaitCycles or the given limit) raises the block's abort flag, and the
// warp's later waits return at once.  Every branch is on a vote, so that the compiler knows
// the warp to be converged and keeps what follows (descriptors, addresses, loop counts) in
// uniform registers.
struct Waiter {
    volatile uint32_t* abort;
    bool ok = true;
    __device__ __forceinline__ bool operator()(uint32_t bar, uint32_t parity, int64_t limit = kWaitCycles) {
        if (!ok || __all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return ok;
        const int64_t t0 = clock64();
        while (true) {
            if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
            if (__any_sync(0xffffffffu, *abort != 0 || clock64() - t0 > limit)) break;
        }
        *abort = 1;
        ok = false;
        return false;
    }
};

// Wait for the copies that can still be in flight, whatever became of the block; barriers 8 bytes apart from `bar`.
template <int S>
__device__ __forceinline__ bool land(const Copies<S>& copies, uint32_t bar) {
    bool ok = true;
    copies.in_flight([&](uint32_t slot, uint32_t parity) { ok &= mbar_wait_timed(bar + 8 * slot, parity); });
    return ok;
}

template <int V> using Const = std::integral_constant<int, V>;

// A position in a ring of S slots and the parity of the pass over it.
template <int S>
struct RingPos {
    uint32_t i = 0, phase = 0;
    __device__ __forceinline__ void step() {
        if (++i == S) i = 0, phase ^= 1u;
    }
    __device__ __forceinline__ void skip(uint32_t n) {
        i += n;
        phase ^= (i / S) & 1u;
        i %= S;
    }
};

// Run f in one lane of a converged warp.
template <typename F>
__device__ __forceinline__ void one_lane(F f) {
    if (elect_one()) f();
    __syncwarp();
}

// f in one lane of a converged warp, with waits of that lane alone: a warp's wait takes its vote as well, and between
// two batches of products every cycle counts.
struct LaneWaiter {
    volatile uint32_t* abort;
    bool ok = true;
    __device__ __forceinline__ bool operator()(uint32_t bar, uint32_t parity) {
        if (!ok || mbar_try_wait(bar, parity)) return ok;
        const int64_t t0 = clock64();
        while (!mbar_try_wait(bar, parity)) {
            if (*abort != 0 || clock64() - t0 > kWaitCycles) {
                *abort = 1;
                return ok = false;
            }
        }
        return true;
    }
};
template <typename F>
__device__ __forceinline__ void by_one_lane(Waiter& wait, F f) {
    LaneWaiter w{wait.abort, wait.ok};
    if (elect_one()) f(w);
    wait.ok = __all_sync(0xffffffffu, w.ok);
}

// The value of lane 0 in every lane, as one that the compiler knows to be uniform.
__device__ __forceinline__ int uniform(int v) { return __shfl_sync(0xffffffffu, v, 0); }
__device__ __forceinline__ uint32_t uniform(uint32_t v) { return __shfl_sync(0xffffffffu, v, 0); }

// Work unit of a block: a few ints, found once by the scheduler warp (looking a tile's
// sample up takes a few dependent loads and divisions, some 2,400 cycles) and handed to
// the other warps through a ring of slots in shared memory.
struct Unit {
    int first, rows;   // first row of the unit within its sample, how many it has; rows < 0: no more units
    int head, part;    // head set or key head; part of the split axis
    int lo, hi;        // tiles of the axis that the unit runs along
    int q0, lq;        // the sample's queries
    int k0, lk;        // its keys: first row, valid rows
    uint32_t max_go, max_v;  // fp16 backward: bits of the sample's largest |dO row|, |V row|
};
constexpr int kUnitSlots = 4;

struct UnitRing {
    int4* slots;          // [kUnitSlots][3]
    uint32_t full, empty;  // barriers, 8 bytes apart
    const AttnArgs& a;     // its unit_cycles bounds both waits: the scheduler's for a slot, and a reader's that is ahead
    uint32_t at = 0;

    __device__ __forceinline__ void put(Waiter& wait, const Unit& x) {
        const uint32_t i = at % kUnitSlots;
        wait(empty + 8 * i, ((at / kUnitSlots) & 1u) ^ 1u, a.unit_cycles);
        if ((threadIdx.x & 31) == 0) {
            const int4* src = reinterpret_cast<const int4*>(&x);
            for (int j = 0; j < 3; ++j) slots[3 * i + j] = src[j];
            mbar_arrive(full + 8 * i);
        }
        __syncwarp();
        ++at;
    }
    // The next unit; false at the end, or when the wait gave up.
    __device__ __forceinline__ bool get(Waiter& wait, Unit& x) {
        const uint32_t i = at % kUnitSlots;
        if (!wait(full + 8 * i, (at / kUnitSlots) & 1u, a.unit_cycles)) return false;
        int4* dst = reinterpret_cast<int4*>(&x);
        for (int j = 0; j < 3; ++j) dst[j] = slots[3 * i + j];
        x.first = uniform(x.first);
        x.rows = uniform(x.rows);
        x.head = uniform(x.head);
        x.part = uniform(x.part);
        x.lo = uniform(x.lo);
        x.hi = uniform(x.hi);
        x.q0 = uniform(x.q0);
        x.lq = uniform(x.lq);
        x.k0 = uniform(x.k0);
        x.lk = uniform(x.lk);
        if ((threadIdx.x & 31) == 0) mbar_arrive(empty + 8 * i);
        __syncwarp();
        ++at;
        return x.rows >= 0;
    }
};

}  // namespace attn_tc

}  // namespace vg
