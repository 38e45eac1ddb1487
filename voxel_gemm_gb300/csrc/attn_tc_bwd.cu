// Cross attention backward on the tensor cores (tcgen05 / TMEM), 16-bit types: one
// kernel for the query gradient, one for the key and value gradients.
//
//   P = exp2(c S - lse log2 e), dS = P (dP - delta), dP = dO V^T
//   dQ = scale dS K,   dK = scale dS^T Q,   dV = P^T dO
//
// Two kernels recompute the scores twice (7 products instead of 5) but each keeps its
// gradient in TMEM from its first tile to its last and writes it once: no atomics, no
// fp32 gradient in memory, the same bits every run.
//
// dQ: a persistent block takes 128 packed query rows and runs along the keys in tiles of
// 128.  dK, dV: it takes 128 keys and runs along the packed rows of every query head that
// reads them, 128 at a time, so gradients of shared heads are sums in the same accumulators.
// Both have
//   warps 0 .. 15   softmax: four threads per row of a 128 x 128 tile, 32 columns each
//   then one warp   loader: TMA copies of the block's own tiles and of the tiles it runs along
//   then two warps  issue the products: one S and dP, the other one the gradients (d > 64 in
//                   dK, dV: one warp for all)
//   then one warp   scheduler: finds the block's next units
// The 16-bit dS (and P) go to TMEM columns of their own, as first operands of the gradient
// products: the next S and dP are computed while this tile's exponentials are.  (dK, dV with
// d > 64 has no columns left: there they lie over the scores.)  Tiles are 128 wide because a
// product of two shared-memory operands runs at the tensor cores' rate only from N = 128
// on: at N = 64 it takes 48 cycles instead of 32 to read its operands.
//
// fp16 has no exponent range to spare: P carries 2^15 (P <= 1), and dP - delta is divided by
// a power of two above 2 max|dO row| max|V row|, which bounds it; both leave with the
// fp32 result.  bf16 needs neither.
#include "attn_tc.cuh"

namespace vg {

namespace {

using namespace attn_tc;

constexpr int kM = 128;  // rows of the products
constexpr int kN = 128;  // columns of a step
constexpr int kH = 32;   // columns of a softmax thread
constexpr int kThreads = 512 + 128;
// A thread's 16-bit values take half the columns of its scores: packed when they have a place of their own, else over
// the first half of those scores, which no other thread reads.
template <bool OWN> constexpr int kGap = OWN ? 0 : kH / 2;

// The power of two that dP - delta is multiplied by, and its inverse.
template <bool BF16>
__device__ __forceinline__ float2 grad_lift(const AttnArgs& a) {
    if constexpr (BF16) return make_float2(1.f, 1.f);
    const float bound = 2.f * __uint_as_float(a.err[1]) * __uint_as_float(a.err[2]);
    const int e = (int)(__float_as_uint(bound) >> 23) - 127;
    if (!(bound > 0.f) || e > 120 || e < -120) return make_float2(1.f, 1.f);
    return make_float2(__uint_as_float((uint32_t)(126 - e) << 23), __uint_as_float((uint32_t)(128 + e) << 23));
}

template <bool BF16> constexpr float kLift = BF16 ? 0.f : 15.f;             // exponent added to P
template <bool BF16> constexpr float kDrop = BF16 ? 1.f : 1.f / 32768.f;

// ================================================================ query gradient
template <int DP>
struct CfgQ {
    static constexpr int kBlocks = DP / 64;
    static constexpr int kTile = kM * 128 * kBlocks;       // bytes of a Q, dO, K or V tile
    static constexpr int S = DP == 64 ? 4 : 2;             // ring stages (a K and a V tile each)
    static constexpr int kOCol = 2 * kN, kPCol = kOCol + DP;  // dQ's and dS's first TMEM column
    // q, s, p and o (full, empty), (kv full, kv empty) x S, tail, done x 2, unit ring
    static constexpr int kBars = 8 + 2 * S + 3 + 2 * kUnitSlots;
    static constexpr size_t kSmem = 1024 + (size_t)(2 + 2 * S) * kTile + kUnitSlots * sizeof(Unit) + 8 * kBars + 16;
};
static_assert(CfgQ<128>::kSmem <= 232448 && CfgQ<64>::kSmem <= 232448 && CfgQ<128>::kPCol + kN / 2 <= 512,
              "shared memory, TMEM");

template <bool BF16, int DP>
__global__ void __launch_bounds__(kThreads, 1)
    k_attn_tc_dq(const AttnArgs a, const __grid_constant__ AttnMaps maps) {
    using C = CfgQ<DP>;
    constexpr int S = C::S;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sQ = smem_u32(smem), sG = sQ + C::kTile, sKV = sG + C::kTile;
    int4* s_units = reinterpret_cast<int4*>(smem + (size_t)(2 + 2 * S) * C::kTile);
    uint64_t* bars = reinterpret_cast<uint64_t*>(s_units + 3 * kUnitSlots);
    uint32_t* s_tmem = reinterpret_cast<uint32_t*>(bars + C::kBars);
    volatile uint32_t* s_abort = s_tmem + 1;
    const uint32_t bar0 = smem_u32(bars);
    const uint32_t q_full = bar0, q_empty = bar0 + 8, s_full = bar0 + 16, s_empty = bar0 + 24, p_full = bar0 + 32;
    const uint32_t p_empty = bar0 + 40, o_full = bar0 + 48, o_empty = bar0 + 56;
    const uint32_t kv_full = bar0 + 64, kv_empty = kv_full + 8 * S, tail = kv_empty + 8 * S;
    const uint32_t done = tail + 8, u_full = done + 16, u_empty = u_full + 8 * kUnitSlots;

    const int warp = uniform((int)threadIdx.x >> 5), lane = threadIdx.x & 31;
    constexpr int kLoader = 16, kIssuer = 17, kIssuer2 = 18, kScheduler = 19;
    if (threadIdx.x == 0) {
        mbar_init(q_full, 1);
        mbar_init(q_empty, 1);
        mbar_init(s_full, 1);
        mbar_init(s_empty, 16);
        mbar_init(p_full, 16);
        mbar_init(p_empty, 1);
        mbar_init(o_full, 1);
        mbar_init(o_empty, 16);
        for (int i = 0; i < S; ++i) {
            mbar_init(kv_full + 8 * i, 1);
            mbar_init(kv_empty + 8 * i, 1);
        }
        for (int i = 0; i < kUnitSlots; ++i) {
            mbar_init(u_full + 8 * i, 1);
            mbar_init(u_empty + 8 * i, 16 + 3);  // every reader: softmax warps, loader, issuers
        }
        mbar_init(tail, 1);
        mbar_init(done, 1);
        mbar_init(done + 8, 1);
        *s_abort = 0;
        fence_mbar_init();
    }
    if (warp == kIssuer) {
        tmem_alloc(smem_u32(s_tmem), 512);
        tmem_relinquish();
    }
    if (warp == kLoader && lane == 0) {
        prefetch_map(&maps.q);
        prefetch_map(&maps.k);
        prefetch_map(&maps.v);
        prefetch_map(&maps.go);
    }
    tc_fence_before();
    const bool good = attn_offsets_ok(a);  // a barrier of the whole block
    tc_fence_after();
    const uint32_t tmem = uniform(*s_tmem);

    const int group = a.hq / a.hk;
    Waiter wait{s_abort};
    UnitRing ring{s_units, u_full, u_empty};
    Unit x;
    if (warp == kScheduler) {
        // unit u = (row tile and part, head set): its rows and its key tiles [lo, hi)
        const int sets = a.hq / a.gp;
        for (int64_t u = blockIdx.x; good && wait.ok; u += gridDim.x) {
            const AttnTile t = attn_find_tile<false>(a, kM, u / sets);
            if (t.b < 0) break;
            x = Unit{t.first, min(kM, t.lq * a.gp - t.first), (int)(u % sets), t.part, 0, 0,
                     t.q0, t.lq, t.k0, t.lk, 0, 0};
            attn_split(a, t.lk, t.part, &x.lo, &x.hi);
            ring.put(wait, x);
        }
        x.rows = -1;
        ring.put(wait, x);
    } else if (warp == kLoader) {
        RingPos<S> pos;
        uint32_t n = 0, uc = 0, tc = 0;  // tiles and units loaded
        while (ring.get(wait, x)) {
            if (x.hi <= x.lo) continue;
            wait(q_empty, (uc & 1u) ^ 1u);
            if (!wait.ok) break;
            const int kh = x.head * a.gp / group, row = x.q0 + (x.first >> a.gp_log2);
            one_lane([&] {
                mbar_arrive_expect_tx(q_full, 2 * C::kTile);
                for (int b = 0; b < C::kBlocks; ++b) {
                    tma_load_3d(sQ + b * kM * 128, &maps.q, b * 64, x.head * a.gp, row, q_full);
                    tma_load_3d(sG + b * kM * 128, &maps.go, b * 64, x.head * a.gp, row, q_full);
                }
            });
            ++uc;
            for (int e = x.lo; e < x.hi; ++e) {
                const uint32_t k = sKV + 2 * pos.i * C::kTile;
                wait(kv_empty + 8 * pos.i, pos.phase ^ 1u);
                if (!wait.ok) break;
                const int left = min(kN, x.lk - e * kN), n16 = (left + 15) / 16 * 16;
                const uint32_t bar = n16 != left ? tail : kv_full + 8 * pos.i;
                one_lane([&] {
                    mbar_arrive_expect_tx(bar, 2 * C::kTile);
                    for (int b = 0; b < C::kBlocks; ++b) {
                        tma_load_3d(k + b * kN * 128, &maps.k, b * 64, kh, x.k0 + e * kN, bar);
                        tma_load_3d(k + C::kTile + b * kN * 128, &maps.v, b * 64, kh, x.k0 + e * kN, bar);
                    }
                });
                if (n16 != left) {  // K rows past the sample's keys may hold anything: 0 x them must be 0 in dS K
                    wait(tail, tc++ & 1u);
                    zero_rows(k, left, n16, C::kBlocks, kN * 128);
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(kv_full + 8 * pos.i);
                    __syncwarp();
                }
                pos.step();
                ++n;
            }
        }
        // every copy has landed before the block may exit
        if (uc > 0 && !mbar_wait_timed(q_full, (uc - 1) & 1u)) wait.ok = false;
        for (uint32_t i = 0; i < (uint32_t)S && i < n; ++i) {
            const uint32_t last = n - 1 - i;
            if (!mbar_wait_timed(kv_full + 8 * (last % S), (last / S) & 1u)) wait.ok = false;
        }
        if (!wait.ok && lane == 0) atomicOr(a.err, kErrTimeout);
    } else if (warp == kIssuer || warp == kIssuer2) {
        const int ksteps = (a.d + 15) / 16;
        const uint32_t idesc_s = idesc_f16(BF16, kN), idesc_o = idesc_f16_bn(BF16, ksteps * 16);
        const uint64_t dq = sw128_kmajor_desc(sQ), dg = sw128_kmajor_desc(sG), dk = sw128_kmajor_desc(sKV);
        const uint64_t dv = sw128_kmajor_desc(sKV + C::kTile), dkt = sw128_mnmajor_desc(sKV, kN * 128);
        RingPos<S> pos;
        uint32_t uc = 0, n = 0;  // units and tiles done
        while (ring.get(wait, x)) {
            if (x.hi <= x.lo) continue;
            const int last16 = (min(kN, x.lk - (x.hi - 1) * kN) + 15) / 16;   // K = 16 steps of the last tile
            wait(warp == kIssuer ? q_full : o_empty, warp == kIssuer ? uc & 1u : (uc & 1u) ^ 1u);
            for (int e = x.lo; e < x.hi; ++e, ++n) {
                const bool last = e + 1 == x.hi;
                const uint32_t stage = pos.i * (2 * C::kTile >> 4);
                wait(kv_full + 8 * pos.i, pos.phase);
                if (warp == kIssuer) {  // S = Q K^T and dP = dO V^T, once the last ones have been read
                    if (!wait(s_empty, (n & 1u) ^ 1u)) break;
                    tc_fence_after();
                    one_lane([&] {
                        const uint32_t id = last ? idesc_f16(BF16, last16 * 16) : idesc_s;
                        mma_channels<DP / 16, kM * 128, kN * 128>(tmem, dq, dk + stage, id, ksteps);
                        mma_channels<DP / 16, kM * 128, kN * 128>(tmem + kN, dg, dv + stage, id, ksteps);
                        mma_commit(s_full);
                        if (last) mma_commit(q_empty);
                    });
                } else {                // dQ += dS K
                    if (!wait(p_full, n & 1u)) break;
                    tc_fence_after();
                    one_lane([&] {
                        mma_rows<kN / 16>(tmem + C::kOCol, tmem + C::kPCol, dkt + stage, idesc_o,
                                          last ? last16 : kN / 16, e > x.lo);
                        mma_commit(p_empty);
                        mma_commit(kv_empty + 8 * pos.i);
                        if (last) mma_commit(o_full);
                    });
                }
                pos.step();
            }
            if (!wait.ok) break;
            ++uc;
        }
        // every product has finished before TMEM is released
        const uint32_t mine = done + 8 * (warp - kIssuer);
        one_lane([&] { mma_commit(mine); });
        if (!mbar_wait_timed(mine, 0)) wait.ok = false;
        if (!wait.ok && lane == 0) {
            *s_abort = 1;
            atomicOr(a.err, kErrTimeout);
        }
    } else if (warp < kLoader) {
        const int quarter = warp >> 2, quad = warp & 3;
        const uint32_t t_lane = tmem + ((uint32_t)(quad * 32) << 16);
        const uint32_t t_s = t_lane + quarter * kH, t_p = t_lane + C::kPCol + quarter * (kH / 2);
        const float c = a.scale_log2;
        const float2 lift = grad_lift<BF16>(a);
        const bool v8ok = lines_ok(a.gq);
        const int row = quad * 32 + lane;  // within the unit
        uint32_t n = 0, uc = 0;            // tiles and units done
        while (ring.get(wait, x)) {
            const bool any = x.rows > quad * 32, mine = row < x.rows;  // the warp, the thread has a row
            const int pr = x.first + row;                              // packed row of the sample
            float2 st = make_float2(0.f, 0.f);
            if (mine) st = a.stats[((int64_t)x.head * a.n_q + x.q0) * a.gp + pr];
            const float base = kLift<BF16> - st.x, delta = -st.y * lift.x;
            const float2 c2 = make_float2(c, c), base2 = make_float2(base, base);
            const float2 lift2 = make_float2(lift.x, lift.x), delta2 = make_float2(delta, delta);
            for (int e = x.lo; e < x.hi; ++e, ++n) {
                if (!wait(s_full, n & 1u)) break;
                tc_fence_after();
                uint32_t d[kH / 2];
                if (any) {
                    uint32_t s[kH], g[kH];
                    tmem_ld32(t_s, s);
                    tmem_ld32(t_s + kN, g);
                    tmem_ld_wait();
                    tmem_ld_done(s);
                    tmem_ld_done(g);
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(s_empty);
                    const int left = x.lk - e * kN - quarter * kH;  // columns from there on are not scores: weight 0,
                    if (left < kH) {                                // gradient 0
#pragma unroll
                        for (int i = 0; i < kH; ++i)
                            if (i >= left) s[i] = 0xff800000u, g[i] = 0u;
                    }
#pragma unroll
                    for (int j = 0; j < kH / 2; ++j) {
                        float2 p = fma2(two(s + 2 * j), c2, base2);
                        p = make_float2(ex2(p.x), ex2(p.y));
                        const float2 dp = two(g + 2 * j);
                        const float2 ds = mul2(p, BF16 ? add2(dp, delta2) : fma2(dp, lift2, delta2));
                        d[j] = pack2<BF16>(ds.x, ds.y);
                    }
                } else if (lane == 0) {
                    mbar_arrive(s_empty);
                }
                // The product that reads the last dS has finished.  Warps without rows wait as well: ahead of the
                // others, their arrivals for two tiles would add up to one early phase.
                if (n > 0 && !wait(p_empty, (n - 1) & 1u)) break;
                tc_fence_after();
                if (any) {
                    tmem_st16(t_p, d);
                    tmem_st_wait();
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(p_full);
            }
            if (x.hi > x.lo) {
                if (!wait(o_full, uc++ & 1u)) break;
                tc_fence_after();
            }
            if (any) {
                const int64_t qi = x.q0 + (pr >> a.gp_log2);
                const int h = x.head * a.gp + (pr & (a.gp - 1));
                float* part = a.part + (((size_t)x.part * a.n_q + qi) * a.hq + h) * a.d;
                store_row<BF16, DP>(a, x.hi > x.lo, t_lane + C::kOCol, a.scale * kDrop<BF16> * lift.y, mine && wait.ok,
                                    head_row<uint16_t>(a.gq, qi, h), part, lane, v8ok, true, quarter, 4);
            }
            if (x.hi > x.lo) {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(o_empty);
            }
        }
        if (!wait.ok && lane == 0) atomicOr(a.err, kErrTimeout);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kIssuer) tmem_dealloc(tmem, 512);
}

// ================================================================ key and value gradients
template <int DP>
struct CfgKV {
    static constexpr int kBlocks = DP / 64;
    static constexpr int kTile = kM * 128 * kBlocks;     // bytes of a K, V, Q or dO tile
    static constexpr int S = DP == 64 ? 4 : 2;           // ring stages (a Q and a dO step each)
    static constexpr int kVCol = 2 * kN, kKCol = kVCol + DP;
    // P and dS in columns of their own where there is room (d <= 64), else over the scores
    static constexpr bool kOwn = DP == 64;
    static constexpr int kPCol = kKCol + DP;
    // k, s, p and o (full, empty), (ring full, empty) x S, tail, done x 2, unit ring
    static constexpr int kBars = 8 + 2 * S + 3 + 2 * kUnitSlots;
    static constexpr size_t kStats = 16 * 2 * 2 * kH * sizeof(float);  // sixteen warps, two steps, two numbers a row
    static constexpr size_t kSmem =
        1024 + (size_t)(2 + 2 * S) * kTile + kStats + kUnitSlots * sizeof(Unit) + 8 * kBars + 16;
};
static_assert(CfgKV<128>::kSmem <= 232448 && CfgKV<64>::kSmem <= 232448 && CfgKV<128>::kKCol + 128 <= 512 &&
                  CfgKV<64>::kPCol + kN <= 512,
              "shared memory, TMEM");

template <bool BF16, int DP>
__global__ void __launch_bounds__(kThreads, 1)
    k_attn_tc_dkv(const AttnArgs a, const __grid_constant__ AttnMaps maps, float* part_dv) {
    using C = CfgKV<DP>;
    constexpr int S = C::S;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sK = smem_u32(smem), sV = sK + C::kTile, sQG = sV + C::kTile;
    float* s_stats = reinterpret_cast<float*>(smem + (size_t)(2 + 2 * S) * C::kTile);
    int4* s_units = reinterpret_cast<int4*>(s_stats + 64 * kH);
    uint64_t* bars = reinterpret_cast<uint64_t*>(s_units + 3 * kUnitSlots);
    uint32_t* s_tmem = reinterpret_cast<uint32_t*>(bars + C::kBars);
    volatile uint32_t* s_abort = s_tmem + 1;
    const uint32_t bar0 = smem_u32(bars);
    const uint32_t k_full = bar0, k_empty = bar0 + 8, s_full = bar0 + 16, s_empty = bar0 + 24, p_full = bar0 + 32;
    const uint32_t p_empty = bar0 + 40, o_full = bar0 + 48, o_empty = bar0 + 56;
    const uint32_t r_full = bar0 + 64, r_empty = r_full + 8 * S, tail = r_empty + 8 * S;
    const uint32_t done = tail + 8, u_full = done + 16, u_empty = u_full + 8 * kUnitSlots;

    const int warp = uniform((int)threadIdx.x >> 5), lane = threadIdx.x & 31;
    constexpr int kLoader = 16, kIssuer = 17, kIssuer2 = 18, kScheduler = 19;
    if (threadIdx.x == 0) {
        mbar_init(k_full, 1);
        mbar_init(k_empty, 1);
        mbar_init(s_full, 1);
        mbar_init(s_empty, 16);
        mbar_init(p_full, 16);
        mbar_init(p_empty, 1);
        mbar_init(o_full, 1);
        mbar_init(o_empty, 16);
        for (int i = 0; i < S; ++i) {
            mbar_init(r_full + 8 * i, 1);
            mbar_init(r_empty + 8 * i, 1);
        }
        for (int i = 0; i < kUnitSlots; ++i) {
            mbar_init(u_full + 8 * i, 1);
            mbar_init(u_empty + 8 * i, 16 + 2 + C::kOwn);  // every reader: softmax warps, loader, issuers
        }
        mbar_init(tail, 1);
        mbar_init(done, 1);
        mbar_init(done + 8, 1);
        *s_abort = 0;
        fence_mbar_init();
    }
    if (warp == kIssuer) {
        tmem_alloc(smem_u32(s_tmem), 512);
        tmem_relinquish();
    }
    if (warp == kLoader && lane == 0) {
        prefetch_map(&maps.q);
        prefetch_map(&maps.k);
        prefetch_map(&maps.v);
        prefetch_map(&maps.go);
    }
    tc_fence_before();
    const bool good = attn_offsets_ok(a);  // a barrier of the whole block
    tc_fence_after();
    const uint32_t tmem = uniform(*s_tmem);

    const int sets = a.hq / a.hk / a.gp;  // head sets that read a key head
    // A unit is (part and key tile, key head): rows = key rows of the tile, valid or not, [lo, hi) its row tiles of
    // each head set.  Its steps run over (head set, row tile).
    Waiter wait{s_abort};
    UnitRing ring{s_units, u_full, u_empty};
    Unit x;
    if (warp == kScheduler) {
        for (int64_t u = blockIdx.x; good && wait.ok; u += gridDim.x) {
            const AttnTile t = attn_find_tile<true>(a, kM, u / a.hk);
            if (t.b < 0) break;
            x = Unit{t.first, min(kM, t.krows - t.first), (int)(u % a.hk), t.part, 0, 0, t.q0, t.lq, t.k0, t.lk, 0, 0};
            if (t.first < t.lk) attn_split(a, (int64_t)t.lq * a.gp, t.part, &x.lo, &x.hi);
            ring.put(wait, x);
        }
        x.rows = -1;
        ring.put(wait, x);
    } else if (warp == kLoader) {
        RingPos<S> pos;
        uint32_t n = 0, uc = 0, tc = 0;  // steps and units loaded
        while (ring.get(wait, x)) {
            if (x.hi <= x.lo) continue;
            wait(k_empty, (uc & 1u) ^ 1u);
            if (!wait.ok) break;
            one_lane([&] {
                mbar_arrive_expect_tx(k_full, 2 * C::kTile);
                for (int b = 0; b < C::kBlocks; ++b) {
                    tma_load_3d(sK + b * kM * 128, &maps.k, b * 64, x.head, x.k0 + x.first, k_full);
                    tma_load_3d(sV + b * kM * 128, &maps.v, b * 64, x.head, x.k0 + x.first, k_full);
                }
            });
            ++uc;
            for (int hs = 0; hs < sets && wait.ok; ++hs)
                for (int e = x.lo; e < x.hi; ++e) {
                    const uint32_t q = sQG + 2 * pos.i * C::kTile;
                    wait(r_empty + 8 * pos.i, pos.phase ^ 1u);
                    if (!wait.ok) break;
                    const int left = min(kN, x.lq * a.gp - e * kN), n16 = (left + 15) / 16 * 16;
                    const uint32_t bar = n16 != left ? tail : r_full + 8 * pos.i;
                    const int head = (x.head * sets + hs) * a.gp, row = x.q0 + ((e * kN) >> a.gp_log2);
                    one_lane([&] {
                        mbar_arrive_expect_tx(bar, 2 * C::kTile);
                        for (int b = 0; b < C::kBlocks; ++b) {
                            tma_load_3d(q + b * kN * 128, &maps.q, b * 64, head, row, bar);
                            tma_load_3d(q + C::kTile + b * kN * 128, &maps.go, b * 64, head, row, bar);
                        }
                    });
                    if (n16 != left) {  // rows of the next sample: 0 x them must be 0 in dS^T Q and P^T dO
                        wait(tail, tc++ & 1u);
                        zero_rows(q, left, n16, C::kBlocks, kN * 128);
                        zero_rows(q + C::kTile, left, n16, C::kBlocks, kN * 128);
                        fence_proxy_async_smem();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(r_full + 8 * pos.i);
                        __syncwarp();
                    }
                    pos.step();
                    ++n;
                }
        }
        // every copy has landed before the block may exit
        if (uc > 0 && !mbar_wait_timed(k_full, (uc - 1) & 1u)) wait.ok = false;
        for (uint32_t i = 0; i < (uint32_t)S && i < n; ++i) {
            const uint32_t last = n - 1 - i;
            if (!mbar_wait_timed(r_full + 8 * (last % S), (last / S) & 1u)) wait.ok = false;
        }
        if (!wait.ok && lane == 0) atomicOr(a.err, kErrTimeout);
    } else if (warp == kIssuer || (C::kOwn && warp == kIssuer2)) {
        const int ksteps = (a.d + 15) / 16;
        const uint32_t idesc_s = idesc_f16(BF16, kN), idesc_o = idesc_f16_bn(BF16, ksteps * 16);
        const uint64_t dk = sw128_kmajor_desc(sK), dv = sw128_kmajor_desc(sV), dq = sw128_kmajor_desc(sQG);
        const uint64_t dqt = sw128_mnmajor_desc(sQG, kN * 128);
        constexpr uint32_t kStage = 2 * C::kTile >> 4, kSecond = C::kTile >> 4;  // to the next stage, to dO
        constexpr int G = kGap<C::kOwn>;
        const uint32_t t_p = C::kOwn ? tmem + C::kPCol : tmem, t_d = C::kOwn ? t_p + kN / 2 : tmem + kN;
        const bool do_scores = warp == kIssuer, do_grads = !C::kOwn || warp == kIssuer2;
        RingPos<S> ahead, pos;                // stages of the scores and of the gradients
        uint32_t uc = 0, n = 0;               // units and steps done
        while (ring.get(wait, x)) {
            if (x.hi <= x.lo) continue;
            const int per = x.hi - x.lo, steps = per * sets;
            const int last16 = (min(kN, x.lq * a.gp - (x.hi - 1) * kN) + 15) / 16;
            int ea = 0, eg = 0;               // row tiles (from lo) of the next scores and gradients
            // S^T = K Q^T and dP^T = V dO^T
            auto s_product = [&] {
                const uint32_t id = ea + 1 == per ? idesc_f16(BF16, last16 * 16) : idesc_s;
                mma_channels<DP / 16, kM * 128, kN * 128>(tmem, dk, dq + ahead.i * kStage, id, ksteps);
            };
            auto dp_product = [&](bool last) {
                const uint32_t id = ea + 1 == per ? idesc_f16(BF16, last16 * 16) : idesc_s;
                mma_channels<DP / 16, kM * 128, kN * 128>(tmem + kN, dv, dq + ahead.i * kStage + kSecond, id, ksteps);
                mma_commit(s_full);
                if (last) mma_commit(k_empty);
            };
            auto advance = [&] {
                ahead.step();
                if (++ea == per) ea = 0;
            };
            if (do_scores) {
                wait(k_full, uc & 1u);
                const int first = C::kOwn ? steps : 1;
                for (int i = 0; i < first; ++i) {
                    wait(r_full + 8 * ahead.i, ahead.phase);
                    if (C::kOwn) wait(s_empty, ((n + i) & 1u) ^ 1u);  // the last ones have been read
                    if (!wait.ok) break;
                    tc_fence_after();
                    one_lane([&] {
                        s_product();
                        dp_product(i + 1 == steps);
                    });
                    advance();
                }
            }
            if (do_grads) {
                wait(o_empty, (uc & 1u) ^ 1u);
                for (int i = 0; i < steps && wait.ok; ++i) {
                    const bool next = !C::kOwn && i + 1 < steps;
                    const int k16 = eg + 1 == per ? last16 : kN / 16;
                    if (C::kOwn) wait(r_full + 8 * pos.i, pos.phase);
                    if (next) wait(r_full + 8 * ahead.i, ahead.phase);
                    if (!wait(p_full, (n + i) & 1u)) break;
                    tc_fence_after();
                    // dV += P^T dO and dK += dS^T Q; over the scores' columns, the next scores follow in issue order
                    one_lane([&] {
                        const uint64_t q = dqt + pos.i * kStage;
                        mma_rows<kN / 16, G>(tmem + C::kVCol, t_p, q + kSecond, idesc_o, k16, i > 0);
                        if (next) s_product();
                        mma_rows<kN / 16, G>(tmem + C::kKCol, t_d, q, idesc_o, k16, i > 0);
                        if (C::kOwn) mma_commit(p_empty);
                        mma_commit(r_empty + 8 * pos.i);
                        if (next) dp_product(i + 2 == steps);
                        if (i + 1 == steps) mma_commit(o_full);
                    });
                    if (next) advance();
                    pos.step();
                    if (++eg == per) eg = 0;
                }
            }
            if (!wait.ok) break;
            n += steps;
            ++uc;
        }
        // every product has finished before TMEM is released
        const uint32_t mine = done + 8 * (warp - kIssuer);
        one_lane([&] { mma_commit(mine); });
        if (!mbar_wait_timed(mine, 0)) wait.ok = false;
        if (!wait.ok && lane == 0) {
            *s_abort = 1;
            atomicOr(a.err, kErrTimeout);
        }
    } else if (warp < kLoader) {
        const int quarter = warp >> 2, quad = warp & 3;
        const uint32_t t_lane = tmem + ((uint32_t)(quad * 32) << 16);
        const uint32_t t_s = t_lane + quarter * kH;
        const uint32_t t_p = C::kOwn ? t_lane + C::kPCol + quarter * (kH / 2) : t_s;
        const uint32_t t_d = t_p + (C::kOwn ? kN / 2 : kN);
        const float c = a.scale_log2;
        const float2 lift = grad_lift<BF16>(a);
        const float2 c2 = make_float2(c, c), lift2 = make_float2(lift.x, lift.x);
        // quarters 0 and 1 write dV, 2 and 3 dK
        const vg_heads grad = quarter < 2 ? a.gv : a.gk;
        float* part = quarter < 2 ? part_dv : a.part;
        const bool v8ok = lines_ok(grad);
        float* my_stats = s_stats + warp * 4 * kH;
        uint32_t n = 0, uc = 0;  // steps and units done
        while (ring.get(wait, x)) {
            const int rows = x.lq * a.gp, per = x.hi - x.lo, steps = per * sets;
            // Statistics (lse log2 e, delta) of the warp's 32 rows of a row tile, one per lane, kept negated.  (hs, e):
            // head set and row tile of the next step
            int hs = x.head * sets, e = x.lo;
            auto stat = [&](bool have) {
                const int r = e * kN + quarter * kH + lane;
                float2 v = make_float2(0.f, 0.f);
                if (have && r < rows) v = a.stats[((int64_t)hs * a.n_q + x.q0) * a.gp + r];
                return v;
            };
            float2 next = stat(steps > 0);
            for (int i = 0; i < steps; ++i, ++n) {
                const int left = rows - e * kN - quarter * kH;
                float* cur = my_stats + (n & 1u) * 2 * kH;  // [kH] of the first number, [kH] of the second
                cur[lane] = kLift<BF16> - next.x;
                cur[lane + kH] = -next.y * lift.x;
                __syncwarp();
                if (++e == x.hi) e = x.lo, ++hs;
                next = stat(i + 1 < steps);
                if (!wait(s_full, n & 1u)) break;
                tc_fence_after();
                uint32_t s[kH], g[kH], p[kH / 2], d[kH / 2];
                tmem_ld32(t_s, s);
                tmem_ld32(t_s + kN, g);
                tmem_ld_wait();
                tmem_ld_done(s);
                tmem_ld_done(g);
                if (C::kOwn) {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(s_empty);
                }
                if (left < kH) {  // columns from there on are no rows of the sample: weight 0, gradient 0
#pragma unroll
                    for (int j = 0; j < kH; ++j)
                        if (j >= left) s[j] = 0xff800000u, g[j] = 0u;
                }
#pragma unroll
                for (int j = 0; j < kH / 2; j += 2) {
                    const float4 lse = *reinterpret_cast<const float4*>(cur + 2 * j);
                    const float4 del = *reinterpret_cast<const float4*>(cur + kH + 2 * j);
#pragma unroll
                    for (int t = 0; t < 2; ++t) {
                        const float2 base = t == 0 ? make_float2(lse.x, lse.y) : make_float2(lse.z, lse.w);
                        float2 pr = fma2(two(s + 2 * (j + t)), c2, base);
                        pr = make_float2(ex2(pr.x), ex2(pr.y));
                        const float2 minus = t == 0 ? make_float2(del.x, del.y) : make_float2(del.z, del.w);
                        const float2 dp = two(g + 2 * (j + t));
                        const float2 ds = mul2(pr, BF16 ? add2(dp, minus) : fma2(dp, lift2, minus));
                        p[j + t] = pack2<BF16>(pr.x, pr.y);
                        d[j + t] = pack2<BF16>(ds.x, ds.y);
                    }
                }
                if (C::kOwn && n > 0) {  // the products that read the last P and dS have finished
                    if (!wait(p_empty, (n - 1) & 1u)) break;
                    tc_fence_after();
                }
                tmem_st16(t_p, p);
                tmem_st16(t_d, d);
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(p_full);
            }
            if (steps > 0) {
                if (!wait(o_full, uc++ & 1u)) break;
                tc_fence_after();
            }
            const int r = quad * 32 + lane;  // key rows past the valid ones get zeros
            const int64_t row = x.k0 + x.first + r;
            const float mul = quarter < 2 ? kDrop<BF16> : a.scale * kDrop<BF16> * lift.y;
            store_row<BF16, DP>(a, steps > 0, t_lane + (quarter < 2 ? C::kVCol : C::kKCol), mul, r < x.rows && wait.ok,
                                head_row<uint16_t>(grad, row, x.head),
                                part + (((size_t)x.part * a.n_k + row) * a.hk + x.head) * a.d, lane, v8ok,
                                x.first + r < x.lk, quarter & 1, 2);
            if (steps > 0) {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(o_empty);
            }
        }
        if (!wait.ok && lane == 0) atomicOr(a.err, kErrTimeout);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kIssuer) tmem_dealloc(tmem, 512);
}

template <bool BF16, int DP>
int launch_dq(const AttnArgs& a, const AttnMaps& maps, int sms, cudaStream_t s) {
    using C = CfgQ<DP>;
    auto kernel = k_attn_tc_dq<BF16, DP>;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)C::kSmem) != cudaSuccess)
        return VG_ERR_CUDA;
    const int64_t units = attn_max_tiles(a.n_q, a.batch, a.gp, kM) * (a.hq / a.gp) * a.splits;
    kernel<<<(unsigned)std::min<int64_t>(units, sms), kThreads, C::kSmem, s>>>(a, maps);
    return cudaPeekAtLastError() == cudaSuccess ? VG_OK : VG_ERR_CUDA;
}

template <bool BF16, int DP>
int launch_dkv(const AttnArgs& a, const AttnMaps& maps, float* part_dv, int sms, cudaStream_t s) {
    using C = CfgKV<DP>;
    auto kernel = k_attn_tc_dkv<BF16, DP>;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)C::kSmem) != cudaSuccess)
        return VG_ERR_CUDA;
    const int64_t units = attn_max_tiles(a.n_k, a.batch, 1, kM) * a.hk * a.splits;
    kernel<<<(unsigned)std::min<int64_t>(units, sms), kThreads, C::kSmem, s>>>(a, maps, part_dv);
    return cudaPeekAtLastError() == cudaSuccess ? VG_OK : VG_ERR_CUDA;
}

// Maps of the four operands, in boxes of 128 (packed) rows.
int make_maps(AttnMaps* m, const AttnArgs& a, int dtype) {
    int st = VG_OK;
    if (a.n_q > 0) {
        if ((st = attn_make_map(&m->q, a.q, a.n_q, a.hq, a.d, dtype, a.gp, kM / a.gp)) != VG_OK) return st;
        if ((st = attn_make_map(&m->go, a.go, a.n_q, a.hq, a.d, dtype, a.gp, kM / a.gp)) != VG_OK) return st;
    }
    if (a.n_k > 0) {
        if ((st = attn_make_map(&m->k, a.k, a.n_k, a.hk, a.d, dtype, 1, kM)) != VG_OK) return st;
        st = attn_make_map(&m->v, a.v, a.n_k, a.hk, a.d, dtype, 1, kM);
    }
    return st;
}

}  // namespace

int attn_tc_dq(const AttnArgs& a, int dtype, int sms, cudaStream_t s) {
    AttnMaps m{};
    const int st = make_maps(&m, a, dtype);
    if (st != VG_OK) return st;
    if (dtype == VG_BF16) return a.d <= 64 ? launch_dq<true, 64>(a, m, sms, s) : launch_dq<true, 128>(a, m, sms, s);
    return a.d <= 64 ? launch_dq<false, 64>(a, m, sms, s) : launch_dq<false, 128>(a, m, sms, s);
}

int attn_tc_dkv(const AttnArgs& a, float* part_dv, int dtype, int sms, cudaStream_t s) {
    AttnMaps m{};
    const int st = make_maps(&m, a, dtype);
    if (st != VG_OK) return st;
    if (dtype == VG_BF16)
        return a.d <= 64 ? launch_dkv<true, 64>(a, m, part_dv, sms, s) : launch_dkv<true, 128>(a, m, part_dv, sms, s);
    return a.d <= 64 ? launch_dkv<false, 64>(a, m, part_dv, sms, s) : launch_dkv<false, 128>(a, m, part_dv, sms, s);
}

}  // namespace vg
