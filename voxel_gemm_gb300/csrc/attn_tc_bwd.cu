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
// reads them, 64 at a time, so gradients of shared heads are sums in the same accumulators.
// Both have softmax warps, one warp that loads with TMA, one that finds the block's next
// units, and two that issue the products: one S and dP, the other one the gradients.
//   dQ        16 softmax warps, four threads per row, 32 columns each
//   dK, dV    two groups of four, one thread per row, each group every second step
// The 16-bit dS (and P) go to TMEM columns of their own, as first operands of the gradient
// products: the next S and dP are computed while this tile's exponentials are.  dK, dV with
// d > 64 has no columns left: there they lie over the scores, and one warp issues all.
// dQ's tiles are 128 wide because a product of two shared-memory operands runs at the tensor
// cores' rate only from N = 128 on: at N = 64 it takes 48 cycles instead of 32 to read its
// operands.
//
// delta is the sum of dO O, with O as the caller has it, rounded to 16 bits.  Where many keys
// share the weight that is exact enough (O is an average, small beside V), over few it is not:
// over five keys it adds as much to dQ's error as the rounding of dS.  So a sample of at most
// one tile of keys gets delta as the row's sum of P dP, which the dQ kernel has in registers
// there; it hands it to the dK, dV kernel too.  A row over more keys that gives nearly all of
// its weight to a few has the larger error: half an ulp of |dO| |O| in delta, which P weighs.
// (Its sum of P dP would take a second pass over the keys.)
//
// Bound by the exponentials' warps and the hand-overs to and from the issuers (the products
// alone would take half the time).  100,003 queries over 2 x 1,370 keys, 16 heads of 64,
// bf16: dQ 692 us (1.2 PFLOP/s), dK and dV 1090 us (1.0 PFLOP/s); fp16: 758 and 1109; the scores' columns for
// P and dS at d = 64 too, 1540 and later 1196 us; 128-wide steps with 16 warps, 1117 us.
//
// fp16 has no exponent range to spare: P carries 2^15 (P <= 1), and dP - delta is divided by
// a power of two above 2 |dO row| max|V row|, which bounds it; both leave with the fp32 result.
// V's rows are the sample's; dO's is the row itself in dQ, the sample's largest in dK, whose sums run
// over rows.  So nothing in one sample, however large, takes range from another's, nor one
// row from another one's dQ.  bf16 needs neither.
#include "attn_tc.cuh"

namespace vg {

namespace {

using namespace attn_tc;

constexpr int kM = 128;  // rows of the products
constexpr int kN = 128;  // columns of dQ's steps
constexpr int kH = 32;   // columns of its softmax threads
constexpr int kThreads = 512 + 128;

// The power of two that dP - delta is multiplied by where |dO row| <= go, and its inverse.
template <bool BF16>
__device__ __forceinline__ float2 grad_lift(const Unit& x, float go) {
    if constexpr (BF16) return make_float2(1.f, 1.f);
    const float bound = 2.f * go * __uint_as_float(x.max_v);
    const int e = (int)(__float_as_uint(bound) >> 23) - 127;
    if (!(bound > 0.f) || e > 120 || e < -120) return make_float2(1.f, 1.f);
    return make_float2(__uint_as_float((uint32_t)(126 - e) << 23), __uint_as_float((uint32_t)(128 + e) << 23));
}

// The norms that the bounds come from, of sample b.
template <bool BF16>
__device__ __forceinline__ void put_bounds(const AttnArgs& a, int b, Unit& x) {
    if constexpr (!BF16) x.max_go = a.bound[2 * b], x.max_v = a.bound[2 * b + 1];
}

template <bool BF16> constexpr float kDrop = BF16 ? 1.f : 1.f / (1 << (int)kHalfLift);  // what P carries, taken out

// ================================================================ query gradient
template <int DP>
struct CfgQ {
    static constexpr int kBlocks = DP / 64;
    static constexpr int kTile = kM * 128 * kBlocks;       // bytes of a Q, dO, K or V tile
    static constexpr int S = DP == 64 ? 4 : 2;             // ring stages (a K and a V tile each)
    static constexpr int kOCol = 2 * kN, kPCol = kOCol + DP;  // dQ's and dS's first TMEM column
    // q, s, p and o (full, empty), (kv full, kv empty) x S, tail, done x 2, unit ring, exchanges x 4
    static constexpr int kBars = 8 + 2 * S + 3 + 2 * kUnitSlots + 4;
    static constexpr size_t kSums = 2 * 4 * kM * sizeof(float);  // two exchanges between the threads of a row
    static constexpr size_t kSmem =
        1024 + (size_t)(2 + 2 * S) * kTile + kSums + kUnitSlots * sizeof(Unit) + 8 * kBars + 16;
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
    float* s_sums = reinterpret_cast<float*>(smem + (size_t)(2 + 2 * S) * C::kTile);
    int4* s_units = reinterpret_cast<int4*>(s_sums + 2 * 4 * kM);
    uint64_t* bars = reinterpret_cast<uint64_t*>(s_units + 3 * kUnitSlots);
    uint32_t* s_tmem = reinterpret_cast<uint32_t*>(bars + C::kBars);
    volatile uint32_t* s_abort = s_tmem + 1;
    const uint32_t bar0 = smem_u32(bars);
    const uint32_t q_full = bar0, q_empty = bar0 + 8, s_full = bar0 + 16, s_empty = bar0 + 24, p_full = bar0 + 32;
    const uint32_t p_empty = bar0 + 40, o_full = bar0 + 48, o_empty = bar0 + 56;
    const uint32_t kv_full = bar0 + 64, kv_empty = kv_full + 8 * S, tail = kv_empty + 8 * S;
    const uint32_t done = tail + 8, u_full = done + 16, u_empty = u_full + 8 * kUnitSlots;
    const uint32_t summed = u_empty + 8 * kUnitSlots;

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
        for (int i = 0; i < 4; ++i) mbar_init(summed + 8 * i, 4);
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
    UnitRing ring{s_units, u_full, u_empty, a};
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
            put_bounds<BF16>(a, t.b, x);
            ring.put(wait, x);
        }
        x.rows = -1;
        ring.put(wait, x);
    } else if (warp == kLoader) {
        RingPos<S> pos;
        Copies<1> qs, tails;  // tiles that end the sample's keys land on the tail's barrier
        Copies<S> kvs;
        while (ring.get(wait, x)) {
            if (x.hi <= x.lo) continue;
            wait(q_empty, (qs.n & 1u) ^ 1u);
            if (!wait.ok) break;
            const int kh = x.head * a.gp / group, row = x.q0 + (x.first >> a.gp_log2);
            one_lane([&] {
                mbar_arrive_expect_tx(q_full, 2 * C::kTile);
                for (int b = 0; b < C::kBlocks; ++b) {
                    tma_load_3d(sQ + b * kM * 128, &maps.q, b * 64, x.head * a.gp, row, q_full);
                    tma_load_3d(sG + b * kM * 128, &maps.go, b * 64, x.head * a.gp, row, q_full);
                }
            });
            qs.issued();
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
                    tails.issued();
                    wait(tail, (tails.n - 1) & 1u);
                    zero_rows(k, left, n16, C::kBlocks, kN * 128);
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(kv_full + 8 * pos.i);
                    __syncwarp();
                }
                kvs.issued();
                pos.step();
            }
        }
        // every copy has landed before the block may exit
        wait.ok &= land(qs, q_full);
        wait.ok &= land(kvs, kv_full);
        wait.ok &= land(tails, tail);
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
        const bool v8ok = lines_ok(a.gq);
        const int row = quad * 32 + lane;  // within the unit
        uint32_t n = 0, uc = 0, sums = 0;  // tiles, units and exchanges done
        while (ring.get(wait, x)) {
            const bool any = x.rows > quad * 32, mine = row < x.rows;  // the warp, the thread has a row
            const int pr = x.first + row;                              // packed row of the sample
            const int64_t at = ((int64_t)x.head * a.n_q + x.q0) * a.gp + pr;
            const float2 st = mine ? attn_stats(a, at) : make_float2(0.f, 0.f);
            const float2 lift = grad_lift<BF16>(x, !BF16 && mine ? a.stats[2 * a.n_q * a.hq + at] : 0.f);
            const float base = st.x, delta = st.y * lift.x;
            const float2 c2 = make_float2(c, c), base2 = make_float2(base, base);
            const float2 lift2 = make_float2(lift.x, lift.x), delta2 = make_float2(delta, delta);
            if (x.lk <= kN && x.lo < x.hi && any) {  // the one tile of a sample
                if (!wait(s_full, n & 1u)) break;
                tc_fence_after();
                uint32_t s[kH], g[kH];
                tmem_ld32(t_s, s);
                tmem_ld32(t_s + kN, g);
                tmem_ld_wait();
                tmem_ld_done(s);
                tmem_ld_done(g);
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(s_empty);
                float w[kH], sum = 0.f;
                const int left = x.lk - quarter * kH;
#pragma unroll
                for (int i = 0; i < kH; ++i) {
                    const float dp = i < left ? __uint_as_float(g[i]) : 0.f;
                    w[i] = i < left ? ex2(fmaf(__uint_as_float(s[i]), c, base)) : 0.f;
                    sum = fmaf(w[i], dp, sum);
                    g[i] = __float_as_uint(dp);
                }
                // delta, to all threads of the row
                float* slot = s_sums + (sums & 1u) * 4 * kM + row;
                slot[quarter * kM] = sum;
                __syncwarp();
                if (lane == 0) mbar_arrive(summed + 8 * quad);
                if (!wait(summed + 8 * quad, sums++ & 1u)) break;
                sum = -kDrop<BF16> * (slot[0] + slot[kM] + (slot[2 * kM] + slot[3 * kM]));
                if (mine && quarter == 0)
                    a.stats[a.n_q * a.hq + at] = sum;
                if (n > 0 && !wait(p_empty, (n - 1) & 1u)) break;
                tc_fence_after();
                uint32_t d[kH / 2];
#pragma unroll
                for (int i = 0; i < kH / 2; ++i) {
                    const float d0 = w[2 * i] * ((__uint_as_float(g[2 * i]) + sum) * lift.x);
                    const float d1 = w[2 * i + 1] * ((__uint_as_float(g[2 * i + 1]) + sum) * lift.x);
                    d[i] = pack2<BF16>(d0, d1);
                }
                tmem_st16(t_p, d);
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(p_full);
                ++n;
            } else {
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
                        // columns from there on are not scores: weight 0, gradient 0
                        const int left = x.lk - e * kN - quarter * kH;
                        if (left < kH) {
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
constexpr int kNK = 64;  // rows of a step
constexpr int kThreadsKV = 2 * 128 + 128;

template <int DP>
struct CfgKV {
    static constexpr int kBlocks = DP / 64;
    static constexpr int kKeyTile = kM * 128 * kBlocks;  // bytes of the K or V tile
    static constexpr int kRowTile = kNK * 128 * kBlocks;  // bytes of a Q or dO step
    static constexpr int S = DP == 64 ? 8 : 4;           // ring stages (a Q and a dO step each)
    static constexpr int kVCol = 4 * kNK, kKCol = kVCol + DP;
    // P and dS in columns of their own where there is room (d <= 64), else over the scores
    static constexpr bool kOwn = DP == 64;
    static constexpr int kPCol = kKCol + DP;
    static constexpr int kTmem = 512;
    // key tiles full, empty; (S full, S empty, P full, P empty) x 2; gradients full, empty; (ring full, empty) x S;
    // tail; done; unit ring
    static constexpr int kBars = 2 + 8 + 2 + 2 * S + 3 + 2 * kUnitSlots;
    static constexpr size_t kStats = S * 2 * kNK * sizeof(float);  // two numbers per row of a ring stage
    static constexpr size_t kSmem = 1024 + 2 * kKeyTile + (size_t)2 * S * kRowTile + kStats +
                                    kUnitSlots * sizeof(Unit) + 8 * kBars + 16;
    static constexpr int kSoft = 200, kAux = 104;
    static_assert(256 * kSoft + 128 * kAux <= kThreadsKV * 168, "register split");
};
static_assert((CfgKV<64>::S & (CfgKV<64>::S - 1)) == 0 && (CfgKV<128>::S & (CfgKV<128>::S - 1)) == 0, "ring stages");
static_assert(CfgKV<128>::kSmem <= 232448 && CfgKV<64>::kSmem <= 232448 && CfgKV<128>::kKCol + 128 <= 512,
              "shared memory, TMEM");

template <bool BF16, int DP>
__global__ void __launch_bounds__(kThreadsKV, 1)
    k_attn_tc_dkv(const AttnArgs a, const __grid_constant__ AttnMaps maps, float* part_dv) {
    using C = CfgKV<DP>;
    constexpr int S = C::S;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sK = smem_u32(smem), sV = sK + C::kKeyTile, sQG = sV + C::kKeyTile;
    float* s_stats = reinterpret_cast<float*>(smem + 2 * C::kKeyTile + (size_t)2 * S * C::kRowTile);
    int4* s_units = reinterpret_cast<int4*>(s_stats + S * 2 * kNK);
    uint64_t* bars = reinterpret_cast<uint64_t*>(s_units + 3 * kUnitSlots);
    uint32_t* s_tmem = reinterpret_cast<uint32_t*>(bars + C::kBars);
    volatile uint32_t* s_abort = s_tmem + 1;
    const uint32_t bar0 = smem_u32(bars);
    const uint32_t k_full = bar0, k_empty = bar0 + 8, s_full = bar0 + 16, p_full = bar0 + 32;
    const uint32_t s_empty = bar0 + 48, p_empty = bar0 + 64, o_full = bar0 + 80, o_empty = bar0 + 88;
    const uint32_t r_full = bar0 + 96, r_empty = r_full + 8 * S;
    const uint32_t tail = r_empty + 8 * S, done = tail + 8, u_full = done + 16, u_empty = u_full + 8 * kUnitSlots;

    const int warp = uniform((int)threadIdx.x >> 5), lane = threadIdx.x & 31;
    constexpr int kLoader = 8, kIssuer = 9, kIssuer2 = 10, kScheduler = 11;
    if (threadIdx.x == 0) {
        mbar_init(k_full, 1);
        mbar_init(k_empty, 1);
        for (int w = 0; w < 2; ++w) {
            mbar_init(s_full + 8 * w, 1);
            mbar_init(p_full + 8 * w, 4);
            mbar_init(s_empty + 8 * w, 4);
            mbar_init(p_empty + 8 * w, 1);
        }
        mbar_init(o_full, 1);
        mbar_init(o_empty, 8);
        for (int i = 0; i < S; ++i) {
            mbar_init(r_full + 8 * i, 1 + 32);  // the tiles, and each lane's statistics
            mbar_init(r_empty + 8 * i, 1);
        }
        for (int i = 0; i < kUnitSlots; ++i) {
            mbar_init(u_full + 8 * i, 1);
            mbar_init(u_empty + 8 * i, 8 + 2 + C::kOwn);  // every reader: softmax warps, loader, issuers
        }
        mbar_init(tail, 1);
        mbar_init(done, 1);
        mbar_init(done + 8, 1);
        *s_abort = 0;
        fence_mbar_init();
    }
    if (warp == kIssuer) {
        tmem_alloc(smem_u32(s_tmem), C::kTmem);
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
    const int64_t plane = a.n_q * a.hq;   // from a row's first statistic to its second
    // A unit is (part and key tile, key head): rows = key rows of the tile, valid or not, [lo, hi) its row tiles of
    // each head set.  Its steps run over (head set, row tile).
    Waiter wait{s_abort};
    UnitRing ring{s_units, u_full, u_empty, a};
    Unit x;
    if (warp >= kLoader) reg_shrink<C::kAux>();
    if (warp == kScheduler) {
        for (int64_t u = blockIdx.x; good && wait.ok; u += gridDim.x) {
            const AttnTile t = attn_find_tile<true>(a, kM, u / a.hk);
            if (t.b < 0) break;
            x = Unit{t.first, min(kM, t.krows - t.first), (int)(u % a.hk), t.part, 0, 0, t.q0, t.lq, t.k0, t.lk, 0, 0};
            if (t.first < t.lk) attn_split(a, (int64_t)t.lq * a.gp, t.part, &x.lo, &x.hi);
            put_bounds<BF16>(a, t.b, x);
            ring.put(wait, x);
        }
        x.rows = -1;
        ring.put(wait, x);
    } else if (warp == kLoader) {
        RingPos<S> pos;
        Copies<1> keys, tails;  // row tiles that end the sample's queries land on the tail's barrier
        Copies<S> steps;
        while (ring.get(wait, x)) {
            if (x.hi <= x.lo) continue;
            wait(k_empty, (keys.n & 1u) ^ 1u);
            if (!wait.ok) break;
            one_lane([&] {
                mbar_arrive_expect_tx(k_full, 2 * C::kKeyTile);
                for (int b = 0; b < C::kBlocks; ++b) {
                    tma_load_3d(sK + b * kM * 128, &maps.k, b * 64, x.head, x.k0 + x.first, k_full);
                    tma_load_3d(sV + b * kM * 128, &maps.v, b * 64, x.head, x.k0 + x.first, k_full);
                }
            });
            keys.issued();
            for (int hs = 0; hs < sets && wait.ok; ++hs)
                for (int e = x.lo; e < x.hi; ++e) {
                    const uint32_t q = sQG + 2 * pos.i * C::kRowTile;
                    wait(r_empty + 8 * pos.i, pos.phase ^ 1u);
                    if (!wait.ok) break;
                    const int left = min(kNK, x.lq * a.gp - e * kNK), n16 = (left + 15) / 16 * 16;
                    const uint32_t bar = n16 != left ? tail : r_full + 8 * pos.i;
                    const int head = (x.head * sets + hs) * a.gp, row = x.q0 + ((e * kNK) >> a.gp_log2);
                    one_lane([&] {
                        mbar_arrive_expect_tx(bar, 2 * C::kRowTile);
                        for (int b = 0; b < C::kBlocks; ++b) {
                            tma_load_3d(q + b * kNK * 128, &maps.q, b * 64, head, row, bar);
                            tma_load_3d(q + C::kRowTile + b * kNK * 128, &maps.go, b * 64, head, row, bar);
                        }
                    });
                    const float* st = a.stats + ((int64_t)(x.head * sets + hs) * a.n_q + x.q0) * a.gp + e * kNK;
                    const uint32_t to = smem_u32(s_stats + pos.i * 2 * kNK);
                    for (int r = lane; r < kNK; r += 32) {  // rows past the sample: 0
                        const bool in = r < left;
                        cp_async4(to + 4 * r, in ? st + r : a.stats, in ? 4 : 0);
                        cp_async4(to + 4 * (kNK + r), in ? st + plane + r : a.stats, in ? 4 : 0);
                    }
                    cp_async_arrive_noinc(r_full + 8 * pos.i);
                    __syncwarp();
                    if (n16 != left) {  // rows of the next sample: 0 x them must be 0 in dS^T Q and P^T dO
                        tails.issued();
                        wait(tail, (tails.n - 1) & 1u);
                        zero_rows(q, left, n16, C::kBlocks, kNK * 128);
                        zero_rows(q + C::kRowTile, left, n16, C::kBlocks, kNK * 128);
                        fence_proxy_async_smem();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(r_full + 8 * pos.i);
                        __syncwarp();
                    }
                    steps.issued();
                    pos.step();
                }
        }
        // every copy has landed before the block may exit
        wait.ok &= land(keys, k_full);
        wait.ok &= land(steps, r_full);
        wait.ok &= land(tails, tail);
        cp_async_wait_all();  // the statistics of a step whose tiles never landed
        if (!wait.ok && lane == 0) atomicOr(a.err, kErrTimeout);
    } else if (warp == kIssuer || (C::kOwn && warp == kIssuer2)) {
        const int ksteps = (a.d + 15) / 16;
        const uint32_t idesc_s = idesc_f16(BF16, kNK), idesc_o = idesc_f16_bn(BF16, ksteps * 16);
        const uint64_t dk = sw128_kmajor_desc(sK), dv = sw128_kmajor_desc(sV), dq = sw128_kmajor_desc(sQG);
        const uint64_t dqt = sw128_mnmajor_desc(sQG, kNK * 128);
        constexpr uint32_t kStage = 2 * C::kRowTile >> 4, kSecond = C::kRowTile >> 4;  // to the next stage, to dO
        RingPos<S> ahead, pos;                // of the scores, two steps ahead, and of the gradients
        uint32_t uc = 0, it = 0;              // it: steps of the block; step `it` uses score buffer it & 1
        while (ring.get(wait, x)) {
            if (x.hi <= x.lo) continue;
            const int per = x.hi - x.lo, steps = per * sets;
            const int rest = min(kNK, x.lq * a.gp - (x.hi - 1) * kNK), last16 = (rest + 15) / 16;
            by_one_lane(wait, [&](LaneWaiter& w) {
                RingPos<S> ra = ahead, rg = pos;
                uint32_t na = it, ng = it;    // steps of the block: of the next scores, of the next gradients
                int ea = 0, eg = 0;           // their row tiles (from lo)
                // S^T = K Q^T and dP^T = V dO^T of the next step
                auto scores = [&](bool last) {
                    const uint32_t id = ea + 1 == per ? idesc_f16(BF16, last16 * 16) : idesc_s, b = na++ & 1u;
                    const uint32_t d = tmem + b * 2 * kNK;
                    const uint64_t q = dq + ra.i * kStage;
                    mma_channels<DP / 16, kM * 128, kNK * 128>(d, dk, q, id, ksteps);
                    mma_channels<DP / 16, kM * 128, kNK * 128>(d + kNK, dv, q + kSecond, id, ksteps);
                    mma_commit(s_full + 8 * b);
                    if (last) mma_commit(k_empty);
                    ra.step();
                    if (++ea == per) ea = 0;
                };
                if (!C::kOwn || warp == kIssuer) {
                    w(k_full, uc & 1u);
                    for (int i = 0; i < (C::kOwn ? steps : min(2, steps)); ++i) {
                        w(r_full + 8 * ra.i, ra.phase);
                        if (C::kOwn) w(s_empty + 8 * (na & 1u), ((na >> 1) & 1u) ^ 1u);  // the last ones have been read
                        if (!w.ok) return;
                        tc_fence_after();
                        scores(i + 1 == steps);
                    }
                }
                if (C::kOwn && warp == kIssuer) return;
                w(o_empty, (uc & 1u) ^ 1u);
                for (int i = 0; i < steps; ++i, ++ng) {
                    const uint32_t b = ng & 1u, sw = tmem + b * 2 * kNK;
                    const uint32_t pt = C::kOwn ? tmem + C::kPCol + b * kNK : sw;
                    const uint32_t st = C::kOwn ? pt + kNK / 2 : sw + kNK;
                    const bool more = !C::kOwn && i + 2 < steps;
                    const int n16 = eg + 1 == per ? last16 : kNK / 16;
                    if (C::kOwn) w(r_full + 8 * rg.i, rg.phase);
                    if (more) w(r_full + 8 * ra.i, ra.phase);
                    if (!w(p_full + 8 * b, (ng >> 1) & 1u)) return;
                    tc_fence_after();
                    const uint64_t q = dqt + rg.i * kStage;
                    mma_rows<kNK / 16>(tmem + C::kVCol, pt, q + kSecond, idesc_o, n16, i > 0);
                    mma_rows<kNK / 16>(tmem + C::kKCol, st, q, idesc_o, n16, i > 0);
                    mma_commit(r_empty + 8 * rg.i);
                    if (C::kOwn) mma_commit(p_empty + 8 * b);
                    if (more) scores(i + 3 == steps);
                    if (i + 1 == steps) mma_commit(o_full);
                    rg.step();
                    if (++eg == per) eg = 0;
                }
            });
            if (!wait.ok) break;
            ahead.skip(steps);
            pos.skip(steps);
            it += steps;
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
        reg_grow<C::kSoft>();
        const int w = warp >> 2, quad = warp & 3;
        const uint32_t t_lane = tmem + ((uint32_t)(quad * 32) << 16);
        const uint32_t t_s = t_lane + w * 2 * kNK;
        const float c = a.scale_log2;
        const float2 c2 = make_float2(c, c);
        const bool v8ok = lines_ok(w == 0 ? a.gv : a.gk);
        const uint32_t t_p = C::kOwn ? t_lane + C::kPCol + w * kNK : t_s, t_d = C::kOwn ? t_p + kNK / 2 : t_s + kNK;
        uint32_t it = 0, sc = 0, uc = 0;
        while (ring.get(wait, x)) {
            const int rows = x.lq * a.gp, per = x.hi - x.lo, steps = per * sets;
            const float2 lift = grad_lift<BF16>(x, __uint_as_float(x.max_go)), lift2 = make_float2(lift.x, lift.x);
            // this group's steps of the unit: every second one
            int i = (int)((w ^ it) & 1u), e = x.lo + (per == 1 ? 0 : i);
            for (; i < steps; i += 2) {
                const int left = rows - e * kNK;
                for (e += 2; e >= x.hi; e -= per) {}
                const uint32_t stage = (it + i) & (S - 1);
                const float* cur = s_stats + stage * 2 * kNK;
                if (!wait(s_full + 8 * w, sc & 1u)) break;
                wait(r_full + 8 * stage, (it + i) / S & 1u);  // the statistics: the scores waited for it as well
                ++sc;
                tc_fence_after();
                uint32_t s[2][32], g[2][32], p[32], d[32];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    tmem_ld32(t_s + 32 * h, s[h]);
                    tmem_ld32(t_s + kNK + 32 * h, g[h]);
                }
                tmem_ld_wait();
#pragma unroll
                for (int h = 0; h < 2; ++h) tmem_ld_done(s[h]), tmem_ld_done(g[h]);
                if (left < kNK) {  // columns from there on are no rows of the sample: weight 0, gradient 0
#pragma unroll
                    for (int j = 0; j < kNK; ++j)
                        if (j >= left) s[j >> 5][j & 31] = 0xff800000u, g[j >> 5][j & 31] = 0u;
                }
                if (C::kOwn) {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(s_empty + 8 * w);
                }
#pragma unroll
                for (int j = 0; j < 32; j += 2) {
                    const float4 lse = *reinterpret_cast<const float4*>(cur + 2 * j);
                    const float4 del = *reinterpret_cast<const float4*>(cur + kNK + 2 * j);
#pragma unroll
                    for (int t = 0; t < 2; ++t) {
                        const int h = (j + t) >> 4, k = 2 * ((j + t) & 15);
                        const float2 base = t == 0 ? make_float2(lse.x, lse.y) : make_float2(lse.z, lse.w);
                        float2 pr = fma2(two(&s[h][k]), c2, base);
                        pr = make_float2(ex2(pr.x), ex2(pr.y));
                        const float2 minus = t == 0 ? make_float2(del.x, del.y) : make_float2(del.z, del.w);
                        const float2 dp = two(&g[h][k]);
                        float2 ds = add2(dp, minus);
                        if (!BF16) ds = mul2(ds, lift2);
                        ds = mul2(pr, ds);
                        p[j + t] = pack2<BF16>(pr.x, pr.y);
                        d[j + t] = pack2<BF16>(ds.x, ds.y);
                    }
                }
                if (C::kOwn && sc > 1) {  // the products that read the buffer's last P and dS have finished
                    if (!wait(p_empty + 8 * w, sc & 1u)) break;
                    tc_fence_after();
                }
                tmem_st32(t_p, p);
                tmem_st32(t_d, d);
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(p_full + 8 * w);
            }
            it += steps;
            if (steps > 0) {
                if (!wait(o_full, uc & 1u)) break;
                ++uc;
                tc_fence_after();
            }
            // group 0 writes dV, group 1 dK; key rows past the valid ones get zeros
            const int r = quad * 32 + lane;
            const int64_t row = x.k0 + x.first + r;
            const float mul = w == 0 ? kDrop<BF16> : a.scale * kDrop<BF16> * lift.y;
            float* dst_p = (w == 0 ? part_dv : a.part) + (((size_t)x.part * a.n_k + row) * a.hk + x.head) * a.d;
            store_row<BF16, DP>(a, steps > 0, t_lane + (w == 0 ? C::kVCol : C::kKCol), mul, r < x.rows && wait.ok,
                                head_row<uint16_t>(w == 0 ? a.gv : a.gk, row, x.head), dst_p, lane, v8ok,
                                x.first + r < x.lk);
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
    if (warp == kIssuer) tmem_dealloc(tmem, C::kTmem);
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
    kernel<<<(unsigned)std::min<int64_t>(units, sms), kThreadsKV, C::kSmem, s>>>(a, maps, part_dv);
    return cudaPeekAtLastError() == cudaSuccess ? VG_OK : VG_ERR_CUDA;
}

// Maps of the four operands; queries in boxes of `qrows` packed rows.
int make_maps(AttnMaps* m, const AttnArgs& a, int dtype, int qrows) {
    int st = VG_OK;
    if (a.n_q > 0) {
        if ((st = attn_make_map(&m->q, a.q, a.n_q, a.hq, a.d, dtype, a.gp, qrows / a.gp)) != VG_OK) return st;
        if ((st = attn_make_map(&m->go, a.go, a.n_q, a.hq, a.d, dtype, a.gp, qrows / a.gp)) != VG_OK) return st;
    }
    if (a.n_k > 0) {
        if ((st = attn_make_map(&m->k, a.k, a.n_k, a.hk, a.d, dtype, 1, kM)) != VG_OK) return st;
        st = attn_make_map(&m->v, a.v, a.n_k, a.hk, a.d, dtype, 1, kM);
    }
    return st;
}

}  // namespace

int attn_tc_dq(AttnArgs a, int dtype, int sms, cudaStream_t s) {
    AttnMaps m{};
    a.unit_cycles = unit_wait_cycles(unit_steps(a.splits, a.per_part, a.n_k, kN, 1));
    const int st = make_maps(&m, a, dtype, kM);
    if (st != VG_OK) return st;
    if (dtype == VG_BF16) return a.d <= 64 ? launch_dq<true, 64>(a, m, sms, s) : launch_dq<true, 128>(a, m, sms, s);
    return a.d <= 64 ? launch_dq<false, 64>(a, m, sms, s) : launch_dq<false, 128>(a, m, sms, s);
}

int attn_tc_dkv(AttnArgs a, float* part_dv, int dtype, int sms, cudaStream_t s) {
    AttnMaps m{};
    a.unit_cycles = unit_wait_cycles(unit_steps(a.splits, a.per_part, a.n_q * a.gp, kNK, a.hq / a.hk / a.gp));
    const int st = make_maps(&m, a, dtype, kNK);
    if (st != VG_OK) return st;
    if (dtype == VG_BF16)
        return a.d <= 64 ? launch_dkv<true, 64>(a, m, part_dv, sms, s) : launch_dkv<true, 128>(a, m, part_dv, sms, s);
    return a.d <= 64 ? launch_dkv<false, 64>(a, m, part_dv, sms, s) : launch_dkv<false, 128>(a, m, part_dv, sms, s);
}

}  // namespace vg
