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
// dQ: a persistent block takes NQ x 128 packed query rows and runs along the keys in
// tiles of 64.  dK, dV: it takes 128 keys and runs along the packed rows of every query
// head that reads them, 64 at a time, so gradients of shared heads are sums in the same
// accumulators.  Both have groups of four softmax warps (one thread per row of the
// products), a loader warp and an MMA-issuing warp; the 16-bit dS (and P) replaces
// the scores in TMEM and is the next product's first operand.  Two tiles are in flight
// (dQ: the block's two row tiles; dK, dV: two consecutive steps), so one's products
// run while the other's exponentials do.
//
// fp16 has no exponent range to spare: P carries 2^15 (P <= 1), and dP - delta is divided by
// a power of two above 2 max|dO row| max|V row|, which bounds it; both leave with the
// fp32 result.  bf16 needs neither.
#include "attn_tc.cuh"

namespace vg {

namespace {

using namespace attn_tc;

constexpr int kM = 128;  // rows of the products
constexpr int kN = 64;   // columns of a step

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
template <int DP, int NQ>
struct CfgQ {
    static constexpr int kThreads = NQ * 128 + 64;
    static constexpr int kBlocks = DP / 64;
    static constexpr int kRowTile = kM * 128 * kBlocks;    // bytes of a Q or dO tile
    static constexpr int kKeyTile = kN * 128 * kBlocks;    // bytes of a K or V tile
    static constexpr int S = DP == 64 ? 4 : 3;             // ring stages (a K and a V tile each)
    static constexpr int kOCol = NQ * 2 * kN;
    static constexpr int kTmem = NQ * (2 * kN + DP) <= 256 ? 256 : 512;
    static constexpr int kPerSm = NQ == 1 && DP == 64 ? 2 : 1;
    static constexpr int kBars = 2 + 4 * NQ + 2 * S + 1;
    static constexpr size_t kSmem = 1024 + (size_t)2 * NQ * kRowTile + (size_t)2 * S * kKeyTile + 8 * kBars + 16;
};
static_assert(CfgQ<128, 2>::kSmem <= 232448 && 2 * (CfgQ<64, 1>::kSmem + 1024) <= 233472, "shared memory");

template <bool BF16, int DP, int NQ>
__global__ void __launch_bounds__(NQ * 128 + 64, CfgQ<DP, NQ>::kPerSm)
    k_attn_tc_dq(const AttnArgs a, const __grid_constant__ AttnMaps maps, const int tiles) {
    using C = CfgQ<DP, NQ>;
    constexpr int S = C::S;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sQ = smem_u32(smem), sG = sQ + NQ * C::kRowTile, sKV = sG + NQ * C::kRowTile;
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + (size_t)2 * NQ * C::kRowTile + (size_t)2 * S * C::kKeyTile);
    uint32_t* s_tmem = reinterpret_cast<uint32_t*>(bars + C::kBars);
    volatile uint32_t* s_abort = s_tmem + 1;
    const uint32_t bar0 = smem_u32(bars);
    const uint32_t q_full = bar0, q_empty = bar0 + 8;
    const uint32_t s_full = bar0 + 16, p_full = s_full + 8 * NQ, o_full = p_full + 8 * NQ, o_empty = o_full + 8 * NQ;
    const uint32_t kv_full = o_empty + 8 * NQ, kv_empty = kv_full + 8 * S, done = kv_empty + 8 * S;

    const int warp = uniform((int)threadIdx.x >> 5), lane = threadIdx.x & 31;
    constexpr int kLoader = NQ * 4, kIssuer = NQ * 4 + 1;
    if (threadIdx.x == 0) {
        mbar_init(q_full, 1);
        mbar_init(q_empty, 1);
        for (int w = 0; w < NQ; ++w) {
            mbar_init(s_full + 8 * w, 1);
            mbar_init(p_full + 8 * w, 4);
            mbar_init(o_full + 8 * w, 1);
            mbar_init(o_empty + 8 * w, 4);
        }
        for (int i = 0; i < S; ++i) {
            mbar_init(kv_full + 8 * i, 1);
            mbar_init(kv_empty + 8 * i, 1);
        }
        mbar_init(done, 1);
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

    const int sets = a.hq / a.gp;
    const int group = a.hq / a.hk;
    const int64_t units = good ? (int64_t)tiles * sets * a.splits : 0;
    struct Unit {
        AttnTile t;
        int hs, part, lo, hi, rows;
    };
    auto find = [&](int64_t u) {
        Unit x;
        x.t = attn_find_tile<false>(a, NQ * kM, u / sets);
        x.hs = (int)(u % sets);
        x.part = x.t.part;
        x.rows = 0;
        x.lo = x.hi = 0;
        if (x.t.b >= 0) {
            x.rows = min(NQ * kM, x.t.lq * a.gp - x.t.first);
            attn_split(a, x.t.lk, x.part, &x.lo, &x.hi);
        }
        return x;
    };
    Waiter wait{s_abort};

    if (warp == kLoader) {
        uint32_t it = 0, uc = 0;
        for (int64_t u = blockIdx.x; u < units && wait.ok; u += gridDim.x) {
            const Unit x = find(u);
            if (x.hi <= x.lo) continue;
            wait(q_empty, (uc & 1u) ^ 1u);
            if (!wait.ok) break;
            const int nq = x.rows > kM ? NQ : 1;
            one_lane([&] {
                mbar_arrive_expect_tx(q_full, 2 * nq * C::kRowTile);
                for (int w = 0; w < nq; ++w)
                    for (int b = 0; b < C::kBlocks; ++b) {
                        const int row = x.t.q0 + (x.t.first + w * kM) / a.gp;
                        const uint32_t off = w * C::kRowTile + b * kM * 128;
                        tma_load_3d(sQ + off, &maps.q, b * 64, x.hs * a.gp, row, q_full);
                        tma_load_3d(sG + off, &maps.go, b * 64, x.hs * a.gp, row, q_full);
                    }
            });
            ++uc;
            const int kh = x.hs * a.gp / group;
            for (int e = x.lo; e < x.hi; ++e, ++it) {
                const uint32_t st = it % S;
                wait(kv_empty + 8 * st, ((it / S) & 1u) ^ 1u);
                if (!wait.ok) break;
                one_lane([&] {
                    mbar_arrive_expect_tx(kv_full + 8 * st, 2 * C::kKeyTile);
                    for (int b = 0; b < C::kBlocks; ++b) {
                        const uint32_t dst = sKV + 2 * st * C::kKeyTile + b * kN * 128;
                        tma_load_3d(dst, &maps.k, b * 64, kh, x.t.k0 + e * kN, kv_full + 8 * st);
                        tma_load_3d(dst + C::kKeyTile, &maps.v, b * 64, kh, x.t.k0 + e * kN, kv_full + 8 * st);
                    }
                });
            }
        }
        // every copy has landed before the block may exit
        if (uc > 0 && !mbar_wait_timed(q_full, (uc - 1) & 1u)) wait.ok = false;
        for (uint32_t i = 0; i < (uint32_t)S && i < it; ++i) {
            const uint32_t last = it - 1 - i;
            if (!mbar_wait_timed(kv_full + 8 * (last % S), (last / S) & 1u)) wait.ok = false;
        }
        if (!wait.ok && lane == 0) atomicOr(a.err, kErrTimeout);
    } else if (warp == kIssuer) {
        const int ksteps = (a.d + 15) / 16;
        const uint32_t idesc_o = idesc_f16_bn(BF16, ksteps * 16);
        uint32_t it = 0, uc = 0, pc[NQ] = {}, oc[NQ] = {};
        auto scores = [&](int w, uint32_t st, int n) {  // S_w = Q_w K^T and dP_w = dO_w V^T
            const uint32_t id = idesc_f16(BF16, n), d = tmem + w * 2 * kN;
            const uint32_t k = sKV + 2 * st * C::kKeyTile;
            mma_channels<DP / 16, kM * 128, kN * 128>(d, sw128_kmajor_desc(sQ + w * C::kRowTile),
                                                      sw128_kmajor_desc(k), id, ksteps);
            mma_channels<DP / 16, kM * 128, kN * 128>(d + kN, sw128_kmajor_desc(sG + w * C::kRowTile),
                                                      sw128_kmajor_desc(k + C::kKeyTile), id, ksteps);
            mma_commit(s_full + 8 * w);
        };
        for (int64_t u = blockIdx.x; u < units && wait.ok; u += gridDim.x) {
            const Unit x = find(u);
            if (x.hi <= x.lo) continue;
            const int nq = x.rows > kM ? NQ : 1;
            auto left = [&](int e) { return min(kN, x.t.lk - e * kN); };
            auto padded = [&](int e) { return (left(e) + 15) / 16 * 16; };
            // K rows past the sample's keys may hold anything, and 0 x them must be 0 in dS K
            auto arrive = [&](int e, uint32_t i) {
                wait(kv_full + 8 * (i % S), (i / S) & 1u);
                if (wait.ok && padded(e) != left(e)) {
                    zero_rows(sKV + 2 * (i % S) * C::kKeyTile, left(e), padded(e), C::kBlocks, kN * 128);
                    fence_proxy_async_smem();
                    __syncwarp();
                }
            };
            wait(q_full, uc & 1u);
            arrive(x.lo, it);
            if (!wait.ok) break;
            tc_fence_after();
            one_lane([&] {
                for (int w = 0; w < nq; ++w) scores(w, it % S, padded(x.lo));
                if (x.hi - x.lo == 1) mma_commit(q_empty);
            });
            for (int e = x.lo; e < x.hi; ++e, ++it) {
                const uint32_t st = it % S, nx = (it + 1) % S;
                const bool more = e + 1 < x.hi;
                if (more) arrive(e + 1, it + 1);
                const int n16 = padded(e);
                for (int w = 0; w < nq; ++w) {
                    wait(p_full + 8 * w, pc[w]++ & 1u);
                    if (e == x.lo) wait(o_empty + 8 * w, (oc[w] & 1u) ^ 1u);
                    if (!wait.ok) break;
                    tc_fence_after();
                    one_lane([&] {
                        mma_rows<kN / 16>(tmem + C::kOCol + w * DP, tmem + w * 2 * kN,
                                          sw128_mnmajor_desc(sKV + 2 * st * C::kKeyTile, kN * 128), idesc_o, n16 / 16,
                                          e > x.lo);
                        if (more) scores(w, nx, padded(e + 1));
                        else mma_commit(o_full + 8 * w);
                        if (w + 1 == nq) {
                            mma_commit(kv_empty + 8 * st);
                            if (e + 2 == x.hi) mma_commit(q_empty);
                        }
                    });
                    if (!more) ++oc[w];
                }
                if (!wait.ok) break;
            }
            ++uc;
        }
        // every product has finished before TMEM is released
        one_lane([&] { mma_commit(done); });
        if (!mbar_wait_timed(done, 0)) wait.ok = false;
        if (!wait.ok && lane == 0) {
            *s_abort = 1;
            atomicOr(a.err, kErrTimeout);
        }
    } else {
        const int w = warp >> 2, quad = warp & 3;
        const uint32_t t_lane = tmem + ((uint32_t)(quad * 32) << 16);
        const uint32_t t_s = t_lane + w * 2 * kN, t_o = t_lane + C::kOCol + w * DP;
        const float c = a.scale_log2;
        const float2 lift = grad_lift<BF16>(a);
        uint32_t sc = 0, oc = 0;
        for (int64_t u = blockIdx.x; u < units && wait.ok; u += gridDim.x) {
            const Unit x = find(u);
            if (x.rows <= w * kM) continue;
            const int row = w * kM + quad * 32 + lane;
            const bool any = x.rows > w * kM + quad * 32, mine = row < x.rows;
            const int pr = x.t.first + row;
            float2 st = make_float2(0.f, 0.f);
            if (mine) st = a.stats[((int64_t)x.hs * a.n_q + x.t.q0) * a.gp + pr];
            const float base = st.x - kLift<BF16>, delta = st.y * lift.x;
            const float2 c2 = make_float2(c, c), base2 = make_float2(-base, -base);
            const float2 lift2 = make_float2(lift.x, lift.x), delta2 = make_float2(-delta, -delta);
            for (int e = x.lo; e < x.hi; ++e) {
                wait(s_full + 8 * w, sc & 1u);
                if (!wait.ok) break;
                ++sc;
                tc_fence_after();
                if (any) {
                    uint32_t s[2][32], g[2][32];
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        tmem_ld32(t_s + 32 * i, s[i]);
                        tmem_ld32(t_s + kN + 32 * i, g[i]);
                    }
                    tmem_ld_wait();
#pragma unroll
                    for (int i = 0; i < 2; ++i) tmem_ld_done(s[i]), tmem_ld_done(g[i]);
                    const int left = x.t.lk - e * kN;
                    uint32_t d[32];
#pragma unroll
                    for (int j = 0; j < 32; ++j) {
                        const int r = j >> 4, i = 2 * (j & 15);
                        float2 p = fma2(two(&s[r][i]), c2, base2);
                        p = make_float2(ex2(p.x), ex2(p.y));
                        float2 ds = BF16 ? add2(two(&g[r][i]), delta2) : fma2(two(&g[r][i]), lift2, delta2);
                        ds = mul2(p, ds);
                        if (2 * j >= left) ds.x = 0.f;
                        if (2 * j + 1 >= left) ds.y = 0.f;
                        d[j] = pack2<BF16>(ds.x, ds.y);
                    }
                    tmem_st32(t_s, d);
                    tmem_st_wait();
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(p_full + 8 * w);
            }
            if (x.hi > x.lo) {
                wait(o_full + 8 * w, oc & 1u);
                if (!wait.ok) break;
                ++oc;
                tc_fence_after();
            }
            if (any) {
                const int64_t qi = x.t.q0 + pr / a.gp;
                const int h = x.hs * a.gp + pr % a.gp;
                const float mul = a.scale * kDrop<BF16> * lift.y;
                float* dst_p = a.part + (((size_t)x.part * a.n_q + qi) * a.hq + h) * a.d;
                uint16_t* dst = head_row<uint16_t>(a.gq, qi, h);
#pragma unroll
                for (int i = 0; i < DP / 32; ++i) {
                    if (32 * i >= a.d) break;
                    uint32_t o[32];
                    if (x.hi > x.lo) {
                        tmem_ld32(t_o + 32 * i, o);
                        tmem_ld_wait();
                        tmem_ld_done(o);
                    } else {
#pragma unroll
                        for (int j = 0; j < 32; ++j) o[j] = 0u;
                    }
                    if (mine) {
                        if (a.splits > 1) store_cols32_f32(dst_p + 32 * i, o, mul, a.d - 32 * i);
                        else store_cols32<BF16>(dst + 32 * i, o, mul, a.d - 32 * i);
                    }
                    __syncwarp();
                }
            }
            if (x.hi > x.lo) {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(o_empty + 8 * w);
            }
        }
        if (!wait.ok && lane == 0) atomicOr(a.err, kErrTimeout);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kIssuer) tmem_dealloc(tmem, C::kTmem);
}

// ================================================================ key and value gradients
constexpr int kThreadsKV = 2 * 128 + 64;

template <int DP>
struct CfgKV {
    static constexpr int kBlocks = DP / 64;
    static constexpr int kKeyTile = kM * 128 * kBlocks;  // bytes of the K or V tile
    static constexpr int kRowTile = kN * 128 * kBlocks;  // bytes of a Q or dO step
    static constexpr int S = 4;                          // ring stages (a Q and a dO step each)
    static constexpr int kVCol = 4 * kN, kKCol = kVCol + DP;
    static constexpr int kTmem = 512;
    // key tiles full, empty; S full x 2, P full x 2; gradients full, empty; ring full, empty; done
    static constexpr int kBars = 2 + 4 + 2 + 2 * S + 1;
    static constexpr size_t kStats = 8 * 2 * kN * sizeof(float2);  // eight warps, two steps each
    static constexpr size_t kSmem = 1024 + 2 * kKeyTile + (size_t)2 * S * kRowTile + kStats + 8 * kBars + 16;
};
static_assert(CfgKV<128>::kSmem <= 232448 && CfgKV<128>::kKCol + 128 <= 512, "shared memory, TMEM");

template <bool BF16, int DP>
__global__ void __launch_bounds__(kThreadsKV, 1)
    k_attn_tc_dkv(const AttnArgs a, const __grid_constant__ AttnMaps maps, const int tiles, float* part_dv) {
    using C = CfgKV<DP>;
    constexpr int S = C::S;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sK = smem_u32(smem), sV = sK + C::kKeyTile, sQG = sV + C::kKeyTile;
    float2* s_stats = reinterpret_cast<float2*>(smem + 2 * C::kKeyTile + (size_t)2 * S * C::kRowTile);
    uint64_t* bars = reinterpret_cast<uint64_t*>(s_stats + 16 * kN);
    uint32_t* s_tmem = reinterpret_cast<uint32_t*>(bars + C::kBars);
    volatile uint32_t* s_abort = s_tmem + 1;
    const uint32_t bar0 = smem_u32(bars);
    const uint32_t k_full = bar0, k_empty = bar0 + 8, s_full = bar0 + 16, p_full = bar0 + 32;
    const uint32_t o_full = bar0 + 48, o_empty = bar0 + 56, r_full = bar0 + 64, r_empty = r_full + 8 * S;
    const uint32_t done = r_empty + 8 * S;

    const int warp = uniform((int)threadIdx.x >> 5), lane = threadIdx.x & 31;
    constexpr int kLoader = 8, kIssuer = 9;
    if (threadIdx.x == 0) {
        mbar_init(k_full, 1);
        mbar_init(k_empty, 1);
        for (int w = 0; w < 2; ++w) {
            mbar_init(s_full + 8 * w, 1);
            mbar_init(p_full + 8 * w, 4);
        }
        mbar_init(o_full, 1);
        mbar_init(o_empty, 8);
        for (int i = 0; i < S; ++i) {
            mbar_init(r_full + 8 * i, 1);
            mbar_init(r_empty + 8 * i, 1);
        }
        mbar_init(done, 1);
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

    const int sets_per_key = a.hq / a.hk / a.gp;  // head sets that read a key head
    const int64_t units = good ? (int64_t)tiles * a.hk * a.splits : 0;
    // unit u = (part, key head, key tile); its steps run over (head set, row tile in [lo, hi))
    struct Unit {
        AttnTile t;
        int kh, part, lo, hi, steps;
    };
    auto find = [&](int64_t u) {
        Unit x;
        x.t = attn_find_tile<true>(a, kM, u / a.hk);
        x.kh = (int)(u % a.hk);
        x.part = x.t.part;
        x.lo = x.hi = 0;
        if (x.t.b >= 0 && x.t.first < x.t.lk) attn_split(a, (int64_t)x.t.lq * a.gp, x.part, &x.lo, &x.hi);
        x.steps = (x.hi - x.lo) * sets_per_key;
        return x;
    };
    Waiter wait{s_abort};

    if (warp == kLoader) {
        uint32_t it = 0, uc = 0;
        for (int64_t u = blockIdx.x; u < units && wait.ok; u += gridDim.x) {
            const Unit x = find(u);
            if (x.steps == 0) continue;
            wait(k_empty, (uc & 1u) ^ 1u);
            if (!wait.ok) break;
            one_lane([&] {
                mbar_arrive_expect_tx(k_full, 2 * C::kKeyTile);
                for (int b = 0; b < C::kBlocks; ++b) {
                    tma_load_3d(sK + b * kM * 128, &maps.k, b * 64, x.kh, x.t.k0 + x.t.first, k_full);
                    tma_load_3d(sV + b * kM * 128, &maps.v, b * 64, x.kh, x.t.k0 + x.t.first, k_full);
                }
            });
            ++uc;
            for (int hs = 0; hs < sets_per_key && wait.ok; ++hs)
                for (int e = x.lo; e < x.hi; ++e, ++it) {
                    const uint32_t st = it % S;
                    wait(r_empty + 8 * st, ((it / S) & 1u) ^ 1u);
                    if (!wait.ok) break;
                    const int head = (x.kh * sets_per_key + hs) * a.gp, row = x.t.q0 + e * kN / a.gp;
                    one_lane([&] {
                        mbar_arrive_expect_tx(r_full + 8 * st, 2 * C::kRowTile);
                        for (int b = 0; b < C::kBlocks; ++b) {
                            const uint32_t dst = sQG + 2 * st * C::kRowTile + b * kN * 128;
                            tma_load_3d(dst, &maps.q, b * 64, head, row, r_full + 8 * st);
                            tma_load_3d(dst + C::kRowTile, &maps.go, b * 64, head, row, r_full + 8 * st);
                        }
                    });
                }
        }
        // every copy has landed before the block may exit
        if (uc > 0 && !mbar_wait_timed(k_full, (uc - 1) & 1u)) wait.ok = false;
        for (uint32_t i = 0; i < (uint32_t)S && i < it; ++i) {
            const uint32_t last = it - 1 - i;
            if (!mbar_wait_timed(r_full + 8 * (last % S), (last / S) & 1u)) wait.ok = false;
        }
        if (!wait.ok && lane == 0) atomicOr(a.err, kErrTimeout);
    } else if (warp == kIssuer) {
        const int ksteps = (a.d + 15) / 16;
        const uint32_t idesc_o = idesc_f16_bn(BF16, ksteps * 16);
        uint32_t it = 0, uc = 0, pc[2] = {0, 0};
        // steps alternate between the two score buffers across units too: step i of the block uses i & 1
        auto scores = [&](uint32_t i, int n) {  // S^T = K Q^T and dP^T = V dO^T of step i
            const uint32_t id = idesc_f16(BF16, n), st = i % S, w = i & 1u, d = tmem + w * 2 * kN;
            const uint32_t q = sQG + 2 * st * C::kRowTile;
            mma_channels<DP / 16, kM * 128, kN * 128>(d, sw128_kmajor_desc(sK), sw128_kmajor_desc(q), id, ksteps);
            mma_channels<DP / 16, kM * 128, kN * 128>(d + kN, sw128_kmajor_desc(sV),
                                                      sw128_kmajor_desc(q + C::kRowTile), id, ksteps);
            mma_commit(s_full + 8 * w);
        };
        for (int64_t u = blockIdx.x; u < units && wait.ok; u += gridDim.x) {
            const Unit x = find(u);
            if (x.steps == 0) continue;
            const int rows = x.t.lq * a.gp, per = x.hi - x.lo;
            auto left = [&](int i) { return min(kN, rows - (x.lo + i % per) * kN); };  // rows of step i of the unit
            auto padded = [&](int i) { return (left(i) + 15) / 16 * 16; };
            // the last rows of a step may be the next sample's, and 0 x them must be 0 in dS^T Q and P^T dO
            auto arrive = [&](int i, uint32_t n) {
                wait(r_full + 8 * (n % S), (n / S) & 1u);
                if (wait.ok && padded(i) != left(i)) {
                    const uint32_t q = sQG + 2 * (n % S) * C::kRowTile;
                    zero_rows(q, left(i), padded(i), C::kBlocks, kN * 128);
                    zero_rows(q + C::kRowTile, left(i), padded(i), C::kBlocks, kN * 128);
                    fence_proxy_async_smem();
                    __syncwarp();
                }
            };
            wait(k_full, uc & 1u);
            for (int i = 0; i < 2 && i < x.steps; ++i) {
                arrive(i, it + i);
                if (!wait.ok) break;
                tc_fence_after();
                one_lane([&] {
                    scores(it + i, padded(i));
                    if (x.steps <= 2 && i + 1 == x.steps) mma_commit(k_empty);
                });
            }
            if (!wait.ok) break;
            wait(o_empty, (uc & 1u) ^ 1u);
            for (int i = 0; i < x.steps; ++i, ++it) {
                const uint32_t st = it % S, w = it & 1u;
                const uint32_t q = sQG + 2 * st * C::kRowTile, g = q + C::kRowTile;
                const int n16 = padded(i);
                if (i + 2 < x.steps) arrive(i + 2, it + 2);
                wait(p_full + 8 * w, pc[w]++ & 1u);
                if (!wait.ok) break;
                tc_fence_after();
                const uint32_t pt = tmem + w * 2 * kN;
                one_lane([&] {
                    mma_rows<kN / 16>(tmem + C::kVCol, pt, sw128_mnmajor_desc(g, kN * 128), idesc_o, n16 / 16, i > 0);
                    mma_rows<kN / 16>(tmem + C::kKCol, pt + kN, sw128_mnmajor_desc(q, kN * 128), idesc_o, n16 / 16,
                                      i > 0);
                    mma_commit(r_empty + 8 * st);
                    if (i + 2 < x.steps) scores(it + 2, padded(i + 2));
                    if (i + 3 == x.steps) mma_commit(k_empty);
                    if (i + 1 == x.steps) mma_commit(o_full);
                });
            }
            ++uc;
        }
        // every product has finished before TMEM is released
        one_lane([&] { mma_commit(done); });
        if (!mbar_wait_timed(done, 0)) wait.ok = false;
        if (!wait.ok && lane == 0) {
            *s_abort = 1;
            atomicOr(a.err, kErrTimeout);
        }
    } else {
        const int w = warp >> 2, quad = warp & 3;
        const uint32_t t_lane = tmem + ((uint32_t)(quad * 32) << 16);
        const uint32_t t_s = t_lane + w * 2 * kN;
        const float c = a.scale_log2;
        const float2 lift = grad_lift<BF16>(a);
        const float2 c2 = make_float2(c, c), lift2 = make_float2(lift.x, lift.x);
        float2* my_stats = s_stats + warp * 2 * kN;
        uint32_t it = 0, sc = 0, uc = 0;
        for (int64_t u = blockIdx.x; u < units && wait.ok; u += gridDim.x) {
            const Unit x = find(u);
            if (x.t.b < 0) continue;
            const int rows = x.t.lq * a.gp, per = x.hi - x.lo;
            // statistics (lse log2 e, delta) of rows lane and lane + 32 of step i, kept negated, a copy per warp
            auto stat = [&](int i, int r0) {
                float2 v = make_float2(0.f, 0.f);
                if (i < x.steps) {
                    const int hs = x.kh * sets_per_key + i / per, r = (x.lo + i % per) * kN + r0 + lane;
                    if (r < rows) v = a.stats[((int64_t)hs * a.n_q + x.t.q0) * a.gp + r];
                }
                return v;
            };
            int i = (int)((w ^ it) & 1u);  // this group's first step of the unit
            float2 next0 = stat(i, 0), next1 = stat(i, 32);
            for (; i < x.steps; i += 2) {
                float2* cur = my_stats + (sc & 1u) * kN;
                cur[lane] = make_float2(kLift<BF16> - next0.x, -next0.y * lift.x);
                cur[lane + 32] = make_float2(kLift<BF16> - next1.x, -next1.y * lift.x);
                __syncwarp();
                next0 = stat(i + 2, 0);
                next1 = stat(i + 2, 32);
                wait(s_full + 8 * w, sc & 1u);
                if (!wait.ok) break;
                ++sc;
                tc_fence_after();
                const int left = rows - (x.lo + i % per) * kN;
#pragma unroll 1
                for (int half = 0; half < 2; ++half) {
                    uint32_t s[32], g[32], p[16], d[16];
                    tmem_ld32(t_s + 32 * half, s);
                    tmem_ld32(t_s + kN + 32 * half, g);
                    tmem_ld_wait();
                    tmem_ld_done(s);
                    tmem_ld_done(g);
#pragma unroll
                    for (int j = 0; j < 16; ++j) {
                        const float4 st = *reinterpret_cast<const float4*>(cur + 32 * half + 2 * j);
                        float2 pr = fma2(two(s + 2 * j), c2, make_float2(st.x, st.z));
                        pr = make_float2(ex2(pr.x), ex2(pr.y));
                        const float2 minus = make_float2(st.y, st.w);
                        float2 ds = BF16 ? add2(two(g + 2 * j), minus) : fma2(two(g + 2 * j), lift2, minus);
                        ds = mul2(pr, ds);
                        if (32 * half + 2 * j >= left) pr.x = ds.x = 0.f;
                        if (32 * half + 2 * j + 1 >= left) pr.y = ds.y = 0.f;
                        p[j] = pack2<BF16>(pr.x, pr.y);
                        d[j] = pack2<BF16>(ds.x, ds.y);
                    }
                    tmem_st16(t_s + 16 * half, p);
                    tmem_st16(t_s + kN + 16 * half, d);
                }
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(p_full + 8 * w);
            }
            it += x.steps;
            if (x.steps > 0) {
                wait(o_full, uc & 1u);
                if (!wait.ok) break;
                ++uc;
                tc_fence_after();
            }
            // group 0 writes dV, group 1 dK
            const int r = x.t.first + quad * 32 + lane;
            const bool mine = r < x.t.krows, live = r < x.t.lk && x.steps > 0;
            const int64_t row = x.t.k0 + r;
            const float mul = w == 0 ? kDrop<BF16> : a.scale * kDrop<BF16> * lift.y;
            float* dst_p = (w == 0 ? part_dv : a.part) + (((size_t)x.part * a.n_k + row) * a.hk + x.kh) * a.d;
            uint16_t* dst = head_row<uint16_t>(w == 0 ? a.gv : a.gk, row, x.kh);
#pragma unroll
            for (int i2 = 0; i2 < DP / 32; ++i2) {
                if (32 * i2 >= a.d) break;
                uint32_t o[32];
                if (x.steps > 0) {
                    tmem_ld32(t_lane + (w == 0 ? C::kVCol : C::kKCol) + 32 * i2, o);
                    tmem_ld_wait();
                    tmem_ld_done(o);
                }
                if (!live)
#pragma unroll
                    for (int j = 0; j < 32; ++j) o[j] = 0u;
                if (mine) {
                    if (a.splits > 1) store_cols32_f32(dst_p + 32 * i2, o, mul, a.d - 32 * i2);
                    else store_cols32<BF16>(dst + 32 * i2, o, mul, a.d - 32 * i2);
                }
                __syncwarp();
            }
            if (x.steps > 0) {
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

template <bool BF16, int DP, int NQ>
int launch_dq(const AttnArgs& a, const AttnMaps& maps, int sms, cudaStream_t s) {
    using C = CfgQ<DP, NQ>;
    auto kernel = k_attn_tc_dq<BF16, DP, NQ>;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)C::kSmem) != cudaSuccess)
        return VG_ERR_CUDA;
    const int64_t tiles = attn_max_tiles(a.n_q, a.batch, a.gp, NQ * kM);
    const int64_t units = tiles * (a.hq / a.gp) * a.splits;
    const int64_t grid = std::min<int64_t>(units, (int64_t)sms * C::kPerSm);
    kernel<<<(unsigned)grid, C::kThreads, C::kSmem, s>>>(a, maps, (int)tiles);
    return cudaPeekAtLastError() == cudaSuccess ? VG_OK : VG_ERR_CUDA;
}

template <bool BF16, int DP>
int launch_dkv(const AttnArgs& a, const AttnMaps& maps, float* part_dv, int sms, cudaStream_t s) {
    using C = CfgKV<DP>;
    auto kernel = k_attn_tc_dkv<BF16, DP>;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)C::kSmem) != cudaSuccess)
        return VG_ERR_CUDA;
    const int64_t tiles = attn_max_tiles(a.n_k, a.batch, 1, kM);
    const int64_t units = tiles * a.hk * a.splits;
    kernel<<<(unsigned)std::min<int64_t>(units, sms), kThreadsKV, C::kSmem, s>>>(a, maps, (int)tiles, part_dv);
    return cudaPeekAtLastError() == cudaSuccess ? VG_OK : VG_ERR_CUDA;
}

// Maps of the four operands: queries' boxes of `qrows` packed rows, keys' of `krows`.
int make_maps(AttnMaps* m, const AttnArgs& a, int dtype, int qrows, int krows) {
    int st = VG_OK;
    if (a.n_q > 0) {
        if ((st = attn_make_map(&m->q, a.q, a.n_q, a.hq, a.d, dtype, a.gp, qrows / a.gp)) != VG_OK) return st;
        if ((st = attn_make_map(&m->go, a.go, a.n_q, a.hq, a.d, dtype, a.gp, qrows / a.gp)) != VG_OK) return st;
    }
    if (a.n_k > 0) {
        if ((st = attn_make_map(&m->k, a.k, a.n_k, a.hk, a.d, dtype, 1, krows)) != VG_OK) return st;
        st = attn_make_map(&m->v, a.v, a.n_k, a.hk, a.d, dtype, 1, krows);
    }
    return st;
}

}  // namespace

int attn_tc_dq(const AttnArgs& a, int dtype, int nq, int sms, cudaStream_t s) {
    AttnMaps m{};
    const int st = make_maps(&m, a, dtype, kM, kN);
    if (st != VG_OK) return st;
    if (dtype == VG_BF16) {
        if (a.d <= 64) return nq == 2 ? launch_dq<true, 64, 2>(a, m, sms, s) : launch_dq<true, 64, 1>(a, m, sms, s);
        return nq == 2 ? launch_dq<true, 128, 2>(a, m, sms, s) : launch_dq<true, 128, 1>(a, m, sms, s);
    }
    if (a.d <= 64) return nq == 2 ? launch_dq<false, 64, 2>(a, m, sms, s) : launch_dq<false, 64, 1>(a, m, sms, s);
    return nq == 2 ? launch_dq<false, 128, 2>(a, m, sms, s) : launch_dq<false, 128, 1>(a, m, sms, s);
}

int attn_tc_dkv(const AttnArgs& a, float* part_dv, int dtype, int sms, cudaStream_t s) {
    AttnMaps m{};
    const int st = make_maps(&m, a, dtype, kN, kM);
    if (st != VG_OK) return st;
    if (dtype == VG_BF16)
        return a.d <= 64 ? launch_dkv<true, 64>(a, m, part_dv, sms, s) : launch_dkv<true, 128>(a, m, part_dv, sms, s);
    return a.d <= 64 ? launch_dkv<false, 64>(a, m, part_dv, sms, s) : launch_dkv<false, 128>(a, m, part_dv, sms, s);
}

}  // namespace vg
