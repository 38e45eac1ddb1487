// Cross attention forward on the tensor cores (tcgen05 / TMEM), 16-bit types.
//
//   S = Q K^T, m = running row maximum, P = exp2(c S - c m), l = running sum of P,
//   O = (sum over tiles of P V) / l, lse = scale m + ln l          (c = scale log2 e)
//
// A persistent block takes units of NQ x 128 packed query rows of one sample and head
// set, and runs along the sample's keys in tiles of 128:
//   warps 0 .. 4 NQ - 1  softmax: one thread per row.  Reads its 128 scores from TMEM,
//                        writes P as 16-bit pairs over them, and at the end scales and
//                        stores its row of O.
//   then one warp        loader: TMA copies of Q (per unit) and of K and V tiles (a ring).
//   then one warp        issues the products: S into TMEM, then O += P V with P read from
//                        TMEM, then the next S over P.
//   then one warp        scheduler: finds the block's next units.
//   one idle warp        fills the last warpgroup, whose registers go to the softmax warps.
// With NQ = 2 the two row tiles take turns: one's products run while the other's
// exponentials do, and both read each K and V tile from the same copy.  NQ = 1 leaves
// room for two blocks on an SM and serves calls with few rows per sample.
//
// The row maximum only keeps the weights in range, and O and l carry the same factor
// whatever it is.  So it is taken from the first tile and kept: later tiles are weighed
// with it right away, and only where a row's sum of weights over a tile leaves the range (2^32 in
// bf16, so that products with values of up to 2^90 stay inside fp32's range; 2^14 in fp16) are
// the maximum renewed, O (in TMEM) and l rescaled and the tile weighed again.  P is rounded to
// the inputs' type for the second product (l sums the unrounded values); fp16 weights carry a
// factor 2^7 more, so that a weight down to 2^-31 of the row's largest is not lost below fp16's
// range.
//
// Bound by the exponentials' warps, of which an SM holds eight: they take some 1,200 cycles
// for a tile's weights and wait some 700 for the next scores, which lie in the same columns
// and so come after the product with V (scores beside the weights' own columns took that
// wait away and made the warps slower by as much: 622 us against 601 at the time; four threads
// to a row in 16 warps, 1361; all of a row's weights stored at once in place of each half
// when it is done, 571).  100,003 queries over 2 x 1,370 keys, 16 heads of 64, bf16: 573 us
// (0.98 PFLOP/s); 25,179 over 4 x 1,024, 16 heads of 128, fp16: 118 us (1.2 PFLOP/s).
// 2 queries over 2 x 159,528 keys: 97 us, 6.7 TB/s, the memory's rate.
#include "attn_tc.cuh"

namespace vg {

namespace {

using namespace attn_tc;

constexpr int kM = 128;   // rows of an MMA tile
constexpr int kN = 128;   // keys of a tile

template <int DP, int NQ>
struct Cfg {
    static constexpr int kSoftWarps = NQ * 4;
    static constexpr int kThreads = 32 * kSoftWarps + 128;
    static constexpr int kBlocks = DP / 64;
    static constexpr int kTile = kM * 128 * kBlocks;       // bytes of a Q, K or V tile
    static constexpr int S = DP == 64 && NQ == 2 ? 5 : 2;  // ring stages, a K and a V tile each
    static constexpr int kPerSm = DP == 64 && NQ == 1 ? 2 : 1;
    static constexpr int kOCol = NQ * kN;                   // O's first TMEM column
    static constexpr int kTmem = NQ * 256;
    // q full, q empty, (s full, p full, o full, o empty) x NQ, (k full, v full, k empty, v empty) x S, tail, done,
    // unit ring
    static constexpr int kBars = 2 + 4 * NQ + 4 * S + 2 + 2 * kUnitSlots;
    static constexpr size_t kSmem = 1024 + (size_t)(NQ + 2 * S) * kTile + kUnitSlots * sizeof(Unit) + 8 * kBars + 16;
    // registers: launched with kRegs a thread; the softmax warps take what the last warpgroup gives up
    static constexpr int kRegs = NQ == 2 ? 168 : 128, kSoft = NQ == 2 ? 200 : 184, kAux = NQ == 2 ? 104 : 72;
    static_assert(32 * kSoftWarps * kSoft + 128 * kAux <= kThreads * kRegs, "register split");
};
static_assert(Cfg<128, 2>::kSmem <= 232448 && 2 * (Cfg<64, 1>::kSmem + 1024) <= 233472 &&
                  Cfg<128, 1>::kSmem <= 232448, "shared memory");

template <bool BF16, int DP, int NQ>
__global__ void __launch_bounds__(Cfg<DP, NQ>::kThreads, Cfg<DP, NQ>::kPerSm)
    k_attn_tc_fwd(const AttnArgs a, const __grid_constant__ AttnMaps maps) {
    using C = Cfg<DP, NQ>;
    constexpr int S = C::S;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sQ = smem_u32(smem), sKV = sQ + NQ * C::kTile;
    int4* s_units = reinterpret_cast<int4*>(smem + (size_t)(NQ + 2 * S) * C::kTile);
    uint64_t* bars = reinterpret_cast<uint64_t*>(s_units + 3 * kUnitSlots);
    uint32_t* s_tmem = reinterpret_cast<uint32_t*>(bars + C::kBars);
    volatile uint32_t* s_abort = s_tmem + 1;
    const uint32_t bar0 = smem_u32(bars);
    const uint32_t q_full = bar0, q_empty = bar0 + 8;
    const uint32_t s_full = bar0 + 16, p_full = s_full + 8 * NQ, o_full = p_full + 8 * NQ, o_empty = o_full + 8 * NQ;
    const uint32_t k_full = o_empty + 8 * NQ, v_full = k_full + 8 * S, k_empty = v_full + 8 * S;
    const uint32_t v_empty = k_empty + 8 * S, tail = v_empty + 8 * S;
    const uint32_t done = tail + 8, u_full = done + 8, u_empty = u_full + 8 * kUnitSlots;

    const int warp = uniform((int)threadIdx.x >> 5), lane = threadIdx.x & 31;
    constexpr int kLoader = C::kSoftWarps, kIssuer = kLoader + 1, kScheduler = kLoader + 2;
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
            mbar_init(k_full + 8 * i, 1);
            mbar_init(v_full + 8 * i, 1);
            mbar_init(k_empty + 8 * i, 1);
            mbar_init(v_empty + 8 * i, 1);
        }
        for (int i = 0; i < kUnitSlots; ++i) {
            mbar_init(u_full + 8 * i, 1);
            mbar_init(u_empty + 8 * i, C::kSoftWarps + 2);  // every reader: softmax warps, loader, issuer
        }
        mbar_init(tail, 1);
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
    }
    tc_fence_before();
    const bool good = attn_offsets_ok(a);  // a barrier of the whole block
    tc_fence_after();
    const uint32_t tmem = uniform(*s_tmem);

    const int group = a.hq / a.hk;
    Waiter wait{s_abort};
    UnitRing ring{s_units, u_full, u_empty, a};
    Unit x;
    if (warp >= kLoader) reg_shrink<C::kAux>();
    if (warp == kScheduler) {
        // unit u = (row tile and part, head set): its rows and its key tiles [lo, hi)
        const int sets = a.hq / a.gp;
        for (int64_t u = blockIdx.x; good && wait.ok; u += gridDim.x) {
            const AttnTile t = attn_find_tile<false>(a, NQ * kM, u / sets);
            if (t.b < 0) break;
            x = Unit{t.first, min(NQ * kM, t.lq * a.gp - t.first), (int)(u % sets), t.part, 0, 0,
                     t.q0, t.lq, t.k0, t.lk, 0, 0};
            attn_split(a, t.lk, t.part, &x.lo, &x.hi);
            ring.put(wait, x);
        }
        x.rows = -1;
        ring.put(wait, x);
    } else if (warp == kLoader) {
        Copies<1> qs, tails;  // V tiles that end the sample's keys land on the tail's barrier
        Copies<S> ks, vs;
        while (ring.get(wait, x)) {
            if (x.hi <= x.lo) continue;
            wait(q_empty, (qs.n & 1u) ^ 1u);
            if (!wait.ok) break;
            const int nq = x.rows > kM ? NQ : 1, kh = x.head * a.gp / group;
            one_lane([&] {
                mbar_arrive_expect_tx(q_full, nq * C::kTile);
                for (int w = 0; w < nq; ++w)
                    for (int b = 0; b < C::kBlocks; ++b)
                        tma_load_3d(sQ + w * C::kTile + b * kM * 128, &maps.q, b * 64, x.head * a.gp,
                                    x.q0 + ((x.first + w * kM) >> a.gp_log2), q_full);
            });
            qs.issued();
            for (int e = x.lo; e < x.hi; ++e) {
                const uint32_t at = ks.slot(), parity = ks.pass() ^ 1u;
                const uint32_t k = sKV + 2 * at * C::kTile, v = k + C::kTile;
                wait(k_empty + 8 * at, parity);
                if (!wait.ok) break;
                one_lane([&] {
                    mbar_arrive_expect_tx(k_full + 8 * at, C::kTile);
                    for (int b = 0; b < C::kBlocks; ++b)
                        tma_load_3d(k + b * kN * 128, &maps.k, b * 64, kh, x.k0 + e * kN, k_full + 8 * at);
                });
                ks.issued();
                wait(v_empty + 8 * at, parity);
                if (!wait.ok) break;
                const int left = min(kN, x.lk - e * kN), n16 = (left + 15) / 16 * 16;
                const uint32_t bar = n16 != left ? tail : v_full + 8 * at;
                one_lane([&] {
                    mbar_arrive_expect_tx(bar, C::kTile);
                    for (int b = 0; b < C::kBlocks; ++b)
                        tma_load_3d(v + b * kN * 128, &maps.v, b * 64, kh, x.k0 + e * kN, bar);
                });
                if (n16 != left) {  // V rows past the sample's keys may hold anything: 0 x them must be 0 in P V
                    tails.issued();
                    wait(tail, (tails.n - 1) & 1u);
                    zero_rows(v, left, n16, C::kBlocks, kN * 128);
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(v_full + 8 * at);
                    __syncwarp();
                }
                vs.issued();
            }
        }
        // every copy has landed before the block may exit
        wait.ok &= land(qs, q_full);
        wait.ok &= land(ks, k_full);
        wait.ok &= land(vs, v_full);
        wait.ok &= land(tails, tail);
        if (!wait.ok && lane == 0) atomicOr(a.err, kErrTimeout);
    } else if (warp == kIssuer) {
        const int ksteps = (a.d + 15) / 16;          // K = 16 steps over the channels
        const uint32_t idesc_s = idesc_f16(BF16, kN), idesc_o = idesc_f16_bn(BF16, ksteps * 16);
        const uint64_t dq = sw128_kmajor_desc(sQ), dk = sw128_kmajor_desc(sKV);
        const uint64_t dv = sw128_mnmajor_desc(sKV + C::kTile, kN * 128);
        RingPos<S> pos;
        uint32_t uc = 0, pc[NQ] = {}, oc[NQ] = {};
        while (ring.get(wait, x)) {
            if (x.hi <= x.lo) continue;
            const bool both = NQ == 2 && x.rows > kM;
            const int last16 = (min(kN, x.lk - (x.hi - 1) * kN) + 15) / 16;   // K = 16 steps of the last tile
            // S_w = Q_w K^T of the stage at `at`
            auto scores = [&](auto wc, uint32_t at, bool last) {
                constexpr int w = decltype(wc)::value;
                mma_channels<DP / 16, kM * 128, kN * 128>(tmem + w * kN, dq + w * (C::kTile >> 4),
                                                          dk + at * (2 * C::kTile >> 4),
                                                          last ? idesc_f16(BF16, last16 * 16) : idesc_s, ksteps);
                mma_commit(s_full + 8 * w);
            };
            // O_w += P_w V of tile e in the stage at `at`, then the next scores, over P's columns
            auto values = [&](auto wc, int e, uint32_t at, uint32_t next, bool final) {
                constexpr int w = decltype(wc)::value;
                const bool more = e + 1 < x.hi;
                if (e == x.lo) wait(o_empty + 8 * w, (oc[w]++ & 1u) ^ 1u);
                if (!wait(p_full + 8 * w, pc[w]++ & 1u)) return;
                tc_fence_after();
                one_lane([&] {
                    mma_rows<kN / 16>(tmem + C::kOCol + w * DP, tmem + w * kN, dv + at * (2 * C::kTile >> 4), idesc_o,
                                      more ? kN / 16 : last16, e > x.lo);
                    if (more) scores(wc, next, e + 2 == x.hi);
                    else mma_commit(o_full + 8 * w);
                    if (final) {
                        mma_commit(v_empty + 8 * at);
                        if (more) mma_commit(k_empty + 8 * next);
                        if (e + 2 == x.hi) mma_commit(q_empty);
                    }
                });
            };
            const Const<0> first;
            const Const<NQ - 1> second;
            const bool single = x.hi - x.lo == 1;
            wait(q_full, uc & 1u);
            wait(k_full + 8 * pos.i, pos.phase);
            if (!wait.ok) break;
            tc_fence_after();
            one_lane([&] {
                scores(first, pos.i, single);
                if (both) scores(second, pos.i, single);
                mma_commit(k_empty + 8 * pos.i);
                if (single) mma_commit(q_empty);
            });
            for (int e = x.lo; e < x.hi && wait.ok; ++e) {
                const uint32_t at = pos.i;
                wait(v_full + 8 * at, pos.phase);
                pos.step();
                if (e + 1 < x.hi) wait(k_full + 8 * pos.i, pos.phase);
                values(first, e, at, pos.i, !both);
                if (both) values(second, e, at, pos.i, true);
            }
            if (!wait.ok) break;
            ++uc;
        }
        // every product has finished before TMEM is released
        one_lane([&] { mma_commit(done); });
        if (!mbar_wait_timed(done, 0)) wait.ok = false;
        if (!wait.ok && lane == 0) {
            *s_abort = 1;
            atomicOr(a.err, kErrTimeout);
        }
    } else if (warp < kLoader) {
        reg_grow<C::kSoft>();
        const int w = warp >> 2, quad = warp & 3;
        const uint32_t t_lane = tmem + ((uint32_t)(quad * 32) << 16);
        const uint32_t t_s = t_lane + w * kN, t_o = t_lane + C::kOCol + w * DP;
        const float c = a.scale_log2;
        constexpr float kLift = BF16 ? 0.f : 7.f;            // exponent added to the weights
        constexpr float kMost = BF16 ? 0x1p32f : 0x1p14f;    // of a tile's sum before the maximum is replaced
        const bool v8ok = lines_ok(a.o);
        const int row = w * kM + quad * 32 + lane;           // within the unit
        uint32_t sc = 0, oc = 0;
        while (ring.get(wait, x)) {
            if (x.rows <= w * kM) continue;
            const bool any = x.rows > w * kM + quad * 32, mine = row < x.rows;  // the warp, the thread has a row
            float m = -INFINITY, l = 0.f;
            for (int e = x.lo; e < x.hi; ++e) {
                if (!wait(s_full + 8 * w, sc++ & 1u)) break;
                tc_fence_after();
                if (any) {
                    const int left = x.lk - e * kN;                   // valid keys of the tile
                    uint32_t s[kN / 32][32], p[kN / 64][32];
                    float sum;
                    auto load = [&] {
#pragma unroll
                        for (int i = 0; i < kN / 32; ++i) tmem_ld32(t_s + 32 * i, s[i]);
                        tmem_ld_wait();
#pragma unroll
                        for (int i = 0; i < kN / 32; ++i) tmem_ld_done(s[i]);
                        if (left < kN) {
#pragma unroll
                            for (int i = 0; i < kN; ++i)
                                if (i >= left) s[i >> 5][i & 31] = 0xff800000u;
                        }
                    };
                    auto weights = [&] {
                        const float base = kLift - (m == -INFINITY ? 0.f : m * c);
                        const float2 c2 = make_float2(c, c), base2 = make_float2(base, base);
                        float2 acc[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
                        for (int j = 0; j < kN / 2; ++j) {
                            float2 x2 = fma2(two(&s[j >> 4][2 * (j & 15)]), c2, base2);
                            x2 = make_float2(ex2(x2.x), ex2(x2.y));
                            acc[j & 1] = add2(acc[j & 1], x2);
                            p[j >> 5][j & 31] = pack2<BF16>(x2.x, x2.y);
                        }
                        const float2 both = add2(acc[0], acc[1]);
                        sum = both.x + both.y;
                    };
                    auto renew_max = [&](bool rescale) {
                        float top[kN / 32];
#pragma unroll
                        for (int i = 0; i < kN / 32; ++i) {
                            top[i] = fmaxf(__uint_as_float(s[i][0]), __uint_as_float(s[i][1]));
#pragma unroll
                            for (int j = 2; j < 32; j += 2)
                                top[i] = max3(top[i], __uint_as_float(s[i][j]), __uint_as_float(s[i][j + 1]));
                        }
                        const float next = fmaxf(m, fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])));
                        const float f = next == m ? 1.f : ex2((m - next) * c);
                        m = next;
                        l *= f;
                        if (rescale) {  // O holds the earlier tiles' sum, whose products have finished
#pragma unroll 1
                            for (int i = 0; i < DP / 16; ++i) {
                                uint32_t o[16];
                                const uint32_t at = t_o + 16 * i;
                                tmem_ld16(at, o);
                                tmem_ld_wait();
                                tmem_ld_done(o);
#pragma unroll
                                for (int j = 0; j < 16; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * f);
                                tmem_st16(at, o);
                            }
                        }
                    };
                    // a second pass only where the maximum has to be renewed (P is not yet over the scores)
                    for (bool renew = e == x.lo;; renew = true) {
                        load();
                        if (renew) renew_max(e > x.lo);
                        weights();
                        if (renew || !__any_sync(0xffffffffu, mine && (!(sum <= kMost) || m == -INFINITY))) break;
                    }
                    l += sum;
#pragma unroll
                    for (int i = 0; i < kN / 64; ++i) tmem_st32(t_s + 32 * i, p[i]);
                    tmem_st_wait();
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(p_full + 8 * w);
            }
            if (x.hi > x.lo) {
                if (!wait(o_full + 8 * w, oc++ & 1u)) break;
                tc_fence_after();
            }
            if (any) {
                const bool store = mine && wait.ok;
                const int pr = x.first + row;                       // packed row of the sample
                const int64_t qi = x.q0 + (pr >> a.gp_log2);
                const int h = x.head * a.gp + (pr & (a.gp - 1));
                // a part of weight zero has no sum to be normalised by
                const float inv = x.hi <= x.lo ? 0.f : a.splits > 1 && l == 0.f ? 1.f : 1.f / l;
                const float lse = x.hi > x.lo ? (m * c + (log2f(l) - kLift)) * kLn2 : -INFINITY;
                float* dst_l = a.splits > 1 ? a.part_lse + (size_t)x.part * a.hq * a.n_q : a.lse;
                if (store && dst_l) dst_l[(int64_t)h * a.n_q + qi] = lse;
                store_row<BF16, DP>(a, x.hi > x.lo, t_o, inv, store, head_row<uint16_t>(a.o, qi, h),
                                    a.part + (((size_t)x.part * a.n_q + qi) * a.hq + h) * a.d, lane, v8ok);
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

template <bool BF16, int DP, int NQ>
int launch(const AttnArgs& a, const AttnMaps& maps, int sms, cudaStream_t s) {
    using C = Cfg<DP, NQ>;
    auto kernel = k_attn_tc_fwd<BF16, DP, NQ>;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)C::kSmem) != cudaSuccess)
        return VG_ERR_CUDA;
    const int64_t units = attn_max_tiles(a.n_q, a.batch, a.gp, NQ * kM) * (a.hq / a.gp) * a.splits;
    const int64_t grid = std::min<int64_t>(units, (int64_t)sms * C::kPerSm);
    kernel<<<(unsigned)grid, C::kThreads, C::kSmem, s>>>(a, maps);
    return cudaPeekAtLastError() == cudaSuccess ? VG_OK : VG_ERR_CUDA;
}

}  // namespace

int attn_make_map(CUtensorMap* map, const vg_heads& h, int64_t rows, int heads, int d, int dtype, int box_heads,
                  int box_rows) {
    using Encode = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
    static const Encode encode = [] {
        void* f = nullptr;
        cudaDriverEntryPointQueryResult r;
        const cudaError_t e =
            cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &r);
        return e == cudaSuccess && r == cudaDriverEntryPointSuccess ? reinterpret_cast<Encode>(f) : nullptr;
    }();
    if (!encode) return VG_ERR_CUDA;
    const cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)heads, (cuuint64_t)rows};
    // the stride of an axis of one element is never used, but has to be a valid one
    const int64_t hs = heads > 1 ? h.head_stride : d, rs = rows > 1 ? h.row_stride : (int64_t)d * heads;
    const cuuint64_t strides[2] = {(cuuint64_t)hs * 2, (cuuint64_t)rs * 2};
    const cuuint32_t box[3] = {64, (cuuint32_t)box_heads, (cuuint32_t)box_rows}, ones[3] = {1, 1, 1};
    const auto type = dtype == VG_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
    const CUresult r = encode(map, type, 3, h.data, dims, strides, box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
                              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? VG_OK : VG_ERR_UNSUPPORTED;
}

int attn_tc_fwd(AttnArgs a, int dtype, int nq, int sms, cudaStream_t s) {
    AttnMaps maps{};
    a.unit_cycles = unit_wait_cycles(unit_steps(a.splits, a.per_part, a.n_k, kN, 1));
    int st = attn_make_map(&maps.q, a.q, a.n_q, a.hq, a.d, dtype, a.gp, kM / a.gp);
    if (st != VG_OK) return st;
    if (a.n_k > 0) {
        if ((st = attn_make_map(&maps.k, a.k, a.n_k, a.hk, a.d, dtype, 1, kN)) != VG_OK) return st;
        if ((st = attn_make_map(&maps.v, a.v, a.n_k, a.hk, a.d, dtype, 1, kN)) != VG_OK) return st;
    }
    if (dtype == VG_BF16) {
        if (a.d <= 64) return nq == 2 ? launch<true, 64, 2>(a, maps, sms, s) : launch<true, 64, 1>(a, maps, sms, s);
        return nq == 2 ? launch<true, 128, 2>(a, maps, sms, s) : launch<true, 128, 1>(a, maps, sms, s);
    }
    if (a.d <= 64) return nq == 2 ? launch<false, 64, 2>(a, maps, sms, s) : launch<false, 64, 1>(a, maps, sms, s);
    return nq == 2 ? launch<false, 128, 2>(a, maps, sms, s) : launch<false, 128, 1>(a, maps, sms, s);
}

}  // namespace vg
