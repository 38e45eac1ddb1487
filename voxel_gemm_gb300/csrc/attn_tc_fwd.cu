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
//   then one warp        the MMA-issuing thread: S into TMEM, then O += P V with P read
//                        from TMEM.
//   two idle warps       fill the last warpgroup, whose registers go to the softmax warps.
// With NQ = 2 the two row tiles take turns: one's products run while the other's
// exponentials do, and both read each K and V tile from the same copy.  NQ = 1 leaves
// room for two blocks on an SM and serves calls with few rows per sample.
//
// The running maximum is only replaced when a row's scores exceed it by 2^8 (its
// exact value does not matter: O and l carry the same factor), so O, which stays in
// TMEM, is rescaled a few times per row at most instead of once per tile.  P is
// rounded to the inputs' type for the second product (l sums the unrounded values);
// fp16 weights carry a factor 2^7 more, so that a weight down to 2^-31 of the row's
// largest is not lost below fp16's range.
#include "attn_tc.cuh"

namespace vg {

namespace {

using namespace attn_tc;

constexpr int kM = 128;   // rows of an MMA tile
constexpr int kN = 128;   // keys of a tile

template <int DP, int NQ>
struct Cfg {
    static constexpr int kThreads = NQ * 128 + 128;
    static constexpr int kBlocks = DP / 64;
    static constexpr int kTile = kM * 128 * kBlocks;               // bytes of a Q, K or V tile
    static constexpr int S = NQ == 2 ? (DP == 64 ? 6 : 4) : (DP == 64 ? 4 : 2);  // ring stages
    static constexpr int kOCol = NQ * kN;                           // O's first TMEM column
    static constexpr int kTmem = NQ * (kN + DP) <= 256 ? 256 : 512;
    // q full, q empty, (s full, p full, o full, o empty) x NQ, kv full x S, kv empty x S, done
    static constexpr int kBars = 2 + 4 * NQ + 2 * S + 1;
    static constexpr size_t kSmem = 1024 + (size_t)(NQ + S) * kTile + 8 * kBars + 16;
};
static_assert(Cfg<128, 2>::kSmem <= 232448 && 2 * (Cfg<128, 1>::kSmem + 1024) <= 233472, "shared memory");

template <bool BF16, int DP, int NQ>
__global__ void __launch_bounds__(NQ * 128 + 128, NQ == 1 ? 2 : 1)
    k_attn_tc_fwd(const AttnArgs a, const __grid_constant__ AttnMaps maps, const int tiles) {
    using C = Cfg<DP, NQ>;
    constexpr int S = C::S;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sQ = smem_u32(smem), sKV = sQ + NQ * C::kTile;
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + (size_t)(NQ + S) * C::kTile);
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
    }
    tc_fence_before();
    const bool good = attn_offsets_ok(a);  // a barrier of the whole block
    tc_fence_after();
    const uint32_t tmem = uniform(*s_tmem);

    const int sets = a.hq / a.gp;
    const int group = a.hq / a.hk;
    const int64_t units = good ? (int64_t)tiles * sets * a.splits : 0;
    // unit u = (part, head set, row tile); its key tiles [lo, hi) and the row tiles it fills
    struct Unit {
        AttnTile t;
        int hs, part, lo, hi, rows;
    };
    auto find = [&](int64_t u) {
        Unit x;
        const int64_t v = u / tiles;
        x.t = attn_find_tile(a, a.q_off, a.gp, NQ * kM, (int)(u - v * tiles));
        x.hs = (int)(v % sets);
        x.part = (int)(v / sets);
        x.rows = 0;
        x.lo = x.hi = 0;
        if (x.t.b >= 0) {
            x.rows = min(NQ * kM, x.t.lq * a.gp - x.t.first);
            attn_split((x.t.lk + kN - 1) / kN, a.splits, x.part, &x.lo, &x.hi);
        }
        return x;
    };
    Waiter wait{s_abort};
    // the block was launched with 168 registers a thread (NQ = 1: 128); the softmax warps,
    // which hold a row of scores each, take what the last warpgroup leaves
    if (warp >= kLoader) reg_shrink<NQ == 2 ? 88 : 72>();
    if (warp == kLoader) {
        uint32_t it = 0, uc = 0;
        for (int64_t u = blockIdx.x; u < units && wait.ok; u += gridDim.x) {
            const Unit x = find(u);
            if (x.hi <= x.lo) continue;
            wait(q_empty, (uc & 1u) ^ 1u);
            if (!wait.ok) break;
            const int nq = x.rows > kM ? NQ : 1;
            one_lane([&] {
                mbar_arrive_expect_tx(q_full, nq * C::kTile);
                for (int w = 0; w < nq; ++w)
                    for (int b = 0; b < C::kBlocks; ++b)
                        tma_load_3d(sQ + w * C::kTile + b * kM * 128, &maps.q, b * 64, x.hs * a.gp,
                                    x.t.q0 + (x.t.first + w * kM) / a.gp, q_full);
            });
            ++uc;
            const int kh = x.hs * a.gp / group;
            for (int e = 2 * x.lo; e < 2 * x.hi; ++e, ++it) {  // K and V tiles in turn
                const uint32_t st = it % S;
                wait(kv_empty + 8 * st, ((it / S) & 1u) ^ 1u);
                if (!wait.ok) break;
                one_lane([&] {
                    mbar_arrive_expect_tx(kv_full + 8 * st, C::kTile);
                    for (int b = 0; b < C::kBlocks; ++b)
                        tma_load_3d(sKV + st * C::kTile + b * kN * 128, e & 1 ? &maps.v : &maps.k, b * 64, kh,
                                    x.t.k0 + (e >> 1) * kN, kv_full + 8 * st);
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
        const int ksteps = (a.d + 15) / 16;          // K = 16 steps over the channels
        const int o_cols = ksteps * 16;              // columns of O
        const uint32_t idesc_o = idesc_f16_bn(BF16, o_cols);
        uint32_t it = 0, uc = 0, pc[NQ] = {}, oc[NQ] = {};
        // S_w = Q_w K^T of the tile in stage st, `n` keys
        auto scores = [&](int w, uint32_t st, int n) {
            mma_channels<DP / 16, kM * 128, kN * 128>(tmem + w * kN, sw128_kmajor_desc(sQ + w * C::kTile),
                                                      sw128_kmajor_desc(sKV + st * C::kTile), idesc_f16(BF16, n),
                                                      ksteps);
            mma_commit(s_full + 8 * w);
        };
        for (int64_t u = blockIdx.x; u < units && wait.ok; u += gridDim.x) {
            const Unit x = find(u);
            if (x.hi <= x.lo) continue;
            const int nq = x.rows > kM ? NQ : 1;
            auto left = [&](int e) { return min(kN, x.t.lk - e * kN); };           // keys of tile e
            auto padded = [&](int e) { return (left(e) + 15) / 16 * 16; };
            wait(q_full, uc & 1u);
            wait(kv_full + 8 * (it % S), (it / S) & 1u);
            if (!wait.ok) break;
            tc_fence_after();
            one_lane([&] {
                for (int w = 0; w < nq; ++w) scores(w, it % S, padded(x.lo));
                mma_commit(kv_empty + 8 * (it % S));
                if (x.hi - x.lo == 1) mma_commit(q_empty);
            });
            ++it;
            for (int e = x.lo; e < x.hi; ++e) {
                const uint32_t sv = it % S, pv = (it / S) & 1u;
                const uint32_t sk = (it + 1) % S, pk = ((it + 1) / S) & 1u;
                const bool more = e + 1 < x.hi;
                wait(kv_full + 8 * sv, pv);
                if (more) wait(kv_full + 8 * sk, pk);
                if (!wait.ok) break;
                const int n16 = padded(e);
                if (n16 != left(e)) {  // V rows past the sample's keys may hold anything: 0 x them must be 0
                    zero_rows(sKV + sv * C::kTile, left(e), n16, C::kBlocks, kN * 128);
                    fence_proxy_async_smem();
                    __syncwarp();
                }
                for (int w = 0; w < nq; ++w) {
                    wait(p_full + 8 * w, pc[w]++ & 1u);
                    if (e == x.lo) wait(o_empty + 8 * w, (oc[w] & 1u) ^ 1u);
                    if (!wait.ok) break;
                    tc_fence_after();
                    one_lane([&] {
                        mma_rows<kN / 16>(tmem + C::kOCol + w * DP, tmem + w * kN,
                                          sw128_mnmajor_desc(sKV + sv * C::kTile, kN * 128), idesc_o, n16 / 16,
                                          e > x.lo);
                        if (more) scores(w, sk, padded(e + 1));
                        else mma_commit(o_full + 8 * w);
                        if (w + 1 == nq) {
                            mma_commit(kv_empty + 8 * sv);
                            if (more) mma_commit(kv_empty + 8 * sk);
                            if (e + 2 == x.hi) mma_commit(q_empty);
                        }
                    });
                    if (!more) ++oc[w];
                }
                if (!wait.ok) break;
                it += more ? 2 : 1;
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
    } else if (warp < kLoader) {
        reg_grow<NQ == 2 ? 208 : 184>();
        const int w = warp >> 2, quad = warp & 3;
        const uint32_t t_lane = tmem + ((uint32_t)(quad * 32) << 16);
        const uint32_t t_s = t_lane + w * kN, t_o = t_lane + C::kOCol + w * DP;
        const float c = a.scale_log2;
        constexpr float kLift = BF16 ? 0.f : 7.f;  // exponent added to the weights
        const float lazy = 8.f / c;                // scores above the maximum that do not replace it
        uint32_t sc = 0, oc = 0;
        for (int64_t u = blockIdx.x; u < units && wait.ok; u += gridDim.x) {
            const Unit x = find(u);
            if (x.rows <= w * kM) continue;
            const int row = w * kM + quad * 32 + lane;                // within the unit
            const bool any = x.rows > w * kM + quad * 32;             // the warp has rows
            float m = -INFINITY, l = 0.f;
            for (int e = x.lo; e < x.hi; ++e) {
                wait(s_full + 8 * w, sc & 1u);
                if (!wait.ok) break;
                ++sc;
                tc_fence_after();
                if (any) {
                    uint32_t s[4][32];
#pragma unroll
                    for (int i = 0; i < 4; ++i) tmem_ld32(t_s + 32 * i, s[i]);
                    tmem_ld_wait();
#pragma unroll
                    for (int i = 0; i < 4; ++i) tmem_ld_done(s[i]);
                    const int left = x.t.lk - e * kN;
                    if (left < kN) {
#pragma unroll
                        for (int i = 0; i < kN; ++i)
                            if (i >= left) s[i >> 5][i & 31] = 0xff800000u;
                    }
                    float top[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        top[i] = fmaxf(__uint_as_float(s[i][0]), __uint_as_float(s[i][1]));
#pragma unroll
                        for (int j = 2; j < 32; j += 2)
                            top[i] = max3(top[i], __uint_as_float(s[i][j]), __uint_as_float(s[i][j + 1]));
                    }
                    const float big = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
                    const bool grow = big > m + lazy || (m == -INFINITY && big > m);
                    if (__any_sync(0xffffffffu, grow)) {
                        const float next = grow ? big : m;
                        const float f = next == m ? 1.f : ex2((m - next) * c);
                        m = next;
                        l *= f;
                        if (e > x.lo) {  // O holds the earlier tiles' sum; its products have finished
#pragma unroll 1
                            for (int i = 0; i < DP / 16; ++i) {
                                uint32_t o[16];
                                tmem_ld16(t_o + 16 * i, o);
                                tmem_ld_wait();
                                tmem_ld_done(o);
#pragma unroll
                                for (int j = 0; j < 16; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * f);
                                tmem_st16(t_o + 16 * i, o);
                            }
                        }
                    }
                    const float base = (m == -INFINITY ? 0.f : m * c) - kLift;
                    const float2 c2 = make_float2(c, c), base2 = make_float2(-base, -base);
                    float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        uint32_t p[32];
#pragma unroll
                        for (int j = 0; j < 32; ++j) {
                            float2 x2 = fma2(two(&s[2 * i + (j >> 4)][2 * (j & 15)]), c2, base2);
                            x2 = make_float2(ex2(x2.x), ex2(x2.y));
                            sum[j & 1] = add2(sum[j & 1], x2);
                            p[j] = pack2<BF16>(x2.x, x2.y);
                        }
                        tmem_st32(t_s + 32 * i, p);
                    }
                    const float2 both = add2(sum[0], sum[1]);
                    l += both.x + both.y;
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
                const bool mine = row < x.rows;
                const int pr = x.t.first + row;                       // packed row of the sample
                const int64_t qi = x.t.q0 + pr / a.gp;
                const int h = x.hs * a.gp + pr % a.gp;
                const float inv = x.hi > x.lo ? 1.f / l : 0.f;
                const float lse = x.hi > x.lo ? (m * c + (log2f(l) - kLift)) * kLn2 : -INFINITY;
                float* dst_l = a.splits > 1 ? a.part_lse + (size_t)x.part * a.hq * a.n_q : a.lse;
                if (mine && dst_l) dst_l[(int64_t)h * a.n_q + qi] = lse;
                float* dst_p = a.part + (((size_t)x.part * a.n_q + qi) * a.hq + h) * a.d;
                uint16_t* dst = head_row<uint16_t>(a.o, qi, h);
                __syncwarp();
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
                        if (a.splits > 1) store_cols32_f32(dst_p + 32 * i, o, inv, a.d - 32 * i);
                        else store_cols32<BF16>(dst + 32 * i, o, inv, a.d - 32 * i);
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

template <bool BF16, int DP, int NQ>
int launch(const AttnArgs& a, const AttnMaps& maps, int sms, cudaStream_t s) {
    using C = Cfg<DP, NQ>;
    auto kernel = k_attn_tc_fwd<BF16, DP, NQ>;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)C::kSmem) != cudaSuccess)
        return VG_ERR_CUDA;
    const int64_t tiles = attn_max_tiles(a.n_q, a.batch, a.gp, NQ * kM);
    const int64_t units = tiles * (a.hq / a.gp) * a.splits;
    const int64_t grid = std::min<int64_t>(units, (int64_t)sms * (NQ == 1 ? 2 : 1));
    kernel<<<(unsigned)grid, C::kThreads, C::kSmem, s>>>(a, maps, (int)tiles);
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

int attn_tc_fwd(const AttnArgs& a, int dtype, int nq, int sms, cudaStream_t s) {
    AttnMaps maps{};
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
