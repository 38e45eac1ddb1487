// Cross attention forward on the tensor cores (tcgen05 / TMEM), 16-bit types.
//
//   S = Q K^T, m = running row maximum, P = exp2(c S - c m), l = running sum of P,
//   O = (sum over tiles of P V) / l, lse = scale m + ln l          (c = scale log2 e)
//
// A persistent block takes units of NQ x 128 packed query rows of one sample and head
// set, and runs along the sample's keys in tiles of 128:
//   warps 0 .. 8 NQ - 1  softmax: two threads per row, 64 keys of a tile each.  A thread
//                        reads its scores from TMEM, writes P as 16-bit pairs over them,
//                        and at the end scales and stores a part of its row of O.
//   then one warp        loader: TMA copies of Q (per unit) and of K and V tiles (a ring).
//   then one warp        issues the products: S into TMEM, then O += P V with P read from
//                        TMEM.
//   two idle warps       fill the last warpgroup, whose registers go to the softmax warps.
// With NQ = 2 the two row tiles take turns: one's products run while the other's
// exponentials do, and both read each K and V tile from the same copy.  NQ = 1 leaves
// room for two blocks on an SM and serves calls with few rows per sample.
//
// The row maximum only keeps the weights in range, and O and l carry the same factor
// whatever it is.  So it is taken from the first tile and kept: later tiles are weighed
// with it right away, and only where a half row's sum of weights leaves the range (2^64 in
// bf16, 2^14 in fp16) are the maximum renewed, O (in TMEM) and l rescaled and the tile
// weighed again.  P is rounded to the inputs' type for the second product (l sums
// the unrounded values); fp16 weights carry a factor 2^7 more, so that a weight down to
// 2^-31 of the row's largest is not lost below fp16's range.
#include "attn_tc.cuh"

namespace vg {

namespace {

using namespace attn_tc;

constexpr int kM = 128;   // rows of an MMA tile
constexpr int kN = 128;   // keys of a tile

constexpr int kH = kN / 2;  // keys of a softmax thread

template <int DP, int NQ>
struct Cfg {
    static constexpr int kThreads = NQ * 256 + 128;
    static constexpr int kBlocks = DP / 64;
    static constexpr int kTile = kM * 128 * kBlocks;               // bytes of a Q, K or V tile
    static constexpr int S = NQ == 2 ? (DP == 64 ? 6 : 4) : (DP == 64 ? 4 : 2);  // ring stages
    static constexpr int kOCol = NQ * kN;                           // O's first TMEM column
    static constexpr int kTmem = NQ * (kN + DP) <= 256 ? 256 : 512;
    // q full, q empty, (s full, p full, o full, o empty) x NQ, kv full x S, kv empty x S, tail, done
    static constexpr int kBars = 2 + 4 * NQ + 2 * S + 2;
    static constexpr size_t kSwap = (size_t)NQ * 2 * 2 * kM * sizeof(float);  // maxima and sums of the row halves
    static constexpr size_t kSmem = 1024 + (size_t)(NQ + S) * kTile + kSwap + 8 * kBars + 16;
    // registers: launched with kRegs a thread; the softmax warps take what the last warpgroup gives up
    static constexpr int kRegs = NQ == 2 ? 96 : 80, kSoft = NQ == 2 ? 104 : 96, kAux = NQ == 2 ? 64 : 48;
    static_assert(NQ * 256 * kSoft + 128 * kAux <= kThreads * kRegs, "register split");
};
static_assert(Cfg<128, 2>::kSmem <= 232448 && 2 * (Cfg<128, 1>::kSmem + 1024) <= 233472, "shared memory");

template <bool BF16, int DP, int NQ>
__global__ void __launch_bounds__(NQ * 256 + 128, NQ == 1 ? 2 : 1)
    k_attn_tc_fwd(const AttnArgs a, const __grid_constant__ AttnMaps maps, const int tiles) {
    using C = Cfg<DP, NQ>;
    constexpr int S = C::S;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sQ = smem_u32(smem), sKV = sQ + NQ * C::kTile;
    float* s_swap = reinterpret_cast<float*>(smem + (size_t)(NQ + S) * C::kTile);
    uint64_t* bars = reinterpret_cast<uint64_t*>(reinterpret_cast<uint8_t*>(s_swap) + C::kSwap);
    uint32_t* s_tmem = reinterpret_cast<uint32_t*>(bars + C::kBars);
    volatile uint32_t* s_abort = s_tmem + 1;
    const uint32_t bar0 = smem_u32(bars);
    const uint32_t q_full = bar0, q_empty = bar0 + 8;
    const uint32_t s_full = bar0 + 16, p_full = s_full + 8 * NQ, o_full = p_full + 8 * NQ, o_empty = o_full + 8 * NQ;
    const uint32_t kv_full = o_empty + 8 * NQ, kv_empty = kv_full + 8 * S, tail = kv_empty + 8 * S, done = tail + 8;

    const int warp = uniform((int)threadIdx.x >> 5), lane = threadIdx.x & 31;
    constexpr int kLoader = NQ * 8, kIssuer = NQ * 8 + 1;
    if (threadIdx.x == 0) {
        mbar_init(q_full, 1);
        mbar_init(q_empty, 1);
        for (int w = 0; w < NQ; ++w) {
            mbar_init(s_full + 8 * w, 1);
            mbar_init(p_full + 8 * w, 8);
            mbar_init(o_full + 8 * w, 1);
            mbar_init(o_empty + 8 * w, 8);
        }
        for (int i = 0; i < S; ++i) {
            mbar_init(kv_full + 8 * i, 1);
            mbar_init(kv_empty + 8 * i, 1);
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
    if (warp >= kLoader) reg_shrink<C::kAux>();
    if (warp == kLoader) {
        uint32_t it = 0, uc = 0, tc = 0;
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
                const uint32_t st = it % S, dst = sKV + st * C::kTile;
                wait(kv_empty + 8 * st, ((it / S) & 1u) ^ 1u);
                if (!wait.ok) break;
                const int left = min(kN, x.t.lk - (e >> 1) * kN), n16 = (left + 15) / 16 * 16;
                const bool cut = (e & 1) && n16 != left;
                const void* map = e & 1 ? &maps.v : &maps.k;
                const uint32_t bar = cut ? tail : kv_full + 8 * st;
                one_lane([&] {
                    mbar_arrive_expect_tx(bar, C::kTile);
                    for (int b = 0; b < C::kBlocks; ++b)
                        tma_load_3d(dst + b * kN * 128, map, b * 64, kh, x.t.k0 + (e >> 1) * kN, bar);
                });
                if (cut) {  // V rows past the sample's keys may hold anything, and 0 x them must be 0 in P V
                    wait(tail, tc++ & 1u);
                    zero_rows(dst, left, n16, C::kBlocks, kN * 128);
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(kv_full + 8 * st);
                    __syncwarp();
                }
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
            auto padded = [&](int e) { return (min(kN, x.t.lk - e * kN) + 15) / 16 * 16; };  // keys of tile e
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
        reg_grow<C::kSoft>();
        // Thread (tile w, quadrant quad, lane) and half: 64 keys of one row.  The two warps that share a
        // quadrant's rows meet at a named barrier, so none of them may leave its loops early: after a wait that
        // gave up they only skip work.
        const int w = warp >> 3, half = (warp >> 2) & 1, quad = warp & 3;
        const uint32_t pair = 1 + w * 4 + quad;
        float* swap_max = s_swap + w * 4 * kM + quad * 32 + lane;  // [half][row] maxima, then [half][row] sums
        float* swap_sum = swap_max + 2 * kM;
        const uint32_t t_lane = tmem + ((uint32_t)(quad * 32) << 16);
        const uint32_t t_s = t_lane + w * kN + half * kH, t_p = t_lane + w * kN + half * (kH / 2);
        const uint32_t t_o = t_lane + C::kOCol + w * DP;
        const float c = a.scale_log2;
        constexpr float kLift = BF16 ? 0.f : 7.f;            // exponent added to the weights
        constexpr float kMost = BF16 ? 0x1p64f : 0x1p14f;    // of a half row's sum before the maximum is replaced
        const bool v8ok = ((reinterpret_cast<uintptr_t>(a.o.data) | (uintptr_t)(a.o.row_stride * 2) |
                            (uintptr_t)(a.o.head_stride * 2)) & 31u) == 0;
        uint32_t sc = 0, oc = 0;
        for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
            const Unit x = find(u);
            if (x.rows <= w * kM) continue;
            const int row = w * kM + quad * 32 + lane;                // within the unit
            const bool any = x.rows > w * kM + quad * 32, mine = row < x.rows;  // the warp, the thread has a row
            float m = -INFINITY, l = 0.f;
            for (int e = x.lo; e < x.hi; ++e) {
                wait(s_full + 8 * w, sc++ & 1u);
                tc_fence_after();
                if (any) {
                    const int left = x.t.lk - e * kN - half * kH;     // valid keys of the half
                    uint32_t s[2][32], p[32];
                    float sum;
                    auto load = [&] {
#pragma unroll
                        for (int i = 0; i < 2; ++i) tmem_ld32(t_s + 32 * i, s[i]);
                        tmem_ld_wait();
#pragma unroll
                        for (int i = 0; i < 2; ++i) tmem_ld_done(s[i]);
                        if (left < kH) {
#pragma unroll
                            for (int i = 0; i < kH; ++i)
                                if (i >= left) s[i >> 5][i & 31] = 0xff800000u;
                        }
                    };
                    auto weights = [&] {
                        const float base = kLift - (m == -INFINITY ? 0.f : m * c);
                        const float2 c2 = make_float2(c, c), base2 = make_float2(base, base);
                        float2 acc[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
                        for (int j = 0; j < 32; ++j) {
                            float2 x2 = fma2(two(&s[j >> 4][2 * (j & 15)]), c2, base2);
                            x2 = make_float2(ex2(x2.x), ex2(x2.y));
                            acc[j & 1] = add2(acc[j & 1], x2);
                            p[j] = pack2<BF16>(x2.x, x2.y);
                        }
                        const float2 both = add2(acc[0], acc[1]);
                        sum = both.x + both.y;
                    };
                    load();
                    bool renew = e == x.lo;
                    if (!renew) {
                        weights();
                        renew = named_bar_or(pair, 64, mine && (!(sum <= kMost) || m == -INFINITY));
                        if (renew) load();  // nobody has written P over the scores yet
                    }
                    if (renew) {
                        float top[2];
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            top[i] = fmaxf(__uint_as_float(s[i][0]), __uint_as_float(s[i][1]));
#pragma unroll
                            for (int j = 2; j < 32; j += 2)
                                top[i] = max3(top[i], __uint_as_float(s[i][j]), __uint_as_float(s[i][j + 1]));
                        }
                        swap_max[half * kM] = fmaxf(top[0], top[1]);
                        named_bar_sync(pair, 64);
                        const float next = fmaxf(m, fmaxf(swap_max[0], swap_max[kM]));
                        const float f = next == m ? 1.f : ex2((m - next) * c);
                        m = next;
                        l *= f;
                        if (e > x.lo) {  // O holds the earlier tiles' sum, whose products have finished
#pragma unroll 1
                            for (int i = 0; i < DP / 32; ++i) {
                                uint32_t o[16];
                                const uint32_t at = t_o + half * (DP / 2) + 16 * i;
                                tmem_ld16(at, o);
                                tmem_ld_wait();
                                tmem_ld_done(o);
#pragma unroll
                                for (int j = 0; j < 16; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * f);
                                tmem_st16(at, o);
                            }
                        }
                        weights();
                    }
                    l += sum;
                    tmem_st32(t_p, p);
                    tmem_st_wait();
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(p_full + 8 * w);
            }
            if (x.hi > x.lo) {
                wait(o_full + 8 * w, oc++ & 1u);
                tc_fence_after();
            }
            if (any) {
                if (x.hi > x.lo) {  // the row's sum is both halves'
                    swap_sum[half * kM] = l;
                    named_bar_sync(pair, 64);
                    l = swap_sum[0] + swap_sum[kM];
                }
                const bool store = mine && wait.ok;
                const int pr = x.t.first + row;                       // packed row of the sample
                const int64_t qi = x.t.q0 + pr / a.gp;
                const int h = x.hs * a.gp + pr % a.gp;
                const float inv = x.hi > x.lo ? 1.f / l : 0.f;
                const float lse = x.hi > x.lo ? (m * c + (log2f(l) - kLift)) * kLn2 : -INFINITY;
                float* dst_l = a.splits > 1 ? a.part_lse + (size_t)x.part * a.hq * a.n_q : a.lse;
                if (store && half == 0 && dst_l) dst_l[(int64_t)h * a.n_q + qi] = lse;
                float* dst_p = a.part + (((size_t)x.part * a.n_q + qi) * a.hq + h) * a.d;
                uint16_t* dst = head_row<uint16_t>(a.o, qi, h);
                __syncwarp();
                auto columns = [&](int col, uint32_t (&o)[32]) {
                    if (x.hi > x.lo) {
                        tmem_ld32(t_o + col, o);
                        tmem_ld_wait();
                        tmem_ld_done(o);
                    } else {
#pragma unroll
                        for (int j = 0; j < 32; ++j) o[j] = 0u;
                    }
                };
                if (a.splits == 1 && a.d == DP) {
                    // whole 128-byte lines of 64 columns: d = 128 one line a half, d = 64 the row by half 0
                    if (DP == 128 || half == 0) {
                        uint32_t z[32];
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            uint32_t o[32];
                            columns(half * 64 + 32 * i, o);
#pragma unroll
                            for (int j = 0; j < 16; ++j) {
                                const float2 v = two(o + 2 * j);
                                z[16 * i + j] = pack2<BF16>(v.x * inv, v.y * inv);
                            }
                        }
                        store_lines_quad(store ? reinterpret_cast<uint8_t*>(dst + half * 64) : nullptr, z, lane, v8ok);
                    }
                } else {
#pragma unroll 1
                    for (int col = half * (DP / 2); col < min(a.d, (half + 1) * (DP / 2)); col += 32) {
                        uint32_t o[32];
                        columns(col, o);
                        if (store) {
                            if (a.splits > 1) store_cols32_f32(dst_p + col, o, inv, a.d - col);
                            else store_cols32<BF16>(dst + col, o, inv, a.d - col);
                        }
                        __syncwarp();
                    }
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
