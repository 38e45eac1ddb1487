// Cross attention: what the fp32 and the tensor-core kernels share -- arguments,
// the layout of the work, the lookup of a tile's sample and the joins of split
// work.
//
// Rows of work.  G = heads_q / heads_k query heads read one key head.  When G is a
// power of two up to 16, a sample's queries and those G heads are taken together
// as "packed rows" r = i * gp + g (query i, head g of the group; gp = G), so the
// keys and values are read once for all of them; otherwise gp = 1 and each query
// head is its own list of rows.  A "head set" hs in [0, heads_q / gp) is gp
// consecutive query heads; its key head is hs * gp / G.
#pragma once
#include "common.cuh"
#include "internal.h"

namespace vg {

struct AttnArgs {
    // shapes
    int64_t n_q, n_k;
    int batch, hq, hk, d;
    int gp, gp_log2;             // query heads packed into rows
    const int32_t* q_off;        // [batch + 1]
    const int32_t* k_off;        // [batch + 1]
    const int32_t* k_len;        // [batch] or null: every row between offsets is valid
    float scale;                 // of the scores
    float scale_log2;            // scale * log2(e)
    // tensors ([rows][heads][d], strides in elements)
    vg_heads q, k, v, o, go, gq, gk, gv;
    float* lse;                  // [hq][n_q]
    // workspace
    uint32_t* err;               // error record
    uint32_t* bound;             // fp16: fp32 bits of each sample's largest |dO row| and |V row|
    // [2][hq / gp][n_q * gp], negated: lse * log2 e and sum_d dO O of every packed row; fp16: a third, |dO row|
    float* stats;
    // The axis that a kernel runs along is cut into parts of `per_part` tiles of `tile` rows, so that a sample has
    // attn_parts of them; splits bounds that number (1: not cut, results go to their place at once).
    int splits, per_part, tile;
    float* part;                 // results of the parts (layouts at their kernels)
    float* part_lse;
    int64_t unit_cycles;         // limit of a wait that lasts as long as a unit of work (tensor cores)
};

// fp16 has no exponent range to spare: the backward pass's weights (<= 1) carry 2^15.
constexpr float kHalfLift = 15.f;

// A packed row's statistics.
__device__ __forceinline__ float2 attn_stats(const AttnArgs& a, int64_t row) {
    return make_float2(a.stats[row], a.stats[a.n_q * a.hq + row]);
}

// The tile of one sample that a block works on.
struct AttnTile {
    int b;          // sample, -1: none
    int first;      // first row of the tile within the sample's rows
    int part;       // part of the other axis
    int q0, lq;     // the sample's queries
    int k0, lk;     // its keys: first row, valid rows
    int krows;      // its key rows, valid or not
};

// Whether the offsets are a partition of the rows and the lengths fit it; by all
// threads of the block, the same answer in each.  A bad array is recorded and the
// kernel writes nothing, so that no wrong offset becomes a wrong address.
__device__ __forceinline__ bool attn_offsets_ok(const AttnArgs& a) {
    bool bad = false;
    for (int b = threadIdx.x; b < a.batch; b += blockDim.x) {
        const int q = a.q_off[b], q1 = a.q_off[b + 1], k = a.k_off[b], k1 = a.k_off[b + 1];
        bad |= q < 0 || q1 < q || q1 > a.n_q || k < 0 || k1 < k || k1 > a.n_k;
        bad |= b == 0 && (q != 0 || k != 0);
        bad |= b == a.batch - 1 && (q1 != a.n_q || k1 != a.n_k);
        if (a.k_len) bad |= a.k_len[b] < 0 || a.k_len[b] > k1 - k;
    }
    bad = __syncthreads_or(bad);
    if (bad && threadIdx.x == 0) atomicOr(a.err, kErrRange);
    return !bad;
}

// Parts of an axis of `len` rows.
__device__ __forceinline__ int attn_parts(const AttnArgs& a, int64_t len) {
    if (a.splits == 1) return 1;
    const int64_t step = (int64_t)a.per_part * a.tile;
    return max(1, (int)((len + step - 1) / step));
}

// Tile `t` of the work: sample by sample, the sample's tiles of `rows` rows (its queries times gp; kKeys: its key
// rows) for each part of the other axis.  By a whole warp, every lane gets the answer: lanes take 32 samples at a
// time and prefix-sum their tile counts.
template <bool kKeys>
__device__ __forceinline__ AttnTile attn_find_tile(const AttnArgs& a, int rows, int64_t t) {
    const int lane = threadIdx.x & 31;
    AttnTile r;
    r.b = -1;
    for (int b0 = 0; b0 < a.batch; b0 += 32) {
        const int b = b0 + lane;
        int64_t lq = 0, lk = 0, kr = 0;
        if (b < a.batch) {
            lq = (int64_t)(a.q_off[b + 1] - a.q_off[b]) * a.gp;
            kr = a.k_off[b + 1] - a.k_off[b];
            lk = a.k_len ? a.k_len[b] : kr;
        }
        const int tiles = (int)(((kKeys ? kr : lq) + rows - 1) / rows);
        const int64_t count = (int64_t)tiles * attn_parts(a, kKeys ? lq : lk);
        int64_t incl = count;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t up = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += up;
        }
        const uint32_t at = __ballot_sync(0xffffffffu, t < incl);
        if (at) {
            const int src = __ffs(at) - 1;
            const int n = __shfl_sync(0xffffffffu, tiles, src);
            const int64_t i = t - __shfl_sync(0xffffffffu, incl - count, src);
            r.b = b0 + src;
            r.part = (int)(i / n);
            r.first = (int)(i - (int64_t)r.part * n) * rows;
            // one load each, shared out by a shuffle: the compiler knows the result to be uniform
            const int32_t* p = lane < 2 ? a.q_off + r.b + lane : lane < 4 ? a.k_off + r.b + (lane - 2)
                               : a.k_len ? a.k_len + r.b : nullptr;
            const int v = p ? *p : 0;
            r.q0 = __shfl_sync(0xffffffffu, v, 0);
            r.lq = __shfl_sync(0xffffffffu, v, 1) - r.q0;
            r.k0 = __shfl_sync(0xffffffffu, v, 2);
            r.krows = __shfl_sync(0xffffffffu, v, 3) - r.k0;
            r.lk = a.k_len ? __shfl_sync(0xffffffffu, v, 4) : r.krows;
            return r;
        }
        t -= __shfl_sync(0xffffffffu, incl, 31);
    }
    return r;
}

// Most tiles that `total` rows in `batch` samples can make.
inline int64_t attn_max_tiles(int64_t total, int batch, int mult, int rows) {
    return total * mult / rows + std::min<int64_t>(batch, total);
}

// How a call is cut and where its scratch lies (byte offsets in the workspace; the
// first 256 bytes are the error record).
struct AttnShape {
    int64_t n_q, n_k;
    int batch, hq, hk, d, dtype;
    bool backward;
};
struct AttnPlan {
    int sms = 0;
    int tc = 0;                          // 16-bit types: tensor cores
    int gp = 1;                          // query heads packed into rows
    int nq = 1;                          // row tiles of a forward block
    // most parts of the key axis (forward, dQ) and of the query axis (dK, dV), and the tiles of a part
    int s_fwd = 1, s_dq = 1, s_dkv = 1;
    int per_fwd = 0, per_dq = 0, per_dkv = 0;
    size_t off_lse = 0, off_bound = 0, off_dq = 0, off_dk = 0, off_dv = 0, total = 0;
};
int attn_plan(const AttnShape& c, AttnPlan* P);
int attn_fwd(AttnArgs a, const AttnPlan& p, int dtype, char* ws, cudaStream_t s);
int attn_bwd(AttnArgs a, const AttnPlan& p, int dtype, char* ws, cudaStream_t s);

// Tiles [lo, hi) of part `part` of an axis of `len` rows.
__device__ __forceinline__ void attn_split(const AttnArgs& a, int64_t len, int part, int* lo, int* hi) {
    const int n = (int)((len + a.tile - 1) / a.tile);
    *lo = a.splits == 1 ? 0 : min(n, a.per_part * part);
    *hi = a.splits == 1 ? n : min(n, *lo + a.per_part);
}

template <typename T>
__device__ __forceinline__ T* head_row(const vg_heads& h, int64_t row, int head) {
    return static_cast<T*>(h.data) + row * h.row_stride + head * h.head_stride;
}

// ---- fp32 path (attn_simt.cu) ----
int attn_simt_fwd(const AttnArgs& a, cudaStream_t s);
int attn_simt_dq(const AttnArgs& a, cudaStream_t s);
int attn_simt_dkv(const AttnArgs& a, float* part_dv, cudaStream_t s);

// ---- 16-bit path (attn_tc_fwd.cu, attn_tc_bwd.cu); nq: row tiles of a forward block ----
int attn_tc_fwd(AttnArgs a, int dtype, int nq, int sms, cudaStream_t s);
int attn_tc_dq(AttnArgs a, int dtype, int sms, cudaStream_t s);
int attn_tc_dkv(AttnArgs a, float* part_dv, int dtype, int sms, cudaStream_t s);

}  // namespace vg
