// Gated linear recurrence of each channel along each sequence, and its gradient.
//
//   a = sigmoid(gate),  h_t = a_t h_{t-1} + b_t,  b_t = (1 - a_t) x_t  (or x_t)
// backward: lam_t = dy_t + mu_{t+1}, mu_t = a_t lam_t;  db = lam, da = h_{t-1} lam (- x lam)
//
// A run of tokens maps the state that enters it to the one that leaves it, h -> A h + B, and two
// runs after one another make (A2 A1, A2 B1 + B2): so the positions are cut into tiles that work
// side by side.  A block takes a tile of positions and 128 bytes of channels: 8 lanes hold a
// token's channels as 16-byte vectors, 32 rows of lanes hold a few tokens each.  Each thread finds
// the map of its tokens, the block joins them in shared memory, publishes the tile's map, collects
// those of the tiles before it, and goes through its tokens again from the state that enters.
// Bound by memory: gate and x are read once, out written once.
//
// The maps of earlier tiles are collected through a tree: node (l, i) is the map of the 8^l tiles
// from i 8^l on; tile j reads, at each level, the siblings before its own ancestor, at most 7,
// and the last tile below a node publishes that node.  So the shape of every sum depends on the
// sizes alone (the same bits in every run), and a tile waits for about as many hand-overs as there
// are levels.  A node's word holds A and B, 64 bits that are stored at once; words are all ones
// before they are written (a NaN that no result has), so the data is its own flag.  Blocks
// take their tiles in order from a counter: whatever a tile waits for was taken by a block that
// runs already.  Waits are bounded by time; a block that gives up records it and goes on with NaN.
//
// Where a sequence begins, the map is constant (A = -1 marks it, h -> B), so that nothing, not
// even a NaN, passes from one sequence to the next.
#include "common.cuh"
#include "internal.h"
#include "tc_ptx.cuh"

namespace vg {

namespace {

using namespace ptx;

constexpr int kThreads = 256;
constexpr int kLanes = 8;                    // 16-byte vectors of a token in a block: 128 bytes of channels
constexpr int kRows = kThreads / kLanes;     // rows of lanes
constexpr int kFwdTokens = 8, kBwdTokens = 4;  // tokens of a thread
constexpr int kFwdTile = kRows * kFwdTokens, kBwdTile = kRows * kBwdTokens;
constexpr int kFan = 3;                      // log2 of a node's children
constexpr int kMaxLevels = 8;                // 128 * 8^8 positions are more than 2^31
constexpr uint64_t kUnset = ~0ull;
constexpr uint64_t kGiveUpNs = 2000000000;
static_assert(kBwdTile == kScanCarryRows && kFwdTile % kBwdTile == 0, "states are kept where the backward tiles begin");

// Workspace: word 0 the error record, word 1 this call's verdict on its offsets, word 2 the
// counter of work units; nodes from byte 256 on.
struct Tree {
    int levels;
    int64_t tiles;
    int64_t base[kMaxLevels];  // first node of a level, in units of channels
};

struct ScanArgs {
    int64_t n;
    int c, batch, blocks_c;    // blocks_c: blocks of channels
    const int32_t* off;
    const int32_t* order;
    int reverse, free_input;
    const char *gate, *x, *gy;
    char *out, *gg;            // out: grad_x in the backward pass
    int64_t gate_s, x_s, gy_s, out_s, gg_s;
    const float* first;
    const float* glast;
    float *last, *carries, *gfirst;
    uint32_t* head;
    uint64_t* nodes;
    Tree tree;
    int64_t units;
};

// sigmoid(g) by its smaller side, m = e / (1 + e) with e = exp(-|g|), of which all else follows
// without cancellation: a = m for g < 0, 1 - m else.  Returned as m or, for g >= 0, as -m, so the
// sign bit says which.
template <typename T>
__device__ __forceinline__ float side(float g) {
    const float e = sizeof(T) == 4 ? expf(-fabsf(g)) : __expf(-fabsf(g));
    const float m = __fdividef(e, 1.f + e);
    return g < 0.f ? m : -m;
}
__device__ __forceinline__ bool near_one(float m) { return signbit(m); }
__device__ __forceinline__ float kept(float m, float h) { return fmaf(m, h, near_one(m) ? h : 0.f); }  // a h
__device__ __forceinline__ float added(float m) { return near_one(m) ? -m : 1.f - m; }               // 1 - a
__device__ __forceinline__ float slope(float m) { return near_one(m) ? -m * (1.f + m) : m * (1.f - m); }  // a (1 - a)

// Maps h -> A h + B; A = -1: h -> B.
struct Map {
    float a, b;
};
__device__ __forceinline__ float through(Map m, float h) { return m.a < 0.f ? m.b : fmaf(m.a, h, m.b); }
__device__ __forceinline__ Map then(Map first, Map second) {
    if (second.a < 0.f) return second;
    return Map{first.a < 0.f ? -1.f : first.a * second.a, fmaf(second.a, first.b, second.b)};
}
__device__ __forceinline__ void publish(uint64_t* node, Map m) {
    uint64_t w = (uint64_t)__float_as_uint(m.b) << 32 | __float_as_uint(m.a);
    if (w == kUnset) w = (uint64_t)0x7fc00000u << 32 | 0x7fc00000u;
    asm volatile("st.relaxed.gpu.global.u64 [%0], %1;" ::"l"(node), "l"(w) : "memory");
}
__device__ __forceinline__ uint64_t look(const uint64_t* node) {
    uint64_t w;
    asm volatile("ld.relaxed.gpu.global.u64 %0, [%1];" : "=l"(w) : "l"(node) : "memory");
    return w;
}
__device__ __forceinline__ Map map_of(uint64_t w) {
    return Map{__uint_as_float((uint32_t)w), __uint_as_float((uint32_t)(w >> 32))};
}
// The node's map once it is there.  Where another block gave up (its record is set), or after
// kGiveUpNs, a constant NaN.
__device__ __forceinline__ Map awaited(const uint64_t* node, uint64_t w, uint32_t* record) {
    if (w != kUnset) return map_of(w);
    const uint64_t t0 = globaltimer();
    for (int spins = 0;; ++spins) {
        w = look(node);
        if (w != kUnset) return map_of(w);
        if ((spins & 63) == 63) {
            const bool late = globaltimer() - t0 > kGiveUpNs;
            if (late) atomicOr(record, kErrTimeout);
            if (late || (*reinterpret_cast<volatile uint32_t*>(record) & kErrTimeout))
                return Map{-1.f, __uint_as_float(0x7fc00000u)};
        }
    }
}

// Where sequence b begins in the order of the visits (a sequence's visits are its positions,
// downwards all of them counted from the end), and which sequence that is.
__device__ __forceinline__ int64_t begins(const ScanArgs& a, int b) {
    return a.reverse ? a.n - a.off[a.batch - b] : a.off[b];
}
__device__ __forceinline__ int sequence(const ScanArgs& a, int b) { return a.reverse ? a.batch - 1 - b : b; }

// What a tile of visits [lo, hi) holds of beginnings and ends.
template <int TILE>
struct Cuts {
    uint32_t begin[TILE / 32], end[TILE / 32];  // a bit per visit
    int32_t begin_seq[TILE], end_seq[TILE];     // the sequence, where the bit is set
};

// Fill in `s`.  Sequences without tokens that lie here hand `in` on to `out` (each may be null).
template <int TILE>
__device__ __forceinline__ void find_cuts(const ScanArgs& a, Cuts<TILE>& s, int64_t lo, int64_t hi, bool last_tile,
                                          int c0, int channels, const float* in, float* out) {
    for (int i = threadIdx.x; i < TILE / 32; i += kThreads) s.begin[i] = s.end[i] = 0;
    // the number of sequences that begin before lo, 256 probes at a time
    int from = 0, to = a.batch;
    while (to > from) {
        const int step = (to - from + kThreads - 1) / kThreads;
        const int b = from + (int)threadIdx.x * step;
        const int before = __syncthreads_count(b < to && begins(a, b) < lo);
        if (before == 0) {
            to = from;
        } else {
            const int hit = from + (before - 1) * step;  // begins before lo; the next probe does not
            from = hit + 1;
            to = min(to, hit + step);
        }
    }
    __syncthreads();
    // those that begin here, and the one before them, which may end here
    for (int b = max(from - 1, 0) + (int)threadIdx.x; b < a.batch; b += kThreads) {
        const int64_t p = begins(a, b), q = begins(a, b + 1);
        if (p >= hi && !(last_tile && p == a.n)) break;
        const int seq = sequence(a, b);
        if (q > p) {
            if (p >= lo && p < hi) {
                atomicOr(&s.begin[(p - lo) >> 5], 1u << ((p - lo) & 31));
                s.begin_seq[p - lo] = seq;
            }
            if (q > lo && q <= hi) {
                atomicOr(&s.end[(q - 1 - lo) >> 5], 1u << ((q - 1 - lo) & 31));
                s.end_seq[q - 1 - lo] = seq;
            }
        } else if (p >= lo && out) {
            for (int i = c0; i < c0 + channels; ++i)
                out[(int64_t)seq * a.c + i] = in ? in[(int64_t)seq * a.c + i] : 0.f;
        }
    }
    __syncthreads();
}

// Bits [at, at + COUNT) of a tile's mask, COUNT a power of two up to 32.
template <int COUNT>
__device__ __forceinline__ uint32_t bits(const uint32_t* mask, int at) {
    return (mask[at >> 5] >> (at & 31)) & ((1u << COUNT) - 1);
}

// Nodes of the tree: siblings of tile v's ancestor at level l that come before it.
__device__ __forceinline__ int64_t node_at(const ScanArgs& a, int l, int64_t i, int c) {
    return a.tree.base[l] + i * a.c + c;
}

// Maps of the rows of lanes, and what the block makes of them.
template <int CH>
struct Joint {
    static constexpr int kGroups = kThreads / CH;     // groups of rows that are gone through side by side
    static constexpr int kSpan = kRows / kGroups;     // rows of a group
    float a[kRows][CH], b[kRows][CH];                 // a row's map, then that of the rows of its group before it
    float ga[kGroups][CH], gb[kGroups][CH];           // a group's map
    float la[kMaxLevels][CH], lb[kMaxLevels][CH];     // the maps of a level's siblings, joined
    float enter[kGroups][CH];                         // the state that enters a group
};

// From the rows' maps (in the order in which they are applied: `down`, the last row first) to the
// state that enters each group.  v: the tile's place among the tiles; alone: nothing reaches into
// it from earlier tiles; sealed: its own map is constant.
template <int CH>
__device__ __forceinline__ void join(const ScanArgs& a, Joint<CH>& s, int64_t v, int c0, bool down, bool alone,
                                     bool sealed) {
    using J = Joint<CH>;
    const int c = threadIdx.x % CH, g = threadIdx.x / CH;
    const bool real = c0 + c < a.c;
    __syncthreads();
    Map m{1.f, 0.f};
    for (int k = 0; k < J::kSpan; ++k) {
        const int i = g * J::kSpan + k, r = down ? kRows - 1 - i : i;
        const Map mine{s.a[r][c], s.b[r][c]};
        s.a[r][c] = m.a;
        s.b[r][c] = m.b;
        m = then(m, mine);
    }
    s.ga[g][c] = m.a;
    s.gb[g][c] = m.b;
    __syncthreads();
    Map own{1.f, 0.f};
    const bool more = a.tree.tiles > 1;
    if (g == 0 && more) {
        for (int i = 0; i < J::kGroups; ++i) own = then(own, Map{s.ga[i][c], s.gb[i][c]});
        if (real) publish(a.nodes + node_at(a, 0, v, c0 + c), own);
    }
    // the siblings before this tile's ancestors, a level to a group
    const bool parent = (v & ((1 << kFan) - 1)) == (1 << kFan) - 1;
    const bool wanted = more && (!alone || (parent && !sealed));
    if (wanted) {
        for (int l = g; l < a.tree.levels; l += J::kGroups) {
            const int64_t at = v >> (kFan * l), first = at >> kFan << kFan;
            Map lm{1.f, 0.f};
            if (real) {
                uint64_t w[(1 << kFan) - 1];
#pragma unroll
                for (int i = 0; i < (1 << kFan) - 1; ++i)
                    if (first + i < at) w[i] = look(a.nodes + node_at(a, l, first + i, c0 + c));
#pragma unroll
                for (int i = 0; i < (1 << kFan) - 1; ++i)
                    if (first + i < at)
                        lm = then(lm, awaited(a.nodes + node_at(a, l, first + i, c0 + c), w[i], a.head));
            }
            s.la[l][c] = lm.a;
            s.lb[l][c] = lm.b;
        }
    }
    if (more && (wanted || parent)) {
        __syncthreads();
        if (g == 0 && real) {
            // the nodes that end with this tile
            Map node = own;
            for (int l = 0; l + 1 < a.tree.levels; ++l) {
                if (((v >> (kFan * l)) & ((1 << kFan) - 1)) != (1 << kFan) - 1) break;
                if (!sealed) node = then(Map{s.la[l][c], s.lb[l][c]}, node);
                publish(a.nodes + node_at(a, l + 1, v >> (kFan * (l + 1)), c0 + c), node);
            }
        }
    }
    if (g == 0) {
        float h = 0.f;
        if (wanted && !alone)
            for (int l = a.tree.levels - 1; l >= 0; --l) h = through(Map{s.la[l][c], s.lb[l][c]}, h);
        for (int i = 0; i < J::kGroups; ++i) {
            s.enter[i][c] = h;
            h = through(Map{s.ga[i][c], s.gb[i][c]}, h);
        }
    }
    __syncthreads();
}

template <typename T>
__device__ __forceinline__ void unpack(uint4 v, float (&x)[16 / sizeof(T)]) {
    const T* e = reinterpret_cast<const T*>(&v);
#pragma unroll
    for (int j = 0; j < 16 / (int)sizeof(T); ++j) x[j] = to_f32<T>(e[j]);
}
template <typename T>
__device__ __forceinline__ uint4 pack(const float (&x)[16 / sizeof(T)]) {
    uint4 v;
    T* e = reinterpret_cast<T*>(&v);
#pragma unroll
    for (int j = 0; j < 16 / (int)sizeof(T); ++j) e[j] = from_f32<T>(x[j]);
    return v;
}
template <int V>
__device__ __forceinline__ void load_state(const float* p, float (&h)[V]) {
#pragma unroll
    for (int j = 0; j < V; j += 4) {
        const float4 f = p ? *reinterpret_cast<const float4*>(p + j) : make_float4(0.f, 0.f, 0.f, 0.f);
        h[j] = f.x, h[j + 1] = f.y, h[j + 2] = f.z, h[j + 3] = f.w;
    }
}
template <int V>
__device__ __forceinline__ void store_state(float* p, const float (&h)[V]) {
#pragma unroll
    for (int j = 0; j < V; j += 4) *reinterpret_cast<float4*>(p + j) = make_float4(h[j], h[j + 1], h[j + 2], h[j + 3]);
}

// Row of visit v, or -1 where the order names none.
__device__ __forceinline__ int64_t row_of(const ScanArgs& a, int64_t v) {
    const int64_t p = a.reverse ? a.n - 1 - v : v;
    if (!a.order) return p;
    const int32_t r = a.order[p];
    return r >= 0 && r < a.n ? r : -1;
}

// The block's next unit of work, in the order of the counter.
__device__ __forceinline__ int64_t next_unit(const ScanArgs& a) {
    __shared__ uint32_t s_unit;
    if (threadIdx.x == 0) s_unit = atomicAdd(a.head + 2, 1u);
    __syncthreads();
    return s_unit;
}

template <typename T>
__global__ void __launch_bounds__(kThreads, 2) k_scan_fwd(const ScanArgs a) {
    constexpr int V = 16 / (int)sizeof(T), CH = kLanes * V, S = kFwdTokens;
    __shared__ Cuts<kFwdTile> s_cuts;
    extern __shared__ float4 s_dyn[];
    Joint<CH>& s = *reinterpret_cast<Joint<CH>*>(s_dyn);
    if (a.head[1] != 0) return;  // bad offsets
    const int64_t unit = next_unit(a);
    const int64_t v = unit / a.blocks_c;
    const int c0 = (int)(unit - v * a.blocks_c) * CH;
    const int64_t lo = v * kFwdTile, hi = min(lo + kFwdTile, a.n);
    const int lane = threadIdx.x % kLanes, row = threadIdx.x / kLanes;
    const int c = c0 + lane * V;
    const bool real = c < a.c;

    int64_t at[S];
    uint4 gv[S], xv[S];
    const int64_t t0 = lo + row * S;
#pragma unroll
    for (int k = 0; k < S; ++k) {
        at[k] = t0 + k < hi && real ? row_of(a, t0 + k) : -1;
        if (at[k] < 0 && t0 + k < hi && real) atomicOr(a.head, kErrRange);
        gv[k] = xv[k] = make_uint4(0, 0, 0, 0);
        if (at[k] >= 0) {
            gv[k] = *reinterpret_cast<const uint4*>(a.gate + (at[k] * a.gate_s + c) * (int)sizeof(T));
            xv[k] = *reinterpret_cast<const uint4*>(a.x + (at[k] * a.x_s + c) * (int)sizeof(T));
        }
    }
    find_cuts<kFwdTile>(a, s_cuts, lo, hi, hi == a.n, c0, min(CH, a.c - c0), a.first, a.last);
    const uint32_t begin = bits<S>(s_cuts.begin, row * S), end = bits<S>(s_cuts.end, row * S);
    const int count = (int)max((int64_t)0, min((int64_t)S, hi - t0));

    float A[V], B[V];
#pragma unroll
    for (int j = 0; j < V; ++j) A[j] = 1.f, B[j] = 0.f;
#pragma unroll
    for (int k = 0; k < S; ++k) {
        if (k < count) {
            float g[V], x[V];
            unpack<T>(gv[k], g);
            unpack<T>(xv[k], x);
            if (begin >> k & 1) {
                float h[V];
                load_state<V>(a.first && real ? a.first + (int64_t)s_cuts.begin_seq[row * S + k] * a.c + c : nullptr, h);
#pragma unroll
                for (int j = 0; j < V; ++j) A[j] = -1.f, B[j] = h[j];
            }
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float m = side<T>(g[j]);
                B[j] = kept(m, B[j]) + (a.free_input ? x[j] : added(m) * x[j]);
                if (!(A[j] < 0.f)) A[j] = kept(m, A[j]);
            }
        }
    }
#pragma unroll
    for (int j = 0; j < V; ++j) s.a[row][lane * V + j] = A[j], s.b[row][lane * V + j] = B[j];

    uint32_t any = 0;
    for (int i = 0; i < kFwdTile / 32; ++i) any |= s_cuts.begin[i];
    join<CH>(a, s, v, c0, false, s_cuts.begin[0] & 1, any != 0);

    float h[V];
#pragma unroll
    for (int j = 0; j < V; ++j) {
        const int i = lane * V + j;
        h[j] = through(Map{s.a[row][i], s.b[row][i]}, s.enter[row / Joint<CH>::kSpan][i]);
    }
    if (!real) return;
    if (a.carries && count > 0 && t0 % kScanCarryRows == 0)
        store_state<V>(a.carries + t0 / kScanCarryRows * a.c + c, h);
#pragma unroll
    for (int k = 0; k < S; ++k) {
        if (k < count) {
            float g[V], x[V];
            unpack<T>(gv[k], g);
            unpack<T>(xv[k], x);
            if (begin >> k & 1)
                load_state<V>(a.first ? a.first + (int64_t)s_cuts.begin_seq[row * S + k] * a.c + c : nullptr, h);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float m = side<T>(g[j]);
                h[j] = kept(m, h[j]) + (a.free_input ? x[j] : added(m) * x[j]);
            }
            if (at[k] >= 0) *reinterpret_cast<uint4*>(a.out + (at[k] * a.out_s + c) * (int)sizeof(T)) = pack<T>(h);
            if (a.last && (end >> k & 1))
                store_state<V>(a.last + (int64_t)s_cuts.end_seq[row * S + k] * a.c + c, h);
        }
    }
}

// The backward pass goes through the tiles, and through each tile's rows, from the end.  The
// states are found again from those that the forward pass kept at the tiles' beginnings.
template <typename T>
__global__ void __launch_bounds__(kThreads, 2) k_scan_bwd(const ScanArgs a) {
    constexpr int V = 16 / (int)sizeof(T), CH = kLanes * V, S = kBwdTokens;
    using J = Joint<CH>;
    __shared__ Cuts<kBwdTile> s_cuts;
    extern __shared__ float4 s_dyn[];
    J& s = *reinterpret_cast<J*>(s_dyn);
    float(*fa)[CH] = reinterpret_cast<float(*)[CH]>(&s + 1);  // the forward maps of the rows
    float(*fb)[CH] = fa + kRows;
    float(*ge)[CH] = fb + kRows;                              // [2][kGroups] the groups' forward maps
    if (a.head[1] != 0) return;
    const int64_t unit = next_unit(a);
    const int64_t v = unit / a.blocks_c;                      // 0: the last tile
    const int c0 = (int)(unit - v * a.blocks_c) * CH;
    const int64_t tile = a.tree.tiles - 1 - v;
    const int64_t lo = tile * kBwdTile, hi = min(lo + kBwdTile, a.n);
    const int lane = threadIdx.x % kLanes, row = threadIdx.x / kLanes;
    const int c = c0 + lane * V;
    const bool real = c < a.c;

    int64_t at[S];
    uint4 gv[S], xv[S], yv[S];
    const int64_t t0 = lo + row * S;
#pragma unroll
    for (int k = 0; k < S; ++k) {
        at[k] = t0 + k < hi && real ? row_of(a, t0 + k) : -1;
        if (at[k] < 0 && t0 + k < hi && real) atomicOr(a.head, kErrRange);
        gv[k] = xv[k] = yv[k] = make_uint4(0, 0, 0, 0);
        if (at[k] >= 0) {
            gv[k] = *reinterpret_cast<const uint4*>(a.gate + (at[k] * a.gate_s + c) * (int)sizeof(T));
            xv[k] = *reinterpret_cast<const uint4*>(a.x + (at[k] * a.x_s + c) * (int)sizeof(T));
            yv[k] = *reinterpret_cast<const uint4*>(a.gy + (at[k] * a.gy_s + c) * (int)sizeof(T));
        }
    }
    float enter[V];
    load_state<V>(real && lo < hi ? a.carries + tile * a.c + c : nullptr, enter);
    find_cuts<kBwdTile>(a, s_cuts, lo, hi, hi == a.n, c0, min(CH, a.c - c0), a.glast, a.gfirst);
    const uint32_t begin = bits<S>(s_cuts.begin, row * S), end = bits<S>(s_cuts.end, row * S);
    const int count = (int)max((int64_t)0, min((int64_t)S, hi - t0));

    {
        float A[V], B[V], G[V], D[V];  // h -> A h + B forwards, mu -> G mu + D backwards
#pragma unroll
        for (int j = 0; j < V; ++j) A[j] = G[j] = 1.f, B[j] = D[j] = 0.f;
#pragma unroll
        for (int k = 0; k < S; ++k) {
            if (k < count) {
                float g[V], x[V], y[V];
                unpack<T>(gv[k], g);
                unpack<T>(xv[k], x);
                unpack<T>(yv[k], y);
                if (begin >> k & 1) {
                    float h[V];
                    load_state<V>(a.first && real ? a.first + (int64_t)s_cuts.begin_seq[row * S + k] * a.c + c : nullptr,
                                  h);
#pragma unroll
                    for (int j = 0; j < V; ++j) A[j] = -1.f, B[j] = h[j];
                }
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    const float m = side<T>(g[j]);
                    B[j] = kept(m, B[j]) + (a.free_input ? x[j] : added(m) * x[j]);
                    if (!(A[j] < 0.f)) A[j] = kept(m, A[j]);
                }
            }
        }
#pragma unroll
        for (int k = S - 1; k >= 0; --k) {
            if (k < count) {
                float g[V], y[V];
                unpack<T>(gv[k], g);
                unpack<T>(yv[k], y);
                if (end >> k & 1) {
                    float h[V];
                    load_state<V>(a.glast && real ? a.glast + (int64_t)s_cuts.end_seq[row * S + k] * a.c + c : nullptr,
                                  h);
#pragma unroll
                    for (int j = 0; j < V; ++j) G[j] = -1.f, D[j] = h[j];
                }
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    const float m = side<T>(g[j]);
                    D[j] = kept(m, y[j] + D[j]);
                    if (!(G[j] < 0.f)) G[j] = kept(m, G[j]);
                }
            }
        }
#pragma unroll
        for (int j = 0; j < V; ++j) {
            s.a[row][lane * V + j] = G[j];
            s.b[row][lane * V + j] = D[j];
            fa[row][lane * V + j] = A[j];
            fb[row][lane * V + j] = B[j];
        }
    }
    __syncthreads();
    {   // the forward maps: rows of a group, then groups
        const int cc = threadIdx.x % CH, g = threadIdx.x / CH;
        Map m{1.f, 0.f};
        for (int i = g * J::kSpan; i < (g + 1) * J::kSpan; ++i) {
            const Map mine{fa[i][cc], fb[i][cc]};
            fa[i][cc] = m.a;
            fb[i][cc] = m.b;
            m = then(m, mine);
        }
        ge[g][cc] = m.a;
        ge[J::kGroups + g][cc] = m.b;
    }
    uint32_t any = 0;
    for (int i = 0; i < kBwdTile / 32; ++i) any |= s_cuts.end[i];
    const int lastv = (int)(hi - 1 - lo);
    const bool alone = hi == lo || (s_cuts.end[lastv >> 5] >> (lastv & 31) & 1);
    join<CH>(a, s, v, c0, true, alone, any != 0);
    if (!real) return;

    float before[S][V], h[V], mu[V];
#pragma unroll
    for (int j = 0; j < V; ++j) {
        const int i = lane * V + j;
        h[j] = enter[j];
        for (int g = 0; g < row / J::kSpan; ++g) h[j] = through(Map{ge[g][i], ge[J::kGroups + g][i]}, h[j]);
        h[j] = through(Map{fa[row][i], fb[row][i]}, h[j]);
        mu[j] = through(Map{s.a[row][i], s.b[row][i]}, s.enter[(kRows - 1 - row) / J::kSpan][i]);
    }
#pragma unroll
    for (int k = 0; k < S; ++k) {
        if (k < count) {
            float g[V], x[V];
            unpack<T>(gv[k], g);
            unpack<T>(xv[k], x);
            if (begin >> k & 1)
                load_state<V>(a.first ? a.first + (int64_t)s_cuts.begin_seq[row * S + k] * a.c + c : nullptr, h);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float m = side<T>(g[j]);
                before[k][j] = h[j];
                h[j] = kept(m, h[j]) + (a.free_input ? x[j] : added(m) * x[j]);
            }
        }
    }
#pragma unroll
    for (int k = S - 1; k >= 0; --k) {
        if (k < count) {
            float g[V], x[V], y[V], dg[V], dx[V];
            unpack<T>(gv[k], g);
            unpack<T>(xv[k], x);
            unpack<T>(yv[k], y);
            if (end >> k & 1)
                load_state<V>(a.glast ? a.glast + (int64_t)s_cuts.end_seq[row * S + k] * a.c + c : nullptr, mu);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float m = side<T>(g[j]);
                const float lam = y[j] + mu[j];
                dg[j] = slope(m) * (a.free_input ? before[k][j] : before[k][j] - x[j]) * lam;
                dx[j] = a.free_input ? lam : added(m) * lam;
                mu[j] = kept(m, lam);
            }
            if (at[k] >= 0) {
                *reinterpret_cast<uint4*>(a.gg + (at[k] * a.gg_s + c) * (int)sizeof(T)) = pack<T>(dg);
                *reinterpret_cast<uint4*>(a.out + (at[k] * a.out_s + c) * (int)sizeof(T)) = pack<T>(dx);
            }
            if (a.gfirst && (begin >> k & 1))
                store_state<V>(a.gfirst + (int64_t)s_cuts.begin_seq[row * S + k] * a.c + c, mu);
        }
    }
}

// Before the pass: nodes unset, counter at zero, and the verdict on the offsets, which the first
// block alone reaches (0 and n at the ends, never falling).
__global__ void __launch_bounds__(1024) k_scan_begin(const ScanArgs a, int64_t words) {
    for (int64_t i = (int64_t)blockIdx.x * 1024 + threadIdx.x; i < words; i += (int64_t)gridDim.x * 1024)
        a.nodes[i] = kUnset;
    if (blockIdx.x > 0) return;
    bool bad = false;
    for (int64_t i = threadIdx.x; i < a.batch; i += 1024) {
        const int32_t p = a.off[i], q = a.off[i + 1];
        bad |= p > q || (i == 0 && p != 0) || (i == a.batch - 1 && q != a.n);
    }
    const int any = __syncthreads_or(bad);
    if (threadIdx.x == 0) {
        a.head[1] = any ? 1u : 0u;
        a.head[2] = 0;
        if (any) atomicOr(a.head, kErrRange);
    }
}

template <typename T>
__global__ void __launch_bounds__(kThreads) k_scan_step(int64_t vectors, int per_row, int c, int free_input,
                                                        const char* gate, int64_t gate_s, const char* x, int64_t x_s,
                                                        float* state, char* out, int64_t out_s) {
    constexpr int V = 16 / (int)sizeof(T);
    for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < vectors; i += (int64_t)gridDim.x * kThreads) {
        const int64_t r = i / per_row;
        const int at = (int)(i - r * per_row) * V;
        float g[V], xx[V], h[V];
        unpack<T>(*reinterpret_cast<const uint4*>(gate + (r * gate_s + at) * (int)sizeof(T)), g);
        unpack<T>(*reinterpret_cast<const uint4*>(x + (r * x_s + at) * (int)sizeof(T)), xx);
        float* sp = state + r * c + at;
        load_state<V>(sp, h);
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const float m = side<T>(g[j]);
            h[j] = kept(m, h[j]) + (free_input ? xx[j] : added(m) * xx[j]);
        }
        store_state<V>(sp, h);
        *reinterpret_cast<uint4*>(out + (r * out_s + at) * (int)sizeof(T)) = pack<T>(h);
    }
}

Tree tree_of(int64_t n, int c, int tile, int64_t* words) {
    Tree t{};
    t.tiles = std::max<int64_t>(1, (n + tile - 1) / tile);
    int64_t at = 0;
    for (t.levels = 0; t.levels < kMaxLevels; ++t.levels) {
        if (t.levels > 0 && ((t.tiles - 1) >> (kFan * t.levels)) == 0) break;
        t.base[t.levels] = at;
        at += ((t.tiles - 1) >> (kFan * t.levels)) * c + c;
    }
    *words = t.tiles > 1 ? at : 0;
    return t;
}

template <typename T>
int launch(const ScanArgs& a, bool bwd, cudaStream_t s) {
    constexpr int CH = kLanes * 16 / (int)sizeof(T);
    const size_t smem = sizeof(Joint<CH>) + (bwd ? (size_t)(2 * kRows + 2 * Joint<CH>::kGroups) * CH * 4 : 0);
    auto kernel = bwd ? k_scan_bwd<T> : k_scan_fwd<T>;
    if (smem > 32 * 1024 &&
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess)
        return VG_ERR_CUDA;
    kernel<<<(unsigned)a.units, kThreads, smem, s>>>(a);
    return cudaPeekAtLastError() == cudaSuccess ? VG_OK : VG_ERR_CUDA;
}

}  // namespace

size_t gated_scan_workspace_bytes(int64_t n, int c) {
    int64_t words;
    tree_of(n, c, kBwdTile, &words);
    return align_up(256 + (size_t)words * 8, 256);
}

int gated_scan(const GatedScan& q, bool bwd, cudaStream_t s) {
    ScanArgs a{};
    const int es = q.s->dtype == VG_F32 ? 4 : 2;
    a.n = q.s->n;
    a.c = q.s->channels;
    a.batch = q.s->batch;
    a.blocks_c = (a.c * es + 127) / 128;
    a.off = q.s->offsets;
    a.order = q.s->order;
    a.reverse = (q.s->flags & VG_SCAN_REVERSE) != 0;
    a.free_input = (q.s->flags & VG_SCAN_FREE_INPUT) != 0;
    const auto in = [](const vg_rows* r, const char** p, int64_t* stride) {
        *p = r ? static_cast<const char*>(r->data) : nullptr;
        *stride = r ? r->row_stride : 0;
    };
    const auto out = [](const vg_rows* r, char** p, int64_t* stride) {
        *p = r ? static_cast<char*>(r->data) : nullptr;
        *stride = r ? r->row_stride : 0;
    };
    in(q.gate, &a.gate, &a.gate_s);
    in(q.x, &a.x, &a.x_s);
    in(q.grad_out, &a.gy, &a.gy_s);
    out(q.out, &a.out, &a.out_s);
    out(q.grad_gate, &a.gg, &a.gg_s);
    a.first = q.first;
    a.glast = q.grad_last;
    a.last = q.last;
    a.carries = q.carries;
    a.gfirst = q.grad_first;
    a.head = reinterpret_cast<uint32_t*>(q.ws);
    a.nodes = reinterpret_cast<uint64_t*>(q.ws + 256);
    int64_t words;
    a.tree = tree_of(a.n, a.c, bwd ? kBwdTile : kFwdTile, &words);
    a.units = a.tree.tiles * a.blocks_c;
    if (a.units >= (int64_t(1) << 31)) return VG_ERR_UNSUPPORTED;
    const int64_t fill = std::max<int64_t>(1, std::min<int64_t>((words + 4095) / 4096, q.sms));
    k_scan_begin<<<(unsigned)fill, 1024, 0, s>>>(a, words);
    if (cudaPeekAtLastError() != cudaSuccess) return VG_ERR_CUDA;
    return q.s->dtype == VG_F32   ? launch<float>(a, bwd, s)
           : q.s->dtype == VG_F16 ? launch<__half>(a, bwd, s)
                                  : launch<__nv_bfloat16>(a, bwd, s);
}

int gated_scan_step(int64_t n, int c, int dtype, bool free_input, const vg_rows& gate, const vg_rows& x, float* state,
                    const vg_rows& out, cudaStream_t s) {
    const int v = dtype == VG_F32 ? 4 : 8;
    const int64_t vectors = n * (c / v);
    const int grid = (int)std::min<int64_t>((vectors + kThreads - 1) / kThreads, 152 * 8);
    const auto run = [&](auto kernel) {
        kernel<<<grid, kThreads, 0, s>>>(vectors, c / v, c, (int)free_input, static_cast<const char*>(gate.data),
                                         gate.row_stride, static_cast<const char*>(x.data), x.row_stride, state,
                                         static_cast<char*>(out.data), out.row_stride);
        return cudaPeekAtLastError() == cudaSuccess ? VG_OK : VG_ERR_CUDA;
    };
    return dtype == VG_F32   ? run(k_scan_step<float>)
           : dtype == VG_F16 ? run(k_scan_step<__half>)
                             : run(k_scan_step<__nv_bfloat16>);
}

}  // namespace vg
