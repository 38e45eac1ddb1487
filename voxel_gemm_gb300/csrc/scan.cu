// Gated linear recurrence of each channel along each sequence, and its gradient.
//
//   a = sigmoid(gate),  h_t = a_t h_{t-1} + b_t,  b_t = (1 - a_t) x_t  (or x_t)
// backward: lam_t = dy_t + mu_{t+1}, mu_t = a_t lam_t;  db = lam, da = h_{t-1} lam (- x lam)
//
// A run of tokens maps the state that enters it to the one that leaves it, h -> A h + B, and two
// runs after one another make (A2 A1, A2 B1 + B2): so the positions are cut into tiles that work
// side by side.  A block takes a tile of 128 positions and 128 bytes of channels: a warp's lanes hold
// a token's channels, 4 bytes each, and a warp goes along 16 tokens.  It finds the map of its
// tokens; the block joins the warps' maps in shared memory, publishes the tile's map, collects
// those of the tiles before it, and each warp goes through its tokens again from the state that
// enters.  What a token's gate gives stays in registers between the two passes.
// Bound by memory: gate and x are read once, out written once.  Each warp copies its own tokens of
// the block's next tile into shared memory while it works on this one.
//
// The maps of earlier tiles are collected through a tree: node (l, i) is the map of the 8^l tiles
// from i 8^l on; tile j reads, at each level, the siblings before its own ancestor, at most 7,
// and the last tile below a node publishes that node.  So the shape of every sum depends on the
// sizes alone (the same bits in every run), and a tile waits for about as many hand-overs as there
// are levels.  A node's word holds A and B, 64 bits that are stored at once; words are all ones
// before they are written (a NaN that no result has), so the data is its own flag.  Blocks
// take their tiles in order from a counter, the next one when this one's tokens are there: the
// first tile that is not done was taken by a block that works on it and has all that it waits for.
// (Two tiles taken at once at the start left every second tile to a block still waiting for the
// first, a chain through all blocks: 602k tokens of 512 channels took 4.5 ms.)  Waits are bounded by time; a block that
// gives up records it and goes on with NaN.
//
// Where a sequence begins, the map is constant (A = -1 marks it, h -> B), so that nothing, not
// even a NaN, passes from one sequence to the next.  A warp's tokens are the same for all of its
// lanes, so such places cost a branch that no lane takes alone.
#include "common.cuh"
#include "internal.h"
#include "tc_ptx.cuh"

namespace vg {

namespace {

using namespace ptx;

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kTokens = 16;                  // of a warp
constexpr int kTile = kWarps * kTokens;
constexpr int kRowBytes = 128;               // of a token in a block: 64 16-bit or 32 fp32 channels
constexpr int kTileBytes = kTile * kRowBytes;
constexpr int kFan = 3;                      // log2 of a node's children
constexpr int kSiblings = (1 << kFan) - 1;
constexpr int kMaxLevels = 8;                // 128 * 8^8 positions are more than 2^31
constexpr uint64_t kUnset = ~0ull;
constexpr uint64_t kGiveUpNs = 2000000000;
static_assert(kTile == kScanCarryRows, "states are kept where the tiles begin");
static_assert(kMaxLevels <= kWarps, "a warp collects a level");
constexpr int kFwdStages = 3;                // tiles in shared memory: being read, finished, waited for
constexpr int kBlocksPerSm = 2;              // by shared memory (96 KB of tiles) and registers (128 a thread)

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
    uint32_t gate_s, x_s, gy_s, out_s, gg_s;  // strides in bytes
    const float* first;
    const float* glast;
    float *last, *carries, *gfirst;
    uint32_t* head;
    uint64_t* nodes;
    Tree tree;
    uint32_t units;
};

// ---------------------------------------------------------------- a lane's channels
// Two channels (16-bit types) or one, in fp32; two are worked on by paired instructions.
__device__ __forceinline__ float2 fma_(float2 a, float2 b, float2 c) { return fma2(a, b, c); }
__device__ __forceinline__ float fma_(float a, float b, float c) { return fmaf(a, b, c); }
__device__ __forceinline__ float2 add_(float2 a, float2 b) { return add2(a, b); }
__device__ __forceinline__ float add_(float a, float b) { return a + b; }
__device__ __forceinline__ float2 mul_(float2 a, float2 b) { return mul2(a, b); }
__device__ __forceinline__ float mul_(float a, float b) { return a * b; }
__device__ __forceinline__ float2 neg_(float2 a) { return make_float2(-a.x, -a.y); }
__device__ __forceinline__ float neg_(float a) { return -a; }

template <typename N> struct Side;
struct Rest;
template <typename T> struct Lane;
template <> struct Lane<float> {
    using Num = float;
    static constexpr int V = 1;
    static __device__ __forceinline__ float unpack(uint32_t w) { return __uint_as_float(w); }
    static __device__ __forceinline__ uint32_t pack(float x) { return __float_as_uint(x); }
    static __device__ __forceinline__ float fill(float x) { return x; }
    using Fast = Side<float>;
    static __device__ __forceinline__ float load(const float* p) { return *p; }
    static __device__ __forceinline__ void store(float* p, float x) { *p = x; }
};
template <typename T> struct Lane16 {
    using Num = float2;
    using Fast = Rest;
    static constexpr int V = 2;
    static __device__ __forceinline__ float2 fill(float x) { return make_float2(x, x); }
    static __device__ __forceinline__ float2 load(const float* p) { return *reinterpret_cast<const float2*>(p); }
    static __device__ __forceinline__ void store(float* p, float2 x) { *reinterpret_cast<float2*>(p) = x; }
};
template <> struct Lane<__half> : Lane16<__half> {
    static __device__ __forceinline__ float2 unpack(uint32_t w) {
        return __half22float2(*reinterpret_cast<const __half2*>(&w));
    }
    static __device__ __forceinline__ uint32_t pack(float2 x) {
        const __half2 h = __floats2half2_rn(x.x, x.y);
        return *reinterpret_cast<const uint32_t*>(&h);
    }
};
template <> struct Lane<__nv_bfloat16> : Lane16<__nv_bfloat16> {
    static __device__ __forceinline__ float2 unpack(uint32_t w) {
        return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
    }
    static __device__ __forceinline__ uint32_t pack(float2 x) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(x.x, x.y);
        return *reinterpret_cast<const uint32_t*>(&h);
    }
};

// What a token's gate does to a state.  Two forms:
//
// Side: m = e / (1 + e) with e = exp(-|g|), the smaller of a = sigmoid(g) and 1 - a, held as m
// (a = m, for g < 0) or as -m (a = 1 - m).  Everything follows without cancellation, but each use
// has to look at the sign: 13 instructions an element to find a run's map, 8 to apply it.
//
// Rest: s = 1 - a = 1 / (1 + exp(g)), and a h = h - s h in one rounding.  Exact at s = 0 and 1,
// and no coarser than the other where a is near one, so long memories keep their length; near s = 1 what is
// left of a state is off by 2^-24 of the state (of h_{t-1}, not of what is left).  8 and 5
// instructions.  The forward pass takes it for 16-bit types, which have a floor of 6 bytes an
// element, or some 30 instructions; fp32 (12 bytes) and the backward pass (10), whose slope a (1 - a) would
// lose its small values, take the first.
//
// 16-bit types take the fast exponential and reciprocal, off by 2 units and |g| / 2^24, and by 1:
// 1e-6 of m for |g| < 10, where the inputs have 2^-9 or 2^-12.
template <typename N> struct Side {
    using Held = N;
    N m, one;  // one: 1 where a is 1 - m, 0 where it is m
    static __device__ __forceinline__ float with_side(float m, float g) {
        return __uint_as_float((__float_as_uint(m) & 0x7fffffffu) | (~__float_as_uint(g) & 0x80000000u));
    }
    static __device__ __forceinline__ float hold(float g) {
        const float e = expf(-fabsf(g));
        return with_side(e / (1.f + e), g);
    }
    static __device__ __forceinline__ float2 hold(float2 g) {
        float2 e, r;
        asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.x) : "f"(fabsf(g.x) * -1.4426950408889634f));
        asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.y) : "f"(fabsf(g.y) * -1.4426950408889634f));
        const float2 d = add2(e, make_float2(1.f, 1.f));
        asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r.x) : "f"(d.x));
        asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r.y) : "f"(d.y));
        const float2 m = mul2(e, r);
        return make_float2(with_side(m.x, g.x), with_side(m.y, g.y));
    }
    static __device__ __forceinline__ float near_one(float m) {
        return __uint_as_float((uint32_t)((int32_t)__float_as_uint(m) >> 31) & 0x3f800000u);
    }
    static __device__ __forceinline__ float2 near_one(float2 m) { return make_float2(near_one(m.x), near_one(m.y)); }
    static __device__ __forceinline__ float rest(float m, float one) { return (1.f - one) - m; }
    static __device__ __forceinline__ float2 rest(float2 m, float2 one) {
        const float2 n = make_float2(-1.f, -1.f), u = make_float2(1.f, 1.f);
        return fma2(m, n, fma2(one, n, u));
    }
    static __device__ __forceinline__ float slope(float m) { return fmaf(-fabsf(m), fabsf(m), fabsf(m)); }
    static __device__ __forceinline__ float2 slope(float2 m) { return make_float2(slope(m.x), slope(m.y)); }

    __device__ __forceinline__ explicit Side(Held held) : m(held), one(near_one(held)) {}
    __device__ __forceinline__ N kept(N h) const { return fma_(m, h, mul_(one, h)); }  // a h
    __device__ __forceinline__ N rest() const { return rest(m, one); }                 // 1 - a
    __device__ __forceinline__ N slope() const { return slope(m); }                    // a (1 - a)
};
struct Rest {
    using Held = float2;
    float2 s, minus;
    static __device__ __forceinline__ float2 hold(float2 g) {
        float2 e, s;
        const float2 y = mul2(g, make_float2(1.4426950408889634f, 1.4426950408889634f));
        asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.x) : "f"(y.x));
        asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.y) : "f"(y.y));
        const float2 d = add2(e, make_float2(1.f, 1.f));
        asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(s.x) : "f"(d.x));
        asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(s.y) : "f"(d.y));
        return s;
    }
    __device__ __forceinline__ explicit Rest(Held held) : s(held), minus(mul2(held, make_float2(-1.f, -1.f))) {}
    __device__ __forceinline__ float2 kept(float2 h) const { return fma2(minus, h, h); }
    __device__ __forceinline__ float2 rest() const { return s; }
};
// The state after a token.
template <bool FREE, typename G, typename N> __device__ __forceinline__ N next_state(const G& g, N x, N h) {
    if constexpr (FREE) return add_(g.kept(h), x);
    return fma_(g.rest(), x, g.kept(h));
}

// ---------------------------------------------------------------- maps of runs of tokens
// h -> A h + B; A = -1: h -> B.
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
__device__ __noinline__ uint64_t awaited(const uint64_t* node, uint32_t* record) {
    const uint64_t t0 = globaltimer();
    for (int spins = 0;; ++spins) {
        const uint64_t w = look(node);
        if (w != kUnset) return w;
        if ((spins & 63) == 63) {
            const bool late = globaltimer() - t0 > kGiveUpNs;
            if (late) atomicOr(record, kErrTimeout);
            if (late || (*reinterpret_cast<volatile uint32_t*>(record) & kErrTimeout))
                return (uint64_t)0x7fc00000u << 32 | 0xbf800000u;
        }
    }
}
__device__ __forceinline__ uint64_t* node_at(const ScanArgs& a, int l, int64_t i, int c) {
    return a.nodes + a.tree.base[l] + i * a.c + c;
}

// ---------------------------------------------------------------- beginnings and ends of sequences
// Where sequence b begins in the order of the visits (a sequence's visits are its positions,
// downwards all of them counted from the end), and which sequence that is.
__device__ __forceinline__ int64_t begins(const ScanArgs& a, int b) {
    return a.reverse ? a.n - a.off[a.batch - b] : a.off[b];
}
__device__ __forceinline__ int sequence(const ScanArgs& a, int b) { return a.reverse ? a.batch - 1 - b : b; }

// What a warp's visits [lo, lo + count) hold of them: a bit per visit, and the sequences.
struct Cuts {
    uint32_t begin, end;
};
struct CutSeqs {
    int32_t begin[kTokens];  // the sequence that begins there
    int32_t entering;        // the one that goes on into the visits
    __device__ __forceinline__ int end(const Cuts& c, int k) const {  // the one that ends there
        const uint32_t until = c.begin & ((2u << k) - 1);
        return until ? begin[31 - __clz(until)] : entering;
    }
};

// Positions of the sequence that a warp looked up last: visits inside of it need no search.
struct Within {
    int64_t from = 0, to = 0;
};

// Sequences without tokens that lie here hand their state `in` on to `out` (each may be null).
template <int V>
__device__ __forceinline__ Cuts find_cuts(const ScanArgs& a, CutSeqs& s, Within& w, int64_t lo, int count, int c,
                                          const float* in, float* out) {
    const int lane = threadIdx.x & 31;
    const int64_t hi = lo + count;
    Cuts r{0u, 0u};
    if (lo > w.from && hi < w.to) return r;
    const bool last = hi == a.n && (count > 0 || (lo == 0 && threadIdx.x < 32));  // the visits' end lies here
    if (count == 0 && !last) return r;
    // the number of sequences that begin before lo, 32 probes at a time
    int from = 0, to = a.batch;
    while (to > from) {
        const int step = (to - from + 31) / 32;
        const int b = from + lane * step;
        const int before = __popc(__ballot_sync(0xffffffffu, b < to && begins(a, b) < lo));
        if (before == 0) {
            to = from;
        } else {
            const int hit = from + (before - 1) * step;  // begins before lo; the next probe does not
            from = hit + 1;
            to = min(to, hit + step);
        }
    }
    if (from > 0) {
        w.from = begins(a, from - 1);
        w.to = begins(a, from);
        s.entering = sequence(a, from - 1);
    }
    // those that begin here, and the one before them, which may end here
    for (int b0 = max(from - 1, 0);; b0 += 32) {
        const int b = b0 + lane;
        const bool real = b < a.batch;
        const int64_t p = real ? begins(a, b) : a.n, q = real ? begins(a, b + 1) : a.n;
        const bool here = real && (p < hi || (last && p == a.n));  // or before
        const int seq = sequence(a, b);
        const bool begin = real && q > p && p >= lo && p < hi, end = real && q > p && q > lo && q <= hi;
        if (begin) s.begin[p - lo] = seq;
        r.begin |= __reduce_or_sync(0xffffffffu, begin ? 1u << (p - lo) : 0u);
        r.end |= __reduce_or_sync(0xffffffffu, end ? 1u << (q - 1 - lo) : 0u);
        uint32_t none = __ballot_sync(0xffffffffu, here && q == p && p >= lo);
        while (out && none) {
            const int64_t at = (int64_t)__shfl_sync(0xffffffffu, seq, __ffs(none) - 1) * a.c + c;
            none &= none - 1;
            if (c < a.c) {
#pragma unroll
                for (int j = 0; j < V; ++j) out[at + j] = in ? in[at + j] : 0.f;
            }
        }
        if (!(__ballot_sync(0xffffffffu, here) >> 31)) break;
    }
    __syncwarp();
    return r;
}

// ---------------------------------------------------------------- the work of a block
// Maps of the warps (h -> A h + B), sealed ones marked, of two tiles, and the joined maps of the
// levels' siblings.
template <int CH, bool BWD>
struct Joint {
    float a[2][kWarps][CH], b[2][kWarps][CH];  // in the direction that goes from tile to tile
    float fa[BWD ? kWarps : 1][CH], fb[BWD ? kWarps : 1][CH];  // backward pass: along the visits
    CutSeqs seqs[2][kWarps];
    uint32_t unit;
    int reached;      // something reaches into the tile
    float la[1][CH];  // of each level, a and b in turn

    static constexpr size_t bytes(int levels) { return sizeof(Joint) + (2 * (size_t)levels - 1) * CH * 4; }
};

// A warp's tokens of a unit.
struct Share {
    uint32_t v;           // the tile's place in the order of the work
    int32_t lo, count;    // the warp's first visit, its tokens
    int32_t c0;           // the block's first channel
    int32_t row;          // of the token of this lane's number: -1 where there is none
    Cuts cuts;
    bool simple;          // all tokens there, nothing begins or ends among them
    bool reached, sealed; // of the tile: something reaches into it; its map is constant
};
template <int CH>
__device__ __forceinline__ Share share_of(const ScanArgs& a, uint32_t unit, bool from_end) {
    Share s;
    s.v = unit / (uint32_t)a.blocks_c;
    s.c0 = (int)(unit - s.v * (uint32_t)a.blocks_c) * CH;
    const int64_t tile = from_end ? a.tree.tiles - 1 - s.v : s.v;
    s.lo = (int32_t)min(tile * kTile + (threadIdx.x >> 5) * kTokens, a.n);
    s.count = min(kTokens, (int32_t)a.n - s.lo);
    const int lane = threadIdx.x & 31;
    s.row = -1;
    if (lane < s.count) {
        const int32_t p = a.reverse ? (int32_t)a.n - 1 - (s.lo + lane) : s.lo + lane;
        s.row = p;
        if (a.order) {
            s.row = a.order[p];
            if (s.row < 0 || s.row >= a.n) {
                s.row = -1;
                atomicOr(a.head, kErrRange);
            }
        }
    }
    return s;
}
// Copy the tokens' channels of one operand, [kTokens][128 bytes]; zeros where there is no row or channel.
template <typename T>
__device__ __forceinline__ void fetch(uint32_t to, const char* from, uint32_t stride, const Share& s, int c) {
    const int lane = threadIdx.x & 31, chunk = lane & 7;
    const int at = s.c0 * (int)sizeof(T) + chunk * 16;
#pragma unroll
    for (int i = 0; i < kTokens / 4; ++i) {
        const int r = i * 4 + (lane >> 3);
        const int row = __shfl_sync(0xffffffffu, s.row, r);
        const bool have = row >= 0 && at < c * (int)sizeof(T);
        cp_async16(to + r * kRowBytes + chunk * 16, have ? from + (uint64_t)(uint32_t)row * stride + at : from, have ? 16 : 0);
    }
}

// The block's units: the first at `first`, the others from the counter, one ahead.
__device__ __forceinline__ uint32_t claim(const ScanArgs& a) { return atomicAdd(a.head + 2, 1u); }

// False if the call's offsets are no partition of the positions.  With one tile (and no launch
// before this one) the block sees for itself.
__device__ __forceinline__ bool good_offsets(const ScanArgs& a) {
    if (a.tree.tiles > 1) return a.head[1] == 0;
    bool bad = false;
    for (int64_t i = threadIdx.x; i < a.batch; i += kThreads) {
        const int32_t p = a.off[i], q = a.off[i + 1];
        bad |= p > q || (i == 0 && p != 0) || (i == a.batch - 1 && q != a.n);
    }
    if (!__syncthreads_or(bad)) return true;
    if (threadIdx.x == 0) atomicOr(a.head, kErrRange);
    return false;
}

// The joined maps of the siblings before tile v's ancestor at a level, waited for.
template <int V>
__device__ __forceinline__ void siblings(const ScanArgs& a, int64_t v, int level, int c, Map (&m)[V]) {
#pragma unroll
    for (int j = 0; j < V; ++j) m[j] = Map{1.f, 0.f};
    if (c >= a.c) return;
    const int64_t at = v >> (kFan * level);
    const int before = (int)(at & kSiblings);
    const uint64_t* node = node_at(a, level, at - before, c);
    uint64_t w[kSiblings][V];
#pragma unroll
    for (int i = 0; i < kSiblings; ++i)
#pragma unroll
        for (int j = 0; j < V; ++j) w[i][j] = i < before ? look(node + (int64_t)i * a.c + j) : 0;
#pragma unroll
    for (int i = 0; i < kSiblings; ++i)
        if (i < before) {
#pragma unroll
            for (int j = 0; j < V; ++j) {
                if (w[i][j] == kUnset) w[i][j] = awaited(node + (int64_t)i * a.c + j, a.head);
                m[j] = then(m[j], map_of(w[i][j]));
            }
        }
}

// The first warp publishes the tile's map (the joined maps of the warps; BWD: the last one's first), and
// the nodes that end with the tile, each as soon as the levels below it are there.  (When a block
// waited for all levels before it published any, each group of 8 tiles waited for the one before:
// 4.9 M tokens of 64 channels took 7.1 ms.)
template <int CH, bool BWD>
__device__ __forceinline__ void publish_nodes(const ScanArgs& a, const Joint<CH, BWD>& s, int parity, uint32_t v,
                                              int c0, bool sealed) {
    constexpr int V = CH / 32;
    const int cl = (int)threadIdx.x * V, c = c0 + cl;
    Map own[V];
#pragma unroll
    for (int j = 0; j < V; ++j) {
        own[j] = Map{1.f, 0.f};
#pragma unroll
        for (int i = 0; i < kWarps; ++i) {
            const int w = BWD ? kWarps - 1 - i : i;
            own[j] = then(own[j], Map{s.a[parity][w][cl + j], s.b[parity][w][cl + j]});
        }
        if (c < a.c) publish(node_at(a, 0, v, c + j), own[j]);
    }
    for (int l = 0; l + 1 < a.tree.levels && ((v >> (kFan * l)) & kSiblings) == kSiblings; ++l) {
        if (!sealed) {
            Map m[V];
            siblings<V>(a, v, l, c, m);
#pragma unroll
            for (int j = 0; j < V; ++j) own[j] = then(m[j], own[j]);
        }
#pragma unroll
        for (int j = 0; j < V; ++j)
            if (c < a.c) publish(node_at(a, l + 1, v >> (kFan * (l + 1)), c + j), own[j]);
    }
}

// Collect the maps of the tiles before this one, a level to a warp.
template <int CH, bool BWD>
__device__ __forceinline__ void collect(const ScanArgs& a, Joint<CH, BWD>& s, uint32_t v, int c0) {
    constexpr int V = CH / 32;
    const int level = kWarps - 1 - (threadIdx.x >> 5), cl = (threadIdx.x & 31) * V;
    if (level >= a.tree.levels) return;
    Map m[V];
    siblings<V>(a, v, level, c0 + cl, m);
#pragma unroll
    for (int j = 0; j < V; ++j) {
        s.la[2 * level][cl + j] = m[j].a;
        s.la[2 * level + 1][cl + j] = m[j].b;
    }
}

// h through a map of the lane's channels.
__device__ __forceinline__ float step_through(const float* a, const float* b, float h) {
    return through(Map{*a, *b}, h);
}
__device__ __forceinline__ float2 step_through(const float* a, const float* b, float2 h) {
    const float2 x = *reinterpret_cast<const float2*>(a), y = *reinterpret_cast<const float2*>(b);
    return make_float2(through(Map{x.x, y.x}, h.x), through(Map{x.y, y.y}, h.y));
}
// What enters this warp's tokens, from the levels' maps and those of the warps before it.
template <typename L, int CH, bool BWD>
__device__ __forceinline__ typename L::Num entering(const ScanArgs& a, const Joint<CH, BWD>& s, int parity,
                                                    bool reached) {
    const int warp = threadIdx.x >> 5, cl = (threadIdx.x & 31) * L::V;
    typename L::Num h = L::fill(0.f);
    if (reached)
        for (int l = a.tree.levels - 1; l >= 0; --l) h = step_through(&s.la[2 * l][cl], &s.la[2 * l + 1][cl], h);
    if constexpr (BWD) {
        for (int w = kWarps - 1; w > warp; --w) h = step_through(&s.a[parity][w][cl], &s.b[parity][w][cl], h);
    } else {
        for (int w = 0; w < warp; ++w) h = step_through(&s.a[parity][w][cl], &s.b[parity][w][cl], h);
    }
    return h;
}

// A block's first unit (one tile in all: its only one).
template <typename J>
__device__ __forceinline__ uint32_t first_unit(const ScanArgs& a, J& s) {
    if (a.tree.tiles == 1) return blockIdx.x;
    if (threadIdx.x == 0) s.unit = claim(a);
    __syncthreads();
    return s.unit;
}

__device__ __forceinline__ bool all_rows(const Share& s) {
    return __all_sync(0xffffffffu, s.row >= 0 || (threadIdx.x & 31) >= kTokens) && s.count == kTokens;
}
template <typename L>
__device__ __forceinline__ void put(char* base, int32_t row, uint32_t stride, typename L::Num x) {
    *reinterpret_cast<uint32_t*>(base + (uint64_t)(uint32_t)row * stride) = L::pack(x);
}
// The states of sequence `seq`, zero where there are none.
template <typename L>
__device__ __forceinline__ typename L::Num state_of(const ScanArgs& a, const float* states, int seq, int c) {
    return states && c < a.c ? L::load(states + (int64_t)seq * a.c + c) : L::fill(0.f);
}

// A block finds and publishes a tile's map before it finishes the tile before: by the time it wants
// to know what enters a tile, the blocks of the earlier tiles have long published theirs.  (With one
// tile at a time all blocks went through their phases in step, and waited together: 602k tokens
// of 512 channels took 1732 us forward and 1955 backward.)
template <typename T, bool FREE>
__global__ void __launch_bounds__(kThreads, kBlocksPerSm) k_scan_fwd(const ScanArgs a) {
    using L = Lane<T>;
    using N = typename L::Num;
    using G = typename L::Fast;
    constexpr int CH = 32 * L::V, kStep = kRowBytes / 4, kStage = 2 * kTileBytes;
    extern __shared__ __align__(128) char s_dyn[];  // [kFwdStages][gate, x][kTile][128 bytes], then the maps
    using J = Joint<CH, false>;
    J& s = *reinterpret_cast<J*>(s_dyn + kFwdStages * kStage);
    if (!good_offsets(a)) return;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, cl = lane * L::V;
    const bool many = a.tree.tiles > 1;
    const uint32_t unit = first_unit(a, s);
    if (unit >= a.units) return;
    char* const mine = s_dyn + warp * kTokens * kRowBytes;  // this warp's tokens in a stage
    const auto fetch_all = [&](int stage, const Share& of) {
        const uint32_t to = smem_u32(mine) + stage * kStage;
        fetch<T>(to, a.gate, a.gate_s, of, a.c);
        fetch<T>(to + kTileBytes, a.x, a.x_s, of, a.c);
    };
    Within within;
    Share now = share_of<CH>(a, unit, false), last{};
    typename G::Held held[kTokens];  // of the last tile
    fetch_all(0, now);
    bool have = true, pending = false;

    for (int turn = 0, stage = 0; have || pending; ++turn) {
        const int parity = turn & 1, next_stage = stage == kFwdStages - 1 ? 0 : stage + 1;
        typename G::Held fresh[kTokens];
        Share ahead{};
        uint32_t next = a.units;
        if (have) {
            const int c = now.c0 + cl;
            CutSeqs& seqs = s.seqs[parity][warp];
            now.cuts = find_cuts<L::V>(a, seqs, within, now.lo, now.count, c, a.first, a.last);
            now.simple = all_rows(now) && (now.cuts.begin | now.cuts.end) == 0;
            cp_async_wait_all();
            __syncwarp();
            if (many && threadIdx.x == 0) next = claim(a);
            const uint32_t* gw = reinterpret_cast<const uint32_t*>(mine + stage * kStage) + lane;
            const uint32_t* xw = gw + kTileBytes / 4;
            N A = L::fill(1.f), B = L::fill(0.f);
            if (now.simple) {
#pragma unroll
                for (int k = 0; k < kTokens; ++k) {
                    fresh[k] = G::hold(L::unpack(gw[k * kStep]));
                    const G g(fresh[k]);
                    B = next_state<FREE>(g, L::unpack(xw[k * kStep]), B);
                    A = g.kept(A);
                }
            } else {
#pragma unroll 1
                for (int k = 0; k < now.count; ++k) {
                    if (now.cuts.begin >> k & 1) B = state_of<L>(a, a.first, seqs.begin[k], c);
                    const G g(G::hold(L::unpack(gw[k * kStep])));
                    B = next_state<FREE>(g, L::unpack(xw[k * kStep]), B);
                    A = g.kept(A);
                }
                if (now.cuts.begin) A = L::fill(-1.f);
            }
            L::store(&s.a[parity][warp][cl], A);
            L::store(&s.b[parity][warp][cl], B);
            if (threadIdx.x == 0) {
                s.reached = many && !(now.cuts.begin & 1);
                s.unit = next;
            }
        }
        now.sealed = __syncthreads_or(have && now.cuts.begin != 0);
        if (have) {
            now.reached = s.reached;
            next = s.unit;
            if (next < a.units) {
                ahead = share_of<CH>(a, next, false);
                fetch_all(next_stage, ahead);
            }
            if (many && warp == 0) publish_nodes<CH, false>(a, s, parity, now.v, now.c0, now.sealed);
        }
        if (pending) {
            const int before = stage == 0 ? kFwdStages - 1 : stage - 1, c = last.c0 + cl;
            const CutSeqs& seqs = s.seqs[parity ^ 1][warp];
            if (last.reached) collect<CH, false>(a, s, last.v, last.c0);
            __syncthreads();
            N h = entering<L, CH, false>(a, s, parity ^ 1, last.reached);
            const bool real = c < a.c;
            if (real && a.carries && warp == 0 && last.count > 0) L::store(a.carries + (int64_t)last.v * a.c + c, h);
            const uint32_t* gw = reinterpret_cast<const uint32_t*>(mine + before * kStage) + lane;
            const uint32_t* xw = gw + kTileBytes / 4;
            char* const out = a.out + c * (int)sizeof(T);
            if (last.simple) {
#pragma unroll
                for (int k = 0; k < kTokens; ++k) {
                    const int32_t row = __shfl_sync(0xffffffffu, last.row, k);
                    h = next_state<FREE>(G(held[k]), L::unpack(xw[k * kStep]), h);
                    if (real) put<L>(out, row, a.out_s, h);
                }
            } else {
#pragma unroll 1
                for (int k = 0; k < last.count; ++k) {
                    const int32_t row = __shfl_sync(0xffffffffu, last.row, k);
                    if (last.cuts.begin >> k & 1) h = state_of<L>(a, a.first, seqs.begin[k], c);
                    const G g(G::hold(L::unpack(gw[k * kStep])));
                    h = next_state<FREE>(g, L::unpack(xw[k * kStep]), h);
                    if (real && row >= 0) put<L>(out, row, a.out_s, h);
                    if (a.last && real && (last.cuts.end >> k & 1))
                        L::store(a.last + (int64_t)seqs.end(last.cuts, k) * a.c + c, h);
                }
            }
        }
        __syncthreads();  // the last tile's maps and stage have been read
        pending = have;
        have = next < a.units;
        last = now;
        now = ahead;
#pragma unroll
        for (int k = 0; k < kTokens; ++k) held[k] = fresh[k];
        stage = next_stage;
    }
}

// The backward pass takes the tiles from the end, and joins the warps' maps from the last.  The
// states are found again from those that the forward pass kept at the tiles' beginnings.
template <typename T, bool FREE>
__global__ void __launch_bounds__(kThreads, kBlocksPerSm) k_scan_bwd(const ScanArgs a) {
    using L = Lane<T>;
    using N = typename L::Num;
    using G = Side<N>;
    constexpr int CH = 32 * L::V, kStep = kRowBytes / 4, kStage = 3 * kTileBytes;
    extern __shared__ __align__(128) char s_dyn[];  // [2][gate, x, dy][kTile][128 bytes], then the maps
    using J = Joint<CH, true>;
    J& s = *reinterpret_cast<J*>(s_dyn + 2 * kStage);
    if (!good_offsets(a)) return;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, cl = lane * L::V;
    const bool many = a.tree.tiles > 1;
    const uint32_t unit = first_unit(a, s);
    if (unit >= a.units) return;
    char* const mine = s_dyn + warp * kTokens * kRowBytes;
    const auto fetch_all = [&](int stage, const Share& of) {
        const uint32_t to = smem_u32(mine) + stage * kStage;
        fetch<T>(to, a.gate, a.gate_s, of, a.c);
        fetch<T>(to + kTileBytes, a.x, a.x_s, of, a.c);
        fetch<T>(to + 2 * kTileBytes, a.gy, a.gy_s, of, a.c);
    };
    Within within;
    Share now = share_of<CH>(a, unit, true), last{};
    N from_before = L::fill(0.f);  // the state that enters the last tile's tokens of this warp
    fetch_all(0, now);
    bool have = true, pending = false;

    for (int turn = 0; have || pending; ++turn) {
        const int parity = turn & 1;
        Share ahead{};
        uint32_t next = a.units;
        N h = L::fill(0.f);
        if (have) {
            const int c = now.c0 + cl;
            CutSeqs& seqs = s.seqs[parity][warp];
            if (c < a.c && now.count > 0) h = L::load(a.carries + (a.tree.tiles - 1 - now.v) * a.c + c);
            now.cuts = find_cuts<L::V>(a, seqs, within, now.lo, now.count, c, a.glast, a.gfirst);
            now.simple = all_rows(now) && (now.cuts.begin | now.cuts.end) == 0;
            cp_async_wait_all();
            __syncwarp();
            if (many && threadIdx.x == 0) next = claim(a);
            const uint32_t* gw = reinterpret_cast<const uint32_t*>(mine + parity * kStage) + lane;
            const uint32_t* xw = gw + kTileBytes / 4;
            const uint32_t* yw = xw + kTileBytes / 4;
            N A = L::fill(1.f), B = L::fill(0.f), D = L::fill(0.f);
            if (now.simple) {
                typename G::Held held[kTokens];
#pragma unroll
                for (int k = 0; k < kTokens; ++k) {
                    held[k] = G::hold(L::unpack(gw[k * kStep]));
                    const G g(held[k]);
                    B = next_state<FREE>(g, L::unpack(xw[k * kStep]), B);
                    A = g.kept(A);
                }
#pragma unroll
                for (int k = kTokens - 1; k >= 0; --k) D = G(held[k]).kept(add_(D, L::unpack(yw[k * kStep])));
            } else {
#pragma unroll 1
                for (int k = 0; k < now.count; ++k) {
                    if (now.cuts.begin >> k & 1) B = state_of<L>(a, a.first, seqs.begin[k], c);
                    const G g(G::hold(L::unpack(gw[k * kStep])));
                    B = next_state<FREE>(g, L::unpack(xw[k * kStep]), B);
                    A = g.kept(A);
                }
#pragma unroll 1
                for (int k = now.count - 1; k >= 0; --k) {
                    if (now.cuts.end >> k & 1) D = state_of<L>(a, a.glast, seqs.end(now.cuts, k), c);
                    D = G(G::hold(L::unpack(gw[k * kStep]))).kept(add_(D, L::unpack(yw[k * kStep])));
                }
            }
            L::store(&s.fa[warp][cl], now.cuts.begin ? L::fill(-1.f) : A);
            L::store(&s.fb[warp][cl], B);
            L::store(&s.a[parity][warp][cl], now.cuts.end ? L::fill(-1.f) : A);
            L::store(&s.b[parity][warp][cl], D);
            // the last visit of all is an end, so a tile that is not full is not reached
            if (threadIdx.x == kThreads - 1)
                s.reached = many && now.count == kTokens && !(now.cuts.end >> (kTokens - 1) & 1);
            if (threadIdx.x == 0) s.unit = next;
        }
        now.sealed = __syncthreads_or(have && now.cuts.end != 0);
        if (have) {
            now.reached = s.reached;
            next = s.unit;
            if (many && warp == 0) publish_nodes<CH, true>(a, s, parity, now.v, now.c0, now.sealed);
            for (int w = 0; w < warp; ++w) h = step_through(&s.fa[w][cl], &s.fb[w][cl], h);
        }
        if (pending) {
            const int c = last.c0 + cl;
            const CutSeqs& seqs = s.seqs[parity ^ 1][warp];
            if (last.reached) collect<CH, true>(a, s, last.v, last.c0);
            __syncthreads();
            N mu = entering<L, CH, true>(a, s, parity ^ 1, last.reached);
            const bool real = c < a.c;
            const uint32_t* gw = reinterpret_cast<const uint32_t*>(mine + (parity ^ 1) * kStage) + lane;
            const uint32_t* xw = gw + kTileBytes / 4;
            const uint32_t* yw = xw + kTileBytes / 4;
            char* const gg = a.gg + c * (int)sizeof(T);
            char* const gx = a.out + c * (int)sizeof(T);
            // a token's gradients, from the state before it and the gradient that comes from behind it
            const auto gradients = [&](const G& g, N x, N y, N before, N& dg, N& dx) {
                const N lam = add_(mu, y);
                dg = mul_(mul_(g.slope(), FREE ? before : add_(before, neg_(x))), lam);
                dx = FREE ? lam : mul_(g.rest(), lam);
                mu = g.kept(lam);
            };
            if (last.simple) {
                typename G::Held held[kTokens];
                N before[kTokens], state = from_before;
#pragma unroll
                for (int k = 0; k < kTokens; ++k) {
                    held[k] = G::hold(L::unpack(gw[k * kStep]));
                    before[k] = state;
                    state = next_state<FREE>(G(held[k]), L::unpack(xw[k * kStep]), state);
                }
#pragma unroll
                for (int k = kTokens - 1; k >= 0; --k) {
                    const int32_t row = __shfl_sync(0xffffffffu, last.row, k);
                    N dg, dx;
                    gradients(G(held[k]), L::unpack(xw[k * kStep]), L::unpack(yw[k * kStep]), before[k], dg, dx);
                    if (real) {
                        put<L>(gg, row, a.gg_s, dg);
                        put<L>(gx, row, a.out_s, dx);
                    }
                }
            } else {
                // the state before a token is found from the warp's first one, or the last beginning, each time
#pragma unroll 1
                for (int k = last.count - 1; k >= 0; --k) {
                    N before = from_before;
                    int from = 0;
                    const uint32_t until = last.cuts.begin & ((2u << k) - 1);
                    if (until) {
                        from = 31 - __clz(until);
                        before = state_of<L>(a, a.first, seqs.begin[from], c);
                    }
#pragma unroll 1
                    for (int i = from; i < k; ++i)
                        before = next_state<FREE>(G(G::hold(L::unpack(gw[i * kStep]))), L::unpack(xw[i * kStep]),
                                                  before);
                    if (last.cuts.end >> k & 1) mu = state_of<L>(a, a.glast, seqs.end(last.cuts, k), c);
                    N dg, dx;
                    gradients(G(G::hold(L::unpack(gw[k * kStep]))), L::unpack(xw[k * kStep]),
                              L::unpack(yw[k * kStep]), before, dg, dx);
                    const int32_t row = __shfl_sync(0xffffffffu, last.row, k);
                    if (real && row >= 0) {
                        put<L>(gg, row, a.gg_s, dg);
                        put<L>(gx, row, a.out_s, dx);
                    }
                    if (a.gfirst && real && (last.cuts.begin >> k & 1))
                        L::store(a.gfirst + (int64_t)seqs.begin[k] * a.c + c, mu);
                }
            }
        }
        __syncthreads();  // the last tile's maps and stage have been read
        if (next < a.units) {
            ahead = share_of<CH>(a, next, true);
            fetch_all(parity ^ 1, ahead);
        }
        pending = have;
        have = next < a.units;
        last = now;
        now = ahead;
        from_before = h;
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

// 16 bytes of a lane's channels.
template <typename T, bool FREE>
__global__ void __launch_bounds__(kThreads) k_scan_step(int64_t vectors, int per_row, int c, const char* gate,
                                                        int64_t gate_s, const char* x, int64_t x_s, float* state,
                                                        char* out, int64_t out_s) {
    using L = Lane<T>;
    using G = Side<typename L::Num>;
    for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < vectors; i += (int64_t)gridDim.x * kThreads) {
        const int64_t r = i / per_row;
        const int at = (int)(i - r * per_row);
        uint4 g = *reinterpret_cast<const uint4*>(gate + r * gate_s + at * 16);
        uint4 xv = *reinterpret_cast<const uint4*>(x + r * x_s + at * 16);
        float* sp = state + r * c + at * 4 * L::V;
        float4 h[L::V];
#pragma unroll
        for (int j = 0; j < L::V; ++j) h[j] = reinterpret_cast<const float4*>(sp)[j];
        typename L::Num* hn = reinterpret_cast<typename L::Num*>(h);
        uint32_t* gw = reinterpret_cast<uint32_t*>(&g);
        uint32_t* xw = reinterpret_cast<uint32_t*>(&xv);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const G g(G::hold(L::unpack(gw[j])));
            hn[j] = next_state<FREE>(g, L::unpack(xw[j]), hn[j]);
            gw[j] = L::pack(hn[j]);
        }
#pragma unroll
        for (int j = 0; j < L::V; ++j) reinterpret_cast<float4*>(sp)[j] = h[j];
        *reinterpret_cast<uint4*>(out + r * out_s + at * 16) = g;
    }
}

Tree tree_of(int64_t n, int c, int64_t* words) {
    Tree t{};
    t.tiles = std::max<int64_t>(1, (n + kTile - 1) / kTile);
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
int launch(const ScanArgs& a, bool bwd, int sms, cudaStream_t s) {
    constexpr int CH = 32 * Lane<T>::V;
    const size_t maps = bwd ? Joint<CH, true>::bytes(a.tree.levels) : Joint<CH, false>::bytes(a.tree.levels);
    const size_t smem = 6 * (size_t)kTileBytes + maps;
    static_assert(kFwdStages * 2 == 6, "as many operands' tiles as two backward stages");
    auto kernel = a.free_input ? (bwd ? k_scan_bwd<T, true> : k_scan_fwd<T, true>)
                               : (bwd ? k_scan_bwd<T, false> : k_scan_fwd<T, false>);
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess)
        return VG_ERR_CUDA;
    const int grid = a.tree.tiles == 1 ? (int)a.units : (int)std::min<int64_t>(a.units, (int64_t)sms * kBlocksPerSm);
    kernel<<<grid, kThreads, smem, s>>>(a);
    return cudaPeekAtLastError() == cudaSuccess ? VG_OK : VG_ERR_CUDA;
}

}  // namespace

size_t gated_scan_workspace_bytes(int64_t n, int c) {
    int64_t words;
    tree_of(n, c, &words);
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
    const auto in = [&](const vg_rows* r, const char** p, uint32_t* stride) {
        *p = r ? static_cast<const char*>(r->data) : nullptr;
        *stride = r && q.s->n > 1 ? (uint32_t)(r->row_stride * es) : 0;
    };
    const auto out = [&](const vg_rows* r, char** p, uint32_t* stride) {
        *p = r ? static_cast<char*>(r->data) : nullptr;
        *stride = r && q.s->n > 1 ? (uint32_t)(r->row_stride * es) : 0;
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
    a.tree = tree_of(a.n, a.c, &words);
    if (a.tree.tiles * a.blocks_c >= (int64_t(1) << 31)) return VG_ERR_UNSUPPORTED;
    a.units = (uint32_t)(a.tree.tiles * a.blocks_c);
    if (a.tree.tiles > 1) {
        const int64_t fill = std::max<int64_t>(1, std::min<int64_t>((words + 4095) / 4096, q.sms));
        k_scan_begin<<<(unsigned)fill, 1024, 0, s>>>(a, words);
        if (cudaPeekAtLastError() != cudaSuccess) return VG_ERR_CUDA;
    }
    return q.s->dtype == VG_F32   ? launch<float>(a, bwd, q.sms, s)
           : q.s->dtype == VG_F16 ? launch<__half>(a, bwd, q.sms, s)
                                  : launch<__nv_bfloat16>(a, bwd, q.sms, s);
}

int gated_scan_step(int64_t n, int c, int dtype, bool free_input, const vg_rows& gate, const vg_rows& x, float* state,
                    const vg_rows& out, cudaStream_t s) {
    const int v = dtype == VG_F32 ? 4 : 8;
    const int64_t vectors = n * (c / v);
    const int grid = (int)std::min<int64_t>((vectors + kThreads - 1) / kThreads, 152 * 8);
    const auto run = [&](auto kernel) {
        kernel<<<grid, kThreads, 0, s>>>(vectors, c / v, c, static_cast<const char*>(gate.data),
                                         gate.row_stride * 16 / v, static_cast<const char*>(x.data),
                                         x.row_stride * 16 / v, state, static_cast<char*>(out.data),
                                         out.row_stride * 16 / v);
        return cudaPeekAtLastError() == cudaSuccess ? VG_OK : VG_ERR_CUDA;
    };
    if (dtype == VG_F32) return free_input ? run(k_scan_step<float, true>) : run(k_scan_step<float, false>);
    if (dtype == VG_F16) return free_input ? run(k_scan_step<__half, true>) : run(k_scan_step<__half, false>);
    return free_input ? run(k_scan_step<__nv_bfloat16, true>) : run(k_scan_step<__nv_bfloat16, false>);
}

}  // namespace vg
