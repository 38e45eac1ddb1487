// Gated linear recurrence of each channel along each sequence, and its gradient.
//
//   a = sigmoid(gate),  h_t = a_t h_{t-1} + b_t,  b_t = (1 - a_t) x_t  (or x_t)
// backward: lam_t = dy_t + mu_{t+1}, mu_t = a_t lam_t;  db = lam, da = h_{t-1} lam (- x lam)
//
// A run of tokens maps the state that enters it to the one that leaves it, h -> A h + B, and two
// runs after one another make (A2 A1, A2 B1 + B2).  So a pass has three steps: every warp finds the
// map of its tokens (up to 256; a lane has 4 bytes of channels, two 16-bit ones), and the block those of
// its warps; the blocks' maps are joined, in a fixed order, into the state that enters each block; every
// warp goes through its tokens from the state that enters it.  A warp copies its next 16 tokens into shared memory
// while it works on these, and needs nothing of other warps, so loads stream.  The forward pass
// keeps the state before every 16th token, from which the backward pass finds the others again.
//
// Gate and x (backward: gate and dy) are read twice: 602,492 tokens of 512 channels in bf16 take 204 us for the
// maps (6.1 TB/s), 7 for the join and 299 for the pass (6.4 TB/s), backward 202, 7 and 514 (6.2 TB/s); the maps issue in
// 73 % of the cycles, the passes in 60.  Single passes, in which blocks publish their maps and wait for those of the blocks
// before, were built first and read everything once: with a tree of maps, tiles held in shared memory and each tile's map
// published before the last tile was finished, the forward pass took 950 us, and 600 with the waits left out, so that
// its body too was slower than these steps; 4.9 M tokens of 64 channels took 1790, so 520.  None has been built around the
// present body.  Smaller pieces that stay in the L2 between the steps gain nothing: with all of its data there the last
// step is as slow (8.4 M more elements cost 6.5 us).  Blocks that go from unit to unit without a pause, each warp's next
// tokens sent for across them, took 581 and 851 us.
//
// Where a sequence begins, the map is constant (A = -1 marks it, h -> B), so that nothing, not
// even a NaN, passes from one sequence to the next.  A warp's tokens are the same for all of its
// lanes, so such places cost a branch that no lane takes alone.
#include <type_traits>

#include "common.cuh"
#include "internal.h"
#include "tc_ptx.cuh"

namespace vg {

namespace {

using namespace ptx;

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kTokens = kScanCarryRows;      // looked up and loaded at once; a state is kept for each such run
constexpr int kHalf = kTokens / 2;           // unrolled: more straight code did not stay in the instruction cache
constexpr int kMaxRuns = 16;                 // runs of a warp (ScanArgs::runs), at most
constexpr int kRowBytes = 128, kRunBytes = kTokens * kRowBytes;  // of an operand in a block
constexpr int kStep = kRowBytes / 4, kOperand = kRunBytes / 4;  // words from a token, an operand to the next
// Blocks per SM, by their shared memory and registers.
constexpr int per_sm(bool bwd) { return bwd ? 2 : 3; }
// Shared memory of a block: two runs of `operands` a warp.
constexpr size_t stage_bytes(int operands) { return (size_t)kWarps * 2 * operands * kRunBytes; }
constexpr int kFoldTiles = 256;              // up to so many, blocks join the maps before them themselves
constexpr int kJoinChannels = 4, kJoinParts = 256;  // of a block of k_scan_join
static_assert(kTokens == 16, "a lane holds the row of one token, half of the lanes none");

// Workspace: word 0 the error record, word 1 this call's verdict on its offsets; from byte 256 on the
// tiles' maps [tiles][c], the warps' [tiles][warps][c] (of the warps before each in its tile), and
// the states that enter the tiles, fp32 [tiles][c].
struct Map {
    float a, b;  // h -> a h + b; a = -1: h -> b
};

struct ScanArgs {
    int64_t n;
    int c, batch, blocks_c;    // blocks_c: blocks of channels
    int tiles, runs;           // tiles of kWarps * runs * kTokens tokens
    const int32_t* off;
    const int32_t* order;
    int reverse;
    const char *gate, *x, *gy;
    char *out, *gg;            // out: grad_x in the backward pass
    uint32_t gate_s, x_s, gy_s, out_s, gg_s;  // strides in bytes
    const float* first;
    const float* glast;
    float *last, *carries, *gfirst;
    uint32_t* head;
    Map *tile_maps, *warp_maps;
    float* states;
};

// ---------------------------------------------------------------- a lane's channels
// Two channels (16-bit types) or one, in fp32; two are worked on by paired instructions.
__device__ __forceinline__ float2 fma_(float2 a, float2 b, float2 c) { return fma2(a, b, c); }
__device__ __forceinline__ float fma_(float a, float b, float c) { return fmaf(a, b, c); }
__device__ __forceinline__ float2 add_(float2 a, float2 b) { return add2(a, b); }
__device__ __forceinline__ float add_(float a, float b) { return a + b; }
__device__ __forceinline__ float2 mul_(float2 a, float2 b) { return mul2(a, b); }
__device__ __forceinline__ float mul_(float a, float b) { return a * b; }
__device__ __forceinline__ float2 sub_(float2 a, float2 b) { return fma2(b, make_float2(-1.f, -1.f), a); }
__device__ __forceinline__ float sub_(float a, float b) { return a - b; }

// What a token's gate does to a state.  No form lets a h lose what is small beside h, nor 1 - a what is small beside 1.
//
// Side, for fp32: m = e / (1 + e) with e = exp(-|g|), the smaller of a = sigmoid(g) and 1 - a, held as m
// (a = m, for g < 0) or as -m (a = 1 - m).  Each use has to look at the sign.
//
// 16-bit types, with s = 1 - a = 1 / (1 + e), e = exp(g), do with fewer instructions.  s is good to 2^-22 of its size, and
// h - s h has what an open gate leaves; of a nearly closed one's it misses what the rounding of s to 32 bits took, s d with
// the reciprocal's residual d = s (1 + e) - 1, which one fused operation finds from s - 1 (s - 1 is exact for
// s >= 1/2, and below its rounding is a share 2^-25 of s).
// Rest adds s d h where a run of tokens has a gate below -3 (CLOSED): four instructions a pair of gates and one a use.
// Above, h - s h alone is good to 3e-6 of a h.  (Without it all of a was lost at gates below -17, and 0.1 % of it at
// -10; with it for every run 100,000 tokens of 256 channels took 54 and 90 us, forward and backward, so 50 and 77.)
// The backward pass holds 16 gates, as one number each: Halves, 1 - a for an open gate and -a, a = e s, for the others.
//
// 16-bit types take the fast exponential and reciprocal, off by 2 units and |g| / 2^23, and by 1 (and exact at 1):
// 1e-6 of a and s for |g| < 10, where the inputs have 2^-9 or 2^-12.  Gates are bounded at 88, where s is
// already 0, so that the exponential stays finite.
struct Side {
    float m, one;  // one: 1 where a is 1 - m, 0 where it is m
    static __device__ __forceinline__ uint32_t sign(float x) { return (int32_t)__float_as_uint(x) >> 31; }  // 0 or all ones
    static __device__ __forceinline__ float hold(uint32_t word) {
        const float g = __uint_as_float(word), e = expf(-fabsf(g)), m = e / (1.f + e);
        return __uint_as_float((__float_as_uint(m) & 0x7fffffffu) | (~__float_as_uint(g) & 0x80000000u));
    }
    // also a (1 - a) and 1 - a
    static __device__ __forceinline__ float hold(uint32_t word, float& slope, float& rest) {
        const float m = hold(word);
        slope = fmaf(-fabsf(m), fabsf(m), fabsf(m));
        rest = Side(m).rest();
        return m;
    }
    __device__ __forceinline__ explicit Side(uint32_t word) : Side(hold(word)) {}
    __device__ __forceinline__ explicit Side(float held) : m(held) { one = __uint_as_float(sign(held) & 0x3f800000u); }
    __device__ __forceinline__ float kept(float h) const { return fmaf(m, h, one * h); }  // a h
    __device__ __forceinline__ float rest() const { return (1.f - one) - m; }             // 1 - a
    __device__ __forceinline__ float rest_of(float h) const { return rest() * h; }
};

__device__ __forceinline__ float2 negated(float2 x) { return mul2(x, make_float2(-1.f, -1.f)); }
// Two gates' exp(g), and s.
template <typename T> struct Exp {
    float2 e, s;
    // Bounded at 88 (NaN stays).
    static __device__ __forceinline__ uint32_t bounded(uint32_t word) {
        if constexpr (std::is_same_v<T, __half>)
            asm("min.NaN.f16x2 %0, %0, %1;" : "+r"(word) : "r"(0x55805580u));
        else
            asm("min.NaN.bf16x2 %0, %0, %1;" : "+r"(word) : "r"(0x42b042b0u));
        return word;
    }
    // The smaller ones of two words' numbers, passing over NaN.
    static __device__ __forceinline__ uint32_t smaller(uint32_t a, uint32_t b) {
        if constexpr (std::is_same_v<T, __half>)
            asm("min.f16x2 %0, %0, %1;" : "+r"(a) : "r"(b));
        else
            asm("min.bf16x2 %0, %0, %1;" : "+r"(a) : "r"(b));
        return a;
    }
    __device__ __forceinline__ explicit Exp(uint32_t word) {
        const float2 y = mul2(Pair<T>::unpack(word), make_float2(1.4426950408889634f, 1.4426950408889634f));
        asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.x) : "f"(y.x));
        asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.y) : "f"(y.y));
        const float2 d = add2(e, make_float2(1.f, 1.f));
        asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(s.x) : "f"(d.x));
        asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(s.y) : "f"(d.y));
    }
};
template <typename T, bool CLOSED> struct Rest {
    float2 s, minus, missed;
    __device__ __forceinline__ explicit Rest(uint32_t word) {
        const Exp<T> x(CLOSED ? Exp<T>::bounded(word) : word);
        s = x.s;
        minus = negated(s);
        if constexpr (CLOSED) missed = mul2(fma2(x.e, s, add2(s, make_float2(-1.f, -1.f))), s);
    }
    __device__ __forceinline__ float2 kept(float2 h) const {
        const float2 left = fma2(minus, h, h);
        if constexpr (CLOSED) return fma2(missed, h, left);
        return left;
    }
    __device__ __forceinline__ float2 rest() const { return s; }
};
template <bool CLOSED> struct Halves {
    float2 v;
    uint32_t closed_x, closed_y;  // all ones where v is -a
    template <typename T>
    static __device__ __forceinline__ float2 hold(uint32_t word, float2& slope, float2& rest) {
        const Exp<T> x(Exp<T>::bounded(word));
        const float2 a = mul2(x.e, x.s);
        slope = mul2(a, x.s);
        rest = x.s;
        if constexpr (!CLOSED) return x.s;
        return make_float2(x.e.x < 1.f ? -a.x : x.s.x, x.e.y < 1.f ? -a.y : x.s.y);
    }
    __device__ __forceinline__ explicit Halves(float2 held) : v(held) {
        closed_x = CLOSED ? Side::sign(held.x) : 0u;
        closed_y = CLOSED ? Side::sign(held.y) : 0u;
    }
    static __device__ __forceinline__ float2 masked(float2 h, uint32_t x, uint32_t y) {
        return make_float2(__uint_as_float(__float_as_uint(h.x) & x), __uint_as_float(__float_as_uint(h.y) & y));
    }
    __device__ __forceinline__ float2 kept(float2 h) const {
        return fma2(negated(v), h, CLOSED ? masked(h, ~closed_x, ~closed_y) : h);
    }
    __device__ __forceinline__ float2 rest_of(float2 h) const {
        if constexpr (!CLOSED) return mul2(v, h);
        return fma2(v, h, masked(h, closed_x, closed_y));
    }
};

// A lane's word of T, its gates (CLOSED: nearly closed ones may be among them; Kept: as the backward pass holds them),
// and its states.
template <typename T> struct Lane : Pair<T> {
    using Num = float2;
    template <bool CLOSED> using Gate = Rest<T, CLOSED>;
    template <bool CLOSED> using Kept = Halves<CLOSED>;
    static constexpr int V = 2;
    template <bool CLOSED> static __device__ __forceinline__ float2 hold(uint32_t gate, float2& slope, float2& rest) {
        return Halves<CLOSED>::template hold<T>(gate, slope, rest);
    }
    // Whether a gate of a run's tokens, for any lane, is below -3.
    static __device__ __forceinline__ bool any_closed(const uint32_t* w) {
        uint32_t least[kTokens];
#pragma unroll
        for (int k = 0; k < kTokens; ++k) least[k] = w[k * kStep];
#pragma unroll
        for (int d = kTokens / 2; d > 0; d /= 2)
#pragma unroll
            for (int k = 0; k < d; ++k) least[k] = Exp<T>::smaller(least[k], least[k + d]);
        const float2 g = Pair<T>::unpack(least[0]);
        return __any_sync(0xffffffffu, fminf(g.x, g.y) < -3.f);
    }
    // Numbers in place of a token's gate and input.
    static __device__ __forceinline__ void stash(uint32_t* w, float2 x) {
        w[0] = __float_as_uint(x.x);
        w[kOperand] = __float_as_uint(x.y);
    }
    static __device__ __forceinline__ float2 stashed(const uint32_t* w) {
        return make_float2(__uint_as_float(w[0]), __uint_as_float(w[kOperand]));
    }
    static __device__ __forceinline__ float2 fill(float x) { return make_float2(x, x); }
    static __device__ __forceinline__ float2 load(const float* p) { return *reinterpret_cast<const float2*>(p); }
    static __device__ __forceinline__ void store(float* p, float2 x) { *reinterpret_cast<float2*>(p) = x; }
};
template <> struct Lane<float> {
    using Num = float;
    template <bool CLOSED> using Gate = Side;
    template <bool CLOSED> using Kept = Side;
    static constexpr int V = 1;
    template <bool CLOSED> static __device__ __forceinline__ float hold(uint32_t gate, float& slope, float& rest) {
        return Side::hold(gate, slope, rest);
    }
    static __device__ __forceinline__ bool any_closed(const uint32_t*) { return true; }
    static __device__ __forceinline__ void stash(uint32_t* w, float x) { w[0] = __float_as_uint(x); }
    static __device__ __forceinline__ float stashed(const uint32_t* w) { return __uint_as_float(w[0]); }
    static __device__ __forceinline__ float unpack(uint32_t w) { return __uint_as_float(w); }
    static __device__ __forceinline__ uint32_t pack(float x) { return __float_as_uint(x); }
    static __device__ __forceinline__ float fill(float x) { return x; }
    static __device__ __forceinline__ float load(const float* p) { return *p; }
    static __device__ __forceinline__ void store(float* p, float x) { *p = x; }
};
// go(simple, closed, ..) for a run, by what its tokens are.
template <typename L, typename R, typename Go>
__device__ __forceinline__ void by_kind(const R& r, const uint32_t* w, const Go& go) {
    if (!r.simple)
        go(std::false_type{}, std::true_type{});
    else if (L::any_closed(w))
        go(std::true_type{}, std::true_type{});
    else
        go(std::true_type{}, std::false_type{});
}

// The state after a token.
template <bool FREE, typename G, typename N> __device__ __forceinline__ N next_state(const G& g, N rest, N x, N h) {
    if constexpr (FREE) return add_(g.kept(h), x);
    return fma_(rest, x, g.kept(h));
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
    const bool last = hi == a.n && (count > 0 || (a.n == 0 && threadIdx.x < 32));  // the visits' end lies here
    if (count == 0 && !last) return r;
    // the number of sequences that begin before lo, 32 probes at a time (up to 32 of them: none, for
    // all are looked at below)
    int from = 0, to = a.batch > 32 ? a.batch : 0;
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
    // those that begin here, and the one before them, which goes on into the visits and may end here
    for (int b0 = max(from - 1, 0);; b0 += 32) {
        const int b = b0 + lane;
        const bool real = b < a.batch;
        const int64_t p = real ? begins(a, b) : a.n, q = real ? begins(a, b + 1) : a.n;
        const bool here = real && (p < hi || (last && p == a.n));  // or before
        const int seq = sequence(a, b);
        const bool begin = real && q > p && p >= lo && p < hi, end = real && q > p && q > lo && q <= hi;
        if (begin) s.begin[p - lo] = seq;
        const uint32_t over = __ballot_sync(0xffffffffu, real && p < lo && q > lo);
        if (over) {  // one at most
            const int l = __ffs(over) - 1;
            w.from = __shfl_sync(0xffffffffu, p, l);
            w.to = __shfl_sync(0xffffffffu, q, l);
            if (lane == l) s.entering = seq;
        }
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

// ---------------------------------------------------------------- maps of runs of tokens
__device__ __forceinline__ bool constant(Map m) { return m.a < -0.5f; }
__device__ __forceinline__ float through(Map m, float h) { return constant(m) ? m.b : fmaf(m.a, h, m.b); }
__device__ __forceinline__ Map then(Map first, Map second) {
    if (constant(second)) return second;
    return Map{constant(first) ? -1.f : first.a * second.a, fmaf(second.a, first.b, second.b)};
}
// Of a lane's channels.
template <int V> struct Maps {
    Map m[V];
};
template <int V> __device__ __forceinline__ Maps<V> load_maps(const Map* p) {
    Maps<V> r;
    if constexpr (V == 2) {
        const float4 f = *reinterpret_cast<const float4*>(p);
        r.m[0] = Map{f.x, f.y};
        r.m[1] = Map{f.z, f.w};
    } else {
        const float2 f = *reinterpret_cast<const float2*>(p);
        r.m[0] = Map{f.x, f.y};
    }
    return r;
}
template <int V> __device__ __forceinline__ void store_maps(Map* p, const Maps<V>& r) {
    if constexpr (V == 2)
        *reinterpret_cast<float4*>(p) = make_float4(r.m[0].a, r.m[0].b, r.m[1].a, r.m[1].b);
    else
        *reinterpret_cast<float2*>(p) = make_float2(r.m[0].a, r.m[0].b);
}
template <int V> __device__ __forceinline__ Maps<V> then(const Maps<V>& first, const Maps<V>& second) {
    Maps<V> r;
#pragma unroll
    for (int j = 0; j < V; ++j) r.m[j] = then(first.m[j], second.m[j]);
    return r;
}
template <int V> __device__ __forceinline__ Maps<V> no_change() {
    Maps<V> r;
#pragma unroll
    for (int j = 0; j < V; ++j) r.m[j] = Map{1.f, 0.f};
    return r;
}
__device__ __forceinline__ float through(const Maps<1>& m, float h) { return through(m.m[0], h); }
__device__ __forceinline__ float2 through(const Maps<2>& m, float2 h) {
    return make_float2(through(m.m[0], h.x), through(m.m[1], h.y));
}
__device__ __forceinline__ Maps<1> maps_of(float a, float b, bool constant) {
    return Maps<1>{{Map{constant ? -1.f : a, b}}};
}
__device__ __forceinline__ Maps<2> maps_of(float2 a, float2 b, bool constant) {
    return Maps<2>{{Map{constant ? -1.f : a.x, b.x}, Map{constant ? -1.f : a.y, b.y}}};
}

// ---------------------------------------------------------------- the tokens of a warp
// What a lane of a warp knows of its place.
struct Place {
    int c;       // its first channel
    bool real;   // there is such a channel
    int32_t lo;  // the warp's first visit
};
template <typename L>
__device__ __forceinline__ Place place_of(const ScanArgs& a, int tile, int block_c) {
    Place p;
    p.c = (block_c * 32 + (int)(threadIdx.x & 31)) * L::V;
    p.real = p.c < a.c;
    p.lo = (int32_t)min(((int64_t)tile * kWarps + (threadIdx.x >> 5)) * a.runs * kTokens, a.n);
    return p;
}
// The row of the token of this lane's number in run q, as the order names it (unchecked, so that
// the load need not be waited for here).
__device__ __forceinline__ int32_t row_of(const ScanArgs& a, const Place& p, int q) {
    const int lane = threadIdx.x & 31;
    const int64_t v = (int64_t)p.lo + q * kTokens + lane;
    if (lane >= kTokens || q < 0 || q >= a.runs || v >= a.n) return -1;
    const int64_t at = a.reverse ? a.n - 1 - v : v;
    return a.order ? a.order[at] : (int32_t)at;
}
// A run of the warp's tokens.
struct Run {
    int32_t lo, count;
    int32_t row;   // of the token of this lane's number, -1 where there is none
    Cuts cuts;
    bool simple;   // all tokens there, nothing begins or ends among them
};

// Copy a run's channels of P operands, [kTokens][128 bytes] each, into a stage; zeros where there is
// no row or channel.  16 bytes a lane, 8 lanes a token.
template <typename T, int P>
__device__ __forceinline__ void fetch(const ScanArgs& a, const char* const (&from)[P], const uint32_t (&stride)[P],
                                      uint32_t to, int32_t row, int first_channel) {
    const int lane = threadIdx.x & 31;
    const int at = first_channel * (int)sizeof(T) + (lane & 7) * 16;
    const bool inside = at < a.c * (int)sizeof(T);
    const char* const nowhere = reinterpret_cast<const char*>(a.head);  // not read
    to += lane * 16;
#pragma unroll
    for (int i = 0; i < kTokens / 4; ++i) {
        const int32_t r = __shfl_sync(0xffffffffu, row, i * 4 + (lane >> 3));
        const bool have = inside && r >= 0;
        const uint64_t rr = (uint32_t)r;
#pragma unroll
        for (int p = 0; p < P; ++p)
            cp_async16(to + p * kRunBytes + i * 512, have ? from[p] + at + rr * stride[p] : nowhere, have ? 16 : 0);
    }
}

// A warp's way through its runs, DOWN from the last, the next run's tokens always on their way.
template <typename T, int P, bool DOWN>
struct Walk {
    static constexpr int V = Lane<T>::V;
    const ScanArgs& a;
    const Place& p;
    const char* from[P];   // operands
    uint32_t stride[P];
    char* stages;
    int32_t row, next;     // this lane's token of the current run, and of the one that follows

    __device__ __forceinline__ int run(int i) const { return DOWN ? a.runs - 1 - i : i; }
    __device__ __forceinline__ int32_t check(int32_t r, int i) const {
        const int lane = threadIdx.x & 31;
        const int64_t v = (int64_t)p.lo + run(i) * kTokens + lane;
        if (i < a.runs && lane < kTokens && v < a.n && (r < 0 || r >= a.n)) {
            atomicOr(a.head, kErrRange);
            return -1;
        }
        return r;
    }
    __device__ __forceinline__ void fetch_run(int i, int32_t r) {
        fetch<T, P>(a, from, stride, smem_u32(stages) + (i & 1) * P * kRunBytes, r, p.c - (int)(threadIdx.x & 31) * V);
    }
    // Send for the first run.
    __device__ __forceinline__ void start() {
        const int32_t first = row_of(a, p, run(0));
        next = row_of(a, p, run(1));
        row = check(first, 0);
        fetch_run(0, row);
        cp_async_commit();
    }
    // use(run, words) for each run, with its tokens of the first operand at words[k * kStep], the next
    // operand's kOperand further.
    template <typename Use>
    __device__ __forceinline__ void go(CutSeqs& seqs, const float* in, float* out, const Use& use) {
        const int lane = threadIdx.x & 31;
        Within within;
#pragma unroll 1
        for (int i = 0; i < a.runs; ++i) {
            const int32_t later = i + 2 < a.runs ? row_of(a, p, run(i + 2)) : -1;
            next = check(next, i + 1);
            if (i + 1 < a.runs) fetch_run(i + 1, next);
            cp_async_commit();
            Run r;
            r.lo = (int32_t)min((int64_t)p.lo + run(i) * kTokens, a.n);
            r.count = min(kTokens, (int32_t)a.n - r.lo);
            r.row = row;
            r.cuts = find_cuts<V>(a, seqs, within, r.lo, r.count, p.c, in, out);
            r.simple = r.count == kTokens && (r.cuts.begin | r.cuts.end) == 0 &&
                       __all_sync(0xffffffffu, row >= 0 || lane >= kTokens);
            cp_async_wait<1>();
            __syncwarp();
            use(r, reinterpret_cast<uint32_t*>(stages + (i & 1) * P * kRunBytes) + lane);
            __syncwarp();
            row = next;
            next = later;
        }
    }
};

template <typename L>
__device__ __forceinline__ void put(char* base, int32_t row, uint32_t stride, typename L::Num x) {
    *reinterpret_cast<uint32_t*>(base + (uint64_t)(uint32_t)row * stride) = L::pack(x);
}
__device__ __forceinline__ int32_t row_at(const Run& r, int k) { return __shfl_sync(0xffffffffu, r.row, k); }
// The states of sequence `seq`, zero where there are none.
template <typename L>
__device__ __forceinline__ typename L::Num state_of(const ScanArgs& a, const float* states, int seq, const Place& p) {
    return states && p.real ? L::load(states + (int64_t)seq * a.c + p.c) : L::fill(0.f);
}

// The map of a warp's tokens: of the state along the visits, or (BWD) of the gradient against them.
template <typename T, bool FREE, bool BWD>
__device__ __forceinline__ Maps<Lane<T>::V> warp_map(const ScanArgs& a, const Place& p, char* s_stages,
                                                     CutSeqs& seqs) {
    using L = Lane<T>;
    using N = typename L::Num;
    N A = L::fill(1.f), B = L::fill(0.f);
    bool constant = false;
    const auto go = [&](auto simple, auto closed, const Run& r, const uint32_t* w) {
        const uint32_t resets = BWD ? r.cuts.end : r.cuts.begin;
#pragma unroll 1
        for (int b = 0; b < kTokens; b += kHalf) {
#pragma unroll
            for (int j = 0; j < kHalf; ++j) {
                const int k = BWD ? kTokens - 1 - b - j : b + j;
                if (simple || k < r.count) {
                    const typename L::template Gate<closed> g(w[k * kStep]);
                    const N v = L::unpack(w[kOperand + k * kStep]);
                    if (!simple && (resets >> k & 1))
                        B = BWD ? state_of<L>(a, a.glast, seqs.end(r.cuts, k), p)
                                : state_of<L>(a, a.first, seqs.begin[k], p);
                    B = BWD ? g.kept(add_(B, v)) : next_state<FREE>(g, g.rest(), v, B);
                    A = g.kept(A);
                }
            }
        }
        constant |= resets != 0;
    };
    Walk<T, 2, BWD> walk{a, p, {a.gate, BWD ? a.gy : a.x}, {a.gate_s, BWD ? a.gy_s : a.x_s}, s_stages};
    walk.start();
    walk.go(seqs, nullptr, nullptr, [&](const Run& r, const uint32_t* w) {
        by_kind<L>(r, w, [&](auto simple, auto closed) { go(simple, closed, r, w); });
    });
    return maps_of(A, B, constant);
}

// Each warp's map in shared memory becomes, for each warp, that of the warps before it (BWD: behind
// it); `all`: the block's.
template <int V>
__device__ __forceinline__ Maps<V> before_warp(const Map (*s_maps)[32 * V], bool bwd, Maps<V>& all) {
    const int warp = threadIdx.x >> 5, cl = (threadIdx.x & 31) * V;
    Maps<V> m = no_change<V>(), mine = m;
#pragma unroll
    for (int i = 0; i < kWarps; ++i) {
        const int w = bwd ? kWarps - 1 - i : i;
        if (w == warp) mine = m;
        m = then(m, load_maps<V>(&s_maps[w][cl]));
    }
    all = m;
    return mine;
}

// False if the call's offsets are no partition of the positions.
__device__ __forceinline__ bool good_offsets(const ScanArgs& a) {
    bool bad = false;
    for (int64_t i = threadIdx.x; i < a.batch; i += kThreads) {
        const int32_t p = a.off[i], q = a.off[i + 1];
        bad |= p > q || (i == 0 && p != 0) || (i == a.batch - 1 && q != a.n);
    }
    return !__syncthreads_or(bad);
}

// Step 1.  (Offsets that are no partition lead it to wrong maps, but to no wrong address; the first
// block leaves its verdict for step 3.)
template <typename T, bool FREE, bool BWD>
__global__ void __launch_bounds__(kThreads, per_sm(false)) k_scan_map(const ScanArgs a) {
    using L = Lane<T>;
    constexpr int V = L::V;
    __shared__ Map s_maps[kWarps][32 * V];
    __shared__ CutSeqs s_seqs[kWarps];
    extern __shared__ __align__(128) char s_dyn[];  // [warps][2 stages][operands][tokens][128 bytes]
    dependents_may_start();
    const int warp = threadIdx.x >> 5, cl = (threadIdx.x & 31) * V;
    const int tile = blockIdx.x / a.blocks_c, block_c = blockIdx.x - tile * a.blocks_c;
    const Place p = place_of<L>(a, tile, block_c);
    store_maps<V>(&s_maps[warp][cl], warp_map<T, FREE, BWD>(a, p, s_dyn + warp * 4 * kRunBytes, s_seqs[warp]));
    __syncthreads();
    Maps<V> all;
    const Maps<V> mine = before_warp<V>(s_maps, BWD, all);
    if (p.real) {
        store_maps<V>(a.warp_maps + ((int64_t)tile * kWarps + warp) * a.c + p.c, mine);
        if (warp == 0) store_maps<V>(a.tile_maps + (int64_t)tile * a.c + p.c, all);
    }
    if (blockIdx.x == 0) {
        const bool good = good_offsets(a);
        if (threadIdx.x == 0) {
            a.head[1] = good ? 0u : 1u;
            if (!good) atomicOr(a.head, kErrRange);
        }
    }
}

// Step 2, for many tiles: the states that enter them.  kJoinParts threads a channel take a range of
// tiles each, join the ranges' maps by doubling the distance, and go through their ranges again.
template <bool BWD>
__global__ void __launch_bounds__(kJoinChannels* kJoinParts) k_scan_join(const ScanArgs a) {
    __shared__ Map s[2][kJoinParts][kJoinChannels];
    const int cl = threadIdx.x % kJoinChannels, part = threadIdx.x / kJoinChannels;
    const int c = blockIdx.x * kJoinChannels + cl;
    const int span = (a.tiles + kJoinParts - 1) / kJoinParts;
    const int t0 = min(part * span, a.tiles), t1 = min(t0 + span, a.tiles);
    const auto tile = [&](int i) { return (int64_t)(BWD ? a.tiles - 1 - i : i) * a.c + c; };
    dependents_may_start();
    wait_for_previous();
    // `use(i, map)` for the range's tiles, some loads ahead
    const auto each = [&](const auto& use) {
        constexpr int kAhead = 8;
        for (int i0 = t0; i0 < t1; i0 += kAhead) {
            Map next[kAhead];
#pragma unroll
            for (int j = 0; j < kAhead; ++j) next[j] = a.tile_maps[tile(min(i0 + j, t1 - 1))];
#pragma unroll
            for (int j = 0; j < kAhead; ++j)
                if (i0 + j < t1) use(i0 + j, next[j]);
        }
    };
    Map m{1.f, 0.f};
    each([&](int, Map next) { m = then(m, next); });
    int now = 0;
    s[0][part][cl] = m;
    __syncthreads();
    for (int d = 1; d < kJoinParts; d *= 2) {
        if (part >= d) m = then(s[now][part - d][cl], m);
        now ^= 1;
        s[now][part][cl] = m;
        __syncthreads();
    }
    float h = part > 0 ? s[now][part - 1][cl].b : 0.f;  // all maps from the first visit on are constant
    each([&](int i, Map next) {
        a.states[tile(i)] = h;
        h = through(next, h);
    });
}

// What enters this warp's tokens.  One tile: from the maps that the block has found itself.  A few:
// from the maps of all tiles before, a share of them to each warp.  Many: from k_scan_join.
template <typename T, bool FREE, bool BWD>
__device__ __forceinline__ typename Lane<T>::Num entering(const ScanArgs& a, const Place& p, int tile,
                                                          Map (*s_maps)[32 * Lane<T>::V], char* s_stages,
                                                          CutSeqs& seqs) {
    using L = Lane<T>;
    constexpr int V = L::V;
    const int warp = threadIdx.x >> 5, cl = (threadIdx.x & 31) * V;
    Maps<V> all;
    if (a.tiles == 1) {
        store_maps<V>(&s_maps[warp][cl], warp_map<T, FREE, BWD>(a, p, s_stages, seqs));
        __syncthreads();
        return through(before_warp<V>(s_maps, BWD, all), L::fill(0.f));
    }
    const Maps<V> mine = p.real ? load_maps<V>(a.warp_maps + ((int64_t)tile * kWarps + warp) * a.c + p.c) : no_change<V>();
    if (a.tiles > kFoldTiles)
        return through(mine, p.real ? L::load(a.states + (int64_t)tile * a.c + p.c) : L::fill(0.f));
    const int before = BWD ? a.tiles - 1 - tile : tile, span = (before + kWarps - 1) / kWarps;
    Maps<V> m = no_change<V>();
    if (p.real) {
        constexpr int kAhead = 8;  // loads in flight
        const int i1 = min((warp + 1) * span, before);
        for (int i0 = warp * span; i0 < i1; i0 += kAhead) {
            Maps<V> next[kAhead];
#pragma unroll
            for (int j = 0; j < kAhead; ++j) {
                const int i = min(i0 + j, i1 - 1);
                next[j] = load_maps<V>(a.tile_maps + (int64_t)(BWD ? a.tiles - 1 - i : i) * a.c + p.c);
            }
#pragma unroll
            for (int j = 0; j < kAhead; ++j)
                if (i0 + j < i1) m = then(m, next[j]);
        }
    }
    store_maps<V>(&s_maps[warp][cl], m);
    __syncthreads();
    before_warp<V>(s_maps, false, all);
    return through(mine, through(all, L::fill(0.f)));
}

// Blocks of step 3 send for their first tokens while the steps before still run.  False if the call's
// offsets are bad.
template <typename W>
__device__ __forceinline__ bool begin_step(const ScanArgs& a, W& walk) {
    if (a.tiles > 1) {
        walk.start();
        wait_for_previous();
        if (a.head[1] == 0) return true;
        cp_async_wait_all();
        return false;
    }
    const bool good = good_offsets(a);
    if (!good && threadIdx.x == 0) atomicOr(a.head, kErrRange);
    return good;
}

// Step 3.
template <typename T, bool FREE>
__global__ void __launch_bounds__(kThreads, per_sm(false)) k_scan_fwd(const ScanArgs a) {
    using L = Lane<T>;
    using N = typename L::Num;
    __shared__ Map s_maps[kWarps][32 * L::V];
    __shared__ CutSeqs s_seqs[kWarps];
    extern __shared__ __align__(128) char s_dyn[];
    const int tile = blockIdx.x / a.blocks_c, block_c = blockIdx.x - tile * a.blocks_c;
    const Place p = place_of<L>(a, tile, block_c);
    CutSeqs& seqs = s_seqs[threadIdx.x >> 5];
    char* const s_stages = s_dyn + (threadIdx.x >> 5) * 4 * kRunBytes;
    Walk<T, 2, false> walk{a, p, {a.gate, a.x}, {a.gate_s, a.x_s}, s_stages};
    if (!begin_step(a, walk)) return;
    N h = entering<T, FREE, false>(a, p, tile, s_maps, s_stages, seqs);
    if (a.tiles == 1) walk.start();
    char* const out = a.out + p.c * (int)sizeof(T);
    const auto go = [&](auto simple, auto closed, const Run& r, const uint32_t* w) {
#pragma unroll
        for (int k = 0; k < kTokens; ++k) {
            const int32_t row = row_at(r, k);
            if (simple || k < r.count) {
                if (!simple && (r.cuts.begin >> k & 1)) h = state_of<L>(a, a.first, seqs.begin[k], p);
                const typename L::template Gate<closed> g(w[k * kStep]);
                h = next_state<FREE>(g, g.rest(), L::unpack(w[kOperand + k * kStep]), h);
                if (p.real && (simple || row >= 0)) put<L>(out, row, a.out_s, h);
                if (!simple && a.last && p.real && (r.cuts.end >> k & 1))
                    L::store(a.last + (int64_t)seqs.end(r.cuts, k) * a.c + p.c, h);
            }
        }
    };
    walk.go(seqs, a.first, a.last, [&](const Run& r, const uint32_t* w) {
        if (a.carries && p.real && r.count > 0) L::store(a.carries + (int64_t)(r.lo / kTokens) * a.c + p.c, h);
        by_kind<L>(r, w, [&](auto simple, auto closed) { go(simple, closed, r, w); });
    });
}

// The gradients, from the last run to the first; the states of a run's tokens are found again from the
// one that the forward pass kept at its beginning.
template <typename T, bool FREE>
__global__ void __launch_bounds__(kThreads, per_sm(true)) k_scan_bwd(const ScanArgs a) {
    using L = Lane<T>;
    using N = typename L::Num;
    __shared__ Map s_maps[kWarps][32 * L::V];
    __shared__ CutSeqs s_seqs[kWarps];
    extern __shared__ __align__(128) char s_dyn[];
    const int tile = blockIdx.x / a.blocks_c, block_c = blockIdx.x - tile * a.blocks_c;
    const Place p = place_of<L>(a, tile, block_c);
    CutSeqs& seqs = s_seqs[threadIdx.x >> 5];
    char* const s_stages = s_dyn + (threadIdx.x >> 5) * 6 * kRunBytes;
    Walk<T, 3, true> walk{a, p, {a.gate, a.x, a.gy}, {a.gate_s, a.x_s, a.gy_s}, s_stages};
    if (!begin_step(a, walk)) return;
    N mu = entering<T, FREE, true>(a, p, tile, s_maps, s_stages, seqs);
    if (a.tiles == 1) walk.start();
    char* const gg = a.gg + p.c * (int)sizeof(T);
    char* const gx = a.out + p.c * (int)sizeof(T);
    const auto go = [&](auto simple, auto closed, const Run& r, uint32_t* w, N from) {
        using G = typename L::template Kept<closed>;
        // Up the run, the gates held and a (1 - a) (h_{t-1} - x) put where this lane has read a token's gate and
        // input; then down.  (What is held of 16 tokens leaves no registers for these as well, and beside 200 KB of
        // shared memory the L1 has no room for what would be spilled.)  `held` is the half in hand, `other` the other one.
        N held[kHalf], other[kHalf];
#pragma unroll
        for (int k = 0; k < kHalf; ++k) held[k] = L::fill(0.f);
#pragma unroll 1
        for (int b = 0; b < kTokens; b += kHalf) {
            uint32_t* const half = w + b * kStep;
#pragma unroll
            for (int k = 0; k < kHalf; ++k) other[k] = held[k];
#pragma unroll
            for (int k = 0; k < kHalf; ++k) {
                if (simple || b + k < r.count) {
                    if (!simple && (r.cuts.begin >> (b + k) & 1)) from = state_of<L>(a, a.first, seqs.begin[b + k], p);
                    uint32_t* const u = half + k * kStep;
                    const N x = L::unpack(u[kOperand]);
                    N slope, rest;
                    held[k] = L::template hold<closed>(u[0], slope, rest);
                    L::stash(u, mul_(slope, FREE ? from : sub_(from, x)));
                    from = next_state<FREE>(G(held[k]), rest, x, from);
                }
            }
        }
#pragma unroll 1
        for (int b = kTokens - kHalf; b >= 0; b -= kHalf) {
            const uint32_t* const half = w + b * kStep;
#pragma unroll
            for (int k = kHalf - 1; k >= 0; --k) {
                const int32_t row = row_at(r, b + k);
                if (simple || b + k < r.count) {
                    if (!simple && (r.cuts.end >> (b + k) & 1))
                        mu = state_of<L>(a, a.glast, seqs.end(r.cuts, b + k), p);
                    const uint32_t* const u = half + k * kStep;
                    const G g(held[k]);
                    const N lam = add_(mu, L::unpack(u[2 * kOperand]));
                    const N dg = mul_(L::stashed(u), lam), dx = FREE ? lam : g.rest_of(lam);
                    mu = g.kept(lam);
                    if (p.real && (simple || row >= 0)) {
                        put<L>(gg, row, a.gg_s, dg);
                        put<L>(gx, row, a.out_s, dx);
                    }
                    if (!simple && a.gfirst && p.real && (r.cuts.begin >> (b + k) & 1))
                        L::store(a.gfirst + (int64_t)seqs.begin[b + k] * a.c + p.c, mu);
                }
            }
#pragma unroll
            for (int k = 0; k < kHalf; ++k) held[k] = other[k];
        }
    };
    const auto carry = [&](int q) {  // the state before run q
        const int64_t lo = (int64_t)p.lo + q * kTokens;
        return p.real && q >= 0 && lo < a.n ? L::load(a.carries + lo / kTokens * a.c + p.c) : L::fill(0.f);
    };
    int q = a.runs - 1;
    N coming = carry(q);
    walk.go(seqs, a.glast, a.gfirst, [&](const Run& r, uint32_t* w) {
        const N state = coming;
        coming = carry(--q);
        by_kind<L>(r, w, [&](auto simple, auto closed) { go(simple, closed, r, w, state); });
    });
}

// 16 bytes of a lane's channels.
template <typename T, bool FREE>
__global__ void __launch_bounds__(kThreads) k_scan_step(int64_t vectors, int per_row, int c, const char* gate,
                                                        int64_t gate_s, const char* x, int64_t x_s, float* state,
                                                        char* out, int64_t out_s) {
    using L = Lane<T>;
    using G = typename L::template Gate<true>;
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
            const G g(gw[j]);
            hn[j] = next_state<FREE>(g, g.rest(), L::unpack(xw[j]), hn[j]);
            gw[j] = L::pack(hn[j]);
        }
#pragma unroll
        for (int j = 0; j < L::V; ++j) reinterpret_cast<float4*>(sp)[j] = h[j];
        *reinterpret_cast<uint4*>(out + r * out_s + at * 16) = g;
    }
}

// Runs of a warp, 1, 2, 4 .. kMaxRuns: the cut with the least time, reckoned in runs as those of the SM that has the
// most of them, and three more for each round of blocks, in which nothing is at hand yet.  (bf16, both passes:
// 25,179 tokens of 256 channels 63 us with 1 run a warp, 56 with 2, 54 with 2 forward and 4 backward; 319,057 of
// 128 208 us with 4, 211 with 8, 218 with 16; 602,492 of 512 1260 us with 4, 1246 with 8, 1234 with 16.)
struct Cut {
    int runs;
    int64_t tiles;
};
Cut cut_of(int64_t n, int c, int es, bool bwd, int sms) {
    const int64_t blocks_c = (c * es + kRowBytes - 1) / kRowBytes, slots = (int64_t)sms * per_sm(bwd);
    Cut best{};
    int64_t least = INT64_MAX;
    for (int runs = 1; runs <= kMaxRuns; runs *= 2) {
        const int64_t tile = (int64_t)kWarps * kTokens * runs, tiles = std::max<int64_t>(1, (n + tile - 1) / tile);
        const int64_t blocks = tiles * blocks_c;
        const int64_t time = (blocks + sms - 1) / sms * runs + (blocks + slots - 1) / slots * 3;
        if (time < least) {
            least = time;
            best = Cut{runs, tiles};
        }
    }
    return best;
}

// The most tiles that cut_of gives any call of up to n tokens, or a few times that: never fewer for more tokens, so that one
// workspace serves all shorter calls.  With b = tiles * blocks_c, a cut of `runs` is taken only where its time, at least
// b runs / sms + 3 b / slots, is at most that of `more` runs, below (b' / sms + 1) more + 3 (b' / slots + 1) with
// b' <= b runs / more + blocks_c; solved for the tiles.
int64_t most_tiles(int64_t n, int c, int es, bool bwd, int sms) {
    const int64_t blocks_c = (c * es + kRowBytes - 1) / kRowBytes, slots = (int64_t)sms * per_sm(bwd);
    int64_t most = 1;
    for (int runs = 1; runs <= kMaxRuns; runs *= 2) {
        const int64_t tile = (int64_t)kWarps * kTokens * runs;
        int64_t tiles = (n + tile - 1) / tile;
        for (int more = 2 * runs; more <= kMaxRuns; more *= 2)
            tiles = std::min(tiles, ((more + 3) * slots + blocks_c * (more * per_sm(bwd) + 3)) * more /
                                        (3 * blocks_c * (more - runs)));
        most = std::max(most, tiles);
    }
    return most;
}
// Of a call of so many tiles; more for more of them.
size_t workspace_of(int64_t tiles, int c) {
    return align_up(256 + (tiles > 1 ? (size_t)tiles * c * ((1 + kWarps) * sizeof(Map) + sizeof(float)) : 0), 256);
}

template <typename K>
bool allow(K kernel, size_t smem) {
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) == cudaSuccess;
}
template <typename T, bool FREE, bool BWD>
int launch(const ScanArgs& a, cudaStream_t s) {
    const unsigned grid = (unsigned)a.tiles * a.blocks_c;
    if (a.tiles > 1) {
        const auto kernel = k_scan_map<T, FREE, BWD>;
        if (!allow(kernel, stage_bytes(2))) return VG_ERR_CUDA;
        kernel<<<grid, kThreads, stage_bytes(2), s>>>(a);
        if (cudaPeekAtLastError() != cudaSuccess) return VG_ERR_CUDA;
    }
    if (a.tiles > kFoldTiles) {
        if (launch_after(k_scan_join<BWD>, a.c / kJoinChannels, kJoinChannels * kJoinParts, 0, s, a) != cudaSuccess)
            return VG_ERR_CUDA;
    }
    const auto kernel = BWD ? k_scan_bwd<T, FREE> : k_scan_fwd<T, FREE>;
    const size_t smem = stage_bytes(BWD ? 3 : 2);
    if (!allow(kernel, smem)) return VG_ERR_CUDA;
    if (a.tiles > 1) return launch_after(kernel, grid, kThreads, smem, s, a) == cudaSuccess ? VG_OK : VG_ERR_CUDA;
    kernel<<<grid, kThreads, smem, s>>>(a);
    return cudaPeekAtLastError() == cudaSuccess ? VG_OK : VG_ERR_CUDA;
}
template <typename T>
int launch(const ScanArgs& a, bool free_input, bool bwd, cudaStream_t s) {
    if (free_input) return bwd ? launch<T, true, true>(a, s) : launch<T, true, false>(a, s);
    return bwd ? launch<T, false, true>(a, s) : launch<T, false, false>(a, s);
}

}  // namespace

size_t gated_scan_workspace_bytes(int64_t n, int c, int dtype, int sms) {
    const int es = dtype == VG_F32 ? 4 : 2;
    return workspace_of(std::max(most_tiles(n, c, es, false, sms), most_tiles(n, c, es, true, sms)), c);
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
    const Cut cut = cut_of(a.n, a.c, es, bwd, q.sms);
    const int64_t tiles = cut.tiles;
    a.runs = cut.runs;
    if (tiles * a.blocks_c >= (int64_t(1) << 31)) return VG_ERR_UNSUPPORTED;
    if (workspace_of(tiles, a.c) > q.ws_bytes) return VG_ERR_WORKSPACE_TOO_SMALL;
    a.tiles = (int)tiles;
    a.tile_maps = reinterpret_cast<Map*>(q.ws + 256);
    a.warp_maps = a.tile_maps + tiles * a.c;
    a.states = reinterpret_cast<float*>(a.warp_maps + tiles * kWarps * a.c);
    const bool free_input = (q.s->flags & VG_SCAN_FREE_INPUT) != 0;
    return q.s->dtype == VG_F32   ? launch<float>(a, free_input, bwd, s)
           : q.s->dtype == VG_F16 ? launch<__half>(a, free_input, bwd, s)
                                  : launch<__nv_bfloat16>(a, free_input, bwd, s);
}

int gated_scan_step(int64_t n, int c, int dtype, bool free_input, const vg_rows& gate, const vg_rows& x, float* state,
                    const vg_rows& out, int sms, cudaStream_t s) {
    const int v = dtype == VG_F32 ? 4 : 8;
    const int64_t vectors = n * (c / v);
    const int grid = (int)std::min<int64_t>((vectors + kThreads - 1) / kThreads, (int64_t)sms * 8);
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
