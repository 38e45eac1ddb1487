// Cross attention on the tensor cores: the arithmetic of waiting, on the host as on
// the device (plain C++, so that it is tested without a GPU).
#pragma once
#include <cstdint>

#ifdef __CUDACC__
#define VG_HOST_DEVICE __host__ __device__ __forceinline__
#else
#define VG_HOST_DEVICE inline
#endif

namespace vg {

// Copies into a ring of S slots, each of which completes the next phase of its slot's
// barrier.  A slot is used again only once it has been read, so at most the last S can be
// in flight: what a warp that leaves, at the end or because it gave up, has to see land.
// A copy is counted where it is issued, so that no way out skips one.
template <int S>
struct Copies {
    uint32_t n = 0;
    VG_HOST_DEVICE void issued() { ++n; }
    // Slot of the next copy, and the parity of the pass over the ring that it belongs to.
    VG_HOST_DEVICE uint32_t slot() const { return n % S; }
    VG_HOST_DEVICE uint32_t pass() const { return (n / S) & 1u; }
    // f(slot, parity of the phase that its last copy completes)
    template <typename F>
    VG_HOST_DEVICE void in_flight(F f) const {
        for (uint32_t i = n > (uint32_t)S ? n - S : 0u; i < n; ++i) f(i % S, (i / S) & 1u);
    }
};

// A hand-over between two warps takes a step's work, some 1,000 to 3,000 cycles; a wait for one gives up after
// kWaitCycles.  A wait for the next unit, or for the slot of a unit that is being worked on, lasts as long as
// a unit, whose number of steps the caller sets: it has kStepCycles more for each of them.
constexpr int64_t kWaitCycles = 4000000000ll;  // about 2 s of an SM's cycle counter
constexpr int64_t kStepCycles = 1 << 16;

// Most steps of a unit that runs along `rows` rows in tiles of `tile`, `sets` times, in parts of `per_part` tiles if
// there is more than one.
VG_HOST_DEVICE int64_t unit_steps(int splits, int per_part, int64_t rows, int tile, int64_t sets) {
    return (splits > 1 ? (int64_t)per_part : (rows + tile - 1) / tile) * sets;
}
VG_HOST_DEVICE int64_t unit_wait_cycles(int64_t steps) {
    constexpr int64_t most = INT64_MAX / 4 / kStepCycles;
    return kWaitCycles + (steps < most ? steps : most) * kStepCycles;
}

}  // namespace vg
