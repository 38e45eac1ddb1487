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
    // f(slot, parity of the phase that its last copy completes)
    template <typename F>
    VG_HOST_DEVICE void in_flight(F f) const {
        for (uint32_t i = n > (uint32_t)S ? n - S : 0u; i < n; ++i) f(i % S, (i / S) & 1u);
    }
};

}  // namespace vg
