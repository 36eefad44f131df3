// route_layout.h -- dynamic shared memory of the kernel that places routed pairs
// (route_place), computed once for the kernel and for its launch. Plain C++: the
// host tests compile it.
#pragma once

#include <cstddef>

#ifdef __CUDACC__
#define DG_ROUTE_FN __host__ __device__ inline
#else
#define DG_ROUTE_FN inline
#endif

namespace dg {
namespace route {

constexpr int kPlaceThreads = 1024;

// Experts of a row of counts: whole words of four.
DG_ROUTE_FN int pitch_of(int E) { return (E + 3) / 4 * 4; }

// mask     [pitch] 64-bit words at offset 0
// before   [parts][pitch] int, at `before` bytes
// base     [parts][pitch] int, at `base` bytes
// Threads take quads of experts, `parts` of them share a quad; the pitch (not E)
// sizes every array, so that a quad's 16-byte stores are aligned and inside.
struct PlaceLayout {
    int pitch, parts;
    size_t before, base, bytes;
    DG_ROUTE_FN explicit PlaceLayout(int E) {
        pitch = pitch_of(E);
        const int n = kPlaceThreads / (pitch / 4);
        parts = n < 1 ? 1 : n > 32 ? 32 : n;
        before = static_cast<size_t>(pitch) * 8;
        base = before + static_cast<size_t>(parts) * pitch * 4;
        bytes = base + static_cast<size_t>(parts) * pitch * 4;
    }
};

}  // namespace route
}  // namespace dg
