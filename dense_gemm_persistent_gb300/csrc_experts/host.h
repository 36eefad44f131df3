// host.h -- the host-side services of api.cu that the expert operators share:
// device state, launch epochs, tensor maps, and the override fields that apply
// to every bounded wait.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

#include "dgemm.h"

namespace dg {
namespace host {

struct Device {
    int id, num_sms;
    unsigned* status;   // the per-device status word
};

// The current device; DGEMM_ERR_ARCH unless it is sm_103.
dgemm_status_t current_device(Device* out);

// A fresh launch epoch (tags the status word of a workspace).
unsigned long long next_launch_epoch();

// Tiled tensor map with 128-byte swizzle; strides (bytes) has rank - 1 entries.
// Out-of-range coordinates load as zero.
bool encode_map(CUtensorMap* m, CUtensorMapDataType type, const void* ptr, int rank, const uint64_t* dims,
                const uint64_t* strides, const uint32_t* box);

// Limit of every bounded device-side wait, and the testing override that stops
// a producer early (< 0: off).
void wait_settings(uint64_t* wait_ns, long long* stall_after);

// The planner override for CTA pairs: -1 none, 0 never, 1 always.
int pair_override();

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

constexpr int kMaxDevices = 64;

// Launch configuration with programmatic dependent launch: the kernel may start
// while the previous one in the stream finishes, and waits on griddepcontrol
// before touching global memory.
struct Launch {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    Launch(unsigned gx, unsigned gy, unsigned threads, size_t smem, cudaStream_t s, int cluster = 1) {
        cfg.gridDim = dim3(gx, gy);
        cfg.blockDim = dim3(threads);
        cfg.dynamicSmemBytes = smem;
        cfg.stream = s;
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        cfg.numAttrs = 1;
        if (cluster > 1) {
            attr[1].id = cudaLaunchAttributeClusterDimension;
            attr[1].val.clusterDim.x = static_cast<unsigned>(cluster);
            attr[1].val.clusterDim.y = 1;
            attr[1].val.clusterDim.z = 1;
            cfg.numAttrs = 2;
        }
        cfg.attrs = attr;
    }
};

}  // namespace host
}  // namespace dg
