// Host-side helpers shared by the translation units of the C ABI: cached
// device properties, the process-wide switches and pointer checks.  (Defined
// in gnq_api.cu.)
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace gnq {

constexpr int64_t kMaxH = 65536;
constexpr int64_t kMaxM = (int64_t)0x7FFFFFFF / 8;

constexpr int kMaxDevices = 64;

struct DevInfo {
    int dev;
    int sms;
    int smem_optin;     // largest dynamic shared memory a CTA may opt in to
    int smem_sm;        // shared memory of an SM
    unsigned int *err;  // device address of the error word
};

// Properties of the current device (nullptr on error), queried once per device.
const DevInfo *dev_info();

// The switches of gnq_set_pdl, gnq_set_constant_weights and
// gnq_inject_wait_timeout; the CTA that gnq_inject_split_timeout names (-1: off).
bool pdl_on();
bool constant_weights_on();
bool inject_timeout_on();
int inject_split_timeout();

// Clock cycles a bounded wait may spin (shorter under the test hooks).
constexpr long long kWaitLimit = 1LL << 31;      // about a second
constexpr long long kTestWaitLimit = 1LL << 20;  // under a millisecond
long long wait_limit_cycles();

// True if `ptr` is plain device memory (not pinned host, managed or unknown).
bool in_device_memory(const void *ptr);
// ... of this device.
bool on_device(const void *ptr, int dev);

inline bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// Launch `fn` with these dimensions, `cluster` CTAs per cluster along x, as a
// programmatic dependent where the switch is on.
template <typename... P, typename... A>
cudaError_t launch(void (*fn)(P...), int64_t grid, int threads, size_t smem, int cluster,
                   cudaStream_t stream, const A &...args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid, 1, 1);
    cfg.blockDim = dim3((unsigned)threads, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    unsigned n = 0;
    if (cluster > 1) {
        attr[n].id = cudaLaunchAttributeClusterDimension;
        attr[n].val.clusterDim.x = (unsigned)cluster;
        attr[n].val.clusterDim.y = 1;
        attr[n].val.clusterDim.z = 1;
        ++n;
    }
    if (pdl_on()) {
        attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[n].val.programmaticStreamSerializationAllowed = 1;
        ++n;
    }
    cfg.numAttrs = n;
    cfg.attrs = attr;
    return cudaLaunchKernelEx(&cfg, fn, args...);
}

}  // namespace gnq
