// Host-side helpers shared by the translation units of the C ABI: cached
// device properties, the process-wide switches and pointer checks.  (Defined
// in gnq_api.cu.)
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

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
// Kernel that gnq_set_linear_policy forces (0: the automatic choice).
int linear_policy();

// Clock cycles a bounded wait may spin (shorter under the test hooks).
constexpr long long kWaitLimit = 1LL << 31;      // about a second
constexpr long long kTestWaitLimit = 1LL << 20;  // under a millisecond
long long wait_limit_cycles();

// True if `ptr` is plain device memory (not pinned host, managed or unknown).
bool in_device_memory(const void *ptr);
// ... of this device.
bool on_device(const void *ptr, int dev);

inline bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// An answer (0 or more) that `ask` gives once and `slot`, 0 at first, keeps; -1
// where `ask` fails with -1, which is not kept: the next call asks again.
template <typename Ask> int answer_once(std::atomic<int> &slot, Ask ask) {
    int n = slot.load() - 1;
    if (n < 0 && (n = ask()) >= 0) slot.store(n + 1);
    return n;
}

// A stretch of memory of a call: `rows` rows of `width` bytes, `stride` bytes
// apart; empty for a buffer that the call does not use.
struct Extent {
    const void *at;
    int64_t rows, stride, width;
};
inline Extent extent(const void *p, int64_t bytes) { return {p, p ? 1 : 0, 0, bytes}; }

// Whether the contiguous stretch `a` shares a byte with `b`.
inline bool meets(const Extent &a, const Extent &b) {
    if (a.rows <= 0 || b.rows <= 0 || a.width <= 0 || b.width <= 0) return false;
    const uintptr_t a0 = reinterpret_cast<uintptr_t>(a.at), a1 = a0 + (uintptr_t)a.width;
    const uintptr_t b0 = reinterpret_cast<uintptr_t>(b.at);
    if (a1 <= b0) return false;
    if (a0 <= b0 || b.rows == 1) return a0 < b0 + (uintptr_t)b.width;
    // the last row that starts at or before `a`, then the next
    const uintptr_t r = (a0 - b0) / (uintptr_t)b.stride, row = b0 + r * (uintptr_t)b.stride;
    if (r >= (uintptr_t)b.rows) return false;
    return a0 < row + (uintptr_t)b.width || (r + 1 < (uintptr_t)b.rows && a1 > row + (uintptr_t)b.stride);
}

// What a call writes may be neither read by it nor written twice: CTAs run
// in any order.
template <int W, int R> bool outputs_meet(const Extent (&written)[W], const Extent (&read)[R]) {
    for (int i = 0; i < W; ++i) {
        for (int j = 0; j < i; ++j)
            if (meets(written[i], written[j])) return true;
        for (const Extent &r : read)
            if (meets(written[i], r)) return true;
    }
    return false;
}

// Bytes of the codes and block scales that a mode writes (0: none).
inline int64_t code_bytes(int mode, int64_t M, int64_t H) { return mode < 0 ? 0 : mode == 1 ? M * H / 2 : M * H; }
inline int64_t scale_bytes(int mode, int64_t M, int64_t H) {
    return mode == 1 ? (M + 127) / 128 * 8 * H : mode == 2 ? M * (H / 32) : 0;
}

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
