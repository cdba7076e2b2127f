// Host-side checks shared by the entry points: the current device, and who
// owns each buffer a call is given.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <map>
#include <mutex>

#include "internal.h"

namespace muon {

inline int64_t round_up(int64_t x, int64_t q) { return (x + q - 1) / q * q; }

struct DeviceInfo {
    int ok = -1;  // -1 unknown, 0 unsupported, 1 sm_103
    int num_sms = 0;
};

inline muon_status_t device_info(int* num_sms) {
    static std::mutex mu;
    static DeviceInfo info[64];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return MUON_ERR_NO_DEVICE;
    if (dev < 0 || dev >= 64) return MUON_ERR_NO_DEVICE;
    std::lock_guard<std::mutex> lock(mu);
    DeviceInfo& d = info[dev];
    if (d.ok < 0) {
        int major = 0, minor = 0, sms = 0;
        if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
            cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess ||
            cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
            return MUON_ERR_CUDA;
        d.ok = (major == 10 && minor == 3) ? 1 : 0;
        d.num_sms = sms;
    }
    if (d.ok != 1) return MUON_ERR_NO_DEVICE;
    *num_sms = d.num_sms;
    return MUON_OK;
}

// ---------------------------------------------------------------------------
// Whose memory the caller's buffers are.  Every buffer the kernels read or
// write must be memory the current device owns: a device allocation made on
// it, or managed memory.  Host memory (pinned or pageable), another device's
// allocations and unknown addresses are refused with MUON_ERR_INVALID_ARG
// before anything is enqueued, so such a call ends in an error code rather
// than in a memory fault on the device.  Each driver query also looks up the
// bounds of the allocation holding the pointer and remembers them, so the
// views of one large buffer cost a single query.
// ---------------------------------------------------------------------------
typedef CUresult (*AddressRangeFn)(CUdeviceptr*, size_t*, CUdeviceptr);

inline AddressRangeFn address_range_fn() {
    static AddressRangeFn fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void* ptr = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuMemGetAddressRange", &ptr, 12000, cudaEnableDefault, &q) ==
                cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<AddressRangeFn>(ptr);
    });
    return fn;
}

class DeviceMemoryCheck {
  public:
    explicit DeviceMemoryCheck(int device) : dev_(device) {}

    // Whether the buffer starting at p (bytes long) is the current device's.
    bool owns(const void* p, size_t bytes) {
        const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
        auto it = known_.upper_bound(lo);
        if (it != known_.begin()) {
            --it;
            if (lo >= it->first && lo + bytes <= it->second) return true;
        }
        cudaPointerAttributes a;
        if (cudaPointerGetAttributes(&a, p) != cudaSuccess) {
            cudaGetLastError();  // a refused query must not look like a failed launch later
            return false;
        }
        const bool mine = (a.type == cudaMemoryTypeDevice && a.device == dev_) || a.type == cudaMemoryTypeManaged;
        if (!mine) return false;
        CUdeviceptr base = 0;
        size_t size = 0;
        const AddressRangeFn range = address_range_fn();
        if (range && range(&base, &size, static_cast<CUdeviceptr>(lo)) == CUDA_SUCCESS && size > 0)
            known_[static_cast<uintptr_t>(base)] = static_cast<uintptr_t>(base) + size;
        return true;
    }

  private:
    int dev_;
    std::map<uintptr_t, uintptr_t> known_;  // verified allocations, start -> end
};

// Whether `st` is being captured into a graph.  A capture records launches
// only, so the memory checks are left out there (muon_step_graph_create
// checks before it captures); a stream whose state cannot be read counts as
// capturing.
inline bool capturing(cudaStream_t st) {
    cudaStreamCaptureStatus cs = cudaStreamCaptureStatusNone;
    if (cudaStreamIsCapturing(st, &cs) != cudaSuccess) {
        cudaGetLastError();
        return true;
    }
    return cs != cudaStreamCaptureStatusNone;
}

inline muon_status_t from_cuda(cudaError_t e) { return e == cudaSuccess ? MUON_OK : MUON_ERR_CUDA; }

}  // namespace muon
