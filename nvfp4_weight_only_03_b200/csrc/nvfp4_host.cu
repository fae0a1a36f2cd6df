// What the serving operators ask about the current device, looked up once per device.  Threads may
// look at the same time: each finds the same, and what one has stored is complete for the others.
#include <atomic>

#include "nvfp4_host.h"

namespace nvfp4_host {

namespace {
struct DeviceInfo {
    std::atomic<int> ok{-1};  // -1 unknown, 0 not a B200, 1 ok: stored behind the count
    std::atomic<int> sms{0};
};
DeviceInfo g_device[64];
std::atomic<EncodeFn> g_encode{nullptr};
}  // namespace

int device(int* dev, int* sms, EncodeFn* encode) {
    int d = 0;
    if (cudaGetDevice(&d) != cudaSuccess || d < 0 || d >= 64) {
        cudaGetLastError();
        return NVFP4_ERR_ARCH;
    }
    DeviceInfo& di = g_device[d];
    if (di.ok < 0) {
        int major = 0, minor = 0, count = 0;
        if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, d) != cudaSuccess ||
            cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, d) != cudaSuccess ||
            cudaDeviceGetAttribute(&count, cudaDevAttrMultiProcessorCount, d) != cudaSuccess) {
            cudaGetLastError();
            return NVFP4_ERR_ARCH;
        }
        di.sms = count;
        di.ok = (major == 10 && minor == 0) ? 1 : 0;
    }
    if (di.ok != 1) return NVFP4_ERR_ARCH;
    if (!g_encode) {
        void* fn = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &fn, cudaEnableDefault, &q) !=
                cudaSuccess ||
            q != cudaDriverEntryPointSuccess || !fn) {
            cudaGetLastError();
            return NVFP4_ERR_ARCH;
        }
        g_encode = reinterpret_cast<EncodeFn>(fn);
    }
    *dev = d;
    *sms = di.sms;
    *encode = g_encode;
    return NVFP4_OK;
}

}  // namespace nvfp4_host
