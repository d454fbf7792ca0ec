// hip_stub.cpp -- host-only stand-ins for the HIP runtime, for building the
// host halves of the .hip files (their planning code and launches) on the CPU
// under AddressSanitizer and UndefinedBehaviorSanitizer.  A launch is checked
// against what a grid can hold and counted; nothing reaches a device.
// Test infrastructure only: nothing here is part of libq4.so.
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace {
int g_launches = 0, g_bad = 0;
}  // namespace

extern "C" {

int hipstub_launches(void) { return g_launches; }
int hipstub_bad(void) { return g_bad; }

hipError_t hipLaunchKernel(const void *fn, dim3 grid, dim3 block, void **args, size_t, hipStream_t) {
    ++g_launches;
    const uint64_t threads = (uint64_t)block.x * block.y * block.z;
    if (!fn || !args || !grid.x || !grid.y || !grid.z || !threads || threads > 1024 || grid.y > 65535 || grid.z > 65535 ||
        (uint64_t)grid.x * block.x >= UINT64_C(1) << 32)
        ++g_bad;
    return hipSuccess;
}
hipError_t hipMemcpyAsync(void *, const void *, size_t, hipMemcpyKind, hipStream_t) { return hipSuccess; }
hipError_t hipGetDevice(int *dev) {
    *dev = 0;
    return hipSuccess;
}
hipError_t hipDeviceGetAttribute(int *v, hipDeviceAttribute_t, int) {
    *v = 256;
    return hipSuccess;
}
void **__hipRegisterFatBinary(const void *) {
    static void *handle;
    return &handle;
}
void __hipUnregisterFatBinary(void **) {}
void __hipRegisterFunction(void **, const void *, char *, const char *, unsigned, void *, void *, void *, void *, int *) {}
void __hipRegisterVar(void **, void *, char *, const char *, int, size_t, int, int) {}
hipError_t __hipPushCallConfiguration(dim3, dim3, size_t, hipStream_t) { return hipSuccess; }
hipError_t __hipPopCallConfiguration(dim3 *, dim3 *, size_t *, hipStream_t *) { return hipSuccess; }

}  // extern "C"
