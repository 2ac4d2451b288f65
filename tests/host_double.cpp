// A stand-in for the HIP runtime and the kernels' launchers, for running
// zero_api.hip as host code on a machine without a GPU: device memory is heap
// memory whose ranges are known, copies are memcpy, and a launch is counted
// and its arguments kept. Only kernels that move data on their own
// (launch_fill_words) do so here.
#include <hip/hip_runtime_api.h>

#include <cstdlib>
#include <cstring>
#include <map>

#include "zero_internal.h"

namespace {

std::map<uintptr_t, size_t> ranges;
bool capturing;
int launches;                 // of any kernel
int copies;                   // hipMemcpyAsync
bool adamw_streams;           // of the last AdamW step
void *symbol[1 << 18];        // what hipGetSymbolAddress gives

hipError_t launched() {
    ++launches;
    return hipSuccess;
}

}  // namespace

extern "C" {

void double_capturing(int on) { capturing = on != 0; }
int double_launches() { return launches; }
int double_copies() { return copies; }
int double_adamw_streams() { return adamw_streams; }

hipError_t hipMalloc(void **p, size_t n) {
    *p = std::aligned_alloc(256, (n + 255) / 256 * 256);
    if (!*p) return hipErrorOutOfMemory;
    ranges[(uintptr_t)*p] = n;
    return hipSuccess;
}
hipError_t hipFree(void *p) {
    ranges.erase((uintptr_t)p);
    std::free(p);
    return hipSuccess;
}
hipError_t hipMemGetAddressRange(hipDeviceptr_t *base, size_t *size, hipDeviceptr_t p) {
    auto it = ranges.upper_bound((uintptr_t)p);
    if (it == ranges.begin()) return hipErrorNotFound;
    --it;
    if ((uintptr_t)p - it->first >= it->second) return hipErrorNotFound;
    *base = (hipDeviceptr_t)it->first;
    *size = it->second;
    return hipSuccess;
}
hipError_t hipMemset(void *p, int v, size_t n) { std::memset(p, v, n); return hipSuccess; }
hipError_t hipMemcpy(void *d, const void *s, size_t n, hipMemcpyKind) {
    std::memcpy(d, s, n);
    return hipSuccess;
}
hipError_t hipMemcpyAsync(void *d, const void *s, size_t n, hipMemcpyKind, hipStream_t) {
    ++copies;
    std::memcpy(d, s, n);
    return hipSuccess;
}
hipError_t hipGetDevice(int *d) { *d = 0; return hipSuccess; }
hipError_t hipSetDevice(int) { return hipSuccess; }
hipError_t hipDeviceGetAttribute(int *v, hipDeviceAttribute_t, int) { *v = 256; return hipSuccess; }
hipError_t hipDeviceSynchronize() { return hipSuccess; }
hipError_t hipStreamSynchronize(hipStream_t) { return hipSuccess; }
hipError_t hipStreamIsCapturing(hipStream_t, hipStreamCaptureStatus *s) {
    *s = capturing ? hipStreamCaptureStatusActive : hipStreamCaptureStatusNone;
    return hipSuccess;
}
hipError_t hipGetSymbolAddress(void **p, const void *) { *p = symbol; return hipSuccess; }
hipError_t hipGetLastError() { return hipSuccess; }
const char *hipGetErrorString(hipError_t) { return "error of the stand-in"; }

}  // extern "C"

namespace zk {

hipError_t launch_step(const StepArgs &, hipStream_t) { return launched(); }
hipError_t launch_begin_step(DevSchedule *ds, const float *, int64_t, const StepScalars &,
                             StepScalars *, hipStream_t) {
    ++ds->t;
    return launched();
}
hipError_t launch_set_schedule(DevSchedule *ds, int64_t t, float lr, hipStream_t) {
    if (t >= 1) ds->t = t;
    ds->lr = lr;
    return launched();
}
hipError_t launch_fill_words(uint32_t *dst, const WordChunk &c, hipStream_t) {
    std::memcpy(dst, c.w, (size_t)c.n * sizeof(uint32_t));
    return launched();
}
hipError_t launch_fsdp_step(const FsdpArgs &, hipStream_t) { return launched(); }
hipError_t launch_copy_segments(const Segment *, int, int, hipStream_t) { return launched(); }
hipError_t launch_load_master(const void *, bool, float *, float *, float *, int64_t, hipStream_t) {
    return launched();
}
hipError_t launch_adamw(const AdamwArgs &a, hipStream_t) {
    adamw_streams = a.stream_state;
    return launched();
}
hipError_t launch_sumsq(const SumsqArgs &, hipStream_t) { return launched(); }
hipError_t launch_adamw_decode(const AdamwStateRef &, int64_t, float *, float *, hipStream_t) {
    return launched();
}
hipError_t launch_adamw_encode(const AdamwStateRef &, int64_t, const float *, const float *,
                               hipStream_t) {
    return launched();
}
hipError_t launch_adamw_clear(const AdamwStateRef &, int64_t, hipStream_t) { return launched(); }
hipError_t launch_widen(const void *, bool, float *, int64_t, hipStream_t) { return launched(); }

}  // namespace zk
