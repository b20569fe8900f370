// fake_cudart.cpp -- a stand-in for the CUDA runtime's entry points that the library
// calls, so that its host side runs without a GPU: nothing is launched, every launch
// and allocation is written down.  A split kernel's launch takes a while, so that
// what another host thread may put between it and its join does come between.
#include <chrono>
#include <cstdio>
#include <cstring>
#include <map>
#include <mutex>
#include <string>
#include <thread>

#include <cuda.h>
#include <cuda_runtime_api.h>

namespace {

std::mutex mu;
std::map<const void *, std::string> names;
std::string text;
unsigned long long next_address = 1ull << 32, capture = 0;
int capture_objects = 0;
unsigned int word;
thread_local int me = -1;
thread_local bool bound = false;  // this host thread has a context: some runtime calls give it one

CUresult encode(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *, const cuuint64_t *,
                const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                CUtensorMapL2promotion, CUtensorMapFloatOOBfill) {
    return bound ? CUDA_SUCCESS : CUDA_ERROR_INVALID_CONTEXT;
}

void note(const std::string &line) {
    std::lock_guard<std::mutex> lk(mu);
    text += line + "\n";
}

bool joins(const std::string &name) {
    return name.find("merge_kernel") != std::string::npos || name.find("combine_kernel") != std::string::npos;
}

}  // namespace

extern "C" {

// ------------------------------------------------------- for the tests
__attribute__((visibility("default"))) void fake_thread(int id) { me = id; }
__attribute__((visibility("default"))) void fake_clear() {
    std::lock_guard<std::mutex> lk(mu);
    text.clear();
}
// 0: streams are not captured; else the id of their capture
__attribute__((visibility("default"))) void fake_capture(unsigned long long id) { capture = id; }
__attribute__((visibility("default"))) size_t fake_log(char *out, size_t size) {
    std::lock_guard<std::mutex> lk(mu);
    if (out && size > text.size()) memcpy(out, text.c_str(), text.size() + 1);
    return text.size() + 1;
}

// ------------------------------------------------------- registration
void **__cudaRegisterFatBinary(void *) {
    static void *handle;
    return &handle;
}
void __cudaRegisterFatBinaryEnd(void **) {}
void __cudaUnregisterFatBinary(void **) {}
void __cudaRegisterFunction(void **, const char *host, char *, const char *name, int, void *, void *, void *, void *,
                            int *) {
    names[host] = name;
}
void __cudaRegisterVar(void **, char *, char *, const char *, int, size_t, int, int) {}
unsigned __cudaPushCallConfiguration(dim3, dim3, size_t, void *) { return 0; }
cudaError_t __cudaPopCallConfiguration(dim3 *, dim3 *, size_t *, void *) { return cudaSuccess; }
cudaError_t __cudaGetKernel(void **kernel, const void *host) {
    *kernel = const_cast<void *>(host);
    return cudaSuccess;
}
cudaError_t __cudaLaunchKernel(void *, dim3, dim3, void **, size_t, cudaStream_t) { return cudaSuccess; }

// ------------------------------------------------------- the runtime
cudaError_t cudaLaunchKernelExC(const cudaLaunchConfig_t *cfg, const void *host, void **) {
    const std::string name = names.count(host) ? names[host] : "?";
    note("launch " + std::to_string(me) + " " + std::to_string((unsigned long long)(uintptr_t)cfg->stream) + " " + name);
    bound = true;
    if (!joins(name)) std::this_thread::sleep_for(std::chrono::milliseconds(3));
    return cudaSuccess;
}
cudaError_t cudaMalloc(void **p, size_t bytes) {
    std::lock_guard<std::mutex> lk(mu);
    bound = true;
    *p = reinterpret_cast<void *>(next_address);
    next_address += (bytes + 4095) / 4096 * 4096;
    text += "malloc " + std::to_string(me) + " " + std::to_string(bytes) + "\n";
    return cudaSuccess;
}
cudaError_t cudaFree(void *) {
    note("free " + std::to_string(me));
    return cudaSuccess;
}
cudaError_t cudaDeviceSynchronize() {
    note("sync " + std::to_string(me));
    return cudaSuccess;
}
cudaError_t cudaGetDevice(int *d) {
    *d = 0;
    return cudaSuccess;
}
cudaError_t cudaSetDevice(int) {
    bound = true;
    return cudaSuccess;
}
cudaError_t cudaDeviceGetAttribute(int *v, cudaDeviceAttr, int) {
    *v = 152;
    return cudaSuccess;
}
cudaError_t cudaGetSymbolAddress(void **p, const void *) {
    *p = &word;
    return cudaSuccess;
}
cudaError_t cudaFuncSetAttribute(const void *, cudaFuncAttribute, int) { return cudaSuccess; }
cudaError_t cudaGetLastError() { return cudaSuccess; }
const char *cudaGetErrorString(cudaError_t) { return "an error"; }
cudaError_t cudaGetDriverEntryPointByVersion(const char *, void **fn, unsigned, unsigned long long,
                                             cudaDriverEntryPointQueryResult *q) {
    *fn = reinterpret_cast<void *>(encode);
    *q = cudaDriverEntryPointSuccess;
    return cudaSuccess;
}
cudaError_t cudaEventRecord(cudaEvent_t, cudaStream_t) { return cudaSuccess; }
cudaError_t cudaStreamSynchronize(cudaStream_t) { return cudaSuccess; }
cudaError_t cudaMemcpyFromSymbol(void *, const void *, size_t, size_t, cudaMemcpyKind) { return cudaSuccess; }
cudaError_t cudaMemcpyToSymbol(const void *, const void *, size_t, size_t, cudaMemcpyKind) { return cudaSuccess; }
cudaError_t cudaStreamGetCaptureInfo(cudaStream_t, cudaStreamCaptureStatus *st, unsigned long long *id, cudaGraph_t *,
                                     const cudaGraphNode_t **, const cudaGraphEdgeData **, size_t *) {
    *st = capture ? cudaStreamCaptureStatusActive : cudaStreamCaptureStatusNone;
    if (id) *id = capture;
    return cudaSuccess;
}
cudaError_t cudaThreadExchangeStreamCaptureMode(cudaStreamCaptureMode *) { return cudaSuccess; }
cudaError_t cudaUserObjectCreate(cudaUserObject_t *o, void *, cudaHostFn_t, unsigned, unsigned) {
    *o = reinterpret_cast<cudaUserObject_t>(&capture_objects);
    ++capture_objects;
    return cudaSuccess;
}
cudaError_t cudaUserObjectRelease(cudaUserObject_t, unsigned) { return cudaSuccess; }
cudaError_t cudaGraphRetainUserObject(cudaGraph_t, cudaUserObject_t, unsigned, unsigned) { return cudaSuccess; }

}  // extern "C"
