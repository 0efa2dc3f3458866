// A stand-in for the CUDA runtime, for tests of the library's host code on a
// machine without a GPU: launches are counted and checked, nothing runs.  The
// library's object files are linked against it instead of the runtime.
#include <chrono>
#include <condition_variable>
#include <cstdint>
#include <cstring>
#include <map>
#include <mutex>
#include <thread>

#include <cuda_runtime_api.h>

namespace {

std::mutex mu;
std::map<const void *, int> limits;    // dynamic shared memory that each kernel may use
thread_local cudaError_t last = cudaSuccess;
int launches = 0, fail_at = 0;         // fail_at: the launch (counted from 1) that fails
int slow_bytes = 0;                    // setting a limit this large is slow to return
bool in_slow = false;                  // ... and has been entered

thread_local struct {
    dim3 grid, block;
    size_t smem;
    cudaStream_t stream;
} call;

cudaError_t launch(const void *kernel, size_t smem) {
    std::lock_guard<std::mutex> lock(mu);
    ++launches;
    const auto it = limits.find(kernel);
    const size_t limit = it == limits.end() ? 48 * 1024 : (size_t)it->second;
    cudaError_t e = cudaSuccess;
    if (smem > limit) e = cudaErrorInvalidValue;
    if (launches == fail_at) e = cudaErrorLaunchOutOfResources;
    if (e != cudaSuccess) last = e;
    return e;
}

}  // namespace

extern "C" {

void fake_reset() {
    std::lock_guard<std::mutex> lock(mu);
    launches = fail_at = slow_bytes = 0;
    in_slow = false;
    last = cudaSuccess;
}
int fake_launches() {
    std::lock_guard<std::mutex> lock(mu);
    return launches;
}
void fake_fail_at(int n) {
    std::lock_guard<std::mutex> lock(mu);
    launches = 0;
    fail_at = n;
}
void fake_slow_limit(int bytes) {
    std::lock_guard<std::mutex> lock(mu);
    slow_bytes = bytes;
}
int fake_in_slow_limit() {
    std::lock_guard<std::mutex> lock(mu);
    return in_slow;
}

// ---- the runtime
cudaError_t cudaGetLastError() {
    const cudaError_t e = last;
    last = cudaSuccess;
    return e;
}
cudaError_t cudaGetDevice(int *d) {
    *d = 0;
    return cudaSuccess;
}
cudaError_t cudaDeviceGetAttribute(int *v, cudaDeviceAttr a, int) {
    *v = a == cudaDevAttrMultiProcessorCount ? 152 : 0;
    return cudaSuccess;
}
cudaError_t cudaFuncSetAttribute(const void *f, cudaFuncAttribute, int value) {
    bool slow;
    {
        std::lock_guard<std::mutex> lock(mu);
        limits[f] = value;
        slow = slow_bytes > 0 && value >= slow_bytes;
        if (slow) in_slow = true;
    }
    if (slow) std::this_thread::sleep_for(std::chrono::milliseconds(500));
    return cudaSuccess;
}
cudaError_t cudaOccupancyMaxActiveBlocksPerMultiprocessor(int *n, const void *, int, size_t) {
    *n = 1;
    return cudaSuccess;
}
cudaError_t cudaOccupancyMaxActiveBlocksPerMultiprocessorWithFlags(int *n, const void *, int, size_t, unsigned) {
    *n = 1;
    return cudaSuccess;
}
cudaError_t cudaLaunchKernelExC(const cudaLaunchConfig_t *c, const void *f, void **) { return launch(f, c->dynamicSmemBytes); }
cudaError_t cudaMemcpyToSymbol(const void *, const void *, size_t, size_t, cudaMemcpyKind) { return cudaSuccess; }
cudaError_t cudaMemcpyFromSymbol(void *d, const void *, size_t n, size_t, cudaMemcpyKind) {
    std::memset(d, 0, n);
    return cudaSuccess;
}
cudaError_t cudaMemcpyAsync(void *, const void *, size_t, cudaMemcpyKind, cudaStream_t) { return cudaSuccess; }
cudaError_t cudaMemsetAsync(void *, int, size_t, cudaStream_t) { return cudaSuccess; }
cudaError_t cudaStreamSynchronize(cudaStream_t) { return cudaSuccess; }
cudaError_t cudaGetSymbolAddress(void **p, const void *s) {
    *p = const_cast<void *>(s);
    return cudaSuccess;
}
cudaError_t cudaGetDriverEntryPointByVersion(const char *, void **, unsigned, unsigned long long, cudaDriverEntryPointQueryResult *) {
    return cudaErrorNotSupported;
}

// ---- what a <<<>>> launch and the registration of device code call
unsigned __cudaPushCallConfiguration(dim3 grid, dim3 block, size_t smem, cudaStream_t stream) {
    call = {grid, block, smem, stream};
    return 0;
}
cudaError_t __cudaPopCallConfiguration(dim3 *grid, dim3 *block, size_t *smem, void *stream) {
    *grid = call.grid;
    *block = call.block;
    *smem = call.smem;
    *static_cast<cudaStream_t *>(stream) = call.stream;
    return cudaSuccess;
}
cudaError_t __cudaGetKernel(cudaKernel_t *k, const void *f) {
    *k = (cudaKernel_t) const_cast<void *>(f);
    return cudaSuccess;
}
cudaError_t __cudaLaunchKernel(cudaKernel_t k, dim3, dim3, void **, size_t smem, cudaStream_t) {
    return launch((const void *)k, smem);
}
void **__cudaRegisterFatBinary(void *) {
    static void *handle;
    return &handle;
}
void __cudaRegisterFatBinaryEnd(void **) {}
void __cudaUnregisterFatBinary(void **) {}
void __cudaRegisterFunction(void **, const char *, char *, const char *, int, void *, void *, void *, void *, int *) {}
void __cudaRegisterVar(void **, char *, char *, const char *, int, size_t, int, int) {}

}  // extern "C"
