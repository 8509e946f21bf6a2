// fake_cuda.cpp -- the few CUDA calls that the token operators' host code
// makes, without a GPU: launches are written down instead of run, and any
// call can be made to fail. Linked with the operators' own translation units
// into a library of its own (tests/test_tokens_launches_cpu.py).
#include <cuda.h>
#include <cuda_runtime.h>

#include <cstring>
#include <map>
#include <mutex>
#include <string>
#include <vector>

namespace {

struct Launch {
    std::string name;
    dim3 grid, block;
    size_t smem;
};

struct State {
    std::mutex mu;
    std::map<const void *, std::string> names;  // by host function
    std::map<const void *, int> limit;          // dynamic shared memory a function may take
    std::vector<Launch> launches;
    int last_error = 0;
    int launch_to_fail = -1;     // counted from the last reset
    int fail_attributes = 0;
    int attributes = 0;          // calls of cudaFuncSetAttribute
    void (*before_launch)() = nullptr;
};

State &state() {
    static State s;
    return s;
}

cudaError_t fail(int code) {
    state().last_error = code;
    return (cudaError_t)code;
}

CUresult encode(...) { return CUDA_SUCCESS; }

}  // namespace

namespace lmc {
int sm_count() { return 152; }
}  // namespace lmc

extern "C" {

// ---- for the tests ----
__attribute__((visibility("default"))) void fake_reset(void) {
    State &s = state();
    s.launches.clear();
    s.last_error = 0;
    s.launch_to_fail = -1;
    s.fail_attributes = 0;
    s.attributes = 0;
    s.before_launch = nullptr;
}
__attribute__((visibility("default"))) void fake_fail_launch(int n) { state().launch_to_fail = n; }
__attribute__((visibility("default"))) void fake_fail_attributes(int on) { state().fail_attributes = on; }
__attribute__((visibility("default"))) void fake_set_last_error(int code) { state().last_error = code; }
__attribute__((visibility("default"))) int fake_last_error(void) { return state().last_error; }
__attribute__((visibility("default"))) int fake_attributes(void) { return state().attributes; }
__attribute__((visibility("default"))) void fake_before_launch(void (*f)()) { state().before_launch = f; }
__attribute__((visibility("default"))) int fake_launches(void) { return (int)state().launches.size(); }
// (grid x, y, z, threads, dynamic shared memory) of a launch; its kernel's name
__attribute__((visibility("default"))) const char *fake_launch(int i, long long out[5]) {
    const Launch &l = state().launches[i];
    out[0] = l.grid.x;
    out[1] = l.grid.y;
    out[2] = l.grid.z;
    out[3] = l.block.x;
    out[4] = (long long)l.smem;
    return l.name.c_str();
}

// ---- what the operators call ----
cudaError_t cudaGetDevice(int *dev) {
    *dev = 0;
    return cudaSuccess;
}

cudaError_t cudaGetLastError(void) {
    const int e = state().last_error;
    state().last_error = 0;
    return (cudaError_t)e;
}

cudaError_t cudaFuncSetAttribute(const void *f, cudaFuncAttribute attr, int value) {
    State &s = state();
    s.attributes++;
    if (s.fail_attributes || attr != cudaFuncAttributeMaxDynamicSharedMemorySize || value < 0 || value > 227 * 1024)
        return fail(cudaErrorInvalidValue);
    s.limit[f] = value;
    return cudaSuccess;
}

cudaError_t cudaLaunchKernelExC(const cudaLaunchConfig_t *cfg, const void *f, void **) {
    State &s = state();
    if (void (*hook)() = s.before_launch) {
        s.before_launch = nullptr;  // a call made by it does not come here again
        hook();
    }
    const int n = (int)s.launches.size();
    const auto it = s.limit.find(f);
    const size_t most = it == s.limit.end() ? 48 * 1024 : (size_t)it->second;
    if (n == s.launch_to_fail)
        return fail(cudaErrorLaunchOutOfResources);
    if (cfg->dynamicSmemBytes > most || cfg->gridDim.x == 0 || cfg->gridDim.y == 0 || cfg->gridDim.y > 65535)
        return fail(cudaErrorInvalidValue);
    s.launches.push_back(Launch{s.names[f], cfg->gridDim, cfg->blockDim, cfg->dynamicSmemBytes});
    return cudaSuccess;
}

cudaError_t cudaGetDriverEntryPointByVersion(const char *, void **fn, unsigned int, unsigned long long,
                                             cudaDriverEntryPointQueryResult *found) {
    *fn = reinterpret_cast<void *>(encode);
    *found = cudaDriverEntryPointSuccess;
    return cudaSuccess;
}

// ---- what a CUDA translation unit registers when it is loaded ----
void **__cudaRegisterFatBinary(void *) {
    static void *handle;
    return &handle;
}
void __cudaRegisterFatBinaryEnd(void **) {}
void __cudaUnregisterFatBinary(void **) {}
void __cudaRegisterFunction(void **, const char *host, char *, const char *name, int, uint3 *, uint3 *, dim3 *, dim3 *,
                            int *) {
    state().names[host] = name;
}
cudaError_t __cudaGetKernel(cudaKernel_t *k, const void *f) {
    *k = (cudaKernel_t) const_cast<void *>(f);
    return cudaSuccess;
}
cudaError_t __cudaLaunchKernel(cudaKernel_t, dim3, dim3, void **, size_t, cudaStream_t) {
    return fail(cudaErrorNotSupported);
}
unsigned __cudaPushCallConfiguration(dim3, dim3, size_t, struct CUstream_st *) { return 0; }
cudaError_t __cudaPopCallConfiguration(dim3 *, dim3 *, size_t *, void *) { return cudaSuccess; }

}  // extern "C"
