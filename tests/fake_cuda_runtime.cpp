// A stand-in for the CUDA runtime calls that minf_block_tables.cu makes, for tests of its launches on the host: kernels
// never run, limits and errors are kept as the runtime keeps them.
#include <cuda_runtime_api.h>

#include <stdint.h>
#include <map>

namespace {

constexpr int kDefaultLimit = 48 * 1024, kMostOptIn = 227 * 1024;

struct Kernel {
    int limit = -1;         // dynamic bytes that were opted in to (-1: none)
    bool large_cluster = false;
};
std::map<const void *, Kernel> kernels;
cudaError_t last = cudaSuccess;
int static_bytes = 0;       // a kernel's own arrays
int clusters_of_16 = 1;     // what the occupancy query says for them
bool refuse_large_clusters = false;
int launches = 0, last_dynamic = 0, last_cluster = 0;
int32_t (*meanwhile)() = nullptr;  // runs once, after the next setting of a limit: another host thread

cudaError_t end(cudaError_t e) {
    if (e != cudaSuccess) last = e;
    return e;
}

}  // namespace

extern "C" {

void fake_reset(int own_bytes) {
    kernels.clear();
    last = cudaSuccess;
    static_bytes = own_bytes;
    clusters_of_16 = 1;
    refuse_large_clusters = false;
    launches = last_dynamic = last_cluster = 0;
    meanwhile = nullptr;
}
void fake_meanwhile(int32_t (*f)()) { meanwhile = f; }
void fake_clusters_of_16(int n) { clusters_of_16 = n; }
void fake_refuse_large_clusters() { refuse_large_clusters = true; }
int fake_launches() { return launches; }
int fake_dynamic() { return last_dynamic; }
int fake_cluster() { return last_cluster; }
int fake_last_error() { return last; }

void **__cudaRegisterFatBinary(void *) {
    static void *handle;
    return &handle;
}
void __cudaRegisterFatBinaryEnd(void **) {}
void __cudaUnregisterFatBinary(void **) {}
void __cudaRegisterFunction(void **, const char *, char *, const char *, int, void *, void *, void *, void *, int *) {}
unsigned __cudaPushCallConfiguration(dim3, dim3, size_t, void *) { return 0; }
cudaError_t __cudaPopCallConfiguration(dim3 *, dim3 *, size_t *, void *) { return cudaSuccess; }
cudaError_t __cudaGetKernel(void **, const void *) { return end(cudaErrorNotSupported); }
cudaError_t __cudaLaunchKernel(void *, dim3, dim3, void **, size_t, cudaStream_t) { return end(cudaErrorNotSupported); }

cudaError_t cudaGetLastError() {
    const cudaError_t e = last;
    last = cudaSuccess;
    return e;
}
cudaError_t cudaPeekAtLastError() { return last; }

cudaError_t cudaFuncSetAttribute(const void *f, cudaFuncAttribute what, int value) {
    if (what == cudaFuncAttributeNonPortableClusterSizeAllowed) {
        if (refuse_large_clusters) return end(cudaErrorNotSupported);
        kernels[f].large_cluster = value != 0;
        return cudaSuccess;
    }
    if (value < 0 || value + static_bytes > kMostOptIn) return end(cudaErrorInvalidValue);
    kernels[f].limit = value;
    if (meanwhile) {
        auto other = meanwhile;
        meanwhile = nullptr;
        other();
    }
    return cudaSuccess;
}

static int cluster_of(const cudaLaunchConfig_t *c) {
    for (unsigned i = 0; i < c->numAttrs; ++i)
        if (c->attrs[i].id == cudaLaunchAttributeClusterDimension) return static_cast<int>(c->attrs[i].val.clusterDim.x);
    return 1;
}
static bool fits(const void *f, const cudaLaunchConfig_t *c) {
    const Kernel &k = kernels[f];
    const int dynamic = static_cast<int>(c->dynamicSmemBytes);
    // (what is not opted in to is limited together with the kernel's own arrays)
    return dynamic <= k.limit || dynamic + static_bytes <= kDefaultLimit;
}

cudaError_t cudaOccupancyMaxActiveClusters(int *n, const void *f, const cudaLaunchConfig_t *c) {
    if (!fits(f, c)) return end(cudaErrorInvalidValue);
    *n = cluster_of(c) > 8 ? clusters_of_16 : 8;
    return *n < 0 ? end(cudaErrorInvalidClusterSize) : cudaSuccess;
}

cudaError_t cudaLaunchKernelExC(const cudaLaunchConfig_t *c, const void *f, void **) {
    if (!fits(f, c)) return end(cudaErrorInvalidValue);
    if (cluster_of(c) > 8 && (!kernels[f].large_cluster || clusters_of_16 <= 0)) return end(cudaErrorInvalidClusterSize);
    ++launches;
    last_dynamic = static_cast<int>(c->dynamicSmemBytes);
    last_cluster = cluster_of(c);
    return cudaSuccess;
}

}  // extern "C"
