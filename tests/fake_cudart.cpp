// A stand-in for the CUDA runtime on machines without a GPU: the library's
// objects linked against it make their calls as ever, and nothing runs.  It
// keeps what the launch tests ask about (each kernel's shared-memory opt-in,
// each launch) and refuses a launch that asks for more than the device or its
// opt-in gives, as the runtime does.
#include <cuda.h>
#include <cuda_runtime.h>

#include <map>
#include <string>

namespace {

constexpr int kDefaultShared = 48 * 1024, kMostShared = 227 * 1024;

struct Kernel {
    std::string name;
    int opt_in = -1;                   // bytes, once it has been set
    int fixed = 0;                     // declared shared memory, told by the test
};

std::map<const void *, Kernel> kernels;
std::string lines;
std::string fail_call;                 // name of the call that fails
int fail_times = 0;
cudaError_t last = cudaSuccess;
int registers = 168;

dim3 pushed_grid, pushed_block;
size_t pushed_shared;

bool fails(const char *call)
{
    if (fail_times > 0 && fail_call == call) {
        --fail_times;
        last = cudaErrorUnknown;
        return true;
    }
    return false;
}

cudaError_t launched(const void *f, dim3 grid, dim3 block, size_t shared, unsigned cluster)
{
    Kernel &k = kernels[f];
    const bool fits = (int)shared <= (k.opt_in < 0 ? kDefaultShared - k.fixed : k.opt_in);
    lines += "launch " + k.name + " " + std::to_string(grid.x) + " " + std::to_string(block.x) + " " +
             std::to_string(shared) + " " + std::to_string(cluster) + (fits ? " ok\n" : " refused\n");
    if (fits && !fails("launch"))
        return cudaSuccess;
    return last = cudaErrorInvalidValue;
}

CUresult encode(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *, const cuuint64_t *,
                const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle, CUtensorMapL2promotion,
                CUtensorMapFloatOOBfill)
{
    return CUDA_SUCCESS;
}

}  // namespace

extern "C" {

// ---- what the tests call
const char *fake_lines() { return lines.c_str(); }
void fake_clear() { lines.clear(); }
void fake_fail(const char *call, int times)
{
    fail_call = call;
    fail_times = times;
}
void fake_last_error(int e) { last = (cudaError_t)e; }
int fake_peek() { return last; }
void fake_fixed(const char *name, int bytes)
{
    for (auto &k : kernels)
        if (k.second.name.find(name) != std::string::npos)
            k.second.fixed = bytes;
}

// ---- what the compiler's stubs call
void **__cudaRegisterFatBinary(void *)
{
    static void *handle;
    return &handle;
}
void __cudaRegisterFatBinaryEnd(void **) {}
void __cudaUnregisterFatBinary(void **) {}
void __cudaRegisterFunction(void **, const char *host, char *, const char *name, int, uint3 *, uint3 *, dim3 *, dim3 *, int *)
{
    kernels[host].name = name;
}
void __cudaRegisterVar(void **, char *, char *, const char *, int, size_t, int, int) {}
unsigned __cudaPushCallConfiguration(dim3 grid, dim3 block, size_t shared, cudaStream_t)
{
    pushed_grid = grid;
    pushed_block = block;
    pushed_shared = shared;
    return 0;
}
cudaError_t __cudaPopCallConfiguration(dim3 *grid, dim3 *block, size_t *shared, void *stream)
{
    *grid = pushed_grid;
    *block = pushed_block;
    *shared = pushed_shared;
    *static_cast<cudaStream_t *>(stream) = nullptr;
    return cudaSuccess;
}

// ---- the runtime
cudaError_t cudaFuncSetAttribute(const void *f, cudaFuncAttribute attr, int value)
{
    Kernel &k = kernels[f];
    if (fails("cudaFuncSetAttribute"))
        return cudaErrorUnknown;
    if (attr != cudaFuncAttributeMaxDynamicSharedMemorySize || value < 0 || value + k.fixed > kMostShared)
        return last = cudaErrorInvalidValue;
    k.opt_in = value;
    lines += "opt_in " + k.name + " " + std::to_string(value) + "\n";
    return cudaSuccess;
}
cudaError_t cudaFuncGetAttributes(cudaFuncAttributes *at, const void *)
{
    if (fails("cudaFuncGetAttributes"))
        return cudaErrorUnknown;
    *at = cudaFuncAttributes{};
    at->numRegs = registers;
    return cudaSuccess;
}
cudaError_t cudaLaunchKernel(const void *f, dim3 grid, dim3 block, void **, size_t shared, cudaStream_t)
{
    return launched(f, grid, block, shared, 1);
}
cudaError_t cudaLaunchKernelExC(const cudaLaunchConfig_t *c, const void *f, void **)
{
    unsigned cluster = 1;
    for (unsigned i = 0; i < c->numAttrs; ++i)
        if (c->attrs[i].id == cudaLaunchAttributeClusterDimension)
            cluster = c->attrs[i].val.clusterDim.x;
    return launched(f, c->gridDim, c->blockDim, c->dynamicSmemBytes, cluster);
}
cudaError_t cudaGetLastError()
{
    const cudaError_t e = last;
    last = cudaSuccess;
    return e;
}
cudaError_t cudaGetDevice(int *dev)
{
    *dev = 0;
    return cudaSuccess;
}
cudaError_t cudaDeviceGetAttribute(int *value, cudaDeviceAttr, int)
{
    *value = 148;
    return cudaSuccess;
}
cudaError_t cudaGetDriverEntryPoint(const char *, void **fn, unsigned long long, cudaDriverEntryPointQueryResult *q)
{
    if (fails("cudaGetDriverEntryPoint"))
        return cudaErrorUnknown;
    *fn = reinterpret_cast<void *>(encode);
    if (q)
        *q = cudaDriverEntryPointSuccess;
    return cudaSuccess;
}
cudaError_t cudaEventRecord(cudaEvent_t, cudaStream_t) { return cudaSuccess; }
cudaError_t cudaMemcpyAsync(void *, const void *, size_t, cudaMemcpyKind, cudaStream_t) { return cudaSuccess; }
cudaError_t cudaMemsetAsync(void *, int, size_t, cudaStream_t) { return cudaSuccess; }
cudaError_t cudaStreamSynchronize(cudaStream_t) { return cudaSuccess; }
cudaError_t cudaGetSymbolAddress(void **p, const void *)
{
    *p = reinterpret_cast<void *>((size_t)1 << 20);
    return cudaSuccess;
}

}
