// The tile list of a ragged batch: the rows of every sequence cut into tiles
// of a fixed size, the tiles with the most keys first.
//
// One block sums the sequences' tile counts, then every thread finds the
// sequence of its tiles by bisection.  The order is a counting sort over the
// number of 128-key steps (at most 1024 classes, longest first), so that the
// work handed out last is the shortest.  The order inside a class depends on
// the atomics; no result does, since every row belongs to one tile.
#include "ragged.cuh"

namespace kvattn {
namespace ragged {

namespace {

constexpr int kClasses = 1024;

__global__ void __launch_bounds__(kThreads, 1) plan_kernel(const PlanArgs a)
{
    extern __shared__ int32_t start[];          // [batch + 1] first tile of each sequence
    __shared__ long long sh_scan[32];
    __shared__ int count[kClasses];
    const int tid = threadIdx.x;
    pdl_launch_dependents();
    const int per = (a.batch + kThreads - 1) / kThreads;
    const int b0 = min(tid * per, a.batch), b1 = min(b0 + per, a.batch);
    count[tid] = 0;
    static_assert(kClasses == kThreads, "one class a thread");
    long long tiles = 0, total;
    bool bad = false;
    for (int b = b0; b < b1; ++b) {
        int q0, nq, k0, nk;
        bad |= !ranges(a, b, q0, nq, k0, nk);
        tiles += (nq + a.rows_per_tile - 1) / a.rows_per_tile;
    }
    long long at = block_scan(tiles, total, sh_scan);
    for (int b = b0; b < b1; ++b) {
        int q0, nq, k0, nk;
        ranges(a, b, q0, nq, k0, nk);
        start[b] = (int)min(at, (long long)a.capacity);
        at += (nq + a.rows_per_tile - 1) / a.rows_per_tile;
    }
    // overlapping ranges can ask for more tiles than the list holds
    const int n = (int)min(total, (long long)a.capacity);
    if ((bad || total > n) && a.err)
        atomicOr(a.err, KVATTN_DEVERR_BAD_LENGTH);
    if (tid == 0) {
        start[a.batch] = n;
        a.header[0] = n;
        a.header[1] = 0;
    }
    __syncthreads();

    int shift = 0;
    while (((a.max_kv / 128 + 1) >> shift) >= kClasses)
        ++shift;
    auto tile_of = [&](int i, Tile &t) -> int {
        const int b = find(start, a.batch, i);
        int q0, nq, k0, nk;
        ranges(a, b, q0, nq, k0, nk);
        t = make_tile(a, b, q0, nq, k0, nk, (i - start[b]) * a.rows_per_tile);
        const int last = a.causal ? min(nk, max(t.lim0 + t.nq - 1, 0)) : nk;
        return kClasses - 1 - (((last + 127) / 128) >> shift);
    };
    for (int i = tid; i < n; i += kThreads) {
        Tile t;
        atomicAdd(&count[tile_of(i, t)], 1);
    }
    __syncthreads();
    long long unused;
    const long long first = block_scan(count[tid], unused, sh_scan);
    __syncthreads();
    count[tid] = (int)first;
    __syncthreads();
    for (int i = tid; i < n; i += kThreads) {
        Tile t;
        const int c = tile_of(i, t);
        a.tiles[atomicAdd(&count[c], 1)] = t;
    }
}

}  // namespace

cudaError_t launch_plan(const PlanArgs &a, cudaStream_t st)
{
    const size_t smem = (size_t)(a.batch + 1) * sizeof(int32_t);
    if (smem > 40 * 1024) {
        // for the largest batch: the opt-in is the kernel's, and calls at the
        // same time share it
        const cudaError_t e = cudaFuncSetAttribute(plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   (int)((kMaxBatch + 1) * sizeof(int32_t)));
        if (e != cudaSuccess)
            return e;
    }
    // (launched so that the status is this launch's, not an earlier call's)
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(1);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    return cudaLaunchKernelEx(&cfg, plan_kernel, a);
}

}  // namespace ragged
}  // namespace kvattn
