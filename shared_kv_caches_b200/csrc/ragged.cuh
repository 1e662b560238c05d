// Pieces shared by the kernels over ragged batches (tables, expand, prefill):
// sums over the requests and the lookup of the request an index falls in.
#pragma once

#include "kvattn_internal.cuh"
#include "sm100.cuh"

namespace kvattn {
namespace ragged {

constexpr int kThreads = 1024;           // threads of a block that sums over the requests
constexpr int kMaxBatch = 16384;         // requests whose sums fit its shared memory
constexpr int kMaxRows = INT32_MAX - 4096;   // rows of a batch: a tile past the last one still has a 32-bit number

// Exclusive sums over a block of kThreads threads; the total in `sum`.
// sh: 32 values of shared memory.
__device__ __forceinline__ long long block_scan(long long v, long long &sum, long long *sh)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const long long v0 = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long x = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o)
            v += x;
    }
    __syncthreads();                      // sh may still be read by the scan before
    if (lane == 31)
        sh[warp] = v;
    __syncthreads();
    long long w = sh[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long x = __shfl_up_sync(0xffffffffu, w, o);
        if (lane >= o)
            w += x;
    }
    sum = __shfl_sync(0xffffffffu, w, 31);
    const long long before = __shfl_sync(0xffffffffu, w, (warp + 31) & 31);
    return v - v0 + (warp ? before : 0);
}

// The last index i in [0, n) with start[i] <= x (start ascending, start[0] <= x).
__device__ __forceinline__ int find(const int32_t *start, int n, int x)
{
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (start[mid] <= x)
            lo = mid;
        else
            hi = mid;
    }
    return lo;
}

// MMAs and commits issued by one elected lane (always the same one) in code
// that the whole warp runs.  What the descriptors are made of is then the same
// in every lane and stays in uniform registers: issued from a branch that only
// lane 0 takes, every operand is moved there first, and an MMA of 64 cycles
// took 140 to issue (clock trace of an 8K prompt); so, about 70.
__device__ __forceinline__ void elect_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc)
{
    asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\telect.sync _|q, 0xffffffff;\n\t"
                 "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
                 "l"(a), "l"(b), "r"(idesc), "r"(acc)
                 : "memory");
}

__device__ __forceinline__ void elect_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc)
{
    asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\telect.sync _|q, 0xffffffff;\n\t"
                 "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
                 "r"(a), "l"(b), "r"(idesc), "r"(acc)
                 : "memory");
}

__device__ __forceinline__ void elect_commit(uint64_t *bar)
{
    asm volatile("{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\t"
                 "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_u32(bar))
                 : "memory");
}

// One tile of a ragged batch, as the plan kernel lists them.
struct Tile {
    int32_t q0;       // first row of the tile
    int32_t nq;       // rows of the tile
    int32_t k0;       // first key row of the sequence
    int32_t nk;       // keys of the sequence
    int32_t lim0;     // keys that the tile's first row attends, before the clip to [0, nk]
    int32_t seq;      // sequence
    int32_t tok0;     // position of the first row in its sequence's rows
    int32_t pad;
};

constexpr size_t kPlanHeader = 256;      // bytes in front of the tile list: [0] its length, [1] 0 (a count for its reader)

struct PlanArgs {
    int batch, rows_per_tile;
    int max_q, max_kv;
    int capacity;                        // tiles the list has room for
    int causal;
    const int32_t *q_start;              // [batch + 1]
    const int32_t *kv_start;             // [batch + 1]
    int32_t *header;
    Tile *tiles;
    int32_t *err;
};

// Rows and keys of sequence b.  A range that runs backwards or out of the
// arrays is taken as empty (false).
__device__ __forceinline__ bool ranges(const PlanArgs &a, int b, int &q0, int &nq, int &k0, int &nk)
{
    q0 = a.q_start[b];
    const int q1 = a.q_start[b + 1];
    k0 = a.kv_start[b];
    const int k1 = a.kv_start[b + 1];
    const bool ok = q0 >= 0 && q0 <= q1 && q1 <= a.max_q && k0 >= 0 && k0 <= k1 && k1 <= a.max_kv;
    nq = ok ? q1 - q0 : 0;
    nk = ok ? k1 - k0 : 0;
    return ok;
}

// Tile of the rows from `off` on of sequence b.
__device__ __forceinline__ Tile make_tile(const PlanArgs &a, int b, int q0, int nq, int k0, int nk, int off)
{
    Tile t;
    t.q0 = q0 + off;
    t.nq = min(nq - off, a.rows_per_tile);
    t.k0 = k0;
    t.nk = nk;
    t.lim0 = a.causal ? nk - nq + off + 1 : nk;
    t.seq = b;
    t.tok0 = off;
    t.pad = 0;
    return t;
}

// Small batches: their tiles, in the sequences' order, listed by one warp of
// every CTA in its shared memory.  It saves the plan's launch (two 512-token
// prompts of 8 heads: 16.2 -> 14.1 us on the device, the call on the host 9.5 ->
// 5.5).
constexpr int kSmallBatch = 32, kSmallTiles = 16;

inline bool small_plan(int batch, long long capacity) { return batch <= kSmallBatch && capacity <= kSmallTiles; }

// Returns the number of tiles (to every lane).  tiles: room for kSmallTiles.
__device__ __forceinline__ int list_tiles(const PlanArgs &a, Tile *tiles, bool report)
{
    const int lane = threadIdx.x & 31;
    int q0 = 0, nq = 0, k0 = 0, nk = 0;
    const bool ok = lane >= a.batch || ranges(a, lane, q0, nq, k0, nk);
    const int mine = (nq + a.rows_per_tile - 1) / a.rows_per_tile;
    // overlapping ranges can ask for more tiles than there is room for
    int at = min(mine, kSmallTiles + 1);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, at, o);
        if (lane >= o)
            at += x;
    }
    const int total = __shfl_sync(0xffffffffu, at, 31);
    at -= min(mine, kSmallTiles + 1);
    for (int i = 0; i < mine && at + i < a.capacity; ++i)
        tiles[at + i] = make_tile(a, lane, q0, nq, k0, nk, i * a.rows_per_tile);
    const bool bad = __any_sync(0xffffffffu, !ok) || total > a.capacity;
    if (bad && report && lane == 0 && a.err)
        atomicOr(a.err, KVATTN_DEVERR_BAD_LENGTH);
    __syncwarp();
    return min(total, a.capacity);
}

// Most tiles a batch can have: every sequence may end in one of its own.
inline long long tile_capacity(long long rows, int batch, int rows_per_tile)
{
    return (rows + rows_per_tile - 1) / rows_per_tile + batch;
}

cudaError_t launch_plan(const PlanArgs &a, cudaStream_t st);

}  // namespace ragged
}  // namespace kvattn
