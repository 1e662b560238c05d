// Expanded keys and values of cached latents (kvattn_expand_kv).
//
// With c the latent of a cached token (for GLA the one of head h's group),
//   k^C_h = W_UK[h] c      v_h = c W_UV[h]
// for every head: the two products whose weights kvattn_head_proj folds into
// the query and the output for single tokens, here applied to the cache, so
// that a chunk of many new tokens attends keys of 128 + 64 and values of 128
// instead of 576 and 512.  Per (query, key) pair that is 2 (192 + 128) flops a
// head against 2 (576 + 512); expanding a token costs 2 * 512 * 256 a head, so
// the expanded form does less work from about 170 new tokens on.
//
// A GEMM whose A rows are gathered by the block table.  A tile is 128 tokens of
// one sequence (two pages, one TMA box each).  Two CTAs of a cluster work on
// two tiles and two heads: each keeps all of its own tile's latent columns in
// shared memory and streams its own head's weights past them in 64-wide chunks
// of the contraction, first W_UK, then W_UV; tcgen05 MMAs of the pair
// (cta_group::2, 256 x 256 x 16) multiply both tiles with both heads, into one
// of two TMEM accumulators, so that one is stored while the other fills.  With
// latents in place and a head's weights read once for two tiles, an SM reads
// 32 bytes a cycle from L2 while its MMAs run; one CTA on its own needs 64, and
// the 96 KB that it can have in flight are then no more than the latency
// times that (ragged MLA prompts, 22 thousand tokens, calls repeated back to
// back: 818 us; so, 678).  Every cluster takes the same number of (tile pair,
// group, head pair) units, in order, and loads latents only where the tiles or
// the group change.
#include <math.h>

#include "ragged.cuh"

namespace kvattn {

namespace {

bool is_aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

constexpr int kRows = 128;                      // tokens of a tile
constexpr int kThreads = 256;
constexpr int kChunk = 64;                      // contraction elements per stage
constexpr int kBox = kRows * kChunk * 2;        // 16 KB: one chunk of the tile's latents, or of a head's weight
constexpr int kMaxChunks = 8;                   // 512 latent columns
constexpr int kMaxStages = 8;                   // as many 16 KB stages as fit beside the latents
constexpr int kOutBox = 32 * 128;               // 32 rows x 64 columns on their way out, two for each storing warp
constexpr int kOutBytes = 4 * 2 * kOutBox;
constexpr int kSmemMax = 227 * 1024;
constexpr uint32_t kCols = 256;                 // accumulator columns: 128 of each head

// The barriers that the MMAs wait on are the leader's (rank 0): both CTAs' TMA
// loads count on them.  The others are each CTA's own, arrived on by commits
// that go to both.
struct Bars {
    uint64_t a_full[kMaxChunks], a_empty;
    uint64_t b_full[kMaxStages], b_empty[kMaxStages];
    uint64_t d_full[2], d_empty[2];
    uint64_t done;
    uint32_t tmem_base;
    int32_t ntiles;
    ragged::Tile tiles[ragged::kSmallTiles];
};

constexpr int stages_of(int chunks)
{
    const int fit = (kSmemMax - (int)sizeof(Bars) - kOutBytes) / kBox - chunks;
    return fit < kMaxStages ? fit : kMaxStages;
}

// The pair's forms of the tcgen05 instructions (both CTAs allocate and free).
__device__ __forceinline__ void tmem_alloc2(uint32_t *dst, uint32_t ncols)
{
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(dst)), "r"(ncols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}

__device__ __forceinline__ void tmem_dealloc2(uint32_t taddr, uint32_t ncols)
{
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}

__device__ __forceinline__ void elect_ss2(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc)
{
    asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\telect.sync _|q, 0xffffffff;\n\t"
                 "@q tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
                 "l"(a), "l"(b), "r"(idesc), "r"(acc)
                 : "memory");
}

// Arrive on the barrier at this place in both CTAs once the MMAs so far are done.
__device__ __forceinline__ void elect_commit2(uint64_t *bar)
{
    asm volatile("{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\t"
                 "@q tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], "
                 "%1;\n\t}" ::"r"(smem_u32(bar)),
                 "h"((uint16_t)3)
                 : "memory");
}

// TMA loads into this CTA's shared memory that count on a barrier of the
// leader (bar: its shared::cluster address).
__device__ __forceinline__ void pair_load_2d(void *dst, const CUtensorMap *map, int x, int y, uint32_t bar)
{
    asm volatile("cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, "
                 "{%2, %3}], [%4];" ::"r"(smem_u32(dst)),
                 "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar)
                 : "memory");
}

__device__ __forceinline__ void pair_load_3d(void *dst, const CUtensorMap *map, int x, int y, int z, uint32_t bar,
                                             uint64_t policy)
{
    asm volatile("cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint "
                 "[%0], [%1, {%2, %3, %4}], [%5], %6;" ::"r"(smem_u32(dst)),
                 "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar), "l"(policy)
                 : "memory");
}

struct ExpandArgs {
    ragged::PlanArgs plan;
    int listed;                                 // the plan kernel has listed the tiles; else every CTA does
    const int32_t *block_table;                 // nullptr: contiguous
    const __nv_bfloat16 *cache;
    __nv_bfloat16 *k, *v, *k_rope;
    int32_t *err;
    int heads_per_group, groups, branches, pairs_per_group, d_c, d_k, d_v, d_rope, row;
    int mpps, num_pages, max_kv;
};

// Physical page of the sequence's page pi; num_pages (nothing there: the load
// fills zeros) for a bad id.
__device__ __forceinline__ int page_or_none(const ExpandArgs &a, int seq, int pi, bool report)
{
    const long long page = pi >= a.mpps ? -1
                           : a.block_table ? (long long)a.block_table[(long long)seq * a.mpps + pi]
                                           : (long long)seq * a.mpps + pi;
    if (page < 0 || page >= a.num_pages) {
        if (report && a.err)
            atomicOr(a.err, KVATTN_DEVERR_PAGE_OUT_OF_RANGE);
        return a.num_pages;
    }
    return (int)page;
}

// L2 keeps the weights, which every cluster reads again for every tile pair,
// rather than the outputs, which are more than it holds (calls repeated back
// to back: GLA 16K 393 -> 360 us, ragged MLA prompts 701 -> 678).
__device__ __forceinline__ uint64_t keep_policy()
{
    uint64_t p;
    asm volatile("createpolicy.fractional.L2::evict_last.b64 %0, 1.0;" : "=l"(p));
    return p;
}

__device__ __forceinline__ uint64_t pass_policy()
{
    uint64_t p;
    asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(p));
    return p;
}

// TMA store of a box from shared memory, and the groups that such stores are
// waited for in.
__device__ __forceinline__ void tma_store_3d(const CUtensorMap *map, int x, int y, int z, const void *src, uint64_t policy)
{
    asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.bulk_group.L2::cache_hint [%0, {%1, %2, %3}], [%4], %5;" ::"l"(
                     reinterpret_cast<uint64_t>(map)),
                 "r"(x), "r"(y), "r"(z), "r"(smem_u32(src)), "l"(policy)
                 : "memory");
    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}

// All but the last group have been read from shared memory.
__device__ __forceinline__ void tma_store_wait_read1() { asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory"); }
__device__ __forceinline__ void tma_store_wait_all() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }

// The units of this cluster, in order; every role walks them on its own.  While
// there are tile pairs for all clusters, each takes one whole, so that they
// stream the same weights at about the same time (out of L2, where the outputs
// would push weights out between uses far apart); what is left is cut into
// equal runs of units.
struct Walk {
    int unit, whole, end;                        // units done, of whole tile pairs, and in all
    int first;                                   // where the run of what is left starts
    int pairs, groups;
    int tiles, group, pair;
    __device__ __forceinline__ Walk(const ExpandArgs &a, int ntiles)
        : unit(0), pairs(a.pairs_per_group), groups(a.groups), tiles(blockIdx.x / 2), group(0), pair(0)
    {
        const int c = blockIdx.x / 2, n = gridDim.x / 2, all = (ntiles + 1) / 2, each = groups * pairs;
        const int rounds = all / n;
        const long long left = (long long)(all - rounds * n) * each;
        const int from = (int)(left * c / n), to = (int)(left * (c + 1) / n);
        whole = rounds * each;
        end = whole + to - from;
        first = rounds * n * each + from;
        if (rounds == 0)
            start_rest();
    }
    __device__ __forceinline__ void start_rest()
    {
        pair = first % pairs;
        group = first / pairs % groups;
        tiles = first / pairs / groups;
    }
    __device__ __forceinline__ bool more() const { return unit < end; }
    // whether the unit after this one has other latents (or there is none)
    __device__ __forceinline__ bool last_of_latents() const { return pair + 1 == pairs || unit + 1 == end; }
    __device__ __forceinline__ void next()
    {
        if (++unit == whole) {
            start_rest();
        } else if (++pair == pairs) {
            pair = 0;
            if (++group == groups) {
                group = 0;
                tiles += unit < whole ? (int)gridDim.x / 2 : 1;
            }
        }
    }
};

// The tile of CTA `rank` in the walk's tile pair (no rows where the list ends).
__device__ __forceinline__ ragged::Tile pair_tile(const ragged::Tile *tiles, const Walk &w, int ntiles, int rank)
{
    const int i = 2 * w.tiles + rank;
    ragged::Tile t = tiles[min(i, ntiles - 1)];
    if (i >= ntiles)
        t.nq = 0;
    return t;
}

__device__ __forceinline__ int pages_in(const ragged::Tile &t) { return (t.nq + kPage - 1) / kPage; }

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    expand_kernel(const __grid_constant__ CUtensorMap cmap, const __grid_constant__ CUtensorMap kmap,
                  const __grid_constant__ CUtensorMap vmap, const __grid_constant__ CUtensorMap kout,
                  const __grid_constant__ CUtensorMap vout, const ExpandArgs a)
{
    extern __shared__ __align__(1024) unsigned char smem[];
    const int chunks = a.d_c / kChunk, stages = stages_of(chunks);
    unsigned char *const wts = smem + chunks * kBox;
    unsigned char *const outs = wts + stages * kBox;
    Bars &B = *reinterpret_cast<Bars *>(outs + kOutBytes);
    const int rank = (int)cluster_ctarank();
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    if (smem_u32(smem) & 1023u) {
        if (threadIdx.x == 0 && a.err)
            atomicOr(a.err, KVATTN_DEVERR_WAIT_TIMEOUT);
        return;
    }
    if (threadIdx.x == 0) {
        for (int c = 0; c < kMaxChunks; ++c)
            mbar_init(&B.a_full[c], 1);
        mbar_init(&B.a_empty, 1);
        for (int s = 0; s < kMaxStages; ++s) {
            mbar_init(&B.b_full[s], 1);
            mbar_init(&B.b_empty[s], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&B.d_full[i], 1);
            mbar_init(&B.d_empty[i], 8);
        }
        mbar_init(&B.done, 1);
        fence_mbar_init();
    }
    if (warp == 0)
        tmem_alloc2(&B.tmem_base, 512);
    if (warp == 1 && !a.listed) {
        const int n = ragged::list_tiles(a.plan, B.tiles, blockIdx.x == 0);
        if (lane == 0)
            B.ntiles = n;
    }
    tc_fence_before();
    cluster_sync_all();
    tc_fence_after();
    const uint32_t tbase = B.tmem_base;
    if (a.listed)
        pdl_wait_primary();                      // the tile list
    const int ntiles = a.listed ? a.plan.header[0] : B.ntiles;
    const ragged::Tile *const tiles = a.listed ? a.plan.tiles : B.tiles;
    Walk w(a, ntiles);
    bool ok = true;

    if (warp == 0) {
        // ---------------------------------------------------------------- TMA
        if (lane == 0) {
            const uint64_t policy = keep_policy();
            uint32_t nb = 0, na = 0;             // weight chunks, latent tiles loaded
            bool fresh = true;
            for (; ok && w.more(); w.next()) {
                if (fresh) {
                    if (na > 0 && !mbar_wait(&B.a_empty, (na - 1) & 1)) {
                        ok = false;
                        break;
                    }
                    ++na;
                    const ragged::Tile t = pair_tile(tiles, w, ntiles, rank);
                    const int subs = pages_in(t), both = subs + pages_in(pair_tile(tiles, w, ntiles, rank ^ 1));
                    int y[2] = {0, 0};
                    for (int s = 0; s < subs; ++s)
                        y[s] = page_or_none(a, t.seq, t.tok0 / kPage + s, w.group == 0) * kPage;
                    for (int c = 0; c < chunks; ++c) {
                        const uint32_t bar = mapa_shared(smem_u32(&B.a_full[c]), 0);
                        if (rank == 0)
                            mbar_arrive_expect_tx(&B.a_full[c], (uint32_t)(both * (kBox / 2)));
                        for (int s = 0; s < subs; ++s)
                            pair_load_2d(smem + c * kBox + s * (kBox / 2), &cmap, w.group * a.d_c + c * kChunk, y[s], bar);
                    }
                }
                fresh = w.last_of_latents();
                // MLRA: the branch's columns of every head's weight; else the group's heads
                const int h = (a.branches > 1 ? 0 : w.group * a.heads_per_group) + 2 * w.pair + rank;
                const int c0 = a.branches > 1 ? w.group * a.d_c : 0;
                for (int kind = 0; ok && kind < 2; ++kind)
                    for (int c = 0; c < chunks; ++c, ++nb) {
                        const uint32_t st = nb % stages;
                        if (nb >= (uint32_t)stages && !mbar_wait(&B.b_empty[st], (nb / stages - 1) & 1)) {
                            ok = false;
                            break;
                        }
                        unsigned char *dst = wts + st * kBox;
                        const uint32_t bar = mapa_shared(smem_u32(&B.b_full[st]), 0);
                        if (rank == 0)
                            mbar_arrive_expect_tx(&B.b_full[st], 2 * kBox);
                        if (kind == 0) {
                            pair_load_3d(dst, &kmap, c0 + c * kChunk, 0, h, bar, policy);
                        } else {
                            pair_load_3d(dst, &vmap, 0, c0 + c * kChunk, h, bar, policy);
                            pair_load_3d(dst + kBox / 2, &vmap, 64, c0 + c * kChunk, h, bar, policy);
                        }
                    }
            }
            // every copy that counts on the leader's barriers has landed before
            // it comes to the cluster's last barrier, and so before either exits
            if (rank == 0) {
                for (uint32_t s = 0; s < (uint32_t)stages; ++s)
                    if (nb > s && !mbar_wait(&B.b_full[s], ((nb - 1 - s) / stages) & 1))
                        ok = false;
                for (int c = 0; c < chunks; ++c)
                    if (na > 0 && !mbar_wait(&B.a_full[c], (na - 1) & 1))
                        ok = false;
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        // ------------------------------------------------- MMA (of the leader)
        const uint64_t cdesc = smem_desc(smem_u32(smem), 16, 1024, 2);            // K-major latents
        const uint64_t kdesc = smem_desc(smem_u32(wts), 16, 1024, 2);             // K-major rows of W_UK
        const uint64_t vdesc = smem_desc(smem_u32(wts), kBox / 2, 1024, 2);       // N-major rows of W_UV
        uint32_t nb = 0, na = 0, nd = 0;                 // weight chunks, latent tiles, accumulators
        bool fresh = true;
        for (; ok && rank == 0 && w.more(); w.next()) {
            na += fresh;
            const bool last = w.last_of_latents();
#pragma unroll 1
            for (int kind = 0; ok && kind < 2; ++kind, ++nd) {
                const uint32_t buf = nd & 1, d = tbase + buf * kCols;
                bool in = nd < 2 || mbar_wait_cluster(&B.d_empty[buf], ((nd >> 1) - 1) & 1);
                const uint32_t idesc = idesc_bf16_f32(2 * kRows, kCols, false, false) | (kind ? 1u << 16 : 0u);   // N-major W_UV
                const uint64_t step = kind ? 128 : 2;    // sixteen rows of W_UV, sixteen columns of W_UK
#pragma unroll 1
                for (int c = 0; c < chunks; ++c, ++nb) {
                    const uint32_t st = nb % stages;
                    if (fresh && kind == 0)
                        in = in && mbar_wait(&B.a_full[c], (na - 1) & 1);
                    in = in && mbar_wait(&B.b_full[st], (nb / stages) & 1);
                    ok = __all_sync(0xffffffffu, in);
                    if (!ok)
                        break;
                    tc_fence_after();
                    const uint64_t ad = cdesc + (uint64_t)(c * (kBox >> 4));
                    const uint64_t bd = (kind ? vdesc : kdesc) + (uint64_t)(st * (kBox >> 4));
#pragma unroll
                    for (int i = 0; i < kChunk / 16; ++i)
                        elect_ss2(d, ad + i * 2, bd + i * step, idesc, (c | i) ? 1u : 0u);
                    elect_commit2(&B.b_empty[st]);
                }
                if (ok)
                    elect_commit2(&B.d_full[buf]);
            }
            if (ok && last)
                elect_commit2(&B.a_empty);
            fresh = last;
        }
        // every MMA has completed, and every commit has arrived, before either
        // CTA frees its TMEM and exits
        if (rank == 0)
            elect_commit2(&B.done);
        ok = __all_sync(0xffffffffu, mbar_wait(&B.done, 0)) && ok;
    } else if (warp == 2) {
        // the shared rope keys of a tile's tokens, copied once, with its first unit
        const int vecs = a.d_rope / 8;
        for (; w.more(); w.next()) {
            if (w.group || w.pair || !vecs)
                continue;
            const ragged::Tile t = pair_tile(tiles, w, ntiles, rank);
            for (int i = lane; i < t.nq * vecs; i += 32) {
                const int r = i / vecs, p = i % vecs;
                const int page = page_or_none(a, t.seq, (t.tok0 + r) / kPage, false);
                uint4 x = make_uint4(0, 0, 0, 0);
                if (page < a.num_pages)
                    x = *reinterpret_cast<const uint4 *>(
                        a.cache + ((long long)page * kPage + (t.tok0 + r) % kPage) * a.row + a.groups * a.d_c + 8 * p);
                *reinterpret_cast<uint4 *>(a.k_rope + (long long)(t.q0 + r) * a.d_rope + 8 * p) = x;
            }
        }
    } else if (warp >= 4) {
        // ----------------------------------------------- accumulators to memory
        // A warp stores its 32 rows in boxes of 64 columns by TMA, through
        // shared memory; where the sequence ends inside them, row by row (the
        // rows behind are the next sequence's).
        const uint32_t lane_addr = (uint32_t)((warp & 3) * 32) << 16;
        const int r0 = (warp & 3) * 32 + lane;           // row of the tile
        unsigned char *const out_box = outs + (warp & 3) * 2 * kOutBox;
        const uint64_t policy = pass_policy();
        uint32_t nd = 0, no = 0;
        for (; ok && w.more(); w.next()) {
            const ragged::Tile t = pair_tile(tiles, w, ntiles, rank);
            const int q0 = t.q0, nq = t.nq;
            const bool whole = (warp & 3) * 32 + 32 <= nq;
            const int heads = min(2, a.heads_per_group - 2 * w.pair);
            // output block of head p of the pair: h0 + p * step
            const int step = a.branches;
            const int h0 = step > 1 ? 2 * w.pair * step + w.group : w.group * a.heads_per_group + 2 * w.pair;
#pragma unroll 1
            for (int kind = 0; kind < 2; ++kind, ++nd) {
                const uint32_t buf = nd & 1;
                ok = __all_sync(0xffffffffu, mbar_wait(&B.d_full[buf], (nd >> 1) & 1));
                if (!ok)
                    break;
                tc_fence_after();
                const int width = kind ? a.d_v : a.d_k;
                __nv_bfloat16 *const rows = (kind ? a.v : a.k) + ((long long)h0 * a.max_kv + q0 + r0) * width;
#pragma unroll 1
                for (int c = 0; c < 256; c += 64) {
                    uint32_t r[64];
                    tmem_ld64(tbase + buf * kCols + lane_addr + c, r);
                    if (c == 192) {
                        // the accumulator is in registers: the MMAs may have it
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0)
                            mbar_arrive_cluster(mapa_shared(smem_u32(&B.d_empty[buf]), 0));
                    }
                    if ((c >> 7) >= heads || (c & 64) >= width)
                        continue;
                    uint4 v[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        uint32_t pk[4];
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const __nv_bfloat162 x = __floats2bfloat162_rn(__uint_as_float(r[8 * i + 2 * j]),
                                                                           __uint_as_float(r[8 * i + 2 * j + 1]));
                            pk[j] = *reinterpret_cast<const uint32_t *>(&x);
                        }
                        v[i] = make_uint4(pk[0], pk[1], pk[2], pk[3]);
                    }
                    if (whole) {
                        unsigned char *const box = out_box + (no++ & 1) * kOutBox;
                        if (lane == 0)
                            tma_store_wait_read1();      // the box before last has been read
                        __syncwarp();
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            *reinterpret_cast<uint4 *>(box + lane * 128 + ((i ^ (lane & 7)) << 4)) = v[i];
                        fence_proxy_async_smem();
                        __syncwarp();
                        if (lane == 0)
                            tma_store_3d(kind ? &vout : &kout, c & 64, q0 + (warp & 3) * 32, h0 + (c >> 7) * step, box,
                                         policy);
                    } else if (r0 < nq) {
                        __nv_bfloat16 *const out = rows + (long long)((c >> 7) * step) * a.max_kv * width + (c & 64);
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            if ((c & 64) + 8 * i < width)
                                *reinterpret_cast<uint4 *>(out + 8 * i) = v[i];
                    }
                    __syncwarp();
                }
            }
        }
        if (lane == 0)
            tma_store_wait_all();
        __syncwarp();
    }
    if (!ok && lane == 0 && a.err)
        atomicOr(a.err, KVATTN_DEVERR_WAIT_TIMEOUT);
    __syncwarp();
    tc_fence_before();
    cluster_sync_all();
    tc_fence_after();
    if (warp == 0)
        tmem_dealloc2(tbase, 512);
}

}  // namespace
}  // namespace kvattn

using namespace kvattn;

extern "C" int kvattn_expand_workspace_size(int32_t variant, const kvattn_params *p, int32_t max_kv_tokens,
                                            size_t *bytes)
{
    Problem pr;
    const int st = validate_params(variant, p, &pr);
    if (st)
        return st;
    if (!bytes || max_kv_tokens < 0)
        return KVATTN_ERR_INVALID_ARG;
    if (!pr.latent || max_kv_tokens > ragged::kMaxRows)
        return KVATTN_ERR_UNSUPPORTED;
    const long long cap = ragged::tile_capacity(max_kv_tokens, p->batch, kRows);
    *bytes = ragged::small_plan(p->batch, cap) ? 0 : ragged::kPlanHeader + (size_t)cap * sizeof(ragged::Tile);
    return KVATTN_OK;
}

extern "C" int kvattn_expand_kv(int32_t variant, const kvattn_params *p, const void *kv_cache,
                                const int32_t *block_table, const int32_t *kv_start, int32_t max_kv_tokens,
                                int32_t d_k, int32_t d_v, const void *w_uk, const void *w_uv, void *k_nope, void *v,
                                void *k_rope, void *workspace, size_t workspace_bytes, int32_t *device_error,
                                void *stream)
{
    size_t need = 0;
    const int st = kvattn_expand_workspace_size(variant, p, max_kv_tokens, &need);
    if (st)
        return st;
    Problem pr;
    validate_params(variant, p, &pr);
    if (!kv_cache || !kv_start || !w_uk || !w_uv || !k_nope || !v || (need && !workspace) || (pr.dr > 0 && !k_rope) ||
        d_k < 1 || d_v < 1)
        return KVATTN_ERR_INVALID_ARG;
    if (d_k % 8 || d_v % 8 || d_k > 128 || d_v > 128 || pr.dn % 64 || p->batch > ragged::kMaxBatch ||
        pr.num_pages > INT32_MAX / kPage - 1)
        return KVATTN_ERR_UNSUPPORTED;
    if (!is_aligned(kv_cache, 16) || !is_aligned(w_uk, 16) || !is_aligned(w_uv, 16) || !is_aligned(k_nope, 16) ||
        !is_aligned(v, 16) || !is_aligned(k_rope, 16) || !is_aligned(workspace, 256) || !is_aligned(block_table, 4) ||
        !is_aligned(kv_start, 4) || !is_aligned(device_error, 4))
        return KVATTN_ERR_MISALIGNED;
    if (workspace_bytes < need)
        return KVATTN_ERR_WORKSPACE_TOO_SMALL;
    const long long cap = ragged::tile_capacity(max_kv_tokens, p->batch, kRows);
    const int pairs = (pr.HPU + 1) / 2;
    if (cap * pr.NU * pairs > INT32_MAX)
        return KVATTN_ERR_UNSUPPORTED;
    if (max_kv_tokens == 0)
        return KVATTN_OK;
    const auto bf16 = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    const auto swz = CU_TENSOR_MAP_SWIZZLE_128B;
    CUtensorMap cm, km, vm, ko, vo;
    // latent columns that a head's weights have, and blocks of keys and values there are
    const cuuint64_t cols = (cuuint64_t)(pr.mlra ? pr.NU : 1) * pr.dn, blocks = (cuuint64_t)pr.HU;
    {
        const cuuint64_t dims[2] = {(cuuint64_t)pr.row, (cuuint64_t)pr.num_pages * kPage};
        const cuuint64_t strides[1] = {(cuuint64_t)pr.row * 2};
        const cuuint32_t box[2] = {kChunk, kPage};
        if (encode_tiled(&cm, bf16, 2, const_cast<void *>(kv_cache), dims, strides, box, swz) != CUDA_SUCCESS)
            return KVATTN_ERR_UNSUPPORTED;
    }
    {
        const cuuint64_t dims[3] = {cols, (cuuint64_t)d_k, (cuuint64_t)pr.H};
        const cuuint64_t strides[2] = {cols * 2, cols * d_k * 2};
        const cuuint32_t box[3] = {kChunk, 128, 1};
        if (encode_tiled(&km, bf16, 3, const_cast<void *>(w_uk), dims, strides, box, swz) != CUDA_SUCCESS)
            return KVATTN_ERR_UNSUPPORTED;
    }
    {
        const cuuint64_t dims[3] = {(cuuint64_t)d_v, cols, (cuuint64_t)pr.H};
        const cuuint64_t strides[2] = {(cuuint64_t)d_v * 2, cols * d_v * 2};
        const cuuint32_t box[3] = {64, kChunk, 1};
        if (encode_tiled(&vm, bf16, 3, const_cast<void *>(w_uv), dims, strides, box, swz) != CUDA_SUCCESS)
            return KVATTN_ERR_UNSUPPORTED;
    }
    for (int i = 0; i < 2; ++i) {
        const cuuint64_t width = (cuuint64_t)(i ? d_v : d_k);
        const cuuint64_t dims[3] = {width, (cuuint64_t)max_kv_tokens, blocks};
        const cuuint64_t strides[2] = {width * 2, (cuuint64_t)max_kv_tokens * width * 2};
        const cuuint32_t box[3] = {64, 32, 1};
        if (encode_tiled(i ? &vo : &ko, bf16, 3, i ? v : k_nope, dims, strides, box, swz) != CUDA_SUCCESS)
            return KVATTN_ERR_UNSUPPORTED;
    }
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    char *ws = static_cast<char *>(workspace);
    ragged::PlanArgs pa{};
    pa.batch = p->batch;
    pa.rows_per_tile = kRows;
    pa.max_q = pa.max_kv = max_kv_tokens;
    pa.capacity = (int)cap;
    pa.q_start = pa.kv_start = kv_start;
    pa.header = reinterpret_cast<int32_t *>(ws);
    pa.tiles = reinterpret_cast<ragged::Tile *>(ws + ragged::kPlanHeader);
    pa.err = device_error;
    const bool listed = !ragged::small_plan(pa.batch, cap);
    cudaError_t e = listed ? ragged::launch_plan(pa, s) : cudaSuccess;
    if (e != cudaSuccess)
        return launch_status(e);
    ExpandArgs a{};
    a.plan = pa;
    a.listed = listed;
    a.block_table = block_table;
    a.cache = static_cast<const __nv_bfloat16 *>(kv_cache);
    a.k = static_cast<__nv_bfloat16 *>(k_nope);
    a.v = static_cast<__nv_bfloat16 *>(v);
    a.k_rope = static_cast<__nv_bfloat16 *>(k_rope);
    a.err = device_error;
    a.heads_per_group = pr.HPU;
    a.groups = pr.NU;
    a.branches = pr.mlra ? pr.NU : 1;
    a.pairs_per_group = pairs;
    a.d_c = pr.dn;
    a.d_k = d_k;
    a.d_v = d_v;
    a.d_rope = pr.dr;
    a.row = pr.row;
    a.mpps = pr.mpps;
    a.num_pages = pr.num_pages;
    a.max_kv = max_kv_tokens;
    const int chunks = pr.dn / kChunk;
    const size_t smem = (size_t)(chunks + stages_of(chunks)) * kBox + kOutBytes + sizeof(Bars);
    // the opt-in is the kernel's, not the call's: the same for every width, so
    // that no call lowers it under another one's launch
    e = cudaFuncSetAttribute(expand_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemMax);
    if (e != cudaSuccess)
        return launch_status(e);
    const long long units = (cap + 1) / 2 * pr.NU * pairs, most = sm_count() / 2;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)(2 * (units < most ? units : most)));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = listed ? 1 : 0;
    return launch_status(cudaLaunchKernelEx(&cfg, expand_kernel, cm, km, vm, ko, vo, (const ExpandArgs)a));
}
