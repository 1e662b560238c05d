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
// A GEMM whose A rows are gathered by the block table: a tile is 128 tokens of
// one sequence (two pages, one TMA box each), staged with the head's weights in
// 64-wide chunks of the contraction; tcgen05 MMAs (M = 128, N = 128, K = 16)
// accumulate keys and values side by side in TMEM.
#include <math.h>

#include "ragged.cuh"

namespace kvattn {

namespace {

bool is_aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

constexpr int kRows = 128;                      // tokens of a tile
constexpr int kThreads = 128;
constexpr int kChunk = 64;                      // contraction elements per stage
constexpr int kBox = kRows * kChunk * 2;        // 16 KB: the tile's latents, W_UK or W_UV of one chunk
constexpr int kStage = 3 * kBox;
constexpr int kStages = 2;                      // 96 KB a CTA: two on an SM, one storing while the other multiplies
constexpr uint32_t kCols = 256;                 // TMEM: 128 key and 128 value columns
constexpr size_t kSmem = (size_t)kStages * kStage + 64;

struct ExpandArgs {
    const int32_t *header;
    const ragged::Tile *tiles;
    const int32_t *block_table;                 // nullptr: contiguous
    const __nv_bfloat16 *cache;
    __nv_bfloat16 *k, *v, *k_rope;
    int32_t *err;
    int heads, heads_per_group, groups, d_c, d_k, d_v, d_rope, row;
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

__global__ void __launch_bounds__(kThreads)
    expand_kernel(const __grid_constant__ CUtensorMap cmap, const __grid_constant__ CUtensorMap kmap,
                  const __grid_constant__ CUtensorMap vmap, const ExpandArgs a)
{
    extern __shared__ __align__(1024) unsigned char smem[];
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + kStages * kStage);
    uint64_t *empty = full + kStages;
    uint64_t *done = empty + kStages;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(done + 1);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (smem_u32(smem) & 1023u) {
        if (threadIdx.x == 0 && a.err)
            atomicOr(a.err, KVATTN_DEVERR_WAIT_TIMEOUT);
        return;
    }
    pdl_wait_primary();
    if ((int)blockIdx.y >= a.header[0])
        return;
    const ragged::Tile t = a.tiles[blockIdx.y];
    const int h = blockIdx.x, group = h / a.heads_per_group;
    const int chunks = a.d_c / kChunk;
    const int subs = t.nq > kPage ? 2 : 1;       // pages that hold rows of the tile
    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        mbar_init(done, 1);
        fence_mbar_init();
    }
    if (warp == 0)
        tmem_alloc(tmem_slot, kCols);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tacc = *tmem_slot;
    bool ok = true;

    if (warp == 0) {
        if (lane == 0) {
            int y[2] = {0, 0};
            for (int s = 0; s < subs; ++s)
                y[s] = page_or_none(a, t.seq, t.tok0 / kPage + s, h == 0) * kPage;
            int issued = 0;
            for (int c = 0; c < chunks; ++c) {
                const int st = c % kStages;
                if (c >= kStages && !mbar_wait(&empty[st], ((c / kStages) - 1) & 1)) {
                    ok = false;
                    break;
                }
                unsigned char *base = smem + st * kStage;
                mbar_arrive_expect_tx(&full[st], (uint32_t)(subs * (kBox / 2) + 2 * kBox));
                for (int s = 0; s < subs; ++s)
                    tma_load_2d(base + s * (kBox / 2), &cmap, group * a.d_c + c * kChunk, y[s], &full[st]);
                tma_load_3d(base + kBox, &kmap, c * kChunk, 0, h, &full[st]);
                tma_load_3d(base + 2 * kBox, &vmap, 0, c * kChunk, h, &full[st]);
                tma_load_3d(base + 2 * kBox + kBox / 2, &vmap, 64, c * kChunk, h, &full[st]);
                issued = c + 1;
            }
            // every copy started here has landed before the CTA can exit
            for (int st = 0; st < kStages && st < issued; ++st) {
                const int cl = st + ((issued - 1 - st) / kStages) * kStages;
                if (!mbar_wait(&full[st], (cl / kStages) & 1))
                    ok = false;
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        constexpr uint32_t kidesc = idesc_bf16_f32(kRows, 128, false, false);
        constexpr uint32_t videsc = idesc_bf16_f32(kRows, 128, false, true);
        const uint64_t cdesc = smem_desc(smem_u32(smem), 16, 1024, 2);                    // K-major latents
        const uint64_t kdesc = smem_desc(smem_u32(smem) + kBox, 16, 1024, 2);             // K-major rows of W_UK
        const uint64_t vdesc = smem_desc(smem_u32(smem) + 2 * kBox, kBox / 2, 1024, 2);   // N-major rows of W_UV
        for (int c = 0; c < chunks; ++c) {
            const int st = c % kStages;
            if (!__all_sync(0xffffffffu, mbar_wait(&full[st], (c / kStages) & 1))) {
                ok = false;
                break;
            }
            tc_fence_after();
            if (lane == 0) {
                const uint64_t o = (uint64_t)(st * (kStage >> 4));
#pragma unroll
                for (int i = 0; i < kChunk / 16; ++i) {
                    umma_ss(tacc, cdesc + o + i * 2, kdesc + o + i * 2, kidesc, (c | i) ? 1u : 0u);
                    umma_ss(tacc + 128, cdesc + o + i * 2, vdesc + o + i * 128, videsc, (c | i) ? 1u : 0u);
                }
                umma_commit(&empty[st]);
            }
            __syncwarp();
        }
        if (lane == 0)
            umma_commit(done);
        __syncwarp();
    } else if (h == 0) {
        // the shared rope keys of the tile's tokens, copied once
        const int vecs = a.d_rope / 8;
        for (int i = threadIdx.x - 64; i < t.nq * vecs; i += 64) {
            const int r = i / vecs, p = i % vecs;
            const int page = page_or_none(a, t.seq, (t.tok0 + r) / kPage, false);
            uint4 x = make_uint4(0, 0, 0, 0);
            if (page < a.num_pages)
                x = *reinterpret_cast<const uint4 *>(a.cache + ((long long)page * kPage + (t.tok0 + r) % kPage) * a.row +
                                                     a.groups * a.d_c + 8 * p);
            *reinterpret_cast<uint4 *>(a.k_rope + (long long)(t.q0 + r) * a.d_rope + 8 * p) = x;
        }
    }

    // thread r of the CTA stores row r of the tile
    const bool have = __all_sync(0xffffffffu, mbar_wait(done, 0));
    tc_fence_after();
    const int r0 = threadIdx.x;
    const uint32_t lane_addr = (uint32_t)(warp * 32) << 16;
#pragma unroll 1
    for (int half = 0; half < 2; ++half) {
        const int width = half ? a.d_v : a.d_k;
        __nv_bfloat16 *out = (half ? a.v : a.k) + ((long long)h * a.max_kv + t.q0 + r0) * width;
#pragma unroll 1
        for (int c = 0; c < 128; c += 32) {
            if (c >= width)
                break;
            uint32_t r[32];
            if (have)
                tmem_ld32(tacc + lane_addr + 128 * half + c, r);
            if (r0 < t.nq && have) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    uint32_t pk[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const __nv_bfloat162 v = __floats2bfloat162_rn(__uint_as_float(r[8 * i + 2 * j]),
                                                                       __uint_as_float(r[8 * i + 2 * j + 1]));
                        pk[j] = *reinterpret_cast<const uint32_t *>(&v);
                    }
                    if (c + 8 * i < width)
                        *reinterpret_cast<uint4 *>(out + c + 8 * i) = make_uint4(pk[0], pk[1], pk[2], pk[3]);
                }
            }
        }
    }
    if ((!ok || !have) && lane == 0 && a.err)
        atomicOr(a.err, KVATTN_DEVERR_WAIT_TIMEOUT);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 0)
        tmem_dealloc(tacc, kCols);
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
    if (variant != KVATTN_MLA && variant != KVATTN_GLA)
        return KVATTN_ERR_UNSUPPORTED;
    *bytes = ragged::kPlanHeader +
             (size_t)ragged::tile_capacity(max_kv_tokens, p->batch, kRows) * sizeof(ragged::Tile);
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
    if (!kv_cache || !kv_start || !w_uk || !w_uv || !k_nope || !v || !workspace || (pr.dr > 0 && !k_rope) ||
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
    if (cap > 65535)
        return KVATTN_ERR_UNSUPPORTED;
    if (max_kv_tokens == 0)
        return KVATTN_OK;
    const auto bf16 = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    const auto swz = CU_TENSOR_MAP_SWIZZLE_128B;
    CUtensorMap cm, km, vm;
    {
        const cuuint64_t dims[2] = {(cuuint64_t)pr.row, (cuuint64_t)pr.num_pages * kPage};
        const cuuint64_t strides[1] = {(cuuint64_t)pr.row * 2};
        const cuuint32_t box[2] = {kChunk, kPage};
        if (encode_tiled(&cm, bf16, 2, const_cast<void *>(kv_cache), dims, strides, box, swz) != CUDA_SUCCESS)
            return KVATTN_ERR_UNSUPPORTED;
    }
    {
        const cuuint64_t dims[3] = {(cuuint64_t)pr.dn, (cuuint64_t)d_k, (cuuint64_t)pr.H};
        const cuuint64_t strides[2] = {(cuuint64_t)pr.dn * 2, (cuuint64_t)pr.dn * d_k * 2};
        const cuuint32_t box[3] = {kChunk, 128, 1};
        if (encode_tiled(&km, bf16, 3, const_cast<void *>(w_uk), dims, strides, box, swz) != CUDA_SUCCESS)
            return KVATTN_ERR_UNSUPPORTED;
    }
    {
        const cuuint64_t dims[3] = {(cuuint64_t)d_v, (cuuint64_t)pr.dn, (cuuint64_t)pr.H};
        const cuuint64_t strides[2] = {(cuuint64_t)d_v * 2, (cuuint64_t)pr.dn * d_v * 2};
        const cuuint32_t box[3] = {64, kChunk, 1};
        if (encode_tiled(&vm, bf16, 3, const_cast<void *>(w_uv), dims, strides, box, swz) != CUDA_SUCCESS)
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
    if (ragged::launch_plan(pa, s) != cudaSuccess)
        return KVATTN_ERR_CUDA;
    ExpandArgs a{};
    a.header = pa.header;
    a.tiles = pa.tiles;
    a.block_table = block_table;
    a.cache = static_cast<const __nv_bfloat16 *>(kv_cache);
    a.k = static_cast<__nv_bfloat16 *>(k_nope);
    a.v = static_cast<__nv_bfloat16 *>(v);
    a.k_rope = static_cast<__nv_bfloat16 *>(k_rope);
    a.err = device_error;
    a.heads = pr.H;
    a.heads_per_group = pr.HPU;
    a.groups = pr.NU;
    a.d_c = pr.dn;
    a.d_k = d_k;
    a.d_v = d_v;
    a.d_rope = pr.dr;
    a.row = pr.row;
    a.mpps = pr.mpps;
    a.num_pages = pr.num_pages;
    a.max_kv = max_kv_tokens;
    if (cudaFuncSetAttribute(expand_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmem) != cudaSuccess)
        return KVATTN_ERR_CUDA;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(pr.H, (unsigned)cap);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kSmem;
    cfg.stream = s;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, expand_kernel, cm, km, vm, (const ExpandArgs)a) == cudaSuccess ? KVATTN_OK
                                                                                                   : KVATTN_ERR_CUDA;
}
