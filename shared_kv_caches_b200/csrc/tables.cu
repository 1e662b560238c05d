// A step's bookkeeping on the GPU: pages, positions and slots of the new
// tokens of every request (kvattn_build_tables), and the write of their rows
// into the paged cache by slot (kvattn_append_slots).
//
// build_tables.  With c_b cached and n_b new tokens of request b, request b
// holds ceil(c_b / 64) pages and needs d_b = ceil((c_b + n_b) / 64) -
// ceil(c_b / 64) more.  Three exclusive prefix sums over the requests (new
// tokens, pages, context) give every chunk's start and every request's first
// place in the free list; after them each token and each new page is a lookup
// of its own:
//   pos(t)  = c_b + t - q_start_b
//   page(i) = i-th entry from the top of the free list for the request's new
//             pages, the table's entry for the page it already holds
// The whole call is one launch: every CTA repeats the sums (a few thousand
// integers) and takes a share of the tokens and pages.  Where the lengths and
// the free count are updated in place (a captured decode step advances by
// itself on each replay), the CTAs are one thread-block cluster, and the new
// values are written after its barrier, when every CTA has read the old.
#include <cuda_fp8.h>
#include <math.h>

#include "ragged.cuh"
#include "rope.cuh"

namespace kvattn {

namespace {

bool is_aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

constexpr int kTableThreads = ragged::kThreads;
constexpr int kTableMaxCtas = 8;           // the portable cluster size
constexpr int kTokensPerCta = 4096;

struct TableArgs {
    int batch, mpps, num_pages, max_tokens;
    int vectors;                                    // pos and slots start on 16 bytes
    const int32_t *cached, *fresh, *free_pages, *free_count;
    int32_t *table, *seq_lens, *free_left, *q_start, *kv_start, *pos, *slots, *err;
};

// Shared memory of the sums over the requests.
constexpr size_t table_smem(int batch) { return (3 * (size_t)batch + 2) * sizeof(int32_t); }

__device__ __forceinline__ int pages_of(long long n) { return (int)((n + kPage - 1) / kPage); }

__global__ void __launch_bounds__(kTableThreads, 1) build_tables_kernel(const TableArgs a)
{
    extern __shared__ int32_t sh_i[];
    __shared__ long long sh_scan[32];
    __shared__ int sh_taken, sh_served;
    int32_t *tok = sh_i;                            // [B + 1] first token of each chunk (at most max_tokens)
    int32_t *pgs = sh_i + a.batch + 1;              // [B + 1] new pages of the requests before
    int32_t *cch = sh_i + 2 * (a.batch + 1);        // [B] cached tokens, or -1 - cached where the request gets nothing
    const int tid = threadIdx.x, rank = blockIdx.x, ctas = gridDim.x;
    const long long capacity = min((long long)a.mpps * kPage, (long long)INT32_MAX);   // lengths are 32-bit numbers
    const int raw_free = *a.free_count;
    const int nfree = min(max(raw_free, 0), a.num_pages);
    int bits = raw_free == nfree ? 0 : KVATTN_DEVERR_BAD_LENGTH;

    const int per = (a.batch + kTableThreads - 1) / kTableThreads;
    const int b0 = min(tid * per, a.batch), b1 = min(b0 + per, a.batch);
    // what request b asks for: its token count, and its pages if the lengths can be served at all
    auto request = [&](int b, int &c, int &n, int &pages) -> bool {
        c = a.cached[b];
        n = a.fresh[b];
        pages = 0;
        if (c < 0 || n < 0) {
            bits |= KVATTN_DEVERR_BAD_LENGTH;
            c = max(c, 0);
            n = max(n, 0);
            return false;
        }
        if ((long long)c + n > capacity) {
            bits |= KVATTN_DEVERR_SEQ_TOO_LONG;
            return false;
        }
        pages = pages_of((long long)c + n) - pages_of(c);
        return true;
    };
    long long ntok = 0, npg = 0, tok_total, pg_total;
    for (int b = b0; b < b1; ++b) {
        int c, n, pages;
        request(b, c, n, pages);
        ntok += n;
        npg += pages;
    }
    ntok = ragged::block_scan(ntok, tok_total, sh_scan);
    npg = ragged::block_scan(npg, pg_total, sh_scan);
    long long ctx = 0, ctx_total;
    int taken = 0;
    bool late = false;                              // requests here that want pages, but whose tokens do not fit
    {
        long long t = ntok, p = npg;
        for (int b = b0; b < b1; ++b) {
            int c, n, pages;
            bool ok = request(b, c, n, pages);
            tok[b] = (int)min(t, (long long)a.max_tokens);
            pgs[b] = (int)min(p, (long long)a.num_pages);
            t += n;
            p += pages;
            if (n > 0 && t > a.max_tokens) {
                bits |= KVATTN_DEVERR_TOO_MANY_TOKENS;
                ok = false;
                late |= pages > 0;
                if (t - n <= a.max_tokens)          // the first of them
                    sh_served = (int)min(p - pages, (long long)INT32_MAX);
            } else if (pages > 0 && p > nfree) {
                bits |= KVATTN_DEVERR_POOL_EXHAUSTED;
                ok = false;
            }
            cch[b] = ok ? c : -1 - c;
            ctx += ok ? (long long)c + n : c;
            // the requests that get pages are the first ones that ask for any
            // (both sums only grow), so the list's top `taken` entries go
            if (ok && pages > 0)
                taken = (int)p;
        }
    }
    const int total = (int)min(tok_total, (long long)a.max_tokens);
    if (tid == 0) {
        tok[a.batch] = total;
        pgs[a.batch] = (int)min(pg_total, (long long)a.num_pages);
        sh_taken = 0;
    }
    ctx = ragged::block_scan(ctx, ctx_total, sh_scan);
    // a request whose tokens do not fit takes no pages: the list is too short
    // for it only where it lacks pages beside those of the requests before
    // the first such one
    if (late) {
        long long t = ntok;
        for (int b = b0; b < b1; ++b) {
            int c, n, pages;
            request(b, c, n, pages);
            t += n;
            if (n > 0 && t > a.max_tokens && pages > 0 && (long long)sh_served + pages > nfree)
                bits |= KVATTN_DEVERR_POOL_EXHAUSTED;
        }
    }
    if (taken > 0)
        atomicMax(&sh_taken, taken);
    if (rank == 0 && bits && a.err)
        atomicOr(a.err, bits);
    // every CTA of the cluster (or this one alone) has read the lengths and the free count
    cluster_sync_all();
    taken = sh_taken;

    if (rank == 0) {
        for (int b = b0; b < b1; ++b) {
            const int c = cch[b], n = max(a.fresh[b], 0);
            const int len = c >= 0 ? c + n : -1 - c;
            a.seq_lens[b] = len;
            a.q_start[b] = tok[b];
            if (a.kv_start)
                a.kv_start[b] = (int)min(ctx, (long long)INT32_MAX);
            ctx += len;
        }
        if (tid == 0) {
            a.q_start[a.batch] = total;
            if (a.kv_start)
                a.kv_start[a.batch] = (int)min(ctx_total, (long long)INT32_MAX);
            *a.free_left = nfree - taken;
        }
    }
    bits = 0;
    for (int i = rank * kTableThreads + tid; i < taken; i += ctas * kTableThreads) {
        const int b = ragged::find(pgs, a.batch, i);
        const int page = a.free_pages[nfree - 1 - i];
        if (page < 0 || page >= a.num_pages)
            bits = KVATTN_DEVERR_PAGE_OUT_OF_RANGE;
        a.table[(long long)b * a.mpps + pages_of(cch[b]) + i - pgs[b]] = page;
    }
    // four tokens at a time: one search, and one page looked up, for most
    for (int t0 = 4 * (rank * kTableThreads + tid); t0 < a.max_tokens; t0 += 4 * ctas * kTableThreads) {
        int pos[4], slot[4];
        int b = t0 < total ? ragged::find(tok, a.batch, t0) : 0;
        int c = 0, at = -1, page = -1;                  // the request's cached tokens; the page looked up last
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int t = t0 + k;
            pos[k] = 0;
            slot[k] = -1;
            if (t >= total)
                continue;
            if (k == 0 || t >= tok[b + 1]) {
                while (t >= tok[b + 1])
                    ++b;
                c = cch[b];
                at = -1;
            }
            const long long p = (long long)(c >= 0 ? c : -1 - c) + t - tok[b];
            pos[k] = (int)min(p, (long long)INT32_MAX);
            if (c < 0)
                continue;
            const int pi = (int)(p / kPage), held = pages_of(c);
            if (pi != at) {
                at = pi;
                page = pi < held ? a.table[(long long)b * a.mpps + pi] : a.free_pages[nfree - 1 - (pgs[b] + pi - held)];
            }
            if (page < 0 || page >= a.num_pages)
                bits = KVATTN_DEVERR_PAGE_OUT_OF_RANGE;
            else
                slot[k] = page * kPage + (int)(p % kPage);
        }
        if (a.vectors && t0 + 4 <= a.max_tokens) {
            *reinterpret_cast<int4 *>(a.pos + t0) = make_int4(pos[0], pos[1], pos[2], pos[3]);
            *reinterpret_cast<int4 *>(a.slots + t0) = make_int4(slot[0], slot[1], slot[2], slot[3]);
        } else {
            for (int k = 0; k < 4 && t0 + k < a.max_tokens; ++k) {
                a.pos[t0 + k] = pos[k];
                a.slots[t0 + k] = slot[k];
            }
        }
    }
    if (bits && a.err)
        atomicOr(a.err, bits);
}

// ------------------------------------------------------- append by slot

constexpr int kAppendThreads = 256;

struct SlotAppendArgs {
    const __nv_bfloat16 *src;     // [tokens][planes][row]
    const int32_t *pos;           // [tokens]; read only where rows are turned
    const int32_t *slots;         // [tokens]
    void *cache;
    int32_t *err;                 // may be null
    int tokens, planes, row;
    int copy;                     // leading elements of plane 0 taken as they are
    int rot_width, rot_count;     // RoPE over rot_count slices of rot_width after `copy`
    long long num_slots;
    double log2_base;
    float k_scale, v_scale;       // fp8: what a stored value is multiplied by when it is read
};

// x / scale in fp32; exactly the product with 1 / scale where that is a power of two.
__device__ __forceinline__ float unscaled(float x, float scale, float inverse, bool exact)
{
    return exact ? x * inverse : x / scale;
}

// Two values as e4m3 bytes, nearest even, saturated at +-448.
__device__ __forceinline__ uint16_t e4m3_pair(float x, float y)
{
    return (uint16_t)__nv_cvt_float2_to_fp8x2(make_float2(x, y), __NV_SATFINITE, __NV_E4M3);
}

// Eight bf16 values divided by scale, as e4m3 bytes.
__device__ __forceinline__ uint2 e4m3_oct(uint4 v, float scale)
{
    // a product is a tenth of a division's instructions (fp8 append of 9001
    // tokens: 31 -> 20 us)
    const bool exact = (__float_as_uint(scale) & 0x7fffffu) == 0 && scale > 1e-30f && scale < 1e30f;
    const float inverse = 1.f / scale;
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    uint32_t r[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        r[i] = e4m3_pair(unscaled(__uint_as_float(w[i] << 16), scale, inverse, exact),
                         unscaled(__uint_as_float(w[i] & 0xffff0000u), scale, inverse, exact));
    return make_uint2(r[0] | (r[1] << 16), r[2] | (r[3] << 16));
}

// Four 16-byte vectors a lane at a time: 2 KB of a row on their way per warp.
constexpr int kAppendVecs = 4;
// Heads whose pairs a lane loads before it forms their angle.
constexpr int kAppendHeads = 8;

// One warp per token: 16-byte copies of what is stored as it is; a turned
// pair belongs to one lane, which forms its angle once for the token and turns
// the pair of every slice (every K head) with it.  The angle and the turn are
// in double precision with one rounding to the stored type, by the routine that
// kvattn_rope uses; a lane's first two rates (all it has for slices up to 128
// wide) stay in registers over its tokens.  Bound by memory latency: a row's
// loads do not wait for its slot or for the angles, which are formed while they
// are under way.
template <bool FP8>
__global__ void __launch_bounds__(kAppendThreads, 4) append_slots_kernel(const SlotAppendArgs a)
{
    const int lane = threadIdx.x & 31;
    const unsigned warps = gridDim.x * (kAppendThreads / 32);
    const int half = a.rot_width / 2;
    double rate0 = 0.0, rate1 = 0.0;
    if (a.rot_count > 0) {
        rate0 = rope_rate(lane, a.rot_width, a.log2_base);
        if (half > 32)
            rate1 = rope_rate(lane + 32, a.rot_width, a.log2_base);
    }
    // (unsigned: the step past the last of 2^31 - 1 tokens stays in front of 2^32)
    for (unsigned t = blockIdx.x * (kAppendThreads / 32) + (threadIdx.x >> 5); t < (unsigned)a.tokens; t += warps) {
        const int slot = a.slots[t];
        const int pos = a.rot_count > 0 ? a.pos[t] : 0;
        const bool valid = slot >= 0 && slot < a.num_slots;
        const long long page = slot / kPage;
        const int off = slot % kPage;
        for (int pl = 0; pl < a.planes; ++pl) {
            const __nv_bfloat16 *src = a.src + ((long long)t * a.planes + pl) * a.row;
            const long long at = ((page * a.planes + pl) * kPage + off) * (long long)a.row;
            const bool turn = a.rot_count > 0 && pl == 0;
            const int copy = turn ? a.copy : a.row, vecs = copy / 8;
            const float scale = pl == 0 ? a.k_scale : a.v_scale;
            for (int i0 = lane; i0 < vecs; i0 += 32 * kAppendVecs) {
                uint4 v[kAppendVecs];
#pragma unroll
                for (int x = 0; x < kAppendVecs; ++x)
                    if (i0 + 32 * x < vecs)
                        v[x] = __ldcs(reinterpret_cast<const uint4 *>(src) + i0 + 32 * x);
                if (!valid)
                    break;
#pragma unroll
                for (int x = 0; x < kAppendVecs; ++x) {
                    const int i = i0 + 32 * x;
                    if (i >= vecs)
                        break;
                    if constexpr (FP8)
                        reinterpret_cast<uint2 *>(static_cast<uint8_t *>(a.cache) + at)[i] = e4m3_oct(v[x], scale);
                    else
                        reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(a.cache) + at)[i] = v[x];
                }
            }
            if (!turn || !valid)
                continue;
            const double unscale = 1.0 / (double)scale;
            for (int i = lane; i < half; i += 32) {
                const double rate = i == lane ? rate0 : i == lane + 32 ? rate1 : rope_rate(i, a.rot_width, a.log2_base);
                double s = 0.0, c = 1.0;
                for (int n0 = 0; n0 < a.rot_count; n0 += kAppendHeads) {
                    __nv_bfloat162 v[kAppendHeads];
#pragma unroll
                    for (int n = 0; n < kAppendHeads; ++n)
                        if (n0 + n < a.rot_count)
                            v[n] = *reinterpret_cast<const __nv_bfloat162 *>(src + copy + (n0 + n) * a.rot_width + 2 * i);
                    if (n0 == 0)
                        rope_angle(pos, rate, &s, &c);
#pragma unroll
                    for (int n = 0; n < kAppendHeads; ++n) {
                        if (n0 + n >= a.rot_count)
                            break;
                        const int e = copy + (n0 + n) * a.rot_width + 2 * i;
                        double rx, ry;
                        rope_turn((double)__bfloat162float(v[n].x), (double)__bfloat162float(v[n].y), s, c, &rx, &ry);
                        if constexpr (FP8) {
                            // one rounding to e4m3 but for the one to fp32 in
                            // front of it, 20 bits finer
                            *reinterpret_cast<uint16_t *>(static_cast<uint8_t *>(a.cache) + at + e) =
                                e4m3_pair((float)(rx * unscale), (float)(ry * unscale));
                        } else {
                            __nv_bfloat162 r;
                            r.x = __double2bfloat16(rx);
                            r.y = __double2bfloat16(ry);
                            *reinterpret_cast<__nv_bfloat162 *>(static_cast<__nv_bfloat16 *>(a.cache) + at + e) = r;
                        }
                    }
                }
            }
        }
        if (!valid && slot != -1 && lane == 0 && a.err)
            atomicOr(a.err, KVATTN_DEVERR_PAGE_OUT_OF_RANGE);
    }
}

}  // namespace

}  // namespace kvattn

using namespace kvattn;

extern "C" int kvattn_build_tables(int32_t batch, int32_t max_pages_per_seq, int32_t num_pages, int32_t max_tokens,
                                   const int32_t *cached_lens, const int32_t *new_lens, const int32_t *free_pages,
                                   const int32_t *free_count, int32_t *block_table, int32_t *seq_lens,
                                   int32_t *free_left, int32_t *q_start, int32_t *kv_start, int32_t *pos,
                                   int32_t *slots, int32_t *device_error, void *stream)
{
    if (batch < 1 || max_pages_per_seq < 1 || num_pages < 1 || max_tokens < 0)
        return KVATTN_ERR_INVALID_ARG;
    if (!cached_lens || !new_lens || !free_pages || !free_count || !block_table || !seq_lens || !free_left ||
        !q_start || (max_tokens > 0 && (!pos || !slots)))
        return KVATTN_ERR_INVALID_ARG;
    if (batch > ragged::kMaxBatch || num_pages > INT32_MAX / kPage || max_tokens > (1 << 30))
        return KVATTN_ERR_UNSUPPORTED;
    for (const void *p : {static_cast<const void *>(cached_lens), static_cast<const void *>(new_lens),
                          static_cast<const void *>(free_pages), static_cast<const void *>(free_count),
                          static_cast<const void *>(block_table), static_cast<const void *>(seq_lens),
                          static_cast<const void *>(free_left), static_cast<const void *>(q_start),
                          static_cast<const void *>(kv_start), static_cast<const void *>(pos),
                          static_cast<const void *>(slots), static_cast<const void *>(device_error)})
        if (!is_aligned(p, 4))
            return KVATTN_ERR_MISALIGNED;
    TableArgs a{batch, max_pages_per_seq, num_pages, max_tokens,
                is_aligned(pos, 16) && is_aligned(slots, 16), cached_lens, new_lens, free_pages, free_count,
                block_table, seq_lens, free_left, q_start, kv_start, pos, slots, device_error};
    int ctas = (max_tokens + kTokensPerCta - 1) / kTokensPerCta;
    // in place, what one CTA writes others read: a cluster of up to eight.
    // Otherwise as many as there are tokens for (150 thousand: 13 us with
    // eight, 6 with 37)
    const bool in_place = seq_lens == cached_lens || free_left == free_count;
    const int most = in_place ? kTableMaxCtas : sm_count();
    ctas = ctas < 1 ? 1 : ctas > most ? most : ctas;
    const size_t smem = table_smem(batch);
    // the 48 KB of a launch without an opt-in hold what the kernel declares
    // itself (272 bytes) too; the opt-in is for the largest batch, so that no
    // call lowers it under another one's launch
    if (smem > 40 * 1024) {
        const cudaError_t e = cudaFuncSetAttribute(build_tables_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   (int)table_smem(ragged::kMaxBatch));
        if (e != cudaSuccess)
            return launch_status(e);
    }
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3(kTableThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = static_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = ctas;
    attr.val.clusterDim.y = 1;
    attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = in_place && ctas > 1 ? 1 : 0;
    return launch_status(cudaLaunchKernelEx(&cfg, build_tables_kernel, (const TableArgs)a));
}

extern "C" int kvattn_append_slots(int32_t variant, const kvattn_params *p, const void *new_kv, int32_t num_tokens,
                                   const int32_t *pos, const int32_t *slots, void *kv_cache, float rope_base,
                                   int32_t *device_error, void *stream)
{
    Problem pr;
    const int st = validate_params(variant, p, &pr);
    if (st)
        return st;
    if (num_tokens < 0 || !new_kv || !slots || !kv_cache)
        return KVATTN_ERR_INVALID_ARG;
    if (!(rope_base == 0.f || (rope_base > 1.f && isfinite(rope_base))))
        return KVATTN_ERR_INVALID_ARG;
    if (rope_base > 0.f && !pos)
        return KVATTN_ERR_INVALID_ARG;
    const bool tied = !pr.latent && pr.kv_planes == 1;
    if (tied && rope_base != 0.f)
        return KVATTN_ERR_INVALID_ARG;      // the row is the value too (as in kvattn_append_kv)
    if (pr.num_pages > INT32_MAX / kPage)
        return KVATTN_ERR_UNSUPPORTED;
    if (!is_aligned(new_kv, 16) || !is_aligned(kv_cache, 16) || !is_aligned(pos, 4) || !is_aligned(slots, 4) ||
        !is_aligned(device_error, 4))
        return KVATTN_ERR_MISALIGNED;
    if (num_tokens == 0)
        return KVATTN_OK;
    const bool fp8 = p->cache_dtype == KVATTN_CACHE_FP8_E4M3;
    SlotAppendArgs a{};
    a.src = static_cast<const __nv_bfloat16 *>(new_kv);
    a.pos = pos;
    a.slots = slots;
    a.cache = kv_cache;
    a.err = device_error;
    a.tokens = num_tokens;
    a.row = pr.row;
    a.planes = pr.latent || tied ? 1 : 2;
    a.num_slots = (long long)pr.num_pages * kPage;
    a.log2_base = rope_base > 0.f ? log2((double)rope_base) : 0.0;
    a.k_scale = fp8 ? p->k_scale : 1.f;
    a.v_scale = fp8 ? p->v_scale : 1.f;
    if (rope_base > 0.f) {
        a.copy = pr.latent ? pr.NU * pr.dn : 0;
        a.rot_width = pr.latent ? pr.dr : pr.dn;
        a.rot_count = pr.latent ? (pr.dr > 0 ? 1 : 0) : pr.NU;
    }
    const int per = kAppendThreads / 32;
    const long long want = ((long long)num_tokens + per - 1) / per;
    const long long most = 4LL * sm_count();      // the blocks that are resident: rates are formed once a warp
    const int grid = (int)(want < most ? want : most);
    // (launched so that the status is this launch's, not an earlier call's)
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(kAppendThreads);
    cfg.stream = static_cast<cudaStream_t>(stream);
    return launch_status(cudaLaunchKernelEx(&cfg, fp8 ? append_slots_kernel<true> : append_slots_kernel<false>,
                                            (const SlotAppendArgs)a));
}
