// Attention of ragged chunks of new tokens over per-head keys and values
// (kvattn_prefill): the expanded form of latent attention, and grouped heads
// without a rope part.
//
//   s_ij = sm_scale (q_nope_i . k_nope_j + q_rope_i . k_rope_j)
//   o_i  = sum_j softmax_j(s_ij) v_j        over j < nk (causal: j <= i + nk - nq)
//
// One CTA works off 256 query rows of one head (two MMA tiles of 128) against
// key tiles of 96 tokens in one pass with a running maximum and sum.  Per key
// tile and query tile, for a key of 192 and a value of 128, shared memory gives
// the operands of the scores (12 MMAs of N = 96 that read 7 KB each, at 128
// bytes a cycle) in 672 cycles, P.V (6 MMAs of N = 128, P from TMEM) takes 384,
// and the special-function units 768 for 128 x 96 exponentials at 16 a cycle.
// A softmax step from start to end takes longer than the MMAs of a tile, so
// everything that can is taken off the path between two steps of a query tile:
// its next scores are formed while its softmax runs (the scores' columns are
// free as soon as they are in registers), and the other query tile's MMAs fill
// what is left.  Measured: 1150 cycles per key tile and query tile (1056 of
// MMAs) in the middle of an 8K prompt; the whole call, causal, 128 heads, takes
// 2.24 ms when repeated back to back, at the power cap (1.23 PFLOP/s), and 1.95
// to 2.0 ms for the first few calls after a pause.
// Forming a part of the exponentials on the FMA pipe makes the softmax shorter
// and the call longer (8K prompt 2263 us without, 2321 with a quarter of them).
//
// TMEM (512 columns): outputs of the two query tiles (128 each), their scores
// (96 each), and one tile of bf16 probabilities (48) that the two take turns
// with; keys come in tiles of 96, not 128, so that all of it fits.  Shared
// memory: the two query tiles, two key tiles and two value tiles, in boxes of 64
// columns (128-byte swizzle).
//
// Warp roles (384 threads):
//   warp 0     one thread hands out the items and streams queries, keys and
//              values with TMA
//   warp 1     issues the MMAs of the scores, S0(j) S1(j) S0(j+1) ...
//   warp 2     issues those of P.V, PV0(j) PV1(j) PV0(j+1) ... (a warp of its
//              own: one that issued both spent more time on the waits and
//              commits between them than the MMAs take)
//   warp 3     guards the value tiles that some row does not attend whole: what
//              is not finite there must not reach the rows that leave it out
//   warps 4-11 one thread per query row: scores from TMEM, mask, online softmax
//              in fp32 (base 2), probabilities back to TMEM in bf16, output
//              rescaled when the maximum grows by more than 2^8 (lazily: the
//              reference maximum only scales numerator and denominator alike)
// P is rounded to bf16 for the MMA, as in the decode kernels (off by at most 2^-8
// of the weight, as much as the output's own rounding); the sum uses the unrounded values; scores, maxima, sums and outputs stay in
// fp32.
//
// The work list (tiles by falling number of keys) comes from ragged.cu; the
// CTAs, one per SM, take its items as they get to them, ordered by groups of
// eight heads, then tiles, then heads, so that the CTAs at work share a few
// heads' keys and values in L2.  The last group is 16 heads or more: the items
// handed out last are then short ones (4K prompt, 74 heads, repeated: 378 us with
// eight, 370; 24 heads or more gain there and lose on longer prompts).
#include <math.h>

#include <atomic>

#include "latent_common.cuh"
#include "ragged.cuh"

namespace kvattn {

namespace {

using ragged::elect_commit;
using ragged::elect_ss;
using ragged::elect_ts;
using latent::exp2_approx;
using latent::fadd2;
using latent::ffma2;
using latent::kLn2;
using latent::kRescaleThreshold;
using latent::reduce_extreme;

bool is_aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

constexpr int kTile = 128;                        // query rows of an MMA tile
constexpr int kKeys = 96;                         // keys of a key tile
constexpr int kItemRows = 2 * kTile;              // query rows of a work item
constexpr int kThreads = 384;
// Registers: 384 threads are launched with 168 each (the most that fit), the
// two softmax warpgroups, which hold a row of scores a thread, take theirs
// from the one that only issues.  88 + 2 * 208 = 3 * 168.
constexpr int kLaunchRegs = 168, kIssueRegs = 88, kSoftmaxRegs = 208;
static_assert(kIssueRegs + 2 * kSoftmaxRegs <= 3 * kLaunchRegs, "register split");
constexpr int kQBox = kTile * 128;                // 128 query rows x 64 bf16
constexpr int kBox = kKeys * 128;                 // 96 keys x 64 bf16
constexpr float kFarReference = 1073741824.f;     // 2^30
constexpr int kHeadGroup = 8, kLastHeads = 16;    // heads of a group, and at least in the last one
constexpr int kBarBytes = 2048;
constexpr int kSmemMax = 227 * 1024;

struct PrefillArgs {
    ragged::PlanArgs plan;                        // header: [0] tiles, [1] items handed out (0 at the start)
    int listed;                                   // the plan kernel has listed the tiles; else every CTA does
    void *out;
    float *lse;                                   // may be null
    int32_t *err;                                 // may be null
    int head_groups;                              // groups of kHeadGroup heads in front of the last, larger one
    int heads, heads_per_kv, heads_per_q;         // heads that share a key head, and a q_nope head
    int d_v, out_fp32, causal;
    int wide;                                     // output rows start on 32 bytes
    long long out_token_stride, out_head_stride;
    const __nv_bfloat16 *v;
    long long v_token_stride, v_head_stride;
    float scale_log2;                             // of the scale's magnitude
    uint32_t negate;                              // a negative scale: the MMAs take -q (the instruction descriptor's bit)
};

struct Maps {
    CUtensorMap q, qr, k, kr, v;
};

// NKB key boxes (the last one the rope part if ROPE), NVB value boxes.
template <int NKB, int NVB>
struct Layout {
    static constexpr int kKeyTile = NKB * kBox, kValueTile = NVB * kBox;
    static constexpr size_t kKeysAt = (size_t)2 * NKB * kQBox;
    static constexpr size_t kValuesAt = kKeysAt + 2 * kKeyTile;
    static constexpr size_t kBarsAt = kValuesAt + 2 * kValueTile;
    static constexpr size_t kBytes = kBarsAt + kBarBytes;
    static_assert(kBytes <= kSmemMax, "shared memory");
};

// A work item: a tile of the list, a head, and the keys of its two query tiles.
struct Item {
    int32_t q0, nq, k0, nk, lim0;                 // as in ragged::Tile
    int32_t head;                                 // -1: no more items
    int32_t end0, end1;                           // keys that the last row of each query tile attends

    int32_t all;                                  // keys that every row attends

    __device__ __forceinline__ int tiles0() const { return (end0 + kKeys - 1) / kKeys; }
    __device__ __forceinline__ int tiles1() const { return (end1 + kKeys - 1) / kKeys; }
};

// The items that the TMA thread hands out stand here until all have read them.
constexpr int kItems = 4;
constexpr int kItemReaders = 11;                  // the MMA, guard and softmax warps
// Key tiles of an item that some row does not attend, or that end behind the
// sequence: the rows' limits span 256 keys.
constexpr int kEdgeTiles = 5;

struct Bars {
    uint64_t k_full[2], k_empty[2], v_full[2], v_empty[2];
    uint64_t item_full[kItems], item_empty[kItems];
    Item item[kItems];
    uint32_t bad[kItems][kEdgeTiles][kKeys / 32]; // tokens of the edge tiles whose values are not finite
    uint64_t edge_full[2];                        // an edge tile's values have landed (the guard looks them over)
    ragged::Tile tiles[ragged::kSmallTiles];
    uint64_t q_full[2], q_empty[2];
    uint64_t s_full[2], s_free[2];                // scores formed; scores in registers
    uint64_t p_full[2];                           // probabilities stored
    uint64_t p_free[2];                           // every P.V before this query tile's next one is done
    uint64_t o_full[2];                           // the item's last P.V of the query tile is done
    uint64_t mma_done[2];
    uint32_t tmem_base;
};
static_assert(sizeof(Bars) <= kBarBytes, "barrier space");

template <int N>
__device__ __forceinline__ void set_regs_up()
{
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}

template <int N>
__device__ __forceinline__ void set_regs_down()
{
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// 16 columns of this thread's TMEM lane; the store is waited for with tmem_st_wait.
__device__ __forceinline__ void tmem_st16_start(uint32_t taddr, const uint32_t *r)
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15, %16};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}

// 32 columns; the values may be used after tmem_ld_wait, which names them.
__device__ __forceinline__ void tmem_ld32_start(uint32_t taddr, float *r)
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]), "=f"(r[7]), "=f"(r[8]),
          "=f"(r[9]), "=f"(r[10]), "=f"(r[11]), "=f"(r[12]), "=f"(r[13]), "=f"(r[14]), "=f"(r[15]), "=f"(r[16]),
          "=f"(r[17]), "=f"(r[18]), "=f"(r[19]), "=f"(r[20]), "=f"(r[21]), "=f"(r[22]), "=f"(r[23]), "=f"(r[24]),
          "=f"(r[25]), "=f"(r[26]), "=f"(r[27]), "=f"(r[28]), "=f"(r[29]), "=f"(r[30]), "=f"(r[31])
        : "r"(taddr)
        : "memory");
}

__device__ __forceinline__ void tmem_ld_wait(float *r)
{
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
    for (int i = 0; i < 32; ++i)
        asm volatile("" : "+f"(r[i]));
}

__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ int key_end(const PrefillArgs &a, const ragged::Tile &t, int rows_before, int rows)
{
    // keys that the last of `rows` rows from rows_before on attends
    if (rows <= 0)
        return 0;
    return a.causal ? min(t.nk, max(t.lim0 + rows_before + rows - 1, 0)) : t.nk;
}

// Of two bf16 values: the top bit of each that is infinite or NaN; and the word
// with those set to 0.
__device__ __forceinline__ uint32_t exponent_ones(uint32_t w) { return ((w & 0x7f807f80u) + 0x00800080u) & 0x80008000u; }

__device__ __forceinline__ uint32_t finite_only(uint32_t w)
{
    const uint32_t e = exponent_ones(w);
    return w & ~((e & 0x8000u ? 0xffffu : 0u) | (e & 0x80000000u ? 0xffff0000u : 0u));
}

// N words of a row: with `wide` (rows that start on 32 bytes) a whole sector at a time.
template <int N>
__device__ __forceinline__ void store_row(void *p, const uint32_t *r, bool wide)
{
    if constexpr (N == 8) {
        if (wide) {
            asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(r[0]), "r"(r[1]),
                         "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                         : "memory");
            return;
        }
        static_cast<uint4 *>(p)[1] = make_uint4(r[4], r[5], r[6], r[7]);
    }
    static_cast<uint4 *>(p)[0] = make_uint4(r[0], r[1], r[2], r[3]);
}

// Item i of the list: groups of kHeadGroup heads (the rest in one group), then tiles, then heads.
__device__ __forceinline__ Item get_item(const PrefillArgs &a, const ragged::Tile *tiles, int ntiles, int i)
{
    const int per_group = ntiles * kHeadGroup;
    const int g = min(i / per_group, a.head_groups), r = i - g * per_group;
    const int hc = g < a.head_groups ? kHeadGroup : a.heads - g * kHeadGroup;
    const ragged::Tile t = tiles[r / hc];
    Item it;
    it.q0 = t.q0;
    it.nq = t.nq;
    it.k0 = t.k0;
    it.nk = t.nk;
    it.lim0 = t.lim0;
    it.head = g * kHeadGroup + r % hc;
    it.end0 = key_end(a, t, 0, min(t.nq, kTile));
    it.end1 = key_end(a, t, kTile, t.nq - kTile);
    it.all = a.causal ? min(t.nk, max(t.lim0 + (it.end0 > 0 ? 0 : kTile), 0)) : t.nk;
    return it;
}

template <int NKB, bool ROPE, int NVB>
__global__ void __launch_bounds__(kThreads, 1)
    prefill_kernel(const __grid_constant__ Maps m, const PrefillArgs a)
{
    using Lay = Layout<NKB, NVB>;
    constexpr int NKN = ROPE ? NKB - 1 : NKB;
    constexpr int kDv = NVB * 64;
    constexpr uint32_t kIdescS = idesc_bf16_f32(kTile, kKeys, false, false);
    constexpr uint32_t kIdescPV = idesc_bf16_f32(kTile, kDv, false, true);
    extern __shared__ __align__(1024) unsigned char smem[];
    Bars &B = *reinterpret_cast<Bars *>(smem + Lay::kBarsAt);
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    if (smem_u32(smem) & 1023u) {
        if (threadIdx.x == 0 && a.err)
            atomicOr(a.err, KVATTN_DEVERR_WAIT_TIMEOUT);
        return;
    }
    if (threadIdx.x == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(&B.k_full[i], 1);
            mbar_init(&B.k_empty[i], 1);
            mbar_init(&B.v_full[i], 1);
            mbar_init(&B.v_empty[i], 1);
            mbar_init(&B.edge_full[i], 1);
            mbar_init(&B.q_full[i], 1);
            mbar_init(&B.q_empty[i], 1);
            mbar_init(&B.s_full[i], 1);
            mbar_init(&B.s_free[i], 4);
            mbar_init(&B.p_full[i], 4);
            mbar_init(&B.p_free[i], 1);
            mbar_init(&B.o_full[i], 1);
        }
        for (int i = 0; i < kItems; ++i) {
            mbar_init(&B.item_full[i], 1);
            mbar_init(&B.item_empty[i], kItemReaders);
        }
        mbar_init(&B.mma_done[0], 1);
        mbar_init(&B.mma_done[1], 1);
        fence_mbar_init();
    }
    if (warp == 0)
        tmem_alloc(&B.tmem_base, 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tbase = B.tmem_base;
    const uint32_t tO = tbase;                           // + 128 for the second query tile
    const uint32_t tS = tbase + 256;                     // + kKeys for the second query tile
    const uint32_t tP = tS + 2 * kKeys;
    pdl_wait_primary();                                  // the tile list
    bool ok = true;
    // The next item, for a whole warp: null at the end or where a wait ran out.
    // It stays until the warp has called done_item.
    uint32_t taken = 0;
    auto next_item = [&]() -> const Item * {
        const uint32_t slot = taken % kItems;
        if (!__all_sync(0xffffffffu, mbar_wait(&B.item_full[slot], (taken / kItems) & 1))) {
            ok = false;
            return nullptr;
        }
        return B.item[slot].head < 0 ? nullptr : &B.item[slot];
    };
    auto done_item = [&]() {
        __syncwarp();
        if (lane == 0)
            mbar_arrive(&B.item_empty[taken % kItems]);
        ++taken;
    };
    // Every MMA that this warp issued has completed (before TMEM is freed).
    auto finish = [&]() {
        elect_commit(&B.mma_done[warp - 1]);
        ok = __all_sync(0xffffffffu, mbar_wait(&B.mma_done[warp - 1], 0)) && ok;
        if (!ok && lane == 0 && a.err)
            atomicOr(a.err, KVATTN_DEVERR_WAIT_TIMEOUT);
    };

    if (warp < 4) {
        set_regs_down<kIssueRegs>();
        if (warp == 0) {
            // ---------------------------------------------------------------- TMA
            const int ntiles = a.listed ? a.plan.header[0] : ragged::list_tiles(a.plan, B.tiles, blockIdx.x == 0);
            if (lane == 0) {
                uint32_t kn = 0, vn = 0;                     // key and value tiles loaded
                uint32_t qn[2] = {0, 0};                     // query tiles loaded
                uint32_t edge_seen = 0;                      // bit st: an edge tile was loaded; bit 2 + st: an odd number
                auto load_q = [&](const Item &it, int i) {
                    if (qn[i] > 0 && !mbar_wait(&B.q_empty[i], (qn[i] - 1) & 1)) {
                        ok = false;
                        return;
                    }
                    ++qn[i];
                    mbar_arrive_expect_tx(&B.q_full[i], NKB * kQBox);
                    const int row = it.q0 + i * kTile;
#pragma unroll
                    for (int b = 0; b < NKB; ++b) {
                        unsigned char *dst = smem + (i * NKB + b) * kQBox;
                        if (b < NKN)
                            tma_load_3d(dst, &m.q, 64 * b, it.head / a.heads_per_q, row, &B.q_full[i]);
                        else
                            tma_load_3d(dst, &m.qr, 0, it.head, row, &B.q_full[i]);
                    }
                };
                auto load_k = [&](const Item &it, int j) {
                    const int row = it.k0 + j * kKeys, kvh = it.head / a.heads_per_kv, st = kn & 1;
                    if (kn >= 2 && !mbar_wait(&B.k_empty[st], ((kn >> 1) - 1) & 1)) {
                        ok = false;
                        return;
                    }
                    ++kn;
                    unsigned char *dst = smem + Lay::kKeysAt + st * Lay::kKeyTile;
                    mbar_arrive_expect_tx(&B.k_full[st], Lay::kKeyTile);
#pragma unroll
                    for (int b = 0; b < NKB; ++b) {
                        if (b < NKN)
                            tma_load_3d(dst + b * kBox, &m.k, 64 * b, kvh, row, &B.k_full[st]);
                        else
                            tma_load_2d(dst + b * kBox, &m.kr, 0, row, &B.k_full[st]);
                    }
                };
                auto load_v = [&](const Item &it, int j) {
                    const int row = it.k0 + j * kKeys, kvh = it.head / a.heads_per_kv, st = vn & 1;
                    if (vn >= 2 && !mbar_wait(&B.v_empty[st], ((vn >> 1) - 1) & 1)) {
                        ok = false;
                        return;
                    }
                    ++vn;
                    unsigned char *dst = smem + Lay::kValuesAt + st * Lay::kValueTile;
                    const bool edge = (j + 1) * kKeys > it.all;
                    if (edge)
                        edge_seen = (edge_seen | 1u << st) ^ 4u << st;
                    uint64_t *const full = edge ? &B.edge_full[st] : &B.v_full[st];
                    mbar_arrive_expect_tx(full, Lay::kValueTile);
#pragma unroll
                    for (int b = 0; b < NVB; ++b)
                        tma_load_3d(dst + b * kBox, &m.v, 64 * b, kvh, row, full);
                };
                // items are handed out as CTAs get to them: the first by the block's
                // number, then by a count that the plan kernel sets to 0
                // (an item is looked up while the one before is loaded)
                const ragged::Tile *const tiles = a.listed ? a.plan.tiles : B.tiles;
                const int items = ntiles * a.heads;
                auto look_up = [&](int i) -> Item {
                    Item it{};
                    it.head = -1;
                    return i < items ? get_item(a, tiles, ntiles, i) : it;
                };
                Item next = look_up(blockIdx.x);
                for (uint32_t given = 0; ok; ++given) {
                    const uint32_t slot = given % kItems;
                    const Item it = next;
                    if (given >= kItems && !mbar_wait(&B.item_empty[slot], (given / kItems - 1) & 1)) {
                        ok = false;
                        break;
                    }
                    B.item[slot] = it;
                    mbar_arrive(&B.item_full[slot]);
                    if (it.head < 0)
                        break;
                    // (a batch that is not listed has a CTA for every item)
                    const int after = a.listed ? (int)gridDim.x + atomicAdd(&a.plan.header[1], 1) : items;
                    const int n0 = it.tiles0(), n1 = it.tiles1(), n = max(n0, n1);
                    if (n == 0) {
                        next = look_up(after);
                        continue;
                    }
                    if (n0 > 0)
                        load_q(it, 0);
                    if (ok)
                        load_k(it, 0);
                    if (ok && n1 > 0)
                        load_q(it, 1);
                    for (int j = 0; ok && j < n; ++j) {
                        if (j + 1 < n)
                            load_k(it, j + 1);
                        if (ok)
                            load_v(it, j);
                        if (j == 0)
                            next = look_up(after);
                    }
                }
                // every copy started here has landed before the CTA can exit
                for (uint32_t st = 0; st < 2; ++st) {
                    // phase of the stage's last load
                    if (kn > st && !mbar_wait(&B.k_full[st], ((kn - 1 - st) >> 1) & 1))
                        ok = false;
                    if (vn > st && !mbar_wait(&B.v_full[st], ((vn - 1 - st) >> 1) & 1))
                        ok = false;
                    if ((edge_seen >> st & 1) && !mbar_wait(&B.edge_full[st], (edge_seen >> (2 + st) & 1) ^ 1))
                        ok = false;
                    if (qn[st] > 0 && !mbar_wait(&B.q_full[st], (qn[st] - 1) & 1))
                        ok = false;
                }
                if (!ok && a.err)
                    atomicOr(a.err, KVATTN_DEVERR_WAIT_TIMEOUT);
            }
            __syncwarp();
        } else if (warp == 1) {
            // ------------------------------------------------------------- scores
            const uint64_t qdesc = smem_desc(smem_u32(smem), 16, 1024, 2);                           // K-major query boxes
            const uint64_t kdesc = smem_desc(smem_u32(smem) + (uint32_t)Lay::kKeysAt, 16, 1024, 2);  // K-major key boxes
            uint32_t t = 0;                                  // key tiles of the items before
            // phase bit i of query tile i: queries, scores taken to registers (the
            // first tile's columns are free from the start)
            uint32_t qpar = 0, fpar = 3;
            for (const Item *it; ok && (it = next_item());) {
                const int end0 = __shfl_sync(0xffffffffu, it->end0, 0), end1 = __shfl_sync(0xffffffffu, it->end1, 0);
                done_item();
                const int n0 = (end0 + kKeys - 1) / kKeys, n1 = (end1 + kKeys - 1) / kKeys, n = max(n0, n1);
#pragma unroll 1
                for (int x = 0; x < 2 * n; ++x) {
                    const int j = x >> 1, i = x & 1;
                    const int mine = i ? n1 : n0, other = i ? n0 : n1;
                    if (j >= mine)
                        continue;
                    const uint32_t st = (t + j) & 1;
                    bool in = true;
                    if (i == 0 || j >= other)                // the first of the tile's uses
                        in = mbar_wait(&B.k_full[st], ((t + j) >> 1) & 1);
                    if (j == 0) {
                        in = in && mbar_wait(&B.q_full[i], (qpar >> i) & 1);
                        qpar ^= 1u << i;
                    }
                    in = in && mbar_wait(&B.s_free[i], (fpar >> i) & 1);
                    fpar ^= 1u << i;
                    ok = __all_sync(0xffffffffu, in);
                    if (!ok)
                        break;
                    tc_fence_after();
                    // the last tile's scores only as far as a row attends (in
                    // steps of 16; what stands in the other columns is masked)
                    const int keys = min(kKeys, ((i ? end1 : end0) - j * kKeys + 15) & ~15);
                    const uint32_t idesc = (kIdescS & ~(0x3Fu << 17)) | (uint32_t)(keys >> 3) << 17 | a.negate;
                    const uint64_t qd = qdesc + (uint64_t)(i * NKB * (kQBox >> 4));
                    const uint64_t kd = kdesc + (uint64_t)(st * (Lay::kKeyTile >> 4));
#pragma unroll
                    for (int k = 0; k < 4 * NKB; ++k)
                        elect_ss(tS + i * kKeys, qd + (k / 4) * (kQBox >> 4) + (k % 4) * 2,
                                 kd + (k / 4) * (kBox >> 4) + (k % 4) * 2, idesc, k ? 1u : 0u);
                    elect_commit(&B.s_full[i]);
                    if (i == 1 || j >= other)                // the last of the tile's uses
                        elect_commit(&B.k_empty[st]);
                    if (j + 1 == mine)
                        elect_commit(&B.q_empty[i]);
                }
                t += (uint32_t)n;
            }
            finish();
        } else if (warp == 2) {
            // ---------------------------------------------------------------- P.V
            const uint64_t vdesc = smem_desc(smem_u32(smem) + (uint32_t)Lay::kValuesAt, kBox, 1024, 2);  // N-major value boxes
            uint32_t t = 0;                                  // value tiles of the items before
            uint32_t ppar = 0;                               // phase bit i: probabilities of query tile i
            for (const Item *it; ok && (it = next_item());) {
                const int end0 = __shfl_sync(0xffffffffu, it->end0, 0), end1 = __shfl_sync(0xffffffffu, it->end1, 0);
                done_item();
                const int n0 = (end0 + kKeys - 1) / kKeys, n1 = (end1 + kKeys - 1) / kKeys, n = max(n0, n1);
                // the first to store probabilities waits for all items before
                if (n > 0)
                    elect_commit(&B.p_free[n0 > 0 ? 0 : 1]);
#pragma unroll 1
                for (int x = 0; x < 2 * n; ++x) {
                    const int j = x >> 1, i = x & 1;
                    const int mine = i ? n1 : n0, other = i ? n0 : n1;
                    if (j >= mine)
                        continue;
                    const uint32_t st = (t + j) & 1;
                    bool in = true;
                    if (i == 0 || j >= other)                // the first of the tile's uses
                        in = mbar_wait(&B.v_full[st], ((t + j) >> 1) & 1);
                    in = in && mbar_wait(&B.p_full[i], (ppar >> i) & 1);
                    ppar ^= 1u << i;
                    ok = __all_sync(0xffffffffu, in);
                    if (!ok)
                        break;
                    tc_fence_after();
                    const uint64_t vd = vdesc + (uint64_t)(st * (Lay::kValueTile >> 4));
#pragma unroll
                    for (int k = 0; k < kKeys / 16; ++k)
                        if (j * kKeys + 16 * k < (i ? end1 : end0))
                            elect_ts(tO + i * kTile, tP + 8 * k, vd + (uint64_t)(k * 128), kIdescPV,
                                     (j > 0 || k > 0) ? 1u : 0u);
                    // who is next to store probabilities: the other query tile
                    // where it has this tile (1) or the next one (0) to work off,
                    // else this one while it has more; after the item's last, see
                    // the item's start
                    const int next = j + i < other ? i ^ 1 : j + 1 < mine ? i : -1;
                    if (next >= 0)
                        elect_commit(&B.p_free[next]);
                    if (i == 1 || j >= other)                // the last of the tile's uses
                        elect_commit(&B.v_empty[st]);
                    if (j + 1 == mine)
                        elect_commit(&B.o_full[i]);
                }
                t += (uint32_t)n;
            }
            finish();
        } else {
            // -------------------------------------------------------------- guard
            // Values that a row's mask leaves out have the weight 0, and 0 * NaN
            // or 0 * infinity in P.V would still spoil it.  In the tiles that
            // some row does not attend whole, rows past the sequence become 0,
            // and so do values that are not finite; their tokens are noted, and
            // the rows that do attend them add those values in the end.
            uint32_t t = 0, epar = 0;                        // value tiles of the items before; phase bits of edge_full
            for (const Item *it; ok && (it = next_item());) {
                const int n = max(it->tiles0(), it->tiles1()), nk = it->nk, all = it->all;
                uint32_t(*const bad)[kKeys / 32] = B.bad[taken % kItems];
                if (lane < kEdgeTiles * (kKeys / 32))
                    bad[lane / (kKeys / 32)][lane % (kKeys / 32)] = 0;
                __syncwarp();
                for (int j = all / kKeys; j < n; ++j) {
                    const uint32_t st = (t + j) & 1;
                    ok = __all_sync(0xffffffffu, mbar_wait(&B.edge_full[st], (epar >> st) & 1));
                    if (!ok)
                        break;
                    epar ^= 1u << st;
                    unsigned char *const v0 = smem + Lay::kValuesAt + st * Lay::kValueTile;
                    // a 16-byte piece of four rows a lane, six times at once: P.V may be waiting
                    const int tok0 = j * kKeys, ntok = min(nk - tok0, kKeys);
                    auto piece = [&](int r, int b) -> uint4 * {
                        return reinterpret_cast<uint4 *>(v0 + b * kBox + r * 128 + (lane & 7) * 16);
                    };
                    for (int r0 = max(all - tok0, 0) / 24 * 24; r0 < ntok; r0 += 24) {
                        uint4 x[6][NVB];
                        uint32_t ones = 0;
#pragma unroll
                        for (int y = 0; y < 6; ++y)
#pragma unroll
                            for (int b = 0; b < NVB; ++b)
                                x[y][b] = *piece(r0 + 4 * y + (lane >> 3), b);
#pragma unroll
                        for (int y = 0; y < 6; ++y)
#pragma unroll
                            for (int b = 0; b < NVB; ++b)
                                ones |= exponent_ones(x[y][b].x) | exponent_ones(x[y][b].y) | exponent_ones(x[y][b].z) |
                                        exponent_ones(x[y][b].w);
                        if (!__any_sync(0xffffffffu, ones != 0))
                            continue;
                        for (int y = 0; y < 6; ++y) {
                            const int r = r0 + 4 * y + (lane >> 3);
                            for (int b = 0; b < NVB; ++b) {
                                const uint4 w = *piece(r, b);
                                if (r < ntok && (exponent_ones(w.x) | exponent_ones(w.y) | exponent_ones(w.z) | exponent_ones(w.w))) {
                                    *piece(r, b) = make_uint4(finite_only(w.x), finite_only(w.y), finite_only(w.z), finite_only(w.w));
                                    atomicOr(&bad[j - all / kKeys][r >> 5], 1u << (r & 31));
                                }
                            }
                        }
                    }
                    for (int idx = lane; idx < (kKeys - ntok) * 8 * NVB; idx += 32)    // (lane & 7: the column)
                        *piece(ntok + idx / (8 * NVB), idx / 8 % NVB) = make_uint4(0, 0, 0, 0);
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0)
                        mbar_arrive(&B.v_full[st]);
                }
                t += (uint32_t)n;
                done_item();
            }
            if (!ok && lane == 0 && a.err)
                atomicOr(a.err, KVATTN_DEVERR_WAIT_TIMEOUT);
        }
    } else {
        set_regs_up<kSoftmaxRegs>();
        // ------------------------------------------------------------ softmax
        const int i = (warp >> 2) - 1;                   // query tile
        const int quarter = warp & 3;
        const int row = i * kTile + quarter * 32 + lane; // of the item
        const uint32_t lane_addr = (uint32_t)(quarter * 32) << 16;
        const uint32_t s_addr = tS + i * kKeys + lane_addr, o_addr = tO + i * kTile + lane_addr;
        const uint32_t p_addr = tP + lane_addr;
        const float c = a.scale_log2;
        uint32_t sn = 0, on = 0;                         // score tiles and outputs taken
        for (const Item *it; ok && (it = next_item());) {
            const int n = i ? it->tiles1() : it->tiles0();
            const int lim = a.causal ? min(it->nk, it->lim0 + row) : it->nk;
            const int lim_first = __shfl_sync(0xffffffffu, lim, 0);     // limits grow with the row
            float m_ref = -INFINITY, l = 0.f;
            for (int j = 0; j < n; ++j) {
                ok = __all_sync(0xffffffffu, mbar_wait(&B.s_full[i], sn & 1));
                if (!ok)
                    break;
                ++sn;
                tc_fence_after();
                const int nvalid = lim - j * kKeys;
                const bool partial = lim_first - j * kKeys < kKeys;
                float s[kKeys], mx[3];
#pragma unroll
                for (int x = 0; x < kKeys; x += 32)
                    tmem_ld32_start(s_addr + x, s + x);
#pragma unroll
                for (int x = 0; x < kKeys; x += 32)
                    tmem_ld_wait(s + x);
                // the scores are in registers: the next ones may come
                tc_fence_before();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(&B.s_free[i]);
#pragma unroll
                for (int x = 0; x < kKeys; x += 32) {
                    // raw scores: the scale is folded into the exponent's FMA
                    if (partial) {
#pragma unroll
                        for (int y = x; y < x + 32; ++y)
                            s[y] = y < nvalid ? s[y] : -INFINITY;
                    }
                    mx[x / 32] = reduce_extreme<true, 32>(s + x);
                }
                const float e = latent::fmax3(mx[0], mx[1], mx[2]);
                const float mt = e == -INFINITY ? -INFINITY : c * e;
                float alpha = 1.f;
                bool rescale = false;
                if (mt > m_ref + kRescaleThreshold) {
                    if (m_ref != -INFINITY) {
                        alpha = exp2f(m_ref - mt);
                        rescale = true;
                    }
                    m_ref = mt;
                }
                float nm = m_ref == -INFINITY ? 0.f : -m_ref;
                // Past 2^30 the reference's own rounding is 64 or more, and the
                // FMA, which has c * s exactly, would turn that into 2^64: there
                // (hardly ever) the raw maximum comes off first.
                const bool far = fabsf(nm) > kFarReference;
                if (__any_sync(0xffffffffu, far)) {
                    const float off = far && e != -INFINITY ? e : 0.f;
                    nm = far ? mt - m_ref : nm;
#pragma unroll
                    for (int y = 0; y < kKeys; ++y)
                        s[y] -= off;
                }
                float sx[4] = {0.f, 0.f, 0.f, 0.f}, sy[4] = {0.f, 0.f, 0.f, 0.f};
                uint32_t pk[kKeys / 2];
#pragma unroll
                for (int x = 0; x < kKeys / 2; ++x) {
                    float x0, x1;
                    ffma2(x0, x1, s[2 * x], s[2 * x + 1], c, c, nm, nm);
                    const float e0 = exp2_approx(x0), e1 = exp2_approx(x1);
                    fadd2(sx[x & 3], sy[x & 3], sx[x & 3], sy[x & 3], e0, e1);
                    const __nv_bfloat162 v2 = __floats2bfloat162_rn(e0, e1);
                    pk[x] = *reinterpret_cast<const uint32_t *>(&v2);
                }
                // the probabilities' columns are free, and the output holds all
                // tiles before this one, when every P.V before this tile's is
                // done; TMEM accesses are warp-wide: the warp's rows are
                // rescaled when any needs it
                ok = __all_sync(0xffffffffu, mbar_wait(&B.p_free[i], (sn - 1) & 1));
                if (!ok)
                    break;
                tc_fence_after();
                if (__any_sync(0xffffffffu, rescale)) {
                    uint32_t r[32];
#pragma unroll 1
                    for (int x = 0; x < kDv / 32; ++x) {
                        tmem_ld32(o_addr + 32 * x, r);
#pragma unroll
                        for (int y = 0; y < 32; ++y)
                            r[y] = __float_as_uint(__uint_as_float(r[y]) * alpha);
                        tmem_st32(o_addr + 32 * x, r);
                    }
                }
#pragma unroll
                for (int x = 0; x < kKeys / 2; x += 16)
                    tmem_st16_start(p_addr + x, pk + x);
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(&B.p_full[i]);
                l = l * alpha + (((sx[0] + sy[0]) + (sx[1] + sy[1])) + ((sx[2] + sy[2]) + (sx[3] + sy[3])));
            }
            if (!ok)
                break;
            if (n > 0) {
                ok = __all_sync(0xffffffffu, mbar_wait(&B.o_full[i], on & 1));
                if (!ok)
                    break;
                ++on;
                tc_fence_after();
            }
            const bool valid = row < it->nq;
            const int head = it->head;
            const long long grow = (long long)it->q0 + row;
            // values that are not finite, of tokens near the rows' ends: rare.
            // The guard's notes are read of this query tile's own edge tiles
            // alone: it was done with those before their P.V.  An item without
            // one may be stored before the guard has taken it, and the other
            // query tile's may still be written.
            const int noted = n > 0 ? n - it->all / kKeys : 0;
            static_assert(kEdgeTiles * (kKeys / 32) <= 32, "a word of the notes a lane");
            const bool any_bad =
                __any_sync(0xffffffffu, lane < noted * (kKeys / 32) &&
                                            B.bad[taken % kItems][lane / (kKeys / 32)][lane % (kKeys / 32)] != 0);
            const bool any = n > 0 && l != 0.f;          // a row without keys has l = 0 (NaN passes)
            const float inv = any ? 1.f / l : 0.f;
            const long long at = grow * a.out_token_stride + head * a.out_head_stride;
#pragma unroll 1
            for (int x = 0; x < kDv; x += 64) {
                float f[64];
                if (n > 0) {
                    tmem_ld32_start(o_addr + x, f);
                    tmem_ld32_start(o_addr + x + 32, f + 32);
                    tmem_ld_wait(f);
                    tmem_ld_wait(f + 32);
                }
#pragma unroll
                for (int y = 0; y < 64; ++y)
                    f[y] = any ? f[y] * inv : 0.f;
                if (any_bad) {
                    // P.V took them as 0: the rows that attend their tokens get them here
                    const int edge = it->all / kKeys;
                    const __nv_bfloat16 *const v0 = a.v + (long long)it->k0 * a.v_token_stride +
                                                    (head / a.heads_per_kv) * a.v_head_stride + x;
#pragma unroll 1
                    for (int e = 0; e < noted * kKeys; ++e) {
                        const int tok = edge * kKeys + e;
                        if (!(B.bad[taken % kItems][e / kKeys][e % kKeys / 32] >> (e % 32) & 1) || tok >= lim)
                            continue;
#pragma unroll
                        for (int y = 0; y < 64; y += 8) {
                            if (x + y >= a.d_v)
                                continue;
                            const uint4 u = *reinterpret_cast<const uint4 *>(v0 + tok * a.v_token_stride + y);
                            const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
                            for (int z = 0; z < 4; ++z) {
                                const uint32_t ones = exponent_ones(w[z]);
                                f[y + 2 * z] += ones & 0x8000u ? __uint_as_float(w[z] << 16) : 0.f;
                                f[y + 2 * z + 1] += ones & 0x80000000u ? __uint_as_float(w[z] & 0xffff0000u) : 0.f;
                            }
                        }
                    }
                    __syncwarp();
                }
                if (valid && x < a.d_v) {
                    if (a.out_fp32) {
                        float *const dst = static_cast<float *>(a.out) + at + x;
#pragma unroll
                        for (int y = 0; y < 64; y += 8)
                            if (x + y < a.d_v)
                                store_row<8>(dst + y, reinterpret_cast<const uint32_t *>(f + y), a.wide);
                    } else {
                        __nv_bfloat16 *const dst = static_cast<__nv_bfloat16 *>(a.out) + at + x;
#pragma unroll
                        for (int y = 0; y < 64; y += 16) {
                            uint32_t p[8];
#pragma unroll
                            for (int z = 0; z < 8; ++z) {
                                const __nv_bfloat162 v2 = __floats2bfloat162_rn(f[y + 2 * z], f[y + 2 * z + 1]);
                                p[z] = *reinterpret_cast<const uint32_t *>(&v2);
                            }
                            if (x + y + 8 < a.d_v)
                                store_row<8>(dst + y, p, a.wide);
                            else if (x + y < a.d_v)
                                store_row<4>(dst + y, p, false);
                        }
                    }
                }
                __syncwarp();
            }
            if (valid && a.lse)
                a.lse[grow * a.heads + head] = any ? (m_ref + log2f(l)) * kLn2 : -INFINITY;
            done_item();
            // the next item's first P.V overwrites the output: it follows this
            // warp's next arrival, which follows these loads
            tc_fence_before();
        }
        if (!ok && lane == 0 && a.err)
            atomicOr(a.err, KVATTN_DEVERR_WAIT_TIMEOUT);
    }
    __syncwarp();

    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 0)
        tmem_dealloc(tbase, 512);
}

struct Call {
    Maps maps;
    PrefillArgs args;
    long long most_items;
    cudaStream_t stream;
};

template <int NKB, bool ROPE, int NVB>
cudaError_t launch(const Call &c)
{
    auto kern = prefill_kernel<NKB, ROPE, NVB>;
    const size_t smem = Layout<NKB, NVB>::kBytes;
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess)
        return e;
    // the register split waits for good if the kernel is launched with fewer
    static std::atomic<bool> checked{false};
    if (!checked.load(std::memory_order_relaxed)) {
        cudaFuncAttributes at;
        const cudaError_t q = cudaFuncGetAttributes(&at, reinterpret_cast<const void *>(kern));
        if (q != cudaSuccess)
            return q;                        // asked again by the next call
        if (at.numRegs != kLaunchRegs)
            return cudaErrorInvalidConfiguration;
        checked.store(true, std::memory_order_relaxed);
    }
    const long long most = c.args.listed ? sm_count() : c.most_items;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)(c.most_items < most ? c.most_items : most));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = c.stream;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = c.args.listed ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kern, c.maps, c.args);
}

// Strides (elements) with the dense defaults filled in; false if one cannot be used.
bool strides(const int64_t *given, long long token, long long head, long long *out)
{
    out[0] = given[0] ? given[0] : token;
    out[1] = given[1] ? given[1] : head;
    for (int i = 0; i < 2; ++i)
        if (out[i] < 1 || out[i] % 8 || out[i] >= (1LL << 38))
            return false;
    return true;
}

// Tensor map of x [tokens][heads][d] in boxes of `rows` tokens x 64 columns (zeros past d and past the last token).
bool rows_map(CUtensorMap *map, const void *x, int d, int heads, long long tokens, const long long *st, int rows)
{
    const cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)heads, (cuuint64_t)tokens};
    const cuuint64_t bytes[2] = {(cuuint64_t)st[1] * 2, (cuuint64_t)st[0] * 2};
    const cuuint32_t box[3] = {64, 1, (cuuint32_t)rows};
    return encode_tiled(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(x), dims, bytes, box,
                        CU_TENSOR_MAP_SWIZZLE_128B) == CUDA_SUCCESS;
}

// Whether the plan kernel lists the tiles.  Else every item has a CTA of its
// own, and every CTA lists them: up to as many as a B200 runs at once.
bool needs_plan(const kvattn_prefill_params *p)
{
    const long long cap = ragged::tile_capacity(p->max_q_tokens, p->batch, kItemRows);
    return !ragged::small_plan(p->batch, cap) || cap * p->num_q_heads > kDefaultSMs;
}

int validate_prefill(const kvattn_prefill_params *p)
{
    if (!p || p->batch < 1 || p->num_q_heads < 1 || p->num_kv_heads < 1 || p->d_nope < 1 || p->d_rope < 0 ||
        p->d_v < 1 || p->max_q_tokens < 0 || p->max_kv_tokens < 0 || (p->causal != 0 && p->causal != 1) ||
        p->num_q_heads % p->num_kv_heads || p->num_q_nope_heads < 0 ||
        (p->num_q_nope_heads > 0 && p->num_q_heads % p->num_q_nope_heads))
        return KVATTN_ERR_INVALID_ARG;
    if (p->out_dtype != KVATTN_OUT_BF16 && p->out_dtype != KVATTN_OUT_FP32)
        return KVATTN_ERR_INVALID_ARG;
    if (p->d_nope % 8 || p->d_rope % 8 || p->d_v % 8 || p->d_nope > 128 || p->d_rope > 64 || p->d_v > 128 ||
        p->batch > ragged::kMaxBatch || p->num_q_heads > 65535 || p->max_q_tokens > ragged::kMaxRows ||
        p->max_kv_tokens > ragged::kMaxRows)
        return KVATTN_ERR_UNSUPPORTED;
    const long long cap = ragged::tile_capacity(p->max_q_tokens, p->batch, kItemRows);
    if (cap * ((p->num_q_heads + kHeadGroup - 1) / kHeadGroup * kHeadGroup) > INT32_MAX / 2)
        return KVATTN_ERR_UNSUPPORTED;
    return KVATTN_OK;
}

}  // namespace
}  // namespace kvattn

using namespace kvattn;

extern "C" int kvattn_prefill_workspace_size(const kvattn_prefill_params *p, size_t *bytes)
{
    const int st = validate_prefill(p);
    if (st)
        return st;
    if (!bytes)
        return KVATTN_ERR_INVALID_ARG;
    *bytes = !needs_plan(p) ? 0
                            : ragged::kPlanHeader + (size_t)ragged::tile_capacity(p->max_q_tokens, p->batch, kItemRows) *
                                                        sizeof(ragged::Tile);
    return KVATTN_OK;
}

extern "C" int kvattn_prefill(const kvattn_prefill_params *p, const void *q_nope, const void *q_rope,
                              const void *k_nope, const void *k_rope, const void *v, const int32_t *q_start,
                              const int32_t *kv_start, float sm_scale, void *out, float *lse, void *workspace,
                              size_t workspace_bytes, int32_t *device_error, void *stream)
{
    size_t need = 0;
    const int st = kvattn_prefill_workspace_size(p, &need);
    if (st)
        return st;
    const bool keys = p->max_kv_tokens > 0;      // without any, key and value pointers may be null
    if (!q_nope || !q_start || !kv_start || !out || (need && !workspace) || (keys && (!k_nope || !v)) ||
        (p->d_rope > 0 && (!q_rope || (keys && !k_rope))) || !isfinite(sm_scale))
        return KVATTN_ERR_INVALID_ARG;
    if (!is_aligned(q_nope, 16) || !is_aligned(q_rope, 16) || !is_aligned(k_nope, 16) || !is_aligned(k_rope, 16) ||
        !is_aligned(v, 16) || !is_aligned(out, 16) || !is_aligned(lse, 4) || !is_aligned(workspace, 256) ||
        !is_aligned(q_start, 4) || !is_aligned(kv_start, 4) || !is_aligned(device_error, 4))
        return KVATTN_ERR_MISALIGNED;
    if (workspace_bytes < need)
        return KVATTN_ERR_WORKSPACE_TOO_SMALL;
    const long long H = p->num_q_heads, KH = p->num_kv_heads, QH = p->num_q_nope_heads ? p->num_q_nope_heads : H;
    const long long tq = p->max_q_tokens, tk = p->max_kv_tokens;
    long long sq[2], sqr[2] = {8, 8}, sk[2], sv[2], so[2];
    const int64_t kr_given[2] = {p->k_rope_stride, 8};
    long long skr[2] = {8, 8};
    if (!strides(p->q_nope_stride, QH * p->d_nope, p->d_nope, sq) ||
        !strides(p->k_stride, p->d_nope, (keys ? tk : 1) * p->d_nope, sk) ||
        !strides(p->v_stride, p->d_v, (keys ? tk : 1) * p->d_v, sv) || !strides(p->out_stride, H * p->d_v, p->d_v, so) ||
        (p->d_rope > 0 && (!strides(p->q_rope_stride, H * p->d_rope, p->d_rope, sqr) || !strides(kr_given, p->d_rope, 8, skr))))
        return KVATTN_ERR_INVALID_ARG;
    if (tq == 0)
        return KVATTN_OK;

    Call c;
    Maps &m = c.maps;
    // without keys there is nothing to load: the maps only have to be well formed
    const long long rows = keys ? tk : 1;
    if (!keys)
        k_nope = v = k_rope = q_nope;
    bool fine = rows_map(&m.q, q_nope, p->d_nope, (int)QH, tq, sq, kTile) && rows_map(&m.k, k_nope, p->d_nope, (int)KH, rows, sk, kKeys) &&
                rows_map(&m.v, v, p->d_v, (int)KH, rows, sv, kKeys);
    if (fine && p->d_rope > 0) {
        fine = rows_map(&m.qr, q_rope, p->d_rope, (int)H, tq, sqr, kTile);
        const cuuint64_t dims[2] = {(cuuint64_t)p->d_rope, (cuuint64_t)rows};
        const cuuint64_t bytes[1] = {(cuuint64_t)skr[0] * 2};
        const cuuint32_t box[2] = {64, kKeys};
        fine = fine && encode_tiled(&m.kr, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void *>(k_rope), dims, bytes,
                                    box, CU_TENSOR_MAP_SWIZZLE_128B) == CUDA_SUCCESS;
    } else {
        m.qr = m.q;
        m.kr = m.k;
    }
    if (!fine)
        return KVATTN_ERR_UNSUPPORTED;

    char *ws = static_cast<char *>(workspace);
    ragged::PlanArgs pa{};
    pa.batch = p->batch;
    pa.rows_per_tile = kItemRows;
    pa.max_q = (int)tq;
    pa.max_kv = (int)tk;
    pa.capacity = (int)ragged::tile_capacity(tq, p->batch, kItemRows);
    pa.causal = p->causal;
    pa.q_start = q_start;
    pa.kv_start = kv_start;
    pa.header = reinterpret_cast<int32_t *>(ws);
    pa.tiles = reinterpret_cast<ragged::Tile *>(ws + ragged::kPlanHeader);
    pa.err = device_error;
    c.stream = static_cast<cudaStream_t>(stream);
    c.most_items = pa.capacity * H;
    const bool listed = needs_plan(p);
    cudaError_t e = listed ? ragged::launch_plan(pa, c.stream) : cudaSuccess;
    if (e != cudaSuccess)
        return launch_status(e);
    PrefillArgs &a = c.args;
    a.plan = pa;
    a.listed = listed;
    a.out = out;
    a.lse = lse;
    a.err = device_error;
    a.heads = (int)H;
    a.head_groups = (int)(H > kLastHeads ? (H - kLastHeads) / kHeadGroup : 0);
    a.heads_per_kv = (int)(H / KH);
    a.heads_per_q = (int)(H / QH);
    a.d_v = p->d_v;
    a.out_fp32 = p->out_dtype == KVATTN_OUT_FP32;
    a.causal = p->causal;
    a.wide = is_aligned(out, 32) && so[0] % (a.out_fp32 ? 8 : 16) == 0 && so[1] % (a.out_fp32 ? 8 : 16) == 0;
    a.out_token_stride = so[0];
    a.out_head_stride = so[1];
    a.v = static_cast<const __nv_bfloat16 *>(v);
    a.v_token_stride = sv[0];
    a.v_head_stride = sv[1];
    // masked scores are infinite, so a scale of 0 (every key weighs the same)
    // is taken as the smallest there is: times any finite score it is below
    // 2^-20, too small to show in a weight
    a.scale_log2 = sm_scale == 0.f ? 1.4e-45f : fabsf(sm_scale) * 1.4426950408889634f;
    a.negate = sm_scale < 0.f ? 1u << 13 : 0u;

    const int nkn = (p->d_nope + 63) / 64, nvb = (p->d_v + 63) / 64;
    const bool rope = p->d_rope > 0;
    if (nvb == 2)
        e = nkn == 2 ? (rope ? launch<3, true, 2>(c) : launch<2, false, 2>(c))
                     : (rope ? launch<2, true, 2>(c) : launch<1, false, 2>(c));
    else
        e = nkn == 2 ? (rope ? launch<3, true, 1>(c) : launch<2, false, 1>(c))
                     : (rope ? launch<2, true, 1>(c) : launch<1, false, 1>(c));
    return launch_status(e);
}
