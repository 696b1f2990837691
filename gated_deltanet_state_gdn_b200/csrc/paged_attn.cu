// paged_attn.cu -- attention of each request's last T tokens over its paged keys and values.
//
// Mathematics.  For one head of the cache the T * (Hq / H) query rows that read it are a matrix
// Q; over the tokens j in order, with x = scale log2(e) Q k_j,
//     m' = max(m, x),  l' = l 2^(m - m') + 2^(x - m'),  O' = O 2^(m - m') + 2^(x - m') v_j
// and out = O / l.  Two parts (m1, l1, O1), (m2, l2, O2) of one row join by the same rule, which
// is what lets the tokens of a row be cut anywhere.
//
// What bounds it: a key or value meets T Hq / H rows, T Hq / H operations a byte in 16 bits, and is
// read once for every 64 of them (32 where heads are wider than 128).  Up to 16 rows a head HBM is
// the bound, and warp mma keeps up with the tensor pipe 18 % busy, so tcgen05 (64 or 128 rows, of
// which one token's group would fill 1 to 16) is not used.  Measured on a B200 (copy rate 6.46
// TB/s): 243 rows of 1 to 4096 tokens, 32 heads on 8 of 128, bf16: 308 to 322 us, 6.3 to 6.6 TB/s;
// over e4m3 195 us, 5.3 TB/s, where the steps of the computing warps (conversions, warp mma) are
// nearly as long as the memory's; one row of 131072, 16 heads on 2 of 256, fp16: 55 us, 4.9 TB/s,
// 10 us of them start and join; 16 tokens a row of the first case (64 rows a head): 631 us, bound by
// the rate of warp mma, 206 TFLOP/s.
//
// Layout of the work.
//   - A unit is (request, head, block of 16 WR rows); its tokens are cut into tiles of 16 KB of
//     keys and 16 KB of values.  All tiles of all units in a row are dealt to the resident
//     blocks (two an SM) in equal runs, found on the device from the lengths: one long request
//     and many short ones fill the GPU alike, and the host reads nothing.
//   - In a block up to four warps walk the run: they look the tile's tokens up in the page table
//     and fetch their pages with TMA (boxes of as many tokens as a power of two that divides the
//     page size allows, 128-byte swizzle) into one of three stages of shared memory.
//   - Four warps share a tile: WR over blocks of 16 rows, the others over the tokens (each with
//     its own m, l, O, joined in shared memory at the end of the unit), and for 256-wide heads
//     two over the halves of the values.  They wait for a stage each for itself; no barrier of
//     the block is in the loop.
//   - A unit that lies in one block is finished there.  Parts of the others go to the workspace
//     and a second kernel joins them in the order of the tokens: no atomics, the same result in
//     every run.
#include <cudaTypedefs.h>
#include <float.h>

#include <algorithm>
#include <type_traits>
#include <cuda_runtime.h>

#include "cache.cuh"

namespace gdn_attn {

using namespace gdn_cache;
using gdn::in_range;
using sm100::ex2_approx;
using sm100::smem_u32;

constexpr int kConsumers = 128;     // threads that compute: four warps
constexpr int kThreads = 256;       // and up to four that fetch: 128 registers a thread at launch,
constexpr int kFetchRegs = 56;      // then 56 and 200
constexpr int kComputeRegs = 200;
static_assert(kFetchRegs + kComputeRegs == 2 * 128, "the block's registers, two blocks an SM");
constexpr int kHalfStage = 16384;   // bytes of keys (or values) in a stage
constexpr int kStages = 3;
constexpr int kMergeBytes = 8192;
constexpr int kAlign = 1024;        // of a stage: where the swizzle's pattern begins
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

enum Kind { kBF16 = 0, kF16 = 1, kE4M3 = 2 };

template <int KIND, int DP, int WR>
struct Cfg {
    static constexpr int ESZ = KIND == kE4M3 ? 1 : 2;
    static constexpr int RB = DP * ESZ;              // bytes of a token's row in a stage
    static constexpr int IB = RB < 128 ? RB : 128;   // bytes of a row in a box
    static constexpr int HB = RB / IB;               // boxes side by side
    static constexpr int TILE = kHalfStage / RB;     // tokens a tile
    static constexpr int WD = DP == 256 ? 2 : 1;     // warps over the values' dimensions
    static constexpr int WT = 4 / (WR * WD);         // warps over tokens
    // Warps that fetch a tile, a share of its tokens each: looking 256 tokens up takes one warp
    // longer than the memory takes for them.
    static constexpr int FETCH = TILE / 32 < 4 ? TILE / 32 : 4;
    static constexpr int FW = TILE / 32 / FETCH;     // 32 tokens each of a warp's share
    // tokens a warp takes at a time: two blocks of 16, twice the independent products, where it
    // has them and the registers hold them
    static constexpr int STEP = ESZ == 1 && DP == 64 && WT == 4 ? 64 : (ESZ == 1 || DP == 64 ? 32 : 16);
    using Mask = typename std::conditional<STEP == 64, uint64_t, uint32_t>::type;   // a bit a token
    static constexpr int NS = TILE / WT / STEP;      // such steps of a warp in a tile
    static constexpr int NX = STEP / 8;              // blocks of 8 columns of scores
    static constexpr int DW = DP / WD;               // dimensions a warp accumulates
    static constexpr int RMAX = 16 * WR;             // rows of a unit
    // Weights are 2^(x - base) with the base this far below the running maximum: those that meet
    // the values in fp16 are at most 2^15 (fp16 ends at 65504), so that fp16 holds weights down to
    // 2^-29 of the largest as normal numbers, not to 2^-14 (bf16 has the range of fp32).
    static constexpr int UP = KIND == kBF16 ? 0 : 15;
    static constexpr int SMEM = kStages * 2 * kHalfStage + kMergeBytes + kAlign;
    static_assert(WT >= 1 && NS >= 1, "four warps");
};

struct alignas(16) Desc {
    int b, h, rt, base;             // request, head, block of rows, first position
    int len, tile, nt, last;        // last: of the block's run
    int64_t place;                  // in the deal
};

struct Split {              // a unit whose parts lie in blocks [c0, c1]
    int u_lo, b, c0, c1;    // c1 < 0: nothing to join
};

// What a unit costs beside its tiles (its queries, its end), in tiles, when work is dealt out.
// 256 rows of 1 to 4096 tokens, four tokens each, with 0, 2, 3, 4: 358, 336, 320, 317 us; one token
// each over e4m3: 241, 218, 208, 205 us; equal rows do not care, few tiles in all lose with more.
constexpr int kUnitCost = 3;

// W places in a row dealt to G blocks: the first `more` get one more than the others
struct Deal {
    int64_t W;
    int each, more;
    __device__ __forceinline__ Deal(int64_t w, int G) : W(w)
    {
        if (w < ((int64_t)1 << 31)) {
            each = (int)w / G;
            more = (int)w - each * G;
        } else {
            each = (int)(w / G);
            more = (int)(w - (int64_t)each * G);
        }
    }
    __device__ __forceinline__ int64_t first(int c) const { return (int64_t)c * each + min(c, more); }
    __device__ __forceinline__ int count(int c) const { return each + (c < more); }
    __device__ __forceinline__ int owner(int64_t t) const
    {
        const int64_t long_ones = (int64_t)more * (each + 1);
        if (t < long_ones) return (int)(t / (each + 1));
        return more + (int)((t - long_ones) / each);
    }
};

// rows of the batch: slot (or -1 for padding) and length
struct RowInfo {
    int slot, len;
};

__device__ __forceinline__ RowInfo row_info(const GdnAttnArgs &a, int b, bool tell)
{
    RowInfo r;
    r.slot = a.slots ? __ldg(a.slots + b) : b;
    r.len = 0;
    if (r.slot < 0) {
        r.slot = -1;
        return r;
    }
    if (r.slot >= a.cache.rows) {
        if (tell && a.dev_status) atomicOr(a.dev_status, GDN_DEV_BAD_SLOT);
        r.slot = 0;
        return r;
    }
    const int64_t cap = (int64_t)a.cache.width * a.cache.page_size;
    const int n = __ldg(a.cache.seq_lens + r.slot);
    r.len = n < 0 ? 0 : (n > cap ? (int)cap : n);
    if (tell && r.len != n && a.dev_status) atomicOr(a.dev_status, GDN_DEV_BAD_LENGTH);
    return r;
}

// elements from the first to past the last of q
__device__ __forceinline__ int64_t q_elements(const GdnAttnArgs &a)
{
    return ((int64_t)a.B * a.T - 1) * a.q_token_stride + (a.Hq - 1) * a.q_head_stride + a.cache.head_dim;
}

// first position that some token of the request sees
__device__ __forceinline__ int first_seen(const GdnAttnArgs &a, int len)
{
    return a.window > 0 ? max(0, (int)max((int64_t)len - a.T - a.window + 1, (int64_t)0)) : 0;
}

// first position of the first tile: boxes do not cross pages
__device__ __forceinline__ int first_tile(const GdnAttnArgs &a, int len, int box)
{
    return first_seen(a, len) & ~(box - 1);
}

// places of a unit in the deal: kUnitCost, then its tiles; none if it has no tile
template <int TILE>
__device__ __forceinline__ int places_of(const GdnAttnArgs &a, int len, int box)
{
    return len > first_seen(a, len) ? kUnitCost + (len - first_tile(a, len, box) + TILE - 1) / TILE : 0;
}

// inclusive prefix sum over the block's threads; *total is the same in all.  With
// `small` the values are of one request each, at most 2^25 + kUnitCost, and a warp's sum fits 32
// bits.
__device__ __forceinline__ int64_t block_scan(int64_t x, bool small, int64_t *s, int64_t *total)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (small) {
        int y = (int)x;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int z = __shfl_up_sync(0xffffffffu, y, d);
            if (lane >= d) y += z;
        }
        x = y;
    } else {
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int64_t z = __shfl_up_sync(0xffffffffu, x, d);
            if (lane >= d) x += z;
        }
    }
    if (lane == 31) s[warp] = x;
    __syncthreads();
    int64_t all = 0;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) {
        if (w < warp) x += s[w];
        all += s[w];
    }
    *total = all;
    __syncthreads();
    return x;
}

// Wait for a phase of a barrier, about a second at most: then GDN_DEV_TIMEOUT is set and the warps
// of the block leave at their next wait that has to wait (its outputs are invalid).  Whether the
// phase came, for the whole warp.
__device__ __forceinline__ bool wait_phase(uint32_t bar, uint32_t parity, volatile int *abort, int32_t *status)
{
    bool came = sm100::mbar_try_wait(bar, parity);
    if (!came) {
        const long long start = clock64();
        while (!(came = sm100::mbar_try_wait(bar, parity)) && !*abort)
            if (clock64() - start > (1ll << 31)) {
                *abort = 1;
                if (status) atomicOr(status, GDN_DEV_TIMEOUT);
            }
    }
    return __all_sync(0xffffffffu, came);
}

// What the weights of a row with running maximum m are relative to.  Any base does as long as m, l
// and O of a part go by the same; without a maximum (-inf) it is finite, so that scores of -inf
// weigh nothing.
template <class C>
__device__ __forceinline__ float base_of(float m)
{
    return fmaxf(m, -FLT_MAX) - C::UP;
}

// two weights for a product in 16 bits (where scores come in steps of 8 or 16 the base may be rounded
// to 16 below the maximum, and that weight, 2^16, becomes 65504: 2^-11 of it less)
template <bool BF16>
__device__ __forceinline__ uint32_t pack_weights(float lo, float hi)
{
    if constexpr (BF16) {
        return gdn::pack_bf16x2(lo, hi);
    } else {
        uint32_t d;
        asm("cvt.rn.satfinite.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
        return d;
    }
}

__device__ __forceinline__ uint32_t pack_out(bool bf16, float lo, float hi)
{
    return bf16 ? gdn::pack_bf16x2(lo, hi) : pack_f16x2(lo, hi);
}

// byte of 16-byte piece c of token r in the keys or values of a stage
template <class C>
__device__ __forceinline__ int piece(int r, int c)
{
    if constexpr (C::IB == 64) return r * 64 + (c ^ ((r >> 1) & 3)) * 16;
    return (c >> 3) * (C::TILE * 128) + r * 128 + ((c & 7) ^ (r & 7)) * 16;
}

// Token (of the step's) that column `col` of the n-th block of 8 stands for.  In 8 bits the order
// is such that the four tokens of a byte-wise transposed load are the two pairs that a thread's
// probabilities of two blocks make, that the two tokens whose keys eight threads read together
// lie in different banks, and so do the eight whose values are loaded together.
template <class C>
__device__ __forceinline__ int token_of(int n, int col)
{
    if constexpr (C::ESZ == 2) return n * 8 + col;
    const int i = n & 1, j = col & 1, t = col >> 1;
    return 16 * (n >> 1) + (t >> 1) * 8 + (t & 1) * 2 + (C::RB == 64 ? j + 4 * i : 4 * j + i);
}

template <int KIND, int DP, int WR>
__global__ void __launch_bounds__(kThreads, 2)
paged_attn_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                  const __grid_constant__ GdnAttnArgs a, const int box, const int RT, Split *const splits,
                  const int n_splits, float2 *const part_ml, float *const part_o)
{
    using C = Cfg<KIND, DP, WR>;
    constexpr int TILE = C::TILE;
    constexpr bool BF16 = KIND == kBF16;
    extern __shared__ unsigned char smem_raw[];
    unsigned char *const smem = smem_raw + (kAlign - (smem_u32(smem_raw) & (kAlign - 1))) % kAlign;
    float4 *const s_merge = reinterpret_cast<float4 *>(smem + kStages * 2 * kHalfStage);
    __shared__ __align__(8) uint64_t s_full[kStages], s_empty[kStages];
    __shared__ int64_t s_sum[kThreads / 32];
    __shared__ int s_found[3];
    __shared__ Desc s_desc[kStages];
    __shared__ uint32_t s_valid[kStages][TILE / 32];
    __shared__ float4 s_stat[2][32];
    __shared__ __align__(8) uint64_t s_meet;    // of the warps that compute
    __shared__ __align__(8) uint64_t s_read;    // a unit's joining has been read
    __shared__ volatile int s_abort;

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int c = blockIdx.x, G = gridDim.x;
    const gdn_paged_cache &kv = a.cache;
    const int H = kv.heads, D = kv.head_dim, group = a.Hq / H, rows_all = a.T * group;
    const int U = H * RT;                              // units of a request
    const bool by_unit = (int64_t)a.B * U <= n_splits; // one Split a unit, else one a block
    const uint32_t full0 = smem_u32(s_full), empty0 = smem_u32(s_empty);

    launch_dependents();
    if (tid == 0) {
        s_abort = 0;
        for (int s = 0; s < kStages; ++s) {
            sm100::mbar_init(full0 + 8 * s, C::FETCH);
            sm100::mbar_init(empty0 + 8 * s, kConsumers / 32);
        }
        sm100::mbar_init(smem_u32(&s_meet), kConsumers / 32);
        sm100::mbar_init(smem_u32(&s_read), WR * C::WD);
        sm100::fence_mbar_init();
        sm100::prefetch_tmap(&kmap);
        sm100::prefetch_tmap(&vmap);
        if (!by_unit && in_range(c, 1, n_splits, a.dev_status)) splits[c].c1 = -1;
    }

    // ---- this block's run of places
    int64_t S = 0, incl0;      // of the batch, a unit of each request; up to this thread's
    const int nt0 = tid < a.B ? places_of<TILE>(a, row_info(a, tid, c == 0).len, box) : 0;
    {
        int64_t mine = nt0;
        for (int b = tid + kThreads; b < a.B; b += kThreads)
            mine += places_of<TILE>(a, row_info(a, b, c == 0).len, box);
        incl0 = block_scan(mine, a.B <= kThreads, s_sum, &S);
    }
    const Deal deal(S * U, G);
    const int64_t t0 = deal.first(c);
    const int n_places = deal.count(c);

    // the request, unit and place where it begins
    if (n_places > 0) {
        int64_t before = 0;
        for (int b0 = 0; b0 < a.B; b0 += kThreads) {
            const int b = b0 + tid;
            int nt = nt0;
            int64_t incl = incl0, all = S;
            if (a.B > kThreads) {       // the sum above was over more than a request a thread
                nt = b < a.B ? places_of<TILE>(a, row_info(a, b, false).len, box) : 0;
                incl = before + block_scan(nt, true, s_sum, &all);
            }
            if (nt > 0 && t0 >= (incl - nt) * U && t0 < incl * U) {
                const int64_t past = t0 - (incl - nt) * U;
                s_found[0] = b;
                s_found[1] = (int)(past / nt);
                s_found[2] = (int)(past % nt);
            }
            before += all;
            if (t0 < before * U) break;
        }
    }
    __syncthreads();
    // a run that ends before the first tile of the unit it begins in has none
    const bool idle = n_places == 0 || n_places <= kUnitCost - s_found[2];

    if (warp >= kConsumers / 32) {
        // ================================================================ the warps that fetch
        registers_down<kFetchRegs>();
        const int fw = warp - kConsumers / 32;
        if (idle || fw >= C::FETCH) return;
        int cb = s_found[0], win = cb;     // request; lane i knows about request win + i
        RowInfo mine = cb + lane < a.B ? row_info(a, cb + lane, false) : RowInfo{-1, 0};
        int len = __shfl_sync(0xffffffffu, mine.len, 0), slot = __shfl_sync(0xffffffffu, mine.slot, 0);
        int cnt = places_of<TILE>(a, len, box);
        int cu = s_found[1], cp = s_found[2];
        int64_t place = t0;
        int i = 0;
        for (bool more = true; more; ++i) {
            if (cp < kUnitCost) {               // the run holds a tile of the unit, or it had ended
                place += kUnitCost - cp;
                cp = kUnitCost;
            }
            const int st = i % kStages, ct = cp - kUnitCost;
            const int left = (int)(t0 + n_places - place) - 1;      // places after this tile's
            more = left > (cp + 1 == cnt ? kUnitCost : 0);
            const int base = first_tile(a, len, box) + ct * TILE, lo = first_seen(a, len);
            const int h = cu / RT;
            // a lane looks up a token of each 32
            const int32_t *const row = kv.block_table + (int64_t)slot * kv.table_stride;
            const int first = base + fw * C::FW * 32 + lane;
            int page[C::FW];
#pragma unroll
            for (int w = 0; w < C::FW; ++w) {
                const int j = first + w * 32;
                const int pg = (int)((uint32_t)j / (uint32_t)kv.page_size);
                page[w] = j < len && in_range(pg, 1, kv.width, a.dev_status) ? __ldg(row + pg) : -1;
            }
            if (i >= kStages && !wait_phase(empty0 + 8 * st, ((i / kStages) & 1) ^ 1, &s_abort, a.dev_status)) break;
            int boxes = 0;
#pragma unroll
            for (int w = 0; w < C::FW; ++w) {
                const int j = first + w * 32;
                const bool ok = (uint32_t)page[w] < (uint32_t)kv.num_pages;
                if (j < len && j >= lo && !ok && a.dev_status) atomicOr(a.dev_status, GDN_DEV_BAD_PAGE);
                const uint32_t seen = __ballot_sync(0xffffffffu, ok && j >= lo);
                if (lane == 0) s_valid[st][fw * C::FW + w] = seen;
                if (!ok || ((j - base) & (box - 1)) != 0) page[w] = -1;    // not first of a box
                boxes += __popc(__ballot_sync(0xffffffffu, page[w] >= 0));
            }
            if (lane == 0) {
                if (fw == 0) {
                    Desc d;
                    d.b = cb; d.h = h; d.rt = cu - h * RT; d.base = base; d.len = len; d.tile = ct; d.nt = cnt - kUnitCost;
                    d.last = !more; d.place = place;
                    s_desc[st] = d;
                }
                const uint32_t extra = place == kUnitCost && fw == 0 && gdn::test_stall_requested(a.dev_status) ? 16 : 0;
                sm100::mbar_arrive_expect_tx(full0 + 8 * st, (uint32_t)(boxes * box * C::RB * 2) + extra);
            }
            __syncwarp();
            const uint32_t ks = smem_u32(smem + st * 2 * kHalfStage), vs = ks + kHalfStage;
#pragma unroll
            for (int w = 0; w < C::FW; ++w)
                if (page[w] >= 0) {
                    const int j = first + w * 32;
                    const uint32_t to = (j - base) * C::IB;
                    const int at = (int)((uint32_t)j % (uint32_t)kv.page_size);
#pragma unroll
                    for (int k = 0; k < C::HB; ++k) {
                        tma_load_4d(ks + k * TILE * 128 + to, &kmap, full0 + 8 * st, k * 128 / C::ESZ, at, h, page[w]);
                        tma_load_4d(vs + k * TILE * 128 + to, &vmap, full0 + 8 * st, k * 128 / C::ESZ, at, h, page[w]);
                    }
                }
            // a unit's query rows are brought near while its first tile is on the way
            if (i == 0 || ct == 0) {
                const int r0 = (cu - h * RT) * C::RMAX, lines = (D * 2 + 127) / 128;
                const int n = min(C::RMAX, rows_all - r0) * lines;
                for (int k = fw * 32 + lane; k < n; k += C::FETCH * 32) {
                    const int r = r0 + k / lines, t = r / group;
                    if constexpr (gdn::kChecked)
                        if (!in_range(((int64_t)cb * a.T + t) * a.q_token_stride +
                                          (int64_t)(h * group + r - t * group) * a.q_head_stride + (k % lines) * 64,
                                      2, q_elements(a), a.dev_status))
                            continue;
                    touch_l1(static_cast<const uint16_t *>(a.q) + ((int64_t)cb * a.T + t) * a.q_token_stride +
                             (int64_t)(h * group + r - t * group) * a.q_head_stride + (k % lines) * 64);
                }
            }
            // the next place of the run (past the last one the cursor may stand anywhere)
            ++place;
            if (++cp == cnt) {
                cp = 0;
                if (++cu == U) {
                    cu = 0;
                    do {
                        if (++cb >= a.B) break;
                        if (cb - win >= 32) {
                            win = cb;
                            mine = cb + lane < a.B ? row_info(a, cb + lane, false) : RowInfo{-1, 0};
                        }
                        len = __shfl_sync(0xffffffffu, mine.len, cb - win);
                        slot = __shfl_sync(0xffffffffu, mine.slot, cb - win);
                        cnt = places_of<TILE>(a, len, box);
                    } while (cnt == 0);
                }
            }
        }
        // no copy may land after the block is gone, whoever gives up: a wait for the last ones, far
        // longer than they take and not for good
        const long long start = clock64();
        for (int k = i > kStages ? i - kStages : 0; k < i; ++k)
            while (!sm100::mbar_try_wait(full0 + 8 * (k % kStages), (k / kStages) & 1) &&
                   clock64() - start < (1ll << 26)) {
            }
        return;
    }

    // ==================================================================== the warps that compute
    registers_up<kComputeRegs>();
    // requests with nothing to see: zeros for a row of the cache, nothing (or zeros) for padding
    for (int b = c; b < a.B; b += G) {
        const RowInfo ri = row_info(a, b, false);
        if (places_of<TILE>(a, ri.len, box) > 0) continue;
        if (by_unit)
            for (int u = tid; u < U; u += kConsumers)
                if (in_range((int64_t)b * U + u, 1, n_splits, a.dev_status))
                    splits[(int64_t)b * U + u].c1 = -1;
        if (ri.slot < 0 && !a.zero_padding) continue;
        const int64_t rows = (int64_t)a.T * a.Hq, words = rows * D / 2;
        const int64_t total = (int64_t)a.B * rows;
        uint32_t *const o = static_cast<uint32_t *>(a.out) + b * words;
        if (in_range(b * words, words, total * D / 2, a.dev_status))
            for (int64_t i = tid; i < words; i += kConsumers) o[i] = 0u;
        if (a.lse && in_range(b * rows, rows, total, a.dev_status))
            for (int64_t i = tid; i < rows; i += kConsumers) a.lse[b * rows + i] = -INFINITY;
    }

    if (idle) return;

    const uint32_t meet = smem_u32(&s_meet);
    uint32_t met = 0;       // parity of the next meeting
    // all four warps are here (or, after a timeout, need not be)
    bool together = true;
    auto meet_all = [&]() {
        __syncwarp();
        if (lane == 0) sm100::mbar_arrive(meet);
        together = wait_phase(meet, met, &s_abort, a.dev_status) && together;
        met ^= 1;
    };
    const int tq = lane & 3, lr = lane >> 2;
    const int wr = warp % WR, wd = (warp / WR) % C::WD, wt = warp / (WR * C::WD);
    // ---- the run
    constexpr int E = 2, NX = C::NX;
    float m[E], l[E], o[C::DW / 8][4];      // rows lr (and lr + 8) of the warp's
    uint32_t qf[DP / 16][4];
    float xs[E];                            // what a raw score is multiplied by
    int hi[E], lo[E];                       // a row sees lo < j <= hi
    int seg_tile = 0;                       // where the unit's part in this block began
    int units = 0;                          // done
#pragma unroll 1
    for (int i = 0;; ++i) {
        const int st = i % kStages;
        if (!wait_phase(full0 + 8 * st, (i / kStages) & 1, &s_abort, a.dev_status)) break;
        const Desc d = s_desc[st];
        const int h = d.h, rt = d.rt;
        if constexpr (gdn::kChecked)        // of the request, and of the heads (and their scales)
            if (!in_range(d.b, 1, a.B, a.dev_status) || !in_range(h, 1, H, a.dev_status)) break;

        if (i == 0 || d.tile == 0) {        // a unit begins: its query rows
            seg_tile = d.tile;
            const float x2 = a.scale * kLog2e * (KIND == kE4M3 && kv.k_scale ? __ldg(kv.k_scale + h) : 1.f);
            const uint32_t *qr[E];
            bool has[E];
#pragma unroll
            for (int e = 0; e < E; ++e) {
                m[e] = -INFINITY;
                l[e] = 0.f;
                xs[e] = x2;
                const int r = rt * C::RMAX + wr * 16 + lr + 8 * e;
                has[e] = r < rows_all;
                const int t = has[e] ? r / group : 0, g = has[e] ? r - t * group : 0;
                qr[e] = reinterpret_cast<const uint32_t *>(
                    static_cast<const uint16_t *>(a.q) + ((int64_t)d.b * a.T + t) * a.q_token_stride +
                    (int64_t)(h * group + g) * a.q_head_stride);
                if constexpr (gdn::kChecked)
                    has[e] = has[e] && in_range(reinterpret_cast<const uint16_t *>(qr[e]) - static_cast<const uint16_t *>(a.q),
                                                D, q_elements(a), a.dev_status);
                const int64_t pos = (int64_t)d.len - a.T + t;
                hi[e] = has[e] ? (int)pos : -1;
                lo[e] = has[e] && a.window > 0 && pos >= a.window ? (int)(pos - a.window) : -1;
            }
#pragma unroll
            for (int n = 0; n < C::DW / 8; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[n][e] = 0.f;
            // (rows 8 to 15 of a warp, where the unit has none, cost nothing but zeros)
            const bool two = rows_all - rt * C::RMAX - wr * 16 > 8;
            if constexpr (KIND != kE4M3) {
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    if (e == 0 || two) {
#pragma unroll
                        for (int k = 0; k < DP / 8; ++k) {
                            const int dd = k * 8 + 2 * tq;
                            qf[k / 2][e + 2 * (k & 1)] = has[e] && dd < D ? __ldg(qr[e] + dd / 2) : 0u;
                        }
                    } else {
#pragma unroll
                        for (int k = 0; k < DP / 8; ++k) qf[k / 2][e + 2 * (k & 1)] = 0u;
                    }
                }
            } else {
                // Rows of q become halves, scaled by the power of two that brings the largest
                // element to [2^7, 2^8): a bf16 or fp16 number down to 2^-22 of it is kept
                // exactly, smaller ones to 2^-33 of it.  The order of the dimensions is that of
                // the keys' 16-byte pieces: thread tq of a quad has 16 of each 64 in a row.
                auto load = [&](auto bf16) {
                    auto value = [&](uint32_t x, int half) {
                        if constexpr (decltype(bf16)::value)
                            return __uint_as_float(half ? x & 0xffff0000u : x << 16);
                        else
                            return __half2float(__ushort_as_half((unsigned short)(half ? x >> 16 : x & 0xffffu)));
                    };
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        if (e == 1 && !two) {
#pragma unroll
                            for (int k = 0; k < DP / 8; ++k) qf[k / 2][e + 2 * (k & 1)] = 0u;
                            break;
                        }
                        auto pair = [&](int s, int k) {
                            const int dd = s * 64 + tq * 16 + 2 * k;
                            return has[e] && dd < D ? __ldg(qr[e] + dd / 2) : 0u;
                        };
                        // two passes over the row, so that it need not be held twice
                        float top = 0.f;
#pragma unroll
                        for (int s = 0; s < DP / 64; ++s)
#pragma unroll
                            for (int k = 0; k < 8; ++k) {
                                const uint32_t w = pair(s, k);
                                top = fmaxf(top, fmaxf(fabsf(value(w, 0)), fabsf(value(w, 1))));
                            }
                        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
                        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
                        const int ex = min(max((int)(__float_as_uint(top) >> 23), 8), 254);
                        const float up = __uint_as_float((uint32_t)(261 - ex) << 23);
                        xs[e] = x2 * __uint_as_float((uint32_t)(ex - 7) << 23);
#pragma unroll
                        for (int s = 0; s < DP / 64; ++s)
#pragma unroll
                            for (int k = 0; k < 8; ++k) {
                                const uint32_t w = pair(s, k);
                                qf[s * 4 + k / 2][e + 2 * (k & 1)] = pack_f16x2(value(w, 0) * up, value(w, 1) * up);
                            }
                    }
                };
                if (a.q_bf16)
                    load(std::true_type{});
                else
                    load(std::false_type{});
            }
        }

        const uint32_t ks = smem_u32(smem + st * 2 * kHalfStage), vs = ks + kHalfStage;
        const int see_all = d.len - a.T;                                     // j <= this: causally seen by all rows
        const int64_t see_from = a.window > 0 ? (int64_t)d.len - a.window : 0;   // j >= this: in every window
#pragma unroll 1
        for (int s = 0; s < C::NS; ++s) {
            const int tok = (s * C::WT + wt) * C::STEP;
            using Mask = typename C::Mask;
            constexpr Mask kAll = (Mask)~(Mask)0 >> (sizeof(Mask) * 8 - C::STEP);
            Mask ok = (s_valid[st][tok >> 5] >> (tok & 31)) & kAll;
            if constexpr (C::STEP == 64) ok |= (Mask)s_valid[st][(tok >> 5) + 1] << 32;
            if (ok == 0) continue;
            const int j0 = d.base + tok;
            const bool ragged = j0 + C::STEP - 1 > see_all || j0 < see_from;    // rows may see different tokens

            // scores of the rows and STEP tokens
            float x[NX][4] = {};
            if constexpr (KIND != kE4M3) {
                // four chains of products: two blocks of 16 tokens, or even and odd steps of one
                const int r = tok + (lane & 7) + ((lane >> 4) << 3);
                float y[NX][4] = {};
#pragma unroll
                for (int k = 0; k < DP / 16; ++k)
#pragma unroll
                    for (int u = 0; u < NX / 2; ++u) {
                        uint32_t b[4];
                        ldmatrix_x4(b, ks + piece<C>(r + 16 * u, 2 * k + ((lane >> 3) & 1)));
                        float(&x0)[4] = NX == 2 && (k & 1) ? y[0] : x[2 * u];
                        float(&x1)[4] = NX == 2 && (k & 1) ? y[1] : x[2 * u + 1];
                        mma_16816<BF16>(x0, qf[k][0], qf[k][1], qf[k][2], qf[k][3], b[0], b[1]);
                        mma_16816<BF16>(x1, qf[k][0], qf[k][1], qf[k][2], qf[k][3], b[2], b[3]);
                    }
                if constexpr (NX == 2) {
#pragma unroll
                    for (int n = 0; n < 2; ++n)
#pragma unroll
                        for (int k = 0; k < 4; ++k) x[n][k] += y[n][k];
                }
            } else {
#pragma unroll
                for (int q4 = 0; q4 < DP / 64; ++q4) {
                    uint32_t w[NX][4];
#pragma unroll
                    for (int n = 0; n < NX; ++n) {
                        const uint4 v = lds128(ks + piece<C>(tok + token_of<C>(n, lr), q4 * 4 + tq));
                        w[n][0] = v.x; w[n][1] = v.y; w[n][2] = v.z; w[n][3] = v.w;
                    }
#pragma unroll
                    for (int k = 0; k < 4; ++k)
#pragma unroll
                        for (int n = 0; n < NX; ++n) {
                            const uint32_t(&q)[4] = qf[q4 * 4 + k];
                            uint32_t b0, b1;
                            e4m3x4_to_f16x2(w[n][k], b0, b1);
                            mma_16816<false>(x[n], q[0], q[1], q[2], q[3], b0, b1);
                        }
                }
            }
#pragma unroll
            for (int n = 0; n < NX; ++n)
#pragma unroll
                for (int k = 0; k < 2 * E; ++k) x[n][k] *= xs[k >> 1];
            if (ok != kAll || ragged) {
#pragma unroll
                for (int n = 0; n < NX; ++n)
#pragma unroll
                    for (int k = 0; k < 2 * E; ++k) {
                        const int t = token_of<C>(n, 2 * tq + (k & 1)), j = j0 + t;
                        const bool seen = ((ok >> t) & 1) && j <= hi[k >> 1] && j > lo[k >> 1];
                        if (!seen) x[n][k] = -INFINITY;
                    }
            }

            // running maximum and sum
            float mn[E];
            bool up = false;
#pragma unroll
            for (int e = 0; e < E; ++e) {
                float t = fmaxf(x[0][2 * e], x[0][2 * e + 1]);
#pragma unroll
                for (int n = 1; n < NX; ++n) t = fmaxf(t, fmaxf(x[n][2 * e], x[n][2 * e + 1]));
                t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 1));
                t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 2));
                mn[e] = fmaxf(m[e], t);
                up = up || mn[e] > m[e];
            }
            if (__any_sync(0xffffffffu, up)) {
                float f[E];
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    f[e] = ex2_approx(base_of<C>(m[e]) - base_of<C>(mn[e]));
                    m[e] = mn[e];
                    l[e] *= f[e];
                }
#pragma unroll
                for (int n = 0; n < C::DW / 8; ++n)
#pragma unroll
                    for (int k = 0; k < 4; ++k) o[n][k] *= f[(k >> 1) % E];
            }
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const float mm = base_of<C>(m[e]);
#pragma unroll
                for (int n = 0; n < NX; ++n)
#pragma unroll
                    for (int k = 2 * e; k < 2 * e + 2; ++k) {
                        x[n][k] = ex2_approx(x[n][k] - mm);
                        l[e] += x[n][k];
                    }
            }

            if (ok != kAll) {
                // what was fetched along with the tokens (or left in the stage) is no value:
                // nothing, so that weight 0 times it is 0
                for (int t = lane / C::HB / 4; t < C::STEP; t += 32 / C::HB / 4)
                    if (!((ok >> t) & 1))
                        for (int p = lane % (C::HB * 4); p < C::RB / 16; p += C::HB * 4)
                            sts128_zero(vs + piece<C>(tok + t, p));
                sm100::fence_proxy_async_smem();
                __syncwarp();
            }
            // Times the values: the weights rounded to the 16-bit type of the product (off by 2^-8
            // of it at most for bf16, 2^-11 for fp16, to nearest, so over many tokens well below
            // the rounding of the output; in fp16 those below 2^-29 of the row's largest by 2^-40
            // of that one); l keeps them unrounded.
            auto values = [&](auto clean) {
                // `clean`: infinities and NaN are taken out before the product, where a row must
                // not meet the values of a token that another row sees
                bool bad = false;
                auto scrub = [&](uint32_t w) {
                    if constexpr (!decltype(clean)::value) {
                        return w;
                    } else if constexpr (KIND == kE4M3) {
                        const uint32_t nan = __vcmpeq4(w & 0x7f7f7f7fu, 0x7f7f7f7fu);
                        bad = bad || nan;
                        return w & ~nan;
                    } else {
                        const uint32_t nan = __vcmpeq2(w & (BF16 ? 0x7f807f80u : 0x7c007c00u),
                                                       BF16 ? 0x7f807f80u : 0x7c007c00u);
                        bad = bad || nan;
                        return w & ~nan;
                    }
                };
                uint32_t p[NX / 2][4];
#pragma unroll
                for (int u = 0; u < NX / 2; ++u)
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        p[u][k] = pack_weights<BF16>(x[2 * u + k / 2][2 * (k & 1)], x[2 * u + k / 2][2 * (k & 1) + 1]);
                if constexpr (KIND != kE4M3) {
#pragma unroll
                    for (int u = 0; u < NX / 2; ++u) {
                        const int vr = tok + 16 * u + (lane & 15);
#pragma unroll
                        for (int n = 0; n < C::DW / 8; n += 2) {
                            uint32_t b[4];
                            ldmatrix_x4_trans(b, vs + piece<C>(vr, wd * (C::DW / 8) + n + (lane >> 4)));
                            mma_16816<BF16>(o[n], p[u][0], p[u][1], p[u][2], p[u][3], scrub(b[0]), scrub(b[1]));
                            mma_16816<BF16>(o[n + 1], p[u][0], p[u][1], p[u][2], p[u][3], scrub(b[2]), scrub(b[3]));
                        }
                    }
                } else {
#pragma unroll
                    for (int v = 0; v < NX / 4; ++v) {      // 32 tokens
                        const int vr = tok + 32 * v + token_of<C>(2 * (lane >> 4) + ((lane >> 1) & 1),
                                                                  2 * ((lane >> 2) & 3) + (lane & 1));
#pragma unroll
                        for (int n = 0; n < C::DW / 8; n += 2) {
                            uint32_t b[4];
                            ldmatrix_b8_x2_trans(b, vs + piece<C>(vr, wd * (C::DW / 16) + n / 2));
#pragma unroll
                            for (int u = 0; u < 2; ++u)
#pragma unroll
                                for (int k = 0; k < 2; ++k) {
                                    const uint32_t(&q)[4] = p[2 * v + u];
                                    uint32_t b0, b1;
                                    e4m3x4_to_f16x2(scrub(b[2 * u + k]), b0, b1);
                                    mma_16816<false>(o[n + k], q[0], q[1], q[2], q[3], b0, b1);
                                }
                        }
                    }
                }
                return bad;
            };
            if (!ragged || a.T == 1) {
                values(std::false_type{});
            } else if (__any_sync(0xffffffffu, values(std::true_type{}))) {
                // the taken-out values, for the rows that do see them
#pragma unroll
                for (int nj = 0; nj < NX; ++nj)
#pragma unroll 1
                    for (int jj = 0; jj < 8; ++jj) {
                        const int src = (lane & ~3) | (jj >> 1), tj = token_of<C>(nj, jj), j = j0 + tj;
                        float p[E];
#pragma unroll
                        for (int e = 0; e < E; ++e)
                            p[e] = __shfl_sync(0xffffffffu, (jj & 1) ? x[nj][2 * e + 1] : x[nj][2 * e], src);
                        if (!((ok >> tj) & 1)) continue;
                        const unsigned char *const vb = smem + st * 2 * kHalfStage + kHalfStage;
#pragma unroll
                        for (int n = 0; n < C::DW / 8; ++n)
#pragma unroll
                            for (int k = 0; k < 2; ++k) {
                                const int at = (wd * C::DW + n * 8 + 2 * tq + k) * C::ESZ;
                                const unsigned char *const e0 = vb + piece<C>(tok + tj, at / 16) + at % 16;
                                float v;
                                if constexpr (KIND == kBF16)
                                    v = __uint_as_float((uint32_t)*reinterpret_cast<const uint16_t *>(e0) << 16);
                                else if constexpr (KIND == kF16)
                                    v = __half2float(__ushort_as_half(*reinterpret_cast<const uint16_t *>(e0)));
                                else
                                    v = (*e0 & 0x7f) == 0x7f ? __uint_as_float(0x7fc00000u) : 0.f;
                                if (isfinite(v)) continue;
#pragma unroll
                                for (int e = 0; e < E; ++e)
                                    if (j <= hi[e] && j > lo[e]) o[n][2 * e + k] += p[e] * v;
                            }
                    }
            }
        }
        __syncwarp();
        if (lane == 0) sm100::mbar_arrive(empty0 + 8 * st);

        if (d.tile == d.nt - 1 || d.last) {   // the unit, or its part here, is done
#pragma unroll
            for (int e = 0; e < E; ++e) {
                l[e] += __shfl_xor_sync(0xffffffffu, l[e], 1);
                l[e] += __shfl_xor_sync(0xffffffffu, l[e], 2);
                m[e] = base_of<C>(m[e]);        // what l and O are relative to, from here on
            }
            if constexpr (KIND == kE4M3) {
                float vsc = kv.v_scale ? __ldg(kv.v_scale + h) : 1.f;
                // O may be 2^24 times the tokens.  Where that would take the scaled sum past the range
                // of fp32 (scales above 2^64), the 2^15 of the weights go first, out of l too.
                if (fabsf(vsc) > 0x1p64f) {
                    vsc *= 0x1p-15f;
#pragma unroll
                    for (int e = 0; e < E; ++e) {
                        l[e] *= 0x1p-15f;
                        m[e] += C::UP;
                    }
                }
#pragma unroll
                for (int n = 0; n < C::DW / 8; ++n)
#pragma unroll
                    for (int k = 0; k < 4; ++k) o[n][k] *= vsc;
            }
            // The other warps of the same rows and dimensions join into wt = 0, halving their
            // number; rows 8 to 15 only where the unit has them.  A writer's 4 KB are those that it
            // has just read itself, or of the unit before, whose last reader says so (s_read).
            constexpr int kQ = C::DW / 16;              // float4 of a row's
            const int halves = rows_all - rt * C::RMAX > 8 ? 2 : 1;
            const bool two = rows_all - rt * C::RMAX - wr * 16 > 8;
            if (C::WT > 1 && wt > 0)
                together = wait_phase(smem_u32(&s_read), units & 1 ^ 1, &s_abort, a.dev_status) && together;
            float fj[2][2][2];      // weights of the two parts, by step and row
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                if (C::WT == 1 || e >= halves) break;
                if (e == 1) meet_all();             // the first halves have been read
#pragma unroll
                for (int half = C::WT / 2; half > 0; half >>= 1) {
                    // four warps: 2 and 3 write places 0 and 1 for 0 and 1, then 1 writes place 1 for 0
                    const int at = C::WT == 4 && half == 1 ? 1 : warp % (half * WR * C::WD);
                    float4 *const buf = s_merge + at * kQ * 32 + lane;
                    float4 *const stat = &s_stat[at][lane];
                    float(&f)[2][2] = fj[half / 2];
                    if (wt >= half && wt < 2 * half && (e == 0 || two)) {
                        if (e == 0) *stat = make_float4(m[0], m[1], l[0], l[1]);
#pragma unroll
                        for (int k = 0; k < kQ; ++k)
                            buf[k * 32] = make_float4(o[2 * k][2 * e], o[2 * k][2 * e + 1], o[2 * k + 1][2 * e],
                                                      o[2 * k + 1][2 * e + 1]);
                    }
                    meet_all();
                    if (wt < half && (e == 0 || two)) {
                        if (e == 0) {
                            const float4 y = *stat;
#pragma unroll
                            for (int r = 0; r < 2; ++r) {
                                const float ym = r ? y.y : y.x, yl = r ? y.w : y.z;
                                const float mx = fmaxf(m[r], ym), ms = mx == -INFINITY ? 0.f : mx;
                                f[r][0] = ex2_approx(m[r] - ms);
                                f[r][1] = ex2_approx(ym - ms);
                                m[r] = mx;
                                l[r] = l[r] * f[r][0] + yl * f[r][1];
                            }
                        }
#pragma unroll
                        for (int k = 0; k < kQ; ++k) {
                            const float4 y = buf[k * 32];
                            o[2 * k][2 * e] = o[2 * k][2 * e] * f[e][0] + y.x * f[e][1];
                            o[2 * k][2 * e + 1] = o[2 * k][2 * e + 1] * f[e][0] + y.y * f[e][1];
                            o[2 * k + 1][2 * e] = o[2 * k + 1][2 * e] * f[e][0] + y.z * f[e][1];
                            o[2 * k + 1][2 * e + 1] = o[2 * k + 1][2 * e + 1] * f[e][0] + y.w * f[e][1];
                        }
                    }
                }
            }
            if (C::WT > 1 && wt == 0) {
                __syncwarp();
                if (lane == 0) sm100::mbar_arrive(smem_u32(&s_read));
            }
            ++units;
            if (!together) break;
            const bool whole = seg_tile == 0 && d.tile == d.nt - 1;
            if (wt == 0) {
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    const int rl = wr * 16 + lr + 8 * e, r = rt * C::RMAX + rl;
                    if (whole) {
                        if (r >= rows_all) continue;
                        const int t = r / group, hq = h * group + r - t * group;
                        const int64_t row = ((int64_t)d.b * a.T + t) * a.Hq + hq;
                        if (!in_range(row, 1, (int64_t)a.B * a.T * a.Hq, a.dev_status)) continue;
                        const float inv = l[e] == 0.f ? 0.f : 1.f / l[e];
                        uint16_t *const out = static_cast<uint16_t *>(a.out) + row * D;
#pragma unroll
                        for (int n = 0; n < C::DW / 8; ++n) {
                            const int dd = wd * C::DW + n * 8 + 2 * tq;
                            if (dd < D)
                                *reinterpret_cast<uint32_t *>(out + dd) =
                                    pack_out(KIND == kE4M3 ? a.q_bf16 : BF16, o[n][2 * e] * inv, o[n][2 * e + 1] * inv);
                        }
                        if (a.lse && wd == 0 && tq == 0)
                            a.lse[row] = l[e] == 0.f ? -INFINITY : (m[e] + log2f(l[e])) * kLn2;
                    } else {
                        const int64_t p = ((int64_t)c * 2 + (seg_tile > 0 ? 0 : 1)) * C::RMAX + rl;
                        if (!in_range(p, 1, (int64_t)G * 2 * C::RMAX, a.dev_status)) continue;
                        if (wd == 0 && tq == 0) part_ml[p] = make_float2(m[e], l[e]);
                        float *const po = part_o + p * DP + wd * C::DW;
#pragma unroll
                        for (int n = 0; n < C::DW / 8; ++n)
                            *reinterpret_cast<float2 *>(po + n * 8 + 2 * tq) = make_float2(o[n][2 * e], o[n][2 * e + 1]);
                    }
                }
            }
            // the block where a unit begins says who holds its parts
            if (tid == 0 && seg_tile == 0) {
                const int u = h * RT + rt;
                const int64_t unit = (int64_t)d.b * U + u;
                const int64_t end = d.place + (d.nt - 1 - d.tile);   // the unit's last tile
                const int last = deal.owner(end);
                const int64_t at = by_unit ? unit : c;
                if ((by_unit || !whole) && in_range(at, 1, n_splits, a.dev_status)) {
                    Split sp;
                    sp.u_lo = u; sp.b = d.b; sp.c0 = c; sp.c1 = whole ? -1 : last;
                    splits[at] = sp;
                }
            }
        }
        if (d.last) break;
    }
}

// Joins the rows of units that several blocks worked on.  `per` == kJoinRows (many units): eight
// rows a block, one warp a row of up to kFew parts.  Otherwise, and for rows of more parts, the
// whole block takes a row, 64 dimensions at a time, sixteen groups of threads every sixteenth
// part; with `per` == 1 a block has one row and 64 dimensions.
constexpr int kJoin = 256;
constexpr int kJoinGroups = 16;
constexpr int kMaxBlocks = 1024;
constexpr int kFew = 8;
constexpr int kJoinRows = kJoin / 32;

template <int DP>
__global__ void __launch_bounds__(kJoin)
paged_attn_join_kernel(const GdnAttnArgs a, const int RT, const int RMAX, const int per,
                       const int blocks, const Split *const splits, const float2 *const part_ml, const float *const part_o)
{
    __shared__ float s_w[kMaxBlocks];                   // weights of the parts
    __shared__ float s_red[2][kJoin / 32];
    __shared__ float4 s_o[kJoinGroups][16];
    wait_primary();
    const Split sp = splits[blockIdx.x];
    const int H = a.cache.heads, D = a.cache.head_dim, group = a.Hq / H;
    // (a block that gave up waiting wrote nothing: what is there then need not make sense)
    if (sp.c1 < 0 || sp.c0 < 0 || sp.c0 > sp.c1 || sp.c1 >= blocks || (uint32_t)sp.b >= (uint32_t)a.B ||
        (uint32_t)sp.u_lo >= (uint32_t)(H * RT))
        return;
    const int h = sp.u_lo / RT, rt = sp.u_lo - h * RT;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int np = sp.c1 - sp.c0 + 1;
    const int rows = min(RMAX, a.T * group - rt * RMAX);        // of the unit
    auto place = [&](int rl) {
        const int r = rt * RMAX + rl, t = r / group;
        return ((int64_t)sp.b * a.T + t) * a.Hq + h * group + r - t * group;
    };
    // part k: the first block's is its second, the others' are their first
    // (a checked build reads the first row for one that is none)
    auto at = [&](int k, int rl) {
        if constexpr (gdn::kChecked)
            if (!in_range(((int64_t)(sp.c0 + k) * 2 + (k == 0 ? 1 : 0)) * RMAX + rl, 1, (int64_t)blocks * 2 * RMAX,
                          a.dev_status))
                return (int64_t)0;
        return ((int64_t)(sp.c0 + k) * 2 + (k == 0 ? 1 : 0)) * RMAX + rl;
    };
    auto store = [&](int64_t row, int d, float4 y, float sum) {
        const float inv = sum == 0.f ? 0.f : 1.f / sum;
        uint32_t *const out = reinterpret_cast<uint32_t *>(static_cast<uint16_t *>(a.out) + row * D + d);
        out[0] = pack_out(a.q_bf16, y.x * inv, y.y * inv);
        out[1] = pack_out(a.q_bf16, y.z * inv, y.w * inv);
    };
    const int64_t all_rows = (int64_t)a.B * a.T * a.Hq;

    if (per == kJoinRows && np <= kFew) {
        const int rl = blockIdx.y * per + warp;
        if (rl >= rows) return;
        constexpr int PER = (DP + 127) / 128;           // float4 a thread
        float4 y[PER][kFew];
#pragma unroll
        for (int k = 0; k < kFew; ++k)
#pragma unroll
            for (int e = 0; e < PER; ++e)
                y[e][k] = k < np && (e * 32 + lane) * 4 < DP
                              ? __ldcg(reinterpret_cast<const float4 *>(part_o + at(k, rl) * DP) + e * 32 + lane)
                              : make_float4(0.f, 0.f, 0.f, 0.f);
        float2 ml = make_float2(-INFINITY, 0.f);
        if (lane < np) ml = __ldcg(part_ml + at(lane, rl));
        float top = ml.x;
#pragma unroll
        for (int s = 16; s > 0; s >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, s));
        const float ms = top == -INFINITY ? 0.f : top;
        const float w = ex2_approx(ml.x - ms);
        const float sum = gdn::warp_sum(ml.y * w);
        const int64_t row = place(rl);
        const bool ok = in_range(row, 1, all_rows, a.dev_status);
#pragma unroll
        for (int e = 0; e < PER; ++e) {
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int k = 0; k < kFew; ++k) {
                const float wk = __shfl_sync(0xffffffffu, w, k);
                if (k < np) {
                    acc.x += wk * y[e][k].x;
                    acc.y += wk * y[e][k].y;
                    acc.z += wk * y[e][k].z;
                    acc.w += wk * y[e][k].w;
                }
            }
            const int d = (e * 32 + lane) * 4;
            if (ok && d < D) store(row, d, acc, sum);
        }
        if (ok && a.lse && lane == 0) a.lse[row] = sum == 0.f ? -INFINITY : (top + log2f(sum)) * kLn2;
        return;
    }

    const int grp = tid / 16, d4 = tid % 16;
    constexpr int kAhead = 10;
    constexpr int kMl = kMaxBlocks / kJoin;             // np <= kMaxBlocks
    for (int rl = blockIdx.y * per; rl < min(rows, (int)(blockIdx.y + 1) * per); ++rl)
        for (int d0 = blockIdx.z * 64; d0 < D; d0 += 64 * gridDim.z) {
            // the values come first: they do not depend on the weights
            float4 y[kAhead];
            auto fetch = [&](int k0) {
#pragma unroll
                for (int u = 0; u < kAhead; ++u) {
                    const int k = k0 + u * kJoinGroups;
                    y[u] = k < np ? __ldcg(reinterpret_cast<const float4 *>(part_o + at(k, rl) * DP + d0) + d4)
                                  : make_float4(0.f, 0.f, 0.f, 0.f);
                }
            };
            fetch(grp);
            float top = -INFINITY;
            float2 ml[kMl];
#pragma unroll
            for (int u = 0; u < kMl; ++u) {
                const int k = tid + u * kJoin;
                ml[u] = k < np ? __ldcg(part_ml + at(k, rl)) : make_float2(-INFINITY, 0.f);
                top = fmaxf(top, ml[u].x);
            }
#pragma unroll
            for (int s = 16; s > 0; s >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, s));
            if (lane == 0) s_red[0][warp] = top;
            __syncthreads();
#pragma unroll
            for (int w = 0; w < kJoin / 32; ++w) top = fmaxf(top, s_red[0][w]);
            const float ms = top == -INFINITY ? 0.f : top;
            float sum = 0.f;
#pragma unroll
            for (int u = 0; u < kMl; ++u) {
                const int k = tid + u * kJoin;
                const float w = ex2_approx(ml[u].x - ms);
                if (k < np) {
                    s_w[k] = w;
                    sum += ml[u].y * w;
                }
            }
            sum = gdn::warp_sum(sum);
            if (lane == 0) s_red[1][warp] = sum;
            __syncthreads();
            sum = 0.f;
#pragma unroll
            for (int w = 0; w < kJoin / 32; ++w) sum += s_red[1][w];

            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
            for (int k0 = grp; k0 < np; k0 += kAhead * kJoinGroups) {
                if (k0 != grp) fetch(k0);
#pragma unroll
                for (int u = 0; u < kAhead; ++u) {
                    const int k = k0 + u * kJoinGroups;
                    if (k >= np) break;
                    const float w = s_w[k];
                    acc.x += w * y[u].x;
                    acc.y += w * y[u].y;
                    acc.z += w * y[u].z;
                    acc.w += w * y[u].w;
                }
            }
            s_o[grp][d4] = acc;
            __syncthreads();
            const int64_t row = place(rl);
            const bool ok = in_range(row, 1, all_rows, a.dev_status);
            if (ok && tid < 16 && d0 + 4 * tid < D) {
                acc = s_o[0][tid];
#pragma unroll
                for (int g = 1; g < kJoinGroups; ++g) {
                    const float4 z = s_o[g][tid];
                    acc.x += z.x;
                    acc.y += z.y;
                    acc.z += z.z;
                    acc.w += z.w;
                }
                store(row, d0 + 4 * tid, acc, sum);
            }
            if (ok && a.lse && tid == 0 && d0 == 0) a.lse[row] = sum == 0.f ? -INFINITY : (top + log2f(sum)) * kLn2;
            __syncthreads();        // the shared arrays are used again
        }
}

// ------------------------------------------------------------------ host
int padded(int D) { return D <= 64 ? 64 : (D <= 128 ? 128 : 256); }
// warps over rows: as few as hold them; 256-wide heads leave room for two
int row_warps(int rows, int DP) { return rows <= 16 ? 1 : (rows <= 32 || DP == 256 ? 2 : 4); }
int max_blocks() { return std::min(2 * sm_count(), kMaxBlocks); }

struct Layout {
    int RT, RMAX, n_splits;
    uint64_t ml_at, o_at, bytes;
};

// `DP` as the kernel pads the head
Layout layout(int B, int T, int Hq, int H, int DP, int blocks)
{
    const int rows = T * (Hq / H);
    Layout y;
    y.RMAX = 16 * row_warps(rows, DP);
    y.RT = (rows + y.RMAX - 1) / y.RMAX;
    const int64_t units = (int64_t)B * H * y.RT;
    y.n_splits = (int)(units < blocks ? units : blocks);
    y.ml_at = ((uint64_t)y.n_splits * sizeof(Split) + 15) / 16 * 16;
    y.o_at = y.ml_at + (uint64_t)blocks * 2 * y.RMAX * sizeof(float2);
    y.bytes = y.o_at + (uint64_t)blocks * 2 * y.RMAX * DP * sizeof(float);
    return y;
}

PFN_cuTensorMapEncodeTiled_v12000 get_encode()
{
    static const PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            p = nullptr;
        return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
    }();
    return fn;
}

// keys or values as (dimension, token of a page, head, page), in boxes of `box` tokens of a head
cudaError_t encode(CUtensorMap *map, const void *base, const gdn_paged_cache &kv, int es, int row_bytes, int box)
{
    const PFN_cuTensorMapEncodeTiled_v12000 fn = get_encode();
    if (!fn) return cudaErrorNotSupported;
    const cuuint64_t dims[4] = {(cuuint64_t)kv.head_dim, (cuuint64_t)kv.page_size, (cuuint64_t)kv.heads,
                                (cuuint64_t)kv.num_pages};
    const cuuint64_t none = (cuuint64_t)kv.head_dim * es;   // the stride of a dimension of one
    const cuuint64_t strides[3] = {kv.page_size > 1 ? (cuuint64_t)kv.token_stride * es : none,
                                   kv.heads > 1 ? (cuuint64_t)kv.head_stride * es : none,
                                   kv.num_pages > 1 ? (cuuint64_t)kv.page_stride * es : none};
    const int inner = row_bytes < 128 ? row_bytes : 128;
    const cuuint32_t boxes[4] = {(cuuint32_t)(inner / es), (cuuint32_t)box, 1, 1};
    const cuuint32_t steps[4] = {1, 1, 1, 1};
    // whole tokens side by side are fetched 256 bytes at a time; the rows of one head between
    // those of others no further than they reach
    const int reach = kv.page_size > 1 && kv.token_stride != kv.head_dim ? kv.head_dim * es : 256;
    const CUtensorMapL2promotion l2 = reach % 256 == 0   ? CU_TENSOR_MAP_L2_PROMOTION_L2_256B
                                      : reach % 128 == 0 ? CU_TENSOR_MAP_L2_PROMOTION_L2_128B
                                                         : CU_TENSOR_MAP_L2_PROMOTION_L2_64B;
    const CUresult r = fn(map, es == 1 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_UINT16, 4,
                          const_cast<void *>(base), dims, strides, boxes, steps, CU_TENSOR_MAP_INTERLEAVE_NONE,
                          inner == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
                          l2, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

// tokens of a box: the largest power of two that divides the page size, a tile's at most
int box_tokens(int page_size, int tile)
{
    const int p = page_size & -page_size;
    return p < tile ? p : tile;
}

template <int KIND, int DP, int WR>
cudaError_t launch(const GdnAttnArgs &a, cudaStream_t stream)
{
    using C = Cfg<KIND, DP, WR>;
    static DeviceOnce once;
    cudaError_t e = once.run([] {
        // the warps that compute wait for registers that the block must have been launched with
        cudaFuncAttributes at;
        cudaError_t e = cudaFuncGetAttributes(&at, paged_attn_kernel<KIND, DP, WR>);
        if (e != cudaSuccess) return e;
        if (at.numRegs * 2 < kFetchRegs + kComputeRegs) return cudaErrorInvalidKernelImage;
        return cudaFuncSetAttribute(paged_attn_kernel<KIND, DP, WR>,
                                    cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
    });
    if (e != cudaSuccess) return e;
    const gdn_paged_cache &kv = a.cache;
    const int box = box_tokens(kv.page_size, C::TILE);
    CUtensorMap kmap, vmap;
    e = encode(&kmap, kv.k, kv, C::ESZ, C::RB, box);
    if (e == cudaSuccess) e = encode(&vmap, kv.v, kv, C::ESZ, C::RB, box);
    if (e != cudaSuccess) return e;
    const Layout y = layout(a.B, a.T, a.Hq, kv.heads, DP, max_blocks());
    // no more blocks than there can be places in the deal
    const int64_t cap = (int64_t)kv.width * kv.page_size;
    const double tiles = (double)a.B * kv.heads * y.RT * (double)((cap + C::TILE - 1) / C::TILE + 1 + kUnitCost);
    const int blocks = tiles < max_blocks() ? (int)tiles : max_blocks();
    unsigned char *const ws = static_cast<unsigned char *>(a.workspace);
    Split *const splits = reinterpret_cast<Split *>(ws);
    float2 *const ml = reinterpret_cast<float2 *>(ws + y.ml_at);
    float *const o = reinterpret_cast<float *>(ws + y.o_at);
    const int64_t units = (int64_t)a.B * kv.heads * y.RT;
    const int n_splits = (int)(units < blocks ? units : blocks);
    paged_attn_kernel<KIND, DP, WR><<<blocks, kThreads, C::SMEM, stream>>>(kmap, vmap, a, box, y.RT, splits,
                                                                           n_splits, ml, o);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    // many units have two or three parts each as a rule, few many
    const int rows = std::min(y.RMAX, a.T * (a.Hq / kv.heads));
    const int per = units * kFew >= blocks ? kJoinRows : 1;
    return launch_dependent(paged_attn_join_kernel<DP>,
                            dim3(n_splits, (rows + per - 1) / per, per == 1 ? DP / 64 : 1), dim3(kJoin), 0,
                            stream, a, y.RT, y.RMAX, per, blocks, splits, ml, o);
}

// A box starts on 128 bytes of shared memory: 64-byte rows need an even number of tokens, so
// 8-bit heads of at most 64 dimensions on pages of an odd number of tokens run 128 wide (the
// dimensions past the head's are zeros).
int padded(const gdn_paged_cache &kv)
{
    const bool odd64 = kv.dtype == GDN_E4M3 && kv.head_dim <= 64 && kv.page_size % 2 != 0;
    return odd64 ? 128 : padded(kv.head_dim);
}

template <int KIND>
cudaError_t dispatch(const GdnAttnArgs &a, cudaStream_t stream)
{
    const int DP = padded(a.cache);
    const int WR = row_warps(a.T * (a.Hq / a.cache.heads), DP);
    switch (DP + WR) {
    case 64 + 1: return launch<KIND, 64, 1>(a, stream);
    case 64 + 2: return launch<KIND, 64, 2>(a, stream);
    case 64 + 4: return launch<KIND, 64, 4>(a, stream);
    case 128 + 1: return launch<KIND, 128, 1>(a, stream);
    case 128 + 2: return launch<KIND, 128, 2>(a, stream);
    case 128 + 4: return launch<KIND, 128, 4>(a, stream);
    case 256 + 1: return launch<KIND, 256, 1>(a, stream);
    default: return launch<KIND, 256, 2>(a, stream);
    }
}

}  // namespace gdn_attn

int gdn_cache::sm_count()
{
    static std::atomic<int> known[32];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return 0;
    if (dev < 32) {
        const int k = known[dev].load(std::memory_order_relaxed);
        if (k > 0) return k;
    }
    int n = 0;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
    if (dev < 32) known[dev].store(n, std::memory_order_relaxed);
    return n;
}

uint64_t paged_attn_workspace_bytes(int32_t B, int32_t T, int32_t Hq, int32_t heads, int32_t D,
                                    int32_t cache_dtype)
{
    using namespace gdn_attn;
    const int blocks = max_blocks(), DP = padded(D);
    if (blocks == 0) return 0;
    // (8-bit heads of at most 64 dimensions may run 128 wide, by the page size)
    const uint64_t n = layout(B, T, Hq, heads, DP, blocks).bytes;
    return cache_dtype == GDN_E4M3 && DP == 64 ? std::max(n, layout(B, T, Hq, heads, 128, blocks).bytes) : n;
}

cudaError_t launch_paged_attn(const GdnAttnArgs &a, cudaStream_t stream)
{
    switch (a.cache.dtype) {
    case GDN_BF16: return gdn_attn::dispatch<gdn_attn::kBF16>(a, stream);
    case GDN_F16: return gdn_attn::dispatch<gdn_attn::kF16>(a, stream);
    default: return gdn_attn::dispatch<gdn_attn::kE4M3>(a, stream);
    }
}
