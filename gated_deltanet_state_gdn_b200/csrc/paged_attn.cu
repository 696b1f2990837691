// paged_attn.cu -- attention of each request's last T tokens over its paged keys and values.
//
// Mathematics.  For one head of the cache the T * (Hq / H) query rows that read it are a matrix
// Q; over the tokens j in order, with x = scale log2(e) Q k_j,
//     m' = max(m, x),  l' = l 2^(m - m') + 2^(x - m'),  O' = O 2^(m - m') + 2^(x - m') v_j
// and out = O / l.  Two parts (m1, l1, O1), (m2, l2, O2) of one row join by the same rule, which
// is what lets the tokens of a row be cut anywhere.
//
// What bounds it: every key and value is read once and meets T Hq / H rows, 2 T Hq / H
// operations a byte in 16 bits; below about 100 rows a head HBM is the bound, and warp mma feeds
// it with the tensor pipe a quarter busy, so tcgen05 (128 rows at least, of which one token's
// group would fill 1 to 16) is not used.
//
// Layout of the work.
//   - A unit is (request, head, block of 16 WR rows); its tokens are cut into tiles of 16 KB of
//     keys and 16 KB of values.  All tiles of all units in a row are dealt to the resident
//     blocks (two an SM) in equal runs, found on the device from the lengths: one long request
//     and many short ones fill the GPU alike, and the host reads nothing.
//   - A block streams its run through three stages of shared memory with 16-byte asynchronous
//     copies, rows of a tile looked up in the page table one tile ahead; tokens that no row sees
//     are zero-filled, never read.
//   - Four warps share a tile: WR over blocks of 16 rows, the others over the tokens (each with
//     its own m, l, O, joined in shared memory at the end of the unit), and for 256-wide heads
//     two over the halves of the values.
//   - A unit that lies in one block is finished there.  Parts of the others go to the workspace
//     and a second kernel joins them in the order of the tokens: no atomics, the same result in
//     every run.
#include <cuda_runtime.h>

#include "cache.cuh"

namespace gdn_attn {

using namespace gdn_cache;
using gdn::in_range;
using gdn::in_smem;
using sm100::ex2_approx;
using sm100::smem_u32;

constexpr int kThreads = 128;
constexpr int kHalfStage = 16384;   // bytes of keys (or values) in a stage
constexpr int kStages = 3;
constexpr int kRing = 4;            // tile descriptors alive at once
constexpr int kMergeBytes = 8192;
constexpr int kRowsWindow = 64;     // rows of the batch whose lengths are at hand
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

enum Kind { kBF16 = 0, kF16 = 1, kE4M3 = 2 };

template <int KIND, int DP, int WR>
struct Cfg {
    static constexpr int ESZ = KIND == kE4M3 ? 1 : 2;
    static constexpr int RB = DP * ESZ;              // bytes of a token's row in a stage
    static constexpr int CPR = RB / 16;              // 16-byte pieces of it
    static constexpr int TILE = kHalfStage / RB;     // tokens a tile
    static constexpr int WD = DP == 256 ? 2 : 1;     // warps over the values' dimensions
    static constexpr int WT = 4 / (WR * WD);         // warps over tokens
    static constexpr int NS = TILE / 16 / WT;        // 16-token steps of a warp in a tile
    static constexpr int DW = DP / WD;               // dimensions a warp accumulates
    static constexpr int RMAX = 16 * WR;             // rows of a unit
    static constexpr int SMEM = kStages * 2 * kHalfStage + kMergeBytes + 2 * TILE * 8;
    static_assert(WT >= 1 && NS >= 1, "four warps");
};

struct Desc {
    int b, u, base, len, tile, nt;
};

struct Split {              // a unit whose parts lie in blocks [c0, c1]
    int u_lo, b, c0, c1;    // c1 < 0: nothing to join
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

// first position that some token of the request sees
__device__ __forceinline__ int first_seen(const GdnAttnArgs &a, int len)
{
    return a.window > 0 ? max(0, (int)max((int64_t)len - a.T - a.window + 1, (int64_t)0)) : 0;
}

template <int TILE>
__device__ __forceinline__ int tiles_of(const GdnAttnArgs &a, int len)
{
    const int lo = first_seen(a, len);
    return len > lo ? (len - lo + TILE - 1) / TILE : 0;
}

__device__ __forceinline__ int64_t block_sum(int64_t x, int64_t *s)
{
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
    if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = x;
    __syncthreads();
    x = s[0] + s[1] + s[2] + s[3];
    __syncthreads();
    return x;
}

// rows and dimensions of a finished or partial result
template <int KIND, int DP, int WR>
struct Where {
    using C = Cfg<KIND, DP, WR>;
    // first of the pair of dimensions held in o[n][e], o[n][e + 1] (16 bits), or of the four in
    // o[n][e], o[n + 1][e], o[n][e + 1], o[n + 1][e + 1] (e4m3, n even)
    static __device__ __forceinline__ int dim(int n, int tq)
    {
        return KIND == kE4M3 ? n * 8 + 4 * tq : n * 8 + 2 * tq;
    }
};

template <bool BF16>
__device__ __forceinline__ uint32_t pack16(float lo, float hi)
{
    if constexpr (BF16)
        return gdn::pack_bf16x2(lo, hi);
    else
        return pack_f16x2(lo, hi);
}

__device__ __forceinline__ uint32_t pack_out(bool bf16, float lo, float hi)
{
    return bf16 ? gdn::pack_bf16x2(lo, hi) : pack_f16x2(lo, hi);
}

// 16-byte piece c of token row r of a stage: keys and values of 16 bits and values of 8 are read
// by ldmatrix (eight rows, one piece), keys of 8 bits four pieces of two rows at a time
template <int RB, bool QUADS>
__device__ __forceinline__ int piece(int r, int c)
{
    if constexpr (QUADS) return RB == 64 ? c : c ^ ((r & 1) << 2);
    return RB == 64 ? c ^ ((r >> 1) & 3) : c ^ (r & 7);
}

template <int KIND, int DP, int WR>
__global__ void __launch_bounds__(kThreads, 2)
paged_attn_kernel(const GdnAttnArgs a, const int RT, Split *const splits, const int n_splits,
                  float2 *const part_ml, float *const part_o)
{
    using C = Cfg<KIND, DP, WR>;
    constexpr int TILE = C::TILE, RB = C::RB, CPR = C::CPR;
    constexpr bool BF16 = KIND == kBF16;
    extern __shared__ __align__(128) unsigned char smem[];
    unsigned char *const s_stage = smem;
    float *const s_merge = reinterpret_cast<float *>(smem + kStages * 2 * kHalfStage);
    int64_t *const s_off = reinterpret_cast<int64_t *>(smem + kStages * 2 * kHalfStage + kMergeBytes);
    __shared__ int64_t s_sum[4];
    __shared__ int64_t s_found[2];
    __shared__ Desc s_desc[kRing];
    __shared__ uint32_t s_valid[kRing][TILE / 32];
    __shared__ RowInfo s_rows[kRowsWindow];
    __shared__ float4 s_stat[2][32];

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int tq = lane & 3, lr = lane >> 2;
    const int wr = warp % WR, wd = (warp / WR) % C::WD, wt = warp / (WR * C::WD);
    const int c = blockIdx.x, G = gridDim.x;
    const gdn_paged_cache &kv = a.cache;
    const int H = kv.heads, D = kv.head_dim, group = a.Hq / H, rows_all = a.T * group;
    const int U = H * RT;                              // units of a request
    const bool by_unit = (int64_t)a.B * U <= n_splits; // one Split a unit, else one a block

    launch_dependents();

    // ---- this block's run of tiles
    int64_t mine = 0;
    for (int b = tid; b < a.B; b += kThreads) mine += tiles_of<TILE>(a, row_info(a, b, c == 0).len);
    const int64_t W = block_sum(mine, s_sum) * U;
    const int64_t Ge = W < G ? W : G;
    const int64_t t0 = c < Ge ? c * W / Ge : 0, t1 = c < Ge ? (c + 1) * W / Ge : 0;
    const int n_tiles = (int)(t1 - t0);
    if (!by_unit && tid == 0 && in_range(c, 1, n_splits, a.dev_status)) splits[c].c1 = -1;

    // requests with nothing to see: zeros for a row of the cache, nothing (or zeros) for padding
    for (int b = c; b < a.B; b += G) {
        const RowInfo ri = row_info(a, b, false);
        if (tiles_of<TILE>(a, ri.len) > 0) continue;
        if (by_unit)
            for (int u = tid; u < U; u += kThreads)
                if (in_range((int64_t)b * U + u, 1, n_splits, a.dev_status))
                    splits[(int64_t)b * U + u].c1 = -1;
        if (ri.slot < 0 && !a.zero_padding) continue;
        const int64_t rows = (int64_t)a.T * a.Hq, words = rows * D / 2;
        const int64_t total = (int64_t)a.B * rows;
        uint32_t *const o = static_cast<uint32_t *>(a.out) + b * words;
        if (in_range(b * words, words, total * D / 2, a.dev_status))
            for (int64_t i = tid; i < words; i += kThreads) o[i] = 0u;
        if (a.lse && in_range(b * rows, rows, total, a.dev_status))
            for (int64_t i = tid; i < rows; i += kThreads) a.lse[b * rows + i] = -INFINITY;
    }
    if (n_tiles == 0) return;

    // the request, unit and tile where it begins
    {
        int64_t before = 0;
        for (int b0 = 0; b0 < a.B; b0 += kThreads) {
            const int b = b0 + tid;
            const int nt = b < a.B ? tiles_of<TILE>(a, row_info(a, b, false).len) : 0;
            int64_t incl = nt;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int64_t y = __shfl_up_sync(0xffffffffu, incl, d);
                if (lane >= d) incl += y;
            }
            if (lane == 31) s_sum[warp] = incl;
            __syncthreads();
            int64_t all = 0;
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                if (w < warp) incl += s_sum[w];
                all += s_sum[w];
            }
            incl += before;
            if (nt > 0 && t0 >= (incl - nt) * U && t0 < incl * U) {
                s_found[0] = b;
                s_found[1] = t0 - (incl - nt) * U;
            }
            before += all;
            __syncthreads();
            if (t0 < before * U) break;
        }
    }

    // cursor over the run (the same in every thread): where the next tile to prepare is
    int cb = (int)s_found[0], win = cb;
    auto fill_window = [&]() {
        __syncthreads();
        win = cb;
        if (tid < kRowsWindow && win + tid < a.B) s_rows[tid] = row_info(a, win + tid, false);
        __syncthreads();
    };
    fill_window();
    RowInfo cr = s_rows[0];
    int cnt = tiles_of<TILE>(a, cr.len);
    int cu = (int)(s_found[1] / cnt), ct = (int)(s_found[1] - (int64_t)cu * cnt);
    auto advance = [&]() {
        if (++ct < cnt) return;
        ct = 0;
        if (++cu < U) return;
        cu = 0;
        do {
            if (++cb >= a.B) return;  // past the last tile (never prepared)
            if (cb - win >= kRowsWindow) fill_window();
            cr = s_rows[cb - win];
            cnt = tiles_of<TILE>(a, cr.len);
        } while (cnt == 0);
    };

    // ---- a tile's rows: page lookups, then (a step later) its copies
    constexpr int LPT = (TILE + kThreads - 1) / kThreads;   // lookups a thread
    const int64_t cache_bytes = ((int64_t)(kv.num_pages - 1) * kv.page_stride +
                                 (int64_t)(kv.page_size - 1) * kv.token_stride +
                                 (int64_t)(H - 1) * kv.head_stride + D) * C::ESZ;
    int64_t look[LPT];
    auto lookup = [&]() {     // byte offset of each of this thread's token rows, or -1
        const int base = first_seen(a, cr.len) + ct * TILE;
        const int h = cu / RT;
        const int32_t *const row = kv.block_table + (int64_t)cr.slot * kv.table_stride;
#pragma unroll
        for (int i = 0; i < LPT; ++i) {
            const int j = base + tid + i * kThreads;
            look[i] = -1;
            if (tid + i * kThreads < TILE && j < cr.len) {
                const int pg = (int)((uint32_t)j / (uint32_t)kv.page_size);
                const int id = in_range(pg, 1, kv.width, a.dev_status) ? __ldg(row + pg) : -1;
                if ((uint32_t)id < (uint32_t)kv.num_pages)
                    look[i] = (id * kv.page_stride + (j - pg * kv.page_size) * kv.token_stride +
                               h * kv.head_stride) * C::ESZ;
                else if (a.dev_status)
                    atomicOr(a.dev_status, GDN_DEV_BAD_PAGE);
            }
        }
    };
    auto note = [&](int n, const Desc &d) {   // write down tile n of the run
#pragma unroll
        for (int i = 0; i < LPT; ++i) {
            const int r = tid + i * kThreads;
            if (r < TILE) {      // whole warps: TILE is a multiple of 32
                s_off[(n & 1) * TILE + r] = look[i];
                const uint32_t ok = __ballot_sync(0xffffffffu, look[i] >= 0);
                if (lane == 0) s_valid[n % kRing][r >> 5] = ok;
            }
        }
        if (tid == 0) s_desc[n % kRing] = d;
    };
    auto here = [&]() {
        Desc d;
        d.b = cb; d.u = cu; d.base = first_seen(a, cr.len) + ct * TILE; d.len = cr.len;
        d.tile = ct; d.nt = cnt;
        return d;
    };
    const unsigned char *const kp = static_cast<const unsigned char *>(kv.k);
    const unsigned char *const vp = static_cast<const unsigned char *>(kv.v);
    auto issue = [&](int n) {
        unsigned char *const st = s_stage + (n % kStages) * 2 * kHalfStage;
        const uint32_t ks = smem_u32(st), vs = ks + kHalfStage;
        const int ch = tid % CPR;
        const bool has = ch * 16 < D * C::ESZ;
#pragma unroll
        for (int i = 0; i < kHalfStage / 16 / kThreads; ++i) {
            const int r = tid / CPR + i * (kThreads / CPR);
            const int64_t off = s_off[(n & 1) * TILE + r];
            const bool ok = off >= 0 && has && in_range(off + ch * 16, 16, cache_bytes, a.dev_status);
            const int64_t src = ok ? off + ch * 16 : 0;
            const uint32_t bytes = ok ? 16u : 0u;
            cp_async16(ks + r * RB + piece<RB, KIND == kE4M3>(r, ch) * 16, kp + src, bytes);
            cp_async16(vs + r * RB + piece<RB, false>(r, ch) * 16, vp + src, bytes);
        }
    };

    lookup();
    note(0, here());
    if (n_tiles > 1) {
        advance();
        lookup();
        note(1, here());
    }
    __syncthreads();
    issue(0);
    cp_async_commit();
    if (n_tiles > 1) issue(1);
    cp_async_commit();
    if (n_tiles > 2) {
        __syncthreads();
        advance();
        lookup();
        note(2, here());
    }

    // ---- the run
    float m[2], l[2], o[C::DW / 8][4];      // rows lr and lr + 8 of the warp's 16
    uint32_t qf[DP / 16][4];
    float xs[2];                            // what a raw score is multiplied by
    int hi[2], lo[2];                       // a row sees lo < j <= hi
    int seg_tile = 0;                       // where the unit's part in this block began
#pragma unroll 1
    for (int i = 0; i < n_tiles; ++i) {
        cp_async_wait<kStages - 2>();
        __syncthreads();
        if (i + 2 < n_tiles) issue(i + 2);
        cp_async_commit();
        const bool more = i + 3 < n_tiles;
        Desc next;
        if (more) {
            advance();
            lookup();
            next = here();
        }
        const Desc d = s_desc[i % kRing];
        const int h = d.u / RT, rt = d.u - h * RT;

        if (i == 0 || d.tile == 0) {        // a unit begins: its query rows
            seg_tile = d.tile;
            const float x2 = a.scale * kLog2e * (KIND == kE4M3 && kv.k_scale ? __ldg(kv.k_scale + h) : 1.f);
            const uint32_t *qr[2];
            bool has[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                m[e] = -INFINITY;
                l[e] = 0.f;
                xs[e] = x2;
                const int r = rt * C::RMAX + wr * 16 + lr + 8 * e;
                has[e] = r < rows_all;
                const int t = has[e] ? r / group : 0, g = has[e] ? r - t * group : 0;
                qr[e] = reinterpret_cast<const uint32_t *>(
                    static_cast<const uint16_t *>(a.q) + ((int64_t)d.b * a.T + t) * a.q_token_stride +
                    (int64_t)(h * group + g) * a.q_head_stride);
                const int64_t pos = (int64_t)d.len - a.T + t;
                hi[e] = has[e] ? (int)pos : -1;
                lo[e] = has[e] && a.window > 0 && pos >= a.window ? (int)(pos - a.window) : -1;
            }
#pragma unroll
            for (int n = 0; n < C::DW / 8; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[n][e] = 0.f;
            if constexpr (KIND != kE4M3) {
#pragma unroll
                for (int k = 0; k < DP / 16; ++k)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int dd = k * 16 + (e >> 1) * 8 + 2 * tq;
                        qf[k][e] = has[e & 1] && dd < D ? __ldg(qr[e & 1] + dd / 2) : 0u;
                    }
            } else {
                // Rows of q become halves, scaled by the power of two that brings the largest
                // element to [2^7, 2^8): a bf16 or fp16 number down to 2^-22 of it is kept
                // exactly, smaller ones to 2^-33 of it.  The order of the dimensions is that of
                // the keys' 16-byte pieces: thread tq of a quad has 16 of each 64 in a row.
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    uint32_t w[DP / 64][8];
                    float top = 0.f;
#pragma unroll
                    for (int s = 0; s < DP / 64; ++s)
#pragma unroll
                        for (int k = 0; k < 8; ++k) {
                            const int dd = s * 64 + tq * 16 + 2 * k;
                            w[s][k] = has[e] && dd < D ? __ldg(qr[e] + dd / 2) : 0u;
                        }
                    auto value = [&](uint32_t x, int half) {
                        const uint16_t v = (uint16_t)(half ? x >> 16 : x & 0xffffu);
                        return a.q_bf16 ? __uint_as_float((uint32_t)v << 16)
                                        : __half2float(__ushort_as_half(v));
                    };
#pragma unroll
                    for (int s = 0; s < DP / 64; ++s)
#pragma unroll
                        for (int k = 0; k < 8; ++k)
                            top = fmaxf(top, fmaxf(fabsf(value(w[s][k], 0)), fabsf(value(w[s][k], 1))));
                    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
                    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
                    const int ex = min(max((int)(__float_as_uint(top) >> 23), 8), 254);
                    const float up = __uint_as_float((uint32_t)(261 - ex) << 23);
                    xs[e] = x2 * __uint_as_float((uint32_t)(ex - 7) << 23);
#pragma unroll
                    for (int s = 0; s < DP / 64; ++s)
#pragma unroll
                        for (int k = 0; k < 8; ++k)
                            qf[s * 4 + k / 2][e + 2 * (k & 1)] =
                                pack_f16x2(value(w[s][k], 0) * up, value(w[s][k], 1) * up);
                }
            }
        }

        const uint32_t ks = smem_u32(s_stage + (i % kStages) * 2 * kHalfStage), vs = ks + kHalfStage;
        const int see_all = d.len - a.T;                                     // j <= this: causally seen by all rows
        const int64_t see_from = a.window > 0 ? (int64_t)d.len - a.window : 0;   // j >= this: in every window
#pragma unroll 1
        for (int s = 0; s < C::NS; ++s) {
            const int tok = (s * C::WT + wt) * 16;
            const uint32_t ok = (s_valid[i % kRing][tok >> 5] >> (tok & 16)) & 0xffffu;
            if (ok == 0) continue;
            const int j0 = d.base + tok;
            const bool ragged = j0 + 15 > see_all || j0 < see_from;   // rows may see different tokens

            // scores of 16 rows x 16 tokens
            float x[2][4] = {};
            if constexpr (KIND != kE4M3) {
                const int r = tok + (lane & 7) + ((lane >> 4) << 3);
                const uint32_t row = ks + r * RB;
#pragma unroll
                for (int k = 0; k < DP / 16; ++k) {
                    uint32_t b[4];
                    ldmatrix_x4(b, row + piece<RB, false>(r, 2 * k + ((lane >> 3) & 1)) * 16);
                    mma_16816<BF16>(x[0], qf[k][0], qf[k][1], qf[k][2], qf[k][3], b[0], b[1]);
                    mma_16816<BF16>(x[1], qf[k][0], qf[k][1], qf[k][2], qf[k][3], b[2], b[3]);
                }
            } else {
#pragma unroll
                for (int n = 0; n < 2; ++n) {
                    const int r = tok + n * 8 + lr;
#pragma unroll
                    for (int q4 = 0; q4 < DP / 64; ++q4) {
                        const uint4 w = lds128(ks + r * RB + piece<RB, true>(r, q4 * 4 + tq) * 16);
                        const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            mma_16816<false>(x[n], qf[q4 * 4 + k][0], qf[q4 * 4 + k][1], qf[q4 * 4 + k][2],
                                             qf[q4 * 4 + k][3], e4m3x2_to_f16x2((uint16_t)(ww[k] & 0xffffu)),
                                             e4m3x2_to_f16x2((uint16_t)(ww[k] >> 16)));
                    }
                }
            }
#pragma unroll
            for (int n = 0; n < 2; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) x[n][e] *= xs[e >> 1];
            if (ok != 0xffffu || ragged) {
#pragma unroll
                for (int n = 0; n < 2; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int col = n * 8 + 2 * tq + (e & 1), j = j0 + col;
                        const bool seen = ((ok >> col) & 1) && j <= hi[e >> 1] && j > lo[e >> 1];
                        if (!seen) x[n][e] = -INFINITY;
                    }
            }

            // running maximum and sum
            float mn[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float t = fmaxf(fmaxf(x[0][2 * e], x[0][2 * e + 1]), fmaxf(x[1][2 * e], x[1][2 * e + 1]));
                t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 1));
                t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 2));
                mn[e] = fmaxf(m[e], t);
            }
            if (__any_sync(0xffffffffu, mn[0] > m[0] || mn[1] > m[1])) {
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float f = ex2_approx(m[e] - (mn[e] == -INFINITY ? 0.f : mn[e]));
                    m[e] = mn[e];
                    l[e] *= f;
#pragma unroll
                    for (int n = 0; n < C::DW / 8; ++n) {
                        o[n][2 * e] *= f;
                        o[n][2 * e + 1] *= f;
                    }
                }
            }
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const float mm = m[e] == -INFINITY ? 0.f : m[e];
#pragma unroll
                for (int n = 0; n < 2; ++n)
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        x[n][2 * e + k] = ex2_approx(x[n][2 * e + k] - mm);
                        l[e] += x[n][2 * e + k];
                    }
            }

            // times the values: the probabilities, rounded to the 16-bit type of the product
            // (off by 2^-8 of it at most for bf16, 2^-11 for fp16, to nearest, so over many tokens well
            // below the rounding of the output); l keeps them unrounded
            const uint32_t p0 = pack16<BF16>(x[0][0], x[0][1]), p1 = pack16<BF16>(x[0][2], x[0][3]);
            const uint32_t p2 = pack16<BF16>(x[1][0], x[1][1]), p3 = pack16<BF16>(x[1][2], x[1][3]);
            const int vr = tok + (lane & 15);
            const uint32_t vrow = vs + vr * RB;
            auto values = [&](auto clean) {
                // `clean`: infinities and NaN are taken out before the product, where a row must
                // not meet the values of a token that another row sees
                bool bad = false;
                auto scrub = [&](uint32_t w) {
                    if constexpr (!decltype(clean)::value) return w;
                    const uint32_t E = BF16 ? 0x7f80u : 0x7c00u;
                    if ((w & E) == E) { w &= 0xffff0000u; bad = true; }
                    if ((w & (E << 16)) == E << 16) { w &= 0xffffu; bad = true; }
                    return w;
                };
                if constexpr (KIND != kE4M3) {
#pragma unroll
                    for (int n = 0; n < C::DW / 8; n += 2) {
                        uint32_t b[4];
                        ldmatrix_x4_trans(b, vrow + piece<RB, false>(vr, wd * (C::DW / 8) + n + (lane >> 4)) * 16);
                        mma_16816<BF16>(o[n], p0, p1, p2, p3, scrub(b[0]), scrub(b[1]));
                        mma_16816<BF16>(o[n + 1], p0, p1, p2, p3, scrub(b[2]), scrub(b[3]));
                    }
                } else {
#pragma unroll
                    for (int n = 0; n < C::DW / 8; n += 4) {
                        // a piece holds 16 dimensions: as pairs of bytes, ldmatrix hands thread
                        // (lr, tq) dimensions 2 lr, 2 lr + 1 of tokens 2 tq, 2 tq + 1
                        uint32_t b[4];
                        ldmatrix_x4_trans(b, vrow + piece<RB, false>(vr, wd * (C::DW / 16) + n / 2 + (lane >> 4)) * 16);
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            const uint32_t w0 = __byte_perm(b[2 * k], 0, 0x3120);
                            const uint32_t w1 = __byte_perm(b[2 * k + 1], 0, 0x3120);
                            mma_16816<false>(o[n + 2 * k], p0, p1, p2, p3,
                                             scrub(e4m3x2_to_f16x2((uint16_t)(w0 & 0xffffu))),
                                             scrub(e4m3x2_to_f16x2((uint16_t)(w1 & 0xffffu))));
                            mma_16816<false>(o[n + 2 * k + 1], p0, p1, p2, p3,
                                             scrub(e4m3x2_to_f16x2((uint16_t)(w0 >> 16))),
                                             scrub(e4m3x2_to_f16x2((uint16_t)(w1 >> 16))));
                        }
                    }
                }
                return bad;
            };
            if (!ragged || a.T == 1) {
                values(std::false_type{});
            } else if (__any_sync(0xffffffffu, values(std::true_type{}))) {
                // the taken-out values, for the rows that do see them
#pragma unroll 1
                for (int jj = 0; jj < 16; ++jj) {
                    const int src = (lane & ~3) | ((jj & 7) >> 1);
                    float p[2];
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const float y0 = jj < 8 ? x[0][2 * e] : x[1][2 * e];
                        const float y1 = jj < 8 ? x[0][2 * e + 1] : x[1][2 * e + 1];
                        p[e] = __shfl_sync(0xffffffffu, (jj & 1) ? y1 : y0, src);
                    }
                    const int j = j0 + jj;
                    if (!((ok >> jj) & 1)) continue;
                    const unsigned char *const vb = s_stage + (i % kStages) * 2 * kHalfStage + kHalfStage +
                                                    (tok + jj) * RB;
#pragma unroll
                    for (int n = 0; n < C::DW / 8; ++n)
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            const int dd = wd * C::DW + (KIND == kE4M3 ? (n & ~1) * 8 + 4 * tq + 2 * k + (n & 1)
                                                                       : n * 8 + 2 * tq + k);
                            const int at = dd * C::ESZ;
                            const unsigned char *const e0 = vb + piece<RB, false>(tok + jj, at / 16) * 16 + at % 16;
                            float v;
                            if constexpr (KIND == kBF16)
                                v = __uint_as_float((uint32_t)*reinterpret_cast<const uint16_t *>(e0) << 16);
                            else if constexpr (KIND == kF16)
                                v = __half2float(__ushort_as_half(*reinterpret_cast<const uint16_t *>(e0)));
                            else
                                v = (*e0 & 0x7f) == 0x7f ? __uint_as_float(0x7fc00000u) : 0.f;
                            if (isfinite(v)) continue;
#pragma unroll
                            for (int e = 0; e < 2; ++e)
                                if (j <= hi[e] && j > lo[e]) o[n][2 * e + k] += p[e] * v;
                        }
                }
            }
        }

        if (d.tile == d.nt - 1 || i == n_tiles - 1) {   // the unit, or its part here, is done
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                l[e] += __shfl_xor_sync(0xffffffffu, l[e], 1);
                l[e] += __shfl_xor_sync(0xffffffffu, l[e], 2);
            }
            // the other warps of the same rows and dimensions join into wt = 0, one after the other
            constexpr int kWriters = WR * C::WD;
            constexpr int kRegs = C::DW / 2;
            constexpr int kAtOnce = kRegs < 64 / kWriters ? kRegs : 64 / kWriters;
#pragma unroll 1
            for (int src = 1; src < C::WT; ++src) {
                float f0[2] = {1.f, 1.f}, f1[2] = {0.f, 0.f};
                float *const buf = s_merge + (warp % kWriters) * kAtOnce * 32 + lane;
#pragma unroll
                for (int part = 0; part < kRegs / kAtOnce; ++part) {
                    if (wt == src) {
                        if (part == 0) s_stat[warp % kWriters][lane] = make_float4(m[0], m[1], l[0], l[1]);
#pragma unroll
                        for (int k = 0; k < kAtOnce; ++k) {
                            const int g = part * kAtOnce + k;
                            buf[k * 32] = o[g / 4][g % 4];
                        }
                    }
                    __syncthreads();
                    if (wt == 0) {
                        if (part == 0) {
                            const float4 y = s_stat[warp % kWriters][lane];
                            const float ym[2] = {y.x, y.y}, yl[2] = {y.z, y.w};
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                const float mx = fmaxf(m[e], ym[e]), ms = mx == -INFINITY ? 0.f : mx;
                                f0[e] = ex2_approx(m[e] - ms);
                                f1[e] = ex2_approx(ym[e] - ms);
                                m[e] = mx;
                                l[e] = l[e] * f0[e] + yl[e] * f1[e];
                            }
                        }
#pragma unroll
                        for (int k = 0; k < kAtOnce; ++k) {
                            const int g = part * kAtOnce + k, e = (g >> 1) & 1;
                            o[g / 4][g % 4] = o[g / 4][g % 4] * f0[e] + buf[k * 32] * f1[e];
                        }
                    }
                    __syncthreads();
                }
            }
            const bool whole = seg_tile == 0 && d.tile == d.nt - 1;
            const int slot2 = seg_tile > 0 ? 0 : 1;
            if (wt == 0) {
                const float vsc = KIND == kE4M3 && kv.v_scale ? __ldg(kv.v_scale + h) : 1.f;
                if (whole) {
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int r = rt * C::RMAX + wr * 16 + lr + 8 * e;
                        if (r >= rows_all) continue;
                        const int t = r / group, hq = h * group + r - t * group;
                        const int64_t row = ((int64_t)d.b * a.T + t) * a.Hq + hq;
                        const int64_t total = (int64_t)a.B * a.T * a.Hq;
                        if (!in_range(row, 1, total, a.dev_status)) continue;
                        const float inv = l[e] == 0.f ? 0.f : vsc / l[e];
                        uint16_t *const out = static_cast<uint16_t *>(a.out) + row * D;
                        if constexpr (KIND != kE4M3) {
#pragma unroll
                            for (int n = 0; n < C::DW / 8; ++n) {
                                const int dd = wd * C::DW + n * 8 + 2 * tq;
                                if (dd < D)
                                    *reinterpret_cast<uint32_t *>(out + dd) =
                                        pack16<BF16>(o[n][2 * e] * inv, o[n][2 * e + 1] * inv);
                            }
                        } else {
#pragma unroll
                            for (int n = 0; n < C::DW / 8; n += 2) {
                                const int dd = wd * C::DW + n * 8 + 4 * tq;
                                if (dd < D) {
                                    uint32_t *const w = reinterpret_cast<uint32_t *>(out + dd);
                                    w[0] = pack_out(a.q_bf16, o[n][2 * e] * inv, o[n + 1][2 * e] * inv);
                                    w[1] = pack_out(a.q_bf16, o[n][2 * e + 1] * inv, o[n + 1][2 * e + 1] * inv);
                                }
                            }
                        }
                        if (a.lse && wd == 0 && tq == 0)
                            a.lse[row] = l[e] == 0.f ? -INFINITY : (m[e] + log2f(l[e])) * kLn2;
                    }
                } else {
                    const int64_t p = (int64_t)c * 2 + slot2;
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int64_t r = p * C::RMAX + wr * 16 + lr + 8 * e;
                        if (!in_range(r, 1, (int64_t)G * 2 * C::RMAX, a.dev_status)) continue;
                        if (wd == 0 && tq == 0) part_ml[r] = make_float2(m[e], l[e]);
                        float *const po = part_o + r * DP + wd * C::DW;
                        if constexpr (KIND != kE4M3) {
#pragma unroll
                            for (int n = 0; n < C::DW / 8; ++n)
                                *reinterpret_cast<float2 *>(po + n * 8 + 2 * tq) =
                                    make_float2(o[n][2 * e], o[n][2 * e + 1]);
                        } else {
#pragma unroll
                            for (int n = 0; n < C::DW / 8; n += 2)
                                *reinterpret_cast<float4 *>(po + n * 8 + 4 * tq) =
                                    make_float4(o[n][2 * e] * vsc, o[n + 1][2 * e] * vsc,
                                                o[n][2 * e + 1] * vsc, o[n + 1][2 * e + 1] * vsc);
                        }
                    }
                }
            }
            // the block where a unit begins says who holds its parts
            if (tid == 0 && seg_tile == 0) {
                const int64_t unit = (int64_t)d.b * U + d.u;
                const int64_t end = t0 + i + (d.nt - 1 - d.tile);   // the unit's last tile
                const int last = (int)(((end + 1) * Ge - 1) / W);
                const int64_t at = by_unit ? unit : c;
                if ((by_unit || !whole) && in_range(at, 1, n_splits, a.dev_status)) {
                    Split sp;
                    sp.u_lo = d.u; sp.b = d.b; sp.c0 = c; sp.c1 = whole ? -1 : last;
                    splits[at] = sp;
                }
            }
        }
        if (more) note(i + 3, next);
    }
    cp_async_wait<0>();
}

// One block joins one row of one unit that several blocks worked on.
template <int DP>
__global__ void __launch_bounds__(kThreads)
paged_attn_join_kernel(const GdnAttnArgs a, const int RT, const int RMAX, const Split *const splits,
                       const float2 *const part_ml, const float *const part_o)
{
    wait_primary();
    __shared__ float s_o[4][DP];
    const Split sp = splits[blockIdx.x];
    if (sp.c1 < 0) return;
    const int H = a.cache.heads, D = a.cache.head_dim, group = a.Hq / H;
    const int h = sp.u_lo / RT, rt = sp.u_lo - h * RT;
    const int rl = blockIdx.y, r = rt * RMAX + rl;
    if (r >= a.T * group) return;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int np = sp.c1 - sp.c0 + 1;
    // part k: the first block's is its second, the others' are their first
    auto at = [&](int k) { return ((int64_t)(sp.c0 + k) * 2 + (k == 0 ? 1 : 0)) * RMAX + rl; };

    float top = -INFINITY;
    for (int k = lane; k < np; k += 32) top = fmaxf(top, part_ml[at(k)].x);
#pragma unroll
    for (int s = 16; s > 0; s >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, s));
    const float ms = top == -INFINITY ? 0.f : top;
    float sum = 0.f;
    for (int k = lane; k < np; k += 32) {
        const float2 ml = part_ml[at(k)];
        sum += ml.y * ex2_approx(ml.x - ms);
    }
    sum = gdn::warp_sum(sum);

    constexpr int PER = DP / 32;
    float acc[PER] = {};
#pragma unroll 4
    for (int k = warp; k < np; k += 4) {
        const float w = ex2_approx(part_ml[at(k)].x - ms);
        const float2 *const src = reinterpret_cast<const float2 *>(part_o + at(k) * DP) + lane;
#pragma unroll
        for (int e = 0; e < PER / 2; ++e) {
            const float2 y = src[e * 32];
            acc[2 * e] += w * y.x;
            acc[2 * e + 1] += w * y.y;
        }
    }
#pragma unroll
    for (int e = 0; e < PER / 2; ++e) {
        s_o[warp][e * 64 + 2 * lane] = acc[2 * e];
        s_o[warp][e * 64 + 2 * lane + 1] = acc[2 * e + 1];
    }
    __syncthreads();
    const int t = r / group, hq = h * group + r - t * group;
    const int64_t row = ((int64_t)sp.b * a.T + t) * a.Hq + hq;
    if (!in_range(row, 1, (int64_t)a.B * a.T * a.Hq, a.dev_status)) return;
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    for (int w = tid; w < D / 2; w += kThreads) {
        float y[2];
#pragma unroll
        for (int e = 0; e < 2; ++e)
            y[e] = (s_o[0][2 * w + e] + s_o[1][2 * w + e] + s_o[2][2 * w + e] + s_o[3][2 * w + e]) * inv;
        reinterpret_cast<uint32_t *>(static_cast<uint16_t *>(a.out) + row * D)[w] = pack_out(a.q_bf16, y[0], y[1]);
    }
    if (a.lse && tid == 0) a.lse[row] = sum == 0.f ? -INFINITY : (top + log2f(sum)) * kLn2;
}

// ------------------------------------------------------------------ host
int padded(int D) { return D <= 64 ? 64 : (D <= 128 ? 128 : 256); }
// warps over rows: as few as hold them; a 256-wide head leaves registers for 32 rows
int row_warps(int rows, int DP) { return rows <= 16 ? 1 : (rows <= 32 || DP == 256 ? 2 : 4); }
int max_blocks() { return 2 * sm_count(); }

struct Layout {
    int RT, RMAX, n_splits;
    uint64_t ml_at, o_at, bytes;
};

Layout layout(int B, int T, int Hq, int H, int D, int blocks)
{
    const int DP = padded(D), rows = T * (Hq / H);
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

template <int KIND, int DP, int WR>
cudaError_t launch(const GdnAttnArgs &a, cudaStream_t stream)
{
    using C = Cfg<KIND, DP, WR>;
    static DeviceOnce once;
    cudaError_t e = once.run([] {
        return cudaFuncSetAttribute(paged_attn_kernel<KIND, DP, WR>,
                                    cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
    });
    if (e != cudaSuccess) return e;
    const gdn_paged_cache &kv = a.cache;
    const Layout y = layout(a.B, a.T, a.Hq, kv.heads, kv.head_dim, max_blocks());
    // no more blocks than there can be tiles
    const int64_t cap = (int64_t)kv.width * kv.page_size;
    const double tiles = (double)a.B * kv.heads * y.RT * (double)((cap + C::TILE - 1) / C::TILE);
    const int blocks = tiles < max_blocks() ? (tiles < 1 ? 1 : (int)tiles) : max_blocks();
    unsigned char *const ws = static_cast<unsigned char *>(a.workspace);
    Split *const splits = reinterpret_cast<Split *>(ws);
    float2 *const ml = reinterpret_cast<float2 *>(ws + y.ml_at);
    float *const o = reinterpret_cast<float *>(ws + y.o_at);
    const int64_t units = (int64_t)a.B * kv.heads * y.RT;
    const int n_splits = (int)(units < blocks ? units : blocks);
    paged_attn_kernel<KIND, DP, WR><<<blocks, kThreads, C::SMEM, stream>>>(a, y.RT, splits, n_splits, ml, o);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    return launch_dependent(paged_attn_join_kernel<DP>, dim3(n_splits, y.RMAX), dim3(kThreads), 0,
                            stream, a, y.RT, y.RMAX, splits, ml, o);
}

template <int KIND>
cudaError_t dispatch(const GdnAttnArgs &a, cudaStream_t stream)
{
    const int DP = padded(a.cache.head_dim);
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
    (void)cache_dtype;
    const int blocks = gdn_attn::max_blocks();
    return blocks == 0 ? 0 : gdn_attn::layout(B, T, Hq, heads, D, blocks).bytes;
}

cudaError_t launch_paged_attn(const GdnAttnArgs &a, cudaStream_t stream)
{
    switch (a.cache.dtype) {
    case GDN_BF16: return gdn_attn::dispatch<gdn_attn::kBF16>(a, stream);
    case GDN_F16: return gdn_attn::dispatch<gdn_attn::kF16>(a, stream);
    default: return gdn_attn::dispatch<gdn_attn::kE4M3>(a, stream);
    }
}
