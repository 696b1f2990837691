// pages.cu -- the page table of the paged cache: growing, shrinking, forking and compacting its
// rows, with the copies of pages and states that follow.
//
// The tables are integers of a few megabytes at most; a call's time is the latency of its
// dependent steps.  Resize and compact run them in one cluster of blocks, whose barrier orders the
// steps (about half a microsecond each where a launch a step would cost two to three).
// The copies are HBM-bound (each byte read once and written once) and run in a second kernel
// over the whole GPU, brought up while the first one drains.  Everything is decided by scans in
// the order of the lists and of the page numbers, so a call has one result; atomics only count
// integers.
// Measured on a B200: 40000 pages of 64 KB in order, half used: 427 us, 6.15 TB/s of 6.46 (copy
// rate); 64 children of 16 requests with 6.4 MB of states each: 115 us with their growth, of which the
// states take 107 (80 were each parent read once from HBM: its children, pieces apart, make that twice);
// a decoding step's growth of 256 rows 8 to 11 us on up to 16384 pages, which one block passes over at
// once, and 20 us on 300000; 262144 pages given back and as many handed out 33 us.
#include <cooperative_groups.h>

#include "cache.cuh"

namespace gdn_pages {

namespace cg = cooperative_groups;
using namespace gdn_cache;
using gdn::in_range;

constexpr int kCluster = 16;            // planning blocks at most
constexpr int kThreads = 1024;          // of one
constexpr int kChunk = 256;             // table entries a warp takes at a time
constexpr int kPer = 16;                // pages a thread takes at a time at most, 32 apart
constexpr int kNear = 1024;             // listed rows whose plan is kept in shared memory
constexpr int kFewEntries = 24 * 1024;  // of the table, that one block changes faster than a cluster
constexpr int kSlots = 4096;            // of the table that finds rows listed twice
constexpr int kHashed = 3000;           // listed rows that it is used for
constexpr int kCopyThreads = 256;
constexpr int kCopyBytes = 16384;       // of a row a block copies at a time
constexpr int kMaxPools = 96;           // a launch (a kernel's arguments hold 4 KB)

struct Pool {
    unsigned char *data;
    int64_t stride, bytes;
    int first, width;                   // first piece of a row among all pools'; access width
};
struct Pools {
    Pool p[kMaxPools];
    int n, pieces;                      // pieces of a row over all pools
};

struct alignas(16) Row {                // what resize does to a listed row
    int row, had, want, first;          // pages before and after; first new page's place
    int len, copied, last, need;        // new length; a shared page is replaced, that page; new pages
};

__device__ __forceinline__ void tell(int32_t *status, int bit)
{
    if (status) atomicOr(status, bit);
}

__device__ __forceinline__ int pages_of(int len, int page) { return (int)(((int64_t)len + page - 1) / page); }

__device__ __forceinline__ bool length_ok(const gdn_page_table &t, int len)
{
    return len >= 0 && len <= (int64_t)t.width * t.page_size;
}

// exclusive prefix sum over the block's threads; *total is the same in all
template <typename T>
__device__ __forceinline__ T block_scan(T x, T *s_warp, T *total)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
    T incl = x;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const T y = __shfl_up_sync(0xffffffffu, incl, d);
        if (lane >= d) incl += y;
    }
    if (lane == 31) s_warp[warp] = incl;
    __syncthreads();
    T w = lane < nw ? s_warp[lane] : 0, wi = w;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const T y = __shfl_up_sync(0xffffffffu, wi, d);
        if (lane >= d) wi += y;
    }
    const T before = __shfl_sync(0xffffffffu, wi - w, warp);
    *total = __shfl_sync(0xffffffffu, wi, 31);
    __syncthreads();                    // s_warp is used again
    return before + incl - x;
}

// Which of the next 32 `per` pages from p on (below end) are used: bit `lane` of word e is page
// p + 32 e + lane.  A block takes 1024 `per` pages at a time, as few a warp as its share allows.
struct Used {
    uint32_t w[kPer];
    int left;                           // pages there are
    __device__ __forceinline__ uint32_t in(int e) const
    {
        const int n = left - 32 * e;
        return n >= 32 ? 0xffffffffu : (n <= 0 ? 0u : (1u << n) - 1);
    }
    __device__ __forceinline__ uint32_t open(int e) const { return in(e) & ~w[e]; }
    __device__ __forceinline__ void look(const int32_t *ref, int p, int end, int per)
    {
        const int lane = threadIdx.x & 31;
        left = min(max(end - p, 0), 32 * per);
        int v[kPer];
#pragma unroll
        for (int e = 0; e < kPer; ++e) v[e] = 32 * e + lane < left ? __ldcg(ref + p + 32 * e + lane) : 0;
#pragma unroll
        for (int e = 0; e < kPer; ++e) {
            w[e] = 0;
            if (32 * e < left) w[e] = __ballot_sync(0xffffffffu, v[e] > 0);
        }
    }
    __device__ __forceinline__ int used() const
    {
        int n = 0;
#pragma unroll
        for (int e = 0; e < kPer; ++e)
            if (32 * e < left) n += __popc(w[e]);
        return n;
    }
};
__device__ __forceinline__ int words_of(int pages) { return min(kPer, (pages + kThreads - 1) / kThreads); }

// exclusive prefix sum over the block's warps of a value that a warp's lanes share
__device__ __forceinline__ int warps_scan(int x, int *s_warp, int *total)
{
    return block_scan<int>((threadIdx.x & 31) == 0 ? x : 0, s_warp, total);
}

// copy piece `item` of row src to row dst
__device__ __forceinline__ void copy_piece(const Pools &ps, int item, int64_t src, int64_t dst, int32_t *status)
{
    int lo = 0, hi = ps.n - 1;          // the last pool whose first piece is <= item
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (ps.p[mid].first <= item) lo = mid; else hi = mid - 1;
    }
    const Pool &p = ps.p[lo];
    const int64_t at = (int64_t)(item - p.first) * kCopyBytes;
    const int64_t n = p.bytes - at < kCopyBytes ? p.bytes - at : kCopyBytes;
    if (!in_range(at, n, p.bytes, status)) return;
    const unsigned char *const s = p.data + src * p.stride + at;
    unsigned char *const d = p.data + dst * p.stride + at;
    const int tid = threadIdx.x;
    if (p.width == 16) {
        constexpr int kHold = kCopyBytes / 16 / kCopyThreads;
        const uint4 *const s16 = reinterpret_cast<const uint4 *>(s);
        uint4 *const d16 = reinterpret_cast<uint4 *>(d);
        const int w = (int)(n / 16);
        uint4 x[kHold];
#pragma unroll
        for (int k = 0; k < kHold; ++k)
            if (tid + k * kCopyThreads < w) x[k] = __ldcs(s16 + tid + k * kCopyThreads);
#pragma unroll
        for (int k = 0; k < kHold; ++k)
            if (tid + k * kCopyThreads < w) __stcs(d16 + tid + k * kCopyThreads, x[k]);
    } else if (p.width == 4) {
        const uint32_t *const s4 = reinterpret_cast<const uint32_t *>(s);
        for (int i = tid; i < (int)(n / 4); i += kCopyThreads) reinterpret_cast<uint32_t *>(d)[i] = __ldcs(s4 + i);
    } else if (p.width == 2) {
        const uint16_t *const s2 = reinterpret_cast<const uint16_t *>(s);
        for (int i = tid; i < (int)(n / 2); i += kCopyThreads) reinterpret_cast<uint16_t *>(d)[i] = __ldcs(s2 + i);
    } else {
        for (int i = tid; i < (int)n; i += kCopyThreads) d[i] = __ldcs(s + i);
    }
}

// Table entries renamed by `map` (compact): a warp takes a row of the table at a time.
__device__ __noinline__ void rename_rows(const gdn_page_table &t, const int32_t *map, int32_t *status)
{
    const int lane = threadIdx.x & 31;
    for (int s = blockIdx.x * (kCopyThreads / 32) + (threadIdx.x >> 5); s < t.rows;
         s += gridDim.x * (kCopyThreads / 32)) {
        const int len = __ldg(t.seq_lens + s);
        if (!length_ok(t, len)) {
            if (lane == 0) tell(status, GDN_DEV_BAD_LENGTH);
            continue;
        }
        int32_t *const e = t.block_table + s * t.table_stride;
        const int had = pages_of(len, t.page_size);
        for (int j = lane; j < had; j += 32) {
            const int id = in_range(j, 1, t.width, status) ? e[j] : -1;
            const int to = (uint32_t)id < (uint32_t)t.num_pages ? __ldcg(map + id) : -1;
            if (to < 0)
                tell(status, GDN_DEV_BAD_PAGE);
            else if (to != id)
                e[j] = to;
        }
    }
}

// The copies that a plan wrote down: pairs[k] = (src, dst), disjoint.  With a map, the table's
// entries are renamed too.
__global__ void __launch_bounds__(kCopyThreads)
copy_pairs_kernel(const __grid_constant__ Pools ps, const int2 *pairs, const int *count,
                  const int num_rows, const __grid_constant__ gdn_page_table t, const int32_t *map, int32_t *status)
{
    wait_primary();
    const int64_t items = (int64_t)*count * ps.pieces;
    for (int64_t i = blockIdx.x; i < items; i += gridDim.x) {
        const int2 p = pairs[i / ps.pieces];
        if (in_range(p.x, 1, num_rows, status) && in_range(p.y, 1, num_rows, status))
            copy_piece(ps, (int)(i % ps.pieces), p.x, p.y, status);
    }
    if (map) rename_rows(t, map, status);
}

// ------------------------------------------------------------------ resize
// Workspace: count | pairs [n] | a copy of the rows for each block [8][n] | free pages [P]
struct ResizeWork {
    int *count;
    int2 *pairs;
    Row *rows;
    int *free_list;
};

__global__ void __launch_bounds__(kThreads, 1)
resize_kernel(const __grid_constant__ gdn_page_table t, const int32_t *row_list, const int32_t *new_lens,
              const int n, const ResizeWork ws, int32_t *status)
{
    cg::cluster_group cluster = cg::this_cluster();
    int blocks = (int)cluster.num_blocks();
    const int rank = (int)cluster.block_rank();
    const int tid = threadIdx.x, lane = tid & 31;
    __shared__ int s_warp[32];
    __shared__ long long s_wide[32];
    __shared__ int s_most[2];
    __shared__ int s_free;
    __shared__ Row s_rows[kNear];
    static_assert(kSlots * sizeof(int) <= sizeof(s_rows), "the table and the rows share their place");
    int *const s_key = reinterpret_cast<int *>(s_rows);
    constexpr int kTwice = (int)0x80000000;     // (-1 is a free slot: no row is 0x7fffffff)
    Row *const rows = n <= kNear ? s_rows : ws.rows + (int64_t)rank * n;
    launch_dependents();
    // the steps' order: among the blocks, or the threads of the only one
    auto meet = [&]() {
        if (blocks > 1) cluster.sync(); else __syncthreads();
    };

    // 1. what is asked of each row (every block works it out for itself).  Rows listed twice meet in
    //    a table in shared memory, or, of more than kHashed, are looked for one by one.
    if (tid == 0) s_most[0] = s_most[1] = 0;
    if (n <= kHashed) {
        for (int k = tid; k < kSlots; k += kThreads) s_key[k] = -1;
        __syncthreads();
        for (int i = tid; i < n; i += kThreads) {
            const int r = __ldg(row_list + i);
            if (r < 0 || r >= t.rows) continue;
            // (at most kHashed rows: a free slot is found)
            for (uint32_t h = (uint32_t)r * 2654435769u >> 20;; h = (h + 1) % kSlots) {
                const int was = atomicCAS(s_key + h, -1, r);
                if (was == r || was == (r | kTwice)) {
                    s_key[h] = r | kTwice;      // (whoever writes it, writes the same)
                    break;
                }
                if (was == -1) break;
            }
        }
        __syncthreads();
    }
    auto listed_twice = [&](int r) {
        for (uint32_t h = (uint32_t)r * 2654435769u >> 20;; h = (h + 1) % kSlots) {
            const int k = s_key[h];
            if (k == r) return false;
            if (k == (r | kTwice)) return true;
        }
    };
    for (int i0 = 0; i0 < n; i0 += kThreads) {
        const int i = i0 + tid;
        const int r = i < n ? __ldg(row_list + i) : -1;
        const bool there = r >= 0 && r < t.rows;
        const int old = there ? __ldcg(t.seq_lens + r) : 0, len = i < n ? __ldg(new_lens + i) : 0;
        bool twice = false;
        if (n <= kHashed) {
            twice = there && listed_twice(r);
        } else {
            int times = 0;
            for (int k0 = 0; k0 < n; k0 += kSlots) {
                __syncthreads();
                for (int k = tid; k < kSlots; k += kThreads) s_key[k] = k0 + k < n ? __ldg(row_list + k0 + k) : -1;
                __syncthreads();
                for (int k = 0; k < kSlots / 4 && i < n; ++k) {
                    const int4 q = reinterpret_cast<const int4 *>(s_key)[k];
                    times += (q.x == r) + (q.y == r) + (q.z == r) + (q.w == r);
                }
            }
            twice = times > 1;
        }
        Row x = {-1, 0, 0, 0, 0, 0, 0, 0};
        int bad = 0;
        if (r >= t.rows) {
            bad = GDN_DEV_BAD_SLOT;
        } else if (r >= 0) {
            if (twice) {
                bad = GDN_DEV_CONFLICT;
            } else if (!length_ok(t, old) || !length_ok(t, len)) {
                bad = GDN_DEV_BAD_LENGTH;
            } else {
                x.row = r;
                x.had = pages_of(old, t.page_size);
                x.want = pages_of(len, t.page_size);
                x.len = len;
                x.copied = len > old && old % t.page_size != 0;   // until the count is seen
                if (x.had > x.want) atomicMax(&s_most[0], x.had - x.want);
                if (x.want > x.had || x.copied) atomicMax(&s_most[1], x.want - x.had + 1);
            }
        }
        if (bad && rank == 0) tell(status, bad);
        if (n <= kNear) __syncthreads();        // the table has been read: the rows take its place
        if (i < n) rows[i] = x;
    }
    __syncthreads();
    const int most_gone = s_most[0], most_new = s_most[1];
    // a wide table of which little changes (a step of decoding): the first block does it alone
    if (blocks > 1 && t.num_pages <= kThreads * kPer && n * ((int64_t)most_gone + most_new) <= kFewEntries) {
        if (rank > 0) return;
        blocks = 1;
    }
    const int warps = blocks * (kThreads / 32), gw = (tid >> 5) * blocks + rank;    // of those at work

    // 2. pages past the new lengths go back; a warp takes kChunk entries of a row at a time
    for (int j00 = 0; j00 < most_gone; j00 += kChunk)
        for (int i = gw; i < n; i += warps) {
            const Row x = rows[i];
            const int j0 = x.want + j00;
            if (x.row < 0 || j0 >= x.had) continue;
            int32_t *const e = t.block_table + x.row * t.table_stride;
            int id[kChunk / 32];
#pragma unroll
            for (int k = 0; k < kChunk / 32; ++k) {
                const int j = j0 + k * 32 + lane;
                id[k] = j < x.had && in_range(j, 1, t.width, status) ? e[j] : 0;
            }
#pragma unroll
            for (int k = 0; k < kChunk / 32; ++k) {
                const int j = j0 + k * 32 + lane;
                if (j >= x.had) continue;
                if ((uint32_t)id[k] < (uint32_t)t.num_pages)
                    atomicSub(t.ref_count + id[k], 1);
                else
                    tell(status, GDN_DEV_BAD_PAGE);
                if (in_range(j, 1, t.width, status)) e[j] = -1;
            }
        }
    meet();

    // 3. how many pages each row takes, and where its share begins (every block for itself); what is
    //    asked for may pass 32 bits, what there is does not
    long long total = 0;
    int copies = 0;
    if (most_new > 0) {
        for (int i0 = 0; i0 < n; i0 += kThreads) {
            const int i = i0 + tid;
            int need = 0;
            Row x;
            if (i < n) {
                x = rows[i];
                if (x.row >= 0 && x.copied && in_range(x.had - 1, 1, t.width, status)) {
                    x.last = __ldcg(t.block_table + x.row * t.table_stride + x.had - 1);
                    if ((uint32_t)x.last >= (uint32_t)t.num_pages) {
                        if (rank == 0) tell(status, GDN_DEV_BAD_PAGE);
                        x.row = -1;
                    } else {
                        x.copied = __ldcg(t.ref_count + x.last) > 1;
                    }
                }
                if (x.row >= 0) need = max(x.want - x.had, 0) + x.copied;
            }
            long long sum;
            const long long before = total + block_scan<long long>(need, s_wide, &sum);
            if (i < n) {
                x.first = (int)(before < t.num_pages ? before : t.num_pages);
                x.need = need;
                rows[i] = x;
            }
            total += sum;
        }
    }

    // 4. the lowest free pages, in order: each block counts its share of the pages, the counts
    //    are exchanged, then it writes its part of the list
    int free_all = 0;
    if (total > 0) {
        const int share = ((t.num_pages + blocks - 1) / blocks + 31) / 32 * 32;
        const int p0 = min(rank * share, t.num_pages), p1 = min(p0 + share, t.num_pages);
        const int per = words_of(p1 - p0), pass = kThreads * per;
        const bool once = p1 - p0 <= pass;      // what is counted need not be read again
        const int warp_at = (tid >> 5) * 32 * per;
        Used u;
        int at = 0, sum;
        if (blocks > 1) {
            int mine = 0;
            for (int q = p0; q < p1; q += pass) {
                u.look(t.ref_count, q + warp_at, p1, per);
                mine += u.left - u.used();
            }
            warps_scan(mine, s_warp, &sum);
            if (tid == 0) s_free = sum;
            cluster.sync();
            for (int k = 0; k < blocks; ++k) {
                const int f = *cluster.map_shared_rank(&s_free, k);
                if (k < rank) at += f;
                free_all += f;
            }
        }
        for (int q = p0; q < p1 && at < total; q += pass) {
            const int p = q + warp_at;
            if (blocks == 1 || !once) u.look(t.ref_count, p, p1, per);
            int k = at + warps_scan(u.left - u.used(), s_warp, &sum);
            k = __shfl_sync(0xffffffffu, k, 0);
#pragma unroll
            for (int e = 0; e < kPer; ++e) {
                if (32 * e >= u.left) break;
                const uint32_t open = u.open(e);
                const int kk = k + __popc(open & ((1u << lane) - 1));
                if ((open >> lane & 1) && kk < total && in_range(kk, 1, t.num_pages, status))
                    ws.free_list[kk] = p + 32 * e + lane;
                k += __popc(open);
            }
            at += sum;
        }
        if (blocks == 1) free_all = at;     // as many as are needed, or all there are
    }
    meet();

    // 5. rows that fit take their pages
    for (int i0 = 0; i0 < n; i0 += kThreads) {
        const int i = i0 + tid;
        int copy = 0;
        Row x;
        if (i < n) {
            x = rows[i];
            if (x.row >= 0 && x.need > free_all - x.first && x.need > 0) {
                if (rank == 0) tell(status, GDN_DEV_NO_PAGES);
                rows[i].row = x.row = -1;
            }
            copy = x.row >= 0 && x.need > 0 && x.copied;
        }
        int sum;
        const int k = copies + block_scan<int>(copy, s_warp, &sum);
        copies += sum;
        if (rank == 0 && i < n && x.row >= 0) {
            t.seq_lens[x.row] = x.len;
            if (copy && in_range(k, 1, n, status) && in_range(x.first, 1, t.num_pages, status)) {
                atomicSub(t.ref_count + x.last, 1);
                ws.pairs[k] = make_int2(x.last, __ldcg(ws.free_list + x.first));
            }
        }
    }
    if (rank == 0 && tid == 0) *ws.count = copies;
    __syncthreads();
    for (int j00 = 0; total > 0 && j00 < most_new; j00 += kChunk)
        for (int i = gw; i < n; i += warps) {
            const Row x = rows[i];
            if (x.row < 0 || j00 >= x.need) continue;
            int32_t *const e = t.block_table + x.row * t.table_stride + x.had - x.copied;
            int id[kChunk / 32];
#pragma unroll
            for (int k = 0; k < kChunk / 32; ++k) {
                const int j = j00 + k * 32 + lane;
                id[k] = j < x.need && in_range(x.had - x.copied + j, 1, t.width, status) &&
                                in_range(x.first + j, 1, t.num_pages, status)
                            ? __ldcg(ws.free_list + x.first + j) : -1;
            }
#pragma unroll
            for (int k = 0; k < kChunk / 32; ++k)
                if (id[k] >= 0 && in_range(id[k], 1, t.num_pages, status)) {
                    e[j00 + k * 32 + lane] = id[k];
                    t.ref_count[id[k]] = 1;
                }
        }
    if (blocks > 1) cluster.sync();     // no block leaves while another may read its shared memory
}

// ------------------------------------------------------------------ compact
// Workspace: count, rank of page U | pairs [P] | used pages by rank [P] | free pages by rank [P]
struct CompactWork {
    int *count;
    int2 *pairs;
    int *used, *open;
};

__global__ void __launch_bounds__(kThreads, 1)
compact_kernel(const __grid_constant__ gdn_page_table t, int32_t *const map, const CompactWork ws, int32_t *status)
{
    cg::cluster_group cluster = cg::this_cluster();
    const int blocks = (int)cluster.num_blocks(), rank = (int)cluster.block_rank(), tid = threadIdx.x;
    __shared__ int s_warp[32];
    __shared__ int s_used;
    launch_dependents();
    const int P = t.num_pages, lane = tid & 31;
    const int share = ((P + blocks - 1) / blocks + 31) / 32 * 32;
    const int p0 = min(rank * share, P), p1 = min(p0 + share, P);
    const int per = words_of(p1 - p0), pass = kThreads * per;
    const bool once = p1 - p0 <= pass;          // what is counted need not be read again
    const int warp_at = (tid >> 5) * 32 * per;
    // the steps' order: among the blocks, or the threads of the only one
    auto meet = [&]() {
        if (blocks > 1) cluster.sync(); else __syncthreads();
    };
    Used u;
    int mine = 0, sum;
    for (int q = p0; q < p1; q += pass) {
        u.look(t.ref_count, q + warp_at, p1, per);
        mine += u.used();
    }
    const int mine_at = warps_scan(mine, s_warp, &sum);
    int at = 0, U = sum;
    if (blocks > 1) {
        if (tid == 0) s_used = sum;
        cluster.sync();
        U = 0;
        for (int k = 0; k < blocks; ++k) {
            const int f = *cluster.map_shared_rank(&s_used, k);
            if (k < rank) at += f;
            U += f;
        }
    }
    // Of the pages in order, `at` are used before p.  A used page of number >= U is the
    // (at - used before U)-th to move, a free one below U the (p - at)-th place.
    for (int q0 = p0; q0 < p1; q0 += pass) {
        const int p = q0 + warp_at;
        int k = at + mine_at;
        if (!once) {
            u.look(t.ref_count, p, p1, per);
            k = at + warps_scan(u.used(), s_warp, &sum);
            at += sum;
        }
        k = __shfl_sync(0xffffffffu, k, 0);
#pragma unroll
        for (int e = 0; e < kPer; ++e) {
            if (32 * e >= u.left) break;
            const int q = p + 32 * e + lane, kk = k + __popc(u.w[e] & ((1u << lane) - 1));
            k += __popc(u.w[e]);
            if (!(u.in(e) >> lane & 1)) continue;
            const bool is = u.w[e] >> lane & 1;
            if (q == U) ws.count[1] = kk;
            map[q] = is ? q : -1;
            if (is && q >= U && in_range(kk, 1, P, status)) ws.used[kk] = q;
            if (!is && q < U && in_range(q - kk, 1, P, status)) ws.open[q - kk] = q;
        }
    }
    meet();
    const int below = U < P ? __ldcg(ws.count + 1) : U;     // used pages of number < U
    const int moves = U - below;
    for (int k = rank * kThreads + tid; k < moves; k += blocks * kThreads) {
        if (!in_range(below + k, 1, P, status)) continue;
        const int src = __ldcg(ws.used + below + k), dst = __ldcg(ws.open + k);
        if (!in_range(src, 1, P, status) || !in_range(dst, 1, P, status)) continue;
        t.ref_count[dst] = __ldcg(t.ref_count + src);
        t.ref_count[src] = 0;
        map[src] = dst;
        ws.pairs[k] = make_int2(src, dst);
    }
    if (rank == 0 && tid == 0) ws.count[0] = moves;
    if (blocks > 1) cluster.sync();     // no block leaves while another may read its shared memory
}

// ------------------------------------------------------------------ fork
// Blocks [0, n) rename table rows, the others copy pieces of the pools.  Which pairs stand
// depends on the two lists alone, so every block checks its own pair.
__global__ void __launch_bounds__(kCopyThreads)
fork_kernel(const __grid_constant__ Pools ps, const gdn_page_table t, const int32_t *parents,
            const int32_t *children, const int n, const int table_blocks, int32_t *status)
{
    const int tid = threadIdx.x;
    const int64_t items = table_blocks + (int64_t)n * ps.pieces;
    for (int64_t i = blockIdx.x; i < items; i += gridDim.x) {
        const bool table = i < table_blocks;
        const int k = table ? (int)i : (int)((i - table_blocks) / ps.pieces);
        const int p = __ldg(parents + k), c = __ldg(children + k);
        if (p < 0 || c < 0) continue;
        if (p >= t.rows || c >= t.rows) {
            if (table && tid == 0) tell(status, GDN_DEV_BAD_SLOT);
            continue;
        }
        const int len = __ldg(t.seq_lens + p);      // a parent is no child: nobody writes it
        bool clash = p == c;
        for (int q = tid; q < n; q += kCopyThreads) {
            const int qp = __ldg(parents + q), qc = __ldg(children + q);
            if (q != k && qp >= 0 && qc >= 0 && (qc == c || qp == c || qc == p)) clash = true;
        }
        clash = __syncthreads_or(clash);
        if (clash || !length_ok(t, len)) {
            if (table && tid == 0) tell(status, clash ? GDN_DEV_CONFLICT : GDN_DEV_BAD_LENGTH);
            continue;
        }
        if (!table) {
            copy_piece(ps, (int)((i - table_blocks) % ps.pieces), p, c, status);
            continue;
        }
        const int old = *reinterpret_cast<const volatile int32_t *>(t.seq_lens + c);
        __syncthreads();                            // read by all before it is written
        const int want = pages_of(len, t.page_size);
        const int had = length_ok(t, old) ? pages_of(old, t.page_size) : 0;
        const int32_t *const from = t.block_table + p * t.table_stride;
        int32_t *const to = t.block_table + c * t.table_stride;
        for (int j = tid; j < max(had, want); j += kCopyThreads) {
            if (!in_range(j, 1, t.width, status)) break;
            const int give = j < had ? to[j] : 0, take = j < want ? __ldg(from + j) : -1;
            if (j < had) {
                if ((uint32_t)give < (uint32_t)t.num_pages)
                    atomicSub(t.ref_count + give, 1);
                else
                    tell(status, GDN_DEV_BAD_PAGE);
            }
            if (j < want) {
                if ((uint32_t)take < (uint32_t)t.num_pages)
                    atomicAdd(t.ref_count + take, 1);
                else
                    tell(status, GDN_DEV_BAD_PAGE);
            }
            to[j] = take;
        }
        if (tid == 0) {
            t.seq_lens[c] = len;
            if (!length_ok(t, old)) tell(status, GDN_DEV_BAD_LENGTH);
        }
    }
}

// ------------------------------------------------------------------ host
int access_width(const gdn_pool &p)
{
    const uint64_t x = (uint64_t)(uintptr_t)p.data | (uint64_t)p.row_stride | (uint64_t)p.row_bytes;
    return x % 16 == 0 ? 16 : (x % 4 == 0 ? 4 : (x % 2 == 0 ? 2 : 1));
}

// pools [first, first + kMaxPools) of the call
Pools take_pools(const gdn_pool *pools, int n_pools, int first)
{
    Pools ps;
    ps.n = ps.pieces = 0;
    for (int i = first; i < n_pools && ps.n < kMaxPools; ++i) {
        Pool &p = ps.p[ps.n++];
        p.data = static_cast<unsigned char *>(pools[i].data);
        p.stride = pools[i].row_stride;
        p.bytes = pools[i].row_bytes;
        p.first = ps.pieces;
        p.width = access_width(pools[i]);
        ps.pieces += (int)((p.bytes + kCopyBytes - 1) / kCopyBytes);
    }
    return ps;
}

unsigned copy_blocks(int64_t items)
{
    const int64_t most = 8 * (int64_t)sm_count();   // resident blocks of kCopyThreads
    return (unsigned)(items < 1 ? 1 : (items < most ? items : most));
}

cudaError_t launch_copies(const gdn_page_table &t, const gdn_pool *pools, int n_pools,
                          const int2 *pairs, const int *count, int64_t most_pairs,
                          const int32_t *map, int32_t *status, cudaStream_t stream)
{
    for (int first = 0; first < n_pools || (first == 0 && map); first += kMaxPools) {
        const Pools ps = take_pools(pools, n_pools, first);
        int64_t items = most_pairs * ps.pieces;
        const int32_t *const m = first == 0 ? map : nullptr;
        if (m) {
            const int64_t renames = t.rows / (kCopyThreads / 32) + 1;
            items = items > renames ? items : renames;
        }
        const cudaError_t e = launch_dependent(copy_pairs_kernel, dim3(copy_blocks(items)),
                                               dim3(kCopyThreads), 0, stream, ps, pairs, count,
                                               t.num_pages, t, m, status);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

// Blocks of a large plan: sixteen where the device can place such a cluster (more than the eight
// that every one can), asked once per device.
template <typename K>
cudaError_t largest_cluster(K kernel, std::atomic<int> (&known)[32], int *blocks)
{
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    *blocks = dev < 32 ? known[dev].load(std::memory_order_acquire) : 0;
    if (*blocks > 0) return cudaSuccess;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(kCluster);
    cfg.blockDim = dim3(kThreads);
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = kCluster;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess || n < 1) {
        cudaGetLastError();
        *blocks = 8;
    } else {
        *blocks = kCluster;
    }
    if (dev < 32) known[dev].store(*blocks, std::memory_order_release);
    return cudaSuccess;
}

template <typename... KA, typename... A>
cudaError_t launch_cluster(void (*kernel)(KA...), int blocks, cudaStream_t stream, A &&...args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(blocks);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = stream;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = blocks;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, KA(args)...);
}

// One block for tables that it passes over at once and lists that may change up to kFewEntries
// entries; else a cluster.  Two calls of 16, 128, 200, 400 rows on rows of 129 entries: 18, 24, 29,
// 41 us on one block, 26, 28, 29, 30 us on a cluster.
bool small_resize(const gdn_page_table &t, int n)
{
    return t.num_pages <= kThreads * kPer && (int64_t)n * t.width <= kFewEntries;
}
// 3000, 6000, 12000 pages in order: 12, 19.5, 31 us on one block, 16, 21, 31 us on a cluster.
bool small_compact(const gdn_page_table &t) { return t.num_pages <= kThreads * 8; }

uint64_t up16(uint64_t x) { return (x + 15) / 16 * 16; }

}  // namespace gdn_pages

uint64_t page_workspace_bytes(int32_t num_pages, int32_t n)
{
    using namespace gdn_pages;
    if (n > 0)
        return 16 + up16((uint64_t)n * sizeof(int2)) + (uint64_t)kCluster * n * sizeof(Row) +
               up16((uint64_t)num_pages * 4);
    return 16 + up16((uint64_t)num_pages * sizeof(int2)) + 2 * up16((uint64_t)num_pages * 4);
}

cudaError_t launch_page_resize(const gdn_page_table &t, const int32_t *row_list,
                               const int32_t *new_lens, int32_t n, const gdn_pool *pools,
                               int32_t n_pools, void *workspace, int32_t *dev_status,
                               cudaStream_t stream)
{
    using namespace gdn_pages;
    unsigned char *const w = static_cast<unsigned char *>(workspace);
    ResizeWork ws;
    ws.count = reinterpret_cast<int *>(w);
    ws.pairs = reinterpret_cast<int2 *>(w + 16);
    unsigned char *const r = w + 16 + up16((uint64_t)n * sizeof(int2));
    ws.rows = reinterpret_cast<Row *>(r);
    ws.free_list = reinterpret_cast<int *>(r + (uint64_t)kCluster * n * sizeof(Row));
    static std::atomic<int> known[32];
    int blocks = 1;
    cudaError_t e = small_resize(t, n) ? cudaSuccess : largest_cluster(resize_kernel, known, &blocks);
    if (e == cudaSuccess)
        e = launch_cluster(resize_kernel, blocks, stream, t, row_list, new_lens, n, ws, dev_status);
    if (e != cudaSuccess) return e;
    return launch_copies(t, pools, n_pools, ws.pairs, ws.count, n, nullptr, dev_status, stream);
}

cudaError_t launch_page_compact(const gdn_page_table &t, int32_t *page_map, const gdn_pool *pools,
                                int32_t n_pools, void *workspace, int32_t *dev_status,
                                cudaStream_t stream)
{
    using namespace gdn_pages;
    unsigned char *const w = static_cast<unsigned char *>(workspace);
    CompactWork ws;
    ws.count = reinterpret_cast<int *>(w);
    ws.pairs = reinterpret_cast<int2 *>(w + 16);
    unsigned char *const u = w + 16 + up16((uint64_t)t.num_pages * sizeof(int2));
    ws.used = reinterpret_cast<int *>(u);
    ws.open = reinterpret_cast<int *>(u + up16((uint64_t)t.num_pages * 4));
    static std::atomic<int> known[32];
    int blocks = 1;
    cudaError_t e = small_compact(t) ? cudaSuccess : largest_cluster(compact_kernel, known, &blocks);
    if (e == cudaSuccess) e = launch_cluster(compact_kernel, blocks, stream, t, page_map, ws, dev_status);
    if (e != cudaSuccess) return e;
    return launch_copies(t, pools, n_pools, ws.pairs, ws.count, t.num_pages / 2, page_map,
                         dev_status, stream);
}

cudaError_t launch_page_fork(const gdn_page_table &t, const int32_t *parents,
                             const int32_t *children, int32_t n, const gdn_pool *pools,
                             int32_t n_pools, int32_t *dev_status, cudaStream_t stream)
{
    using namespace gdn_pages;
    for (int first = 0; first == 0 || first < n_pools; first += kMaxPools) {
        const Pools ps = take_pools(pools, n_pools, first);
        const int table_blocks = first == 0 ? n : 0;
        const int64_t items = table_blocks + (int64_t)n * ps.pieces;
        fork_kernel<<<copy_blocks(items), kCopyThreads, 0, stream>>>(ps, t, parents, children, n,
                                                                     table_blocks, dev_status);
        const cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}
