// kv_append.cu -- new keys and values to the pages of their positions.
//
// HBM-bound: every value is read once and written once, 4 bytes a value in 16 bits and 3 into 8.
// A block takes a few tokens, all their heads, keys and values.  Its first loads are issued
// before the tokens' places are known (a chain of four dependent loads: offsets, slot, length,
// page), so the two latencies overlap; then each thread stores what it holds.
#include "cache.cuh"

namespace gdn_append {

using namespace gdn_cache;
using gdn::in_range;

constexpr int kThreads = 256;
constexpr int kHold = 4;         // 16-byte pieces a thread holds at a time
constexpr int kMaxTokens = 32;   // tokens a block

// eight 16-bit values -> eight e4m3 numbers of x / scale
__device__ __forceinline__ uint2 quantise(const uint4 &w, bool bf16, float scale)
{
    const uint32_t in[4] = {w.x, w.y, w.z, w.w};
    uint32_t out[2] = {0u, 0u};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        float lo, hi;
        if (bf16) {
            lo = __uint_as_float(in[k] << 16);
            hi = __uint_as_float(in[k] & 0xffff0000u);
        } else {
            lo = __half2float(__ushort_as_half((unsigned short)(in[k] & 0xffffu)));
            hi = __half2float(__ushort_as_half((unsigned short)(in[k] >> 16)));
        }
        // one rounding to float32, then one to e4m3 (to nearest even; past 448, infinities too,
        // to the largest number; a NaN stays one)
        const __nv_fp8x2_storage_t y = __nv_cvt_float2_to_fp8x2(
            make_float2(__fdiv_rn(lo, scale), __fdiv_rn(hi, scale)), __NV_SATFINITE, __NV_E4M3);
        out[k / 2] |= (uint32_t)y << (16 * (k & 1));
    }
    return make_uint2(out[0], out[1]);
}

// where token n goes: element offset of its head 0 in the cache, or -1
__device__ int64_t place(const GdnAppendArgs &a, int64_t n)
{
    const gdn_paged_cache &kv = a.cache;
    int b;
    int64_t end;
    if (a.row_offsets) {
        // The request with s <= n < e; offsets ascend, so it is the last whose s is <= n (empty
        // requests before it end at or before n).
        int lo = 0, hi = a.B;        // offsets[lo] <= n < offsets[hi], were they sentinels
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (__ldg(a.row_offsets + mid) <= n)
                lo = mid;
            else
                hi = mid;
        }
        b = lo;
        if (n < __ldg(a.row_offsets + b)) return -1;    // ahead of the first request
        end = __ldg(a.row_offsets + b + 1);
        if (end > a.N) end = a.N;
        if (n >= end) return -1;                        // behind the last one
    } else {
        const int64_t T = a.N / a.B;
        b = (int)(n / T);
        end = (int64_t)(b + 1) * T;
    }
    const int slot = a.slots ? __ldg(a.slots + b) : b;
    if (slot < 0) return -1;
    int bad = 0;
    int64_t at = -1;
    if (slot >= kv.rows) {
        bad = GDN_DEV_BAD_SLOT;
    } else {
        const int64_t pos = (int64_t)__ldg(kv.seq_lens + slot) - (end - n);
        if (pos < 0 || pos >= (int64_t)kv.width * kv.page_size) {
            bad = GDN_DEV_BAD_LENGTH;
        } else {
            const int pg = (int)((uint32_t)pos / (uint32_t)kv.page_size);
            const int id = __ldg(kv.block_table + slot * kv.table_stride + pg);
            if ((uint32_t)id < (uint32_t)kv.num_pages)
                at = id * kv.page_stride + (pos - (int64_t)pg * kv.page_size) * kv.token_stride;
            else
                bad = GDN_DEV_BAD_PAGE;
        }
    }
    if (bad && a.dev_status) atomicOr(a.dev_status, bad);
    return at;
}

template <bool E4M3>
__global__ void __launch_bounds__(kThreads) kv_append_kernel(const GdnAppendArgs a, const int tokens)
{
    __shared__ int64_t s_at[kMaxTokens];
    const gdn_paged_cache &kv = a.cache;
    const int tid = threadIdx.x, D8 = kv.head_dim / 8, per_token = 2 * kv.heads * D8;
    const int64_t n0 = (int64_t)blockIdx.x * tokens;
    const int here = (int)(a.N - n0 < tokens ? a.N - n0 : tokens);
    const int pieces = here * per_token;
    const int64_t cache_n = (int64_t)(kv.num_pages - 1) * kv.page_stride +
                            (int64_t)(kv.page_size - 1) * kv.token_stride +
                            (int64_t)(kv.heads - 1) * kv.head_stride + kv.head_dim;

    // piece i of the block: token, keys or values, head, 8 dimensions
    struct Piece { int t, v, h, d; };
    auto piece = [&](int i) {
        Piece p;
        p.t = i / per_token;
        int r = i - p.t * per_token;
        const int half = kv.heads * D8;
        p.v = r >= half;
        r -= p.v ? half : 0;
        p.h = r / D8;
        p.d = (r - p.h * D8) * 8;
        return p;
    };
    bool placed = false;
    for (int i0 = tid; i0 - tid < pieces; i0 += kThreads * kHold) {
        uint4 w[kHold];
#pragma unroll
        for (int k = 0; k < kHold; ++k) {
            const int i = i0 + k * kThreads;
            if (i >= pieces) continue;
            const Piece p = piece(i);
            const uint16_t *const x = static_cast<const uint16_t *>(p.v ? a.v : a.k);
            const int64_t ts = p.v ? a.v_token_stride : a.k_token_stride;
            const int64_t hs = p.v ? a.v_head_stride : a.k_head_stride;
            w[k] = __ldcs(reinterpret_cast<const uint4 *>(x + (n0 + p.t) * ts + p.h * hs + p.d));
        }
        if (!placed) {
            if (tid < here) s_at[tid] = place(a, n0 + tid);
            __syncthreads();
            placed = true;
        }
#pragma unroll
        for (int k = 0; k < kHold; ++k) {
            const int i = i0 + k * kThreads;
            if (i >= pieces) continue;
            const Piece p = piece(i);
            if (s_at[p.t] < 0) continue;
            const int64_t to = s_at[p.t] + p.h * kv.head_stride + p.d;
            if (!in_range(to, 8, cache_n, a.dev_status)) continue;
            if constexpr (E4M3) {
                const float *const sc = p.v ? kv.v_scale : kv.k_scale;
                const float s = sc ? __ldg(sc + p.h) : 1.f;
                *reinterpret_cast<uint2 *>(static_cast<unsigned char *>(p.v ? kv.v : kv.k) + to) =
                    quantise(w[k], a.bf16 != 0, s);
            } else {
                *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(p.v ? kv.v : kv.k) + to) = w[k];
            }
        }
    }
}

}  // namespace gdn_append

cudaError_t launch_kv_append(const GdnAppendArgs &a, cudaStream_t stream)
{
    using namespace gdn_append;
    // tokens a block: up to what its threads hold at once, fewer when that leaves SMs idle
    const int64_t per_token = 2 * (int64_t)a.cache.heads * (a.cache.head_dim / 8);
    int64_t tokens = kThreads * kHold / per_token;
    const int64_t spread = a.N / (4 * gdn_cache::sm_count() + 1);
    if (tokens > spread) tokens = spread;
    if (tokens > kMaxTokens) tokens = kMaxTokens;
    if (tokens < 1) tokens = 1;
    const int64_t blocks = (a.N + tokens - 1) / tokens;
    if (a.cache.dtype == GDN_E4M3)
        kv_append_kernel<true><<<(unsigned)blocks, kThreads, 0, stream>>>(a, (int)tokens);
    else
        kv_append_kernel<false><<<(unsigned)blocks, kThreads, 0, stream>>>(a, (int)tokens);
    return cudaGetLastError();
}
