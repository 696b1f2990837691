// kv_append.cu -- new keys and values to the pages of their positions.
//
// HBM-bound: every value is read once and written once, 4 bytes a value in 16 bits and 3 into 8.
// Where a token goes hangs on a chain of four dependent loads (offsets, slot, length, page), so a
// block has a warp for it that works a chunk of tokens ahead of the eight that copy; blocks stay
// and take every so-many-th chunk of equal size.  A copying thread keeps one column (keys or values, head, 8
// dimensions) and walks the tokens, so that nothing is divided in the loop; its loads are issued
// before it waits for the places.
// Measured on a B200: 16384 ragged tokens of 8 heads of 128, bf16: 27 us, 5.0 TB/s; into e4m3 23
// us, 4.4 TB/s; one token each of 243 rows 4 us.  With 3, 4, 5, 6 blocks an SM (8, 4, 4, 4 pieces
// held) the second takes 30, 24, 29, 40 us: more blocks spill registers, fewer leave loads out.
#include "cache.cuh"

namespace gdn_append {

using namespace gdn_cache;
using gdn::in_range;

constexpr int kThreads = 256;     // that copy
constexpr int kHold = 4;          // 16-byte pieces a thread holds at a time
constexpr int kMaxTokens = 32;    // of a chunk: a lane of the placing warp each
constexpr int kBlocksSM = 4;
constexpr int kOffsets = 1024;    // offsets that a block searches in shared memory

// x / scale to nearest for a scale > 0, for a quotient within +-1024 (past 448 every quotient is
// stored as 448, so there the product with the reciprocal will do, infinities included).  With r the
// reciprocal rounded to nearest, one step of the remainder from x r gives the rounded quotient
// (Markstein, "Computation of elementary functions on the IBM RISC System/6000 processor", 1990).
// The remainder is taken as q scale - x: where it is zero it is +0, its product with -r is -0, and a
// quotient of -0 stays one.
__device__ __forceinline__ float quotient(float x, float scale, float r)
{
    const float q = x * r;
    const float y = fmaf(fmaf(q, scale, -x), -r, q);
    return fabsf(q) < 1024.f ? y : q;
}

// eight 16-bit values -> eight e4m3 numbers of x / scale, the sign of a negative scale in `flip`
__device__ __forceinline__ uint2 quantise(const uint4 &w, bool bf16, float scale, float r, bool plain, uint32_t flip)
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
        const float2 y = plain ? make_float2(quotient(lo, scale, r), quotient(hi, scale, r))
                               : make_float2(__fdiv_rn(lo, scale), __fdiv_rn(hi, scale));
        // one rounding to float32, then one to e4m3 (to nearest even; past 448, infinities too,
        // to the largest number; a NaN stays one)
        out[k / 2] |= (uint32_t)__nv_cvt_float2_to_fp8x2(y, __NV_SATFINITE, __NV_E4M3) << (16 * (k & 1));
    }
    return make_uint2(out[0] ^ flip, out[1] ^ flip);
}

// The request with s <= n < e among the offsets, or -1.  Where they ascend, which is how they are
// searched, it is the last whose s is <= n (empty requests before it end at or before n).
__device__ int request_of(const GdnAppendArgs &a, int64_t n, const int32_t *offsets)
{
    int lo = 0, hi = a.B;        // offsets[lo] <= n < offsets[hi], were they sentinels
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (in_range(mid, 1, a.B + 1, a.dev_status) && offsets[mid] <= n)
            lo = mid;
        else
            hi = mid;
    }
    return in_range(lo, 2, a.B + 1, a.dev_status) && offsets[lo] <= n && n < offsets[lo + 1] ? lo : -1;
}

// The same, by a whole warp for a token (or none: n < 0) each, where offsets may fall back, as those
// do behind the last one in use of a list of fixed size: what is empty then may lead the search
// astray, which it shows by finding nothing.  Offsets in shared memory (`own`) are raised to the
// largest up to each, which leaves every other request what it is; others are gone through.
__device__ int warp_request_of(const GdnAppendArgs &a, int64_t n, const int32_t *offsets, int32_t *own, int &falls)
{
    const int lane = threadIdx.x & 31;
    int b = n >= 0 ? request_of(a, n, offsets) : -1;
    if (!__any_sync(0xffffffffu, n >= 0 && b < 0)) return b;
    if (falls < 0) {             // not known yet
        bool down = false;
        for (int i = lane; i < a.B; i += 32) down = down || offsets[i] > offsets[i + 1];
        falls = __any_sync(0xffffffffu, down);
    }
    if (!falls) return b;        // ahead of the first request or behind the last one
    if (own) {
        int top = own[0];
        for (int i0 = 0; i0 <= a.B; i0 += 32) {
            const int i = i0 + lane;
            int x = i <= a.B ? max(own[i], top) : top;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) x = max(x, __shfl_up_sync(0xffffffffu, x, d));
            if (i <= a.B) own[i] = x;
            top = __shfl_sync(0xffffffffu, x, 31);
        }
        __syncwarp();
        falls = 0;
        return n >= 0 && b < 0 ? request_of(a, n, own) : b;
    }
    for (int k = 0; n >= 0 && b < 0 && k < a.B; ++k)
        if (offsets[k] <= n && n < offsets[k + 1]) b = k;
    return b;
}

// where token n of request b goes: element offset of its head 0 in the cache, or -1
__device__ int64_t place(const GdnAppendArgs &a, int64_t n, int b, const int32_t *offsets)
{
    const gdn_paged_cache &kv = a.cache;
    int32_t *const status = a.dev_status;
    const int64_t end = offsets ? min((int64_t)offsets[b + 1], a.N) : (int64_t)(b + 1) * (a.N / a.B);
    if (!in_range(b, 1, a.B, status)) return -1;
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
            if (!in_range(pg, 1, kv.width, status)) return -1;
            const int id = __ldg(kv.block_table + slot * kv.table_stride + pg);
            if ((uint32_t)id < (uint32_t)kv.num_pages)
                at = id * kv.page_stride + (pos - (int64_t)pg * kv.page_size) * kv.token_stride;
            else
                bad = GDN_DEV_BAD_PAGE;
        }
    }
    if (bad && status) atomicOr(status, bad);
    return at;
}

template <bool E4M3>
__global__ void __launch_bounds__(kThreads + 32, kBlocksSM)
kv_append_kernel(const __grid_constant__ GdnAppendArgs a, const int tokens, const int64_t chunks)
{
    __shared__ int64_t s_at[2][kMaxTokens];
    __shared__ int32_t s_offsets[kOffsets];
    const gdn_paged_cache &kv = a.cache;
    const int tid = threadIdx.x, D8 = kv.head_dim / 8, per_token = 2 * kv.heads * D8;
    auto size_of = [&](int64_t chunk) { return (int)min(a.N - chunk * tokens, (int64_t)tokens); };

    if (tid >= kThreads) {
        const int lane = tid - kThreads;
        const bool staged = a.row_offsets && a.B < kOffsets;
        if (staged)
            for (int i = lane; i <= a.B; i += 32) s_offsets[i] = __ldg(a.row_offsets + i);
        __syncwarp();
        const int32_t *const offsets = staged ? s_offsets : a.row_offsets;
        const int each = (int)(a.N / a.B);      // tokens a request, without offsets
        int buf = 0, falls = -1;
        for (int64_t chunk = blockIdx.x; chunk < chunks; chunk += gridDim.x, buf ^= 1) {
            // (the chunk before the last one has been copied: the others are past its meeting)
            const int64_t n = lane < size_of(chunk) ? chunk * tokens + lane : -1;
            const int b = !offsets ? (int)n / each : warp_request_of(a, n, offsets, staged ? s_offsets : nullptr, falls);
            if (n >= 0) s_at[buf][lane] = b < 0 ? -1 : place(a, n, b, offsets);
            __syncthreads();
        }
        return;
    }

    const int64_t cache_n = (int64_t)(kv.num_pages - 1) * kv.page_stride +
                            (int64_t)(kv.page_size - 1) * kv.token_stride +
                            (int64_t)(kv.heads - 1) * kv.head_stride + kv.head_dim;
    // tokens side by side in the block, and this thread's column
    const int side = per_token < kThreads ? kThreads / per_token : 1;
    const int t0 = per_token < kThreads ? tid / per_token : 0;
    const int col0 = per_token < kThreads ? tid - t0 * per_token : tid;
    int buf = 0;
    for (int64_t chunk = blockIdx.x; chunk < chunks; chunk += gridDim.x, buf ^= 1) {
        const int64_t n0 = chunk * tokens;
        const int here = size_of(chunk);
#pragma unroll 1
        for (int c0 = 0; c0 < per_token; c0 += kThreads) {
            const int col = c0 + col0;
            const bool mine = col < per_token && t0 < side;
            const int v = col >= kv.heads * D8, r = col - (v ? kv.heads * D8 : 0), h = r / D8, d = (r - h * D8) * 8;
            const int64_t ts = v ? a.v_token_stride : a.k_token_stride;
            const int64_t hs = v ? a.v_head_stride : a.k_head_stride;
            const uint16_t *const x0 = static_cast<const uint16_t *>(v ? a.v : a.k);
            const uint16_t *x = x0 + (n0 + t0) * ts + h * hs + d;
            const int64_t x_n = (a.N - 1) * ts + (kv.heads - 1) * hs + kv.head_dim;
            const int64_t off = h * kv.head_stride + d;
            unsigned char *const y = static_cast<unsigned char *>(v ? kv.v : kv.k) + off * (E4M3 ? 1 : 2);
            float scale = 1.f, inv = 1.f;
            uint32_t flip = 0u;
            if (E4M3 && mine) {
                const float *const sc = v ? kv.v_scale : kv.k_scale;
                if (sc && in_range(h, 1, kv.heads, a.dev_status)) scale = __ldg(sc + h);
                if (signbit(scale)) flip = 0x80808080u;
                scale = fabsf(scale);
                inv = __frcp_rn(scale);
            }
            // (a scale whose reciprocal is no normal number is divided by)
            const bool plain = scale > 0x1p-120f && scale < 0x1p120f;
#pragma unroll 1
            for (int i = t0; i - t0 < here; i += side * kHold) {
                uint4 w[kHold];
#pragma unroll
                for (int k = 0; k < kHold; ++k) {
                    if (mine && i + k * side < here)
                        w[k] = in_range(x - x0, 8, x_n, a.dev_status) ? __ldcs(reinterpret_cast<const uint4 *>(x))
                                                                      : make_uint4(0u, 0u, 0u, 0u);
                    x += side * ts;
                }
                if (c0 == 0 && i == t0) __syncthreads();        // the places are known
#pragma unroll
                for (int k = 0; k < kHold; ++k) {
                    const int t = i + k * side;
                    const int64_t at = mine && t < here ? s_at[buf][t] : -1;
                    if (at < 0 || !in_range(at + off, 8, cache_n, a.dev_status)) continue;
                    if constexpr (E4M3)
                        *reinterpret_cast<uint2 *>(y + at) = quantise(w[k], a.bf16 != 0, scale, inv, plain, flip);
                    else
                        *reinterpret_cast<uint4 *>(y + 2 * at) = w[k];
                }
            }
        }
    }
}

}  // namespace gdn_append

cudaError_t launch_kv_append(const GdnAppendArgs &a, cudaStream_t stream)
{
    using namespace gdn_append;
    // equal chunks of at most kMaxTokens, in as few rounds of the resident blocks as that takes
    const int64_t resident = (int64_t)kBlocksSM * gdn_cache::sm_count();
    if (resident == 0) {        // no device, or one that does not answer
        const cudaError_t e = cudaGetLastError();
        return e == cudaSuccess ? cudaErrorNoDevice : e;
    }
    const int64_t rounds = (a.N + resident * kMaxTokens - 1) / (resident * kMaxTokens);
    const int64_t tokens = (a.N + resident * rounds - 1) / (resident * rounds);
    const int64_t chunks = (a.N + tokens - 1) / tokens;
    const unsigned blocks = (unsigned)(chunks < resident ? chunks : resident);
    if (a.cache.dtype == GDN_E4M3)
        kv_append_kernel<true><<<blocks, kThreads + 32, 0, stream>>>(a, (int)tokens, chunks);
    else
        kv_append_kernel<false><<<blocks, kThreads + 32, 0, stream>>>(a, (int)tokens, chunks);
    return cudaGetLastError();
}
