// cache.cuh -- what the paged key-value cache's kernels share: launcher arguments and thin
// inline-PTX wrappers (rank-4 tensor loads, ldmatrix, 16-bit warp mma, dependent launches).
#pragma once

#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "common.cuh"
#include "sm100.cuh"

namespace gdn_cache {

// a box of a rank-4 tensor -> shared memory (128-byte aligned), completing on an mbarrier
__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap *map, uint32_t bar,
                                            int x, int y, int z, int w)
{
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y), "r"(z), "r"(w)
        : "memory");
}

__device__ __forceinline__ void ldmatrix_x4(uint32_t (&r)[4], uint32_t addr)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldmatrix_x4_trans(uint32_t (&r)[4], uint32_t addr)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
// two 16x16 blocks of bytes, transposed: thread (g, t) of a quad row gets rows 4t..4t+3 of
// columns g (r[0]) and 8 + g (r[1]) of the block whose rows lanes 0-15 point at; r[2], r[3] of
// the one of lanes 16-31
__device__ __forceinline__ void ldmatrix_b8_x2_trans(uint32_t (&r)[4], uint32_t addr)
{
    asm volatile("ldmatrix.sync.aligned.m16n16.x2.trans.shared.b8 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void sts128_zero(uint32_t addr)
{
    asm volatile("st.shared.v4.u32 [%0], {%1,%1,%1,%1};" ::"r"(addr), "r"(0u) : "memory");
}
__device__ __forceinline__ uint4 lds128(uint32_t addr)
{
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(addr)
                 : "memory");
    return v;
}

// C(16x8) += A(16x16, row) * B(16x8, col), 16-bit inputs of one type, fp32 accumulate
template <bool BF16>
__device__ __forceinline__ void mma_16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                          uint32_t a3, uint32_t b0, uint32_t b1)
{
    if constexpr (BF16)
        asm(
            "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 "
            "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm(
            "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
            "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// bring the line that holds p into L1 (a load that nobody waits for)
__device__ __forceinline__ void touch_l1(const void *p)
{
    asm volatile("{\n\t.reg .b32 x;\n\tld.global.nc.b32 x, [%0];\n\t}" ::"l"(p));
}

// four e4m3 numbers -> halves (every e4m3 number is one)
__device__ __forceinline__ void e4m3x4_to_f16x2(uint32_t w, uint32_t &lo, uint32_t &hi)
{
    asm("{\n\t.reg .b16 l, h;\n\t"
        "mov.b32 {l, h}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, l;\n\t"
        "cvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi)
{
    const __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&v);
}

// the warpgroup's registers a thread from here on (of those that the block was launched with)
template <int N>
__device__ __forceinline__ void registers_down() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N>
__device__ __forceinline__ void registers_up() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }

// dependent launches: the next kernel of the stream may begin / wait for the one before
__device__ __forceinline__ void launch_dependents()
{
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
__device__ __forceinline__ void wait_primary() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// Launch of a kernel that calls wait_primary() before it touches anything that the kernel
// before it in the stream wrote: it may be brought up while that one drains.
template <typename... KA, typename... A>
cudaError_t launch_dependent(void (*kernel)(KA...), dim3 grid, dim3 block, size_t smem,
                             cudaStream_t stream, A &&...args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, KA(args)...);
}

// SMs of the current device (0 without one); looked up once per device
int sm_count();

}  // namespace gdn_cache

struct GdnAttnArgs {
    const void *q;
    int64_t q_token_stride, q_head_stride;
    gdn_paged_cache cache;
    const int32_t *slots;
    int32_t B, T, Hq;
    int32_t q_bf16;         // q and out are bf16 (else fp16)
    float scale;
    int32_t window;
    void *out;
    float *lse;
    int32_t zero_padding;
    void *workspace;
    uint64_t workspace_bytes;
    int32_t *dev_status;
};

struct GdnAppendArgs {
    const void *k, *v;
    int64_t k_token_stride, k_head_stride, v_token_stride, v_head_stride;
    gdn_paged_cache cache;
    const int32_t *slots, *row_offsets;
    int32_t B;
    int64_t N;
    int32_t bf16;           // k and v are bf16 (else fp16)
    int32_t *dev_status;
};

cudaError_t launch_paged_attn(const GdnAttnArgs &a, cudaStream_t stream);
uint64_t paged_attn_workspace_bytes(int32_t B, int32_t T, int32_t Hq, int32_t heads, int32_t D,
                                    int32_t cache_dtype);
cudaError_t launch_kv_append(const GdnAppendArgs &a, cudaStream_t stream);
cudaError_t launch_page_resize(const gdn_page_table &t, const int32_t *row_list,
                               const int32_t *new_lens, int32_t n, const gdn_pool *pools,
                               int32_t n_pools, void *workspace, int32_t *dev_status,
                               cudaStream_t stream);
cudaError_t launch_page_fork(const gdn_page_table &t, const int32_t *parents,
                             const int32_t *children, int32_t n, const gdn_pool *pools,
                             int32_t n_pools, int32_t *dev_status, cudaStream_t stream);
cudaError_t launch_page_compact(const gdn_page_table &t, int32_t *page_map, const gdn_pool *pools,
                                int32_t n_pools, void *workspace, int32_t *dev_status,
                                cudaStream_t stream);
uint64_t page_workspace_bytes(int32_t num_pages, int32_t n);
