// wq_prompt.cuh -- device helpers of the prompt-side kernels.
#pragma once

#include "wq_common.cuh"
#include "wq_sm100.cuh"

namespace wq {

// A 16-byte load in a kernel that starts before the previous one has ended: what that one wrote is not read-only for
// the kernel's whole life, so this is an ordinary load and not one through the read-only path.
__device__ __forceinline__ uint4 ld_written_v4(const void *p)
{
    uint4 r;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
                 : "l"(p)
                 : "memory");
    return r;
}

// Two binary32 in a bf16x2 word (lo = a, hi = b), each rounded to nearest even: one instruction, where two single
// conversions would go through the special-function units.
__device__ __forceinline__ uint32_t pack2_bf16(float a, float b)
{
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
    return r;
}

// mbar_wait by a whole warp, with one answer for all lanes: what follows a wait (tensor-memory loads, votes, barriers) needs
// every lane, and lanes that gave up one by one would leave the others waiting for them without a bound.
__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t parity, int *status, volatile int *abort)
{
    return __all_sync(0xffffffffu, mbar_wait(bar, parity, status, abort));
}

// named_bar_sync whose threads learn whether `ok` held for all of them.
__device__ __forceinline__ bool named_bar_and(int id, int threads, bool ok)
{
    uint32_t all;
    asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.u32 q, %3, 0;\n\tbar.red.and.pred p, %1, %2, q;\n\tselp.u32 %0, 1, 0, p;\n\t}"
                 : "=r"(all)
                 : "r"(id), "r"(threads), "r"((uint32_t)ok)
                 : "memory");
    return all != 0;
}

// One lane of the (whole) warp.
__device__ __forceinline__ bool elect_one()
{
    uint32_t p;
    asm volatile("{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\tselp.u32 %0, 1, 0, q;\n\t}" : "=r"(p));
    return p != 0;
}

// The 3-D form of tma_load_2d (x innermost).
__device__ __forceinline__ void tma_load_3d(void *dst, const CUtensorMap *map, uint64_t *bar, int x, int y, int z)
{
    asm volatile("cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], [%2];"
                 ::"r"(smem_u32(dst)), "l"(map), "r"(smem_u32(bar)), "r"(x), "r"(y), "r"(z)
                 : "memory");
}

// D[tmem] (+)= A[smem] * B[smem]^T, kind::f16 (bf16 inputs, f32 accumulate).
__device__ __forceinline__ void tc_mma_ss(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                          uint32_t accumulate)
{
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
                 "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
                 "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
                 : "memory");
}

// encode_tmap_2d for rows of `mid` adjacent vectors of `inner` values (tokens of heads): mid_stride_bytes between
// vectors, row_stride_bytes between rows (wq_gemv_tma.cu).
bool encode_tmap_3d(CUtensorMap *map, CUtensorMapDataType dtype, const void *base, uint64_t inner, uint64_t mid,
                    uint64_t outer, uint64_t mid_stride_bytes, uint64_t row_stride_bytes, uint32_t box_inner,
                    uint32_t box_mid, uint32_t box_outer, CUtensorMapSwizzle swizzle);

}  // namespace wq
