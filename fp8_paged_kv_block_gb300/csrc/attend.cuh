// attend.cuh -- device helpers shared by the attention kernels that keep P in FP16
// (tree.cu, window.cu): waits, FP16 tensor operations, runs of equal weight.
#pragma once

#include "common.cuh"

#include <cuda_fp16.h>
#include <cuda_fp8.h>

namespace pa {

// ---- runs ----
// Run c of `ctas` over `total`: the first total % ctas runs are one longer.
__device__ __forceinline__ uint32_t run_begin(uint32_t total, uint32_t c, uint32_t ctas)
{
    return c * (total / ctas) + min(c, total % ctas);
}
// the CTA whose run holds position pos
__device__ __forceinline__ int cta_of(uint32_t total, uint32_t pos, uint32_t ctas)
{
    const uint32_t q = total / ctas, r = total % ctas, longer = r * (q + 1);
    return static_cast<int>(pos < longer ? pos / (q + 1) : r + (pos - longer) / q);
}

// ---- waits -----------------------------------------------------------------------
// mbar_wait with a shorter body: the kernel's parts run at once out of one
// instruction cache. Each lane polls and leaves for itself: a __syncwarp (or a
// vote) stands between a wait and the next tensor memory operation or named
// barrier, which are for a converged warp. (One in here, for every wait, cost 2%
// on 16 x 8 drafted tokens, 1% on long contexts.)
__device__ __forceinline__ bool wait_for(uint64_t* bar, uint32_t parity, int* err, int code, volatile int* abort)
{
    if (mbar_try_wait(bar, parity)) return true;
    const uint32_t t0 = static_cast<uint32_t>(globaltimer_ns());
    while (!mbar_try_wait(bar, parity)) {
        if (*abort) return false;
        if (static_cast<uint32_t>(globaltimer_ns()) - t0 > static_cast<uint32_t>(kWaitLimitNs)) {
            *abort = 1;
            atomicOr(err, code);
            return false;
        }
    }
    return true;
}

// ---- small device helpers ------------------------------------------------------------
__host__ __device__ constexpr uint32_t idesc_f16(int M, int N, int a_mn, int b_mn)
{
    return (1u << 4) | (static_cast<uint32_t>(a_mn) << 15) | (static_cast<uint32_t>(b_mn) << 16) |
           (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24);
}

// D(tmem) (+)= A(tmem, FP16 pairs) * B(smem, FP16): K = 16 per MMA.
__device__ __forceinline__ void umma_f16_ta(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                            uint32_t accumulate)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t* v)
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(
            taddr),
        "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
        "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
        : "memory");
}

__device__ __forceinline__ uint32_t half2_bits(float lo, float hi)
{
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}

__device__ __forceinline__ uint32_t codes_to_half2(uint32_t two)
{
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(two), __NV_E4M3);
    return *reinterpret_cast<const uint32_t*>(&h);
}

__device__ __forceinline__ void named_bar_arrive(int id, int nthreads)
{
    asm volatile("bar.arrive %0, %1;" ::"r"(id), "r"(nthreads) : "memory");
}

__device__ __forceinline__ float max3(float a, float b, float c)
{
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

__device__ __forceinline__ uint64_t l2_keep_policy()
{
    uint64_t p;
    asm volatile("createpolicy.fractional.L2::evict_unchanged.b64 %0, 1.0;" : "=l"(p));
    return p;
}

// True in one thread of the (converged) warp.
__device__ __forceinline__ bool elect_one()
{
    uint32_t is;
    asm volatile(
        "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(is));
    return is != 0;
}

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

}  // namespace pa
