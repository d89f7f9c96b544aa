// few_rows.cuh -- what the kernels share that take up to 32 query rows of a KV head through
// mma.sync: fragments, waits, and the exchange between the CTAs of a cluster (sm_103a).
#pragma once

#include "common.cuh"

namespace magicdec {

constexpr float kFewLazy = 24.0f;    // log2 growth of a row's maximum that is put up with

__device__ __forceinline__ uint32_t few_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ uint32_t few_ctas() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void few_cluster_sync() {
    __syncwarp();
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// The address of `p` in the shared memory of CTA `rank` of the cluster, and loads from there.
__device__ __forceinline__ uint32_t few_at(const void *p, uint32_t rank) {
    uint32_t a;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
    return a;
}
__device__ __forceinline__ float2 few_ld2(uint32_t a) {
    float2 v;
    asm volatile("ld.shared::cluster.v2.f32 {%0,%1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ float4 few_ld4(uint32_t a) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(a)
                 : "memory");
    return v;
}
// A warp's wait, with one outcome for all lanes; once one has given up, the later ones return at once.
__device__ __forceinline__ bool few_wait(uint64_t *bar, uint32_t parity, int *err, bool ok, int lane) {
    if (__all_sync(0xffffffffu, ok && mbar_try_sleep(bar, parity))) return true;
    int got = ok ? 1 : 0;
    if (ok && lane == 0) got = mbar_poll_on(bar, parity, err) ? 1 : 0;
    return __shfl_sync(0xffffffffu, got, 0) != 0;
}

// D(16x8) += A(16x16) B(16x8); with 8 real rows (HR = 1) the lower half of A and of D is not there.
template <int HR>
__device__ __forceinline__ void few_mma(float (&c)[2 * HR], const uint32_t (&a)[2 * HR], uint32_t b0, uint32_t b1) {
    if constexpr (HR == 2) {
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
            "{%0,%1,%2,%3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    } else {
        asm volatile(
            "{\n\t.reg .f32 x, y;\n\t"
            "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,x,y}, {%2,%3,%4,%5}, {%6,%7}, "
            "{%0,%1,%8,%8};\n\t}"
            : "+f"(c[0]), "+f"(c[1])
            : "r"(a[0]), "r"(0u), "r"(a[1]), "r"(0u), "r"(b0), "r"(b1), "f"(0.f));
    }
}

// Bits of the bf16 of a word that are not finite: the carry of an exponent of ones tells.
__device__ __forceinline__ uint32_t few_odd_bits(uint32_t x) {
    return ((((x & 0x7f807f80u) + 0x00800080u) & 0x80008000u) >> 15) * 0xffffu;
}

// Whether any value of rows [row, row + rows) of a tile of V is not finite: 64-channel halves `half`
// bytes apart, rows of 128 bytes, swizzled.  By a warp.
template <int HV>
__device__ __forceinline__ bool few_not_finite(const uint8_t *v, int half, int row, int rows, int lane) {
    uint32_t any = 0;
    for (int i = lane; i < rows * HV * 8; i += 32) {
        const int r = row + i / (HV * 8), c = i % (HV * 8);
        const uint4 x = *reinterpret_cast<const uint4 *>(v + (c >> 3) * half + swz128(r, c & 7));
        any |= few_odd_bits(x.x) | few_odd_bits(x.y) | few_odd_bits(x.z) | few_odd_bits(x.w);
    }
    return __any_sync(0xffffffffu, any != 0);
}

}  // namespace magicdec
