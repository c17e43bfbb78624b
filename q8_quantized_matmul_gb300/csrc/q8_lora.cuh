// q8_lora.cuh -- device helpers shared by the adapter kernels.
#pragma once

#include "q8_attn.cuh"
#include "q8_kv.h"
#include "q8_layer.h"

namespace q8 {

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
__device__ __forceinline__ uint32_t cluster_addr(const void *p, uint32_t cta) {
    uint32_t a;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_addr(p)), "r"(cta));
    return a;
}
__device__ __forceinline__ float ld_cluster(uint32_t a) {
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ float4 ld_cluster4(uint32_t a) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(a) : "memory");
    return v;
}

__device__ __forceinline__ float value16(uint32_t bits, bool bf16) {
    return bf16 ? __uint_as_float(bits << 16) : half_bits_to_float((uint16_t)bits);
}
__device__ __forceinline__ void values16(float (&v)[8], const uint4 &r, bool bf16) {
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        v[2 * e] = value16(w[e] & 0xffffu, bf16);
        v[2 * e + 1] = value16(w[e] >> 16, bf16);
    }
}

// A rank as given; one outside [0, max_rank] is cut and raises Q8_ERANGE (by the thread that says so).
__device__ __forceinline__ int32_t given_rank(const LoraParams &p, int32_t id) { return p.ranks ? p.ranks[id] : (int32_t)p.max_rank; }
__device__ __forceinline__ uint32_t cut_rank(const LoraParams &p, int32_t r, bool tell) {
    if (r >= 0 && r <= (int32_t)p.max_rank) return (uint32_t)r;
    if (tell) raise_error(p.err, DEV_ERANGE);
    return r < 0 ? 0u : p.max_rank;
}

// 16-bit values 0 .. keep - 1 of a chunk of 8, the others zero.
__device__ __forceinline__ uint4 first_values(uint4 v, int keep) {
    uint32_t *w = reinterpret_cast<uint32_t *>(&v);
#pragma unroll
    for (int e = 0; e < 4; ++e) w[e] &= (2 * e < keep ? 0xffffu : 0u) | (2 * e + 1 < keep ? 0xffff0000u : 0u);
    return v;
}

}  // namespace q8
