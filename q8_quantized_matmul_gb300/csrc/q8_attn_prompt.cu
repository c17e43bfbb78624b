// q8_attn_prompt.cu -- attention over whole packed prompts, causal, grouped heads: the
// mma.sync kernel, for the calls that q8_attn_prompt_tc.cu does not take (attn_prompt_on_tc).
//
// k_attn_prompt_mma: 64 query rows of one head per CTA (16 a warp), keys in tiles of 64 (32 for heads
// of more than 128 values) through a double buffer of asynchronous copies; running maximum, sum and
// unnormalised output in registers, fp32.  Heads of more than 128 values give each CTA a slice of 128
// of V's dimensions; the slices compute the scores again.
//
// What a query may not see never reaches its result.  Keys: the score is replaced.  Values: rows of
// other sequences are staged as zeros, and in tiles where some rows see a key and others do not, a
// value that is not finite is staged as zero and added at the end, to the rows that see it (0 times
// infinity would otherwise reach the rows that do not).
#include "q8_attn.cuh"
#include "q8_attn_prompt.cuh"
#include "q8_kv.h"

namespace q8 {
namespace {

template <int D> struct Pm {
    static constexpr int BM = 64, BN = D > 128 ? 32 : 64, DV = D > 128 ? 128 : D;
    static constexpr int QB_ = D > 128 ? BM * D * 2 : 0;      // q in shared memory for the larger heads
    static constexpr int KB = BN * D * 2, VB = BN * DV * 2;
    static constexpr int ST = KB + VB;
    static constexpr int OB = BM * DV * 4;
    static constexpr int SMEM = QB_ + (2 * ST > OB ? 2 * ST : OB) + 128;
};

template <int D, bool BF16> __global__ void __launch_bounds__(128) k_attn_prompt_mma(const AttnPromptParams p) {
    using C = Pm<D>;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ int sh[10];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, c = lane & 3;
    grid_dep_wait();
    PromptTile w;
    if (!prompt_tile<128>(p, C::BM, blockIdx.x, blockIdx.x + blockIdx.y + blockIdx.z == 0, w, sh)) return;
    const uint32_t head = blockIdx.y, kvh = head / (p.n_heads / p.n_kv);
    const int dv0 = blockIdx.z * C::DV;
    const uint16_t *qp = static_cast<const uint16_t *>(p.q) + (uint64_t)(w.q0 + w.row0) * p.q_stride + (uint64_t)head * D;
    const uint16_t *kp = static_cast<const uint16_t *>(p.k) + (uint64_t)w.k0 * p.k_stride + (uint64_t)kvh * D;
    const uint16_t *vp = static_cast<const uint16_t *>(p.v) + (uint64_t)w.k0 * p.v_stride + (uint64_t)kvh * D + dv0;
    uint8_t *qs = smem, *ring = smem + C::QB_;
    const uint32_t qs_s = smem_addr(qs), ring_s = smem_addr(ring);
    if (tid == 0) sh[9] = 0;   // a masked tile held a value that is not finite

    const int n0 = w.first(0, p.window) / C::BN, n1 = w.rows ? (w.last(w.rows - 1) + C::BN) / C::BN : 0;   // key tiles [n0, n1)
    auto stage = [&](int n) {
        if (n < n1) {
            const uint32_t st = ring_s + (n & 1) * C::ST;
#pragma unroll 4
            for (int i = tid; i < C::BN * (D / 8); i += 128) {
                const int r = i / (D / 8), ch = i % (D / 8);
                const bool ok = n * C::BN + r < w.lk;
                cp_async16(st + r * (D * 2) + (ch ^ (r & 7)) * 16, ok ? kp + (uint64_t)(n * C::BN + r) * p.k_stride + ch * 8 : kp, ok);
            }
#pragma unroll 4
            for (int i = tid; i < C::BN * (C::DV / 8); i += 128) {
                const int r = i / (C::DV / 8), ch = i % (C::DV / 8);
                const bool ok = n * C::BN + r < w.lk;
                cp_async16(st + C::KB + r * (C::DV * 2) + (ch ^ (r & 7)) * 16,
                           ok ? vp + (uint64_t)(n * C::BN + r) * p.v_stride + ch * 8 : vp, ok);
            }
        }
        cp_async_commit();
    };
    // a row of this thread: g and g + 8 of the warp's sixteen
    uint32_t qr[D <= 128 ? D / 16 : 1][4];
    if constexpr (D <= 128) {
        const int ra = warp * 16 + g, rb = ra + 8;
        const uint16_t *qa = qp + (uint64_t)ra * p.q_stride, *qb = qp + (uint64_t)rb * p.q_stride;
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
            const int k = ks * 16 + 2 * c;
            qr[ks][0] = ra < w.rows ? *reinterpret_cast<const uint32_t *>(qa + k) : 0u;
            qr[ks][1] = rb < w.rows ? *reinterpret_cast<const uint32_t *>(qb + k) : 0u;
            qr[ks][2] = ra < w.rows ? *reinterpret_cast<const uint32_t *>(qa + k + 8) : 0u;
            qr[ks][3] = rb < w.rows ? *reinterpret_cast<const uint32_t *>(qb + k + 8) : 0u;
        }
    } else {
#pragma unroll 4
        for (int i = tid; i < C::BM * (D / 8); i += 128) {
            const int r = i / (D / 8), ch = i % (D / 8);
            const bool ok = r < w.rows;
            cp_async16(qs_s + r * (D * 2) + (ch ^ (r & 7)) * 16, ok ? qp + (uint64_t)r * p.q_stride + ch * 8 : qp, ok);
        }
    }
    float o[C::DV / 8][4];
#pragma unroll
    for (int i = 0; i < C::DV / 8; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.0f;
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f};
    const int row_a = warp * 16 + g;
    stage(n0);
    for (int n = n0; n < n1; ++n) {
        stage(n + 1);
        cp_async_wait<1>();
        __syncthreads();
        const uint32_t st = ring_s + (n & 1) * C::ST;
        const bool masked = w.masked(n * C::BN, C::BN, p.window);
        if (masked) {
            // values that are not finite leave the tile; see the end of the kernel
            uint8_t *vt = ring + (n & 1) * C::ST + C::KB;
            for (int i = tid; i < C::VB / 16; i += 128) {
                uint4 x = reinterpret_cast<uint4 *>(vt)[i];
                if (prompt_scrub<BF16>(x)) {
                    reinterpret_cast<uint4 *>(vt)[i] = x;
                    sh[9] = 1;
                }
            }
            __syncthreads();
        }
        float z[C::BN / 8][4];
#pragma unroll
        for (int i = 0; i < C::BN / 8; ++i) z[i][0] = z[i][1] = z[i][2] = z[i][3] = 0.0f;
        {
            const int r = (lane >> 4) * 8 + (lane & 7), hc = (lane >> 3) & 1;
            const int qrow = warp * 16 + (lane & 15), qc = lane >> 4;
#pragma unroll(D <= 128 ? D / 16 : 4)
            for (int ks = 0; ks < D / 16; ++ks) {
                uint32_t a[4];
                if constexpr (D <= 128) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) a[i] = qr[ks][i];
                } else {
                    ldsm4(a, qs_s + qrow * (D * 2) + ((ks * 2 + qc) ^ (qrow & 7)) * 16);
                }
#pragma unroll
                for (int t = 0; t < C::BN / 16; ++t) {
                    uint32_t b[4];
                    const int rr = t * 16 + r;
                    ldsm4(b, st + rr * (D * 2) + ((ks * 2 + hc) ^ (rr & 7)) * 16);
                    mma16<BF16>(z[2 * t], a, b[0], b[1]);
                    mma16<BF16>(z[2 * t + 1], a, b[2], b[3]);
                }
            }
        }
        float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
        for (int i = 0; i < C::BN / 8; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                float v = z[i][e] * p.scale_log2;
                if (masked && !w.sees(row_a + (e >> 1) * 8, n * C::BN + 8 * i + 2 * c + (e & 1), p.window)) v = -INFINITY;
                z[i][e] = v;
                mx[e >> 1] = fmaxf(mx[e >> 1], v);
            }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            mx[h] = fmaxf(mx[h], __shfl_xor_sync(0xffffffffu, mx[h], 1));
            mx[h] = fmaxf(mx[h], __shfl_xor_sync(0xffffffffu, mx[h], 2));
            const float mn = fmaxf(m[h], mx[h]), f = m[h] == -INFINITY ? 0.0f : ex2(m[h] - mn);
            m[h] = mn;
            l[h] *= f;
#pragma unroll
            for (int i = 0; i < C::DV / 8; ++i) {
                o[i][2 * h] *= f;
                o[i][2 * h + 1] *= f;
            }
            const float s = mn == -INFINITY ? 0.0f : mn;
#pragma unroll
            for (int i = 0; i < C::BN / 8; ++i) {
                z[i][2 * h] = ex2(z[i][2 * h] - s);
                z[i][2 * h + 1] = ex2(z[i][2 * h + 1] - s);
                l[h] += z[i][2 * h] + z[i][2 * h + 1];
            }
        }
        {
            const int r = ((lane >> 3) & 1) * 8 + (lane & 7), hc = lane >> 4;
#pragma unroll
            for (int t = 0; t < C::BN / 16; ++t) {
                const uint32_t a[4] = {pack16<BF16>(z[2 * t][0], z[2 * t][1]), pack16<BF16>(z[2 * t][2], z[2 * t][3]),
                                       pack16<BF16>(z[2 * t + 1][0], z[2 * t + 1][1]),
                                       pack16<BF16>(z[2 * t + 1][2], z[2 * t + 1][3])};
#pragma unroll
                for (int i = 0; i < C::DV / 16; ++i) {
                    uint32_t b[4];
                    const int rr = t * 16 + r;
                    ldsm4t(b, st + C::KB + rr * (C::DV * 2) + ((i * 2 + hc) ^ (rr & 7)) * 16);
                    mma16<BF16>(o[2 * i], a, b[0], b[1]);
                    mma16<BF16>(o[2 * i + 1], a, b[2], b[3]);
                }
            }
        }
        __syncthreads();   // the stage is free
    }
    cp_async_wait<0>();
    __syncthreads();
    float *mo = reinterpret_cast<float *>(ring) + warp * 16 * C::DV;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
        l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
        float lse;
        const float f = softmax_finish(m[h], l[h], p.sinks != nullptr, p.sinks ? p.sinks[head] * 1.4426950408889634f : 0.0f, lse);
        const int row = row_a + 8 * h;
#pragma unroll
        for (int i = 0; i < C::DV / 8; ++i) {
            mo[(g + 8 * h) * C::DV + 8 * i + 2 * c] = f == 0.0f ? 0.0f : o[i][2 * h] * f;
            mo[(g + 8 * h) * C::DV + 8 * i + 2 * c + 1] = f == 0.0f ? 0.0f : o[i][2 * h + 1] * f;
        }
        if (p.lse && c == 0 && dv0 == 0 && row < w.rows)
            p.lse[(uint64_t)(w.q0 + w.row0 + row) * p.n_heads + head] = lse;
    }
    __syncwarp();
    const bool dirty = sh[9] != 0;
    for (int i = lane; i < 16 * (C::DV / 8); i += 32) {
        const int r = i / (C::DV / 8), d0 = i % (C::DV / 8) * 8, row = warp * 16 + r;
        const bool act = row < w.rows;
        float y[8];
        load8s(y, mo + r * C::DV + d0);
        if (dirty && act) prompt_restore<BF16>(p, w, vp + d0, row, C::BN, y);
        store_out8(p.out, p.out_type, ((uint64_t)(w.q0 + w.row0 + (act ? row : 0)) * p.n_heads + head) * D + dv0 + d0, y, act);
    }
}

template <int D, bool BF16> cudaError_t launch_one(const AttnPromptParams &p, cudaStream_t st) {
    static bool attr_done = false;
    if (!attr_done) {
        const cudaError_t e = cudaFuncSetAttribute(k_attn_prompt_mma<D, BF16>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   Pm<D>::SMEM);
        if (e != cudaSuccess) return e;
        attr_done = true;
    }
    const dim3 grid(p.n_q / Pm<D>::BM + p.n_seq, p.n_heads, D / Pm<D>::DV);
    return launch_dependent(k_attn_prompt_mma<D, BF16>, p, grid, 128, Pm<D>::SMEM, st);
}

template <bool BF16> cudaError_t launch_type(const AttnPromptParams &p, cudaStream_t st) {
    switch (p.dim) {
        case 64: return launch_one<64, BF16>(p, st);
        case 128: return launch_one<128, BF16>(p, st);
        case 256: return launch_one<256, BF16>(p, st);
        case 512: return launch_one<512, BF16>(p, st);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace

cudaError_t launch_attn_prompt_mma(const AttnPromptParams &p, cudaStream_t st) {
    return p.type == Q8_TYPE_BF16 ? launch_type<true>(p, st) : launch_type<false>(p, st);
}

}  // namespace q8
