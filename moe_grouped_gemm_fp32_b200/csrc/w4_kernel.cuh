// w4_kernel.cuh -- products of a few BF16 rows with 4-bit weights:
//
//   D[m,n] = sum_j s[j,n] * sum_{k in group j} (q[n,k] - z[j,n]) * x[m,k]
//
// q: codes 0..15, two per byte along K; s (BF16) and z (8 where absent): one
// for each row n and group j of kGs consecutive k, stored [K/kGs][N].  Dense,
// or with expert g's weights for the rows offsets[g] .. offsets[g+1).
//
// The weights' bytes are the floor (half a byte and 2/kGs of scale per weight,
// read once), so the kernel is laid out around streaming them:
//   * a CTA owns 128 weight rows and a range of K, each of its 8 warps 16 rows;
//     stages of 256 k (128 bytes of every row, with their x, scales and zero
//     points) arrive by 16-byte asynchronous copies, kStages in flight;
//   * a cluster of `split` CTAs shares the 128 rows along K where there are too
//     few row blocks to fill the GPU; the FP32 partial sums are added in rank
//     order through distributed shared memory.
// Arithmetic.  A code pair becomes two BF16 numbers by one logic operation
// (0x4300 | q is 128 + q) and one subtraction of 128 + z, both exact: q - z is
// an integer of at most 8 bits.  mma.m16n8k16 multiplies 16 weight rows with 8
// rows of x into an FP32 partial sum of the group, which is then scaled in
// FP32: no weight is ever rounded.  (At one to a few tokens the products cost
// a small part of the tensor cores, whichever instruction issues them; what
// counts is that the sums leave the CUDA cores free to unpack codes.)
// A lane's word holds 8 consecutive codes; (w >> 4 i) & 0x000F000F takes codes
// i and i + 4, so x is paired (i, i + 4) too -- the order inside a product is
// free as long as both operands share it.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "ptx.cuh"

namespace dg {

constexpr int kW4Threads = 256;
constexpr int kW4Rows = 128;            // weight rows per CTA
constexpr int kW4StageK = 256;          // k per stage: 128 bytes of each row
constexpr int kW4XPitch = kW4StageK * 2 + 64;   // bytes; 8 rows' 16-byte reads hit distinct banks
constexpr unsigned kW4SiteBadOffsets = 14;

struct W4Params {
    const __nv_bfloat16 *x;     // [M, K]
    const uint8_t *w;           // [G][N][K/2]
    const __nv_bfloat16 *s;     // [G][K/kGs][N]
    const uint8_t *z;           // [G][K/kGs][N] or null
    __nv_bfloat16 *d;           // [M, N]
    const int32_t *offsets;     // [G + 1]; null: dense
    unsigned *status;
    int M, N, K, G;
};

template <int kGs, int kNT>
struct W4Smem {
    static constexpr int kGroups = kW4StageK / kGs;
    static constexpr int kWBytes = kW4Rows * (kW4StageK / 2);
    static constexpr int kXBytes = 8 * kNT * kW4XPitch;
    static constexpr int kSBytes = kGroups * kW4Rows * 2;
    static constexpr int kZBytes = kGroups * kW4Rows;
    static constexpr int kXOffset = kWBytes;
    static constexpr int kSOffset = kXOffset + kXBytes;
    static constexpr int kZOffset = kSOffset + kSBytes;
    static constexpr int kStageBytes = kZOffset + kZBytes;
    static constexpr int kStages = kNT == 4 ? 3 : 4;
    static constexpr int kAlloc = kStages * kStageBytes;
    // partial sums, [8 kNT][kRedPitch] floats, over the stages
    static constexpr int kRedPitch = kW4Rows + 4;
    static_assert(8 * kNT * kRedPitch * 4 <= kAlloc, "partial sums live in the stages");
    static_assert(kStageBytes % 16 == 0, "16-byte copies");
};

namespace w4 {

// 16 (8) bytes global -> shared; `bytes` of them read, the rest zero
__device__ __forceinline__ void cp16(uint32_t dst, const void *src, uint32_t bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp8(uint32_t dst, const void *src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int n>
__device__ __forceinline__ void cp_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(n) : "memory");
}
__device__ __forceinline__ uint32_t lds32(uint32_t a) {
    uint32_t v;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a));
    return v;
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
    return v;
}
__device__ __forceinline__ uint32_t lds16(uint32_t a) {
    uint16_t v;
    asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(a));
    return v;
}
__device__ __forceinline__ uint32_t lds8(uint32_t a) {
    uint32_t v;
    asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(a));
    return v;
}
__device__ __forceinline__ uint32_t sub_bf16x2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
// codes i and i + 4 of a word as 128 + q, then minus 128 + z
template <int i>
__device__ __forceinline__ uint32_t codes(uint32_t w, uint32_t zero) {
    return sub_bf16x2(((w >> (4 * i)) & 0x000F000Fu) | 0x43004300u, zero);
}
__device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ float4 ld_cluster_f4(uint32_t a) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(a)
                 : "memory");
    return v;
}
// 16-byte chunk `c` of weight row `r` (128 bytes) in a stage: chunks are
// permuted by the row so that 8 rows' chunks at the same k hit distinct banks
__device__ __forceinline__ uint32_t w_at(int r, int c) {
    return static_cast<uint32_t>(r * 128 + ((c ^ (r & 7)) << 4));
}

}  // namespace w4

// grid (split, row blocks, experts), cluster (split, 1, 1)
template <int kGs, int kNT>
__global__ void __launch_bounds__(kW4Threads)
w4_gemv_kernel(const W4Params p) {
    using L = W4Smem<kGs, kNT>;
    constexpr int kTok = 8 * kNT;
    extern __shared__ __align__(128) uint8_t smem[];
    const uint32_t s_base = ptx::smem_u32(smem);
    const int tid = threadIdx.x;
    const int warp = tid / 32, lane = tid % 32;
    const int g8 = lane >> 2, t4 = lane & 3;
    const int split = static_cast<int>(gridDim.x), rank = static_cast<int>(blockIdx.x);
    const int n0 = static_cast<int>(blockIdx.y) * kW4Rows;

    int first = 0, end = p.M;
    const size_t e = blockIdx.z;
    if (p.offsets) {
        // this expert's rows: clamped to the buffer, never before an earlier offset
        const int g = static_cast<int>(e);
        int lo = 0;
        for (int i = lane; i <= g; i += 32) {
            const int raw = __ldg(p.offsets + i);
            lo = max(lo, min(max(raw, 0), p.M));
        }
        lo = __reduce_max_sync(0xffffffffu, lo);
        const int raw_lo = __ldg(p.offsets + g), raw_hi = __ldg(p.offsets + g + 1);
        first = lo;
        end = max(lo, min(max(raw_hi, 0), p.M));
        if ((raw_lo != first || raw_hi != end) && tid == 0) atomicCAS(p.status, 0u, 1u | (kW4SiteBadOffsets << 8));
    }
    if (first >= end) return;                       // the whole cluster: its CTAs share the expert

    const int num_st = (p.K + kW4StageK - 1) / kW4StageK;
    const int st0 = num_st * rank / split, st1 = num_st * (rank + 1) / split;
    const size_t groups = static_cast<size_t>(p.K / kGs);
    const uint8_t *w = p.w + (e * p.N) * static_cast<size_t>(p.K / 2);
    const __nv_bfloat16 *sc = p.s + e * groups * p.N + n0;
    const uint8_t *zp = p.z ? p.z + e * groups * p.N + n0 : nullptr;
    const int rows_left = p.N - n0;

    for (int m0 = first; m0 < end; m0 += kTok) {
        const int ntok = min(kTok, end - m0);
        auto issue = [&](int st) {
            const uint32_t base = s_base + (st - st0) % L::kStages * L::kStageBytes;
            const int k0 = st * kW4StageK;
            const int kv = min(kW4StageK, p.K - k0);
            {
                const int c = tid & 7, r0 = tid >> 3;
                if (c * 32 < kv) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int r = r0 + 32 * i;
                        const int n = min(r, rows_left - 1);        // rows past N: any row, not stored
                        w4::cp16(base + w4::w_at(r, c),
                                 w + (static_cast<size_t>(n0 + n) * p.K + k0) / 2 + c * 16, 16u);
                    }
                }
            }
#pragma unroll
            for (int i = 0; i < kNT; ++i) {
                const int tok = (tid >> 5) + 8 * i, c = tid & 31;
                if (c * 8 < kv) {
                    const bool ok = tok < ntok;                     // tokens past the expert's: zeros
                    w4::cp16(base + L::kXOffset + tok * kW4XPitch + c * 16,
                             p.x + static_cast<size_t>(m0 + (ok ? tok : 0)) * p.K + k0 + c * 8, ok ? 16u : 0u);
                }
            }
            const int c = tid & 15, j = tid >> 4;
            if (j < kv / kGs && c * 8 < rows_left) {
                const size_t at = static_cast<size_t>(k0 / kGs + j) * p.N + c * 8;
                w4::cp16(base + L::kSOffset + j * (kW4Rows * 2) + c * 16, sc + at, 16u);
                if (zp) w4::cp8(base + L::kZOffset + j * kW4Rows + c * 8, zp + at);
            }
        };

        float acc[kNT][4];
#pragma unroll
        for (int i = 0; i < kNT; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[i][j] = 0.f;

#pragma unroll
        for (int i = 0; i < L::kStages - 1; ++i) {
            if (st0 + i < st1) issue(st0 + i);
            w4::cp_commit();
        }
        const int r = warp * 16 + g8;
        for (int st = st0; st < st1; ++st) {
            w4::cp_wait<L::kStages - 2>();
            __syncthreads();                       // stage st has landed; stage st - 1 is free
            if (st + L::kStages - 1 < st1) issue(st + L::kStages - 1);
            w4::cp_commit();
            const uint32_t base = s_base + (st - st0) % L::kStages * L::kStageBytes;
            const int kv = min(kW4StageK, p.K - st * kW4StageK);
#pragma unroll
            for (int j = 0; j < L::kGroups; ++j) {
                if (j * kGs >= kv) break;
                uint32_t z_lo = 0x43084308u, z_hi = 0x43084308u;
                if (zp) {
                    z_lo = (0x4300u | (w4::lds8(base + L::kZOffset + j * kW4Rows + r) & 0x7Fu)) * 0x10001u;
                    z_hi = (0x4300u | (w4::lds8(base + L::kZOffset + j * kW4Rows + r + 8) & 0x7Fu)) * 0x10001u;
                }
                float c[kNT][4];
#pragma unroll
                for (int i = 0; i < kNT; ++i)
#pragma unroll
                    for (int q = 0; q < 4; ++q) c[i][q] = 0.f;
#pragma unroll
                for (int b = j * kGs / 32; b < (j + 1) * kGs / 32; ++b) {
                    const uint32_t lo = w4::lds32(base + w4::w_at(r, b) + t4 * 4);
                    const uint32_t hi = w4::lds32(base + w4::w_at(r + 8, b) + t4 * 4);
                    const uint32_t l0 = w4::codes<0>(lo, z_lo), l1 = w4::codes<1>(lo, z_lo),
                                   l2 = w4::codes<2>(lo, z_lo), l3 = w4::codes<3>(lo, z_lo);
                    const uint32_t h0 = w4::codes<0>(hi, z_hi), h1 = w4::codes<1>(hi, z_hi),
                                   h2 = w4::codes<2>(hi, z_hi), h3 = w4::codes<3>(hi, z_hi);
#pragma unroll
                    for (int i = 0; i < kNT; ++i) {
                        const uint4 x = w4::lds128(base + L::kXOffset + (8 * i + g8) * kW4XPitch + b * 64 + t4 * 16);
                        w4::mma(c[i], l0, h0, l1, h1, __byte_perm(x.x, x.z, 0x5410), __byte_perm(x.x, x.z, 0x7632));
                        w4::mma(c[i], l2, h2, l3, h3, __byte_perm(x.y, x.w, 0x5410), __byte_perm(x.y, x.w, 0x7632));
                    }
                }
                const float s_lo = __uint_as_float(w4::lds16(base + L::kSOffset + (j * kW4Rows + r) * 2) << 16);
                const float s_hi = __uint_as_float(w4::lds16(base + L::kSOffset + (j * kW4Rows + r + 8) * 2) << 16);
#pragma unroll
                for (int i = 0; i < kNT; ++i) {
                    acc[i][0] = fmaf(s_lo, c[i][0], acc[i][0]);
                    acc[i][1] = fmaf(s_lo, c[i][1], acc[i][1]);
                    acc[i][2] = fmaf(s_hi, c[i][2], acc[i][2]);
                    acc[i][3] = fmaf(s_hi, c[i][3], acc[i][3]);
                }
            }
        }
        // partial sums [token][row] over the stages, then the sum over the cluster
        w4::cp_wait<0>();
        __syncthreads();
        float *red = reinterpret_cast<float *>(smem);
#pragma unroll
        for (int i = 0; i < kNT; ++i) {
            float *at = red + (8 * i + 2 * t4) * L::kRedPitch + r;
            at[0] = acc[i][0];
            at[L::kRedPitch] = acc[i][1];
            at[8] = acc[i][2];
            at[L::kRedPitch + 8] = acc[i][3];
        }
        if (split > 1) ptx::cluster_sync_all();
        else __syncthreads();
        const int quads = kW4Rows / 4 / split;      // this CTA's runs of 4 rows
        for (int i = tid; i < quads * ntok; i += kW4Threads) {
            const int tok = i / quads, q = rank * quads + i % quads;
            const uint32_t at = s_base + static_cast<uint32_t>(tok * L::kRedPitch + 4 * q) * 4u;
            float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
            for (int c = 0; c < split; ++c) {
                const float4 v = split > 1 ? w4::ld_cluster_f4(ptx::map_cluster(at, static_cast<uint32_t>(c)))
                                           : *reinterpret_cast<const float4 *>(red + tok * L::kRedPitch + 4 * q);
                sum.x += v.x; sum.y += v.y; sum.z += v.z; sum.w += v.w;
            }
            if (4 * q < rows_left) {
                const __nv_bfloat162 a = __floats2bfloat162_rn(sum.x, sum.y), b = __floats2bfloat162_rn(sum.z, sum.w);
                uint2 o;
                o.x = *reinterpret_cast<const uint32_t *>(&a);
                o.y = *reinterpret_cast<const uint32_t *>(&b);
                *reinterpret_cast<uint2 *>(p.d + static_cast<size_t>(m0 + tok) * p.N + n0 + 4 * q) = o;
            }
        }
        // the partial sums are read before the stages are written again or the CTA leaves
        if (split > 1) ptx::cluster_sync_all();
        else __syncthreads();
    }
}

}  // namespace dg
