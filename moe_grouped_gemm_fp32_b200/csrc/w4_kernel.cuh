// w4_kernel.cuh -- products of a few BF16 rows with 4-bit weights:
//
//   D[m,n] = sum_j s[j,n] * sum_{k in group j} (q[n,k] - z[j,n]) * x[m,k]
//
// q: codes 0..15, two per byte along K; s (BF16) and z (8 where absent): one
// for each row n and group j of kGs consecutive k, stored [K/kGs][N].  Dense,
// or with expert g's weights for the rows offsets[g] .. offsets[g+1).
//
// The weights' bytes are the floor (half a byte and 2/kGs of scale per weight,
// read once); what stands in the way is the number of instructions that unpack
// them: at the memory's rate an SM has 2.8 lane instructions for each weight.
//   * A CTA owns 128 weight rows and a range of K, each of its 4 warps 32 rows.
//     A warp copies its own rows asynchronously, two blocks of 128 k ahead, and
//     waits for nobody; x and the scales come in chunks of 4 blocks, copied by the
//     whole CTA a chunk ahead (staged when its turn came, a chunk held up all warps for
//     a trip to L2: one token, 4096 x 7168, 8.8 us against 7.8).  x is paired for the
//     products once, on its way between two places in shared memory: paired after each
//     read it costs 16 more instructions a block, and 16384 x 7168 took 24.5 us, not 19.3.
//   * A cluster of `split` CTAs shares the 128 rows along K where there are too
//     few row blocks to fill the GPU; each CTA stores its FP32 partial sums into
//     the shared memory of the rows' owners, which add them in rank order.
// Arithmetic.  A code pair becomes two BF16 numbers by one logic operation
// (0x4300 | q is 128 + q) and one subtraction of 128 + z, both exact: q - z is
// an integer of at most 8 bits (a zero point above 127 is recorded, and its low seven
// bits are used).  mma.m16n8k16 multiplies 16 weight rows with 8
// rows of x into an FP32 partial sum of the group, which is then scaled in
// FP32: no weight is ever rounded.
//
// Order of K inside a block of 128.  Both operands of a product may share any
// order, as long as a product stays inside one scale group.  Word i (8 codes) of
// lane t of a quad holds the codes from
//   kGs 128: 32 t + 8 i     kGs 64: 64 (i / 2) + 16 t + 8 (i % 2)     kGs 32: 32 i + 8 t
// -- one 16-byte, two 8-byte or four 4-byte reads a row -- and x lies in shared
// memory at [i][t].  (w >> 4 j) & 0x000F000F takes codes j and j + 4 of a word, so
// each 8 values of x are in pair order (0,4) (1,5) (2,6) (3,7).
// Rows in shared memory: row 4 g + i of a warp at 64 (8 i + g), its 16-byte
// pieces permuted by g, so that the copies and all three reads are free of bank
// conflicts.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "pdl.cuh"
#include "ptx.cuh"

namespace dg {

constexpr int kW4Threads = 128;
constexpr int kW4Rows = 128;            // weight rows per CTA
constexpr int kW4BlockK = 128;          // k per block: 16 bytes of a row for each lane of a quad
constexpr int kW4Depth = 2;             // blocks in flight per warp, a power of two
constexpr int kW4WarpBlock = 32 * (kW4BlockK / 2);                  // bytes of a warp's rows in a block
constexpr unsigned kW4SiteBadOffsets = 14, kW4SiteBadZeros = 15;

struct W4Params {
    const __nv_bfloat16 *x;     // [M, K]
    const uint8_t *w;           // [G][N][K/2]
    const __nv_bfloat16 *s;     // [G][K/kGs][N]
    const uint8_t *z;           // [G][K/kGs][N] or null
    __nv_bfloat16 *d;           // [M, N]
    const int32_t *offsets;     // [G + 1]; null: dense
    unsigned *status;
    int M, N, K, G;
    int tok_cap;                // tokens that shared memory holds: min(8 kNT, M)
    int bufs;                   // chunks of scales that it holds: 2, or 1 where a CTA has no more
};

// x and scales arrive in chunks of 4 blocks, the next one while this one is used.
constexpr int kW4Chunk = 4;
constexpr int kW4XPitch = kW4Chunk * kW4BlockK * 2 + 64;       // bytes; 8 rows' reads are free of bank conflicts

// Byte offsets: the warps' weight blocks, x paired (and a row of zeros), x as it
// arrives, scales, zero points, partial sums.
template <int kGs>
struct W4Smem {
    static constexpr int kSBlock = kW4BlockK / kGs * kW4Rows * 2;   // scales of a block
    static constexpr int kZBlock = kW4BlockK / kGs * kW4Rows;
    static constexpr int kXOffset = kW4Threads / 32 * kW4Depth * kW4WarpBlock;
    __host__ __device__ static int raw_offset(int tok_cap) { return kXOffset + (tok_cap + 1) * kW4XPitch; }
    __host__ __device__ static int s_offset(int tok_cap) { return raw_offset(tok_cap) + tok_cap * kW4Chunk * kW4BlockK * 2; }
    __host__ __device__ static int z_offset(int tok_cap, int bufs) { return s_offset(tok_cap) + bufs * kW4Chunk * kSBlock; }
    __host__ __device__ static int red_offset(int tok_cap, int bufs, bool zeros) {
        return z_offset(tok_cap, bufs) + (zeros ? bufs * kW4Chunk * kZBlock : 0);
    }
    static int bytes(int tok_cap, int bufs, bool zeros) { return red_offset(tok_cap, bufs, zeros) + tok_cap * kW4Rows * 4; }
};

namespace w4 {

// 16 (8) bytes global -> shared; `bytes` of them read, the rest zero
__device__ __forceinline__ void cp16(uint32_t dst, const void *src, uint32_t bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp16(uint32_t dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp8(uint32_t dst, const void *src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int n>
__device__ __forceinline__ void cp_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(n) : "memory");
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
    return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
    uint2 v;
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
    return v;
}
__device__ __forceinline__ uint32_t lds32(uint32_t a) {
    uint32_t v;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a));
    return v;
}
__device__ __forceinline__ void sts128(uint32_t a, uint4 v) {
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
__device__ __forceinline__ uint32_t sub_bf16x2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
// codes i and i + 4 of a word as 128 + q (`bias` 0x43004300), then minus 128 + z
template <int i>
__device__ __forceinline__ uint32_t codes(uint32_t w, uint32_t bias, uint32_t zero) {
    uint32_t d;
    asm("lop3.b32 %0, %1, 0x000F000F, %2, 0xEA;" : "=r"(d) : "r"(w >> (4 * i)), "r"(bias));   // (a & b) | c
    return sub_bf16x2(d, zero);
}
__device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// the first product of a sum
__device__ __forceinline__ void mma_first(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                          uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%10, %10, %10, %10};"
        : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}

// 16-byte piece `c` of row 4 g + i of a warp's block
__device__ __forceinline__ uint32_t w_at(int i, int g, int c) {
    return static_cast<uint32_t>((8 * i + g) * 64 + ((c ^ ((g & 2) | (g >> 2))) << 4));
}
// Place [i][t] of the 8 values from k = 8 c of a block, as i * 4 + t.
template <int kGs>
__device__ __forceinline__ int x_slot(int c) {
    if (kGs == 128) return (c & 3) * 4 + (c >> 2);
    if (kGs == 64) return ((c >> 3) * 2 + (c & 1)) * 4 + ((c >> 1) & 3);
    return c;
}

// The z-th run of at most run_rows rows of an expert: the expert, the run's first row
// and its end; false if there are fewer runs.  Offsets are used clamped to [0, M] and raised to the largest
// before; `record` marks those that were not so.
__device__ __forceinline__ bool find_expert(const W4Params &p, int run_rows, int z, bool record, int lane, int &expert, int &first,
                                            int &end) {
    int run = 0, seen = 0;
    bool found = false;
    for (int base = 0; base <= p.G; base += 128) {      // four offsets a lane, their loads in flight together
        int raw[4], v[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int i = base + 4 * lane + j;
            raw[j] = i <= p.G ? p.offsets[i] : 0;
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            v[j] = min(max(raw[j], 0), p.M);
            if (j) v[j] = max(v[j], v[j - 1]);
        }
        int incl = v[3];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int u = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl = max(incl, u);
        }
        int before = __shfl_up_sync(0xffffffffu, incl, 1);
        before = max(run, lane ? before : 0);            // offset base + 4 lane - 1
        int count = 0, last = before;
#pragma unroll
        for (int j = 0; j < 4; ++j) {                    // offset i closes expert i - 1
            const int i = base + 4 * lane + j;
            v[j] = max(v[j], before);
            if (record && i <= p.G && v[j] != raw[j]) atomicCAS(p.status, 0u, 1u | (kW4SiteBadOffsets << 8));
            if (i >= 1 && i <= p.G) count += (v[j] - last + run_rows - 1) / run_rows;
            last = v[j];
        }
        int upto = count;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int u = __shfl_up_sync(0xffffffffu, upto, o);
            if (lane >= o) upto += u;
        }
        const int rank = z - seen - (upto - count);       // of the expert sought among this lane's
        const bool here = rank >= 0 && rank < count;
        int at = 0, from = 0, to = 0, k = 0;
        last = before;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int i = base + 4 * lane + j;
            if (i >= 1 && i <= p.G && v[j] > last) {
                const int runs = (v[j] - last + run_rows - 1) / run_rows;
                if (rank >= k && rank < k + runs) {
                    at = i - 1;
                    from = last + (rank - k) * run_rows;
                    to = min(v[j], from + run_rows);
                }
                k += runs;
            }
            last = v[j];
        }
        const unsigned mask = __ballot_sync(0xffffffffu, here);
        if (mask != 0u) {
            const int src = __ffs(static_cast<int>(mask)) - 1;
            expert = __shfl_sync(0xffffffffu, at, src);
            first = __shfl_sync(0xffffffffu, from, src);
            end = __shfl_sync(0xffffffffu, to, src);
            found = true;
            if (!record) return true;
        }
        seen += __shfl_sync(0xffffffffu, upto, 31);
        run = max(run, __shfl_sync(0xffffffffu, incl, 31));
    }
    return found;
}

}  // namespace w4

// grid (split, row blocks, runs of 8 kNT tokens), cluster (split, 1, 1)
template <int kGs, int kNT, bool kZeros>
__global__ void __launch_bounds__(kW4Threads, kNT == 4 ? 3 : kNT == 2 ? 4 : 5)
w4_gemv_kernel(const W4Params p) {
    using L = W4Smem<kGs>;
    constexpr int kTok = 8 * kNT;
    constexpr int kGroups = kW4BlockK / kGs;        // scale groups of a block
    constexpr int kWords = 4 / kGroups;             // words of a lane in a group
    constexpr int kRawTok = kW4Chunk * kW4BlockK * 2;   // bytes of a token's x in a chunk
    extern __shared__ __align__(128) uint8_t smem[];   // the reads' permutation wants 64
    const uint32_t s_base = ptx::smem_u32(smem);
    const int tid = threadIdx.x;
    const int warp = tid / 32, lane = tid % 32;
    const int g8 = lane >> 2, t4 = lane & 3;
    const int split = static_cast<int>(gridDim.x), rank = static_cast<int>(blockIdx.x);
    const int n0 = static_cast<int>(blockIdx.y) * kW4Rows;

    // The launch may overlap the end of the kernel before it in the stream: from here on
    // that kernel is done and its writes are visible.
    pdl::grid_dependency_wait();
    int expert = 0, first = static_cast<int>(blockIdx.z) * kTok, end = min(p.M, first + kTok);
    if (p.offsets) {
        const int z = static_cast<int>(blockIdx.z);
        const bool record = z == 0 && rank == 0 && n0 == 0 && warp == 0;
        if (!w4::find_expert(p, kTok, z, record, lane, expert, first, end)) return;   // the whole cluster: it shares z
    }

    const int num_blk = (p.K + kW4BlockK - 1) / kW4BlockK;
    const int blk0 = static_cast<int>(static_cast<long long>(num_blk) * rank / split);
    const int blk1 = static_cast<int>(static_cast<long long>(num_blk) * (rank + 1) / split);
    const size_t e = static_cast<size_t>(expert);
    const size_t groups = static_cast<size_t>(p.K / kGs);
    const __nv_bfloat16 *sc = p.s + e * groups * p.N + n0;
    const uint8_t *zp = kZeros ? p.z + e * groups * p.N + n0 : nullptr;
    const int rows_left = p.N - n0;
    const int r0 = warp * 32 + 4 * g8;              // this lane's rows r0 .. r0 + 3 of the CTA's (rows past N: row N - 1)
    const uint8_t *wrow[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        wrow[i] = p.w + (e * p.N + n0 + min(r0 + i, rows_left - 1)) * static_cast<size_t>(p.K / 2) + t4 * 16;
    const uint32_t s_off = s_base + L::s_offset(p.tok_cap) + r0 * 2;
    const uint32_t z_off = s_base + L::z_offset(p.tok_cap, p.bufs) + r0;

    // first of this lane's reads of a row: a 16-byte piece, 8 bytes or a word of one
    const uint32_t w_read = s_base + warp * (kW4Depth * kW4WarpBlock) +
                            (kGs == 128 ? w4::w_at(0, g8, t4)
                             : kGs == 64 ? w4::w_at(0, g8, t4 >> 1) + (t4 & 1) * 8 : w4::w_at(0, g8, 0) + t4 * 4);
    const uint32_t w_off = s_base + warp * (kW4Depth * kW4WarpBlock);
    const uint32_t red_off = s_base + L::red_offset(p.tok_cap, p.bufs, kZeros);
    const uint32_t zero_row = s_base + L::kXOffset + p.tok_cap * kW4XPitch;
    uint32_t bias;
    asm volatile("mov.u32 %0, 0x43004300;" : "=r"(bias));
    for (int i = tid * 16; i < kW4XPitch; i += kW4Threads * 16)
        w4::sts128(zero_row + i, make_uint4(0u, 0u, 0u, 0u));
    if (split > 1) ptx::cluster_arrive_relaxed();   // waited for before the first store into another CTA

    // A warp's rows of block `blk`, whose slot `u` is its place in its chunk modulo kW4Depth, from
    // `ahead` bytes past wptr; zeros past K.
    const uint8_t *wptr[4];
    const int full = min(blk1, p.K / kW4BlockK);
    const uint32_t w_copy = w_off + w4::w_at(0, g8, t4);
    auto copy = [&](int blk, int u, int ahead) {
        if (blk < full) {
#pragma unroll
            for (int i = 0; i < 4; ++i) w4::cp16(w_copy + u * kW4WarpBlock + i * 512, wptr[i] + ahead);
        } else if (blk < blk1) {                   // the last block, where K ends inside it
            const uint32_t bytes = blk * kW4BlockK + t4 * 32 < p.K ? 16u : 0u;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                w4::cp16(w_copy + u * kW4WarpBlock + i * 512, bytes ? wptr[i] + ahead : p.w, bytes);
        }
        w4::cp_commit();
    };

    const int m0 = first, ntok = end - first;
    float acc[2][kNT][4];
#pragma unroll
    for (int r = 0; r < 2; ++r)
#pragma unroll
        for (int i = 0; i < kNT; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[r][i][j] = 0.f;
    const uint32_t raw = s_base + L::raw_offset(p.tok_cap) + (tid >> 4) * kRawTok + (tid & 15) * 16;
    // x of the blocks c .. c + 3 as it is, their scales into buffer `buf`
    auto stage = [&](int c, int buf) {
        const int nblk = min(kW4Chunk, blk1 - c);
        // x in pieces of 8 values; zeros past K.  Thread: piece tid % 16 of a block, tokens
        // tid / 16, tid / 16 + 8, ..., which it alone reads again (pair).
        const int left = p.K - (c * kW4BlockK + (tid & 15) * 8);
#pragma unroll
        for (int n = 0; n < kNT; ++n) {
            const int tok = 8 * n + (tid >> 4);
            if (tok < ntok) {
                const __nv_bfloat16 *src = p.x + static_cast<size_t>(m0 + tok) * p.K + static_cast<size_t>(c) * kW4BlockK + (tid & 15) * 8;
                const uint32_t dst = raw + n * (8 * kRawTok);
#pragma unroll
                for (int b = 0; b < kW4Chunk; ++b)
                    if (b < nblk) {
                        const bool ok = b * kW4BlockK < left;
                        w4::cp16(dst + b * 256, ok ? src + b * kW4BlockK : p.x, ok ? 16u : 0u);
                    }
            }
        }
        // scales and zero points; scales of groups past K: zero
        for (int i = tid; i < nblk * kGroups * 16; i += kW4Threads) {
            const int j = i >> 4, q = i & 15;
            if (q * 8 < rows_left) {
                const int grp = c * kGroups + j;
                const bool ok = grp < static_cast<int>(groups);
                const size_t at = static_cast<size_t>(ok ? grp : 0) * p.N + q * 8;
                w4::cp16(s_base + L::s_offset(p.tok_cap) + buf * (kW4Chunk * L::kSBlock) + j * (kW4Rows * 2) + q * 16,
                         sc + at, ok ? 16u : 0u);
                if (kZeros)
                    w4::cp8(s_base + L::z_offset(p.tok_cap, p.bufs) + buf * (kW4Chunk * L::kZBlock) + j * kW4Rows + q * 8, zp + at);
            }
        }
    };

    // this thread's pieces of x to where the products want them, in pair order
    auto pair = [&](int nblk) {
#pragma unroll
        for (int n = 0; n < kNT; ++n) {
            const int tok = 8 * n + (tid >> 4);
            if (tok < ntok) {
                const uint32_t src = raw + n * (8 * kRawTok);
                const uint32_t dst = s_base + L::kXOffset + tok * kW4XPitch + w4::x_slot<kGs>(tid & 15) * 16;
#pragma unroll
                for (int b = 0; b < kW4Chunk; ++b)
                    if (b < nblk) {
                        const uint4 v = w4::lds128(src + b * 256);
                        w4::sts128(dst + b * 256, make_uint4(__byte_perm(v.x, v.z, 0x5410), __byte_perm(v.x, v.z, 0x7632),
                                                             __byte_perm(v.y, v.w, 0x5410), __byte_perm(v.y, v.w, 0x7632)));
                    }
            }
        }
    };

    // where this lane's rows of x lie: tokens past the run's read zeros
    uint32_t xa[kNT];
#pragma unroll
    for (int n = 0; n < kNT; ++n)
        xa[n] = (8 * n + g8 < ntok ? s_base + L::kXOffset + (8 * n + g8) * kW4XPitch : zero_row) + t4 * 16;
#pragma unroll
    for (int i = 0; i < 4; ++i) wptr[i] = wrow[i] + static_cast<size_t>(blk0) * (kW4BlockK / 2);
    stage(blk0, 0);
    w4::cp_commit();
#pragma unroll
    for (int d = 0; d < kW4Depth; ++d) copy(blk0 + d, d, d * (kW4BlockK / 2));
    w4::cp_wait<kW4Depth>();                       // the first chunk has landed

    int buf = 0;
    // All bits of this lane's zero points: one OR a group (8 of 64 experts, 4096 x 2048, groups
    // of 32: 14.2 -> 14.4 us; looked through once as they land: 14.6).
    uint32_t seen = 0;
    for (int c0 = blk0; c0 < blk1; c0 += kW4Chunk) {
        if (c0 != blk0) __syncthreads();           // the chunk before has been read
        pair(min(kW4Chunk, blk1 - c0));
        __syncthreads();
        if (c0 + kW4Chunk < blk1) stage(c0 + kW4Chunk, buf ^ 1);
        w4::cp_commit();
        const uint32_t sa = s_off + buf * (kW4Chunk * L::kSBlock), za = z_off + buf * (kW4Chunk * L::kZBlock);
#pragma unroll
        for (int u = 0; u < kW4Chunk; ++u) {
            if (c0 + u >= blk1) break;
            // this block's copies have landed: behind them are those of the next block
            // and, until kW4Depth blocks of the chunk are done, the next chunk's (which
            // has landed, too, when the last wait of four is over)
            if (u < kW4Depth) w4::cp_wait<kW4Depth>();
            else w4::cp_wait<kW4Depth - 1>();
            __syncwarp();                      // of every lane
#pragma unroll
            for (int j = 0; j < kGroups; ++j) {
                uint32_t zero[4] = {0x43084308u, 0x43084308u, 0x43084308u, 0x43084308u};
                if constexpr (kZeros) {
                    const uint32_t z4 = w4::lds32(za + u * L::kZBlock + j * kW4Rows);
                    const uint32_t zb = z4 & 0x7F7F7F7Fu;
                    seen |= z4;
#pragma unroll
                    for (int i = 0; i < 4; ++i) zero[i] = __byte_perm(zb, 0x43u, 0x4040 + i * 0x0101);   // 128 + z
                }
                uint32_t w[4][kWords];
                const uint32_t wa = (w_read ^ (j * (64 / kGroups))) + u % kW4Depth * kW4WarpBlock;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if constexpr (kGs == 128) {
                        const uint4 v = w4::lds128(wa + i * 512);
                        w[i][0] = v.x; w[i][1] = v.y; w[i][2] = v.z; w[i][3] = v.w;
                    } else if constexpr (kGs == 64) {
                        const uint2 v = w4::lds64(wa + i * 512);
                        w[i][0] = v.x; w[i][1] = v.y;
                    } else {
                        w[i][0] = w4::lds32(wa + i * 512);
                    }
                }
                float c[2][kNT][4];
#pragma unroll
                for (int k = 0; k < kWords; ++k) {
                    uint4 x[kNT];
#pragma unroll
                    for (int n = 0; n < kNT; ++n) x[n] = w4::lds128(xa[n] + u * 256 + (j * kWords + k) * 64);
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        const uint32_t lo = w[2 * r][k], hi = w[2 * r + 1][k];
                        const uint32_t zl = zero[2 * r], zh = zero[2 * r + 1];
                        const uint32_t l0 = w4::codes<0>(lo, bias, zl), l1 = w4::codes<1>(lo, bias, zl),
                                       l2 = w4::codes<2>(lo, bias, zl), l3 = w4::codes<3>(lo, bias, zl);
                        const uint32_t h0 = w4::codes<0>(hi, bias, zh), h1 = w4::codes<1>(hi, bias, zh),
                                       h2 = w4::codes<2>(hi, bias, zh), h3 = w4::codes<3>(hi, bias, zh);
#pragma unroll
                        for (int n = 0; n < kNT; ++n) {
                            if (k == 0) w4::mma_first(c[r][n], l0, h0, l1, h1, x[n].x, x[n].y);
                            else w4::mma(c[r][n], l0, h0, l1, h1, x[n].x, x[n].y);
                            w4::mma(c[r][n], l2, h2, l3, h3, x[n].z, x[n].w);
                        }
                    }
                }
                const uint2 sv = w4::lds64(sa + u * L::kSBlock + j * (kW4Rows * 2));
                const float s4[4] = {__uint_as_float(sv.x << 16), __uint_as_float(sv.x & 0xFFFF0000u),
                                     __uint_as_float(sv.y << 16), __uint_as_float(sv.y & 0xFFFF0000u)};
#pragma unroll
                for (int r = 0; r < 2; ++r)
#pragma unroll
                    for (int n = 0; n < kNT; ++n) {
                        acc[r][n][0] = fmaf(s4[2 * r], c[r][n][0], acc[r][n][0]);
                        acc[r][n][1] = fmaf(s4[2 * r], c[r][n][1], acc[r][n][1]);
                        acc[r][n][2] = fmaf(s4[2 * r + 1], c[r][n][2], acc[r][n][2]);
                        acc[r][n][3] = fmaf(s4[2 * r + 1], c[r][n][3], acc[r][n][3]);
                    }
            }
            __syncwarp();                  // every lane has read this block
            copy(c0 + u + kW4Depth, u % kW4Depth, (u + kW4Depth) * (kW4BlockK / 2));
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) wptr[i] += kW4Chunk * (kW4BlockK / 2);
        buf ^= 1;
    }
    if (kZeros && (seen & 0x80808080u) != 0u && r0 < rows_left) atomicCAS(p.status, 0u, 1u | (kW4SiteBadZeros << 8));
    // This lane's sums of 4 rows for 2 kNT tokens go to the rows' owner: rank
    // r adds rows 128 r / split .. and keeps [source rank][token][its rows].
    const int own = kW4Rows / split;            // rows per owner, at least 16
    const uint32_t slot = red_off + static_cast<uint32_t>(rank * p.tok_cap * own + (r0 & (own - 1))) * 4u;
    const uint32_t dst = split > 1 ? ptx::map_cluster(slot, static_cast<uint32_t>(r0 / own)) : slot;
    if (split > 1) ptx::cluster_wait_acquire();     // every CTA of the cluster has started
#pragma unroll
    for (int n = 0; n < kNT; ++n)
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            const int tok = 8 * n + 2 * t4 + q;
            if (tok < ntok)
                ptx::st_cluster_v4(dst + static_cast<uint32_t>(tok * own) * 4u, acc[0][n][q], acc[0][n][2 + q],
                                   acc[1][n][q], acc[1][n][2 + q]);
        }
    if (split > 1) ptx::cluster_sync_all();
    else __syncthreads();
    const int quads = own / 4;                  // this CTA's runs of 4 rows
    const float *red = reinterpret_cast<const float *>(smem + (red_off - s_base));
    for (int i = tid; i < quads * ntok; i += kW4Threads) {
        const int tok = i / quads, q = i - tok * quads;
        float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int c = 0; c < split; ++c) {
            const float4 v = *reinterpret_cast<const float4 *>(red + (c * p.tok_cap + tok) * own + 4 * q);
            sum.x += v.x; sum.y += v.y; sum.z += v.z; sum.w += v.w;
        }
        const int row = rank * own + 4 * q;
        if (row < rows_left) {
            const __nv_bfloat162 a = __floats2bfloat162_rn(sum.x, sum.y), b = __floats2bfloat162_rn(sum.z, sum.w);
            uint2 o;
            o.x = *reinterpret_cast<const uint32_t *>(&a);
            o.y = *reinterpret_cast<const uint32_t *>(&b);
            *reinterpret_cast<uint2 *>(p.d + static_cast<size_t>(m0 + tok) * p.N + n0 + row) = o;
        }
    }
}

}  // namespace dg
