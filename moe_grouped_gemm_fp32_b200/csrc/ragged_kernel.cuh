// ragged_kernel.cuh -- the sm_100a kernel of the ragged grouped BF16 products:
// experts own runs of a token buffer given by offsets on the device, with no
// padding between them.  Three directions share one kernel:
//
//   kNT  D[r,n]    = sum_k A[r,k] * B[g(r)][n,k]        forward
//   kNN  D[r,n]    = sum_k A[r,k] * B[g(r)][k,n]        input gradient
//   kTN  D[g][m,n] = sum_{r in g} A[r,m] * B[r,n]       weight gradient
//
// Operands.  tcgen05.mma reads either operand K-major (the reduced index
// innermost) or MN-major; both come straight from the caller's layout by TMA
// with 128-byte swizzle, nothing is transposed in memory:
//   K-major   box {64 K, rows}: one 128-byte line per row (kNT: A and B, kNN: A)
//   MN-major  boxes {64 M or N, 64 K}: one 128-byte line per reduced index, 64
//             columns wide; 8192 bytes between boxes, 1024 bytes between
//             groups of 8 reduced indices (kNN: B, kTN: A and B)
//
// Ragged edges.
//   kNT, kNN: a tile's token rows start at the expert's offset (TMA row
//     coordinates need no alignment) and may run past its end: those rows are
//     computed from the neighbour's tokens and not stored.  Rows of the product
//     do not mix, so a NaN there stays there.
//   kTN: the last block of 64 tokens of an expert may run into the next one's.
//     Its MMAs stop at the last started group of 16 tokens, and the rows between
//     the expert's end and that group's end have to be zeros, in both operands (0 *
//     NaN would be NaN).  They come by TMA like the tokens themselves: such a block is
//     put together from boxes of tail_rows(i) tokens, and for the zeros from boxes
//     that lie behind the buffer's last row.  So whatever the MMAs read, the
//     second CTA of a pair included, has arrived on the one barrier that they wait
//     for.  (Rows that a warp clears by plain stores have to be released to the other
//     CTA's tensor core at cluster scope: weight gradient of 64 experts of 62 tokens,
//     1000 x 2112, BF16, 80.6 us against 70.3.  Boxes of 32, 16, 8, 4, 2 and 1 tokens:
//     70.4, and 1 us more on the host for their maps.)
//
// Output.  A lane holds one row of the accumulator; stored straight from there,
// each instruction touches 32 lines (weight gradient of 64 experts, 62 tokens each,
// 1000 x 2112, BF16: 174 us, against 46 for its bytes).  So a warp turns 32 x 32
// boxes (single CTAs of kNT, kNN: 32 weights x 16 tokens) around in shared memory and
// stores runs of a row.
//
// Roles: warp 0 producer (TMA), warp 1 TMEM and MMA issue, warps 4.. epilogue: warp w
// drains TMEM lanes 32 (w % 4), columns of half (w / 4 - 1) % 2.  Persistent; two accumulators in rotation, so the next
// tile's MMAs overlap this tile's stores; with one-level sums a group of 8 epilogue
// warps for each, so that tiles of few tokens store two at a time.
//
// CTA pairs (kCtaGroup == 2): 256 x kBN tiles, each CTA stages its 128 rows of
// A and half of B's columns.  Single CTAs take over where experts have few
// rows: there A comes in boxes of 32 rows, only those that the expert has, so
// that weight bytes, not token tiles, fill the memory pipeline.  Where experts have
// a few rows, or the call few tiles, they are thin (kRows 32): a stage keeps 4 KB for
// A and not 16, and twice as many weight bytes are in flight (64 rows over 16 experts,
// 4096 x 7168, in a graph: 155 us in tiles of 128 rows, 138 in thin ones, the copy rate).
//
// Single CTAs of kNT and kNN make the weights the MMA's 128 rows and the tokens its
// columns, as many as the expert has, rounded up to 16: the other way round, products
// of rows that no expert has cost time and the clock (in a loop of calls, where the GPU
// is hotter than in a graph of few, those 64 rows: 165 -> 141 us; 64 experts of 62 rows on
// average, 1000 x 2112: 66 -> 61; both with one-level sums).  Tiles of 64 weights leave
// the MMA's upper rows whatever follows in shared memory (the next stage, in the middle
// of being written perhaps); nobody reads those accumulator rows.
//
// Precision.  The tensor core's FP32 accumulator truncates: measured against 64
// bits, a sum of 8192 products loses 9e-6 (relative, 2-norm) and 32768 products
// 1.9e-5, where rounded FP32 sums lose 1e-6 and 2.3e-6; products of one sign lose in
// proportion to their number (16.8 million of them: 9.7 %).  So sums have two
// levels: every kSegBlocks K-blocks the accumulator is read out and added, rounded, to
// FP32 registers of the epilogue warps.  A segment is 512 products for FP32 results
// (5e-7) and 1024 for BF16 ones (1e-6): each costs the tensor core a pause of 0.2 us,
// seen where one tile's latency is the call's (one expert of 64 rows, 512 x 8192:
// 17.2 us in one level, 20.4 with 512, 18.8 with 1024, 17.9 with 2048) and not
// elsewhere (64 rows, 16 experts, 4096 x 7168: 137 each; 64 experts of 62 rows, 1000 x
// 2112: 59.0 and 59.9; 32768 rows in a loop 1538 and 1555, whatever the segments'
// length).  Only short BF16 weight gradients go without (rule and figures in
// ragged_api.cu).
//
// Every wait is bounded (BoundedWait).
#pragma once

#include "gemm_kernel.cuh"
#include "pdl.cuh"

namespace dg {

enum RaggedDir : int { kNT = 0, kNN = 1, kTN = 2 };

// 4 warps that load and multiply, and 8 warps for each accumulator in rotation;
// two-level sums take one such group, with more registers
__host__ __device__ constexpr int ragged_threads(bool two_level) { return two_level ? 384 : 640; }
constexpr int kRaggedBlockK = 64;
// Row blocks per L2 raster band at most; an expert's bands are equally high (33 row
// blocks of 8192 tokens and a few: 11 each).  Bands of 8, 12, 16, 32 on the prompt's
// input gradient: 1413, 1359, 1369, 1496 us.
constexpr int kRaggedBand = 16;
constexpr unsigned kSiteBadOffsets = 12;
// kTN: tokens of the boxes that an expert's last block is put together from
constexpr int kTailMaps = 3;
__host__ __device__ constexpr int tail_rows(int i) { return i == 0 ? 16 : i == 1 ? 4 : 1; }

struct RaggedParams {
    void *d;
    const int32_t *offsets;   // [G + 1]
    unsigned *status;
    long long timeout_cycles;
    int T;                    // rows of the token buffer
    int M, N, K;              // kTN: output rows M; kNT, kNN: reduced size K
    int G;
    int accumulate;           // kTN: add to d
    // When the next grid's blocks may be placed: once this grid's blocks are set up, or
    // each when its tiles are done.  (The first thread of a block that says so counts.)
    int signal_early;
    int debug_flags;
};

// The operands' tensor maps; kNT, kNN single CTAs: A boxes of 32 rows.
template <int kDir>
struct RaggedMaps {
    CUtensorMap a, b;
};
template <>
struct RaggedMaps<kTN> {
    CUtensorMap a, b;                                 // boxes of kRaggedBlockK tokens
    CUtensorMap a_tail[kTailMaps], b_tail[kTailMaps]; // of tail_rows(i)
};

template <int kDir, int kBN, int kStages, int kCtaGroup, bool kF32, int kRows, bool kTwoLevel>
struct RaggedSmem {
    static constexpr int kABytes = kRows * 128;
    static constexpr int kBCols = kBN / kCtaGroup;            // this CTA's columns of B
    static constexpr int kBBytes = kBCols * 128;
    // K-blocks of 64 in a stage: two in thin tiles of 64 columns, where few tiles wait on
    // a block's barriers and issue (0.2 us) rather than on its bytes: 4 rows, 1024 x
    // 8192, 26.2 -> 17.6 us (18.5 with two-level sums); four a stage, of which then three
    // fit: 19.7
    static constexpr int kSub = kRows == 32 && kBN == 64 ? 2 : 1;
    static constexpr int kSubBytes = kABytes + kBBytes;
    static constexpr int kStageBytes = kSub * kSubBytes;
    static constexpr int kAccBufs = 2;
    static constexpr int kBarOffset = kStages * kStageBytes;
    static constexpr int kNumBars = 2 * kStages + 2 * kAccBufs + 1;
    static constexpr int kMiscOffset = kBarOffset + kNumBars * 8;   // tmem addr, abort flag
    static constexpr int kOffsOffset = (kMiscOffset + 16 + 15) / 16 * 16;
    static constexpr int kPrefixOffset = kOffsOffset + (kMaxGroups + 1) * 4;
    // epilogue: 32 rows by 32 columns for each of its warps
    static constexpr int kBoxBytes = 32 * 32 * (kF32 ? 4 : 2);
    static constexpr int kOutOffset = (kPrefixOffset + (kMaxGroups + 1) * 4 + 1023) / 1024 * 1024;
    static constexpr int kUsed = kOutOffset + (ragged_threads(kTwoLevel) / 32 - 4) * kBoxBytes;
    static constexpr int kAlloc = (kUsed + 1024 > kMinSmem) ? kUsed + 1024 : kMinSmem;
    static constexpr bool kSwap = kDir != kTN && kCtaGroup == 1;     // weights are rows, tokens columns
    static constexpr int kAccCols = kSwap ? kRows : kBN;
    static constexpr int kTmemCols = kAccBufs * kAccCols <= 128 ? kAccBufs * kAccCols
                                     : kAccBufs * kAccCols <= 256 ? 256 : 512;
    static_assert(kBN == 64 || kBN == 128 || kBN == 256, "tile N");
    static_assert(kBCols % 64 == 0, "MN-major boxes are 64 columns wide");
    static_assert(kAlloc <= 227 * 1024, "shared memory budget");
};

// MN-major, 128-byte swizzle: boxes of 64 columns by 64 reduced indices, 8192
// bytes apart (leading offset); 1024 bytes between groups of 8 reduced indices.
__device__ __forceinline__ uint64_t sw128_mn_desc(uint32_t saddr) {
    uint64_t d = 0;
    d |= static_cast<uint64_t>((saddr & 0x3FFFF) >> 4);
    d |= static_cast<uint64_t>(8192 >> 4) << 16;
    d |= static_cast<uint64_t>(1024 >> 4) << 32;
    d |= static_cast<uint64_t>(1) << 46;
    d |= static_cast<uint64_t>(2) << 61;
    return d;
}

// kind::f16, D = F32, A = B = BF16; bits 15 and 16 mark MN-major A and B.
__host__ __device__ constexpr uint32_t ragged_idesc(int m, int n, bool a_mn, bool b_mn) {
    return (1u << 4) | (1u << 7) | (1u << 10) | (a_mn ? 1u << 15 : 0u) | (b_mn ? 1u << 16 : 0u) |
           (static_cast<uint32_t>(n >> 3) << 17) | (static_cast<uint32_t>(m >> 4) << 24);
}

// The tiles of the experts in order, and where the walk stands: every role goes
// through its CTA's tiles (t ascending) by itself.  What holds for an expert is kept
// while its tiles last, and divisions are by a reciprocal: the walk is one thread's
// chain of dependent instructions once a tile, which bounds tiles with few K-blocks.
template <int kDir, int kBN, int kCtaGroup, int kCtaRows>
struct RaggedTile {
    static constexpr int kRows = kCtaRows * kCtaGroup;
    // the tile
    int g;
    int row0;      // kNT, kNN: first token row of the tile (in the buffer); kTN: first output row
    int row_end;   // exclusive bound of its valid rows
    int n0;
    int num_kb;    // K-blocks of 64
    int tail;      // kTN: tokens in the last K-block (1..64), 64 elsewhere
    int tok0;      // first token of the expert
    // the expert
    int base, next;        // its tiles [base, next)
    unsigned rb, height;   // row blocks, and those of a band
    float inv;             // 1 / height

    __device__ static int row_blocks(const RaggedParams &p, const int *offs, int g) {
        const int rows = kDir == kTN ? p.M : offs[g + 1] - offs[g];
        return (rows + kRows - 1) / kRows;
    }
    // n / d with inv = 1 / d, put right by a step (small n)
    __device__ static unsigned quotient(unsigned n, unsigned d, float inv) {
        if (n >= (1u << 22)) return n / d;
        unsigned q = static_cast<unsigned>(static_cast<float>(n) * inv);
        if (q * d > n) --q;
        if (n - q * d >= d) ++q;
        return q;
    }

    __device__ __forceinline__ RaggedTile() : g(-1), base(0), next(0) {}

    __device__ __forceinline__ void decode(int t, const RaggedParams &p, const int *offs, const int *prefix) {
        const unsigned nb = (p.N + kBN - 1) / kBN;
        if (t >= next) {
            do {
                ++g;
                base = next;
                if (kDir == kTN) next += row_blocks(p, offs, 0) * static_cast<int>(nb);    // alike for all
                else next = prefix[g + 1];
            } while (t >= next);
            tok0 = offs[g];
            const int end = offs[g + 1];
            rb = row_blocks(p, offs, g);
            height = rb;
            if (rb > kRaggedBand) {
                const unsigned bands = (rb + kRaggedBand - 1) / kRaggedBand;
                height = (rb + bands - 1) / bands;
            }
            inv = __fdividef(1.f, static_cast<float>(height));
            if (kDir == kTN) {
                row_end = p.M;
                num_kb = (end - tok0 + kRaggedBlockK - 1) / kRaggedBlockK;
                tail = end - tok0 - (num_kb - 1) * kRaggedBlockK;
            } else {
                row_end = end;
                num_kb = (p.K + kRaggedBlockK - 1) / kRaggedBlockK;
                tail = kRaggedBlockK;
            }
        }
        unsigned in_band = t - base, first = 0, width = height;
        float inv_w = inv;
        if (rb > kRaggedBand) {
            const unsigned band = in_band / (height * nb);
            first = band * height;
            in_band -= first * nb;
            if (rb - first < height) {
                width = rb - first;
                inv_w = __fdividef(1.f, static_cast<float>(width));
            }
        }
        const unsigned col = quotient(in_band, width, inv_w);
        const int row = static_cast<int>(first + in_band - col * width) * kRows;
        n0 = static_cast<int>(col) * kBN;
        row0 = kDir == kTN ? row : tok0 + row;
    }
};

__device__ __forceinline__ uint32_t pack_bf16x2(float a, float b) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
}

// Adds eight columns to a row of BF16: widened exactly, added in FP32, rounded once.
__device__ __forceinline__ void add8(__nv_bfloat16 *d, const float *v) {
    uint4 *o = reinterpret_cast<uint4 *>(d);
    const uint4 x = *o;
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
    float s[8];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        s[2 * j] = v[2 * j] + __uint_as_float(w[j] << 16);
        s[2 * j + 1] = v[2 * j + 1] + __uint_as_float(w[j] & 0xFFFF0000u);
    }
    *o = make_uint4(pack_bf16x2(s[0], s[1]), pack_bf16x2(s[2], s[3]), pack_bf16x2(s[4], s[5]), pack_bf16x2(s[6], s[7]));
}

// A warp's way from accumulator rows (one a lane) to runs of a row in memory, 32
// columns at a time: `put` writes a box of 32 rows to shared memory, its 16-byte
// pieces permuted by the row against bank conflicts, and stores it in runs of 64 (BF16)
// or 128 bytes of a row.  Addresses that do not change are kept.
template <bool kF32>
struct BoxWriter {
    static constexpr int kElem = kF32 ? 4 : 2;
    static constexpr int kPieces = kF32 ? 8 : 4;        // 16-byte pieces of a row
    static constexpr int kRowsAt = 32 / kPieces;        // rows of one store instruction
    uint32_t in[kPieces], out[kPieces];                 // this lane's pieces in shared memory
    uint8_t *dst[kPieces];                              // and in memory, for the tile's first columns
    uint32_t row_ok;                                    // a bit for each of them
    int col;                                            // its first column in a box

    __device__ __forceinline__ BoxWriter(uint32_t box, int lane) {
        col = lane % kPieces * (16 / kElem);
#pragma unroll
        for (int i = 0; i < kPieces; ++i) {
            const int r = lane / kPieces + i * kRowsAt;
            in[i] = box + lane * (32 * kElem) + ((i ^ swizzle(lane)) << 4);
            out[i] = box + r * (32 * kElem) + ((lane % kPieces ^ swizzle(r)) << 4);
        }
    }
    __device__ __forceinline__ static int swizzle(int row) { return kF32 ? row & 7 : (row >> 1) & 3; }

    // base: the warp's first row and the tile's first column; ld: bytes between rows;
    // rows: how many of the 32 exist
    __device__ __forceinline__ void tile(uint8_t *base, size_t ld, int rows, int lane) {
        row_ok = 0;
        uint8_t *d = base + static_cast<size_t>(lane / kPieces) * ld + col * kElem;
#pragma unroll
        for (int i = 0; i < kPieces; ++i) {
            dst[i] = d;
            d += kRowsAt * ld;
            if (lane / kPieces + i * kRowsAt < rows) row_ok |= 1u << i;
        }
    }

    // v: 32 columns of this lane's row, from column `c` of the tile's first; `cols` of
    // them exist (a multiple of 8)
    __device__ __forceinline__ void put(int c, const float *v, int cols, bool add) const {
#pragma unroll
        for (int i = 0; i < kPieces; ++i) {
            uint4 x;
            if constexpr (kF32)
                x = make_uint4(__float_as_uint(v[4 * i]), __float_as_uint(v[4 * i + 1]), __float_as_uint(v[4 * i + 2]),
                               __float_as_uint(v[4 * i + 3]));
            else
                x = make_uint4(pack_bf16x2(v[8 * i], v[8 * i + 1]), pack_bf16x2(v[8 * i + 2], v[8 * i + 3]),
                               pack_bf16x2(v[8 * i + 4], v[8 * i + 5]), pack_bf16x2(v[8 * i + 6], v[8 * i + 7]));
            asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(in[i]), "r"(x.x), "r"(x.y), "r"(x.z), "r"(x.w)
                         : "memory");
        }
        __syncwarp();
        uint4 x[kPieces];
#pragma unroll
        for (int i = 0; i < kPieces; ++i)
            asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(x[i].x), "=r"(x[i].y), "=r"(x[i].z), "=r"(x[i].w)
                         : "r"(out[i])
                         : "memory");
        if (col < cols) {
#pragma unroll
            for (int i = 0; i < kPieces; ++i) {
                if ((row_ok >> i) & 1u) {
                    uint4 *o = reinterpret_cast<uint4 *>(dst[i] + c * kElem);
                    if (kF32 && add) {
                        const float4 y = *reinterpret_cast<const float4 *>(o);
                        x[i].x = __float_as_uint(__uint_as_float(x[i].x) + y.x);
                        x[i].y = __float_as_uint(__uint_as_float(x[i].y) + y.y);
                        x[i].z = __float_as_uint(__uint_as_float(x[i].z) + y.z);
                        x[i].w = __float_as_uint(__uint_as_float(x[i].w) + y.w);
                    }
                    if constexpr (kF32) __stcs(o, x[i]);        // large, and not read soon: 118 -> 114 us for 64 experts
                    else *o = x[i];
                }
            }
        }
        __syncwarp();
    }
};

// kRows: rows of a CTA's tile (32 or 128).
template <int kDir, int kBN, int kStages, int kCtaGroup, bool kF32, int kRows, bool kTwoLevel>
__global__ void __launch_bounds__(ragged_threads(kTwoLevel), 1)
ragged_gemm_kernel(const __grid_constant__ RaggedMaps<kDir> maps, const RaggedParams p) {
    using L = RaggedSmem<kDir, kBN, kStages, kCtaGroup, kF32, kRows, kTwoLevel>;
    using Tile = RaggedTile<kDir, kBN, kCtaGroup, kRows>;
    static_assert(!kF32 || kDir == kTN, "FP32 output: weight gradient");
    static_assert(kTwoLevel || (kDir == kTN && !kF32), "one-level sums: short BF16 weight gradients");
    static_assert(kRows == kTileX || (kRows == 32 && kDir != kTN && kCtaGroup == 1), "thin tiles: one CTA, K-major A");
    constexpr bool kSwap = L::kSwap;
    // the weight descriptor of a tile of 64 runs on over as many rows that follow
    static_assert(!kSwap || kTileX * 128 - L::kBBytes <= L::kUsed - L::kBarOffset, "reads stay inside shared memory");
    constexpr bool kPair = kCtaGroup == 2;
    constexpr bool kAMn = kDir == kTN, kBMn = kDir != kNT;
    constexpr int kAccBufs = L::kAccBufs;
    constexpr int kEpiWarp0 = 4;
    constexpr int kHalf = kBN / 2;                 // columns per epilogue warp
    constexpr bool kRebalance = kTwoLevel && !kSwap && kHalf >= 128;   // see kRegsLaunch
    constexpr int kSegBlocks = kF32 ? 8 : 16;      // K-blocks per accumulator segment of two-level sums
    static_assert(kSegBlocks % L::kSub == 0, "a segment is whole stages");

    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    const uint32_t s_base = ptx::smem_u32(smem);
    const uint32_t bar_base = s_base + L::kBarOffset;
    auto full_bar = [&](int s) { return bar_base + 8u * s; };
    auto empty_bar = [&](int s) { return bar_base + 8u * (kStages + s); };
    auto tfull_bar = [&](int b) { return bar_base + 8u * (2 * kStages + b); };
    auto tempty_bar = [&](int b) { return bar_base + 8u * (2 * kStages + kAccBufs + b); };
    const uint32_t mma_done_bar = bar_base + 8u * (2 * kStages + 2 * kAccBufs);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + L::kMiscOffset);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + L::kMiscOffset + 4);
    int *offs = reinterpret_cast<int *>(smem + L::kOffsOffset);
    int *prefix = reinterpret_cast<int *>(smem + L::kPrefixOffset);

    const int warp = threadIdx.x / 32;
    const int lane = threadIdx.x % 32;
    const BoundedWait wait{abort_flag, p.status, p.timeout_cycles};
    const int pair_rank = kPair ? static_cast<int>(ptx::cluster_rank() & 1u) : 0;
    const bool mma_cta = pair_rank == 0;
    auto leader_addr = [&](uint32_t local) { return kPair ? ptx::map_cluster(local, 0) : local; };

    if (threadIdx.x == 0) {
        ptx::prefetch_tmap(&maps.a);
        ptx::prefetch_tmap(&maps.b);
        for (int i = 0; i < kStages; ++i) {
            ptx::mbar_init(full_bar(i), 1);
            ptx::mbar_init(empty_bar(i), 1);
        }
        for (int b = 0; b < kAccBufs; ++b) {
            ptx::mbar_init(tfull_bar(b), 1);
            ptx::mbar_init(tempty_bar(b), 8 * kCtaGroup);   // one arrival per epilogue warp of the pair
        }
        ptx::mbar_init(mma_done_bar, 1);
        *abort_flag = 0;
        ptx::fence_mbar_init();
    }
    if constexpr (kDir == kTN) {
        if (warp == 2 && lane < kTailMaps) {
            ptx::prefetch_tmap(&maps.a_tail[lane]);
            ptx::prefetch_tmap(&maps.b_tail[lane]);
        }
    }
    // The launch may overlap the end of the kernel before it in the stream: from here on
    // that kernel is done and its writes are visible.
    pdl::grid_dependency_wait();
    if (warp == kEpiWarp0) {
        // offsets as the tiles use them: clamped to [0, T] and made non-decreasing.  Four
        // of them a lane, so that their loads are in flight together.
        int run = 0;
        for (int base = 0; base <= p.G; base += 128) {
            int raw[4], v[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int i = base + 4 * lane + j;
                raw[j] = i <= p.G ? p.offsets[i] : 0;
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                v[j] = min(max(raw[j], 0), p.T);
                if (j) v[j] = max(v[j], v[j - 1]);
            }
            int incl = v[3];
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int u = __shfl_up_sync(0xffffffffu, incl, o);
                if (lane >= o) incl = max(incl, u);
            }
            int before = __shfl_up_sync(0xffffffffu, incl, 1);
            before = max(run, lane ? before : 0);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int i = base + 4 * lane + j;
                v[j] = max(v[j], before);
                if (i <= p.G) {
                    offs[i] = v[j];
                    if (v[j] != raw[j]) record_status(p.status, kStatusInvalid, kSiteBadOffsets);
                }
            }
            run = max(run, __shfl_sync(0xffffffffu, incl, 31));
        }
        __syncwarp();
        // exclusive prefix of tiles per expert
        const int nb = (p.N + kBN - 1) / kBN;
        int carry = 0;
        for (int base = 0; base < p.G; base += 32) {
            const int g = base + lane;
            const int tiles = g < p.G ? Tile::row_blocks(p, offs, g) * nb : 0;
            int incl = tiles;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int u = __shfl_up_sync(0xffffffffu, incl, o);
                if (lane >= o) incl += u;
            }
            if (g < p.G) prefix[g] = carry + incl - tiles;
            carry += __shfl_sync(0xffffffffu, incl, 31);
        }
        if (lane == 0) prefix[p.G] = carry;
    }
    if (warp == 1) {
        if constexpr (kPair) {
            ptx::tmem_alloc_pair(ptx::smem_u32(tmem_slot), L::kTmemCols);
            ptx::tmem_relinquish_pair();
        } else {
            ptx::tmem_alloc(ptx::smem_u32(tmem_slot), L::kTmemCols);
            ptx::tmem_relinquish();
        }
    }
    ptx::tc_fence_before();
    __syncthreads();
    if constexpr (kPair) ptx::cluster_sync_all();   // the peer's barriers exist before any remote use
    ptx::tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;
    if (p.signal_early && threadIdx.x == 0) pdl::grid_launch_dependents();

    const int num_tiles = prefix[p.G];
    const int t_first = static_cast<int>(blockIdx.x) / kCtaGroup;
    const int t_step = static_cast<int>(gridDim.x) / kCtaGroup;

    if (warp < kEpiWarp0) {
        if constexpr (kRebalance) ptx::regs_dec<kRegsIssue>();
        if (warp == 0) {
            // ======================================================== producer
            if (ptx::elect_one()) {
                int stage = 0;
                uint32_t phase = 0;
                long long issued = 0;
                bool ok = (p.debug_flags & kDebugProducerIdle) == 0;
                Tile tl;
                for (int t = t_first; ok && t < num_tiles; t += t_step) {
                    tl.decode(t, p, offs, prefix);
                    // kNT, kNN: rows of A that this CTA loads, in boxes of 32 (single CTAs) or 128
                    const int a_boxes = (kDir != kTN && !kPair) ? (min(tl.row_end - tl.row0, kRows) + 31) / 32 : 0;
                    const uint32_t bytes = (kDir != kTN && !kPair) ? L::kSub * (a_boxes * 4096u + L::kBBytes)
                                                                   : static_cast<uint32_t>(L::kStageBytes);
                    const int nb0 = tl.n0 + pair_rank * L::kBCols;
                    for (int kb = 0; kb < tl.num_kb; kb += L::kSub) {
                        if (!wait(empty_bar(stage), phase ^ 1u, kSiteProducerEmpty)) { ok = false; break; }
                        const uint32_t sa = s_base + stage * L::kStageBytes;
                        const uint32_t sb = sa + L::kABytes;
                        const int k0 = kb * kRaggedBlockK;
                        // an expert's last tokens, where they end inside a group of 16
                        const bool ragged = kDir == kTN && kb == tl.num_kb - 1 && (tl.tail & 15) != 0;
                        const uint32_t expect = ragged ? (tl.tail + 15) / 16 * 16 * ((2 + L::kBCols / 64) * 128u) : bytes;
                        const uint32_t bar = leader_addr(full_bar(stage));
                        if (mma_cta) ptx::mbar_arrive_expect_tx(full_bar(stage), kCtaGroup * expect);
                        auto load = [&](uint32_t dst, const CUtensorMap *m, int c0, int c1, int c2) {
                            if constexpr (kPair) ptx::tma_load_3d_pair(dst, m, bar, c0, c1, c2);
                            else ptx::tma_load_3d(dst, m, bar, c0, c1, c2);
                        };
                        if constexpr (kDir == kTN) {
                            // rows of all boxes from `row` on, the tokens from `tok` on
                            auto load_rows = [&](const CUtensorMap *a, const CUtensorMap *b, int row, int tok) {
                                for (int i = 0; i < 2; ++i)
                                    load(sa + i * 8192u + row * 128u, a, tl.row0 + pair_rank * kTileX + 64 * i, tok, 0);
                                for (int i = 0; i < L::kBCols / 64; ++i)
                                    load(sb + i * 8192u + row * 128u, b, nb0 + 64 * i, tok, 0);
                            };
                            const int tok = tl.tok0 + k0;
                            if (!ragged) {
                                load_rows(&maps.a, &maps.b, 0, tok);
                            } else {
                                int row = 0;
#pragma unroll
                                for (int i = 0; i < kTailMaps; ++i)
                                    for (; row + tail_rows(i) <= tl.tail; row += tail_rows(i))
                                        load_rows(&maps.a_tail[i], &maps.b_tail[i], row, tok + row);
                                const int end = (tl.tail + 15) / 16 * 16;
#pragma unroll
                                for (int i = 1; i < kTailMaps; ++i)                  // zeros: behind the last token
                                    for (; row + tail_rows(i) <= end; row += tail_rows(i))
                                        load_rows(&maps.a_tail[i], &maps.b_tail[i], row, p.T);
                            }
                        } else {
#pragma unroll
                            for (int s = 0; s < L::kSub; ++s) {          // (past K: zeros)
                                const uint32_t a = sa + s * L::kSubBytes, b = a + L::kABytes;
                                const int k = k0 + s * kRaggedBlockK;
                                if constexpr (kPair) {
                                    load(a, &maps.a, k, tl.row0 + pair_rank * kTileX, 0);
                                } else {
                                    for (int i = 0; i < a_boxes; ++i)
                                        load(a + i * 4096u, &maps.a, k, tl.row0 + 32 * i, 0);
                                }
                                if constexpr (kDir == kNT) {
                                    load(b, &maps.b, k, nb0, tl.g);
                                } else {
                                    for (int i = 0; i < L::kBCols / 64; ++i)
                                        load(b + i * 8192u, &maps.b, nb0 + 64 * i, k, tl.g);
                                }
                            }
                        }
                        ++issued;
                        if (++stage == kStages) { stage = 0; phase ^= 1u; }
                    }
                }
                // never leave with TMA writes into shared memory in flight.  A pair's
                // second CTA cannot see its other bytes land; for it the final
                // cluster barrier, reached after the MMA CTA consumed every stage (or
                // ran out of time waiting for it), covers them.
                auto drain = [&](uint32_t bar, uint32_t par) {
                    const long long start = clock64();
                    while (!ptx::mbar_try_wait(bar, par)) {
                        if (clock64() - start > p.timeout_cycles) {
                            record_status(p.status, kStatusTimeout, kSiteTeardownLoads);
                            break;
                        }
                    }
                };
                const long long first = !mma_cta ? issued : (issued > kStages ? issued - kStages : 0);
                for (long long i = first; i < issued; ++i)
                    drain(full_bar(static_cast<int>(i % kStages)), static_cast<uint32_t>((i / kStages) & 1));
            }
            __syncwarp();
        } else if (warp == 1) {
            // ======================================================== MMA issuer
            if (mma_cta && ptx::elect_one()) {
                int stage = 0, buf = 0;
                uint32_t phase = 0, tphase = 0;
                bool ok = true;
                constexpr uint32_t kStepA = kAMn ? 2048 >> 4 : 32 >> 4;   // 16 reduced indices
                constexpr uint32_t kStepB = kBMn ? 2048 >> 4 : 32 >> 4;
                Tile tl;
                for (int t = t_first; ok && t < num_tiles; t += t_step) {
                    tl.decode(t, p, offs, prefix);
                    const int columns = (min(tl.row_end - tl.row0, kRows) + 15) / 16 * 16;
                    const uint32_t idesc = kSwap ? ragged_idesc(kTileX, columns, kBMn, kAMn)
                                                 : ragged_idesc(kTileX * kCtaGroup, kBN, kAMn, kBMn);
                    // one accumulator for the tile (nothing in it for an expert without tokens), or
                    // one for each segment
                    const int seg = kTwoLevel ? kSegBlocks : max(tl.num_kb, 1);
                    for (int kb0 = 0; ok && kb0 < max(tl.num_kb, 1); kb0 += seg) {
                        if (!wait(tempty_bar(buf), tphase ^ 1u, kSiteMmaTmemEmpty)) { ok = false; break; }
                        ptx::tc_fence_after();
                        const uint32_t dtm = tmem_base + static_cast<uint32_t>(buf * L::kAccCols);
                        const int kb1 = min(kb0 + seg, tl.num_kb);
                        for (int kb = kb0; kb < kb1; kb += L::kSub) {
                            if (!wait(full_bar(stage), phase, kSiteMmaFull)) { ok = false; break; }
                            const bool last = kDir == kTN && kb == tl.num_kb - 1;
                            ptx::tc_fence_after();
                            const int steps = last ? (tl.tail + 15) / 16 : kRaggedBlockK / 16;
#pragma unroll
                            for (int s = 0; s < L::kSub; ++s) {
                                const uint32_t sa = s_base + stage * L::kStageBytes + s * L::kSubBytes;
                                const uint64_t da = kAMn ? sw128_mn_desc(sa) : sw128_desc(sa);
                                const uint64_t db = kBMn ? sw128_mn_desc(sa + L::kABytes) : sw128_desc(sa + L::kABytes);
#pragma unroll
                                for (int k = 0; k < kRaggedBlockK / 16; ++k) {
                                    if (k < steps) {
                                        const uint32_t acc = (kb > kb0 || s > 0 || k > 0) ? 1u : 0u;
                                        if constexpr (kPair) ptx::mma_f16_pair(dtm, da + kStepA * k, db + kStepB * k, idesc, acc);
                                        else if constexpr (kSwap) ptx::mma_f16(dtm, db + kStepB * k, da + kStepA * k, idesc, acc);
                                        else ptx::mma_f16(dtm, da + kStepA * k, db + kStepB * k, idesc, acc);
                                    }
                                }
                            }
                            if constexpr (kPair) ptx::mma_commit_pair(empty_bar(stage), 0x3);
                            else ptx::mma_commit(empty_bar(stage));
                            if (++stage == kStages) { stage = 0; phase ^= 1u; }
                        }
                        if (!ok) break;
                        if constexpr (kPair) ptx::mma_commit_pair(tfull_bar(buf), 0x3);
                        else ptx::mma_commit(tfull_bar(buf));
                        if (++buf == kAccBufs) { buf = 0; tphase ^= 1u; }
                    }
                }
                // the commit is issued even when nothing ran, so every wait on it is uniform
                if constexpr (kPair) ptx::mma_commit_pair(mma_done_bar, 0x3);
                else ptx::mma_commit(mma_done_bar);
            }
            __syncwarp();
        }
    } else {
        // ============================================================ epilogue
        if constexpr (kRebalance) ptx::regs_inc<kRegsPromo>();
        const int quarter = warp & 3;
        const int half = ((warp - kEpiWarp0) >> 2) & 1;
        const int group = (warp - kEpiWarp0) >> 3;          // of the accumulators' rotation (FP32: one group for both)
        const int wrow = pair_rank * kTileX + quarter * 32;  // the warp's first row in a tile
        BoxWriter<kF32> writer(s_base + L::kOutOffset + (warp - kEpiWarp0) * L::kBoxBytes, lane);
        constexpr int kElem = kF32 ? 4 : 2;
        const bool add = kDir == kTN && p.accumulate;
        int buf = group;
        uint32_t tphase = 0;
        bool ok = true;
        auto release = [&]() {
            // the accumulator is free for the MMA warp (on the MMA CTA's barrier)
            ptx::tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                if (kPair && !mma_cta) ptx::mbar_arrive_remote(leader_addr(tempty_bar(buf)));
                else ptx::mbar_arrive(tempty_bar(buf));
            }
            if (kTwoLevel) buf ^= 1;
            if (!kTwoLevel || buf == 0) tphase ^= 1u;
        };
        Tile tl;
        const int e_step = kTwoLevel ? t_step : 2 * t_step;
        for (int t = t_first + group * t_step; ok && t < num_tiles; t += e_step) {
            tl.decode(t, p, offs, prefix);
            if constexpr (kSwap) {
                // lanes are weights, columns tokens: a warp turns 32 weights by 16 tokens round
                const int first = half * (kRows / 2);                  // of the warp's tokens
                const int tokens = min(tl.row_end - tl.row0 - first, kRows / 2);
                const int n = tl.n0 + quarter * 32;
                const bool mine = quarter * 32 < kBN && n < p.N;
                float acc[kRows / 2];
#pragma unroll
                for (int j = 0; j < kRows / 2; ++j) acc[j] = 0.f;
                for (int kb0 = 0; kb0 < tl.num_kb; kb0 += kSegBlocks) {
                    if (!wait(tfull_bar(buf), tphase, kSitePromoFull)) { ok = false; break; }
                    ptx::tc_fence_after();
                    if (mine) {
#pragma unroll
                        for (int c = 0; c < kRows / 2; c += 16) {
                            if (c < tokens) {
                                float v[16];
                                ptx::tmem_ld16(tmem_base + (static_cast<uint32_t>(quarter * 32) << 16) +
                                               static_cast<uint32_t>(buf * L::kAccCols + first + c), v);
                                ptx::tmem_wait_ld();
#pragma unroll
                                for (int j = 0; j < 16; ++j) acc[c + j] += v[j];
                            }
                        }
                    }
                    release();
                }
                if (!ok) break;
                if (mine) {
                    uint8_t *box = smem + L::kOutOffset + (warp - kEpiWarp0) * L::kBoxBytes;
                    const int piece = lane % 4 * 8;
                    uint8_t *dst = static_cast<uint8_t *>(p.d) +
                                   (static_cast<size_t>(tl.row0 + first + lane / 4) * p.N + n + piece) * 2;
                    const size_t step = static_cast<size_t>(p.N) * 16;                 // 8 tokens
#pragma unroll
                    for (int c = 0; c < kRows / 2; c += 16) {
                        if (c >= tokens) break;
#pragma unroll
                        for (int j = 0; j < 16; ++j)
                            *reinterpret_cast<__nv_bfloat16 *>(box + j * 64 + lane * 2) = __float2bfloat16_rn(acc[c + j]);
                        __syncwarp();
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const uint4 x = *reinterpret_cast<const uint4 *>(box + (i * 8 + lane / 4) * 64 + piece * 2);
                            if (c + i * 8 + lane / 4 < tokens && n + piece < p.N) *reinterpret_cast<uint4 *>(dst) = x;
                            dst += step;
                        }
                        __syncwarp();
                    }
                }
                continue;
            }
            const int rows = min(tl.row_end, tl.row0 + pair_rank * kTileX + kRows) - (tl.row0 + wrow);   // of the warp's 32
            const int c0 = tl.n0 + half * kHalf;
            const size_t row0 = (kDir == kTN ? static_cast<size_t>(tl.g) * p.M : 0) + tl.row0 + wrow;
            writer.tile(static_cast<uint8_t *>(p.d) + (row0 * p.N + c0) * kElem, static_cast<size_t>(p.N) * kElem, rows, lane);
            auto put = [&](int c, const float *v) {      // columns c0 + c .. + 31 of this lane's row
                if (c0 + c >= p.N || rows <= 0) return;
                if (kDir == kTN && !kF32 && add) {       // BF16 is added in FP32: before it is rounded
                    if (lane < rows)
#pragma unroll
                        for (int j = 0; j < 32; j += 8)
                            if (c0 + c + j < p.N)
                                add8(static_cast<__nv_bfloat16 *>(p.d) + (row0 + lane) * p.N + c0 + c + j, v + j);
                    return;
                }
                writer.put(c, v, p.N - c0 - c, add);
            };
            if constexpr (kTwoLevel) {
                float acc[kHalf];
#pragma unroll
                for (int j = 0; j < kHalf; ++j) acc[j] = 0.f;
                for (int kb0 = 0; kb0 < max(tl.num_kb, 1); kb0 += kSegBlocks) {
                    if (!wait(tfull_bar(buf), tphase, kSitePromoFull)) { ok = false; break; }
                    ptx::tc_fence_after();
                    const uint32_t taddr = tmem_base + (static_cast<uint32_t>(quarter * 32) << 16) +
                                           static_cast<uint32_t>(buf * kBN + half * kHalf);
                    if (tl.num_kb > 0) {
#pragma unroll
                        for (int c = 0; c < kHalf; c += 16) {
                            float v[16];
                            ptx::tmem_ld16(taddr + c, v);
                            ptx::tmem_wait_ld();
#pragma unroll
                            for (int j = 0; j < 16; ++j) acc[c + j] += v[j];
                        }
                    }
                    release();
                }
                if (!ok) break;
                if (tl.num_kb > 0 || !add) {
#pragma unroll
                    for (int c = 0; c < kHalf; c += 32) put(c, acc + c);
                }
            } else {
                if (!wait(tfull_bar(buf), tphase, kSitePromoFull)) { ok = false; break; }
                ptx::tc_fence_after();
                const uint32_t taddr = tmem_base + (static_cast<uint32_t>(quarter * 32) << 16) +
                                       static_cast<uint32_t>(buf * kBN + half * kHalf);
                if (tl.num_kb > 0 || !add) {
#pragma unroll
                    for (int c = 0; c < kHalf; c += 32) {
                        float v[32];
                        if (kDir != kTN || tl.num_kb > 0) {
                            ptx::tmem_ld32p(taddr + c, v);
                            ptx::tmem_wait_ld();
                        } else {                           // an expert without tokens
#pragma unroll
                            for (int j = 0; j < 32; ++j) v[j] = 0.f;
                        }
                        put(c, v);
                    }
                }
                release();
            }
        }
    }

    // ---------------------------------------------------------------- teardown
    ptx::tc_fence_before();
    __syncthreads();
    // The next grid's blocks may be placed (see RaggedParams::signal_early).
    if (threadIdx.x == 0) pdl::grid_launch_dependents();
    // (After the barrier: a pair's second CTA issues no MMAs, and would wait here from its
    // start, so that the limit bounded the call.)
    if (warp == 1 && ptx::elect_one()) {
        const long long start = clock64();
        while (!ptx::mbar_try_wait(mma_done_bar, 0)) {
            if (clock64() - start > p.timeout_cycles) {
                record_status(p.status, kStatusTimeout, kSiteTeardownMma);
                break;
            }
        }
    }
    __syncwarp();
    if constexpr (kPair) ptx::cluster_sync_all();   // no CTA leaves while its peer may touch its smem
    if (warp == 1) {
        ptx::tc_fence_after();
        if constexpr (kPair) ptx::tmem_dealloc_pair(tmem_base, L::kTmemCols);
        else ptx::tmem_dealloc(tmem_base, L::kTmemCols);
    }
}

}  // namespace dg
