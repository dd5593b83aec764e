// ragged_api.cu -- host side of the ragged grouped BF16 products declared in
// include/dg.h (dg_m_grouped_bf16_gemm_nt_ragged, dg_m_grouped_bf16_gemm_nn_ragged,
// dg_k_grouped_bf16_gemm_tn_ragged): argument validation, TMA descriptors, tile
// choice, launch.  Nothing here synchronises the host or allocates memory.
#include <cuda.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstdio>

#include "dg.h"
#include "api_common.h"
#include "ragged_kernel.cuh"

namespace {
using namespace dg_host;

constexpr long long kMaxInt = (1LL << 31) - 1;

// rows: the token buffer's; p, q: the two other sizes, both innermost somewhere
dg_status_t check_ragged(const void *a, const void *b, const void *d, const int32_t *offsets, int rows, int p, int q,
                         int G) {
    if (!b || !offsets || (rows > 0 && (!a || !d))) return DG_ERR_INVALID_VALUE;
    if (rows < 0 || p <= 0 || q <= 0 || G <= 0) return DG_ERR_INVALID_VALUE;
    if (p % 8 != 0 || q % 8 != 0) return DG_ERR_UNSUPPORTED_SHAPE;        // 16-byte rows
    if (G > dg::kMaxGroups || p > (1 << 30) || q > (1 << 30)) return DG_ERR_UNSUPPORTED_SHAPE;
    if (rows > kMaxInt - 1024) return DG_ERR_UNSUPPORTED_SHAPE;           // a tile's rows past the end stay 32-bit
    if (!aligned16(a) || !aligned16(b) || !aligned16(d)) return DG_ERR_MISALIGNED;
    return DG_SUCCESS;
}

template <int kDir, int kBN, int kStages, int kCtaGroup, bool kF32, int kRows = 128, bool kTwoLevel = true>
struct Launch {
    using L = dg::RaggedSmem<kDir, kBN, kStages, kCtaGroup, kF32, kRows, kTwoLevel>;

    static auto kernel() { return dg::ragged_gemm_kernel<kDir, kBN, kStages, kCtaGroup, kF32, kRows, kTwoLevel>; }

    static void config(cudaLaunchConfig_t &cfg, cudaLaunchAttribute *attr, int grid, cudaStream_t stream) {
        cfg = {};
        cfg.gridDim = dim3(grid, 1, 1);
        cfg.blockDim = dim3(dg::ragged_threads(kTwoLevel), 1, 1);
        cfg.dynamicSmemBytes = L::kAlloc;
        cfg.stream = stream;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;      // see pdl.cuh
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        if (kCtaGroup > 1) {
            attr[1].id = cudaLaunchAttributeClusterDimension;
            attr[1].val.clusterDim.x = kCtaGroup;
            attr[1].val.clusterDim.y = 1;
            attr[1].val.clusterDim.z = 1;
            cfg.numAttrs = 2;
        }
    }

    // One-time set-up per device; resident tiles (CTAs or CTA pairs) in *units.
    // Idempotent: the atomic keeps racing first calls defined.
    static dg_status_t setup(const DeviceInfo *info, int *units) {
        static std::atomic<int> cache[kMaxDevices] = {};
        int dev = 0;
        cudaGetDevice(&dev);
        if ((*units = cache[dev].load(std::memory_order_acquire)) > 0) return DG_SUCCESS;
        cudaError_t e = cudaFuncSetAttribute(kernel(), cudaFuncAttributeMaxDynamicSharedMemorySize, L::kAlloc);
        if (e != cudaSuccess) return cuda_fail(e, "cudaFuncSetAttribute(ragged smem)");
        if (kTwoLevel && kBN == 256) {
            // the register hand-over between warpgroups adds up only for this launch size
            cudaFuncAttributes fa;
            if ((e = cudaFuncGetAttributes(&fa, kernel())) != cudaSuccess) return cuda_fail(e, "cudaFuncGetAttributes");
            if (fa.numRegs != dg::kRegsLaunch) return cuda_fail(cudaErrorLaunchOutOfResources, "ragged kernel registers");
        }
        int n = info->num_sms;
        if (kCtaGroup > 1) {
            cudaLaunchConfig_t cfg;
            cudaLaunchAttribute attr[2];
            config(cfg, attr, kCtaGroup, nullptr);
            if ((e = cudaOccupancyMaxActiveClusters(&n, kernel(), &cfg)) != cudaSuccess)
                return cuda_fail(e, "cudaOccupancyMaxActiveClusters(ragged)");
            if (n <= 0) return cuda_fail(cudaErrorLaunchOutOfResources, "ragged CTA pairs");
        }
        *units = n;
        cache[dev].store(n, std::memory_order_release);
        return DG_SUCCESS;
    }

    // tiles: an upper bound of the tile count
    static dg_status_t run(const dg::RaggedMaps<kDir> &maps, dg::RaggedParams p, long long tiles,
                           const DeviceInfo *info, cudaStream_t stream) {
        int units = 0;
        dg_status_t st = setup(info, &units);
        if (st != DG_SUCCESS) return st;
        // The next launch is let in early by pairs with several tiles each: the low-numbered
        // blocks, which have a tile more, then come to the SMs that are done first (forward
        // calls in a row, 4096 x 7168, 4 experts: 2048 rows 139 us against 147, 8192 rows 399 and
        // 427, 32768 rows 1550 and 1600; a 4-bit call behind them takes as long either way).
        // Elsewhere blocks that come while some SMs are done fill the SMs unevenly: a 4-bit
        // call of 8 tokens, 16384 x 7168, behind a forward of one expert of 16 rows, 1024 x
        // 1024: 28.3 us for both with the early signal, 25.1 with the late one, 25.1 without; that
        // forward and its input gradient: 11.4, 11.6, 12.1; a weight gradient of 8 experts of
        // 100 tokens, 256 x 512, on pairs, and the 4-bit call: 30.7, 28.8, 28.0.
        p.signal_early = kCtaGroup == 2 && tiles >= 4LL * units;
        const int grid = kCtaGroup * static_cast<int>(tiles < units ? tiles : units);
        if (verbose())
            std::fprintf(stderr, "[dg] ragged dir=%d rows=%d bn=%d stages=%d ctas/mma=%d f32=%d levels=%d grid=%d smem=%d\n",
                         kDir, kRows, kBN, kStages, kCtaGroup, kF32 ? 1 : 0, kTwoLevel ? 2 : 1, grid, L::kAlloc);
        cudaLaunchConfig_t cfg;
        cudaLaunchAttribute attr[2];
        config(cfg, attr, grid, stream);
        cudaError_t e = cudaLaunchKernelEx(&cfg, kernel(), maps, p);
        return e == cudaSuccess ? DG_SUCCESS : cuda_fail(e, "ragged_gemm_kernel launch");
    }
};

long long ceil_div(long long a, long long b) { return (a + b - 1) / b; }

dg::RaggedParams ragged_params(void *d, const int32_t *offsets, int T, int M, int N, int K, int G, int accumulate,
                               const DeviceInfo *info) {
    dg::RaggedParams p = {};
    p.d = d;
    p.offsets = offsets;
    p.status = info->status;
    p.timeout_cycles = timeout_cycles();
    p.T = T;
    p.M = M;
    p.N = N;
    p.K = K;
    p.G = G;
    p.accumulate = accumulate;
    p.debug_flags = debug_flags();
    return p;
}

// Forward and input gradient: a [T, K], b [G, N, K] (kNT) or [G, K, N] (kNN).
template <int kDir>
dg_status_t m_grouped(const void *a, const void *b, void *d, const int32_t *offsets, int T, int N, int K, int G,
                      cudaStream_t stream) {
    dg_status_t st = check_ragged(a, b, d, offsets, T, N, K, G);
    if (st != DG_SUCCESS) return st;
    const int used = T < G ? T : G;              // experts that can have a row
    if ((ceil_div(T, 32) + used) * ceil_div(N, 64) > kMaxInt) return DG_ERR_UNSUPPORTED_SHAPE;
    const DeviceInfo *info = nullptr;
    if ((st = device_info(&info)) != DG_SUCCESS) return st;
    if (T == 0) return DG_SUCCESS;
    const dg::RaggedParams p = ragged_params(d, offsets, T, 0, N, K, G, 0, info);
    // 256-row CTA pairs where an expert has 128 rows or more on average and there are a
    // few of their tiles: 8 experts of 128 rows, 2048 x 4096: 34.0 us in pair tiles, 42.6 in
    // single ones; one expert of 512 rows, 1024 x 1024: 8 pair tiles 10.5 us, 64 single
    // ones 8.4.  Thin tiles of 32 rows where experts have 24 or fewer on average, so that
    // few need several (16 experts of 4096 x 7168, tiles of 128 rows against thin ones: 24
    // rows on average, skewed, 157 and 146 us, 48 rows 161 and 176), or where the thin ones
    // fill no more than the SMs once: a call of few tiles takes as long as one tile does
    // (one expert of 256 rows, 1024 x 8192, 128 thin tiles: 33 and 19.7; 192 rows, 4096 x
    // 4096, 384 of them: 19.5 and 28.3).  Tiles 64 wide where 128 would leave SMs without one
    // (one expert of 16 rows, 4096 x 7168: 18.0 us, 23.0 in the wider ones).
    const long long pair_tiles = ceil_div(T, 256) * ceil_div(N, 256);
    const bool pair = N > 128 && T / used >= 128 && 8 * pair_tiles >= info->num_sms;
    const bool thin = !pair && (T / used <= 24 || ceil_div(T, 32) * ceil_div(N, 64) <= info->num_sms);
    const int rows = pair ? 256 : thin ? 32 : 128;
    const long long filled = ceil_div(T, rows) > used ? ceil_div(T, rows) : used;     // row blocks, about
    const int bn = pair ? 256 : ceil_div(N, 128) * filled >= info->num_sms ? 128 : 64;
    dg::RaggedMaps<kDir> maps;
    if ((st = make_kmajor_map(&maps.a, a, 2, K, T, 1, pair ? 128 : 32)) != DG_SUCCESS) return st;
    st = kDir == dg::kNT ? make_kmajor_map(&maps.b, b, 2, K, N, G, pair ? bn / 2 : bn)
                         : make_kmajor_map(&maps.b, b, 2, N, K, G, dg::kRaggedBlockK);
    if (st != DG_SUCCESS) return st;
    const long long tiles = (ceil_div(T, rows) + used) * ceil_div(N, bn);
    if (pair) return Launch<kDir, 256, 5, 2, false>::run(maps, p, tiles, info, stream);
    if (thin && bn == 128) return Launch<kDir, 128, 9, 1, false, 32>::run(maps, p, tiles, info, stream);
    if (thin) return Launch<kDir, 64, 7, 1, false, 32>::run(maps, p, tiles, info, stream);
    if (bn == 128) return Launch<kDir, 128, 5, 1, false>::run(maps, p, tiles, info, stream);
    return Launch<kDir, 64, 7, 1, false>::run(maps, p, tiles, info, stream);
}

// Most tokens of a call whose BF16 weight gradient is summed in one level.  What the
// tensor core's accumulator then loses, 4.7e-5 of a sum of products of one sign, is 1/80
// of a BF16 result's half step, and two groups of epilogue warps can take turns: 64
// experts of 62 tokens, 1000 x 2112, 70.4 us and 77.5 in two levels; of 125, 84.1 and
// 89.9; 8 experts of 1024 tokens, 2048 x 4096, 107.5 and 109.0.
constexpr int kOneLevelTokens = 8192;

template <bool kF32, bool kTwoLevel>
dg_status_t k_grouped(const void *a, const void *b, const dg::RaggedParams &p, const DeviceInfo *info,
                      cudaStream_t stream) {
    dg::RaggedMaps<dg::kTN> maps;
    dg_status_t st = DG_SUCCESS;
    auto encode = [&](CUtensorMap *ma, CUtensorMap *mb, int tokens) {
        if (st == DG_SUCCESS) st = make_kmajor_map(ma, a, 2, p.M, p.T, 1, tokens);
        if (st == DG_SUCCESS) st = make_kmajor_map(mb, b, 2, p.N, p.T, 1, tokens);
    };
    encode(&maps.a, &maps.b, dg::kRaggedBlockK);
    for (int i = 0; i < dg::kTailMaps; ++i) encode(&maps.a_tail[i], &maps.b_tail[i], dg::tail_rows(i));
    if (st != DG_SUCCESS) return st;
    if (p.M > 128 && p.N > 128)
        return Launch<dg::kTN, 256, 5, 2, kF32, 128, kTwoLevel>::run(
            maps, p, p.G * ceil_div(p.M, 256) * ceil_div(p.N, 256), info, stream);
    return Launch<dg::kTN, 128, 5, 1, kF32, 128, kTwoLevel>::run(
        maps, p, p.G * ceil_div(p.M, 128) * ceil_div(p.N, 128), info, stream);
}

}  // namespace

extern "C" {

dg_status_t dg_m_grouped_bf16_gemm_nt_ragged(const void *a, const void *b, void *d, const int32_t *m_offsets,
                                             int M_total, int N, int K, int G, void *stream) {
    return m_grouped<dg::kNT>(a, b, d, m_offsets, M_total, N, K, G, static_cast<cudaStream_t>(stream));
}

dg_status_t dg_m_grouped_bf16_gemm_nn_ragged(const void *a, const void *b, void *d, const int32_t *m_offsets,
                                             int M_total, int N, int K, int G, void *stream) {
    return m_grouped<dg::kNN>(a, b, d, m_offsets, M_total, N, K, G, static_cast<cudaStream_t>(stream));
}

dg_status_t dg_k_grouped_bf16_gemm_tn_ragged(const void *a, const void *b, void *d, int d_is_fp32,
                                             const int32_t *k_offsets, int G, int M, int N, int K_total,
                                             int accumulate, void *stream) {
    if (!d) return DG_ERR_INVALID_VALUE;
    dg_status_t st = check_ragged(a, K_total > 0 ? b : d, d, k_offsets, K_total, M, N, G);
    if (st != DG_SUCCESS) return st;
    if (G * ceil_div(M, 128) * ceil_div(N, 128) > kMaxInt) return DG_ERR_UNSUPPORTED_SHAPE;
    const DeviceInfo *info = nullptr;
    if ((st = device_info(&info)) != DG_SUCCESS) return st;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (K_total == 0) {                           // no tokens: zeros, or nothing to add
        if (accumulate) return DG_SUCCESS;
        const size_t bytes = static_cast<size_t>(G) * M * N * (d_is_fp32 ? 4 : 2);
        cudaError_t e = cudaMemsetAsync(d, 0, bytes, s);
        return e == cudaSuccess ? DG_SUCCESS : cuda_fail(e, "cudaMemsetAsync");
    }
    const dg::RaggedParams p = ragged_params(d, k_offsets, K_total, M, N, 0, G, accumulate ? 1 : 0, info);
    if (d_is_fp32) return k_grouped<true, true>(a, b, p, info, s);
    if (K_total > kOneLevelTokens) return k_grouped<false, true>(a, b, p, info, s);
    return k_grouped<false, false>(a, b, p, info, s);
}

}  // extern "C"
