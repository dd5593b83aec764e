// w4_api.cu -- host side of the 4-bit weight products declared in include/dg.h
// (dg_w4_gemv_nt, dg_m_grouped_w4_gemv_nt_ragged): argument validation, choice
// of token tile and K split, launch.  Nothing here synchronises the host or
// allocates memory.
#include <cuda_runtime.h>

#include <atomic>
#include <cstdio>

#include "dg.h"
#include "api_common.h"
#include "w4_kernel.cuh"

namespace {
using namespace dg_host;

constexpr int kMaxRows = 2000000;   // their runs of 32, and one more for each expert, are grid.z (65535 at most)

dg_status_t check_w4(const void *x, const void *w, const void *s, const void *z, const void *d, int M, int N, int K,
                     int G, int group_size) {
    if (!w || !s || (M > 0 && (!x || !d))) return DG_ERR_INVALID_VALUE;
    if (M < 0 || N <= 0 || K <= 0 || G <= 0) return DG_ERR_INVALID_VALUE;
    if (group_size != 32 && group_size != 64 && group_size != 128) return DG_ERR_UNSUPPORTED_SHAPE;
    if (K % group_size != 0 || N % 8 != 0 || G > 1024) return DG_ERR_UNSUPPORTED_SHAPE;
    if (M > kMaxRows) return DG_ERR_UNSUPPORTED_SHAPE;
    if (K > (1 << 30) || (N + dg::kW4Rows - 1) / dg::kW4Rows > 65535) return DG_ERR_UNSUPPORTED_SHAPE;   // grid.y
    if (!aligned16(x) || !aligned16(w) || !aligned16(s) || !aligned16(z) || !aligned16(d)) return DG_ERR_MISALIGNED;
    return DG_SUCCESS;
}

template <int kGs, int kNT, bool kZeros>
dg_status_t launch_w4(dg::W4Params p, int split, int runs, cudaStream_t stream) {
    using L = dg::W4Smem<kGs>;
    auto kernel = dg::w4_gemv_kernel<kGs, kNT, kZeros>;
    const int blocks = (p.K + dg::kW4BlockK - 1) / dg::kW4BlockK;
    const int per_cta = (blocks + split - 1) / split;
    p.tok_cap = p.M < 8 * kNT ? p.M : 8 * kNT;
    p.bufs = per_cta > dg::kW4Chunk ? 2 : 1;
    const int smem = L::bytes(p.tok_cap, p.bufs, kZeros);
    // one-time per-device set-up (idempotent; the atomic flag keeps racing first calls defined)
    static std::atomic<bool> configured[kMaxDevices] = {};
    int dev = 0;
    cudaGetDevice(&dev);
    if (!configured[dev].load(std::memory_order_acquire)) {
        const int most = L::bytes(8 * kNT, 2, kZeros);
        cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
        if (e != cudaSuccess) return cuda_fail(e, "cudaFuncSetAttribute(w4 smem)");
        configured[dev].store(true, std::memory_order_release);
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(split, (p.N + dg::kW4Rows - 1) / dg::kW4Rows, runs);
    cfg.blockDim = dim3(dg::kW4Threads, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;      // see pdl.cuh
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = split;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = split > 1 ? 2 : 1;
    if (verbose())
        std::fprintf(stderr, "[dg] w4_gemv group=%d tokens=%d split=%d grid=%ux%ux%u bufs=%d smem=%d\n", kGs, 8 * kNT,
                     split, cfg.gridDim.x, cfg.gridDim.y, cfg.gridDim.z, p.bufs, smem);
    cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, p);
    return e == cudaSuccess ? DG_SUCCESS : cuda_fail(e, "w4_gemv_kernel launch");
}

// CTAs that share a row block along K: the count with the least cost of the fullest SM,
// in times that an SM with enough CTAs takes for a block of K.  It works through the blocks
// of all of its CTAs; a wave of resident ones takes at least the latency of a CTA's blocks,
// 2.5 such times each (2 with 16 or 32 tokens); and each CTA costs 3 to start and hand over.
// Measured for 4 to 1000 row blocks, 4 to 128 blocks of K, 1 to 30 tokens (400 shapes, splits
// of 1, 2, 4, 8): the choice takes 0.5 % more than the best one on average, 10 % at
// worst.  512 row blocks of 55 K blocks, one token: 56.1 us whole, 50.1 halved.
int k_split(long long row_blocks, int k_blocks, int tokens, int num_sms) {
    const int resident = tokens <= 8 ? 5 : tokens <= 16 ? 4 : 3, latency = tokens <= 8 ? 5 : 4;    // in halves
    int best = 1;
    long long least = 0;
    for (int split = 1; split <= 8 && (split == 1 || k_blocks >= 2 * split); split *= 2) {
        const long long ctas = (row_blocks * split + num_sms - 1) / num_sms;
        const long long waves = (ctas + resident - 1) / resident, blocks = (k_blocks + split - 1) / split;
        const long long work = 2 * ctas * blocks, wait = waves * blocks * latency;
        const long long cost = (work > wait ? work : wait) + 6 * ctas;
        if (split == 1 || cost < least) {
            least = cost;
            best = split;
        }
    }
    return best;
}

// runs of `rows` rows that M rows of `experts` experts can make at most
int runs_of(int M, int experts, int rows) { return experts + (M - experts) / rows; }

// experts: those that can have rows (0: dense)
template <int kGs, bool kZeros>
dg_status_t dispatch_tokens(const dg::W4Params &p, int tokens, int experts, int split, cudaStream_t stream) {
    auto runs = [&](int rows) { return experts ? runs_of(p.M, experts, rows) : (p.M + rows - 1) / rows; };
    if (tokens <= 8) return launch_w4<kGs, 1, kZeros>(p, split, runs(8), stream);
    if (tokens <= 16) return launch_w4<kGs, 2, kZeros>(p, split, runs(16), stream);
    return launch_w4<kGs, 4, kZeros>(p, split, runs(32), stream);
}

template <int kGs>
dg_status_t dispatch(const dg::W4Params &p, int tokens, int experts, int split, cudaStream_t stream) {
    if (p.z) return dispatch_tokens<kGs, true>(p, tokens, experts, split, stream);
    return dispatch_tokens<kGs, false>(p, tokens, experts, split, stream);
}

dg_status_t w4_gemv(const void *x, const void *w, const void *s, const void *z, void *d, const int32_t *offsets, int M,
                    int N, int K, int G, int group_size, cudaStream_t stream) {
    dg_status_t st = check_w4(x, w, s, z, d, M, N, K, G, group_size);
    if (st != DG_SUCCESS) return st;
    const DeviceInfo *info = nullptr;
    if ((st = device_info(&info)) != DG_SUCCESS) return st;
    if (M == 0) return DG_SUCCESS;
    dg::W4Params p = {};
    p.x = static_cast<const __nv_bfloat16 *>(x);
    p.w = static_cast<const uint8_t *>(w);
    p.s = static_cast<const __nv_bfloat16 *>(s);
    p.z = static_cast<const uint8_t *>(z);
    p.d = static_cast<__nv_bfloat16 *>(d);
    p.offsets = offsets;
    p.status = info->status;
    p.M = M;
    p.N = N;
    p.K = K;
    p.G = G;
    // tokens a CTA takes at once: all (dense), or what an expert has on average and as much again
    const int experts = offsets ? (M < G ? M : G) : 0;
    const int tokens = M <= 8 || !experts ? M : 2 * ((M + experts - 1) / experts);
    const long long blocks = static_cast<long long>((N + dg::kW4Rows - 1) / dg::kW4Rows) * (experts ? experts : 1);
    const int split = k_split(blocks, (K + dg::kW4BlockK - 1) / dg::kW4BlockK, tokens, info->num_sms);
    if (group_size == 32) return dispatch<32>(p, tokens, experts, split, stream);
    if (group_size == 64) return dispatch<64>(p, tokens, experts, split, stream);
    return dispatch<128>(p, tokens, experts, split, stream);
}

}  // namespace

extern "C" {

dg_status_t dg_w4_gemv_nt(const void *x, const uint8_t *w, const void *scales, const uint8_t *zeros, void *d, int M,
                          int N, int K, int group_size, void *stream) {
    return w4_gemv(x, w, scales, zeros, d, nullptr, M, N, K, 1, group_size, static_cast<cudaStream_t>(stream));
}

dg_status_t dg_m_grouped_w4_gemv_nt_ragged(const void *x, const uint8_t *w, const void *scales, const uint8_t *zeros,
                                           void *d, const int32_t *m_offsets, int M_total, int N, int K, int G,
                                           int group_size, void *stream) {
    if (!m_offsets) return DG_ERR_INVALID_VALUE;
    return w4_gemv(x, w, scales, zeros, d, m_offsets, M_total, N, K, G, group_size, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
