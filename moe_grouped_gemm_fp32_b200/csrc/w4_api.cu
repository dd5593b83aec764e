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

dg_status_t check_w4(const void *x, const void *w, const void *s, const void *z, const void *d, int M, int N, int K,
                     int G, int group_size) {
    if (!w || !s || (M > 0 && (!x || !d))) return DG_ERR_INVALID_VALUE;
    if (M < 0 || N <= 0 || K <= 0 || G <= 0) return DG_ERR_INVALID_VALUE;
    if (group_size != 32 && group_size != 64 && group_size != 128) return DG_ERR_UNSUPPORTED_SHAPE;
    if (K % group_size != 0 || N % 8 != 0 || G > 1024) return DG_ERR_UNSUPPORTED_SHAPE;
    if (K > (1 << 30) || (N + dg::kW4Rows - 1) / dg::kW4Rows > 65535) return DG_ERR_UNSUPPORTED_SHAPE;   // grid.y
    if (!aligned16(x) || !aligned16(w) || !aligned16(s) || !aligned16(z) || !aligned16(d)) return DG_ERR_MISALIGNED;
    return DG_SUCCESS;
}

template <int kGs, int kNT>
dg_status_t launch_w4(const dg::W4Params &p, int split, cudaStream_t stream) {
    using L = dg::W4Smem<kGs, kNT>;
    auto kernel = dg::w4_gemv_kernel<kGs, kNT>;
    // one-time per-device set-up (idempotent; the atomic flag keeps racing first calls defined)
    static std::atomic<bool> configured[kMaxDevices] = {};
    int dev = 0;
    cudaGetDevice(&dev);
    if (!configured[dev].load(std::memory_order_acquire)) {
        cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kAlloc);
        if (e != cudaSuccess) return cuda_fail(e, "cudaFuncSetAttribute(w4 smem)");
        configured[dev].store(true, std::memory_order_release);
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(split, (p.N + dg::kW4Rows - 1) / dg::kW4Rows, p.offsets ? p.G : 1);
    cfg.blockDim = dim3(dg::kW4Threads, 1, 1);
    cfg.dynamicSmemBytes = L::kAlloc;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = split;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = split > 1 ? 1 : 0;
    if (verbose())
        std::fprintf(stderr, "[dg] w4_gemv group=%d tokens=%d split=%d grid=%ux%ux%u smem=%d\n", kGs, 8 * kNT, split,
                     cfg.gridDim.x, cfg.gridDim.y, cfg.gridDim.z, L::kAlloc);
    cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, p);
    return e == cudaSuccess ? DG_SUCCESS : cuda_fail(e, "w4_gemv_kernel launch");
}

template <int kGs>
dg_status_t dispatch(const dg::W4Params &p, int tokens, int split, cudaStream_t stream) {
    if (tokens <= 8) return launch_w4<kGs, 1>(p, split, stream);
    if (tokens <= 16) return launch_w4<kGs, 2>(p, split, stream);
    return launch_w4<kGs, 4>(p, split, stream);
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
    const int used = offsets ? (M < G ? M : G) : 1;
    const int tokens = M <= 8 ? M : offsets ? 2 * ((M + used - 1) / used) : M;
    // K split: the least that gives every SM two CTAs
    const long long blocks = static_cast<long long>((N + dg::kW4Rows - 1) / dg::kW4Rows) * used;
    const int stages = (K + dg::kW4StageK - 1) / dg::kW4StageK;
    int split = 1;
    while (split < 8 && blocks * split < 2 * info->num_sms && 2 * split <= stages) split *= 2;
    if (group_size == 32) return dispatch<32>(p, tokens, split, stream);
    if (group_size == 64) return dispatch<64>(p, tokens, split, stream);
    return dispatch<128>(p, tokens, split, stream);
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
