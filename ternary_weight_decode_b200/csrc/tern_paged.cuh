// tern_paged.cuh -- device view of a paged 8-bit KV cache and of a batch over
// it (tern_paged_cache, tern_paged_batch), shared by the append, read and
// attention kernels.
#pragma once

#include <cuda_fp8.h>
#include <stdint.h>

#include "tern_common.cuh"
#include "tern_internal.h"

namespace tern {

constexpr int kPD = 128;                 // head dimension
constexpr int kPB = TERN_KV_BLOCK;       // tokens that share a scale
constexpr int kMaxBatch = 4096;          // sequences of a batch

// Division of 0 <= n < 2^31 by a number fixed at the launch, by the method of
// Granlund and Montgomery (Division by Invariant Integers using Multiplication,
// 1994): multiply, add, shift (with l = ceil(log2 d): mul = floor(2^32 (2^l - d)
// / d) + 1).
struct FastDiv {
    uint32_t d, mul, shift;
    __device__ __forceinline__ int quot(int n) const {
        return static_cast<int>((__umulhi(static_cast<uint32_t>(n), mul) + static_cast<uint32_t>(n)) >> shift);
    }
};
inline FastDiv fast_div(int d) {
    FastDiv f;
    f.d = static_cast<uint32_t>(d);
    f.shift = 0;
    while ((1ull << f.shift) < f.d) ++f.shift;
    f.mul = static_cast<uint32_t>(((1ull << 32) * ((1ull << f.shift) - f.d)) / f.d + 1);
    return f;
}

struct PagedView {
    int kind, Hkv, page_size, bpp, n_pages;  // bpp: blocks of 16 tokens per page
    FastDiv by_bpp;
    uint8_t *kc, *vc;
    float *ks, *vs;
    int B, T, pages_ld;
    const int32_t *row_start, *ctx, *pages;
};

inline PagedView paged_view(const tern_paged_batch &B, const tern_paged_cache &C) {
    PagedView v;
    v.kind = C.kind;
    v.Hkv = C.Hkv;
    v.page_size = C.page_size;
    v.bpp = C.page_size / kPB;
    v.by_bpp = fast_div(v.bpp);
    v.n_pages = C.n_pages;
    v.kc = C.k_codes;
    v.vc = C.v_codes;
    v.ks = C.k_scales;
    v.vs = C.v_scales;
    v.B = B.B;
    v.T = B.T;
    v.pages_ld = B.pages_ld;
    v.row_start = B.row_start;
    v.ctx = B.ctx;
    v.pages = B.pages;
    return v;
}

// Index of block `blk` (16 tokens) of sequence b and KV head 0 in the scale
// arrays, counted per head as (page * Hkv) * bpp + block of the page; -1 when
// the page table has no valid page there.  Head g lies g * bpp further on, and
// the codes of the block start at 2048 times its index.
__device__ __forceinline__ int64_t block_index(const PagedView &v, int b, int blk) {
    if (blk < 0) return -1;
    const int e = v.by_bpp.quot(blk);
    if (e >= v.pages_ld) return -1;
    const int page = v.pages[static_cast<int64_t>(b) * v.pages_ld + e];
    if (page < 0 || page >= v.n_pages) return -1;
    return static_cast<int64_t>(page) * v.Hkv * v.bpp + (blk - e * v.bpp);
}

// The sequence of row t, by bisection over row_start (in shared or global
// memory); -1 for a row behind the last sequence (or before the first).
__device__ __forceinline__ int row_sequence(const int32_t *row_start, int B, int t) {
    if (t < row_start[0] || t >= row_start[B]) return -1;
    int lo = 0, hi = B;  // row_start[lo] <= t < row_start[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (row_start[mid] <= t) lo = mid; else hi = mid;
    }
    return lo;
}

// Launch with programmatic dependent launch.
template <typename... P, typename... A>
cudaError_t launch_pdl(void (*kernel)(P...), dim3 grid, int threads, size_t smem, cudaStream_t s, A... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, args...);
    if (e != cudaSuccess) return e;
    return cudaGetLastError();
}

}  // namespace tern
