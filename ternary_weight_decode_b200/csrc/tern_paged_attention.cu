// tern_paged_attention.cu -- attention over the paged 8-bit KV cache.
//
// out = sum_j softmax_j(scale q . k_j) v_j, one pass over the tokens with the
// running maximum m and sum z of the softmax: a new maximum m' scales what was
// summed before by 2^(m - m') (scores are held times log2 e).
//
// attn_split_paged_kernel.  The rows of one sequence that share a KV head (its
// tokens times the query heads of the group) are taken eight at a time: an
// item.  An item's work is its visible tiles of 16 tokens (one scale block
// each).  All tiles of all items form one line, cut into equal ranges, one per
// CTA, so that uneven contexts fill the GPU evenly; the lengths are read on the
// device.  An item cut by a range's end leaves partial results (m, z and the
// unnormalised sum) in the workspace; the CTA that finishes its last part
// merges them in the order of the ranges, so the result does not depend on
// timing.
//
// A warp takes every kWarps-th tile of its CTA's part of an item: TMA brings
// the 16 key and 16 value rows (2 KB each, 128-byte swizzle) into the warp's
// own ring of stages, and the warp multiplies on the tensor cores with fp16
// operands and fp32 accumulators (m16n8k16).  Codes of 8 bits are exact in
// fp16.  Queries and softmax weights are fp32 values, held as two fp16 parts
// hi + lo (22 bits, the query row first scaled by a power of two): the eight
// rows' hi parts fill rows 0-7 of the 16-row operand and their lo parts rows
// 8-15, so the second part costs no further matrix instruction, and the two
// halves of a result lie in one thread.  The value product of each tile starts
// from zero and is added to the fp32 sum with the block's scale, so that no
// long chain of sums runs inside the tensor cores.
//
// The order of the 128 dimensions inside a score's sum is free: lane (g, t)
// (g = lane / 4, t = lane % 4) feeds bytes 32t .. 32t+31 of key g, two 16-byte
// loads; likewise output column n of value product i is dimension 16 n + i, so
// a lane's value operands are 16 contiguous bytes of four tokens.
#include <cuda_fp16.h>

#include <algorithm>

#include "tern_paged.cuh"

namespace tern {

namespace {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kCtasPerSm = 4;
constexpr int kRows = 8;         // rows of an item
constexpr int kStages = 3;       // tiles in flight per warp
constexpr int kTileBytes = kPB * kPD;       // 2048: one block's codes of K or of V
constexpr int kStageBytes = 2 * kTileBytes;
constexpr int kMaxCtas = 1024;   // CTAs of a launch (counters of the workspace)
constexpr float kPScale = 8.0f;  // softmax weights are held times 2^8: their lo parts stay normal in fp16

// Workspace: kMaxCtas counters (zero at rest), then per CTA two partial records.
constexpr int kRecFloats = kRows * (kPD + 2);

struct AttnParams {
    PagedView v;
    const float *q;
    int ldq, Hq, GQ;
    int window, sinks;
    float scale_log2;
    float *out;
    int ldo;
    int *counters;
    float *part;
};

// One sequence as this call sees it.
struct Seq {
    int start, rows;  // first row, rows x query heads of a group
    int first;        // token of the first row
    int end;          // tokens that may be read: min(ctx, page table)
};

__device__ __forceinline__ Seq sequence(const AttnParams &p, int b) {
    const PagedView &v = p.v;
    const int s0 = v.row_start[b], s1 = v.row_start[b + 1], ctx = v.ctx[b];
    Seq s;
    s.start = s0;
    s.rows = s0 < 0 || s0 > v.T || s1 <= s0 ? 0 : (min(s1, v.T) - s0) * p.GQ;
    s.first = ctx - (s1 - s0);
    const long long cap = static_cast<long long>(v.pages_ld) * v.page_size;
    s.end = static_cast<int>(min(static_cast<long long>(min(ctx, 0x7FFFFF00)), cap));
    return s;
}

// Visible tiles of row tile rt: tile k is k below `sink`, else lo + k - sink.
struct Tiles {
    int n, sink, lo;
};

__device__ __forceinline__ Tiles tiles_of(const AttnParams &p, const Seq &s, int rt) {
    const int r1 = min(kRows * rt + kRows, s.rows) - 1;
    const int p0 = s.first + kRows * rt / p.GQ, p1 = s.first + r1 / p.GQ;
    const int hi = max(0, min(p1 + 1, s.end));
    const int hit = (hi + kPB - 1) / kPB;
    Tiles t;
    t.lo = t.sink = 0;
    if (p.window > 0) {
        t.lo = min(max(0, p0 - p.window + 1) / kPB, hit);
        t.sink = min((min(p.sinks, hi) + kPB - 1) / kPB, t.lo);
    }
    t.n = t.sink + hit - t.lo;
    return t;
}

// Tiles of one KV head of a sequence (an item that sees nothing still counts
// one: its rows are written as 0).
__device__ __forceinline__ long long head_units(const AttnParams &p, const Seq &s) {
    long long u = 0;
    for (int rt = 0; rt * kRows < s.rows; ++rt) u += max(1, tiles_of(p, s, rt).n);
    return u;
}

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t as_u32(__half2 h) { return *reinterpret_cast<uint32_t *>(&h); }

// Two fp32 values as fp16 pairs hi + lo.
__device__ __forceinline__ void split2(float x, float y, uint32_t &hi, uint32_t &lo) {
    const __half2 h = __floats2half2_rn(x, y);
    const float2 f = __half22float2(h);
    hi = as_u32(h);
    lo = as_u32(__floats2half2_rn(x - f.x, y - f.y));
}

// Codes c0 c1 (low half of the pair's bytes) as fp16 x 2.  int8: 1024 + (c +
// 128) has the code's bits as its low byte (fp16 spacing 1 there), and one
// subtraction leaves c; the caller has flipped the sign bits.  e4m3: the
// conversion instruction.
template <int KIND, int SEL>
__device__ __forceinline__ uint32_t code_pair(uint32_t w) {
    if constexpr (KIND == TERN_KV_INT8) {
        const uint32_t m = __byte_perm(w, 0x64646464u, SEL ? 0x4342 : 0x4140);
        return as_u32(__hsub2(*reinterpret_cast<const __half2 *>(&m), __half2(__half(1152.0f), __half(1152.0f))));
    } else {
        uint32_t r;
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(static_cast<unsigned short>(SEL ? w >> 16 : w & 0xFFFFu)));
        return r;
    }
}
template <int KIND>
__device__ __forceinline__ uint32_t flip(uint32_t w) {
    return KIND == TERN_KV_INT8 ? w ^ 0x80808080u : w;
}

// The running softmax of one warp: row g's reference (its maximum less
// kPScale; weights are 2^(score - m)) and this lane's part of its sum, and the
// lane's output columns (dimensions 32 t + i and 32 t + 16 + i).
struct State {
    float m, z;
    float o[16][2];
};

template <int KIND>
__global__ void __launch_bounds__(kThreads, kCtasPerSm)
    attn_split_paged_kernel(AttnParams p, const __grid_constant__ CUtensorMap kmap,
                            const __grid_constant__ CUtensorMap vmap) {
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    __shared__ uint64_t bars[kWarps][kStages];
    __shared__ long long scan[kWarps];
    __shared__ long long s_total, s_off;
    __shared__ int s_b, s_last;
    __shared__ float wm[kWarps][kRows], wz[kWarps][kRows];
    uint8_t *ring = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    float *merge = reinterpret_cast<float *>(ring);  // [kWarps][kRows][kPD], between segments
    const PagedView &v = p.v;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int g = lane >> 2, t = lane & 3;
    const int c = blockIdx.x;

    if (tid == 0) {
        prefetch_tmap(&kmap);
        prefetch_tmap(&vmap);
        for (int w = 0; w < kWarps; ++w)
            for (int s = 0; s < kStages; ++s) mbar_init(&bars[w][s], 1);
        fence_mbar_init();
    }
    pdl_wait();

    // ---- this CTA's range of the line of tiles
    const int per = (v.B + kThreads - 1) / kThreads;
    const int b0 = tid * per, b1 = min(v.B, b0 + per);
    long long mine = 0;
    for (int b = b0; b < b1; ++b) mine += v.Hkv * head_units(p, sequence(p, b));
    long long incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long x = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += x;
    }
    if (lane == 31) scan[warp] = incl;
    __syncthreads();
    long long before = 0, total = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        if (w < warp) before += scan[w];
        total += scan[w];
    }
    const int G = static_cast<int>(min(static_cast<long long>(gridDim.x), total));  // no range is empty
    long long u = c < G ? total * c / G : 0;
    const long long u_end = c < G ? total * (c + 1) / G : 0;
    {
        const long long base = before + incl - mine;
        if (c < G && u >= base && u < base + mine) {
            long long off = u - base;
            int b = b0;
            for (; b < b1; ++b) {
                const long long n = v.Hkv * head_units(p, sequence(p, b));
                if (off < n) break;
                off -= n;
            }
            s_b = b;
            s_off = off;
        }
    }
    __syncthreads();

    uint32_t phases = 0;  // parity of each of this warp's stages
    uint8_t *my_ring = ring + warp * kStages * kStageBytes;
    int b = u < u_end ? s_b : 0;
    long long off = u < u_end ? s_off : 0;

    while (u < u_end) {
        // ---- the segment: tiles [k0, k1) of item (b, head, rt)
        const Seq s = sequence(p, b);
        const long long per_head = head_units(p, s);
        if (off >= per_head * v.Hkv) {  // the next sequence
            off -= per_head * v.Hkv;
            ++b;
            continue;
        }
        const int head = static_cast<int>(off / per_head);
        long long rem = off - head * per_head;
        int rt = 0;
        Tiles tl = tiles_of(p, s, 0);
        while (rem >= max(1, tl.n)) {
            rem -= max(1, tl.n);
            tl = tiles_of(p, s, ++rt);
        }
        const int item_units = max(1, tl.n);
        const int k0 = static_cast<int>(rem);
        const int k1 = static_cast<int>(min(static_cast<long long>(item_units), rem + (u_end - u)));
        const long long item_u0 = u - k0;

        // ---- queries: row g of the item, dimensions 32 t .. 32 t + 31
        const int r = kRows * rt + g;
        const bool row_ok = r < s.rows;
        const int pos = s.first + (row_ok ? r / p.GQ : 0);
        uint32_t qhi[8][2], qlo[8][2];
        float rowf;
        {
            const float *qp = p.q + static_cast<int64_t>(s.start + r / p.GQ) * p.ldq +
                              (head * p.GQ + r % p.GQ) * kPD + 32 * t;
            float4 x[8];
            float amax = 0.0f;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                x[i] = row_ok ? *reinterpret_cast<const float4 *>(qp + 4 * i) : make_float4(0, 0, 0, 0);
                amax = fmaxf(amax, fmaxf(fmaxf(fabsf(x[i].x), fabsf(x[i].y)), fmaxf(fabsf(x[i].z), fabsf(x[i].w))));
            }
            amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
            amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
            // the row times 2^e: its largest value in [2^7, 2^8)
            const int e = max(-120, min(120, 134 - static_cast<int>(__float_as_uint(amax) >> 23)));
            const float up = __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
            rowf = p.scale_log2 * __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                split2(x[i].x * up, x[i].y * up, qhi[i][0], qlo[i][0]);
                split2(x[i].z * up, x[i].w * up, qhi[i][1], qlo[i][1]);
            }
        }

        // ---- this warp's tiles of the segment: k0 + warp, k0 + warp + kWarps, ...
        State st;
        st.m = -INFINITY;
        st.z = 0.0f;
#pragma unroll
        for (int i = 0; i < 16; ++i) st.o[i][0] = st.o[i][1] = 0.0f;
        const int k_real = min(k1, tl.n);  // an item without tiles has no real one
        const int count = k0 + warp < k_real ? (k_real - k0 - warp + kWarps - 1) / kWarps : 0;
        const int p_min = s.first + kRows * rt / p.GQ, p_max = s.first + (min(kRows * rt + kRows, s.rows) - 1) / p.GQ;
        int bi_lane = -1;             // block of tile (group of 32) + lane
        float ks_lane = 0.0f, vs_lane = 0.0f;
        int bi_next = -1;             // the same of the next group
        float ks_next = 0.0f, vs_next = 0.0f;
        auto tile_at = [&](int i) {
            const int k = k0 + warp + i * kWarps;
            return k < tl.sink ? k : tl.lo + k - tl.sink;
        };
        auto fetch = [&](int i0, int &bi, float &ks, float &vs) {
            bi = -1;
            if (i0 + lane < count) {
                const int64_t x = block_index(v, b, tile_at(i0 + lane));
                if (x >= 0) {
                    bi = static_cast<int>(x) + head * v.bpp;
                    ks = __ldg(v.ks + bi);
                    vs = __ldg(v.vs + bi);
                }
            }
        };
        fetch(0, bi_lane, ks_lane, vs_lane);
        fetch(32, bi_next, ks_next, vs_next);
        auto start = [&](int i, int bi) {
            if (lane == 0 && bi >= 0) {
                uint8_t *dst = my_ring + (i % kStages) * kStageBytes;
                uint64_t *bar = &bars[warp][i % kStages];
                mbar_arrive_expect_tx(bar, kStageBytes);
                tma_load_2d_nohint(dst, &kmap, 0, bi * kPB, bar);
                tma_load_2d_nohint(dst + kTileBytes, &vmap, 0, bi * kPB, bar);
            }
        };
        // the merge buffer of the segment before lay where the stages are
        fence_proxy_async_smem();
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kStages; ++i) start(i, __shfl_sync(0xffffffffu, bi_lane, i));

        for (int i = 0; i < count; ++i) {
            if ((i & 31) == 0 && i > 0) {
                bi_lane = bi_next;
                ks_lane = ks_next;
                vs_lane = vs_next;
                fetch(i + 32, bi_next, ks_next, vs_next);
            }
            const int bi = __shfl_sync(0xffffffffu, bi_lane, i & 31);
            const float ks = __shfl_sync(0xffffffffu, ks_lane, i & 31);
            const float vs = __shfl_sync(0xffffffffu, vs_lane, i & 31);
            const int stage = i % kStages;
            if (bi >= 0) {
                mbar_wait_bounded(&bars[warp][stage], (phases >> stage) & 1u);
                phases ^= 1u << stage;
                const uint8_t *kt = my_ring + stage * kStageBytes, *vt = kt + kTileBytes;
                const int tile = tile_at(i), j0 = tile * kPB;
                // scores: tokens j0 + 2t, + 1 (n = 0) and j0 + 8 + 2t, + 1 (n = 1) of row g
                float sc[2][4];
#pragma unroll
                for (int n = 0; n < 2; ++n) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) sc[n][e] = 0.0f;
                    const uint8_t *row = kt + (8 * n + g) * kPD;
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const uint4 w4 = lds128(row + (((2 * t + h) ^ g) << 4));
                        const uint32_t w[4] = {w4.x, w4.y, w4.z, w4.w};
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int i8 = 4 * h + e;
                            const uint32_t f = flip<KIND>(w[e]);
                            const uint32_t a[4] = {qhi[i8][0], qlo[i8][0], qhi[i8][1], qlo[i8][1]};
                            mma_f16(sc[n], a, code_pair<KIND, 0>(f), code_pair<KIND, 1>(f));
                        }
                    }
                }
                const float f = rowf * ks;
                float x[4] = {(sc[0][0] + sc[0][2]) * f, (sc[0][1] + sc[0][3]) * f, (sc[1][0] + sc[1][2]) * f,
                              (sc[1][1] + sc[1][3]) * f};
                const bool whole = j0 + kPB - 1 <= p_min &&
                                   (p.window == 0 || j0 > p_max - p.window || j0 + kPB <= p.sinks);
                if (!whole) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int j = j0 + (e >> 1) * 8 + 2 * t + (e & 1);
                        if (j > pos || (p.window > 0 && j <= pos - p.window && j >= p.sinks)) x[e] = -INFINITY;
                    }
                }
                float mx = fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3]));
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
                const float mn = fmaxf(st.m, mx - kPScale);
                const float ref = mn == -INFINITY ? 0.0f : mn;
                if (__any_sync(0xffffffffu, mn != st.m)) {
                    const float corr = ex2(st.m - ref);  // 0 when nothing was seen before
                    st.z *= corr;
#pragma unroll
                    for (int k = 0; k < 16; ++k) {
                        st.o[k][0] *= corr;
                        st.o[k][1] *= corr;
                    }
                    st.m = mn;
                }
                float w[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) w[e] = ex2(x[e] - ref);
                st.z += (w[0] + w[1]) + (w[2] + w[3]);
                uint32_t a[4];
                split2(w[0], w[1], a[0], a[1]);
                split2(w[2], w[3], a[2], a[3]);
                // values: tokens 2t, 2t + 1, 2t + 8, 2t + 9 of the tile, dimensions 16 g .. 16 g + 15
                uint32_t vw[4][4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int rr = 2 * t + (k & 1) + 8 * (k >> 1);
                    const uint4 w4 = lds128(vt + rr * kPD + ((g ^ (rr & 7)) << 4));
                    vw[k][0] = w4.x;
                    vw[k][1] = w4.y;
                    vw[k][2] = w4.z;
                    vw[k][3] = w4.w;
                    if (j0 + kPB > s.end && j0 + rr >= s.end)  // slots behind the context hold anything
                        vw[k][0] = vw[k][1] = vw[k][2] = vw[k][3] = 0;
                }
#pragma unroll
                for (int q4 = 0; q4 < 4; ++q4) {
                    const uint32_t x0 = flip<KIND>(vw[0][q4]), x1 = flip<KIND>(vw[1][q4]);
                    const uint32_t y0 = flip<KIND>(vw[2][q4]), y1 = flip<KIND>(vw[3][q4]);
                    const uint32_t xl = __byte_perm(x0, x1, 0x5140), xh = __byte_perm(x0, x1, 0x7362);
                    const uint32_t yl = __byte_perm(y0, y1, 0x5140), yh = __byte_perm(y0, y1, 0x7362);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        float d[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                        if (e == 0) mma_f16(d, a, code_pair<KIND, 0>(xl), code_pair<KIND, 0>(yl));
                        if (e == 1) mma_f16(d, a, code_pair<KIND, 1>(xl), code_pair<KIND, 1>(yl));
                        if (e == 2) mma_f16(d, a, code_pair<KIND, 0>(xh), code_pair<KIND, 0>(yh));
                        if (e == 3) mma_f16(d, a, code_pair<KIND, 1>(xh), code_pair<KIND, 1>(yh));
                        float(&o)[2] = st.o[4 * q4 + e];
                        o[0] = fmaf(vs, d[0] + d[2], o[0]);
                        o[1] = fmaf(vs, d[1] + d[3], o[1]);
                    }
                }
                fence_proxy_async_smem();  // these reads before the refill of the stage
                __syncwarp();
            }
            const int in = i + kStages;
            if (in < count) {
                // tile in's block: of this group of 32, or of the next
                const int cur = __shfl_sync(0xffffffffu, bi_lane, in & 31);
                const int nxt = __shfl_sync(0xffffffffu, bi_next, in & 31);
                start(in, (in >> 5) == (i >> 5) ? cur : nxt);
            }
        }

        // ---- the warps' results, merged in warp order
        st.z += __shfl_xor_sync(0xffffffffu, st.z, 1);
        st.z += __shfl_xor_sync(0xffffffffu, st.z, 2);
        __syncthreads();  // the stages are free
        if (t == 0) {
            wm[warp][g] = st.m;
            wz[warp][g] = st.z;
        }
        {
            float *mg = merge + (warp * kRows + g) * kPD + 32 * t;
#pragma unroll
            for (int i = 0; i < 16; i += 4) {
                *reinterpret_cast<float4 *>(mg + i) =
                    make_float4(st.o[i][0], st.o[i + 1][0], st.o[i + 2][0], st.o[i + 3][0]);
                *reinterpret_cast<float4 *>(mg + 16 + i) =
                    make_float4(st.o[i][1], st.o[i + 1][1], st.o[i + 2][1], st.o[i + 3][1]);
            }
        }
        __syncthreads();
        const bool complete = k0 == 0 && k1 == item_units;
        float *rec = p.part + static_cast<int64_t>(2 * c + (k0 == 0 ? 1 : 0)) * kRecFloats;
        for (int rr = warp; rr < kRows; rr += kWarps) {
            const int row = kRows * rt + rr;
            if (row >= s.rows) break;
            float M = -INFINITY;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) M = fmaxf(M, wm[w][rr]);
            const float ref = M == -INFINITY ? 0.0f : M;
            float z = 0.0f;
            float4 o = make_float4(0, 0, 0, 0);
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const float f = ex2(wm[w][rr] - ref);
                const float4 x = *reinterpret_cast<const float4 *>(merge + (w * kRows + rr) * kPD + 4 * lane);
                z = fmaf(f, wz[w][rr], z);
                o.x = fmaf(f, x.x, o.x);
                o.y = fmaf(f, x.y, o.y);
                o.z = fmaf(f, x.z, o.z);
                o.w = fmaf(f, x.w, o.w);
            }
            if (complete) {
                const float iz = z > 0.0f ? 1.0f / z : 0.0f;
                *reinterpret_cast<float4 *>(p.out + static_cast<int64_t>(s.start + row / p.GQ) * p.ldo +
                                            (head * p.GQ + row % p.GQ) * kPD + 4 * lane) =
                    make_float4(o.x * iz, o.y * iz, o.z * iz, o.w * iz);
            } else {
                *reinterpret_cast<float4 *>(rec + rr * kPD + 4 * lane) = o;
                if (lane == 0) {
                    rec[kRows * kPD + 2 * rr] = M;
                    rec[kRows * kPD + 2 * rr + 1] = z;
                }
            }
        }

        // ---- a cut item: whoever finishes its last part merges all of them
        if (!complete) {
            // the ranges that hold its first and its last tile (range c begins at floor(c * total / G))
            const int c_first = static_cast<int>(((item_u0 + 1) * G + total - 1) / total) - 1;
            const int c_last = static_cast<int>(((item_u0 + item_units) * G + total - 1) / total) - 1;
            __threadfence();
            __syncthreads();
            if (tid == 0) {
                const int done = atomicAdd(p.counters + c_first, 1);
                s_last = done == c_last - c_first;
                if (s_last) p.counters[c_first] = 0;  // zero at rest
            }
            __syncthreads();
            if (s_last) {
                __threadfence();
                for (int rr = warp; rr < kRows; rr += kWarps) {
                    const int row = kRows * rt + rr;
                    if (row >= s.rows) break;
                    const int parts = c_last - c_first + 1;
                    auto record = [&](int i) {
                        return p.part + static_cast<int64_t>(i == 0 ? 2 * c_first + 1 : 2 * (c_first + i)) * kRecFloats;
                    };
                    float M = -INFINITY;
                    for (int i = lane; i < parts; i += 32)
                        M = fmaxf(M, __ldcg(record(i) + kRows * kPD + 2 * rr));
                    M = warp_max(M);
                    const float ref = M == -INFINITY ? 0.0f : M;
                    float z = 0.0f;
                    float4 o = make_float4(0, 0, 0, 0);
#pragma unroll 4
                    for (int i = 0; i < parts; ++i) {
                        const float *rc = record(i);
                        const float2 mz = __ldcg(reinterpret_cast<const float2 *>(rc + kRows * kPD + 2 * rr));
                        const float4 x = __ldcg(reinterpret_cast<const float4 *>(rc + rr * kPD + 4 * lane));
                        const float f = ex2(mz.x - ref);
                        z = fmaf(f, mz.y, z);
                        o.x = fmaf(f, x.x, o.x);
                        o.y = fmaf(f, x.y, o.y);
                        o.z = fmaf(f, x.z, o.z);
                        o.w = fmaf(f, x.w, o.w);
                    }
                    const float iz = z > 0.0f ? 1.0f / z : 0.0f;
                    *reinterpret_cast<float4 *>(p.out + static_cast<int64_t>(s.start + row / p.GQ) * p.ldo +
                                                (head * p.GQ + row % p.GQ) * kPD + 4 * lane) =
                        make_float4(o.x * iz, o.y * iz, o.z * iz, o.w * iz);
                }
            }
        }
        u += k1 - k0;
        off += k1 - k0;
        __syncthreads();  // the merge buffer and the shared words are free
    }
    pdl_launch_dependents();
}

constexpr size_t kSplitSmem = kWarps * kStages * kStageBytes + 1024;

template <int KIND>
cudaError_t launch_split(const AttnParams &p, const CUtensorMap &km, const CUtensorMap &vm, int ctas, cudaStream_t s) {
    static DeviceOnce once;
    int dev = 0;
    cudaError_t e = current_device(&dev);
    if (e != cudaSuccess) return e;
    e = once.run(dev, [] {
        return cudaFuncSetAttribute(attn_split_paged_kernel<KIND>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    static_cast<int>(kSplitSmem));
    });
    if (e != cudaSuccess) return e;
    return launch_pdl(attn_split_paged_kernel<KIND>, dim3(ctas), kThreads, kSplitSmem, s, p, km, vm);
}

}  // namespace

size_t attention_paged_workspace_bytes(int Hq, int Hkv, int num_sms) {
    (void)Hq;
    (void)Hkv;
    (void)num_sms;
    return kMaxCtas * sizeof(int) + static_cast<size_t>(2) * kMaxCtas * kRecFloats * sizeof(float);
}

cudaError_t launch_attention_paged(const PagedAttentionLaunch &A, cudaStream_t s, const char **why) {
    AttnParams p;
    p.v = paged_view(A.batch, A.cache);
    p.q = A.q;
    p.ldq = A.ldq;
    p.Hq = A.Hq;
    p.GQ = A.Hq / A.cache.Hkv;
    p.window = std::min(A.window, 1 << 30);  // positions minus a window stay in 32 bits
    p.sinks = std::min(A.sinks, 1 << 30);
    p.scale_log2 = A.scale * 1.4426950408889634f;
    p.out = A.out;
    p.ldo = A.ldo;
    p.counters = reinterpret_cast<int *>(A.workspace);
    p.part = A.workspace + kMaxCtas;
    CUtensorMap km, vm;
    const uint64_t rows = static_cast<uint64_t>(A.cache.n_pages) * A.cache.Hkv * A.cache.page_size;
    if (!make_u8_tmap_2d(&km, A.cache.k_codes, kPD, rows, kPD, kPD, kPB) ||
        !make_u8_tmap_2d(&vm, A.cache.v_codes, kPD, rows, kPD, kPD, kPB)) {
        *why = "cuTensorMapEncodeTiled failed or is unavailable";
        return cudaErrorInvalidValue;
    }
    // one CTA per resident slot, fewer when the tiles are few
    const int64_t rowtiles = ceil_div(static_cast<int64_t>(std::min(A.batch.max_rows, A.batch.T)) * p.GQ, kRows);
    const int64_t span = A.window > 0 ? std::min<int64_t>(A.batch.max_ctx, static_cast<int64_t>(A.window) + A.sinks + 32)
                                      : A.batch.max_ctx;
    const int64_t units = std::min<int64_t>(A.batch.B, A.batch.T) * A.cache.Hkv * rowtiles * ceil_div(span, kPB);
    int64_t ctas = std::min<int64_t>(kCtasPerSm * A.num_sms, ceil_div(units, kWarps));
    ctas = std::max<int64_t>(1, std::min<int64_t>(ctas, kMaxCtas));
    if (A.cache.kind == TERN_KV_INT8) return launch_split<TERN_KV_INT8>(p, km, vm, static_cast<int>(ctas), s);
    return launch_split<TERN_KV_E4M3>(p, km, vm, static_cast<int>(ctas), s);
}

}  // namespace tern
