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
// warp of the grid, so that uneven contexts fill the GPU evenly; the lengths
// are read on the device.  A warp walks its range without waiting for others:
// the ring of TMA stages runs on across items.  An item that lies inside one
// warp's range is written out by it; the pieces of the others (m, z and the
// unnormalised sum) are merged in the order of the ranges, first those of a
// CTA through shared memory, then those of several CTAs through the workspace,
// by the CTA that finishes the last of them, so the result does not depend on
// timing.
//
// TMA brings the 16 key and 16 value rows of a tile (2 KB each, 128-byte
// swizzle) into the warp's own stages, and the warp multiplies on the tensor
// cores with fp16 operands and fp32 accumulators (m16n8k16).  Codes of 8 bits
// are exact in fp16.  Queries and softmax weights are fp32 values, held as two
// fp16 parts hi + lo (22 bits, the query row first scaled by a power of two):
// the eight rows' hi parts fill rows 0-7 of the 16-row operand and their lo
// parts rows 8-15, so the second part costs no further matrix instruction, and
// the two halves of a result lie in one thread.  The value product of each
// tile starts from zero and is added to the fp32 sum with the block's scale,
// so that no long chain of sums runs inside the tensor cores.
//
// The order of the 128 dimensions inside a score's sum is free: lane (g, t)
// (g = lane / 4, t = lane % 4) feeds bytes 32t .. 32t+31 of key g, two 16-byte
// loads; likewise output column n of value product i is dimension 16 n + i, so
// a lane's value operands are 16 contiguous bytes of four tokens.
#include <cuda_fp16.h>

#include <algorithm>

#include "tern_paged_attention.cuh"

namespace tern {

namespace {

constexpr int kWarps = 12;
constexpr int kThreads = 32 * kWarps;
constexpr int kRows = 8;         // rows of an item
constexpr int kStages = 3;       // tiles in flight per warp
constexpr int kBatch = 16;       // tiles whose places are looked up at a time, one a lane
constexpr int kTileBytes = kPB * kPD;       // 2048: one block's codes of K or of V
constexpr int kStageBytes = 2 * kTileBytes;
constexpr float kPScale = 8.0f;  // softmax weights are held times 2^8: their lo parts stay normal in fp16

__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// The same from zero.
__device__ __forceinline__ void mma_f16_zero(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%10, %10, %10, %10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.0f));
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
    float2 o[16];
};

// What a warp's walk needs of one tile.
struct __align__(16) TileInfo {
    int bi;          // scale block of K and V (its 16 rows begin at 16 bi), -1: none
    float ks, vs;
    int j0;          // first token
    int b, head, rt; // item
    int k;           // tile of the item, times 2, + 1 for the item's last tile
};

// A warp's piece of an item that others share.
struct Piece {
    int valid, ends;   // ends: holds the item's last tile
    int head, rt, units;
    Seq s;
    long long u0;      // line index of the item's first tile
};

constexpr int kRingBytes = kWarps * kStages * kStageBytes;
constexpr int kPieceFloats = kRows * kPD;
struct SplitShared {
    float first[kWarps][kPieceFloats];  // the piece a warp's range begins with (its last piece lies in its ring)
    TileInfo info[kWarps][2][kBatch];
    float m[kWarps][2][kRows], z[kWarps][2][kRows];
    Piece piece[kWarps][2];
    uint64_t bars[kWarps][kStages];
    LineShared line;
    CutItem cut[2];
    int last[2];
};
constexpr size_t kSplitSmem = kRingBytes + sizeof(SplitShared) + 1024;
static_assert(kSplitSmem <= 227 * 1024, "shared memory of one CTA");

template <int KIND>
__global__ void __launch_bounds__(kThreads, 1)
    attn_split_paged_kernel(AttnParams p, const __grid_constant__ CUtensorMap kmap,
                            const __grid_constant__ CUtensorMap vmap) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t *ring = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    SplitShared &S = *reinterpret_cast<SplitShared *>(ring + kRingBytes);
    const PagedView &v = p.v;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int g = lane >> 2, t = lane & 3;
    const int c = blockIdx.x;
    uint8_t *my_ring = ring + warp * kStages * kStageBytes;

    if (tid == 0) {
        prefetch_tmap(&kmap);
        prefetch_tmap(&vmap);
    }
    if (lane == 0) {
        for (int s = 0; s < kStages; ++s) mbar_init(&S.bars[warp][s], 1);
        fence_mbar_init();
        S.piece[warp][0].valid = S.piece[warp][1].valid = 0;
        S.piece[warp][0].ends = 0;
        if (warp < 2) S.cut[warp].valid = 0;
    }
    pdl_wait();

    // ---- the line of tiles, and this warp's range of it
    const Line L = make_line<kRows, 1>(p, S.line);
    const long long total = L.total;
    auto seq_of = [&](int b) { return L.per == 1 ? S.line.seq[b] : sequence(p, b); };
    const int nw = static_cast<int>(min(static_cast<long long>(gridDim.x) * kWarps, total));
    Ranges R = {0, 0};
    if (total > 0) {
        R.base = quot(total, nw);
        R.more = total - R.base * nw;
    }
    const int wi = c * kWarps + warp;  // this warp's range
    const long long u0 = wi < nw ? R.begin(wi) : 0;
    const int count = wi < nw ? static_cast<int>(R.begin(wi + 1) - u0) : 0;

    if (count > 0) {
        Cursor<1> cur = find_place<kRows, 1>(p, S.line, L, u0, seq_of);
        // lane l < kBatch keeps the cursor of tiles l, l + kBatch, ...: tile i of the range is in
        // info[i / kBatch % 2][i % kBatch]
        auto info = [&](int i) -> TileInfo & { return S.info[warp][(i / kBatch) & 1][i % kBatch]; };
        int step = lane;
        auto fill = [&](int i0) {
            if (lane < kBatch && i0 + lane < count) {
                advance<kRows>(p, cur, step, seq_of);
                step = kBatch;
                TileInfo x;
                x.j0 = cur.tl.block(cur.k) * kPB;
                x.b = cur.b;
                x.head = cur.head;
                x.rt = cur.rt;
                x.k = 2 * cur.k + (cur.k + 1 == cur.units() ? 1 : 0);
                x.bi = -1;
                x.ks = x.vs = 0.0f;
                if (cur.tl.n > 0) {
                    const int64_t bi = block_index(v, cur.b, cur.tl.block(cur.k));
                    if (bi >= 0) {
                        x.bi = static_cast<int>(bi) + cur.head * v.bpp;
                        x.ks = v.ks[x.bi];
                        x.vs = v.vs[x.bi];
                    }
                }
                info(i0 + lane) = x;
            }
            __syncwarp();
        };
        auto start = [&](int i) {  // tile i's copies into its stage
            if (lane == 0 && i < count) {
                const int bi = info(i).bi;
                if (bi >= 0) {
                    uint8_t *dst = my_ring + (i % kStages) * kStageBytes;
                    uint64_t *bar = &S.bars[warp][i % kStages];
                    mbar_arrive_expect_tx(bar, kStageBytes);
                    tma_load_2d_nohint(dst, &kmap, 0, bi * kPB, bar);
                    tma_load_2d_nohint(dst + kTileBytes, &vmap, 0, bi * kPB, bar);
                }
            }
        };

        State st;
        uint32_t qhi[8][2], qlo[8][2];
        Seq s = {};
        float rowf = 0.0f;
        int pos = 0, p_min = 0, p_max = 0, k_first = 0;
        uint32_t phases = 0;  // parity of each stage
        int stage = 0;
#pragma unroll 1
        for (int i = -1; i < count; ++i) {
            // look up the first batch, and the batch behind the next while this one is worked off
            if (i < 0 || (i % kBatch == 0 && i + kBatch < count)) fill(i < 0 ? 0 : i + kBatch);
            if (i < 0) {
#pragma unroll 1
                for (int e = 0; e < kStages; ++e) start(e);
                continue;
            }
            const TileInfo x = info(i);
            if (i == 0 || (x.k >> 1) == 0) {
                // ---- a new item: row g's query, dimensions 32 t .. 32 t + 31, as hi + lo operands
                s = seq_of(x.b);
                k_first = x.k >> 1;
                const int r = kRows * x.rt + g;
                const bool row_ok = r < s.rows;
                const int ri = row_ok ? p.by_gq.quot(r) : 0;
                pos = s.first + ri;
                p_min = s.first + p.by_gq.quot(kRows * x.rt);
                p_max = s.first + p.by_gq.quot(min(kRows * x.rt + kRows, s.rows) - 1);
                const float *qp = p.q + static_cast<int64_t>(s.start + ri) * p.ldq +
                                  (x.head * p.GQ + (row_ok ? r : 0) - ri * p.GQ) * kPD + 32 * t;
                float4 q4[8];
                float amax = 0.0f;
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    q4[e] = row_ok ? *reinterpret_cast<const float4 *>(qp + 4 * e) : make_float4(0, 0, 0, 0);
                    amax = fmaxf(amax, fmaxf(fmaxf(fabsf(q4[e].x), fabsf(q4[e].y)), fmaxf(fabsf(q4[e].z), fabsf(q4[e].w))));
                }
                amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
                amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
                // the row times 2^e: its largest value in [2^7, 2^8)
                const int e = max(-120, min(120, 134 - static_cast<int>(__float_as_uint(amax) >> 23)));
                const float up = __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
                rowf = p.scale_log2 * __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
#pragma unroll
                for (int n = 0; n < 8; ++n) {
                    split2(q4[n].x * up, q4[n].y * up, qhi[n][0], qlo[n][0]);
                    split2(q4[n].z * up, q4[n].w * up, qhi[n][1], qlo[n][1]);
                }
                st.m = -INFINITY;
                st.z = 0.0f;
#pragma unroll
                for (int n = 0; n < 16; ++n) st.o[n] = make_float2(0.0f, 0.0f);
            }
            if (x.bi >= 0) {
                mbar_wait_bounded(&S.bars[warp][stage], (phases >> stage) & 1u);
                phases ^= 1u << stage;
                const uint8_t *kt = my_ring + stage * kStageBytes, *vt = kt + kTileBytes;
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
                const float f = rowf * x.ks;
                float y[4] = {(sc[0][0] + sc[0][2]) * f, (sc[0][1] + sc[0][3]) * f, (sc[1][0] + sc[1][2]) * f,
                              (sc[1][1] + sc[1][3]) * f};
                const bool whole = x.j0 + kPB - 1 <= p_min &&
                                   (p.window == 0 || x.j0 > p_max - p.window || x.j0 + kPB <= p.sinks);
                if (!whole) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int j = x.j0 + (e >> 1) * 8 + 2 * t + (e & 1);
                        if (j > pos || (p.window > 0 && j <= pos - p.window && j >= p.sinks)) y[e] = -INFINITY;
                    }
                }
                float mx = fmaxf(fmaxf(y[0], y[1]), fmaxf(y[2], y[3]));
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
                const float mn = fmaxf(st.m, mx - kPScale);
                const float ref = mn == -INFINITY ? 0.0f : mn;
                if (__any_sync(0xffffffffu, mn != st.m)) {
                    const float corr = ex2(st.m - ref);  // 0 when nothing was seen before
                    st.z *= corr;
#pragma unroll
                    for (int k = 0; k < 16; ++k) st.o[k] = __fmul2_rn(st.o[k], make_float2(corr, corr));
                    st.m = mn;
                }
                float w[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) w[e] = ex2(y[e] - ref);
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
                    if (x.j0 + kPB > s.end && x.j0 + rr >= s.end)  // slots behind the context hold anything
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
                        float d[4];
                        if (e == 0) mma_f16_zero(d, a, code_pair<KIND, 0>(xl), code_pair<KIND, 0>(yl));
                        if (e == 1) mma_f16_zero(d, a, code_pair<KIND, 1>(xl), code_pair<KIND, 1>(yl));
                        if (e == 2) mma_f16_zero(d, a, code_pair<KIND, 0>(xh), code_pair<KIND, 0>(yh));
                        if (e == 3) mma_f16_zero(d, a, code_pair<KIND, 1>(xh), code_pair<KIND, 1>(yh));
                        const float2 sum = __fadd2_rn(make_float2(d[0], d[1]), make_float2(d[2], d[3]));
                        st.o[4 * q4 + e] = __ffma2_rn(make_float2(x.vs, x.vs), sum, st.o[4 * q4 + e]);
                    }
                }
                fence_proxy_async_smem();  // these reads before the refill of the stage
                __syncwarp();
            }
            start(i + kStages);
            stage = stage + 1 == kStages ? 0 : stage + 1;

            const bool ends = (x.k & 1) != 0;
            if (ends || i + 1 == count) {
                // ---- the item, or this warp's piece of it, is done
                st.z += __shfl_xor_sync(0xffffffffu, st.z, 1);
                st.z += __shfl_xor_sync(0xffffffffu, st.z, 2);
                const int r = kRows * x.rt + g;
                if (k_first == 0 && ends) {
                    if (r < s.rows) {
#pragma unroll
                        for (int n = 0; n < 16; n += 4) {
                            write_row(p, s.start, x.head, r,
                                      make_float4(st.o[n].x, st.o[n + 1].x, st.o[n + 2].x, st.o[n + 3].x), st.z, 32 * t + n);
                            write_row(p, s.start, x.head, r,
                                      make_float4(st.o[n].y, st.o[n + 1].y, st.o[n + 2].y, st.o[n + 3].y), st.z,
                                      32 * t + 16 + n);
                        }
                    }
                } else {
                    const int slot = k_first > 0 ? 0 : 1;  // a range's first piece, or its last
                    float *dst = (slot == 0 ? S.first[warp] : reinterpret_cast<float *>(my_ring)) + g * kPD + 32 * t;
#pragma unroll
                    for (int n = 0; n < 16; n += 4) {
                        *reinterpret_cast<float4 *>(dst + n) =
                            make_float4(st.o[n].x, st.o[n + 1].x, st.o[n + 2].x, st.o[n + 3].x);
                        *reinterpret_cast<float4 *>(dst + 16 + n) =
                            make_float4(st.o[n].y, st.o[n + 1].y, st.o[n + 2].y, st.o[n + 3].y);
                    }
                    if (t == 0) {
                        S.m[warp][slot][g] = st.m;
                        S.z[warp][slot][g] = st.z;
                    }
                    if (lane == 0) {
                        Piece pc;
                        pc.valid = 1;
                        pc.ends = ends;
                        pc.s = s;
                        pc.head = x.head;
                        pc.rt = x.rt;
                        pc.u0 = u0 + i - (x.k >> 1);
                        pc.units = tile_count<1>(tiles_of<kRows>(p, s, x.rt));
                        S.piece[warp][slot] = pc;
                    }
                }
            }
        }
    }
    __syncthreads();

    // ---- pieces of this CTA's warps: group a begins with a warp's last piece
    // (a = warp) or with the first piece of warp 0 (a = -1), and goes on with
    // the first pieces of the warps behind it until the item ends
    const bool is_warp = lane < kWarps;
    const unsigned first_ok = __ballot_sync(0xffffffffu, is_warp && S.piece[is_warp ? lane : 0][0].valid);
    const unsigned first_ends = __ballot_sync(0xffffffffu, is_warp && S.piece[is_warp ? lane : 0][0].ends);
    const unsigned last_ok = __ballot_sync(0xffffffffu, is_warp && S.piece[is_warp ? lane : 0][1].valid);
    // bit 0: the first piece of warp 0, bit a + 1: the last piece of warp a
#pragma unroll 1
    for (unsigned groups = (first_ok & 1u) | last_ok << 1; groups != 0; groups &= groups - 1) {
        const int a = __ffs(groups) - 2, w0 = max(a, 0), slot0 = a < 0 ? 0 : 1;
        const Piece pc = S.piece[w0][slot0];
        // last warp of the group: the first behind w0 whose first piece ends the item, else the last of those that have one
        bool ends = pc.ends;
        int w1 = w0;
        if (!ends) {
            const int run = __ffs(~(first_ok >> (w0 + 1))) - 1, e = __ffs(first_ends >> (w0 + 1));
            ends = e != 0 && e <= run;
            w1 += ends ? e : run;
        }
        const bool complete = a >= 0 && ends;
        if (!complete && tid == 0) note_cut(S.cut[slot0], R, kWarps, pc.head, pc.rt, pc.s, pc.u0, pc.units);
        const Seq s = pc.s;
        for (int rr = warp; rr < kRows; rr += kWarps) {
            const int row = kRows * pc.rt + rr;
            if (row >= s.rows) break;
            const bool mine = lane >= w0 && lane <= w1;
            const int slot = lane == w0 ? slot0 : 0;
            const float m = mine ? S.m[lane][slot][rr] : -INFINITY;
            const float M = warp_max(m);
            const float f = ex2(m - (M == -INFINITY ? 0.0f : M));
            const float z = warp_sum(mine ? f * S.z[lane][slot][rr] : 0.0f);
            float4 o = make_float4(0, 0, 0, 0);
            float unused = 0.0f;
#pragma unroll 4
            for (int w = w0; w <= w1; ++w) {
                const float *src = w == w0 && slot0 == 1 ? reinterpret_cast<const float *>(ring + w * kStages * kStageBytes)
                                                         : S.first[w];
                add_scaled(o, unused, __shfl_sync(0xffffffffu, f, w),
                           *reinterpret_cast<const float4 *>(src + rr * kPD + 4 * lane), 0.0f);
            }
            if (complete) {
                write_row(p, s.start, pc.head, row, o, z, 4 * lane);
            } else {
                float *rec = p.part + static_cast<int64_t>(2 * c + slot0) * rec_floats(kRows);
                *reinterpret_cast<float4 *>(rec + rr * kPD + 4 * lane) = o;
                if (lane == 0) *reinterpret_cast<float2 *>(rec + kRows * kPD + 2 * rr) = make_float2(M, z);
            }
        }
    }

    __syncthreads();
    merge_cut_items<kRows, kThreads>(p, S.cut, S.last, nullptr);
    pdl_launch_dependents();
}

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
    // the counters, and two partial records a CTA (one CTA per SM)
    return kMaxCtas * sizeof(int) + static_cast<size_t>(2) * std::min(num_sms, kMaxCtas) * rec_floats(kMaxRows) * sizeof(float);
}

cudaError_t launch_attention_paged(const PagedAttentionLaunch &A, cudaStream_t s, const char **why) {
    AttnParams p;
    p.v = paged_view(A.batch, A.cache);
    p.q = A.q;
    p.ldq = A.ldq;
    p.Hq = A.Hq;
    p.GQ = A.Hq / A.cache.Hkv;
    p.by_gq = fast_div(p.GQ);
    p.window = std::min(A.window, 1 << 30);  // positions minus a window stay in 32 bits
    p.sinks = std::min(A.sinks, 1 << 30);
    p.scale_log2 = A.scale * 1.4426950408889634f;
    p.out = A.out;
    p.ldo = A.ldo;
    p.counters = reinterpret_cast<int *>(A.workspace);
    p.part = A.workspace + kMaxCtas;
    CacheMaps maps;
    const uint64_t cache_rows = static_cast<uint64_t>(A.cache.n_pages) * A.cache.Hkv * A.cache.page_size;
    // boxes of more blocks than the cache holds are never used, and not made
    for (int i = 0; i < (A.cache.kind == TERN_KV_INT8 ? 4 : 1); ++i) {
        const uint32_t box = static_cast<uint32_t>(std::min<uint64_t>(kPB << i, cache_rows));
        if (!make_u8_tmap_2d(&maps.k[i], A.cache.k_codes, kPD, cache_rows, kPD, kPD, box) ||
            !make_u8_tmap_2d(&maps.v[i], A.cache.v_codes, kPD, cache_rows, kPD, kPD, box)) {
            *why = "cuTensorMapEncodeTiled failed or is unavailable";
            return cudaErrorInvalidValue;
        }
    }
    const int64_t span = A.window > 0 ? std::min<int64_t>(A.batch.max_ctx, static_cast<int64_t>(A.window) + A.sinks + 32)
                                      : A.batch.max_ctx;
    const int64_t rows = std::min<int64_t>(static_cast<int64_t>(std::min(A.batch.max_rows, A.batch.T)) * p.GQ, 1 << 30);
    if (A.cache.kind == TERN_KV_INT8)
        return launch_attention_tc(p, maps, static_cast<int>(rows), span, A.num_sms, s);
    // one CTA per SM, fewer when the tiles are few
    const int64_t units = std::min<int64_t>(A.batch.B, A.batch.T) * A.cache.Hkv * ceil_div(rows, kRows) * ceil_div(span, kPB);
    int64_t ctas = std::min<int64_t>(A.num_sms, ceil_div(units, kWarps));
    ctas = std::max<int64_t>(1, std::min<int64_t>(ctas, kMaxCtas));
    return launch_split<TERN_KV_E4M3>(p, maps.k[0], maps.v[0], static_cast<int>(ctas), s);
}

}  // namespace tern
