// tern_paged_attention.cu -- attention over the paged 8-bit KV cache on the
// 5th-generation tensor cores, the codes used as they lie.
//
// out = sum_j softmax_j(scale q . k_j) v_j, one pass over the tokens with the
// running maximum m and sum z of the softmax.  Both products are matrix
// products of the 8-bit codes with an fp32 operand written as 8-bit digits, so
// no code is ever converted:
//   S^T[token][row] = K[token][d] . Q[row][d]^T
//   O^T[d][row]     = V[token][d]^T . P[token][row]
// with 128 tokens (of S) and 128 dimensions (of O) as the 128 accumulator
// lanes.  K is the A operand as TMA brings it (tokens x 128 bytes, K-major,
// 128-byte swizzle), V the same bytes read the other way (M-major).
// int8 codes (tcgen05.mma kind::i8, exact int32 sums):
//  * A query row is scaled by a power of two to 23 bits and split into three
//    signed 8-bit digits, q = d2 2^16 + d1 2^8 + d0 (error at most 2^-22.9 of the
//    row's largest element): three columns of the B operand per row.  A digit's
//    product is an exact int32 of at most 2^21.
//  * A softmax weight times its block's value scale, relative to the row's
//    reference, is an unsigned 32-bit fixed-point number, and its four bytes are
//    four unsigned digits: the word is stored as it is, four columns per row.
//    The sums over tokens are exact int32, so they stay in tensor memory from
//    tile to tile.
// e4m3 codes (kind::f8f6f4, fp32 sums):
//  * A query row is scaled below 2^8 and each element written as five e4m3
//    digits, x = d0 + (d1 + (d2 + ...) / 16) / 16, each the nearest to what is
//    left: a digit is off by 2^-4 of it, so the five by 2^-20 of the element.
//  * A softmax weight times its block's value scale, relative to the row's
//    reference below 2^8 (2^2 for a new reference's largest), likewise: off by
//    2^-20 of itself or, where the digits' subnormals begin, 2^-26.
//    The fp32 sums stay in tensor memory for at most 16 tiles.
//  A weight of 0 does not undo a NaN code: value rows that some query row does
//  not see (the rest of a block may hold anything) lose theirs in shared memory.
// References: the digits hold the product 2^y of a row's weight and the token's
// value scale, y = score + log2(scale) (its exponent, relative to that of the
// item; the mantissa is multiplied on), as 2^(y - m_r) with m_r at least the
// largest y so far, and z sums 2^(y - m_r) / scale.  When a tile has a larger y,
// or a chain of sums ends, the sums are read, added to fp32 registers and begun
// again.  m_r is set six above the largest y, so that happens a few times per
// item (26 of int8's 32 bits remain).
// With weights and scales held by references of their own, a first token of a
// large weight and a small value (what sinks are kept for) set both against
// itself, and weights below 2^-27 of the one or scales' share of the other were
// lost: at 65536 tokens and a value scale of 1/64, 2.3e-5 of the output (normal
// scores, the first 2^24 above the largest), by a model up to 6.6e-3 (all others
// 2^27.5 below).  So a reference
// may fall as well: new references are taken from the present tile, wherever
// that one's largest y lies 12 or more below the one that set m_r; and they are
// taken behind a y that stands 12 above what came before it or above another 32
// tokens of its tile, and when a chain ends.  (A test of every eighth tile cost
// prompts 12 %.)  The error is then below that of plain fp32 on such inputs too.
//
// One CTA per SM.  Warps of their own look the tiles up, copy K, copy V, issue
// QK, issue PV and make the query digits: a thread takes some 450 cycles to
// issue a product, and look-up and K's copies in one warp took 1570 cycles a
// tile of 16-token pages, more than the 1430 in which memory delivers it (24
// ragged sequences 114 us; with a warp for each 98).  With 32 rows one warp
// looks up and copies, which leaves 96 registers a thread.  Two softmax groups
// (thread = token of S, dimension of O; with 32 rows each group is two
// warpgroups of 16) take the tiles in turn, each with its own accumulators,
// references and weight buffer, so that one group's waits, fences and barriers
// pass under the other's arithmetic; what they have of an item is put together
// at its end.  A tile is eight visible blocks of 16 tokens of an item, from
// anywhere in the sequence, so sinks and a window fill whole tiles.  Everything
// runs ahead across items: K and V by rings of their own (a K stage is free
// after QK, a V stage after PV), QK of the next tiles before PV of this one, the
// next item's digits while this one's tiles are worked off.
//
// Measured (device time; the floor is the codes at the measured copy rate): 24
// sequences of up to 20011 tokens, 40 heads on 8, 98 us of 86 (int8 103; 16-token
// pages); one of 65536 35 of 20.5, of 4096 13 of 1.3 (some 8 us are launch,
// look-up and the merging of divided items); 16 sequences of which a window and
// sinks show 4100 tokens 35 of 20.6; three sequences of 16 drafted tokens 60 of
// 8.0 (e4m3 66) and a prompt's 2048 rows of 4096 tokens 525 of 79 (e4m3 1000):
// there some 20 instructions an element of the softmax, and the ends of items.
// All the loops together fill the instruction cache; a few hundred bytes more in
// one of them have cost 5 to 25 %.
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <float.h>

#include <algorithm>

#include "tern_paged_attention.cuh"
#include "tern_tc.cuh"

namespace tern {

namespace {

constexpr int kTok = kTB * kPB;           // 128 tokens
constexpr int kTileBytes = kTok * kPD;    // 16 KB of K or V codes
constexpr int kInfo = 16;                 // tile infos kept: the copies want at most kStages + kSBufs + 2 tiles ahead of the softmax
constexpr int kItems = 16;                // items kept for the query warp, and whose score scales are kept.  (Tile t's item, which
                                          // may be item t, is noted before the scales of t - 11 are: at least 10, or the
                                          // look-up waits for digits that wait for it)
constexpr float kHeadroom = 6.0f;         // a new reference lies this far (log2) above the largest score
constexpr int kChainInt8 = 32;            // tiles summed in int32, at most 256: 256 * 128 * 255 * 127 < 2^31
constexpr int kChainE4m3 = 16;            // tiles summed in fp32 inside the tensor cores (16 or 64: the same time)
constexpr float kFallBelow = 18.0f;       // a reference this far above a tile's largest product falls (12 below what set it)
constexpr float kLowest = 48.0f;          // how far references may fall below the highest
constexpr float kLowestAtOnce = 64.0f;    // and at once: tokens of far smaller value scales, as blocks of zeros have, may have set one
constexpr int kScaleRange = 24;           // largest block scale of a tile (log2), relative to the item's
constexpr int kScaleLowest = -30;         // least block scale that a reference is told apart by

template <int R, int KIND>
struct Shape {
    static constexpr bool kInt = KIND == TERN_KV_INT8;
    static constexpr int kHalves = R == 32 ? 2 : 1;   // warpgroups of a softmax group
    static constexpr int kRW = R / kHalves;           // rows of each
    static constexpr int kHelpers = R == 32 ? 4 : 8;  // warps in front of the softmax warps
    static constexpr int kThreads = 32 * kHelpers + 2 * kHalves * 128;
    static constexpr int kGroup = 128 * kHalves;      // threads of a softmax group
    // warps: look-up of the tiles (with 4 helpers their copies too), copies of K, of V, issue of QK, of PV, query digits
    static constexpr bool kCopyWarps = kHelpers == 8;
    static constexpr int kWarpLook = 0, kWarpK = kCopyWarps ? 1 : -1, kWarpV = kCopyWarps ? 2 : -1,
                         kWarpQK = kCopyWarps ? 3 : 1, kWarpPV = kCopyWarps ? 4 : 2, kWarpQ = kCopyWarps ? 5 : 3;
    static constexpr int kQWarps = kCopyWarps ? 3 : 1;  // from kWarpQ on
    static constexpr int kSBufs = R == 32 ? 2 : 4;    // S accumulators
    static constexpr int kQD = kInt ? 3 : 5;          // digits of a query, columns of S per row
    static constexpr int kVD = kInt ? 4 : 5;         // digits of a weight, columns of O per row
    static constexpr int kNS = (kQD * R + 15) / 16 * 16;
    static constexpr int kNP = (kVD * R + 15) / 16 * 16;
    static constexpr int kPRow = kNP == 32 ? 32 : 128;  // bytes of a token's row of weight digits
    static constexpr int kStages = R == 32 ? 3 : kInt && R == 8 ? 6 : 5;    // of K
    static constexpr int kVStages = R == 32 || R == 16 ? 4 : kInt ? 6 : 5;  // of V (held longer: until PV)
    static constexpr int kQBytes = kNS * 128;
    static constexpr int kPBytes = kTok * kPRow;      // (also holds a group's own R x 128 sums at the end of an item)
    static constexpr int kSumBytes = R * kPD * 4;     // the sums that one group hands to the other
    static constexpr uint32_t kO = kSBufs * kNS;      // first column of O
    static constexpr uint32_t kTmemCols = kSBufs * kNS + 2 * kNP <= 256 ? 256 : 512;
    static_assert(kSBufs * kNS + 2 * kNP <= kTmemCols && kSumBytes <= kPBytes, "tensor memory; sums in the weight buffer");
    static_assert(kQBytes % 1024 == 0 && kPBytes % 1024 == 0, "operand tiles begin on 1024 bytes");
};

// One tile, as the softmax and MMA warps see it.
struct TileInfo {
    float ks[kTB], vm[kTB];
    int ve[kTB];      // value scales: 2^ve times vm, which is in (1/2, 1] (0: no scale) times what a weight of 1 is held as
    int j0[kTB];      // first token of each block
    int row[kTB];     // its first code row, for the block that begins a copy
    int size[kTB];    // log2 of the blocks that this copy takes, -1: none begins here
    int valid;        // bit j: block j is there
    int flags;
    int vtop;         // largest ve
    int head, rt, k, units, ord;
    Seq s;
};
// An item, as the query warp sees it.
struct ItemInfo {
    int head, rt;
    int tiles;        // of this CTA
    Seq s;
};
enum : int {
    kFirst = 1,       // the first tile of its item in this CTA
    kLast = 2,        // the last
    kGroupFirst = 4,  // the first of its item that its group has here
    kGroupLast = 8,   // the last
    kBoth = 16,       // both groups have tiles of the item
    kEdge = 32,       // masks needed
    kEnds = 64,       // the item's last tile
};

template <int R, int KIND>
struct AttnShared {
    using Sh = Shape<R, KIND>;
    TileInfo info[kInfo];
    ItemInfo item[kItems], first_item;
    float4 rowf[kItems][R / 4];        // score scale of each row's digits
    float4 m[2][R / 4], top[2][R / 4];  // each group's references, and the highest they have been
    float4 back[2][R / 4];            // what new references make of the sums before
    float wmax[2][4][R];
    float zsum[2][4][R];
    float sum_m[R], sum_z[R];         // references and sums of the part of an item that a group hands to the other
    float2 factors[2][R];             // of the parts at an item's end
    LineShared line;
    uint64_t k_full[Sh::kStages], k_empty[Sh::kStages], v_full[Sh::kVStages], v_empty[Sh::kVStages];
    uint64_t info_full[kInfo], scales_full[kInfo], info_empty[kInfo], item_full[kItems], item_empty[kItems];
    uint64_t s_full[Sh::kSBufs], s_empty[Sh::kSBufs], p_full[2], p_empty[2], q_full[2], q_empty[2], sum_full, sum_empty;
    CutItem cut[2];
    uint32_t tmem;
    int accumulate[2];
    int last[2];
};

template <int R, int KIND>
constexpr size_t attn_smem() {
    using Sh = Shape<R, KIND>;
    return (Sh::kStages + Sh::kVStages) * kTileBytes + 2 * Sh::kPBytes + 2 * Sh::kQBytes + Sh::kSumBytes +
           sizeof(AttnShared<R, KIND>) + 1024;
}
static_assert(attn_smem<8, TERN_KV_INT8>() <= 227 * 1024 && attn_smem<16, TERN_KV_INT8>() <= 227 * 1024 &&
                  attn_smem<32, TERN_KV_INT8>() <= 227 * 1024 &&
                  attn_smem<8, TERN_KV_E4M3>() <= 227 * 1024 && attn_smem<16, TERN_KV_E4M3>() <= 227 * 1024,
              "shared memory of one CTA");

// B operand descriptor of the weight digits, N-major: a token's row of ROW
// bytes, 128 (128-byte swizzle, layout 2) or 32 (32-byte swizzle, layout 6:
// 16-byte chunk c of row k stored at c ^ (k / 4 % 2)), groups of 8 tokens 8 rows apart.
template <int ROW>
__device__ __forceinline__ uint64_t weights_desc(uint32_t saddr) {
    if constexpr (ROW == 32)
        return static_cast<uint64_t>((saddr >> 4) & 0x3FFFu) | (1ull << 16) | (static_cast<uint64_t>(256u >> 4) << 32) |
               (1ull << 46) | (6ull << 61);
    return smem_desc_sw128(saddr);
}
template <int ROW>
__device__ __forceinline__ int weights_chunk(int c, int k) {
    return ROW == 32 ? c ^ (k >> 2 & 1) : c ^ (k & 7);
}

// Two values as their next e4m3 digits (two bytes), and what is left of them,
// times 16 (|x| <= 256; a digit is off by at most 2^-4 of the value).
__device__ __forceinline__ uint32_t e4m3_digit(float2 &x) {
    const __nv_fp8x2_storage_t d = __nv_cvt_float2_to_fp8x2(x, __NV_SATFINITE, __NV_E4M3);
    const float2 f = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2(d, __NV_E4M3)));
    x = __fmul2_rn(__fadd2_rn(x, make_float2(-f.x, -f.y)), make_float2(16.0f, 16.0f));
    return d;
}

// Waits.  One that runs out records the device error, and its thread waits no
// more.  What a wait would have handed over (a tile's info, an item, a product)
// is then not used for an address, a copy or a product: each warp of one role,
// and each softmax group as a whole, leaves its loop, and waits once more for
// the copies or products that it has in flight.  Those that wait for it run out
// in turn, so the CTA ends, its tensor memory is given back, and its rows may
// hold anything.
__constant__ long long c_wait_budget = kWaitBudgetCycles;  // (a test shortens it)
__device__ __noinline__ bool wait_slow(uint64_t *bar, uint32_t parity) { return mbar_wait_bounded(bar, parity, c_wait_budget); }
__device__ __forceinline__ void wait(uint64_t *bar, uint32_t parity, bool &ok) {
    if (ok && !mbar_try_wait(bar, parity)) ok = wait_slow(bar, parity);
}
// The same, polled in line: what 16 warps wait for in the kernel's largest loop is better not waited for in another place
// of the code (16 and 32 rows, a prompt of e4m3 1013 -> 989 us, 24 sequences of 80 heads on 8 133 -> 122; elsewhere, or of
// 8 rows, the longer code costs more than that).
__device__ __forceinline__ void wait_in_line(uint64_t *bar, uint32_t parity, bool &ok) {
    const long long start = clock64();
    while (ok && !mbar_try_wait(bar, parity)) {
        __nanosleep(kWaitBackoffNs);
        if (clock64() - start > c_wait_budget) {
            atomicExch(&g_device_error, kErrTmaTimeout);
            ok = false;
        }
    }
}
// The wait for what a warp has in flight, which needs no other warp to end.
__device__ __noinline__ bool land(uint64_t *bar, uint32_t parity) { return mbar_wait_bounded(bar, parity); }
// Whether no lane's wait has run out (warp-collective).
__device__ __forceinline__ bool all_ok(bool ok) { return __all_sync(0xffffffffu, ok); }

// An int32 of at most 22 bits as fp32, exactly, without the conversion unit.
__device__ __forceinline__ float small_int(uint32_t c) {
    return __uint_as_float(c + 0x4B400000u) - 12582912.0f;
}

// 2^e, -127 < e < 128; 0 below.
__device__ __forceinline__ float exp2i(int e) { return __uint_as_float(static_cast<uint32_t>(max(127 + e, 0)) << 23); }

__device__ __forceinline__ uint32_t to_u32_sat(float x) {
    uint32_t u;
    asm("cvt.rni.u32.f32 %0, %1;" : "=r"(u) : "f"(x));
    return u;
}

__device__ __forceinline__ float redux_max(float x) {
    float y;
    asm("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(y) : "f"(x));
    return y;
}

// Whether a tile whose largest value scale is 2^vtop needs another value
// reference than 2^lref.
__device__ __forceinline__ bool other_scale(int vtop, int lref) {
    return vtop > -127 && static_cast<unsigned>(vtop - lref + kScaleRange) > 2 * kScaleRange;
}

// Barrier over the N threads of softmax group g, with the "or" of x.
template <int N>
__device__ __forceinline__ bool any_of(bool x, int g) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 p, %1, 0;\n\t"
        "barrier.cta.red.or.pred q, %2, %3, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"(static_cast<uint32_t>(x)), "r"(1 + g), "n"(N)
        : "memory");
    return r != 0;
}

// Sums of each z[r] over the warp; lane l ends up with that of row l % R.
template <int R>
__device__ __forceinline__ float sum_rows(float (&z)[R], int lane) {
#pragma unroll
    for (int h = R / 2; h >= 1; h >>= 1) {
        const bool up = (lane & h) != 0;
#pragma unroll
        for (int j = 0; j < h; ++j) {
            const float other = __shfl_xor_sync(0xffffffffu, up ? z[j] : z[j + h], h);
            z[j] = (up ? z[j + h] : z[j]) + other;
        }
    }
#pragma unroll
    for (int h = R; h < 32; h <<= 1) z[0] += __shfl_xor_sync(0xffffffffu, z[0], h);
    return z[0];
}

// Adds what PV has summed to o, times the value reference: of int8, four digit
// columns a row, of value 2^(8 k - 32); of e4m3, R columns a digit, of value
// 2^(-8 - 4 k).
template <int R, int KIND>
__device__ __forceinline__ void add_sums(uint32_t taddr, float vref, float (&o)[Shape<R, KIND>::kRW]) {
    constexpr int RW = Shape<R, KIND>::kRW;
    if constexpr (KIND == TERN_KV_INT8) {
#pragma unroll
        for (int h = 0; h < RW / 8; ++h) {
            uint32_t ov[32];
            tmem_ld32(taddr + 32 * h, ov);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                float t = static_cast<float>(static_cast<int>(ov[4 * e])) * 0x1p-32f;
                t = fmaf(static_cast<float>(static_cast<int>(ov[4 * e + 1])), 0x1p-24f, t);
                t = fmaf(static_cast<float>(static_cast<int>(ov[4 * e + 2])), 0x1p-16f, t);
                t = fmaf(static_cast<float>(static_cast<int>(ov[4 * e + 3])), 0x1p-8f, t);
                o[8 * h + e] = fmaf(t, vref, o[8 * h + e]);
            }
        }
    } else {
#pragma unroll
        for (int h = 0; h < RW / 8; ++h) {
            uint32_t ov[5][8];
#pragma unroll
            for (int k = 0; k < 5; ++k) tmem_ld8(taddr + R * k + 8 * h, ov[k]);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                float t = 0.0f;
#pragma unroll
                for (int k = 4; k >= 0; --k) t = fmaf(t, 0.0625f, __uint_as_float(ov[k][e]));
                o[8 * h + e] = fmaf(t, vref * 0x1p-8f, o[8 * h + e]);
            }
        }
    }
}

// Copies of tile i's keys, or values, by its info; lanes 0-7 a block each.
// False when a wait ran out, here or before: nothing is copied.
template <int R, int KIND, bool K>
__device__ __forceinline__ bool copy_tile(const CacheMaps &maps, AttnShared<R, KIND> &S, uint8_t *ring, int i, bool &ok) {
    constexpr int kSt = K ? Shape<R, KIND>::kStages : Shape<R, KIND>::kVStages;
    const int lane = threadIdx.x & 31, stage = i % kSt;
    uint64_t *full = K ? &S.k_full[stage] : &S.v_full[stage];
    const TileInfo &f = S.info[i % kInfo];
    const int size = lane < kTB ? f.size[lane] : -1, row = lane < kTB ? f.row[lane] : 0;
    const uint32_t bytes = __popc(f.valid) * kPB * kPD;
    wait(K ? &S.k_empty[stage] : &S.v_empty[stage], ((i / kSt) + 1) & 1, ok);
    if (!all_ok(ok)) return false;
    if (lane == 0) {
        mbar_arrive_expect_tx(full, bytes);
        if (!K) mbar_arrive(&S.info_empty[i % kInfo]);  // (the softmax is done with a tile only after K's copy)
    }
    __syncwarp();
    if (size >= 0)
        tma_load_2d_nohint(ring + stage * kTileBytes + lane * kPB * kPD, K ? &maps.k[size] : &maps.v[size], 0, row, full);
    return true;
}

// Before a warp that copied n tiles ends: none of its copies is in flight.
template <int R, int KIND, bool K>
__device__ __forceinline__ void copies_land(AttnShared<R, KIND> &S, int n) {
    constexpr int kSt = K ? Shape<R, KIND>::kStages : Shape<R, KIND>::kVStages;
#pragma unroll 1
    for (int i = max(0, n - kSt); i < n; ++i)
        if (!land(K ? &S.k_full[i % kSt] : &S.v_full[i % kSt], (i / kSt) & 1)) break;
}

// All copies of K, or of V.
template <int R, int KIND, bool K>
__device__ __forceinline__ void copy_codes(const CacheMaps &maps, AttnShared<R, KIND> &S, uint8_t *ring, int count) {
    bool ok = true;
    int n = 0;
#pragma unroll 1
    for (; n < count; ++n) {
        wait(&S.info_full[n % kInfo], (n / kInfo) & 1, ok);
        if (!copy_tile<R, KIND, K>(maps, S, ring, n, ok)) break;
    }
    copies_land<R, KIND, K>(S, n);
}

// (Out of line: with at most kLineThreads sequences they are in shared memory.)
__device__ __noinline__ Seq far_sequence(const AttnParams &p, int b) { return sequence(p, b); }

// Look-up of a range's tiles: writes the infos of the items and tiles.  Four
// tiles at a time (lane = 8 * tile + block), in three steps that overlap, so
// that no load is waited for while another could be on its way: page numbers;
// places and masks, which the copies start from, and loads of the scales; the
// scales, and then, without warps for them, the copies.
template <int R, int KIND, typename SeqOf>
__device__ __forceinline__ void look_up(const AttnParams &p, const CacheMaps &maps, AttnShared<R, KIND> &S, uint8_t *kring,
                                        uint8_t *vring, const Line &L, const Ranges &ranges, long long u0, int count,
                                        SeqOf seq_of) {
    const PagedView &v = p.v;
    const int lane = threadIdx.x & 31, sub = lane >> 3, j = lane & 7;
    bool ok = true;
    Cursor cur = find_place<R>(p, S.line, L, u0, seq_of);
    const int k_first = cur.k;
    if (lane == 0) S.first_item = {cur.head, cur.rt, cur.units(), cur.s};
    int step = sub, page = -1, in_page = 0, j0 = 0;
    int nk = 0, nv = 0;  // tiles whose K, V are copied here
    float ks = 0.0f, vs = 0.0f;
    int i0 = 0;
#pragma unroll 1
    for (; i0 < count + 8; i0 += 4) {
        const Cursor it = cur;
        const int page_now = page, in_page_now = in_page, j0_now = j0;
        const float ks_now = ks, vs_now = vs;
        // ---- tiles i0 ..: page numbers
        page = -1;
        if (i0 + sub < count) {
            advance<R>(p, cur, step, seq_of);
            step = 4;
            if (j == 0 && (cur.k == 0 || i0 + sub == 0)) {
                const int slot = cur.ord % kItems;
                wait(&S.item_empty[slot], ((cur.ord / kItems) + 1) & 1, ok);
                if (ok) {
                    S.item[slot].head = cur.head;
                    S.item[slot].rt = cur.rt;
                    S.item[slot].tiles = min(cur.units() - cur.k, count - i0 - sub);
                    S.item[slot].s = cur.s;
                    mbar_arrive(&S.item_full[slot]);
                }
            }
            const int kb = kTB * cur.k + j;
            if (kb < cur.tl.n) {
                const int blk = cur.tl.block(kb), e = v.by_bpp.quot(blk);
                j0 = blk * kPB;
                in_page = blk - e * v.bpp;
                if (e < v.pages_ld) page = v.pages[static_cast<int64_t>(cur.b) * v.pages_ld + e];
            }
        }
        __syncwarp();
        // ---- tiles i0 - 4 ..: places and masks
        if (i0 >= 4) {
            const int i = i0 - 4 + sub;
            const int bi = page_now >= 0 && page_now < v.n_pages ? (page_now * v.Hkv + it.head) * v.bpp + in_page_now : -1;
            ks = vs = 0.0f;
            if (bi >= 0) {
                ks = v.ks[bi];
                vs = v.vs[bi];
            }
            const unsigned there = __ballot_sync(0xffffffffu, bi >= 0) >> (8 * sub) & 255;
            // runs of blocks that lie behind one another in the cache: one copy each for 8, 4, 2 or 1 of them
            // (copies of 16 rows: 2150 cycles a tile, of 64 rows 1690)
            const int before = __shfl_up_sync(0xffffffffu, bi, 1);
            const unsigned follows = __ballot_sync(0xffffffffu, continues_block(before, bi)) >> (8 * sub) & 255;
            const int size = copy_size(follows, j, bi);
            // masks: a block whose tokens not every row sees, or that is missing
            const int p_min = it.s.first + p.by_gq.quot(R * it.rt);
            const int p_max = it.s.first + p.by_gq.quot(min(R * it.rt + R, it.s.rows) - 1);
            const bool whole = bi >= 0 && j0_now + kPB - 1 <= p_min &&
                               (p.window == 0 || j0_now > p_max - p.window || j0_now + kPB <= p.sinks);
            const unsigned not_whole = __ballot_sync(0xffffffffu, !whole) >> (8 * sub) & 255;
            if (i < count) wait(&S.info_empty[i % kInfo], ((i / kInfo) + 1) & 1, ok);
            if (!all_ok(ok)) break;
            if (i < count) {
                TileInfo &f = S.info[i % kInfo];
                f.j0[j] = j0_now;
                f.row[j] = bi * kPB;
                f.size[j] = size;
                if (j == 0) {
                    const int since = min(it.k, i), left = min(it.units() - 1 - it.k, count - 1 - i);
                    f.valid = there;
                    f.flags = (since == 0 ? kFirst : 0) | (left == 0 ? kLast : 0) | (since < 2 ? kGroupFirst : 0) |
                              (left < 2 ? kGroupLast : 0) | (since + left > 0 ? kBoth : 0) | (not_whole ? kEdge : 0) |
                              (it.k + 1 == it.units() ? kEnds : 0);
                    f.head = it.head;
                    f.rt = it.rt;
                    f.k = it.k;
                    f.units = it.units();
                    f.ord = it.ord;
                    f.s = it.s;
                }
            }
            __syncwarp();
            if (j == 0 && i < count) mbar_arrive(&S.info_full[i % kInfo]);
        }
        // ---- tiles i0 - 8 ..: scales
        if (i0 >= 8) {
            const int i = i0 - 8 + sub;
            // the exponent rounded up; of no scale (0), and of subnormal ones, -127
            const int ve = min(127, static_cast<int>((__float_as_uint(vs_now) + 0x7FFFFFu) >> 23) - 127);
            int vtop = ve;
#pragma unroll
            for (int o = 1; o < 8; o <<= 1) vtop = max(vtop, __shfl_xor_sync(0xffffffffu, vtop, o));
            if (i < count) {
                TileInfo &f = S.info[i % kInfo];
                f.ks[j] = ks_now;
                f.vm[j] = vs_now * exp2i(-ve) * (Shape<R, KIND>::kInt ? 0x1p32f : 0x1p8f);
                f.ve[j] = ve;
                if (j == 0) f.vtop = vtop;
            }
            __syncwarp();
            if (j == 0 && i < count) mbar_arrive(&S.scales_full[i % kInfo]);
            if constexpr (!Shape<R, KIND>::kCopyWarps) {
#pragma unroll 1
                for (int e = i0 - 8; e < min(i0 - 4, count); ++e) {
                    if (!copy_tile<R, KIND, true>(maps, S, kring, e, ok)) break;
                    ++nk;
                    if (!copy_tile<R, KIND, false>(maps, S, vring, e, ok)) break;
                    ++nv;
                }
                ok = all_ok(ok);  // (then the next step's vote ends the loop)
            }
        }
    }
    // the items that other CTAs have parts of
    if (lane == 0 && k_first > 0) {
        const ItemInfo &it = S.first_item;
        note_cut(S.cut[0], ranges, it.head, it.rt, it.s, u0 - k_first, it.tiles);
    }
    // (the last tile's item, as the lane that looked it up has it: cut if it goes on and began in this range)
    if (i0 >= count + 8 && j == 0 && sub == (count - 1) % 4 && cur.k + 1 < cur.units() && cur.k <= count - 1)
        note_cut(S.cut[1], ranges, cur.head, cur.rt, cur.s, u0 + count - 1 - cur.k, cur.units());
    if constexpr (!Shape<R, KIND>::kCopyWarps) {
        copies_land<R, KIND, true>(S, nk);
        copies_land<R, KIND, false>(S, nv);
    }
}

template <int KIND>
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    if constexpr (KIND == TERN_KV_INT8)
        mma_i8_ss(d, a, b, idesc, accumulate);
    else
        mma_e4m3_ss(d, a, b, idesc, accumulate);
}

template <int R, int KIND>
__global__ void __launch_bounds__(Shape<R, KIND>::kThreads, 1)
    attn_paged_kernel(const __grid_constant__ AttnParams p, const __grid_constant__ CacheMaps maps) {
    using Sh = Shape<R, KIND>;
    constexpr bool kInt = Sh::kInt;
    constexpr int kSt = Sh::kStages, kRW = Sh::kRW, kGroup = Sh::kGroup;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *kring = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
    uint8_t *vring = kring + kSt * kTileBytes;
    uint8_t *pbuf = vring + Sh::kVStages * kTileBytes;
    uint8_t *qbuf = pbuf + 2 * Sh::kPBytes;
    float *handed = reinterpret_cast<float *>(qbuf + 2 * Sh::kQBytes);
    AttnShared<R, KIND> &S = *reinterpret_cast<AttnShared<R, KIND> *>(qbuf + 2 * Sh::kQBytes + Sh::kSumBytes);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int c = blockIdx.x;
    bool ok = true;

    if (tid == 0) {
        for (int i = 0; i < 4; ++i) {
            prefetch_tmap(&maps.k[i]);
            prefetch_tmap(&maps.v[i]);
        }
        for (int i = 0; i < kSt; ++i) {
            mbar_init(&S.k_full[i], 1);
            mbar_init(&S.k_empty[i], 1);
        }
        for (int i = 0; i < Sh::kVStages; ++i) {
            mbar_init(&S.v_full[i], 1);
            mbar_init(&S.v_empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&S.p_full[i], 4 * Sh::kHalves);
            mbar_init(&S.p_empty[i], 1);
            mbar_init(&S.q_full[i], Sh::kQWarps);
            mbar_init(&S.q_empty[i], 1);
            S.cut[i].valid = 0;
        }
        mbar_init(&S.sum_full, 4 * Sh::kHalves);
        mbar_init(&S.sum_empty, 4 * Sh::kHalves);
        for (int i = 0; i < kInfo; ++i) {
            mbar_init(&S.info_full[i], 1);
            mbar_init(&S.scales_full[i], 1);
            mbar_init(&S.info_empty[i], 4 * Sh::kHalves + 1);
        }
        for (int i = 0; i < kItems; ++i) {
            mbar_init(&S.item_full[i], 1);
            mbar_init(&S.item_empty[i], Sh::kQWarps);
        }
        for (int i = 0; i < Sh::kSBufs; ++i) {
            mbar_init(&S.s_full[i], 2);
            mbar_init(&S.s_empty[i], 4 * Sh::kHalves);
        }
        fence_mbar_init();
    }
    if (warp == Sh::kWarpQK) {
        tmem_alloc(&S.tmem, Sh::kTmemCols);
        tmem_relinquish();
    }
    pdl_wait();
    tc_fence_before_sync();
    const Line L = make_line<R>(p, S.line);
    tc_fence_after_sync();
    const int G = static_cast<int>(min(static_cast<long long>(gridDim.x), L.total));
    Ranges ranges = {0, 0};
    if (L.total > 0) {
        ranges.base = quot(L.total, G);
        ranges.more = L.total - ranges.base * G;
    }
    const long long u0 = c < G ? ranges.begin(c) : 0;
    const int count = c < G ? static_cast<int>(ranges.begin(c + 1) - u0) : 0;
    const uint32_t tmem = S.tmem;

    if (count == 0) {
    } else if (warp == Sh::kWarpLook) {
        look_up<R, KIND>(p, maps, S, kring, vring, L, ranges, u0, count,
                         [&](int b) { return L.per == 1 ? S.line.seq[b] : far_sequence(p, b); });
    } else if (warp == Sh::kWarpK) {
        copy_codes<R, KIND, true>(maps, S, kring, count);
    } else if (warp == Sh::kWarpV) {
        copy_codes<R, KIND, false>(maps, S, vring, count);
    } else if (warp == Sh::kWarpQK) {
        // ---- S of each tile, as soon as its keys are there and its accumulator has been read
        if (lane == 0) {
            constexpr uint32_t id_s = kInt ? idesc_i8(128, Sh::kNS, 1, 1) : idesc_e4m3(128, Sh::kNS);
            int item = -1, i = 0, asked = -1;  // asked: the last item whose last tile was issued
#pragma unroll 1
            for (; i < count; ++i) {
                const int stage = i % kSt, buf = i % Sh::kSBufs;
                wait(&S.k_full[stage], (i / kSt) & 1, ok);
                wait(&S.scales_full[i % kInfo], (i / kInfo) & 1, ok);
                if (!ok) break;
                const int flags = S.info[i % kInfo].flags;
                if (flags & kFirst) {
                    ++item;
                    wait(&S.q_full[item & 1], (item >> 1) & 1, ok);
                }
                wait(&S.s_empty[buf], ((i / Sh::kSBufs) + 1) & 1, ok);
                if (!ok) break;
                tc_fence_after_sync();
                const uint32_t a = smem_u32(kring + stage * kTileBytes), b = smem_u32(qbuf + (item & 1) * Sh::kQBytes);
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    mma_ss<KIND>(tmem + buf * Sh::kNS, smem_desc_sw128(a + 32 * k), smem_desc_sw128(b + 32 * k), id_s, k > 0);
                tc_commit(&S.s_full[buf]);
                tc_commit(&S.k_empty[stage]);
                if (flags & kLast) {
                    tc_commit(&S.q_empty[item & 1]);
                    asked = item;
                }
                mbar_arrive(&S.s_full[buf]);  // (hands on the tile's info and the rows' scales, which this thread has acquired)
            }
            if (i < count && i > 0) {  // (each arrival that these products make)
                land(&S.s_full[(i - 1) % Sh::kSBufs], ((i - 1) / Sh::kSBufs) & 1);
                land(&S.k_empty[(i - 1) % kSt], ((i - 1) / kSt) & 1);
                if (asked >= 0) land(&S.q_empty[asked & 1], (asked >> 1) & 1);
            }
        }
        __syncwarp();
    } else if (warp == Sh::kWarpPV) {
        // ---- O of each tile, added to its group's sums
        if (lane == 0) {
            constexpr uint32_t id_o = (kInt ? idesc_i8(128, Sh::kNP, 1, 0) : idesc_e4m3(128, Sh::kNP)) | (1u << 15) |
                                      (1u << 16);  // both operands M/N-major
            int i = 0;
#pragma unroll 1
            for (; i < count; ++i) {
                const int stage = i % Sh::kVStages, g = i & 1;
                wait(&S.v_full[stage], (i / Sh::kVStages) & 1, ok);
                wait(&S.p_full[g], (i >> 1) & 1, ok);
                if (!ok) break;
                tc_fence_after_sync();
                const uint32_t a = smem_u32(vring + stage * kTileBytes), b = smem_u32(pbuf + g * Sh::kPBytes);
                const uint32_t acc = S.accumulate[g];
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    mma_ss<KIND>(tmem + Sh::kO + g * Sh::kNP, smem_desc_sw128(a + 4096 * k),
                                 weights_desc<Sh::kPRow>(b + 32 * Sh::kPRow * k), id_o, k > 0 || acc);
                tc_commit(&S.p_empty[g]);
                tc_commit(&S.v_empty[stage]);
            }
            if (i < count && i > 0) {
                land(&S.p_empty[(i - 1) & 1], ((i - 1) >> 1) & 1);
                land(&S.v_empty[(i - 1) % Sh::kVStages], ((i - 1) / Sh::kVStages) & 1);
            }
        }
        __syncwarp();
    } else if (warp >= Sh::kWarpQ && warp < Sh::kWarpQ + Sh::kQWarps) {
        // ---- query digits of each item, ahead of its tiles
#pragma unroll 1
        for (int done = 0, item = 0; done < count; ++item) {
            const int slot = item % kItems;
            wait(&S.item_full[slot], (item / kItems) & 1, ok);
            wait(&S.q_empty[item & 1], ((item >> 1) + 1) & 1, ok);
            if (!all_ok(ok)) break;
            const ItemInfo it = S.item[slot];
            uint8_t *qb = qbuf + (item & 1) * Sh::kQBytes;
            // one or two rows at a time, the next ones on their way (a loop of four rows written out crowds the
            // instruction cache)
            constexpr int kAt = Sh::kQWarps == 1 ? 2 : 1, kStep = kAt * Sh::kQWarps;
            auto load_row = [&](int rr) {
                const int row = R * it.rt + rr, ri = p.by_gq.quot(row);
                if (rr >= R || row >= it.s.rows) return make_float4(0, 0, 0, 0);
                return *reinterpret_cast<const float4 *>(p.q + static_cast<int64_t>(it.s.start + ri) * p.ldq +
                                                         (it.head * p.GQ + row - ri * p.GQ) * kPD + 4 * lane);
            };
            float4 x[kAt], next[2][kAt];
            const int first = kAt * (warp - Sh::kWarpQ);
#pragma unroll
            for (int h = 0; h < kAt; ++h) {
                next[0][h] = load_row(first + h);
                next[1][h] = load_row(first + kStep + h);
            }
#pragma unroll 1
            for (int rr0 = first; rr0 < R; rr0 += kStep) {
#pragma unroll
                for (int h = 0; h < kAt; ++h) {
                    x[h] = next[0][h];
                    next[0][h] = next[1][h];
                    next[1][h] = load_row(rr0 + 2 * kStep + h);
                }
                float up[kAt];
#pragma unroll
                for (int h = 0; h < kAt; ++h) {
                    // (the largest bits: those of a NaN or an infinity lie above all others)
                    const uint32_t amax = __reduce_max_sync(
                        0xffffffffu, max(max(__float_as_uint(fabsf(x[h].x)), __float_as_uint(fabsf(x[h].y))),
                                         max(__float_as_uint(fabsf(x[h].z)), __float_as_uint(fabsf(x[h].w)))));
                    // the row times 2^e: its largest value in (1.984 * 2^21, 1.984 * 2^22], which three signed int8 digits
                    // hold (127 * (2^16 + 2^8 + 1) is 1.992 * 2^22), or in [2^7, 2^8), below the largest e4m3 value
                    const int e = max(-120, min(120, kInt ? 149 - static_cast<int>((amax + 0x1FFFFu) >> 23)
                                                          : 134 - static_cast<int>(amax >> 23)));
                    up[h] = __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
                    if (lane == 0) {
                        float down = R * it.rt + rr0 + h < it.s.rows
                                         ? p.scale_log2 * __uint_as_float(static_cast<uint32_t>(127 - e) << 23)
                                         : 0.0f;
                        if (amax >= 0x7F800000u) down = NAN;  // no digits hold such a row: all its scores are NaN
                        reinterpret_cast<float *>(S.rowf[slot])[rr0 + h] = down;
                    }
                }
#pragma unroll
                for (int h = 0; h < kAt; ++h) {
                    const int rr = rr0 + h;
                    // digit k of the four dimensions as one word; column of digit k of row rr: 2 kQD (rr / 2) + 2 k + rr % 2,
                    // so that two rows' digits are neighbours
                    const float f[4] = {x[h].x * up[h], x[h].y * up[h], x[h].z * up[h], x[h].w * up[h]};
                    uint32_t w[Sh::kQD];
                    if constexpr (kInt) {
                        // (n + 0x8080) ^ 0x8080 has the signed digits d0, d1 as its low bytes, d2 above
                        uint32_t n[4];
#pragma unroll
                        for (int d = 0; d < 4; ++d) n[d] = static_cast<uint32_t>(__float2int_rn(f[d]) + 0x8080) ^ 0x8080u;
                        const uint32_t lo0 = __byte_perm(n[0], n[1], 0x5140), lo1 = __byte_perm(n[2], n[3], 0x5140);
                        const uint32_t hi0 = __byte_perm(n[0], n[1], 0x0062), hi1 = __byte_perm(n[2], n[3], 0x0062);
                        w[0] = __byte_perm(lo0, lo1, 0x5410);
                        w[1] = __byte_perm(lo0, lo1, 0x7632);
                        w[2] = __byte_perm(hi0, hi1, 0x5410);
                    } else {
                        float2 a = make_float2(f[0], f[1]), b = make_float2(f[2], f[3]);
#pragma unroll
                        for (int k = 0; k < Sh::kQD; ++k) {
                            const uint32_t lo = e4m3_digit(a);
                            w[k] = lo | e4m3_digit(b) << 16;
                        }
                    }
#pragma unroll
                    for (int k = 0; k < Sh::kQD; ++k)
                        *reinterpret_cast<uint32_t *>(qb + sw128_offset(2 * Sh::kQD * (rr >> 1) + 2 * k + (rr & 1), 4 * lane)) =
                            w[k];
                }
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&S.q_full[item & 1]);
                mbar_arrive(&S.item_empty[slot]);
            }
            done += it.tiles;
        }
    } else if (warp >= Sh::kHelpers) {
        // ---- softmax group g: tiles g, g + 2, ...; thread = token of the tile and dimension of the output, rows
        // r0 .. r0 + kRW - 1
        const int in = tid - 32 * Sh::kHelpers, g = in / kGroup, gt = in % kGroup, w4 = warp & 3, me = tid & 127;
        const int r0 = kRW * (gt >> 7);
        const uint32_t lanes = static_cast<uint32_t>(w4) << 21;  // this warp's quarter of tensor memory
        const uint32_t ts = tmem + lanes + Sh::kQD * r0, to = tmem + lanes + Sh::kO + g * Sh::kNP + 4 * r0;
        uint8_t *my_p = pbuf + g * Sh::kPBytes;
        float2 z[kRW / 2];
        float o[kRW];
        int lref = 0;   // value reference (log2)
        bool again = false;  // the next tile takes new references, in case they fall
        int chain = 0, k_first = 0;
        int handovers = 0;  // items of which both groups had parts
#pragma unroll 1
        for (int i = g; i < count; i += 2) {
            const TileInfo &f = S.info[i % kInfo];
            const int buf = i % Sh::kSBufs;
            if constexpr (R >= 16)
                wait_in_line(&S.s_full[buf], (i / Sh::kSBufs) & 1, ok);
            else
                wait(&S.s_full[buf], (i / Sh::kSBufs) & 1, ok);
            tc_fence_after_sync();
            const int flags = f.flags;
            if (flags & kGroupFirst) {
                k_first = f.k - ((flags & kFirst) ? 0 : 1);  // the first tile that the CTA has of the item
#pragma unroll
                for (int r = 0; r < kRW; ++r) o[r] = 0.0f;
#pragma unroll
                for (int r = 0; r < kRW / 2; ++r) z[r] = make_float2(0.0f, 0.0f);
                lref = f.vtop;
                if (gt < R)  // (no barrier: whatever the others find in m, they take new references below)
                    reinterpret_cast<float *>(S.m[g])[gt] = reinterpret_cast<float *>(S.top[g])[gt] = -FLT_MAX;
            }
            // scores of this token plus its value scale, in log2: the products that the weights' digits hold
            float x[kRW];
            {
                const float ks = f.ks[me >> 4], lvf = small_int(max(f.ve[me >> 4] - lref, kScaleLowest));
                const float2 ks2 = make_float2(ks, ks), lv2 = make_float2(lvf, lvf);
#pragma unroll
                for (int h = 0; h < kRW / 8; ++h) {
                    uint32_t sv[8 * Sh::kQD];
#pragma unroll
                    for (int e = 0; e < Sh::kQD; ++e)
                        tmem_ld8(ts + buf * Sh::kNS + 8 * Sh::kQD * h + 8 * e, *reinterpret_cast<uint32_t(*)[8]>(sv + 8 * e));
                    tmem_wait_ld();
                    const float4 ra = S.rowf[f.ord & (kItems - 1)][r0 / 4 + 2 * h], rb = S.rowf[f.ord & (kItems - 1)][r0 / 4 + 2 * h + 1];
                    const float2 rf[4] = {make_float2(ra.x, ra.y), make_float2(ra.z, ra.w), make_float2(rb.x, rb.y),
                                          make_float2(rb.z, rb.w)};
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const uint32_t *d = sv + 2 * Sh::kQD * r;
                        float2 t;
                        if constexpr (kInt) {  // (d2 2^8 + d1) 2^8 + d0: the first sum is an integer of at most 2^29 + 2^21, rounded to fp32
                            t = make_float2(static_cast<float>(static_cast<int>(256 * d[4] + d[2])),
                                            static_cast<float>(static_cast<int>(256 * d[5] + d[3])));
                            t = __ffma2_rn(t, make_float2(256.0f, 256.0f), make_float2(small_int(d[0]), small_int(d[1])));
                        } else {  // d0 + (d1 + ...) / 16
                            const float2 down = make_float2(0.0625f, 0.0625f);
                            t = make_float2(__uint_as_float(d[8]), __uint_as_float(d[9]));
#pragma unroll
                            for (int k = 3; k >= 0; --k)
                                t = __ffma2_rn(t, down, make_float2(__uint_as_float(d[2 * k]), __uint_as_float(d[2 * k + 1])));
                        }
                        const float2 s2 = __ffma2_rn(t, __fmul2_rn(rf[r], ks2), lv2);
                        x[8 * h + 2 * r] = s2.x;
                        x[8 * h + 2 * r + 1] = s2.y;
                    }
                }
                tc_fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(&S.s_empty[buf]);
            }
            if (flags & kEdge) {
                const Seq s = f.s;
                const int tok = f.j0[me >> 4] + (me & 15);
                const bool there = f.valid >> (me >> 4) & 1;
#pragma unroll
                for (int r = 0; r < kRW; ++r) {
                    const int pos = s.first + p.by_gq.quot(min(R * f.rt + r0 + r, s.rows - 1));
                    if (!there || tok > pos || (p.window > 0 && tok <= pos - p.window && tok >= p.sinks)) x[r] = -INFINITY;
                }
                if constexpr (!kInt) {
                    // a weight of 0 would not undo a NaN code of a token that not every row sees: its value row is set to 0
                    // where no row sees it (it may hold anything), and loses its NaN codes where some do, whose scores
                    // become NaN instead
                    bool unseen = true, hidden = false;
#pragma unroll
                    for (int r = 0; r < kRW; ++r) {
                        unseen &= x[r] == -INFINITY;
                        hidden |= x[r] == -INFINITY;
                    }
                    const int vs = i % Sh::kVStages;
                    if (hidden) wait(&S.v_full[vs], (i / Sh::kVStages) & 1, ok);
                    if (hidden && ok) {
                        uint4 *vrow = reinterpret_cast<uint4 *>(vring + vs * kTileBytes + me * kPD);
                        uint32_t nan = 0;
#pragma unroll 1
                        for (int k = 0; k < kPD / 16; ++k) {
                            uint4 c = vrow[k];
                            uint32_t *w = &c.x;
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const uint32_t is = unseen ? 0xFFFFFFFFu : __vcmpeq4(w[e] & 0x7F7F7F7Fu, 0x7F7F7F7Fu);
                                w[e] &= ~is;
                                nan |= is;
                            }
                            if (nan) vrow[k] = c;
                        }
                        if (nan)
#pragma unroll
                            for (int r = 0; r < kRW; ++r) x[r] = x[r] == -INFINITY ? x[r] : NAN;
                    }
                }
            }
            bool flush = !ok || again || (flags & kGroupFirst) || chain >= (kInt ? kChainInt8 : kChainE4m3) || other_scale(f.vtop, lref);
#pragma unroll
            for (int h = 0; h < kRW / 4; ++h) {
                const float4 m = S.m[g][r0 / 4 + h];
                flush |= x[4 * h] > m.x || x[4 * h + 1] > m.y || x[4 * h + 2] > m.z || x[4 * h + 3] > m.w;
            }
            if (any_of<kGroup>(flush, g)) {
                // ---- new references: each row's largest product of the tile over all 128 tokens
                const int scale_was = lref;
                if (other_scale(f.vtop, lref)) {  // another value reference from here on
                    lref = f.vtop;
                    const int ve = f.ve[me >> 4];
                    const float by = small_int(max(ve - lref, kScaleLowest) - max(ve - scale_was, kScaleLowest));
#pragma unroll
                    for (int r = 0; r < kRW; ++r) x[r] += by;
                }
#pragma unroll
                for (int r = 0; r < kRW; ++r) {
                    const float y = redux_max(x[r]);
                    if (lane == 0) S.wmax[g][w4][r0 + r] = y;
                }
                // the maxima of all warps are there; the group ends together when a wait of one of its threads has run out
                if (any_of<kGroup>(!ok, g)) break;
                if (chain > 0) {
                    wait(&S.p_empty[g], ((i - 2) >> 1) & 1, ok);  // PV of this group's last tile
                    tc_fence_after_sync();
                    add_sums<R, KIND>(to, exp2i(scale_was), o);
                    tc_fence_before_sync();
                }
                // each row's new reference, and what it makes of the sums so far
                bool far = false;
                if (gt < R) {
                    float *mp = reinterpret_cast<float *>(S.m[g]) + gt, *hp = reinterpret_cast<float *>(S.top[g]) + gt;
                    const float w0 = S.wmax[g][0][gt], w1 = S.wmax[g][1][gt], w2 = S.wmax[g][2][gt], w3 = S.wmax[g][3][gt];
                    const float was = *mp, top = fmaxf(fmaxf(w0, w1), fmaxf(w2, w3));
                    const float by = static_cast<float>(lref - scale_was), high = *hp - by;
                    // (o, up to 2^25 value references, is to stay finite when it is raised by the fall)
                    const float lowest = fminf(fmaxf(70.0f - static_cast<float>(lref), 0.0f), kLowest);
                    float m = was - by;
                    // far above what came before it, or what stands beside it
                    const float low = fminf(fminf(w0, w1), fminf(w2, w3));
                    far = (top > m + kHeadroom && m > -FLT_MAX) || (low < top - (kFallBelow - kHeadroom) && low > -FLT_MAX);
                    if (top > m || (top < m - kFallBelow && top > -FLT_MAX)) 
                        m = fmaxf(fmaxf(top + kHeadroom, high - lowest), was - kLowestAtOnce);
                    *mp = m;
                    *hp = fmaxf(high, m);
                    reinterpret_cast<float *>(S.back[g])[gt] = ex2(was - m);
                }
                again = any_of<kGroup>(far, g);
                if (!(flags & kGroupFirst)) {
#pragma unroll
                    for (int h = 0; h < kRW / 4; ++h) {
                        const float4 back = S.back[g][r0 / 4 + h];
                        const float bk[4] = {back.x, back.y, back.z, back.w};
#pragma unroll
                        for (int e = 0; e < 4; ++e) o[4 * h + e] *= bk[e];
                        z[2 * h] = __fmul2_rn(z[2 * h], make_float2(back.x, back.y));
                        z[2 * h + 1] = __fmul2_rn(z[2 * h + 1], make_float2(back.z, back.w));
                    }
                }
                chain = 0;
            }
            // weights and their digits
            const int lv = f.ve[me >> 4] - lref;
            float up = f.vm[me >> 4];
            if (lv < kScaleLowest) up *= exp2i(lv - kScaleLowest);
            const float down = __uint_as_float(static_cast<uint32_t>(127 - max(lv, kScaleLowest)) << 23);
            const float2 up2 = make_float2(up, up), down2 = make_float2(down, down);
            wait(&S.p_empty[g], ((i >> 1) + 1) & 1, ok);  // PV of this group's last tile has read the buffer
            uint8_t *row = my_p + me * Sh::kPRow;
            float2 u[kRW / 2];
#pragma unroll
            for (int h = 0; h < kRW / 4; ++h) {
                const float4 m = S.m[g][r0 / 4 + h];
                const float2 x0 = __fadd2_rn(make_float2(x[4 * h], x[4 * h + 1]), make_float2(-m.x, -m.y));
                const float2 x1 = __fadd2_rn(make_float2(x[4 * h + 2], x[4 * h + 3]), make_float2(-m.z, -m.w));
                const float2 w0 = make_float2(ex2(x0.x), ex2(x0.y)), w1 = make_float2(ex2(x1.x), ex2(x1.y));
                z[2 * h] = __ffma2_rn(w0, down2, z[2 * h]);
                z[2 * h + 1] = __ffma2_rn(w1, down2, z[2 * h + 1]);
                u[2 * h] = __fmul2_rn(w0, up2);
                u[2 * h + 1] = __fmul2_rn(w1, up2);
                if constexpr (kInt)
                    *reinterpret_cast<uint4 *>(row + (weights_chunk<Sh::kPRow>(r0 / 4 + h, me) << 4)) =
                        make_uint4(to_u32_sat(u[2 * h].x), to_u32_sat(u[2 * h].y), to_u32_sat(u[2 * h + 1].x),
                                   to_u32_sat(u[2 * h + 1].y));
            }
            if constexpr (!kInt) {
                // column of digit k of row r: R k + r.  (A loop of 16 rows' digits written out five times does not stay in the
                // instruction cache beside the helpers' loops: 24 sequences of 80 heads on 8 148 us instead of 126)
#pragma unroll(R == 8 ? Sh::kVD : 1)
                for (int k = 0; k < Sh::kVD; ++k) {
                    uint32_t d[kRW / 4];
#pragma unroll
                    for (int h = 0; h < kRW / 4; ++h) {
                        const uint32_t lo = e4m3_digit(u[2 * h]);
                        d[h] = lo | e4m3_digit(u[2 * h + 1]) << 16;
                    }
                    if constexpr (R == 16)
                        *reinterpret_cast<uint4 *>(row + (weights_chunk<128>(k, me) << 4)) = make_uint4(d[0], d[1], d[2], d[3]);
                    else
                        *reinterpret_cast<uint2 *>(row + (weights_chunk<128>(k >> 1, me) << 4) + 8 * (k & 1)) =
                            make_uint2(d[0], d[1]);
                }
            }
            if (gt == 0) S.accumulate[g] = chain > 0;
            ++chain;
            fence_proxy_async_smem();
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(&S.p_full[g]);

            if (flags & kGroupLast) {
                // ---- this group's part of the item is done
                float zs[kRW];
#pragma unroll
                for (int r = 0; r < kRW / 2; ++r) {
                    zs[2 * r] = z[r].x;
                    zs[2 * r + 1] = z[r].y;
                }
                const float zw = sum_rows<kRW>(zs, lane);
                if (lane < kRW) S.zsum[g][w4][r0 + lane] = zw;
                wait(&S.p_empty[g], (i >> 1) & 1, ok);
                tc_fence_after_sync();
                add_sums<R, KIND>(to, exp2i(lref), o);
                tc_fence_before_sync();
                chain = 0;
                // the sums by dimension: where the weights lay, or, when the other group has the item's last tile, handed
                // over to it once it has taken what it was handed before
                const bool hand = !(flags & kLast);
                if (hand) wait(&S.sum_empty, (handovers + 1) & 1, ok);
                float *own = (hand ? handed : reinterpret_cast<float *>(my_p)) + me;
#pragma unroll
                for (int r = 0; r < kRW; ++r) own[(r0 + r) * kPD] = o[r];
                any_of<kGroup>(false, g);
                float zr = gt < R ? (S.zsum[g][0][gt] + S.zsum[g][1][gt]) + (S.zsum[g][2][gt] + S.zsum[g][3][gt]) : 0.0f;
                if (zr > FLT_MAX) zr = FLT_MAX;  // (of references that fell twice by the most; its output is 0 all the same)
                if (hand) {
                    if (gt < R) {
                        S.sum_z[gt] = zr;
                        S.sum_m[gt] = reinterpret_cast<const float *>(S.m[g])[gt];
                    }
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&S.sum_full);
                } else {
                    const bool both = (flags & kBoth) != 0, ends = (flags & kEnds) != 0, complete = k_first == 0 && ends;
                    const int slot = k_first > 0 ? 0 : 1;
                    if (both) wait(&S.sum_full, handovers & 1, ok);
                    float *rec = p.part + static_cast<int64_t>(2 * c + slot) * rec_floats(R);
                    if (gt < R) {
                        // factors of the two parts, the final division included
                        const float m0 = reinterpret_cast<const float *>(S.m[g])[gt], m1 = both ? S.sum_m[gt] : -INFINITY;
                        const float M = fmaxf(m0, m1), ref = M == -INFINITY ? 0.0f : M;
                        float2 fac = make_float2(ex2(m0 - ref), ex2(m1 - ref));
                        const float zz = zr * fac.x + (both ? S.sum_z[gt] * fac.y : 0.0f);
                        if (complete) {
                            const float iz = recip(zz);
                            fac = make_float2(fac.x * iz, fac.y * iz);
                        } else {
                            *reinterpret_cast<float2 *>(rec + R * kPD + 2 * gt) = make_float2(M, zz);
                        }
                        S.factors[g][gt] = fac;
                    }
                    any_of<kGroup>(false, g);
                    const Seq s = f.s;
                    const int rows = min(R, s.rows - R * f.rt);
                    // a warp a row, four dimensions a lane
                    const float4 *mine = reinterpret_cast<const float4 *>(my_p) + lane;
                    const float4 *other = reinterpret_cast<const float4 *>(handed) + lane;
#pragma unroll 2
                    for (int r = gt >> 5; r < rows; r += kGroup / 32) {
                        const float2 fac = S.factors[g][r];
                        float4 t = mine[r * (kPD / 4)];
                        t = make_float4(t.x * fac.x, t.y * fac.x, t.z * fac.x, t.w * fac.x);
                        if (both) {
                            const float4 y = other[r * (kPD / 4)];
                            t = make_float4(fmaf(y.x, fac.y, t.x), fmaf(y.y, fac.y, t.y), fmaf(y.z, fac.y, t.z),
                                            fmaf(y.w, fac.y, t.w));
                        }
                        const int rw = R * f.rt + r, ri = p.by_gq.quot(rw);
                        float *dst = complete ? p.out + static_cast<int64_t>(s.start + ri) * p.ldo +
                                                    (f.head * p.GQ + rw - ri * p.GQ) * kPD
                                              : rec + r * kPD;
                        *reinterpret_cast<float4 *>(dst + 4 * lane) = t;
                    }
                    if (both) {
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&S.sum_empty);
                    }
                }
                if (flags & kBoth) ++handovers;
                any_of<kGroup>(false, g);  // the sums have been read
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&S.info_empty[i % kInfo]);
        }
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    if (warp == Sh::kWarpQK) tmem_dealloc(tmem, Sh::kTmemCols);
    merge_cut_items<R, Sh::kThreads>(p, S.cut, S.last, reinterpret_cast<float *>(pbuf));
    pdl_launch_dependents();
}

template <int R, int KIND>
cudaError_t launch_rows(const AttnParams &p, const CacheMaps &maps, int ctas, cudaStream_t s) {
    static DeviceOnce once;
    int dev = 0;
    cudaError_t e = current_device(&dev);
    if (e != cudaSuccess) return e;
    e = once.run(dev, [] {
        return cudaFuncSetAttribute(attn_paged_kernel<R, KIND>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    static_cast<int>(attn_smem<R, KIND>()));
    });
    if (e != cudaSuccess) return e;
    return launch_pdl(attn_paged_kernel<R, KIND>, dim3(ctas), Shape<R, KIND>::kThreads, attn_smem<R, KIND>(), s, p, maps);
}

}  // namespace

cudaError_t set_paged_wait_budget(long long cycles) {
    return cudaMemcpyToSymbol(c_wait_budget, &cycles, sizeof(cycles));
}

void paged_copies(const int32_t *at, int32_t *size) {
    unsigned follows = 0;
    for (int j = 1; j < kTB; ++j) follows |= continues_block(at[j - 1], at[j]) ? 1u << j : 0u;
    for (int j = 0; j < kTB; ++j) size[j] = copy_size(follows, j, at[j]);
}

size_t attention_paged_workspace_bytes(int num_sms) {
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
    for (int i = 0; i < 4; ++i) {
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
    const bool int8 = A.cache.kind == TERN_KV_INT8;
    // Items of 8, 16 or, of int8, 32 rows (e4m3's digits take five columns of tensor memory a row).  In us with 8 / 16 /
    // 32 rows, and e4m3 with 8 / 16: one token, context 65536, of 40 heads on 8 34.9 / 39.1 / 48.5, 33.6 / 39.4, of 128
    // heads on 8 49.2 / 43.1 / 53.4, 52 / 44; three sequences of 2 drafted tokens, 40 heads, context 8191 27.6 / 26.3 /
    // 33.1, 30.0 / 27.7, of 16 tokens 79 / 59 / 60, 84 / 66; a prompt's last 2048 of 4096 tokens 1078 / 862 / 525,
    // 1300 / 1003.
    const int R = rows <= 8 ? 8 : int8 && rows > 16 ? 32 : 16;
    // one CTA per SM, fewer when the tiles are few
    const int64_t tiles = std::min<int64_t>(A.batch.B, A.batch.T) * A.cache.Hkv * ceil_div(rows, R) * ceil_div(span, kTok);
    const int ctas = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>({tiles, A.num_sms, kMaxCtas})));
    if (int8)
        return R == 8    ? launch_rows<8, TERN_KV_INT8>(p, maps, ctas, s)
               : R == 16 ? launch_rows<16, TERN_KV_INT8>(p, maps, ctas, s)
                         : launch_rows<32, TERN_KV_INT8>(p, maps, ctas, s);
    return R == 8 ? launch_rows<8, TERN_KV_E4M3>(p, maps, ctas, s) : launch_rows<16, TERN_KV_E4M3>(p, maps, ctas, s);
}

}  // namespace tern
