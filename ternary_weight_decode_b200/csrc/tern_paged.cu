// tern_paged.cu -- rotary embedding, and the append to and read of the paged
// 8-bit KV cache (the attention over it is in tern_paged_attention.cu).
//
//  * rope_kernel: a thread owns four pairs of one row's heads (eight floats of
//    each: the two halves' float4, or two adjacent float4 when pairs are
//    interleaved), so rows may be rotated in place and a row's cosines are read
//    once per thread.
//  * append_paged_kernel: some CTAs rotate the queries the same way; the others
//    take the new blocks of the cache, four warps per (block of 16
//    tokens, KV head, K or V): half a warp per token, eight elements a lane, all
//    of the block's new tokens in registers, so each input is read once and the
//    block's maximum is a warp reduction and four words of shared memory.
//  * read_paged_kernel: codes times scales, four elements a thread.
//
// Arithmetic: products, sums and differences of the rotation are rounded one
// by one (no fused multiply-add), the scales are powers of two (their
// reciprocal and every rescaling factor are exact), so that the codes are
// reproducible bit for bit.
//
// All three are bound by memory at large sizes and by latency at small ones.
// Measured (device time, and the bytes at the measured copy rate): rotation of
// 2048 rows of 48 heads 19.9 us (15.5), of 777 rows of 32 heads, 64 of 128
// elements, 8.5 (3.9); append and read back of 4096 rows of 40 + 2 x 8 heads
// 41.1 + 11.6 (38.7; the cache's CTAs behind the queries' instead of among
// them 47.0), of 33 ragged sequences of up to 16 rows 9.5 + 3.0 (2.8),
// of one row 3.4 + 2.1.
#include <algorithm>

#include "tern_paged.cuh"

namespace tern {

namespace {

constexpr int kRopeThreads = 256;

struct RopeView {
    const float2 *table;
    int n_pos, half;     // half: pairs of a head
    int end0, end1;      // first pair of axis 1 and of axis 2
    int interleaved;
    float sign;          // -1 for the inverse rotation
};

RopeView rope_view(const tern_rope_plan &R) {
    RopeView v;
    v.table = reinterpret_cast<const float2 *>(R.table);
    v.n_pos = R.n_pos;
    v.half = R.rot_dim / 2;
    v.end0 = R.section[0];
    v.end1 = R.section[0] + R.section[1];
    v.interleaved = (R.flags & TERN_ROPE_INTERLEAVED) != 0;
    v.sign = (R.flags & TERN_ROPE_INVERSE) ? -1.0f : 1.0f;
    return v;
}

// The positions of row t; false when one of them (of any axis: the whole row is
// refused, whichever pairs a thread owns) lies outside the table.
__device__ __forceinline__ bool load_positions(const RopeView &R, const int32_t *pos, int T, int axes, int t, int (&p)[3]) {
    bool ok = true;
#pragma unroll
    for (int a = 0; a < 3; ++a) {
        p[a] = a < axes ? pos[static_cast<int64_t>(a) * T + t] : 0;
        ok = ok && p[a] >= 0 && p[a] < R.n_pos;
    }
    return ok;
}

// Cosine and sine of pairs 4j .. 4j+3 at positions p (inside the table).
__device__ __forceinline__ void load_turns(const RopeView &R, const int (&p)[3], int j, float (&c)[4], float (&s)[4]) {
    if (4 * j >= R.half) return;  // past the rotated elements
    const int a0 = 4 * j < R.end0 ? 0 : 4 * j < R.end1 ? 1 : 2;
    const int a3 = 4 * j + 3 < R.end0 ? 0 : 4 * j + 3 < R.end1 ? 1 : 2;
    if (a0 == a3) {  // one axis: 32 contiguous bytes
        const int at = a0 == 0 ? p[0] : a0 == 1 ? p[1] : p[2];
        const float4 *q = reinterpret_cast<const float4 *>(R.table + static_cast<int64_t>(at) * R.half + 4 * j);
        const float4 u = __ldg(q), w = __ldg(q + 1);
        c[0] = u.x, c[1] = u.z, c[2] = w.x, c[3] = w.z;
        s[0] = R.sign * u.y, s[1] = R.sign * u.w, s[2] = R.sign * w.y, s[3] = R.sign * w.w;
        return;
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const int i = 4 * j + e;
        const int at = i < R.end0 ? p[0] : i < R.end1 ? p[1] : p[2];
        const float2 cs = __ldg(R.table + static_cast<int64_t>(at) * R.half + i);
        c[e] = cs.x;
        s[e] = R.sign * cs.y;
    }
}

// First elements of the two float4 that unit j (of D/8) of a head owns.
__device__ __forceinline__ void unit_offsets(const RopeView &R, int j, int &o0, int &o1) {
    const bool halves = !R.interleaved && 4 * j < R.half;
    o0 = halves ? 4 * j : 8 * j;
    o1 = halves ? R.half + 4 * j : 8 * j + 4;
}

// Rotates the eight elements of unit j in place (a, b: the float4 at
// unit_offsets).
__device__ __forceinline__ void turn(const RopeView &R, int j, float (&a)[4], float (&b)[4], const float (&c)[4],
                                     const float (&s)[4]) {
    if (4 * j >= R.half) return;
    if (R.interleaved) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const float a0 = a[2 * e], a1 = a[2 * e + 1], b0 = b[2 * e], b1 = b[2 * e + 1];
            a[2 * e] = __fsub_rn(__fmul_rn(a0, c[e]), __fmul_rn(a1, s[e]));
            a[2 * e + 1] = __fadd_rn(__fmul_rn(a1, c[e]), __fmul_rn(a0, s[e]));
            b[2 * e] = __fsub_rn(__fmul_rn(b0, c[2 + e]), __fmul_rn(b1, s[2 + e]));
            b[2 * e + 1] = __fadd_rn(__fmul_rn(b1, c[2 + e]), __fmul_rn(b0, s[2 + e]));
        }
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float x0 = a[e], x1 = b[e];
            a[e] = __fsub_rn(__fmul_rn(x0, c[e]), __fmul_rn(x1, s[e]));
            b[e] = __fadd_rn(__fmul_rn(x1, c[e]), __fmul_rn(x0, s[e]));
        }
    }
}

__device__ __forceinline__ void load4(const float *p, float (&v)[4]) {
    const float4 t = *reinterpret_cast<const float4 *>(p);
    v[0] = t.x;
    v[1] = t.y;
    v[2] = t.z;
    v[3] = t.w;
}
__device__ __forceinline__ void store4(float *p, const float (&v)[4]) {
    *reinterpret_cast<float4 *>(p) = make_float4(v[0], v[1], v[2], v[3]);
}

// Unit j of the heads slot, slot + hs, ... of row t: the row's cosines and
// sines are read once, and kHeadsAtOnce heads are in flight.  The first heads'
// loads go out before the positions are waited for.  Three heads keep four CTAs
// resident (2048 x 48 heads: 19.9 us; two heads 20.0, five heads 23.4, one 22.5).  Rows outside [*first, *last) are left alone (null: none are).
constexpr int kHeadsAtOnce = 3;
__device__ __forceinline__ void rotate_row(const RopeView &R, const int32_t *pos, int T, int axes, int t, int j, int slot,
                                           int hs, int H, int D, const float *x, float *y, int32_t *d_invalid,
                                           const int32_t *first, const int32_t *last) {
    float c[4], s[4];
    int o0, o1, at[3];
    unit_offsets(R, j, o0, o1);
    bool ok = true, mine = true;
#pragma unroll 1
    for (int h = slot; h < H; h += kHeadsAtOnce * hs) {
        float a[kHeadsAtOnce][4], b[kHeadsAtOnce][4];
#pragma unroll
        for (int e = 0; e < kHeadsAtOnce; ++e)
            if (h + e * hs < H) {
                load4(x + (h + e * hs) * D + o0, a[e]);
                load4(x + (h + e * hs) * D + o1, b[e]);
            }
        if (h == slot) {
            ok = load_positions(R, pos, T, axes, t, at);
            mine = !first || (t >= *first && t < *last);
            if (ok) load_turns(R, at, j, c, s);
            if (!ok && mine && d_invalid && j == 0 && slot == 0) atomicAdd(d_invalid, 1);
        }
#pragma unroll
        for (int e = 0; e < kHeadsAtOnce; ++e)
            if (h + e * hs < H && mine) {
                if (ok) {
                    turn(R, j, a[e], b[e], c, s);
                } else {
#pragma unroll
                    for (int i = 0; i < 4; ++i) a[e][i] = b[e][i] = 0.0f;
                }
                store4(y + (h + e * hs) * D + o0, a[e]);
                store4(y + (h + e * hs) * D + o1, b[e]);
            }
    }
}

// How a CTA of kRopeThreads shares out rows of H heads: hs head slots a row.
struct RowShare {
    FastDiv units, slots;
    int hs, rows;  // head slots of a row, rows of a CTA
};
RowShare row_share(int H, int units) {
    // the fewest slots (a power of two, so that rows fill the CTA) whose threads take their heads at once
    const int most = kRopeThreads / units;
    RowShare w;
    w.hs = 1;
    while (2 * w.hs <= most && w.hs * kHeadsAtOnce < H) w.hs *= 2;
    w.rows = std::max(1, most / w.hs);
    w.units = fast_div(units);
    w.slots = fast_div(w.hs);
    return w;
}

__global__ void __launch_bounds__(kRopeThreads, 4)
    rope_kernel(RopeView R, RowShare w, const int32_t *__restrict__ pos, int T, int axes, int H, int units, const float *x,
                int ldx, float *y, int ldy, int32_t *d_invalid) {
    pdl_wait();
    const int q = w.units.quot(threadIdx.x), j = threadIdx.x - q * units;
    const int rl = w.slots.quot(q), slot = q - rl * w.hs;
    const int64_t t = static_cast<int64_t>(blockIdx.x) * w.rows + rl;
    if (rl < w.rows && t < T)
        rotate_row(R, pos, T, axes, static_cast<int>(t), j, slot, w.hs, H, units * 8, x + t * ldx, y + t * ldy, d_invalid,
                   nullptr, nullptr);
    pdl_launch_dependents();
}

__global__ void rope_table_kernel(double theta, double scale, int half, int n_pos, float2 *table) {
    pdl_wait();
    const int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
    if (i >= static_cast<int64_t>(n_pos) * half) return;
    const int64_t p = i / half;
    const int e = static_cast<int>(i - p * half);
    double s, c;
    sincos(static_cast<double>(p) * scale * pow(theta, -static_cast<double>(e) / half), &s, &c);
    table[i] = make_float2(static_cast<float>(c), static_cast<float>(s));
}

// ---------------------------------------------------------------- codes
// Four values (of at most the largest code) as codes.
template <int KIND>
__device__ __forceinline__ uint32_t to_codes(float y0, float y1, float y2, float y3) {
    uint32_t lo, hi;
    if constexpr (KIND == TERN_KV_INT8) {
        asm("cvt.pack.sat.s8.s32.b32 %0, %1, %2, 0;" : "=r"(hi) : "r"(__float2int_rn(y3)), "r"(__float2int_rn(y2)));
        asm("cvt.pack.sat.s8.s32.b32 %0, %1, %2, %3;"
            : "=r"(lo)
            : "r"(__float2int_rn(y1)), "r"(__float2int_rn(y0)), "r"(hi));
        return lo;
    } else {
        lo = __nv_cvt_float2_to_fp8x2(make_float2(y0, y1), __NV_SATFINITE, __NV_E4M3);
        hi = __nv_cvt_float2_to_fp8x2(make_float2(y2, y3), __NV_SATFINITE, __NV_E4M3);
        return lo | hi << 16;
    }
}
template <int KIND>
__device__ __forceinline__ float4 from_codes(uint32_t w) {
    if constexpr (KIND == TERN_KV_INT8) {
        return make_float4(static_cast<int8_t>(w), static_cast<int8_t>(w >> 8), static_cast<int8_t>(w >> 16),
                           static_cast<int8_t>(w >> 24));
    } else {
        const float2 lo = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(w), __NV_E4M3)));
        const float2 hi =
            __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(w >> 16), __NV_E4M3)));
        return make_float4(lo.x, lo.y, hi.x, hi.y);
    }
}

// The least power of two s, 2^-100 <= s <= 2^120, with amax <= s * top (top =
// 127 = 1.984375 * 2^6 or 448 = 1.75 * 2^8), from the bits of amax = f * 2^E.
template <int KIND>
__device__ __forceinline__ float pow2_scale(float amax) {
    const uint32_t u = __float_as_uint(amax);
    const uint32_t frac = KIND == TERN_KV_INT8 ? 0x7E0000u : 0x600000u;
    int e = static_cast<int>(u >> 23) - 127 - (KIND == TERN_KV_INT8 ? 6 : 8) + ((u & 0x7FFFFFu) > frac ? 1 : 0);
    e = max(-100, min(120, e));
    return __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
}

struct AppendParams {
    PagedView v;
    RopeView R;
    int axes, Hq;
    const float *q, *k, *vv;
    int ldq, ldk, ldv;
    const int32_t *pos;
    float *q_out;
    int ldqo;
    int32_t *d_invalid;
    int kv_ctas;     // CTAs of the cache: every `every`-th of the first every * kv_ctas; the others rotate queries
    int every;
    FastDiv by_every;
    RowShare share;
    int group;       // rows of a KV CTA
};

constexpr int kAppendThreads = 256;

// Rescales rows r0, r0 + step, ... below slot0 of a block's codes by r: lane l
// dimensions 4l .. 4l+3, up to eight tokens' codes in flight.
template <int KIND>
__device__ __forceinline__ void rescale_rows(uint8_t *codes, int slot0, float r, int lane, int r0, int step) {
    uint32_t *row4 = reinterpret_cast<uint32_t *>(codes) + lane;
#pragma unroll 1
    for (int i0 = r0; i0 < slot0; i0 += 8 * step) {
        uint32_t w[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = i0 + i * step < slot0 ? row4[(i0 + i * step) * (kPD / 4)] : 0u;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float4 y = from_codes<KIND>(w[i]);
            if (i0 + i * step < slot0)
                row4[(i0 + i * step) * (kPD / 4)] = to_codes<KIND>(y.x * r, y.y * r, y.z * r, y.w * r);
        }
    }
}

// The rows of block `blk` that this call appends (tokens [lo, hi) of sequence
// b, row `row` holding token lo), one KV head, K or V, by one of four warps (w):
// a warp's own chain of instructions is what counts (16 rows by one warp 10.4
// us, by four 3.7).  A warp has rows 2 (w + 4 i) + sub, i = 0, 1, in registers;
// the four share the maximum.
template <int KIND>
__device__ __forceinline__ void append_block(const AppendParams &p, int b, int blk, int lo, int hi, int row, int g,
                                                    bool is_k, int lane, int w, float *shared_max) {
    const PagedView &v = p.v;
    const int sub = lane >> 4, j = lane & 15;  // token parity, unit of 8 elements
    const int n = hi - lo;
    int o0, o1;
    unit_offsets(p.R, j, o0, o1);
    const float *x = (is_k ? p.k + static_cast<int64_t>(row) * p.ldk : p.vv + static_cast<int64_t>(row) * p.ldv) + g * kPD;
    const int ld = is_k ? p.ldk : p.ldv;
    float a[2][4], c8[2][4];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int r = 2 * (w + 4 * i) + sub;
#pragma unroll
        for (int e = 0; e < 4; ++e) a[i][e] = c8[i][e] = 0.0f;
        if (r < n) {
            load4(x + static_cast<int64_t>(r) * ld + o0, a[i]);
            load4(x + static_cast<int64_t>(r) * ld + o1, c8[i]);
        }
    }
    const int64_t bi0 = block_index(v, b, blk), bi = bi0 + static_cast<int64_t>(g) * v.bpp;
    const int slot0 = lo - blk * kPB;
    float *sp = (is_k ? v.ks : v.vs) + bi;
    const float old = bi0 >= 0 && slot0 > 0 ? *sp : 0.0f;
    float amax = 0.0f;
    int bad = 0;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int r = 2 * (w + 4 * i) + sub;
        if (r < n) {
            int at[3];
            float c[4], s[4];
            const bool ok = load_positions(p.R, p.pos, v.T, p.axes, row + r, at);
            if (!ok) {  // a row outside the table is appended as 0
#pragma unroll
                for (int e = 0; e < 4; ++e) a[i][e] = c8[i][e] = 0.0f;
            } else if (is_k) {
                load_turns(p.R, at, j, c, s);
                turn(p.R, j, a[i], c8[i], c, s);
            }
            bad += !ok || bi0 < 0;
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) amax = fmaxf(amax, fmaxf(fabsf(a[i][e]), fabsf(c8[i][e])));
    }
    if (j == 0 && bad > 0 && g == 0 && is_k && p.d_invalid) atomicAdd(p.d_invalid, bad);
    amax = warp_max(amax);
    if (lane == 0) shared_max[w] = amax;
    asm volatile("barrier.cta.sync %0, 128;" ::"r"(is_k ? 1 : 2) : "memory");  // also: every lane has read the old scale
    const float top = fmaxf(fmaxf(shared_max[0], shared_max[1]), fmaxf(shared_max[2], shared_max[3]));
    asm volatile("barrier.cta.sync %0, 128;" ::"r"(is_k ? 1 : 2) : "memory");  // the words are free for the next block
    if (bi0 < 0) return;
    if (KIND == TERN_KV_INT8 && top > 0x1.FCp126f) {  // past 127 of the largest scale the code is 127 or -127, not -128
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                a[i][e] = fmaxf(a[i][e], -0x1.FCp126f);
                c8[i][e] = fmaxf(c8[i][e], -0x1.FCp126f);
            }
    }
    uint8_t *cp = (is_k ? v.kc : v.vc) + bi * (kPB * kPD);
    float scale = pow2_scale<KIND>(top);
    if (slot0 > 0) {  // earlier tokens: keep their scale, or rescale their codes
        scale = fmaxf(old, scale);
        if (scale != old) rescale_rows<KIND>(cp, slot0, old * (1.0f / scale), lane, w, 4);
    }
    const float inv = 1.0f / scale;
    if (w == 0 && lane == 0) *sp = scale;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int r = 2 * (w + 4 * i) + sub;
        if (r < n) {
            uint8_t *dst = cp + (slot0 + r) * kPD;
            *reinterpret_cast<uint32_t *>(dst + o0) = to_codes<KIND>(a[i][0] * inv, a[i][1] * inv, a[i][2] * inv, a[i][3] * inv);
            *reinterpret_cast<uint32_t *>(dst + o1) =
                to_codes<KIND>(c8[i][0] * inv, c8[i][1] * inv, c8[i][2] * inv, c8[i][3] * inv);
        }
    }
}

// Row t's sequence, token, and (where the row is the first of a block) the
// token behind the block's last one that this call appends.
struct RowPlace {
    int b, tok, hi;
    bool leads;
};
__device__ __forceinline__ RowPlace row_place(const PagedView &v, const int32_t *starts, int t, int32_t *d_invalid) {
    RowPlace r = {row_sequence(starts, v.B, t), 0, 0, false};
    if (r.b < 0) return r;
    const int end = min(starts[r.b + 1], v.T), ctx = v.ctx[r.b];
    r.tok = ctx - (starts[r.b + 1] - t);
    if (r.tok < 0) {
        if (d_invalid) atomicAdd(d_invalid, 1);
    } else if (r.tok % kPB == 0 || t == starts[r.b]) {
        r.leads = true;
        r.hi = min(min((r.tok / kPB + 1) * kPB, ctx), r.tok + (end - t));
    }
    return r;
}

template <int KIND>
__global__ void __launch_bounds__(kAppendThreads, 4) append_paged_kernel(AppendParams p) {
    extern __shared__ int32_t starts[];  // row_start
    __shared__ float shared_max[2][4];
    __shared__ RowPlace place[kPB];
    __shared__ unsigned leaders;
    const PagedView &v = p.v;
    const int tid = threadIdx.x, lane = tid & 31;
    pdl_wait();
    const int kv = min(p.by_every.quot(blockIdx.x), p.kv_ctas), in = static_cast<int>(blockIdx.x) - kv * p.every;
    if (kv == p.kv_ctas || in != 0) {
        const int q = tid >> 4, j = tid & 15;
        const int rl = p.share.slots.quot(q), slot = q - rl * p.share.hs;
        const int64_t t = (static_cast<int64_t>(kv) * (p.every - 1) + (kv == p.kv_ctas ? in : in - 1)) * p.share.rows + rl;
        if (rl < p.share.rows && t < v.T)
            rotate_row(p.R, p.pos, v.T, p.axes, static_cast<int>(t), j, slot, p.share.hs, p.Hq, kPD, p.q + t * p.ldq,
                       p.q_out + t * p.ldqo, nullptr, v.row_start, v.row_start + v.B);
        pdl_launch_dependents();
        return;
    }
    for (int i = tid; i <= v.B; i += kAppendThreads) starts[i] = v.row_start[i];
    __syncthreads();
    const int64_t u = kv;
    // a CTA per (p.group rows, KV head), four warps for K and four for V; each row that is the first of a block is one
    // block's work
    const int64_t rg = u / v.Hkv, t0 = rg * p.group;
    const int g = static_cast<int>(u - rg * v.Hkv), warp = tid >> 5;
    if (warp == 0) {
        RowPlace mine = {-1, 0, 0, false};
        if (lane < p.group && t0 + lane < v.T)
            mine = row_place(v, starts, static_cast<int>(t0) + lane, g == 0 ? p.d_invalid : nullptr);
        if (lane < kPB) place[lane] = mine;
        const unsigned m = __ballot_sync(0xffffffffu, mine.leads);
        if (lane == 0) leaders = m;
    }
    __syncthreads();
#pragma unroll 1
    for (unsigned m = leaders; m != 0; m &= m - 1) {
        const int l = __ffs(m) - 1;
        const RowPlace r = place[l];
        append_block<KIND>(p, r.b, r.tok / kPB, r.tok, r.hi, static_cast<int>(t0) + l, g, warp < 4, lane, warp & 3,
                           shared_max[warp >> 2]);
    }
    pdl_launch_dependents();
}

template <int KIND>
__global__ void __launch_bounds__(256)
    read_paged_kernel(PagedView v, float *k_out, int ldk, float *v_out, int ldv, int32_t *d_invalid) {
    extern __shared__ int32_t starts[];
    const int tid = threadIdx.x;
    pdl_wait();
    for (int i = tid; i <= v.B; i += 256) starts[i] = v.row_start[i];
    __syncthreads();
    // a thread per four elements of K and of V
    const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + tid;
    const int per_row = v.Hkv * (kPD / 4);
    const int64_t row = i / per_row;
    const int b = row < v.T ? row_sequence(starts, v.B, static_cast<int>(row)) : -1;
    if (b >= 0) {
        const int t = static_cast<int>(row), r = static_cast<int>(i - row * per_row);
        const int g = r / (kPD / 4), d = 4 * (r % (kPD / 4));
        const int tok = v.ctx[b] - starts[b + 1] + t;
        const int64_t bi0 = tok >= 0 ? block_index(v, b, tok / kPB) : -1;
        float kk[4] = {}, vv[4] = {};
        if (bi0 >= 0) {
            const int64_t bi = bi0 + static_cast<int64_t>(g) * v.bpp;
            const int64_t at = (bi * kPB + tok % kPB) * kPD + d;
            const uint32_t kw = *reinterpret_cast<const uint32_t *>(v.kc + at);
            const uint32_t vw = *reinterpret_cast<const uint32_t *>(v.vc + at);
            const float ks = v.ks[bi], vs = v.vs[bi];
            const float4 kf = from_codes<KIND>(kw), vf = from_codes<KIND>(vw);
            kk[0] = kf.x * ks, kk[1] = kf.y * ks, kk[2] = kf.z * ks, kk[3] = kf.w * ks;
            vv[0] = vf.x * vs, vv[1] = vf.y * vs, vv[2] = vf.z * vs, vv[3] = vf.w * vs;
        } else if (r == 0 && d_invalid) {
            atomicAdd(d_invalid, 1);
        }
        store4(k_out + static_cast<int64_t>(t) * ldk + g * kPD + d, kk);
        store4(v_out + static_cast<int64_t>(t) * ldv + g * kPD + d, vv);
    }
    pdl_launch_dependents();
}

unsigned blocks_of(int64_t n, int per) { return static_cast<unsigned>(ceil_div(n, per)); }

}  // namespace

cudaError_t launch_rope_table(double theta, double scale, int rot_dim, int n_pos, float *table, cudaStream_t s) {
    const int half = rot_dim / 2;
    return launch_pdl(rope_table_kernel, dim3(blocks_of(static_cast<int64_t>(n_pos) * half, 128)), 128, 0, s, theta,
                      scale, half, n_pos, reinterpret_cast<float2 *>(table));
}

cudaError_t launch_rope(const tern_rope_plan &R, const int32_t *pos, int T, int H, int D, const float *x, int ldx,
                        float *y, int ldy, int32_t *d_invalid, cudaStream_t s) {
    const RowShare w = row_share(H, D / 8);
    return launch_pdl(rope_kernel, dim3(blocks_of(T, w.rows)), kRopeThreads, 0, s, rope_view(R), w, pos, T, R.axes, H, D / 8,
                      x, ldx, y, ldy, d_invalid);
}

cudaError_t launch_kv_append_paged(const AppendLaunch &A, cudaStream_t s) {
    AppendParams p;
    p.v = paged_view(A.batch, A.cache);
    p.R = rope_view(A.rope);
    p.axes = A.rope.axes;
    p.Hq = A.Hq;
    p.q = A.q;
    p.k = A.k;
    p.vv = A.v;
    p.ldq = A.ldq;
    p.ldk = A.ldk;
    p.ldv = A.ldv;
    p.pos = A.pos;
    p.q_out = A.q_out;
    p.ldqo = A.ldqo;
    p.d_invalid = A.d_invalid;
    const int64_t T = A.batch.T;
    p.share = row_share(A.Hq, 16);
    // a CTA per 16 rows and KV head, but per row where sequences have few (there nearly every row is the first of its
    // block, and 16 of them one after another took longer).  251 rows of one sequence: 5.6 us per 16, 7.3 us per row.
    p.group = A.batch.max_rows >= kPB ? kPB : 1;
    const int64_t kv_ctas = ceil_div(T, p.group) * A.cache.Hkv, ctas = blocks_of(T, p.share.rows) + kv_ctas;
    // the cache's CTAs, whose time is latency, spread among those of the queries, whose time is memory's
    p.kv_ctas = static_cast<int>(kv_ctas);
    p.every = static_cast<int>(std::max<int64_t>(1, ctas / kv_ctas));
    p.by_every = fast_div(p.every);
    return launch_pdl(A.cache.kind == TERN_KV_INT8 ? append_paged_kernel<TERN_KV_INT8> : append_paged_kernel<TERN_KV_E4M3>,
                      dim3(static_cast<unsigned>(ctas)), kAppendThreads,
                      static_cast<size_t>(A.batch.B + 1) * sizeof(int32_t), s, p);
}

cudaError_t launch_kv_read_paged(const tern_paged_batch &B, const tern_paged_cache &C, float *k_out, int ldk,
                                 float *v_out, int ldv, int32_t *d_invalid, cudaStream_t s) {
    const int64_t n = static_cast<int64_t>(B.T) * C.Hkv * (kPD / 4);
    return launch_pdl(C.kind == TERN_KV_INT8 ? read_paged_kernel<TERN_KV_INT8> : read_paged_kernel<TERN_KV_E4M3>, dim3(blocks_of(n, 256)), 256, static_cast<size_t>(B.B + 1) * sizeof(int32_t), s,
                      paged_view(B, C), k_out, ldk, v_out, ldv, d_invalid);
}

}  // namespace tern
