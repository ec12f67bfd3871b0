// tern_paged.cu -- rotary embedding, and the append to and read of the paged
// 8-bit KV cache (the attention over it is in tern_paged_attention.cu).
//
//  * rope_kernel: a thread owns four pairs of one head of one row (eight
//    floats: the two halves' float4, or two adjacent float4 when pairs are
//    interleaved), so rows may be rotated in place.
//  * append_paged_kernel: the first CTAs rotate the queries the same way; the
//    others take the new blocks of the cache, a warp per (block of 16 tokens,
//    KV head, K or V): half a warp per token, eight elements a lane, all of the
//    block's new tokens in registers, so the block's maximum is one warp
//    reduction and each input is read once.
//  * read_paged_kernel: codes times scales, four elements a thread.
//
// Arithmetic: products, sums and differences of the rotation are rounded one
// by one (no fused multiply-add), the scales are powers of two (their
// reciprocal and every rescaling factor are exact), so that the codes are
// reproducible bit for bit.
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

// Cosine and sine of pairs 4j .. 4j+3 of row t; false when one of the row's
// positions (of any axis: the whole row is refused, whichever pairs a thread
// owns) lies outside the table.
__device__ __forceinline__ bool load_turns(const RopeView &R, const int32_t *pos, int T, int axes, int t, int j,
                                           float (&c)[4], float (&s)[4]) {
    int p[3] = {0, 0, 0};
    bool ok = true;
#pragma unroll
    for (int a = 0; a < 3; ++a)
        if (a < axes) {
            p[a] = pos[static_cast<int64_t>(a) * T + t];
            ok = ok && p[a] >= 0 && p[a] < R.n_pos;
        }
    if (!ok) return false;
    if (4 * j >= R.half) return true;  // past the rotated elements
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const int i = 4 * j + e;
        const int at = i < R.end0 ? p[0] : i < R.end1 ? p[1] : p[2];
        const float2 cs = __ldg(R.table + static_cast<int64_t>(at) * R.half + i);
        c[e] = cs.x;
        s[e] = R.sign * cs.y;
    }
    return true;
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

// One unit of one head of one row: load, turn, store.
__device__ __forceinline__ void rotate_unit(const RopeView &R, const int32_t *pos, int T, int axes, int t, int j,
                                            const float *x, float *y, int32_t *d_invalid, bool counts) {
    float c[4], s[4], a[4] = {}, b[4] = {};
    int o0, o1;
    unit_offsets(R, j, o0, o1);
    if (load_turns(R, pos, T, axes, t, j, c, s)) {
        load4(x + o0, a);
        load4(x + o1, b);
        turn(R, j, a, b, c, s);
    } else if (counts && d_invalid) {
        atomicAdd(d_invalid, 1);
    }
    store4(y + o0, a);
    store4(y + o1, b);
}

__global__ void __launch_bounds__(kRopeThreads)
    rope_kernel(RopeView R, const int32_t *__restrict__ pos, int T, int axes, int H, int units, const float *x, int ldx,
                float *y, int ldy, int32_t *d_invalid) {
    pdl_wait();
    const int64_t i = static_cast<int64_t>(blockIdx.x) * kRopeThreads + threadIdx.x;
    const int per_row = H * units;
    const int64_t row = i / per_row;
    if (row < T) {
        const int t = static_cast<int>(row), r = static_cast<int>(i - row * per_row);
        const int h = r / units, j = r - h * units;
        rotate_unit(R, pos, T, axes, t, j, x + static_cast<int64_t>(t) * ldx + h * units * 8,
                    y + static_cast<int64_t>(t) * ldy + h * units * 8, d_invalid, r == 0);
    }
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
__device__ __forceinline__ uint8_t to_code(float y, int kind) {
    if (kind == TERN_KV_INT8) return static_cast<uint8_t>(max(-127, min(127, __float2int_rn(y))));
    return __nv_cvt_float_to_fp8(y, __NV_SATFINITE, __NV_E4M3);
}
__device__ __forceinline__ float from_code(uint8_t c, int kind) {
    if (kind == TERN_KV_INT8) return static_cast<float>(static_cast<int8_t>(c));
    return __half2float(__half(__nv_cvt_fp8_to_halfraw(c, __NV_E4M3)));
}

// The least power of two s, 2^-100 <= s <= 2^120, with amax <= s * top (top =
// 127 = 1.984375 * 2^6 or 448 = 1.75 * 2^8), from the bits of amax = f * 2^E.
__device__ __forceinline__ float pow2_scale(float amax, int kind) {
    const uint32_t u = __float_as_uint(amax);
    const uint32_t frac = kind == TERN_KV_INT8 ? 0x7E0000u : 0x600000u;
    int e = static_cast<int>(u >> 23) - 127 - (kind == TERN_KV_INT8 ? 6 : 8) + ((u & 0x7FFFFFu) > frac ? 1 : 0);
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
    int q_ctas;  // CTAs that rotate queries
};

constexpr int kAppendThreads = 256;

// The rows of block `blk` that this call appends (tokens [lo, hi) of sequence
// b, row `row` holding token lo), one KV head, K or V.
__device__ void append_block(const AppendParams &p, int b, int blk, int lo, int hi, int row, int g, bool is_k,
                             int lane) {
    const PagedView &v = p.v;
    const int64_t bi0 = block_index(v, b, blk);
    const int sub = lane >> 4, j = lane & 15;  // token parity, unit of 8 elements
    const int n = hi - lo;
    float a[8][4], c8[8][4];
    bool bad = false;
    int o0, o1;
    unit_offsets(p.R, j, o0, o1);
    float amax = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int r = 2 * i + sub;
#pragma unroll
        for (int e = 0; e < 4; ++e) a[i][e] = c8[i][e] = 0.0f;
        if (r < n) {
            const int t = row + r;
            const float *x = (is_k ? p.k + static_cast<int64_t>(t) * p.ldk : p.vv + static_cast<int64_t>(t) * p.ldv) +
                             g * kPD;
            float c[4], s[4];
            const bool ok = load_turns(p.R, p.pos, v.T, p.axes, t, j, c, s);
            if (ok) {
                load4(x + o0, a[i]);
                load4(x + o1, c8[i]);
                if (is_k) turn(p.R, j, a[i], c8[i], c, s);
            }
            bad = (!ok || bi0 < 0);
            if (bad && g == 0 && is_k && j == 0 && p.d_invalid) atomicAdd(p.d_invalid, 1);
#pragma unroll
            for (int e = 0; e < 4; ++e) amax = fmaxf(amax, fmaxf(fabsf(a[i][e]), fabsf(c8[i][e])));
        }
    }
    if (bi0 < 0) return;
    amax = warp_max(amax);
    const int64_t bi = bi0 + static_cast<int64_t>(g) * v.bpp;
    float *sp = (is_k ? v.ks : v.vs) + bi;
    uint8_t *cp = (is_k ? v.kc : v.vc) + bi * (kPB * kPD);
    const int slot0 = lo - blk * kPB;
    float scale = pow2_scale(amax, v.kind);
    if (slot0 > 0) {  // earlier tokens: keep their scale, or rescale their codes
        const float old = *sp;
        __syncwarp();  // every lane has read the scale before it is written
        scale = fmaxf(old, scale);
        if (scale != old) {
            const float r = old * (1.0f / scale);
            for (int i = lane; i < slot0 * (kPD / 4); i += 32) {
                uint32_t w = reinterpret_cast<uint32_t *>(cp)[i], o = 0;
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    o |= static_cast<uint32_t>(to_code(from_code(static_cast<uint8_t>(w >> (8 * e)), v.kind) * r, v.kind))
                         << (8 * e);
                reinterpret_cast<uint32_t *>(cp)[i] = o;
            }
        }
    }
    const float inv = 1.0f / scale;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int r = 2 * i + sub;
        if (r < n) {
            uint32_t w0 = 0, w1 = 0;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                w0 |= static_cast<uint32_t>(to_code(a[i][e] * inv, v.kind)) << (8 * e);
                w1 |= static_cast<uint32_t>(to_code(c8[i][e] * inv, v.kind)) << (8 * e);
            }
            uint8_t *dst = cp + (slot0 + r) * kPD;
            *reinterpret_cast<uint32_t *>(dst + o0) = w0;
            *reinterpret_cast<uint32_t *>(dst + o1) = w1;
        }
    }
    if (lane == 0) *sp = scale;
}

__global__ void __launch_bounds__(kAppendThreads) append_paged_kernel(AppendParams p) {
    extern __shared__ int32_t starts[];  // row_start
    const PagedView &v = p.v;
    const int tid = threadIdx.x;
    pdl_wait();
    for (int i = tid; i <= v.B; i += kAppendThreads) starts[i] = v.row_start[i];
    __syncthreads();
    if (static_cast<int>(blockIdx.x) < p.q_ctas) {
        const int64_t i = static_cast<int64_t>(blockIdx.x) * kAppendThreads + tid;
        const int per_row = p.Hq * 16;
        const int64_t row = i / per_row;
        if (row < v.T && row >= starts[0] && row < starts[v.B]) {
            const int t = static_cast<int>(row), r = static_cast<int>(i - row * per_row);
            const int h = r >> 4, j = r & 15;
            rotate_unit(p.R, p.pos, v.T, p.axes, t, j, p.q + static_cast<int64_t>(t) * p.ldq + h * kPD,
                        p.q_out + static_cast<int64_t>(t) * p.ldqo + h * kPD, nullptr, false);
        }
    } else {
        // a warp per (row, KV head, K or V); the block's first row does its work
        const int64_t u = static_cast<int64_t>(blockIdx.x - p.q_ctas) * (kAppendThreads / 32) + (tid >> 5);
        const int per_row = 2 * v.Hkv;
        const int64_t row = u / per_row;
        if (row < v.T) {
            const int t = static_cast<int>(row), r = static_cast<int>(u - row * per_row);
            const int b = row_sequence(starts, v.B, t);
            if (b >= 0) {
                const int end = min(starts[b + 1], v.T), ctx = v.ctx[b];
                const int first = ctx - (starts[b + 1] - starts[b]);  // token of the sequence's first row
                const int tok = first + (t - starts[b]);
                if (tok < 0) {
                    if (r == 0 && (tid & 31) == 0 && p.d_invalid) atomicAdd(p.d_invalid, 1);
                } else if (tok % kPB == 0 || t == starts[b]) {
                    const int blk = tok / kPB;
                    const int hi = min(min((blk + 1) * kPB, ctx), tok + (end - t));
                    append_block(p, b, blk, tok, hi, t, r >> 1, (r & 1) == 0, tid & 31);
                }
            }
        }
    }
    pdl_launch_dependents();
}

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
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                kk[e] = from_code(static_cast<uint8_t>(kw >> (8 * e)), v.kind) * ks;
                vv[e] = from_code(static_cast<uint8_t>(vw >> (8 * e)), v.kind) * vs;
            }
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
    return launch_pdl(rope_kernel, dim3(blocks_of(static_cast<int64_t>(T) * H * (D / 8), kRopeThreads)), kRopeThreads, 0,
                      s, rope_view(R), pos, T, R.axes, H, D / 8, x, ldx, y, ldy, d_invalid);
}

cudaError_t launch_kv_append_paged(const AppendLaunch &A, int num_sms, cudaStream_t s) {
    (void)num_sms;
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
    p.q_ctas = static_cast<int>(blocks_of(T * A.Hq * 16, kAppendThreads));
    const unsigned kv_ctas = blocks_of(T * A.cache.Hkv * 2, kAppendThreads / 32);
    return launch_pdl(append_paged_kernel, dim3(p.q_ctas + kv_ctas), kAppendThreads,
                      static_cast<size_t>(A.batch.B + 1) * sizeof(int32_t), s, p);
}

cudaError_t launch_kv_read_paged(const tern_paged_batch &B, const tern_paged_cache &C, float *k_out, int ldk,
                                 float *v_out, int ldv, int32_t *d_invalid, cudaStream_t s) {
    const int64_t n = static_cast<int64_t>(B.T) * C.Hkv * (kPD / 4);
    return launch_pdl(read_paged_kernel, dim3(blocks_of(n, 256)), 256, static_cast<size_t>(B.B + 1) * sizeof(int32_t), s,
                      paged_view(B, C), k_out, ldk, v_out, ldv, d_invalid);
}

}  // namespace tern
