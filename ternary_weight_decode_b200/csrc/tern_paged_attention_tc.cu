// tern_paged_attention_tc.cu -- attention over the paged cache's int8 codes on
// the 5th-generation tensor cores, the codes used as they lie.
//
// Both products of the attention are integer matrix products of the codes with
// an fp32 operand written as fixed-point digits, so no code is ever converted:
//   S^T[token][row] = K[token][d] . Q[row][d]^T      (tcgen05.mma kind::i8)
//   O^T[d][row]     = V[token][d]^T . P[token][row]
// with 128 tokens (of S) and 128 dimensions (of O) as the 128 accumulator
// lanes.  K is the A operand as TMA brings it (tokens x 128 bytes, K-major,
// 128-byte swizzle), V the same bytes read the other way (M-major).
//  * A query row is scaled by a power of two to 23 bits and split into three
//    signed 8-bit digits, q = d2 2^16 + d1 2^8 + d0 (error at most 2^-24 of the
//    row's largest element): three columns of the B operand per row.  A digit's
//    product is an exact int32 below 2^21.
//  * A softmax weight times its block's value scale, relative to a reference of
//    each, is an unsigned 32-bit fixed-point number, and its four bytes are
//    four unsigned digits: the word is stored as it is, four columns per row.
//    The sums over tokens are exact int32, so they stay in tensor memory from
//    tile to tile.
// References: row r's weights are 2^(score - m_r) with m_r at least the largest
// score so far; when a tile has a larger one (or block scales leave the
// reference's range, or int32 could overflow), the sums are read, added to fp32
// registers and begun again.  m_r is set four above the largest score, so that
// happens a few times per item (28 of 32 bits remain; block scales may cost 8
// more).
//
// One CTA per SM; warps: 0 TMA and block look-up, 1 MMA issue, 2-3 query
// digits, then one or two warpgroups of softmax (16 or 8 rows each; thread =
// token of S, dimension of O).  A tile is eight visible blocks of 16 tokens of
// an item, from anywhere in the sequence, so sinks and a window fill whole
// tiles.  Everything runs ahead across items: TMA by the ring of stages, QK of
// the next tile before PV of this one, the next item's digits while this one's
// tiles are worked off.
#include <algorithm>

#include "tern_paged_attention.cuh"
#include "tern_tc.cuh"

namespace tern {

namespace {

constexpr int kTB = 8;                    // blocks of a tile
constexpr int kTok = kTB * kPB;           // 128 tokens
constexpr int kTileBytes = kTok * kPD;    // 16 KB of K or V codes
constexpr int kStageBytes = 2 * kTileBytes;
constexpr int kPBytes = kTok * 128;       // weight digits: a token's row of 128 bytes
constexpr float kHeadroom = 4.0f;         // a new reference lies this far (log2) above the largest score
constexpr int kMaxChain = 256;            // tiles summed in int32: 256 * 128 * 255 * 127 < 2^31
constexpr float kVRange = 1.0f / 256.0f;  // largest block scale of a tile, relative to the reference

template <int R>
struct Shape {
    static constexpr int kWG = R > 8 ? 2 : 1;         // softmax warpgroups
    static constexpr int kRW = R / kWG;               // rows of each
    static constexpr int kThreads = 128 + 128 * kWG;
    static constexpr int kNS = R == 8 ? 32 : 3 * R;   // columns of S: 3 per row, a multiple of 16
    static constexpr int kNP = 4 * R;                 // columns of O
    static constexpr int kStages = R > 8 ? 4 : 5;
    static constexpr int kQBytes = kNS * 128;
    static constexpr uint32_t kTmemCols = 2 * kNS + kNP <= 128 ? 128 : 512;
    static constexpr uint32_t kO = 2 * kNS;           // first column of O
};

// One tile, as the softmax and MMA warps see it.
struct TileInfo {
    float ks[kTB], vs[kTB];
    int j0[kTB];      // first token of each block
    int valid;        // bit j: block j is there
    int flags;        // kFirst, kLast, kEdge, kEnds
    float vmax;       // largest value scale
    int b, head, rt, k, units;
};
constexpr int kFirst = 1, kLast = 2, kEdge = 4, kEnds = 8;  // first / last tile of the item here, masks needed, item's end

template <int R>
struct TcShared {
    using Sh = Shape<R>;
    TileInfo info[Sh::kStages];
    float rowf[2][R];                 // score scale of each row's digits
    float wmax[Sh::kWG][4][Sh::kRW];
    float zsum[Sh::kWG][4][Sh::kRW];
    LineShared<Sh::kThreads> line;
    uint64_t kv_full[Sh::kStages], kv_empty[Sh::kStages];
    uint64_t s_full[2], s_empty[2], p_full[2], p_empty[2], q_full[2], q_empty[2];
    Piece piece[2];
    uint32_t tmem;
    int accumulate[2];
    int last[2];
};

template <int R>
constexpr size_t tc_smem() {
    using Sh = Shape<R>;
    return Sh::kStages * kStageBytes + 2 * kPBytes + 2 * Sh::kQBytes + sizeof(TcShared<R>) + 1024;
}
static_assert(tc_smem<8>() <= 227 * 1024 && tc_smem<32>() <= 227 * 1024, "shared memory of one CTA");

// A wait of this thread; once one has run out, none of the later ones waits.
__device__ __forceinline__ void wait(uint64_t *bar, uint32_t parity, bool &ok) {
    if (ok) ok = mbar_wait_bounded(bar, parity);
}

// An int32 of at most 22 bits as fp32, exactly, without the conversion unit.
__device__ __forceinline__ float small_int(uint32_t c) {
    return __uint_as_float(c + 0x4B400000u) - 12582912.0f;
}

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

template <int N>
__device__ __forceinline__ bool any_of(bool x) {  // named barrier 1 over the N softmax threads
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 p, %1, 0;\n\t"
        "barrier.cta.red.or.pred q, 1, %2, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"(static_cast<uint32_t>(x)), "n"(N)
        : "memory");
    return r != 0;
}

template <int R>
__global__ void __launch_bounds__(Shape<R>::kThreads, 1)
    attn_tc_paged_kernel(AttnParams p, const __grid_constant__ CUtensorMap kmap,
                         const __grid_constant__ CUtensorMap vmap) {
    using Sh = Shape<R>;
    constexpr int kSt = Sh::kStages, kNT = Sh::kThreads, kSoft = 128 * Sh::kWG, kRW = Sh::kRW;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *kv = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
    uint8_t *pbuf = kv + kSt * kStageBytes;
    uint8_t *qbuf = pbuf + 2 * kPBytes;
    TcShared<R> &S = *reinterpret_cast<TcShared<R> *>(qbuf + 2 * Sh::kQBytes);
    const PagedView &v = p.v;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int c = blockIdx.x;
    bool ok = true;

    if (tid == 0) {
        prefetch_tmap(&kmap);
        prefetch_tmap(&vmap);
        for (int i = 0; i < kSt; ++i) {
            mbar_init(&S.kv_full[i], 1);
            mbar_init(&S.kv_empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&S.s_full[i], 1);
            mbar_init(&S.s_empty[i], 4 * Sh::kWG);
            mbar_init(&S.p_full[i], 4 * Sh::kWG);
            mbar_init(&S.p_empty[i], 1);
            mbar_init(&S.q_full[i], 2);
            mbar_init(&S.q_empty[i], 1 + 4 * Sh::kWG);
            S.piece[i].valid = 0;
        }
        fence_mbar_init();
    }
    if (warp == 1) {
        tmem_alloc(&S.tmem, Sh::kTmemCols);
        tmem_relinquish();
    }
    pdl_wait();
    tc_fence_before_sync();
    const Line L = make_line<R, kTB>(p, S.line);  // (holds two __syncthreads)
    tc_fence_after_sync();
    auto seq_of = [&](int b) { return L.per == 1 ? S.line.seq[b] : sequence(p, b); };
    const int G = static_cast<int>(min(static_cast<long long>(gridDim.x), L.total));
    Ranges ranges = {0, 0};
    if (L.total > 0) {
        ranges.base = quot(L.total, G);
        ranges.more = L.total - ranges.base * G;
    }
    const long long u0 = c < G ? ranges.begin(c) : 0;
    const int count = c < G ? static_cast<int>(ranges.begin(c + 1) - u0) : 0;
    const uint32_t tmem = S.tmem;

    if (warp == 0 && count > 0) {
        // ---- blocks of the tiles, four tiles at a time (lane = 8 * tile + block), and their copies
        Cursor<kTB> cur = find_place<R, kTB>(p, S.line, L, u0, seq_of);
        const int sub = lane >> 3, j = lane & 7;
        if (sub < count) advance<R>(p, cur, sub, seq_of);
        int bi = -1, j0 = 0;
        float ks = 0.0f, vs = 0.0f;
        Cursor<kTB> at = cur;
        auto look_up = [&](int i0) {  // this lane's block of tile i0 + sub
            bi = -1;
            ks = vs = 0.0f;
            if (i0 + sub >= count) return;
            at = cur;
            const int kb = kTB * cur.k + j;
            if (kb < cur.tl.n) {
                const int blk = cur.tl.block(kb);
                j0 = blk * kPB;
                const int64_t x = block_index(v, cur.b, blk);
                if (x >= 0) {
                    bi = static_cast<int>(x) + cur.head * v.bpp;
                    ks = v.ks[bi];
                    vs = v.vs[bi];
                }
            }
            if (i0 + 4 + sub < count) advance<R>(p, cur, 4, seq_of);
        };
        look_up(0);
        for (int i0 = 0; i0 < count; i0 += 4) {
            const int b_now = bi, j0_now = j0;
            const float ks_now = ks, vs_now = vs;
            const Cursor<kTB> it = at;
            // masks: a block whose tokens not every row sees, or that is missing
            const int p_min = it.s.first + p.by_gq.quot(R * it.rt);
            const int p_max = it.s.first + p.by_gq.quot(min(R * it.rt + R, it.s.rows) - 1);
            const bool whole = b_now >= 0 && j0_now + kPB - 1 <= p_min &&
                               (p.window == 0 || j0_now > p_max - p.window || j0_now + kPB <= p.sinks);
            const unsigned not_whole = __ballot_sync(0xffffffffu, !whole);
            const unsigned there = __ballot_sync(0xffffffffu, b_now >= 0);
            float vmax = vs_now;
#pragma unroll
            for (int o = 1; o < 8; o <<= 1) vmax = fmaxf(vmax, __shfl_xor_sync(0xffffffffu, vmax, o));
            if (i0 + 4 < count) look_up(i0 + 4);  // in flight while the stages come free
            for (int e = 0; e < 4 && i0 + e < count; ++e) {
                const int i = i0 + e, stage = i % kSt;
                wait(&S.kv_empty[stage], ((i / kSt) + 1) & 1, ok);
                TileInfo &f = S.info[stage];
                if (sub == e) {
                    f.ks[j] = ks_now;
                    f.vs[j] = vs_now;
                    f.j0[j] = j0_now;
                    if (j == 0) {
                        f.valid = there >> (8 * e) & 255;
                        f.flags = (i == 0 || it.k == 0 ? kFirst : 0) | (it.k + 1 == it.units() ? kEnds | kLast : 0) |
                                  (i + 1 == count ? kLast : 0) | ((not_whole >> (8 * e) & 255) ? kEdge : 0);
                        f.vmax = vmax;
                        f.b = it.b;
                        f.head = it.head;
                        f.rt = it.rt;
                        f.k = it.k;
                        f.units = it.units();
                    }
                }
                __syncwarp();
                if (lane == 8 * e)
                    mbar_arrive_expect_tx(&S.kv_full[stage], __popc(there >> (8 * e) & 255) * 2 * kPB * kPD);
                __syncwarp();
                if (sub == e && b_now >= 0) {
                    uint8_t *dst = kv + stage * kStageBytes + j * kPB * kPD;
                    tma_load_2d_nohint(dst, &kmap, 0, b_now * kPB, &S.kv_full[stage]);
                    tma_load_2d_nohint(dst + kTileBytes, &vmap, 0, b_now * kPB, &S.kv_full[stage]);
                }
            }
        }
        // no copy is in flight when the CTA ends, even after a wait that ran out
        bool land = true;
        for (int i = max(0, count - kSt); i < count; ++i) wait(&S.kv_full[i % kSt], (i / kSt) & 1, land);
    } else if (warp == 1 && count > 0) {
        // ---- matrix products: QK of tile i + 1 before PV of tile i
        if (lane == 0) {
            constexpr uint32_t id_s = idesc_i8(128, Sh::kNS, 1, 1);
            constexpr uint32_t id_o = idesc_i8(128, Sh::kNP, 1, 0) | (1u << 15) | (1u << 16);  // both operands M/N-major
            int item = -1;
            auto qk = [&](int i) {
                const int stage = i % kSt;
                wait(&S.kv_full[stage], (i / kSt) & 1, ok);
                const int flags = S.info[stage].flags;
                if (flags & kFirst) {
                    ++item;
                    wait(&S.q_full[item & 1], (item >> 1) & 1, ok);
                }
                wait(&S.s_empty[i & 1], ((i >> 1) + 1) & 1, ok);
                tc_fence_after_sync();
                const uint32_t a = smem_u32(kv + stage * kStageBytes), b = smem_u32(qbuf + (item & 1) * Sh::kQBytes);
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    mma_i8_ss(tmem + (i & 1) * Sh::kNS, smem_desc_sw128(a + 32 * k), smem_desc_sw128(b + 32 * k), id_s, k > 0);
                tc_commit(&S.s_full[i & 1]);
                if (flags & kLast) tc_commit(&S.q_empty[item & 1]);
            };
            qk(0);
            for (int i = 0; i < count; ++i) {
                if (i + 1 < count) qk(i + 1);
                const int stage = i % kSt;
                wait(&S.p_full[i & 1], (i >> 1) & 1, ok);
                tc_fence_after_sync();
                const uint32_t a = smem_u32(kv + stage * kStageBytes + kTileBytes), b = smem_u32(pbuf + (i & 1) * kPBytes);
                const uint32_t acc = S.accumulate[i & 1];
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    mma_i8_ss(tmem + Sh::kO, smem_desc_sw128(a + 4096 * k), smem_desc_sw128(b + 4096 * k), id_o,
                              k > 0 || acc);
                tc_commit(&S.kv_empty[stage]);
                tc_commit(&S.p_empty[i & 1]);
            }
        }
        __syncwarp();
    } else if (warp < 4 && count > 0) {
        // ---- query digits of each item, ahead of its tiles; warp 2 the even rows, warp 3 the odd ones
        Cursor<kTB> cur = find_place<R, kTB>(p, S.line, L, u0, seq_of);
        for (int done = 0, item = 0; done < count; ++item) {
            wait(&S.q_empty[item & 1], ((item >> 1) + 1) & 1, ok);
            uint8_t *qb = qbuf + (item & 1) * Sh::kQBytes;
#pragma unroll 4
            for (int rr = warp - 2; rr < R; rr += 2) {
                const int row = R * cur.rt + rr;
                float4 x = make_float4(0, 0, 0, 0);
                if (row < cur.s.rows) {
                    const int ri = p.by_gq.quot(row);
                    x = *reinterpret_cast<const float4 *>(p.q + static_cast<int64_t>(cur.s.start + ri) * p.ldq +
                                                          (cur.head * p.GQ + row - ri * p.GQ) * kPD + 4 * lane);
                }
                const float amax = warp_max(fmaxf(fmaxf(fabsf(x.x), fabsf(x.y)), fmaxf(fabsf(x.z), fabsf(x.w))));
                // the row times 2^e: its largest value in [2^21, 2^22), so that three signed digits hold it
                const int e = max(-120, min(120, 148 - static_cast<int>(__float_as_uint(amax) >> 23)));
                const float up = __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
                const int n[4] = {__float2int_rn(x.x * up), __float2int_rn(x.y * up), __float2int_rn(x.z * up),
                                  __float2int_rn(x.w * up)};
                // digits: (n + 0x8080) ^ 0x8080 has the signed digits d0, d1 as its low bytes, d2 above
                uint32_t w[3] = {0, 0, 0};
#pragma unroll
                for (int d = 0; d < 4; ++d) {
                    const uint32_t t = static_cast<uint32_t>(n[d] + 0x8080) ^ 0x8080u;
#pragma unroll
                    for (int k = 0; k < 3; ++k) w[k] |= (t >> (8 * k) & 255u) << (8 * d);
                }
                // column of digit k of row rr: 6 (rr / 2) + 2 k + rr % 2, so that two rows' digits are neighbours
#pragma unroll
                for (int k = 0; k < 3; ++k)
                    *reinterpret_cast<uint32_t *>(qb + sw128_offset(6 * (rr >> 1) + 2 * k + (rr & 1), 4 * lane)) = w[k];
                if (lane == 0)
                    S.rowf[item & 1][rr] =
                        row < cur.s.rows ? p.scale_log2 * __uint_as_float(static_cast<uint32_t>(127 - e) << 23) : 0.0f;
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&S.q_full[item & 1]);
            const int n = min(count - done, cur.units() - cur.k);
            done += n;
            if (done < count) advance<R>(p, cur, n, seq_of);
        }
    } else if (count > 0) {
        // ---- softmax: thread = token of the tile and dimension of the output
        const int wg = (warp - 4) >> 2, w4 = warp & 3, me = tid & 127;
        const uint32_t lanes = static_cast<uint32_t>(w4) << 21;  // this warp's quarter of tensor memory
        float m[kRW], z[kRW], o[kRW], rowf[kRW];
        float vref = 1.0f, inv_vref = 1.0f;
        int chain = 0, item = -1, k_first = 0;
        for (int i = 0; i < count; ++i) {
            const int stage = i % kSt;
            const TileInfo &f = S.info[stage];
            wait(&S.kv_full[stage], (i / kSt) & 1, ok);  // the tile's info
            wait(&S.s_full[i & 1], (i >> 1) & 1, ok);
            tc_fence_after_sync();
            const int flags = f.flags;
            if (flags & kFirst) {
                ++item;
                k_first = f.k;
#pragma unroll
                for (int r = 0; r < kRW; ++r) {
                    rowf[r] = S.rowf[item & 1][kRW * wg + r];
                    m[r] = -INFINITY;
                    z[r] = o[r] = 0.0f;
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&S.q_empty[item & 1]);
            }
            // scores of this token: x[r], in log2
            float x[kRW];
            {
                uint32_t sv[3 * kRW];
                const uint32_t a = tmem + lanes + (i & 1) * Sh::kNS + 3 * kRW * wg;
#pragma unroll
                for (int h = 0; h < 3 * kRW / 8; ++h) tmem_ld8(a + 8 * h, *reinterpret_cast<uint32_t(*)[8]>(sv + 8 * h));
                tmem_wait_ld();
                tc_fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(&S.s_empty[i & 1]);
                const float ks = f.ks[me >> 4];
#pragma unroll
                for (int r = 0; r < kRW; r += 2) {
                    const uint32_t *d = sv + 3 * r;
                    const float2 d0 = make_float2(small_int(d[0]), small_int(d[1]));
                    const float2 d1 = make_float2(small_int(d[2]), small_int(d[3]));
                    const float2 d2 = make_float2(small_int(d[4]), small_int(d[5]));
                    const float2 up = make_float2(256.0f, 256.0f);
                    const float2 s2 = __fmul2_rn(__ffma2_rn(__ffma2_rn(d2, up, d1), up, d0),
                                                 __fmul2_rn(make_float2(rowf[r], rowf[r + 1]), make_float2(ks, ks)));
                    x[r] = s2.x;
                    x[r + 1] = s2.y;
                }
            }
            if (flags & kEdge) {
                const Seq s = seq_of(f.b);
                const int tok = f.j0[me >> 4] + (me & 15);
                const bool there = f.valid >> (me >> 4) & 1;
#pragma unroll
                for (int r = 0; r < kRW; ++r) {
                    const int pos = s.first + p.by_gq.quot(min(R * f.rt + kRW * wg + r, s.rows - 1));
                    if (!there || tok > pos || (p.window > 0 && tok <= pos - p.window && tok >= p.sinks)) x[r] = -INFINITY;
                }
            }
            const float vmax = f.vmax;
            bool flush = (flags & kFirst) || chain >= kMaxChain || vmax > vref || (vmax > 0.0f && vmax < vref * kVRange);
#pragma unroll
            for (int r = 0; r < kRW; ++r) flush |= x[r] > m[r];
            if (any_of<kSoft>(flush)) {
                // ---- new references: each row's largest score of the tile over all 128 tokens
#pragma unroll
                for (int r = 0; r < kRW; ++r) {
                    const float y = redux_max(x[r]);
                    if (lane == 0) S.wmax[wg][w4][r] = y;
                }
                if (!(flags & kFirst)) {
                    // what PV of the tiles before has summed: digits o_k of value 2^(8 k - 32), in units of the references
                    wait(&S.p_empty[(i - 1) & 1], ((i - 1) >> 1) & 1, ok);
                    tc_fence_after_sync();
#pragma unroll
                    for (int h = 0; h < kRW / 2; ++h) {
                        uint32_t ov[8];
                        tmem_ld8(tmem + lanes + Sh::kO + 4 * kRW * wg + 8 * h, ov);
                        tmem_wait_ld();
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            float t = static_cast<float>(static_cast<int>(ov[4 * e])) * 0x1p-32f;
                            t = fmaf(static_cast<float>(static_cast<int>(ov[4 * e + 1])), 0x1p-24f, t);
                            t = fmaf(static_cast<float>(static_cast<int>(ov[4 * e + 2])), 0x1p-16f, t);
                            t = fmaf(static_cast<float>(static_cast<int>(ov[4 * e + 3])), 0x1p-8f, t);
                            o[2 * h + e] = fmaf(t, vref, o[2 * h + e]);
                        }
                    }
                    tc_fence_before_sync();
                }
                any_of<kSoft>(false);  // the maxima of all warps are there
#pragma unroll
                for (int r = 0; r < kRW; ++r) {
                    const float top = fmaxf(fmaxf(S.wmax[wg][0][r], S.wmax[wg][1][r]),
                                            fmaxf(S.wmax[wg][2][r], S.wmax[wg][3][r]));
                    if (top > m[r]) {
                        const float mn = top + kHeadroom, back = ex2(m[r] - mn);
                        z[r] *= back;
                        o[r] *= back;
                        m[r] = mn;
                    }
                }
                if (vmax > 0.0f) {
                    vref = vmax;
                    inv_vref = 1.0f / vmax;
                }
                chain = 0;
                any_of<kSoft>(false);  // the maxima have been read
            }
            // weights and their digits
            uint32_t u[kRW];
            {
                const float up = f.vs[me >> 4] * inv_vref * 0x1p32f;
#pragma unroll
                for (int r = 0; r < kRW; ++r) {
                    const float w = ex2(x[r] - (m[r] == -INFINITY ? 0.0f : m[r]));
                    z[r] += w;
                    u[r] = to_u32_sat(w * up);
                }
            }
            wait(&S.p_empty[i & 1], ((i >> 1) + 1) & 1, ok);  // PV of tile i - 2 has read this buffer
            {
                uint8_t *row = pbuf + (i & 1) * kPBytes + me * 128;
#pragma unroll
                for (int h = 0; h < kRW / 4; ++h)
                    *reinterpret_cast<uint4 *>(row + (((kRW / 4 * wg + h) ^ (me & 7)) << 4)) =
                        make_uint4(u[4 * h], u[4 * h + 1], u[4 * h + 2], u[4 * h + 3]);
            }
            // (read before the weights are handed on: the stage and its info are free once PV has run)
            Piece pc;
            pc.valid = 1;
            pc.ends = (flags & kEnds) != 0;
            pc.b = f.b;
            pc.head = f.head;
            pc.rt = f.rt;
            pc.units = f.units;
            pc.u0 = u0 + i - f.k;
            if (tid == 128) S.accumulate[i & 1] = chain > 0;
            ++chain;
            fence_proxy_async_smem();
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(&S.p_full[i & 1]);

            if (flags & kLast) {
                // ---- the item, or this CTA's piece of it, is done
                const Seq s = seq_of(pc.b);
#pragma unroll
                for (int r = 0; r < kRW; ++r) {
                    const float y = warp_sum(z[r]);
                    if (lane == 0) S.zsum[wg][w4][r] = y;
                }
                any_of<kSoft>(false);
                wait(&S.p_empty[i & 1], (i >> 1) & 1, ok);
                tc_fence_after_sync();
                const bool complete = k_first == 0 && pc.ends;
                const int slot = k_first > 0 ? 0 : 1;
                float *rec = p.part + static_cast<int64_t>(2 * c + slot) * rec_floats(R);
#pragma unroll
                for (int h = 0; h < kRW / 2; ++h) {
                    uint32_t ov[8];
                    tmem_ld8(tmem + lanes + Sh::kO + 4 * kRW * wg + 8 * h, ov);
                    tmem_wait_ld();
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int r = 2 * h + e, rr = kRW * wg + r, row = R * pc.rt + rr;
                        float t = static_cast<float>(static_cast<int>(ov[4 * e])) * 0x1p-32f;
                        t = fmaf(static_cast<float>(static_cast<int>(ov[4 * e + 1])), 0x1p-24f, t);
                        t = fmaf(static_cast<float>(static_cast<int>(ov[4 * e + 2])), 0x1p-16f, t);
                        t = fmaf(static_cast<float>(static_cast<int>(ov[4 * e + 3])), 0x1p-8f, t);
                        t = fmaf(t, vref, o[r]);
                        const float zz = (S.zsum[wg][0][r] + S.zsum[wg][1][r]) + (S.zsum[wg][2][r] + S.zsum[wg][3][r]);
                        if (row < s.rows) {
                            if (complete) {
                                const int ri = p.by_gq.quot(row);
                                p.out[static_cast<int64_t>(s.start + ri) * p.ldo + (pc.head * p.GQ + row - ri * p.GQ) * kPD + me] =
                                    zz > 0.0f ? t / zz : 0.0f;
                            } else {
                                rec[rr * kPD + me] = t;
                                if (me == 0) *reinterpret_cast<float2 *>(rec + R * kPD + 2 * rr) = make_float2(m[r], zz);
                            }
                        }
                    }
                }
                tc_fence_before_sync();
                if (!complete && tid == 128) S.piece[slot] = pc;
                chain = 0;
                any_of<kSoft>(false);  // the sums have been read
            }
        }
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    if (warp == 1) tmem_dealloc(tmem, Sh::kTmemCols);
    const Piece pieces[2] = {S.piece[0], S.piece[1]};
    const bool cut[2] = {pieces[0].valid != 0, pieces[1].valid != 0};
    merge_cut_items<R, kNT>(p, cut, pieces, ranges, 1, S.last, seq_of);
    pdl_launch_dependents();
}

template <int R>
cudaError_t launch_rows(const AttnParams &p, const CUtensorMap &km, const CUtensorMap &vm, int ctas, cudaStream_t s) {
    static DeviceOnce once;
    int dev = 0;
    cudaError_t e = current_device(&dev);
    if (e != cudaSuccess) return e;
    e = once.run(dev, [] {
        return cudaFuncSetAttribute(attn_tc_paged_kernel<R>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    static_cast<int>(tc_smem<R>()));
    });
    if (e != cudaSuccess) return e;
    return launch_pdl(attn_tc_paged_kernel<R>, dim3(ctas), Shape<R>::kThreads, tc_smem<R>(), s, p, km, vm);
}

}  // namespace

cudaError_t launch_attention_tc(const AttnParams &p, const CUtensorMap &km, const CUtensorMap &vm, int max_rows,
                                int64_t span, int num_sms, cudaStream_t s) {
    const int R = max_rows <= 8 ? 8 : 32;
    const int64_t tiles = std::min<int64_t>(p.v.B, p.v.T) * p.v.Hkv * ceil_div(max_rows, R) * ceil_div(span, kTok);
    const int ctas = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>({tiles, num_sms, kMaxCtas})));
    return R == 8 ? launch_rows<8>(p, km, vm, ctas, s) : launch_rows<32>(p, km, vm, ctas, s);
}

}  // namespace tern
