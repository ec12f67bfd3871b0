// tern_paged_attention.cuh -- how the paged attention divides its work: the
// items of a batch, their visible blocks of 16 tokens, the line of all their
// tiles that the grid divides evenly, and the merging of divided items.
//
// The rows of one sequence that share a KV head (its tokens times the query
// heads of the group) are taken R at a time: an item.  An item's work is its
// visible blocks of 16 tokens (one scale each), eight blocks to a tile.  All
// tiles of all items form one line (by sequence, head, row tile, tile), cut
// into equal ranges, so that uneven contexts fill the GPU evenly; the lengths
// are read on the device.
#pragma once

#include "tern_paged.cuh"

namespace tern {

constexpr int kTB = 8;           // blocks of a tile
constexpr int kMaxRows = 32;     // rows of an item, at most
constexpr int kMaxCtas = 1024;   // CTAs of a launch (counters at the workspace's start)

// The copies of a tile: block j of the tile lies at place at[j] of the cache
// (in blocks of one head), -1 when it is missing.  Blocks that lie behind one
// another there are copied together, 8, 4, 2 or 1 at a time, each copy at a
// place of the tile that its size divides.
// Whether block j continues block j - 1 (a missing block is continued by none,
// not even by place 0, which is one above its -1).
__host__ __device__ constexpr bool continues_block(int before, int at) { return before >= 0 && at == before + 1; }
// log2 of the blocks that the copy beginning at block j takes, -1 when none
// begins there (the block is missing, or another's copy takes it).  follows:
// bit i when block i continues block i - 1.
__host__ __device__ constexpr int copy_size(unsigned follows, int j, int at) {
    const int size = (follows & 0xFEu) == 0xFEu ? 3 : (follows >> (j & 4) & 0xEu) == 0xEu ? 2 : follows >> (j & 6) & 2u ? 1 : 0;
    return at < 0 || (j & ((1 << size) - 1)) ? -1 : size;
}

// A partial record: [rows][kPD] sums, then (m, z) of each row.
__host__ __device__ constexpr int rec_floats(int rows) { return rows * (kPD + 2); }

// Tensor maps of the code arrays, boxes of 16 << i rows.
struct CacheMaps {
    CUtensorMap k[4], v[4];
};

struct AttnParams {
    PagedView v;
    const float *q;
    int ldq, Hq, GQ;
    FastDiv by_gq;
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

// Visible blocks of row tile rt: the k-th is block k below `sink`, else lo + k
// - sink.
struct Tiles {
    int n, sink, lo;
    __device__ __forceinline__ int block(int k) const { return k < sink ? k : lo + k - sink; }
};

template <int R>
__device__ __forceinline__ Tiles tiles_of(const AttnParams &p, const Seq &s, int rt) {
    const int r1 = min(R * rt + R, s.rows) - 1;
    const int p0 = s.first + p.by_gq.quot(R * rt), p1 = s.first + p.by_gq.quot(r1);
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
__device__ __forceinline__ int tile_count(const Tiles &t) {
    return max(1, (t.n + kTB - 1) / kTB);
}
template <int R>
__device__ __forceinline__ long long head_units(const AttnParams &p, const Seq &s) {
    long long u = 0;
#pragma unroll 1
    for (int rt = 0; rt * R < s.rows; ++rt) u += tile_count(tiles_of<R>(p, s, rt));
    return u;
}

// 1 / x within a rounding error (x not subnormal), 0 for x = 0, NaN for NaN.
__device__ __forceinline__ float recip(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return x == 0.0f ? 0.0f : y;
}

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Quotient of nonnegative numbers; 64-bit division is a long routine that
// nearly every call can do without.
__device__ __forceinline__ long long quot(long long a, long long b) {
    if (((a | b) >> 32) == 0) return static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
    return a / b;
}

// The line of `total` tiles in n ranges: the first `more` hold base + 1 tiles,
// the others base (n <= total, so none is empty).
struct Ranges {
    long long base, more;
    __device__ __forceinline__ long long begin(int i) const { return base * i + min(static_cast<long long>(i), more); }
    __device__ __forceinline__ int owner(long long u) const {
        const long long big = more * (base + 1);
        return static_cast<int>(u < big ? quot(u, base + 1) : more + quot(u - big, base));
    }
};

// A place on the line: tile k of an item.
struct Cursor {
    int b, head, rt, k;
    int ord;  // items passed since the range's first
    Seq s;
    Tiles tl;
    __device__ __forceinline__ int units() const { return tile_count(tl); }
};

template <int R, typename SeqOf>
__device__ __forceinline__ void advance(const AttnParams &p, Cursor &x, int n, SeqOf seq_of) {
    x.k += n;
#pragma unroll 1
    while (x.k >= x.units()) {
        x.k -= x.units();
        ++x.ord;
        if ((x.rt + 1) * R < x.s.rows) {
            ++x.rt;
        } else {
            x.rt = 0;
            if (++x.head == p.v.Hkv) {
                x.head = 0;
#pragma unroll 1
                do {
                    if (++x.b >= p.v.B) return;  // past the line: the caller counts its tiles
                    x.s = seq_of(x.b);
                } while (x.s.rows == 0);
            }
        }
        x.tl = tiles_of<R>(p, x.s, x.rt);
    }
}

// The line of a launch, as a CTA finds it: its first kLineThreads threads share
// out the sequences.
constexpr int kLineThreads = 256;
struct LineShared {
    long long chunk[kLineThreads];  // line index where each thread's sequences begin
    long long scan[kLineThreads / 32];
    Seq seq[kLineThreads];          // with one sequence a thread at most: the sequences
};
struct Line {
    long long total;
    int per;  // sequences of a thread
};

// (All threads of the CTA, at least kLineThreads; holds several __syncthreads.)
template <int R>
__device__ __forceinline__ Line make_line(const AttnParams &p, LineShared &S) {
    const PagedView &v = p.v;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const bool counts = tid < kLineThreads;
    Line L;
    L.per = (v.B + kLineThreads - 1) / kLineThreads;
    Seq s = {0, 0, 0, 0};
    if (counts && L.per == 1) {
        if (tid < v.B) s = sequence(p, tid);
        S.seq[tid] = s;
    }
    // sequences of many row tiles (prompts) are counted by a warp each, a row tile a lane
    const bool many = __syncthreads_or(s.rows > 2 * R);
    long long mine = 0, incl = 0;
    if (counts && L.per > 1) {
#pragma unroll 1
        for (int b = tid * L.per; b < min(v.B, tid * L.per + L.per); ++b)
            mine += v.Hkv * head_units<R>(p, sequence(p, b));
    } else if (counts && !many) {
        S.chunk[tid] = head_units<R>(p, s);  // (for now: the tiles of one KV head)
    } else if (counts) {
#pragma unroll 1
        for (int b = warp; b < v.B; b += kLineThreads / 32) {
            const Seq t = S.seq[b];
            long long n = 0;
#pragma unroll 1
            for (int rt = lane; rt * R < t.rows; rt += 32) n += tile_count(tiles_of<R>(p, t, rt));
#pragma unroll
            for (int o = 16; o >= 1; o >>= 1) n += __shfl_xor_sync(0xffffffffu, n, o);
            if (lane == 0) S.chunk[b] = n;
        }
    }
    __syncthreads();
    if (counts) {
        if (L.per == 1 && tid < v.B) mine = v.Hkv * S.chunk[tid];
        incl = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long x = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += x;
        }
        if (lane == 31) S.scan[warp] = incl;
    }
    __syncthreads();
    long long before = 0;
    L.total = 0;
#pragma unroll
    for (int w = 0; w < kLineThreads / 32; ++w) {
        if (w < warp) before += S.scan[w];
        L.total += S.scan[w];
    }
    if (counts) S.chunk[tid] = before + incl - mine;
    __syncthreads();
    return L;
}

// The place of line index u < total (warp-collective).
template <int R, typename SeqOf>
__device__ __forceinline__ Cursor find_place(const AttnParams &p, const LineShared &S, const Line &L, long long u,
                                                 SeqOf seq_of) {
    const int lane = threadIdx.x & 31;
    Cursor cur;
    int lo = 0;  // the last thread whose sequences begin at or before u
#pragma unroll 1
    for (int i = 0; i < kLineThreads / 32 && 32 * i * L.per < p.v.B; ++i) {
        const unsigned le = __ballot_sync(0xffffffffu, S.chunk[32 * i + lane] <= u && (32 * i + lane) * L.per < p.v.B);
        if (le) lo = 32 * i + 31 - __clz(le);
    }
    long long off = u - S.chunk[lo], ph;
    int b = lo * L.per;
#pragma unroll 1
    for (;; ++b) {
        cur.s = seq_of(b);
        ph = L.per == 1 ? quot((b + 1 < kLineThreads ? S.chunk[b + 1] : L.total) - S.chunk[b], p.v.Hkv)
                        : head_units<R>(p, cur.s);
        if (off < ph * p.v.Hkv || b + 1 == p.v.B) break;  // (the second: lengths that changed under the kernel end here)
        off -= ph * p.v.Hkv;
    }
    cur.b = b;
    cur.head = min(static_cast<int>(quot(off, max(ph, 1LL))), p.v.Hkv - 1);
    long long k = off - cur.head * ph;
    // the row tile, 32 at a time
#pragma unroll 1
    for (int rt0 = 0;; rt0 += 32) {
        const int rt = rt0 + lane, n = rt * R < cur.s.rows ? tile_count(tiles_of<R>(p, cur.s, rt)) : 0;
        int incl = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int x = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += x;
        }
        const unsigned past = __ballot_sync(0xffffffffu, incl > k);
        if (past || (rt0 + 32) * R >= cur.s.rows) {
            const int l = past ? __ffs(past) - 1 : 0;
            cur.rt = rt0 + l;
            cur.k = static_cast<int>(k) - (__shfl_sync(0xffffffffu, incl, l) - __shfl_sync(0xffffffffu, n, l));
            break;
        }
        k -= __shfl_sync(0xffffffffu, incl, 31);
    }
    cur.tl = tiles_of<R>(p, cur.s, cur.rt);
    cur.ord = 0;
    return cur;
}

// Row rr of an item to its place in out: four dimensions a lane.
__device__ __forceinline__ void write_row(const AttnParams &p, int start, int head, int row, float4 o, float z, int d) {
    const float iz = recip(z);
    const int i = p.by_gq.quot(row);
    *reinterpret_cast<float4 *>(p.out + static_cast<int64_t>(start + i) * p.ldo +
                                (head * p.GQ + row - i * p.GQ) * kPD + d) =
        make_float4(o.x * iz, o.y * iz, o.z * iz, o.w * iz);
}

__device__ __forceinline__ void add_scaled(float4 &o, float &z, float f, float4 x, float xz) {
    z = fmaf(f, xz, z);
    o.x = fmaf(f, x.x, o.x);
    o.y = fmaf(f, x.y, o.y);
    o.z = fmaf(f, x.z, o.z);
    o.w = fmaf(f, x.w, o.w);
}

// An item that the CTA shares with others: its range begins inside item 0
// (record in slot 2c), or ends inside item 1, which began in it (slot 2c + 1;
// the middle CTAs of an item have slot 2c alone).
struct CutItem {
    int valid;
    int head, rt;
    Seq s;
    int first, parts;  // the CTA with the item's first part, and how many have one
};

// item: the CTA's first (a = 0) or last (a = 1) item, whose first tile has line
// index u0.
__device__ __forceinline__ void note_cut(CutItem &x, const Ranges &ranges, int head, int rt, const Seq &s,
                                         long long u0, int units) {
    x.head = head;
    x.rt = rt;
    x.s = s;
    x.first = ranges.owner(u0);
    x.parts = ranges.owner(u0 + units - 1) - x.first + 1;
    x.valid = 1;
}

constexpr int kMergeParts = 10;  // records that a warp has in flight

// Items cut between CTAs: whoever finishes an item's last part merges all of
// them, in range order.  All threads of the CTA, after its records have been
// written and a __syncthreads; scratch: shared memory, R * (kPD + 4) floats, 16-byte aligned.
template <int R, int NT>
__device__ __forceinline__ void merge_cut_items(const AttnParams &p, const CutItem (&cut)[2], int (&last)[2], float *scratch) {
    constexpr int kSplit = NT / 32 >= 2 * R ? 2 : 1;  // warps of a row
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (!cut[0].valid && !cut[1].valid) return;
    if (tid < 2 && cut[tid].valid) {
        __threadfence();  // the CTA's records (ordered before this thread by the barrier) before its arrival
        const int done = atomicAdd(p.counters + cut[tid].first, 1);
        const int l = done + 1 == cut[tid].parts;
        if (l) p.counters[cut[tid].first] = 0;  // zero at rest
        __threadfence();
        last[tid] = l;
    }
    __syncthreads();
#pragma unroll 1
    for (int a = 0; a < 2; ++a) {
        if (!cut[a].valid || !last[a]) continue;
        const Seq s = cut[a].s;
        const int parts = cut[a].parts, head = cut[a].head, rt = cut[a].rt;
        // part i's record: slot 2 first + 1 for the first, 2 (first + i) behind it
        const float *base = p.part + static_cast<int64_t>(2 * cut[a].first) * rec_floats(R);
        auto offset = [](int i) { return (i == 0 ? 1 : 2 * i) * rec_floats(R); };
        const int half = (parts + kSplit - 1) / kSplit, mine = kSplit == 1 ? 0 : warp / R;
        const int begin = mine * half, end = min(parts, begin + half);
#pragma unroll 1
        for (int rr = kSplit == 1 ? warp : warp % R; rr < R && mine < kSplit; rr += kSplit == 1 ? NT / 32 : R) {
            const int row = R * rt + rr;
            if (row >= s.rows) break;
            const float *sums = base + rr * kPD + 4 * lane, *stats = base + R * kPD + 2 * rr;
            float z = 0.0f, M = -INFINITY;
            float4 o = make_float4(0, 0, 0, 0);
#pragma unroll 1
            for (int i0 = begin; i0 < end; i0 += kMergeParts) {
                const int n = min(kMergeParts, end - i0);
                float2 mz = make_float2(-INFINITY, 0.0f);
                if (lane < n) mz = __ldcg(reinterpret_cast<const float2 *>(stats + offset(i0 + lane)));
                float4 x[kMergeParts];
#pragma unroll
                for (int i = 0; i < kMergeParts; ++i)
                    x[i] = __ldcg(reinterpret_cast<const float4 *>(sums + offset(i0 + min(i, n - 1))));
                const float Mn = fmaxf(M, warp_max(mz.x));
                const float ref = Mn == -INFINITY ? 0.0f : Mn;
                const float back = ex2(M - ref);
                M = Mn;
                const float f = ex2(mz.x - ref);  // 0 past the last part
                z = z * back + warp_sum(f * mz.y);
                o = make_float4(o.x * back, o.y * back, o.z * back, o.w * back);
#pragma unroll
                for (int i = 0; i < kMergeParts; ++i) {
                    const float fi = __shfl_sync(0xffffffffu, f, i);
                    o.x = fmaf(fi, x[i].x, o.x);
                    o.y = fmaf(fi, x[i].y, o.y);
                    o.z = fmaf(fi, x[i].z, o.z);
                    o.w = fmaf(fi, x[i].w, o.w);
                }
            }
            if constexpr (kSplit == 2) {  // the second half's sums to the first half's warp
                float *sc = scratch + rr * (kPD + 4);
                if (mine == 1) {
                    *reinterpret_cast<float4 *>(sc + 4 * lane) = o;
                    if (lane == 0) *reinterpret_cast<float2 *>(sc + kPD) = make_float2(M, z);
                }
                asm volatile("barrier.cta.sync %0, 64;" ::"r"(1 + rr) : "memory");
                if (mine == 0) {
                    const float4 x = *reinterpret_cast<const float4 *>(sc + 4 * lane);
                    const float2 mz = *reinterpret_cast<const float2 *>(sc + kPD);
                    const float Mn = fmaxf(M, mz.x), ref = Mn == -INFINITY ? 0.0f : Mn, back = ex2(M - ref);
                    o = make_float4(o.x * back, o.y * back, o.z * back, o.w * back);
                    z *= back;
                    add_scaled(o, z, ex2(mz.x - ref), x, mz.y);
                }
                asm volatile("barrier.cta.sync %0, 64;" ::"r"(1 + rr) : "memory");
                if (mine == 1) continue;
            }
            write_row(p, s.start, head, row, o, z, 4 * lane);
        }
    }
}

}  // namespace tern
