// la_paged.cuh -- the paged key/value cache of global softmax attention: the
// write of new tokens into pages, one-token attention over the cache, and
// eviction by accumulated attention weight.
#pragma once

#include <cooperative_groups.h>
#include <limits.h>
#include <type_traits>

#include "la_device.cuh"
#include "sm100.cuh"

namespace la {

// The cache of one layer (layouts in la.h) as the kernels see it.
struct PagedCache {
    void *kp, *vp;
    const int *table, *lens;
    int B, Hkv, dqk, dv, num_pages, page, max_pages;
    int shift;   // log2(page) if page is a power of two, else -1
    __host__ __device__ __forceinline__ long long cap() const { return (long long)max_pages * page; }
};

// Row of slot t of (b, h) in the pool seen as [num_pages * Hkv * page] rows,
// or -1 if the table's entry is out of range.
__device__ __forceinline__ int paged_row(const PagedCache &c, int b, int h, int t)
{
    const int i = c.shift >= 0 ? t >> c.shift : t / c.page;
    const int pg = c.table[(size_t)b * c.max_pages + i];
    if ((unsigned)pg >= (unsigned)c.num_pages) return -1;
    return (pg * c.Hkv + h) * c.page + (t - i * c.page);
}

// ------------------------------------------------------------------ append

constexpr int kPagedFillThreads = 256;
constexpr int kPagedFillRows = 64;
// Blocks that a head's N tokens take, for every N (N + 63 may pass 31 bits).
__host__ __device__ constexpr int paged_fill_tiles(int N) { return (N - 1) / kPagedFillRows + 1; }
static_assert(paged_fill_tiles(1) == 1 && paged_fill_tiles(64) == 1 && paged_fill_tiles(65) == 2, "paged_fill_tiles");
static_assert(paged_fill_tiles(INT_MAX) == 1 << 25, "paged_fill_tiles");

struct PagedFillParams {
    PagedCache c;
    const void *k, *v;
    const int *n_new, *pos;
    float *weights;
    int *positions;
    int N;
    int elem;    // bytes of an element
    int width;   // bytes a copy moves at once: 16 if both rows allow it, else an element
};

// Rows `src` + i of k and v to rows[i] of the pool, for this warp's eight of the
// block's 64: a power of two of lanes copies a row pair, eight pairs in flight.
template <typename V>
__device__ __forceinline__ void fill_rows(const PagedFillParams &p, size_t src, const int *rows, int m)
{
    constexpr int U = 8;
    const PagedCache &c = p.c;
    const int pk = c.dqk * p.elem / (int)sizeof(V), pv = c.dv * p.elem / (int)sizeof(V), np = pk + pv;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int per_row = 1;
    while (per_row < np && per_row < 32) per_row <<= 1;
    const int groups = 32 / per_row, sub = lane / per_row, piece0 = lane & (per_row - 1);
    const V *k = (const V *)p.k + src * pk, *v = (const V *)p.v + src * pv;
    V *kp = (V *)c.kp, *vp = (V *)c.vp;
    constexpr int WARPS = kPagedFillThreads / 32;
    for (int i0 = warp * U * groups; i0 < m; i0 += WARPS * U * groups)
        for (int q = piece0; q < np; q += per_row) {
            const bool isk = q < pk;
            const V *from = isk ? k + q : v + (q - pk);
            V *to = isk ? kp + q : vp + (q - pk);
            const size_t stride = isk ? pk : pv;
            V x[U];
            int row[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int i = i0 + u * groups + sub;
                row[u] = i < m ? rows[i] : -1;
                if (row[u] >= 0) x[u] = from[i * stride];
            }
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (row[u] >= 0) to[row[u] * stride] = x[u];
        }
}

// One block per 64 new tokens of a (b, h): slot lens[b] + i <- token i.  A copy,
// bound by HBM: 8 prompts of 4096 tokens, 8 heads, bf16 d = 128 (268 MB read and
// written) take 43 us, 6.2 TB/s; with one pair in flight per eight lanes, 53 us.
__global__ void __launch_bounds__(kPagedFillThreads) paged_fill_kernel(const PagedFillParams p)
{
    sm100::grid_dependency_wait();
    sm100::launch_dependents();
    __shared__ int rows[kPagedFillRows];
    const PagedCache &c = p.c;
    const int tiles = paged_fill_tiles(p.N);
    const int bh = blockIdx.x / tiles, i0 = (blockIdx.x - bh * tiles) * kPagedFillRows;
    const int b = bh / c.Hkv, h = bh - b * c.Hkv;
    const int tid = threadIdx.x;
    const int len = c.lens[b], n = p.n_new ? p.n_new[b] : p.N, pos = p.pos ? p.pos[b] : 0;
    if (len < 0 || n < 0 || n > p.N || (long long)len + n > c.cap() || pos < 0) {
        if (tid == 0) report(kStatusCheck);
        return;
    }
    const int m = min(kPagedFillRows, n - i0);
    if (m <= 0) return;
    for (int i = tid; i < m; i += kPagedFillThreads) {
        const int t = len + i0 + i, row = paged_row(c, b, h, t);
        rows[i] = row;
        if (row < 0) {
            report(kStatusCheck);
            continue;
        }
        if (p.weights) p.weights[bh * c.cap() + t] = 0.f;
        if (p.positions) p.positions[bh * c.cap() + t] = pos + i0 + i;
    }
    __syncthreads();
    const size_t src = bh * (size_t)p.N + i0;
    if (p.width == 16) fill_rows<uint4>(p, src, rows, m);
    else if (p.width == 4) fill_rows<uint32_t>(p, src, rows, m);
    else fill_rows<uint16_t>(p, src, rows, m);
}

// ------------------------------------------------------- one-token attention
//
// For every sequence b and key/value head h, up to 16 query heads that share
// the head form a unit (groups of more than 16 heads are several units), and a
// unit's slots are cut into tiles of 64 or 128.  All tiles of the call, in
// (b, h, tile) order, are dealt out in contiguous ranges of equal cost, one per
// block: one long sequence or many ragged ones load every SM alike, and each
// block finds its range from lens by one scan.  A tile counts 4 and the end of a
// unit 3, as they take (1.7 and 1.3 us at d = 64 with three blocks on an SM); a
// tile belongs to the range in which its cost begins.
//
// Inside a tile each of the four warps owns a quarter of the slots, with its own
// running maximum, sum and accumulators, so warps meet only where a unit ends.  A
// unit inside one range is finished there; the parts of one that crosses ranges
// go to the workspace and the join kernel adds them, in the order of the ranges:
// with M = max m_i,
//     y = sum_i 2^(m_i - M) O_i / sum_i 2^(m_i - M) l_i      (scores in log2 units).
// O and l are formed before the division, so values above the type's largest over
// the number of slots can overflow.
// The same launch then adds the normalised weights, from the step's scores
// kept in the workspace: a weight needs the whole row's sum.

constexpr int kPagedThreads = 128;
constexpr int kPagedWarps = kPagedThreads / 32;
constexpr int kPagedJoinThreads = 128;     // of the join
constexpr int kPagedWeightBlocks = 3;      // more blocks of it per range where weights are kept (all run at once)
constexpr int kPagedRows = 16;       // query heads of a unit
constexpr int kPagedMaxGroup = 128;  // query heads per key/value head

constexpr int kTileCost = 4, kUnitCost = 3;

// A unit that crosses ranges, as the join needs it: its tiles' costs begin at
// first, first + kTileCost, ..
struct PagedSpan {
    long long first;
    int nt, b, u;   // b < 0: none
};
// What a block of the decode kernel leaves for the block of the join: where
// its range starts, and the units it shares with the ranges before and after.
struct PagedRecord {
    PagedSpan head, tail;
    int b, u, tile, tiles;   // start of the range, and its length in tiles (0: idle)
    long long at, chunk;     // where the first tile's cost begins, and the cost of a range
};

struct PagedDecodeParams {
    PagedCache c;
    const void *q, *k, *v;   // k, v: the new token, or null
    void *y;
    float *lse;
    const float *w_in;
    float *w_out;
    int *positions;
    const int *pos;
    int Hq, g, nsub, gs;     // query heads; per key/value head; units per head; heads per unit
    int tile;                // log2 of the slots per tile
    bool aligned;            // one unit per block, nothing to join
    float scale_log2;        // log2(e) / sqrt(dqk)
    int box_rows;            // slots per TMA box: 32, 16, 8 or 4, or below 4: gathered by fours
    PagedRecord *rec;        // [grid]
    float2 *ml;              // [grid][2][16]: running maximum and sum of the head and tail parts
    float *part;             // [grid][2][16][dv]: their accumulators
    float *lse2;             // [B * Hq]: log2 of the sum of exponentials (with weights)
    float *scores;           // [B * Hq][stride]: the scores in log2 units (with weights)
    long long stride;
};

// Slots that sequence b attends to, or -1 if its length or position is bad.
__device__ __forceinline__ int paged_count(const PagedDecodeParams &p, int len, int pos)
{
    const int more = p.k ? 1 : 0;
    return len < 0 || len > p.c.cap() - more || pos < 0 ? -1 : len + more;
}
__device__ __forceinline__ int paged_count(const PagedDecodeParams &p, int b)
{
    return paged_count(p, p.c.lens[b], p.pos ? p.pos[b] : 0);
}
__device__ __forceinline__ int paged_tiles(const PagedDecodeParams &p, int n)
{
    return n <= 0 ? 1 : ((n - 1) >> p.tile) + 1;
}

// Exclusive prefix of x over the block in thread order, and the total.
template <int NT, typename I>
__device__ __forceinline__ I block_scan(I x, I *part, I &total)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    I s = x;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const I o = __shfl_up_sync(0xffffffffu, s, off);
        if (lane >= off) s += o;
    }
    __syncthreads();
    if (lane == 31) part[warp] = s;
    __syncthreads();
    I before = 0;
    total = 0;
#pragma unroll
    for (int i = 0; i < NT / 32; ++i) {
        if (i < warp) before += part[i];
        total += part[i];
    }
    return before + s - x;
}

// A position in the (b, h, sub, tile) order; (h, sub) is a unit, u = h nsub + sub.
struct PagedWalk {
    int b, h, sub, tile, nt, n;
    __device__ __forceinline__ int rows(const PagedDecodeParams &p) const { return min(p.gs, p.g - sub * p.gs); }
    // its first query head, and its key/value head, of all sequences
    __device__ __forceinline__ size_t hq(const PagedDecodeParams &p) const
    {
        return (size_t)b * p.Hq + h * p.g + sub * p.gs;
    }
    __device__ __forceinline__ size_t bh(const PagedDecodeParams &p) const { return (size_t)b * p.c.Hkv + h; }
    __device__ __forceinline__ void set(const PagedDecodeParams &p, int count)
    {
        n = count;
        nt = paged_tiles(p, count);
    }
    // to the next tile (not past the last sequence); `count` gives a sequence's slots
    template <typename F>
    __device__ __forceinline__ void next(const PagedDecodeParams &p, F count)
    {
        if (++tile < nt) return;
        tile = 0;
        if (++sub < p.nsub) return;
        sub = 0;
        if (++h < p.c.Hkv) return;
        h = 0;
        ++b;
        set(p, count(b));
    }
};

// This block's range: tiles whose cost begins in [at, stop).  Sets the walk to the
// first of them; false if there is none.  `part`: kPagedWarps + 2 words of shared memory.
__device__ __forceinline__ bool paged_range(const PagedDecodeParams &p, PagedWalk &w, long long &at, long long &stop,
                                            long long *part)
{
    long long *found = part + kPagedWarps;
    const int B = p.c.B, U = p.c.Hkv * p.nsub, tid = threadIdx.x;
    if (p.aligned) {   // one unit per block
        const int u = blockIdx.x % U;
        w.b = blockIdx.x / U;
        w.h = u / p.nsub;
        w.sub = u - w.h * p.nsub;
        w.tile = 0;
        w.set(p, paged_count(p, w.b));
        at = 0;
        stop = (long long)w.nt * kTileCost;
        return true;
    }
    const int slab = (B + kPagedThreads - 1) / kPagedThreads, b0 = min(B, tid * slab), b1 = min(B, b0 + slab);
    long long mine = 0, total;
#pragma unroll 4
    for (int b = b0; b < b1; ++b) mine += (long long)paged_tiles(p, paged_count(p, b)) * kTileCost + kUnitCost;
    long long before = block_scan<kPagedThreads>(mine, part, total);
    total *= U;
    const bool small = total < INT_MAX / 2;   // (a 32-bit division is a fraction of a 64-bit one)
    long long chunk = small ? ((unsigned)total + gridDim.x - 1) / gridDim.x : (total + gridDim.x - 1) / gridDim.x;
    if (chunk < kTileCost) chunk = kTileCost;   // so that no range between two parts of a unit is without a tile
    const long long first = blockIdx.x * chunk;
    if (tid == 0) {
        PagedRecord &r = p.rec[blockIdx.x];
        r.head.b = r.tail.b = -1;
        r.tiles = 0;
        r.chunk = chunk;
    }
    if (first >= total) return false;
    stop = first + chunk < total ? first + chunk : total;
    const long long x = small ? (unsigned)first / (unsigned)U : first / U;
    if (x >= before && x < before + mine) {
        int b = b0;
        for (;; ++b) {
            const long long cost = (long long)paged_tiles(p, paged_count(p, b)) * kTileCost + kUnitCost;
            if (x < before + cost) break;
            before += cost;
        }
        found[0] = b;
        found[1] = before;
    }
    __syncthreads();
    w.b = (int)found[0];
    w.set(p, paged_count(p, w.b));
    const long long off = first - U * found[1], per = (long long)w.nt * kTileCost + kUnitCost;   // off < U * per
    int u = small ? (int)((unsigned)off / (unsigned)per) : (int)(off / per);
    const long long rem = off - u * per;
    w.tile = (int)((rem + kTileCost - 1) / kTileCost);
    at = first - rem + (long long)w.tile * kTileCost;
    if (w.tile >= w.nt) {   // the range begins at a unit's end: the next one
        at = first - rem + per;
        w.tile = 0;
        if (++u == U) {
            u = 0;
            if (++w.b == B) return false;
            w.set(p, paged_count(p, w.b));
        }
    }
    w.h = u / p.nsub;
    w.sub = u - w.h * p.nsub;
    if (at >= stop) return false;
    if (tid == 0) {
        PagedRecord &r = p.rec[blockIdx.x];
        r.b = w.b;
        r.u = u;
        r.tile = w.tile;
        r.at = at;
    }
    return true;
}

// 2^x to within 2^-22 of itself, four half steps of fp32, in one instruction: a
// score's own error is larger.  Results below 2^-126 are 0.
__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// The merge buffer: [warp][OR rows][64 columns] floats, four columns to a piece.
// Piece q of row r lies at piece q ^ (q >> 3) ^ 2 (r mod 2): the MMA kernel's
// threads write pieces 4 c + i (c = lane % 4) of rows 2 k, 2 k + 1 at once, and
// so touch every bank.
constexpr int kPagedMergeCols = 64;
__device__ __forceinline__ int paged_piece(int q, int r) { return q ^ (q >> 3 & 1) ^ (r & 1) << 1; }

// Where one unit's part of a range ends: columns col0 .. col0 + 63 of the four
// warps' rows r0 .. r0 + OR - 1 lie in obuf and their maxima and sums in mls
// [warp][16].  Finishes the rows (`whole`) or leaves them to the join as part `slot`.
template <typename T, int OR>
__device__ __forceinline__ void paged_merge(const PagedDecodeParams &p, const PagedWalk &w, const float *obuf,
                                            const float2 *mls, int r0, int col0, int rows, bool whole, int slot)
{
    const int tid = threadIdx.x, col = tid % kPagedMergeCols;
    const size_t hq0 = w.hq(p);
#pragma unroll
    for (int r = tid / kPagedMergeCols; r < OR; r += kPagedThreads / kPagedMergeCols) {
        if (r0 + r >= rows) break;
        float2 e[kPagedWarps];
        float x[kPagedWarps], M = -INFINITY, L = 0.f, acc = 0.f;
#pragma unroll
        for (int i = 0; i < kPagedWarps; ++i) {
            e[i] = mls[i * kPagedRows + r0 + r];
            x[i] = obuf[(i * OR + r) * kPagedMergeCols + 4 * paged_piece(col >> 2, r) + (col & 3)];
            M = fmaxf(M, e[i].x);
        }
        const float base = M == -INFINITY ? 0.f : M;
#pragma unroll
        for (int i = 0; i < kPagedWarps; ++i) {
            const float f = ex2(e[i].x - base);
            L = fmaf(f, e[i].y, L);
            acc = fmaf(f, x[i], acc);
        }
        if (whole) {
            const bool none = L == 0.f;   // nothing to attend to
            if (col0 + col < p.c.dv) st((T *)p.y + (hq0 + r0 + r) * p.c.dv + col0 + col, none ? 0.f : acc / L);
            if (col0 + col == 0) {
                if (p.lse) p.lse[hq0 + r0 + r] = none ? -INFINITY : M * 0.693147180559945309f + logf(L);
                if (p.lse2) p.lse2[hq0 + r0 + r] = none ? -INFINITY : M + log2f(L);
            }
        } else {
            const size_t at = ((size_t)blockIdx.x * 2 + slot) * kPagedRows + r0 + r;
            if (col0 + col < p.c.dv) p.part[at * p.c.dv + col0 + col] = acc;
            if (col0 + col == 0) p.ml[at] = make_float2(M, L);
        }
    }
}

// The end of a unit's part [t0, w.tile] of a range, at the tile that begins at
// `at`: whether it is whole, and what the join has to know if it is not.  Returns
// the slot of the part.
__device__ __forceinline__ int paged_part(const PagedDecodeParams &p, const PagedWalk &w, int t0, long long at,
                                          bool &whole)
{
    whole = t0 == 0 && w.tile == w.nt - 1;
    if (whole) return 0;
    const int slot = t0 == 0 ? 1 : 0;
    if (threadIdx.x == 0) {
        PagedSpan &s = slot ? p.rec[blockIdx.x].tail : p.rec[blockIdx.x].head;
        s.first = at - (long long)w.tile * kTileCost;
        s.nt = w.nt;
        s.b = w.b;
        s.u = w.h * p.nsub + w.sub;
    }
    return slot;
}

// The table's entry for slot t of the walk's unit, and the slot's row in the pool
// with that entry: -1 past the end or on a bad page.
__device__ __forceinline__ int paged_entry(const PagedDecodeParams &p, const PagedWalk &w, int t)
{
    if (t >= w.n) return -1;
    return p.c.table[(size_t)w.b * p.c.max_pages + (p.c.shift >= 0 ? t >> p.c.shift : t / p.c.page)];
}
__device__ __forceinline__ int paged_entry_row(const PagedDecodeParams &p, const PagedWalk &w, int t, int entry)
{
    const PagedCache &c = p.c;
    if (t >= w.n) return -1;
    if ((unsigned)entry >= (unsigned)c.num_pages) {
        report(kStatusCheck);
        return -1;
    }
    const int off = c.shift >= 0 ? t & (c.page - 1) : t % c.page;
    return (entry * c.Hkv + w.h) * c.page + off;
}

// The first `bytes` of 16 bytes from global to shared memory, zeros after them.
__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, int bytes)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
// 2D tiled load of one box into shared memory, completing on `bar`, under
// an L2 policy.
__device__ __forceinline__ void tma_load_2d_hint(void *dst, const CUtensorMap *map, uint64_t *bar, int x, int y,
                                                 uint64_t policy)
{
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint"
        " [%0], [%1, {%3, %4}], [%2], %5;" ::"r"(sm100::smem_addr(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(sm100::smem_addr(bar)), "r"(x), "r"(y), "l"(policy)
        : "memory");
}

// Four rows of a 2D tensor, from column x, into four consecutive rows of shared
// memory (the map's box is one row high), completing on `bar`.
__device__ __forceinline__ void tma_gather4(void *dst, const CUtensorMap *map, uint64_t *bar, int x, int y0, int y1,
                                            int y2, int y3)
{
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile::gather4.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5, %6, %7}], [%2];" ::"r"(sm100::smem_addr(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(sm100::smem_addr(bar)), "r"(x), "r"(y0), "r"(y1), "r"(y2), "r"(y3)
        : "memory");
}

__device__ __forceinline__ uint4 lds128(uint32_t a)
{
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
    return v;
}

// D += A B, A 16 x 16 and B 16 x 8 bf16, fp32 accumulators.
__device__ __forceinline__ void mma_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                          uint32_t b0, uint32_t b1)
{
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                 "{%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t word(const uint4 &v, int i) { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; }
__device__ __forceinline__ uint32_t bf16x2(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
// What bf16x2(lo, hi) rounded off, as bf16 again.
__device__ __forceinline__ uint32_t bf16x2_rest(float lo, float hi, uint32_t r)
{
    return bf16x2(lo - __uint_as_float(r << 16), hi - __uint_as_float(r & 0xffff0000u));
}

// Two numbers of at least 0 cut off to bf16, and what that took off, raised by 2^-23
// of the number: above 0 wherever the number is (from 2^-110 on).
__device__ __forceinline__ uint32_t bf16x2_cut(float lo, float hi)
{
    return __byte_perm(__float_as_uint(lo), __float_as_uint(hi), 0x7632u);
}
__device__ __forceinline__ uint32_t bf16x2_cut_rest(float lo, float hi, uint32_t r)
{
    constexpr float more = 1.f + 0x1p-23f;
    return bf16x2(fmaf(lo, more, -__uint_as_float(r << 16)), fmaf(hi, more, -__uint_as_float(r & 0xffff0000u)));
}

// ---- a warp's keys and values, from the pool to shared memory
//
// Each warp brings the keys, then the values, of its quarter of the next tiles
// (SLOTS slots) into its own ring of shared memory, ST loads deep.  A place of
// the ring holds blocks of 128 bytes per slot, in the 128-byte swizzle: 16-byte
// piece i of slot t lies at piece i ^ (t mod 8).  By TMA, with one mbarrier per
// place: slots of a page are neighbouring rows of the pool, so a box of
// `box_rows` rows (32, 16, 8 or 4, whichever divides the page size) is one copy
// per block; pages of other sizes gather four rows by index.  Rows that do not
// start on 16 bytes cannot be copied by TMA: the 16-byte pieces that cover a run
// of rows come by cp.async into a ring of their own, and the lanes spread the
// elements into one place, as floats, when they are needed.
// Nothing but the wait for its own copies orders a warp inside a unit.
//
// What the consumer has to know of a tile (below) lies beside the ring, so only
// the loads walk through the sequences; the length of the sequence after the
// walk's is on its way while the walk is in this one.
struct PagedTile {
    uint32_t mask;     // slots attended to
    uint32_t copies;   // copies that fill them: 0, nothing to wait for
    int newrow;        // row of the new token if it is among them, else -1
    int n, b, h, sub, tile;
    bool last;         // of the range (kept in the top bit of sub)
};

// Tiles kept beside the ring: with at most four places, the keys of tile i + 2
// are asked for after tile i has been read, and tile i + 1 is still there.
constexpr int kPagedAhead = 2;
constexpr int kPagedTileBytes = 32;   // of a tile beside the ring

template <typename T, typename E, int KB, int VB, int SLOTS, int ST, bool TMA>
struct PagedFeed {
    static_assert(ST <= 4, "kPagedAhead");
    static constexpr uint32_t ALL = 0xffffffffu;
    static constexpr int BLOCK = SLOTS * 128, PLACE = (KB > VB ? KB : VB) * BLOCK;
    static constexpr int COLS = 128 / sizeof(E);   // elements of a block's row: E in shared memory, T in the pool
    // a warp's shared memory: the ring; or one place, the ring of raw rows (at worst
    // every row a run of its own) and where each slot's row begins in it
    static constexpr int RAW = SLOTS * ((KB > VB ? KB : VB) * COLS * (int)sizeof(T) + 30) / 16 * 16;
    static constexpr int BYTES = TMA ? ST * PLACE : (PLACE + ST * (RAW + SLOTS * 2) + 127) / 128 * 128;
    const PagedDecodeParams &p;
    const CUtensorMap *tm_k, *tm_v;
    uint8_t *ring;
    uint64_t *full;
    int4 *tiles_at;
    PagedWalk w;                 // the tile whose loads are next, and where its cost begins
    long long at, stop;
    bool done, values;           // no tile is left to begin; its values are next
    int issued, place_in, place_out, warp, lane, entry, row;
    int next_len, next_pos;      // of sequence w.b + 1
    uint32_t copies, pending, phases;
    bool alive;                  // false once a wait ran out: tiles go by without loads and without slots

    __device__ __forceinline__ PagedFeed(const PagedDecodeParams &p_, const CUtensorMap *k, const CUtensorMap *v,
                                         uint8_t *ring_, uint64_t *full_, uint8_t *tiles_, const PagedWalk &w_,
                                         long long at_, long long stop_)
        : p(p_), tm_k(k), tm_v(v), ring(ring_), full(full_), tiles_at(reinterpret_cast<int4 *>(tiles_)), w(w_), at(at_),
          stop(stop_), done(false), values(false), issued(0), place_in(0), place_out(0), warp(threadIdx.x >> 5),
          lane(threadIdx.x & 31), row(-1), copies(0), pending(0), phases(0), alive(true)
    {
        ahead();
        entry = paged_entry(p, w, slot());
    }
    __device__ __forceinline__ int slot() const
    {
        return SLOTS == 32 || lane < SLOTS ? (w.tile * 4 + warp) * SLOTS + lane : INT_MAX;
    }
    __device__ __forceinline__ void ahead()
    {
        next_len = next_pos = 0;
        if (w.b + 1 < p.c.B) {
            next_len = p.c.lens[w.b + 1];
            if (p.pos) next_pos = p.pos[w.b + 1];
        }
    }
    __device__ __forceinline__ void advance()
    {
        const int b = w.b;
        w.next(p, [&](int) { return paged_count(p, next_len, next_pos); });
        if (w.b != b) ahead();
        entry = paged_entry(p, w, slot());
    }
    // the next load into the ring, if there is one
    __device__ __forceinline__ void issue()
    {
        using namespace sm100;
        if (done && !values) {
            if (!TMA) cp_async_commit();   // every load is a group, so that the wait can count them
            return;
        }
        const bool isv = values;
        values = !values;
        const int group = p.box_rows < 4 ? 4 : p.box_rows < SLOTS ? p.box_rows : SLOTS;   // slots per copy
        if (!isv) {
            row = alive ? paged_entry_row(p, w, slot(), entry) : -1;
            const uint32_t mask = __ballot_sync(ALL, row >= 0);
            const bool fresh = p.k && row >= 0 && slot() == w.n - 1;   // the new token: not in the pool yet
            const uint32_t newmask = __ballot_sync(ALL, fresh), held = mask & ~newmask;
            const int newrow = newmask ? __shfl_sync(ALL, row, __ffs(newmask) - 1) : -1;
            // a box lies in one page: its first slot is held if any is; four gathered
            // rows are brought in if any is held
            copies = 0;
            if (TMA) copies = __ballot_sync(ALL, (lane & (group - 1)) == 0 && (held >> lane & (group == 32 ? ALL : (1u << group) - 1)));
            else if (fresh) row = -1;
            if (!TMA) copies = held;
            at += kTileCost + (w.tile + 1 < w.nt ? 0 : kUnitCost);
            done = at >= stop;
            if (lane == 0) {
                int4 *to = tiles_at + issued % kPagedAhead * 2;
                to[0] = make_int4((int)mask, (int)copies, newrow, w.n);
                to[1] = make_int4(w.b, w.h, w.sub | (done ? INT_MIN : 0), w.tile);
            }
            ++issued;
            if (!done) advance();
        }
        if (!alive) copies = 0;
        if (copies) {
            uint8_t *dst = ring + place_in * PLACE;
            if constexpr (TMA) {
                const CUtensorMap *map = isv ? tm_v : tm_k;
                if (lane == 0) mbar_arrive_expect_tx(full + place_in, __popc(copies) * group * 128 * (isv ? VB : KB));
                int y1, y2, y3;   // of rows that are not held: row 0 or the new token's, whose places are not used
                if (p.box_rows < 4) {
                    y1 = max(__shfl_down_sync(ALL, row, 1), 0);
                    y2 = max(__shfl_down_sync(ALL, row, 2), 0);
                    y3 = max(__shfl_down_sync(ALL, row, 3), 0);
                }
                __syncwarp();
                if (copies >> lane & 1) {
                    const uint64_t policy = policy_evict_first();
#pragma unroll
                    for (int j = 0; j < (KB > VB ? KB : VB); ++j) {
                        if (j >= (isv ? VB : KB)) break;
                        if (p.box_rows < 4)
                            tma_gather4(dst + j * BLOCK + lane * 128, map, full + place_in, j * COLS, max(row, 0), y1, y2, y3);
                        else
                            tma_load_2d_hint(dst + j * BLOCK + lane * 128, map, full + place_in, j * COLS, row, policy);
                    }
                }
                pending |= 1u << place_in;
            } else {
                const int rb = (isv ? p.c.dv : p.c.dqk) * (int)sizeof(T), run = p.box_rows < SLOTS ? p.box_rows : SLOTS;
                const int stride = (run * rb + 30) / 16 * 16;   // a run and what its alignment adds
                const uint8_t *pool = (const uint8_t *)(isv ? p.c.vp : p.c.kp);
                const size_t end = (size_t)p.c.num_pages * p.c.Hkv * p.c.page * rb;
                const uint32_t raw = sm100::smem_addr(ring + PLACE + place_in * RAW);
                for (int s = 0; s < SLOTS; s += run) {
                    // a run lies in one page: its first slot is held if any is
                    const int first = __shfl_sync(ALL, row, s);
                    if (first < 0) continue;
                    const size_t start = (size_t)first * rb, from = start & ~(size_t)15;
                    const int skip = (int)(start - from), at = s / run * stride;
                    for (int i = lane * 16; i < skip + run * rb; i += 512)
                        cp_async16(raw + at + i, pool + from + i, from + i + 16 <= end ? 16 : (int)(end - from - i));
                    if (lane < run) offsets()[place_in * SLOTS + s + lane] = (uint16_t)(at + skip + lane * rb);
                }
            }
        }
        if (!TMA) cp_async_commit();
        if (++place_in == ST) place_in = 0;
    }
    __device__ __forceinline__ uint16_t *offsets() const { return reinterpret_cast<uint16_t *>(ring + PLACE + ST * RAW); }
    // the next place of the ring, once its copies (a mask of them) have landed; rows of d elements
    __device__ __forceinline__ uint8_t *take(uint32_t copied, int d)
    {
        uint8_t *at = ring;
        if constexpr (TMA) {
            if (copied && alive) {
                alive = __all_sync(ALL, sm100::mbar_wait(full + place_out, phases >> place_out & 1));
                if (alive) {
                    phases ^= 1u << place_out;
                    pending &= ~(1u << place_out);
                }
            }
            at += place_out * PLACE;
        } else {
            cp_async_wait<ST - 2>();
            __syncwarp();
            const T *raw = reinterpret_cast<const T *>(ring + PLACE + place_out * RAW);
#pragma unroll 4
            for (int s = 0; s < SLOTS; ++s) {
                const T *from = raw + offsets()[place_out * SLOTS + s] / sizeof(T);
                float *to = reinterpret_cast<float *>(ring + s * 128 + ((lane >> 2 ^ (s & 7)) << 4)) + (lane & 3);
                if (copied >> s & 1)
                    for (int j = 0; j * 32 + lane < (d + 31) / 32 * 32; ++j)
                        to[j * (BLOCK / 4)] = j * 32 + lane < d ? ld(from + j * 32 + lane) : 0.f;
            }
            __syncwarp();
        }
        if (++place_out == ST) place_out = 0;
        return at;
    }
    // The new token's row of a place is stale: the caller's k or v takes its
    // place (zeros past d, as in a copy), and goes to its row of the pool.
    __device__ __forceinline__ void patch(uint8_t *dst, const T *src, T *pool, int d, int blocks, const PagedTile &t)
    {
        const int s = t.n - 1 - (t.tile * 4 + warp) * SLOTS;
        constexpr int PE = 16 / sizeof(E);   // elements of a 16-byte piece
        for (int i = lane; i < blocks * 8; i += 32) {
            E x[PE];
#pragma unroll
            for (int e = 0; e < PE; ++e) x[e] = E(0.f);
            if constexpr (TMA) {
                if (i * PE < d) *reinterpret_cast<uint4 *>(x) = *reinterpret_cast<const uint4 *>(src + i * PE);
                if (i * PE < d && t.sub == 0)
                    *reinterpret_cast<uint4 *>(pool + (size_t)t.newrow * d + i * PE) = *reinterpret_cast<const uint4 *>(x);
            } else {
#pragma unroll
                for (int e = 0; e < PE; ++e)
                    if (i * PE + e < d) {
                        const T y = src[i * PE + e];
                        x[e] = E(ld(&y));
                        if (t.sub == 0) pool[(size_t)t.newrow * d + i * PE + e] = y;
                    }
            }
            *reinterpret_cast<uint4 *>(dst + (i >> 3) * BLOCK + s * 128 + (((i ^ s) & 7) << 4)) = *reinterpret_cast<const uint4 *>(x);
        }
        if (TMA) sm100::fence_proxy_async();   // before a later copy writes this place
        __syncwarp();
    }
    // Masked slots have no weight, but their rows of a place may hold anything,
    // and 0 * NaN is NaN: zeros.
    __device__ __forceinline__ void clear(uint8_t *dst, int blocks, uint32_t mask)
    {
        if (lane < SLOTS && !(mask >> lane & 1))
            for (int i = 0; i < blocks * 8; ++i)
                *reinterpret_cast<uint4 *>(dst + (i >> 3) * BLOCK + lane * 128 + (((i ^ lane) & 7) << 4)) = make_uint4(0u, 0u, 0u, 0u);
        if (TMA) sm100::fence_proxy_async();   // before a later copy writes this place
        __syncwarp();
    }
    __device__ __forceinline__ PagedTile tile(int it) const
    {
        const int4 *from = tiles_at + it % kPagedAhead * 2;
        const int4 x = from[0], y = from[1];
        PagedTile t;
        t.mask = (uint32_t)x.x;
        t.copies = (uint32_t)x.y;
        t.newrow = x.z;
        t.n = x.w;
        t.b = y.x;
        t.h = y.y;
        t.sub = y.z & INT_MAX;
        t.tile = y.w;
        t.last = y.z < 0;
        return t;
    }
    // after a wait that ran out, let this warp's own copies land before leaving (bounded)
    __device__ __forceinline__ void drain()
    {
        if (TMA && !alive)
            for (int i = 0; i < ST; ++i)
                if (pending >> i & 1) sm100::mbar_wait(full + i, phases >> i & 1, 100000000ull);
    }
};

__device__ __forceinline__ PagedWalk paged_unit(const PagedDecodeParams &p, const PagedTile &t)
{
    PagedWalk w;
    w.b = t.b;
    w.h = t.h;
    w.sub = t.sub;
    w.tile = t.tile;
    w.set(p, t.n);
    return w;
}

// The new token's position goes beside its slot.
__device__ __forceinline__ void paged_store_position(const PagedDecodeParams &p, const PagedWalk &w)
{
    if (p.positions && threadIdx.x == 0 && w.sub == 0 && w.n > 0 && w.tile == w.nt - 1 &&
        paged_row(p.c, w.b, w.h, w.n - 1) >= 0)
        p.positions[w.bh(p) * p.c.cap() + w.n - 1] = p.pos[w.b];
}

// A permutation of 0..7: the slot (of eight) whose key thread lane / 4 reads.
// With the swizzle it lets the reads of both kernels touch every bank once:
// eight lanes read 16 bytes each at a time, and they are rows slot(2i),
// slot(2i+1) (which differ in bit 2) for keys, and rows slot(0), slot(2),
// slot(4), slot(6) (which differ above bit 0) for the values of the MMA kernel.
__device__ __forceinline__ int paged_slot(int r)
{
    return ((r ^ r >> 2) & 1) << 2 | (r & 2) | r >> 2;
}

// bf16, dqk and dv multiples of 8, on the tensor cores with mma.sync: the work
// per byte (2 * heads FLOP) is far below what a tcgen05 tile is for, and its 16
// rows hold the query heads.
//
// The operands go from shared memory to the MMA's registers without a
// transpose, because a sum does not depend on the order of its terms and a
// matrix product not on the order of its columns:
//   S = Q K^T  thread (r = lane / 4, c = lane % 4) reads 8 consecutive
//       coordinates 32 j + 8 c .. + 7 of key slot(r) (+ 8 i): the two k-steps
//       2j, 2j + 1 take them as their coordinates 2c, 2c+1, 2c+8, 2c+9; Q is
//       held in the same order.
//   O = P V    thread (r, c) reads the values 64 j + 8 r .. + 7 of the slots
//       slot(2c), slot(2c+1) (+ 8 i): a byte permutation pairs two slots, and
//       column block e of the product is the values 64 j + 8 r + e.
// P enters as two bf16 halves, p = hi + lo.  With at most 8 heads (HI false) the
// low half takes the rows 8..15, which are free, and costs no further MMA.
// An infinite value v asks that hi v + lo v is p v: hi has p's sign, and is 0 only
// where p is, but a low half of 0 would give NaN, and one below 0 (hi rounded up)
// the other infinity.  With at most 8 heads the halves' sums lie apart, and where
// the high one is not finite the low one is left out; hi is rounded to nearest
// (error of p 2^-17; 2^-9 without a low half).  With more, both halves go to one
// sum, so p is cut off and the low half kept above 0 (error 2^-16).  Finding
// infinite values by a vote instead, which keeps 2^-17, took 35 us instead of 31
// (16 sequences of 8192, 16 heads, d = 128) and 76 instead of 63 (4096, 72 on 8).
// A score's products are exact and its sum is the tensor core's, which adds 16 of
// them at a time in fp32 and may cut off where FMA would round.  Neither these nor
// P's halves show beside y's own rounding (2^-9): against 64 bits y is 0.0017 of
// its norm off, as is a form that holds all of them in fp32.
//
// Bound by HBM at long contexts: 131,072 slots, 32 query heads on 8, d = 128
// (537 MB) take 90 us a step, join included, 5.9 TB/s.  A chunk of 32 slots is
// about 750 warp instructions; with chunks of 16 (590 each) eight warps per SM
// issued too slowly, 127 us.  Short contexts are bound by a block's chain of
// latencies: about 3 us to its first rows, 1.7 us a tile, 1.3 us a unit's end.
// With 9 to 16 heads two warps on a scheduler do not hide their own latencies: 16
// sequences of 4096, 128 heads on 8, d = 128 (268 MB) take 74 us a step, 56 % of
// the measured copy bandwidth, with the tensor pipe at 23 % and a scheduler issuing
// in one cycle of three; an instruction waits 2.1 cycles for fixed latencies, 0.6 for
// shared memory.  Groups above 16 read their keys again for each 16 heads, from L2: 8
// sequences of 16,384, 128 heads on one, 104 us, DRAM 78 MB for 67 of keys and values.

// Shared memory to ask for so that not more than `blocks` blocks fit an SM.  The
// ranges are dealt out for so many: a launch that begins while the last one's
// join is still leaving some SMs could otherwise put more blocks on the others.
constexpr int paged_smem(int need, int blocks)
{
    const int least = 228 * 1024 / (blocks + 1) - 1024 + 128;
    return need > least ? need : least;
}

template <int DQ, int DV, bool HI>
struct PagedMma {
    static constexpr int KB = DQ / 64, VB = DV / 64;           // 64-column blocks
    static constexpr int ST = KB > 1 || VB > 1 ? 3 : 4;
    using Feed = PagedFeed<__nv_bfloat16, __nv_bfloat16, KB, VB, 32, ST, true>;
    static constexpr int BLOCK = Feed::BLOCK;
    static constexpr int OFF_O = kPagedWarps * Feed::BYTES;
    static constexpr int OFF_ML = OFF_O + kPagedWarps * 8 * kPagedMergeCols * 4;
    static constexpr int OFF_TILE = OFF_ML + kPagedWarps * kPagedRows * 8;
    static constexpr int OFF_BAR = OFF_TILE + kPagedWarps * kPagedAhead * kPagedTileBytes;
    static constexpr int BLOCKS = KB > 1 || VB > 1 ? 2 : 3;    // per SM
    static constexpr int SMEM = paged_smem(OFF_BAR + kPagedWarps * ST * 8, BLOCKS);
    static constexpr int REGS = BLOCKS == 3 ? 168 : HI ? 248 : 224;   // 224: the join fits beside two blocks
    static_assert(BLOCKS * (SMEM + 1024) <= 228 * 1024, "shared memory of an SM");
};

template <int DQ, int DV, bool HI>
__global__ void __launch_bounds__(kPagedThreads) __maxnreg__((PagedMma<DQ, DV, HI>::REGS))
paged_decode_mma_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                        const PagedDecodeParams p)
{
    using Cfg = PagedMma<DQ, DV, HI>;
    using T = __nv_bfloat16;
    using namespace sm100;
    constexpr uint32_t ALL = 0xffffffffu;
    extern __shared__ __align__(1024) uint8_t smem[];   // swizzled tiles from the start; no static shared memory before it
    const PagedCache &c = p.c;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, r = lane >> 2, cq = lane & 3;
    float *obuf = reinterpret_cast<float *>(smem + Cfg::OFF_O);
    float2 *mls = reinterpret_cast<float2 *>(smem + Cfg::OFF_ML);
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + Cfg::OFF_BAR) + warp * Cfg::ST;
    if (lane == 0) {
        for (int i = 0; i < Cfg::ST; ++i) mbar_init(full + i, 1);
        mbar_init_fence();
        if (warp == 0) {
            prefetch_tensormap(&tm_k);
            prefetch_tensormap(&tm_v);
        }
    }
    grid_dependency_wait();
    launch_dependents();

    PagedWalk w;
    long long at, stop;
    if (!paged_range(p, w, at, stop, reinterpret_cast<long long *>(obuf))) return;
    __syncthreads();   // the barriers are set, and obuf is free
    typename Cfg::Feed feed(p, &tm_k, &tm_v, smem + warp * Cfg::Feed::BYTES, full,
                            smem + Cfg::OFF_TILE + warp * kPagedAhead * kPagedTileBytes, w, at, stop);
#pragma unroll 1
    for (int s = 0; s < Cfg::ST - 1; ++s) feed.issue();

    const int sk = paged_slot(r), sv0 = paged_slot(2 * cq), sv1 = paged_slot(2 * cq + 1);
    const uint32_t off_k = sk * 128 + ((cq ^ sk) << 4);   // coordinates 32 j + ..: ^ 64 for odd j, + a block per two
    const uint32_t off_v0 = sv0 * 128 + ((r ^ sv0) << 4), off_v1 = sv1 * 128 + ((r ^ sv1) << 4);

    constexpr int NR = HI ? 2 : 1;   // rows of a thread: r and r + 8
    uint4 qf[DQ / 32][NR];
    float o[DV / 8][4], m[NR], l[NR];
    auto load_q = [&](const PagedWalk &u) {
        const int rows = u.rows(p);
        const T *q = (const T *)p.q + u.hq(p) * c.dqk;
#pragma unroll
        for (int j = 0; j < DQ / 32; ++j)
#pragma unroll
            for (int i = 0; i < NR; ++i) {
                const int col = j * 32 + cq * 8, row = r + 8 * i;
                qf[j][i] = make_uint4(0u, 0u, 0u, 0u);
                if (row < rows && col < c.dqk) qf[j][i] = *reinterpret_cast<const uint4 *>(q + row * c.dqk + col);
            }
    };
    load_q(w);
    int t0 = 0;
    for (int it = 0;; ++it) {
        __syncwarp();
        const PagedTile t = feed.tile(it);
        w = paged_unit(p, t);
        if (it == 0 || w.tile == 0) {   // a new unit
            t0 = w.tile;
#pragma unroll
            for (int i = 0; i < DV / 8; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
#pragma unroll
            for (int i = 0; i < NR; ++i) {
                m[i] = -INFINITY;
                l[i] = 0.f;
            }
        }
        const uint32_t mask = t.mask;
        const int rows = w.rows(p);
        float *const sc = p.scores ? p.scores + (w.hq(p) + r) * p.stride + (w.tile << 7) + warp * 32 : nullptr;
        uint8_t *kp = feed.take(t.copies, c.dqk);
        feed.issue();   // into the place before, which every lane has used; with it the next tile is known
        uint32_t hi[4][NR], lo[4][NR];   // P: [slots 8 i + sv.][row]
        if (mask && feed.alive) {
            if (t.newrow >= 0) feed.patch(kp, (const T *)p.k + w.bh(p) * c.dqk, (T *)c.kp, c.dqk, Cfg::KB, t);
            const uint32_t ks = smem_addr(kp);
            float s[4][4];
#pragma unroll
            for (int i = 0; i < 4; ++i) s[i][0] = s[i][1] = s[i][2] = s[i][3] = 0.f;
#pragma unroll
            for (int j = 0; j < DQ / 32; ++j) {
                const uint4 a = qf[j][0], b = HI ? qf[j][NR - 1] : make_uint4(0u, 0u, 0u, 0u);
                uint4 kk[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) kk[i] = lds128(ks + (j >> 1) * Cfg::BLOCK + i * 1024 + (off_k ^ (j & 1) * 64));
#pragma unroll
                for (int i = 0; i < 4; ++i) mma_16816(s[i], a.x, b.x, a.y, b.y, kk[i].x, kk[i].y);
#pragma unroll
                for (int i = 0; i < 4; ++i) mma_16816(s[i], a.z, b.z, a.w, b.w, kk[i].z, kk[i].w);
            }
            // scores in log2 units; slot of s[i][e] (and s[i][e + 2]): 8 i + sv_e
            float mn[NR];
#pragma unroll
            for (int n = 0; n < NR; ++n) {
                mn[n] = -INFINITY;
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float &x = s[i][n * 2 + e];
                        x = mask >> (8 * i + (e ? sv1 : sv0)) & 1 ? x * p.scale_log2 : -INFINITY;
                        mn[n] = fmaxf(mn[n], x);
                    }
                mn[n] = fmaxf(mn[n], __shfl_xor_sync(ALL, mn[n], 1));
                mn[n] = fmaxf(mn[n], __shfl_xor_sync(ALL, mn[n], 2));
                mn[n] = fmaxf(mn[n], m[n]);
                if (sc && r + 8 * n < rows)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        sc[8 * n * p.stride + 8 * i + sv0] = s[i][n * 2];
                        sc[8 * n * p.stride + 8 * i + sv1] = s[i][n * 2 + 1];
                    }
            }
            bool grew = mn[0] != m[0];
            if (HI) grew |= mn[NR - 1] != m[NR - 1];
            if (__any_sync(ALL, grew)) {
                float al[NR];
#pragma unroll
                for (int n = 0; n < NR; ++n) {
                    al[n] = ex2(m[n] - (mn[n] == -INFINITY ? 0.f : mn[n]));
                    l[n] *= al[n];
                    m[n] = mn[n];
                }
#pragma unroll
                for (int i = 0; i < DV / 8; ++i) {
                    o[i][0] *= al[0];
                    o[i][1] *= al[0];
                    o[i][2] *= al[NR - 1];
                    o[i][3] *= al[NR - 1];
                }
            }
#pragma unroll
            for (int n = 0; n < NR; ++n) {
                const float base = m[n] == -INFINITY ? 0.f : m[n];
                float sum = 0.f;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float e0 = ex2(s[i][n * 2] - base), e1 = ex2(s[i][n * 2 + 1] - base);
                    sum += e0 + e1;
                    hi[i][n] = HI ? bf16x2_cut(e0, e1) : bf16x2(e0, e1);
                    lo[i][n] = HI ? bf16x2_cut_rest(e0, e1, hi[i][n]) : bf16x2_rest(e0, e1, hi[i][n]);
                }
                l[n] += sum;
            }
        } else if (sc && w.n > 0) {   // slots past the end, or on bad pages: no weight
#pragma unroll
            for (int n = 0; n < NR; ++n)
                if (r + 8 * n < rows)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        sc[8 * n * p.stride + 8 * i + sv0] = sc[8 * n * p.stride + 8 * i + sv1] = -INFINITY;
        }
        // the next unit's queries are on their way while this one is finished
        if (!t.last && w.tile == w.nt - 1) {
            __syncwarp();
            load_q(paged_unit(p, feed.tile(it + 1)));
        }
        uint8_t *vp = feed.take(t.copies, c.dv);
        feed.issue();
        if (mask && feed.alive) {
            if (t.newrow >= 0) feed.patch(vp, (const T *)p.v + w.bh(p) * c.dv, (T *)c.vp, c.dv, Cfg::VB, t);
            if (mask != ALL) feed.clear(vp, Cfg::VB, mask);
            const uint32_t vs = smem_addr(vp);
#pragma unroll
            for (int j = 0; j < DV / 64; ++j) {
                if (j * 64 >= c.dv) break;
#pragma unroll
                for (int kk = 0; kk < 2; ++kk) {
                    uint4 vv[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        vv[i] = lds128(vs + (i & 1 ? off_v1 : off_v0) + (2 * kk + (i >> 1)) * 1024 + j * Cfg::BLOCK);
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const uint32_t sel = e & 1 ? 0x7632u : 0x5410u;
                        const uint32_t b0 = __byte_perm(word(vv[0], e / 2), word(vv[1], e / 2), sel);
                        const uint32_t b1 = __byte_perm(word(vv[2], e / 2), word(vv[3], e / 2), sel);
                        float(&d)[4] = o[j * 8 + e];
                        if (HI) {
                            mma_16816(d, hi[2 * kk][0], hi[2 * kk][NR - 1], hi[2 * kk + 1][0], hi[2 * kk + 1][NR - 1], b0, b1);
                            mma_16816(d, lo[2 * kk][0], lo[2 * kk][NR - 1], lo[2 * kk + 1][0], lo[2 * kk + 1][NR - 1], b0, b1);
                        } else {
                            mma_16816(d, hi[2 * kk][0], lo[2 * kk][0], hi[2 * kk + 1][0], lo[2 * kk + 1][0], b0, b1);
                        }
                    }
                }
            }
        }
        if (w.tile == w.nt - 1 || t.last) {   // the unit, or its part in this range, ends
            bool whole;
            const int slot = paged_part(p, w, t0, at, whole);
            if (w.n < 0) {
                if (w.h == 0 && w.sub == 0 && tid == 0) report(kStatusCheck);
            } else {
#pragma unroll
                for (int n = 0; n < NR; ++n) {
                    l[n] += __shfl_xor_sync(ALL, l[n], 1);
                    l[n] += __shfl_xor_sync(ALL, l[n], 2);
                    if (cq == 0) mls[warp * kPagedRows + r + 8 * n] = make_float2(m[n], l[n]);
                }
#pragma unroll
                for (int n = 0; n < NR; ++n)
#pragma unroll
                    for (int j = 0; j < DV / 64; ++j) {
                        float4 *to = reinterpret_cast<float4 *>(obuf + (warp * 8 + r) * kPagedMergeCols);
                        if (r + 8 * n < rows)
#pragma unroll
                            for (int e = 0; e < 2; ++e)
#pragma unroll
                                for (int f = 0; f < 2; ++f) {
                                    float x[4];
#pragma unroll
                                    for (int i = 0; i < 4; ++i) {
                                        const float *oo = o[j * 8 + f * 4 + i];
                                        x[i] = HI || !(fabsf(oo[e]) < INFINITY) ? oo[n * 2 + e] : oo[e] + oo[e + 2];
                                    }
                                    to[paged_piece(cq * 4 + e * 2 + f, r)] = make_float4(x[0], x[1], x[2], x[3]);
                                }
                        __syncthreads();
                        paged_merge<T, 8>(p, w, obuf, mls, 8 * n, 64 * j, rows, whole, slot);
                        __syncthreads();
                    }
                paged_store_position(p, w);
            }
        }
        at += kTileCost + (w.tile + 1 < w.nt ? 0 : kUnitCost);
        if (t.last) {
            if (tid == 0 && !p.aligned) p.rec[blockIdx.x].tiles = it + 1;
            break;
        }
    }
    feed.drain();
}

// fp32, and bf16 rows that do not start on 16-byte boundaries: the same walk
// with fp32 FMA on four floats per 16-byte piece.  A quad of lanes shares a slot
// in the scores (lane c holds the coordinates 16 j + 4 c .. + 3 of slots slot(r)
// and 8 + slot(r)), and a lane owns four columns of the output.  The queries are
// scaled to log2 units in fp32 before the products, one rounding of each, where the
// scores would take one each.
// Bound by HBM with a head of keys for each query head (16 sequences of up to 4096
// slots, 16 heads, d = 64, 303 MB: 57 us a step, 5.3 TB/s), with shared heads by the
// latencies that two warps on a scheduler leave open: 16 sequences of 2048, 64 heads
// on 8, d = 128 (268 MB) take 97 us a step, the FMA pipe at 22 % and a scheduler
// issuing in two cycles of five; an instruction waits 1.2 cycles for fixed latencies
// and 1.1 for shared memory (a query read of 16 bytes feeds 8 FMA).  Rows off 16
// bytes are bound the same way by their spreading: bf16 d = 127, 16 sequences of
// 4096, 8 heads (266 MB) 243 us, fixed latencies 1.9 cycles, shared memory 1.4.
template <typename T, int D, int GM, bool TMA>
struct PagedSimt {
    static constexpr int NB = D / 32;                // 32-column blocks
    static constexpr int ST = !TMA || (D > 64 && GM > 8) ? 2 : 3;
    static constexpr int OR = GM < 8 ? GM : 8;       // rows merged at once
    using Feed = PagedFeed<T, float, NB, NB, 16, ST, TMA>;
    static constexpr int BLOCK = Feed::BLOCK;
    static constexpr int LR = D / 4, TP = 32 / LR;   // lanes per value row, rows per pass
    static constexpr int OFF_O = kPagedWarps * Feed::BYTES;
    static constexpr int OFF_Q = OFF_O + kPagedWarps * OR * kPagedMergeCols * 4;   // [GM][D] queries, shared by the warps
    static constexpr int OFF_P = OFF_Q + GM * D * 4;                       // [warp][16][GM] weights
    static constexpr int OFF_ML = OFF_P + kPagedWarps * 16 * GM * 4;
    static constexpr int OFF_TILE = OFF_ML + kPagedWarps * kPagedRows * 8;
    static constexpr int OFF_BAR = OFF_TILE + kPagedWarps * kPagedAhead * kPagedTileBytes;
    static constexpr int BLOCKS = D > 64 && GM > 4 && !TMA && sizeof(T) == 4 ? 1 : D > 64 || GM > 8 ? 2 : 3;   // per SM
    static constexpr int SMEM = paged_smem(OFF_BAR + kPagedWarps * ST * 8, BLOCKS);
    static_assert(BLOCKS * (SMEM + 1024) <= 228 * 1024, "shared memory of an SM");
};

__device__ __forceinline__ float4 lds_f4(uint32_t a)
{
    const uint4 v = lds128(a);
    return make_float4(__uint_as_float(v.x), __uint_as_float(v.y), __uint_as_float(v.z), __uint_as_float(v.w));
}

template <typename T, int D, int GM, bool TMA>
__global__ void __launch_bounds__(kPagedThreads, PagedSimt<T, D, GM, TMA>::BLOCKS)
paged_decode_simt_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                         const PagedDecodeParams p)
{
    using Cfg = PagedSimt<T, D, GM, TMA>;
    using namespace sm100;
    constexpr uint32_t ALL = 0xffffffffu;
    extern __shared__ __align__(1024) uint8_t smem[];
    const PagedCache &c = p.c;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, r = lane >> 2, cq = lane & 3;
    const int vcol = (lane % Cfg::LR) * 4, vrow = lane / Cfg::LR;
    float *obuf = reinterpret_cast<float *>(smem + Cfg::OFF_O);
    float *qs = reinterpret_cast<float *>(smem + Cfg::OFF_Q);
    float *ps = reinterpret_cast<float *>(smem + Cfg::OFF_P) + warp * 16 * GM;
    float2 *mls = reinterpret_cast<float2 *>(smem + Cfg::OFF_ML);
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + Cfg::OFF_BAR) + warp * Cfg::ST;
    if (TMA && lane == 0) {
        for (int i = 0; i < Cfg::ST; ++i) mbar_init(full + i, 1);
        mbar_init_fence();
        if (warp == 0) {
            prefetch_tensormap(&tm_k);
            prefetch_tensormap(&tm_v);
        }
    }
    grid_dependency_wait();
    launch_dependents();

    PagedWalk w;
    long long at, stop;
    if (!paged_range(p, w, at, stop, reinterpret_cast<long long *>(obuf))) return;
    __syncthreads();
    typename Cfg::Feed feed(p, &tm_k, &tm_v, smem + warp * Cfg::Feed::BYTES, full,
                            smem + Cfg::OFF_TILE + warp * kPagedAhead * kPagedTileBytes, w, at, stop);
#pragma unroll 1
    for (int s = 0; s < Cfg::ST - 1; ++s) feed.issue();

    const int sk = paged_slot(r);
    const uint32_t off_k = sk * 128 + ((cq ^ sk) << 4);   // coordinates 16 j + ..: ^ 64 for odd j, + a block per two
    const uint32_t off_v = (vcol / 32) * Cfg::BLOCK;
    constexpr int F = GM < 4 ? GM : 4;
    float4 o[GM];
    float m[GM], l[GM];
    int t0 = 0;
    for (int it = 0;; ++it) {
        __syncwarp();
        const PagedTile t = feed.tile(it);
        w = paged_unit(p, t);
        const int rows = w.rows(p);
        const size_t hq0 = w.hq(p);
        if (it == 0 || w.tile == 0) {
            t0 = w.tile;
            __syncthreads();   // the queries of the last unit are read
            for (int i = tid; i < GM * D; i += kPagedThreads) {
                const int row = i / D, col = i - row * D;
                qs[i] = row < rows && col < c.dqk ? ld((const T *)p.q + (hq0 + row) * c.dqk + col) * p.scale_log2 : 0.f;
            }
            __syncthreads();
#pragma unroll
            for (int n = 0; n < GM; ++n) {
                o[n] = make_float4(0.f, 0.f, 0.f, 0.f);
                m[n] = -INFINITY;
                l[n] = 0.f;
            }
        }
        const uint32_t mask = t.mask;
        uint8_t *kp = feed.take(t.copies, c.dqk);
        feed.issue();
        if (mask && feed.alive) {
            if (t.newrow >= 0) feed.patch(kp, (const T *)p.k + w.bh(p) * c.dqk, (T *)c.kp, c.dqk, Cfg::NB, t);
            const uint32_t ks = smem_addr(kp);
            // heads go by in groups of four without a branch between them, so that
            // their loads and sums overlap (a head past `rows` has zeros for a query)
            float s[2][GM];
#pragma unroll
            for (int n = 0; n < GM; ++n) s[0][n] = s[1][n] = 0.f;
#pragma unroll
            for (int j = 0; j < D / 16; ++j) {
                if (j * 16 >= c.dqk) break;
                const float4 k0 = lds_f4(ks + (j >> 1) * Cfg::BLOCK + (off_k ^ (j & 1) * 64));
                const float4 k1 = lds_f4(ks + (j >> 1) * Cfg::BLOCK + 1024 + (off_k ^ (j & 1) * 64));
#pragma unroll
                for (int n0 = 0; n0 < GM; n0 += F) {
                    if (n0 >= rows) break;
                    float4 x[F];
#pragma unroll
                    for (int n = 0; n < F; ++n) x[n] = *reinterpret_cast<const float4 *>(qs + (n0 + n) * D + j * 16 + cq * 4);
#pragma unroll
                    for (int n = 0; n < F; ++n) {
                        float &s0 = s[0][n0 + n], &s1 = s[1][n0 + n];
                        s0 = fmaf(x[n].x, k0.x, fmaf(x[n].y, k0.y, fmaf(x[n].z, k0.z, fmaf(x[n].w, k0.w, s0))));
                        s1 = fmaf(x[n].x, k1.x, fmaf(x[n].y, k1.y, fmaf(x[n].z, k1.z, fmaf(x[n].w, k1.w, s1))));
                    }
                }
            }
#pragma unroll
            for (int n0 = 0; n0 < GM; n0 += F) {
                if (n0 >= rows) break;
                float mx[F];
#pragma unroll
                for (int n = 0; n < F; ++n) {
                    mx[n] = m[n0 + n];
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        float x = s[i][n0 + n];
                        x += __shfl_xor_sync(ALL, x, 1);
                        x += __shfl_xor_sync(ALL, x, 2);
                        s[i][n0 + n] = x = mask >> (i * 8 + sk) & 1 ? x : -INFINITY;
                        mx[n] = fmaxf(mx[n], x);
                        if (p.scores && cq == 0 && n0 + n < rows)
                            p.scores[(hq0 + n0 + n) * p.stride + (w.tile << 6) + warp * 16 + i * 8 + sk] = x;
                    }
                }
#pragma unroll
                for (int off = 4; off < 32; off <<= 1)
#pragma unroll
                    for (int n = 0; n < F; ++n) mx[n] = fmaxf(mx[n], __shfl_xor_sync(ALL, mx[n], off));
#pragma unroll
                for (int n = 0; n < F; ++n) {
                    const int nn = n0 + n;
                    const float base = mx[n] == -INFINITY ? 0.f : mx[n], al = ex2(m[nn] - base);
                    m[nn] = mx[n];
                    const float e0 = ex2(s[0][nn] - base), e1 = ex2(s[1][nn] - base);
                    l[nn] = l[nn] * al + e0 + e1;
                    if (cq == (nn & 3)) {
                        ps[sk * GM + nn] = e0;
                        ps[(8 + sk) * GM + nn] = e1;
                    }
                    o[nn].x *= al;
                    o[nn].y *= al;
                    o[nn].z *= al;
                    o[nn].w *= al;
                }
            }
            __syncwarp();
            uint8_t *vp = feed.take(t.copies, c.dv);
            feed.issue();
            if (t.newrow >= 0 && feed.alive) feed.patch(vp, (const T *)p.v + w.bh(p) * c.dv, (T *)c.vp, c.dv, Cfg::NB, t);
            const uint32_t vs = smem_addr(vp) + off_v;
            if (feed.alive) {
                if (mask != 0xffffu) feed.clear(vp, Cfg::NB, mask);
#pragma unroll
                for (int i = 0; i < 16 / Cfg::TP; ++i) {
                    const int row = i * Cfg::TP + vrow;
                    const float4 x = lds_f4(vs + row * 128 + (((lane ^ row) & 7) << 4));
                    const float *pp = ps + row * GM;
#pragma unroll
                    for (int n0 = 0; n0 < GM; n0 += F) {
                        if (n0 >= rows) break;
                        __align__(16) float f[F];
                        if constexpr (F == 4) *reinterpret_cast<float4 *>(f) = *reinterpret_cast<const float4 *>(pp + n0);
                        else f[0] = pp[0];
#pragma unroll
                        for (int n = n0; n < n0 + F; ++n) {
                            o[n].x = fmaf(f[n - n0], x.x, o[n].x);
                            o[n].y = fmaf(f[n - n0], x.y, o[n].y);
                            o[n].z = fmaf(f[n - n0], x.z, o[n].z);
                            o[n].w = fmaf(f[n - n0], x.w, o[n].w);
                        }
                    }
                }
            }
            __syncwarp();   // the weights are read before the next tile's
        } else {
            if (p.scores && w.n > 0 && cq == 0)
                for (int n = 0; n < rows; ++n)
                    for (int i = 0; i < 2; ++i)
                        p.scores[(hq0 + n) * p.stride + (w.tile << 6) + warp * 16 + i * 8 + r] = -INFINITY;
            feed.take(0, c.dv);
            feed.issue();
        }
        if (w.tile == w.nt - 1 || t.last) {
            bool whole;
            const int slot = paged_part(p, w, t0, at, whole);
            if (w.n < 0) {
                if (w.h == 0 && w.sub == 0 && tid == 0) report(kStatusCheck);
            } else {
#pragma unroll
                for (int n = 0; n < GM; ++n) {   // a slot's weight is held by its quad's four lanes alike
#pragma unroll
                    for (int off = 4; off < 32; off <<= 1) l[n] += __shfl_xor_sync(ALL, l[n], off);
                    if (Cfg::TP == 2) {
                        o[n].x += __shfl_xor_sync(ALL, o[n].x, 16);
                        o[n].y += __shfl_xor_sync(ALL, o[n].y, 16);
                        o[n].z += __shfl_xor_sync(ALL, o[n].z, 16);
                        o[n].w += __shfl_xor_sync(ALL, o[n].w, 16);
                    }
                    if (lane == 0) mls[warp * kPagedRows + n] = make_float2(m[n], l[n]);
                }
#pragma unroll
                for (int n0 = 0; n0 < GM; n0 += 8)
#pragma unroll
                    for (int c0 = 0; c0 < D; c0 += kPagedMergeCols) {
#pragma unroll
                        for (int n = n0; n < GM && n < n0 + 8; ++n)
                            if (vrow == 0 && vcol >= c0 && vcol < c0 + kPagedMergeCols)
                                *reinterpret_cast<float4 *>(obuf + (warp * Cfg::OR + n - n0) * kPagedMergeCols +
                                                            4 * paged_piece((vcol - c0) >> 2, n - n0)) = o[n];
                        __syncthreads();
                        paged_merge<T, Cfg::OR>(p, w, obuf, mls, n0, c0, min(rows, GM), whole, slot);
                        __syncthreads();
                    }
                paged_store_position(p, w);
            }
        }
        at += kTileCost + (w.tile + 1 < w.nt ? 0 : kUnitCost);
        if (t.last) {
            if (tid == 0 && !p.aligned) p.rec[blockIdx.x].tiles = it + 1;
            break;
        }
    }
    feed.drain();
}

// a / b of non-negative numbers (a 32-bit division is a fraction of a 64-bit one)
__device__ __forceinline__ int paged_div(long long a, long long b)
{
    return (int)(a <= INT_MAX && b <= INT_MAX ? (unsigned)a / (unsigned)b : a / b);
}

// Maximum and sum of row `row` over the parts of a unit that crosses ranges.
__device__ __forceinline__ float2 paged_part_ml(const PagedDecodeParams &p, int g0, int i, int row)
{
    return p.ml[((size_t)(g0 + i) * 2 + (i == 0 ? 1 : 0)) * kPagedRows + row];
}

// Joins a unit's parts.  The K ranges that hold them share the work: their
// blocks take equal slices of the unit's rows x dv outputs, and KL neighbouring
// lanes share one output's parts (as many as leave one output to each group, so
// that the loads of a lane, one after the other, are few).
template <typename T>
__device__ __forceinline__ void paged_join(const PagedDecodeParams &p, const PagedSpan &s, long long chunk, int range)
{
    const int g0 = paged_div(s.first, chunk), g1 = paged_div(s.first + (s.nt - 1ll) * kTileCost, chunk);
    const int K = g1 - g0 + 1, dv = p.c.dv;
    const int h = s.u / p.nsub, sub = s.u - h * p.nsub, rows = min(p.gs, p.g - sub * p.gs);
    const size_t hq0 = (size_t)s.b * p.Hq + h * p.g + sub * p.gs;
    const int E = rows * dv, per = (E + K - 1) / K, e0 = (range - g0) * per, e1 = min(E, e0 + per);
    int KL = 1;
    while (KL < K && KL < 32 && per * KL * 2 <= kPagedJoinThreads) KL <<= 1;
    const int mine = threadIdx.x & (KL - 1);
    for (int base = e0; base < e1; base += kPagedJoinThreads / KL) {   // the same count for every thread
        const int e = base + threadIdx.x / KL;
        const bool on = e < e1;
        const int row = on ? e / dv : 0, col = on ? e - row * dv : 0;
        // one pass: maximum, sum and accumulator of eight parts at a time
        float M = -INFINITY, L = 0.f, acc = 0.f;
        for (int i0 = mine; i0 < K; i0 += 8 * KL) {
            float2 ml[8];
            float x[8], mx = M;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int i = i0 + j * KL;
                ml[j] = make_float2(-INFINITY, 0.f);
                x[j] = 0.f;
                if (i < K) {
                    ml[j] = paged_part_ml(p, g0, i, row);
                    x[j] = p.part[(((size_t)(g0 + i) * 2 + (i == 0 ? 1 : 0)) * kPagedRows + row) * dv + col];
                }
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) mx = fmaxf(mx, ml[j].x);
            const float base = mx == -INFINITY ? 0.f : mx, f = ex2(M - base);
            L *= f;
            acc *= f;
            M = mx;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float e = ex2(ml[j].x - base);
                L = fmaf(e, ml[j].y, L);
                acc = fmaf(e, x[j], acc);
            }
        }
        for (int off = 1; off < KL; off <<= 1) {
            const float m2 = __shfl_xor_sync(0xffffffffu, M, off), l2 = __shfl_xor_sync(0xffffffffu, L, off);
            const float a2 = __shfl_xor_sync(0xffffffffu, acc, off), mx = fmaxf(M, m2);
            const float base = mx == -INFINITY ? 0.f : mx, f = ex2(M - base), f2 = ex2(m2 - base);
            L = L * f + l2 * f2;
            acc = acc * f + a2 * f2;
            M = mx;
        }
        if (on && mine == 0) {
            const bool none = L == 0.f;
            st((T *)p.y + (hq0 + row) * dv + col, none ? 0.f : acc / L);
            if (col == 0 && p.lse) p.lse[hq0 + row] = none ? -INFINITY : M * 0.693147180559945309f + logf(L);
        }
    }
}

// One block per range joins; with weights kPagedWeightBlocks more add the
// weights of a part of the range's tiles each.  A chain of three loads (record,
// parts, output): about 5 us after the decode kernel; with weights 10 us at 64
// sequences of 2112 slots and 32 heads (scores of 17 MB).
template <typename T, bool WEIGHTS>
__global__ void __launch_bounds__(kPagedJoinThreads, 9) paged_join_kernel(const PagedDecodeParams p)
{
    sm100::grid_dependency_wait();
    sm100::launch_dependents();
    constexpr int PER = WEIGHTS ? kPagedWeightBlocks + 1 : 1;
    const int range = blockIdx.x / PER, share = blockIdx.x % PER;
    const PagedRecord &rec = p.rec[range];
    const int tiles = rec.tiles;
    if (!tiles) return;
    const long long per_range = rec.chunk;
    if (share == PER - 1) {
        const PagedSpan head = rec.head, tail = rec.tail;
        if (head.b >= 0) paged_join<T>(p, head, per_range, range);
        if (tail.b >= 0) paged_join<T>(p, tail, per_range, range);
        return;
    }
    if constexpr (!WEIGHTS) return;
    __shared__ float lse2[kPagedMaxGroup];
    // weights of the range's slots, each head's first unit for all its units
    const PagedCache &c = p.c;
    const int tid = threadIdx.x;
    PagedWalk w;
    w.b = rec.b;
    w.h = rec.u / p.nsub;
    w.sub = rec.u - w.h * p.nsub;
    w.tile = rec.tile;
    w.set(p, paged_count(p, w.b));
    auto count = [&](int b) { return paged_count(p, b); };
    // this block's tiles of the range
    const int from = (int)((long long)tiles * share / kPagedWeightBlocks);
    int left = (int)((long long)tiles * (share + 1) / kPagedWeightBlocks) - from;
    long long at = rec.at;
    auto step = [&](int here) {   // past `here` tiles of the unit
        at += (long long)here * kTileCost + (w.tile + here < w.nt ? 0 : kUnitCost);
        w.tile += here - 1;
        w.next(p, count);
    };
    for (int skip = from; skip > 0;) {
        const int here = min(skip, w.nt - w.tile);
        step(here);
        skip -= here;
    }
    while (left > 0) {
        const int here = min(left, w.nt - w.tile);
        if (w.sub == 0 && w.n > 0) {
            const size_t hq0 = w.hq(p), bh = w.bh(p);
            __syncthreads();
            for (int j = tid; j < p.g; j += kPagedJoinThreads) {
                const int sub = j / p.gs;
                // where this head's unit begins: the units of a sequence follow one another
                const long long cost = (long long)w.nt * kTileCost;
                const long long first = at - (long long)w.tile * kTileCost + sub * (cost + kUnitCost);
                const int g0 = paged_div(first, per_range), g1 = paged_div(first + cost - kTileCost, per_range);
                if (g0 == g1) {
                    const float x = p.lse2[hq0 + j];
                    lse2[j] = x == -INFINITY ? INFINITY : x;   // nothing attended to: 2^(s - inf) = 0
                } else {
                    float M = -INFINITY, L = 0.f;
#pragma unroll 8
                    for (int i = 0; i <= g1 - g0; ++i) M = fmaxf(M, paged_part_ml(p, g0, i, j - sub * p.gs).x);
#pragma unroll 8
                    for (int i = 0; i <= g1 - g0; ++i) {
                        const float2 e = paged_part_ml(p, g0, i, j - sub * p.gs);
                        L = fmaf(ex2(e.x - (M == -INFINITY ? 0.f : M)), e.y, L);
                    }
                    lse2[j] = L == 0.f ? INFINITY : M + log2f(L);
                }
            }
            __syncthreads();
            // four neighbouring slots per thread: a tile's scores start on 16 bytes
            const int end = min((long long)w.n, (long long)(w.tile + here) << p.tile);
            const float *wi = p.w_in + bh * c.cap();
            float *wo = p.w_out + bh * c.cap();
            const bool vec = ((reinterpret_cast<uintptr_t>(wi) | reinterpret_cast<uintptr_t>(wo)) & 15) == 0;
            const int fresh = p.k ? w.n - 1 : -1;
            for (int t = (w.tile << p.tile) + 4 * tid; t < end; t += 4 * kPagedJoinThreads) {
                __align__(16) float sum[4], old[4];
                const bool four = vec && t + 4 <= end;
                if (four) {
                    *reinterpret_cast<float4 *>(old) = *reinterpret_cast<const float4 *>(wi + t);
                } else {
#pragma unroll
                    for (int e = 0; e < 4; ++e) old[e] = t + e < end ? wi[t + e] : 0.f;
                }
#pragma unroll
                for (int e = 0; e < 4; ++e) sum[e] = 0.f;
                const float *sc = p.scores + hq0 * p.stride + t;
#pragma unroll 4
                for (int j = 0; j < p.g; ++j, sc += p.stride) {
                    const float4 s = *reinterpret_cast<const float4 *>(sc);
                    const float L = lse2[j];
                    sum[0] += ex2(s.x - L);
                    sum[1] += ex2(s.y - L);
                    sum[2] += ex2(s.z - L);
                    sum[3] += ex2(s.w - L);
                }
#pragma unroll
                for (int e = 0; e < 4; ++e) old[e] = (t + e == fresh ? 0.f : old[e]) + sum[e];
                if (four) {
                    *reinterpret_cast<float4 *>(wo + t) = *reinterpret_cast<const float4 *>(old);
                } else {
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (t + e < end) wo[t + e] = old[e];
                }
            }
        }
        left -= here;
        if (left > 0) step(here);
    }
}

// ------------------------------------------------------------------ eviction

struct PagedEvictParams {
    PagedCache c;
    int *lens_out;
    const float *w_in;
    float *w_out;
    const int *pos_in;
    int *pos_out;
    const int *pos;
    int *holes, *movers;   // [B*Hkv, maxmoves] each
    int *newlen;           // [B]; null: lens_out is written by the first kernel
    int budget, recent, maxmoves;
    int elem;              // bytes of an element
    int width;             // bytes a row copy moves at once: 16 if both rows allow it, else an element
    int keys;              // keys that fit the block's shared memory
};

constexpr int kEvictThreads = 256;
constexpr int kEvictWarps = kEvictThreads / 32;
constexpr int kEvictMaxKeys = 12288;
constexpr int kEvictMaxCluster = 8;

// Blocks per (b, h) of an eviction, `units` of them, of tables of `cap` slots: more
// while
//   - all blocks run at once, with at least 1024 slots each.  Clusters have two
//     blocks on an SM and lie within a GPC: 144 of 2 and 64 of 4 ran at once, 32 of
//     8 mostly did; 152, 74 and 40 did not.  2112 -> 2048 slots, 152 heads: 12 us
//     alone, 23 in clusters of 2; 8256 -> 8192, 74 heads: 23 alone, 19 of 2, 27 of 4;
//     64 heads of 32,768 -> 4096: 76 of 4, 86 of 8.  (Where a fourth of the slots
//     stays, the rows weigh more and a second round is about even: 8192 -> 2048, 200
//     heads: 108 alone, 96 of 2; 512 heads 215 and 205.)  Blocks of fewer slots cost
//     more than they save (1088 -> 1024: 9.4 alone, 11.7 of 2; at 2112 -> 2048 it is
//     11 to 13, but where half the slots go, 22 to 18).
//   - or the table's keys do not fit the blocks' shared memory and the blocks run in
//     two rounds: keys are then made anew in each sweep (32,768 -> 4096, 144 heads:
//     310 of 2, 177 of 4).
//   - or the keys of twice the budget do not fit, however many blocks that takes.
//     A longer sequence is right too; that cap itself fits is not asked for, since a
//     table may be far wider than what it holds (512 heads of 32,768 -> 4096: 1396
//     alone, 506 of 4; but 4160 -> 4096 in the same table 22 and 102).
constexpr int paged_evict_cluster(long long units, long long cap, long long budget)
{
    const long long likely = cap < 2 * budget + 1024 ? cap : 2 * budget + 1024;
    int cs = 1;
    while (cs < kEvictMaxCluster) {
        const long long more = cs * 2, keys = (long long)cs * kEvictMaxKeys;
        const bool at_once = units * more <= (more == 2 ? 288 : 256) && cap >= more * 1024;
        const bool two_rounds = cap > keys && units * more <= 592;
        if (!at_once && !two_rounds && likely <= keys) break;
        cs = (int)more;
    }
    return cs;
}
static_assert(paged_evict_cluster(512, 2112, 2048) == 1 && paged_evict_cluster(152, 2112, 2048) == 1 &&
                  paged_evict_cluster(144, 2112, 2048) == 2 && paged_evict_cluster(32, 32768, 4096) == 8 &&
                  paged_evict_cluster(64, 32768, 4096) == 4 && paged_evict_cluster(74, 8256, 8192) == 2 &&
                  paged_evict_cluster(144, 32768, 4096) == 4 && paged_evict_cluster(512, 32768, 4096) == 1 &&
                  paged_evict_cluster(4096, 1 << 20, 1 << 19) == 8,
              "paged_evict_cluster");

// Weight as an unsigned key of the same order: larger weight, larger key; NaN
// counts as -inf and -0 as +0.  No weight has the key 0 or 2^32 - 1.
__device__ __forceinline__ uint32_t weight_key(float w)
{
    if (!(w == w)) w = -INFINITY;
    const uint32_t u = __float_as_uint(w + 0.f);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// Moves this block's share of the list.  A warp takes up to 32 moves, one lane
// looks up each of them and moves its weight and position, and then a power of
// two of lanes copies each row pair, U pairs in flight.
template <typename V, int U>
__device__ __forceinline__ void evict_rows(const PagedEvictParams &p, int b, int h, const int *holes,
                                           const int *movers, int m, int rank, int blocks)
{
    constexpr uint32_t ALL = 0xffffffffu;
    const PagedCache &c = p.c;
    const int pk = c.dqk * p.elem / (int)sizeof(V), pv = c.dv * p.elem / (int)sizeof(V), np = pk + pv;
    const int lane = threadIdx.x & 31, warps = blocks * kEvictWarps, wid = rank * kEvictWarps + (threadIdx.x >> 5);
    int per_row = 1;
    while (per_row < np && per_row < 32) per_row <<= 1;
    const int groups = 32 / per_row, sub = lane / per_row, piece0 = lane & (per_row - 1);
    const int share = min(32, (m + warps - 1) / warps);
    V *kp = (V *)c.kp, *vp = (V *)c.vp;
    for (int i0 = wid * share; i0 < m; i0 += warps * share) {
        const int cnt = min(share, m - i0);
        int to = 0, from = 0;
        if (lane < cnt) {
            const int hole = holes[i0 + lane], mover = movers[i0 + lane];
            to = paged_row(c, b, h, hole);
            from = paged_row(c, b, h, mover);
            const size_t base = ((size_t)b * c.Hkv + h) * c.cap();
            p.w_out[base + hole] = p.w_in[base + mover];
            if (p.pos_out) p.pos_out[base + hole] = p.pos_in[base + mover];
        }
        for (int i = 0; i < cnt; i += U * groups) {
            int rt[U], rf[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int j = i + u * groups + sub;
                rt[u] = __shfl_sync(ALL, to, j & 31);
                rf[u] = __shfl_sync(ALL, from, j & 31);
                if (j >= cnt) rt[u] = -1;
            }
            for (int q = piece0; q < np; q += per_row) {
                V x[U];
                const bool isk = q < pk;
                V *base = isk ? kp + q : vp + (q - pk);
                const size_t stride = isk ? pk : pv;
#pragma unroll
                for (int u = 0; u < U; ++u)
                    if (rt[u] >= 0) x[u] = base[rf[u] * stride];
#pragma unroll
                for (int u = 0; u < U; ++u)
                    if (rt[u] >= 0) base[rt[u] * stride] = x[u];
            }
        }
    }
}

// The sum of a warp's value over the warps before this one, and over all.
// `part` (kEvictWarps words) must not be in use: two buffers in turn.
__device__ __forceinline__ int warps_before(int x, int *part, int &total)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (lane == 0) part[warp] = x;
    __syncthreads();
    int s = lane < kEvictWarps ? part[lane] : 0;
#pragma unroll
    for (int off = 1; off < kEvictWarps; off <<= 1) {
        const int o = __shfl_up_sync(0xffffffffu, s, off);
        if (lane >= off) s += o;
    }
    total = __shfl_sync(0xffffffffu, s, kEvictWarps - 1);
    return __shfl_sync(0xffffffffu, s, warp) - x;
}

// One block, or a cluster of them, per (b, h), each block with a slice of the slots.
// The order is one of 32-bit keys: a recent token's is the largest, the others
// follow their weights.  A radix select (one block: digits of 11, 11 and 10 bits; a
// cluster: four of 8, its blocks adding their histograms over distributed shared
// memory) finds the smallest key that is kept and how many slots of that key are;
// sweeps in slot order then rank the ties, list the dropped slots below the budget
// and the kept ones above it, and move rows, weights and positions along the two
// lists.  Sources lie at or above the budget and destinations below it, so moves
// need no order.
//
// One page over a budget of 2048, 512 heads of d = 128: 16.7 us a call in a row (20
// through the binding, 21 in place, with lens written by a second launch).  All
// blocks run at once, each a chain of latencies: its average end is at 13.1 us
// (start 0.7, keys and table 2.8, select 3.8, counts 1.7, lists 2.0, rows 2.1), the
// last at 16.2; the select's end alone lies between 4.8 and 9.6.  32,768 slots to
// 4096, 32 heads, clusters of 8: 48 us in a row, 50 through the binding.  The blocks
// end at 36 on average and the last at 41 (start 0.6, keys and table 6.0, select 8.0,
// counts 2.0, lists 5.6, rows 13.3), but in about one call of three a cluster finds
// no place and begins at 31.  Seven cluster barriers are in these figures, and the
// rows (117 MB) alone would take 18 at the measured copy rate.
template <int U, int BLOCKS, bool CLUSTER>
__global__ void __launch_bounds__(kEvictThreads, BLOCKS) paged_evict_kernel(const PagedEvictParams p)
{
    extern __shared__ __align__(16) int evict_smem[];
    constexpr int BITS = CLUSTER ? 8 : 11, BINS = 1 << BITS;   // digits of the radix select
    __shared__ __align__(16) int hist[2][BINS];
    __shared__ int part[2][kEvictWarps], pick[3];
    __shared__ int xch[5];   // read by the cluster's other blocks
    namespace cg = cooperative_groups;
    sm100::grid_dependency_wait();
    sm100::launch_dependents();
    // a cluster of up to kEvictMaxCluster blocks, or one block alone
    const int CS = CLUSTER ? (int)cg::this_cluster().num_blocks() : 1;
    const int rank = CLUSTER ? (int)cg::this_cluster().block_rank() : 0;
    auto sync_all = [&]() {
        if constexpr (CLUSTER) cg::this_cluster().sync();
        else __syncthreads();
    };
    const PagedCache &c = p.c;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const size_t bh = blockIdx.x / CS;
    const int b = (int)(bh / c.Hkv), h = (int)(bh - (size_t)b * c.Hkv);
    const int n = c.lens[b], budget = p.budget;
    const long long last = p.recent ? (long long)p.pos[b] : 0;
    const float *w = p.w_in + bh * c.cap();
    float *wo = p.w_out + bh * c.cap();
    const int *ps = p.pos_in ? p.pos_in + bh * c.cap() : nullptr;
    int *po = p.pos_out ? p.pos_out + bh * c.cap() : nullptr;
    const bool first = rank == 0 && h == 0 && tid == 0;   // writes the sequence's length
    int *const len_to = p.newlen ? p.newlen : p.lens_out;

    // every block of a cluster sees the same n, so all of them leave here or none
    if (n < 0 || n > c.cap() || last < 0 || n <= budget) {
        const bool bad = n < 0 || n > c.cap() || last < 0;
        if (bad && rank == 0 && tid == 0) report(kStatusCheck);
        if (first && (!bad || p.newlen)) len_to[b] = n;
        if (!bad)
            for (int t = rank * kEvictThreads + tid; t < n; t += CS * kEvictThreads) {
                if (wo != w) wo[t] = w[t];
                if (po != ps) po[t] = ps[t];
            }
        return;
    }

    // slots [s0, s1) of this block, a whole number of 32 per warp: [a0, a1)
    const int per = (n + CS * kEvictThreads - 1) / (CS * kEvictThreads) * kEvictThreads;
    const int s0 = min(n, rank * per), s1 = min(n, s0 + per);
    const int a0 = s0 + warp * (per / kEvictWarps), a1 = min(s1, a0 + per / kEvictWarps);
    uint32_t *keys = reinterpret_cast<uint32_t *>(evict_smem);
    const bool cached = per <= p.keys;
    auto is_recent = [&](int t) { return p.recent && ps[t] >= last - p.recent; };
    // if the recent tokens alone exceed the budget, their weights decide and the others' keys are 0
    bool crowded = false;
    auto make_key = [&](int t) {
        const bool late = is_recent(t);
        if (crowded) return late ? weight_key(w[t]) : 0u;
        return late ? 0xffffffffu : weight_key(w[t]);
    };
    auto key_of = [&](int t) { return cached ? keys[t - s0] : make_key(t); };
    // the sum over the cluster's blocks of their xch[slot], written before a cluster
    // barrier; also the sum over the blocks before this one
    auto gather = [&](int slot, int &before) {
        before = 0;
        if constexpr (!CLUSTER) {
            return xch[slot];
        } else {
            int x[kEvictMaxCluster], all = 0;
#pragma unroll
            for (int i = 0; i < kEvictMaxCluster; ++i) x[i] = i < CS ? *cg::this_cluster().map_shared_rank(&xch[slot], i) : 0;
#pragma unroll
            for (int i = 0; i < kEvictMaxCluster; ++i) {
                if (i < rank) before += x[i];
                all += x[i];
            }
            return all;
        }
    };

    // f(t0, key, in) for this warp's slots, 32 at a time from t0 on (slot t0 + lane,
    // `in` if it exists), their keys loaded four times 32 at once
    auto sweep = [&](auto f) {
        for (int t = a0; t < a1; t += 128) {
            uint32_t key[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) key[j] = t + 32 * j + lane < a1 ? key_of(t + 32 * j + lane) : 0u;
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (t + 32 * j < a1) f(t + 32 * j, key[j], t + 32 * j + lane < a1);
        }
    };
    // the keys, the number of recent tokens, and the table's entries
    for (int i = tid; i < 2 * BINS / 4; i += kEvictThreads) reinterpret_cast<int4 *>(hist)[i] = make_int4(0, 0, 0, 0);
    constexpr int KU = 6;   // loads in flight per lane
    int late = 0, none;
    for (int t = a0 + lane; t < a1; t += 32 * KU) {
        float x[KU];
        int y[KU];
#pragma unroll
        for (int j = 0; j < KU; ++j) {
            x[j] = 0.f;
            y[j] = 0;
            if (t + 32 * j < a1) {
                x[j] = w[t + 32 * j];
                if (ps) y[j] = ps[t + 32 * j];
            }
        }
#pragma unroll
        for (int j = 0; j < KU; ++j) {
            const int at = t + 32 * j;
            if (at >= a1) break;
            const bool l = p.recent && y[j] >= last - p.recent;
            late += l;
            if (cached) keys[at - s0] = l ? 0xffffffffu : weight_key(x[j]);
            if (at < budget) {   // other buffers: entries that may stay (those of dropped slots are written again below)
                if (wo != w) wo[at] = x[j];
                if (po != ps) po[at] = y[j];
            }
        }
    }
    bool bad = false;
    const int used = (n - 1) / c.page + 1;
#pragma unroll 4
    for (int i = rank * kEvictThreads + tid; i < used; i += CS * kEvictThreads)
        bad |= (unsigned)c.table[(size_t)b * c.max_pages + i] >= (unsigned)c.num_pages;
    int total;
    (void)warps_before(__reduce_add_sync(0xffffffffu, late), part[0], total);
    bad = __syncthreads_or(bad);
    if (tid == 0) {
        xch[0] = bad;
        xch[1] = total;
    }
    sync_all();
    if (gather(0, none)) {   // a bad entry: the sequence stays as it was
        if (rank == 0 && tid == 0) report(kStatusCheck);
        if (first && p.newlen) len_to[b] = n;
        sync_all();   // no block leaves while another reads its xch
        return;
    }
    if (gather(1, none) > budget) {
        crowded = true;
        if (cached)
            for (int t = a0 + lane; t < a1; t += 32) keys[t - s0] = make_key(t);
        __syncthreads();
    }
    // the radix select, from the top; it ends early when a whole bin stays.  Kept
    // are the keys whose `known` bits are above thr, and `need` of the `ties`
    // slots where they are thr.
    uint32_t thr = 0, known = 0;
    int need = budget, ties = 0;
    for (int pass = 0, top = 32; top > 0 && need != ties; ++pass) {
        const int bits = top < BITS ? top : BITS, shift = top - bits;
        top = shift;
        int *hs = hist[pass & 1];
        if (pass >= 2) {   // (the other blocks have read it: they have passed the barrier of the last pass)
            for (int i = tid; i < BINS; i += kEvictThreads) hs[i] = 0;
            __syncthreads();
        }
        sweep([&](int, uint32_t key, bool in) {
            if (in && (key & known) == thr) atomicAdd(&hs[key >> shift & ((1u << bits) - 1)], 1);
        });
        sync_all();
        // thread i owns BP bins, larger keys first
        constexpr int BP = BINS / kEvictThreads;
        const int bin = BINS - BP * (tid + 1);
        int cnt[BP], mine = 0;
        if constexpr (CLUSTER) {
            static_assert(BP == 1, "one bin per thread");
            int x[kEvictMaxCluster];
#pragma unroll
            for (int i = 0; i < kEvictMaxCluster; ++i)
                x[i] = i < CS ? cg::this_cluster().map_shared_rank(hs, i)[bin] : 0;
            cnt[0] = 0;
#pragma unroll
            for (int i = 0; i < kEvictMaxCluster; ++i) cnt[0] += x[i];
        } else {
#pragma unroll
            for (int j = 0; j < BP; j += 4) *reinterpret_cast<int4 *>(cnt + j) = *reinterpret_cast<const int4 *>(hs + bin + j);
        }
#pragma unroll
        for (int j = 0; j < BP; ++j) mine += cnt[j];
        int scan = mine;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int o = __shfl_up_sync(0xffffffffu, scan, off);
            if (lane >= off) scan += o;
        }
        int left = need - (scan - mine) - warps_before(__shfl_sync(0xffffffffu, scan, 31), part[pass & 1 ? 0 : 1], total);
        if (left > 0 && left <= mine) {   // one thread: the bins add up to at least `need`
            bool found = false;
#pragma unroll
            for (int j = BP - 1; j >= 0; --j) {
                if (found) continue;
                if (left <= cnt[j]) {
                    pick[0] = bin + j;
                    pick[1] = left;
                    pick[2] = cnt[j];
                    found = true;
                } else {
                    left -= cnt[j];
                }
            }
        }
        __syncthreads();
        thr |= (uint32_t)pick[0] << shift;
        known |= ((1u << bits) - 1) << shift;
        need = pick[1];
        ties = pick[2];
    }

    // of the ties, the lowest slots stay
    int rank0 = 0;   // ties before this warp's slots
    __syncthreads();   // part[0] may have been read last in the select
    if (need < ties) {
        int mine = 0;
        sweep([&](int, uint32_t key, bool in) { mine += __popc(__ballot_sync(0xffffffffu, in && (key & known) == thr)); });
        const int before = warps_before(mine, part[0], total);
        if (tid == 0) xch[2] = total;
        sync_all();
        int blocks_before;
        (void)gather(2, blocks_before);
        rank0 = blocks_before + before;
    }
    // Of the 1024 slots from `base` on, 32 for each lane: those dropped below the
    // budget, and those kept above it.
    int seen = 0;   // ties before them
    auto find = [&](int base, uint32_t &hole, uint32_t &mover) {
        uint32_t k = 0;
        for (int i0 = 0; i0 < 32 && base + 32 * i0 < a1; i0 += 4) {
            uint32_t key[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int t = base + 32 * (i0 + j) + lane;
                key[j] = t < a1 ? key_of(t) & known : 0u;
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const bool in = base + 32 * (i0 + j) + lane < a1;
                bool eq = in && key[j] == thr;
                if (need < ties) {
                    const uint32_t all = __ballot_sync(0xffffffffu, eq);
                    eq = eq && rank0 + seen + __popc(all & ((1u << lane) - 1)) < need;
                    seen += __popc(all);
                }
                const uint32_t keep = __ballot_sync(0xffffffffu, in && (key[j] > thr || eq));
                if (lane == i0 + j) k = keep;
            }
        }
        const int t0 = base + 32 * lane;
        const uint32_t exist = t0 + 32 <= a1 ? 0xffffffffu : t0 >= a1 ? 0u : (1u << (a1 - t0)) - 1;
        const uint32_t below = t0 + 32 <= budget ? 0xffffffffu : t0 >= budget ? 0u : (1u << (budget - t0)) - 1;
        hole = ~k & exist & below;
        mover = k & ~below;
    };
    uint32_t hole = 0, mover = 0;
    int nh = 0, nm = 0;
    for (int base = a0; base < a1; base += 1024) {
        find(base, hole, mover);
        nh += __popc(hole);
        nm += __popc(mover);
    }
    const bool one = a1 - a0 <= 1024;   // (then the masks are still there below)
    int ih = warps_before(__reduce_add_sync(0xffffffffu, nh), part[1], total), blocks_before;
    if (tid == 0) xch[3] = total;
    __syncthreads();
    int im = warps_before(__reduce_add_sync(0xffffffffu, nm), part[0], total);
    if (tid == 0) xch[4] = total;
    sync_all();
    const int m = gather(3, blocks_before);
    ih += blocks_before;
    (void)gather(4, blocks_before);
    im += blocks_before;
    int *holes = p.holes + bh * p.maxmoves, *movers = p.movers + bh * p.maxmoves;
    seen = 0;
    for (int base = a0; base < a1; base += 1024) {
        if (!one) find(base, hole, mover);
        int sh = __popc(hole), sm = __popc(mover);
        const int ch = sh, cm = sm;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int x = __shfl_up_sync(0xffffffffu, sh, off), y = __shfl_up_sync(0xffffffffu, sm, off);
            if (lane >= off) {
                sh += x;
                sm += y;
            }
        }
        int *to = holes + ih + sh - ch, t0 = base + 32 * lane;
        for (uint32_t x = hole; x; x &= x - 1) *to++ = t0 + __ffs(x) - 1;
        to = movers + im + sm - cm;
        for (uint32_t x = mover; x; x &= x - 1) *to++ = t0 + __ffs(x) - 1;
        ih += __shfl_sync(0xffffffffu, sh, 31);
        im += __shfl_sync(0xffffffffu, sm, 31);
    }
    sync_all();   // the lists are complete, all keys are read, and no block reads another's memory any more
    if (first) len_to[b] = budget;
    if (p.width == 16) evict_rows<uint4, U>(p, b, h, holes, movers, m, rank, CS);
    else if (p.width == 4) evict_rows<uint32_t, U>(p, b, h, holes, movers, m, rank, CS);
    else evict_rows<uint16_t, U>(p, b, h, holes, movers, m, rank, CS);
}

// lens in place: no block of the kernel above may still read it when it is written.
__global__ void paged_evict_lens_kernel(const PagedEvictParams p)
{
    sm100::grid_dependency_wait();
    sm100::launch_dependents();
    const int b = blockIdx.x * blockDim.x + threadIdx.x;
    if (b < p.c.B) p.lens_out[b] = p.newlen[b];
}

}  // namespace la
