// la_paged.cuh -- the paged key/value cache of global softmax attention: the
// write of new tokens into pages, one-token attention over the cache, and
// eviction by accumulated attention weight.
#pragma once

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

// 16-byte copies where every row starts on a 16-byte boundary, elements otherwise.
template <typename T, int LANES>
__device__ __forceinline__ void copy_row(T *dst, const T *src, int d, bool vec, int lane)
{
    if (vec) {
        constexpr int E = 16 / sizeof(T);
        for (int i = lane; i < d / E; i += LANES)
            reinterpret_cast<uint4 *>(dst)[i] = reinterpret_cast<const uint4 *>(src)[i];
    } else {
        for (int i = lane; i < d; i += LANES) dst[i] = src[i];
    }
}

// ------------------------------------------------------------------ append

constexpr int kPagedFillThreads = 256;
constexpr int kPagedFillRows = 64;

struct PagedFillParams {
    PagedCache c;
    const void *k, *v;
    const int *n_new, *pos;
    float *weights;
    int *positions;
    int N;
    bool vec_k, vec_v;
};

// One block per 64 new tokens of a (b, h): slot lens[b] + i <- token i.
template <typename T>
__global__ void __launch_bounds__(kPagedFillThreads) paged_fill_kernel(const PagedFillParams p)
{
    sm100::grid_dependency_wait();
    sm100::launch_dependents();
    __shared__ int rows[kPagedFillRows];
    const PagedCache &c = p.c;
    const int tiles = (p.N + kPagedFillRows - 1) / kPagedFillRows;
    const long long bh = blockIdx.x / tiles;
    const int i0 = (int)(blockIdx.x - bh * tiles) * kPagedFillRows;
    const int b = (int)(bh / c.Hkv), h = (int)(bh - (long long)b * c.Hkv);
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
    constexpr int G = 8;   // threads per row
    const int lane = tid % G;
    for (int i = tid / G; i < m; i += kPagedFillThreads / G) {
        const int row = rows[i];
        if (row < 0) continue;
        const size_t src = bh * (size_t)p.N + i0 + i;
        copy_row<T, G>((T *)c.kp + (size_t)row * c.dqk, (const T *)p.k + src * c.dqk, c.dqk, p.vec_k, lane);
        copy_row<T, G>((T *)c.vp + (size_t)row * c.dv, (const T *)p.v + src * c.dv, c.dv, p.vec_v, lane);
    }
}

// ------------------------------------------------------- one-token attention

struct PagedDecodeParams {
    PagedCache c;
    const void *q, *k, *v;   // k, v: the new token, or null
    void *y;
    float *lse;
    const float *w_in;
    float *w_out;
    int *positions;
    const int *pos;
    int Hq;
    float scale;
};

constexpr int kPagedThreads = 128;

template <int NT>
__device__ __forceinline__ float block_reduce(float x, bool is_max, float *red)
{
#pragma unroll
    for (int off = 16; off; off >>= 1) {
        const float o = __shfl_xor_sync(0xffffffffu, x, off);
        x = is_max ? fmaxf(x, o) : x + o;
    }
    __syncthreads();
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = x;
    __syncthreads();
    x = red[0];
#pragma unroll
    for (int i = 1; i < NT / 32; ++i) x = is_max ? fmaxf(x, red[i]) : x + red[i];
    return x;
}

// One block per (b, key/value head): for each query head a pass over the cache
// in tiles of 128 tokens with the running maximum and sum, then, if weights
// are kept, a second one that adds the normalised weights.
template <typename T>
__global__ void __launch_bounds__(kPagedThreads) paged_decode_simple_kernel(const PagedDecodeParams p)
{
    sm100::grid_dependency_wait();
    sm100::launch_dependents();
    __shared__ float qs[128], sc[kPagedThreads], red[kPagedThreads / 32];
    __shared__ int rows[kPagedThreads];
    const PagedCache &c = p.c;
    const int tid = threadIdx.x;
    const size_t bh = blockIdx.x;
    const int b = (int)(bh / c.Hkv), h = (int)(bh - (size_t)b * c.Hkv), g = p.Hq / c.Hkv;
    const int len = c.lens[b], pos = p.pos ? p.pos[b] : 0;
    if (len < 0 || len > c.cap() - (p.k ? 1 : 0) || pos < 0) {
        if (tid == 0) report(kStatusCheck);
        return;
    }
    const int n = len + (p.k ? 1 : 0);
    T *kp = (T *)c.kp, *vp = (T *)c.vp;
    if (p.k) {
        const int row = paged_row(c, b, h, len);
        if (row >= 0) {
            if (tid < c.dqk) kp[(size_t)row * c.dqk + tid] = ((const T *)p.k)[bh * c.dqk + tid];
            if (tid < c.dv) vp[(size_t)row * c.dv + tid] = ((const T *)p.v)[bh * c.dv + tid];
        }
        if (p.positions && tid == 0 && row >= 0) p.positions[bh * c.cap() + len] = pos;
        __syncthreads();
    }
    for (int j = 0; j < g; ++j) {
        const size_t hq = (size_t)b * p.Hq + h * g + j;
        __syncthreads();
        if (tid < c.dqk) qs[tid] = ld((const T *)p.q + hq * c.dqk + tid);
        __syncthreads();
        auto score = [&](int t, int &row) {
            row = t < n ? paged_row(c, b, h, t) : -1;
            if (t < n && row < 0) report(kStatusCheck);
            if (row < 0) return -INFINITY;
            float s = 0.f;
            for (int i = 0; i < c.dqk; ++i) s = fmaf(qs[i], ld(kp + (size_t)row * c.dqk + i), s);
            return s * p.scale;
        };
        float m = -INFINITY, z = 0.f, acc = 0.f;
        for (int t0 = 0; t0 < n; t0 += kPagedThreads) {
            int row;
            const float s = score(t0 + tid, row);
            const float mn = fmaxf(m, block_reduce<kPagedThreads>(s, true, red));
            const float base = mn == -INFINITY ? 0.f : mn;   // nothing but -inf so far: exp(-inf) = 0
            const float e = expf(s - base), a = expf(m - base);
            sc[tid] = e;
            rows[tid] = row;
            z = z * a + block_reduce<kPagedThreads>(row < 0 ? 0.f : e, false, red);
            m = mn;
            acc *= a;
            if (tid < c.dv)
                for (int i = 0; i < min(kPagedThreads, n - t0); ++i)
                    if (rows[i] >= 0) acc = fmaf(sc[i], ld(vp + (size_t)rows[i] * c.dv + tid), acc);
        }
        if (tid < c.dv) st((T *)p.y + hq * c.dv + tid, n ? acc / z : 0.f);
        const float lse = n ? m + logf(z) : -INFINITY;
        if (p.lse && tid == 0) p.lse[hq] = lse;
        if (p.w_out)
            for (int t = tid; t < n; t += kPagedThreads) {
                int row;
                const float s = score(t, row);
                const size_t at = bh * c.cap() + t;
                const float old = j ? p.w_out[at] : t == len ? 0.f : p.w_in[at];
                p.w_out[at] = old + (row < 0 ? 0.f : expf(s - lse));
            }
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
    int *count, *newlen;   // [B*Hkv], [B]
    int budget, recent, maxmoves;
    bool vec_k, vec_v;
};

constexpr int kEvictThreads = 512;

// Weight as an unsigned key of the same order: larger weight, larger key; NaN
// counts as -inf and -0 as +0.
__device__ __forceinline__ uint32_t weight_key(float w)
{
    if (!(w == w)) w = -INFINITY;
    const uint32_t u = __float_as_uint(w + 0.f);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// Exclusive prefix of x over the block in thread order, and the total.
template <int NT>
__device__ __forceinline__ int block_scan(int x, int *part, int &total)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int s = x;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int o = __shfl_up_sync(0xffffffffu, s, off);
        if (lane >= off) s += o;
    }
    __syncthreads();
    if (lane == 31) part[warp] = s;
    __syncthreads();
    int before = 0;
    total = 0;
#pragma unroll
    for (int i = 0; i < NT / 32; ++i) {
        if (i < warp) before += part[i];
        total += part[i];
    }
    return before + s - x;
}

// One block per (b, h): a radix select over the weights' keys (four passes of
// 8 bits) finds the smallest key that is kept, then one pass in slot order
// lists the dropped slots below the budget and the kept ones above it, and
// moves their weights and positions.
__global__ void __launch_bounds__(kEvictThreads) paged_evict_select_kernel(const PagedEvictParams p)
{
    sm100::grid_dependency_wait();
    sm100::launch_dependents();
    __shared__ int hist[256], part[kEvictThreads / 32], pick[2];
    const PagedCache &c = p.c;
    const int tid = threadIdx.x;
    const size_t bh = blockIdx.x;
    const int b = (int)(bh / c.Hkv), h = (int)(bh - (size_t)b * c.Hkv);
    const int n = c.lens[b], budget = p.budget;
    const long long last = p.recent ? p.pos[b] : 0;
    bool bad = n < 0 || n > c.cap() || last < 0;
    if (!bad && n > budget) {
        const int used = (n - 1) / c.page + 1;
        for (int i = tid; i < used; i += kEvictThreads)
            if ((unsigned)c.table[(size_t)b * c.max_pages + i] >= (unsigned)c.num_pages) bad = true;
    }
    bad = __syncthreads_or(bad);
    if (tid == 0) {
        if (bad) report(kStatusCheck);
        if (h == 0) p.newlen[b] = bad ? n : min(n, budget);
        if (bad || n <= budget) p.count[bh] = 0;
    }
    if (bad) return;
    const float *w = p.w_in + bh * c.cap();
    float *wo = p.w_out + bh * c.cap();
    const int *ps = p.pos_in ? p.pos_in + bh * c.cap() : nullptr;
    int *po = p.pos_out ? p.pos_out + bh * c.cap() : nullptr;
    if (n <= budget) {
        for (int t = tid; t < n; t += kEvictThreads) {
            if (wo != w) wo[t] = w[t];
            if (po != ps) po[t] = ps[t];
        }
        return;
    }
    auto recent = [&](int t) { return p.recent && ps[t] >= last - p.recent; };
    // the class the cut falls into: the recent tokens if they alone exceed the
    // budget (then the others are all dropped), else the others (the recent all stay)
    int nrec = 0;
    for (int t = tid; t < n; t += kEvictThreads) nrec += recent(t);
    int total;
    (void)block_scan<kEvictThreads>(nrec, part, total);
    const bool cls = total >= budget;
    int need = cls ? budget : budget - total;
    uint32_t thr = 0, known = 0;
    for (int shift = 24; shift >= 0; shift -= 8) {
        __syncthreads();
        if (tid < 256) hist[tid] = 0;
        __syncthreads();
        for (int t = tid; t < n; t += kEvictThreads)
            if (recent(t) == cls) {
                const uint32_t key = weight_key(w[t]);
                if ((key & known) == thr) atomicAdd(&hist[key >> shift & 255], 1);
            }
        __syncthreads();
        if (tid == 0) {
            int bin = 255, left = need;
            while (hist[bin] < left) left -= hist[bin--];   // the counts add up to at least `need`
            pick[0] = bin;
            pick[1] = left;
        }
        __syncthreads();
        thr |= (uint32_t)pick[0] << shift;
        known |= 255u << shift;
        need = pick[1];
    }
    // slot order: `need` slots with key == thr stay, the lowest ones
    int ties = 0, nh = 0, nm = 0;
    int *holes = p.holes + bh * p.maxmoves, *movers = p.movers + bh * p.maxmoves;
    for (int t0 = 0; t0 < n; t0 += kEvictThreads) {
        const int t = t0 + tid;
        const bool in = t < n, r = in && recent(t);
        const uint32_t key = in && r == cls ? weight_key(w[t]) : 0;
        const bool eq = in && r == cls && key == thr;
        const int rank = ties + block_scan<kEvictThreads>(eq, part, total);
        ties += total;
        const bool keep = in && (r == cls ? key > thr || (eq && rank < need) : r);
        const bool hole = in && t < budget && !keep, mover = keep && t >= budget;
        const int ih = nh + block_scan<kEvictThreads>(hole, part, total);
        nh += total;
        const int im = nm + block_scan<kEvictThreads>(mover, part, total);
        nm += total;
        if (hole) holes[ih] = t;
        if (mover) movers[im] = t;
        if (keep && !mover) {
            if (wo != w) wo[t] = w[t];
            if (po != ps) po[t] = ps[t];
        }
    }
    __syncthreads();   // the lists are complete and visible to the block
    for (int i = tid; i < nm; i += kEvictThreads) {
        wo[holes[i]] = w[movers[i]];
        if (po) po[holes[i]] = ps[movers[i]];
    }
    if (tid == 0) p.count[bh] = nm;
}

// Copies the moved rows; the sources lie at or above the budget and the
// destinations below it, so no order is needed.  The first blocks write lens.
template <typename T>
__global__ void __launch_bounds__(256) paged_evict_move_kernel(const PagedEvictParams p, int splits)
{
    sm100::grid_dependency_wait();
    sm100::launch_dependents();
    const PagedCache &c = p.c;
    const size_t bh = blockIdx.x / splits;
    const int s = (int)(blockIdx.x - bh * splits);
    const int b = (int)(bh / c.Hkv), h = (int)(bh - (size_t)b * c.Hkv);
    if (h == 0 && s == 0 && threadIdx.x == 0) p.lens_out[b] = p.newlen[b];
    const int m = p.count[bh];
    constexpr int G = 8;
    const int lane = threadIdx.x % G;
    for (int i = s * (256 / G) + threadIdx.x / G; i < m; i += splits * (256 / G)) {
        const int to = paged_row(c, b, h, p.holes[bh * p.maxmoves + i]);
        const int from = paged_row(c, b, h, p.movers[bh * p.maxmoves + i]);
        T *kp = (T *)c.kp, *vp = (T *)c.vp;
        copy_row<T, G>(kp + (size_t)to * c.dqk, kp + (size_t)from * c.dqk, c.dqk, p.vec_k, lane);
        copy_row<T, G>(vp + (size_t)to * c.dv, vp + (size_t)from * c.dv, c.dv, p.vec_v, lane);
    }
}

}  // namespace la
