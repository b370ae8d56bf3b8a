// Page pool of a paged cache: mapping, sharing, freeing, copying and
// compacting pages (include/jsv.h, "Page pool").
//
// A pool's state is one reference count per page and nothing else: a free
// page is a page with count 0, taken lowest index first.  No free list is
// kept between calls, so the result of a call does not depend on the order in
// which atomics land, and a call that is skipped or refused leaves no list
// to repair.  What it costs is a look at every count per allocating call:
// 4 bytes a page, a quarter of a megabyte for the 70,000 pages that 180 GB
// hold of a 36-layer 8-head bf16 cache.
//
// The allocating calls run as ONE cluster of eight CTAs of 1024 threads: the
// counts are split over the CTAs, each thread scans a run of them, and the
// cluster barrier (which also orders global memory inside the cluster) takes
// the place of a second launch between the scan and its use.  Bound by
// latency: two or three rounds of dependent loads and as many barriers (alloc
// 8-10 us, fork 10 us for 4 rows and 21 for 64, compact 11-14 us under ncu on
// pools of 300 to 20,000 pages; rows' entries are read eight to a lane at a time,
// which took the fork of 64 rows from 30 us to 21).  Trimming (4-5 us) and copying need no order between
// CTAs and use plain grids.
#include "jsv_internal.cuh"
#include "kv_internal.cuh"
#include "sm100.cuh"

#include <algorithm>

namespace jsv {

using sm100::cluster_ctarank;

namespace {

constexpr int kPoolCtas = 8;                 // one cluster (the portable size)
constexpr int kPoolThreads = 1024;
constexpr int kPoolWarps = kPoolThreads / 32;
constexpr int kPageSlots = 16;
constexpr int kRowBatch = 8;                 // row entries a lane reads at a time
constexpr int kCounts = 64;                  // ints of exchanged counts at the workspace's start

// Barrier over the cluster; the block's own barrier in front reconverges the
// warps, which the aligned cluster barrier asks for.
__device__ __forceinline__ void pool_sync() {
    __syncthreads();
    sm100::cluster_sync();
}

__device__ __forceinline__ int pages_up(int slots) { return (int)(((long long)slots + kPageSlots - 1) / kPageSlots); }

// Workspace of one call: counts exchanged between the CTAs, one number per
// row (or fork), one per page.
struct PoolScratch {
    int *counts, *rows, *pages;
};
__host__ __device__ inline size_t rows_ints(int rows) { return ((size_t)rows + 3) / 4 * 4; }
__device__ __forceinline__ PoolScratch scratch_of(void *ws, int rows) {
    PoolScratch s;
    s.counts = static_cast<int *>(ws);
    s.rows = s.counts + kCounts;
    s.pages = s.rows + rows_ints(rows);
    return s;
}

// Exclusive scan over the block; `total` gets the sum.  Every thread calls it.
template <typename T>
__device__ T block_scan(T v, T &total) {
    __shared__ T sums[kPoolWarps];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    T incl = v;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const T u = __shfl_up_sync(0xffffffffu, incl, off);
        if (lane >= off) incl += u;
    }
    __syncthreads();                         // an earlier scan's sums have been read
    if (lane == 31) sums[warp] = incl;
    __syncthreads();
    if (warp == 0) {
        T w = sums[lane];
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const T u = __shfl_up_sync(0xffffffffu, w, off);
            if (lane >= off) w += u;
        }
        sums[lane] = w;
    }
    __syncthreads();
    total = sums[kPoolWarps - 1];
    return incl - v + (warp ? sums[warp - 1] : T(0));
}

// Exclusive prefix of rows[0..n) into shared memory, the same in every CTA.
template <typename T>
__device__ T prefix_rows(const int *rows, int n, T *out) {
    const int per = (n + kPoolThreads - 1) / kPoolThreads;
    const int lo = min((int)threadIdx.x * per, n), hi = min(lo + per, n);
    T sum = 0, total;
    for (int i = lo; i < hi; ++i) sum += (T)__ldcg(rows + i);
    T at = block_scan(sum, total);
    for (int i = lo; i < hi; ++i) {
        out[i] = at;
        at += (T)__ldcg(rows + i);
    }
    __syncthreads();
    return total;
}

// The run of pages this thread scans: the cluster's CTAs take equal parts of
// the pool in order, a CTA's threads equal parts of its own.
__device__ __forceinline__ void page_run(int num_pages, int rank, int &lo, int &hi) {
    const long long per = ((long long)num_pages + kPoolCtas - 1) / kPoolCtas;
    const long long run = (per + kPoolThreads - 1) / kPoolThreads;
    const long long end = min(per * (rank + 1), (long long)num_pages);
    const long long l = min(per * rank + run * threadIdx.x, end);
    lo = (int)l;
    hi = (int)min(l + run, end);
}

__device__ __forceinline__ int count_free(const int *refcount, int lo, int hi) {
    int n = 0;
    for (int p = lo; p < hi; ++p) n += refcount[p] == 0;
    return n;
}

// Sum of the CTAs' counts before this one's, and of all.
__device__ __forceinline__ int counts_before(const int *counts, int rank, int &total) {
    int before = 0;
    total = 0;
    for (int c = 0; c < kPoolCtas; ++c) {
        const int v = __ldcg(counts + c);
        if (c < rank) before += v;
        total += v;
    }
    return before;
}

// Writes the first `limit` free pages, ascending, to list.  `mine` is this
// thread's first rank.
__device__ __forceinline__ void list_free(const int *refcount, int lo, int hi, int mine, long long limit, int *list,
                                          int num_pages, int32_t *status) {
    for (int p = lo; p < hi && mine < limit; ++p)
        if (refcount[p] == 0) {
            if (JSV_IN_BOUNDS(mine, num_pages, status)) list[mine] = p;
            ++mine;
        }
}

}  // namespace

size_t pages_workspace_bytes(int num_pages, int rows) {
    return (kCounts + rows_ints(rows) + (size_t)num_pages + 3) / 4 * 16;
}

// ---------------------------------------------------------------------------
// Map fresh pages
// ---------------------------------------------------------------------------
__global__ void __launch_bounds__(kPoolThreads)
pages_alloc_kernel(int num_pages, int32_t *__restrict__ refcount, int32_t *status, int32_t *__restrict__ table, int B,
                   int max_pages, const int32_t *__restrict__ begin, const int32_t *__restrict__ end, int full_only,
                   void *ws) {
    pdl_allow_dependents();
    pdl_wait_predecessor();
    extern __shared__ long long prefix[];                 // [B]
    const PoolScratch s = scratch_of(ws, B);
    const int rank = (int)cluster_ctarank(), warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    // a row's range of logical pages; lo > hi: refused
    auto range = [&](int b, int &lo, int &hi) {
        const int f = begin ? begin[b] : 0, t = end[b];
        const bool ok = f >= 0 && f <= t && (long long)t <= (long long)max_pages * kPageSlots;
        lo = ok ? f / kPageSlots : 1;
        hi = ok ? (full_only ? t / kPageSlots : pages_up(t)) : 0;
        return ok;
    };
    // how many entries of each row lack a page; how many pages are free
    for (int b = rank * kPoolWarps + warp; b < B; b += kPoolCtas * kPoolWarps) {
        int lo, hi, n = 0;
        if (!range(b, lo, hi) && lane == 0) flag_error(status, JSV_ERR_DEVICE_INPUT);
        for (int i = lo + lane; i < hi; i += 32) n += table[(size_t)b * max_pages + i] == -1;
        n = __reduce_add_sync(0xffffffffu, n);
        if (lane == 0) s.rows[b] = n;
    }
    int lo, hi, mine_total, free_pages;
    page_run(num_pages, rank, lo, hi);
    const int mine = block_scan(count_free(refcount, lo, hi), mine_total);
    if (threadIdx.x == 0) s.counts[rank] = mine_total;
    pool_sync();

    const int before = counts_before(s.counts, rank, free_pages);
    const long long need = prefix_rows(s.rows, B, prefix);
    list_free(refcount, lo, hi, before + mine, need, s.pages, num_pages, status);
    pool_sync();

    for (int b = rank * kPoolWarps + warp; b < B; b += kPoolCtas * kPoolWarps) {
        const int n = __ldcg(s.rows + b);
        if (n == 0) continue;
        if (prefix[b] + n > free_pages) {                  // does not fit after the rows before it
            if (lane == 0) flag_error(status, JSV_ERR_NO_PAGES);
            continue;
        }
        int l, h, at = (int)prefix[b];
        range(b, l, h);
        for (int i0 = l; i0 < h; i0 += 32) {
            const int i = i0 + lane;
            const size_t e = (size_t)b * max_pages + i;
            const bool take = i < h && table[e] == -1;
            const unsigned m = __ballot_sync(0xffffffffu, take);
            const int r = at + __popc(m & ((1u << lane) - 1));
            if (take && JSV_IN_BOUNDS(r, num_pages, status)) {
                const int page = __ldcg(s.pages + r);
                table[e] = page;
                refcount[page] = 1;
            }
            at += __popc(m);
        }
    }
}

// ---------------------------------------------------------------------------
// Fork rows
// ---------------------------------------------------------------------------
__global__ void __launch_bounds__(kPoolThreads)
pages_fork_kernel(int num_pages, int32_t *__restrict__ refcount, int32_t *status, int32_t *__restrict__ table, int B,
                  int max_pages, int n, const int32_t *__restrict__ src, const int32_t *__restrict__ dst,
                  const int32_t *__restrict__ len, int full_only, int32_t *__restrict__ copy_src,
                  int32_t *__restrict__ copy_dst, void *ws) {
    pdl_allow_dependents();
    pdl_wait_predecessor();
    extern __shared__ int fork_smem[];
    int *first = fork_smem, *prefix = fork_smem + B;       // [B] first fork into a row, [n]
    const PoolScratch s = scratch_of(ws, n);
    const int rank = (int)cluster_ctarank(), warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    // the first fork into each row, by its own arguments (every CTA alike)
    for (int b = threadIdx.x; b < B; b += kPoolThreads) first[b] = n;
    __syncthreads();
    auto sound = [&](int i) {
        const int a = src[i], d = dst[i], l = len[i];
        return a >= 0 && a < B && d >= 0 && d < B && a != d && l >= 0 && (long long)l <= (long long)max_pages * kPageSlots;
    };
    for (int i = threadIdx.x; i < n; i += kPoolThreads)
        if (sound(i)) atomicMin(&first[dst[i]], i);
    __syncthreads();

    // each fork's entries: 0 = refused, 1 = shares only, 2 = needs a page.
    // rows[] holds state - 1 clipped to 0 for the prefix, with -1 = refused
    // kept in the list of copies
    for (int i = rank * kPoolWarps + warp; i < n; i += kPoolCtas * kPoolWarps) {
        int bad = !sound(i), part = 0;
        if (!bad) bad = first[dst[i]] != i || first[src[i]] != n;
        if (!bad) {
            const int a = src[i], d = dst[i], l = len[i];
            const int full = l / kPageSlots;
            part = !full_only && l % kPageSlots;
            // kRowBatch entries a lane at a time, so that their loads overlap
            const int32_t *from = table + (size_t)a * max_pages, *to = table + (size_t)d * max_pages;
            for (int e0 = lane; e0 < max_pages; e0 += 32 * kRowBatch) {
                int p[kRowBatch];
#pragma unroll
                for (int k = 0; k < kRowBatch; ++k) {
                    const int e = e0 + 32 * k;
                    p[k] = e < full + part ? from[e] : -1;
                    if (e < max_pages && to[e] != -1) bad = 1;
                }
#pragma unroll
                for (int k = 0; k < kRowBatch; ++k) {
                    if (p[k] == -1) bad |= part && e0 + 32 * k == full;
                    else if (p[k] < 0 || p[k] >= num_pages || refcount[p[k]] <= 0) bad = 1;
                }
            }
        }
        bad = __any_sync(0xffffffffu, bad);
        if (lane == 0) {
            if (bad) flag_error(status, JSV_ERR_DEVICE_INPUT);
            s.rows[i] = !bad && part;
            copy_src[i] = bad ? -2 : -1;                    // -2: refused, replaced below
            copy_dst[i] = -1;
        }
    }
    int lo, hi, mine_total, free_pages;
    page_run(num_pages, rank, lo, hi);
    const int mine = block_scan(count_free(refcount, lo, hi), mine_total);
    if (threadIdx.x == 0) s.counts[rank] = mine_total;
    pool_sync();

    const int before = counts_before(s.counts, rank, free_pages);
    const int need = prefix_rows(s.rows, n, prefix);
    list_free(refcount, lo, hi, before + mine, need, s.pages, num_pages, status);
    pool_sync();

    for (int i = rank * kPoolWarps + warp; i < n; i += kPoolCtas * kPoolWarps) {
        const bool part = __ldcg(s.rows + i) != 0;
        const bool refused = copy_src[i] == -2, lacks = part && prefix[i] >= free_pages;
        __syncwarp();                                      // every lane has read copy_src[i]
        if (refused || lacks) {
            if (lane == 0) {
                if (lacks) flag_error(status, JSV_ERR_NO_PAGES);
                copy_src[i] = -1;
            }
            continue;
        }
        const int full = len[i] / kPageSlots;
        const int32_t *from = table + (size_t)src[i] * max_pages;
        int32_t *to = table + (size_t)dst[i] * max_pages;
        for (int e0 = lane; e0 < full; e0 += 32 * kRowBatch) {
            int p[kRowBatch];
#pragma unroll
            for (int k = 0; k < kRowBatch; ++k) p[k] = e0 + 32 * k < full ? from[e0 + 32 * k] : -1;
#pragma unroll
            for (int k = 0; k < kRowBatch; ++k) {
                if (p[k] < 0) continue;
                if (JSV_IN_BOUNDS(p[k], num_pages, status)) atomicAdd(&refcount[p[k]], 1);
                to[e0 + 32 * k] = p[k];
            }
        }
        if (part && lane == 0 && JSV_IN_BOUNDS(prefix[i], num_pages, status)) {
            const int p = __ldcg(s.pages + prefix[i]);
            refcount[p] = 1;
            to[full] = p;
            copy_src[i] = from[full];
            copy_dst[i] = p;
        }
    }
}

// ---------------------------------------------------------------------------
// Free pages: one thread a table entry; the counts' atomics commute, so the
// result has no order in it.
// ---------------------------------------------------------------------------
constexpr int kTrimThreads = 256;

__global__ void __launch_bounds__(kTrimThreads)
pages_trim_kernel(int num_pages, int32_t *__restrict__ refcount, int32_t *status, int32_t *__restrict__ table, int B,
                  int max_pages, const int32_t *__restrict__ keep_begin, const int32_t *__restrict__ keep_end) {
    pdl_allow_dependents();
    pdl_wait_predecessor();
    const int per_row = (max_pages + kTrimThreads - 1) / kTrimThreads;
    for (long long w = blockIdx.x; w < (long long)B * per_row; w += gridDim.x) {
        const int b = (int)(w / per_row), e = (int)(w % per_row) * kTrimThreads + threadIdx.x;
        if (e >= max_pages) continue;
        const int f = keep_begin ? keep_begin[b] : 0, t = keep_end[b];
        if (f < 0 || t < f || (long long)t > (long long)max_pages * kPageSlots) {
            if (e == 0) flag_error(status, JSV_ERR_DEVICE_INPUT);
            continue;
        }
        if (e >= f / kPageSlots && e < pages_up(t)) continue;
        const size_t i = (size_t)b * max_pages + e;
        const int p = table[i];
        if (p == -1) continue;
        table[i] = -1;
        if (p < 0 || p >= num_pages) {
            flag_error(status, JSV_ERR_DEVICE_INPUT);
        } else if (atomicSub(&refcount[p], 1) <= 0) {
            atomicAdd(&refcount[p], 1);                     // was free already
            flag_error(status, JSV_ERR_DEVICE_INPUT);
        }
    }
}

// ---------------------------------------------------------------------------
// Compaction plan.  U = pages in use.  The i-th used page at or past U (a
// mover) goes to the i-th free page below U (a hole); there are as many of
// one as of the other, since U pages are used in all.
// ---------------------------------------------------------------------------
__global__ void __launch_bounds__(kPoolThreads)
pages_compact_kernel(int num_pages, const int32_t *__restrict__ refcount, int32_t *status, const int32_t *table, int B,
                     int max_pages, int32_t *new_table, int32_t *__restrict__ new_refcount, int32_t *copy_src,
                     int32_t *copy_dst, int max_copies, int32_t *num_copies, void *ws) {
    pdl_allow_dependents();
    pdl_wait_predecessor();
    const PoolScratch s = scratch_of(ws, B);               // s.pages: where each page goes
    const int rank = (int)cluster_ctarank();
    int lo, hi, total, used = 0;
    page_run(num_pages, rank, lo, hi);
    for (int p = lo; p < hi; ++p) used += refcount[p] > 0;
    block_scan(used, total);
    if (threadIdx.x == 0) s.counts[rank] = total;
    pool_sync();

    int U;
    counts_before(s.counts, rank, U);
    int moves = 0, holes = 0, m_total, h_total;
    for (int p = lo; p < hi; ++p) {
        const bool u = refcount[p] > 0;
        moves += u && p >= U;
        holes += !u && p < U;
    }
    const int m_mine = block_scan(moves, m_total), h_mine = block_scan(holes, h_total);
    if (threadIdx.x == 0) {
        s.counts[kPoolCtas + rank] = m_total;
        s.counts[2 * kPoolCtas + rank] = h_total;
    }
    pool_sync();

    int M, H;
    const int m0 = counts_before(s.counts + kPoolCtas, rank, M) + m_mine;
    int h = counts_before(s.counts + 2 * kPoolCtas, rank, H) + h_mine, m = m0;
    for (int p = lo; p < hi; ++p) {
        const bool u = refcount[p] > 0;
        if (u && p >= U && JSV_IN_BOUNDS(m, max_copies, status)) copy_src[m++] = p;
        if (!u && p < U && JSV_IN_BOUNDS(h, max_copies, status)) copy_dst[h++] = p;
    }
    const int all = kPoolCtas * kPoolThreads, me = rank * kPoolThreads + threadIdx.x;
    for (int i = M + me; i < max_copies; i += all) copy_src[i] = copy_dst[i] = -1;
    if (me == 0) *num_copies = M;
    pool_sync();

    m = m0;
    for (int p = lo; p < hi; ++p) {
        const int r = refcount[p];
        if (r > 0 && p >= U) {
            const int to = JSV_IN_BOUNDS(m, max_copies, status) ? __ldcg(copy_dst + m) : -1;
            ++m;
            s.pages[p] = to;
            if (JSV_IN_BOUNDS(to, num_pages, status)) new_refcount[to] = r;
            new_refcount[p] = 0;
        } else if (r > 0) {
            s.pages[p] = p;
            new_refcount[p] = r;
        } else {
            s.pages[p] = -1;                                // a free page: no entry may hold it
            if (p >= U) new_refcount[p] = 0;                // below U a hole, filled by its mover
        }
    }
    pool_sync();

    for (long long i = me; i < (long long)B * max_pages; i += all) {
        const int p = table[i];
        int to = -1;
        if (p != -1) {
            if (p >= 0 && p < num_pages) to = __ldcg(s.pages + p);
            if (to < 0) flag_error(status, JSV_ERR_DEVICE_INPUT);
        }
        new_table[i] = to;
    }
}

// ---------------------------------------------------------------------------
// Page contents.  One launch covers up to kCopyBuffers buffers; a CTA takes
// (pair, 16 KB segment) items, each thread four 16-byte vectors at a time
// (all loads before the stores).  Bound by HBM traffic once there are enough
// pairs to fill the machine: the copies of a pool of 7,000 pages of 32 KB in four
// buffers, a third of it free, move 600 MB at 5.5 TB/s.  More CTAs than are
// resident at once, so that none walks many items (8, 16, 32 and 64 an SM: 139,
// 134, 130 and 126 us, the plan's 13 us included).
// ---------------------------------------------------------------------------
constexpr int kCopyBuffers = 64;
constexpr int kCopyThreads = 256;
constexpr int kCopyUnroll = 4;

struct CopyBuffers {
    void *base[kCopyBuffers];
    long long bytes[kCopyBuffers];
};

template <typename V>
__device__ __forceinline__ void copy_segment(const V *from, V *to, long long n, long long at) {
    V v[kCopyUnroll];
#pragma unroll
    for (int k = 0; k < kCopyUnroll; ++k) {
        const long long i = at + k * kCopyThreads + threadIdx.x;
        if (i < n) v[k] = from[i];
    }
#pragma unroll
    for (int k = 0; k < kCopyUnroll; ++k) {
        const long long i = at + k * kCopyThreads + threadIdx.x;
        if (i < n) to[i] = v[k];
    }
}

__global__ void __launch_bounds__(kCopyThreads)
pages_copy_kernel(int num_pages, int32_t *status, const CopyBuffers bufs, const int32_t *__restrict__ copy_src,
                  const int32_t *__restrict__ copy_dst, int n, const int32_t *__restrict__ num_copies) {
    pdl_allow_dependents();
    pdl_wait_predecessor();
    char *base = static_cast<char *>(bufs.base[blockIdx.y]);
    const long long bytes = bufs.bytes[blockIdx.y];
    const bool wide = bytes % 16 == 0 && (reinterpret_cast<uintptr_t>(base) & 15) == 0;
    const long long vecs = bytes / (wide ? 16 : 4);
    const int segs = (int)((vecs + kCopyThreads * kCopyUnroll - 1) / (kCopyThreads * kCopyUnroll));
    if (num_copies) n = min(n, *num_copies);
    for (long long w = blockIdx.x; w < (long long)n * segs; w += gridDim.x) {
        const int i = (int)(w / segs);
        const int a = copy_src[i], d = copy_dst[i];
        if (a < 0) continue;
        if (a >= num_pages || d < 0 || d >= num_pages) {
            if (threadIdx.x == 0) flag_error(status, JSV_ERR_DEVICE_INPUT);
            continue;
        }
        if (a == d) continue;
        const long long at = (w % segs) * (kCopyThreads * kCopyUnroll);
        if (wide)
            copy_segment(reinterpret_cast<const uint4 *>(base + a * bytes), reinterpret_cast<uint4 *>(base + d * bytes),
                         vecs, at);
        else
            copy_segment(reinterpret_cast<const uint32_t *>(base + a * bytes),
                         reinterpret_cast<uint32_t *>(base + d * bytes), vecs, at);
    }
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------
template <typename K, typename... Args>
static cudaError_t launch_pool(K *kernel, PerDeviceOnce &once, size_t most_smem, size_t smem, cudaStream_t st,
                               Args... args) {
    cudaError_t e = once.run([&]() {
        cudaError_t r = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)most_smem);
        if (r == cudaSuccess)
            r = cudaFuncSetAttribute(kernel, cudaFuncAttributePreferredSharedMemoryCarveout,
                                     (int)cudaSharedmemCarveoutMaxShared);
        return r;
    });
    if (e != cudaSuccess) return e;
    e = launch_pdl_cluster(kernel, dim3(kPoolCtas), dim3(kPoolThreads), smem, st, kPoolCtas, args...);
    count_launches(1);
    return e;
}

cudaError_t launch_pages_alloc(const jsv_page_pool &pool, int32_t *table, int B, int max_pages, const int32_t *begin,
                               const int32_t *end, bool full_only, void *ws, cudaStream_t st) {
    static PerDeviceOnce once;
    return launch_pool(pages_alloc_kernel, once, JSV_PAGES_MAX_ROWS * sizeof(long long), B * sizeof(long long), st,
                       pool.num_pages, pool.refcount, pool.dev_status, table, B, max_pages, begin, end,
                       full_only ? 1 : 0, ws);
}

cudaError_t launch_pages_fork(const jsv_page_pool &pool, int32_t *table, int B, int max_pages, int n,
                              const int32_t *src, const int32_t *dst, const int32_t *len, bool full_only,
                              int32_t *copy_src, int32_t *copy_dst, void *ws, cudaStream_t st) {
    static PerDeviceOnce once;
    return launch_pool(pages_fork_kernel, once, 2 * JSV_PAGES_MAX_ROWS * sizeof(int), ((size_t)B + n) * sizeof(int),
                       st, pool.num_pages, pool.refcount, pool.dev_status, table, B, max_pages, n, src, dst, len,
                       full_only ? 1 : 0, copy_src, copy_dst, ws);
}

cudaError_t launch_pages_compact(const jsv_page_pool &pool, const int32_t *table, int B, int max_pages,
                                 int32_t *new_table, int32_t *new_refcount, int32_t *copy_src, int32_t *copy_dst,
                                 int max_copies, int32_t *num_copies, void *ws, cudaStream_t st) {
    static PerDeviceOnce once;
    return launch_pool(pages_compact_kernel, once, 0, 0, st, pool.num_pages, (const int32_t *)pool.refcount,
                       pool.dev_status, table, B, max_pages, new_table, new_refcount, copy_src, copy_dst, max_copies,
                       num_copies, ws);
}

cudaError_t launch_pages_trim(const jsv_page_pool &pool, int32_t *table, int B, int max_pages,
                              const int32_t *keep_begin, const int32_t *keep_end, cudaStream_t st) {
    static PerDeviceOnce once;
    cudaError_t e = prefer_max_shared(pages_trim_kernel, once);
    if (e != cudaSuccess) return e;
    const long long blocks = (long long)B * ((max_pages + kTrimThreads - 1) / kTrimThreads);
    e = launch_pdl(pages_trim_kernel, dim3((unsigned)std::min<long long>(blocks, 8 * device_sm_count())),
                   dim3(kTrimThreads), 0, st, pool.num_pages, pool.refcount, pool.dev_status, table, B, max_pages,
                   keep_begin, keep_end);
    count_launches(1);
    return e;
}

cudaError_t launch_pages_copy(const jsv_page_pool &pool, void *const *buffers, const int64_t *page_bytes,
                              int n_buffers, const int32_t *copy_src, const int32_t *copy_dst, int n,
                              const int32_t *num_copies, cudaStream_t st) {
    static PerDeviceOnce once;
    cudaError_t e = prefer_max_shared(pages_copy_kernel, once);
    if (e != cudaSuccess) return e;
    for (int b0 = 0; b0 < n_buffers; b0 += kCopyBuffers) {
        CopyBuffers bufs = {};
        const int nb = std::min(kCopyBuffers, n_buffers - b0);
        long long most = 0;
        for (int i = 0; i < nb; ++i) {
            bufs.base[i] = buffers[b0 + i];
            bufs.bytes[i] = page_bytes[b0 + i];
            const long long seg = (page_bytes[b0 + i] % 16 ? 4 : 16) * kCopyThreads * kCopyUnroll;
            most = std::max(most, (page_bytes[b0 + i] + seg - 1) / seg);
        }
        const long long per_buffer = std::max(1, 64 * device_sm_count() / nb);
        e = launch_pdl(pages_copy_kernel, dim3((unsigned)std::min<long long>(n * most, per_buffer), nb),
                       dim3(kCopyThreads), 0, st, pool.num_pages, pool.dev_status, bufs, copy_src, copy_dst, n,
                       num_copies);
        if (e != cudaSuccess) return e;
        count_launches(1);
    }
    return cudaSuccess;
}

}  // namespace jsv
