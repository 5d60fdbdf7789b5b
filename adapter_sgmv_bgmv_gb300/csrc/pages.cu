// Page tables in device memory: sequences get pages, share them, give them back, and the pages
// that are held move to the front of the pool.  Integers only; every result is determined by
// the inputs (the lowest free page first, lists in order), not by who comes first.
//
// refs[page] counts the sequences that hold a page; 0 is free, LORA_PAGE_PINNED and more stays where it
// is.  Extend and compact have to
// rank the free (or held) pages of the whole pool: one cluster of up to eight CTAs, each warp
// a run of pages, counts first, exchanges the counts through shared memory and walks its run
// again with its rank at hand.  Every wait in between is a hardware barrier of the block or the cluster.
//
// Bound: latency, launch and the chain lengths, counts, ranks, table; refs are 4 bytes a page
// (a pool of a million pages 4 MB, which eight SMs read in some microseconds).
//
// Measured: 64 sequences cut back and grown by up to eight tokens (pool of 20,000 pages) 9.8 us for
// both calls; 200 sequences freed and forked anew from one of 1876 pages 13.0 us, the 750,000
// atomic counts; compaction's table of 128 sequences and 24,000 pages 9.7 us, three launches.
#include <cuda_runtime.h>

#include <algorithm>
#include <type_traits>

#include "../../include/lora.h"
#include "kv.h"
#include "launch.cuh"
#include "ptx.cuh"

namespace lora {

namespace {

constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCluster = 8;
constexpr int kUnroll = 16;        // loads of refs a lane has under way

// All threads of all CTAs; lanes that took different ways meet first.
__device__ __forceinline__ void cluster_barrier()
{
    __syncwarp();
    cluster_sync();
}

__device__ __forceinline__ int ceil_div(int a, int b) { return int((unsigned(a) + unsigned(b) - 1) / unsigned(b)); }

// Inclusive scan over the block of one value a thread.
__device__ long long block_scan(long long v, long long *sums, long long &total)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, v, d);
        if (lane >= d)
            v += y;
    }
    __syncthreads();
    if (lane == 31)
        sums[warp] = v;
    __syncthreads();
    long long x = sums[lane];          // kWarps is 32
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, x, d);
        if (lane >= d)
            x += y;
    }
    total = __shfl_sync(0xffffffffu, x, 31);
    const long long before = __shfl_sync(0xffffffffu, x, max(warp - 1, 0));
    return v + (warp ? before : 0);
}

// A cluster's view of the pool: warp w of the cluster's warps has pages [lo, hi).
struct Run {
    int lo, hi;
};

__device__ __forceinline__ Run my_run(int n_pages, int n_cta)
{
    const int warps = n_cta * kWarps, w = int(cluster_ctarank()) * kWarps + int(threadIdx.x >> 5);
    const int64_t chunk = (int64_t(n_pages) + warps * 32 - 1) / (warps * 32) * 32;
    return {int(min(w * chunk, int64_t(n_pages))), int(min((w + 1) * chunk, int64_t(n_pages)))};
}

// Pages of the run with refs > 0, and the bits that any count has; the same in all lanes.
__device__ __forceinline__ int count_held(const int32_t *refs, const Run &r, int &bits)
{
    const int lane = threadIdx.x & 31;
    int n = 0, seen = 0;
    for (int base = r.lo; base < r.hi; base += 32 * kUnroll) {
        int v[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u)
            v[u] = base + u * 32 + lane < r.hi ? refs[base + u * 32 + lane] : 0;
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            n += v[u] > 0;
            seen |= v[u];
        }
    }
    bits = __reduce_or_sync(0xffffffffu, seen);
    return __reduce_add_sync(0xffffffffu, n);
}

// Pages of the run that are pinned.
__device__ __noinline__ int count_pinned(const int32_t *refs, const Run &r)
{
    int n = 0;
    for (int id = r.lo + int(threadIdx.x & 31); id < r.hi; id += 32)
        n += refs[id] >= LORA_PAGE_PINNED;
    return __reduce_add_sync(0xffffffffu, n);
}

// What all warps counted, K numbers each: the sums ahead of this warp's and over the cluster.  `counts`
// is K entries a warp in every CTA's shared memory; ends behind a cluster barrier, and the caller has
// to pass another before it leaves.
template <int K>
__device__ __forceinline__ void rank_warps(const int (&mine)[K], int (*counts)[kWarps], int n_cta, int (&before)[K], int (&total)[K])
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, rank = int(cluster_ctarank());
#pragma unroll
    for (int k = 0; k < K; ++k) {
        if (lane == 0)
            counts[k][warp] = mine[k];
        before[k] = total[k] = 0;
    }
    if (n_cta == 1)
        __syncthreads();
    else
        cluster_barrier();
    for (int c = 0; c < n_cta; ++c)
#pragma unroll
        for (int k = 0; k < K; ++k) {
            int v = counts[k][lane];
            if (n_cta > 1)
                asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(map_cluster(smem_u32(&counts[k][lane]), c)) : "memory");
            total[k] += v;
            before[k] += c < rank || (c == rank && lane < warp) ? v : 0;
        }
#pragma unroll
    for (int k = 0; k < K; ++k) {
        total[k] = __reduce_add_sync(0xffffffffu, total[k]);
        before[k] = __reduce_add_sync(0xffffffffu, before[k]);
    }
}

// ---------------------------------------------------------------- extend

// Per sequence, in the dynamic shared memory of every CTA.
struct Want {
    int upto;                 // pages wanted up to and with this one
    int first;                // first column that gets a page; the sign bit: it is a copy
};

struct ExtendArgs {
    TableView t;
    const int32_t *grow;
    int32_t *got, *src, *dst, *cells;
};

__global__ void __launch_bounds__(kThreads) k_pages_extend(const __grid_constant__ ExtendArgs a, int n_cta)
{
    extern __shared__ __align__(16) uint8_t smem[];
    const TableView &t = a.t;
    Want *want = reinterpret_cast<Want *>(smem);
    int *mark = reinterpret_cast<int *>(want + t.n_seqs);        // the shared page a sequence would write into, or -1
    __shared__ long long sums[kWarps];
    __shared__ int counts[1][kWarps];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, rank = int(cluster_ctarank());
    unsigned *status = rank == 0 ? t.status : nullptr;
    grid_dep_wait();
    grid_dep_launch();

    const Run run = my_run(t.n_pages, n_cta);
    int bits;
    const int held[1] = {count_held(t.refs, run, bits)};

    // What each sequence wants: every CTA works it out for itself.
    int any = 0;
    for (int s = threadIdx.x; s < t.n_seqs; s += kThreads) {
        const int len = t.lens[s], grow = a.grow[s];
        bool ok = grow > 0;
        if (ok && (len < 0 || len > t.capacity)) {
            raise_status(status, kDevBadBatch);
            ok = false;
        }
        ok = ok && grow <= t.capacity - len;
        int m = -1;
        if (ok && len % t.page_size) {
            const int page = t.pages[s * t.ld_pages + len / t.page_size];
            if (page < 0 || page >= t.n_pages) {
                raise_status(status, kDevBadPage);
                ok = false;
            } else if (t.refs[page] > 1) {
                m = page;
                any = 1;
            }
        }
        mark[s] = m;
        want[s].upto = ok ? ceil_div(len + grow, t.page_size) - ceil_div(len, t.page_size) : -1;
        want[s].first = ok ? ceil_div(len, t.page_size) : 0;
    }
    any = __syncthreads_or(any);
    // Writers of one shared page: all but the last take a copy; all, where others hold it too.
    if (any) {
        for (int s = warp; s < t.n_seqs; s += kWarps) {
            const int m = mark[s];
            if (m < 0)
                continue;
            int writers = 0, later = 0;
            for (int o = lane; o < t.n_seqs; o += 32) {
                const bool same = mark[o] == m;
                writers += same;
                later |= same && o > s;
            }
            writers = __reduce_add_sync(0xffffffffu, writers);
            later = __any_sync(0xffffffffu, later);
            if (lane)
                continue;
            if (writers > t.refs[m]) {               // more than are counted: the table is wrong
                raise_status(status, kDevBadPage);
                want[s].upto = -1;
            } else if (later || writers < t.refs[m]) {
                want[s].upto += 1;
                want[s].first = (want[s].first - 1) | int(0x80000000u);
            }
        }
        __syncthreads();
    }
    // Needs to running sums; a sequence that wants nothing is told by its need of -1.
    long long carry = 0;
    for (int base = 0; base < t.n_seqs; base += kThreads) {
        const int s = base + threadIdx.x;
        const int need = s < t.n_seqs ? want[s].upto : 0;
        long long total;
        const long long x = carry + block_scan(max(need, 0), sums, total);
        carry += total;
        if (s < t.n_seqs) {
            want[s].upto = int(min(x, (long long)0x7fffffff));
            mark[s] = need;
        }
    }

    int held_before[1], held_all[1];
    rank_warps(held, counts, n_cta, held_before, held_all);      // behind it nobody reads lens or another's refs
    const int free_all = t.n_pages - held_all[0];

    if (rank == 0)
        for (int s = threadIdx.x; s < t.n_seqs; s += kThreads) {
            const bool served = mark[s] >= 0 && want[s].upto <= free_all, copy = served && want[s].first < 0;
            const int len = t.lens[s], grow = served ? a.grow[s] : 0;
            a.got[s] = grow;
            a.cells[s] = copy ? len % t.page_size : 0;
            if (!copy)
                a.src[s] = a.dst[s] = -1;
            if (served)
                t.lens[s] = len + grow;
        }
    // The free pages in order, each to whoever wants one of its rank.
    const int wanted = t.n_seqs ? want[t.n_seqs - 1].upto : 0;
    int next = run.lo - held_before[0];
    if (held[0] < run.hi - run.lo)
        for (int base = run.lo; base < run.hi && next < wanted; base += 32) {
            const int id = base + lane;
            const bool is_free = id < run.hi && t.refs[id] <= 0;
            const unsigned m = __ballot_sync(0xffffffffu, is_free);
            const int k = next + __popc(m & ((1u << lane) - 1));
            next += __popc(m);
            if (!is_free || k >= wanted)
                continue;
            int lo = 0, hi = t.n_seqs - 1;           // the first sequence with upto > k
            while (lo < hi) {
                const int mid = (lo + hi) >> 1;
                if (want[mid].upto > k)
                    hi = mid;
                else
                    lo = mid + 1;
            }
            if (want[lo].upto > free_all)
                continue;
            const int nth = k - (want[lo].upto - mark[lo]), first = want[lo].first;
            int32_t *at = t.pages + lo * t.ld_pages + (first & 0x7fffffff) + nth;
            if (first < 0 && nth == 0) {
                const int old = *at;
                atomicSub(&t.refs[old], 1);
                a.src[lo] = old;
                a.dst[lo] = id;
            }
            *at = id;
            t.refs[id] = 1;
        }
    if (n_cta > 1)
        cluster_barrier();                           // others may still read this CTA's counts
}

// ---------------------------------------------------------------- fork, free

// Whether an earlier entry of a list holds the same value; every thread of the block calls it.
__device__ __forceinline__ bool seen_before(const int32_t *list, int i, int value)
{
    int hit = 0;
    for (int j = threadIdx.x; j < i; j += blockDim.x)
        hit |= list[j] == value;
    return __syncthreads_or(hit);
}

constexpr int kBatch = 4;          // columns a thread has under way

__global__ void __launch_bounds__(kThreads) k_pages_fork(const __grid_constant__ TableView t, const int32_t *from,
                                                         const int32_t *to, int n)
{
    grid_dep_wait();
    grid_dep_launch();
    const int i = blockIdx.x, parent = from[i], child = to[i];
    bool bad = parent < 0 || parent >= t.n_seqs || child < 0 || child >= t.n_seqs;
    bad = seen_before(to, i, child) || bad;          // twice the same child: the first one counts
    bad = seen_before(to, n, parent) || bad;         // a row that this call writes
    int len = 0;
    if (!bad) {
        len = t.lens[parent];
        bad = len < 0 || len > t.capacity || t.lens[child] != 0;
    }
    __syncthreads();                                 // all have read the child's length
    if (bad) {
        if (threadIdx.x == 0)
            raise_status(t.status, kDevBadBatch);
        return;
    }
    const int cols = ceil_div(len, t.page_size);
    const int32_t *src = t.pages + parent * t.ld_pages;
    int32_t *dst = t.pages + child * t.ld_pages;
    for (int c0 = threadIdx.x; c0 < cols; c0 += blockDim.x * kBatch) {
        int page[kBatch];
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
            const int c = c0 + b * int(blockDim.x);
            page[b] = c < cols ? src[c] : -1;
        }
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
            const int c = c0 + b * int(blockDim.x);
            if (c >= cols)
                continue;
            if (page[b] < 0 || page[b] >= t.n_pages)
                raise_status(t.status, kDevBadPage);
            else
                atomicAdd(&t.refs[page[b]], 1);
            dst[c] = page[b];
        }
    }
    if (threadIdx.x == 0)
        t.lens[child] = len;
}

__global__ void __launch_bounds__(kThreads) k_pages_free(const __grid_constant__ TableView t, const int32_t *seqs,
                                                         const int32_t *keeps, int n)
{
    grid_dep_wait();
    grid_dep_launch();
    const int i = blockIdx.x, s = seqs[i];
    bool bad = s < 0 || s >= t.n_seqs;
    bad = seen_before(seqs, i, s) || bad;            // twice the same sequence: the first one counts
    int len = 0, keep = 0;
    if (!bad) {
        len = t.lens[s];
        keep = keeps ? keeps[i] : 0;
        bad = len < 0 || len > t.capacity || keep < 0;
    }
    __syncthreads();                                 // all have read the length
    if (bad) {
        if (threadIdx.x == 0)
            raise_status(t.status, kDevBadBatch);
        return;
    }
    if (keep >= len)
        return;
    const int cols = ceil_div(len, t.page_size);
    int32_t *row = t.pages + s * t.ld_pages;
    for (int c0 = ceil_div(keep, t.page_size) + threadIdx.x; c0 < cols; c0 += blockDim.x * kBatch) {
        int page[kBatch];
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
            const int c = c0 + b * int(blockDim.x);
            page[b] = c < cols ? row[c] : -1;
        }
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
            const int c = c0 + b * int(blockDim.x);
            if (c >= cols)
                continue;
            if (page[b] < 0 || page[b] >= t.n_pages) {
                raise_status(t.status, kDevBadPage);
            } else {
                const int was = atomicSub(&t.refs[page[b]], 1);
                // no sequence holds it (others may just be finding out the same): the table is wrong
                if (was <= 0 || (was <= LORA_PAGE_PINNED && was > LORA_PAGE_PINNED - kMaxTableSeqs)) {
                    atomicAdd(&t.refs[page[b]], 1);
                    raise_status(t.status, kDevBadPage);
                }
            }
            row[c] = -1;
        }
    }
    if (threadIdx.x == 0)
        t.lens[s] = keep;
}

// ---------------------------------------------------------------- compact

// A pinned page stays where it is and takes no part: the others have their places between them,
// place = id - pinned pages before it.  With L held ones of those, the held ones at places from L on
// move to the free places below L: the highest to the lowest.  A free page at place p < L is
// the (p - held before it)-th hole, a held one at p >= L has L - 1 - held before it higher movers:
// both know their position in the lists.
__global__ void __launch_bounds__(kThreads) k_pages_compact(const __grid_constant__ TableView t, int32_t *src,
                                                            int32_t *dst, int n, int32_t *top, int n_cta)
{
    __shared__ int counts[2][kWarps];
    const int lane = threadIdx.x & 31, at = int(cluster_ctarank()) * kThreads + int(threadIdx.x), all = n_cta * kThreads;
    grid_dep_wait();
    grid_dep_launch();
    for (int k = at; k < n; k += all)
        src[k] = dst[k] = -1;
    const Run run = my_run(t.n_pages, n_cta);
    int bits, first[2], sums[2];
    const int held_here = count_held(t.refs, run, bits);
    const int mine[2] = {held_here, bits & LORA_PAGE_PINNED ? count_pinned(t.refs, run) : 0};
    rank_warps(mine, counts, n_cta, first, sums);
    const int pinned = mine[1], held = mine[0] - pinned, total = sums[0] - sums[1];
    const int held0 = first[0] - first[1], pinned0 = first[1];
    const bool pins_there = sums[1] > 0;
    if (at == 0 && top)
        *top = pins_there ? 0 : total;               // and where there are pins, or a mover stays, what these say below
    int end = 0;                                     // of the highest page that this lane knows is held in the end
    auto walk = [&](auto with_pins) {
        constexpr bool kPins = decltype(with_pins)::value;
        int before = held0, pins = pinned0;
        for (int base = run.lo; base < run.hi; base += 32 * 4) {
            int v[4];
#pragma unroll
            for (int u = 0; u < 4; ++u)
                v[u] = base + u * 32 + lane < run.hi ? t.refs[base + u * 32 + lane] : 0;
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const int id = base + u * 32 + lane;
                const bool pin = kPins && v[u] >= LORA_PAGE_PINNED, on = v[u] > 0 && !pin;
                const unsigned below = (1u << lane) - 1, m = __ballot_sync(0xffffffffu, on);
                const int ahead = before + __popc(m & below);
                before += __popc(m);
                int place = id - pins;
                if (kPins) {
                    const unsigned mp = __ballot_sync(0xffffffffu, pin);
                    place -= __popc(mp & below);
                    pins += __popc(mp);
                }
                if (id >= run.hi)
                    continue;
                if (kPins && (pin || place == total - 1))
                    end = id + 1;
                if (pin)
                    continue;
                if (place < total) {
                    if (!on && place - ahead < n)
                        dst[place - ahead] = id;
                } else if (on && total - 1 - ahead < n) {
                    src[total - 1 - ahead] = id;
                }
            }
        }
    };
    // The last place below L is held if all move; else a page that stays is higher.
    if (pinned) {
        walk(std::true_type());
    } else {
        const int last = total - 1 + pinned0;
        if (pins_there && last >= run.lo && last < run.hi)
            end = last + 1;
        // a run of free pages at or above L, or of held ones below it, has nothing to move
        if (!(held == 0 && run.lo - pinned0 >= total) && !(held == run.hi - run.lo && run.hi - pinned0 <= total))
            walk(std::false_type());
    }
    cluster_barrier();
    // Where the lists are full, the mover with n higher ones is the highest that stays.
    if (top && (n == 0 || src[n - 1] >= 0) && held > 0 && run.hi > total) {
        int b = held0;
        for (int base = run.lo; base < run.hi; base += 32) {
            const int id = base + lane;
            const int v = id < run.hi ? t.refs[id] : 0;
            const bool on = v > 0 && v < LORA_PAGE_PINNED;
            const unsigned m = __ballot_sync(0xffffffffu, on);
            const int ahead = b + __popc(m & ((1u << lane) - 1));
            b += __popc(m);
            if (on && total - 1 - ahead == n)
                end = max(end, id + 1);
        }
    }
    if (top) {
        end = __reduce_max_sync(0xffffffffu, end);
        if (lane == 0 && end)
            atomicMax(top, end);
    }
    cluster_barrier();
    // The counts move; the old place holds where to (as its complement) until the tables know.
    for (int k = at; k < n; k += all) {
        const int s = src[k], d = dst[k];
        if (s >= 0) {
            t.refs[d] = t.refs[s];
            t.refs[s] = ~d;
        }
    }
}

__global__ void __launch_bounds__(256) k_pages_moved(const __grid_constant__ TableView t)
{
    grid_dep_wait();
    grid_dep_launch();
    const int s = blockIdx.x, len = t.lens[s];
    if (len < 0 || len > t.capacity) {
        if (threadIdx.x == 0 && blockIdx.y == 0)
            raise_status(t.status, kDevBadBatch);
        return;
    }
    const int cols = ceil_div(len, t.page_size), step = int(gridDim.y * blockDim.x);
    int32_t *row = t.pages + s * t.ld_pages;
    for (int c0 = int(blockIdx.y * blockDim.x + threadIdx.x); c0 < cols; c0 += step * kBatch) {
        int page[kBatch], to[kBatch];
#pragma unroll
        for (int b = 0; b < kBatch; ++b)
            page[b] = c0 + b * step < cols ? row[c0 + b * step] : -1;
#pragma unroll
        for (int b = 0; b < kBatch; ++b)
            to[b] = page[b] >= 0 && page[b] < t.n_pages ? t.refs[page[b]] : 0;
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
            if (c0 + b * step >= cols)
                continue;
            if (page[b] < 0 || page[b] >= t.n_pages)
                raise_status(t.status, kDevBadPage);
            else if (to[b] < 0 && ~to[b] < t.n_pages)
                row[c0 + b * step] = ~to[b];
        }
    }
}

__global__ void __launch_bounds__(256) k_pages_moved_end(const __grid_constant__ TableView t, const int32_t *src, int n)
{
    grid_dep_wait();
    grid_dep_launch();
    const int k = int(blockIdx.x * blockDim.x + threadIdx.x);
    if (k < n && src[k] >= 0)
        t.refs[src[k]] = 0;
}

// A CTA for each 512 pages a warp, up to the largest cluster that every GPU takes.
int cluster_for(int n_pages)
{
    int c = 1;
    while (c < kMaxCluster && int64_t(c) * kWarps * 32 * kUnroll < n_pages)
        c *= 2;
    return c;
}

// Threads of a CTA that walks one sequence's row.
int threads_for(int n_cols) { return n_cols <= 1024 ? 256 : kThreads; }

}  // namespace

cudaError_t launch_pages_extend(const TableView &t, const int32_t *grow, int32_t *got, int32_t *src,
                                int32_t *dst, int32_t *cells, cudaStream_t stream)
{
    static OncePerDevice once;
    const cudaError_t e = allow_shared(once, k_pages_extend, kMaxTableSeqs * (sizeof(Want) + sizeof(int)));
    if (e != cudaSuccess)
        return e;
    const int c = cluster_for(t.n_pages);
    return start(k_pages_extend, dim3(unsigned(c)), kThreads, size_t(t.n_seqs) * (sizeof(Want) + sizeof(int)), c, stream,
                 ExtendArgs{t, grow, got, src, dst, cells}, c);
}

cudaError_t launch_pages_fork(const TableView &t, const int32_t *from, const int32_t *to, int n, cudaStream_t stream)
{
    return start(k_pages_fork, dim3(unsigned(n)), threads_for(t.n_cols), 0, 0, stream, t, from, to, n);
}

cudaError_t launch_pages_free(const TableView &t, const int32_t *seqs, const int32_t *keep, int n, cudaStream_t stream)
{
    return start(k_pages_free, dim3(unsigned(n)), threads_for(t.n_cols), 0, 0, stream, t, seqs, keep, n);
}

cudaError_t launch_pages_compact(const TableView &t, int32_t *src, int32_t *dst, int n, int32_t *top, int *launches,
                                 cudaStream_t stream)
{
    const int c = cluster_for(t.n_pages);
    cudaError_t e = start(k_pages_compact, dim3(unsigned(c)), kThreads, 0, c, stream, t, src, dst, n, top, c);
    *launches = e == cudaSuccess;
    if (e == cudaSuccess && t.n_seqs && n) {
        const int parts = std::max(1, std::min(t.n_cols / 1024, 32));
        e = start(k_pages_moved, dim3(unsigned(t.n_seqs), unsigned(parts)), 256, 0, 0, stream, t);
        *launches += e == cudaSuccess;
    }
    if (e == cudaSuccess && n) {
        e = start(k_pages_moved_end, dim3(unsigned((n + 255) / 256)), 256, 0, 0, stream, t, static_cast<const int32_t *>(src), n);
        *launches += e == cudaSuccess;
    }
    return e;
}

}  // namespace lora
