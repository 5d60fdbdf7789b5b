// Copies of pages within caches of one shape (a model's layers share one page table, so one list
// of pairs serves them all): keys, values, scales and bounds of page src[i] to page dst[i].
//
// The list may be long and mostly empty (one entry a sequence, few of them forked), so the
// grid is fixed and each CTA first gathers the pairs that are there, kList entries at a time;
// then its warps take items of up to 2 KB (a pair's keys or values in one cache, a part of
// the page), all of an item's loads under way before its first store.
//
// Bound: DRAM, every byte read and written once.  4640 pages of 16 KB in each of four caches, 608 MB:
// 102 us, 6.0 TB/s (0.88 of a copy's rate).  48 to 64 KB under way a SM are best: 128 KB (16 warps of
// 4 KB twice) take 117 us, 192 KB 207; one CTA of 16 warps of 4 KB 99, but 0.7 us more for a few pages.
#include <cuda_runtime.h>

#include <algorithm>

#include "kv.h"
#include "launch.cuh"
#include "ptx.cuh"

namespace lora {

namespace {

constexpr int kThreads = 256;
constexpr int kCtas = 3;                     // a SM
constexpr int kWarps = kThreads / 32;
constexpr int kList = 4096;                  // entries looked at at once
constexpr int kItem = 2048;                  // bytes of an item
constexpr int kUnits = kItem / 16 / 32;      // 16-byte units of it a lane

struct Shape {
    Divider per_cell;                        // by the heads
    int parts;                               // items of a page's keys
    int unit_shift;                          // log2 of a vector's 16-byte units
};

// The caches travel in the launch's parameters: up to eight in an eighth of the bytes that 64 take, half a
// microsecond less on the host.
template <int CACHES>
struct Params : KvCopyLists {
    KvView kv[CACHES];
    int n_kv;
    unsigned *status;
};

template <int CACHES>
__global__ void __launch_bounds__(kThreads, kCtas) k_kv_copy(const __grid_constant__ Params<CACHES> p, Shape sh)
{
    __shared__ int pairs[kList];
    __shared__ int counts[kWarps];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const KvView &kv0 = p.kv[0];
    const int vecs = kItem / 16 >> sh.unit_shift;            // vectors of an item
    const int all_vecs = kv0.page_size * kv0.heads;          // of a page
    grid_dep_wait();
    grid_dep_launch();
    for (int base = 0; base < p.n; base += kList) {
        // in the same order in every CTA: the items are dealt out by number
        constexpr int kRounds = kList / kThreads;
        unsigned there[kRounds];
        int mine = 0;
#pragma unroll
        for (int u = 0; u < kRounds; ++u) {
            const int i = base + (warp * kRounds + u) * 32 + lane;
            there[u] = __ballot_sync(0xffffffffu, i < p.n && p.src[i] >= 0);
            mine += __popc(there[u]);
        }
        if (lane == 0)
            counts[warp] = mine;
        __syncthreads();
        int at_pair = 0, n_pairs = 0;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            at_pair += w < warp ? counts[w] : 0;
            n_pairs += counts[w];
        }
#pragma unroll
        for (int u = 0; u < kRounds; ++u) {
            if (there[u] >> lane & 1)
                pairs[at_pair + __popc(there[u] & ((1u << lane) - 1))] = base + (warp * kRounds + u) * 32 + lane;
            at_pair += __popc(there[u]);
        }
        __syncthreads();
        const int per_pair = p.n_kv * 2 * sh.parts;
        const int64_t items = int64_t(n_pairs) * per_pair;
        for (int64_t it = int64_t(blockIdx.x) + int64_t(warp) * gridDim.x; it < items; it += int64_t(gridDim.x) * kWarps) {
            const int slot = int(items >> 31 ? it / per_pair : int64_t(unsigned(it) / unsigned(per_pair)));
            int rest = int(it - int64_t(slot) * per_pair);
            const int part = rest % sh.parts;
            rest /= sh.parts;
            const KvView &kv = p.kv[rest >> 1];
            const bool is_v = rest & 1;
            const int i = pairs[slot], s = p.src[i], d = p.dst[i];
            const int cells = p.cells ? min(p.cells[i], kv.page_size) : kv.page_size;
            if (s >= kv.n_pages || d < 0 || d >= kv.n_pages) {
                if (lane == 0)
                    raise_status(p.status, kDevBadPage);
                continue;
            }
            uint8_t *pool = is_v ? kv.v : kv.k;
            const uint8_t *from = pool + s * kv.page_stride;
            uint8_t *to = pool + d * kv.page_stride;
            const int vec0 = part * vecs, cell0 = vec0 / kv.heads, head0 = vec0 - cell0 * kv.heads;
            const int n_vec = min(vecs, min(all_vecs, max(cells, 0) * kv.heads) - vec0);
            uint4 x[kUnits];
            int64_t at[kUnits];
#pragma unroll
            for (int u = 0; u < kUnits; ++u) {
                const int unit = lane + 32 * u, vec = unit >> sh.unit_shift;
                const int c = sh.per_cell.quotient(head0 + vec), head = head0 + vec - c * kv.heads;
                at[u] = vec < n_vec ? (cell0 + c) * kv.cell_stride + head * kv.head_stride + ((unit - (vec << sh.unit_shift)) << 4) : -1;
                if (at[u] >= 0)
                    x[u] = *reinterpret_cast<const uint4 *>(from + at[u]);
            }
#pragma unroll
            for (int u = 0; u < kUnits; ++u)
                if (at[u] >= 0)
                    *reinterpret_cast<uint4 *>(to + at[u]) = x[u];
            if (kv.format != kKvBf16) {
                float *scale = is_v ? kv.v_scale : kv.k_scale;
                for (int vec = lane; vec < n_vec; vec += 32) {
                    const int c = sh.per_cell.quotient(head0 + vec), head = head0 + vec - c * kv.heads;
                    const int64_t o = (cell0 + c) * kv.s_cell + head * kv.s_head;
                    scale[d * kv.s_page + o] = scale[s * kv.s_page + o];
                }
            }
            if (kv.bounds && part == 0 && !is_v) {
                const int64_t bytes = int64_t(kv.heads) * 2 * kv.dim;
                for (int64_t o = lane * 16; o < bytes; o += 512)
                    *reinterpret_cast<uint4 *>(kv.bounds + d * bytes + o) = *reinterpret_cast<const uint4 *>(kv.bounds + s * bytes + o);
                for (int h = lane; h < kv.heads; h += 32)
                    kv.unit[int64_t(d) * kv.heads + h] = kv.unit[int64_t(s) * kv.heads + h];
            }
        }
        __syncthreads();
    }
}

template <int CACHES>
cudaError_t launch(const KvView *kv, int n_kv, const KvCopyLists &lists, unsigned *status, const Shape &sh, unsigned ctas, cudaStream_t stream)
{
    Params<CACHES> p;
    static_cast<KvCopyLists &>(p) = lists;
    std::copy(kv, kv + n_kv, p.kv);
    p.n_kv = n_kv;
    p.status = status;
    return start(k_kv_copy<CACHES>, dim3(ctas), kThreads, 0, 0, stream, p, sh);
}

}  // namespace

cudaError_t launch_kv_copy(const KvView *kv, int n_kv, const KvCopyLists &lists, unsigned *status, int sms, cudaStream_t stream)
{
    const int bytes = kv->dim * (kv->format == kKvBf16 ? 2 : 1);
    Shape sh;
    sh.per_cell = Divider(kv->heads);
    sh.unit_shift = bytes == 256 ? 4 : bytes == 128 ? 3 : 2;
    const int64_t vecs = int64_t(kv->page_size) * kv->heads;
    sh.parts = int((vecs * bytes + kItem - 1) / kItem);
    const int64_t items = int64_t(lists.n) * n_kv * 2 * sh.parts;
    const unsigned ctas = unsigned(std::min<int64_t>(int64_t(kCtas) * sms, items));
    return n_kv <= 8 ? launch<8>(kv, n_kv, lists, status, sh, ctas, stream)
                     : launch<kMaxCopyCaches>(kv, n_kv, lists, status, sh, ctas, stream);
}

}  // namespace lora
