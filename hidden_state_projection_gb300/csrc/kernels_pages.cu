// kernels_pages.cu -- the pages of a cache: sequences grown, cut, freed and forked, live pages
// moved together, pages copied.
//
// All decisions are made on the device from the caller's arrays (block table, lengths, holder
// counts), so a decode step that grows, forks or frees sequences needs no copy to the host
// and can be captured.  They are integers and their outcome does not depend on the order in
// which threads run: pages are handed out lowest first in the order of the request, counts
// change by integer atomics.
//
//   resize  hsp_resize_plan_kernel (one CTA: prefix sum of the pages wanted, the lowest free
//           pages) and hsp_resize_apply_kernel (table, counts, and the copies of shared last
//           pages, over the whole GPU)
//           or, small calls, hsp_resize_team_kernel (one cluster for all of it)
//   fork    hsp_fork_kernel (a CTA per child)
//   compact hsp_compact_plan_kernel (one CTA: the k-th live page past the number of live
//           pages goes to the k-th free page before it, so sources and destinations never
//           meet) and hsp_compact_apply_kernel
//   copy    hsp_copy_pages_kernel (pairs by value, checked on the host)
//
// The plan kernels are bound by latency: a warp takes a contiguous share of the counts, 128 at a
// time (four 4-byte loads of every lane in flight), sums by shuffles, the warps' sums in shared
// memory; resize reads the counts twice (how many are free, which), compaction three times (how
// many are live, how many holes and tails lie in front of a warp's share, which).  The moves are
// bound by memory: 16 KB pieces, four 16-byte loads per thread before the stores, and CTAs that
// take the pieces in order as they get free: 6000 pages of 73,728 bytes took 144 us with a fixed
// stride over a resident grid (6.1 TB/s), 133 us in order (6.67 TB/s, the rate of a plain
// device copy).
#include <stdint.h>

#include "cache_args.h"
#include "ptx.cuh"

namespace hsp {

namespace {

constexpr int kPlanThreads = 1024;
constexpr int kPlanWarps = kPlanThreads / 32;
constexpr int kPagesThreads = 256;

__device__ __forceinline__ int pages_of(int len, int shift) {
    return static_cast<int>((static_cast<int64_t>(len) + (1 << shift) - 1) >> shift);
}

// Exclusive prefix of v over the CTA's threads, and the sum.
__device__ __forceinline__ int64_t block_prefix(int64_t v, int64_t *warp_sums, int64_t *sum) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int64_t incl = v;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int64_t o = __shfl_up_sync(0xffffffffu, incl, d);
        if (lane >= d) incl += o;
    }
    __syncthreads();  // warp_sums of the last call have been read
    if (lane == 31) warp_sums[warp] = incl;
    __syncthreads();
    int64_t before = 0, all = 0;
    for (int w = 0; w < kPlanWarps; ++w) {
        if (w < warp) before += warp_sums[w];
        all += warp_sums[w];
    }
    *sum = all;
    return before + incl - v;
}

// ---- copies ---------------------------------------------------------------------------

// Copies unit u of a list of page pairs: pair u / pieces_total, then pool, layer and piece.
template <typename Pair>
__device__ __forceinline__ void copy_unit(const PoolList &pl, int64_t u, Pair pair) {
    const int64_t k = u / pl.pieces_total;
    int rem = static_cast<int>(u - k * pl.pieces_total);
    int p = 0;
    while (p + 1 < pl.count && rem >= pl.layers[p] * pl.pieces[p]) {
        rem -= pl.layers[p] * pl.pieces[p];
        ++p;
    }
    const int layer = rem / pl.pieces[p];
    const int64_t at = static_cast<int64_t>(rem - layer * pl.pieces[p]) * kCopyPiece;
    const int2 ids = pair(k);
    const char *from = pl.base[p] + layer * pl.layer_stride[p] + ids.x * pl.page_stride[p] + at;
    char *to = pl.base[p] + layer * pl.layer_stride[p] + ids.y * pl.page_stride[p] + at;
    const int n16 = static_cast<int>(min(static_cast<int64_t>(kCopyPiece), pl.page_bytes[p] - at) / 16);
    constexpr int kPer = kCopyPiece / 16 / kPagesThreads;
    uint4 v[kPer];
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
        const int c = threadIdx.x + j * kPagesThreads;
        if (c < n16) v[j] = reinterpret_cast<const uint4 *>(from)[c];
    }
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
        const int c = threadIdx.x + j * kPagesThreads;
        if (c < n16) reinterpret_cast<uint4 *>(to)[c] = v[j];
    }
}

// All page pairs by a team of kTeam CTAs with kPlanThreads threads: the 16-byte lines of all pages, layers and
// pools in one row, four on their way per thread before the first is stored (at most kTeamBytes in all).
template <typename Pair>
__device__ __forceinline__ void copy_by_team(const PoolList &pl, int moves, int rank, Pair pair) {
    constexpr uint32_t kDeep = 4, kStep = kTeam * kPlanThreads;
    uint32_t per = 0;
    for (int p = 0; p < pl.count; ++p) per += static_cast<uint32_t>(pl.layers[p] * (pl.page_bytes[p] / 16));
    const uint32_t lines = static_cast<uint32_t>(moves) * per;
    for (uint32_t f0 = rank * kPlanThreads + threadIdx.x; f0 < lines; f0 += kDeep * kStep) {
        uint4 v[kDeep];
        uint4 *to[kDeep];
#pragma unroll
        for (uint32_t j = 0; j < kDeep; ++j) {
            const uint32_t f = f0 + j * kStep;
            to[j] = nullptr;
            if (f >= lines) continue;
            const uint32_t k = f / per;
            uint32_t rem = f - k * per;
            int p = 0;
            for (; p + 1 < pl.count; ++p) {
                const uint32_t n = static_cast<uint32_t>(pl.layers[p] * (pl.page_bytes[p] / 16));
                if (rem < n) break;
                rem -= n;
            }
            const uint32_t page = static_cast<uint32_t>(pl.page_bytes[p] / 16), layer = rem / page;
            char *const base = pl.base[p] + layer * pl.layer_stride[p] + static_cast<int64_t>(rem - layer * page) * 16;
            const int2 ids = pair(k);
            v[j] = *reinterpret_cast<const uint4 *>(base + ids.x * pl.page_stride[p]);
            to[j] = reinterpret_cast<uint4 *>(base + ids.y * pl.page_stride[p]);
        }
#pragma unroll
        for (uint32_t j = 0; j < kDeep; ++j)
            if (to[j]) *to[j] = v[j];
    }
}

// All units of copy_unit, taken in order from a counter that starts at zero.  All threads call.
template <typename Pair>
__device__ __forceinline__ void copy_in_order(const PoolList &pl, int64_t units, unsigned long long *counter, Pair pair) {
    __shared__ int64_t next;
    if (units == 0) return;
    int64_t mine = 0;
    if (threadIdx.x == 0) mine = static_cast<int64_t>(atomicAdd(counter, 1ull));
    for (;;) {
        if (threadIdx.x == 0) next = mine;
        __syncthreads();
        const int64_t u = next;
        if (u >= units) return;
        if (threadIdx.x == 0) mine = static_cast<int64_t>(atomicAdd(counter, 1ull));  // on its way during the copy
        copy_unit(pl, u, pair);
        __syncthreads();
    }
}

template <int PAIRS>
struct CopyArgs {
    PoolList pools;
    int32_t n;
    int32_t src[PAIRS], dst[PAIRS];
};

template <int PAIRS>
__global__ void __launch_bounds__(kPagesThreads) hsp_copy_pages_kernel(const __grid_constant__ CopyArgs<PAIRS> a) {
    griddep_wait();
    const int64_t units = static_cast<int64_t>(a.n) * a.pools.pieces_total;
    for (int64_t u = blockIdx.x; u < units; u += gridDim.x)
        copy_unit(a.pools, u, [&](int64_t k) { return make_int2(a.src[k], a.dst[k]); });
    cta_release_and_trigger();
}

// ---- resize ---------------------------------------------------------------------------

__global__ void __launch_bounds__(kPlanThreads) hsp_resize_plan_kernel(const __grid_constant__ ResizeArgs a) {
    __shared__ int64_t warp_sums[kPlanWarps];
    __shared__ int warp_free[kPlanWarps];
    __shared__ int pair_count;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const IndexArgs &ix = a.ix;
    const int64_t most = static_cast<int64_t>(ix.max_pages) << ix.page_shift;
    griddep_launch_dependents();  // (the apply kernel, which waits for this one's end)
    griddep_wait();
    // a row named twice counts once: the first of them
    for (int i = tid; i < a.n; i += kPlanThreads) {
        const int r = a.rows[i];
        if (r >= 0 && r < ix.num_rows) a.claims[r] = 0x7fffffff;
    }
    if (tid == 0) pair_count = 0;
    __syncthreads();
    for (int i = tid; i < a.n; i += kPlanThreads) {
        const int r = a.rows[i];
        if (r >= 0 && r < ix.num_rows) atomicMin(&a.claims[r], i);
    }
    __syncthreads();
    int64_t total = 0;
    for (int i0 = 0; i0 < a.n; i0 += kPlanThreads) {
        const int i = i0 + tid;
        RowPlan p;
        p.row = -1;
        p.len = p.have = p.want = p.first = 0;
        p.cow_src = -1;
        int need = 0;
        if (i < a.n) {
            const int r = a.rows[i], want = a.new_lens[i];
            const bool in = r >= 0 && r < ix.num_rows;
            if (!in) atomicCAS(ix.err_word, 0, kDeviceErrIndex);
            if (in && a.claims[r] == i && want >= 0 && want <= most) {
                const int old = ix.lens[r];
                if (old >= 0 && old <= most) {
                    p.row = r;
                    p.len = want;
                    p.have = pages_of(old, ix.page_shift);
                    p.want = pages_of(want, ix.page_shift);
                    if (want > old && (old & ((1 << ix.page_shift) - 1)) != 0) {
                        const int last = ix.table[r * ix.table_stride + p.have - 1];
                        if (last < 0 || last >= ix.num_pages) atomicCAS(ix.err_word, 0, kDeviceErrIndex);
                        else if (ix.refs[last] > 1) p.cow_src = last;
                    }
                    need = max(0, p.want - p.have) + (p.cow_src >= 0 ? 1 : 0);
                } else {
                    atomicCAS(ix.err_word, 0, kDeviceErrIndex);
                }
            }
        }
        int64_t sum;
        const int64_t first = total + block_prefix(need, warp_sums, &sum);
        total += sum;
        p.first = static_cast<int>(min(first, static_cast<int64_t>(0x7fffffff)));
        if (i < a.n) a.plan[i] = p;
    }
    // the lowest free pages, as many as are wanted
    const int goal = static_cast<int>(min(total, static_cast<int64_t>(ix.num_pages)));
    int found = 0;
    if (goal > 0) {
        const int share = ((ix.num_pages + kPlanWarps - 1) / kPlanWarps + 127) / 128 * 128;
        const int lo = min(ix.num_pages, warp * share), hi = min(ix.num_pages, lo + share);
        int mine = 0;
        for (int j0 = lo; j0 < hi; j0 += 128) {
            int z = 0;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int j = j0 + k * 32 + lane;
                z += (j < hi && ix.refs[j] == 0) ? 1 : 0;
            }
            mine += z;
        }
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) mine += __shfl_xor_sync(0xffffffffu, mine, d);
        if (lane == 0) warp_free[warp] = mine;
        __syncthreads();
        int at = 0;
        for (int w = 0; w < kPlanWarps; ++w) {
            if (w < warp) at += warp_free[w];
            found += warp_free[w];
        }
        for (int j0 = lo; j0 < hi && at < goal; j0 += 128) {
            bool z[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int j = j0 + k * 32 + lane;
                z[k] = j < hi && ix.refs[j] == 0;
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const unsigned m = __ballot_sync(0xffffffffu, z[k]);
                const int to = at + __popc(m & ((1u << lane) - 1u));
                if (z[k] && to < goal) a.list[to] = j0 + k * 32 + lane;
                at += __popc(m);
            }
        }
    }
    __syncthreads();
    // rows whose pages were found change, in the order of the call; the others stay as they are (all of the
    // request has been read: new_lens may be seq_lens, or a part of it)
    for (int i = tid; i < a.n; i += kPlanThreads) {
        RowPlan p = a.plan[i];
        int st = 2;
        if (p.row >= 0) {
            const int need = max(0, p.want - p.have) + (p.cow_src >= 0 ? 1 : 0);
            if (need == 0 || static_cast<int64_t>(p.first) + need <= found) {
                st = 0;
                ix.lens[p.row] = p.len;
                if (p.cow_src >= 0) a.pairs[atomicAdd(&pair_count, 1)] = make_int2(p.cow_src, a.list[p.first]);
            } else {
                st = 1;
                a.plan[i].row = -1;
            }
        }
        a.status[i] = st;
    }
    __syncthreads();
    if (tid == 0) {
        a.head[0] = pair_count;
        *a.taken = 0;
    }
}

__device__ __forceinline__ void release_page(const IndexArgs &ix, int id) {
    if (id < 0 || id >= ix.num_pages) {
        atomicCAS(ix.err_word, 0, kDeviceErrIndex);
        return;
    }
    if (atomicSub(&ix.refs[id], 1) <= 0) {  // held by nobody: the caller's arrays do not belong together
        atomicAdd(&ix.refs[id], 1);
        atomicCAS(ix.err_word, 0, kDeviceErrIndex);
    }
}

__global__ void __launch_bounds__(kPagesThreads) hsp_resize_apply_kernel(const __grid_constant__ ResizeArgs a) {
    const IndexArgs &ix = a.ix;
    griddep_wait();
    for (int i = blockIdx.x; i < a.n; i += gridDim.x) {
        const RowPlan p = a.plan[i];
        if (p.row < 0) continue;
        int32_t *t = ix.table + p.row * ix.table_stride;
        const int cow = p.cow_src >= 0 ? 1 : 0;
        for (int j = p.have + threadIdx.x; j < p.want; j += kPagesThreads) {
            const int id = a.list[p.first + cow + j - p.have];
            t[j] = id;
            ix.refs[id] = 1;
        }
        for (int j = p.want + threadIdx.x; j < p.have; j += kPagesThreads) {
            release_page(ix, t[j]);
            t[j] = -1;
        }
        if (cow && threadIdx.x == 0) {
            const int id = a.list[p.first];
            t[p.have - 1] = id;
            ix.refs[id] = 1;
            release_page(ix, p.cow_src);
        }
    }
    const int64_t units = static_cast<int64_t>(a.head[0]) * a.pools.pieces_total;
    copy_in_order(a.pools, units, a.taken, [&](int64_t k) { return a.pairs[k]; });
    cta_release_and_trigger();
}

// A table of the rows named in a request, in shared memory: the first place that names a row.
struct RowsNamed {
    static constexpr int kPlaces = 2 * kTeamRows;  // at most half of them are taken
    int row[kPlaces], first[kPlaces];
    __device__ __forceinline__ void clear() {
        for (int h = threadIdx.x; h < kPlaces; h += kPlanThreads) {
            row[h] = -1;
            first[h] = 0x7fffffff;
        }
    }
    __device__ __forceinline__ int enter(int r, int i) {
        int h = static_cast<int>((static_cast<uint32_t>(r) * 2654435761u) >> 20) & (kPlaces - 1);
        for (;;) {
            const int was = atomicCAS(&row[h], -1, r);
            if (was == -1 || was == r) break;
            h = (h + 1) & (kPlaces - 1);
        }
        atomicMin(&first[h], i);
        return h;
    }
};

// One launch for a small call: every CTA of the cluster reads the same arrays and makes the same plan in its
// own shared memory, and when all have read (the cluster's barrier), each applies its share.  The plan
// follows the rules of hsp_resize_plan_kernel: a thread per row, a warp per 128 pages.  Beam step of 8
// children (two resizes and a fork, 0.3 MB to copy): 17.5 us on the GPU with two launches for either resize, 15.2 so,
// and two launches less for the host, which bounds such calls.
__global__ void __launch_bounds__(kPlanThreads) hsp_resize_team_kernel(const __grid_constant__ ResizeArgs a) {
    __shared__ int64_t warp_sums[kPlanWarps];
    __shared__ int warp_free[kPlanWarps], warp_cow[kPlanWarps];
    __shared__ RowsNamed named;
    __shared__ int list[kTeamPages];
    __shared__ int2 pairs[kTeamRows];
    __shared__ RowPlan plan[kTeamRows];
    static_assert(kTeamPages <= kPlanWarps * 128 && kTeamRows <= kTeam * kPlanWarps && kTeamRows <= kPlanThreads, "one pass");
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, rank = blockIdx.x;
    const IndexArgs &ix = a.ix;
    const int64_t most = static_cast<int64_t>(ix.max_pages) << ix.page_shift;
    named.clear();
    __syncthreads();
    griddep_wait();
    int r = -1, want = 0;
    if (tid < a.n) {
        r = a.rows[tid];
        want = a.new_lens[tid];
    }
    bool z[4];
    int mine = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const int j = warp * 128 + k * 32 + lane;
        z[k] = j < ix.num_pages && ix.refs[j] == 0;
        mine += z[k] ? 1 : 0;
    }
    const bool in = r >= 0 && r < ix.num_rows;
    const int old = in ? ix.lens[r] : 0;
    int h = 0;
    if (in) h = named.enter(r, tid);
    else if (tid < a.n) atomicCAS(ix.err_word, 0, kDeviceErrIndex);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) mine += __shfl_xor_sync(0xffffffffu, mine, d);
    if (lane == 0) warp_free[warp] = mine;
    __syncthreads();
    RowPlan p;
    p.row = p.cow_src = -1;
    p.len = p.have = p.want = p.first = 0;
    int need = 0;
    if (in && named.first[h] == tid && want >= 0 && want <= most) {
        if (old >= 0 && old <= most) {
            p.row = r;
            p.have = pages_of(old, ix.page_shift);
            p.want = pages_of(want, ix.page_shift);
            if (want > old && (old & ((1 << ix.page_shift) - 1)) != 0) {
                const int last = ix.table[r * ix.table_stride + p.have - 1];
                if (last < 0 || last >= ix.num_pages) atomicCAS(ix.err_word, 0, kDeviceErrIndex);
                else if (ix.refs[last] > 1) p.cow_src = last;
            }
            need = max(0, p.want - p.have) + (p.cow_src >= 0 ? 1 : 0);
        } else {
            atomicCAS(ix.err_word, 0, kDeviceErrIndex);
        }
    }
    int64_t total;
    const int64_t first = block_prefix(need, warp_sums, &total);
    int at = 0, found = 0;
    for (int w = 0; w < kPlanWarps; ++w) {
        if (w < warp) at += warp_free[w];
        found += warp_free[w];
    }
    // the free pages, lowest first
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const unsigned m = __ballot_sync(0xffffffffu, z[k]);
        if (z[k]) list[at + __popc(m & ((1u << lane) - 1u))] = warp * 128 + k * 32 + lane;
        at += __popc(m);
    }
    const bool good = p.row >= 0 && (need == 0 || first + need <= found);
    const int status = good ? 0 : p.row >= 0 ? 1 : 2;
    p.first = good ? static_cast<int>(first) : 0;
    const bool cow = good && p.cow_src >= 0;
    const unsigned cows = __ballot_sync(0xffffffffu, cow);
    if (lane == 0) warp_cow[warp] = __popc(cows);
    __syncthreads();
    int pair_at = 0, pair_count = 0;
    for (int w = 0; w < kTeamRows / 32; ++w) {
        if (w < warp) pair_at += warp_cow[w];
        pair_count += warp_cow[w];
    }
    if (cow) pairs[pair_at + __popc(cows & ((1u << lane) - 1u))] = make_int2(p.cow_src, list[p.first]);
    if (tid < a.n) {
        if (!good) p.row = -1;
        plan[tid] = p;
    }
    cluster_sync_all();  // every CTA has read what the others change (and this one's plan is written)
    if (tid < a.n && tid % kTeam == rank) {
        if (good) ix.lens[r] = want;
        a.status[tid] = status;
    }
    const int i = rank + kTeam * warp;
    if (i < a.n && plan[i].row >= 0) {
        const RowPlan q = plan[i];
        int32_t *t = ix.table + q.row * ix.table_stride;
        const int shared = q.cow_src >= 0 ? 1 : 0;
        for (int j = q.have + lane; j < q.want; j += 32) {
            const int id = list[q.first + shared + j - q.have];
            t[j] = id;
            ix.refs[id] = 1;
        }
        for (int j = q.want + lane; j < q.have; j += 32) {
            release_page(ix, t[j]);
            t[j] = -1;
        }
        if (shared && lane == 0) {
            const int id = list[q.first];
            t[q.have - 1] = id;
            ix.refs[id] = 1;
            release_page(ix, q.cow_src);
        }
    }
    copy_by_team(a.pools, pair_count, rank, [&](uint32_t k) { return pairs[k]; });
    cta_release_and_trigger();
}

// ---- fork -----------------------------------------------------------------------------

__global__ void __launch_bounds__(kPagesThreads) hsp_fork_kernel(const __grid_constant__ ForkArgs a) {
    __shared__ int refuse;
    const IndexArgs &ix = a.ix;
    const int i = blockIdx.x;
    if (threadIdx.x == 0) refuse = 0;
    griddep_wait();
    __syncthreads();
    const int p = a.parents[i], c = a.children[i];
    const bool in = p >= 0 && p < ix.num_rows && c >= 0 && c < ix.num_rows;
    // a child named before, or a parent that is a child of this call: refused, whoever runs first
    bool bad = false;
    for (int j = threadIdx.x; j < a.n; j += kPagesThreads) {
        const int o = a.children[j];
        bad = bad || o == p || (j < i && o == c);
    }
    if (bad) refuse = 1;
    __syncthreads();
    int st = 0;
    int len = 0;
    if (!in) {
        st = 2;
        if (threadIdx.x == 0) atomicCAS(ix.err_word, 0, kDeviceErrIndex);
    } else if (refuse) {
        st = 2;
    } else {
        len = ix.lens[p];
        const int64_t most = static_cast<int64_t>(ix.max_pages) << ix.page_shift;
        if (ix.lens[c] != 0 || len < 0 || len > most) st = 2;
    }
    __syncthreads();  // every thread has seen the child's length
    if (st == 0) {
        const int pages = pages_of(len, ix.page_shift);
        const int32_t *from = ix.table + p * ix.table_stride;
        int32_t *to = ix.table + c * ix.table_stride;
        for (int j = threadIdx.x; j < pages; j += kPagesThreads) {
            const int id = from[j];
            to[j] = id;
            if (id >= 0 && id < ix.num_pages) atomicAdd(&ix.refs[id], 1);
            else atomicCAS(ix.err_word, 0, kDeviceErrIndex);
        }
        if (threadIdx.x == 0) ix.lens[c] = len;
    }
    if (threadIdx.x == 0) a.status[i] = st;
    cta_release_and_trigger();
}

// ---- compact --------------------------------------------------------------------------

__global__ void __launch_bounds__(kPlanThreads) hsp_compact_plan_kernel(const __grid_constant__ CompactArgs a) {
    __shared__ int warp_live[kPlanWarps], warp_holes[kPlanWarps], warp_tails[kPlanWarps];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const IndexArgs &ix = a.ix;
    const int N = ix.num_pages;
    griddep_launch_dependents();  // (the apply kernel, which waits for this one's end)
    griddep_wait();
    const int share = ((N + kPlanWarps - 1) / kPlanWarps + 127) / 128 * 128;
    const int lo = min(N, warp * share), hi = min(N, lo + share);
    int live = 0;
    for (int j0 = lo; j0 < hi; j0 += 128) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int j = j0 + k * 32 + lane;
            live += (j < hi && ix.refs[j] > 0) ? 1 : 0;
        }
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) live += __shfl_xor_sync(0xffffffffu, live, d);
    if (lane == 0) warp_live[warp] = live;
    __syncthreads();
    int L = 0;
    for (int w = 0; w < kPlanWarps; ++w) L += warp_live[w];
    // free pages before L, and live pages at or past L, in this warp's share (read again, now that L is known)
    int holes = 0, tails = 0;
    for (int j0 = lo; j0 < hi; j0 += 128) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int j = j0 + k * 32 + lane;
            const bool in = j < hi, alive = in && ix.refs[j] > 0;
            holes += (in && !alive && j < L) ? 1 : 0;
            tails += (alive && j >= L) ? 1 : 0;
        }
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) {
        holes += __shfl_xor_sync(0xffffffffu, holes, d);
        tails += __shfl_xor_sync(0xffffffffu, tails, d);
    }
    if (lane == 0) {
        warp_holes[warp] = holes;
        warp_tails[warp] = tails;
    }
    __syncthreads();
    int hole_at = 0, tail_at = 0, moves = 0;
    for (int w = 0; w < kPlanWarps; ++w) {
        if (w < warp) {
            hole_at += warp_holes[w];
            tail_at += warp_tails[w];
        }
        moves += warp_tails[w];
    }
    for (int j0 = lo; j0 < hi; j0 += 128) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int j = j0 + k * 32 + lane;
            const bool in = j < hi, alive = in && ix.refs[j] > 0;
            const bool hole = in && !alive && j < L, tail = alive && j >= L;
            const unsigned mh = __ballot_sync(0xffffffffu, hole), mt = __ballot_sync(0xffffffffu, tail);
            const unsigned low = (1u << lane) - 1u;
            if (hole) a.pairs[hole_at + __popc(mh & low)].y = j;
            if (tail) a.pairs[tail_at + __popc(mt & low)].x = j;
            if (in && j >= L && !alive) a.list[j] = -1;
            hole_at += __popc(mh);
            tail_at += __popc(mt);
        }
    }
    __syncthreads();
    // where each moved page goes (holes and tails are equally many)
    for (int k = tid; k < moves; k += kPlanThreads) {
        const int2 p = a.pairs[k];
        a.list[p.x] = p.y;
    }
    if (tid == 0) {
        a.head[0] = moves;
        a.head[1] = L;
        *a.taken = 0;
        a.live[0] = L;
    }
}

__global__ void __launch_bounds__(kPagesThreads) hsp_compact_apply_kernel(const __grid_constant__ CompactArgs a) {
    const IndexArgs &ix = a.ix;
    griddep_wait();
    const int moves = a.head[0], L = a.head[1];
    if (moves > 0) {
        const int64_t most = static_cast<int64_t>(ix.max_pages) << ix.page_shift;
        for (int r = blockIdx.x; r < ix.num_rows; r += gridDim.x) {
            int len = ix.lens[r];
            if (len < 0 || len > most) {
                if (threadIdx.x == 0) atomicCAS(ix.err_word, 0, kDeviceErrIndex);
                len = len < 0 ? 0 : static_cast<int>(most);
            }
            const int pages = pages_of(len, ix.page_shift);
            int32_t *t = ix.table + r * ix.table_stride;
            for (int j = threadIdx.x; j < pages; j += kPagesThreads) {
                const int id = t[j];
                const int to = id >= L && id < ix.num_pages ? a.list[id] : id;
                if (id < 0 || id >= ix.num_pages || to < 0) atomicCAS(ix.err_word, 0, kDeviceErrIndex);
                else if (to != id) t[j] = to;
            }
        }
        for (int k = blockIdx.x * kPagesThreads + threadIdx.x; k < moves; k += gridDim.x * kPagesThreads) {
            const int2 p = a.pairs[k];
            ix.refs[p.y] = ix.refs[p.x];
            ix.refs[p.x] = 0;
        }
        const int64_t units = static_cast<int64_t>(moves) * a.pools.pieces_total;
        copy_in_order(a.pools, units, a.taken, [&](int64_t k) { return a.pairs[k]; });
    }
    cta_release_and_trigger();
}

// ---- launches -------------------------------------------------------------------------

template <typename Args>
cudaError_t launch_one(void (*kern)(Args), const Args &a, int64_t ctas, int threads, int pdl, cudaStream_t stream,
                       int cluster = 1) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(ctas < 1 ? 1 : ctas), 1, 1);
    cfg.blockDim = dim3(static_cast<unsigned>(threads), 1, 1);
    cfg.stream = stream;
    cudaLaunchAttribute attrs[2];
    unsigned n = 0;
    if (pdl) {
        attrs[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attrs[n].val.programmaticStreamSerializationAllowed = 1;
        ++n;
    }
    if (cluster > 1) {
        attrs[n].id = cudaLaunchAttributeClusterDimension;
        attrs[n].val.clusterDim.x = static_cast<unsigned>(cluster);
        attrs[n].val.clusterDim.y = attrs[n].val.clusterDim.z = 1;
        ++n;
    }
    cfg.attrs = attrs;
    cfg.numAttrs = n;
    return cudaLaunchKernelEx(&cfg, kern, a);
}

template <int PAIRS>
cudaError_t launch_copy(const PoolList &pools, const int32_t *src, const int32_t *dst, int n, int pdl, cudaStream_t stream) {
    CopyArgs<PAIRS> a;
    a.pools = pools;
    a.n = n;
    for (int i = 0; i < n; ++i) {
        a.src[i] = src[i];
        a.dst[i] = dst[i];
    }
    int64_t ctas = static_cast<int64_t>(n) * pools.pieces_total;  // one each: they start in order
    if (ctas > 0x7fffffff) ctas = 0x7fffffff;
    return launch_one(hsp_copy_pages_kernel<PAIRS>, a, ctas, kPagesThreads, pdl, stream);
}

}  // namespace

cudaError_t launch_copy_pages(const PoolList &pools, const int32_t *src, const int32_t *dst, int n, int pdl, cudaStream_t stream) {
    if (n <= 64) return launch_copy<64>(pools, src, dst, n, pdl, stream);
    return launch_copy<kMaxCopyPairs>(pools, src, dst, n, pdl, stream);
}

cudaError_t launch_resize(const ResizeArgs &a, int sms, int pdl, cudaStream_t stream) {
    if (team_resize(a)) return launch_one(hsp_resize_team_kernel, a, kTeam, kPlanThreads, pdl, stream, kTeam);
    cudaError_t e = launch_one(hsp_resize_plan_kernel, a, 1, kPlanThreads, pdl, stream);
    if (e != cudaSuccess) return e;
    // one CTA per row while rows are few, and as many as the copies of their last pages can use
    int64_t ctas = static_cast<int64_t>(a.n) * (a.pools.pieces_total > 1 ? a.pools.pieces_total : 1);
    if (ctas > sms * 8) ctas = sms * 8;
    return launch_one(hsp_resize_apply_kernel, a, ctas, kPagesThreads, pdl, stream);
}

cudaError_t launch_fork(const ForkArgs &a, int pdl, cudaStream_t stream) {
    return launch_one(hsp_fork_kernel, a, a.n, kPagesThreads, pdl, stream);
}

cudaError_t launch_compact(const CompactArgs &a, int sms, int pdl, cudaStream_t stream) {
    cudaError_t e = launch_one(hsp_compact_plan_kernel, a, 1, kPlanThreads, pdl, stream);
    if (e != cudaSuccess) return e;
    return launch_one(hsp_compact_apply_kernel, a, sms * 8, kPagesThreads, pdl, stream);
}

}  // namespace hsp
