// Page bookkeeping of the paged 4-bit key/value cache: lengths, shared and
// copied sequences, compaction.  The state is the caller's: reference counts
// per page, tables and lengths per sequence; a page is free when its count is
// 0, so the state has one form and every call's result depends on it alone.
//
// A planning kernel (one CTA) decides and writes the tables; pages that have
// to be copied go on a list that a second kernel, over the whole GPU, works
// off.  The plan is bound by latency (a chain of a few dependent loads, and
// one pass over the counts when pages are taken), the copies by HBM traffic.
#include <cuda_runtime.h>

#include "kv4.cuh"

namespace sparstar {
namespace {

constexpr int kPlanThreads = 1024;
constexpr int kWarps = kPlanThreads / 32;

// Scratch (int32): a head, three lists of n_pages, three of n_seqs.
struct Work {
    int32_t *pairs;  // [0] pages to copy, [1] live pages (compact)
    int32_t *to, *from, *moved;
    int32_t *owner, *begin, *rank;
};
constexpr int kHead = 16;
__host__ __device__ inline Work work_of(const Kv4 &c) {
    Work w;
    w.pairs = c.work;
    w.to = c.work + kHead;
    w.from = w.to + c.n_pages;
    w.moved = w.from + c.n_pages;
    w.owner = w.moved + c.n_pages;
    w.begin = w.owner + c.n_seqs;
    w.rank = w.begin + c.n_seqs;
    return w;
}

// Exclusive prefix sum over the CTA; `total` gets the sum.
template <typename N>
__device__ N block_scan(N x, N *sums, N &total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    N y = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const N z = __shfl_up_sync(0xffffffffu, y, o);
        if (lane >= o) y += z;
    }
    __syncthreads();  // sums may still be read by an earlier scan
    if (lane == 31) sums[warp] = y;
    __syncthreads();
    if (warp == 0) {
        N v = sums[lane];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const N z = __shfl_up_sync(0xffffffffu, v, o);
            if (lane >= o) v += z;
        }
        sums[lane] = v;
    }
    __syncthreads();
    total = sums[kWarps - 1];
    return (warp ? sums[warp - 1] : 0) + y - x;
}

// The lowest `want` free pages into list (all, when there are fewer);
// returns how many.
__device__ int find_free(const Kv4 &c, int want, int32_t *list, int32_t *sums) {
    int found = 0;
    for (int base = 0; base < c.n_pages && found < want; base += 4 * kPlanThreads) {
        const int p = base + 4 * threadIdx.x;
        int4 r = make_int4(1, 1, 1, 1);
        if (p + 3 < c.n_pages) {
            r = *reinterpret_cast<const int4 *>(c.refs + p);
        } else {
            if (p < c.n_pages) r.x = c.refs[p];
            if (p + 1 < c.n_pages) r.y = c.refs[p + 1];
            if (p + 2 < c.n_pages) r.z = c.refs[p + 2];
        }
        const int mine = (r.x == 0) + (r.y == 0) + (r.z == 0) + (r.w == 0);
        int total;
        int at = found + block_scan(mine, sums, total);
        if (r.x == 0 && at < want) list[at] = p;
        at += r.x == 0;
        if (r.y == 0 && at < want) list[at] = p + 1;
        at += r.y == 0;
        if (r.z == 0 && at < want) list[at] = p + 2;
        at += r.z == 0;
        if (r.w == 0 && at < want) list[at] = p + 3;
        found += total;
    }
    return found < want ? found : want;
}

// True when no earlier entry names the slot (owner[slot] = the lowest one).
__device__ void mark_owners(const Kv4 &c, const Work &w, const int32_t *slots, int n) {
    for (int i = threadIdx.x; i < n; i += kPlanThreads) {
        const int s = kv4_slot(c, slots, i);
        if (s >= 0) w.owner[s] = 0x7fffffff;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += kPlanThreads) {
        const int s = kv4_slot(c, slots, i);
        if (s >= 0) atomicMin(w.owner + s, i);
    }
    __syncthreads();
}

// What entry i of a resize (src NULL) or deep fork asks for.
struct Ask {
    int slot, from_slot, old_len, new_len;
    bool ok;
};
__device__ Ask ask_of(const Kv4 &c, const Work &w, const int32_t *slots, const int32_t *src,
                      const int32_t *lens, int i) {
    Ask a;
    a.slot = kv4_slot(c, slots, i);
    a.from_slot = -1;
    a.old_len = a.new_len = 0;
    a.ok = a.slot >= 0 && (!slots || __ldcg(w.owner + a.slot) == i);
    if (!a.ok) return a;
    a.old_len = kv4_len(c, a.slot);
    if (src) {
        a.from_slot = kv4_slot(c, src, i);
        a.ok = a.from_slot >= 0 && a.old_len == 0;
        const int have = a.ok ? kv4_len(c, a.from_slot) : 0;
        a.new_len = lens ? __ldg(lens + i) : have;
        a.ok = a.ok && a.new_len >= 0 && a.new_len <= have;
    } else {
        a.new_len = __ldg(lens + i);
        a.ok = a.new_len >= 0 && a.new_len <= (int64_t)c.max_pages * kBlock;
    }
    return a;
}

__device__ __forceinline__ int pages_of(int len) { return (len + kBlock - 1) / kBlock; }
__device__ __forceinline__ bool is_page(const Kv4 &c, int p) { return p >= 0 && p < c.n_pages; }

// A fork entry whose source is one of the call's destinations is left out
// (fork_shared_kernel, whose CTAs run at the same time, needs that rule).
__device__ bool is_dst(const int32_t *dst, int n, int slot) {
    for (int i = 0; i < n; ++i)
        if (__ldg(dst + i) == slot) return true;
    return false;
}

// resize (src NULL: slots, lens) and deep fork (src, slots = dst, lens).
__global__ void __launch_bounds__(kPlanThreads)
    plan_kernel(Kv4 c, const int32_t *slots, const int32_t *src, const int32_t *lens, int n,
                int32_t *status) {
    __shared__ int64_t needs[kWarps];
    __shared__ int32_t sums[kWarps], n_pairs;
    const Work w = work_of(c);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (threadIdx.x == 0) n_pairs = 0;
    if (slots) mark_owners(c, w, slots, n);
    // Pass 1: what each entry needs (negative begin: nothing to take), its
    // first rank among the pages taken.  Reads the counts before any change.
    int64_t wanted = 0;
    for (int base = 0; base < n; base += kPlanThreads) {
        const int i = base + threadIdx.x;
        int64_t need = 0;
        int begin = -1;
        if (i < n) {
            Ask a = ask_of(c, w, slots, src, lens, i);
            if (a.ok && src && is_dst(slots, n, a.from_slot)) a.ok = false;
            if (!a.ok) {
                kv4_flag(status, SPARSTAR_STATUS_BAD_INDEX);
                begin = -2;
            } else if (a.new_len > a.old_len) {
                begin = pages_of(a.old_len);
                if (a.old_len % kBlock) {
                    const int tail = c.table[(int64_t)a.slot * c.max_pages + begin - 1];
                    if (is_page(c, tail) && c.refs[tail] > 1) --begin;
                }
                need = pages_of(a.new_len) - begin;
            }
        }
        int64_t total;
        const int64_t rank = wanted + block_scan(need, needs, total);
        if (i < n) {
            w.begin[i] = begin;
            w.rank[i] = rank <= c.n_pages ? (int)rank : c.n_pages + 1;
        }
        wanted += total;
    }
    // Free pages, lowest first; copies use the same list as their targets.
    const int limit = wanted < c.n_pages ? (int)wanted : c.n_pages;
    const int found = limit > 0 ? find_free(c, limit, w.moved, sums) : 0;
    __syncthreads();
    // Pass 2: one warp an entry.
    for (int i = warp; i < n; i += kWarps) {
        const int begin = __ldcg(w.begin + i), rank = __ldcg(w.rank + i);
        if (begin == -2) continue;
        const Ask a = ask_of(c, w, slots, src, lens, i);
        int32_t *row = c.table + (int64_t)a.slot * c.max_pages;
        const int had = pages_of(a.old_len), have = pages_of(a.new_len);
        if (begin >= 0) {
            const int need = have - begin;
            if (need > 0 && (rank > found || need > found - rank)) {
                if (lane == 0) kv4_flag(status, SPARSTAR_STATUS_NO_PAGES);
                continue;
            }
            const int32_t *from =
                src ? c.table + (int64_t)a.from_slot * c.max_pages : nullptr;
            for (int j = lane; j < need; j += 32) {
                const int page = __ldcg(w.moved + rank + j);
                int copy_of = -1;
                if (from) {
                    copy_of = from[begin + j];
                } else if (begin + j < had) {  // the shared partial page
                    copy_of = row[begin + j];
                    if (is_page(c, copy_of)) atomicSub(c.refs + copy_of, 1);
                }
                row[begin + j] = page;
                c.refs[page] = 1;
                if (is_page(c, copy_of)) {
                    const int p = atomicAdd(&n_pairs, 1);
                    w.to[p] = page;
                    w.from[p] = copy_of;
                }
            }
        } else {
            for (int j = have + lane; j < had; j += 32) {
                const int page = row[j];
                if (is_page(c, page)) atomicSub(c.refs + page, 1);
                row[j] = -1;
            }
        }
        if (lane == 0) c.lens[a.slot] = a.new_len;
    }
    __syncthreads();
    if (threadIdx.x == 0) w.pairs[0] = n_pairs;
}

// Shared fork: one CTA an entry.  No entry reads what another writes: a
// source is no destination, a destination belongs to the lowest entry.
__global__ void __launch_bounds__(256)
    fork_shared_kernel(Kv4 c, const int32_t *src, const int32_t *dst, const int32_t *len, int n,
                       int32_t *status) {
    const int i = blockIdx.x;
    const int s = kv4_slot(c, src, i), d = kv4_slot(c, dst, i);
    bool bad = s < 0 || d < 0;
    int refuse = 0;
    for (int k = threadIdx.x; k < n; k += blockDim.x) {
        const int other = __ldg(dst + k);
        refuse |= other == s || (k < i && other == d);
    }
    bad |= __syncthreads_or(refuse) != 0;
    int L = 0;
    if (!bad) {
        const int have = kv4_len(c, s);
        L = len ? __ldg(len + i) : have;
        bad = L < 0 || L > have || kv4_len(c, d) != 0;
    }
    __syncthreads();  // every thread has read lens[d]
    if (bad) {
        if (threadIdx.x == 0) kv4_flag(status, SPARSTAR_STATUS_BAD_INDEX);
        return;
    }
    const int32_t *from = c.table + (int64_t)s * c.max_pages;
    int32_t *to = c.table + (int64_t)d * c.max_pages;
    for (int j = threadIdx.x; j < pages_of(L); j += blockDim.x) {
        const int page = from[j];
        to[j] = page;
        if (is_page(c, page)) atomicAdd(c.refs + page, 1);
    }
    if (threadIdx.x == 0) c.lens[d] = L;
}

// Which pages move where, the counts after it.
__global__ void __launch_bounds__(kPlanThreads) compact_plan_kernel(Kv4 c, int32_t *n_live) {
    __shared__ int32_t sums[kWarps];
    const Work w = work_of(c);
    int live = 0, total;
    for (int p = threadIdx.x; p < c.n_pages; p += kPlanThreads) live += c.refs[p] > 0;
    block_scan(live, sums, total);
    live = total;
    int holes = 0, movers = 0;
    for (int base = 0; base < c.n_pages; base += kPlanThreads) {
        const int p = base + threadIdx.x;
        const bool is_live = p < c.n_pages && c.refs[p] > 0;
        const bool hole = p < live && !is_live, mover = p >= live && is_live;
        int n_hole, n_mover;
        const int h = holes + block_scan((int)hole, sums, n_hole);
        const int m = movers + block_scan((int)mover, sums, n_mover);
        if (hole) w.to[h] = p;
        if (mover) w.from[m] = p;
        holes += n_hole;
        movers += n_mover;
    }
    __syncthreads();
    for (int k = threadIdx.x; k < movers; k += kPlanThreads) {  // holes == movers
        const int from = __ldcg(w.from + k), to = __ldcg(w.to + k);
        w.moved[from] = to;
        c.refs[to] = c.refs[from];
        c.refs[from] = 0;
    }
    if (threadIdx.x == 0) {
        w.pairs[0] = movers;
        w.pairs[1] = live;
        *n_live = live;
    }
}

// Copies the listed pages; with `remap`, also renames the moved ones in the
// tables.
__global__ void __launch_bounds__(256) copy_kernel(Kv4 c, bool remap) {
    const Work w = work_of(c);
    const int pairs = w.pairs[0];
    if (pairs == 0) return;
    const int64_t bytes = (int64_t)c.Hkv * kv4_page_bytes(c.D), vecs = bytes / 16;
    const int64_t all = vecs * pairs;
    for (int64_t v = blockIdx.x * (int64_t)blockDim.x + threadIdx.x; v < all;
         v += (int64_t)gridDim.x * blockDim.x) {
        const int64_t k = v / vecs, at = v % vecs;
        reinterpret_cast<uint4 *>(c.pages + w.to[k] * bytes)[at] =
            reinterpret_cast<const uint4 *>(c.pages + w.from[k] * bytes)[at];
    }
    if (!remap) return;
    const int live = w.pairs[1];
    const int64_t entries = (int64_t)c.n_seqs * c.max_pages;
    for (int64_t e = blockIdx.x * (int64_t)blockDim.x + threadIdx.x; e < entries;
         e += (int64_t)gridDim.x * blockDim.x) {
        const int slot = (int)(e / c.max_pages), j = (int)(e % c.max_pages);
        if (j >= pages_of(kv4_len(c, slot))) continue;
        const int page = c.table[e];
        if (page >= live && page < c.n_pages) c.table[e] = w.moved[page];
    }
}

constexpr int kCopyCtas = 148 * 8;

}  // namespace

int64_t kv4_work_ints(int64_t n_pages, int64_t n_seqs) {
    return kHead + 3 * n_pages + 3 * n_seqs;
}

cudaError_t launch_kv4_resize(const Kv4 &c, const int32_t *seqs, const int32_t *new_lens, int n,
                              int32_t *status, cudaStream_t stream) {
    plan_kernel<<<1, kPlanThreads, 0, stream>>>(c, seqs, nullptr, new_lens, n, status);
    copy_kernel<<<kCopyCtas, 256, 0, stream>>>(c, false);
    return cudaGetLastError();
}

cudaError_t launch_kv4_fork(const Kv4 &c, const int32_t *src, const int32_t *dst,
                            const int32_t *len, int n, bool deep, int32_t *status,
                            cudaStream_t stream) {
    if (deep) {
        plan_kernel<<<1, kPlanThreads, 0, stream>>>(c, dst, src, len, n, status);
        copy_kernel<<<kCopyCtas, 256, 0, stream>>>(c, false);
    } else {
        fork_shared_kernel<<<n, 256, 0, stream>>>(c, src, dst, len, n, status);
    }
    return cudaGetLastError();
}

cudaError_t launch_kv4_compact(const Kv4 &c, int32_t *n_live, cudaStream_t stream) {
    compact_plan_kernel<<<1, kPlanThreads, 0, stream>>>(c, n_live);
    copy_kernel<<<kCopyCtas, 256, 0, stream>>>(c, true);
    return cudaGetLastError();
}

}  // namespace sparstar
