// Page bookkeeping of the paged 4-bit key/value cache: lengths, shared and
// copied sequences, compaction.  The state is the caller's: reference counts
// per page, tables and lengths per sequence; a page is free when its count is
// 0, so the state has one form and every call's result depends on it alone.
//
// One CTA decides and writes the tables; pages that have to be copied go on
// a list that a second kernel, over the whole GPU, works off: plain loads and
// stores for the few pages of a resize (at most one a sequence), bulk copies
// through shared memory for the many of a deep copy or a compaction.  The
// second kernel is set up while the first runs.  The plan is bound by latency
// (a chain of a few dependent loads, and one pass over the counts when pages
// are taken): two resizes and a fork of eight sequences, five launches, take
// 13.8 us.  The copies are bound by HBM traffic: a deep copy of two sequences
// of 41,012 tokens and a compaction that moves one, 536 MB, take 97 us, 5.5 TB/s.
// A cluster of eight that plans and copies in one launch was slower (the two
// resizes and the fork 19.5 us against 15.9 then).
#include <cuda_runtime.h>

#include "kv4.cuh"

namespace sparstar {
namespace {

constexpr int kPlanThreads = 1024;
constexpr int kWarps = kPlanThreads / 32;

// An entry of a resize or deep fork.
struct Entry {
    int32_t slot, from;  // slot changed, slot copied (-1: none)
    int32_t begin;       // first page taken; kNothing, kRefused
    int32_t rank;        // of it among the pages that the call takes
    int32_t old_len, new_len;
};
constexpr int kNothing = -1, kRefused = -2;

// Scratch (int32): a head, three lists of n_pages, n_seqs entries and owners.
struct Work {
    int32_t *pairs;  // [0] pages to copy, [1] live pages (compact)
    int32_t *to, *from, *moved;
    int32_t *owner;
    Entry *entries;
};
constexpr int kHead = 16;
constexpr int kInside = 512;  // entries that fit shared memory
__host__ __device__ inline Work work_of(const Kv4 &c) {
    Work w;
    w.pairs = c.work;
    w.to = c.work + kHead;
    w.from = w.to + c.n_pages;
    w.moved = w.from + c.n_pages;
    w.owner = w.moved + c.n_pages;
    w.entries = reinterpret_cast<Entry *>(w.owner + c.n_seqs);
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

__device__ __forceinline__ int pages_of(int len) { return (len + kBlock - 1) / kBlock; }
__device__ __forceinline__ bool is_page(const Kv4 &c, int p) { return p >= 0 && p < c.n_pages; }

// Copies the listed pages, a page of one head (17 or 9 KB) at a time: a warp
// has one stage of shared memory, brings the piece in with one bulk copy and
// sends it off with another.  The CTA's 12 or 24 stages (209 KB) are in flight
// at once, which a few hundred registers could not hold.  False in a warp whose
// copy did not arrive in two seconds (`withhold`: the test hook's, which brings
// none in); it waits as long again before it leaves, so that the copy does not
// outlive its stage.
constexpr int kStageBytes = 12 * kv4_page_bytes(128);
constexpr int kMaxStages = kStageBytes / kv4_page_bytes(64);
__device__ bool copy_pages(const Kv4 &c, const Work &w, int pairs, int cta, int ctas,
                           uint64_t *bars, uint8_t *smem, bool withhold) {
    const int bytes = kv4_page_bytes(c.D), stages = kStageBytes / bytes;
    const int warp = threadIdx.x >> 5;
    if (warp >= stages || (threadIdx.x & 31) != 0) return true;
    uint64_t *mbar = bars + warp;
    const uint32_t bar = (uint32_t)__cvta_generic_to_shared(mbar);
    const uint32_t stage = (uint32_t)__cvta_generic_to_shared(smem + warp * bytes);
    asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" ::"r"(bar) : "memory");
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    uint32_t phase = 0;
    const int64_t all = (int64_t)pairs * c.Hkv;
    for (int64_t it = (int64_t)cta * stages + warp; it < all; it += (int64_t)ctas * stages) {
        const int k = (int)(it / c.Hkv), h = (int)(it - (int64_t)k * c.Hkv);
        const int from = __ldcg(w.from + k), to = __ldcg(w.to + k);
        asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar),
                     "r"(bytes)
                     : "memory");
        if (!withhold)
            asm volatile(
                "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, "
                "[%3];" ::"r"(stage),
                "l"(c.pages + ((int64_t)from * c.Hkv + h) * bytes), "r"(bytes), "r"(bar)
                : "memory");
        if (!kv4_wait(bar, phase)) {
            kv4_wait(bar, phase);
            asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
            return false;
        }
        phase ^= 1u;
        asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(
                         c.pages + ((int64_t)to * c.Hkv + h) * bytes),
                     "r"(stage), "r"(bytes)
                     : "memory");
        asm volatile("cp.async.bulk.commit_group;" ::: "memory");
        asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
    }
    asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
    return true;
}

// resize (src NULL: slots, lens) and deep fork (src, slots = dst, lens).
__device__ void plan(const Kv4 &c, const int32_t *slots, const int32_t *src, const int32_t *lens,
                     int n, int32_t *status) {
    __shared__ int64_t needs[kWarps];
    __shared__ int32_t sums[kWarps], n_pairs;
    __shared__ Entry inside[kInside];
    const Work w = work_of(c);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    Entry *entries = n <= kInside ? inside : w.entries;
    if (threadIdx.x == 0) n_pairs = 0;
    for (int i = threadIdx.x; i < n; i += kPlanThreads) {
        entries[i].slot = kv4_slot(c, slots, i);
        entries[i].from = src ? kv4_slot(c, src, i) : -1;
    }
    __syncthreads();
    // A slot belongs to the lowest entry that names it: few entries compare
    // with the ones before, many mark their slots.
    const bool marks = slots && n > kInside;
    if (marks) {
        for (int i = threadIdx.x; i < n; i += kPlanThreads)
            if (entries[i].slot >= 0) w.owner[entries[i].slot] = 0x7fffffff;
        __syncthreads();
        for (int i = threadIdx.x; i < n; i += kPlanThreads)
            if (entries[i].slot >= 0) atomicMin(w.owner + entries[i].slot, i);
        __syncthreads();
    }
    // Pass 1: what each entry needs and its first rank among the pages taken.
    // Reads the counts before any change.
    int64_t wanted = 0;
    for (int base = 0; base < n; base += kPlanThreads) {
        const int i = base + threadIdx.x;
        int64_t need = 0;
        Entry e{-1, -1, kRefused, 0, 0, 0};
        if (i < n) {
            e.slot = entries[i].slot, e.from = entries[i].from;
            bool ok = e.slot >= 0;
            if (ok && marks) ok = __ldcg(w.owner + e.slot) == i;
            else if (ok && slots)
                for (int k = 0; k < i; ++k) ok &= entries[k].slot != e.slot;
            if (ok) {
                e.old_len = kv4_len(c, e.slot);
                if (src) {
                    // An entry whose source is a destination of the call is
                    // left out (fork_shared_kernel's CTAs need that rule).
                    ok = e.from >= 0 && e.old_len == 0;
                    for (int k = 0; k < n && ok; ++k) ok = entries[k].slot != e.from;
                    const int have = ok ? kv4_len(c, e.from) : 0;
                    e.new_len = lens ? __ldca(lens + i) : have;
                    ok = ok && e.new_len >= 0 && e.new_len <= have;
                } else {
                    e.new_len = __ldca(lens + i);
                    ok = e.new_len >= 0 && e.new_len <= (int64_t)c.max_pages * kBlock;
                }
            }
            if (!ok) {
                kv4_flag(status, SPARSTAR_STATUS_BAD_INDEX);
            } else if (e.new_len > e.old_len) {
                e.begin = pages_of(e.old_len);
                if (e.old_len % kBlock) {
                    const int tail = c.table[(int64_t)e.slot * c.max_pages + e.begin - 1];
                    if (is_page(c, tail) && c.refs[tail] > 1) --e.begin;
                }
                need = pages_of(e.new_len) - e.begin;
            } else {
                e.begin = kNothing;
            }
        }
        int64_t total;
        const int64_t rank = wanted + block_scan(need, needs, total);
        e.rank = rank <= c.n_pages ? (int)rank : c.n_pages + 1;
        // Slots and sources stay: other entries compare with them.
        if (i < n) {
            entries[i].begin = e.begin, entries[i].rank = e.rank;
            entries[i].old_len = e.old_len, entries[i].new_len = e.new_len;
        }
        wanted += total;
    }
    // Free pages, lowest first; copies use the same list as their targets.
    const int limit = wanted < c.n_pages ? (int)wanted : c.n_pages;
    const int found = limit > 0 ? find_free(c, limit, w.moved, sums) : 0;
    __syncthreads();
    // Pass 2: tables and counts; a few warps an entry, four pages a lane at once.
    const int per = n >= kWarps ? 1 : kWarps / n;  // warps an entry
    for (int i = warp / per; i < n && warp < per * n; i += kWarps / per) {
        const Entry e = entries[i];
        if (e.begin == kRefused) continue;
        int32_t *row = c.table + (int64_t)e.slot * c.max_pages;
        const int had = pages_of(e.old_len), have = pages_of(e.new_len);
        const bool takes = e.begin >= 0;
        const int first = takes ? e.begin : have, last = takes ? have : had;
        if (takes && last > first && (e.rank > found || last - first > found - e.rank)) {
            if (lane == 0) kv4_flag(status, SPARSTAR_STATUS_NO_PAGES);
            continue;
        }
        const int32_t *from = src ? c.table + (int64_t)e.from * c.max_pages : nullptr;
        for (int j0 = first + (warp % per) * 128 + lane; j0 < last; j0 += per * 128) {
            int fresh[4], old[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int j = j0 + 32 * k;
                fresh[k] = old[k] = -1;
                if (j >= last) continue;
                if (takes) fresh[k] = __ldcg(w.moved + e.rank + j - first);
                // What a page taken is a copy of (a source's page, the shared
                // partial page), or the page given up.
                if (!takes || from || j < had) old[k] = __ldcg((from ? from : row) + j);
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int j = j0 + 32 * k;
                if (j >= last) continue;
                const bool real = is_page(c, old[k]);
                if (real && !from) atomicSub(c.refs + old[k], 1);
                row[j] = fresh[k];
                if (!takes) continue;
                c.refs[fresh[k]] = 1;
                if (real) {
                    const int at = atomicAdd(&n_pairs, 1);
                    w.to[at] = fresh[k];
                    w.from[at] = old[k];
                }
            }
        }
        if (lane == 0 && warp % per == 0) c.lens[e.slot] = e.new_len;
    }
    __syncthreads();
    if (threadIdx.x == 0) w.pairs[0] = n_pairs;
}

__global__ void __launch_bounds__(kPlanThreads)
    plan_kernel(Kv4 c, const int32_t *slots, const int32_t *src, const int32_t *lens, int n,
                int32_t *status) {
    kv4_begin();
    plan(c, slots, src, lens, n, status);
}

// Copies a short list: 16 bytes a thread.
__global__ void __launch_bounds__(256) copy_few_kernel(Kv4 c) {
    kv4_begin();
    const Work w = work_of(c);
    const int pairs = w.pairs[0];
    const int vecs = c.Hkv * (kv4_page_bytes(c.D) / 16);  // of a page
    const int chunks = (vecs + 255) / 256;
    for (int64_t it = blockIdx.x; it < (int64_t)chunks * pairs; it += gridDim.x) {
        const int k = (int)(it / chunks), at = (int)(it - (int64_t)k * chunks) * 256 + threadIdx.x;
        if (at < vecs)
            reinterpret_cast<uint4 *>(c.pages)[(int64_t)w.to[k] * vecs + at] =
                reinterpret_cast<const uint4 *>(c.pages)[(int64_t)w.from[k] * vecs + at];
    }
}

// Shared fork: one CTA an entry.  No entry reads what another writes: a
// source is no destination, a destination belongs to the lowest entry.
__global__ void __launch_bounds__(256)
    fork_shared_kernel(Kv4 c, const int32_t *src, const int32_t *dst, const int32_t *len, int n,
                       int32_t *status) {
    kv4_begin();
    const int i = blockIdx.x;
    const int s = kv4_slot(c, src, i), d = kv4_slot(c, dst, i);
    bool bad = s < 0 || d < 0;
    int refuse = 0;
    for (int k = threadIdx.x; k < n; k += blockDim.x) {
        const int other = __ldca(dst + k);
        refuse |= other == s || (k < i && other == d);
    }
    bad |= __syncthreads_or(refuse) != 0;
    int L = 0;
    if (!bad) {
        const int have = kv4_len(c, s);
        L = len ? __ldca(len + i) : have;
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
    kv4_begin();
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

// Copies the listed pages; for a compaction (n_live given) also renames the
// moved ones in the tables.  A copy that gave up is said in *status and *n_live.
constexpr int kCopyThreads = 32 * kMaxStages;
__global__ void __launch_bounds__(kCopyThreads)
    copy_kernel(Kv4 c, int32_t *n_live, int32_t *status, bool withhold) {
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ uint64_t bars[kMaxStages];
    kv4_begin();
    const Work w = work_of(c);
    const int pairs = w.pairs[0];
    if (pairs == 0) return;
    if (!copy_pages(c, w, pairs, blockIdx.x, gridDim.x, bars, smem, withhold)) {
        kv4_flag(status, SPARSTAR_STATUS_TIMEOUT);
        if (n_live) atomicExch(n_live, -1);
    }
    if (!n_live) return;
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

cudaError_t launch_copy(const Kv4 &c, int32_t *n_live, int32_t *status, bool withhold,
                        cudaStream_t stream) {
    cudaError_t e = cudaFuncSetAttribute(
        copy_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kStageBytes);
    if (e != cudaSuccess) return e;
    return launch_after(copy_kernel, 148, kCopyThreads, kStageBytes, stream, c, n_live, status,
                        withhold);
}

}  // namespace

int64_t kv4_work_ints(int64_t n_pages, int64_t n_seqs) {
    return kHead + 3 * n_pages + 7 * n_seqs;
}

cudaError_t launch_kv4_resize(const Kv4 &c, const int32_t *seqs, const int32_t *new_lens, int n,
                              int32_t *status, cudaStream_t stream) {
    const cudaError_t e = launch_after(plan_kernel, 1, kPlanThreads, 0, stream, c, seqs,
                                       static_cast<const int32_t *>(nullptr), new_lens, n, status);
    if (e != cudaSuccess) return e;
    return launch_after(copy_few_kernel, 148 * 4, 256, 0, stream, c);
}

cudaError_t launch_kv4_fork(const Kv4 &c, const int32_t *src, const int32_t *dst,
                            const int32_t *len, int n, bool deep, int32_t *status,
                            cudaStream_t stream) {
    if (!deep)
        return launch_after(fork_shared_kernel, (unsigned)n, 256, 0, stream, c, src, dst, len, n,
                            status);
    const cudaError_t e =
        launch_after(plan_kernel, 1, kPlanThreads, 0, stream, c, dst, src, len, n, status);
    if (e != cudaSuccess) return e;
    return launch_copy(c, nullptr, status, false, stream);
}

cudaError_t launch_kv4_compact(const Kv4 &c, int32_t *n_live, cudaStream_t stream,
                               bool withhold) {
    const cudaError_t e =
        launch_after(compact_plan_kernel, 1, kPlanThreads, 0, stream, c, n_live);
    if (e != cudaSuccess) return e;
    return launch_copy(c, n_live, nullptr, withhold, stream);
}

}  // namespace sparstar
