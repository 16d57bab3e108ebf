// Attention of few query rows over the paged 4-bit key/value cache: single
// tokens, a few tokens, and every shape the tcgen05 kernel does not take.
//
// Rows.  The query rows that read the same pages form a stripe: the Lq rows
// of the Hq / Hkv heads of one key head (contiguous in q), or one query
// block of one head when there are block lists.  A unit is R = 8 NT rows of
// a stripe.  Its work is one tile a page.
//
// Split.  All units' tiles form one line, cut into equal parts for 148 CTAs
// and again for the parts of a CTA, a warp each, or a pair of warps on one tile:
// lengths from 1 to 144,512 tokens in one batch keep every warp equally busy, and
// one long sequence is spread over the whole GPU.  A part may begin and end inside
// a unit; such partial results (running maximum, sum, accumulator) are joined
// inside the CTA in shared memory, and across CTAs by the last one to arrive
// (in groups first, where they are many), always in the order of the line, so
// results do not depend on timing.
//
// Tile.  Each part has its own ring of half pages (codes and scales of the
// keys, or of the values), filled by one bulk copy each and waited for by its
// own warps alone.  Both products run on mma.m16n8k16 with the cache as the
// 16-row operand and the query rows as the 8 columns: S^T = K q^T (16 tokens
// x 8 rows) and O^T = V^T P^T (16 channels x 8 rows), so one dequantised
// fragment serves all NT column tiles, and few rows waste no tensor work.
// The order of channels (for S) and tokens (for O) along the contraction is
// free as long as both operands agree, so lane j of a quad takes 16
// consecutive bytes of codes: channels 32 j .. 32 j + 31 of a token (D =
// 128), tokens 32 j .. 32 j + 31 of a channel.  P^T comes out of S^T with
// one movmatrix an 8 x 8 tile.
//
// Dequantising costs a shift, a lop3 and an fma a pair of codes and is exact
// (kv4_dequant), so the cache adds no rounding.  fp32 queries and weights
// are split into three bf16 terms each, whose sum is exact to 2^-24, and
// multiplied term by term.
//
// Bounds.  The bytes of the pages at HBM's rate, in principle.  A page and head
// costs a warp 2,500 instructions, half of them on the integer pipe.  With the
// twelve warps that the registers allow, neither that pipe nor the issue slots
// are above 55% busy: waits for the pipe, for results and for a slot come to
// about equal shares.  18,064 pages and heads (144,512 tokens, 16 heads, 315 MB)
// take 83 us, 3.8 TB/s, each further one 3.5 ns, 5.0 TB/s.  At twice that length
// it takes 147 us, and the copies alone took 113 of then 144; without the
// products or without the extraction of codes hardly less, without the
// dequantisation's fma a sixth less.  A short line
// is bound by the latencies in a row: 1 us to find the line, 1.5 the tiles, 1
// the copy, 1.6 a page's arithmetic, 3 the joins; 897 tokens take 11.3 us.
#include <cuda_bf16.h>

#include "kv4.cuh"

namespace sparstar {
namespace {

constexpr int kCtas = 148;
constexpr int kEndRows = 128;  // rows of a CTA's warps, all of them
constexpr int kArrivedBytes = SPARSTAR_KV4_WORK_ZEROS;  // kCtas words and alignment
constexpr uint64_t kTimeoutNs = 2000000000ull;
constexpr int kChunks = 256;  // of sequences, for finding a place on the line
// A unit of more CTAs than kJoined is joined in groups of kFan first, as one CTA
// takes long to read 148 partial results (72,000 tokens, one key head: eight
// rows 22.9 us, so 16.6; sixteen rows 39.3 and 23.0).
constexpr int kFan = 12, kJoined = 32;

struct Plan {
    int heads;       // query heads a key head
    int units;       // units of a sequence
    int row_tiles;   // units of a stripe
    int nqb;         // query blocks of a head (lists)
    float sc;        // |tau| in log2 units; 1 for tau = 0
    uint32_t flip;   // sign bits to flip in q (tau < 0)
    bool flat;       // tau = 0: q is multiplied by 0
    uint32_t *arrived;  // [kCtas]: high half: CTAs (or groups) whose partial result of the
                        // unit that begins in this CTA and goes on is stored; low half:
                        // CTAs of the group that begins here; 0 between calls
    float *joins;       // [kCtas][2][R][D + 2]: a CTA's partial results: of the unit that
                        // goes on from the CTA before, of the one that begins here
    float *ends;        // [kCtas * kParts][R][D + 2]: ends of units inside a part
};

__device__ __forceinline__ uint32_t smem_u32(const void *p) {
    return (uint32_t)__cvta_generic_to_shared(p);
}
__device__ __forceinline__ uint64_t globaltimer() {
    uint64_t t;
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
    return t;
}
__device__ __forceinline__ void mbar_init(uint64_t *bar, uint32_t count) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(smem_u32(bar)), "r"(count)
                 : "memory");
}
__device__ __forceinline__ bool mbar_test(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}
// Bounded wait of a whole warp; false after two seconds.
__device__ __noinline__ bool wait_slow(uint32_t bar, uint32_t parity) {
    const uint64_t t0 = globaltimer();
    while (true) {
        const bool ok = mbar_test(bar, parity);
        if (__all_sync(0xffffffffu, ok)) return true;
        if (__any_sync(0xffffffffu, globaltimer() - t0 > kTimeoutNs)) return false;
    }
}
__device__ __forceinline__ bool wait_warp(uint64_t *mbar, uint32_t parity) {
    const uint32_t bar = smem_u32(mbar);
    if (__all_sync(0xffffffffu, mbar_test(bar, parity))) return true;
    return wait_slow(bar, parity);
}
__device__ __forceinline__ void bulk_load(uint32_t dst, const void *src, uint32_t bytes,
                                          uint64_t *mbar) {
    const uint32_t bar = smem_u32(mbar);
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes)
                 : "memory");
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
        ::"r"(dst), "l"(src), "r"(bytes), "r"(bar)
        : "memory");
}

__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                    uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ uint32_t pack(float lo, float hi) {
    return as_u32(__floats2bfloat162_rn(lo, hi));
}
// A bf16 pair times 0: infinities and NaN give NaN.
__device__ __forceinline__ uint32_t times0(uint32_t x) {
    return as_u32(__hmul2(as_bf162(x), __float2bfloat162_rn(0.0f)));
}
// Takes the bf16 part of two fp32 values off them.
__device__ __forceinline__ uint32_t split(float &lo, float &hi) {
    const uint32_t p = pack(lo, hi);
    lo -= __uint_as_float(p << 16);
    hi -= __uint_as_float(p & 0xffff0000u);
    return p;
}

__device__ __forceinline__ void store(float *p, float x) { *p = x; }
__device__ __forceinline__ void store(__nv_bfloat16 *p, float x) { *p = __float2bfloat16_rn(x); }

// A unit: its rows and what they see.
struct Unit {
    int i, kh, rows, first;  // sequence, key head, rows held, row of the stripe's head
    int64_t row;             // first row in q, out and lse
    int64_t list;            // row of kv_cnt / kv_idx (lists)
};
template <int R>
__device__ Unit unit_of(const Kv4 &c, const Kv4Attn &a, const Plan &p, int uid) {
    Unit u;
    u.i = uid / p.units;
    int rest = uid - u.i * p.units;
    const int rt = rest % p.row_tiles;
    rest /= p.row_tiles;
    if (a.kv_cnt) {
        const int qb = rest % p.nqb, h = rest / p.nqb;
        const int in_block = min(kBlock, a.Lq - qb * kBlock);
        u.kh = h / p.heads;
        u.first = qb * kBlock + rt * R;
        u.rows = min(R, in_block - rt * R);
        u.row = ((int64_t)u.i * a.Hq + h) * a.Lq + u.first;
        u.list = ((int64_t)u.i * a.Hq + h) * p.nqb + qb;
    } else {
        u.kh = rest;
        u.first = rt * R;
        u.rows = min(R, p.heads * a.Lq - u.first);
        u.row = ((int64_t)u.i * a.Hq + u.kh * p.heads) * a.Lq + u.first;
        u.list = 0;
    }
    return u;
}

// Tiles of one unit of sequence i: the pages of its tokens, or list entries.
__device__ __forceinline__ int tiles_of(const Kv4 &c, const Kv4Attn &a, int i, int &L) {
    const int slot = kv4_slot(c, a.seqs, i);
    L = slot >= 0 ? kv4_len(c, slot) : 0;
    if (a.kv_cnt) return slot >= 0 ? a.max_sel : 0;
    return (L + kBlock - 1) / kBlock;
}

// The partition of the line: sequence i's units' tiles begin at
// units * (tiles of the sequences before it).
struct Line {
    int64_t *prefix;  // shared: [kChunks + 1] tiles before each chunk of sequences
    int chunk;        // sequences a chunk
};
__device__ int64_t build_line(const Kv4 &c, const Kv4Attn &a, Line &line, int64_t *shared,
                              int64_t *sums) {
    line.prefix = shared;
    line.chunk = (a.n + kChunks - 1) / kChunks;
    int64_t mine = 0;
    for (int k = 0; k < line.chunk && threadIdx.x < kChunks; ++k) {
        const int i = threadIdx.x * line.chunk + k;
        int L;
        if (i < a.n) mine += tiles_of(c, a, i, L);
    }
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int64_t y = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t z = __shfl_up_sync(0xffffffffu, y, o);
        if (lane >= o) y += z;
    }
    if (lane == 31) sums[warp] = y;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kChunks / 32; ++w)
        if (w < warp) y += sums[w];
    if (threadIdx.x < kChunks) shared[threadIdx.x + 1] = y;
    if (threadIdx.x == 0) shared[0] = 0;
    __syncthreads();
    return shared[kChunks];
}

__device__ __forceinline__ int64_t per_unit(int64_t x, int units) {
    return x < 0x7fffffff ? (uint32_t)x / (uint32_t)units : x / units;
}
// The chunk of sequences that tile x lies in; for a whole warp.
__device__ __forceinline__ int chunk_of(const Line &line, int64_t x, int units) {
    static_assert(kChunks == 8 * 32, "two steps of a warp");
    const int lane = threadIdx.x & 31;
    const int64_t y = per_unit(x, units);
    const uint32_t far = __ballot_sync(0xffffffffu, line.prefix[8 * lane] <= y);
    const int lo = 8 * (31 - __clz(far));
    const uint32_t near = __ballot_sync(0xffffffffu, line.prefix[lo + (lane & 7)] <= y);
    return lo + 31 - __clz(near & 0xffu);
}

// One tile of the line.
struct Tile {
    int64_t src;     // page * Hkv + head; -1: nothing to read
    int uid, block;
    int edge;        // 1: first tile of its unit, 2: last
};
// Tile x, looked up from a chunk `lo` that is not behind its own.
template <int R>
__device__ Tile locate(const Kv4 &c, const Kv4Attn &a, const Plan &p, const Line &line,
                       int64_t x, int lo) {
    const int64_t y = per_unit(x, p.units);
    while (line.prefix[lo + 1] <= y) ++lo;
    int64_t base = line.prefix[lo];
    int i = lo * line.chunk, L, T;
    while (base + (T = tiles_of(c, a, i, L)) <= y) base += T, ++i;
    const int64_t rem = x - base * p.units;
    const int u = (int)(rem < 0x7fffffff ? (uint32_t)rem / (uint32_t)T : rem / T);
    const int t = (int)(rem - (int64_t)u * T);
    Tile tile;
    tile.uid = i * p.units + u;
    tile.edge = (t == 0 ? 1 : 0) | (t == T - 1 ? 2 : 0);
    tile.src = -1;
    const Unit un = unit_of<R>(c, a, p, tile.uid);
    const int blocks = (L + kBlock - 1) / kBlock;
    tile.block = t;
    bool listed = true;
    if (a.kv_cnt) {
        listed = un.rows > 0 && t < __ldca(a.kv_cnt + un.list);
        if (listed) tile.block = __ldca(a.kv_idx + un.list * a.max_sel + t);
    }
    if (!listed) return tile;
    if (tile.block < 0 || tile.block >= blocks) {
        kv4_flag(a.status, SPARSTAR_STATUS_BAD_INDEX);
        return tile;
    }
    // The row of the unit that sees most.
    int seen = L;
    if (a.causal) {
        const int from = un.first % a.Lq, last = from + un.rows - 1;
        seen = L - a.Lq + 1 + min(last, a.Lq - 1);
    }
    if (tile.block * kBlock >= seen) return tile;
    const int slot = kv4_slot(c, a.seqs, i);
    const int page = __ldca(c.table + (int64_t)slot * c.max_pages + tile.block);
    if (page < 0 || page >= c.n_pages) kv4_flag(a.status, SPARSTAR_STATUS_BAD_INDEX);
    else tile.src = (int64_t)page * c.Hkv + un.kh;
    return tile;
}

// Running join of partial results: maximum, sum, four channels.
struct Part4 {
    float top = -INFINITY, sum = 0.0f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    __device__ void scale(float t) {  // to the maximum t >= top
        const float f = top > -INFINITY ? ex2(top - t) : 0.0f;
        top = t;
        sum *= f;
        acc.x *= f, acc.y *= f, acc.z *= f, acc.w *= f;
    }
    __device__ void add(float m, float l, const float4 &x) {  // m <= top
        const float f = m > -INFINITY ? ex2(m - top) : 0.0f;
        sum = fmaf(f, l, sum);
        acc.x = fmaf(f, x.x, acc.x), acc.y = fmaf(f, x.y, acc.y);
        acc.z = fmaf(f, x.z, acc.z), acc.w = fmaf(f, x.w, acc.w);
    }
    // Ends the join: the result, or 0 where no token was seen.
    template <typename T>
    __device__ void write(T *out, float *lse) const {
        const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
        store(out, acc.x * inv), store(out + 1, acc.y * inv);
        store(out + 2, acc.z * inv), store(out + 3, acc.w * inv);
        if (lse) *lse = (top + log2f(sum)) * 0.6931471805599453f;
    }
};

// Counts one more arrival (from bit `shift`) and says whether all have arrived;
// what their CTAs stored can then be read.  The last one sets the count back,
// behind the fence: nobody waits for that.
__device__ __forceinline__ bool arrive(uint32_t *count, int shift, int all) {
    __threadfence();
    const uint32_t before = atomicAdd(count, 1u << shift);
    __threadfence();
    const bool last = ((before >> shift) & 0xffffu) == (uint32_t)(all - 1);
    if (last) atomicSub(count, (uint32_t)all << shift);
    return last;
}

// The result of a unit whose partial results are the records of CTAs from,
// from + step .. to (`begins`: the unit begins in the first), joined in that
// order whichever CTA runs this; without `u` a record in the first one's place.
// A thread has four channels of a row; spare threads take the records in
// pieces.  Eight records a step: their loads overlap.
template <typename T, int D, int R, int kThreads>
__device__ void join(const Plan &p, int from, int to, int step, bool begins, const Unit *u,
                     const Kv4Attn &a, float *shared) {
    constexpr int kRecord = R * (D + 2), kVecs = R * D / 4;
    constexpr int kSplit = kThreads > kVecs ? kThreads / kVecs : 1;
    const int n = (to - from) / step + 1;
    float *first = p.joins + ((int64_t)2 * from + (begins ? 1 : 0)) * kRecord;
    const float *later = p.joins + (int64_t)2 * from * kRecord;  // + 2 kRecord a CTA
    auto *piece = reinterpret_cast<Part4 *>(shared);             // [kSplit][kVecs]
    for (int v = threadIdx.x; v < kVecs * kSplit; v += kThreads) {
        const int vec = v % kVecs, row = vec / (D / 4), s = v / kVecs;
        Part4 part;
        const int k1 = n * (s + 1) / kSplit;
        for (int k0 = n * s / kSplit; k0 < k1; k0 += 8) {
            float m[8], l[8], top = part.top;
            float4 x[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                m[k] = -INFINITY, l[k] = 0.0f, x[k] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (k0 + k >= k1) continue;
                const float *rec = k0 + k ? later + (int64_t)(k0 + k) * 2 * step * kRecord : first;
                m[k] = __ldcg(rec + R * D + row);
                l[k] = __ldcg(rec + R * D + R + row);
                x[k] = __ldcg(reinterpret_cast<const float4 *>(rec) + vec);
            }
#pragma unroll
            for (int k = 0; k < 8; ++k) top = fmaxf(top, m[k]);
            part.scale(top);
#pragma unroll
            for (int k = 0; k < 8; ++k) part.add(m[k], l[k], x[k]);
        }
        piece[v] = part;
    }
    __syncthreads();
    for (int v = threadIdx.x; v < kVecs; v += kThreads) {
        const int row = v / (D / 4), d = v % (D / 4) * 4;
        if (u && row >= u->rows) continue;
        Part4 part = piece[v];
#pragma unroll
        for (int s = 1; s < kSplit; ++s) {
            const Part4 &o = piece[s * kVecs + v];
            part.scale(fmaxf(part.top, o.top));
            part.add(o.top, o.sum, o.acc);
        }
        if (u) {
            part.write(static_cast<T *>(a.out) + (u->row + row) * D + d,
                       d == 0 && a.lse ? a.lse + u->row + row : nullptr);
        } else {
            reinterpret_cast<float4 *>(first)[v] = part.acc;
            if (d == 0) first[R * D + row] = part.top, first[R * D + R + row] = part.sum;
        }
    }
}

template <int D, int NT, bool F32, int kParts, int kPair, int kStages>
__global__ void __launch_bounds__(32 * kParts * kPair, 1) few_kernel(Kv4 c, Kv4Attn a, Plan p) {
    constexpr int R = 8 * NT;
    constexpr int kThreads = 32 * kParts * kPair;
    constexpr int kTerms = F32 ? 3 : 1;
    constexpr int kHalf = kv4_half_bytes(D);
    constexpr int kCodes = kv4_code_bytes(D);
    constexpr int KS = D / 16;                 // k steps of S^T, channel tiles of O^T
    constexpr int kRow = D + 4;                // joined rows: conflict-free stores
    using T = typename std::conditional<F32, float, __nv_bfloat16>::type;
    static_assert(kThreads >= kChunks, "build_line: one chunk a thread");
    static_assert(kParts * R <= kEndRows, "scratch");
    // A pair has one tile (launch_kv4_attn_few), a half of it each warp: all it
    // copies is in the ring at once, and its results stay in registers.
    static_assert(kPair == 1 || kStages >= 2, "a tile's keys and values");
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ uint64_t full[kParts][kStages];
    __shared__ int64_t prefix[kChunks + 1], sums[kParts * kPair];
    // Partial results of the parts, in the order of the line: the end of a
    // unit inside part k (2 k), what the part's end leaves (2 k + 1).
    __shared__ int32_t entry[2 * kParts], edges[2 * kParts];
    // Units with partial results: which entries, first row, rows; flags as edges.
    __shared__ int32_t group_flags[2 * kParts], group_rows[2 * kParts];
    __shared__ uint32_t group_entries[2 * kParts];
    __shared__ int64_t group_row[2 * kParts];
    __shared__ int32_t cross[2], span[2][2], step[2], n_cross, n_groups;
    const int part = (threadIdx.x >> 5) / kPair, member = (threadIdx.x >> 5) % kPair;
    const int lane = threadIdx.x & 31;
    const int r = lane >> 2, j = lane & 3;
    const bool leads = member == 0, copies = leads && !a.withhold;
    if (lane == 0 && leads) {
        for (int s = 0; s < kStages; ++s) mbar_init(&full[part][s], 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    kv4_begin();
    Line line;
    const int64_t total = build_line(c, a, line, prefix, sums) * p.units;
    // Tiles a CTA; CTA k has the tiles from k * share.
    const int64_t share = total < 0x7fffffff - kCtas
                              ? ((uint32_t)total + kCtas - 1) / kCtas
                              : (total + kCtas - 1) / kCtas;
    // Sequences without tiles have no unit on the line.
    for (int i = blockIdx.x; i < a.n; i += gridDim.x) {
        int L;
        if (tiles_of(c, a, i, L) > 0) continue;
        if (threadIdx.x == 0 && kv4_slot(c, a.seqs, i) < 0)
            kv4_flag(a.status, SPARSTAR_STATUS_BAD_INDEX);
        const int64_t rows = (int64_t)a.Hq * a.Lq;
        T *o = static_cast<T *>(a.out) + i * rows * D;
        for (int64_t k = threadIdx.x; k < rows * D; k += kThreads) store(o + k, 0.0f);
        if (a.lse)
            for (int64_t k = threadIdx.x; k < rows; k += kThreads) a.lse[i * rows + k] = -INFINITY;
    }
    // This part: an equal piece of the CTA's tiles or, of one warp, half tiles,
    // the first ones one longer; parts with tiles are neighbours, and two may
    // have a half each of one tile.
    constexpr uint32_t kCut = kPair > 1 ? 1 : 2;
    const int64_t c0 = min(share * blockIdx.x, total), c1 = min(c0 + share, total);
    const uint32_t pieces = kCut * (uint32_t)(c1 - c0), each = pieces / kParts,
                   rest = pieces % kParts;
    const uint32_t h0 = each * part + min((uint32_t)part, rest);
    const uint32_t h1 = h0 + each + ((uint32_t)part < rest ? 1 : 0);
    const int64_t start = c0 + h0 / kCut;
    const int x1 = h1 > h0 ? (int)((h1 + kCut - 1) / kCut - h0 / kCut) : 0;  // tiles of the part
    int x = 0;
    const int slot_id = blockIdx.x * kParts + part;
    uint8_t *ring = smem + part * kStages * kHalf;
    const uint32_t magic = kv4_opaque(kMagic), sixteen = kv4_opaque(16);
    const int tok0 = 32 * (r >> 1) + (r & 1);  // of row r, with 16 hp + 4 u, + 2 for r + 8

    // Tiles 32 at a time, one a lane; the next 32 are looked up ahead.
    Tile now, next;
    auto lookup = [&](int at) {
        Tile t;
        t.src = t.uid = -1;
        t.block = t.edge = 0;
        if (at >= x1) return t;
        const int lo = chunk_of(line, start + at, p.units);
        if (at + lane < x1) t = locate<R>(c, a, p, line, start + at + lane, lo);
        return t;
    };
    auto with_page = [&](const Tile &t) { return __ballot_sync(0xffffffffu, t.src >= 0); };
    int base = 0;
    now = lookup(0);
    next = lookup(32);
    // Which of the 64 tiles in reach have a page, and which of these are still
    // to be copied: halves in order, by the lane that has the tile.
    uint64_t has = (uint64_t)with_page(next) << 32 | with_page(now), todo = has;
    int half_of = 0;  // of the next tile: 0 keys, 1 values
    uint32_t issued = 0, used = 0;
    bool ok = true;
    auto issue = [&]() {  // one half, if there is one in reach
        if (todo == 0) return;
        const int at = __ffsll((long long)todo) - 1;
        const int s = issued % kStages;
        if (copies && lane == (at & 31) && ok)
            bulk_load(smem_u32(ring + s * kHalf),
                      c.pages + (at < 32 ? now.src : next.src) * (2 * kHalf) + half_of * kHalf,
                      kHalf, &full[part][s]);
        ++issued;
        if (half_of) todo &= todo - 1;
        half_of ^= 1;
    };
    for (int s = 0; s < kStages; ++s) issue();
    auto release = [&]() {  // the oldest half is read; refill its stage
        __syncwarp();
        ++used;
        issue();
    };

    uint32_t q[kTerms][NT][KS][2];  // q^T: column r, channels of lane j
    float o[KS][NT][4];             // O^T: channels 16 k + r, + 8; rows 2 j, 2 j + 1
    float m[NT][2], l[NT][2];       // running maxima; this lane's part of the sums
    int seen[NT][2];                // tokens that rows 2 j, 2 j + 1 see
    int seen_min = 0;
    int uid = -1, started = 0;      // unit at work; it began with its first tile
    if (lane == 0 && leads) entry[2 * part] = entry[2 * part + 1] = -1;

    // Sums over the lanes that share rows.
    auto reduce_l = [&]() {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                l[nt][e] += __shfl_xor_sync(0xffffffffu, l[nt][e], 4);
                l[nt][e] += __shfl_xor_sync(0xffffffffu, l[nt][e], 8);
                l[nt][e] += __shfl_xor_sync(0xffffffffu, l[nt][e], 16);
            }
    };

    while (x < x1) {
        if (x == base + 32) {
            base += 32;
            now = next;
            next = lookup(base + 32);
            const uint64_t more = (uint64_t)with_page(next) << 32;
            has = more | has >> 32;
            todo = more | todo >> 32;
        }
        const int at = x - base;
        const bool t_has = (has >> at) & 1u;
        // block and edge in one word
        const int t_meta = __shfl_sync(0xffffffffu, now.block * 4 + now.edge, at);
        const int t_block = t_meta >> 2;
        // The halves of the tile that are this part's, and its unit's edges there.
        const int hp0 = kCut > 1 && x == 0 ? (int)(h0 % kCut) : 0;
        const int hp1 = kCut > 1 && x + 1 == x1 ? 2 - (int)(h1 % kCut) : 2;
        const int t_edge = t_meta & ((hp0 == 0 ? 1 : 0) | (hp1 == 2 ? 2 : 0));
        if (uid < 0) {  // a unit begins (the one before it has been stored)
            uid = __shfl_sync(0xffffffffu, now.uid, at);
            started = t_edge & 1;
            const Unit un = unit_of<R>(c, a, p, uid);
            const int slot = kv4_slot(c, a.seqs, un.i);
            const int L = slot >= 0 ? kv4_len(c, slot) : 0;
            seen_min = 0x7fffffff;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                const int row = nt * 8 + r;
                const T *src = static_cast<const T *>(a.q) + (un.row + row) * D + j * (D / 4);
#pragma unroll
                for (int k = 0; k < KS; ++k) {
                    if constexpr (F32) {
                        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
                        if (row < un.rows) v = __ldca(reinterpret_cast<const float4 *>(src) + k);
                        if (p.flat) v.x *= 0.0f, v.y *= 0.0f, v.z *= 0.0f, v.w *= 0.0f;
#pragma unroll
                        for (int t = 0; t < kTerms; ++t) {
                            q[t][nt][k][0] = split(v.x, v.y) ^ p.flip;
                            q[t][nt][k][1] = split(v.z, v.w) ^ p.flip;
                        }
                    } else {
                        uint2 v = make_uint2(0, 0);
                        if (row < un.rows) v = __ldca(reinterpret_cast<const uint2 *>(src) + k);
                        if (p.flat) v.x = times0(v.x), v.y = times0(v.y);
                        q[0][nt][k][0] = v.x ^ p.flip;
                        q[0][nt][k][1] = v.y ^ p.flip;
                    }
                }
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    m[nt][e] = -INFINITY;
                    l[nt][e] = 0.0f;
                    const int own = nt * 8 + 2 * j + e;
                    seen[nt][e] = a.causal ? L - a.Lq + 1 + (un.first + own) % a.Lq : L;
                    if (own < un.rows) seen_min = min(seen_min, seen[nt][e]);
                }
            }
            seen_min = min(seen_min, __shfl_xor_sync(0xffffffffu, seen_min, 1));
            seen_min = min(seen_min, __shfl_xor_sync(0xffffffffu, seen_min, 2));
#pragma unroll
            for (int k = 0; k < KS; ++k)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 4; ++e) o[k][nt][e] = 0.0f;
        }
        if (t_has) {
            while (issued < used + 2) issue();
            const int sk = used % kStages, sv = (used + 1) % kStages;
            const uint32_t pv = ((used + 1) / kStages) & 1u;
            const uint8_t *kp = ring + sk * kHalf, *vp = ring + sv * kHalf;
            ok = ok && wait_warp(&full[part][sk], (used / kStages) & 1u);
            if (!ok) break;
            // Half a page (64 tokens) at a time, each warp of a pair one; the
            // loop is kept, as the whole page's code would not fit the
            // instruction cache.
#pragma unroll 1
            for (int hp = kPair > 1 ? member : hp0; hp < (kPair > 1 ? member + 1 : hp1); ++hp) {
                float s[4][NT][4];
                // ------------------------------------------ S^T = K q^T
                // Two token tiles at a time: two chains of products.
#pragma unroll
                for (int u0 = 0; u0 < 4; u0 += 2) {
                    uint32_t w[2][2][D / 32], sc[2][2], mi[2][2];
#pragma unroll
                    for (int d = 0; d < 2; ++d)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const int tok = tok0 + 16 * hp + 4 * (u0 + d) + 2 * e;
                            uint32_t(&v)[D / 32] = w[d][e];
                            uint32_t code;
                            if constexpr (D == 128) {
                                const uint4 x4 =
                                    *reinterpret_cast<const uint4 *>(kp + tok * 64 + j * 16);
                                v[0] = x4.x, v[1] = x4.y, v[2] = x4.z, v[3] = x4.w;
                                code = kp[kCodes + tok * 4 + j];
                            } else {
                                const uint2 x2 =
                                    *reinterpret_cast<const uint2 *>(kp + tok * 32 + j * 8);
                                v[0] = x2.x, v[1] = x2.y;
                                code = kp[kCodes + tok * 2 + (j >> 1)];
                            }
                            sc[d][e] = kv4_scale_pair(code * 0x10001u, sixteen);
                            mi[d][e] = kv4_minus136(sc[d][e]);
                        }
#pragma unroll
                    for (int d = 0; d < 2; ++d)
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                            for (int e = 0; e < 4; ++e) s[u0 + d][nt][e] = 0.0f;
#pragma unroll
                    for (int k = 0; k < KS; ++k)
#pragma unroll
                        for (int d = 0; d < 2; ++d) {
                            uint32_t f[4];
#pragma unroll
                            for (int e = 0; e < 2; ++e)
#pragma unroll
                                for (int h = 0; h < 2; ++h)
                                    f[2 * h + e] = kv4_dequant(
                                        kv4_pair128(w[d][e][k / 2], 2 * (k % 2) + h, magic),
                                        sc[d][e], mi[d][e]);
#pragma unroll
                            for (int t = kTerms - 1; t >= 0; --t)
#pragma unroll
                                for (int nt = 0; nt < NT; ++nt)
                                    mma(s[u0 + d][nt], f, q[t][nt][k][0], q[t][nt][k][1]);
                        }
                }
                if (kPair > 1 || hp + 1 == hp1) release();  // the keys
                // --------------------------------------------- softmax
                if ((t_block + 1) * kBlock > seen_min) {
#pragma unroll
                    for (int u = 0; u < 4; ++u)
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const int tok = t_block * kBlock + tok0 + 16 * hp + 4 * u +
                                                2 * (e >> 1);
                                if (tok >= seen[nt][e & 1]) s[u][nt][e] = -INFINITY;
                            }
                }
                uint32_t pw[kTerms][4][NT][2];  // P^T, tokens of the quad's lane j
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    float neg[2];
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float mx = fmaxf(s[0][nt][e], s[0][nt][e + 2]);
#pragma unroll
                        for (int u = 1; u < 4; ++u)
                            mx = fmaxf(mx, fmaxf(s[u][nt][e], s[u][nt][e + 2]));
                        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
                        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
                        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
                        const float top = fmaxf(m[nt][e], mx * p.sc);
                        if (__any_sync(0xffffffffu, top > m[nt][e])) {
                            const float f = top > m[nt][e] ? ex2(m[nt][e] - top) : 1.0f;
                            m[nt][e] = top;
                            l[nt][e] *= f;
#pragma unroll
                            for (int k = 0; k < KS; ++k) {
                                o[k][nt][e] *= f;
                                o[k][nt][e + 2] *= f;
                            }
                        }
                        // While every token was masked, every weight is 0.
                        neg[e] = top > -INFINITY ? -top : 0.0f;
                    }
#pragma unroll
                    for (int u = 0; u < 4; ++u) {
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            s[u][nt][e] = ex2(fmaf(s[u][nt][e], p.sc, neg[e & 1]));
                            l[nt][e & 1] += s[u][nt][e];
                        }
#pragma unroll
                        for (int t = 0; t < kTerms; ++t)
#pragma unroll
                            for (int e = 0; e < 2; ++e)
                                pw[t][u][nt][e] = transpose8x8(
                                    t + 1 < kTerms
                                        ? split(s[u][nt][2 * e], s[u][nt][2 * e + 1])
                                        : pack(s[u][nt][2 * e], s[u][nt][2 * e + 1]));
                    }
                }
                // ------------------------------------- O^T += V^T P^T
                if (kPair > 1 || hp == hp0) {
                    ok = ok && wait_warp(&full[part][sv], pv);
                    if (!ok) break;
                }
#pragma unroll
                for (int g = 0; g < D / kGroup; ++g) {
                    uint32_t sc[8], mi[8];  // of token pairs 32 j + 16 hp + 2 i
                    {
                        const uint4 v = *reinterpret_cast<const uint4 *>(
                            vp + kCodes + g * kBlock + 32 * j + 16 * hp);
                        const uint32_t b[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            sc[i] = kv4_scale_pair(
                                __byte_perm(b[i / 2], 0, (i & 1) ? 0x4342 : 0x4140), sixteen);
                            mi[i] = kv4_minus136(sc[i]);
                        }
                    }
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        const int k = 2 * g + half;
                        uint32_t w[2][2];
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const uint2 v = *reinterpret_cast<const uint2 *>(
                                vp + (16 * k + r + 8 * e) * 64 + j * 16 + 8 * hp);
                            w[e][0] = v.x, w[e][1] = v.y;
                        }
                        // fp32: the sum of 64 tokens apart, joined by rounded
                        // additions (the tensor core's own ones truncate).
                        float part[NT][4];
                        if constexpr (F32) {
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                                for (int e = 0; e < 4; ++e) part[nt][e] = 0.0f;
                        }
#pragma unroll
                        for (int u = 0; u < 4; ++u) {
                            uint32_t f[4];
#pragma unroll
                            for (int e = 0; e < 2; ++e)
#pragma unroll
                                for (int h = 0; h < 2; ++h)
                                    f[2 * h + e] = kv4_dequant(
                                        kv4_pair128(w[e][u / 2], 2 * (u % 2) + h, magic),
                                        sc[2 * u + h], mi[2 * u + h]);
#pragma unroll
                            for (int t = kTerms - 1; t >= 0; --t)
#pragma unroll
                                for (int nt = 0; nt < NT; ++nt) {
                                    if constexpr (F32)
                                        mma(part[nt], f, pw[t][u][nt][0], pw[t][u][nt][1]);
                                    else
                                        mma(o[k][nt], f, pw[t][u][nt][0], pw[t][u][nt][1]);
                                }
                        }
                        if constexpr (F32) {
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                                for (int e = 0; e < 4; ++e) o[k][nt][e] += part[nt][e];
                        }
                    }
                }
            }
            if (!ok) break;
            release();  // the values
        }
        ++x;
        const bool ends = (t_edge & 2) != 0;
        if (kPair == 1 && x < x1 && !ends) continue;
        // The unit ends here, or the part does.
        reduce_l();
        if (kPair > 1 || x == x1) {  // what the part's end leaves stays in registers
            if (lane == 0 && leads) {
                entry[2 * part + 1] = uid;
                edges[2 * part + 1] = started | (t_edge & 2);
            }
            break;
        }
        if (started) {  // whole: straight to the output
            const Unit un = unit_of<R>(c, a, p, uid);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int row = nt * 8 + 2 * j + e;
                    if (row >= un.rows) continue;
                    const float inv = l[nt][e] == 0.0f ? 0.0f : 1.0f / l[nt][e];
                    T *dst = static_cast<T *>(a.out) + (un.row + row) * D + r;
#pragma unroll
                    for (int k = 0; k < KS; ++k) {
                        store(dst + 16 * k, o[k][nt][e] * inv);
                        store(dst + 16 * k + 8, o[k][nt][e + 2] * inv);
                    }
                    if (a.lse && r == 0)
                        a.lse[un.row + row] =
                            (m[nt][e] + log2f(l[nt][e])) * 0.6931471805599453f;
                }
        } else {  // the end of a unit that began before this part
            float *rec = p.ends + (int64_t)slot_id * R * (D + 2);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int row = nt * 8 + 2 * j + e;
#pragma unroll
                    for (int k = 0; k < KS; ++k) {
                        rec[row * D + 16 * k + r] = o[k][nt][e];
                        rec[row * D + 16 * k + r + 8] = o[k][nt][e + 2];
                    }
                    if (r == 0) {
                        rec[R * D + row] = m[nt][e];
                        rec[R * D + R + row] = l[nt][e];
                    }
                }
            if (lane == 0) {
                entry[2 * part] = uid;
                edges[2 * part] = 2;
            }
        }
        uid = -1;
    }
    // Copies in flight land before anything else uses the ring.
    for (; used < issued; ++used)
        ok = wait_warp(&full[part][used % kStages], (used / kStages) & 1u) && ok;
    if (!ok && lane == 0) kv4_flag(a.status, SPARSTAR_STATUS_TIMEOUT);

    // ------------------------------ the parts' partial results, unit by unit
    __syncthreads();
    constexpr int kRecord = R * (D + 2);
    constexpr int kWarps = kParts * kPair, kHeld = kWarps + (kPair == 1 ? kParts : 0);
    // What each warp's registers hold, then the ends inside parts: [kHeld].
    float *so = reinterpret_cast<float *>(smem);  // [kHeld][R][kRow]
    float *sm = so + kHeld * R * kRow, *sl = sm + kHeld * R;
    if (threadIdx.x >= kThreads - 32) {  // the last warp, often idle: an entry a lane
        static_assert(2 * kParts <= 32, "an entry a lane");
        const int id = lane < 2 * kParts ? entry[lane] : -1;
        const int edge = id >= 0 ? edges[lane] : 0;
        const uint32_t same = __match_any_sync(0xffffffffu, id);
        const uint32_t below = (1u << lane) - 1;
        const bool first = id >= 0 && (same & below) == 0;
        const uint32_t firsts = __ballot_sync(0xffffffffu, first);
        const uint32_t enders = __ballot_sync(0xffffffffu, (edge & 2) != 0);
        const int flags = (edge & 1) | ((enders & same) ? 2 : 0);
        // At most two go on in other CTAs: the first and the last.
        const uint32_t crossing = __ballot_sync(0xffffffffu, first && flags != 3);
        if (lane == 0) n_groups = __popc(firsts), n_cross = __popc(crossing);
        if (first) {
            const int g = __popc(firsts & below);
            const Unit un = unit_of<R>(c, a, p, id);
            group_entries[g] = same;
            group_flags[g] = flags;
            group_row[g] = un.row;
            group_rows[g] = un.rows;
        }
        if (first && flags != 3) {  // its CTAs
            const int k = __popc(crossing & below), i = id / p.units;
            int64_t at = line.prefix[i / line.chunk];
            int L;
            for (int s = i / line.chunk * line.chunk; s < i; ++s) at += tiles_of(c, a, s, L);
            const int tiles = tiles_of(c, a, i, L);
            at = at * p.units + (int64_t)(id - i * p.units) * tiles;
            cross[k] = id;
            span[k][0] = (int)(at / share);
            span[k][1] = (int)((at + tiles - 1) / share);
        }
    }
    if (entry[2 * part + 1] >= 0) {
        const int w = part * kPair + member;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int row = nt * 8 + 2 * j + e;
                float *dst = so + (w * R + row) * kRow + r;
#pragma unroll
                for (int k = 0; k < KS; ++k) {
                    dst[16 * k] = o[k][nt][e];
                    dst[16 * k + 8] = o[k][nt][e + 2];
                }
                if (r == 0) {
                    sm[w * R + row] = m[nt][e];
                    sl[w * R + row] = l[nt][e];
                }
            }
    }
    if (kPair == 1 && entry[2 * part] >= 0) {
        const float *rec = p.ends + (int64_t)slot_id * kRecord;
        const int w = kWarps + part;
        for (int v = lane; v < R * D / 4; v += 32)
            *reinterpret_cast<float4 *>(so + (w * R + v / (D / 4)) * kRow + v % (D / 4) * 4) =
                *reinterpret_cast<const float4 *>(rec + 4 * v);
        if (lane < R) {
            sm[w * R + lane] = rec[R * D + lane];
            sl[w * R + lane] = rec[R * D + R + lane];
        }
    }
    __syncthreads();
    for (int it = threadIdx.x; it < n_groups * (R * D / 4); it += kThreads) {
        const int g = it / (R * D / 4), v = it % (R * D / 4);
        const int row = v / (D / 4), d = v % (D / 4) * 4;
        Part4 sum;
        float top = -INFINITY;
        auto each = [&](auto f) {
            for (uint32_t left = group_entries[g]; left; left &= left - 1) {
                const int en = __ffs(left) - 1;
#pragma unroll
                for (int w = 0; w < kPair; ++w) f((en & 1 ? 0 : kWarps) + (en >> 1) * kPair + w);
            }
        };
        each([&](int w) { top = fmaxf(top, sm[w * R + row]); });
        sum.top = top;
        each([&](int w) {
            sum.add(sm[w * R + row], sl[w * R + row],
                    *reinterpret_cast<const float4 *>(so + (w * R + row) * kRow + d));
        });
        if (group_flags[g] != 3) {
            float *rec = p.joins + (int64_t)(blockIdx.x * 2 + (group_flags[g] & 1)) * kRecord;
            *reinterpret_cast<float4 *>(rec + 4 * v) = sum.acc;
            if (d == 0) rec[R * D + row] = sum.top, rec[R * D + R + row] = sum.sum;
        } else if (row < group_rows[g]) {
            const int64_t out_row = group_row[g] + row;
            sum.write(static_cast<T *>(a.out) + out_row * D + d,
                      d == 0 && a.lse ? a.lse + out_row : nullptr);
        }
    }
    // ---------------- units of several CTAs: the last one to arrive joins them
    __syncthreads();
    const int me = blockIdx.x;
    if (threadIdx.x < n_cross) {
        const int k = threadIdx.x, from = span[k][0], to = span[k][1];
        const bool group = to - from >= kJoined;  // its group first
        const int g0 = group ? me - (me - from) % kFan : from;
        const int all = (group ? min(g0 + kFan - 1, to) : to) - g0 + 1;
        const bool last = all == 1 || arrive(p.arrived + g0, group ? 0 : 16, all);
        step[k] = last ? (group ? kFan : 1) : 0;
    }
    __syncthreads();
    float *shared = reinterpret_cast<float *>(smem);
    for (int k = 0; k < n_cross; ++k) {
        if (step[k] == 0) continue;
        const Unit un = unit_of<R>(c, a, p, cross[k]);
        const int from = span[k][0], to = span[k][1], g0 = me - (me - from) % kFan;
        bool group = step[k] == kFan;
        while (true) {  // one copy of the code
            const int r0 = group ? g0 : from, r1 = group ? min(g0 + kFan - 1, to) : to;
            join<T, D, R, kThreads>(p, r0, r1, group ? 1 : step[k], !group || g0 == from,
                                    group ? nullptr : &un, a, shared);
            __syncthreads();
            if (!group) break;
            if (threadIdx.x == 0 && !arrive(p.arrived + from, 16, (to - from) / kFan + 1))
                step[k] = 0;
            __syncthreads();
            if (step[k] == 0) break;
            group = false;
        }
    }
}

template <int D, int NT, bool F32, int kParts, int kPair>
cudaError_t launch(const Kv4 &c, const Kv4Attn &a, const Plan &p, cudaStream_t stream) {
    constexpr int kStages = 24 * (128 / D) / kParts;  // 209 KB
    constexpr int kRing = kParts * kStages * kv4_half_bytes(D);
    constexpr int kHeld = kParts * kPair + (kPair == 1 ? kParts : 0);
    constexpr int kJoin = kHeld * 8 * NT * (D + 4 + 2) * 4;
    constexpr int kBytes = kRing > kJoin ? kRing : kJoin;
    const auto kernel = few_kernel<D, NT, F32, kParts, kPair, kStages>;
    cudaError_t e =
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kBytes);
    if (e != cudaSuccess) return e;
    return launch_after(kernel, kCtas, 32 * kParts * kPair, kBytes, stream, c, a, p);
}

int stripe_rows(int64_t Hq, int64_t Hkv, int64_t Lq, bool lists) {
    return (int)(lists ? (Lq < kBlock ? Lq : kBlock) : Hq / Hkv * Lq);
}

}  // namespace

int64_t kv4_attn_few_work_bytes(int D) {
    return kArrivedBytes + (int64_t)kCtas * (2 * 16 + kEndRows) * (D + 2) * 4;
}

cudaError_t launch_kv4_attn_few(const Kv4 &c, const Kv4Attn &a, int dtype, cudaStream_t stream) {
    const bool lists = a.kv_cnt != nullptr;
    const int rows = stripe_rows(a.Hq, c.Hkv, a.Lq, lists);
    const bool f32 = dtype == SPARSTAR_F32;
    // Eight rows a unit, or sixteen where there are more: the second column
    // tile shares the dequantised fragments.  fp32 has no registers for it.
    const int R = rows <= 8 || f32 ? 8 : 16;
    Plan p;
    p.heads = a.Hq / c.Hkv;
    p.row_tiles = (rows + R - 1) / R;
    p.nqb = (a.Lq + kBlock - 1) / kBlock;
    p.units = p.row_tiles * (lists ? a.Hq * p.nqb : c.Hkv);
    // A scale of 0 would turn masked scores (-inf) into NaN: it goes into the
    // queries instead.  No other tau has a product of 0.
    p.flat = a.tau == 0.0f;
    p.sc = p.flat ? 1.0f : fabsf(a.tau) * 1.4426950408889634f;
    p.flip = a.tau < 0.0f ? 0x80008000u : 0u;
    p.arrived = static_cast<uint32_t *>(a.work);
    p.joins = static_cast<float *>(a.work) + kArrivedBytes / 4;
    p.ends = p.joins + (int64_t)2 * kCtas * R * (c.D + 2);
    // Eight rows: twelve warps, each with (halves of) pages of its own, keep the
    // registers that hide the latencies.  Where that gives some warps one half
    // and some two or three, eight pairs of warps, a page each, take less (16
    // heads: 3,000 tokens 12.2 us against 12.6, 6,000 tokens 14.0 against 18.2,
    // 9,000 tokens 15.7 against 19.9; below, 1,000 tokens, 12.0 and 12.0, 2,000
    // tokens 12.1 and 12.4; above, a pair would have more than one page).  The
    // tables' widths decide, not the lengths, which only the device knows: 6,000
    // tokens in a table of 258 pages take 18.3 us.
    const double most = (double)a.n * p.units * (lists ? a.max_sel : c.max_pages);
    // Not more than 8 * 148 tiles: no part of 8 * 148 has more than one.
    constexpr int kPairs = 8;
    const bool pairs = most > 2.0 * kCtas && most <= (double)kPairs * kCtas;
    if (c.D == 128) {
        if (f32) return launch<128, 1, true, 8, 1>(c, a, p, stream);
        if (R == 16) return launch<128, 2, false, 8, 1>(c, a, p, stream);
        return pairs ? launch<128, 1, false, kPairs, 2>(c, a, p, stream)
                     : launch<128, 1, false, 12, 1>(c, a, p, stream);
    }
    if (f32) return launch<64, 1, true, 8, 1>(c, a, p, stream);
    if (R == 16) return launch<64, 2, false, 8, 1>(c, a, p, stream);
    return pairs ? launch<64, 1, false, kPairs, 2>(c, a, p, stream)
                 : launch<64, 1, false, 12, 1>(c, a, p, stream);
}

}  // namespace sparstar
