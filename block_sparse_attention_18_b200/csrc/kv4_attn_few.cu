// Attention of few query rows over the paged 4-bit key/value cache: single
// tokens, a few tokens, and every shape the tcgen05 kernel does not take.
//
// Rows.  The query rows that read the same pages form a stripe: the Lq rows
// of the Hq / Hkv heads of one key head (contiguous in q), or one query
// block of one head when there are block lists.  A unit is R = 8 NT rows of
// a stripe.  Its work is one tile a page.
//
// Split.  All units' tiles form one line, cut into equal parts for 148 CTAs
// and again for their eight warps: lengths from 1 to 144,512 tokens in one
// batch keep every warp equally busy, and one long sequence is spread over
// the whole GPU.  A warp's part may begin and end inside a unit; such partial
// results (running maximum, sum, accumulator) are joined inside the CTA in
// shared memory and across CTAs by a second kernel, always in the order of
// the line, so results do not depend on timing.
//
// Tile.  Each warp has its own ring of half pages (codes and scales of the
// keys, or of the values), filled by one bulk copy each and waited for by
// this warp alone.  Both products run on mma.m16n8k16 with the cache as the
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
#include <cuda_bf16.h>

#include "kv4.cuh"

namespace sparstar {
namespace {

constexpr int kCtas = 148, kWarps = 8, kThreads = 32 * kWarps;
constexpr int kSlots = kCtas * kWarps;
constexpr uint64_t kTimeoutNs = 2000000000ull;
constexpr int kMaxChunks = kThreads;

struct Plan {
    int heads;       // query heads a key head
    int units;       // units of a sequence
    int row_tiles;   // units of a stripe
    int nqb;         // query blocks of a head (lists)
    float sc;        // |tau| in log2 units
    uint32_t flip;   // sign bits to flip in q (tau < 0)
    int32_t *head;   // [3][kSlots]: unit of the last and of the first partial result, and
                     // of the last: 1 when it begins there and goes on, 2 when it ends there
    float *records;  // [kSlots][2][R][D + 2]
};

__device__ __forceinline__ uint32_t smem_u32(const void *p) {
    return (uint32_t)__cvta_generic_to_shared(p);
}
__device__ __forceinline__ uint64_t globaltimer() {
    uint64_t t;
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
    return t;
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
__device__ __forceinline__ bool wait_warp(uint32_t bar, uint32_t parity) {
    if (__all_sync(0xffffffffu, mbar_test(bar, parity))) return true;
    return wait_slow(bar, parity);
}
__device__ __forceinline__ void bulk_load(uint32_t dst, const void *src, uint32_t bytes,
                                          uint32_t bar) {
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
    int64_t *prefix;  // shared: [kMaxChunks + 1] tiles before each chunk of sequences
    int chunk;        // sequences a chunk
};
__device__ int64_t build_line(const Kv4 &c, const Kv4Attn &a, Line &line, int64_t *shared,
                              int64_t *sums) {
    line.prefix = shared;
    line.chunk = (a.n + kMaxChunks - 1) / kMaxChunks;
    int64_t mine = 0;
    for (int k = 0; k < line.chunk; ++k) {
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
    for (int w = 0; w < warp; ++w) y += sums[w];
    shared[threadIdx.x + 1] = y;
    if (threadIdx.x == 0) shared[0] = 0;
    __syncthreads();
    return shared[kMaxChunks];
}

// One tile of the line.
struct Tile {
    int uid, page, block;  // page -1: nothing to read
    int edge;              // 1: first tile of its unit, 2: last
};
template <int R>
__device__ Tile locate(const Kv4 &c, const Kv4Attn &a, const Plan &p, const Line &line,
                       int64_t x) {
    const int64_t y = x / p.units;
    int lo = 0, hi = kMaxChunks;  // prefix[lo] <= y < prefix[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (line.prefix[mid] <= y) lo = mid;
        else hi = mid;
    }
    int64_t base = line.prefix[lo];
    int i = lo * line.chunk, L, T;
    while (base + (T = tiles_of(c, a, i, L)) <= y) base += T, ++i;
    const int64_t rem = x - base * p.units;
    const int u = (int)(rem / T), t = (int)(rem - (int64_t)u * T);
    Tile tile;
    tile.uid = i * p.units + u;
    tile.edge = (t == 0 ? 1 : 0) | (t == T - 1 ? 2 : 0);
    tile.page = -1;
    const Unit un = unit_of<R>(c, a, p, tile.uid);
    const int blocks = (L + kBlock - 1) / kBlock;
    tile.block = t;
    bool listed = true;
    if (a.kv_cnt) {
        listed = un.rows > 0 && t < __ldg(a.kv_cnt + un.list);
        if (listed) tile.block = __ldg(a.kv_idx + un.list * a.max_sel + t);
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
    const int page = __ldg(c.table + (int64_t)slot * c.max_pages + tile.block);
    if (page < 0 || page >= c.n_pages) kv4_flag(a.status, SPARSTAR_STATUS_BAD_INDEX);
    else tile.page = page;
    return tile;
}

template <int D, int NT, bool F32>
__global__ void __launch_bounds__(kThreads, 1) few_kernel(Kv4 c, Kv4Attn a, Plan p) {
    constexpr int R = 8 * NT;
    constexpr int kTerms = F32 ? 3 : 1;
    constexpr int kHalf = kv4_half_bytes(D);
    constexpr int kCodes = kv4_code_bytes(D);
    constexpr int kStages = D == 128 ? 3 : 6;  // half pages a warp keeps in flight
    constexpr int KS = D / 16;                 // k steps of S^T, channel tiles of O^T
    constexpr int kRow = D + 4;                // joined rows: conflict-free stores
    using T = typename std::conditional<F32, float, __nv_bfloat16>::type;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ uint64_t bars[kWarps][kStages];
    __shared__ int64_t prefix[kMaxChunks + 1], sums[kWarps];
    __shared__ int32_t last_uid[kWarps], last_edge[kWarps];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int r = lane >> 2, j = lane & 3;
    // The joining kernel may start its launch; it waits for this one's end.
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (lane == 0) {
        for (int s = 0; s < kStages; ++s)
            asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" ::"r"(smem_u32(&bars[warp][s]))
                         : "memory");
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    Line line;
    const int64_t total = build_line(c, a, line, prefix, sums) * p.units;
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
    // This warp's part [x, x1) of the line.
    const int64_t c0 = total * blockIdx.x / kCtas, c1 = total * (blockIdx.x + 1) / kCtas;
    // The warps' parts: equal, the last ones shorter or empty, so that parts
    // with tiles are neighbours.
    const int64_t part = (c1 - c0 + kWarps - 1) / kWarps;
    int64_t x = min(c0 + part * warp, c1);
    const int64_t x1 = min(x + part, c1);
    const int slot_id = blockIdx.x * kWarps + warp;
    const uint32_t ring = smem_u32(smem) + warp * kStages * kHalf;
    const uint8_t *ring_ptr = smem + warp * kStages * kHalf;

    // Tiles 32 at a time, one a lane; the next 32 are looked up ahead.
    Tile now, next;
    auto lookup = [&](int64_t at) {
        Tile t;
        t.uid = t.page = -1;
        t.block = t.edge = 0;
        if (at + lane < x1) t = locate<R>(c, a, p, line, at + lane);
        return t;
    };
    int64_t base = x;
    now = lookup(base);
    next = lookup(base + 32);
    // Copies: halves of tiles with a page, in order.
    int64_t ix = x;       // next tile to copy
    int half_of = 0;      // its half: 0 keys, 1 values
    uint32_t issued = 0, used = 0;
    auto issue = [&]() {  // one half, if there is one in reach
        while (ix < x1 && ix < base + 64) {
            const int at = (int)(ix - base);
            const int page = __shfl_sync(0xffffffffu, at < 32 ? now.page : next.page, at & 31);
            if (page >= 0) {
                const int uid = __shfl_sync(0xffffffffu, at < 32 ? now.uid : next.uid, at & 31);
                if (lane == 0) {
                    int rest = (uid % p.units) / p.row_tiles;
                    const int kh = a.kv_cnt ? rest / p.nqb / p.heads : rest;
                    const int s = issued % kStages;
                    bulk_load(ring + s * kHalf,
                              c.pages + ((int64_t)page * c.Hkv + kh) * (2 * kHalf) +
                                  half_of * kHalf,
                              kHalf, smem_u32(&bars[warp][s]));
                }
                ++issued;
                if (half_of) ++ix;
                half_of ^= 1;
                return;
            }
            ++ix;
        }
    };
    for (int s = 0; s < kStages; ++s) issue();

    uint32_t q[kTerms][NT][KS][2];  // q^T: column r, channels of lane j
    float o[KS][NT][4];             // O^T: channels 16 k + r, + 8; rows 2 j, 2 j + 1
    float m[NT][2], l[NT][2];       // running maxima; this lane's part of the sums
    int seen[NT][2];                // tokens that rows 2 j, 2 j + 1 see
    int seen_min = 0;
    int uid = -1, started = 0;      // unit at work; it began with its first tile
    Unit un{};
    bool ok = true;
    if (lane == 0) {
        p.head[slot_id] = p.head[kSlots + slot_id] = -1;
        p.head[2 * kSlots + slot_id] = 0;
        last_uid[warp] = -1;
        last_edge[warp] = 0;
    }

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
        }
        const int at = (int)(x - base);
        const int t_uid = __shfl_sync(0xffffffffu, now.uid, at);
        const int t_page = __shfl_sync(0xffffffffu, now.page, at);
        const int t_block = __shfl_sync(0xffffffffu, now.block, at);
        const int t_edge = __shfl_sync(0xffffffffu, now.edge, at);
        if (t_uid != uid) {  // a unit begins (the one before it has been stored)
            uid = t_uid;
            started = t_edge & 1;
            un = unit_of<R>(c, a, p, uid);
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
                        if (row < un.rows) v = __ldg(reinterpret_cast<const float4 *>(src) + k);
#pragma unroll
                        for (int t = 0; t < kTerms; ++t) {
                            q[t][nt][k][0] = split(v.x, v.y) ^ p.flip;
                            q[t][nt][k][1] = split(v.z, v.w) ^ p.flip;
                        }
                    } else {
                        uint2 v = make_uint2(0, 0);
                        if (row < un.rows) v = __ldg(reinterpret_cast<const uint2 *>(src) + k);
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
        if (t_page >= 0) {
            while (issued < used + 2 && issued - used < kStages) issue();
            // ---------------------------------------------- S^T = K q^T
            int st = used % kStages;
            ok = wait_warp(smem_u32(&bars[warp][st]), (used / kStages) & 1u);
            if (!ok) break;
            const uint8_t *kp = ring_ptr + st * kHalf;
            float s[8][NT][4];
#pragma unroll
            for (int u = 0; u < 8; ++u) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 4; ++e) s[u][nt][e] = 0.0f;
                uint32_t w[2][D / 32], sc[2], mi[2];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int tok = 32 * (r >> 1) + 4 * u + (r & 1) + 2 * e;
                    if constexpr (D == 128) {
                        const uint4 v = *reinterpret_cast<const uint4 *>(kp + tok * 64 + j * 16);
                        w[e][0] = v.x, w[e][1] = v.y, w[e][2] = v.z, w[e][3] = v.w;
                        sc[e] = kv4_scale_pair(kp[kCodes + tok * 4 + j] * 0x10001u);
                    } else {
                        const uint2 v = *reinterpret_cast<const uint2 *>(kp + tok * 32 + j * 8);
                        w[e][0] = v.x, w[e][1] = v.y;
                        sc[e] = kv4_scale_pair(kp[kCodes + tok * 2 + (j >> 1)] * 0x10001u);
                    }
                    mi[e] = kv4_minus136(sc[e]);
                }
#pragma unroll
                for (int k = 0; k < KS; ++k) {
                    uint32_t f[4];
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        f[e] = kv4_dequant(kv4_pair128(w[e][k / 2], 2 * (k % 2)), sc[e], mi[e]);
                        f[2 + e] =
                            kv4_dequant(kv4_pair128(w[e][k / 2], 2 * (k % 2) + 1), sc[e], mi[e]);
                    }
#pragma unroll
                    for (int t = kTerms - 1; t >= 0; --t)
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
                            mma(s[u][nt], f, q[t][nt][k][0], q[t][nt][k][1]);
                }
            }
            __syncwarp();  // the keys' half is read: refill it
            ++used;
            issue();
            // ------------------------------------------------- softmax
            if ((t_block + 1) * kBlock > seen_min) {
#pragma unroll
                for (int u = 0; u < 8; ++u)
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int tok = t_block * kBlock + 32 * (r >> 1) + 4 * u + (r & 1) +
                                            2 * (e >> 1);
                            if (tok >= seen[nt][e & 1]) s[u][nt][e] = -INFINITY;
                        }
            }
            uint32_t pw[kTerms][8][NT][2];  // P^T, tokens of the quad's lane j
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                float neg[2];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float mx = fmaxf(s[0][nt][e], s[0][nt][e + 2]);
#pragma unroll
                    for (int u = 1; u < 8; ++u)
                        mx = fmaxf(mx, fmaxf(s[u][nt][e], s[u][nt][e + 2]));
                    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
                    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
                    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
                    const float top = fmaxf(m[nt][e], mx * p.sc);
                    const float f = top > m[nt][e] ? ex2(m[nt][e] - top) : 1.0f;
                    m[nt][e] = top;
                    l[nt][e] *= f;
                    if (__any_sync(0xffffffffu, f != 1.0f)) {
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
                for (int u = 0; u < 8; ++u) {
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
                                t + 1 < kTerms ? split(s[u][nt][2 * e], s[u][nt][2 * e + 1])
                                               : pack(s[u][nt][2 * e], s[u][nt][2 * e + 1]));
                }
            }
            // --------------------------------------------- O^T += V^T P^T
            st = used % kStages;
            ok = wait_warp(smem_u32(&bars[warp][st]), (used / kStages) & 1u);
            if (!ok) break;
            const uint8_t *vp = ring_ptr + st * kHalf;
#pragma unroll
            for (int g = 0; g < D / kGroup; ++g) {
                uint32_t sc[16], mi[16];  // of token pairs 32 j + 2 i
                {
                    const uint4 *sp = reinterpret_cast<const uint4 *>(vp + kCodes + g * kBlock +
                                                                      32 * j);
                    const uint4 v0 = sp[0], v1 = sp[1];
                    const uint32_t b[8] = {v0.x, v0.y, v0.z, v0.w, v1.x, v1.y, v1.z, v1.w};
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        sc[i] = kv4_scale_pair(
                            __byte_perm(b[i / 2], 0, (i & 1) ? 0x4342 : 0x4140));
                        mi[i] = kv4_minus136(sc[i]);
                    }
                }
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    const int k = 2 * g + half;
                    uint32_t w[2][4];
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const uint4 v = *reinterpret_cast<const uint4 *>(
                            vp + (16 * k + r + 8 * e) * 64 + j * 16);
                        w[e][0] = v.x, w[e][1] = v.y, w[e][2] = v.z, w[e][3] = v.w;
                    }
                    // fp32: the page's sum apart, joined by rounded additions
                    // (the tensor core's own additions truncate).
                    float part[NT][4];
                    if constexpr (F32) {
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                            for (int e = 0; e < 4; ++e) part[nt][e] = 0.0f;
                    }
#pragma unroll
                    for (int u = 0; u < 8; ++u) {
                        uint32_t f[4];
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            f[e] = kv4_dequant(kv4_pair128(w[e][u / 2], 2 * (u % 2)), sc[2 * u],
                                               mi[2 * u]);
                            f[2 + e] = kv4_dequant(kv4_pair128(w[e][u / 2], 2 * (u % 2) + 1),
                                                   sc[2 * u + 1], mi[2 * u + 1]);
                        }
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
            __syncwarp();
            ++used;
            issue();
        }
        ++x;
        const bool ends = (t_edge & 2) != 0;
        if (x < x1 && !ends) continue;
        // The unit ends here, or this warp's part does.
        reduce_l();
        if (ends && started) {  // whole: straight to the output
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
        } else if (x < x1) {  // the end of a unit that began before this part
            float *rec = p.records + ((int64_t)slot_id * 2 + 1) * R * (D + 2);
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
            if (lane == 0) p.head[kSlots + slot_id] = uid;
        } else if (lane == 0) {
            last_uid[warp] = uid;
            last_edge[warp] = started | (ends ? 2 : 0);
        }
        if (ends) uid = -1;
    }
    // Copies in flight land before anything else uses the ring.
    while (used < issued) {
        if (!wait_warp(smem_u32(&bars[warp][used % kStages]), (used / kStages) & 1u)) ok = false;
        ++used;
    }
    if (!ok && lane == 0) kv4_flag(a.status, SPARSTAR_STATUS_TIMEOUT);

    // ---------------------- partial results at the parts' ends, CTA by CTA
    __syncthreads();
    float *so = reinterpret_cast<float *>(smem);       // [kWarps][R][kRow]
    float *sm = so + kWarps * R * kRow, *sl = sm + kWarps * R;
    if (last_uid[warp] >= 0) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int row = nt * 8 + 2 * j + e;
                float *dst = so + (warp * R + row) * kRow + r;
#pragma unroll
                for (int k = 0; k < KS; ++k) {
                    dst[16 * k] = o[k][nt][e];
                    dst[16 * k + 8] = o[k][nt][e + 2];
                }
                if (r == 0) {
                    sm[warp * R + row] = m[nt][e];
                    sl[warp * R + row] = l[nt][e];
                }
            }
    }
    __syncthreads();
    for (int w0 = 0; w0 < kWarps;) {
        const int id = last_uid[w0];
        int w1 = w0 + 1;
        while (w1 < kWarps && id >= 0 && last_uid[w1] == id) ++w1;
        if (id >= 0) {
            const bool begins = (last_edge[w0] & 1) != 0;
            const bool whole = begins && (last_edge[w1 - 1] & 2);
            const Unit g = unit_of<R>(c, a, p, id);
            float *rec = p.records + (int64_t)(blockIdx.x * kWarps + w0) * 2 * R * (D + 2);
            for (int it = threadIdx.x; it < R * D; it += kThreads) {
                const int row = it / D, d = it % D;
                float top = -INFINITY, sum = 0.0f, acc = 0.0f;
                for (int w = w0; w < w1; ++w) top = fmaxf(top, sm[w * R + row]);
                for (int w = w0; w < w1; ++w) {
                    const float mw = sm[w * R + row];
                    const float f = mw > -INFINITY ? ex2(mw - top) : mw == mw ? 0.0f : mw;
                    sum = fmaf(f, sl[w * R + row], sum);
                    acc = fmaf(f, so[(w * R + row) * kRow + d], acc);
                }
                if (!whole) {
                    rec[row * D + d] = acc;
                    if (d == 0) rec[R * D + row] = top, rec[R * D + R + row] = sum;
                } else if (row < g.rows) {
                    store(static_cast<T *>(a.out) + (g.row + row) * D + d,
                          sum == 0.0f ? 0.0f : acc / sum);
                    if (d == 0 && a.lse)
                        a.lse[g.row + row] = (top + log2f(sum)) * 0.6931471805599453f;
                }
            }
            if (!whole && threadIdx.x == 0) {
                for (int w = w0; w < w1; ++w) {
                    p.head[blockIdx.x * kWarps + w] = id;
                    p.head[2 * kSlots + blockIdx.x * kWarps + w] =
                        (last_edge[w] & 2) | (w == w0 && begins ? 1 : 0);
                }
            }
        }
        w0 = w1;
    }
}

// Joins the partial results of the units that no CTA finished: block b takes
// the one that begins in warp part b, if there is one; a warp a row.
template <int D, int NT, bool F32>
__global__ void __launch_bounds__(256 * NT) join_kernel(Kv4 c, Kv4Attn a, Plan p) {
    constexpr int R = 8 * NT, V = D / 32;
    using T = typename std::conditional<F32, float, __nv_bfloat16>::type;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int b = blockIdx.x;
    if (!(p.head[2 * kSlots + b] & 1)) return;
    const int id = p.head[b];
    const Unit u = unit_of<R>(c, a, p, id);
    const int row = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // Records: this one, the first of every later CTA that has the unit, and
    // the end of the unit inside a part.
    float top = -INFINITY, sum = 0.0f, acc[V];
#pragma unroll
    for (int v = 0; v < V; ++v) acc[v] = 0.0f;
    auto add = [&](const float *rec) {
        const float mw = rec[R * D + row], lw = rec[R * D + R + row];
        float x[V];
#pragma unroll
        for (int v = 0; v < V; ++v) x[v] = rec[row * D + 32 * v + lane];
        const float t = fmaxf(top, mw);
        const float f = top > -INFINITY ? ex2(top - t) : 0.0f;
        const float g = mw > -INFINITY ? ex2(mw - t) : mw == mw ? 0.0f : mw;
        top = t;
        sum = fmaf(g, lw, sum * f);
#pragma unroll
        for (int v = 0; v < V; ++v) acc[v] = fmaf(g, x[v], acc[v] * f);
    };
    add(p.records + (int64_t)b * 2 * R * (D + 2));
    int cta = b / kWarps;  // the latest CTA whose record is in
    for (int s = b + 1; s < kSlots; ++s) {
        if (p.head[s] == id) {
            if (s / kWarps != cta) add(p.records + (int64_t)s * 2 * R * (D + 2));
            cta = s / kWarps;
            if (p.head[2 * kSlots + s] & 2) break;
        } else if (p.head[kSlots + s] == id) {
            add(p.records + ((int64_t)s * 2 + 1) * R * (D + 2));
            break;
        }  // else a part without tiles, between parts that have some
    }
    if (row >= u.rows) return;
    T *dst = static_cast<T *>(a.out) + (u.row + row) * D + lane;
#pragma unroll
    for (int v = 0; v < V; ++v) store(dst + 32 * v, sum == 0.0f ? 0.0f : acc[v] / sum);
    if (a.lse && lane == 0) a.lse[u.row + row] = (top + log2f(sum)) * 0.6931471805599453f;
}

template <int D, int NT, bool F32>
cudaError_t launch(const Kv4 &c, const Kv4Attn &a, const Plan &p, cudaStream_t stream) {
    constexpr int kRing = kWarps * (D == 128 ? 3 : 6) * kv4_half_bytes(D);
    constexpr int kJoin = kWarps * 8 * NT * (D + 4 + 2) * 4;
    constexpr int kBytes = kRing > kJoin ? kRing : kJoin;
    cudaError_t e = cudaFuncSetAttribute(few_kernel<D, NT, F32>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, kBytes);
    if (e != cudaSuccess) return e;
    few_kernel<D, NT, F32><<<kCtas, kThreads, kBytes, stream>>>(c, a, p);
    // The joining kernel is set up while this one runs (it waits for its end
    // before it reads anything).
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(kSlots);
    cfg.blockDim = dim3(256 * NT);
    cfg.stream = stream;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, join_kernel<D, NT, F32>, c, a, p);
    return e != cudaSuccess ? e : cudaGetLastError();
}

int stripe_rows(int64_t Hq, int64_t Hkv, int64_t Lq, bool lists) {
    return (int)(lists ? (Lq < kBlock ? Lq : kBlock) : Hq / Hkv * Lq);
}

}  // namespace

int64_t kv4_attn_few_work_bytes(int D) {
    return 3 * kSlots * 4 + (int64_t)kSlots * 2 * 16 * (D + 2) * 4;
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
    // A scale of 0 would turn masked scores (-inf) into NaN; this one leaves
    // every score below 2^-90.
    p.sc = fmaxf(fabsf(a.tau) * 1.4426950408889634f, 1e-37f);
    p.flip = a.tau < 0.0f ? 0x80008000u : 0u;
    p.head = static_cast<int32_t *>(a.work);
    p.records = reinterpret_cast<float *>(p.head + 3 * kSlots);
    if (c.D == 128) {
        if (f32) return launch<128, 1, true>(c, a, p, stream);
        return R == 8 ? launch<128, 1, false>(c, a, p, stream)
                      : launch<128, 2, false>(c, a, p, stream);
    }
    if (f32) return launch<64, 1, true>(c, a, p, stream);
    return R == 8 ? launch<64, 1, false>(c, a, p, stream) : launch<64, 2, false>(c, a, p, stream);
}

}  // namespace sparstar
