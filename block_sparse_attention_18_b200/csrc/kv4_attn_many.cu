// Attention of many query rows over the paged 4-bit key/value cache, bf16
// with head dim 128, on the 5th-generation tensor cores.
//
// The 128 x 128 tiles come from the pages in one of two ways:
//
//   unpacked first: a kernel of its own dequantises every page once (exactly,
//     to bf16) into scratch, as the 32 KB tiles in the 128-byte swizzle that
//     the MMAs read from shared memory, and the attention kernel's producer
//     fetches them with one bulk copy each.  64 KB a page and head are
//     written and, mostly from L2, read again: right where many query blocks
//     read the same pages.  The pipeline is attn_sm100.cu's: one CTA a pair
//     of query blocks A and B (128 rows each), whose scores share one TMEM
//     buffer in turn, with P in tensor memory as the A operand of O += P V.
//     Without block lists A and B are neighbouring blocks of the rows that
//     share a key head (the heads of a group lie one behind the other in q)
//     and walk the same pages: a tile serves 256 rows.  With lists each block
//     walks its own.
//   unpacked in place: the attention kernel brings the packed halves of the
//     pages into a small ring by bulk copies; six warps dequantise them from
//     there into the ring of tiles.  Only the packed bytes cross HBM: right for few
//     query blocks and long caches.  One query block a CTA.  Its softmax has
//     two threads a row, of 64 tokens of each tile, which never meet: each
//     half has its own maximum, sum and accumulator (O of tokens 0-63 and of
//     64-127 of every tile), joined at the end.  Two short chains a tile take
//     half the time of one long one, and 64 scores fit beside the rest in the
//     128 registers of sixteen warps.  One warp issues all products, polling
//     for whichever is ready.
//
// The roles' waits are modelled in tests/test_kv4_ring_protocol.py.
//
// Values lie channel by channel in a page, so both operands are K-major.  Few
// CTAs (short stripes, long caches) split the pages among several; a kernel
// of its own joins the results, in order.
//
// Bounds.  Unpacked first: the tensor and the exponential units in turn, as in
// attn_sm100.cu, and the power cap: 8,000 rows of 16 heads over 16,512 tokens,
// every block, take 796 us on a cool GPU (1.36 PFLOP/s) and 909 in a run of such
// calls; over lists of 83 of the 129 blocks 565 and 650 us, as attn_sm100.cu over
// the values themselves (572 and 650); 28 us of each unpack 135 MB (26 at HBM's
// rate).  In place: the unpacking warps, 1.43 us a page where the MMAs of one
// block need 0.5: 128 rows over 72,000 tokens, 16 heads, 113 to 128 us.
// Short calls: about 14 us of start, epilogue and joining beside the pages.
//
// How the work is cut follows the tables' widths wherever the device does not
// choose (see chooses): 128 rows over 16,512 tokens, 16 heads, take 42 us in
// tables of 129 pages, 63 of 258 and 207 of 1,200.
#include "kv4.cuh"
#include "sm100.cuh"

namespace sparstar {
namespace {

// Query blocks a CTA.
template <bool kPre>
constexpr int kBlocks = kPre ? 2 : 1;
// Warps 0-7: softmax, of blocks A and B or of both halves of the tiles.
// Unpacked first: 8 copies, 9 issues S = Q K^T, 10 O += P V.  In place: 8-13
// unpack, 14 copies, 15 issues both products.
template <bool kPre>
constexpr int kThreads = kPre ? 352 : 512;
template <bool kPre>
constexpr int kLoadWarp = kPre ? 8 : 14;   // Q, tiles or packed halves, barriers
template <bool kPre>
constexpr int kMmaWarp = kPre ? 9 : 15;    // TMEM, S = Q K^T
constexpr int kPvWarp = 10, kUnpackWarp = 8, kUnpackWarps = 6;
constexpr int kUnpackStrips = 3;  // of 16 strips of eight rows, a warp at most
constexpr uint32_t kTmemCols = 512;
// TMEM columns: S; P and O of block (or half) x, P of a half 32 columns.
constexpr uint32_t kColS = 0;
template <bool kPre>
__device__ constexpr uint32_t col_p(int x) {
    return 128u + (kPre ? 64u : 32u) * x;
}
__device__ constexpr uint32_t col_o(int x) { return 256u + 128u * x; }

constexpr int kOffQ = 0;
constexpr int kOffStage = 2 * kTileBytes;
// In place: packed halves of pages, where Q_B would be.
constexpr int kOffPacked = kTileBytes, kPackedStages = 3;
static_assert(kPackedStages * kv4_half_bytes(kHD) <= kTileBytes, "packed ring");
constexpr int kOffBar = kOffStage + kStages * kTileBytes;
struct Bars {
    uint64_t q_full;
    uint64_t st_full[kStages][2];  // [stage][use & 1], see ring_parity
    uint64_t st_empty[kStages];
    uint64_t packed_full[kPackedStages], packed_empty[kPackedStages];
    uint64_t s_full[2];  // S of block A, B; in place: [0]
    uint64_t s_free;
    uint64_t p_full[2][2];  // [block][half of the tile]; in place: [0][half]
    uint64_t pv_done[2];    // of a block, of a half
    uint64_t drain;
    uint32_t tmem_base;
    int32_t abort_flag;
    int32_t n_valid[2];
};
constexpr int kSmemBytes = kOffBar + (int)sizeof(Bars) + 1024;
static_assert(kSmemBytes <= 227 * 1024, "shared memory per CTA");
constexpr uint32_t kIdesc = make_idesc(false);  // both operands K-major

// Partial results of a CTA's rows, up to 256: maxima, sums, and accumulators
// as [kHD / 4][kBlock] fours, which the threads, a row each, store side by side.
constexpr int kPartFloats = kBlock * (kHD + 2);  // a query block
constexpr int kMaxParts = 4 * 148;  // units x splits, bounds the scratch
constexpr int kMaxSplits = 64;
// Scratch: the other kernel's zeros, the chosen chunk, what the joining kernel
// needs to know of each split unit, the parts, the tiles.
constexpr int kChosenBytes = 1024;
constexpr int kHeadBytes = SPARSTAR_KV4_WORK_ZEROS + kChosenBytes + kMaxParts * 16;

struct Plan {
    int heads;      // query heads a key head
    int rows;       // rows of a stripe
    int blocks;     // query blocks a unit: 2 unpacked first, 1 in place
    int per;        // units of a stripe
    int nqb;        // query blocks of a stripe
    int whole;      // units before this one run on one CTA each
    int splits;     // CTAs of each other unit; those behind its last page do nothing
    int chunk;      // entries (pages or list entries) a CTA
    int32_t *chosen;  // unpacked first, without lists: the chunk that the lengths ask for,
                      // then the sequences in order
    float sc;       // tau in log2 units, positive
    int4 *split_units;  // of each unit behind `whole`: parts, stripe, first query block
    int join_rows;  // rows a CTA of the joining kernel
    float *parts;
    uint8_t *tiles;  // unpacked first: [sequence][head][block] pairs of tiles
    int tile_blocks;
};
constexpr int kPairBytes = 2 * kTileBytes;  // a page's keys, then its values

// Whether the phase is complete, without the wait of mbar_test's try_wait.
__device__ __forceinline__ bool mbar_poll(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}
// The pages one query block walks.
struct Walk {
    const int32_t *list;   // block list, or null: every block
    const int32_t *table;  // the sequence's pages
    int lo, hi;            // entries of this CTA
    int blocks;            // blocks of the sequence
    int visible;           // blocks that some row of the query block sees
    int n_pages;
    // The block of an entry and its page; false for one that is skipped.
    __device__ bool at(int t, int &block, int &page) const {
        block = list ? __ldca(list + t) : t;
        if (block < 0 || block >= blocks || block >= visible) return false;
        page = __ldca(table + block);
        return page >= 0 && page < n_pages;
    }
    __device__ int next(int &cur, int &page) const {
        int block = 0;
        while (cur < hi)
            if (at(cur++, block, page)) return block;
        page = 0;
        return 0;  // past the last: callers count first
    }
};

// The blocks (or pages) of a stream of tiles, for the copying lane: the next key
// tile's, looked up ahead, the last key tile's and the one before, whose values
// follow.  A lookup between two copies costs as much as a fifth of a step.
template <bool kPages>
struct Stream {
    const Walk &w;
    const bool every;  // each entry counts
    int cur, next, last, before;
    __device__ Stream(const Walk &w, int n)
        : w(w), every(n == w.hi - w.lo), cur(w.lo), last(0), before(0) {
        next = ahead();
    }
    __device__ int ahead() {
        int page;
        if (!every) {
            const int block = w.next(cur, page);
            return kPages ? page : block;
        }
        if (cur >= w.hi) return 0;
        const int block = w.list ? __ldca(w.list + cur) : cur;
        ++cur;
        return kPages ? __ldca(w.table + block) : block;
    }
    __device__ int key() {
        before = last, last = next;
        next = ahead();
        return last;
    }
};

// Sequences that are put in order, units that are counted (choose_chunk).
constexpr int kOrdered = 240, kChosenUnits = 1024;

// A unit: one or two query blocks of a stripe, and what they walk.
struct Unit {
    int stripe, qb0, seq, kh, slot, L;
    int visible[2];  // blocks that some row of the query block sees
    int count[2];    // entries it walks
    int entries, chunk, parts;
};
// The last blocks of a stripe see most under a causal mask: they come first.
__device__ Unit unit_of(const Kv4 &c, const Kv4Attn &a, const Plan &p, int unit) {
    Unit u;
    u.stripe = unit / p.per;
    u.qb0 = p.blocks * (p.per - 1 - unit % p.per);
    const bool lists = a.kv_cnt != nullptr;
    const int per_seq = lists ? a.Hq : c.Hkv;
    u.seq = u.stripe / per_seq;
    if (p.chosen && a.n <= kOrdered) {  // the longest sequences first
        const int head = u.stripe - u.seq * per_seq;
        u.seq = __ldcg(p.chosen + 1 + u.seq);
        u.stripe = u.seq * per_seq + head;
    }
    u.kh = lists ? u.stripe % per_seq / p.heads : u.stripe % per_seq;
    u.slot = kv4_slot(c, a.seqs, u.seq);
    u.L = u.slot >= 0 ? kv4_len(c, u.slot) : 0;
#pragma unroll
    for (int x = 0; x < 2; ++x) {
        const int first = (u.qb0 + x) * kBlock;
        const int last = x < p.blocks ? min(first + kBlock, p.rows) - 1 : first - 1;
        int seen = u.L;  // by the row that sees most
        if (a.causal) {
            const int in = first % a.Lq + last - first;
            seen = u.L - a.Lq + 1 + (in >= a.Lq ? a.Lq - 1 : in);
        }
        u.visible[x] = last < first || seen <= 0 ? 0 : (seen + kBlock - 1) / kBlock;
        u.count[x] = u.visible[x];
        if (lists) {
            u.count[x] = 0;
            if (last >= first && u.slot >= 0) {
                const int cnt = __ldca(a.kv_cnt + (int64_t)u.stripe * p.nqb + first / kBlock);
                u.count[x] = cnt < 0 ? 0 : (cnt > a.max_sel ? a.max_sel : cnt);
            }
        }
    }
    u.entries = max(u.count[0], u.count[1]);
    u.chunk = p.chosen ? __ldcg(p.chosen) : p.chunk;
    u.parts = max(1, (u.entries + u.chunk - 1) / u.chunk);
    if (unit < p.whole) u.chunk = u.entries, u.parts = 1;
    return u;
}

// The cost of a call whose units' pages are cut into chunks, in steps of a
// pair of blocks over one page (1.55 us): a CTA takes about four steps beside
// its pages, and 1.5 more to store 133 KB where the results are joined, which
// takes 2.5 and 0.01 a CTA.  Equal CTAs run in waves; unequal
// ones follow each other and end about half a chunk apart.
__host__ __device__ inline float cost_of(float ctas, float chunk, float steps, bool joins,
                                         bool equal) {
    const float own = chunk + (joins ? 5.5f : 4.0f);
    const float join = joins ? 2.5f + 0.01f * ctas : 0.0f;
    if (equal || ctas <= 148.0f) return ceilf(ctas / 148.0f) * own + join;
    const float packed = (steps + (joins ? 5.5f : 4.0f) * ctas) / 148.0f + 0.5f * chunk;
    return fmaxf(own, packed) + join;
}

// The chunk for the lengths at hand (no lists): of 32 between the longest
// unit and its split into `splits`, the one of least cost; and the order of
// the sequences, the longest first, so that no long unit starts last.  One
// CTA of 256 threads.
__device__ void choose_chunk(const Kv4 &c, const Kv4Attn &a, const Plan &p) {
    constexpr int kTried = 32;
    __shared__ int32_t longest, ctas[kTried], entries[kChosenUnits], lens[kOrdered];
    __shared__ unsigned long long steps;
    if (threadIdx.x == 0) longest = 1, steps = 0;
    if (threadIdx.x < kTried) ctas[threadIdx.x] = 0;
    __syncthreads();
    // The key heads of a sequence have equal units: one stands for all.
    const int units = a.n * p.per;  // at most kChosenUnits
    Plan q = p;
    q.chosen = nullptr;
    for (int k = threadIdx.x; k < units; k += blockDim.x) {
        const Unit u = unit_of(c, a, q, k / p.per * c.Hkv * p.per + k % p.per);
        entries[k] = u.entries;
        if (k % p.per == 0 && u.seq < kOrdered) lens[u.seq] = u.L;
        atomicMax(&longest, u.entries);
        atomicAdd(&steps, (unsigned long long)u.entries);
    }
    __syncthreads();
    const int tried = threadIdx.x & (kTried - 1);
    const int least_chunk = max(2, (longest + p.splits - 1) / p.splits);
    const int chunk = longest - max(0, longest - least_chunk) * tried / (kTried - 1);
    int n = 0;
    for (int k = threadIdx.x / kTried; k < units; k += blockDim.x / kTried)
        n += max(1, (entries[k] + chunk - 1) / chunk);
    atomicAdd(&ctas[tried], n);
    if (a.n <= kOrdered)
        for (int i = threadIdx.x; i < a.n; i += blockDim.x) {
            int before = 0;
            for (int k = 0; k < a.n; ++k)
                before += lens[k] > lens[i] || (lens[k] == lens[i] && k < i);
            p.chosen[1 + before] = i;
        }
    __syncthreads();
    if (threadIdx.x < kTried) {
        const float all = (float)steps * c.Hkv;
        const bool equal = all >= 0.95f * (float)units * c.Hkv * longest;
        float cost = cost_of((float)ctas[tried] * c.Hkv, (float)chunk, all, chunk < longest,
                             equal);
        int best = chunk;
#pragma unroll
        for (int o = 16; o; o >>= 1) {  // the least cost, then the larger chunk
            const float other = __shfl_xor_sync(0xffffffffu, cost, o);
            const int its = __shfl_xor_sync(0xffffffffu, best, o);
            if (other < cost || (other == cost && its > best)) cost = other, best = its;
        }
        if (threadIdx.x == 0) *p.chosen = best;
    }
}

// Rows of a tile that a lane unpacks: 16 bytes of codes (32 columns from
// 32 g) of row q of strips of eight rows.  The four words go to four of the
// eight 16-byte columns of the row's 128-byte line in the tile's panel; lanes
// of the second panel take words 2, 3, 0, 1, so that the eight lanes of a
// store phase hit eight different columns.
struct Unpack {
    uint32_t off[4];  // byte of word i of strip 0
    uint32_t turn;
    uint32_t magic, sixteen;
    __device__ explicit Unpack(int lane) {
        const int g = lane & 3, q = lane >> 2;
        turn = g & 2;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            off[i] = (uint32_t)((g >> 1) * kPanelBytes + q * 128 +
                                ((((g & 1) * 4 + (i ^ (int)turn)) ^ q) << 4));
        magic = kv4_opaque(kMagic), sixteen = kv4_opaque(16);
    }
    // One row's 32 keys: put(byte in the tile, 16 bytes).
    template <typename Put>
    __device__ void keys(const uint4 &code, uint32_t scale, int strip, Put put) const {
        const uint32_t s = kv4_scale_pair(scale * 0x10001u, sixteen), m = kv4_minus136(s);
        const uint32_t w[4] = {turn ? code.z : code.x, turn ? code.w : code.y,
                               turn ? code.x : code.z, turn ? code.y : code.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint32_t o[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) o[k] = kv4_dequant(kv4_pair128(w[i], k, magic), s, m);
            put(off[i] + strip * 1024, make_uint4(o[0], o[1], o[2], o[3]));
        }
    }
    // Scales of the 32 tokens of the lane's columns, in pairs: 16, ready.
    struct Pairs {
        uint32_t s[16], m[16];
    };
    __device__ void pairs(const uint4 &b0, const uint4 &b1, Pairs &p) const {
        const uint32_t b[8] = {turn ? b1.x : b0.x, turn ? b1.y : b0.y, turn ? b1.z : b0.z,
                               turn ? b1.w : b0.w, turn ? b0.x : b1.x, turn ? b0.y : b1.y,
                               turn ? b0.z : b1.z, turn ? b0.w : b1.w};
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            p.s[i] = kv4_scale_pair(__byte_perm(b[i / 2], 0, (i & 1) ? 0x4342 : 0x4140), sixteen);
            p.m[i] = kv4_minus136(p.s[i]);
        }
    }
    // One channel's 32 values.
    template <typename Put>
    __device__ void values(const uint4 &code, const Pairs &p, int strip, Put put) const {
        const uint32_t w[4] = {turn ? code.z : code.x, turn ? code.w : code.y,
                               turn ? code.x : code.z, turn ? code.y : code.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint32_t o[4];
#pragma unroll
            for (int k = 0; k < 4; ++k)
                o[k] = kv4_dequant(kv4_pair128(w[i], k, magic), p.s[4 * i + k], p.m[4 * i + k]);
            put(off[i] + strip * 1024, make_uint4(o[0], o[1], o[2], o[3]));
        }
    }
};

// Unpacked first: one CTA a page and head of every sequence; four warps the
// keys, four the values, 32 rows each.  The tiles leave through shared memory
// by bulk copies: 28 us for 2,064 pages and heads, 41 with 16-byte stores, which
// the swizzle scatters over half sectors.
__global__ void __launch_bounds__(256) unpack_kernel(Kv4 c, Kv4Attn a, Plan p) {
    kv4_begin();
    if (p.chosen && blockIdx.x == gridDim.x - 1) {  // one CTA behind the pages'
        choose_chunk(c, a, p);
        return;
    }
    const int kh = blockIdx.x % c.Hkv;
    const int block = blockIdx.x / c.Hkv % p.tile_blocks, seq = blockIdx.x / c.Hkv / p.tile_blocks;
    const int slot = kv4_slot(c, a.seqs, seq);
    if (slot < 0 || block * kBlock >= kv4_len(c, slot)) return;
    const int page = __ldca(c.table + (int64_t)slot * c.max_pages + block);
    if (page < 0 || page >= c.n_pages) return;  // the attention kernel says so
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, w = warp & 3;
    const int g = lane & 3, q = lane >> 2;
    const bool values = warp >= 4;
    const uint8_t *half = c.pages + ((int64_t)page * c.Hkv + kh) * kv4_page_bytes(kHD) +
                          (values ? kv4_half_bytes(kHD) : 0);
    const uint8_t *s = half + kv4_code_bytes(kHD);
    uint4 code[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        code[i] = __ldca(reinterpret_cast<const uint4 *>(half) + (32 * w + 8 * i + q) * 4 + g);
    extern __shared__ __align__(128) uint8_t pair[];
    uint8_t *tile = pair + (values ? kTileBytes : 0);
    auto put = [&](uint32_t at, const uint4 &v) { *reinterpret_cast<uint4 *>(tile + at) = v; };
    const Unpack u(lane);
    if (values) {
        Unpack::Pairs pairs;
        const uint4 *sv = reinterpret_cast<const uint4 *>(s + w * kBlock + 32 * g);
        u.pairs(__ldca(sv), __ldca(sv + 1), pairs);
#pragma unroll
        for (int i = 0; i < 4; ++i) u.values(code[i], pairs, 4 * w + i, put);
    } else {
        uint32_t scale[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) scale[i] = __ldca(s + (32 * w + 8 * i + q) * 4 + g);
#pragma unroll
        for (int i = 0; i < 4; ++i) u.keys(code[i], scale[i], 4 * w + i, put);
    }
    // A warp's rows are 4 KB of each panel.
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    __syncwarp();
    if (lane < 2) {
        const int at = (values ? kTileBytes : 0) + lane * kPanelBytes + w * 4096;
        asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(
                         p.tiles +
                         (((int64_t)seq * c.Hkv + kh) * p.tile_blocks + block) * kPairBytes + at),
                     "r"(smem_addr(pair + at)), "r"(4096)
                     : "memory");
        asm volatile("cp.async.bulk.commit_group;" ::: "memory");
        asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
    }
}

template <bool kPre>
__global__ void __launch_bounds__(kThreads<kPre>, 1)
    many_kernel(const __grid_constant__ CUtensorMap tmQ, Kv4 c, Kv4Attn a, Plan p) {
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw_addr = smem_addr(smem_raw);
    const uint32_t base = (raw_addr + 1023u) & ~1023u;
    uint8_t *smem = smem_raw + (base - raw_addr);
    Bars *bars = reinterpret_cast<Bars *>(smem + kOffBar);
    volatile int32_t *abort_flag = &bars->abort_flag;
    int32_t *status = a.status;
    const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;

    // This CTA's pair of query blocks and part of their pages.
    kv4_begin();
    const int tail = (int)blockIdx.x - p.whole;  // CTA of the split units
    const int split = tail < 0 ? 0 : tail % p.splits;
    const Unit un = unit_of(c, a, p, tail < 0 ? blockIdx.x : p.whole + tail / p.splits);
    const int stripe = un.stripe, qb0 = un.qb0, L = un.L;
    const int seq = un.seq, kh = un.kh;
    const bool lists = a.kv_cnt != nullptr;
    if (un.slot < 0 && threadIdx.x == 0) kv4_flag(status, SPARSTAR_STATUS_BAD_INDEX);
    if (split >= un.parts) return;
    if (p.splits > 1 && tail >= 0 && split == 0 && threadIdx.x == 0)
        p.split_units[tail / p.splits] = make_int4(un.parts, stripe, qb0, 0);
    const bool joins = un.parts > 1;  // the result goes to `parts`
    Walk walk[2];
    {
        const int lo = split * un.chunk, hi = min(lo + un.chunk, un.entries);
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            Walk &w = walk[x];
            w.list = lists ? a.kv_idx + ((int64_t)stripe * p.nqb + qb0 + x) * a.max_sel
                           : nullptr;
            w.table = c.table + (int64_t)(un.slot >= 0 ? un.slot : 0) * c.max_pages;
            w.blocks = (L + kBlock - 1) / kBlock;
            w.n_pages = c.n_pages;
            w.visible = un.visible[x];
            w.lo = lo;
            w.hi = max(lo, min(hi, un.count[x]));
        }
    }

    const uint32_t bar_q = smem_addr(&bars->q_full);
    auto bar_full = [&](int e) {
        return smem_addr(&bars->st_full[e % kStages][(e / kStages) & 1]);
    };
    auto bar_empty = [&](int s) { return smem_addr(&bars->st_empty[s]); };
    auto bar_s = [&](int x) { return smem_addr(&bars->s_full[x]); };
    const uint32_t bar_sfree = smem_addr(&bars->s_free);
    auto bar_p = [&](int x, int h) { return smem_addr(&bars->p_full[x][h]); };
    auto bar_pv = [&](int x) { return smem_addr(&bars->pv_done[x]); };
    const uint32_t bar_drain = smem_addr(&bars->drain);

    if (warp == kLoadWarp<kPre>) {
        if (lane == 0) {
            mbar_init(bar_q, 1);
            for (int s = 0; s < kStages; ++s) {
                mbar_init(smem_addr(&bars->st_full[s][0]), kPre ? 1 : kUnpackWarps);
                mbar_init(smem_addr(&bars->st_full[s][1]), kPre ? 1 : kUnpackWarps);
                mbar_init(bar_empty(s), 1);
            }
            for (int s = 0; s < kPackedStages; ++s) {
                mbar_init(smem_addr(&bars->packed_full[s]), 1);
                mbar_init(smem_addr(&bars->packed_empty[s]), kUnpackWarps);
            }
            mbar_init(bar_sfree, kPre ? kBlock : 2 * kBlock);  // the readers of one S
            for (int x = 0; x < 2; ++x) {
                mbar_init(bar_s(x), 1);
                for (int h = 0; h < 2; ++h) mbar_init(bar_p(x, h), kBlock);
                mbar_init(bar_pv(x), 1);
            }
            mbar_init(bar_drain, kPre ? 2 : 1);
            bars->abort_flag = 0;
            asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        }
#pragma unroll
        for (int x = 0; x < kBlocks<kPre>; ++x) {
            int nv = 0;
            bool bad = false;
            for (int t = walk[x].lo + lane; t < walk[x].hi; t += 32) {
                int block, page;
                const bool v = walk[x].at(t, block, page);
                nv += (int)v;
                // A listed block that no row sees is no error.
                bad |= !v && !(block >= walk[x].visible && block < walk[x].blocks);
            }
            if (bad) kv4_flag(status, SPARSTAR_STATUS_BAD_INDEX);
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) nv += __shfl_xor_sync(0xffffffffu, nv, o);
            if (lane == 0) bars->n_valid[x] = nv;
        }
    }
    if (warp == kMmaWarp<kPre>) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                         smem_addr(&bars->tmem_base)),
                     "r"(kTmemCols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = bars->tmem_base;
    const int nA = bars->n_valid[0], nB = kPre ? bars->n_valid[1] : 0;
    const int nmax = nA > nB ? nA : nB;
    // Ring streams: the tiles of A and of B, or one stream for both.
    const bool apart = lists;
    const int sA = apart ? nA : nmax, sB = apart ? nB : 0;
    auto k_slot = [&](int x, int j) { return slot_k(apart ? x : 0, j, sA, sB); };
    auto v_slot = [&](int x, int j) { return slot_v(apart ? x : 0, j, sA, sB); };

    auto bar_packed = [&](int s) { return smem_addr(&bars->packed_full[s]); };
    auto bar_unpacked = [&](int s) { return smem_addr(&bars->packed_empty[s]); };
    auto load_q = [&]() {  // by one lane
        const uint64_t pol = policy_evict_first();
        const int nq = nB > 0 ? 2 : 1;
        mbar_expect_tx(bar_q, nq * kTileBytes);
        for (int x = 0; x < nq; ++x) {
            const uint32_t sQ = base + kOffQ + x * kTileBytes;
            const int row = (qb0 + x) * kBlock;
            tma_load_3d(sQ, &tmQ, bar_q, 0, row, stripe, pol);
            tma_load_3d(sQ + kPanelBytes, &tmQ, bar_q, 64, row, stripe, pol);
        }
    };
    const uint64_t dQ0 = desc_k_major(base + kOffQ);
    const uint64_t dQ1 = desc_k_major(base + kOffQ + kTileBytes);
    // S = Q_x K^T of step j, ring slot e; a shared tile is free after its last
    // reader.
    auto issue_qk = [&](int x, int j, int e) {
        const int stage = e % kStages;
        const uint64_t dK = desc_k_major(base + kOffStage + stage * kTileBytes);
        const uint64_t dQ = x == 0 ? dQ0 : dQ1;
        const bool frees = apart || x == 1 || j >= nB;
        tc_fence_after();
        if (elect_one()) {
#pragma unroll
            for (int kk = 0; kk < kHD / 16; ++kk) {
                const uint64_t o = (uint64_t)(((kk >> 2) * kPanelBytes + (kk & 3) * 32) >> 4);
                mma_ss(tmem + kColS, dQ + o, dK + o, kIdesc, kk > 0 ? 1u : 0u);
            }
            if (frees) mma_commit(bar_empty(stage));
            mma_commit(bar_s(x));
        }
        __syncwarp();
    };
    // O += P V over tokens 64 h .. 64 h + 63 of ring slot e: of block x, or of
    // half h.
    auto issue_pv = [&](int x, int j, int h, int e) {
        const int stage = e % kStages;
        const uint64_t dV = desc_k_major(base + kOffStage + stage * kTileBytes);
        const bool frees = apart || x == 1 || j >= nB;
        const uint32_t dO = tmem + col_o(kPre ? x : h);
        const uint32_t aP = tmem + (kPre ? col_p<kPre>(x) + 32u * h : col_p<kPre>(h));
        const bool fresh = j == 0 && (!kPre || h == 0);
        tc_fence_after();
        if (elect_one()) {
#pragma unroll
            for (int kq = 0; kq < 4; ++kq) {
                const uint64_t o = (uint64_t)((h * kPanelBytes + kq * 32) >> 4);
                mma_ts(dO, aP + 8u * kq, dV + o, kIdesc, fresh && kq == 0 ? 0u : 1u);
            }
            if (h == 1 && frees) mma_commit(bar_empty(stage));
            if (!kPre) mma_commit(bar_pv(h));
            else if (h == 1) mma_commit(bar_pv(x));
        }
        __syncwarp();
    };

    if (kPre && warp == kLoadWarp<kPre>) {
        // ---------------------------------------------------- copying warp
        if (lane == 0 && nmax > 0) {
            load_q();
            const uint8_t *tiles =
                p.tiles + ((int64_t)seq * c.Hkv + kh) * p.tile_blocks * kPairBytes;
            // The stream whose pages A and B share is the longer one's.
            const Walk wa = !apart && nB > nA ? walk[1] : walk[0];
            Stream<false> A(wa, sA), B(walk[1], sB);
            int e = 0;
            bool ok = true;
            auto load = [&](int block, int is_v) {
                if (!ok) return;
                const int stage = e % kStages;
                ok = wait1(bar_empty(stage), ((uint32_t)(e / kStages) & 1u) ^ 1u, abort_flag,
                           status);
                if (!ok) return;
                mbar_expect_tx(bar_full(e), kTileBytes);
                const uint8_t *src = tiles + (int64_t)block * kPairBytes + is_v * kTileBytes;
                if (!a.withhold)
                    asm volatile(
                        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], "
                        "[%1], %2, [%3];" ::"r"(base + kOffStage + stage * kTileBytes),
                        "l"(src), "r"(kTileBytes), "r"(bar_full(e))
                        : "memory");
                ++e;
            };
            if (sA > 0) load(A.key(), 0);
            if (sB > 0) load(B.key(), 0);
            for (int j = 0; j < max(sA, sB) && ok; ++j) {
                if (j + 1 < sA) load(A.key(), 0);
                if (j < sA) load(j + 1 < sA ? A.before : A.last, 1);
                if (j + 1 < sB) load(B.key(), 0);
                if (j < sB) load(j + 1 < sB ? B.before : B.last, 1);
            }
            // Copies in flight land before the CTA may exit.
            drain_wait(bar_q, 0);
            for (int i = e > kStages ? e - kStages : 0; i < e; ++i)
                drain_wait(bar_full(i), ring_parity(i));
        }
    } else if (kPre && warp == kMmaWarp<kPre>) {
        // -------------------------------------------- S = Q K^T MMA issuer
        bool ok = nmax > 0 && wait_warp(bar_q, 0, abort_flag, status);
        int n = 0;
        for (int j = 0; j < nmax && ok; ++j) {
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                if (!ok || j >= (x == 0 ? nA : nB)) continue;
                const int e = k_slot(x, j);
                ok = wait_warp(bar_full(e), ring_parity(e), abort_flag, status) &&
                     (n == 0 ||
                      wait_warp(bar_sfree, (uint32_t)(n - 1) & 1u, abort_flag, status));
                if (!ok) break;
                issue_qk(x, j, e);
                ++n;
            }
        }
        if (nmax > 0) {
            if (elect_one()) mma_commit(bar_drain);
            __syncwarp();
        }
    } else if (kPre && warp == kPvWarp) {
        // ---------------------------------------------- O += P V MMA issuer
        bool ok = nmax > 0;
        for (int j = 0; j < nmax && ok; ++j) {
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                if (!ok || j >= (x == 0 ? nA : nB)) continue;
                const int e = v_slot(x, j);
                ok = wait_warp(bar_p(x, 0), (uint32_t)j & 1u, abort_flag, status) &&
                     wait_warp(bar_full(e), ring_parity(e), abort_flag, status);
                if (!ok) break;
                issue_pv(x, j, 0, e);
                ok = wait_warp(bar_p(x, 1), (uint32_t)j & 1u, abort_flag, status);
                if (!ok) break;
                issue_pv(x, j, 1, e);
            }
        }
        if (nmax > 0) {
            if (elect_one()) mma_commit(bar_drain);
            __syncwarp();
            if (lane == 0) drain_wait(bar_drain, 0);
        }
        __syncwarp();
    } else if (!kPre && warp == kLoadWarp<kPre>) {
        // ------------------------------- copying warp: Q, packed halves
        if (lane == 0 && nmax > 0) {
            load_q();
            constexpr int kHalf = kv4_half_bytes(kHD);
            Stream<true> pages(walk[0], nA);
            int e = 0;
            bool ok = true;
            auto load = [&](int page, int is_v) {
                if (!ok) return;
                const int s = e % kPackedStages;
                ok = wait1(bar_unpacked(s), ((uint32_t)(e / kPackedStages) & 1u) ^ 1u, abort_flag,
                           status);
                if (!ok) return;
                mbar_expect_tx(bar_packed(s), kHalf);
                const uint8_t *src =
                    c.pages + ((int64_t)page * c.Hkv + kh) * (2 * kHalf) + is_v * kHalf;
                if (!a.withhold)
                    asm volatile(
                        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], "
                        "[%1], %2, [%3];" ::"r"(base + kOffPacked + s * kHalf),
                        "l"(src), "r"(kHalf), "r"(bar_packed(s))
                        : "memory");
                ++e;
            };
            load(pages.key(), 0);
            for (int j = 0; j < nA && ok; ++j) {
                if (j + 1 < nA) load(pages.key(), 0);
                load(j + 1 < nA ? pages.before : pages.last, 1);
            }
            // Copies in flight land before the CTA may exit.
            drain_wait(bar_q, 0);
            for (int i = e > kPackedStages ? e - kPackedStages : 0; i < e; ++i)
                drain_wait(bar_packed(i % kPackedStages), (uint32_t)(i / kPackedStages) & 1u);
        }
    } else if (!kPre && warp == kMmaWarp<kPre>) {
        // ----------------------- both products, whichever is ready next
        bool ok = nmax > 0 && wait_warp(bar_q, 0, abort_flag, status);
        auto ready = [&](uint32_t bar, uint32_t parity) {
            return __all_sync(0xffffffffu, mbar_poll(bar, parity));
        };
        // The next S (step qj) and the next half of O (step vj).
        int qj = 0, vj = 0, vh = 0;
        uint64_t idle = globaltimer();
        while (ok && vj < nA) {
            bool moved = false;
            if (qj < nA) {
                const int e = k_slot(0, qj);
                if (ready(bar_full(e), ring_parity(e)) &&
                    (qj == 0 || ready(bar_sfree, (uint32_t)(qj - 1) & 1u))) {
                    issue_qk(0, qj, e);
                    ++qj;
                    moved = true;
                }
            }
            const int e = v_slot(0, vj);
            if (ready(bar_p(0, vh), (uint32_t)vj & 1u) &&
                (vh > 0 || ready(bar_full(e), ring_parity(e)))) {
                issue_pv(0, vj, vh, e);
                vh ^= 1;
                if (vh == 0) ++vj;
                moved = true;
            }
            if (moved) {
                idle = globaltimer();
            } else {
                int give_up = 0;
                if (lane == 0) {
                    if (*abort_flag) {
                        give_up = 1;
                    } else if (globaltimer() - idle > kTimeoutNs) {
                        *abort_flag = 1;
                        kv4_flag(status, SPARSTAR_STATUS_TIMEOUT);
                        give_up = 1;
                    }
                }
                ok = __shfl_sync(0xffffffffu, give_up, 0) == 0;
            }
        }
        if (nmax > 0) {
            if (elect_one()) mma_commit(bar_drain);
            __syncwarp();
            if (lane == 0) drain_wait(bar_drain, 0);
        }
        __syncwarp();
    } else if (!kPre && warp >= kUnpackWarp) {
        // ------------------------------------------------- unpacking warps
        // 16 strips of eight rows: three each, the last two warps two; in two
        // groups of channels at most (a group is four strips).
        const int w = warp - kUnpackWarp, g = lane & 3, q = lane >> 2;
        const int strip0 = w < 5 ? 3 * w : 14, strips = w < 4 ? 3 : 2;
        const int in_first = 4 - (strip0 & 3);  // strips of the first group
        const Unpack u(lane);
        constexpr int kHalf = kv4_half_bytes(kHD);
        for (int e = 0; e < 2 * nA; ++e) {  // K 0, K 1, V 0, K 2, V 1, .. V n - 1
            const bool is_v = e > 0 && (e % 2 == 0 || e == 2 * nA - 1);
            const int s = e % kPackedStages, stage = e % kStages;
            if (!wait_warp(bar_packed(s), (uint32_t)(e / kPackedStages) & 1u, abort_flag, status))
                break;
            const uint8_t *half = smem + kOffPacked + s * kHalf;
            const uint8_t *scales = half + kv4_code_bytes(kHD);
            uint4 code[kUnpackStrips];
#pragma unroll
            for (int i = 0; i < kUnpackStrips; ++i)
                if (i < strips)
                    code[i] =
                        reinterpret_cast<const uint4 *>(half)[((strip0 + i) * 8 + q) * 4 + g];
            if (!wait_warp(bar_empty(stage), ((uint32_t)(e / kStages) & 1u) ^ 1u, abort_flag,
                           status))
                break;
            const uint32_t dst = base + kOffStage + stage * kTileBytes;
            auto put = [&](uint32_t at, const uint4 &v) {
                asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(dst + at),
                             "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w));
            };
            if (is_v) {
                auto pairs_of = [&](int group, Unpack::Pairs &pairs) {
                    const uint4 *sv =
                        reinterpret_cast<const uint4 *>(scales + group * kBlock + 32 * g);
                    u.pairs(sv[0], sv[1], pairs);
                };
                Unpack::Pairs pairs;
                pairs_of(strip0 >> 2, pairs);
#pragma unroll
                for (int i = 0; i < kUnpackStrips; ++i) {
                    if (i >= strips) break;
                    if (i == in_first) pairs_of((strip0 >> 2) + 1, pairs);
                    u.values(code[i], pairs, strip0 + i, put);
                }
            } else {
#pragma unroll
                for (int i = 0; i < kUnpackStrips; ++i)
                    if (i < strips)
                        u.keys(code[i], scales[((strip0 + i) * 8 + q) * 4 + g], strip0 + i, put);
            }
            // The MMAs read through the async proxy.
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(bar_full(e));
                mbar_arrive(bar_unpacked(s));
            }
        }
    } else {
        // ------------------------------- softmax + epilogue (128 per block)
        constexpr int kCols = kPre ? kBlock : kBlock / 2;  // tokens of a tile a thread has
        const int x = warp >> 2;  // block, or half of the tiles
        const int quarter = warp & 3;
        const int row = quarter * 32 + lane;
        const uint32_t lane_base = (uint32_t)(quarter * 32) << 16;
        const uint32_t colO = col_o(x), colP = col_p<kPre>(x);
        const int col0 = kPre ? 0 : kCols * x;
        const int nx = !kPre || x == 0 ? nA : nB;
        const float sc = p.sc;
        const Walk wx = !kPre || x == 0 ? walk[0] : walk[1];
        const int grow = (qb0 + (kPre ? x : 0)) * kBlock + row;  // of the stripe
        const bool real = grow < p.rows;
        // Tokens the row sees; a tile is masked where a row sees part of it.
        const int seen = a.causal ? L - a.Lq + 1 + grow % a.Lq : L;
        const bool plain = nx == wx.hi - wx.lo;  // every entry counts
        float m_ref = -INFINITY, l = 0.0f;
        bool ok = true;
        int cur = wx.lo;
        for (int j = 0; j < nx; ++j) {
            int kb, page;
            if (plain) kb = wx.list ? __ldca(wx.list + wx.lo + j) : wx.lo + j;
            else kb = wx.next(cur, page);
            if (!wait_warp(bar_s(kPre ? x : 0), (uint32_t)j & 1u, abort_flag, status)) {
                ok = false;
                break;
            }
            tc_fence_after();
            float s[kCols];
            {
                uint32_t r[kCols / 32][32];
#pragma unroll
                for (int q = 0; q < kCols / 32; ++q)
                    tmem_ld32(tmem + lane_base + kColS + col0 + 32 * q, r[q]);
                tmem_wait_ld();
#pragma unroll
                for (int q = 0; q < kCols / 32; ++q) reg_fence(r[q]);
#pragma unroll
                for (int q = 0; q < kCols / 32; ++q)
#pragma unroll
                    for (int u = 0; u < 32; ++u) s[32 * q + u] = __uint_as_float(r[q][u]);
            }
            tc_fence_before();
            mbar_arrive(bar_sfree);
            const int valid = seen - kb * kBlock - col0;
            if (__any_sync(0xffffffffu, valid < kCols)) {
#pragma unroll
                for (int q = 0; q < kCols; ++q)
                    if (q >= valid) s[q] = -INFINITY;
            }
            float mx[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
            for (int q = 4; q + 8 <= kCols; q += 8) {
#pragma unroll
                for (int t = 0; t < 4; ++t) mx[t] = max3f(mx[t], s[q + t], s[q + 4 + t]);
            }
#pragma unroll
            for (int t = 0; t < 4; ++t) mx[t] = fmaxf(mx[t], s[kCols - 4 + t]);
            const float m_tile = max3f(mx[0], mx[1], fmaxf(mx[2], mx[3])) * sc;
            const float m_new = fmaxf(m_ref, m_tile);
            bool pv_seen = false;
            if (__any_sync(0xffffffffu, m_new > m_ref + 8.0f)) {
                if (j > 0) {
                    if (!wait_warp(bar_pv(x), (uint32_t)(j - 1) & 1u, abort_flag, status)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    pv_seen = true;
                    const float f = m_new > -INFINITY ? ex2(m_ref - m_new) : 1.0f;
#pragma unroll 1
                    for (int q = 0; q < kHD / 8; ++q) {
                        uint32_t r[8];
                        tmem_ld8(tmem + lane_base + colO + 8 * q, r);
                        tmem_wait_ld();
                        asm volatile("" : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]),
                                     "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]));
#pragma unroll
                        for (int u = 0; u < 8; ++u)
                            r[u] = __float_as_uint(__uint_as_float(r[u]) * f);
                        tmem_st8(tmem + lane_base + colO + 8 * q, r);
                    }
                    tmem_wait_st();
                }
                if (m_new > -INFINITY) {
                    l *= ex2(m_ref - m_new);
                    m_ref = m_new;
                }
            }
            const float neg_m = m_ref > -INFINITY ? -m_ref : 0.0f;
            if (j > 0 && !pv_seen) {
                if (!wait_warp(bar_pv(x), (uint32_t)(j - 1) & 1u, abort_flag, status)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
            }
            const float2 sc2 = make_float2(sc, sc), nm2 = make_float2(neg_m, neg_m);
            float ls[4] = {0.f, 0.f, 0.f, 0.f};
            uint32_t pk[kCols / 2];
#pragma unroll
            for (int h = 0; h < kCols / 64; ++h) {
#pragma unroll
                for (int u = 32 * h; u < 32 * h + 32; u += 2) {
                    const int q = 2 * u;
                    const float2 x01 = __ffma2_rn(make_float2(s[q], s[q + 1]), sc2, nm2);
                    const float2 x23 = __ffma2_rn(make_float2(s[q + 2], s[q + 3]), sc2, nm2);
                    const float2 p01 = make_float2(ex2(x01.x), ex2(x01.y));
                    const float2 p23 = make_float2(ex2(x23.x), ex2(x23.y));
                    ls[0] += p01.x;
                    ls[1] += p01.y;
                    ls[2] += p23.x;
                    ls[3] += p23.y;
                    pk[u] = pack_bf16(p01.x, p01.y);
                    pk[u + 1] = pack_bf16(p23.x, p23.y);
                }
                tmem_st32(tmem + lane_base + colP + 32 * h, pk + 32 * h);
                tmem_wait_st();
                tc_fence_before();
                mbar_arrive(kPre ? bar_p(x, h) : bar_p(0, x));
            }
            l += (ls[0] + ls[1]) + (ls[2] + ls[3]);
        }

        // ---- epilogue
        bool have = nx > 0 && ok &&
                    wait_warp(bar_pv(x), (uint32_t)(nx - 1) & 1u, abort_flag, status);
        if (have) tc_fence_after();
        float fa = 1.0f, fb = 0.0f;  // weights of this half and the other
        float *other = reinterpret_cast<float *>(smem + kOffStage) + row * (kHD + 4);
        if constexpr (!kPre) {
            // The second half's results pass through the ring, which nobody
            // reads any more, to the first half's threads.
            float *rest = reinterpret_cast<float *>(smem + kOffStage) + kBlock * (kHD + 4);
            if (x == 1) {
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    uint32_t r[32];
                    if (have) {
                        tmem_ld32(tmem + lane_base + colO + 32 * q, r);
                        tmem_wait_ld();
                        reg_fence(r);
#pragma unroll
                        for (int u = 0; u < 8; ++u)
                            reinterpret_cast<uint4 *>(other + 32 * q)[u] =
                                make_uint4(r[4 * u], r[4 * u + 1], r[4 * u + 2], r[4 * u + 3]);
                    }
                }
                rest[row] = m_ref, rest[kBlock + row] = l;
                rest[2 * kBlock + row] = have ? 1.0f : 0.0f;
            }
            asm volatile("bar.sync 1, %0;" ::"n"(2 * kBlock) : "memory");
            if (x == 0 && have) {
                const float mb = rest[row], lb = rest[kBlock + row];
                have = rest[2 * kBlock + row] != 0.0f;
                const float top = fmaxf(m_ref, mb);
                fa = m_ref > -INFINITY ? ex2(m_ref - top) : 0.0f;
                fb = mb > -INFINITY ? ex2(mb - top) : 0.0f;
                l = l * fa + lb * fb;
                m_ref = top;
            }
            have = __all_sync(0xffffffffu, have);
        }
        const int64_t out_row = (int64_t)stripe * p.rows + grow;
        float *part = p.parts + (int64_t)(joins ? tail * kBlocks<kPre> + (kPre ? x : 0) : 0) *
                                    kPartFloats;
        uint4 *part_o = reinterpret_cast<uint4 *>(part + 2 * kBlock) + row;
        // A row without a weight (no token seen) gets 0.
        const float inv = l == 0.0f ? 0.0f : 1.0f / l;
        if (kPre || x == 0) {
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                uint32_t r[32];
#pragma unroll
                for (int u = 0; u < 32; ++u) r[u] = 0;
                if (have) {
                    tmem_ld32(tmem + lane_base + colO + 32 * q, r);
                    tmem_wait_ld();
                    reg_fence(r);
                    if constexpr (!kPre) {
#pragma unroll
                        for (int u = 0; u < 8; ++u) {
                            const float4 b = reinterpret_cast<const float4 *>(other + 32 * q)[u];
                            const float v[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                r[4 * u + k] = __float_as_uint(
                                    fmaf(fb, v[k], fa * __uint_as_float(r[4 * u + k])));
                        }
                    }
                }
                if (!real || (nx > 0 && !have)) continue;
                if (joins) {
#pragma unroll
                    for (int u = 0; u < 8; ++u)
                        part_o[(8 * q + u) * kBlock] =
                            make_uint4(r[4 * u], r[4 * u + 1], r[4 * u + 2], r[4 * u + 3]);
                } else {
                    uint4 *o4 = reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(a.out) +
                                                          out_row * kHD + 32 * q);
#pragma unroll
                    for (int u = 0; u < 4; ++u) {
                        uint32_t v[4];
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            v[k] = nx == 0
                                       ? 0u
                                       : pack_bf16(__uint_as_float(r[8 * u + 2 * k]) * inv,
                                                   __uint_as_float(r[8 * u + 2 * k + 1]) * inv);
                        __stcs(o4 + u, make_uint4(v[0], v[1], v[2], v[3]));
                    }
                }
            }
            if (joins) {
                part[row] = m_ref;
                part[kBlock + row] = l;
            } else if (real && a.lse && (nx == 0 || have)) {
                a.lse[out_row] = (m_ref + log2f(l)) * 0.6931471805599453f;
            }
        }
    }

    tc_fence_before();
    __syncthreads();
    if (warp == kMmaWarp<kPre>) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem),
                     "r"(kTmemCols)
                     : "memory");
    }
}

// Joins the parts of every row, in order: the weights first (a row and part a
// thread), then eight rows a step, four channels of one a thread.  Eight rows
// side by side are 128 bytes of a part; 32 bytes of a row's result are stored
// together.
__global__ void __launch_bounds__(256) many_join_kernel(Kv4Attn a, Plan p) {
    // Four parts at a time: most units have two to four (eight: 12.9 against
    // 10.2 us for 96 units of about three).
    constexpr int kMostRows = 32, kTogether = 4;
    __shared__ float weight[kMostRows][kMaxSplits + 1], inverse[kMostRows];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rows = p.blocks * kBlock;  // of a unit
    const int at = blockIdx.x / (rows / p.join_rows);
    const int r0 = blockIdx.x % (rows / p.join_rows) * p.join_rows;  // within one block
    kv4_begin();
    const int4 u = __ldcg(p.split_units + at);
    const int n = u.x, srow0 = u.z * kBlock + r0;  // n <= kMaxSplits
    if (n == 1 || srow0 >= p.rows) return;
    const int64_t out0 = (int64_t)u.y * p.rows + srow0;
    const float *first =
        p.parts + ((int64_t)at * p.splits * p.blocks + r0 / kBlock) * kPartFloats;
    const int row0 = r0 % kBlock;
    const int64_t step = (int64_t)p.blocks * kPartFloats;
    constexpr int kLanes = 16, kEach = kMaxSplits / kLanes;  // lanes of a row
    for (int r = threadIdx.x / kLanes; r < p.join_rows; r += 256 / kLanes) {
        const int k0 = threadIdx.x % kLanes;
        float m[kEach], l[kEach], top = -INFINITY, sum = 0.0f;
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
            const int k = k0 + i * kLanes;
            m[i] = -INFINITY, l[i] = 0.0f;
            if (k < n) {
                const float *rec = first + k * step + row0 + r;
                m[i] = rec[0], l[i] = rec[kBlock];
            }
            top = fmaxf(top, m[i]);
        }
#pragma unroll
        for (int o = kLanes / 2; o; o >>= 1)
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
            const float f = m[i] > -INFINITY ? ex2(m[i] - top) : 0.0f;
            sum += f * l[i];
            weight[r][k0 + i * kLanes] = f;
        }
#pragma unroll
        for (int o = kLanes / 2; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        if (k0 > 0) continue;
        inverse[r] = sum == 0.0f ? 0.0f : 1.0f / sum;
        if (a.lse && srow0 + r < p.rows)
            a.lse[out0 + r] = (top + log2f(sum)) * 0.6931471805599453f;
    }
    __syncthreads();
    const int four = warp * 4 + lane / 8;
#pragma unroll 2
    for (int r = lane % 8; r < p.join_rows; r += 8) {
        if (srow0 + r >= p.rows) break;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        const float4 *src =
            reinterpret_cast<const float4 *>(first + 2 * kBlock) + four * kBlock + row0 + r;
        for (int k0 = 0; k0 < n; k0 += kTogether) {
            float4 x[kTogether];
            float w[kTogether];
#pragma unroll
            for (int k = 0; k < kTogether; ++k) {
                w[k] = k0 + k < n ? weight[r][k0 + k] : 0.0f;
                x[k] = make_float4(0.f, 0.f, 0.f, 0.f);
                // Parts without a seen token have stored nothing.
                if (w[k] != 0.0f) x[k] = src[(k0 + k) * step / 4];
            }
#pragma unroll
            for (int k = 0; k < kTogether; ++k) {
                acc.x = fmaf(w[k], x[k].x, acc.x), acc.y = fmaf(w[k], x[k].y, acc.y);
                acc.z = fmaf(w[k], x[k].z, acc.z), acc.w = fmaf(w[k], x[k].w, acc.w);
            }
        }
        const float inv = inverse[r];
        reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(a.out) + (out0 + r) * kHD)[four] =
            make_uint2(pack_bf16(acc.x * inv, acc.y * inv), pack_bf16(acc.z * inv, acc.w * inv));
    }
}

// Stripes of a call, and the units of one with `blocks` query blocks each.
struct Shape {
    int64_t stripes, rows, blocks, per;
    int64_t units() const { return stripes * per; }
};
Shape shape_of(const Kv4Shape &k, int64_t blocks) {
    Shape s;
    s.stripes = k.n * (k.lists ? k.Hq : k.Hkv);
    s.rows = k.lists ? k.Lq : k.Hq / k.Hkv * k.Lq;
    s.blocks = blocks;
    s.per = ceil_div(s.rows, blocks * kBlock);
    return s;
}

// How a call's units are cut, and what that costs, in the steps of cost_of.
// Where the device chooses the chunk: as many CTAs a unit as the scratch
// holds.  Else, for units of equal length: whole units in full waves first,
// the others split, as cheap as that gets.  `step`: what a step takes.
constexpr float kInPlaceStep = 0.92f;  // one block over a page unpacked in place: 1.43 us
struct Cut {
    int whole, splits;
    float cost;
};
Cut cut_of(int64_t units, int64_t tiles, float step, bool device_chooses) {
    Cut best{0, 1, cost_of((float)units, step * (float)tiles, 0.0f, false, true)};
    const int64_t split = kMaxParts / 2;  // units that can be split at all
    int64_t whole = units > split ? ceil_div(units - split, 148) * 148 : 0;
    if (device_chooses) whole = 0;
    for (; whole < units; whole += 148) {
        const int64_t tail = units - whole;
        const float waves = (float)(whole / 148) * (step * (float)tiles + 4.0f);
        for (int s = 2; s <= kMaxSplits && tail * s <= kMaxParts && tiles >= 2 * s; ++s) {
            const float cost = waves + cost_of((float)(tail * s), step * (float)ceil_div(tiles, s),
                                               0.0f, true, true);
            if (device_chooses || cost < best.cost)
                best = Cut{(int)whole, s, cost < best.cost ? cost : best.cost};
        }
        if (device_chooses) break;
    }
    return best;
}
bool chooses(const Kv4Shape &k, const Shape &s, bool causal) {
    return !k.lists && (k.n > 1 || causal) && k.n * s.per <= kChosenUnits;
}
int64_t entries_of(const Kv4Shape &k) { return k.lists ? k.max_sel : k.max_pages; }

// Scratch for the parts of a call, however it is cut.
int64_t part_bytes(const Shape &s) {
    const int64_t parts = s.units() * kMaxSplits;
    return (parts < kMaxParts ? parts : kMaxParts) * s.blocks * kPartFloats * 4;
}

// Whether the pages are unpacked first: what both ways cost for sequences that
// fill their tables.  Unpacking takes 14 ns a page and head over the whole GPU,
// and one more launch.  Measured, first against in place, 16 heads of one
// sequence: 384 rows a head 94 against 77 us (16,512 tokens) and 35 against 30
// (4,000); 512 rows 97 against 109 and 37 against 38; 1,000 rows 149 against
// 193 and 54 against 56; 128 rows 63 against 38.
bool unpack_first(const Kv4Shape &k) {
    const int64_t tiles = k.n * k.max_pages * k.Hkv;
    if (tiles * kPairBytes > ((int64_t)2 << 30)) return false;
    const Cut in_place = cut_of(shape_of(k, 1).units(), entries_of(k), kInPlaceStep, false);
    const Cut first = cut_of(shape_of(k, 2).units(), entries_of(k), 1.0f, false);
    return first.cost + 1.5f + 0.009f * (float)tiles < in_place.cost;
}

}  // namespace

int64_t kv4_attn_many_rows(const Kv4Shape &k) { return shape_of(k, 1).rows; }

int64_t kv4_attn_many_work_bytes(const Kv4Shape &k) {
    const bool first = unpack_first(k);
    return kHeadBytes + part_bytes(shape_of(k, first ? 2 : 1)) +
           (first ? k.n * k.max_pages * k.Hkv * kPairBytes : 0);
}

cudaError_t launch_kv4_attn_many(const Kv4 &c, const Kv4Attn &a, const Kv4Shape &k,
                                 cudaStream_t stream) {
    const bool first = unpack_first(k);
    const Shape s = shape_of(k, first ? 2 : 1);
    CUtensorMap mq;
    if (!encode(&mq, a.q, s.stripes, s.rows)) return cudaErrorUnknown;
    Plan p;
    p.heads = a.Hq / c.Hkv;
    p.rows = (int)s.rows;
    p.blocks = (int)s.blocks;
    p.per = (int)s.per;
    p.nqb = (int)ceil_div(s.rows, kBlock);
    const int64_t entries = entries_of(k);  // of a unit, at most
    const bool chosen = first && chooses(k, s, a.causal);
    const Cut cut = cut_of(s.units(), entries, first ? 1.0f : kInPlaceStep, chosen);
    p.whole = cut.whole, p.splits = cut.splits;
    p.chunk = (int)ceil_div(entries > 0 ? entries : 1, p.splits);
    p.chosen = chosen && p.splits > 1
                   ? static_cast<int32_t *>(a.work) + SPARSTAR_KV4_WORK_ZEROS / 4
                   : nullptr;
    p.sc = a.tau * 1.4426950408889634f;
    p.split_units = reinterpret_cast<int4 *>(static_cast<uint8_t *>(a.work) +
                                             SPARSTAR_KV4_WORK_ZEROS + kChosenBytes);
    p.parts = static_cast<float *>(a.work) + kHeadBytes / 4;
    p.tiles = static_cast<uint8_t *>(a.work) + kHeadBytes + part_bytes(s);
    p.tile_blocks = c.max_pages;
    const auto kernel = first ? many_kernel<true> : many_kernel<false>;
    cudaError_t e =
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
    if (e != cudaSuccess) return e;
    const int64_t tail = s.units() - p.whole;
    const unsigned grid = (unsigned)(p.whole + tail * p.splits);
    if (first) {
        const int64_t tiles = (int64_t)a.n * c.max_pages * c.Hkv;
        e = cudaFuncSetAttribute(unpack_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 kPairBytes);
        if (e == cudaSuccess)
            e = launch_after(unpack_kernel, (unsigned)(tiles + (p.chosen ? 1 : 0)), 256,
                             kPairBytes, stream, c, a, p);
        if (e != cudaSuccess) return e;
    }
    e = launch_after(kernel, grid, first ? kThreads<true> : kThreads<false>, kSmemBytes, stream,
                     mq, c, a, p);
    if (e != cudaSuccess || p.splits == 1 || tail == 0) return e;
    // Eight rows a CTA while these fit the GPU at once, then 32, which find
    // their unit once.
    const int64_t rows = tail * p.blocks * kBlock;
    p.join_rows = rows / 8 <= 148 * 8 ? 8 : 32;
    return launch_after(many_join_kernel, (unsigned)(rows / p.join_rows), 256, 0, stream, a, p);
}

}  // namespace sparstar
