// The codec of the paged 4-bit key/value cache: tokens into pages (write)
// and the values that pages stand for (read).  Format: sparstar.h.
//
// One CTA a (sequence, touched page, head).  Both directions move 2 D e + D +
// D/16 bytes a token and head.  A read is bound by that traffic: 41,012 tokens
// of 16 heads to bf16, 425 MB, take 79 us, 5.4 TB/s, with the loads of a
// thread's whole share ahead of their use.  A write comes near it: 18,000
// tokens, 187 MB, take 42 us from cold, the integer pipe (packing) 69% and
// shared memory 56% busy.  The keys of a
// page lie token by token, as the inputs do; its values lie channel by
// channel (the contraction of P V runs over tokens, and its operand pairs
// tokens), so they pass through shared memory as words of eight channels and
// are transposed eight tokens by eight channels in registers.
#include <type_traits>

#include <cuda_bf16.h>

#include "kv4.cuh"

namespace sparstar {
namespace {

constexpr int kThreads = 256;

// Scale code of a group whose largest magnitude is a: a / 7 rounded to four
// significant bits.  Two roundings decide as one would: the fp32 quotient can
// only fall on a border M of five bits while a != 7 M if a - 7 M is less than
// half of 2^-23 relative, and it is at least one unit of a's last place.
__device__ __forceinline__ uint32_t scale_code(float a) {
    const uint32_t bits = __float_as_uint(__fdiv_rn(a, 7.0f));
    const int c = (int)((bits + 0x7ffffu + ((bits >> 20) & 1u)) >> 20) - (kScaleExp << 3);
    return (uint32_t)(c < 0 ? 0 : (c > 255 ? 255 : c));
}

constexpr float kRound = 12582912.0f;  // 1.5 * 2^23: adding it rounds to integers, ties to even
constexpr uint32_t kNibbles = 0x000f000fu;

// Joins four pairs of codes (in the low nibbles of the halves) to a word.
__device__ __forceinline__ uint32_t join_pairs(const uint32_t (&p)[4]) {
    return (p[0] & kNibbles) | ((p[1] & kNibbles) << 4) | ((p[2] & kNibbles) << 8) |
           ((p[3] & kNibbles) << 12);
}

// One group of 32 values in registers: bf16 pairs, or fp32.
struct GroupBf16 {
    uint32_t x[16];
    __device__ void load(const __nv_bfloat16 *p) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint4 v = __ldcs(reinterpret_cast<const uint4 *>(p) + i);
            x[4 * i] = v.x, x[4 * i + 1] = v.y, x[4 * i + 2] = v.z, x[4 * i + 3] = v.w;
        }
    }
    // The largest magnitude; NaN when there is one.
    __device__ float largest() const {
        uint32_t m = x[0] & 0x7fff7fffu;
#pragma unroll
        for (int i = 1; i < 16; ++i)
            asm("max.NaN.bf16x2 %0, %0, %1;" : "+r"(m) : "r"(x[i] & 0x7fff7fffu));
        float r;
        asm("max.NaN.f32 %0, %1, %2;"
            : "=f"(r)
            : "f"(__uint_as_float(m << 16)), "f"(__uint_as_float(m & 0xffff0000u)));
        return r;
    }
    __device__ float get(int i) const {
        return __uint_as_float(i & 1 ? x[i / 2] & 0xffff0000u : x[i / 2] << 16);
    }
    __device__ void set(int i, float v) {  // v: a bf16 value
        const uint32_t b = __float_as_uint(v);
        x[i / 2] = i & 1 ? (x[i / 2] & 0xffffu) | (b & 0xffff0000u)
                         : (x[i / 2] & 0xffff0000u) | (b >> 16);
    }
    // Codes of values 8 i .. 8 i + 7.  x / s is a tie or at least 2^-10 of a
    // step away from one (eight and four significant bits), so the products
    // with a reciprocal 2^-20 too large and one 2^-20 too small round alike
    // except for a tie, where they round to its two neighbours: the larger
    // one without its last bit is the even one.
    __device__ uint32_t word(int i, float s) const {
        const float r = __frcp_rn(s);
        const float up = r * (1.0f + 0x1p-20f), down = r * (1.0f - 0x1p-20f);
        uint32_t p[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const float a = get(8 * i + 2 * k), b = get(8 * i + 2 * k + 1);
            const uint32_t u = __byte_perm(__float_as_uint(fmaf(a, up, kRound + 8.0f)),
                                           __float_as_uint(fmaf(b, up, kRound + 8.0f)), 0x5410);
            const uint32_t d = __byte_perm(__float_as_uint(fmaf(a, down, kRound + 8.0f)),
                                           __float_as_uint(fmaf(b, down, kRound + 8.0f)), 0x5410);
            uint32_t m;
            asm("max.u16x2 %0, %1, %2;" : "=r"(m) : "r"(u), "r"(d));
            p[k] = m & ~((u ^ d) & 0x00010001u);
        }
        return join_pairs(p);
    }
};
struct GroupF32 {
    float x[32];
    __device__ void load(const float *p) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float4 v = __ldcs(reinterpret_cast<const float4 *>(p) + i);
            x[4 * i] = v.x, x[4 * i + 1] = v.y, x[4 * i + 2] = v.z, x[4 * i + 3] = v.w;
        }
    }
    __device__ float largest() const {
        float m = fabsf(x[0]);
#pragma unroll
        for (int i = 1; i < 32; ++i) asm("max.NaN.f32 %0, %0, %1;" : "+f"(m) : "f"(fabsf(x[i])));
        return m;
    }
    __device__ float get(int i) const { return x[i]; }
    __device__ void set(int i, float v) { x[i] = v; }
    // n = rint(x * (1/s)) is off by one at most (the product is within 2^-22
    // of the quotient), and x - n s is exact in an fma: its magnitude against
    // s / 2 settles the nearest code, and n's last bit a tie.
    __device__ uint32_t word(int i, float s) const {
        const float r = __frcp_rn(s);
        const uint32_t half = __float_as_uint(0.5f * s);
        uint32_t p[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            uint32_t c[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const float v = x[8 * i + 2 * k + h];
                const float t = fmaf(v, r, kRound + 8.0f);
                const uint32_t bits = __float_as_uint(t);
                const uint32_t d = __float_as_uint(fmaf(-(t - (kRound + 8.0f)), s, v));
                const bool step = (d & 0x7fffffffu) + (bits & 1u) > half;
                c[h] = bits + (step ? ((int)d >> 31) | 1 : 0);
            }
            p[k] = __byte_perm(c[0], c[1], 0x5410);
        }
        return join_pairs(p);
    }
};
template <typename T>
using Group = typename std::conditional<std::is_same<T, float>::value, GroupF32, GroupBf16>::type;

// Quantises one group: four words of codes and the scale code.  Returns
// false when a value was beyond the range or NaN.
template <typename G>
__device__ __forceinline__ bool quantise(G &x, uint32_t (&w)[4], uint32_t &code) {
    float a = x.largest();
    const bool fine = a <= kKv4Limit;  // false for NaN
    if (!fine) {
        a = 0.0f;
#pragma unroll
        for (int i = 0; i < 32; ++i) {
            const float v = x.get(i);
            const float y = v == v ? fminf(fmaxf(v, -kKv4Limit), kKv4Limit) : 0.0f;
            x.set(i, y);
            a = fmaxf(a, fabsf(y));
        }
    }
    code = scale_code(a);
    const float s = kv4_scale(code);
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = x.word(i, s);
    return fine;
}

// What the CTA works on: a page of a sequence, and the tokens t0 <= t < t1
// of the call that lie in it, token t at slot t - shift of the page.
struct Span {
    int i, h, page, t0, t1, shift;
};

// Fills the span; false when the CTA has nothing to do.  `unique`: a slot
// that repeats an earlier entry's is left out.
__device__ bool find_span(const Kv4 &c, int n, int64_t T, int per_seq, const int32_t *seqs,
                          const int32_t *starts, const int32_t *counts, bool write,
                          int32_t *status, Span &sp) {
    const int b = blockIdx.x;
    sp.h = b % c.Hkv;
    const int j = (b / c.Hkv) % per_seq;
    sp.i = b / c.Hkv / per_seq;
    const bool says = sp.h == 0 && j == 0 && threadIdx.x == 0;
    const int slot = kv4_slot(c, seqs, sp.i);
    const int count = counts ? __ldca(counts + sp.i) : (int)T;
    bool bad = slot < 0 || count < 0 || count > T;
    int start = 0;
    if (!bad) {
        const int L = kv4_len(c, slot);
        start = starts ? __ldca(starts + sp.i) : (write ? L - count : 0);
        bad = start < 0 || start > L - count;
    }
    if (write && seqs && !bad) {
        int twice = 0;
        for (int k = threadIdx.x; k < sp.i; k += blockDim.x) twice |= __ldca(seqs + k) == slot;
        bad = __syncthreads_or(twice) != 0;
    }
    if (bad) {
        if (says) kv4_flag(status, SPARSTAR_STATUS_BAD_INDEX);
        return false;
    }
    const int col = start / kBlock + j;
    sp.shift = col * kBlock - start;
    sp.t0 = sp.shift > 0 ? sp.shift : 0;
    sp.t1 = sp.shift + kBlock < count ? sp.shift + kBlock : count;
    if (sp.t0 >= sp.t1) return false;
    sp.page = __ldca(c.table + (int64_t)slot * c.max_pages + col);
    if (sp.page < 0 || sp.page >= c.n_pages) {
        if (threadIdx.x == 0) kv4_flag(status, SPARSTAR_STATUS_BAD_INDEX);
        return false;
    }
    if (write && c.refs[sp.page] > 1) {
        if (threadIdx.x == 0) kv4_flag(status, SPARSTAR_STATUS_SHARED);
        return false;
    }
    return true;
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads)
    write_kernel(Kv4 c, const T *k, const T *v, int n, int64_t tokens, int per_seq,
                 const int32_t *seqs, const int32_t *starts, const int32_t *counts,
                 int32_t *status) {
    constexpr int G = D / kGroup;     // groups of a token
    constexpr int W = D / 8;          // words of eight channels of a token
    constexpr int kStride = W + 1;    // odd: the transpose reads a column of words
    __shared__ uint32_t words[kBlock * kStride];  // value codes, token by token
    __shared__ uint8_t scales[G][kBlock];
    kv4_begin();
    Span sp;
    if (!find_span(c, n, tokens, per_seq, seqs, starts, counts, true, status, sp)) return;
    uint8_t *half_k = c.pages + ((int64_t)sp.page * c.Hkv + sp.h) * kv4_page_bytes(D);
    uint8_t *half_v = half_k + kv4_half_bytes(D);
    const int64_t row = ((int64_t)sp.i * c.Hkv + sp.h) * tokens;
    const int first = sp.t0 - sp.shift, last = sp.t1 - sp.shift;  // slots of the page
    const int items = (last - first) * G;
    bool fine = true;
    for (int it = threadIdx.x; it < 2 * items; it += kThreads) {
        const bool is_v = it >= items;
        const int u = is_v ? it - items : it;
        const int slot = first + u / G, g = u % G;
        Group<T> x;
        uint32_t w[4], code;
        x.load((is_v ? v : k) + (row + slot + sp.shift) * D + g * kGroup);
        fine &= quantise(x, w, code);
        if (is_v) {
#pragma unroll
            for (int q = 0; q < 4; ++q) words[slot * kStride + g * 4 + q] = w[q];
            scales[g][slot] = (uint8_t)code;
        } else {
            reinterpret_cast<uint4 *>(half_k)[slot * G + g] = make_uint4(w[0], w[1], w[2], w[3]);
            half_k[kv4_code_bytes(D) + slot * G + g] = (uint8_t)code;
        }
    }
    if (__syncthreads_or(!fine) && threadIdx.x == 0) kv4_flag(status, SPARSTAR_STATUS_CLAMPED);
    // Eight tokens by eight channels a thread; tokens that the call does not
    // write keep their codes.
    const int w0 = first / 8, w1 = (last + 7) / 8;
    for (int it = threadIdx.x; it < W * (w1 - w0); it += kThreads) {
        const int cw = it / (w1 - w0), tw = w0 + it % (w1 - w0);
        uint32_t r[8], keep = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int slot = tw * 8 + e;
            r[e] = words[slot * kStride + cw];
            if (slot < first || slot >= last) keep |= 0xfu << (4 * kv4_nibble(e));
        }
        kv4_transpose(r);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            uint32_t *p = reinterpret_cast<uint32_t *>(half_v) + (cw * 8 + e) * (kBlock / 8) + tw;
            *p = keep ? (*p & keep) | (r[e] & ~keep) : r[e];
        }
    }
    for (int it = threadIdx.x; it < G * (last - first); it += kThreads) {
        const int g = it / (last - first), slot = first + it % (last - first);
        half_v[kv4_code_bytes(D) + g * kBlock + slot] = scales[g][slot];
    }
}

// Eight values from a word of codes.
__device__ __forceinline__ void store8(__nv_bfloat16 *p, uint32_t w, uint32_t code) {
    const uint32_t s = kv4_scale_pair(code * 0x10001u), m = kv4_minus136(s);
    uint32_t o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = kv4_dequant(kv4_pair128(w, i, kMagic), s, m);
    __stcs(reinterpret_cast<uint4 *>(p), make_uint4(o[0], o[1], o[2], o[3]));
}
__device__ __forceinline__ void store8(float *p, uint32_t w, uint32_t code) {
    const float s = kv4_scale(code);
    float o[8];
#pragma unroll
    for (int e = 0; e < 8; ++e)
        o[e] = s * (float)((int)((w >> (4 * kv4_nibble(e))) & 15u) - 8);
    __stcs(reinterpret_cast<float4 *>(p), make_float4(o[0], o[1], o[2], o[3]));
    __stcs(reinterpret_cast<float4 *>(p) + 1, make_float4(o[4], o[5], o[6], o[7]));
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads)
    read_kernel(Kv4 c, T *k, T *v, int n, int64_t tokens, int per_seq, const int32_t *seqs,
                const int32_t *starts, const int32_t *counts, int32_t *status) {
    constexpr int G = D / kGroup, W = D / 8;
    constexpr int kStride = W + 1;
    __shared__ uint32_t words[kBlock * kStride];
    kv4_begin();
    Span sp;
    if (!find_span(c, n, tokens, per_seq, seqs, starts, counts, false, status, sp)) return;
    const uint8_t *half_k = c.pages + ((int64_t)sp.page * c.Hkv + sp.h) * kv4_page_bytes(D);
    const uint8_t *half_v = half_k + kv4_half_bytes(D);
    const int64_t row = ((int64_t)sp.i * c.Hkv + sp.h) * tokens;
    const int first = sp.t0 - sp.shift, last = sp.t1 - sp.shift;
    // The values' words first: they are on their way while the keys pass.
    const int w0 = first / 8, tiles = W * ((last + 7) / 8 - w0);
    constexpr int kTiles = (W * (kBlock / 8) + kThreads - 1) / kThreads;
    static_assert(kTiles == 1, "eight words a thread, beside four of the keys");
    uint32_t r[kTiles][8];
    auto tile_of = [&](int i, int &cw, int &tw) {
        const int it = threadIdx.x + i * kThreads, n = (last + 7) / 8 - w0;
        cw = it / n, tw = w0 + it % n;
        return it < tiles;
    };
    if (v) {
        const uint32_t *codes = reinterpret_cast<const uint32_t *>(half_v);
#pragma unroll
        for (int i = 0; i < kTiles; ++i) {
            int cw, tw;
            if (!tile_of(i, cw, tw)) continue;
#pragma unroll
            for (int e = 0; e < 8; ++e) r[i][e] = __ldca(codes + (cw * 8 + e) * (kBlock / 8) + tw);
        }
    }
    const int items = (last - first) * W;
    if (k) {
        const uint32_t *codes = reinterpret_cast<const uint32_t *>(half_k);
        const uint8_t *scales = half_k + kv4_code_bytes(D);
        for (int it0 = threadIdx.x; it0 < items; it0 += 4 * kThreads) {
            uint32_t word[4], scale[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int it = it0 + i * kThreads, slot = first + it / W, w = it % W;
                if (it >= items) continue;
                word[i] = __ldca(codes + slot * W + w);
                scale[i] = __ldca(scales + slot * G + w / 4);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int it = it0 + i * kThreads, slot = first + it / W, w = it % W;
                if (it < items)
                    store8(k + (row + slot + sp.shift) * D + w * 8, word[i], scale[i]);
            }
        }
    }
    if (v) {
        const uint8_t *scales = half_v + kv4_code_bytes(D);
#pragma unroll
        for (int i = 0; i < kTiles; ++i) {
            int cw, tw;
            if (!tile_of(i, cw, tw)) continue;
            kv4_transpose(r[i]);
#pragma unroll
            for (int e = 0; e < 8; ++e) words[(tw * 8 + e) * kStride + cw] = r[i][e];
        }
        __syncthreads();
        for (int it0 = threadIdx.x; it0 < items; it0 += 4 * kThreads) {
            uint32_t scale[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int it = it0 + i * kThreads, slot = first + it / W, w = it % W;
                if (it < items) scale[i] = __ldca(scales + (w / 4) * kBlock + slot);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int it = it0 + i * kThreads, slot = first + it / W, w = it % W;
                if (it < items)
                    store8(v + (row + slot + sp.shift) * D + w * 8, words[slot * kStride + w],
                           scale[i]);
            }
        }
    }
}

// Pages that T tokens can touch, whatever the start.
int pages_of(int64_t T) { return (int)((T + kBlock - 2) / kBlock + 1); }

}  // namespace

cudaError_t launch_kv4_write(const Kv4 &c, const void *k, const void *v, int dtype, int n,
                             int64_t T, const int32_t *seqs, const int32_t *starts,
                             const int32_t *counts, int32_t *status, cudaStream_t stream) {
    const int per_seq = pages_of(T);
    const unsigned grid = (unsigned)((int64_t)n * per_seq * c.Hkv);
    auto go = [&](auto kernel, auto type) {
        using E = decltype(type);
        return launch_after(kernel, grid, kThreads, 0, stream, c, static_cast<const E *>(k),
                            static_cast<const E *>(v), n, T, per_seq, seqs, starts, counts,
                            status);
    };
    if (dtype == SPARSTAR_BF16)
        return c.D == 128 ? go(write_kernel<__nv_bfloat16, 128>, __nv_bfloat16())
                          : go(write_kernel<__nv_bfloat16, 64>, __nv_bfloat16());
    return c.D == 128 ? go(write_kernel<float, 128>, float()) : go(write_kernel<float, 64>, float());
}

cudaError_t launch_kv4_read(const Kv4 &c, void *k, void *v, int dtype, int n, int64_t T,
                            const int32_t *seqs, const int32_t *starts, const int32_t *counts,
                            int32_t *status, cudaStream_t stream) {
    const int per_seq = pages_of(T);
    const unsigned grid = (unsigned)((int64_t)n * per_seq * c.Hkv);
    auto go = [&](auto kernel, auto type) {
        using E = decltype(type);
        return launch_after(kernel, grid, kThreads, 0, stream, c, static_cast<E *>(k),
                            static_cast<E *>(v), n, T, per_seq, seqs, starts, counts, status);
    };
    if (dtype == SPARSTAR_BF16)
        return c.D == 128 ? go(read_kernel<__nv_bfloat16, 128>, __nv_bfloat16())
                          : go(read_kernel<__nv_bfloat16, 64>, __nv_bfloat16());
    return c.D == 128 ? go(read_kernel<float, 128>, float()) : go(read_kernel<float, 64>, float());
}

}  // namespace sparstar
