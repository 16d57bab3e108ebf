// The codec of the paged 4-bit key/value cache: tokens into pages (write)
// and the values that pages stand for (read).  Format: sparstar.h.
//
// One CTA a (sequence, touched page, head).  Both directions move 2 D e + D +
// D/16 bytes a token and head and are bound by that traffic.  The keys of a
// page lie token by token, as the inputs do; its values lie channel by
// channel (the contraction of P V runs over tokens, and its operand pairs
// tokens), so they pass through shared memory as words of eight channels and
// are transposed eight tokens by eight channels in registers.
#include <cuda_bf16.h>

#include "kv4.cuh"

namespace sparstar {
namespace {

constexpr int kThreads = 256;

// The 32 values of one group as fp32.
__device__ __forceinline__ void load_group(const __nv_bfloat16 *p, float (&x)[32]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint4 v = __ldcs(reinterpret_cast<const uint4 *>(p) + i);
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            x[8 * i + 2 * j] = __uint_as_float(w[j] << 16);
            x[8 * i + 2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
        }
    }
}
__device__ __forceinline__ void load_group(const float *p, float (&x)[32]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float4 v = __ldcs(reinterpret_cast<const float4 *>(p) + i);
        x[4 * i] = v.x, x[4 * i + 1] = v.y, x[4 * i + 2] = v.z, x[4 * i + 3] = v.w;
    }
}

// Quantises one group: four words of codes and the scale code.  Returns
// false when a value was beyond the range or NaN.
//
// Both decisions are exact.  The scale: a / 7 rounded to fp32 and then to
// four bits can only differ from one rounding if the fp32 quotient falls on
// a border M of five bits while a != 7 M; but then a - 7 M is at least one
// unit of a's last place, 2^-23 relative, and the quotient is off by half of
// 2^-23 at most.  The code: n = rint(x * (1/s)) is off by one at most (the
// product is within 2^-22 of the quotient), and x - n s is exact in an fma,
// so comparing it with s / 2 settles the nearest code and the ties.
__device__ __forceinline__ bool quantise(float (&x)[32], uint32_t (&w)[4], uint32_t &code) {
    bool fine = true;
    float a = 0.0f;
#pragma unroll
    for (int i = 0; i < 32; ++i) {
        fine &= fabsf(x[i]) <= kKv4Limit;  // false for NaN
        a = fmaxf(a, fabsf(x[i]));
    }
    if (!fine) {
        a = 0.0f;
#pragma unroll
        for (int i = 0; i < 32; ++i) {
            x[i] = x[i] == x[i] ? fminf(fmaxf(x[i], -kKv4Limit), kKv4Limit) : 0.0f;
            a = fmaxf(a, fabsf(x[i]));
        }
    }
    const uint32_t bits = __float_as_uint(__fdiv_rn(a, 7.0f));
    int c = (int)((bits + 0x7ffffu + ((bits >> 20) & 1u)) >> 20) - (kScaleExp << 3);
    c = c < 0 ? 0 : (c > 255 ? 255 : c);
    code = (uint32_t)c;
    const float s = kv4_scale(code), r = __frcp_rn(s), half = 0.5f * s;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t word = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float v = x[8 * i + e];
            float n = rintf(v * r);
            const float d = fmaf(-n, s, v);  // exact
            // One step toward v when n is not the nearest, or is odd in a tie.
            const bool odd = ((int)n & 1) != 0;
            if (fabsf(d) > half || (fabsf(d) == half && odd)) n += copysignf(1.0f, d);
            n = fminf(fmaxf(n, -7.0f), 7.0f);
            word |= (uint32_t)((int)n + 8) << (4 * kv4_nibble(e));
        }
        w[i] = word;
    }
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
    const int count = counts ? __ldg(counts + sp.i) : (int)T;
    bool bad = slot < 0 || count < 0 || count > T;
    int start = 0;
    if (!bad) {
        const int L = kv4_len(c, slot);
        start = starts ? __ldg(starts + sp.i) : (write ? L - count : 0);
        bad = start < 0 || start > L - count;
    }
    if (write && seqs && !bad) {
        int twice = 0;
        for (int k = threadIdx.x; k < sp.i; k += blockDim.x) twice |= __ldg(seqs + k) == slot;
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
    sp.page = __ldg(c.table + (int64_t)slot * c.max_pages + col);
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
    write_kernel(Kv4 c, const T *__restrict__ k, const T *__restrict__ v, int n, int64_t tokens,
                 int per_seq, const int32_t *__restrict__ seqs, const int32_t *__restrict__ starts,
                 const int32_t *__restrict__ counts, int32_t *status) {
    constexpr int G = D / kGroup;     // groups of a token
    constexpr int W = D / 8;          // words of eight channels of a token
    constexpr int kStride = W + 1;    // odd: the transpose reads a column of words
    __shared__ uint32_t words[kBlock * kStride];  // value codes, token by token
    __shared__ uint8_t scales[G][kBlock];
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
        float x[32];
        uint32_t w[4], code;
        load_group((is_v ? v : k) + (row + slot + sp.shift) * D + g * kGroup, x);
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
    *reinterpret_cast<uint4 *>(p) = make_uint4(o[0], o[1], o[2], o[3]);
}
__device__ __forceinline__ void store8(float *p, uint32_t w, uint32_t code) {
    const float s = kv4_scale(code);
    float o[8];
#pragma unroll
    for (int e = 0; e < 8; ++e)
        o[e] = s * (float)((int)((w >> (4 * kv4_nibble(e))) & 15u) - 8);
    reinterpret_cast<float4 *>(p)[0] = make_float4(o[0], o[1], o[2], o[3]);
    reinterpret_cast<float4 *>(p)[1] = make_float4(o[4], o[5], o[6], o[7]);
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads)
    read_kernel(Kv4 c, T *__restrict__ k, T *__restrict__ v, int n, int64_t tokens, int per_seq,
                const int32_t *__restrict__ seqs, const int32_t *__restrict__ starts,
                const int32_t *__restrict__ counts, int32_t *status) {
    constexpr int G = D / kGroup, W = D / 8;
    constexpr int kStride = W + 1;
    __shared__ uint32_t words[kBlock * kStride];
    Span sp;
    if (!find_span(c, n, tokens, per_seq, seqs, starts, counts, false, status, sp)) return;
    const uint8_t *half_k = c.pages + ((int64_t)sp.page * c.Hkv + sp.h) * kv4_page_bytes(D);
    const uint8_t *half_v = half_k + kv4_half_bytes(D);
    const int64_t row = ((int64_t)sp.i * c.Hkv + sp.h) * tokens;
    const int first = sp.t0 - sp.shift, last = sp.t1 - sp.shift;
    if (k) {
        const uint32_t *codes = reinterpret_cast<const uint32_t *>(half_k);
        const uint8_t *scales = half_k + kv4_code_bytes(D);
        for (int it = threadIdx.x; it < (last - first) * W; it += kThreads) {
            const int slot = first + it / W, w = it % W;
            store8(k + (row + slot + sp.shift) * D + w * 8, __ldg(codes + slot * W + w),
                   __ldg(scales + slot * G + w / 4));
        }
    }
    if (v) {
        const int w0 = first / 8, w1 = (last + 7) / 8;
        const uint32_t *codes = reinterpret_cast<const uint32_t *>(half_v);
        const uint8_t *scales = half_v + kv4_code_bytes(D);
        for (int it = threadIdx.x; it < W * (w1 - w0); it += kThreads) {
            const int cw = it / (w1 - w0), tw = w0 + it % (w1 - w0);
            uint32_t r[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) r[e] = __ldg(codes + (cw * 8 + e) * (kBlock / 8) + tw);
            kv4_transpose(r);
#pragma unroll
            for (int e = 0; e < 8; ++e) words[(tw * 8 + e) * kStride + cw] = r[e];
        }
        __syncthreads();
        for (int it = threadIdx.x; it < (last - first) * W; it += kThreads) {
            const int slot = first + it / W, w = it % W;
            store8(v + (row + slot + sp.shift) * D + w * 8, words[slot * kStride + w],
                   __ldg(scales + (w / 4) * kBlock + slot));
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
        kernel<<<grid, kThreads, 0, stream>>>(c, static_cast<const E *>(k),
                                              static_cast<const E *>(v), n, T, per_seq, seqs,
                                              starts, counts, status);
    };
    if (dtype == SPARSTAR_BF16) {
        if (c.D == 128) go(write_kernel<__nv_bfloat16, 128>, __nv_bfloat16());
        else go(write_kernel<__nv_bfloat16, 64>, __nv_bfloat16());
    } else {
        if (c.D == 128) go(write_kernel<float, 128>, float());
        else go(write_kernel<float, 64>, float());
    }
    return cudaGetLastError();
}

cudaError_t launch_kv4_read(const Kv4 &c, void *k, void *v, int dtype, int n, int64_t T,
                            const int32_t *seqs, const int32_t *starts, const int32_t *counts,
                            int32_t *status, cudaStream_t stream) {
    const int per_seq = pages_of(T);
    const unsigned grid = (unsigned)((int64_t)n * per_seq * c.Hkv);
    auto go = [&](auto kernel, auto type) {
        using E = decltype(type);
        kernel<<<grid, kThreads, 0, stream>>>(c, static_cast<E *>(k), static_cast<E *>(v), n, T,
                                              per_seq, seqs, starts, counts, status);
    };
    if (dtype == SPARSTAR_BF16) {
        if (c.D == 128) go(read_kernel<__nv_bfloat16, 128>, __nv_bfloat16());
        else go(read_kernel<__nv_bfloat16, 64>, __nv_bfloat16());
    } else {
        if (c.D == 128) go(read_kernel<float, 128>, float());
        else go(read_kernel<float, 64>, float());
    }
    return cudaGetLastError();
}

}  // namespace sparstar
