// Device helpers of the paged 4-bit key/value cache (format: sparstar.h).
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "sparstar.h"
#include "sparstar_internal.h"

namespace sparstar {

constexpr float kKv4Limit = 26880.0f;  // 7 * the largest scale, 3840
constexpr int kScaleExp = 107;         // bf16 exponent field of scale codes 0..7: 2^-20

// Scale code -> scale: four significant bits, so bf16 and fp32 hold it.
__device__ __forceinline__ float kv4_scale(uint32_t code) {
    return __uint_as_float((code + (kScaleExp << 3)) << 20);
}
// Two scale codes in the low bytes of the halves of x -> a bf16 pair.
__device__ __forceinline__ uint32_t kv4_scale_pair(uint32_t x) {
    return (x << 4) + ((uint32_t)kScaleExp << 7) * 0x10001u;
}
// The same with 16 in a register (kv4_opaque): an integer fma, off the pipe
// that the masks and shifts of the codes fill.
__device__ __forceinline__ uint32_t kv4_scale_pair(uint32_t x, uint32_t sixteen) {
    return x * sixteen + ((uint32_t)kScaleExp << 7) * 0x10001u;
}

// Codes 2i and 2i + 1 of a word as the bf16 pair 128 + code (bf16 holds the
// integers up to 256, so the code goes straight into the mantissa).  `magic`
// is kMagic in a register of the caller's (kv4_opaque): the mask and the magic
// then take one lop3, where two constants would take two.
constexpr uint32_t kMagic = 0x43004300u;
__device__ __forceinline__ uint32_t kv4_opaque(uint32_t m) {
    asm volatile("" : "+r"(m));
    return m;
}
__device__ __forceinline__ uint32_t kv4_pair128(uint32_t w, int i, uint32_t magic) {
    uint32_t y;
    asm("lop3.b32 %0, %1, 0x000f000f, %2, 0xea;" : "=r"(y) : "r"(w >> (4 * i)), "r"(magic));
    return y;
}
__device__ __forceinline__ __nv_bfloat162 as_bf162(uint32_t x) {
    return *reinterpret_cast<__nv_bfloat162 *>(&x);
}
__device__ __forceinline__ uint32_t as_u32(__nv_bfloat162 x) {
    return *reinterpret_cast<uint32_t *>(&x);
}
// s * (code - 8) for two codes, as (128 + code) * s - 136 * s.  Exact: 136 s
// has at most 8 significant bits (17 * m for m = 8..15 is below 256), the
// fma rounds once, and its result (7 or fewer bits) needs no rounding.
__device__ __forceinline__ uint32_t kv4_dequant(uint32_t pair128, uint32_t s, uint32_t minus136s) {
    return as_u32(__hfma2(as_bf162(pair128), as_bf162(s), as_bf162(minus136s)));
}
__device__ __forceinline__ uint32_t kv4_minus136(uint32_t s) {
    return as_u32(__hmul2(as_bf162(s), __float2bfloat162_rn(-136.0f)));
}

// Element e of a word: its nibble.
__host__ __device__ constexpr int kv4_nibble(int e) { return (e & 1) * 4 + (e >> 1); }

// Transposes the 8 x 8 nibbles of eight words held by nibble position: word
// p, nibble r goes to word r, nibble p.  Words are given by element (token
// or channel) e at index e; positions follow from kv4_nibble on both sides.
__device__ __forceinline__ void kv4_transpose(uint32_t (&w)[8]) {
    uint32_t r[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) r[kv4_nibble(e)] = w[e];
#pragma unroll
    for (int p = 0; p < 4; ++p) {  // 16-bit halves of rows p and p + 4
        const uint32_t a = r[p], b = r[p + 4];
        r[p] = __byte_perm(a, b, 0x5410);
        r[p + 4] = __byte_perm(a, b, 0x7632);
    }
#pragma unroll
    for (int p = 0; p < 8; ++p) {  // bytes of rows p and p + 2
        if (p & 2) continue;
        const uint32_t a = r[p], b = r[p + 2];
        r[p] = __byte_perm(a, b, 0x6240);
        r[p + 2] = __byte_perm(a, b, 0x7351);
    }
#pragma unroll
    for (int p = 0; p < 8; p += 2) {  // nibbles of rows p and p + 1
        const uint32_t a = r[p], b = r[p + 1];
        r[p] = (a & 0x0f0f0f0fu) | ((b << 4) & 0xf0f0f0f0u);
        r[p + 1] = ((a >> 4) & 0x0f0f0f0fu) | (b & 0xf0f0f0f0u);
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) w[e] = r[kv4_nibble(e)];
}

// Bounded wait of one thread for a phase of an mbarrier; false after two
// seconds.
__device__ __forceinline__ bool kv4_wait(uint32_t bar, uint32_t parity) {
    uint64_t t0 = 0;
    while (true) {
        uint32_t ok;
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(ok)
            : "r"(bar), "r"(parity)
            : "memory");
        if (ok) return true;
        uint64_t t;
        asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
        if (t0 == 0) t0 = t;
        if (t - t0 > 2000000000ull) return false;
    }
}

__device__ __forceinline__ void kv4_flag(int32_t *status, int32_t bits) {
    if (status) atomicOr(status, bits);
}

// Slot of list entry i; -1 when outside the cache.
__device__ __forceinline__ int kv4_slot(const Kv4 &c, const int32_t *seqs, int i) {
    const int s = seqs ? __ldca(seqs + i) : i;
    return s >= 0 && s < c.n_seqs ? s : -1;
}
// Tokens of a slot, whatever the memory holds: 0 .. 128 max_pages.
__device__ __forceinline__ int kv4_len(const Kv4 &c, int slot) {
    const int L = c.lens[slot];
    const int most = c.max_pages * kBlock;
    return L < 0 ? 0 : (L > most ? most : L);
}

// A cache call's kernels follow each other closely (a step resizes, writes and
// attends), so each may be launched while the one before it still runs: its
// CTAs take their places as that one's leave, and each waits for the whole
// grid before it, and for that one's own wait, before it touches memory.  What
// the calls before may have written (pages, tables and lists, but also queries
// and tokens that came from another call) is loaded by ordinary loads behind the
// wait: the read-only path (__ldg, const __restrict__) is defined only for
// memory that nobody writes while the kernel is resident.
__device__ __forceinline__ void kv4_begin() {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
// Launches such a kernel.
template <typename... Args>
inline cudaError_t launch_after(void (*kernel)(Args...), unsigned grid, unsigned block, size_t smem,
                                cudaStream_t stream, Args... args) {
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(block);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

}  // namespace sparstar
