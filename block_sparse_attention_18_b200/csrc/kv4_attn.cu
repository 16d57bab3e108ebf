// Forward attention over the paged 4-bit key/value cache.
//
// One CTA a query row: a page at a time, one thread a token for the scores
// and one thread a channel for the values, with a running maximum and sum.
#include <cuda_bf16.h>

#include "kv4.cuh"

namespace sparstar {
namespace {

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void store(float *p, float x) { *p = x; }
__device__ __forceinline__ void store(__nv_bfloat16 *p, float x) { *p = __float2bfloat16_rn(x); }

template <typename T, int D>
__global__ void __launch_bounds__(kBlock) attn_row_kernel(Kv4 c, Kv4Attn a) {
    constexpr int G = D / kGroup;
    __shared__ float qs[D], ps[kBlock], red[4];
    const int64_t r = blockIdx.x;
    const int row = (int)(r % a.Lq), h = (int)(r / a.Lq % a.Hq), i = (int)(r / a.Lq / a.Hq);
    const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
    const int slot = kv4_slot(c, a.seqs, i);
    const int L = slot >= 0 ? kv4_len(c, slot) : 0;
    if (slot < 0 && t == 0) kv4_flag(a.status, SPARSTAR_STATUS_BAD_INDEX);
    const int seen = a.causal ? L - a.Lq + 1 + row : L;
    const int n_blocks = (L + kBlock - 1) / kBlock;
    const int kh = h / (a.Hq / c.Hkv);
    if (t < D) qs[t] = to_f32(static_cast<const T *>(a.q)[r * D + t]) * a.tau;
    const int32_t *list = nullptr;
    int tiles = n_blocks;
    if (a.kv_cnt) {
        const int64_t lr = ((int64_t)i * a.Hq + h) * ((a.Lq + kBlock - 1) / kBlock) + row / kBlock;
        list = a.kv_idx + lr * a.max_sel;
        tiles = a.kv_cnt[lr];
        tiles = tiles < 0 ? 0 : (tiles > a.max_sel ? a.max_sel : tiles);
    }
    float m = -INFINITY, l = 0.0f, acc = 0.0f;
    for (int j = 0; j < tiles; ++j) {
        const int blk = list ? list[j] : j;
        int page = -1;
        if (blk >= 0 && blk < n_blocks) page = c.table[(int64_t)slot * c.max_pages + blk];
        if (page < 0 || page >= c.n_pages) {
            if (t == 0) kv4_flag(a.status, SPARSTAR_STATUS_BAD_INDEX);
            continue;
        }
        if (blk * kBlock >= seen) continue;
        const uint8_t *half = c.pages + ((int64_t)page * c.Hkv + kh) * kv4_page_bytes(D);
        __syncthreads();  // qs written; ps of the tile before read
        float s = 0.0f;
        for (int w = 0; w < D / 8; ++w) {
            const uint32_t x = reinterpret_cast<const uint32_t *>(half)[t * (D / 8) + w];
            const float sc = kv4_scale(half[kv4_code_bytes(D) + t * G + w / 4]);
            for (int e = 0; e < 8; ++e)
                s = fmaf(qs[8 * w + e],
                         sc * (float)((int)((x >> (4 * kv4_nibble(e))) & 15u) - 8), s);
        }
        if (blk * kBlock + t >= seen) s = -INFINITY;
        float mx = s;
        for (int o = 16; o; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
        if (lane == 0) red[warp] = mx;
        __syncthreads();
        const float m_new = fmaxf(m, fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3])));
        const float p = expf(s - m_new);
        ps[t] = p;
        __syncthreads();
        const float f = expf(m - m_new);
        m = m_new;
        l *= f;
        acc *= f;
        const uint8_t *vh = half + kv4_half_bytes(D);
        for (int u = 0; u < kBlock; ++u) {
            l += ps[u];
            if (t < D) {
                const uint32_t x = reinterpret_cast<const uint32_t *>(vh)[t * 16 + u / 8];
                const float sc = kv4_scale(vh[kv4_code_bytes(D) + (t / kGroup) * kBlock + u]);
                acc = fmaf(ps[u], sc * (float)((int)((x >> (4 * kv4_nibble(u & 7))) & 15u) - 8),
                           acc);
            }
        }
        __syncthreads();
    }
    if (t < D) store(static_cast<T *>(a.out) + r * D + t, l > 0.0f ? acc / l : 0.0f);
    if (t == 0 && a.lse) a.lse[r] = m + logf(l);
}

}  // namespace

int64_t kv4_attn_work_bytes(int64_t, int64_t, int64_t, int64_t, int, int) { return 0; }

cudaError_t launch_kv4_attn(const Kv4 &c, const Kv4Attn &a, int dtype, cudaStream_t stream) {
    const unsigned grid = (unsigned)((int64_t)a.n * a.Hq * a.Lq);
    if (dtype == SPARSTAR_BF16) {
        if (c.D == 128) attn_row_kernel<__nv_bfloat16, 128><<<grid, kBlock, 0, stream>>>(c, a);
        else attn_row_kernel<__nv_bfloat16, 64><<<grid, kBlock, 0, stream>>>(c, a);
    } else {
        if (c.D == 128) attn_row_kernel<float, 128><<<grid, kBlock, 0, stream>>>(c, a);
        else attn_row_kernel<float, 64><<<grid, kBlock, 0, stream>>>(c, a);
    }
    return cudaGetLastError();
}

}  // namespace sparstar
