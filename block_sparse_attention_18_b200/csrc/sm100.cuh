// What the tcgen05 attention kernels (head dim 128, 128 x 128 tiles) share:
// tile constants, PTX helpers, bounded waits, tensor maps.  Every source that
// includes this gets its own copies.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cudaTypedefs.h>

#include "sparstar.h"
#include "sparstar_internal.h"

namespace sparstar {
namespace {

constexpr int kHD = 128;                      // head dim
constexpr int kTileBytes = kBlock * kHD * 2;  // 32 KB: one Q, K or V tile
constexpr int kPanelBytes = kTileBytes / 2;   // 16 KB: 128 rows x 64 columns
constexpr int kStages = 5;                    // K/V ring depth
constexpr uint64_t kTimeoutNs = 2000000000ull;

// Instruction descriptor, kind::f16: D fp32, A and B bf16, M = N = 128.
constexpr uint32_t make_idesc(bool b_mn_major) {
    return (1u << 4) | (1u << 7) | (1u << 10) | ((b_mn_major ? 1u : 0u) << 16) |
           ((uint32_t)(128 >> 3) << 17) | ((uint32_t)(128 >> 4) << 24);
}

// ------------------------------------------------------------ PTX helpers

__device__ __forceinline__ uint32_t smem_addr(const void *p) {
    return (uint32_t)__cvta_generic_to_shared(p);
}

__device__ __forceinline__ uint64_t globaltimer() {
    uint64_t t;
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
    return t;
}

__device__ __forceinline__ void mbar_init(uint32_t bar, uint32_t count) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}
__device__ __forceinline__ void mbar_expect_tx(uint32_t bar, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes)
                 : "memory");
}
__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
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

// Single-thread bounded wait.  False on timeout (flag raised) or when
// another role already raised the abort flag.  The polling loop is out of
// line; the common case (phase already complete) costs one try_wait.
__device__ __noinline__ bool wait1_slow(uint32_t bar, uint32_t parity,
                                        volatile int32_t *abort_flag, int32_t *status) {
    const uint64_t t0 = globaltimer();
    for (uint32_t it = 1;; ++it) {
        if (mbar_test(bar, parity)) return true;
        if ((it & 63u) == 0u) {
            if (*abort_flag) return false;
            if (globaltimer() - t0 > kTimeoutNs) {
                *abort_flag = 1;
                if (status) atomicOr(status, SPARSTAR_STATUS_TIMEOUT);
                return false;
            }
        }
    }
}

__device__ __forceinline__ bool wait1(uint32_t bar, uint32_t parity, volatile int32_t *abort_flag,
                                      int32_t *status) {
    return mbar_test(bar, parity) || wait1_slow(bar, parity, abort_flag, status);
}

// Bounded wait that ignores the abort flag: used on the way out, for work
// already issued (copies in flight, MMAs to drain).
__device__ __noinline__ void drain_wait(uint32_t bar, uint32_t parity) {
    if (mbar_test(bar, parity)) return;
    const uint64_t t0 = globaltimer();
    while (!mbar_test(bar, parity) && globaltimer() - t0 < kTimeoutNs) {
    }
}

// Warp-uniform bounded wait for warp-collective roles: the warp leaves
// together, so the .sync.aligned tcgen05 instructions after it stay
// converged.  Fast path inline (one try_wait per lane); polling out of line.
__device__ __noinline__ bool wait_warp_slow(uint32_t bar, uint32_t parity,
                                            volatile int32_t *abort_flag, int32_t *status) {
    const uint64_t t0 = globaltimer();
    for (uint32_t it = 0;; ++it) {
        const bool ok = mbar_test(bar, parity);
        if (__all_sync(0xffffffffu, ok)) return true;
        if ((it & 63u) == 63u) {
            int give_up = 0;
            if ((threadIdx.x & 31) == 0) {
                if (*abort_flag) {
                    give_up = 1;
                } else if (globaltimer() - t0 > kTimeoutNs) {
                    *abort_flag = 1;
                    if (status) atomicOr(status, SPARSTAR_STATUS_TIMEOUT);
                    give_up = 1;
                }
            }
            if (__shfl_sync(0xffffffffu, give_up, 0)) return false;
        }
    }
}
__device__ __forceinline__ bool wait_warp(uint32_t bar, uint32_t parity,
                                          volatile int32_t *abort_flag, int32_t *status) {
    if (__all_sync(0xffffffffu, mbar_test(bar, parity))) return true;
    return wait_warp_slow(bar, parity, abort_flag, status);
}

// L2 eviction policies for TMA loads: Q tiles are read once per CTA
// (evict first); K/V tiles, re-read by the other query blocks of the head,
// keep the normal policy.
__device__ __forceinline__ uint64_t policy_evict_first() {
    uint64_t p;
    asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(p));
    return p;
}
__device__ __forceinline__ uint64_t policy_evict_normal() {
    uint64_t p;
    asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(p));
    return p;
}

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap *map, uint32_t bar,
                                            int c0, int c1, int c2, uint64_t policy) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        ".L2::cache_hint [%0], [%1, {%3, %4, %5}], [%2], %6;" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1), "r"(c2), "l"(policy)
        : "memory");
}

__device__ __forceinline__ void tc_fence_before() {
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tc_fence_after() {
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}

// Shared-memory matrix descriptors, 128-byte swizzle, sm_100 format
// (version 1 at bit 46, layout type 2 = SWIZZLE_128B at bits 61-63).
// K-major: rows of 128 bytes, 8-row groups 1024 bytes apart (SBO).
__device__ __forceinline__ uint64_t desc_k_major(uint32_t saddr) {
    return (uint64_t)((saddr & 0x3FFFFu) >> 4) | ((uint64_t)1 << 16) |
           ((uint64_t)(1024 >> 4) << 32) | ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}
// MN-major (V as the B operand, N = head dim contiguous): 64-element
// panels 16 KB apart (LBO), 8-row groups along K 1024 bytes apart (SBO).
__device__ __forceinline__ uint64_t desc_mn_major(uint32_t saddr) {
    return (uint64_t)((saddr & 0x3FFFFu) >> 4) | ((uint64_t)(kPanelBytes >> 4) << 16) |
           ((uint64_t)(1024 >> 4) << 32) | ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}

__device__ __forceinline__ void mma_ss(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                       uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}
// A in tensor memory (P), B from shared memory (V).
__device__ __forceinline__ void mma_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc,
                                       uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}
__device__ __forceinline__ void mma_commit(uint32_t bar) {
    asm volatile(
        "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar)
        : "memory");
}

#define SPX_R8(i) "=r"(r[i]), "=r"(r[i + 1]), "=r"(r[i + 2]), "=r"(r[i + 3]), "=r"(r[i + 4]), \
                  "=r"(r[i + 5]), "=r"(r[i + 6]), "=r"(r[i + 7])
#define SPX_W8(i) "r"(r[i]), "r"(r[i + 1]), "r"(r[i + 2]), "r"(r[i + 3]), "r"(r[i + 4]), \
                  "r"(r[i + 5]), "r"(r[i + 6]), "r"(r[i + 7])

// 32 consecutive fp32 columns of this thread's TMEM lane.
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
        "%11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, "
        "%28, %29, %30, %31}, [%32];"
        : SPX_R8(0), SPX_R8(8), SPX_R8(16), SPX_R8(24)
        : "r"(taddr));
}
// 32 consecutive 32-bit columns of this thread's TMEM lane from registers.
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t *r) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, "
        "%10, %11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, "
        "%27, %28, %29, %30, %31, %32};" ::"r"(taddr),
        SPX_W8(0), SPX_W8(8), SPX_W8(16), SPX_W8(24)
        : "memory");
}
__device__ __forceinline__ void tmem_wait_ld() {
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}
// Register fence: the registers a tcgen05.ld wrote are only valid after
// tcgen05.wait::ld; routing them through an empty asm placed after the wait
// keeps the compiler from moving their uses above it.
#define SPX_RW8(i) "+r"(r[i]), "+r"(r[i + 1]), "+r"(r[i + 2]), "+r"(r[i + 3]), "+r"(r[i + 4]), \
                   "+r"(r[i + 5]), "+r"(r[i + 6]), "+r"(r[i + 7])
__device__ __forceinline__ void reg_fence(uint32_t (&r)[32]) {
    asm volatile("" : SPX_RW8(0), SPX_RW8(8), SPX_RW8(16), SPX_RW8(24));
}
__device__ __forceinline__ void tmem_wait_st() {
    asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// True in exactly one lane of the (fully active) warp.
__device__ __forceinline__ bool elect_one() {
    uint32_t pred;
    asm volatile(
        "{\n\t.reg .b32 r;\n\t.reg .pred p;\n\t"
        "elect.sync r|p, 0xffffffff;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(pred));
    return pred != 0;
}

// Three-input maximum (one instruction on sm_100).
__device__ __forceinline__ float max3f(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);  // .x (low half) = lo
    return *reinterpret_cast<uint32_t *>(&h);
}

// 8 consecutive fp32 columns of this thread's TMEM lane (the rare O rescale
// uses these narrow chunks so that a full row of scores stays in registers).
__device__ __forceinline__ void tmem_ld8(uint32_t taddr, uint32_t (&r)[8]) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]),
                   "=r"(r[6]), "=r"(r[7])
                 : "r"(taddr));
}
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t (&r)[8]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};"
                 ::"r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]),
                   "r"(r[6]), "r"(r[7])
                 : "memory");
}

// Producer order (the order the MMA warps consume the tiles): K(A,0),
// K(B,0), then for j = 0, 1, ...: K(A,j+1), V(A,j), K(B,j+1), V(B,j), each
// present while its tile index is below that block's tile count.  The ring
// index of a tile is the number of tiles loaded before it; loads_before(j)
// counts the tiles ahead of step j's group.
__device__ __forceinline__ int imin(int a, int b) { return a < b ? a : b; }
__device__ __forceinline__ int loads_before(int j, int nA, int nB) {
    int c = (nA > 0) + (nB > 0);
    c += imin(j, nA - 1) > 0 ? imin(j, nA - 1) : 0;
    c += imin(j, nA);
    c += imin(j, nB - 1) > 0 ? imin(j, nB - 1) : 0;
    c += imin(j, nB);
    return c;
}
__device__ __forceinline__ int slot_k(int x, int j, int nA, int nB) {
    if (j == 0) return x == 0 ? 0 : (nA > 0 ? 1 : 0);
    const int g = j - 1, b = loads_before(g, nA, nB);
    return x == 0 ? b : b + (g + 1 < nA) + (g < nA);
}
__device__ __forceinline__ int slot_v(int x, int j, int nA, int nB) {
    const int b = loads_before(j, nA, nB);
    return x == 0 ? b + (j + 1 < nA) : b + (j + 1 < nA) + (j < nA) + (j + 1 < nB);
}
// The QK warp consumes the key tiles and the PV warp the value tiles, so a
// stage's previous occupant (slot e - kStages) can be the other warp's tile
// and still be in flight when this warp tests slot e; with one full barrier
// per stage a parity test cannot tell that state from "slot e landed".
// Each stage therefore has two full barriers, for its even and its odd
// uses: slot e waits on barrier (e / kStages) & 1 for that barrier's phase
// e / (2 kStages), whose previous phase is slot e - 2 kStages.  That slot
// has always landed before the test (the waits between the roles guarantee
// it for every pair of list lengths; tests/test_ring_protocol.py checks
// the happens-before chains), so the wait is exact.
__device__ __forceinline__ uint32_t ring_parity(int e) {
    return (uint32_t)(e / (2 * kStages)) & 1u;
}

// ------------------------------------------------------------------- host

PFN_cuTensorMapEncodeTiled_v12000 get_encoder() {
    static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    if (!fn) {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) ==
                cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
    }
    return fn;
}

// [BH, L, 128] bf16 viewed as a 3-D tensor; box = 64 columns x 128 rows x 1.
bool encode(CUtensorMap *map, const void *ptr, int64_t BH, int64_t L) {
    auto fn = get_encoder();
    if (!fn) return false;
    const cuuint64_t dims[3] = {(cuuint64_t)kHD, (cuuint64_t)L, (cuuint64_t)BH};
    const cuuint64_t strides[2] = {(cuuint64_t)kHD * 2, (cuuint64_t)L * kHD * 2};
    const cuuint32_t box[3] = {64, (cuuint32_t)kBlock, 1};
    const cuuint32_t estr[3] = {1, 1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(ptr), dims, strides,
              box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace
}  // namespace sparstar
