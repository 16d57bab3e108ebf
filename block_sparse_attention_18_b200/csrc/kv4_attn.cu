// Attention over the paged 4-bit key/value cache: which kernel takes a call.
#include "kv4.cuh"

namespace sparstar {
namespace {

// Rows of a stripe from which the tcgen05 kernel, which multiplies 128 rows
// whatever it is given, takes over from the other one's 8 or 16 at a time, each
// of which unpacks the pages again.  Measured, 8 key heads, 17 to 32 rows (two
// times 16): four sequences of 8,000 tokens 37 (few) against 35 us, one of
// 72,000 67 against 67, 64 of 1,000 61 against 73; 40 rows, a third time more:
// 53 and 89 against 35 and 67.
constexpr int64_t kManyRows = 33;

bool many(const Kv4Shape &s, float tau) {
    // tau: the kernel takes the maximum of the scores before it scales them.
    // Rows: it counts them in 32 bits, past the last block's end.
    const int64_t rows = kv4_attn_many_rows(s);
    return rows >= kManyRows && rows < (1 << 30) && s.D == 128 && s.dtype == SPARSTAR_BF16 &&
           tau > 1e-30f;
}

}  // namespace

int64_t kv4_attn_work_bytes(const Kv4Shape &s) {
    const int64_t few = kv4_attn_few_work_bytes(s.D);
    const int64_t m = many(s, 1.0f) ? kv4_attn_many_work_bytes(s) : 0;
    return m > few ? m : few;
}

cudaError_t launch_kv4_attn(const Kv4 &c, const Kv4Attn &a, const Kv4Shape &s,
                            cudaStream_t stream) {
    if (many(s, a.tau)) return launch_kv4_attn_many(c, a, s, stream);
    return launch_kv4_attn_few(c, a, s.dtype, stream);
}

}  // namespace sparstar
