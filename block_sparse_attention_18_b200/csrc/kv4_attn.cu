// Attention over the paged 4-bit key/value cache: which kernel takes a call.
#include "kv4.cuh"

namespace sparstar {

int64_t kv4_attn_work_bytes(int64_t, int64_t, int64_t, int64_t, int D, int) {
    return kv4_attn_few_work_bytes(D);
}

cudaError_t launch_kv4_attn(const Kv4 &c, const Kv4Attn &a, int dtype, cudaStream_t stream) {
    return launch_kv4_attn_few(c, a, dtype, stream);
}

}  // namespace sparstar
