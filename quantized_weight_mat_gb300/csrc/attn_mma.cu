// The decode-step attention kernel as pq_attn runs it.

#include "attn_mma.cuh"

namespace pqk {

unsigned attn_mma_wait_timeouts(bool reset) {
    unsigned v = 0;
    if (cudaMemcpyFromSymbol(&v, g_wait_timeouts, sizeof(v)) != cudaSuccess) return 0;
    if (reset) {
        const unsigned z = 0;
        cudaMemcpyToSymbol(g_wait_timeouts, &z, sizeof(z));
    }
    return v;
}

size_t attn_mma_ws_bytes(int d) { return attn_splits_bytes() + 2 * kAttnMaxGrid * attn_part_floats(16, d) * 4; }

cudaError_t launch_attn_mma(int dt, const AttnArgs &a, int rows, cudaStream_t s, const DeviceInfo &dev) {
    return launch_dt<false>(dt, a, rows, s, dev);
}

}  // namespace pqk
