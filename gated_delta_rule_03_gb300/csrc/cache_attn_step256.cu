// cache_attn_step256.cu -- the few-row kernels of cache_attn_step.cuh for heads of 256.
#include "cache_attn_step.cuh"

namespace gdr {
namespace cattn {

int launch_step256(const Attn &a, int codes, int dtype, void *ws, cudaStream_t s) {
    return launch_step_d<256>(a, codes, dtype, ws, s);
}
size_t step_bytes256() { return step_bytes_d<256>(); }

}  // namespace cattn
}  // namespace gdr
