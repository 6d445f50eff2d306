// cache_attn_step64.cu -- the few-row kernels of cache_attn_step.cuh for heads of 64.
#include "cache_attn_step.cuh"

namespace gdr {
namespace cattn {

int launch_step64(const Attn &a, int codes, int dtype, void *ws, cudaStream_t s) {
    return launch_step_d<64>(a, codes, dtype, ws, s);
}
size_t step_bytes64() { return step_bytes_d<64>(); }

}  // namespace cattn
}  // namespace gdr
