// cache_attn_step128.cu -- the few-row kernels of cache_attn_step.cuh for heads of 128.
#include "cache_attn_step.cuh"

namespace gdr {
namespace cattn {

int launch_step128(const Attn &a, int codes, int dtype, void *ws, cudaStream_t s) {
    return launch_step_d<128>(a, codes, dtype, ws, s);
}
size_t step_bytes128() { return step_bytes_d<128>(); }

}  // namespace cattn
}  // namespace gdr
