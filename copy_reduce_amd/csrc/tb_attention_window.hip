// tb_attention_window.hip -- attention over a window of the paged cache, in 16 bits.
#include "tb_attention_kernels.h"

namespace tbk {

hipError_t launch_window_attention(const AttnArgs &g, uint32_t dtype, uint32_t dim, Shape s, uint32_t grid,
        hipStream_t stream) {
    return launch_kernel<true, false>(g, dtype, dim, s, grid, stream);
}

}  // namespace tbk
