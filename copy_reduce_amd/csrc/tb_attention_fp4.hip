// tb_attention_fp4.hip -- attention over a paged cache held in 4 bits, or a window of it.
#include "tb_attention_kernels.h"

namespace tbk {

hipError_t launch_fp4_attention(const AttnArgs &g, uint32_t dtype, uint32_t dim, Shape s, uint32_t grid,
        hipStream_t stream) {
    return launch_kernel<true, true>(g, dtype, dim, s, grid, stream);
}

}  // namespace tbk
