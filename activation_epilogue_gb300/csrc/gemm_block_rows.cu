// E4M3 products in blocks of 128, B with a scale for each row and block: the CTA-pair kernel.
#include "gemm_block_pair.cuh"

namespace gemm_epi {

cudaError_t block_pair_rows(int epilog, const GemmParams& p, int grid, cudaStream_t stream, bool pdl, bool prepare)
{
    return block_pair::launch_epilog<false>(epilog, p, grid, stream, pdl, prepare);
}

}  // namespace gemm_epi
