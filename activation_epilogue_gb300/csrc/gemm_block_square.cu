// E4M3 products in blocks of 128, B with a scale for each 128 x 128 block: the CTA-pair kernel.
#include "gemm_block_pair.cuh"

namespace gemm_epi {

cudaError_t block_pair_square(int epilog, const GemmParams& p, int grid, cudaStream_t stream, bool pdl, bool prepare)
{
    return block_pair::launch_epilog<true>(epilog, p, grid, stream, pdl, prepare);
}

int block_pair_smem() { return block_pair::kSmemBytes; }
int block_pair_stages() { return block_pair::kStages; }

}  // namespace gemm_epi
