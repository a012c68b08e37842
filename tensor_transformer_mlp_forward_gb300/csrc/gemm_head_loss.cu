// gemm_head_loss.cu -- the output head's GEMM instantiations: logits reduced
// to row statistics, the logits' gradient, and dX and dW of the head.
#include "kernels.h"

namespace tpmlp {

cudaError_t launch_head_lse(const GemmMaps& m, const GemmArgs& g, int grid, bool pair,
                            cudaStream_t st) {
    if (g.epi_warps == 8) {
        if (pair) return launch_gemm<false, false, EPI_LSE, true, 8>(m, g, grid, st);
        return launch_gemm<false, false, EPI_LSE, false, 8>(m, g, grid, st);
    }
    if (pair) return launch_gemm<false, false, EPI_LSE, true>(m, g, grid, st);
    return launch_gemm<false, false, EPI_LSE, false>(m, g, grid, st);
}

cudaError_t launch_head_dlogits(const GemmMaps& m, const GemmArgs& g, int grid, bool pair,
                                cudaStream_t st) {
    if (g.epi_warps == 8) {
        if (pair) return launch_gemm<false, false, EPI_DLOGITS, true, 8>(m, g, grid, st);
        return launch_gemm<false, false, EPI_DLOGITS, false, 8>(m, g, grid, st);
    }
    if (pair) return launch_gemm<false, false, EPI_DLOGITS, true>(m, g, grid, st);
    return launch_gemm<false, false, EPI_DLOGITS, false>(m, g, grid, st);
}

// dX reduces over the vocabulary or a piece of it, dW over the tokens: few
// tokens are a short reduction, whose stores eight warps hide better.
cudaError_t launch_head_dx(const GemmMaps& m, const GemmArgs& g, int grid, bool pair,
                           cudaStream_t st) {
    if (g.epi_warps == 8) {
        if (pair) return launch_gemm<false, true, EPI_SCALE, true, 8>(m, g, grid, st);
        return launch_gemm<false, true, EPI_SCALE, false, 8>(m, g, grid, st);
    }
    if (pair) return launch_gemm<false, true, EPI_SCALE, true>(m, g, grid, st);
    return launch_gemm<false, true, EPI_SCALE, false>(m, g, grid, st);
}

cudaError_t launch_head_dw(const GemmMaps& m, const GemmArgs& g, int grid, bool pair,
                           cudaStream_t st) {
    if (g.epi_warps == 8) {
        if (pair) return launch_gemm<true, true, EPI_SCALE, true, 8>(m, g, grid, st);
        return launch_gemm<true, true, EPI_SCALE, false, 8>(m, g, grid, st);
    }
    if (pair) return launch_gemm<true, true, EPI_SCALE, true>(m, g, grid, st);
    return launch_gemm<true, true, EPI_SCALE, false>(m, g, grid, st);
}

}  // namespace tpmlp
