// Tiled FP8 products with binary32 scales of the weights: gemm_fp8_tile.h.  Compiled with the matrix
// instructions' results in vector registers (build_lib.py), where the multiply-adds take them.

#include "gemm_fp8_tile.h"

namespace pdq {

void launch_fp8_tiles_f32(const Fp8TileArgs& a, int epi, int out_dt, Fp8TileShape tile, uint32_t tiles, hipStream_t st) {
    const dim3 grid(tiles), block(256);
    if (epi == kDense && out_dt == kF16) {
        if (tile.rows == 192) hipLaunchKernelGGL((k_fp8_tile<kDense, kF16, 3, 4, true>), grid, block, 0, st, a);
        else hipLaunchKernelGGL((k_fp8_tile<kDense, kF16, 2, 2, true>), grid, block, 0, st, a);
    } else if (epi == kDense) {
        if (tile.rows == 192) hipLaunchKernelGGL((k_fp8_tile<kDense, kBF16, 3, 4, true>), grid, block, 0, st, a);
        else hipLaunchKernelGGL((k_fp8_tile<kDense, kBF16, 2, 2, true>), grid, block, 0, st, a);
    } else if (epi == kGateUp) {
        if (tile.rows == 192) hipLaunchKernelGGL((k_fp8_tile<kGateUp, 0, 3, 4, true>), grid, block, 0, st, a);
        else if (tile.rows == 128) hipLaunchKernelGGL((k_fp8_tile<kGateUp, 0, 2, 4, true>), grid, block, 0, st, a);
        else hipLaunchKernelGGL((k_fp8_tile<kGateUp, 0, 1, 4, true>), grid, block, 0, st, a);
    } else {
        if (tile.rows == 192) hipLaunchKernelGGL((k_fp8_tile<kDown, 0, 3, 4, true>), grid, block, 0, st, a);
        else hipLaunchKernelGGL((k_fp8_tile<kDown, 0, 2, 2, true>), grid, block, 0, st, a);
    }
}

}  // namespace pdq
