// Gate and up of binary16 rows in tiles, the codes widened: gemm_fp8_tile.h.  Compiled with the matrix
// instructions' results in vector registers (build_lib.py), where the multiply-adds take them.

#include "gemm_fp8_tile.h"

namespace pdq {

void launch_fp8_tiles_wide(const Fp8TileArgs& a, int rows, uint32_t tiles, hipStream_t st) {
    const dim3 grid(tiles), block(256);
    if (a.ws_f32) {
        if (rows == 128) hipLaunchKernelGGL((k_fp8_tile<kGateUp, 0, 2, 4, true, true>), grid, block, 0, st, a);
        else hipLaunchKernelGGL((k_fp8_tile<kGateUp, 0, 1, 4, true, true>), grid, block, 0, st, a);
    } else {
        if (rows == 128) hipLaunchKernelGGL((k_fp8_tile<kGateUp, 0, 2, 4, false, true>), grid, block, 0, st, a);
        else hipLaunchKernelGGL((k_fp8_tile<kGateUp, 0, 1, 4, false, true>), grid, block, 0, st, a);
    }
}

}  // namespace pdq
