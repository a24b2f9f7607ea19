// Tiled FP8 products with power-of-two scales, and the launches of both kinds: gemm_fp8_tile.h.

#include <algorithm>

#include "gemm_fp8_tile.h"

namespace pdq {

void launch_fp8_tiles(const Fp8TileArgs& a, int out_dt, int rows, hipStream_t st) {
    const uint32_t tiles = (uint32_t)((int64_t)((a.M + rows - 1) / rows) * ((a.N + BN - 1) / BN));
    if (a.ws_f32) {
        launch_fp8_tiles_f32(a, kDense, out_dt, rows, tiles, st);
        return;
    }
    if (rows == 256) {
        if (out_dt == kF16) hipLaunchKernelGGL((k_fp8_tile<kDense, kF16, 4, false>), dim3(tiles), dim3(256), 0, st, a);
        else hipLaunchKernelGGL((k_fp8_tile<kDense, kBF16, 4, false>), dim3(tiles), dim3(256), 0, st, a);
    } else {
        if (out_dt == kF16) hipLaunchKernelGGL((k_fp8_tile<kDense, kF16, 2, false>), dim3(tiles), dim3(256), 0, st, a);
        else hipLaunchKernelGGL((k_fp8_tile<kDense, kBF16, 2, false>), dim3(tiles), dim3(256), 0, st, a);
    }
}

void launch_fp8_expert_tiles(const Fp8TileArgs& a, bool gate_up, bool wide, int rows, hipStream_t st) {
    const int64_t some = std::min(a.sorted.total, a.sorted.experts);
    const int64_t most = (a.sorted.total + (rows - 1) * some) / rows;  // tiles of rows
    const uint32_t tiles = (uint32_t)(most * (gate_up ? (a.N + 127) / 128 : (a.N + BN - 1) / BN));
    if (wide) {
        launch_fp8_tiles_wide(a, rows, tiles, st);
        return;
    }
    if (a.ws_f32) {
        launch_fp8_tiles_f32(a, gate_up ? kGateUp : kDown, 0, rows, tiles, st);
        return;
    }
    if (rows == 256) {
        if (gate_up) hipLaunchKernelGGL((k_fp8_tile<kGateUp, 0, 4, false>), dim3(tiles), dim3(256), 0, st, a);
        else hipLaunchKernelGGL((k_fp8_tile<kDown, 0, 4, false>), dim3(tiles), dim3(256), 0, st, a);
    } else if (rows == 128) {
        if (gate_up) hipLaunchKernelGGL((k_fp8_tile<kGateUp, 0, 2, false>), dim3(tiles), dim3(256), 0, st, a);
        else hipLaunchKernelGGL((k_fp8_tile<kDown, 0, 2, false>), dim3(tiles), dim3(256), 0, st, a);
    } else {
        if (gate_up) hipLaunchKernelGGL((k_fp8_tile<kGateUp, 0, 1, false>), dim3(tiles), dim3(256), 0, st, a);
        else hipLaunchKernelGGL((k_fp8_tile<kDown, 0, 1, false>), dim3(tiles), dim3(256), 0, st, a);
    }
}

}  // namespace pdq
