// Tiled FP8 products with power-of-two scales, and the launches of both kinds: gemm_fp8_tile.h.

#include <algorithm>

#include "gemm_fp8_tile.h"

namespace pdq {

void launch_fp8_tiles(const Fp8TileArgs& a, int out_dt, Fp8TileShape tile, hipStream_t st) {
    const uint32_t tiles = (uint32_t)((int64_t)((a.M + tile.rows - 1) / tile.rows) * ((a.N + tile.channels - 1) / tile.channels));
    const dim3 grid(tiles), block(256);
    if (a.ws_f32) {
        launch_fp8_tiles_f32(a, kDense, out_dt, tile, tiles, st);
    } else if (tile.rows == 256) {
        if (out_dt == kF16) hipLaunchKernelGGL((k_fp8_tile<kDense, kF16, 4, 4, false>), grid, block, 0, st, a);
        else hipLaunchKernelGGL((k_fp8_tile<kDense, kBF16, 4, 4, false>), grid, block, 0, st, a);
    } else if (tile.channels == 256) {
        if (out_dt == kF16) hipLaunchKernelGGL((k_fp8_tile<kDense, kF16, 2, 4, false>), grid, block, 0, st, a);
        else hipLaunchKernelGGL((k_fp8_tile<kDense, kBF16, 2, 4, false>), grid, block, 0, st, a);
    } else {
        if (out_dt == kF16) hipLaunchKernelGGL((k_fp8_tile<kDense, kF16, 2, 2, false>), grid, block, 0, st, a);
        else hipLaunchKernelGGL((k_fp8_tile<kDense, kBF16, 2, 2, false>), grid, block, 0, st, a);
    }
}

namespace {

// The most tiles that the sorted rows can make.
uint32_t expert_tiles(const Fp8TileArgs& a, Fp8TileShape tile) {
    const int64_t some = std::min(a.sorted.total, a.sorted.experts);
    return (uint32_t)((a.sorted.total + (tile.rows - 1) * some) / tile.rows * ((a.N + tile.channels - 1) / tile.channels));
}

}  // namespace

void launch_fp8_gate_up_tiles(const Fp8TileArgs& a, bool wide, int rows, hipStream_t st) {
    const Fp8TileShape tile{rows, 128};  // of gate, and of up
    const uint32_t tiles = expert_tiles(a, tile);
    const dim3 grid(tiles), block(256);
    if (wide) launch_fp8_tiles_wide(a, rows, tiles, st);
    else if (a.ws_f32) launch_fp8_tiles_f32(a, kGateUp, 0, tile, tiles, st);
    else if (rows == 256) hipLaunchKernelGGL((k_fp8_tile<kGateUp, 0, 4, 4, false>), grid, block, 0, st, a);
    else if (rows == 128) hipLaunchKernelGGL((k_fp8_tile<kGateUp, 0, 2, 4, false>), grid, block, 0, st, a);
    else hipLaunchKernelGGL((k_fp8_tile<kGateUp, 0, 1, 4, false>), grid, block, 0, st, a);
}

void launch_fp8_down_tiles(const Fp8TileArgs& a, Fp8TileShape tile, hipStream_t st) {
    const uint32_t tiles = expert_tiles(a, tile);
    const dim3 grid(tiles), block(256);
    if (a.ws_f32) launch_fp8_tiles_f32(a, kDown, 0, tile, tiles, st);
    else if (tile.rows == 256) hipLaunchKernelGGL((k_fp8_tile<kDown, 0, 4, 4, false>), grid, block, 0, st, a);
    else hipLaunchKernelGGL((k_fp8_tile<kDown, 0, 2, 2, false>), grid, block, 0, st, a);
}

}  // namespace pdq
