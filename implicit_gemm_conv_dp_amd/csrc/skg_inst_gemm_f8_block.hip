// fp8 (OCP E4M3) and bf8 (OCP E5M2) GEMM kernel instances with an fp32 scale for
// each block of 128 elements of K.
#include "skg_f8_block.hpp"
#include "skg_inst_gemm_common.hpp"

namespace skg {
namespace {
template <int FMT, bool ROWS>
GemmInst block_by_tile(int tile_id) {
  switch (tile_id) {
    case SKG_TILE_16x16x128: return f8_direct<1, 1, 4, FMT, ROWS>();
    case SKG_TILE_16x32x128: return f8_direct<1, 2, 3, FMT, ROWS>();
    case SKG_TILE_32x32x128: return f8_direct<2, 2, 2, FMT, ROWS>();
    case SKG_TILE_32x64x128: return f8_direct<2, 4, 3, FMT, ROWS>();
    case SKG_TILE_64x64x128: return f8_direct<4, 4, 2, FMT, ROWS>();
    case SKG_TILE_128x128x128: return f8_ring<128, 128, 4, FMT, ROWS>();
    case SKG_TILE_256x128x128: return f8_ring<256, 128, 3, FMT, ROWS>();
    case SKG_TILE_256x256x128: return f8_ring<256, 256, 2, FMT, ROWS>();
    default: return {nullptr, nullptr};
  }
}
}  // namespace

GemmInst gemm_instance_f8_block(int tile_id, int dtype, bool rows) {
  if (dtype == SKG_F8E4M3) return rows ? block_by_tile<0, true>(tile_id) : block_by_tile<0, false>(tile_id);
  if (dtype == SKG_F8E5M2) return rows ? block_by_tile<1, true>(tile_id) : block_by_tile<1, false>(tile_id);
  return {nullptr, nullptr};
}
}  // namespace skg
