// fp4 (OCP E2M1) GEMM kernel instances with OCP MX block scales: 256x256x256
// and 128x128x256 tiles (128-byte rows, like the 128-deep fp8 tiles).
#include "skg_inst_gemm_common.hpp"

namespace skg {
namespace {
template <int TM, int TN>
GemmInst f4_tile() {
  typedef TileCfg<DT_F4, TM, TN, 256, 2, 2, 32, 128, true> Cfg;
  return {&launch_instance<Cfg, GemmMxProblem<Cfg>>, &occupancy_instance<Cfg, GemmMxProblem<Cfg>>};
}
}  // namespace

GemmInst gemm_instance_f4(int tile_id) {
  if (tile_id == SKG_TILE_256x256x256) return f4_tile<256, 256>();
  if (tile_id == SKG_TILE_128x128x256) return f4_tile<128, 128>();
  return {nullptr, nullptr};
}
hipError_t wait_timeouts_gemm_f4(uint32_t* out, bool reset) { return unit_wait_timeouts(out, reset); }
}  // namespace skg
