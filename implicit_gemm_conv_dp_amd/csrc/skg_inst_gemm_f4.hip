// fp4 (OCP E2M1) GEMM kernel instances with OCP MX block scales: the ring
// kernel's tiles, the two of them that the stream-K engine runs too (128-byte
// rows, like the 128-deep fp8 tiles), and the direct kernel's.
#include "skg_f4_direct.hpp"
#include "skg_f4_tile.hpp"
#include "skg_inst_gemm_common.hpp"

namespace skg {
namespace {
template <class T>
GemmInst f4_ring() {
  return {[](const GemmParams& g, const KPlan& p, const Scratch&, hipStream_t st, hipEvent_t ev0, hipEvent_t ev1) {
            hipError_t e;
            if (ev0 && (e = hipEventRecord(ev0, st)) != hipSuccess) return e;
            if ((e = f4_tile_launch<T>(g, p, st)) != hipSuccess) return e;
            return ev1 ? hipEventRecord(ev1, st) : hipSuccess;
          },
          [](int* out) { return hipOccupancyMaxActiveBlocksPerMultiprocessor(out, f4_tile_kernel<T>, 256, 0); }};
}
// A tile that has the engine's modes too.
template <int TM, int TN, int D>
GemmInst f4_tile() {
  typedef TileCfg<DT_F4, TM, TN, 256, 2, 2, 32, 128, true> Cfg;
  return {[](const GemmParams& g, const KPlan& p, const Scratch& s, hipStream_t st, hipEvent_t ev0, hipEvent_t ev1) {
            return p.mode == MODE_DP ? f4_ring<F4Tile<TM, TN, D>>().launch(g, p, s, st, ev0, ev1)
                                     : launch_instance<Cfg, GemmMxProblem<Cfg>>(g, p, s, st, ev0, ev1);
          },
          &occupancy_instance<Cfg, GemmMxProblem<Cfg>>};
}
}  // namespace

GemmInst gemm_instance_f4(int tile_id) {
  switch (tile_id) {
    case SKG_TILE_256x256x256: return f4_tile<256, 256, 2>();
    case SKG_TILE_128x128x256: return f4_tile<128, 128, 4>();
    case SKG_TILE_16x16x512: return f4_direct<1, 1>();
    case SKG_TILE_16x32x512: return f4_direct<1, 2>();
    case SKG_TILE_16x64x512: return f4_direct<1, 4>();
    case SKG_TILE_32x32x512: return f4_direct<2, 2>();
    case SKG_TILE_32x64x512: return f4_direct<2, 4>();
    case SKG_TILE_48x32x512: return f4_direct<3, 2>();
    case SKG_TILE_64x64x512: return f4_direct<4, 4>();
    case SKG_TILE_256x128x256: return f4_ring<F4Tile<256, 128, 2>>();
    default: return {nullptr, nullptr};
  }
}
hipError_t wait_timeouts_gemm_f4(uint32_t* out, bool reset) { return unit_wait_timeouts(out, reset); }
}  // namespace skg
