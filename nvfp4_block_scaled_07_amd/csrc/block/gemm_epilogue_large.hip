// The unsplit 256-row tiles of the block GEMMs (plan kinds 14 and 16 of the
// plain epilogue, 14 of the gated one), in a source of their own so that they
// take the iterative ILP instruction schedule of the plain GEMM's large tiles.
#include "epilogue_tile.h"

namespace nvfp4 {

typedef Cfg<256, 256, 2, 4, 32, 256, 2, 0, 1, 2, 16, 4> EpiTile256;          // 8 waves of 128x64
typedef Cfg<256, 192, 4, 2, 32, 256, 2, 0, 1, 2, 16, 4> EpiTile256x192;      // 8 waves of 64x96
typedef Cfg<256, 256, 2, 4, 32, 256, 2, 0, 1, 2, 16, 4, 0, 1> GatedTile256;  // 128 gate and 128 up columns

void launch_epilogue_large(int kind, const EpilogueLaunch& p, unsigned grid, hipStream_t stream) {
  if (kind == 16) launch_epilogue_tile<EpiTile256x192, false>(p, grid, stream);
  else launch_epilogue_tile<EpiTile256, false>(p, grid, stream);
}

void launch_gated_large(const EpilogueLaunch& p, bool quantize, unsigned grid, hipStream_t stream) {
  if (quantize) launch_epilogue_tile<GatedTile256, true>(p, grid, stream);
  else launch_epilogue_tile<GatedTile256, false>(p, grid, stream);
}

}  // namespace nvfp4
