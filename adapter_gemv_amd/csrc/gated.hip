// Kernels of the gated half of a feed-forward block with bf16 weights
// (gemm_items.h): both projections, the activation and the product in one.
#include "gemm_items.h"

namespace lora {
namespace {

template <class C, bool GROUPED, int KT>
__global__ __launch_bounds__(C::THREADS) __attribute__((amdgpu_waves_per_eu(C::EU))) void lora_gated_kernel(GemmDesc d) {
  __shared__ __align__(16) uint8_t lds[C::LDS];
  gemm_block<C, GROUPED, KT>(d, lds);
}

// The tiles; NC counts gate's and up's columns.  One MI355X, us of a pass with the
// adapters, gate and up of 8192 x 28672, by tile: 1 row [163], 173, 168, 177; 16
// rows [177], 187, 185, 196; 48 rows 494, 366, [220], 222; 128 rows over 128
// adapters of rank 16 1293, 732, 468, [262], 414 (1.18 GB with their B, 4.7 TB/s of
// the whole call); 7637 rows 256 x 256 [5826], 128 x 128 8596 (1.22 PFLOP/s with
// the epilogue; the matrix cores busy for 60% of the cycles).  128 rows x 96
// columns, two blocks a unit, 343 where 128 x 128 takes 262: not kept.  Registers:
// 256 x 256 by slot spills 2, the others none.
//                   I8     RT   NC  WR WC WK  KB  S EU  PIPE   Q4    GATED
using Gated16 = GemmCfg<false, 16, 64, 1, 1, 4, 512, 2, 2, false, false, true>;
using Gated32 = GemmCfg<false, 32, 64, 1, 1, 4, 256, 3, 2, false, false, true>;
using Gated64 = GemmCfg<false, 64, 64, 2, 2, 1, 256, 2, 2, false, false, true>;
using Gated128 = GemmCfg<false, 128, 128, 4, 2, 1, 128, 4, 2, false, false, true>;
using Gated256 = GemmCfg<false, 256, 256, 2, 2, 1, 128, 2, 1, true, false, true>;

template <class C>
void launch(const GemmDesc &d, GemmKind kind, int blocks, hipStream_t s) {
  if (kind == kGroupedGatedBf16) lora_gated_kernel<C, true, 0><<<blocks, C::THREADS, 0, s>>>(d);
  else if (d.max_rank <= 32) lora_gated_kernel<C, false, 1><<<blocks, C::THREADS, 0, s>>>(d);
  else lora_gated_kernel<C, false, 2><<<blocks, C::THREADS, 0, s>>>(d);
}

}  // namespace

int gated_tiles() { return 5; }

GemmTile gated_tile(int cfg) {
  switch (cfg) {
    case 0: return tile_of<Gated16>(6);
    case 1: return tile_of<Gated32>(6);
    case 2: return tile_of<Gated64>(6);
    case 3: return tile_of<Gated128>(8);
    default: return tile_of<Gated256>(16);
  }
}

void launch_gated(const GemmDesc &d, GemmKind kind, int cfg, int blocks, hipStream_t s) {
  switch (cfg) {
    case 0: launch<Gated16>(d, kind, blocks, s); break;
    case 1: launch<Gated32>(d, kind, blocks, s); break;
    case 2: launch<Gated64>(d, kind, blocks, s); break;
    case 3: launch<Gated128>(d, kind, blocks, s); break;
    default: launch<Gated256>(d, kind, blocks, s); break;
  }
}

}  // namespace lora
