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
