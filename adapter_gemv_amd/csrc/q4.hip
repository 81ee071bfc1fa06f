// Kernels of the products with 4-bit weights and group scales (gemm_items.h).
#include "q4_tiles.h"

namespace lora {
namespace {

template <class C, bool GROUPED, int KT>
__global__ __launch_bounds__(C::THREADS) __attribute__((amdgpu_waves_per_eu(C::EU))) void lora_q4_kernel(GemmDesc d) {
  __shared__ __align__(16) uint8_t lds[C::LDS];
  gemm_block<C, GROUPED, KT>(d, lds);
}

}  // namespace

int q4_tiles() { return kQ4Tiles; }

GemmTile q4_tile(bool gated, int cfg) {
  auto of = [](auto c) { return tile_of<decltype(c)>(c.WK == 8 ? 9 : c.RT <= 64 ? 6 : 16); };
  return gated ? with_q4_tile<true>(cfg, of) : with_q4_tile<false>(cfg, of);
}

void launch_q4(const GemmDesc &d, GemmKind kind, int cfg, int blocks, hipStream_t s) {
  with_q4_tile<false>(cfg, [&](auto c) {
    using C = decltype(c);
    if (kind == kGroupedQ4) lora_q4_kernel<C, true, 0><<<blocks, C::THREADS, 0, s>>>(d);
    else if (d.max_rank <= 32) lora_q4_kernel<C, false, 1><<<blocks, C::THREADS, 0, s>>>(d);
    else lora_q4_kernel<C, false, 2><<<blocks, C::THREADS, 0, s>>>(d);
  });
}

}  // namespace lora
