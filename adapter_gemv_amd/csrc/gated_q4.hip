// Kernels of the gated half of a feed-forward block with 4-bit weights
// (gemm_items.h).
#include "q4_tiles.h"

namespace lora {
namespace {

template <class C, bool GROUPED, int KT>
__global__ __launch_bounds__(C::THREADS) __attribute__((amdgpu_waves_per_eu(C::EU))) void lora_gated_q4_kernel(GemmDesc d) {
  __shared__ __align__(16) uint8_t lds[C::LDS];
  gemm_block<C, GROUPED, KT>(d, lds);
}

}  // namespace

void launch_gated_q4(const GemmDesc &d, GemmKind kind, int cfg, int blocks, hipStream_t s) {
  with_q4_tile<true>(cfg, [&](auto c) {
    using C = decltype(c);
    if (kind == kGroupedGatedQ4) lora_gated_q4_kernel<C, true, 0><<<blocks, C::THREADS, 0, s>>>(d);
    else if (d.max_rank <= 32) lora_gated_q4_kernel<C, false, 1><<<blocks, C::THREADS, 0, s>>>(d);
    else lora_gated_q4_kernel<C, false, 2><<<blocks, C::THREADS, 0, s>>>(d);
  });
}

}  // namespace lora
