// Kernels of the int8 base projection and the grouped dense products
// (gemm_items.h): one kernel per kind and tile configuration, and the row
// quantiser.
#include "gemm_items.h"
#include "shrink_reduce.h"

namespace lora {
namespace {

template <class C, bool GROUPED, int KT>
__global__ __launch_bounds__(C::THREADS) __attribute__((amdgpu_waves_per_eu(C::EU))) void lora_gemm_kernel(GemmDesc d) {
  __shared__ __align__(16) uint8_t lds[C::LDS];
  gemm_block<C, GROUPED, KT>(d, lds);
}

__global__ __launch_bounds__(256) void quantize_rows_kernel(QuantDesc qd) {
  quantize_block(qd, *(const QuantDesc *)(const void *)__builtin_amdgcn_kernarg_segment_ptr(), blockIdx.x);
}

// Between the grouped shrink and the product of an int8 layer call: the rows'
// quantiser and the rows by slot, which need nothing of the shrink, and the sum
// of the shrink's partials, in one launch (each apart is 4 us of a small
// call's 25).
__global__ __launch_bounds__(256) void quantize_reduce_kernel(LayerDesc d, QuantDesc qd, int reduce_blocks,
                                                              const int32_t *ids, int32_t *order) {
  constexpr int kAt = (sizeof(LayerDesc) + 7) / 8 * 8;  // where the second argument lies
  // the rows' order first: its last block counts over all the ids before it
  const int order_blocks = order ? (d.num_rows + 255) / 256 : 0;
  int b = blockIdx.x;
  if (b < order_blocks) {
    order_block(d, ids, order, b);
    return;
  }
  b -= order_blocks;
  if (b < qd.blocks) {
    quantize_block(qd, *(const QuantDesc *)((const char *)(const void *)__builtin_amdgcn_kernarg_segment_ptr() + kAt), b);
  } else {
    const int module = (b - qd.blocks) / reduce_blocks;
    shrink_reduce(d, b - qd.blocks - module * reduce_blocks, module);
  }
}

// The tiles.  Measured on one MI355X (us; in brackets what was taken):
//  * 16 rows: 32 slots, 128 rows, 8192 x 8192 bf16 (4.3 GB of weights), by
//    columns x stages x blocks per unit at 512 bytes of k a stage:
//    [64 x 2 x 2: 749], 32 x 2 x 3: 800, 32 x 3 x 2: 868, 32 x 6 x 1: 1040,
//    128 x 2 x 1: 779; 1024 bytes of k: 859.  Two blocks on a unit overlap one
//    another's start and end, which a deeper ring of one block does not.
//  * 32 rows: 16 slots x 24 rows, 8192 x 8192, int8 and bf16: [64 columns, 256
//    bytes, 3 stages: 191, 385], 8 waves on 512 bytes: 198, 361 to 388, 32
//    columns on 512 bytes: 203, 345.
//  * 64 rows: 16 slots x 64 rows, bf16: [256 bytes, 2 stages: 425], 128 bytes, 4
//    stages: 453; 128 columns: 459; int8 216 to 219 either way.
//  * 128 rows: 128 columns on 8 waves, 4 stages, one block a unit; 96 columns on
//    4 waves, 2 stages, two blocks (see pick_gemm).  A whole layer's int8 base and delta: [676
//    and 712], 128 columns with 5 stages 683, 256 bytes x 2 stages 692, 2
//    stages and two blocks 746, 64 columns 732, 256 columns 780.
//  * 256 x 256 on 4 waves of 128 x 128 (gemm_block): 8192 x 8192 x 8192 bf16 758
//    us (1.45 PFLOP/s; torch.mm on the same card 674), 16384 of each 6.04 ms
//    (1.46 PFLOP/s; 5.50), int8 with the quantiser 446 us and 3.20 ms (2.47 and
//    2.75 POP/s; 441 us and 3.68 ms).  The counters show the matrix cores busy for 70% of the
//    cycles of a prefill at the 1.8 GHz its power leaves.  8 waves of 128 x 64
//    with no operands ahead: 1.05 PFLOP/s on the grouped prefill against 1.2.
//  * Registers: every kernel fits but the 256 x 256 ones, whose sums and operands
//    fill both files, and the 128 x 128 one at ranks above 32.  Spilled before
//    the main loop and read back in the epilogue: int8 base above rank 32, 33
//    (136 bytes a lane; its product takes 4.35 ms of a rank 64 prefill, 4.04 at
//    rank 16); grouped int8 3, grouped bf16 1; the 128 x 128 one 1.
//                                           I8  RT   NC  WR WC WK  KB  S EU
template <bool I8> using Cfg16 = GemmCfg<I8, 16, 64, 1, 1, 4, 512, 2, 2>;
template <bool I8> using Cfg32 = GemmCfg<I8, 32, 64, 1, 1, 4, 256, 3, 2>;
template <bool I8> using Cfg64 = GemmCfg<I8, 64, 64, 2, 2, 1, 256, 2, 2>;
template <bool I8> using Cfg128n = GemmCfg<I8, 128, 96, 2, 2, 1, 128, 2, 2>;
template <bool I8> using Cfg128 = GemmCfg<I8, 128, 128, 4, 2, 1, 128, 4, 2>;
template <bool I8> using Cfg256 = GemmCfg<I8, 256, 256, 2, 2, 1, 128, 2, 1, true>;

template <class C, bool GROUPED, int KT>
void launch(const GemmDesc &d, int blocks, hipStream_t s) {
  lora_gemm_kernel<C, GROUPED, KT><<<blocks, C::THREADS, 0, s>>>(d);
}
template <bool I8, bool GROUPED, int KT>
void pick(const GemmDesc &d, int cfg, int blocks, hipStream_t s) {
  switch (cfg) {
    case 0: launch<Cfg16<I8>, GROUPED, KT>(d, blocks, s); break;
    case 1: launch<Cfg32<I8>, GROUPED, KT>(d, blocks, s); break;
    case 2: launch<Cfg64<I8>, GROUPED, KT>(d, blocks, s); break;
    case 3: launch<Cfg128n<I8>, GROUPED, KT>(d, blocks, s); break;
    case 4: launch<Cfg128<I8>, GROUPED, KT>(d, blocks, s); break;
    default: launch<Cfg256<I8>, GROUPED, KT>(d, blocks, s); break;
  }
}

}  // namespace

namespace {
template <class C>
constexpr GemmTile tile_of(double fixed) {
  return {C::RT, C::NC, 160 * 1024 / C::LDS, fixed, 0.3 * C::MT * C::NTE / C::DT};
}
}  // namespace

GemmTile gemm_tile(int cfg) {
  switch (cfg) {
    case 0: return tile_of<Cfg16<true>>(6);
    case 1: return tile_of<Cfg32<true>>(6);
    case 2: return tile_of<Cfg64<true>>(6);
    case 3: return tile_of<Cfg128n<true>>(8);
    case 4: return tile_of<Cfg128<true>>(8);
    default: return tile_of<Cfg256<true>>(16);
  }
}

hipError_t launch_gemm(const GemmDesc &d, GemmKind kind, int cfg, int blocks, hipStream_t stream) {
  if (blocks <= 0) return hipSuccess;
  switch (kind) {
    case kLinearI8:
      if (d.max_rank <= 32) pick<true, false, 1>(d, cfg, blocks, stream);
      else pick<true, false, 2>(d, cfg, blocks, stream);
      break;
    case kGroupedBf16: pick<false, true, 0>(d, cfg, blocks, stream); break;
    default: pick<true, true, 0>(d, cfg, blocks, stream); break;
  }
  return hipGetLastError();
}

hipError_t launch_quantize(const QuantDesc &d, hipStream_t stream) {
  if (d.blocks <= 0) return hipSuccess;
  quantize_rows_kernel<<<d.blocks, 256, 0, stream>>>(d);
  return hipGetLastError();
}

hipError_t launch_quantize_reduce(const LayerDesc &d, const QuantDesc &q, const int32_t *ids, int32_t *order,
                                  hipStream_t stream) {
  const int64_t reduce = ((int64_t)d.num_rows * d.max_rank + 255) / 256;
  const int64_t blocks = q.blocks + reduce * d.n_active + (order ? (d.num_rows + 255) / 256 : 0);
  if (blocks <= 0) return hipSuccess;
  if (blocks > 0x7fffffff) return hipErrorInvalidValue;
  quantize_reduce_kernel<<<(unsigned)blocks, 256, 0, stream>>>(d, q, (int)reduce, ids, order);
  return hipGetLastError();
}

}  // namespace lora
