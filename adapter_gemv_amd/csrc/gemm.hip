// Kernels of the int8 base projection and the grouped dense products
// (gemm_items.h): one kernel per kind and tile configuration, and the row
// quantiser.
#include "gemm_items.h"

namespace lora {
namespace {

template <class C, bool GROUPED, int KT>
__global__ __launch_bounds__(C::THREADS) __attribute__((amdgpu_waves_per_eu(C::EU))) void lora_gemm_kernel(GemmDesc d) {
  __shared__ __align__(16) uint8_t lds[C::LDS];
  gemm_block<C, GROUPED, KT>(d, lds);
}

__global__ __launch_bounds__(256) void quantize_rows_kernel(QuantDesc qd) {
  __shared__ float red[4];
  __shared__ int badv[4];
  const auto &in = (*(const QuantDesc *)(const void *)__builtin_amdgcn_kernarg_segment_ptr()).in[blockIdx.y];
  const int row = blockIdx.x, t = threadIdx.x;
  if (row >= in.rows) return;  // the grid covers the input with the most rows
  const uint16_t *x = in.x + (int64_t)row * in.ldx;
  const int n8 = in.d_in / 8;  // pieces of 8 values
  u32x4 keep[kQuantRegs];
  float mx = 0.f;
  bool bad = false;
#pragma unroll
  for (int i = 0; i < kQuantRegs; ++i) {
    const int p = i * 256 + t;
    keep[i] = p < n8 ? *(const u32x4 *)(x + (int64_t)p * 8) : zero4();
  }
#pragma unroll
  for (int i = 0; i < kQuantRegs; ++i) mx = abs_max8(keep[i], mx, &bad);
  for (int p = kQuantRegs * 256 + t; p < n8; p += 256) mx = abs_max8(*(const u32x4 *)(x + (int64_t)p * 8), mx, &bad);
#pragma unroll
  for (int k = 32; k >= 1; k /= 2) mx = fmaxf(mx, __shfl_xor(mx, k, 64));
  const bool wbad = __ballot(bad) != 0;
  if ((t & 63) == 0) {
    red[t >> 6] = mx;
    badv[t >> 6] = wbad;
  }
  __syncthreads();
  mx = fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
  const bool nan = badv[0] | badv[1] | badv[2] | badv[3];
  const bool live = mx > 0.f && !nan;
  int8_t *q = in.q + (int64_t)row * in.pitch;
#pragma unroll
  for (int i = 0; i < kQuantRegs; ++i) {
    const int p = i * 256 + t;
    if (p < n8) *(u32x2 *)(q + (int64_t)p * 8) = live ? quant8(keep[i], mx) : u32x2{0u, 0u};
  }
  for (int p = kQuantRegs * 256 + t; p < n8; p += 256)
    *(u32x2 *)(q + (int64_t)p * 8) = live ? quant8(*(const u32x4 *)(x + (int64_t)p * 8), mx) : u32x2{0u, 0u};
  if (t == 0) {
    if (in.d_in < in.pitch) *(u32x2 *)(q + in.d_in) = u32x2{0u, 0u};  // the row's last half piece
    in.s[row] = nan ? __int_as_float(0x7fc00000) : mx / 127.f;
  }
}

//                         I8  RT   NC  WR WC WK  KB  S EU
template <bool I8> using Cfg16 = GemmCfg<I8, 16, 64, 1, 1, 4, 512, 2, 2>;
template <bool I8> using Cfg32 = GemmCfg<I8, 32, 64, 1, 1, 4, 256, 3, 2>;
template <bool I8> using Cfg64 = GemmCfg<I8, 64, 64, 2, 2, 1, 256, 2, 2>;
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
    case 3: launch<Cfg128<I8>, GROUPED, KT>(d, blocks, s); break;
    default: launch<Cfg256<I8>, GROUPED, KT>(d, blocks, s); break;
  }
}

}  // namespace

GemmTile gemm_tile(int cfg) {
  switch (cfg) {
    case 0: return {Cfg16<true>::RT, Cfg16<true>::NC};
    case 1: return {Cfg32<true>::RT, Cfg32<true>::NC};
    case 2: return {Cfg64<true>::RT, Cfg64<true>::NC};
    case 3: return {Cfg128<true>::RT, Cfg128<true>::NC};
    default: return {Cfg256<true>::RT, Cfg256<true>::NC};
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

hipError_t launch_quantize(const QuantDesc &d, int n_inputs, hipStream_t stream) {
  int rows = 0;
  for (int i = 0; i < n_inputs; ++i) rows = d.in[i].rows > rows ? d.in[i].rows : rows;
  if (rows <= 0) return hipSuccess;
  quantize_rows_kernel<<<dim3((unsigned)rows, (unsigned)n_inputs), 256, 0, stream>>>(d);
  return hipGetLastError();
}

}  // namespace lora
