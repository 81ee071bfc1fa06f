// What a base product with adapters (gated.hip, q4.hip, gated_q4.hip) needs of the
// batch's rows before it starts: v = A_a x of every projection, and of each row
// its adapter's B, rank, scale and format.  Found here once, they cost the product
// one load a row; found by its blocks (ids, segments, table, v: four loads that
// wait for one another, behind the weights already requested) they held each block
// back by 2 us before its first product and by 1 to 2 us after its last.
#include "gemm_items.h"
#include "shrink_reduce.h"

namespace lora {
namespace {

__device__ __forceinline__ RowInfo describe(const LayerDesc &d, int b, int a, bool on, const lora_adapter_entry_t &e) {
  RowInfo ri{};
  ri.b = b;
  ri.a = -1;
  if (on && entry_ok(e, d.max_rank)) {  // a malformed entry gives no delta
    ri.a = a;
    ri.rank = e.rank;
    ri.fmt = (int16_t)e.format;
    ri.scale = e.scale;
    ri.B = static_cast<const uint8_t *>(e.B);
  }
  return ri;
}

// Row b of the batch at `place` of its order.
__device__ __forceinline__ void place_row(const RowsDesc &r, int place, int b, int last) {
  const LayerDesc &d = r.L;
  if (r.order) r.order[place] = b;
  const bool in = (unsigned)b < (unsigned)d.num_rows;  // segments of another batch: the place holds no row
  const int a = in ? r.ids[b] : -1;
  const bool on = in && has_segment(d, a, last);
  for (int m = 0; m < d.n_active; ++m) {
    lora_adapter_entry_t e{};
    if (on) e = d.table[(int64_t)a * d.table_cols + kernel_desc().mod[m].col];
    r.info[(int64_t)m * d.num_rows + place] = describe(d, in ? b : -1, a, on, e);
  }
}

// 256 rows.
__device__ __forceinline__ void rows_block(const RowsDesc &r, int block) {
  const int last = last_slot(r.L);
  if (r.order) {
    by_slot_block(r.L, r.ids, block, [&](int place, int b) { place_row(r, place, b, last); });
  } else {
    const int b = block * 256 + threadIdx.x;
    if (b < r.L.num_rows) place_row(r, b, b, last);
  }
}

__global__ __launch_bounds__(256) void rows_kernel(RowsDesc r) {
  int b = blockIdx.x;
  if (b < r.rows_blocks) {
    rows_block(r, b);
    return;
  }
  b -= r.rows_blocks;
  const int module = b / r.reduce_blocks;
  shrink_reduce(r.L, b - module * r.reduce_blocks, module, r.order != nullptr);
}

// A few rows: a block for every row, projection and row of A, straight from the
// ids; instead of the grouped shrink, its partials and their sum (two launches, 16
// us of a token's 4-bit gate and up).  Rows that share an adapter read it again,
// from L2.
__global__ __launch_bounds__(256) void few_rows_kernel(RowsDesc r) {
  __shared__ float red[4];
  const LayerDesc &d = r.L;
  const int t = threadIdx.x, lane = t & 63, w = wave_id();
  const int per = d.num_rows * d.max_rank;
  const int module = (int)blockIdx.x / per, rest = (int)blockIdx.x - module * per;
  const int b = rest / d.max_rank, j = rest - b * d.max_rank;
  const ModuleDesc m = kernel_desc().mod[module];
  // ids and number of segments; then the entry, the last segment and x; then A: what
  // can be read at once is asked for at once
  const int a = uniform(r.ids[b]);
  const int nseg = min(uniform(*d.num_segments), d.max_seg);
  const bool valid = (unsigned)a < (unsigned)d.num_slots;
  const lora_adapter_entry_t raw = d.table[(int64_t)(valid ? a : 0) * d.table_cols + m.col];
  int last = nseg > 0 ? uniform(d.seg_adapter[nseg - 1]) : -1;
  if (nseg > 0 && uniform(d.seg_offsets[nseg]) > d.num_rows) last = uniform(last_slot(d));  // built for more rows
  const bool on = has_segment(d, a, last);
  lora_adapter_entry_t e{};
  if (on) {
    e.A = uniform(raw.A);
    e.B = uniform(raw.B);
    e.rank = uniform(raw.rank);
    e.scale = uniform(raw.scale);
    e.format = uniform(raw.format);
  }
  if (blockIdx.x == 0 && w == 0) {  // segments that do not fit the batch, once a call
    for (int s = lane; s < nseg; s += 64) {
      if (!segment_fits(d.seg_adapter[s], d.seg_offsets[s], d.seg_offsets[s + 1], d.num_slots, d.num_rows))
        atomicAdd(d.status, 1);
    }
  }
  if (j == 0 && t == 0) {
    r.info[(int64_t)module * d.num_rows + b] = describe(d, b, a, on, e);
    if (on && e.rank != 0 && !entry_ok(e, d.max_rank)) {  // counted by the slot's first row
      bool first = true;
      for (int k = 0; k < b; ++k) first &= r.ids[k] != a;
      if (first) atomicAdd(d.status, 1);
    }
  }
  if (!on || !entry_ok(e, d.max_rank) || j >= e.rank) return;  // (columns past the rank are not read)
  const u32x4 *x = reinterpret_cast<const u32x4 *>(m.x + (int64_t)b * m.ldx);
  const int n8 = m.d_in / 8;
  float sum = 0.f, scale = 1.f;
  if (e.format == LORA_FORMAT_BF16) {
    const u32x4 *A = reinterpret_cast<const u32x4 *>(static_cast<const uint16_t *>(e.A) + (int64_t)j * m.d_in);
#pragma unroll 4
    for (int i = t; i < n8; i += 256) sum = dot8_bf16(A[i], x[i], sum);
  } else {
    const uint8_t *A = static_cast<const uint8_t *>(e.A);
    scale = reinterpret_cast<const float *>(A)[j];
    const u32x2 *q = reinterpret_cast<const u32x2 *>(A + q8_values_offset(e.rank) + (int64_t)j * lda8_of(m.d_in));
#pragma unroll 4
    for (int i = t; i < n8; i += 256) sum = dot8_bf16(i8x8_to_bf16x8(q[i]), x[i], sum);
  }
#pragma unroll
  for (int k = 32; k >= 1; k /= 2) sum += __shfl_xor(sum, k, 64);
  if (lane == 0) red[w] = sum;
  __syncthreads();
  if (t == 0)
    d.v_out[((int64_t)module * d.num_rows + b) * d.ldv + j] = ((red[0] + red[1]) + (red[2] + red[3])) * scale;
}

}  // namespace

hipError_t launch_rows(RowsDesc &d, bool few, hipStream_t stream) {
  const int64_t values = (int64_t)d.L.num_rows * d.L.max_rank;
  if (few) {
    few_rows_kernel<<<(unsigned)(values * d.L.n_active), 256, 0, stream>>>(d);
    return hipGetLastError();
  }
  d.rows_blocks = (d.L.num_rows + 255) / 256;
  d.reduce_blocks = (int)((values + 255) / 256);
  const int64_t blocks = d.rows_blocks + (int64_t)d.reduce_blocks * d.L.n_active;
  if (blocks > 0x7fffffff) return hipErrorInvalidValue;
  rows_kernel<<<(unsigned)blocks, 256, 0, stream>>>(d);
  return hipGetLastError();
}

}  // namespace lora
