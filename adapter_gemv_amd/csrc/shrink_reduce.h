// The sum of a shrink's k-chunk partials into one v per row.
#pragma once

#include "device_common.h"

namespace lora {

// Sum the k-chunk partials of each row in a segment into v[b][0..max_rank)
// (zero past the entry's rank), for module `module` into the plane
// v_out + module * num_rows * ldv; `block` counts blocks of 256 values.  The
// LayerDesc is the kernel's first argument (kernel_desc).  by_place: to the row's
// place in the order of the slots instead of its place in the batch.
__device__ __forceinline__ void shrink_reduce(const LayerDesc &d, int block, int module, bool by_place = false) {
  const int nseg = min(*d.num_segments, d.max_seg);
  if (nseg <= 0) return;
  const int nvalid = min(d.seg_offsets[nseg], d.num_rows);
  const int64_t idx = (int64_t)block * 256 + threadIdx.x;
  const int p = (int)(idx / d.max_rank);
  const int j = (int)(idx - (int64_t)p * d.max_rank);
  if (p >= nvalid) return;
  int lo = 0, hi = nseg - 1;  // segment s with seg_offsets[s] <= p < seg_offsets[s+1]
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (d.seg_offsets[mid] <= p) lo = mid;
    else hi = mid - 1;
  }
  const ModuleDesc m = kernel_desc().mod[module];
  float *v_out = d.v_out + (int64_t)module * d.num_rows * d.ldv;
  const int a = d.seg_adapter[lo];
  if ((unsigned)a >= (unsigned)d.num_slots) return;
  const lora_adapter_entry_t e = d.table[(int64_t)a * d.table_cols + m.col];  // varies per lane
  // a segment that does not fit the batch was skipped by the shrink: no delta
  const int o0 = d.seg_offsets[lo], o1 = d.seg_offsets[lo + 1];
  const bool ok = entry_ok(e, d.max_rank) && o0 >= 0 && o0 <= p && p < o1 && o1 <= d.num_rows;
  float sum = 0.f;
  if (ok && j < e.rank)
    for (int c = 0; c < m.n_chunks; ++c) sum += d.part[((int64_t)(m.part_base + c) * d.num_rows + p) * d.rs + j];
  const int b = d.perm[p];
  if ((unsigned)b < (unsigned)d.num_rows) v_out[(int64_t)(by_place ? p : b) * d.ldv + j] = sum;
}

}  // namespace lora
