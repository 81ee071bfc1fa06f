// C ABI of the LoRA-delta library: argument checks, work decomposition and
// launches.  Every check runs before the first HIP call, so a rejected call
// touches neither the device nor the stream.
#include <algorithm>
#include <cmath>
#include <stddef.h>
#include <stdint.h>

#include <mutex>
#include <type_traits>

#include "lora_internal.h"

using namespace lora;

namespace {

bool aligned16(const void *p) { return ((uintptr_t)p & 15) == 0; }

lora_status_t check_segments(const lora_segments_t &seg) {
  if (!seg.perm || !seg.seg_offsets || !seg.seg_adapter || !seg.num_segments || !seg.status || !seg.tile_counts)
    return LORA_ERR_NULL;
  if (seg.max_segments < 0) return LORA_ERR_SHAPE;
  return LORA_OK;
}

// The most segments a batch can have: one per row, one per slot, and the
// caller's bound when it gives one.
int segment_bound(int num_rows, int num_slots, const lora_segments_t &seg) {
  int b = num_rows < num_slots ? num_rows : num_slots;
  if (seg.max_segments > 0 && seg.max_segments < b) b = seg.max_segments;
  return b;
}

size_t ws_need(int num_rows, int num_slots, int max_rank, int64_t sum_d_in) {  // covers every call
  const size_t a = segments_ws_bytes(num_rows, num_slots);
  const size_t b = partials_ws_bytes(num_rows, max_rank, sum_d_in);
  return a > b ? a : b;
}

// The workspace checks of a call whose own scratch is `need` bytes (0: the
// call needs no workspace and *scratch is null).
lora_status_t check_ws(void *ws, size_t ws_bytes, size_t need, void **scratch) {
  *scratch = nullptr;
  if (need == 0) return LORA_OK;
  if (!ws) return LORA_ERR_NULL;
  if (!aligned16(ws)) return LORA_ERR_ALIGN;
  if (ws_bytes < need) return LORA_ERR_WORKSPACE;
  *scratch = ws;
  return LORA_OK;
}

struct ModuleArgs {
  const void *x;
  int64_t ldx;
  void *y;
  int64_t ldy;
  int32_t d_in;
  int32_t d_out;
  int32_t col;
  bool int8_items = false;  // the call's LORA_MASK_INT8_ITEMS: items sized for one-byte factors
};

// Work decomposition: the n-tile of the decode expand.  An item takes the
// largest tile the kernel stages in LDS (2048 outputs at rank class 64, 4096
// below: 256 KiB of bf16 B at the class's rank, half that in int8, where the
// fixed cost of an item weighs more); batches that would give fewer than 1024
// items take smaller tiles (down to one sub-tile of 16 load passes), so the
// work spreads over the device.  Measured on the Zipf batch of 101 adapters
// of mixed rank (q/k/v/o, rank class 64): 512-output tiles 39.7 us, 1024
// 33.9 us, 2048 40.8 us, which a threshold of 2048, 1024 and 512 items
// gives.
int pick_nt(int max_rank, int64_t max_seg, const ModuleArgs *ms, int n) {
  const int cls = max_rank <= 8 ? 8 : max_rank <= 16 ? 16 : max_rank <= 32 ? 32 : 64;
  const int lpr = cls / 8;
  const int sub = 16 * kDecodeThreads / lpr;
  int nt = decode_expand_tile(lpr);
  if (nt < sub) nt = sub;
  while (nt > sub) {
    int64_t items = 0;
    for (int i = 0; i < n; ++i) items += (ms[i].d_out + nt - 1) / nt;
    if (max_seg * items >= 1024) break;
    nt /= 2;
  }
  return nt;
}

// Fill the descriptor for a set of modules; items are k-chunks (shrink) or
// n-tiles (expand).
lora_status_t launched(hipError_t e) { return e == hipSuccess ? LORA_OK : LORA_ERR_LAUNCH; }

// Shrink k-chunk.  Prefill-sized batches: 2 * kKChunkMin (fewer partials to
// write and sum).  Decode batches: about 128 KiB of A per item at the
// launch's rank class (1024 k at rank 64, longer below; four times the k,
// at most 4 * kKChunkMin, when the caller states int8 factors,
// LORA_MASK_INT8_ITEMS), halved while the batch would give fewer than 512
// items, never below kKChunkMin (the workspace is sized for that chunk).
// Measured on the 70B layer at rank 64 with int8 factors: shrink 137 -> 109
// us with 2048 k instead of 1024, and 106 -> 102 us with 4096 (and bf16
// factors 186 -> 196 us at 2048: the hint is the caller's).
int pick_kc(int num_rows, int max_rank, int64_t max_seg, const ModuleArgs *ms, int n) {
  if (num_rows >= kPrefillRows) return 2 * kKChunkMin;
  const int cls = max_rank <= 8 ? 8 : max_rank <= 16 ? 16 : max_rank <= 32 ? 32 : 64;
  int kc = kKChunkMin * (64 / cls) * (n > 0 && ms[0].int8_items ? 4 : 1);
  if (kc > 4 * kKChunkMin) kc = 4 * kKChunkMin;
  while (kc > kKChunkMin) {
    int64_t items = 0;
    for (int i = 0; i < n; ++i) items += (ms[i].d_in + kc - 1) / kc;
    if (max_seg * items >= 512) break;
    kc /= 2;
  }
  return kc;
}

// Fill the descriptor: items per segment are k-chunks (shrink) or decode
// n-tiles (expand); sg_* give the SGMV expand n-tiles per row tile.
void fill_desc(LayerDesc &d, const ModuleArgs *ms, int n, bool shrink, int num_rows, int num_slots, int max_rank,
               int table_cols, const lora_adapter_entry_t *table, const lora_segments_t &seg, void *ws) {
  d = LayerDesc{};
  const int max_seg = segment_bound(num_rows, num_slots, seg);
  d.kc = pick_kc(num_rows, max_rank, max_seg, ms, n);
  d.nt = pick_nt(max_rank, max_seg, ms, n);
  d.sg_nt = num_rows >= kPrefillRows ? kSgmvExpandCols : kSgmvExpandColsSmall;
  int item = 0, chunk = 0, sg = 0;
  for (int i = 0; i < n; ++i) {
    ModuleDesc &m = d.mod[i];
    m.x = static_cast<const uint16_t *>(ms[i].x);
    m.ldx = ms[i].ldx;
    m.y = static_cast<uint16_t *>(ms[i].y);
    m.ldy = ms[i].ldy;
    m.d_in = ms[i].d_in;
    m.d_out = ms[i].d_out;
    m.col = ms[i].col;
    m.n_chunks = m.d_in > 0 ? (m.d_in + d.kc - 1) / d.kc : 0;
    m.part_base = chunk;
    chunk += m.n_chunks;
    m.n_items = shrink ? m.n_chunks : (m.d_out + d.nt - 1) / d.nt;
    m.item_base = item;
    item += m.n_items;
    m.sg_n_items = (m.d_out + d.sg_nt - 1) / d.sg_nt;
    m.sg_item_base = sg;
    sg += m.sg_n_items;
  }
  d.n_active = n;
  d.items_per_seg = item;
  d.sg_items = sg;
  d.table_cols = table_cols;
  d.rs = partial_row_stride(max_rank);
  d.num_rows = num_rows;
  d.num_slots = num_slots;
  d.max_rank = max_rank;
  d.long_min = num_rows >= kLongSegRows ? kLongSegRows : 0x7fffffff;
  d.max_seg = max_seg;
  d.perm = seg.perm;
  d.seg_offsets = seg.seg_offsets;
  d.seg_adapter = seg.seg_adapter;
  d.num_segments = seg.num_segments;
  d.tile_counts = seg.tile_counts;
  d.status = seg.status;
  d.table = table;
  d.part = static_cast<float *>(ws);
}

// The SGMV kernels address an activation matrix with 32-bit byte offsets.
bool fits_u32(int64_t rows, int64_t ld) { return rows * ld * 2 <= (int64_t)0xFFFFFF00; }

// A prefill batch's partials are summed once into their first chunk after
// the shrink (fold_partials_kernel): every SGMV expand tile of a row tile
// (d_out / 1024 of them per projection) would otherwise sum all the chunks
// again, and the tiles of one row tile run on different XCDs, so each
// fetches them from HBM.
bool folds_partials(const LayerDesc &d) {
  if (d.num_rows < kPrefillRows) return false;
  for (int i = 0; i < d.n_active; ++i)
    if (d.mod[i].n_chunks > 1) return true;
  return false;
}

// Launch one phase (shrink or expand) over every module: decode items for
// every possible segment and SGMV items for every row tile that segments of
// at least kLongSegRows rows can produce (the kernels put the tiles the
// build counted first and let the rest of that room exit).  fold: the
// phase's partials pass from this call's shrink to its expand (not to a
// caller's v or the fused kernel's planes), so a prefill batch folds them.
lora_status_t launch_phase(bool shrink, const ModuleArgs *ms, int n, int num_rows, int num_slots, int max_rank,
                           int table_cols, const lora_adapter_entry_t *table, const lora_segments_t &seg, void *ws,
                           const float *v_in, int64_t ldv, hipStream_t s, bool fold = false) {
  LayerDesc d;
  fill_desc(d, ms, n, shrink, num_rows, num_slots, max_rank, table_cols, table, seg, ws);
  d.v = v_in;
  d.ldv = ldv;
  const bool folded = fold && v_in == nullptr && folds_partials(d);
  if (folded && !shrink)
    for (int i = 0; i < n; ++i) d.mod[i].n_chunks = 1;  // the sums wait in each module's first chunk
  // a call counts each bad segment and entry once: the shrink of a layer call,
  // or lora_expand on the caller's v
  d.count_errors = shrink || v_in != nullptr;
  const int64_t dec = (int64_t)d.max_seg * d.items_per_seg;
  int64_t sg = 0;
  if (num_rows >= kLongSegRows)
    sg = (int64_t)long_tiles_max(num_rows, d.max_seg, shrink ? sgmv_shrink_rows() : sgmv_expand_rows()) *
         (shrink ? d.items_per_seg : d.sg_items);
  if (dec + sg > 0x7fffffff) return LORA_ERR_SHAPE;
  const hipError_t e = shrink ? launch_shrink(d, (int)dec, (int)(dec + sg), s) : launch_expand(d, (int)dec, (int)(dec + sg), s);
  const lora_status_t st = launched(e);
  if (st != LORA_OK || !(folded && shrink)) return st;
  return launched(launch_fold_partials(d, s));
}

// Common checks of the layer calls; fills the module list.
lora_status_t check_layer(const lora_module_io_t *io, uint32_t module_mask, int32_t num_rows,
                          const lora_adapter_entry_t *table, int32_t num_slots, const lora_segments_t &seg,
                          int32_t max_rank, void *ws, size_t ws_bytes, ModuleArgs *ms, int *n_out,
                          void **scratch, int64_t *sum_d_in_out = nullptr) {
  if (!io || !table) return LORA_ERR_NULL;
  lora_status_t st = check_segments(seg);
  if (st != LORA_OK) return st;
  const bool int8_items = (module_mask & LORA_MASK_INT8_ITEMS) != 0;
  module_mask &= ~LORA_MASK_INT8_ITEMS;
  if (module_mask == 0 || module_mask >= (1u << LORA_NUM_MODULES)) return LORA_ERR_MODULE;
  if (num_rows < 0 || num_slots < 1) return LORA_ERR_SHAPE;
  if (max_rank < 1 || max_rank > LORA_MAX_RANK) return LORA_ERR_RANK;
  int n = 0;
  int64_t sum_d_in = 0;
  for (int c = 0; c < LORA_NUM_MODULES; ++c) {
    if (!(module_mask & (1u << c))) continue;
    const lora_module_io_t &m = io[c];
    if (!m.x || !m.y) return LORA_ERR_NULL;
    if (m.d_in <= 0 || m.d_out <= 0 || m.ldx < m.d_in || m.ldy < m.d_out) return LORA_ERR_SHAPE;
    if ((m.d_in & 7) || (m.d_out & 7) || (m.ldx & 7) || (m.ldy & 7) || !aligned16(m.x) || !aligned16(m.y))
      return LORA_ERR_ALIGN;
    if (!fits_u32(num_rows, m.ldx) || !fits_u32(num_rows, m.ldy)) return LORA_ERR_SHAPE;
    ms[n] = ModuleArgs{m.x, m.ldx, m.y, m.ldy, m.d_in, m.d_out, c, int8_items};
    sum_d_in += m.d_in;
    ++n;
  }
  st = check_ws(ws, ws_bytes, partials_ws_bytes(num_rows, max_rank, sum_d_in), scratch);
  if (st != LORA_OK) return st;
  *n_out = n;
  if (sum_d_in_out) *sum_d_in_out = sum_d_in;
  return LORA_OK;
}

lora_status_t layer_phase(bool do_shrink, bool do_expand, const lora_module_io_t *io, uint32_t module_mask,
                          int32_t num_rows, const lora_adapter_entry_t *table, int32_t num_slots,
                          lora_segments_t seg, int32_t max_rank, void *ws, size_t ws_bytes, void *stream) {
  ModuleArgs ms[LORA_NUM_MODULES];
  int n = 0;
  void *scratch = nullptr;
  lora_status_t st =
      check_layer(io, module_mask, num_rows, table, num_slots, seg, max_rank, ws, ws_bytes, ms, &n, &scratch);
  if (st != LORA_OK) return st;
  if (num_rows == 0) return LORA_OK;
  ws = scratch;
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (do_shrink) {
    st = launch_phase(true, ms, n, num_rows, num_slots, max_rank, LORA_NUM_MODULES, table, seg, ws, nullptr, 0, s,
                      true);
    if (st != LORA_OK) return st;
  }
  if (do_expand)
    st = launch_phase(false, ms, n, num_rows, num_slots, max_rank, LORA_NUM_MODULES, table, seg, ws, nullptr, 0, s,
                      true);
  return st;
}

// Bytes of a row of int8 values (a multiple of 16), and of the quantised rows
// of sum_d_in inputs in n matrices with their scales.
int i8_pitch(int d_in) { return (d_in + 15) & ~15; }
size_t quant_ws_bytes(int64_t num_rows, int64_t sum_d_in, int n) {
  const size_t per = (size_t)(sum_d_in + 16 * (int64_t)n) * (size_t)num_rows;
  return per + (size_t)n * ((size_t)num_rows * 4 + 512);
}

// The rows by slot.
size_t order_ws_bytes(int num_rows) { return ((size_t)num_rows * 4 + 255) & ~(size_t)255; }

// The end of the v planes of a fused layer call's workspace (a multiple of
// 256): the int8 form's quantised rows follow.
size_t linear_v_end(int num_rows, int max_rank, int64_t sum_d_in, int n_modules) {
  const size_t part = (partials_ws_bytes(num_rows, max_rank, sum_d_in) + 255) & ~(size_t)255;
  return (part + (size_t)n_modules * num_rows * partial_row_stride(max_rank) * 4 + 255) & ~(size_t)255;
}

}  // namespace

extern "C" {

size_t lora_workspace_bytes(int32_t num_rows, int32_t num_slots, int32_t max_rank, int64_t sum_d_in) {
  if (num_rows < 0 || num_slots < 1 || max_rank < 1 || max_rank > LORA_MAX_RANK || sum_d_in < 0) return 0;
  return ws_need(num_rows, num_slots, max_rank, sum_d_in);
}

// The int8 form's: the fused layer's, then the rows by slot and the quantised
// rows.
size_t lora_linear_i8_workspace_bytes(int32_t num_rows, int32_t num_slots, int32_t max_rank, int64_t sum_d_in,
                                      int32_t n_modules) {
  const size_t base = lora_linear_workspace_bytes(num_rows, num_slots, max_rank, sum_d_in, n_modules);
  if (base == 0) return 0;
  const size_t need = linear_v_end(num_rows, max_rank, sum_d_in, n_modules) + order_ws_bytes(num_rows) +
                      quant_ws_bytes(num_rows, sum_d_in, n_modules);
  return need > base ? need : base;
}

size_t lora_grouped_workspace_bytes(int32_t num_rows, int32_t num_slots, int64_t sum_d_in, int32_t n_modules) {
  if (num_rows < 0 || num_slots < 1 || sum_d_in < 0 || n_modules < 1 || n_modules > LORA_NUM_MODULES) return 0;
  const size_t a = quant_ws_bytes(num_rows, sum_d_in, n_modules);
  const size_t b = segments_ws_bytes(num_rows, num_slots);
  return a > b ? a : b;
}

// The fused layer's workspace: the shrink's partials, then one v plane
// [num_rows][rs] per projection (256-byte aligned); at least the segment
// builder's.
size_t lora_linear_workspace_bytes(int32_t num_rows, int32_t num_slots, int32_t max_rank, int64_t sum_d_in,
                                   int32_t n_modules) {
  if (num_rows < 0 || num_slots < 1 || max_rank < 1 || max_rank > LORA_MAX_RANK || sum_d_in < 0 || n_modules < 1 ||
      n_modules > LORA_NUM_MODULES)
    return 0;
  const size_t part = (partials_ws_bytes(num_rows, max_rank, sum_d_in) + 255) & ~(size_t)255;
  const size_t vplanes = (size_t)n_modules * num_rows * partial_row_stride(max_rank) * 4;
  const size_t seg = segments_ws_bytes(num_rows, num_slots);
  return part + vplanes > seg ? part + vplanes : seg;
}

lora_status_t lora_build_segments(const int32_t *row_adapter, int32_t num_rows, int32_t num_slots,
                                  lora_segments_t seg, void *ws, size_t ws_bytes, void *stream) {
  lora_status_t st = check_segments(seg);
  if (st != LORA_OK) return st;
  if (num_rows < 0 || num_slots < 1) return LORA_ERR_SHAPE;
  if (num_rows > 0 && !row_adapter) return LORA_ERR_NULL;
  void *scratch = nullptr;
  st = check_ws(ws, ws_bytes, segments_ws_bytes(num_rows, num_slots), &scratch);
  if (st != LORA_OK) return st;
  return launched(launch_build_segments(row_adapter, 1, num_rows, num_slots, false, seg, scratch,
                                        static_cast<hipStream_t>(stream)));
}

lora_status_t lora_shrink(const void *x, int64_t ldx, int32_t num_rows, int32_t d_in,
                          const lora_adapter_entry_t *table, int32_t num_slots, int32_t n_mod, int32_t module,
                          lora_segments_t seg, int32_t max_rank, float *v, int64_t ldv, void *ws, size_t ws_bytes,
                          void *stream) {
  if (!x || !table || !v) return LORA_ERR_NULL;
  lora_status_t st = check_segments(seg);
  if (st != LORA_OK) return st;
  if (n_mod < 1 || n_mod > LORA_NUM_MODULES || module < 0 || module >= n_mod) return LORA_ERR_MODULE;
  if (max_rank < 1 || max_rank > LORA_MAX_RANK) return LORA_ERR_RANK;
  if (num_rows < 0 || num_slots < 1 || d_in <= 0 || ldx < d_in || ldv < max_rank) return LORA_ERR_SHAPE;
  if ((d_in & 7) || (ldx & 7) || (ldv & 3) || !aligned16(x) || !aligned16(v)) return LORA_ERR_ALIGN;
  if (!fits_u32(num_rows, ldx)) return LORA_ERR_SHAPE;
  void *scratch = nullptr;
  st = check_ws(ws, ws_bytes, partials_ws_bytes(num_rows, max_rank, d_in), &scratch);
  if (st != LORA_OK) return st;
  if (num_rows == 0) return LORA_OK;
  ws = scratch;
  ModuleArgs m{x, ldx, nullptr, 0, d_in, 0, module};
  hipStream_t s = static_cast<hipStream_t>(stream);
  st = launch_phase(true, &m, 1, num_rows, num_slots, max_rank, n_mod, table, seg, ws, nullptr, 0, s);
  if (st != LORA_OK) return st;
  LayerDesc d;
  fill_desc(d, &m, 1, true, num_rows, num_slots, max_rank, n_mod, table, seg, ws);
  d.v_out = v;
  d.ldv = ldv;
  return launched(launch_shrink_reduce(d, s));
}

lora_status_t lora_expand(const float *v, int64_t ldv, int32_t num_rows, int32_t d_out,
                          const lora_adapter_entry_t *table, int32_t num_slots, int32_t n_mod, int32_t module,
                          lora_segments_t seg, int32_t max_rank, void *y, int64_t ldy, void *ws, size_t ws_bytes,
                          void *stream) {
  if (!v || !table || !y) return LORA_ERR_NULL;
  lora_status_t st = check_segments(seg);
  if (st != LORA_OK) return st;
  if (n_mod < 1 || n_mod > LORA_NUM_MODULES || module < 0 || module >= n_mod) return LORA_ERR_MODULE;
  if (max_rank < 1 || max_rank > LORA_MAX_RANK) return LORA_ERR_RANK;
  if (num_rows < 0 || num_slots < 1 || d_out <= 0 || ldy < d_out || ldv < max_rank) return LORA_ERR_SHAPE;
  if ((d_out & 7) || (ldy & 7) || (ldv & 3) || !aligned16(y) || !aligned16(v)) return LORA_ERR_ALIGN;
  if (!fits_u32(num_rows, ldy)) return LORA_ERR_SHAPE;
  (void)ws;
  (void)ws_bytes;  // the expand of a caller-provided v needs no workspace
  if (num_rows == 0) return LORA_OK;
  ModuleArgs m{nullptr, 0, y, ldy, 0, d_out, module};
  return launch_phase(false, &m, 1, num_rows, num_slots, max_rank, n_mod, table, seg, ws, v, ldv,
                      static_cast<hipStream_t>(stream));
}

lora_status_t lora_layer_shrink(const lora_module_io_t *io, uint32_t module_mask, int32_t num_rows,
                                const lora_adapter_entry_t *table, int32_t num_slots, lora_segments_t seg,
                                int32_t max_rank, void *ws, size_t ws_bytes, void *stream) {
  return layer_phase(true, false, io, module_mask, num_rows, table, num_slots, seg, max_rank, ws, ws_bytes, stream);
}

lora_status_t lora_layer_expand(const lora_module_io_t *io, uint32_t module_mask, int32_t num_rows,
                                const lora_adapter_entry_t *table, int32_t num_slots, lora_segments_t seg,
                                int32_t max_rank, void *ws, size_t ws_bytes, void *stream) {
  return layer_phase(false, true, io, module_mask, num_rows, table, num_slots, seg, max_rank, ws, ws_bytes, stream);
}

lora_status_t lora_apply_layer(const lora_module_io_t *io, uint32_t module_mask, int32_t num_rows,
                               const lora_adapter_entry_t *table, int32_t num_slots, lora_segments_t seg,
                               int32_t max_rank, void *ws, size_t ws_bytes, void *stream) {
  return layer_phase(true, true, io, module_mask, num_rows, table, num_slots, seg, max_rank, ws, ws_bytes, stream);
}

}  // extern "C"

namespace {

// The one-launch plan of lora_decode_layer.  Each block of the one-launch
// kernel reads the whole A of its segment (its siblings, one per group of
// expand tiles, read the same lines through L2), so the plan bounds those
// repeated reads: at most kOnePassRepeatBytes over all projections, counting
// one pass over A per block of a segment and one more per 4 further rows
// (segments are at most the caller's bound, else one per row).  Measured on
// one MI355X (steps replayed from a HIP graph, one projection d x d, a
// distinct adapter per row, 16 to 256 rows, d 1024 to 8192, ranks 8 to 32):
// the launch beats the three launches of lora_build_segments +
// lora_apply_layer everywhere, by 2-3x up to 64 rows (4-9 us against 12-16
// us), 18.9 against 27.4 us for 128 rows x 8192 at rank 16, 39 against 42 us
// for 128 rows x 8192 at rank 32 (268 MB of repeated reads), and ties at the
// same 268 MB with 256 rows.  Batches of at most kOnePassMaxRows rows, ranks
// up to 32.  False for any other batch.
constexpr double kOnePassRepeatBytes = 320.0 * (1 << 20);
// Tiles per block grow while the blocks that work (one per row group and
// item) stay at least this many and the widest projection keeps at least
// two blocks per row group: every block of a group reads its A, so fewer
// blocks read A fewer times, until too few blocks share a row's tiles.
// Measured (graph-timed, a distinct adapter per row, 8192 x 8192): rank 32
// at 128 rows 39.5 us with 4 blocks per row, 32.0 with 2; rank 16 at 128
// rows 19.6 with 4, 19.1 with 2, 23.6 with 1 (bench); 256 rows of rank 16 at
// 4096 x 4096 14.9 with 2, 15.7 with 1; 128 rows over 32 adapters at rank 16
// 20.7 with 4 (128 working blocks), 24.7 with 2.
constexpr int64_t kOnePassMinWorking = 256;

bool onepass_plan(const ModuleArgs *ms, int n, int num_rows, const int32_t *ids, int num_slots, int max_rank,
                  const lora_adapter_entry_t *table, const lora_segments_t &seg, OnePassDesc *od, int *grid) {
  if (num_rows < 1 || num_rows > kOnePassMaxRows || max_rank > 32) return false;
  const int lpr = max_rank <= 8 ? 1 : max_rank <= 16 ? 2 : 4;
  const int nt = kOnePassPasses * (kDecodeThreads / lpr);
  const int max_seg = segment_bound(num_rows, num_slots, seg);
  // a bound below min(rows, slots) may drop segments: each block then ranks its slot in a bitmap of the slots
  const bool bound_check = max_seg < (num_rows < num_slots ? num_rows : num_slots);
  if (bound_check && num_slots > kOnePassMaxSlots) return false;
  const double passes = max_seg + (num_rows - max_seg + 3) / 4;
  // tiles per block (each block reads its segment's A once for all its tiles)
  auto items = [&](int tpb) {
    int64_t it = 0;
    for (int i = 0; i < n; ++i) it += ((ms[i].d_out + nt - 1) / nt + tpb - 1) / tpb;
    return it;
  };
  auto widest = [&](int tpb) {  // items of the projection with the most tiles
    int64_t w = 0;
    for (int i = 0; i < n; ++i) {
      const int64_t it = ((ms[i].d_out + nt - 1) / nt + tpb - 1) / tpb;
      w = it > w ? it : w;
    }
    return w;
  };
  int tpb = 1;
  while (tpb < 64 && items(2 * tpb) < items(tpb) && widest(2 * tpb) >= 2 &&
         items(2 * tpb) * passes >= kOnePassMinWorking)
    tpb *= 2;
  double repeat = 0;
  for (int i = 0; i < n; ++i)
    repeat += (double)(((ms[i].d_out + nt - 1) / nt + tpb - 1) / tpb) * ms[i].d_in * (8 * lpr) * 2 * passes;
  if (repeat > kOnePassRepeatBytes) return false;
  *od = OnePassDesc{};
  LayerDesc &d = od->L;
  d.nt = nt;
  int item = 0;
  for (int i = 0; i < n; ++i) {
    ModuleDesc &m = d.mod[i];
    m.x = static_cast<const uint16_t *>(ms[i].x);
    m.ldx = ms[i].ldx;
    m.y = static_cast<uint16_t *>(ms[i].y);
    m.ldy = ms[i].ldy;
    m.d_in = ms[i].d_in;
    m.d_out = ms[i].d_out;
    m.col = ms[i].col;
    m.op_nt = nt;
    m.op_n_tiles = (m.d_out + nt - 1) / nt;
    m.n_items = (m.op_n_tiles + tpb - 1) / tpb;
    m.item_base = item;
    item += m.n_items;
  }
  d.n_active = n;
  d.items_per_seg = item;
  d.table_cols = LORA_NUM_MODULES;
  d.num_rows = num_rows;
  d.num_slots = num_slots;
  d.max_rank = max_rank;
  d.long_min = 0x7fffffff;
  d.max_seg = segment_bound(num_rows, num_slots, seg);
  d.status = seg.status;
  d.table = table;
  od->seg = seg;
  od->ids = ids;
  od->row_slots = (num_rows + 7) / 8 * 8;
  od->bound_check = bound_check;
  od->tiles_per_block = tpb;
  const int64_t blocks = (int64_t)item * od->row_slots + 1;
  if (blocks > 0x7fffffff) return false;
  *grid = (int)blocks;
  return true;
}

}  // namespace

extern "C" {

// Segments and the layer delta of a decode batch: one launch when the batch
// fits the one-launch kernel, else lora_build_segments + lora_apply_layer.
lora_status_t lora_decode_layer(const lora_module_io_t *io, uint32_t module_mask, int32_t num_rows,
                                const int32_t *row_adapter, const lora_adapter_entry_t *table, int32_t num_slots,
                                lora_segments_t seg, int32_t max_rank, void *ws, size_t ws_bytes, void *stream) {
  ModuleArgs ms[LORA_NUM_MODULES];
  int n = 0;
  void *scratch = nullptr;
  lora_status_t st =
      check_layer(io, module_mask, num_rows, table, num_slots, seg, max_rank, ws, ws_bytes, ms, &n, &scratch);
  if (st != LORA_OK) return st;
  if (num_rows > 0 && !row_adapter) return LORA_ERR_NULL;
  void *seg_scratch = nullptr;
  st = check_ws(ws, ws_bytes, segments_ws_bytes(num_rows, num_slots), &seg_scratch);
  if (st != LORA_OK) return st;
  hipStream_t s = static_cast<hipStream_t>(stream);
  OnePassDesc od;
  int grid = 0;
  if (onepass_plan(ms, n, num_rows, row_adapter, num_slots, max_rank, table, seg, &od, &grid))
    return launched(launch_onepass(od, grid, s));
  st = launched(launch_build_segments(row_adapter, 1, num_rows, num_slots, false, seg, seg_scratch, s));
  if (st != LORA_OK || num_rows == 0) return st;
  // the three-launch path
  st = launch_phase(true, ms, n, num_rows, num_slots, max_rank, LORA_NUM_MODULES, table, seg, scratch, nullptr, 0, s,
                    true);
  if (st != LORA_OK) return st;
  return launch_phase(false, ms, n, num_rows, num_slots, max_rank, LORA_NUM_MODULES, table, seg, scratch, nullptr, 0,
                      s, true);
}

int32_t lora_decode_layer_launches(const lora_module_io_t *io, uint32_t module_mask, int32_t num_rows,
                                   int32_t num_slots, lora_segments_t seg, int32_t max_rank) {
  ModuleArgs ms[LORA_NUM_MODULES];
  int n = 0;
  void *scratch = nullptr;
  // the argument checks without a workspace (an aligned stand-in of any size)
  const lora_adapter_entry_t *table = reinterpret_cast<const lora_adapter_entry_t *>(uintptr_t{256});
  if (check_layer(io, module_mask, num_rows, table, num_slots, seg, max_rank, reinterpret_cast<void *>(uintptr_t{256}),
                  ~size_t{0} >> 1, ms, &n, &scratch) != LORA_OK)
    return 0;
  OnePassDesc od;
  int grid = 0;
  const int32_t *ids = reinterpret_cast<const int32_t *>(uintptr_t{256});
  return onepass_plan(ms, n, num_rows, ids, num_slots, max_rank, table, seg, &od, &grid) ? 1 : 3;
}

// One pass per position of the rows' adapter lists: the segments of that
// column, then the layer's shrink and expand, each pass adding its delta to y
// in stream order (a row is in one segment per pass, so no two blocks of a
// launch touch the same y).
lora_status_t lora_apply_layer_stacked(const lora_module_io_t *io, uint32_t module_mask, int32_t num_rows,
                                       const int32_t *row_adapters, int32_t depth, const int32_t *pass_max_rank,
                                       const lora_adapter_entry_t *table, int32_t num_slots, lora_segments_t seg,
                                       int32_t max_rank, void *ws, size_t ws_bytes, void *stream) {
  ModuleArgs ms[LORA_NUM_MODULES];
  int n = 0;
  void *scratch = nullptr;
  lora_status_t st =
      check_layer(io, module_mask, num_rows, table, num_slots, seg, max_rank, ws, ws_bytes, ms, &n, &scratch);
  if (st != LORA_OK) return st;
  if (depth < 1 || depth > LORA_MAX_STACK) return LORA_ERR_SHAPE;
  if (num_rows > 0 && !row_adapters) return LORA_ERR_NULL;
  if (pass_max_rank)
    for (int t = 0; t < depth; ++t)
      if (pass_max_rank[t] < 1 || pass_max_rank[t] > max_rank) return LORA_ERR_RANK;
  void *seg_scratch = nullptr;
  st = check_ws(ws, ws_bytes, segments_ws_bytes(num_rows, num_slots), &seg_scratch);
  if (st != LORA_OK) return st;
  ws = scratch ? scratch : seg_scratch;
  hipStream_t s = static_cast<hipStream_t>(stream);
  for (int t = 0; t < depth; ++t) {
    st = launched(launch_build_segments(row_adapters + t, depth, num_rows, num_slots, t > 0, seg, ws, s));
    if (st != LORA_OK || num_rows == 0) return st;  // no rows: the first pass only resets the segments
    const int r = pass_max_rank ? pass_max_rank[t] : max_rank;  // the pass's launch class
    st = launch_phase(true, ms, n, num_rows, num_slots, r, LORA_NUM_MODULES, table, seg, ws, nullptr, 0, s, true);
    if (st != LORA_OK) return st;
    st = launch_phase(false, ms, n, num_rows, num_slots, r, LORA_NUM_MODULES, table, seg, ws, nullptr, 0, s, true);
    if (st != LORA_OK) return st;
  }
  return LORA_OK;
}

}  // extern "C"

namespace {

// One projection of a fused call, from either io struct.
struct LinearArgs {
  const void *x;
  int64_t ldx;
  const void *W;   // bf16 [d_out][ldw] elements, or 4-bit [d_out][ldw] bytes
  int64_t ldw;
  const float *Ws; // 4-bit: group scales [d_out][ldws]; int8: scales [d_out]
  int64_t ldws;
  void *y;
  int64_t ldy;
  int32_t d_in, d_out;
};

lora_status_t check_linear(const lora_linear_io_t &m, LinearArgs *a) {
  if (!m.x || !m.y || !m.W) return LORA_ERR_NULL;
  if (m.d_in <= 0 || m.d_out <= 0 || m.ldx < m.d_in || m.ldy < m.d_out || m.ldw < m.d_in) return LORA_ERR_SHAPE;
  if ((m.d_in & 7) || (m.d_out & 7) || (m.ldx & 7) || (m.ldy & 7) || (m.ldw & 7) || !aligned16(m.x) ||
      !aligned16(m.y) || !aligned16(m.W))
    return LORA_ERR_ALIGN;
  if (!fits_u32(m.d_out, m.ldw)) return LORA_ERR_SHAPE;
  *a = LinearArgs{m.x, m.ldx, m.W, m.ldw, nullptr, 0, m.y, m.ldy, m.d_in, m.d_out};
  return LORA_OK;
}

lora_status_t check_linear(const lora_linear_q4_io_t &m, LinearArgs *a) {
  if (!m.x || !m.y || !m.Wq || !m.Ws) return LORA_ERR_NULL;
  if (m.d_in <= 0 || m.d_out <= 0 || m.ldx < m.d_in || m.ldy < m.d_out) return LORA_ERR_SHAPE;
  if ((m.d_in % LORA_Q4_GROUP) || (m.d_out & 7) || (m.ldx & 7) || (m.ldy & 7) || (m.ldwq & 15) ||
      !aligned16(m.x) || !aligned16(m.y) || !aligned16(m.Wq) || (reinterpret_cast<uintptr_t>(m.Ws) & 3))
    return LORA_ERR_ALIGN;
  if (m.ldwq < m.d_in / 2 || m.lds < m.d_in / LORA_Q4_GROUP) return LORA_ERR_SHAPE;
  if ((int64_t)m.d_out * m.ldwq > (int64_t)0xFFFFFF00 || (int64_t)m.d_out * m.lds * 4 > (int64_t)0xFFFFFF00)
    return LORA_ERR_SHAPE;
  *a = LinearArgs{m.x, m.ldx, m.Wq, m.ldwq, static_cast<const float *>(m.Ws), m.lds, m.y, m.ldy, m.d_in, m.d_out};
  return LORA_OK;
}

// Widths and leading dimensions beyond this are refused before any product of
// them is formed (a matrix of one such row is 1 GiB of bf16).
constexpr int64_t kMaxDim = 1 << 29;

lora_status_t check_linear(const lora_linear_i8_io_t &m, LinearArgs *a) {
  if (!m.x || !m.y || !m.Wq || !m.Ws) return LORA_ERR_NULL;
  if (m.d_in <= 0 || m.d_out <= 0 || m.ldx < m.d_in || m.ldy < m.d_out || m.ldwq < m.d_in || m.d_in > LORA_I8_MAX_IN ||
      m.ldx > kMaxDim || m.ldy > kMaxDim || m.d_out > kMaxDim)
    return LORA_ERR_SHAPE;
  if ((m.d_in & 7) || (m.d_out & 7) || (m.ldx & 7) || (m.ldy & 7) || (m.ldwq & 15) || !aligned16(m.x) ||
      !aligned16(m.y) || !aligned16(m.Wq) || !aligned16(m.Ws))
    return LORA_ERR_ALIGN;
  // the weight, and a B of the largest rank, below 4 GiB
  if (m.ldwq > (int64_t)0xFFFFFF00 / m.d_out || m.d_out > (int64_t)0xFFFFFF00 / (2 * LORA_MAX_RANK)) return LORA_ERR_SHAPE;
  *a = LinearArgs{m.x, m.ldx, m.Wq, m.ldwq, static_cast<const float *>(m.Ws), 0, m.y, m.ldy, m.d_in, m.d_out};
  return LORA_OK;
}

// ---- the products of gemm_items.h

// One input matrix of a call to quantise, and where its rows go in ws; the
// projections that share it (same pointer, ldx and d_in) share its rows.
struct QuantInputs {
  QuantDesc d{};
  size_t used = 0;
  int add(const void *x, int64_t ldx, int d_in, int64_t rows, void *ws) {
    for (int i = 0; i < d.n; ++i)
      if (d.in[i].x == x && d.in[i].ldx == ldx && d.in[i].d_in == d_in && d.in[i].rows == rows) return i;
    QuantInput &in = d.in[d.n];
    in.x = static_cast<const uint16_t *>(x);
    in.ldx = ldx;
    in.d_in = d_in;
    in.rows = (int)rows;
    in.pitch = i8_pitch(d_in);
    auto take = [&](size_t bytes) {
      void *p = static_cast<char *>(ws) + used;
      used += (bytes + 255) & ~(size_t)255;
      return p;
    };
    in.q = static_cast<int8_t *>(take((size_t)rows * in.pitch));
    in.amax = static_cast<float *>(take((size_t)rows * 4));
    in.rows_per_block = d_in <= kQuantWaveMax ? 4 : 1;
    in.block_base = d.blocks;
    d.blocks += (int)((rows + in.rows_per_block - 1) / in.rows_per_block);  // at most 7 times the rows of a matrix of 16-byte rows below 4 GiB
    return d.n++;
  }
};

// The tile configuration of a product (index into gemm_tile): the one that a
// simple account of its blocks gives the least time.  A block costs a start and
// an end (gemm_tile's `fixed`, and `per_adapter` for each adapter that 16 of
// its rows may have) and, for every byte of k, the bytes of its x and
// W rows at the rate one compute unit fetches and uses them, shared by the
// blocks that run on the unit together; blocks run in rounds.  Row tiles above
// twice the smallest that holds an average group are left out, and the largest
// is for groups of more than 128 rows (16 slots x 128 rows on 8192 x 8192, W
// from HBM once: 254 us with 128 rows a tile, 287 with 256, int8; the account
// knows no HBM).  Measured against it (us), base alone: 128 rows on a whole
// layer's 84000 outputs, 195 expected and 207 to 216 measured by 128 columns,
// 293 and 250 by 96; 256 rows on 18432 outputs, 90 and 59 to 68 by 96 columns
// (384 blocks on 512 places), 109 and 87 by 128 (288 on 256); 8 experts x 16
// rows on average on 2 x 28672 outputs, 590 and 622 by 32 rows, 752 and 780 by
// 16.  With a delta it takes the blocks' waits for the adapters and not the
// bytes of their B, which every tile reads: the whole layer with 128 adapters of
// rank 64 (1.4 GB of B) 224 and 449, the 256 rows with about 100 of rank 32 98
// and 85.
constexpr int kComputeUnits = 256;
constexpr double kUnitBytesPerUs = 45000;

// Row tiles of t rows: every group ends inside one, in its middle on average;
// a group expected to fit in one may be larger than the average.
double row_tiles_expected(int64_t rows, int64_t groups, int t) {
  if (groups == 1) return (double)((rows + t - 1) / t);
  const double per = (double)rows / (double)groups;
  if (per >= t) return (double)groups * (per / t + 0.5);
  const double spread = std::sqrt(per) + 0.15 * per;
  return (double)groups * (1 + std::max(0.0, 0.5 - (t - per) / (3.4 * spread)));
}

int pick_gemm(GemmKind kind, int64_t rows, int64_t groups, int adapters, const GemmModule *m, int n, double *expected_us) {
  const int64_t per = (rows + groups - 1) / groups;
  const int tiles = gemm_tiles(kind);
  // 4-bit: a quarter of the bytes of W, less time for a byte, and time for unpacking
  // and multiplying it that the bytes do not tell: 0.32 ps per row, column and byte
  // of x's k (fitted to blocks of 8192 inputs: 256 x 256 391 us, 128 x 128 by
  // two 219, 64 x 256 by two 244, 32 x 128 by two 74, 16 x 64 by four 45)
  const bool q4 = is_q4(kind);
  // A stage of a block alone on its unit takes a chain of waits (memory, barrier,
  // LDS, products) whatever it holds: where blocks are few, long stages on 8 waves,
  // which leave little room for other blocks (28672 inputs, 8192 outputs, a block or
  // less a unit: one row 46 us with 4 waves and 1024 bytes of x a stage, 30 with 8
  // and 2048; 16 rows 89 with 512 and 64 columns, 42 with 8 waves, 1024 and 32).
  auto work = [&](const GemmTile &t, double share, double kbytes) {
    if (!q4) return share * (t.rows + t.wcols) * kbytes / kUnitBytesPerUs;
    return std::max(kbytes / t.stage_bytes * t.stage_us,
                    share * (0.4 * (t.rows + 0.25 * t.wcols) / kUnitBytesPerUs + 0.32e-6 * std::max(t.rows, 16) * t.wcols) *
                        kbytes);
  };
  int fit = 0;
  while (fit + 1 < tiles && gemm_tile(kind, fit).rows < per) ++fit;
  int best = 0;
  double least = 0;
  for (int cfg = 0; cfg < tiles; ++cfg) {
    const GemmTile t = gemm_tile(kind, cfg);
    if (cfg > 0 && (t.rows > std::max(16, 2 * gemm_tile(kind, fit).rows) || (t.rows > 128 && per <= 128))) continue;
    const double rt = row_tiles_expected(rows, groups, t.rows);
    double blocks = 0;
    for (int i = 0; i < n; ++i) blocks += rt * ((m[i].d_out + t.cols - 1) / t.cols);
    const double share = std::min((double)t.per_unit, std::ceil(blocks / kComputeUnits));
    double sum = 0, longest = 0;
    for (int i = 0; i < n; ++i) {
      const double one = t.fixed + t.per_adapter * std::min(adapters, 16) + work(t, share, (double)m[i].kbytes);
      sum += rt * ((m[i].d_out + t.cols - 1) / t.cols) * one;
      longest = std::max(longest, one);
    }
    const double fill = blocks / (kComputeUnits * t.per_unit);  // rounds; the last of many overlaps the one before
    double us = std::max(longest, sum / blocks * (fill <= 2 ? std::ceil(fill) : fill + 0.4));
    // Blocks of a longer d_in than the others' go on when those are done, with the
    // unit to themselves (16 rows on a whole layer, whose down projection is 3.5
    // times as long as the rest: 150 us with 64 columns, four blocks a unit; 162
    // with 128, two).
    const double others = sum / (kComputeUnits * t.per_unit);
    if (q4 && longest > 1.5 * sum / blocks && longest > others) us = others + (longest - others) / share;
    if (q4) {  // W read again for every row tile, at 5.5 TB/s: what few rows wait for
      double bytes = 0;
      for (int i = 0; i < n; ++i) bytes += rt * m[i].d_out * (double)m[i].kbytes / 4 * (is_gated(kind) ? 2 : 1);
      us = std::max(us, bytes / 5.5e6);
    }
    if (cfg == 0 || us < least) {
      best = cfg;
      least = us;
    }
  }
  if (expected_us) *expected_us = least;
  return best;
}

// The rows of an int8 layer call are multiplied in the order of their slots
// (kOrderRows; a stated bound of nearly a segment per row: nothing to gather).
bool rows_by_slot(int num_rows, const lora_segments_t &seg) {
  return num_rows >= kOrderRows && (seg.max_segments == 0 || 2 * (int64_t)num_rows >= 3 * (int64_t)seg.max_segments);
}

// The tile of a call; adapters among 16 rows: by slot, those that meet there.
int tile_of_call(GemmKind kind, int num_rows, int num_slots, const lora_segments_t &seg, const GemmModule *m, int n,
                 double *expected_us = nullptr) {
  const int segs = segment_bound(num_rows, num_slots, seg);
  if (!has_delta(kind)) return pick_gemm(kind, num_rows, segs, 0, m, n, expected_us);
  const int adapters = rows_by_slot(num_rows, seg) ? (int)std::min<int64_t>(segs, 1 + 16 * (int64_t)segs / num_rows) : segs;
  return pick_gemm(kind, num_rows, 1, adapters, m, n, expected_us);
}

// Number the blocks of n projections (g.mod[0..n), longest d_in first: a
// block's work grows with it and blocks are dispatched in order), fill in what
// is common and launch.  row_tiles: row tiles of a projection (grouped: the
// most the segments can give).
lora_status_t gemm_launch(GemmDesc &g, int n, int64_t row_tiles, int num_rows, int num_slots,
                          const lora_segments_t &seg, GemmKind kind, int cfg, hipStream_t s) {
  std::stable_sort(g.mod, g.mod + n, [](const GemmModule &a, const GemmModule &b) { return a.d_in > b.d_in; });
  const GemmTile tile = gemm_tile(kind, cfg);
  int64_t blocks = 0;
  for (int i = 0; i < n; ++i) {
    g.mod[i].n_tiles = (g.mod[i].d_out + tile.cols - 1) / tile.cols;
    g.mod[i].block_base = (int)blocks;
    blocks += row_tiles * g.mod[i].n_tiles;
    if (blocks > 0x7fffffff) return LORA_ERR_SHAPE;
  }
  g.n_active = n;
  g.num_rows = num_rows;
  g.num_slots = num_slots;
  g.max_seg = segment_bound(num_rows, num_slots, seg);
  g.perm = seg.perm;
  g.seg_offsets = seg.seg_offsets;
  g.seg_adapter = seg.seg_adapter;
  g.num_segments = seg.num_segments;
  g.status = seg.status;
  return launched(launch_gemm(g, kind, cfg, (int)blocks, s));
}

// Base projection + delta: the grouped shrink and the partials summed into one
// v plane per projection (original row order) (do_shrink), then the fused
// kernel (do_fused).  IO: lora_linear_io_t (bf16 base) or lora_linear_q4_io_t.
template <typename IO>
lora_status_t linear_phase(bool do_shrink, bool do_fused, const IO *io, uint32_t module_mask, int32_t num_rows,
                           const int32_t *row_adapter, const lora_adapter_entry_t *table, int32_t num_slots,
                           lora_segments_t seg, int32_t max_rank, void *ws, size_t ws_bytes, void *stream) {
  constexpr bool kQ4 = std::is_same<IO, lora_linear_q4_io_t>::value;
  constexpr bool kI8 = std::is_same<IO, lora_linear_i8_io_t>::value;
  if (!io || !table) return LORA_ERR_NULL;
  lora_status_t st = check_segments(seg);
  if (st != LORA_OK) return st;
  const bool int8_items = (module_mask & LORA_MASK_INT8_ITEMS) != 0;
  module_mask &= ~LORA_MASK_INT8_ITEMS;
  if (module_mask == 0 || module_mask >= (1u << LORA_NUM_MODULES)) return LORA_ERR_MODULE;
  if (num_rows < 0 || num_slots < 1) return LORA_ERR_SHAPE;
  if (max_rank < 1 || max_rank > LORA_MAX_RANK) return LORA_ERR_RANK;
  if (num_rows > 0 && !row_adapter) return LORA_ERR_NULL;
  ModuleArgs ms[LORA_NUM_MODULES];
  LinearArgs la[LORA_NUM_MODULES];
  int n = 0;
  int64_t sum_d_in = 0;
  for (int c = 0; c < LORA_NUM_MODULES; ++c) {
    if (!(module_mask & (1u << c))) continue;
    st = check_linear(io[c], &la[n]);
    if (st != LORA_OK) return st;
    const LinearArgs &m = la[n];
    if (!fits_u32(num_rows, m.ldx) || !fits_u32(num_rows, m.ldy)) return LORA_ERR_SHAPE;
    ms[n] = ModuleArgs{m.x, m.ldx, m.y, m.ldy, m.d_in, m.d_out, c, int8_items};
    sum_d_in += m.d_in;
    ++n;
  }
  const size_t need = kI8 ? lora_linear_i8_workspace_bytes(num_rows, num_slots, max_rank, sum_d_in, n)
                          : lora_linear_workspace_bytes(num_rows, num_slots, max_rank, sum_d_in, n);
  if (!ws) return LORA_ERR_NULL;
  if (!aligned16(ws)) return LORA_ERR_ALIGN;
  if (ws_bytes < need) return LORA_ERR_WORKSPACE;
  const int rs = partial_row_stride(max_rank);
  if ((int64_t)num_rows * rs * 4 > (int64_t)0xFFFFFF00) return LORA_ERR_SHAPE;
  if (num_rows == 0) return LORA_OK;
  hipStream_t s = static_cast<hipStream_t>(stream);
  float *vplanes = reinterpret_cast<float *>(static_cast<char *>(ws) +
                                             ((partials_ws_bytes(num_rows, max_rank, sum_d_in) + 255) & ~(size_t)255));
  QuantInputs quant;
  int quant_of[LORA_NUM_MODULES] = {};
  int32_t *by_slot = nullptr;
  if constexpr (kI8) {  // the rows by slot and the int8 rows of x, behind the v planes
    char *behind = static_cast<char *>(ws) + linear_v_end(num_rows, max_rank, sum_d_in, n);
    if (rows_by_slot(num_rows, seg)) by_slot = reinterpret_cast<int32_t *>(behind);
    void *qws = behind + order_ws_bytes(num_rows);
    for (int i = 0; i < n; ++i) quant_of[i] = quant.add(la[i].x, la[i].ldx, la[i].d_in, num_rows, qws);
  }
  if (do_shrink) {
    // 1. v partials of every projection (segment-grouped: each adapter's A once)
    st = launch_phase(true, ms, n, num_rows, num_slots, max_rank, LORA_NUM_MODULES, table, seg, ws, nullptr, 0, s);
    if (st != LORA_OK) return st;
    // 2. one v plane per projection, rows in their original order
    LayerDesc d;
    fill_desc(d, ms, n, true, num_rows, num_slots, max_rank, LORA_NUM_MODULES, table, seg, ws);
    d.v_out = vplanes;
    d.ldv = rs;
    st = launched(kI8 ? launch_quantize_reduce(d, quant.d, row_adapter, by_slot, s) : launch_shrink_reduce(d, s));
    if (st != LORA_OK) return st;
  }
  if (!do_fused) return LORA_OK;
  if constexpr (kI8) {
    GemmDesc g{};
    for (int i = 0; i < n; ++i) {
      const auto &in = quant.d.in[quant_of[i]];
      GemmModule &gm = g.mod[i];
      gm.x = in.q;
      gm.ldx = in.pitch;
      gm.xs = in.amax;
      gm.x_bytes = (uint32_t)((int64_t)num_rows * in.pitch);
      gm.W = static_cast<const uint8_t *>(la[i].W);
      gm.ldw = la[i].ldw;
      gm.Ws = la[i].Ws;
      gm.y = static_cast<uint16_t *>(la[i].y);
      gm.ldy = la[i].ldy;
      gm.v = vplanes + (int64_t)i * num_rows * rs;
      gm.kbytes = in.pitch;
      gm.d_in = la[i].d_in;
      gm.d_out = la[i].d_out;
      gm.col = ms[i].col;
      gm.rows_per_x = 1;
    }
    const int cfg = tile_of_call(kLinearI8, num_rows, num_slots, seg, g.mod, n);
    g.row_tiles = (num_rows + gemm_tile(kLinearI8, cfg).rows - 1) / gemm_tile(kLinearI8, cfg).rows;
    g.rs = rs;
    g.max_rank = max_rank;
    g.ids = row_adapter;
    g.order = by_slot;
    g.table = table;
    return gemm_launch(g, n, g.row_tiles, num_rows, num_slots, seg, kLinearI8, cfg, s);
  }
  // 3. base projection + delta.  A block's work grows with its module's
  // d_in, and the blocks are dispatched in order, so the modules are numbered
  // longest first: a module of a long d_in (a down projection, 3.5x the
  // others) numbered last would start when the others are done and run
  // alone for most of the launch.
  FusedDesc f{};
  const int row_tiles = (num_rows + kFusedRows - 1) / kFusedRows;
  int order[LORA_NUM_MODULES];
  for (int i = 0; i < n; ++i) order[i] = i;
  std::stable_sort(order, order + n, [&](int a, int b) { return la[a].d_in > la[b].d_in; });
  int64_t blocks = 0;
  for (int j = 0; j < n; ++j) {
    const int i = order[j];
    const LinearArgs &m = la[i];
    FusedModule &fm = f.mod[j];
    fm.x = static_cast<const uint16_t *>(m.x);
    fm.ldx = m.ldx;
    fm.W = m.W;
    fm.ldw = m.ldw;
    fm.Ws = m.Ws;
    fm.ldws = m.ldws;
    fm.y = static_cast<uint16_t *>(m.y);
    fm.ldy = m.ldy;
    fm.v = vplanes + (int64_t)i * num_rows * rs;
    fm.d_in = m.d_in;
    fm.d_out = m.d_out;
    fm.col = ms[i].col;
    fm.n_tiles = (m.d_out + fused_cols(kQ4) - 1) / fused_cols(kQ4);
    fm.block_base = (int)blocks;
    blocks += (int64_t)row_tiles * fm.n_tiles;
  }
  if (blocks > 0x7fffffff) return LORA_ERR_SHAPE;
  f.n_active = n;
  f.num_rows = num_rows;
  f.num_slots = num_slots;
  f.table_cols = LORA_NUM_MODULES;
  f.max_rank = max_rank;
  f.rs = rs;
  f.ids = row_adapter;
  f.status = seg.status;
  f.table = table;
  f.num_segments = seg.num_segments;
  f.seg_adapter = seg.seg_adapter;
  f.max_seg = segment_bound(num_rows, num_slots, seg);
  return launched(launch_fused(f, kQ4, (int)blocks, s));
}

}  // namespace

extern "C" {

lora_status_t lora_linear_layer(const lora_linear_io_t *io, uint32_t module_mask, int32_t num_rows,
                                const int32_t *row_adapter, const lora_adapter_entry_t *table, int32_t num_slots,
                                lora_segments_t seg, int32_t max_rank, void *ws, size_t ws_bytes, void *stream) {
  return linear_phase(true, true, io, module_mask, num_rows, row_adapter, table, num_slots, seg, max_rank, ws,
                      ws_bytes, stream);
}

lora_status_t lora_linear_shrink(const lora_linear_io_t *io, uint32_t module_mask, int32_t num_rows,
                                 const int32_t *row_adapter, const lora_adapter_entry_t *table, int32_t num_slots,
                                 lora_segments_t seg, int32_t max_rank, void *ws, size_t ws_bytes, void *stream) {
  return linear_phase(true, false, io, module_mask, num_rows, row_adapter, table, num_slots, seg, max_rank, ws,
                      ws_bytes, stream);
}

lora_status_t lora_linear_expand(const lora_linear_io_t *io, uint32_t module_mask, int32_t num_rows,
                                 const int32_t *row_adapter, const lora_adapter_entry_t *table, int32_t num_slots,
                                 lora_segments_t seg, int32_t max_rank, void *ws, size_t ws_bytes, void *stream) {
  return linear_phase(false, true, io, module_mask, num_rows, row_adapter, table, num_slots, seg, max_rank, ws,
                      ws_bytes, stream);
}

lora_status_t lora_linear_layer_q4(const lora_linear_q4_io_t *io, uint32_t module_mask, int32_t num_rows,
                                   const int32_t *row_adapter, const lora_adapter_entry_t *table, int32_t num_slots,
                                   lora_segments_t seg, int32_t max_rank, void *ws, size_t ws_bytes, void *stream) {
  return linear_phase(true, true, io, module_mask, num_rows, row_adapter, table, num_slots, seg, max_rank, ws,
                      ws_bytes, stream);
}

lora_status_t lora_linear_shrink_q4(const lora_linear_q4_io_t *io, uint32_t module_mask, int32_t num_rows,
                                    const int32_t *row_adapter, const lora_adapter_entry_t *table,
                                    int32_t num_slots, lora_segments_t seg, int32_t max_rank, void *ws,
                                    size_t ws_bytes, void *stream) {
  return linear_phase(true, false, io, module_mask, num_rows, row_adapter, table, num_slots, seg, max_rank, ws,
                      ws_bytes, stream);
}

lora_status_t lora_linear_expand_q4(const lora_linear_q4_io_t *io, uint32_t module_mask, int32_t num_rows,
                                    const int32_t *row_adapter, const lora_adapter_entry_t *table,
                                    int32_t num_slots, lora_segments_t seg, int32_t max_rank, void *ws,
                                    size_t ws_bytes, void *stream) {
  return linear_phase(false, true, io, module_mask, num_rows, row_adapter, table, num_slots, seg, max_rank, ws,
                      ws_bytes, stream);
}

}  // extern "C"

namespace {

// log2 of a group of 4-bit weights, -1 for a length that is none.
int group_log(int32_t group) { return group == 32 ? 5 : group == 64 ? 6 : group == 128 ? 7 : -1; }

// The activation's constants (gate_act); false for one that is none.
bool set_activation(GemmDesc &g, int32_t activation) {
  if (activation != LORA_ACT_SILU && activation != LORA_ACT_GELU_TANH) return false;
  const double c1 = 1.5957691216057308;  // 2 sqrt(2 / pi)
  g.act_c1 = activation == LORA_ACT_SILU ? 1.f : (float)c1;
  g.act_c3 = activation == LORA_ACT_SILU ? 0.f : (float)(0.044715 * c1);
  return true;
}

// The checks, the quantiser (int8) and the launch of the grouped products; the
// gated kinds take one io (gate's and up's) and a mask of gate alone.
lora_status_t grouped_call(GemmKind kind, const lora_grouped_io_t *io, uint32_t module_mask, int32_t num_rows,
                           const void *weights, int32_t num_slots, const lora_segments_t &seg, void *ws,
                           size_t ws_bytes, void *stream, int32_t group = 0, int32_t activation = LORA_ACT_SILU) {
  const bool i8 = kind == kGroupedI8;
  if (!io || !weights) return LORA_ERR_NULL;
  lora_status_t st = check_segments(seg);
  if (st != LORA_OK) return st;
  if (module_mask == 0 || module_mask >= (1u << LORA_NUM_MODULES)) return LORA_ERR_MODULE;
  if (num_rows < 0 || num_slots < 1) return LORA_ERR_SHAPE;
  GemmDesc g{};
  if (is_q4(kind) && group_log(group) < 0) return LORA_ERR_SHAPE;
  if (is_gated(kind) && !set_activation(g, activation)) return LORA_ERR_SHAPE;
  QuantInputs quant;
  int n = 0;
  int64_t sum_d_in = 0;
  for (int c = 0; c < LORA_NUM_MODULES; ++c) {
    if (!(module_mask & (1u << c))) continue;
    const lora_grouped_io_t &m = is_gated(kind) ? *io : io[c];
    if (!m.x || !m.y) return LORA_ERR_NULL;
    if (m.d_in <= 0 || m.d_out <= 0 || m.ldx < m.d_in || m.ldy < m.d_out || m.rows_per_x < 1 || m.ldx > kMaxDim ||
        m.ldy > kMaxDim)
      return LORA_ERR_SHAPE;
    if ((m.d_in & 7) || (m.d_out & 7) || (m.ldx & 7) || (m.ldy & 7) || !aligned16(m.x) || !aligned16(m.y))
      return LORA_ERR_ALIGN;
    if (i8 && m.d_in > LORA_I8_MAX_IN) return LORA_ERR_SHAPE;
    if (is_q4(kind) && m.d_in % group) return LORA_ERR_ALIGN;
    const int64_t x_rows = ((int64_t)num_rows + m.rows_per_x - 1) / m.rows_per_x;
    if (!fits_u32(x_rows, m.ldx) || !fits_u32(num_rows, m.ldy)) return LORA_ERR_SHAPE;
    GemmModule &gm = g.mod[n];
    gm.x = m.x;
    gm.ldx = m.ldx * 2;
    gm.x_bytes = (uint32_t)(x_rows * m.ldx * 2);
    gm.kbytes = m.d_in * 2;
    if (i8) {
      const auto &in = quant.d.in[quant.add(m.x, m.ldx, m.d_in, x_rows, ws)];
      gm.x = in.q;
      gm.ldx = gm.kbytes = in.pitch;
      gm.xs = in.amax;
      gm.x_bytes = (uint32_t)(x_rows * in.pitch);
    }
    gm.y = static_cast<uint16_t *>(m.y);
    gm.ldy = m.ldy;
    gm.d_in = m.d_in;
    gm.d_out = m.d_out;
    gm.col = c;
    gm.rows_per_x = m.rows_per_x;
    gm.group_log = is_q4(kind) ? group_log(group) : 0;
    gm.row_most = (uint32_t)(0xFFFFFF00u / (uint32_t)m.d_out);
    if (is_gated(kind)) g.mod[1].col = LORA_UP;
    sum_d_in += m.d_in;
    ++n;
  }
  if (i8) {
    void *scratch = nullptr;
    st = check_ws(ws, ws_bytes, lora_grouped_workspace_bytes(num_rows, num_slots, sum_d_in, n), &scratch);
    if (st != LORA_OK) return st;
  }
  if (num_rows == 0) return LORA_OK;
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (i8) {
    st = launched(launch_quantize(quant.d, s));
    if (st != LORA_OK) return st;
  }
  g.weights = static_cast<const lora_weight_entry_t *>(weights);
  const int cfg = tile_of_call(kind, num_rows, num_slots, seg, g.mod, n);
  const int rt = gemm_tile(kind, cfg).rows;
  // every segment's last tile may be partial
  const int64_t row_tiles = std::min<int64_t>(num_rows, (int64_t)num_rows / rt + segment_bound(num_rows, num_slots, seg));
  return gemm_launch(g, n, row_tiles, num_rows, num_slots, seg, kind, cfg, s);
}

// One projection of a call with a base weight and adapters, bf16 (group 0) or
// 4-bit.
lora_status_t check_adapted(const LinearArgs &m, bool q4, int32_t group) {
  if (!m.x || !m.y || !m.W || (q4 && !m.Ws)) return LORA_ERR_NULL;
  if (q4 && group_log(group) < 0) return LORA_ERR_SHAPE;
  if (m.d_in <= 0 || m.d_out <= 0 || m.ldx < m.d_in || m.ldy < m.d_out || m.ldx > kMaxDim || m.ldy > kMaxDim ||
      m.ldw > kMaxDim || m.ldws > kMaxDim)
    return LORA_ERR_SHAPE;
  if ((m.d_in & 7) || (m.d_out & 7) || (m.ldx & 7) || (m.ldy & 7) || !aligned16(m.x) || !aligned16(m.y) || !aligned16(m.W))
    return LORA_ERR_ALIGN;
  if (q4 ? (m.d_in % group) || (m.ldw & 15) || ((uintptr_t)m.Ws & 3) : (m.ldw & 7) != 0) return LORA_ERR_ALIGN;
  if (q4 ? m.ldw < m.d_in / 2 || m.ldws < m.d_in / group : m.ldw < m.d_in) return LORA_ERR_SHAPE;
  // the weight, its scales and a B of the largest rank below 4 GiB
  const int64_t most = (int64_t)0xFFFFFF00 / m.d_out;
  if (m.ldw > (q4 ? most : most / 2) || m.ldws > most / 4 || most < 2 * LORA_MAX_RANK) return LORA_ERR_SHAPE;
  return LORA_OK;
}

// Base products with adapters by the kernels of gemm_items.h: v of the n
// projections with the rows' order and descriptions (rows.hip; a few rows in one
// launch, else behind the grouped shrink), and the product (gated: one of both
// projections).
lora_status_t adapted_call(GemmKind kind, const LinearArgs *la, const int *cols, int n, bool int8_items, int32_t group,
                           int32_t activation, int32_t num_rows, const int32_t *row_adapter,
                           const lora_adapter_entry_t *table, int32_t num_slots, const lora_segments_t &seg,
                           int32_t max_rank, void *ws, size_t ws_bytes, void *stream) {
  if (!table) return LORA_ERR_NULL;
  lora_status_t st = check_segments(seg);
  if (st != LORA_OK) return st;
  GemmDesc g{};
  if (!set_activation(g, activation)) return LORA_ERR_SHAPE;
  if (num_rows < 0 || num_slots < 1) return LORA_ERR_SHAPE;
  if (max_rank < 1 || max_rank > LORA_MAX_RANK) return LORA_ERR_RANK;
  if (num_rows > 0 && !row_adapter) return LORA_ERR_NULL;
  ModuleArgs ms[LORA_NUM_MODULES];
  int64_t sum_d_in = 0;
  for (int i = 0; i < n; ++i) {
    if (!fits_u32(num_rows, la[i].ldx) || !fits_u32(num_rows, la[i].ldy)) return LORA_ERR_SHAPE;
    ms[i] = ModuleArgs{la[i].x, la[i].ldx, la[i].y, la[i].ldy, la[i].d_in, la[i].d_out, cols[i], int8_items};
    sum_d_in += la[i].d_in;
  }
  st = check_ws(ws, ws_bytes, lora_linear_q4g_workspace_bytes(num_rows, num_slots, max_rank, sum_d_in, n), &ws);
  if (st != LORA_OK) return st;
  const int rs = partial_row_stride(max_rank);
  if ((int64_t)num_rows * rs * 4 > (int64_t)0xFFFFFF00) return LORA_ERR_SHAPE;
  if (num_rows == 0) return LORA_OK;
  hipStream_t s = static_cast<hipStream_t>(stream);
  float *vplanes = reinterpret_cast<float *>(static_cast<char *>(ws) +
                                             ((partials_ws_bytes(num_rows, max_rank, sum_d_in) + 255) & ~(size_t)255));
  char *behind = static_cast<char *>(ws) + linear_v_end(num_rows, max_rank, sum_d_in, n);
  const bool few = num_rows < kOrderRows && (double)num_rows * max_rank * sum_d_in * 4 <= kFewBytes;
  RowsDesc rows{};
  if (!few && rows_by_slot(num_rows, seg)) rows.order = reinterpret_cast<int32_t *>(behind);
  rows.info = reinterpret_cast<RowInfo *>(behind + order_ws_bytes(num_rows));
  rows.ids = row_adapter;
  if (!few) {
    st = launch_phase(true, ms, n, num_rows, num_slots, max_rank, LORA_NUM_MODULES, table, seg, ws, nullptr, 0, s);
    if (st != LORA_OK) return st;
  }
  fill_desc(rows.L, ms, n, true, num_rows, num_slots, max_rank, LORA_NUM_MODULES, table, seg, ws);
  rows.L.v_out = vplanes;
  rows.L.ldv = rs;
  st = launched(launch_rows(rows, few, s));
  if (st != LORA_OK) return st;
  for (int i = 0; i < n; ++i) {
    GemmModule &gm = g.mod[i];
    gm.x = la[i].x;
    gm.ldx = la[i].ldx * 2;
    gm.x_bytes = (uint32_t)(num_rows * la[i].ldx * 2);
    gm.W = static_cast<const uint8_t *>(la[i].W);
    gm.ldw = is_q4(kind) ? la[i].ldw : la[i].ldw * 2;
    gm.Ws = la[i].Ws;
    gm.ldws = la[i].ldws;
    gm.group_log = is_q4(kind) ? group_log(group) : 0;
    gm.y = static_cast<uint16_t *>(la[i].y);
    gm.ldy = la[i].ldy;
    gm.v = vplanes + (int64_t)i * num_rows * rs;
    gm.info = rows.info + (int64_t)i * num_rows;
    gm.kbytes = la[i].d_in * 2;
    gm.d_in = la[i].d_in;
    gm.d_out = la[i].d_out;
    gm.col = cols[i];
    gm.rows_per_x = 1;
  }
  const int products = is_gated(kind) ? 1 : n;
  const int cfg = tile_of_call(kind, num_rows, num_slots, seg, g.mod, products);
  g.row_tiles = (num_rows + gemm_tile(kind, cfg).rows - 1) / gemm_tile(kind, cfg).rows;
  g.rs = rs;
  g.max_rank = max_rank;
  g.order = rows.order;
  return gemm_launch(g, products, g.row_tiles, num_rows, num_slots, seg, kind, cfg, s);
}

lora_status_t gated_call(GemmKind kind, const LinearArgs (&la)[2], int32_t group, int32_t activation, int32_t num_rows,
                         const int32_t *row_adapter, const lora_adapter_entry_t *table, int32_t num_slots,
                         const lora_segments_t &seg, int32_t max_rank, void *ws, size_t ws_bytes, void *stream) {
  const int cols[2] = {LORA_GATE, LORA_UP};
  for (const LinearArgs &m : la) {
    const lora_status_t st = check_adapted(m, is_q4(kind), group);
    if (st != LORA_OK) return st;
  }
  return adapted_call(kind, la, cols, 2, false, group, activation, num_rows, row_adapter, table, num_slots, seg, max_rank, ws,
                      ws_bytes, stream);
}

}  // namespace

extern "C" int32_t lora_internal_gemm_tile(int32_t kind, int32_t num_rows, int32_t num_slots, lora_segments_t seg,
                                           const int32_t *d_in, const int32_t *d_out, int32_t n, int32_t *rows,
                                           int32_t *cols, double *expected_us) {
  if (kind < kLinearI8 || kind > kGroupedGatedQ4 || num_rows < 1 || num_slots < 1 || n < 1 || n > kMaxModules) return -1;
  GemmModule m[kMaxModules] = {};
  for (int i = 0; i < n; ++i) {
    m[i].kbytes = kind == kLinearI8 || kind == kGroupedI8 ? i8_pitch(d_in[i]) : d_in[i] * 2;
    m[i].d_out = d_out[i];
  }
  const int cfg = tile_of_call((GemmKind)kind, num_rows, num_slots, seg, m, n, expected_us);
  *rows = gemm_tile((GemmKind)kind, cfg).rows;
  *cols = gemm_tile((GemmKind)kind, cfg).cols;
  return cfg;
}

extern "C" {

lora_status_t lora_linear_layer_i8(const lora_linear_i8_io_t *io, uint32_t module_mask, int32_t num_rows,
                                   const int32_t *row_adapter, const lora_adapter_entry_t *table, int32_t num_slots,
                                   lora_segments_t seg, int32_t max_rank, void *ws, size_t ws_bytes, void *stream) {
  return linear_phase(true, true, io, module_mask, num_rows, row_adapter, table, num_slots, seg, max_rank, ws,
                      ws_bytes, stream);
}

lora_status_t lora_linear_shrink_i8(const lora_linear_i8_io_t *io, uint32_t module_mask, int32_t num_rows,
                                    const int32_t *row_adapter, const lora_adapter_entry_t *table,
                                    int32_t num_slots, lora_segments_t seg, int32_t max_rank, void *ws,
                                    size_t ws_bytes, void *stream) {
  return linear_phase(true, false, io, module_mask, num_rows, row_adapter, table, num_slots, seg, max_rank, ws,
                      ws_bytes, stream);
}

lora_status_t lora_linear_expand_i8(const lora_linear_i8_io_t *io, uint32_t module_mask, int32_t num_rows,
                                    const int32_t *row_adapter, const lora_adapter_entry_t *table,
                                    int32_t num_slots, lora_segments_t seg, int32_t max_rank, void *ws,
                                    size_t ws_bytes, void *stream) {
  return linear_phase(false, true, io, module_mask, num_rows, row_adapter, table, num_slots, seg, max_rank, ws,
                      ws_bytes, stream);
}

lora_status_t lora_grouped_layer(const lora_grouped_io_t *io, uint32_t module_mask, int32_t num_rows,
                                 const lora_weight_entry_t *weights, int32_t num_slots, lora_segments_t seg,
                                 void *stream) {
  return grouped_call(kGroupedBf16, io, module_mask, num_rows, weights, num_slots, seg, nullptr, 0, stream);
}

lora_status_t lora_grouped_layer_i8(const lora_grouped_io_t *io, uint32_t module_mask, int32_t num_rows,
                                    const lora_weight_entry_t *weights, int32_t num_slots, lora_segments_t seg,
                                    void *ws, size_t ws_bytes, void *stream) {
  return grouped_call(kGroupedI8, io, module_mask, num_rows, weights, num_slots, seg, ws, ws_bytes, stream);
}

lora_status_t lora_grouped_layer_q4g(const lora_grouped_io_t *io, uint32_t module_mask, int32_t num_rows,
                                     const lora_weight_q4g_entry_t *weights, int32_t num_slots, int32_t group,
                                     lora_segments_t seg, void *stream) {
  return grouped_call(kGroupedQ4, io, module_mask, num_rows, weights, num_slots, seg, nullptr, 0, stream, group);
}

lora_status_t lora_grouped_gated_layer(const lora_grouped_io_t *io, int32_t activation, int32_t num_rows,
                                       const lora_weight_entry_t *weights, int32_t num_slots, lora_segments_t seg,
                                       void *stream) {
  return grouped_call(kGroupedGatedBf16, io, 1u << LORA_GATE, num_rows, weights, num_slots, seg, nullptr, 0, stream, 0,
                      activation);
}

lora_status_t lora_grouped_gated_layer_q4g(const lora_grouped_io_t *io, int32_t activation, int32_t num_rows,
                                           const lora_weight_q4g_entry_t *weights, int32_t num_slots, int32_t group,
                                           lora_segments_t seg, void *stream) {
  return grouped_call(kGroupedGatedQ4, io, 1u << LORA_GATE, num_rows, weights, num_slots, seg, nullptr, 0, stream, group,
                      activation);
}

size_t lora_linear_q4g_workspace_bytes(int32_t num_rows, int32_t num_slots, int32_t max_rank, int64_t sum_d_in,
                                       int32_t n_modules) {
  const size_t base = lora_linear_workspace_bytes(num_rows, num_slots, max_rank, sum_d_in, n_modules);
  if (base == 0) return 0;
  const size_t need = linear_v_end(num_rows, max_rank, sum_d_in, n_modules) + order_ws_bytes(num_rows) +
                      (size_t)n_modules * num_rows * sizeof(RowInfo);
  return need > base ? need : base;
}

size_t lora_gated_workspace_bytes(int32_t num_rows, int32_t num_slots, int32_t max_rank, int32_t d_in) {
  return lora_linear_q4g_workspace_bytes(num_rows, num_slots, max_rank, 2 * (int64_t)d_in, 2);
}

lora_status_t lora_linear_layer_q4g(const lora_linear_q4g_io_t *io, uint32_t module_mask, int32_t num_rows,
                                    const int32_t *row_adapter, const lora_adapter_entry_t *table, int32_t num_slots,
                                    lora_segments_t seg, int32_t max_rank, void *ws, size_t ws_bytes, void *stream) {
  if (!io) return LORA_ERR_NULL;
  const bool int8_items = (module_mask & LORA_MASK_INT8_ITEMS) != 0;
  module_mask &= ~LORA_MASK_INT8_ITEMS;
  if (module_mask == 0 || module_mask >= (1u << LORA_NUM_MODULES)) return LORA_ERR_MODULE;
  LinearArgs la[LORA_NUM_MODULES];
  int cols[LORA_NUM_MODULES], n = 0, group = 0;
  for (int c = 0; c < LORA_NUM_MODULES; ++c) {
    if (!(module_mask & (1u << c))) continue;
    const lora_linear_q4g_io_t &m = io[c];
    if (n > 0 && m.group != group) return LORA_ERR_SHAPE;
    group = m.group;
    la[n] = LinearArgs{m.x, m.ldx, m.Wq, m.ldwq, static_cast<const float *>(m.Ws), m.lds, m.y, m.ldy, m.d_in, m.d_out};
    const lora_status_t st = check_adapted(la[n], true, group);
    if (st != LORA_OK) return st;
    cols[n++] = c;
  }
  return adapted_call(kLinearQ4, la, cols, n, int8_items, group, LORA_ACT_SILU, num_rows, row_adapter, table, num_slots,
                      seg, max_rank, ws, ws_bytes, stream);
}

lora_status_t lora_gated_layer(const lora_gated_io_t *io, int32_t activation, int32_t num_rows,
                               const int32_t *row_adapter, const lora_adapter_entry_t *table, int32_t num_slots,
                               lora_segments_t seg, int32_t max_rank, void *ws, size_t ws_bytes, void *stream) {
  if (!io) return LORA_ERR_NULL;
  const lora_gated_io_t &m = *io;
  const LinearArgs la[2] = {{m.x, m.ldx, m.Wg, m.ldwg, nullptr, 0, m.h, m.ldh, m.d_in, m.d_ff},
                            {m.x, m.ldx, m.Wu, m.ldwu, nullptr, 0, m.h, m.ldh, m.d_in, m.d_ff}};
  return gated_call(kGatedBf16, la, 0, activation, num_rows, row_adapter, table, num_slots, seg, max_rank, ws, ws_bytes,
                    stream);
}

lora_status_t lora_gated_layer_q4g(const lora_gated_q4g_io_t *io, int32_t activation, int32_t num_rows,
                                   const int32_t *row_adapter, const lora_adapter_entry_t *table, int32_t num_slots,
                                   lora_segments_t seg, int32_t max_rank, void *ws, size_t ws_bytes, void *stream) {
  if (!io) return LORA_ERR_NULL;
  const lora_gated_q4g_io_t &m = *io;
  const LinearArgs la[2] = {
      {m.x, m.ldx, m.Wgq, m.ldwg, static_cast<const float *>(m.Wgs), m.ldsg, m.h, m.ldh, m.d_in, m.d_ff},
      {m.x, m.ldx, m.Wuq, m.ldwu, static_cast<const float *>(m.Wus), m.ldsu, m.h, m.ldh, m.d_in, m.d_ff}};
  return gated_call(kGatedQ4, la, m.group, activation, num_rows, row_adapter, table, num_slots, seg, max_rank, ws, ws_bytes,
                    stream);
}

}  // extern "C"

// ---- lora_apply_layer_noalloc: the k-chunk partials in a static device
// array instead of a caller's workspace.  Each device that loads the library
// holds its own copy until the process ends; in host code `scratch` is only
// a handle, so its device address is looked up once per device and every
// launch takes that address.
static __device__ __align__(256) uint8_t scratch[LORA_STATIC_SCRATCH_BYTES];

namespace {

constexpr int kMaxDevices = 64;
std::mutex g_scratch_mu;
void *g_scratch_addr[kMaxDevices];  // device address of `scratch`, per device

// The address of the current device's `scratch` (looked up on the first call
// on that device, with it current).
lora_status_t scratch_address(void **out) {
  int dev = -1;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= kMaxDevices) return LORA_ERR_LAUNCH;
  std::lock_guard<std::mutex> lock(g_scratch_mu);
  if (g_scratch_addr[dev] == nullptr) {
    void *p = nullptr;
    if (hipGetSymbolAddress(&p, HIP_SYMBOL(scratch)) != hipSuccess || p == nullptr) return LORA_ERR_LAUNCH;
    g_scratch_addr[dev] = p;
  }
  *out = g_scratch_addr[dev];
  return LORA_OK;
}

}  // namespace

extern "C" lora_status_t lora_apply_layer_noalloc(const lora_module_io_t *io, uint32_t module_mask,
                                                  int32_t num_rows, const lora_adapter_entry_t *table,
                                                  int32_t num_slots, lora_segments_t seg, int32_t max_rank,
                                                  void *stream) {
  ModuleArgs ms[LORA_NUM_MODULES];
  int n = 0;
  // the argument checks of lora_apply_layer, with the static array as an
  // aligned workspace of its full size
  void *unused = nullptr;
  lora_status_t st = check_layer(io, module_mask, num_rows, table, num_slots, seg, max_rank,
                                 reinterpret_cast<void *>(uintptr_t{256}), LORA_STATIC_SCRATCH_BYTES, ms, &n, &unused);
  if (st == LORA_ERR_WORKSPACE) return LORA_ERR_SCRATCH;
  if (st != LORA_OK) return st;
  if (num_rows == 0) return LORA_OK;
  void *ws = nullptr;
  st = scratch_address(&ws);
  if (st != LORA_OK) return st;
  hipStream_t s = static_cast<hipStream_t>(stream);
  st = launch_phase(true, ms, n, num_rows, num_slots, max_rank, LORA_NUM_MODULES, table, seg, ws, nullptr, 0, s, true);
  if (st != LORA_OK) return st;
  return launch_phase(false, ms, n, num_rows, num_slots, max_rank, LORA_NUM_MODULES, table, seg, ws, nullptr, 0, s,
                      true);
}
