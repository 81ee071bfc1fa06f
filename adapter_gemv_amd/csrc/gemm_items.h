// Base products on the matrix cores, from int8 or bf16 rows:
//   * the int8 base projection with the adapter delta (lora_linear_layer_i8):
//       y[b] = bf16( s_b * Ws[n] * sum_k q_b[k] Wq[n][k] + scale_a B_a.v[b] )
//     with q_b, s_b the row quantised to int8 (quantize_rows_kernel) and
//     v[b] = A_a.x[b] from the grouped shrink;
//   * the dense products grouped by slot (lora_grouped_layer, _i8):
//       y[b] = bf16( W_a . x[b / rows_per_x] ),  a = the row's slot;
//   * either with 4-bit weights W[n][k] = s[n][k / G] q[n][k] and bf16 rows
//     (lora_linear_layer_q4g, lora_grouped_layer_q4g);
//   * the gated half of a feed-forward block (lora_gated_layer,
//     lora_grouped_gated_layer, and _q4g):
//       h[b] = bf16( act(g) u ),  g and u the sums of gate and up as above: half
//     of a block's rows of W are gate's, half up's, and a wave holds both sums of
//     an output.
//
// One block computes RT rows x NC output columns over the whole input range.
// A product of 16-byte pieces looks the same to memory and LDS for either
// type (64 bytes of k per matrix-core step: 32 bf16 or 64 int8 values), so one
// body serves both and only the matrix-core instruction differs.
//   * x and W go to LDS by direct loads (no registers in between), S stages of
//     KB bytes per row in a ring, S - 1 of them in flight.  The 16-byte pieces
//     of a row are stored at piece ^ (row mod 16) (rows of 128 bytes: mod 8, a
//     row fills half the 64 banks), so that the 16 rows an operand read
//     touches per cycle fall into different banks; the loads write LDS in
//     lane order, so the lanes fetch the pieces in that order.
//   * The loads are issued by inline assembly: they return nothing to
//     registers, and the compiler, which does not know which stage a load
//     fills, would wait for all of them before every LDS read.  A wave waits
//     for its own loads of the stage by count (they complete in order), then
//     the block's barrier covers the other waves' loads.  One barrier per
//     stage: passing it also means that every wave has read the stage before,
//     whose place the next loads take.
//   * W is the matrix-core A operand and x the B operand, so a lane holds 4
//     consecutive outputs of one row and stores them as 8 bytes.
//   * The waves form a WR x WC x WK grid over rows, columns and the k of a
//     stage; with WK > 1 (few rows and columns per block, so that short
//     batches still fill the device) the partial sums meet in LDS, added in
//     wave order.
//   * 4-bit W goes to LDS as it is, a quarter of the bytes, and is unpacked for the
//     matrix cores by the wave that multiplies it: two values an operation
//     (q4x8_shifted), 8 operations a register of 8 weights; converting them took 15
//     and one token's q/k/v/o 46 us instead of 43.  Scales come in batches of 16
//     groups of a row (172 -> 150 us of 16 rows on a layer).
// int8 sums are exact in int32, bf16 sums are fp32; the order of the additions
// is fixed, so results are bit-reproducible.
// Bound: few rows, HBM by the weights (W once per row tile; 4.3 GB of bf16 at 16
// rows a slot 690 us, 6.2 TB/s; 1.1 GB of 4-bit at 4 rows a slot 207 us, 5.5 TB/s);
// many rows, the matrix cores (gemm.hip; 4-bit: with the unpacking beside them).
#pragma once

#include <type_traits>

#include "device_common.h"

namespace lora {

typedef int32_t i32x4_t __attribute__((ext_vector_type(4)));

template <bool I8_, int RT_, int NC_, int WR_, int WC_, int WK_, int KB_, int S_, int EU_, bool PIPE_ = false,
          bool Q4_ = false, bool GATED_ = false>
struct GemmCfg {
  static constexpr bool Q4 = Q4_;                      // 4-bit W, a scale per output and group of inputs; bf16 x
  static constexpr bool GATED = GATED_;                // the first half of the columns is gate's, the second up's
  static constexpr bool PIPE = PIPE_;                  // operands one step ahead in registers
  static constexpr bool I8 = I8_;
  static constexpr int RT = RT_, NC = NC_;             // rows and columns (of both halves) of a block
  static constexpr int HC = GATED_ ? NC_ / 2 : NC_;    // output columns
  static constexpr int WR = WR_, WC = WC_, WK = WK_;   // wave grid: rows, columns, k
  static constexpr int KB = KB_, S = S_;               // bytes of k per stage (of x), stages
  static constexpr int WKB = Q4_ ? KB / 4 : KB;        // the same of W
  static constexpr int EU = EU_;                       // waves per SIMD it is compiled for
  static constexpr int NW = WR * WC * WK, THREADS = NW * 64;
  static constexpr int MT = RT < 16 ? 1 : RT / WR / 16, NT = NC / WC / 16;  // 16 x 16 tiles of a wave
  static constexpr int IR = RT < 16 ? 16 : RT;         // rows of the matrix cores' tiles (beyond RT: never stored)
  // Column tiles a wave finishes (epilogue); gated: as many of each half.
  static constexpr int NTE = GATED_ ? (NT / 2 >= WK ? NT / 2 / WK : 1) : NT >= WK ? NT / WK : 1;
  static constexpr int FIN = GATED_ ? 2 * NTE : NTE;   // their sums
  static constexpr int PIECES = KB / 16;
  static constexpr int SWZ = PIECES >= 16 ? 15 : 7;    // rows whose pieces are moved against one another
  static constexpr int WPIECES = WKB / 16;
  static constexpr int WSWZ = WPIECES >= 16 ? 15 : WPIECES - 1;
  static constexpr int XI = RT * KB / 1024;            // load instructions of x per stage; fewer than waves: some twice
  static constexpr int XL = XI < NW ? 1 : XI / NW, WL = NC * WKB / 1024 / NW;  // loads per wave and stage
  // 4-bit: the scales of SG groups of each row of W (as many as a stage may have, at
  // least 16), and the loads of them per wave.
  static constexpr int SG = KB > 1024 ? KB / 64 : 16;
  static constexpr int SBYTES = Q4_ ? NC * SG * 4 : 0, SL = SBYTES / 256 / NW;
  static constexpr int XBYTES = RT * KB, WBYTES = NC * WKB, STAGE = XBYTES + WBYTES;
  static constexpr int RED = WK > 1 ? NW * MT * NT * 1024 : 0;  // partial sums of the k waves
  // A wave of at least 64 finished columns turns its outputs round in LDS and
  // stores whole lines; 8-byte pieces of 16 rows at a time cost a 256 x 256
  // tile 9 us (8% of an int8 tile of 8192 inputs).
  static constexpr bool TURN = NTE >= 4;
  static constexpr int YROW = NTE * 32 + 16;           // bytes of an output row in LDS
  static constexpr int YWAVE = TURN ? MT * 16 * YROW : 0;
  static constexpr int INFO = (GATED_ ? 64 : 32) * IR;  // the rows' descriptions (gated: of both projections)
  static constexpr int TAIL = RED + INFO + NW * YWAVE;  // and the rows' descriptions, when the ring is done
  static constexpr int RING = PIPE ? 5 * XBYTES : S * (STAGE + SBYTES);  // pipelined: five places of one operand's stage
  static constexpr int LDS = RING > TAIL ? RING : TAIL;
  static constexpr int DT = NTE < 4 ? NTE : Q4_ && RT >= 64 ? 2 : 4;  // column tiles finished at a time
  // Adapters whose B is in flight or in use (delta): rows of one decode tile
  // all differ, and a wave waits for each adapter in turn; the rows of a
  // prefill tile share one, which is kept from row tile to row tile instead.
  static constexpr int AHEAD = RT >= 256 ? 1 : Q4_ && RT >= 64 ? 2 : 4;
  static_assert(WL >= 1 && XI * 1024 == RT * KB && (XI < NW ? NW % XI == 0 : XL * NW == XI) && WL * NW * 1024 == WBYTES, "loads per wave");
  static_assert(!Q4_ || (SL >= 1 && SL * NW * 256 == SBYTES && !I8_ && !PIPE_), "4-bit: scales per wave");
  static_assert(RT >= 16 || (Q4_ && WR == 1 && (RT & (RT - 1)) == 0), "fewer rows than a matrix-core tile");
  static_assert(!GATED_ || (NT % 2 == 0 && NW % 2 == 0 && HC % 16 == 0 && !I8_), "gated: the waves split the halves");
  static_assert(KB % (64 * WK) == 0 && KB >= 128, "k steps per wave");
  static_assert((S - 1) * (XL + WL + SL) < 64, "the load counter holds the stages in flight");
  static_assert(LDS <= 160 * 1024, "LDS");
};

// What the account of the tiles (api.hip) knows of one.
template <class C>
constexpr GemmTile tile_of(double fixed) {
  return {C::RT, C::HC, C::NC, 160 * 1024 / C::LDS, fixed, C::KB, C::Q4 ? (C::KB > 1024 ? 1.0 : C::S > 2 ? 0.72 : 0.78) : 0., 0.3 * C::MT * C::NTE / C::DT * (C::GATED ? 2 : 1)};
}

__device__ __forceinline__ const GemmDesc &gemm_desc() {
  return *(const GemmDesc *)(const void *)__builtin_amdgcn_kernarg_segment_ptr();
}

// A buffer resource as four scalar words (for the inline-assembly loads).
__device__ __forceinline__ u32x4 rsrc_words(const void *base, uint32_t bytes) {
  const uint64_t a = (uint64_t)(uintptr_t)base;
  return u32x4{(uint32_t)uniform((int)(uint32_t)a), (uint32_t)uniform((int)((uint32_t)(a >> 32) & 0xffffu)),
               (uint32_t)uniform((int)bytes), (uint32_t)kBufferWord3};
}

// 16 bytes per lane from r + voff + soff straight to LDS at lds + 16 * lane
// (out-of-range lanes write zeros).  Counted by vmcnt; waits are the caller's.
__device__ __forceinline__ void dma16(u32x4 r, uint32_t voff, uint32_t soff, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds"
               :
               : "s"(lds), "v"(voff), "s"(r), "s"(soff)
               : "memory", "m0");
}

// 4 bytes per lane, to LDS at lds + 4 * lane.
__device__ __forceinline__ void dma4(u32x4 r, uint32_t voff, uint32_t soff, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dword %1, %2, %3 offen lds"
               :
               : "s"(lds), "v"(voff), "s"(r), "s"(soff)
               : "memory", "m0");
}

// Wait until at most N of this wave's loads are outstanding and its LDS reads
// are done, then for the block.
template <int N>
__device__ __forceinline__ void stage_barrier() {
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" : : "n"(N) : "memory");
}

// Segments of at most max_seg, as tiles of RT rows: how many tiles there are,
// and the segment of one.  Every wave does it for itself, 64 segments a step.
struct TileOf {
  int slot, pos0, rows;  // segment's slot, first sorted row and rows
  int first, tiles;      // its first tile's number, and its tiles
};
// AT_ONCE: the arrays are read as far as they may reach, beside the number of
// segments instead of after it.
template <int RT, bool AT_ONCE>
__device__ __forceinline__ int seg_tiles(const GemmDesc &d, int s, int nseg, int *slot, int *o0, int *len) {
  *slot = -1;
  *o0 = 0;
  *len = 0;
  if (s >= (AT_ONCE ? d.max_seg : nseg)) return 0;
  *slot = d.seg_adapter[s];
  *o0 = d.seg_offsets[s];
  const int end = d.seg_offsets[s + 1];
  const bool ok = segment_fits(*slot, *o0, end, d.num_slots, d.num_rows) && (!AT_ONCE || s < nseg);
  *len = ok ? end - *o0 : 0;
  return (*len + RT - 1) / RT;
}
__device__ __forceinline__ int wave_scan(int v, int lane) {  // inclusive
#pragma unroll
  for (int k = 1; k < 64; k *= 2) {
    const int u = __shfl_up(v, k, 64);
    if (lane >= k) v += u;
  }
  return v;
}
template <int RT, bool AT_ONCE>
__device__ __forceinline__ int total_tiles(const GemmDesc &d, int nseg) {
  const int lane = threadIdx.x & 63;
  int total = 0;
  for (int s0 = 0; s0 < nseg; s0 += 64) {
    int slot, o0, len;
    total += __builtin_amdgcn_readlane(wave_scan(seg_tiles<RT, AT_ONCE>(d, s0 + lane, nseg, &slot, &o0, &len), lane), 63);
  }
  return total;
}
template <int RT, bool AT_ONCE>
__device__ __forceinline__ bool find_tile(const GemmDesc &d, int nseg, int t, TileOf *out) {
  const int lane = threadIdx.x & 63;
  int before = 0;
  for (int s0 = 0; s0 < nseg; s0 += 64) {
    int slot, o0, len;
    const int n = seg_tiles<RT, AT_ONCE>(d, s0 + lane, nseg, &slot, &o0, &len);
    const int upto = before + wave_scan(n, lane);
    const uint64_t hit = __ballot(t < upto && n > 0);
    if (hit) {
      const int l = __builtin_ctzll(hit);
      const int start = __builtin_amdgcn_readlane(upto - n, l);
      out->slot = __builtin_amdgcn_readlane(slot, l);
      out->pos0 = __builtin_amdgcn_readlane(o0, l);
      out->rows = __builtin_amdgcn_readlane(len, l);
      out->first = start;
      out->tiles = __builtin_amdgcn_readlane(n, l);
      return true;
    }
    before = __builtin_amdgcn_readlane(upto, 63);
  }
  return false;
}

// Order of a module's tiles over its blocks: blocks go to the 8 XCDs in turn,
// so each XCD takes one contiguous eighth of an order that walks kPatchRows
// row tiles (of one segment) before it moves to the next column tile; the
// tiles an XCD works on at one time then share rows and columns in its L2.
// A segment of up to 8 row tiles is one patch (32 segments of 128 to 2048 rows
// on 8192 x 8192: bf16 4.26 -> 4.15 ms, int8 4.81 -> 4.65; in longer segments
// 8 rows measured up to 10% slower than 4).
constexpr int kPatchRows = 4, kPatchMost = 8;
__device__ __forceinline__ int xcd_order(int local, int n) {  // the local-th block's place in the order of n tiles
  const int xcd = local & 7, i = local >> 3;
  return xcd * (n >> 3) + min(xcd, n & 7) + i;
}
__device__ __forceinline__ void patch_order(int lin, int row_tiles, int col_tiles, int *rt, int *ct) {
  const int patch = row_tiles <= kPatchMost ? row_tiles : kPatchRows;
  const int group = lin / (patch * col_tiles);
  const int in = lin - group * patch * col_tiles;
  const int gr = min(patch, row_tiles - group * patch);
  *ct = in / gr;
  *rt = group * patch + in - *ct * gr;
}

// A slot's weight in the device table, checked.
struct GemmWeight {
  const uint8_t *W;
  const float *Ws;
  int64_t ldw, lds;  // bytes; floats (4-bit)
  bool ok;
};
template <class C>
__device__ __forceinline__ GemmWeight load_weight(const GemmDesc &d, const GemmModule &m, int slot, int col) {
  static_assert(sizeof(lora_weight_q4g_entry_t) == sizeof(lora_weight_entry_t), "one table stride");
  const lora_weight_q4g_entry_t raw = reinterpret_cast<const lora_weight_q4g_entry_t *>(d.weights)[(int64_t)slot * kMaxModules + col];
  auto wide = [](int64_t v) {
    return (int64_t)(((uint64_t)(uint32_t)uniform((int)(uint32_t)((uint64_t)v >> 32)) << 32) |
                     (uint32_t)uniform((int)(uint32_t)v));
  };
  GemmWeight r{uniform(static_cast<const uint8_t *>(raw.W)), nullptr, wide(raw.ldw), 0, false};
  const int64_t most = m.row_most;  // bytes of a row
  if constexpr (C::Q4) {
    r.Ws = uniform(raw.Ws);
    r.lds = wide(raw.lds);
    r.ok = ((uintptr_t)r.W & 15) == 0 && r.ldw >= m.d_in / 2 && r.ldw % 16 == 0 && r.ldw <= most && r.Ws != nullptr &&
           ((uintptr_t)r.Ws & 3) == 0 && r.lds >= (m.d_in >> m.group_log) && r.lds <= most / 4;
  } else {
    r.ok = ((uintptr_t)r.W & 15) == 0 && r.ldw >= m.d_in && r.ldw % 8 == 0 && r.ldw <= most / 2;
    r.ldw *= 2;
  }
  return r;
}

template <bool I8>
struct AccOf {
  typedef f32x4_t type;
};
template <>
struct AccOf<true> {
  typedef i32x4_t type;
};

__device__ __forceinline__ f32x4_t mma(u32x4 a, u32x4 b, f32x4_t c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a), __builtin_bit_cast(bf16x8_t, b), c, 0,
                                                 0, 0);
}
__device__ __forceinline__ i32x4_t mma(u32x4 a, u32x4 b, i32x4_t c) {
  return __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4_t, a), __builtin_bit_cast(i32x4_t, b), c, 0, 0,
                                               0);
}

// The same product with the sums pinned in place in accumulation registers
// (the pipelined loop): a wave's 256 sums fill that file, and left to itself
// the compiler moves them about.  The wait before the sums are read
// (mma_drain) is the caller's.
__device__ __forceinline__ void mma_acc(u32x4 a, u32x4 b, f32x4_t &c) {
  asm volatile("v_mfma_f32_16x16x32_bf16 %0, %1, %2, %0" : "+a"(c) : "v"(a), "v"(b));
}
__device__ __forceinline__ void mma_acc(u32x4 a, u32x4 b, i32x4_t &c) {
  asm volatile("v_mfma_i32_16x16x64_i8 %0, %1, %2, %0" : "+a"(c) : "v"(a), "v"(b));
}
__device__ __forceinline__ void mma_drain() {
  asm volatile("s_nop 15\n\ts_nop 15" : : : "memory");
  __builtin_amdgcn_sched_barrier(0);
}

// Hold results of the matrix cores until they may be read: the compiler counts
// the wait states on one of the paths that lead to the read only, so a branch
// between them can leave too few (seen as wrong first elements of a tile).
template <int N>
__device__ __forceinline__ void mma_settle(f32x4_t (&t)[N]) {
  static_assert(N >= 1 && N <= 4, "tiles");
  if constexpr (N == 1) asm volatile("s_nop 10" : "+v"(t[0]));
  else if constexpr (N == 2) asm volatile("s_nop 10" : "+v"(t[0]), "+v"(t[1]));
  else if constexpr (N == 3) asm volatile("s_nop 10" : "+v"(t[0]), "+v"(t[1]), "+v"(t[2]));
  else asm volatile("s_nop 10" : "+v"(t[0]), "+v"(t[1]), "+v"(t[2]), "+v"(t[3]));
}

// Eight fp32 values of v as bf16 vectors, the largest piece first.  Two rounded
// pieces hold it to 2^-16 (split_v8: the int8 base); three cut ones hold all
// of its 24 bits: 8 a piece, each remainder exact (a value that is infinite or no
// number is its first piece), so that a delta that cancels the base leaves what the
// formula leaves.  It is one matrix-core step more for an adapter and 16 rows: 16
// rows on a layer, rank 32, 149 us either way; 7637 rows of rank 64, gated 6260
// either way, 4-bit 8460 -> 8535.
template <int P>
struct VPieces {
  u32x4 p[P];
};
template <int P>
__device__ __forceinline__ VPieces<P> split_v(const float *v) {
  static_assert(P == 2 || P == 3, "pieces");
  if constexpr (P == 2) {
    const V8Split s = split_v8(v);
    return VPieces<2>{{s.hi, s.lo}};
  } else {
    VPieces<3> r;
    auto cut = [](float f) { return __uint_as_float(__float_as_uint(f) & 0xffff0000u); };
    auto both = [](float a, float b) { return __builtin_amdgcn_perm(__float_as_uint(b), __float_as_uint(a), 0x07060302u); };
    auto rest = [&](float f) { return fabsf(f) < INFINITY ? f - cut(f) : 0.f; };
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float a = v[2 * i], b = v[2 * i + 1], ar = rest(a), br = rest(b);
      r.p[0][i] = both(a, b);
      r.p[1][i] = both(ar, br);
      r.p[2][i] = both(ar - cut(ar), br - cut(br));
    }
    return r;
  }
}

// The B of one adapter for DT column tiles: values and output scales.
template <int DT, int KT>
struct BFrag {
  u32x4 b[DT][KT];
  float s[DT];
  int a = -1;
  bool q8;
};

template <int DT, int KT>
__device__ __forceinline__ void load_b(const GemmModule &m, const RowInfo &ri, int l, bool on, int n0,
                                       BFrag<DT, KT> &f) {
  const int lane = threadIdx.x & 63, r_in = lane & 15, g = lane >> 4;
  f.a = on ? __builtin_amdgcn_readlane(ri.a, l) : -1;
  const int rank = on ? __builtin_amdgcn_readlane(ri.rank, l) : 0;
  f.q8 = __builtin_amdgcn_readlane(ri.fmt, l) == LORA_FORMAT_INT8_ROWS;
  const uint8_t *B = (const uint8_t *)(uintptr_t)(
      (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(uintptr_t)ri.B, l) |
      ((uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)((uintptr_t)ri.B >> 32), l) << 32));
  const uint32_t row_bytes = f.q8 ? (uint32_t)ldb8_of(rank) : (uint32_t)((rank + 7) & ~7) * 2;
  const uint8_t *vals = B + (f.q8 ? q8_values_offset(m.d_out) : 0);
  const rsrc_t rb = make_rsrc(on ? vals : nullptr, on ? (uint32_t)m.d_out * row_bytes : 0u);
  const rsrc_t rs = make_rsrc(on && f.q8 ? B : nullptr, on && f.q8 ? q8_values_offset(m.d_out) : 0u);
#pragma unroll
  for (int nt = 0; nt < DT; ++nt) {
    const int n = n0 + nt * 16 + r_in;
#pragma unroll
    for (int ks = 0; ks < KT; ++ks) {
      const int j = ks * 32 + g * 8;
      const uint32_t at = f.q8 ? (uint32_t)(j & ~15) : (uint32_t)j * 2;
      f.b[nt][ks] = buf_ld16_stream(rb, n < m.d_out && j < rank ? (uint32_t)n * row_bytes + at : kOutOfRange, 0);
    }
    f.s[nt] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(rs, n < m.d_out ? (uint32_t)n * 4 : kOutOfRange, 0, 0));
  }
}

template <int P, int DT, int KT>
__device__ __forceinline__ void use_b(const RowInfo &ri, const VPieces<P> (&v)[KT], const BFrag<DT, KT> &f,
                                      f32x4_t (&acc)[DT]) {
  const int g = (threadIdx.x & 63) >> 4;
  u32x4 b[DT][KT];
  f32x4_t sc[DT];
#pragma unroll
  for (int nt = 0; nt < DT; ++nt) {
#pragma unroll
    for (int ks = 0; ks < KT; ++ks) b[nt][ks] = f.b[nt][ks];
    sc[nt] = f32x4_t{1.f, 1.f, 1.f, 1.f};
  }
  if (f.q8) {
#pragma unroll
    for (int nt = 0; nt < DT; ++nt) {
#pragma unroll
      for (int ks = 0; ks < KT; ++ks)
        b[nt][ks] = i8x8_to_bf16x8((g & 1) ? u32x2{b[nt][ks].z, b[nt][ks].w} : u32x2{b[nt][ks].x, b[nt][ks].y});
#pragma unroll
      for (int i = 0; i < 4; ++i) sc[nt][i] = __shfl(f.s[nt], 4 * g + i, 64);
    }
  }
  const bool mine = ri.a == f.a;
  f32x4_t t[DT];
#pragma unroll
  for (int nt = 0; nt < DT; ++nt) {
    t[nt] = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int ks = 0; ks < KT; ++ks)
#pragma unroll
      for (int k = P - 1; k >= 0; --k) t[nt] = mma(b[nt][ks], v[ks].p[k], t[nt]);
  }
  mma_settle(t);
#pragma unroll
  for (int nt = 0; nt < DT; ++nt)
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[nt][i] = mine ? fmaf(t[nt][i], sc[nt][i], acc[nt][i]) : acc[nt][i];
}

// The delta of one 16-row tile on top of its finished base sums acc[.] (4
// consecutive outputs of a lane's row per column tile, columns n0 + 16 nt).
// For each adapter among the 16 rows in turn, B_a's rows are the matrix-core A
// operand and all 16 rows' v the B operand; the columns of that adapter's rows
// are then added and the others dropped (selected, not multiplied by zero: a
// non-finite factor of one row's adapter must not reach the others).  v, fp32,
// enters in bf16 pieces (VPieces).  The B of the next adapters is
// requested before the current one's products (AHEAD).
// An int8 B (values exact in bf16) comes in the same 16-byte loads: the piece
// that holds a lane's 8 values, of which it keeps its half; the output scales
// come one per lane and are handed round.
// AHEAD == 1: f[0] may hold the last row tile's adapter, which is then not
// loaded again.
// The rows of 16 whose adapter has not been met yet.
struct DeltaRows {
  uint64_t todo;
  __device__ __forceinline__ int next(const RowInfo &ri, bool *on) {  // a row of the next adapter
    *on = todo != 0;
    const int l = *on ? __builtin_ctzll(todo) : 0;
    todo &= ~__ballot(ri.a == __builtin_amdgcn_readlane(ri.a, l));
    return l;
  }
};
__device__ __forceinline__ DeltaRows delta_rows(const RowInfo &ri) { return DeltaRows{__ballot(ri.a >= 0) & 0xffffull}; }

// Request the B of the first AHEAD adapters; then add them and the others.
template <int DT, int KT, int AHEAD>
__device__ __forceinline__ void begin_delta(const GemmModule &m, const RowInfo &ri, int n0, DeltaRows &rows,
                                            BFrag<DT, KT> (&f)[AHEAD]) {
#pragma unroll
  for (int k = 0; k < AHEAD; ++k) {
    bool on;
    const int l = rows.next(ri, &on);
    load_b(m, ri, l, on, n0, f[k]);
  }
}
template <int P, int DT, int KT, int AHEAD>
__device__ __forceinline__ void finish_delta(const GemmModule &m, const RowInfo &ri, const VPieces<P> (&v)[KT], int n0,
                                             DeltaRows &rows, BFrag<DT, KT> (&f)[AHEAD], f32x4_t (&acc)[DT]) {
  for (bool more = true; more;) {
#pragma unroll
    for (int k = 0; k < AHEAD; ++k) {
      if (f[k].a < 0) {
        more = false;
        break;
      }
      use_b(ri, v, f[k], acc);
      bool on;
      const int l = rows.next(ri, &on);
      load_b(m, ri, l, on, n0, f[k]);
    }
  }
}
template <int P, int DT, int KT, int AHEAD>
__device__ __forceinline__ void add_delta(const GemmModule &m, const RowInfo &ri, const VPieces<P> (&v)[KT], int n0,
                                          BFrag<DT, KT> (&f)[AHEAD], f32x4_t (&acc)[DT]) {
  DeltaRows rows = delta_rows(ri);
  if constexpr (AHEAD == 1) {
    while (rows.todo) {
      bool on;
      const int l = rows.next(ri, &on);
      if (__builtin_amdgcn_readlane(ri.a, l) != f[0].a) load_b(m, ri, l, true, n0, f[0]);
      use_b(ri, v, f[0], acc);
    }
  } else {
    begin_delta(m, ri, n0, rows, f);
    finish_delta(m, ri, v, n0, rows, f, acc);
  }
}

// Four outputs rounded to bf16: on the largest tile two by one instruction; on
// the others as pack_bf16x2 does it, in four (there the short form is scheduled
// so that the rank 64 delta of the 128-row tile spills 26 registers, 646 -> 700
// us for a whole layer).
template <class C>
__device__ __forceinline__ u32x2 pack_out(f32x4_t o) {
  typedef __bf16 b16x4_t __attribute__((ext_vector_type(4)));
  if constexpr (C::RT >= 256) return __builtin_bit_cast(u32x2, __builtin_convertvector(o, b16x4_t));
  else return u32x2{pack_bf16x2(o[0], o[1]), pack_bf16x2(o[2], o[3])};
}

// Eight 4-bit weights (value j in bits 4j .. 4j+3, two's complement) as bf16
// values (24 + q) / 16, in the order 0 4 1 5 2 6 3 7: with its top bit turned a
// weight is q + 8, which in the upper four bits of the significand of 1.0 makes 1 +
// (q + 8) / 16.  Two values at a time take a shift and one operation (and, then
// exclusive or with 1.5), eight for a register; converting each value took 15.
// The sum over them is (sum q x + 24 sum x) / 16, so it starts from -24/16 sum x,
// one matrix-core step for every tile of the same x.  Its rounding is that of sums
// of up to (|q| + 48) |x|, times the scale: 2^-24 of them an addition, far below
// a bf16 output's own for weights of any use, but no small part of a sum that is
// itself near 0: a group of zeros leaves up to that, where converted weights leave 0.
constexpr uint32_t kQ4Less = 0xBFC0BFC0u;  // -24/16 twice
__device__ __forceinline__ u32x4 q4x8_shifted(uint32_t q) {
  auto two = [](uint32_t v) { return (v & 0x00780078u) ^ 0x3FC03FC0u; };
  return u32x4{two(q << 3), two(q >> 1), two(q >> 5), two(q >> 9)};
}
// Eight bf16 values in that order.
__device__ __forceinline__ u32x4 pairs_apart(u32x4 x) {
  return u32x4{__builtin_amdgcn_perm(x.z, x.x, 0x05040100u), __builtin_amdgcn_perm(x.z, x.x, 0x07060302u),
               __builtin_amdgcn_perm(x.w, x.y, 0x05040100u), __builtin_amdgcn_perm(x.w, x.y, 0x07060302u)};
}

// act(z) = z sigma(z (c1 + c3 z^2)): SiLU with c1 = 1, c3 = 0; GELU in its tanh form
// with c1 = 2 sqrt(2 / pi), c3 = 0.044715 c1, since (1 + tanh(t)) / 2 = sigma(2t).
// The square is bounded so that 0 * z^2 stays 0; at 1e30 sigma is 0 or 1 already.
// exp and the reciprocal are the hardware's: a few 2^-24 relative, and |t| 2^-24
// (1 - sigma) for each rounding of t and of its product with log2 e (SiLU one, GELU
// four): 2^-17.5 and 2^-15.5 where sigma is smallest (t = -87; below, 0), less than
// a 100th of the output's rounding.
__device__ __forceinline__ float gate_act(float z, float c1, float c3) {
  const float t = z * fmaf(c3, fminf(z * z, 1e30f), c1);
  return z * __builtin_amdgcn_rcpf(1.f + __expf(-t));
}

// KT: 32-wide steps of the ranks of a delta (1: ranks up to 32, 2: up to 64; 0: no delta).
template <class C, bool GROUPED, int KT>
__device__ __forceinline__ void gemm_block(const GemmDesc &d, uint8_t *lds) {
  typedef typename AccOf<C::I8>::type acc_t;
  constexpr bool DELTA = KT > 0;
  const int t = threadIdx.x, lane = t & 63, w = wave_id();
  const int r_in = lane & 15, g = lane >> 4;
  const int wk = w / (C::WR * C::WC), wr = (w / C::WC) % C::WR, wc = w % C::WC;

  int mi = 0;
#pragma unroll
  for (int k = 1; k < kMaxModules; ++k)
    if (k < d.n_active && (int)blockIdx.x >= d.mod[k].block_base) mi = k;
  const GemmModule m = gemm_desc().mod[mi];
  const int half = C::GATED ? w / (C::NW / 2) : 0;  // whose rows of W this wave loads: gate's, up's
  const int local = (int)blockIdx.x - m.block_base;

  // a few rows: v and B are requested before and right behind the main loop
  constexpr bool EARLY = DELTA && (C::Q4 || C::GATED) && C::MT == 1 && C::NTE == C::DT && C::WK > 1;

  // the block's rows and columns
  int row0, rows, ct, slot = 0;
  const uint8_t *W;
  const float *Ws;
  int64_t ldw, lds_ = 0;  // of W, bytes; of 4-bit scales, floats
  auto xload = [&](int i) { return C::XI < C::NW ? w % C::XI : i * C::NW + w; };
  // the row of x, in LDS, of a lane's i-th load, and its 16-byte place in the row
  auto xrow_of = [&](int i) {
    return C::KB > 1024 ? (xload(i) * 64 + lane) / C::PIECES : lane / C::PIECES + xload(i) * (1024 / C::KB);
  };
  auto xslot_of = [&](int i) { return (C::KB > 1024 ? xload(i) * 64 + lane : lane) % C::PIECES; };
  int xperm[C::XL];  // grouped: the rows that this lane loads
  (void)xperm;
  if constexpr (GROUPED) {
    const int nseg = min(uniform(*d.num_segments), d.max_seg);
    if (blockIdx.x == 0 && w == 0)  // segments that do not fit the batch, counted once per call
      for (int s = lane; s < nseg; s += 64) {
        if (!segment_fits(d.seg_adapter[s], d.seg_offsets[s], d.seg_offsets[s + 1], d.num_slots, d.num_rows))
          atomicAdd(d.status, 1);
      }
    int rt;
    TileOf tile;
    if constexpr (C::RT >= 128) {
      const int total = total_tiles<C::RT, C::Q4 || C::GATED>(d, nseg);
      if (local >= total * m.n_tiles) return;
      const int lin = xcd_order(local, total * m.n_tiles);
      if (!find_tile<C::RT, C::Q4 || C::GATED>(d, nseg, lin / m.n_tiles, &tile)) return;
      patch_order(lin - tile.first * m.n_tiles, tile.tiles, m.n_tiles, &rt, &ct);
    } else {
      rt = local / m.n_tiles;
      ct = local - rt * m.n_tiles;
      if (!find_tile<C::RT, C::Q4 || C::GATED>(d, nseg, rt, &tile)) return;
      rt -= tile.first;
    }
    row0 = tile.pos0 + rt * C::RT;
    rows = min(C::RT, tile.rows - rt * C::RT);
    slot = tile.slot;
    if constexpr (C::GATED || C::Q4) {
#pragma unroll
      for (int i = 0; i < C::XL; ++i) xperm[i] = d.perm[row0 + min(xrow_of(i), rows - 1)];
      const GemmWeight own = load_weight<C>(d, m, slot, C::GATED ? gemm_desc().mod[half].col : m.col);
      bool there = own.W != nullptr, ok = own.ok;
      if constexpr (C::GATED) {  // gate and up: both or neither
        const GemmWeight other = load_weight<C>(d, m, slot, gemm_desc().mod[1 - half].col);
        if (there != (other.W != nullptr)) ok = false;
        there |= other.W != nullptr;
        ok &= other.ok;
      }
      if (!there) return;
      if (!ok) {
        if (rt == 0 && ct == 0 && t == 0) atomicAdd(d.status, 1);
        return;
      }
      W = own.W;
      Ws = own.Ws;
      ldw = own.ldw;
      lds_ = own.lds;
    } else {
      const lora_weight_entry_t raw = d.weights[(int64_t)slot * kMaxModules + m.col];
      W = uniform(static_cast<const uint8_t *>(raw.W));
      Ws = uniform(raw.Ws);
      const int64_t ld = raw.ldw;
      ldw = (int64_t)(((uint64_t)(uint32_t)uniform((int)(uint32_t)((uint64_t)ld >> 32)) << 32) |
                      (uint32_t)uniform((int)(uint32_t)ld));
      if (W == nullptr) return;  // this slot has no weight for the projection: its rows stay as they are
      const int elt = C::I8 ? 1 : 2;
      const bool ok = ((uintptr_t)W & 15) == 0 && ldw >= (C::I8 ? (m.d_in + 15) & ~15 : m.d_in) && ldw % (16 / elt) == 0 &&
                      ldw <= (int64_t)0xFFFFFF00 / elt / m.d_out &&
                      (!C::I8 || (Ws != nullptr && ((uintptr_t)Ws & 15) == 0));
      if (!ok) {
        if (rt == 0 && ct == 0 && t == 0) atomicAdd(d.status, 1);
        return;
      }
      ldw *= elt;
    }
  } else {
    int rt;
    if constexpr (C::RT >= 128) {
      patch_order(xcd_order(local, d.row_tiles * m.n_tiles), d.row_tiles, m.n_tiles, &rt, &ct);
    } else {
      rt = local / m.n_tiles;
      ct = local - rt * m.n_tiles;
    }
    row0 = rt * C::RT;
    rows = min(C::RT, d.num_rows - row0);
    if constexpr (C::GATED) {
      const GemmModule &mine = gemm_desc().mod[half];
      W = mine.W;
      Ws = mine.Ws;
      ldw = mine.ldw;
      lds_ = mine.ldws;
    } else {
      W = m.W;
      Ws = m.Ws;
      ldw = m.ldw;
      lds_ = m.ldws;
    }
  }
  const int n0 = ct * C::HC;

  // ---- this lane's pieces of a stage: offsets of the rows it loads
  // (an index past the batch is moved into it for the load; load_info drops its row)
  // this thread's row of the tile: its description (rows.hip) in two pieces, or (grouped) its row
  RowInfo mine{};
  u32x4 desc[C::GATED ? 2 : 1][2];
  int prow = 0;
  (void)mine;
  (void)desc;
  (void)prow;
  f32x4_t vraw[C::GATED ? 2 : 1][DELTA ? KT : 1][2];
  (void)vraw;
  if constexpr (C::Q4 || C::GATED) {
    const int at = row0 + min(t, rows - 1);
    if constexpr (GROUPED) {
      prow = d.perm[at];
    } else {
#pragma unroll
      for (int k = 0; k < (C::GATED ? 2 : 1); ++k) {
        const u32x4 *src = reinterpret_cast<const u32x4 *>((k == 0 ? m.info : gemm_desc().mod[1].info) + at);
        desc[k][0] = src[0];
        desc[k][1] = src[1];
      }
      if constexpr (EARLY) {
        const int64_t row = (int64_t)(row0 + min(r_in, rows - 1)) * d.rs;
#pragma unroll
        for (int ks = 0; ks < KT; ++ks) {
          const int j = min(ks * 32 + g * 8, d.rs - 8);  // columns past the rank are not used
          vraw[0][ks][0] = *(const f32x4_t *)(m.v + row + j);
          vraw[0][ks][1] = *(const f32x4_t *)(m.v + row + j + 4);
          if constexpr (C::GATED) {
            vraw[1][ks][0] = *(const f32x4_t *)(gemm_desc().mod[1].v + row + j);
            vraw[1][ks][1] = *(const f32x4_t *)(gemm_desc().mod[1].v + row + j + 4);
          }
        }
      }
    }
  }
  const u32x4 rx = rsrc_words(m.x, m.x_bytes);
  const u32x4 rw = rsrc_words(W, (uint32_t)(ldw * m.d_out));
  // the resources are written by vector instructions; the assembly that reads
  // them needs 5 wait states after those, which the compiler does not count
  asm volatile("s_nop 4" : : "s"(rx), "s"(rw));
  constexpr int WRPI = 1024 / C::WKB;
  const int wlrow = lane / C::WPIECES, wslot = lane % C::WPIECES;
  // the row of W, in LDS, of a lane's i-th load, and where in LDS the load goes
  auto wload = [&](int i) { return C::GATED ? w * C::WL + i : i * C::NW + w; };
  auto wload_s = [&](int i) { return C::GATED ? w * C::SL + i : i * C::NW + w; };
  auto wrow_of = [&](int i) { return wload(i) * WRPI + wlrow; };
  uint32_t xoff[C::XL], woff[C::WL];
#pragma unroll
  for (int i = 0; i < C::XL; ++i) {
    const int r = xrow_of(i);
    const int rr = min(r, rows - 1);  // past the tile: its last row again (never stored)
    int b = row0 + rr;
    if constexpr (GROUPED && (C::Q4 || C::GATED)) {
      b = (int)min((unsigned)xperm[i], (unsigned)(d.num_rows - 1));
      if (m.rows_per_x > 1) b /= m.rows_per_x;
    } else if constexpr (GROUPED) b = (int)min((unsigned)d.perm[b], (unsigned)(d.num_rows - 1)) / m.rows_per_x;
    else if (d.order) b = (int)min((unsigned)d.order[b], (unsigned)(d.num_rows - 1));
    xoff[i] = (uint32_t)((int64_t)b * m.ldx) + (uint32_t)((xslot_of(i) ^ (r & C::SWZ)) * 16);
    if constexpr (C::Q4 || C::GATED) xoff[i] = r < rows ? xoff[i] : kOutOfRange;  // or nothing: zeros, no fetch
  }
#pragma unroll
  for (int i = 0; i < C::WL; ++i) {
    const int r = wrow_of(i);
    const int n = min(n0 + r - half * C::HC, m.d_out - 1);
    woff[i] = (uint32_t)((int64_t)n * ldw) + (uint32_t)((wslot ^ (r & C::WSWZ)) * 16);
  }
  // 4-bit: the scales of SG groups (a batch), 64 consecutive bytes or more of each
  // row of Ws; in LDS [4 rows][group][row], so that a lane reads its four outputs' in one.
  // (A stage's own, 4 to 32 bytes of a row each time: every load instruction met
  // 64 lines, 7 to 36 us of the calls below.)
  const int glog = C::Q4 ? m.group_log : 0;
  const u32x4 rsc = rsrc_words(C::Q4 ? Ws : nullptr, C::Q4 ? (uint32_t)((lds_ * (m.d_out - 1) + (m.d_in >> glog)) * 4) : 0u);
  if constexpr (C::Q4) asm volatile("s_nop 4" : : "s"(rsc));
  constexpr int SLN = C::SL > 0 ? C::SL : 1;
  uint32_t soffs[SLN];
  auto squad = [&](int i) { return (wload_s(i) * 64 + lane) / (4 * C::SG); };  // its 4 rows
  auto sgroup = [&](int i) { return ((wload_s(i) * 16 + (lane >> 2)) % C::SG) ^ (squad(i) & 3); };
  if constexpr (C::Q4) {
#pragma unroll
    for (int i = 0; i < C::SL; ++i) {
      const int n = min(n0 + squad(i) * 4 + (lane & 3) - half * C::HC, m.d_out - 1);
      soffs[i] = (uint32_t)(((int64_t)n * lds_ + sgroup(i)) * 4);
    }
  }

  const uint32_t lds_base = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t *)lds;
  const int rounds = (m.kbytes + C::KB - 1) / C::KB;
  const int full = m.kbytes / C::KB;
  // the loads of one operand of stage r to LDS at `at`; a last, partial stage
  // and those past the end get zeros beyond the row
  auto issue_x = [&](int r, uint32_t at) {
    const uint32_t soff = (uint32_t)(r * C::KB);
    const int left = m.kbytes - r * C::KB;
    at += lds_base;
    if (r < full) {
#pragma unroll
      for (int i = 0; i < C::XL; ++i) dma16(rx, xoff[i], soff, at + (uint32_t)xload(i) * 1024);
    } else {
#pragma unroll
      for (int i = 0; i < C::XL; ++i) {
        const int piece = xslot_of(i) ^ (xrow_of(i) & C::SWZ);
        const bool on = piece * 16 < left && (!(C::Q4 || C::GATED) || xoff[i] != kOutOfRange);
        dma16(rx, on ? xoff[i] + soff : kOutOfRange, 0, at + (uint32_t)xload(i) * 1024);
      }
    }
  };
  auto issue_w = [&](int r, uint32_t at) {
    const uint32_t soff = (uint32_t)(r * C::WKB);
    const int left = (C::Q4 ? m.kbytes / 4 : m.kbytes) - r * C::WKB;
    at += lds_base;
    if (r < full) {
#pragma unroll
      for (int i = 0; i < C::WL; ++i) dma16(rw, woff[i], soff, at + (uint32_t)wload(i) * 1024);
    } else {
#pragma unroll
      for (int i = 0; i < C::WL; ++i) {
        const int piece = wslot ^ (wrow_of(i) & C::WSWZ);
        dma16(rw, piece * 16 < left ? woff[i] + soff : kOutOfRange, 0, at + (uint32_t)wload(i) * 1024);
      }
    }
  };
  // A stage's batch of scales goes with the first stage that needs it, before its
  // operands (loads complete in order).  A place for each of the stages under way:
  // none of them can need the batch whose place is taken.
  auto batch_of = [&](int r) { return ((r * (C::KB / 2)) >> glog) / C::SG; };
  int s_batch = -1, s_put = 0;
  auto issue_s = [&](int r) {
    const int batch = batch_of(r);
    if (r >= rounds || batch == s_batch) return;
    s_batch = batch;
#pragma unroll
    for (int i = 0; i < C::SL; ++i)
      dma4(rsc, batch * C::SG + sgroup(i) < (m.d_in >> glog) ? soffs[i] + (uint32_t)batch * C::SG * 4 : kOutOfRange, 0,
           lds_base + C::S * C::STAGE + s_put + (uint32_t)wload_s(i) * 256);
    s_put = s_put + C::SBYTES == C::S * C::SBYTES ? 0 : s_put + C::SBYTES;
  };
  auto issue = [&](int r, uint32_t buf) {
    if constexpr (C::Q4) issue_s(r);
    issue_x(r, buf);
    issue_w(r, buf + C::XBYTES);
  };

  // this thread's row of the tile (loaded while the first stages are on their way)
  auto load_info = [&]() {
    if constexpr (C::Q4 || C::GATED) return;
    if (t >= C::RT) return;
    const int at = row0 + min(t, rows - 1);
    const int32_t *order = GROUPED ? d.perm : d.order;
    const int b = order ? order[at] : at;
    const bool in = (unsigned)b < (unsigned)d.num_rows;  // a stray index (segments of another batch) touches nothing
    mine.b = in && t < rows ? b : -1;
    if constexpr (C::I8) mine.xs = m.xs[in ? (GROUPED ? b / m.rows_per_x : b) : 0];
    mine.a = -1;
    if constexpr (DELTA) {
      // segments come in ascending slot order: later slots were dropped by the
      // build, or their segments do not fit the batch and have no v
      const int nseg = fitting_segments(d.num_segments, d.max_seg, d.seg_offsets, d.num_rows);
      const int last_slot = nseg > 0 ? d.seg_adapter[nseg - 1] : -1;
      const int a = mine.b >= 0 ? d.ids[mine.b] : -1;
      if ((unsigned)a < (unsigned)d.num_slots && a <= last_slot) {
        const lora_adapter_entry_t e = d.table[(int64_t)a * kMaxModules + m.col];
        if (entry_ok(e, d.max_rank)) {  // a malformed entry: counted by the shrink
          mine.a = a;
          mine.rank = e.rank;
          mine.fmt = e.format;
          mine.scale = e.scale;
          mine.B = static_cast<const uint8_t *>(e.B);
        }
      }
    }
  };

  acc_t acc[C::NT][C::MT];
#pragma unroll
  for (int nt = 0; nt < C::NT; ++nt)
#pragma unroll
    for (int mt = 0; mt < C::MT; ++mt) acc[nt][mt] = acc_t{0, 0, 0, 0};

  constexpr int KS = C::KB / 64 / C::WK;  // matrix-core steps of a wave per stage
  // the first row of this wave's column tiles in LDS (gated: of its tiles of each half), and of tile nt from there
  const int xin = C::RT < 16 ? r_in & (C::RT - 1) : r_in;  // fewer rows than a tile: each several times
  const int xrow = (wr * C::MT * 16 + xin) * C::KB;
  const int wcol = wc * (C::GATED ? C::NT / 2 : C::NT) * 16;
  const int wrow = C::XBYTES + (wcol + r_in) * C::WKB;
  auto wtile = [](int nt) constexpr { return (C::GATED && nt >= C::NT / 2 ? C::HC + (nt - C::NT / 2) * 16 : nt * 16) * C::WKB; };
  if constexpr (C::PIPE) {
    // The ring has five places of one operand's stage.  In round r: w(r) and
    // x(r) in A and B (the first step's operands already in registers), w(r+1)
    // and x(r+1) in C and D; w(r+2) is sent to E during the first step.  Past
    // the barrier between the steps every wave holds the rest of stage r in
    // registers, so x(r+2) goes to A during the second.  W, which comes from
    // HBM, has a round and a half to arrive, x, mostly in L2, one.  Reads, loads
    // and products are laid out by hand, one of each in turn, and kept so.
    static_assert(!C::PIPE || (C::WK == 1 && KS == 2 && C::RT == C::NC && C::MT == C::NT), "the pipelined loop");
    constexpr int PL = C::XBYTES;                      // bytes of a place
    constexpr int SLOTS = C::MT + C::NT, PER = C::MT * C::NT / SLOTS;  // operand reads of a step, products per read
    static_assert(!C::PIPE || (C::XL * 2 == SLOTS && C::WL * 2 == SLOTS), "a load every second operand read");
    u32x4 xa[C::MT], wa[C::NT], xb[C::MT], wb[C::NT];
    const int s0 = ((0 + g) ^ (r_in & C::SWZ)) * 16, s1 = ((4 + g) ^ (r_in & C::SWZ)) * 16;
    const int wrow0 = wrow - C::XBYTES;
    uint32_t A = 0, B = PL, Cc = 2 * PL, D = 3 * PL, E = 4 * PL;
    issue_w(0, A);
    issue_x(0, B);
    issue_w(1, Cc);
    issue_x(1, D);
    load_info();
    stage_barrier<C::XL + C::WL>();
#pragma unroll
    for (int mt = 0; mt < C::MT; ++mt) xa[mt] = *(const u32x4 *)(lds + B + xrow + mt * 16 * C::KB + s0);
#pragma unroll
    for (int nt = 0; nt < C::NT; ++nt) wa[nt] = *(const u32x4 *)(lds + A + wrow0 + wtile(nt) + s0);
    auto round = [&](int r, bool fast) {
      const uint32_t soff = (uint32_t)((r + 2) * C::KB);
      if (!fast) issue_w(r + 2, E);
#pragma unroll
      for (int i = 0; i < SLOTS; ++i) {
        if (i < C::MT) xb[i] = *(const u32x4 *)(lds + B + xrow + i * 16 * C::KB + s1);
        else wb[i - C::MT] = *(const u32x4 *)(lds + A + wrow0 + wtile(i - C::MT) + s1);
        if (fast && (i & 1) == 0) dma16(rw, woff[i / 2], soff, lds_base + E + (uint32_t)wload(i / 2) * 1024);
#pragma unroll
        for (int k = i * PER; k < (i + 1) * PER; ++k) mma_acc(wa[k / C::MT], xa[k % C::MT], acc[k / C::MT][k % C::MT]);
        __builtin_amdgcn_sched_barrier(0);
      }
      stage_barrier<C::WL>();  // stage r + 1 is there, w(r + 2) may still be on its way
      if (!fast) issue_x(r + 2, A);
#pragma unroll
      for (int i = 0; i < SLOTS; ++i) {
        if (i < C::MT) xa[i] = *(const u32x4 *)(lds + D + xrow + i * 16 * C::KB + s0);
        else wa[i - C::MT] = *(const u32x4 *)(lds + Cc + wrow0 + wtile(i - C::MT) + s0);
        if (fast && (i & 1) == 0) dma16(rx, xoff[i / 2], soff, lds_base + A + (uint32_t)w * 1024 + i / 2 * C::NW * 1024);
#pragma unroll
        for (int k = i * PER; k < (i + 1) * PER; ++k) mma_acc(wb[k / C::MT], xb[k % C::MT], acc[k / C::MT][k % C::MT]);
        __builtin_amdgcn_sched_barrier(0);
      }
      const uint32_t a = A, b = B;
      A = Cc;
      B = D;
      Cc = E;
      D = a;
      E = b;
    };
    int r = 0;
    for (; r + 2 < full; ++r) round(r, true);
    for (; r < rounds; ++r) round(r, false);
    mma_drain();
  } else {
    // Blocks start at different places along k (a ring): rows of W are a power of
    // two apart or near it, and blocks in step would all read the same few
    // channels of HBM.  Few rows: 32 places within an XCD (x is small and stays
    // in L2; 5.8 -> 6.3 TB/s of W at 16 rows).  128 rows: one place per XCD, so
    // that its blocks share each stage of x (221 -> 207 us for the 0.86 GB of a
    // whole layer).
    const int r0 = C::RT >= 128 ? (int)(((local & 7) * rounds) >> 3) : (int)((((local >> 3) & 31) * rounds) >> 5);
    auto stage_of = [&](int r) { return r >= rounds ? rounds : r + r0 >= rounds ? r + r0 - rounds : r + r0; };
    uint32_t put = 0, get = 0;  // ring positions of the next stage to load and to use
#pragma unroll
    for (int s = 0; s < C::S - 1; ++s) {
      issue(stage_of(s), put);
      put += C::STAGE;
    }
    load_info();
    auto wait_stage = [&]() { stage_barrier<(C::S - 2) * (C::XL + C::WL)>(); };
    auto take_stage = [&]() {  // its place in LDS
      const uint8_t *buf = lds + get;
      get = get + C::STAGE == C::S * C::STAGE ? 0 : get + C::STAGE;
      return buf;
    };
    auto refill = [&](int r) {  // the loads of a later stage, to the place of the one before r
      issue(stage_of(r + C::S - 1), put);
      put = put + C::STAGE == C::S * C::STAGE ? 0 : put + C::STAGE;
    };
    if constexpr (C::Q4) {
      // A wave multiplies CH steps of 32 inputs that share their scales, then adds
      // the products to the sums with them: s * (sum_k ((24 + q) / 16) x - 24/16
      // sum_k x), each product exact, the scale in fp32.  CH is as long as the group
      // and the wave's part of a stage allow, or one step, so that a group's sum
      // meets its scale in one part or two.
      const u32x4 less = u32x4{kQ4Less, kQ4Less, kQ4Less, kQ4Less};
      int now = -1, s_get = 0;  // the batch of scales in use and its place
      auto scales_of = [&](int stage) {
        if (batch_of(stage) != now) {
          if (now >= 0) s_get = s_get + C::SBYTES == C::S * C::SBYTES ? 0 : s_get + C::SBYTES;
          now = batch_of(stage);
        }
        return lds + C::S * C::STAGE + s_get + (g * 4 + wcol) * C::SG * 4;
      };
      auto read_x = [&](const uint8_t *buf, int i, int mt) {
        return *(const u32x4 *)(buf + xrow + mt * 16 * C::KB + ((((wk * KS + i) * 4 + g) ^ (xin & C::SWZ)) * 16));
      };
      auto read_w = [&](const uint8_t *buf, int i, int nt) {
        return *(const uint32_t *)(buf + wrow + wtile(nt) + ((wk * KS + i) ^ (r_in & C::WSWZ)) * 16 + g * 4);
      };
      // steps c * CH .. of the stage in buf
      auto multiply = [&](auto chain, int c, int stage, const uint8_t *scales, const uint8_t *buf) {
        constexpr int CH = decltype(chain)::value;
        const int grp = ((stage * (C::KB / 2) + (wk * KS + c * CH) * 32) >> glog) & (C::SG - 1);
        const uint8_t *sc_at = scales + ((grp ^ g) * 16);
        u32x4 xo[CH][C::MT];
        f32x4_t start[C::MT];
#pragma unroll
        for (int mt = 0; mt < C::MT; ++mt) {
          start[mt] = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int i = 0; i < CH; ++i) {
            xo[i][mt] = pairs_apart(read_x(buf, c * CH + i, mt));
            start[mt] = mma(less, xo[i][mt], start[mt]);
          }
        }
#pragma unroll
        for (int nt = 0; nt < C::NT; ++nt) {
          const f32x4_t sc = *(const f32x4_t *)(sc_at + wtile(nt) / C::WKB * C::SG * 4);
          u32x4 wo[CH];
#pragma unroll
          for (int i = 0; i < CH; ++i) wo[i] = q4x8_shifted(read_w(buf, c * CH + i, nt));
#pragma unroll
          for (int mt = 0; mt < C::MT; ++mt) {
            f32x4_t p = start[mt];
#pragma unroll
            for (int i = 0; i < CH; ++i) p = mma(wo[i], xo[i][mt], p);
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[nt][mt][i] = fmaf(p[i], sc[i], acc[nt][mt][i]);
          }
        }
      };
      auto product = [&](auto chain) {
        constexpr int CH = decltype(chain)::value;
        for (int r = 0; r < rounds; ++r) {
          wait_stage();
          refill(r);
          const uint8_t *buf = take_stage();
          const int stage = stage_of(r);
          const uint8_t *scales = scales_of(stage);
#pragma unroll
          for (int c = 0; c < KS / CH; ++c) multiply(chain, c, stage, scales, buf);
        }
      };
      constexpr int CH = KS < 4 ? KS : 4;
      if ((32 * CH) >> glog <= 1) product(std::integral_constant<int, CH>{});
      else product(std::integral_constant<int, 1>{});
#pragma unroll
      for (int nt = 0; nt < C::NT; ++nt)
#pragma unroll
        for (int mt = 0; mt < C::MT; ++mt) acc[nt][mt] *= 16.f;
    } else for (int r = 0; r < rounds; ++r) {
      wait_stage();
      refill(r);
      const uint8_t *buf = take_stage();
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        const int slot16 = (((wk * KS + ks) * 4 + g) ^ (r_in & C::SWZ)) * 16;
        u32x4 xo[C::MT], wo[C::NT];
#pragma unroll
        for (int mt = 0; mt < C::MT; ++mt) xo[mt] = *(const u32x4 *)(buf + xrow + mt * 16 * C::KB + slot16);
#pragma unroll
        for (int nt = 0; nt < C::NT; ++nt) wo[nt] = *(const u32x4 *)(buf + wrow + wtile(nt) + slot16);
#pragma unroll
        for (int nt = 0; nt < C::NT; ++nt)
#pragma unroll
          for (int mt = 0; mt < C::MT; ++mt) acc[nt][mt] = mma(wo[nt], xo[mt], acc[nt][mt]);
      }
    }
  }
  stage_barrier<0>();  // nothing in flight to LDS any more, and every wave is done with it

  // ---- sums of the k waves; the rows' descriptions
  int et0 = 0;  // first column tile this wave finishes
  acc_t fin[C::FIN][C::MT];
  // adapters of the rows whose B is under way (more registers for four rows: 57 -> 73 us of a token's gate and up)
  constexpr int EA = !EARLY ? 1 : C::RT < 16 ? 2 : KT == 1 ? 8 : 4;
  BFrag<C::DT, DELTA ? KT : 1> ebf[C::GATED ? 2 : 1][EA];
  DeltaRows erows[C::GATED ? 2 : 1];
  (void)ebf;
  (void)erows;
  RowInfo *info = reinterpret_cast<RowInfo *>(lds + C::RED);
  if constexpr (C::Q4 || C::GATED) {
    const uint32_t none = 0xffffffffu;
    u32x4 *put = reinterpret_cast<u32x4 *>(info);
    if (t < C::IR) {
#pragma unroll
      for (int k = 0; k < (C::GATED && DELTA ? 2 : 1); ++k) {
        u32x4 lo = u32x4{0u, 0u, none, 0u}, hi = u32x4{0u, 0u, 0u, none};  // no row, no adapter, rank 0
        if constexpr (GROUPED) {
          hi.w = t < rows && (unsigned)prow < (unsigned)d.num_rows ? (uint32_t)prow : none;
        } else if (t < rows) {
          lo = desc[k][0];
          hi = desc[k][1];
        }
        put[(k * C::IR + t) * 2] = lo;
        put[(k * C::IR + t) * 2 + 1] = hi;
      }
    }
  } else if (t < C::RT) {
    if constexpr (C::I8) {
      mine.xe = (int16_t)__builtin_amdgcn_frexp_expf(mine.xs);
      mine.xs = __builtin_amdgcn_frexp_mantf(mine.xs) / 127.f;
    }
    info[t] = mine;
  }
  if constexpr (C::WK > 1) {
    acc_t *red = reinterpret_cast<acc_t *>(lds);
    const int grp = w % (C::WR * C::WC);
#pragma unroll
    for (int nt = 0; nt < C::NT; ++nt)
#pragma unroll
      for (int mt = 0; mt < C::MT; ++mt)
        red[(((wk * C::WR * C::WC + grp) * C::NT + nt) * C::MT + mt) * 64 + lane] = acc[nt][mt];
    __syncthreads();
    et0 = wk * C::NTE;
    if (et0 >= (C::GATED ? C::NT / 2 : C::NT)) return;
    if constexpr (EARLY) {
      const int nw0 = n0 + (wc * (C::GATED ? C::NT / 2 : C::NT) + et0) * 16;
#pragma unroll
      for (int k = 0; k < (C::GATED ? 2 : 1); ++k) {
        const RowInfo ri = info[k * C::IR + r_in];
        erows[k] = delta_rows(ri);
        begin_delta(m, ri, nw0, erows[k], ebf[k]);
      }
    }
#pragma unroll
    for (int e = 0; e < C::FIN; ++e)
#pragma unroll
      for (int mt = 0; mt < C::MT; ++mt) {
        const int nt = et0 + (e >= C::NTE ? C::NT / 2 + e - C::NTE : e);
        acc_t s = acc_t{0, 0, 0, 0};
#pragma unroll
        for (int k = 0; k < C::WK; ++k)
          s += red[(((k * C::WR * C::WC + grp) * C::NT + nt) * C::MT + mt) * 64 + lane];
        fin[e][mt] = s;
      }
  } else {
    __syncthreads();
#pragma unroll
    for (int e = 0; e < C::FIN; ++e)
#pragma unroll
      for (int mt = 0; mt < C::MT; ++mt) fin[e][mt] = acc[e][mt];
  }

  // ---- scales, delta, rounding, store: DT column tiles at a time
  // int8: (sum * s) * Ws with the power of two of s apart and last.  With it a
  // finite result may pass the ends of fp32 on the way (a sum of 2^31 times a row
  // scale of 2^121, a scale of 2^-140); without it sum * s lies between 2^-8 and
  // 2^24, and the three roundings are the same.  The output's power of two apart
  // as well cost the prefills 2.5% (4465 -> 4575 us).
  uint8_t *yw = lds + C::RED + C::INFO + w * C::YWAVE;
  (void)yw;
  constexpr int WNT = C::GATED ? C::NT / 2 : C::NT;  // column tiles of a wave's output
  // v of a row's adapter, scaled, in bf16 pieces
  constexpr int VP = C::I8 ? 2 : 3;
  typedef VPieces<VP> v_t;
  auto scale_v = [&](const f32x4_t (&raw)[DELTA ? KT : 1][2], const RowInfo &ri, v_t *v) {
#pragma unroll
    for (int ks = 0; ks < (DELTA ? KT : 1); ++ks) {
      float vv[8];
      const int j0 = ks * 32 + g * 8;
#pragma unroll
      for (int i = 0; i < 8; ++i) vv[i] = j0 + i < ri.rank ? raw[ks][i / 4][i % 4] * ri.scale : 0.f;
      v[ks] = split_v<VP>(vv);
    }
  };
  typedef f32x4_t raw_t[DELTA ? KT : 1][2];
  auto ask_v = [&](const float *row, const RowInfo &ri, raw_t &raw) {
    const float *src = row + g * 8;
#pragma unroll
    for (int ks = 0; ks < (DELTA ? KT : 1); ++ks) {
      const bool von = ks * 32 + g * 8 < ri.rank;
      raw[ks][0] = von ? *(const f32x4_t *)(src + ks * 32) : f32x4_t{0.f, 0.f, 0.f, 0.f};
      raw[ks][1] = von ? *(const f32x4_t *)(src + ks * 32 + 4) : f32x4_t{0.f, 0.f, 0.f, 0.f};
    }
  };
  auto load_v = [&](const float *row, const RowInfo &ri, v_t *v) {
    raw_t raw;
    ask_v(row, ri, raw);
    scale_v(raw, ri, v);
  };
  // DT column tiles of a row, packed and stored (TURN: put into LDS)
  auto put_out = [&](int mt, int e0, int nw0, int b, const f32x4_t *out) {
    if constexpr (C::TURN) {
      uint8_t *at = yw + (mt * 16 + r_in) * C::YROW + e0 * 32 + g * 8;
#pragma unroll
      for (int e = 0; e < C::DT; ++e)
        *(u32x2 *)(at + e * 32) = pack_out<C>(out[e]);
    } else if (b >= 0) {
      uint16_t *y = m.y + (int64_t)b * m.ldy;
#pragma unroll
      for (int e = 0; e < C::DT; ++e) {
        const int n = nw0 + e * 16 + g * 4;
        if (n < m.d_out)
          *(u32x2 *)(y + n) = pack_out<C>(out[e]);
      }
    }
  };
  if constexpr (C::GATED) {
    const GemmModule &up = gemm_desc().mod[1];
#pragma unroll
    for (int e0 = 0; e0 < C::NTE; e0 += C::DT) {
      const int nw0 = n0 + (wc * WNT + et0 + e0) * 16;
      // (with four of rank 64 the 128-row tile spills 14 registers: 128 rows over as many adapters 455 us, 415 with three)
      constexpr int AH = C::RT == 128 && KT == 2 ? 3 : C::AHEAD;
      BFrag<C::DT, DELTA ? KT : 1> bg[AH], bu[AH];
      (void)bg;
      (void)bu;
#pragma unroll
      for (int mt = 0; mt < C::MT; ++mt) {
        const int r = (wr * C::MT + mt) * 16 + r_in;
        const RowInfo ri = info[r];
        f32x4_t out[C::DT], by[C::DT];
#pragma unroll
        for (int e = 0; e < C::DT; ++e) {
          out[e] = fin[e0 + e][mt];
          by[e] = fin[C::NTE + e0 + e][mt];
        }
        if constexpr (DELTA) {
          v_t v[KT];
          const RowInfo ru = info[C::IR + r];
          if constexpr (EARLY) {
            scale_v(vraw[0], ri, v);
            finish_delta(m, ri, v, nw0, erows[0], ebf[0], out);
            scale_v(vraw[1], ru, v);
            finish_delta(m, ru, v, nw0, erows[1], ebf[1], by);
          } else if constexpr (C::AHEAD == 1) {
            load_v(m.v + (int64_t)(row0 + r) * d.rs, ri, v);
            add_delta(m, ri, v, nw0, bg, out);
            load_v(up.v + (int64_t)(row0 + r) * d.rs, ru, v);
            add_delta(m, ru, v, nw0, bu, by);
          } else {  // both projections' B under way at once
            DeltaRows rg = delta_rows(ri), rup = delta_rows(ru);
            raw_t raw;  // up's v: in pieces when gate's are done with (fewer registers)
            load_v(m.v + (int64_t)(row0 + r) * d.rs, ri, v);
            ask_v(up.v + (int64_t)(row0 + r) * d.rs, ru, raw);
            begin_delta(m, ri, nw0, rg, bg);
            begin_delta(m, ru, nw0, rup, bu);
            finish_delta(m, ri, v, nw0, rg, bg, out);
            scale_v(raw, ru, v);
            finish_delta(m, ru, v, nw0, rup, bu, by);
          }
        }
#pragma unroll
        for (int e = 0; e < C::DT; ++e)
#pragma unroll
          for (int i = 0; i < 4; ++i) out[e][i] = gate_act(out[e][i], d.act_c1, d.act_c3) * by[e][i];
        put_out(mt, e0, nw0, ri.b, out);
      }
    }
  } else {
#pragma unroll
    for (int e0 = 0; e0 < C::NTE; e0 += C::DT) {
      const int nw0 = n0 + (wc * C::NT + et0 + e0) * 16;  // first column
      f32x4_t sw[C::DT];
      if constexpr (C::I8) {
#pragma unroll
        for (int e = 0; e < C::DT; ++e) {
          const int n = nw0 + e * 16 + g * 4;
          sw[e] = n < m.d_out ? *(const f32x4_t *)(Ws + n) : f32x4_t{0.f, 0.f, 0.f, 0.f};
        }
      }
      BFrag<C::DT, DELTA ? KT : 1> bf[C::AHEAD];
      (void)bf;
#pragma unroll
      for (int mt = 0; mt < C::MT; ++mt) {
        const int r = (wr * C::MT + mt) * 16 + r_in;
        const RowInfo ri = info[r];
        f32x4_t out[C::DT];
#pragma unroll
        for (int e = 0; e < C::DT; ++e) {
          if constexpr (C::I8) {
#pragma unroll
            for (int i = 0; i < 4; ++i) out[e][i] = ldexpf((float)fin[e0 + e][mt][i] * ri.xs * sw[e][i], ri.xe);
          } else {
            out[e] = fin[e0 + e][mt];
          }
        }
        if constexpr (DELTA) {
          v_t v[KT];
          if constexpr (EARLY) {
            scale_v(vraw[0], ri, v);
            finish_delta(m, ri, v, nw0, erows[0], ebf[0], out);
          } else {
            load_v(m.v + (int64_t)(C::Q4 ? row0 + r : ri.b) * d.rs, ri, v);
            add_delta(m, ri, v, nw0, bf, out);
          }
        }
        put_out(mt, e0, nw0, ri.b, out);
      }
    }
  }
  if constexpr (C::TURN) {  // the wave's own rows of LDS: no barrier
    constexpr int PPR = C::NTE * 2, STEPS = C::MT * 16 * PPR / 64;  // 16-byte pieces of a row; stores
    const int nw0 = n0 + (wc * WNT + et0) * 16;
#pragma unroll 4
    for (int i = 0; i < STEPS; ++i) {
      const int at = i * 64 + lane, lr = at / PPR, piece = at % PPR;
      const int b = info[wr * C::MT * 16 + lr].b, n = nw0 + piece * 8;
      const u32x4 v = *(const u32x4 *)(yw + lr * C::YROW + piece * 16);
      if (b >= 0 && n < m.d_out) *(u32x4 *)(m.y + (int64_t)b * m.ldy + n) = v;
    }
  }
}

// Rows of x as int8 with one scale each: s = max|x| / 127, q = rint(127 x /
// max|x|), halves to even; what is kept of s is max|x| (the division, by the
// product, is of its significand: s itself may be below the normal numbers).  A
// zero row: q = 0, s = 0.  A row with an infinity or a NaN: NaN for max|x| (its
// outputs are NaN), q = 0.  [d_in, pitch) gets 0.  36534 rows of 8192, two
// inputs: 1.8 GB in 300 us, 6 TB/s.
constexpr int kQuantRegs = 4;
__device__ __forceinline__ float abs_max8(u32x4 p, float m, bool *bad) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float a = fabsf(bf16_lo(p[i])), b = fabsf(bf16_hi(p[i]));
    *bad |= !(a <= 3.4e38f) || !(b <= 3.4e38f);
    m = fmaxf(m, fmaxf(a, b));
  }
  return m;
}
// rint(127 x / amax) for 8 values without a division each: x scaled by amax's
// power of two, times 127 over the rest of amax (one division a row), is within
// 2 units of the last place of the real quotient.  With significands of 8 bits,
// X 2^-k of x beside a of amax, the quotient is
// |254 X - (2j + 1) a 2^k| / (2 a 2^k) from the tie j + 1/2: on it, or at least
// 1 / (510 * 2^k) away, 2^8 units of a quotient below 128 / 2^k (the nearest is
// X = 254 beside a = 255).  Rounded to a multiple of 64 units it is exact on a
// tie and stays on its side otherwise.
struct QuantScale {
  int exp;
  float r;
};
__device__ __forceinline__ QuantScale quant_scale(float amax) {
  int e;
  const float f = frexpf(amax, &e);
  return QuantScale{-e, 127.f / f};
}
__device__ __forceinline__ u32x2 quant8(u32x4 p, QuantScale qs) {
  uint32_t o[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint32_t v = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t u = p[h * 2 + i / 2];
      const float f = (i & 1) ? bf16_hi(u) : bf16_lo(u);
      const uint32_t near = (__float_as_uint(ldexpf(f, qs.exp) * qs.r) + 32u) & ~63u;
      v |= ((uint32_t)(int)rintf(__uint_as_float(near)) & 0xffu) << (8 * i);
    }
    o[h] = v;
  }
  return u32x2{o[0], o[1]};
}

// The slot up to which rows have their delta: segments come in ascending slot
// order; later slots were dropped by the build, or their segments do not fit the
// batch.
__device__ __forceinline__ int last_slot(const LayerDesc &d) {
  const int nseg = fitting_segments(d.num_segments, d.max_seg, d.seg_offsets, d.num_rows);
  return nseg > 0 ? d.seg_adapter[nseg - 1] : -1;
}
__device__ __forceinline__ bool has_segment(const LayerDesc &d, int a, int last) {
  return (unsigned)a < (unsigned)d.num_slots && a <= last;
}

// The batch's rows by slot, put(place, row): first those of the segments, as the
// build sorted them, then the rows whose id has no segment (base only, bad, dropped
// past the caller's bound) in their own order.  A block of 256 places as many of
// each; it counts the rows without a segment before its own from the ids.  Places
// that no row takes (ids other than those that the segments were built from) hold
// row -1.
template <typename F>
__device__ __forceinline__ void by_slot_block(const LayerDesc &d, const int32_t *ids, int block, F put) {
  __shared__ int wsum[4];
  const int t = threadIdx.x, lane = t & 63, w = wave_id();
  const int nseg = fitting_segments(d.num_segments, d.max_seg, d.seg_offsets, d.num_rows);
  const int nvalid = nseg > 0 ? min(max(d.seg_offsets[nseg], 0), d.num_rows) : 0;
  const int last = nseg > 0 ? d.seg_adapter[nseg - 1] : -1;
  const int b = block * 256 + t;
  if (b < nvalid) put(b, d.perm[b]);
  int before = 0;
#pragma unroll 8
  for (int i = t; i < block * 256; i += 256) before += !has_segment(d, ids[i], last);
  const uint64_t mine = __ballot(b < d.num_rows && !has_segment(d, ids[min(b, d.num_rows - 1)], last));
#pragma unroll
  for (int k = 32; k >= 1; k /= 2) before += __shfl_xor(before, k, 64);
  if (lane == 0) wsum[w] = before;
  __syncthreads();
  int base = wsum[0] + wsum[1] + wsum[2] + wsum[3];
  __syncthreads();
  if (lane == 0) wsum[w] = __popcll(mine);
  __syncthreads();
  const int end = nvalid + base + wsum[0] + wsum[1] + wsum[2] + wsum[3];
  for (int k = 0; k < w; ++k) base += wsum[k];
  const int at = nvalid + base + __popcll(mine & ((1ull << lane) - 1));
  if ((mine >> lane & 1) && at < d.num_rows) put(at, b);
  if (block == (d.num_rows + 255) / 256 - 1)
    for (int p = end + t; p < d.num_rows; p += 256) put(p, -1);
}
__device__ __forceinline__ void order_block(const LayerDesc &d, const int32_t *ids, int32_t *order, int block) {
  by_slot_block(d, ids, block, [&](int place, int b) { order[place] = b; });
}

// `lanes` threads (a wave, or a block of 256) quantise one row, keeping REGS
// pieces of 8 values each in registers; longer rows are read again.
template <int LANES, int REGS, typename MAX>
__device__ __forceinline__ void quantize_row(const QuantInput &in, int row, int t, MAX row_max) {
  const uint16_t *x = in.x + (int64_t)row * in.ldx;
  const int n8 = in.d_in / 8;  // pieces of 8 values
  u32x4 keep[REGS];
  float mx = 0.f;
  bool bad = false;
#pragma unroll
  for (int i = 0; i < REGS; ++i) {
    const int p = i * LANES + t;
    keep[i] = p < n8 ? *(const u32x4 *)(x + (int64_t)p * 8) : zero4();
  }
#pragma unroll
  for (int i = 0; i < REGS; ++i) mx = abs_max8(keep[i], mx, &bad);
  for (int p = REGS * LANES + t; p < n8; p += LANES) mx = abs_max8(*(const u32x4 *)(x + (int64_t)p * 8), mx, &bad);
  row_max(&mx, &bad);
  const bool live = mx > 0.f && !bad;
  const QuantScale qs = quant_scale(live ? mx : 1.f);
  int8_t *q = in.q + (int64_t)row * in.pitch;
#pragma unroll
  for (int i = 0; i < REGS; ++i) {
    const int p = i * LANES + t;
    if (p < n8) *(u32x2 *)(q + (int64_t)p * 8) = live ? quant8(keep[i], qs) : u32x2{0u, 0u};
  }
  for (int p = REGS * LANES + t; p < n8; p += LANES)
    *(u32x2 *)(q + (int64_t)p * 8) = live ? quant8(*(const u32x4 *)(x + (int64_t)p * 8), qs) : u32x2{0u, 0u};
  if (t == 0) {
    if (in.d_in < in.pitch) *(u32x2 *)(q + in.d_in) = u32x2{0u, 0u};  // the row's last half piece
    in.amax[row] = bad ? __int_as_float(0x7fc00000) : mx;
  }
}

// One block's rows of a call's inputs; q0 is qd where it lies in the kernel's
// arguments.  A row of up to kQuantWaveMax values takes one wave (4247 rows of
// 600: a block each is 4 times the dispatches), a longer one the block.
__device__ __forceinline__ void quantize_block(const QuantDesc &qd, const QuantDesc &q0, int block) {
  __shared__ float red[4];
  __shared__ int badv[4];
  int k = 0;
#pragma unroll
  for (int i = 1; i < kMaxModules; ++i)
    if (i < qd.n && block >= qd.in[i].block_base) k = i;
  const QuantInput in = q0.in[k];
  const int t = threadIdx.x, lane = t & 63, w = wave_id();
  auto wave_max = [&](float *mx, bool *bad) {
#pragma unroll
    for (int i = 32; i >= 1; i /= 2) *mx = fmaxf(*mx, __shfl_xor(*mx, i, 64));
    *bad = __ballot(*bad) != 0;
  };
  if (in.rows_per_block == 4) {
    const int row = (block - in.block_base) * 4 + w;
    if (row < in.rows) quantize_row<64, kQuantRegs>(in, row, lane, wave_max);
    return;
  }
  quantize_row<256, kQuantRegs>(in, block - in.block_base, t, [&](float *mx, bool *bad) {
    wave_max(mx, bad);
    if (lane == 0) {
      red[w] = *mx;
      badv[w] = *bad;
    }
    __syncthreads();
    *mx = fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
    *bad = badv[0] | badv[1] | badv[2] | badv[3];
  });
}

}  // namespace lora
