// Tiles of the products with 4-bit weights and group scales (gemm_items.h).
#pragma once

#include "gemm_items.h"

namespace lora {

// x is bf16, so that a tile of few columns moves as much x as W: wide tiles where
// W is wide, 4 rows of x where there are no more.  A wave splits k with three or
// seven others up to 32 rows.  Measured on one MI355X, us of a pass (in brackets what
// the rule of pick_gemm takes):
//  * one row, gate and up of 8192 x 28672: 4 x 32 60, 4 x 64 [57], 16 x 64 59;
//    q/k/v/o: [28], 38, 39; with 3 stages (fewer blocks a unit) 64, 4 x 64 on 1024
//    bytes 65.
//  * 32 slots x 4 rows of 8192 x 8192: 16 x 64 209, 16 x 128 [211], 4 x 64 255;
//    16 x 64 with 3 stages 235.  16 rows, gate and up: 16 x 128 [66], 16 x 64 83.
//  * 8 slots x 16 rows, gate and up: 32 x 128 with k by four waves [421], columns and
//    k by two 434 to 469, columns by four 478; 16 x 128 477, 16 x 64 484; 64 rows 605.
//  * 1024 rows, gate and up of 4096 x 8192: 64 x 256 218, 256 x 256 [182], 32 x 128 269;
//    5592 rows of 8192 x 28672: 256 x 256 [5850] (0.9 PFLOP/s; in groups of 32 6914),
//    64 x 256 7086, 256 x 256 on waves of 128 x 64 9047, 256 x 128 on four waves
//    8158.  128 x 128 stays within 3% of 64 x 256 everywhere: not kept.
//  * Registers: 256 x 256 spills, around its epilogue, 4 with adapters of rank up to
//    32 (gated), 8 and 10 above; the others fit.
//  * few blocks (4d, 16d): 8 waves on long stages, see pick_gemm.
//                                                    I8     RT   NC  WR WC WK  KB  S EU  PIPE   Q4
template <bool GATED> using Q4Cfg4n = GemmCfg<false, 4, 32, 1, 1, 4, 1024, 2, 2, false, true, GATED>;
template <bool GATED> using Q4Cfg4d = GemmCfg<false, 4, 32, 1, 1, 8, 2048, 3, 2, false, true, GATED>;
template <bool GATED> using Q4Cfg4 = GemmCfg<false, 4, 64, 1, 1, 4, 512, 2, 2, false, true, GATED>;
template <bool GATED> using Q4Cfg16d = GemmCfg<false, 16, 32, 1, 1, 8, 1024, 3, 2, false, true, GATED>;
template <bool GATED> using Q4Cfg16 = GemmCfg<false, 16, 64, 1, 1, 4, 512, 2, 2, false, true, GATED>;
template <bool GATED> using Q4Cfg16w = GemmCfg<false, 16, 128, 1, 1, 4, 512, 2, 2, false, true, GATED>;
template <bool GATED> using Q4Cfg32 = GemmCfg<false, 32, 128, 1, 1, 4, 512, 2, 2, false, true, GATED>;
template <bool GATED> using Q4Cfg64 = GemmCfg<false, 64, 256, 1, 4, 1, 128, 2, 2, false, true, GATED>;
template <bool GATED> using Q4Cfg256 = GemmCfg<false, 256, 256, 4, 2, 1, 128, 2, 2, false, true, GATED>;
constexpr int kQ4Tiles = 9;

// f(the tile's type) of tile cfg.
template <bool GATED, typename F>
auto with_q4_tile(int cfg, F f) {
  switch (cfg) {
    case 0: return f(Q4Cfg4n<GATED>{});
    case 1: return f(Q4Cfg4d<GATED>{});
    case 2: return f(Q4Cfg4<GATED>{});
    case 3: return f(Q4Cfg16d<GATED>{});
    case 4: return f(Q4Cfg16<GATED>{});
    case 5: return f(Q4Cfg16w<GATED>{});
    case 6: return f(Q4Cfg32<GATED>{});
    case 7: return f(Q4Cfg64<GATED>{});
    default: return f(Q4Cfg256<GATED>{});
  }
}

}  // namespace lora
