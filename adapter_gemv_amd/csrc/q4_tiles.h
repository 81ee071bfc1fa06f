// Tiles of the products with 4-bit weights and group scales (gemm_items.h).
#pragma once

#include "gemm_items.h"

namespace lora {

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
