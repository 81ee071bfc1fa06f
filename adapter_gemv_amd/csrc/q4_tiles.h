// Tiles of the products with 4-bit weights and group scales (gemm_items.h).
#pragma once

#include "gemm_items.h"

namespace lora {

//                                                    I8     RT   NC  WR WC WK  KB  S EU  PIPE   Q4
template <bool GATED> using Q4Cfg4n = GemmCfg<false, 4, 32, 1, 1, 4, 1024, 3, 2, false, true, GATED>;
template <bool GATED> using Q4Cfg4 = GemmCfg<false, 4, 64, 1, 1, 4, 1024, 3, 2, false, true, GATED>;
template <bool GATED> using Q4Cfg16n = GemmCfg<false, 16, 32, 1, 1, 4, 512, 4, 2, false, true, GATED>;
template <bool GATED> using Q4Cfg16 = GemmCfg<false, 16, 64, 1, 1, 4, 512, 3, 2, false, true, GATED>;
template <bool GATED> using Q4Cfg32 = GemmCfg<false, 32, 64, 1, 1, 4, 512, 3, 2, false, true, GATED>;
template <bool GATED> using Q4Cfg64 = GemmCfg<false, 64, 64, 2, 2, 1, 256, 3, 2, false, true, GATED>;
template <bool GATED> using Q4Cfg128 = GemmCfg<false, 128, 128, 2, 2, 1, 128, 3, 2, false, true, GATED>;
template <bool GATED> using Q4Cfg256 = GemmCfg<false, 256, 128, 2, 2, 1, 128, 3, 1, false, true, GATED>;
constexpr int kQ4Tiles = 8;

// f(the tile's type) of tile cfg.
template <bool GATED, typename F>
auto with_q4_tile(int cfg, F f) {
  switch (cfg) {
    case 0: return f(Q4Cfg4n<GATED>{});
    case 1: return f(Q4Cfg4<GATED>{});
    case 2: return f(Q4Cfg16n<GATED>{});
    case 3: return f(Q4Cfg16<GATED>{});
    case 4: return f(Q4Cfg32<GATED>{});
    case 5: return f(Q4Cfg64<GATED>{});
    case 6: return f(Q4Cfg128<GATED>{});
    default: return f(Q4Cfg256<GATED>{});
  }
}

}  // namespace lora
