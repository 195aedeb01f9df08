// attn_tree_tc.cuh -- the tensor core kernel of moe_attn_tree as its host side
// sees it.
#pragma once
#include "attn_tree.cuh"

namespace moe {

constexpr int kTcThreads = 256;
constexpr int kTcShared = 1024;  // bytes beside the tiles

template <int DP>
struct TcCfg {
  static constexpr int ROWS = 128;
  static constexpr int TILE = 64;
  static constexpr int CTAS = DP == 256 ? 1 : 2;  // per SM
  static constexpr int END = 10;                   // what a unit's end costs, in tiles
};

// bf16 and e4m3 caches; ctas of a single wave
cudaError_t launch_tree_tc(int kv, int dp, const TreeArgs& a, int ctas, cudaStream_t st);

}  // namespace moe
