// w8a8.cuh -- the 8-bit product as its callers see it (w8a8.cu; used by api.cu and moe.cu).
#pragma once

#include "internal.h"

namespace awq {

enum W8Epilogue { kW8Store = 0, kW8SiluQuant = 1 };

// y [rows][N] = x [rows][K] . w [N][K]^T on 8-bit matrices.  Dense (groups == 0): all rows of x meet one weight.
// Grouped: w is [groups][wrows][K]; the rows of x are sorted by group, group e's are row_start[e] .. row_start[e + 1],
// and tile_start[e] counts the token tiles (of bt rows) before group e; both tables are on the device.
struct W8Args {
  const uint8_t* xc = nullptr;   // codes and scales of x
  const uint8_t* xs = nullptr;
  const uint16_t* x = nullptr;   // dense, instead of xc and xs where w8a8_quantizes(xrows): x itself, 16-bit of type xdt
  int xdt = 0;
  int xrows = 0;                 // rows of x that exist (grouped: an upper bound)
  const uint8_t* wc = nullptr;   // codes and scales of w
  const uint8_t* wsc = nullptr;
  int N = 0, K = 0;              // N: outputs (kW8SiluQuant: the channels of h; the weight has 2 N rows, gate then up)
  int groups = 0;
  const int* row_start = nullptr;
  const int* tile_start = nullptr;
  int bt = 0;                    // grouped: token tile (w8a8_grouped_bt)
  bool plan_ready = false;       // grouped: the kernel before this one on the stream has itself waited for the tables' kernel
  int epi = kW8Store;
  void* y = nullptr;             // kW8Store: [rows][N] of type dt
  int dt = 0;
  uint8_t* hc = nullptr;         // kW8SiluQuant: h = silu(gate) up as an 8-bit matrix [rows][N]
  uint8_t* hs = nullptr;
  unsigned* status = nullptr;
  cudaStream_t st = nullptr;
};
bool w8a8_quantizes(int tokens);  // whether the dense product takes `tokens` rows of 16-bit x
int w8a8_grouped_bt(long long rows, int groups, int epi);  // token tile for `rows` rows spread over `groups` groups
awq_status w8a8_launch(const W8Args& a);
awq_status fp8_quantize_launch(const void* x, int dt, int R, int K, uint8_t* codes, uint8_t* scales, cudaStream_t st,
                               bool early = false);

}  // namespace awq
