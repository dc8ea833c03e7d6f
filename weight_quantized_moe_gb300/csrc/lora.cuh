// Internal launchers of the low-rank adapters.
#pragma once

#include "common.cuh"

struct LoraArgs {
  bool bf16;                // rows and adapters; else f16
  const void* x;            // [R][K]
  int64_t x_stride;         // elements between rows
  int64_t R;
  int K, N, r, L, E;
  const void* a;            // [L][E][r][K]
  const void* b;            // [L][E][N][r]
  const int32_t* ids;       // [R]: adapter, or -1
  const int32_t* offsets;   // [E + 1], or null: one expert
  const float* scaling;     // [L], or null: 1
  const void* base;         // [R][N] in out_dtype, or null: 0
  int64_t base_stride;
  void* out;                // [R][N]; may be base
  int64_t out_stride;
  int out_dtype;
  uint8_t* workspace;       // of lora_workspace bytes, where the plan has tiles
  unsigned* status;
};
struct LoraPlan {
  bool rows;   // one cluster per row, one launch (else two launches over tiles of rows)
  int height;  // rows of a tile, a multiple of 16
  int splits;  // K splits of the first launch: CTAs of a cluster
  int mparts;  // clusters among which it divides a tile's adapters
  int gparts;  // parts of a tile's adapters in the second launch
};
MQ_HIDDEN size_t lora_workspace(const LoraPlan& pl, int64_t R, int r);
MQ_HIDDEN LoraPlan lora_plan(int64_t R, int K, int N, int r, int L, int E);
// The plan's kernels one by one (which: 0 A x, or both in one; 1 the rest).
MQ_HIDDEN cudaError_t launch_lora(const LoraArgs& g, const LoraPlan& pl, int which, cudaStream_t st);
