// Internal launchers of the 16-bit operators: rows grouped by expert times bf16 or
// f16 weights, the gradients of that product, and low-rank adapters.
#pragma once

#include "common.cuh"

// out[r, m] = sum_k A[r, k] * W[e(r), m, k] (GG_W_K, GG_W_M: how W is stored), or
// out[e, m, n] = sum over e's rows r of Y[r, m] * A[r, n] (GG_ROWS).
enum GgForm {
  GG_W_K = 0,   // W [E][M][K], k contiguous
  GG_W_M = 1,   // W [E][K][M], m contiguous
  GG_ROWS = 2,  // the contraction runs over an expert's rows
};
struct GgGemm {
  GgForm form;
  bool bf16;              // else f16
  const void* w;          // weights; GG_ROWS: Y [R][M]
  int64_t w_stride;       // elements between W's rows (of m, or of k); GG_ROWS: Y's rows
  int64_t w_expert;       // elements between experts
  const void* a;          // rows
  int64_t a_stride;       // elements between rows
  int64_t R;
  int E;
  int M;                  // outputs of a row; GG_ROWS: rows of an expert's result
  int N;                  // GG_ROWS: columns of an expert's result
  int K;                  // contraction of GG_W_K and GG_W_M
  const int32_t* offsets; // first row of each expert, and the last one's end (null: one expert)
  void* out;              // [R][M]; GG_ROWS: [E][M][N]
  int out_dtype;
  bool zero_outside;      // rows of no expert get zeros (else they are left as they are)
  float* part;            // float32 partial sums [split] of out's shape, where split
  unsigned* status;
};
constexpr int kFewRows = 16;  // rows at most of the product that takes one launch (GG_W_K)
struct GgPlan {
  bool few;    // at most kFewRows rows: one launch of gg_few
  int bn;      // columns per tile: rows of A, or GG_ROWS columns of the result
  bool pair;   // CTA pairs (cta_group::2), else single CTAs
  int splits;  // splits of the contraction
};
MQ_HIDDEN GgPlan gg_plan(GgForm form, int64_t R, int E, int M, int N, int K);
MQ_HIDDEN cudaError_t launch_gg(const GgGemm& g, const GgPlan& pl, cudaStream_t st);
MQ_HIDDEN cudaError_t launch_gg_few(const GgGemm& g, cudaStream_t st);
// Both gradients of a product in one launch, and whether that is the better way.
MQ_HIDDEN bool gg_side_by_side(const GgGemm& rows, const GgGemm& weights);
MQ_HIDDEN cudaError_t launch_gg_both(const GgGemm& rows, const GgGemm& weights, cudaStream_t st);
