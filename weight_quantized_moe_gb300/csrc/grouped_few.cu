// A grouped product of a few rows: one read of the weights of the experts that have
// any, in one launch.
//
//   out[r, m] = sum_k A[r, k] * W[e(r), m, k],  R <= kFewRows, W's k contiguous
//
// A CTA has 16 outputs and all rows of one expert; its warps take an eighth of K each and
// their sums are added in shared memory, in the order of the warps.  Bound by the weights,
// which go from memory straight to registers, 16 bytes of two weight rows a lane and
// step, eight steps in flight.  The products are warp-level MMAs (m16n8k16): the sum over k
// does not care for its order, so the eight k that a lane has are the pairs of two
// instructions, for weights and rows alike, and nothing passes through shared memory.  (On
// the CUDA cores eight rows cost more than the weights: one row 8.7 us, four 13.4.)
// tcgen05 would take shared memory, tensor memory and, to read with all SMs at this size,
// a second launch for the sum of its K splits: one row, 4096 x 4096 (33.5 MB), 10.2 us
// there and 7.8 here (4.3 TB/s, of which a launch by itself takes 2 us), 16 rows 10.5 and
// 8.6; with weights of 117 MB they are equal.
#include "grouped.cuh"
#include "pipe.cuh"

#include <algorithm>

namespace {

using namespace mq::pipe;

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kOuts = 16;   // outputs of a CTA at a time
constexpr int kSteps = 8;   // steps of 32 k in flight
constexpr int kTail = 4;    // the same, at the end

template <bool BF16>
__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  if constexpr (BF16)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Elements [8 q, 8 q + 8) of a row of K, zeros behind its end.
__device__ __forceinline__ uint4 last_piece(const uint16_t* row, int q, int K) {
  uint32_t w[4] = {};
  for (int i = 0; q * 8 + i < K && i < 8; ++i) w[i >> 1] |= (uint32_t)row[q * 8 + i] << (i & 1) * 16;
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// At most D steps of 32 k from piece q of two weight rows on, for NT times eight rows, all
// in flight together.  (The tensor core's additions round towards zero: long sums are made
// of short ones.)
template <bool BF16, int NT, int D, bool WHOLE>
__device__ __forceinline__ void steps_of(float (&acc)[NT][4], const uint4* w0, const uint4* w1,
                                         const uint16_t* const (&a)[NT], const bool (&live)[NT], int q, int steps) {
  uint4 v0[D], v1[D];
#pragma unroll
  for (int d = 0; d < D; ++d) {
    v0[d] = v1[d] = make_uint4(0, 0, 0, 0);
    if (WHOLE || d < steps) {
      v0[d] = __ldcs(w0 + q + d * 4);
      v1[d] = __ldcs(w1 + q + d * 4);
    }
  }
  float c[NT][4] = {};
#pragma unroll
  for (int d = 0; d < D; ++d) {
    if (!WHOLE && d >= steps) break;
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      const uint4 x = live[j] ? __ldg(reinterpret_cast<const uint4*>(a[j]) + q + d * 4) : make_uint4(0, 0, 0, 0);
      mma16816<BF16>(c[j], v0[d].x, v1[d].x, v0[d].y, v1[d].y, x.x, x.y);
      mma16816<BF16>(c[j], v0[d].z, v1[d].z, v0[d].w, v1[d].w, x.z, x.w);
    }
  }
#pragma unroll
  for (int j = 0; j < NT; ++j)
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[j][i] += c[j][i];
}

// Grid: (outputs, experts), or (outputs, rows) where there are fewer rows: then the CTAs of
// a row that is its expert's first take all of that expert's rows.  8 NT rows at most at a
// time.  (CTAs that find nothing to do are not free: 16 rows of one expert, 512 x 4096, took
// 11.5 us with one for each row.)
template <bool BF16, int NT>
__global__ void __launch_bounds__(kThreads, 2) gg_few(const GgGemm g) {
  __shared__ int behind[kFewRows];  // experts that end at or before a row
  __shared__ float sums[kWarps][NT * 8][kOuts];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int R = (int)g.R;
  const bool by_expert = g.E <= R;
  const int row = by_expert ? 0 : blockIdx.y;
  mq::pdl_wait();
  mq::pdl_trigger();
  int e = 0, first = 0, rows = R;
  if (g.offsets) {
    if (tid < kFewRows) behind[tid] = 0;
    __syncthreads();
    bool bad = false;
    for (int i = tid; i <= g.E; i += kThreads) {
      const int o = g.offsets[i];
      bad |= o < 0 || o > R || (i < g.E && g.offsets[i + 1] < o);
      if (!by_expert && i > 0 && o >= 0)
        for (int r = o; r < R; ++r) atomicAdd(&behind[r], 1);
    }
    bad = __syncthreads_or(bad);
    if (bad) {
      if (tid == 0 && blockIdx.x == 0 && blockIdx.y == 0) mq::flag(g.status, MQ_DEV_BAD_OFFSETS);
      return;
    }
    const int lo = g.offsets[0], hi = g.offsets[g.E];
    // rows of no expert, by the first CTAs of each (all rows': of the first expert)
    if (g.zero_outside && (!by_expert || blockIdx.y == 0))
      for (int r = row; r < (by_expert ? R : row + 1); ++r)
        if (r < lo || r >= hi)
          for (int64_t m = (int64_t)blockIdx.x * kThreads + tid; m < g.M; m += (int64_t)gridDim.x * kThreads)
            store_out(g.out, g.out_dtype, (int64_t)r * g.M + m, 0.0f);
    if (!by_expert && (row < lo || row >= hi)) return;
    e = by_expert ? blockIdx.y : behind[row];
    first = g.offsets[e];
    rows = g.offsets[e + 1] - first;
    if (rows == 0 || (!by_expert && row != first)) return;
  }
  const uint16_t* we = static_cast<const uint16_t*>(g.w) + (int64_t)e * g.w_expert;
  const int gi = lane >> 2, t = lane & 3;  // of a fragment: row (column of B), pair of k
  const int steps = g.K / 32;  // whole ones
  const int s0 = (int)((int64_t)steps * warp / kWarps), s1 = (int)((int64_t)steps * (warp + 1) / kWarps);
  for (int r0 = 0; r0 < rows; r0 += NT * 8) {
    const uint16_t* a[NT];
    bool live[NT];
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      live[j] = r0 + j * 8 + gi < rows;
      a[j] = static_cast<const uint16_t*>(g.a) + (int64_t)(first + r0 + (live[j] ? j * 8 + gi : 0)) * g.a_stride;
    }
    for (int64_t m0 = (int64_t)blockIdx.x * kOuts; m0 < g.M; m0 += (int64_t)gridDim.x * kOuts) {
      const uint16_t* w0 = we + min(m0 + gi, (int64_t)g.M - 1) * g.w_stride;
      const uint16_t* w1 = we + min(m0 + gi + 8, (int64_t)g.M - 1) * g.w_stride;
      float acc[NT][4] = {};
      const uint4 *p0 = reinterpret_cast<const uint4*>(w0), *p1 = reinterpret_cast<const uint4*>(w1);
      int s = s0;
      for (; s + kSteps <= s1; s += kSteps) steps_of<BF16, NT, kSteps, true>(acc, p0, p1, a, live, s * 4 + t, kSteps);
      if (s + kTail <= s1) {
        steps_of<BF16, NT, kTail, true>(acc, p0, p1, a, live, s * 4 + t, kTail);
        s += kTail;
      }
      if (s < s1) steps_of<BF16, NT, kTail, false>(acc, p0, p1, a, live, s * 4 + t, s1 - s);
      if (warp == kWarps - 1 && steps * 32 < g.K) {
        const int q = steps * 4 + t;
        const uint4 v0 = last_piece(w0, q, g.K), v1 = last_piece(w1, q, g.K);
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          const uint4 x = live[j] ? last_piece(a[j], q, g.K) : make_uint4(0, 0, 0, 0);
          __syncwarp();
          mma16816<BF16>(acc[j], v0.x, v1.x, v0.y, v1.y, x.x, x.y);
          mma16816<BF16>(acc[j], v0.z, v1.z, v0.w, v1.w, x.z, x.w);
        }
      }
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) sums[warp][j * 8 + 2 * t + (i & 1)][gi + (i >> 1) * 8] = acc[j][i];
      __syncthreads();
      for (int i = tid; i < NT * 8 * kOuts; i += kThreads) {
        const int r = i / kOuts, m = i % kOuts;
        float v = 0;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) v += sums[w][r][m];
        if (r0 + r < rows && m0 + m < g.M)
          store_out(g.out, g.out_dtype, (int64_t)(first + r0 + r) * g.M + m0 + m, v);
      }
      __syncthreads();
    }
  }
}

}  // namespace

cudaError_t launch_gg_few(const GgGemm& g, cudaStream_t st) {
  const int64_t ctas = ((int64_t)g.M + kOuts - 1) / kOuts;
  const int64_t groups = std::min<int64_t>(g.R, g.E);
  // two CTAs of each SM at a time; where there are more outputs a CTA goes on to others
  const int64_t most = std::max<int64_t>(1, 2 * tc_num_sms() / groups);
  const dim3 grid((unsigned)std::min(ctas, most), (unsigned)groups), block(kThreads);
  if (g.R <= 8)
    return g.bf16 ? launch_pdl(gg_few<true, 1>, grid, block, 0, st, g) : launch_pdl(gg_few<false, 1>, grid, block, 0, st, g);
  return g.bf16 ? launch_pdl(gg_few<true, 2>, grid, block, 0, st, g) : launch_pdl(gg_few<false, 2>, grid, block, 0, st, g);
}
