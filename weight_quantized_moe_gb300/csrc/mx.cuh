// Microscaled (MX) number formats: blocks of 32 consecutive elements, E2M1
// (4-bit) or E4M3 (8-bit), sharing one power-of-two scale held as the E8M0
// code e + 127.
#pragma once

#include "common.cuh"

#include <cuda_fp4.h>
#include <cuda_fp8.h>

namespace mq {

constexpr int kMxBlock = 32;
constexpr uint32_t kInfBits = 0x7f800000u;

template <int BITS>
struct Mx {
  static_assert(BITS == 4 || BITS == 8, "E2M1 or E4M3");
  static constexpr int kEmax = BITS == 4 ? 2 : 8;  // exponent of the largest element
};

// Scale code of a block whose largest magnitude has these float32 bits:
// floor(log2 amax) - emax + 127 = (biased exponent) - emax, at least 0 (which
// also holds zero and subnormal maxima), and 255 (NaN) where the block holds
// an infinity or NaN.
template <int BITS>
__device__ __forceinline__ uint32_t mx_scale_code(uint32_t amax_bits) {
  const int e = (int)(amax_bits >> 23) - Mx<BITS>::kEmax;
  return amax_bits >= kInfBits ? 255u : (uint32_t)max(e, 0);
}

// 2^-e for scale code e + 127, exact: the code is at most 252, so the
// exponent field 254 - code is a normal float's.  Blocks with a NaN scale
// get 0.
__device__ __forceinline__ float mx_inv_scale(uint32_t code) {
  return code == 255u ? 0.0f : __uint_as_float((254u - code) << 23);
}

// 2^e for scale code e + 127 (code 0: the subnormal 2^-127; 255: NaN).
__device__ __forceinline__ float mx_scale(uint32_t code) {
  const uint32_t b = code == 0u ? 0x00400000u : code == 255u ? 0x7fc00000u : code << 23;
  return __uint_as_float(b);
}

// One element of a block: v * 2^-e (exact but for underflow far below the
// smallest element), or 0 in a block with a NaN scale.
__device__ __forceinline__ float mx_scaled(float v, float inv) {
  return inv == 0.0f ? 0.0f : v * inv;
}

// Larger of each 16-bit half, unsigned: magnitudes of two 16-bit floats (their
// bits without the sign order as they do, NaN above infinity).
__device__ __forceinline__ uint32_t max_halves(uint32_t a, uint32_t b) { return __vmaxu2(a, b); }

// Two elements, rounded to nearest even and clamped to the largest finite
// one; the first goes to the low nibble / byte.
__device__ __forceinline__ uint32_t e2m1x2(float a, float b) {
  return __nv_cvt_float2_to_fp4x2(make_float2(a, b), __NV_E2M1, cudaRoundNearest);
}
__device__ __forceinline__ uint32_t e4m3x2(float a, float b) {
  return __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
}

__device__ __forceinline__ uint32_t max_bits(uint32_t m, float v) {
  return max(m, __float_as_uint(v) & 0x7fffffffu);
}

// Largest of the four adjacent lanes that share a block.
__device__ __forceinline__ uint32_t block_max(uint32_t m) {
  m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
  return max(m, __shfl_xor_sync(0xffffffffu, m, 2));
}

// Bits of the largest of eight magnitudes.
__device__ __forceinline__ uint32_t max8_bits(const float (&v)[8]) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max_bits(m, v[i]);
  return m;
}

// Bits of the largest magnitude of a block of 16-bit floats, eight per lane.
__device__ __forceinline__ uint32_t block_max16(uint4 r) {
  uint32_t m = max_halves(max_halves(r.x & 0x7fff7fffu, r.y & 0x7fff7fffu),
                          max_halves(r.z & 0x7fff7fffu, r.w & 0x7fff7fffu));
  m = max_halves(m, __shfl_xor_sync(0xffffffffu, m, 1));
  m = max_halves(m, __shfl_xor_sync(0xffffffffu, m, 2));
  return max(m >> 16, m & 0xffffu);
}

// Eight consecutive values of type T as float32 (16-byte aligned; 32 bytes of
// float).  Plain loads, not read-only ones: the norm may write its sums where
// its residual came from.
template <typename T>
struct Row8;

template <>
struct Row8<__nv_bfloat16> {
  uint4 r;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) {
    r = *reinterpret_cast<const uint4*>(p);
  }
  __device__ __forceinline__ void get(float (&v)[8]) const {
    v[0] = bf16_lo(r.x); v[1] = bf16_hi(r.x); v[2] = bf16_lo(r.y); v[3] = bf16_hi(r.y);
    v[4] = bf16_lo(r.z); v[5] = bf16_hi(r.z); v[6] = bf16_lo(r.w); v[7] = bf16_hi(r.w);
  }
  // float32 bits of the block's largest magnitude (four adjacent lanes)
  __device__ __forceinline__ uint32_t block_amax() const { return block_max16(r) << 16; }
};

template <>
struct Row8<__half> {
  uint4 r;
  __device__ __forceinline__ void load(const __half* p) {
    r = *reinterpret_cast<const uint4*>(p);
  }
  __device__ __forceinline__ void get(float (&v)[8]) const {
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
      v[2 * i] = f.x;
      v[2 * i + 1] = f.y;
    }
  }
  __device__ __forceinline__ uint32_t block_amax() const {
    return __float_as_uint(__half2float(__ushort_as_half((unsigned short)block_max16(r))));
  }
};

template <>
struct Row8<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = reinterpret_cast<const float4*>(p)[0];
    b = reinterpret_cast<const float4*>(p)[1];
  }
  __device__ __forceinline__ void get(float (&v)[8]) const {
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  }
  __device__ __forceinline__ uint32_t block_amax() const {
    float v[8];
    get(v);
    return block_max(max8_bits(v));
  }
};

// Eight consecutive elements of a block with scale code `code`: their codes in
// q[0] (4 bits) or q[0..1] (8 bits).
template <int BITS>
__device__ __forceinline__ void mx_pack8(const float (&v)[8], uint32_t code, uint32_t (&q)[2]) {
  const float inv = mx_inv_scale(code);
  float t[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) t[i] = v[i] * inv;
  if (BITS == 4) {
    q[0] = e2m1x2(t[0], t[1]) | e2m1x2(t[2], t[3]) << 8 | e2m1x2(t[4], t[5]) << 16 |
           e2m1x2(t[6], t[7]) << 24;
    q[1] = 0;
  } else {
    q[0] = e4m3x2(t[0], t[1]) | e4m3x2(t[2], t[3]) << 16;
    q[1] = e4m3x2(t[4], t[5]) | e4m3x2(t[6], t[7]) << 16;
  }
  if (code == 255u) q[0] = q[1] = 0;  // (infinity times 0 above)
}

// Eight float32 values rounded once (to nearest even) and stored.
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&v)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void store8(__half* p, const float (&v)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __half2 h = __floats2half2_rn(v[2 * i], v[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void store8(float* p, const float (&v)[8]) {
  reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}

}  // namespace mq

// ---------------------------------------------------------------------------
// Internal launchers of the MX operators (dtype: MQ_DTYPE_*).
// ---------------------------------------------------------------------------
MQ_HIDDEN cudaError_t launch_quant_mx(const void* x, int dtype, int64_t rows, int64_t cols,
                                      int64_t row_stride, int bits, uint8_t* q, uint8_t* scale,
                                      cudaStream_t st);
MQ_HIDDEN cudaError_t launch_dequant_mx(const uint8_t* q, const uint8_t* scale, int64_t n,
                                        int bits, void* out, int dtype, cudaStream_t st);
struct NormArgs {
  const void* x;
  const void* residual;  // or null
  const void* weight;
  int dtype;             // of x, residual, residual_out and y
  int weight_f32;        // weight is float32 instead
  int T, H;
  int64_t x_stride, residual_stride;  // elements between rows
  float eps;
  void* residual_out;    // or null
  void* y;               // or null
  int bits;
  uint8_t* q;
  uint8_t* scale;
};
MQ_HIDDEN cudaError_t launch_rmsnorm_mx(const NormArgs& a, cudaStream_t st);

// Rows grouped by expert times each expert's 4-bit weights.
enum MxEpilogue {
  MX_EPI_OUT = 0,    // out[row, n], 16-bit or float32
  MX_EPI_PART = 1,   // float32 partial sums [split][destination row][n]
  MX_EPI_GATED = 2,  // silu(gate) * up as MX codes and scales
};
struct MxGemm {
  int a_bits;                 // 8 (E4M3) or 4 (E2M1) rows
  MxEpilogue epi;
  const uint8_t* a;           // [R, K * a_bits / 8]
  const uint8_t* a_scale;     // [R, K / 32]
  const uint8_t* w;           // [E, wrows, K / 2]
  const uint8_t* w_scale;     // [E, wrows, K / 32]
  int64_t R;                  // rows of a
  int64_t S;                  // live rows at most (the plan's estimate)
  int E, K, N, wrows;         // N outputs; wrows = N, or 2 N when gated
  int64_t weight_bytes;       // codes of the weights that the call can reach (a forward: both products')
  const int32_t* seg_start;   // first row of each expert (null: one expert, all rows)
  const int32_t* seg_count;   // rows of each expert (null: seg_start[e + 1] - seg_start[e])
  void* out;                  // MX_EPI_OUT: [R, N]
  int out_dtype;
  float* part;                // MX_EPI_PART: [splits, part_rows, N]
  int64_t part_rows;
  const int32_t* dest;        // destination row of each row (null: the row itself)
  const float* dest_w;        // factor of each destination row (null: 1)
  uint8_t* act;               // MX_EPI_GATED: [R, N * a_bits / 8]
  uint8_t* act_scale;         // MX_EPI_GATED: [R, N / 32]
  unsigned* status;
};
struct MxPlan {
  int bn;      // rows per tile
  bool pair;   // CTA pairs (cta_group::2), else single CTAs
  int splits;  // K splits (MX_EPI_PART)
};
MQ_HIDDEN MxPlan mx_plan(int64_t S, int E, int K, int N, bool gated, int a_bits);
MQ_HIDDEN cudaError_t launch_mx_gemm(const MxGemm& g, const MxPlan& pl, cudaStream_t st);
// out[r, :] = sum over splits of part[split, r, :], for the rows
// [offsets[0], offsets[E]) (null: all rows).
MQ_HIDDEN cudaError_t launch_mx_reduce(const float* part, int splits, int64_t rows, int N,
                                       const int32_t* offsets, int E, void* out, int out_dtype,
                                       cudaStream_t st);
// The token-slots in expert order (stable), each expert's first row [E + 1], and
// their rows of a with the scales in that order: dst row p = row sorted[p] / k.
MQ_HIDDEN cudaError_t launch_mx_arrange(const int32_t* ids, int S, int k, int E, const uint8_t* a,
                                        const uint8_t* a_scale, int row_bytes, int scale_bytes,
                                        int32_t* sorted, int32_t* offsets, uint8_t* dst,
                                        uint8_t* dst_scale, unsigned* status, cudaStream_t st);
// Rows of a (and their scales) in expert order: dst row p = src row sorted[p] / k.
MQ_HIDDEN cudaError_t launch_mx_gather(const uint8_t* a, const uint8_t* a_scale, int row_bytes,
                                       int scale_bytes, const int32_t* sorted,
                                       const int32_t* num_padded, int k, int S, int64_t cap,
                                       uint8_t* dst, uint8_t* dst_scale, cudaStream_t st);
// The router-weighted sum of each token's slots (weights already applied).
MQ_HIDDEN cudaError_t launch_mx_combine(const float* part, int splits, const int32_t* ids,
                                        int tokens, int k, int E, int H, void* out,
                                        int out_dtype, cudaStream_t st);
