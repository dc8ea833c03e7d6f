// Microscaled quantiser, its inverse, and the residual + RMS norm that writes
// microscaled rows.
#include "mx.cuh"

namespace {

using mq::Row8;

constexpr int kQuantThreads = 256;

// One lane per 8 consecutive elements, so that the four lanes of a block are
// adjacent; U such vectors per thread.  Bound by HBM: each element is read
// and written once (180224 x 2048 bf16 in a loop of 40 calls: to 4 bits 136 us, 6.87
// TB/s; to 8 bits 155 us, 7.22 TB/s; a copy of such rows, with as many bytes
// written as read, 6.73 TB/s).  The block maximum is taken on packed 16-bit
// magnitudes (with eight float maxima per lane 156 us to 4 bits).
template <typename T, int BITS, int U, bool DENSE>
__global__ void __launch_bounds__(kQuantThreads) quant_mx_kernel(const T* __restrict__ x,
                                                                 int64_t nvec, uint32_t vec_per_row,
                                                                 int64_t row_stride,
                                                                 uint8_t* __restrict__ q,
                                                                 uint8_t* __restrict__ scale) {
  mq::pdl_wait();
  mq::pdl_trigger();
  const int64_t i0 = (int64_t)blockIdx.x * (kQuantThreads * U) + threadIdx.x;
  Row8<T> r[U] = {};
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int64_t i = i0 + u * kQuantThreads;
    if (i < nvec) {
      if (DENSE) {
        r[u].load(x + i * 8);
      } else {
        const int64_t row = i / vec_per_row;
        r[u].load(x + row * row_stride + (i - row * vec_per_row) * 8);
      }
    }
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int64_t i = i0 + u * kQuantThreads;
    // (past the end r is 0: whole blocks are past it together)
    const uint32_t code = mq::mx_scale_code<BITS>(r[u].block_amax());
    float v[8];
    r[u].get(v);
    uint32_t w[2];
    mq::mx_pack8<BITS>(v, code, w);
    if (i < nvec) {
      if (BITS == 4) reinterpret_cast<uint32_t*>(q)[i] = w[0];
      else reinterpret_cast<uint2*>(q)[i] = make_uint2(w[0], w[1]);
      if ((threadIdx.x & 3) == 0) scale[i >> 2] = (uint8_t)code;
    }
  }
}

// The inverse: bound by HBM, mostly its writes (180224 x 2048 from 4 bits to
// bf16 134.6 us, 6.94 TB/s; from 8 bits 159 us, 7.03 TB/s).
template <typename T, int BITS>
__global__ void __launch_bounds__(256) dequant_mx_kernel(const uint8_t* __restrict__ q,
                                                         const uint8_t* __restrict__ scale,
                                                         int64_t nvec, T* __restrict__ out) {
  mq::pdl_wait();
  mq::pdl_trigger();
  constexpr int U = 4;
  const int64_t i0 = (int64_t)blockIdx.x * (256 * U) + threadIdx.x;
  uint2 r[U];
  uint32_t sc[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int64_t i = i0 + u * 256;
    if (i < nvec) {
      if (BITS == 4) r[u].x = __ldg(reinterpret_cast<const uint32_t*>(q) + i);
      else r[u] = __ldg(reinterpret_cast<const uint2*>(q) + i);
      sc[u] = __ldg(scale + (i >> 2));
    }
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int64_t i = i0 + u * 256;
    if (i >= nvec) continue;
    const float s = mq::mx_scale(sc[u]);
    float v[8];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      __half2_raw h;
      if (BITS == 4) {
        h = __nv_cvt_fp4x2_to_halfraw2((__nv_fp4x2_storage_t)((r[u].x >> (8 * j)) & 0xff), __NV_E2M1);
      } else {
        const uint32_t w = j < 2 ? r[u].x : r[u].y;
        h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)((w >> (16 * (j & 1))) & 0xffff), __NV_E4M3);
      }
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
      v[2 * j] = f.x * s;
      v[2 * j + 1] = f.y * s;
    }
    mq::store8(out + i * 8, v);
  }
}

// One CTA per row; the row's float32 sums stay in registers (V vectors of 8
// per thread) between the sum of squares and the output, so every input is
// read once.  h = x + residual is rounded only where it is stored; the norm
// and the codes are taken from the float32 values.  Bound by HBM (bf16 with
// residual and 16-bit output: 8192 x 4096 46.4 us, 6.5 TB/s; V = 2, 8192 x 5120 56.0
// us, 4096 x 8192 45.5; V = 4, 4096 x 16384 89.1, 2048 x 32768 95.0, 6.4 TB/s).  V = 1
// up to H = 4096: the rows in flight come from several CTAs per SM.
template <typename T, typename W, int BITS, int V>
__global__ void __launch_bounds__(1024) rmsnorm_mx_kernel(const NormArgs a) {
  __shared__ float s_sum[32];
  mq::pdl_wait();
  mq::pdl_trigger();
  const int64_t row = blockIdx.x;
  const int nvec = a.H >> 3;
  const int nt = blockDim.x;
  const T* x = static_cast<const T*>(a.x) + row * a.x_stride;
  const T* res = a.residual ? static_cast<const T*>(a.residual) + row * a.residual_stride : nullptr;
  float h[V][8];
  {
    Row8<T> rx[V], rr[V];
#pragma unroll
    for (int u = 0; u < V; ++u) {
      const int i = threadIdx.x + u * nt;
      if (i < nvec) {
        rx[u].load(x + i * 8);
        if (res) rr[u].load(res + i * 8);
      }
    }
#pragma unroll
    for (int u = 0; u < V; ++u) {
      const int i = threadIdx.x + u * nt;
#pragma unroll
      for (int j = 0; j < 8; ++j) h[u][j] = 0.0f;
      if (i < nvec) {
        rx[u].get(h[u]);
        if (res) {
          float r[8];
          rr[u].get(r);
#pragma unroll
          for (int j = 0; j < 8; ++j) h[u][j] += r[j];
        }
      }
    }
  }
  float sum = 0.0f;
#pragma unroll
  for (int u = 0; u < V; ++u)
#pragma unroll
    for (int j = 0; j < 8; ++j) sum = fmaf(h[u][j], h[u][j], sum);
#pragma unroll
  for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  const int lane = threadIdx.x & 31;
  if (lane == 0) s_sum[threadIdx.x >> 5] = sum;
  if (a.residual_out) {
    T* ro = static_cast<T*>(a.residual_out) + row * a.H;
#pragma unroll
    for (int u = 0; u < V; ++u) {
      const int i = threadIdx.x + u * nt;
      if (i < nvec) mq::store8(ro + i * 8, h[u]);
    }
  }
  __syncthreads();
  sum = lane < (nt >> 5) ? s_sum[lane] : 0.0f;
#pragma unroll
  for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  const float rstd = rsqrtf(sum / (float)a.H + a.eps);
  const W* wt = static_cast<const W*>(a.weight);
#pragma unroll
  for (int u = 0; u < V; ++u) {
    const int i = threadIdx.x + u * nt;
    if (i < nvec) {
      Row8<W> rw;
      rw.load(wt + i * 8);
      float w[8];
      rw.get(w);
#pragma unroll
      for (int j = 0; j < 8; ++j) h[u][j] = h[u][j] * rstd * w[j];
      if (a.y) mq::store8(static_cast<T*>(a.y) + row * a.H + i * 8, h[u]);
    }
    uint32_t p[2];
    const uint32_t code = mq::mx_scale_code<BITS>(mq::block_max(mq::max8_bits(h[u])));
    mq::mx_pack8<BITS>(h[u], code, p);
    if (i < nvec) {
      const int64_t at = row * nvec + i;
      if (BITS == 4) reinterpret_cast<uint32_t*>(a.q)[at] = p[0];
      else reinterpret_cast<uint2*>(a.q)[at] = make_uint2(p[0], p[1]);
      if ((lane & 3) == 0) a.scale[at >> 2] = (uint8_t)code;
    }
  }
}

template <typename T, int BITS>
cudaError_t quant_t(const void* x, int64_t rows, int64_t cols, int64_t stride, uint8_t* q,
                    uint8_t* scale, cudaStream_t st) {
  const int64_t nvec = rows * (cols / 8);
  // Large inputs: four vectors in flight per thread (180224 x 2048 bf16 to 4 / 8
  // bits 136.1 / 154.9 us, with eight 138.3 / 155.5).  Small ones, up to where the
  // SMs hold one per thread: one (600 x 4096 2.5 us, with four 3.0).
  constexpr int U = 4;
  const bool large = nvec >= (int64_t)tc_num_sms() * 2048;
  const int per = kQuantThreads * (large ? U : 1);
  const dim3 grid((unsigned)((nvec + per - 1) / per));
  const bool dense = stride == cols;
  auto kern = large ? (dense ? quant_mx_kernel<T, BITS, U, true> : quant_mx_kernel<T, BITS, U, false>)
                    : (dense ? quant_mx_kernel<T, BITS, 1, true> : quant_mx_kernel<T, BITS, 1, false>);
  return launch_pdl(kern, grid, dim3(kQuantThreads), 0, st, static_cast<const T*>(x), nvec,
                    (uint32_t)(cols / 8), stride, q, scale);
}

template <typename T>
cudaError_t dequant_t(const uint8_t* q, const uint8_t* scale, int64_t n, int bits, void* out,
                      cudaStream_t st) {
  const int64_t nvec = n / 8;
  const dim3 grid((unsigned)((nvec + 1023) / 1024));
  T* o = static_cast<T*>(out);
  return bits == 4 ? launch_pdl(dequant_mx_kernel<T, 4>, grid, dim3(256), 0, st, q, scale, nvec, o)
                   : launch_pdl(dequant_mx_kernel<T, 8>, grid, dim3(256), 0, st, q, scale, nvec, o);
}

template <typename T, typename W, int BITS>
cudaError_t norm_tw(const NormArgs& a, cudaStream_t st) {
  const int nvec = a.H / 8;
  const int v = nvec <= 512 ? 1 : nvec <= 1024 ? 2 : 4;
  const int nt = ((nvec + v - 1) / v + 31) / 32 * 32;
  const dim3 grid((unsigned)a.T), block(nt);
  switch (v) {
    case 1: return launch_pdl(rmsnorm_mx_kernel<T, W, BITS, 1>, grid, block, 0, st, a);
    case 2: return launch_pdl(rmsnorm_mx_kernel<T, W, BITS, 2>, grid, block, 0, st, a);
    default: return launch_pdl(rmsnorm_mx_kernel<T, W, BITS, 4>, grid, block, 0, st, a);
  }
}

template <typename T>
cudaError_t norm_t(const NormArgs& a, cudaStream_t st) {
  if (a.weight_f32)
    return a.bits == 4 ? norm_tw<T, float, 4>(a, st) : norm_tw<T, float, 8>(a, st);
  return a.bits == 4 ? norm_tw<T, T, 4>(a, st) : norm_tw<T, T, 8>(a, st);
}

}  // namespace

cudaError_t launch_quant_mx(const void* x, int dtype, int64_t rows, int64_t cols,
                            int64_t row_stride, int bits, uint8_t* q, uint8_t* scale,
                            cudaStream_t st) {
#define MQ_QUANT(T)                                                                      \
  return bits == 4 ? quant_t<T, 4>(x, rows, cols, row_stride, q, scale, st)              \
                   : quant_t<T, 8>(x, rows, cols, row_stride, q, scale, st);
  switch (dtype) {
    case MQ_DTYPE_BF16: MQ_QUANT(__nv_bfloat16)
    case MQ_DTYPE_F16: MQ_QUANT(__half)
    default: MQ_QUANT(float)
  }
#undef MQ_QUANT
}

cudaError_t launch_dequant_mx(const uint8_t* q, const uint8_t* scale, int64_t n, int bits,
                              void* out, int dtype, cudaStream_t st) {
  switch (dtype) {
    case MQ_DTYPE_BF16: return dequant_t<__nv_bfloat16>(q, scale, n, bits, out, st);
    case MQ_DTYPE_F16: return dequant_t<__half>(q, scale, n, bits, out, st);
    default: return dequant_t<float>(q, scale, n, bits, out, st);
  }
}

cudaError_t launch_rmsnorm_mx(const NormArgs& a, cudaStream_t st) {
  return a.dtype == MQ_DTYPE_BF16 ? norm_t<__nv_bfloat16>(a, st) : norm_t<__half>(a, st);
}
