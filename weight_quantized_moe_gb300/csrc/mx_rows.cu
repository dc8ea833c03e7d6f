// Around the microscaled product: token-slots and their rows in expert order,
// the sum of K splits, and the router-weighted sum of a token's slots.
#include "mx.cuh"

namespace {

template <typename T>
__device__ __forceinline__ void store4(T* p, float4 v);
template <>
__device__ __forceinline__ void store4(float* p, float4 v) {
  *reinterpret_cast<float4*>(p) = v;
}
template <>
__device__ __forceinline__ void store4(__nv_bfloat16* p, float4 v) {
  __nv_bfloat162 a = __floats2bfloat162_rn(v.x, v.y), b = __floats2bfloat162_rn(v.z, v.w);
  *reinterpret_cast<uint2*>(p) = make_uint2(*reinterpret_cast<uint32_t*>(&a), *reinterpret_cast<uint32_t*>(&b));
}
template <>
__device__ __forceinline__ void store4(__half* p, float4 v) {
  __half2 a = __floats2half2_rn(v.x, v.y), b = __floats2half2_rn(v.z, v.w);
  *reinterpret_cast<uint2*>(p) = make_uint2(*reinterpret_cast<uint32_t*>(&a), *reinterpret_cast<uint32_t*>(&b));
}

// Sums the K splits in their order and rounds once; four outputs per thread.
// With an odd N a group may cross rows and the splits are not 16-byte aligned:
// one at a time then.
template <typename T>
__global__ void __launch_bounds__(256) mx_reduce(const float* __restrict__ part, int splits,
                                                 int64_t rows, int N,
                                                 const int32_t* __restrict__ offsets, int E,
                                                 T* __restrict__ out) {
  mq::pdl_wait();
  mq::pdl_trigger();
  const int64_t n = rows * N;
  const int64_t lo = offsets ? min((int64_t)max(offsets[0], 0), rows) * N : 0;
  const int64_t hi = offsets ? min((int64_t)max(offsets[E], 0), rows) * N : n;
  const int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;
  if ((N & 3) == 0) {
    if (i < lo || i >= hi) return;
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int k = 0; k < splits; ++k) {
      const float4 v = *reinterpret_cast<const float4*>(part + k * n + i);
      s.x += v.x;
      s.y += v.y;
      s.z += v.z;
      s.w += v.w;
    }
    store4(out + i, s);
  } else {
    for (int64_t j = max(i, lo); j < min(i + 4, hi); ++j) {
      float s = 0.f;
      for (int k = 0; k < splits; ++k) s += part[k * n + j];
      out[j] = (T)s;
    }
  }
}

// out[t, :] = sum over the token's valid slots j and the K splits, in the order
// (j, split), of part[split, t k + j, :], rounded once.  A thread sums U groups
// of four outputs and has B slots' groups in flight.  Bound by HBM: with two
// slots per token one group per thread leaves too little in flight (4096
// tokens, k=2, H=4096, between events: 63 us with U = 1, 26 with 4).
template <typename T, int U, int B>
__global__ void __launch_bounds__(256) mx_combine(const float* __restrict__ part, int splits,
                                                  const int32_t* __restrict__ ids, int tokens,
                                                  int k, int E, int H, T* __restrict__ out) {
  mq::pdl_wait();
  mq::pdl_trigger();
  constexpr int per = 256 * U;               // groups of a CTA
  const int ctas = (H / 4 + per - 1) / per;  // of a row
  const int64_t t = blockIdx.x / ctas;
  const int c0 = (int)(blockIdx.x % ctas) * per + threadIdx.x;
  const int64_t slots = (int64_t)tokens * k;
  float4 acc[U];
#pragma unroll
  for (int u = 0; u < U; ++u) acc[u] = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int q0 = 0; q0 < k * splits; q0 += B) {
    float4 v[B][U];
#pragma unroll
    for (int b = 0; b < B; ++b) {
      const int q = q0 + b, j = q / splits;
      const int e = q < k * splits ? ids[t * k + j] : -1;
      const float4* row = reinterpret_cast<const float4*>(
          part + ((q - j * splits) * slots + t * k + j) * H);
#pragma unroll
      for (int u = 0; u < U; ++u)
        v[b][u] = e >= 0 && e < E && c0 + u * 256 < H / 4 ? __ldcs(row + c0 + u * 256)
                                                          : make_float4(0.f, 0.f, 0.f, 0.f);
    }
#pragma unroll
    for (int b = 0; b < B; ++b)
#pragma unroll
      for (int u = 0; u < U; ++u) {
        acc[u].x += v[b][u].x;
        acc[u].y += v[b][u].y;
        acc[u].z += v[b][u].z;
        acc[u].w += v[b][u].w;
      }
  }
#pragma unroll
  for (int u = 0; u < U; ++u)
    if (c0 + u * 256 < H / 4) store4(out + t * H + (int64_t)(c0 + u * 256) * 4, acc[u]);
}

constexpr int kArrangeSlots = 8;

// Rows of a in expert order, and the order itself: a stable counting sort of
// the token-slots by expert and the copy of their rows in one launch.  A CTA
// owns eight consecutive slots; it counts every slot's expert itself (S ids from
// L2), and those of the slots before its own, so that no CTA waits for another.
// That counting bounds it: up to 2048 slots it takes less than the align kernel
// and a gather (T=64 forwards: E=8 147 -> 144 us, E=128 k=8 with Zipf popularity
// 38.3 -> 34.5), at 4096 as much (69.3 and 71.0), at 8192 more (22 us against 18
// between events).
//   sorted [S]: slots in expert order; offsets [E + 1]; dst row p = row
//   sorted[p] / k of a.  Slots with an id outside [0, E) are left out.
__global__ void __launch_bounds__(256) mx_arrange(const int32_t* __restrict__ ids, int S, int k,
                                                  int E, const uint8_t* __restrict__ a,
                                                  const uint8_t* __restrict__ a_scale,
                                                  int row_bytes, int scale_bytes,
                                                  int32_t* __restrict__ sorted,
                                                  int32_t* __restrict__ offsets,
                                                  uint8_t* __restrict__ dst,
                                                  uint8_t* __restrict__ dst_scale,
                                                  unsigned* status) {
  extern __shared__ int arrange_smem[];
  int* total = arrange_smem;  // slots of each expert, then its first row
  int* before = total + E;    // of them, those ahead of this CTA's slots
  __shared__ int place[kArrangeSlots];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int s0 = blockIdx.x * kArrangeSlots;
  for (int e = tid; e < 2 * E; e += 256) arrange_smem[e] = 0;
  mq::pdl_wait();
  mq::pdl_trigger();
  __syncthreads();
  constexpr int kBatch = 4;
  bool bad = false;
  for (int base = warp * 32; base < S; base += 256 * kBatch) {
    int ev[kBatch];
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      const int s = base + b * 256 + lane;
      ev[b] = s < S ? ids[s] : -1;
      bad |= s < S && (ev[b] < 0 || ev[b] >= E);
    }
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      const int s = base + b * 256 + lane;
      if (ev[b] >= 0 && ev[b] < E) {
        atomicAdd(&total[ev[b]], 1);
        if (s < s0) atomicAdd(&before[ev[b]], 1);
      }
    }
  }
  if (blockIdx.x == 0 && __any_sync(0xffffffffu, bad) && lane == 0)
    mq::flag(status, MQ_DEV_BAD_EXPERT_ID);
  __syncthreads();
  if (warp == 0) {
    int run = 0;
    for (int e0 = 0; e0 < E; e0 += 32) {
      const int e = e0 + lane;
      const int mine = e < E ? total[e] : 0;
      int incl = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int t = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += t;
      }
      if (e < E) {
        total[e] = run + incl - mine;
        if (blockIdx.x == 0) offsets[e] = run + incl - mine;
      }
      run += __shfl_sync(0xffffffffu, incl, 31);
    }
    if (blockIdx.x == 0 && lane == 0) offsets[E] = run;
    __syncwarp();
    const int s = s0 + lane;
    int e = lane < kArrangeSlots && s < S ? ids[s] : -1;
    if (e >= E) e = -1;
    const unsigned peers = __match_any_sync(0xffffffffu, e);
    if (lane < kArrangeSlots) {
      int at = -1;
      if (e >= 0) {
        at = total[e] + before[e] + __popc(peers & ((1u << lane) - 1u));
        sorted[at] = s;
      }
      place[lane] = at;
    }
  }
  __syncthreads();
  for (int i = warp; i < kArrangeSlots; i += 8) {
    const int64_t at = place[i];
    if (at < 0) continue;
    const int64_t t = (s0 + i) / k;
    const uint4* src = reinterpret_cast<const uint4*>(a + t * row_bytes);
    uint4* d = reinterpret_cast<uint4*>(dst + at * row_bytes);
#pragma unroll 4
    for (int j = lane; j < row_bytes / 16; j += 32) d[j] = __ldg(src + j);
    const uint32_t* ss = reinterpret_cast<const uint32_t*>(a_scale + t * scale_bytes);
    uint32_t* ds = reinterpret_cast<uint32_t*>(dst_scale + at * scale_bytes);
    for (int j = lane; j < scale_bytes / 4; j += 32) ds[j] = __ldg(ss + j);
  }
}

// Many slots: rows in the align kernel's order.  One warp per row; 16-byte
// pieces of the codes, 4-byte words of the scales.
__global__ void __launch_bounds__(256) mx_gather(const uint8_t* __restrict__ a,
                                                 const uint8_t* __restrict__ a_scale,
                                                 int row_bytes, int scale_bytes,
                                                 const int32_t* __restrict__ sorted,
                                                 const int32_t* __restrict__ num_padded, int k,
                                                 int S, uint8_t* __restrict__ dst,
                                                 uint8_t* __restrict__ dst_scale) {
  mq::pdl_wait();
  mq::pdl_trigger();
  const int64_t row = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  if (row >= *num_padded) return;
  const int s = sorted[row];
  if (s >= S) return;  // padding
  const int lane = threadIdx.x & 31;
  const int64_t t = s / k;
  const uint4* src = reinterpret_cast<const uint4*>(a + t * row_bytes);
  uint4* d = reinterpret_cast<uint4*>(dst + row * row_bytes);
#pragma unroll 4
  for (int i = lane; i < row_bytes / 16; i += 32) d[i] = __ldg(src + i);
  const uint32_t* ss = reinterpret_cast<const uint32_t*>(a_scale + t * scale_bytes);
  uint32_t* ds = reinterpret_cast<uint32_t*>(dst_scale + row * scale_bytes);
  for (int i = lane; i < scale_bytes / 4; i += 32) ds[i] = __ldg(ss + i);
}

template <typename T>
cudaError_t combine_t(const float* part, int splits, const int32_t* ids, int tokens, int k, int E,
                      int H, T* out, cudaStream_t st) {
  // U = 4 once its CTAs still cover the SMs several times
  const bool wide = H >= 4096 && (int64_t)tokens * (H / 4096) >= 4 * tc_num_sms();
  const int per = 256 * (wide ? 4 : 1);
  const int64_t grid = (int64_t)tokens * ((H / 4 + per - 1) / per);
  return launch_pdl(wide ? mx_combine<T, 4, 2> : mx_combine<T, 1, 8>, dim3((unsigned)grid),
                    dim3(256), 0, st, part, splits, ids, tokens, k, E, H, out);
}

}  // namespace

cudaError_t launch_mx_reduce(const float* part, int splits, int64_t rows, int N,
                             const int32_t* offsets, int E, void* out, int out_dtype,
                             cudaStream_t st) {
  const dim3 grid((unsigned)((rows * N + 1023) / 1024)), block(256);
  switch (out_dtype) {
    case MQ_DTYPE_BF16:
      return launch_pdl(mx_reduce<__nv_bfloat16>, grid, block, 0, st, part, splits, rows, N,
                        offsets, E, static_cast<__nv_bfloat16*>(out));
    case MQ_DTYPE_F16:
      return launch_pdl(mx_reduce<__half>, grid, block, 0, st, part, splits, rows, N, offsets, E,
                        static_cast<__half*>(out));
    default:
      return launch_pdl(mx_reduce<float>, grid, block, 0, st, part, splits, rows, N, offsets, E,
                        static_cast<float*>(out));
  }
}

cudaError_t launch_mx_arrange(const int32_t* ids, int S, int k, int E, const uint8_t* a,
                              const uint8_t* a_scale, int row_bytes, int scale_bytes,
                              int32_t* sorted, int32_t* offsets, uint8_t* dst,
                              uint8_t* dst_scale, unsigned* status, cudaStream_t st) {
  return launch_pdl(mx_arrange, dim3((unsigned)((S + kArrangeSlots - 1) / kArrangeSlots)),
                    dim3(256), 2 * (size_t)E * sizeof(int), st, ids, S, k, E, a, a_scale,
                    row_bytes, scale_bytes, sorted, offsets, dst, dst_scale, status);
}

cudaError_t launch_mx_gather(const uint8_t* a, const uint8_t* a_scale, int row_bytes,
                             int scale_bytes, const int32_t* sorted, const int32_t* num_padded,
                             int k, int S, int64_t cap, uint8_t* dst, uint8_t* dst_scale,
                             cudaStream_t st) {
  return launch_pdl(mx_gather, dim3((unsigned)((cap + 7) / 8)), dim3(256), 0, st, a, a_scale,
                    row_bytes, scale_bytes, sorted, num_padded, k, S, dst, dst_scale);
}

cudaError_t launch_mx_combine(const float* part, int splits, const int32_t* ids, int tokens, int k,
                              int E, int H, void* out, int out_dtype, cudaStream_t st) {
  return out_dtype == MQ_DTYPE_F16
             ? combine_t(part, splits, ids, tokens, k, E, H, static_cast<__half*>(out), st)
             : combine_t(part, splits, ids, tokens, k, E, H, static_cast<__nv_bfloat16*>(out), st);
}
