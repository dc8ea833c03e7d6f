// What the tensor-core kernels with one role per warp share: bounded waits on
// the pipeline's barriers, the pair-or-single forms of arrivals and commits, and
// tensor maps.
//
// A kernel's control block `Ctl` has a `volatile int abort_flag`: a wait that
// runs out sets it (and MQ_DEV_WAIT_TIMEOUT), and every other wait of the CTA
// then gives up too.
#pragma once

#include "common.cuh"
#include "sm100_ptx.cuh"

#include <cudaTypedefs.h>

#include <atomic>
#include <mutex>

namespace mq {
namespace pipe {

using namespace mq::ptx;

constexpr unsigned long long kWaitNs = 1000000000ull;

template <int CG, typename Ctl>
__device__ __forceinline__ bool wait_bounded(uint64_t* bar, uint32_t parity, Ctl* ctl,
                                             unsigned* status) {
  const unsigned long long t0 = mq::global_timer_ns();
  for (uint32_t n = 1;; ++n) {
    if (CG == 2 ? mbar_try_wait_cluster(bar, parity) : mbar_try_wait(bar, parity)) return true;
    if ((n & 63u) == 0) {
      if (ctl->abort_flag) return false;
      if (mq::global_timer_ns() - t0 > kWaitNs) {
        ctl->abort_flag = 1;
        mq::flag(status, MQ_DEV_WAIT_TIMEOUT);
        return false;
      }
    }
  }
}

__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
  return p != 0;
}

// CG = 2: the arrivals may come from the other CTA of the pair.
template <int CG = 1, typename Ctl>
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, Ctl* ctl,
                                          unsigned* status) {
  bool ok = CG == 2 ? mbar_try_wait_cluster(bar, parity) : mbar_try_wait(bar, parity);
  if (__all_sync(0xffffffffu, ok)) return true;
  ok = ok || wait_bounded<CG>(bar, parity, ctl, status);
  return __all_sync(0xffffffffu, ok);
}

// Arrives on the barrier of the CTA that issues the MMAs.
template <int CG>
__device__ __forceinline__ void arrive(uint64_t* bar) {
  if (CG == 2) mbar_arrive_cluster(map_rank(bar, 0));
  else mbar_arrive(bar);
}

// Signals the MMAs issued so far: on both CTAs of a pair.
template <int CG>
__device__ __forceinline__ void commit(uint64_t* bar) {
  if (CG == 2) mma_commit_pair(bar);
  else mma_commit(bar);
}

// At the end, or after an abort: lets what is in flight land; bounded, ignores the
// flag.  For whole warps: lanes may see the barrier's phase end at different polls, and
// what follows (barriers, tensor-memory deallocation) takes the warp together.
__device__ __forceinline__ void wait_drain(uint64_t* bar, uint32_t parity) {
  const unsigned long long t0 = mq::global_timer_ns();
  while (!mbar_try_wait(bar, parity))
    if (mq::global_timer_ns() - t0 > kWaitNs) break;
  __syncwarp();
}

// A role's place in a ring of n slots: which slot, and how often round, mod 2.
// (Counted on: a division by n costs more than a short stage.)
struct Ring {
  uint32_t slot = 0, turn = 0;
  __device__ __forceinline__ void next(uint32_t n) {
    if (++slot == n) {
      slot = 0;
      turn ^= 1;
    }
  }
};

__device__ __forceinline__ void store_out(void* out, int dtype, int64_t i, float v) {
  if (dtype == MQ_DTYPE_BF16) static_cast<__nv_bfloat16*>(out)[i] = __float2bfloat16_rn(v);
  else if (dtype == MQ_DTYPE_F16) static_cast<__half*>(out)[i] = __float2half_rn(v);
  else static_cast<float*>(out)[i] = v;
}

// ------------------------------------------------------------ host side --
inline PFN_cuTensorMapEncodeTiled_v12000 map_encoder() {
  static PFN_cuTensorMapEncodeTiled_v12000 encode = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* fn = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault,
                                         &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
  });
  return encode;
}

// Tensor map with the 128-byte swizzle; what lies outside reads as zero.
inline cudaError_t make_map(CUtensorMap* map, CUtensorMapDataType dt, int rank, const void* base,
                            const cuuint64_t* dims, const cuuint64_t* strides,
                            const cuuint32_t* box,
                            CUtensorMapSwizzle swizzle = CU_TENSOR_MAP_SWIZZLE_128B) {
  const auto encode = map_encoder();
  if (!encode) return cudaErrorNotSupported;
  const cuuint32_t ones[4] = {1, 1, 1, 1};
  const auto make = [&] {
    return encode(map, dt, rank, const_cast<void*>(base), dims, strides, box, ones,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
  };
  if (make()) return cudaSuccess;
  // The driver's call needs the device's context bound to this thread, which a
  // thread that has made no other CUDA call (autograd's, say) does not have yet.
  int dev = 0;
  cudaError_t err = cudaGetDevice(&dev);
  if (err == cudaSuccess) err = cudaSetDevice(dev);
  if (err != cudaSuccess) return err;
  return make() ? cudaSuccess : cudaErrorInvalidValue;
}

// Lets a kernel have `bytes` of shared memory on the current device; `ready`: the devices
// where it has them.
template <typename K>
cudaError_t allow_smem(K kern, size_t bytes, std::atomic<uint64_t>& ready) {
  int dev = 0;
  cudaError_t err = cudaGetDevice(&dev);
  if (err != cudaSuccess) return err;
  const uint64_t bit = uint64_t(1) << (dev & 63);
  if (ready.load(std::memory_order_relaxed) & bit) return cudaSuccess;
  err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
  if (err == cudaSuccess) ready.fetch_or(bit, std::memory_order_relaxed);
  return err;
}

}  // namespace pipe
}  // namespace mq
