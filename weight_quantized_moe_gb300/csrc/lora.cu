// Low-rank adapters of many requests beside a projection that is already computed:
//
//   out[t] = base[t] + s[l] * B[l, e] (A[l, e] x[t])     l = ids[t], e the row's expert
//
// A row's group is the pair (l, e).  What bounds the operator is memory: x, base and
// out once, and each adapter in use once.  Two forms:
//
//   rows   A cluster of eight CTAs per row, one launch: each CTA takes an eighth of K,
//          the partial A x are exchanged through distributed shared memory, and each
//          CTA then has an eighth of the outputs.  Float32 arithmetic on the CUDA
//          cores.  For few rows, which seldom share an adapter.
//   tiles  Tiles of 128 consecutive rows, in the order that they come in, and two
//          launches on tcgen05.  Rows are the columns of the accumulators, so that a
//          column has one group whatever its neighbours have: every group of a tile is
//          multiplied with all its columns and each column keeps its own group's sums.
//          Nothing is sorted, gathered or masked, and what another request's adapter
//          holds (infinities, NaN) stays in the columns that are not kept.
//
// Tiles, first launch (lora_down): h = A x in float32.  Groups are packed into the 128
// lanes of an accumulator (eight of rank 16, two of rank 64), x is the other operand.
// Second launch (lora_up): s h is the columns' operand.  It is split into two 16-bit
// parts, h = 2^m (hi + lo), m the exponent of the row's largest |h|: 16 bits of
// precision for bf16 and 22 for f16, whose range it cannot leave either, for twice a
// small product.  base comes by TMA and goes back, with the sums added, the same way.
#include "lora.cuh"
#include "pipe.cuh"

#include <algorithm>
#include <atomic>
#include <cmath>
#include <type_traits>

namespace {

using namespace mq::pipe;

constexpr int kTile = 128;     // rows of a tile
constexpr int kSlot = 16384;   // 128 lines of 128 bytes
constexpr int kMaxE = 1024;
constexpr size_t kSmemMax = 227 * 1024;

// ------------------------------------------------------------------- rows --
constexpr int kCluster = 8;
constexpr int kRowThreads = 256;
constexpr int kMaxRank = 128;

__device__ __forceinline__ void unpack8(const uint4& v, bool bf16, float (&f)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (bf16) {
      f[2 * i] = mq::bf16_lo(w[i]);
      f[2 * i + 1] = mq::bf16_hi(w[i]);
    } else {
      const float2 t = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
      f[2 * i] = t.x;
      f[2 * i + 1] = t.y;
    }
  }
}

__device__ __forceinline__ float load_as(const void* p, int dtype, int64_t i) {
  if (dtype == MQ_DTYPE_BF16) return __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
  if (dtype == MQ_DTYPE_F16) return __half2float(static_cast<const __half*>(p)[i]);
  return static_cast<const float*>(p)[i];
}

// out[i] = base[j], bit for bit; 0 where there is no base.
__device__ __forceinline__ void copy_element(void* out, int64_t i, const void* base, int64_t j, int dtype) {
  if (dtype == MQ_DTYPE_F32)
    static_cast<uint32_t*>(out)[i] = base ? static_cast<const uint32_t*>(base)[j] : 0u;
  else
    static_cast<uint16_t*>(out)[i] = base ? static_cast<const uint16_t*>(base)[j] : (uint16_t)0;
}

__device__ __forceinline__ float dot8(const float (&a)[8], const float (&b)[8], float s) {
#pragma unroll
  for (int i = 0; i < 8; ++i) s = fmaf(a[i], b[i], s);
  return s;
}

// BF16: type of rows and adapters.  LPO: lanes that share an output, r / 8 rounded up
// to a power of two.
template <bool BF16, int LPO>
__global__ void __launch_bounds__(kRowThreads, 4) lora_rows(const LoraArgs p) {
  __shared__ float parts[kCluster][kMaxRank];
  __shared__ float h[kMaxRank];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = (int)cluster_rank();
  const int64_t t = blockIdx.x / kCluster;
  mq::pdl_wait();
  mq::pdl_trigger();
  // the row's group; the whole cluster comes to the same answer
  int l = p.ids[t];
  int e = 0;
  bool outside = false;
  if (p.offsets) {
    int below = 0;
    bool bad = false;
    for (int i = tid; i <= p.E; i += kRowThreads) {
      const int o = p.offsets[i];
      bad |= o < 0 || o > p.R || (i < p.E && p.offsets[i + 1] < o);
      below += i > 0 && o <= t;
    }
    const bool any_bad = __syncthreads_or(bad);
    if (any_bad && tid == 0 && blockIdx.x == 0) mq::flag(p.status, MQ_DEV_BAD_OFFSETS);
    // (a thread has up to five of the offsets)
#pragma unroll
    for (int i = 0; i < (kMaxE + kRowThreads) / kRowThreads; ++i) e += __syncthreads_count(below > i);
    outside = any_bad || t < p.offsets[0] || e >= p.E;
  }
  if (outside) return;
  if (l < -1 || l >= p.L) {
    if (tid == 0 && rank == 0) mq::flag(p.status, MQ_DEV_BAD_ADAPTER_ID);
    l = -1;
  }
  const int n0 = (int)((int64_t)p.N * rank / kCluster), n1 = (int)((int64_t)p.N * (rank + 1) / kCluster);
  if (l < 0) {
    if (p.base == p.out) return;
    for (int n = n0 + tid; n < n1; n += kRowThreads)
      copy_element(p.out, t * p.out_stride + n, p.base, t * p.base_stride + n, p.out_dtype);
    return;
  }
  cluster_arrive();  // (the others' shared memory may be written once all have come here)
  const int64_t g = (int64_t)l * p.E + e;
  const uint16_t* x = static_cast<const uint16_t*>(p.x) + t * p.x_stride;
  const uint16_t* a = static_cast<const uint16_t*>(p.a) + g * p.r * p.K;
  const uint16_t* b = static_cast<const uint16_t*>(p.b) + g * p.r * p.N;

  // The first outputs' rows of B and base are on their way while A x is summed.
  constexpr int kOuts = kRowThreads / LPO;  // outputs of a pass
  constexpr int kAhead = 4;
  const int chunk = tid % LPO;
  const bool has = chunk * 8 < p.r;
  const uint4 zero = make_uint4(0, 0, 0, 0);
  uint4 bv[kAhead];
  float old[kAhead];
  auto fetch = [&](int n, int i) {
    const bool live = n < n1;
    bv[i] = live && has ? __ldg(reinterpret_cast<const uint4*>(b + (int64_t)n * p.r + chunk * 8)) : zero;
    old[i] = live && chunk == 0 && p.base ? load_as(p.base, p.out_dtype, t * p.base_stride + n) : 0.0f;
  };
  const int first = n0 + tid / LPO;
#pragma unroll
  for (int i = 0; i < kAhead; ++i) fetch(first + i * kOuts, i);

  // A x over this CTA's vectors of eight; a warp takes four ranks at a time.
  const int vecs = p.K / 8;
  const int v0 = (int)((int64_t)vecs * rank / kCluster), v1 = (int)((int64_t)vecs * (rank + 1) / kCluster);
  constexpr int kRanks = 4;
  bool met = false;
  for (int j0 = warp; j0 < p.r; j0 += 8 * kRanks) {
    float acc[kRanks] = {};
#pragma unroll 2
    for (int v = v0 + lane; v < v1; v += 32) {
      const uint4 xv = __ldg(reinterpret_cast<const uint4*>(x) + v);
      uint4 av[kRanks];
#pragma unroll
      for (int i = 0; i < kRanks; ++i)
        av[i] = j0 + 8 * i < p.r ? __ldg(reinterpret_cast<const uint4*>(a + (int64_t)(j0 + 8 * i) * p.K) + v) : zero;
      float xf[8], af[8];
      unpack8(xv, BF16, xf);
#pragma unroll
      for (int i = 0; i < kRanks; ++i) {
        unpack8(av[i], BF16, af);
        acc[i] = dot8(xf, af, acc[i]);
      }
    }
    if (!met) cluster_wait();
    met = true;
#pragma unroll
    for (int i = 0; i < kRanks; ++i) {
#pragma unroll
      for (int o = 16; o; o >>= 1) acc[i] += __shfl_xor_sync(0xffffffffu, acc[i], o);
      const int j = j0 + 8 * i;
      if (j < p.r && lane < kCluster)  // to the CTA of rank `lane`
        asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(map_rank(&parts[rank][j], lane)), "f"(acc[i])
                     : "memory");
    }
  }
  if (!met) cluster_wait();
  cluster_sync();
  const float s = p.scaling ? p.scaling[l] : 1.0f;
  if (tid < p.r) {
    float v = 0;
#pragma unroll
    for (int c = 0; c < kCluster; ++c) v += parts[c][tid];
    h[tid] = v * s;
  }
  __syncthreads();
  float hv[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) hv[i] = has ? h[chunk * 8 + i] : 0.0f;
  for (int n = first; n - tid / LPO < n1; n += kAhead * kOuts) {
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      float bf[8];
      unpack8(bv[i], BF16, bf);
      float v = dot8(hv, bf, 0.0f);
#pragma unroll
      for (int o = LPO / 2; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
      const int m = n + i * kOuts;
      if (m < n1 && chunk == 0) store_out(p.out, p.out_dtype, t * p.out_stride + m, old[i] + v);
    }
#pragma unroll
    for (int i = 0; i < kAhead; ++i) fetch(n + (kAhead + i) * kOuts, i);
  }
}

// ------------------------------------------------------------------ tiles --
// Groups of a tile's rows.
struct Table {
  int key[kTile];        // group of a row as an index into the adapters (l E + e); -1 none, -2 not written
  int group_key[kTile];  // key of each of the tile's groups, in order of their first rows
  unsigned blocks[kTile];               // the 16-row blocks that hold rows of a group
  alignas(16) uint8_t slot[kTile];      // a row's group; kNone, kOut
  unsigned first[kTile / 32];
  int groups, rows;
  int inside;            // rows that are written
};
constexpr int kNone = 255, kOut = 254;

// Joins THREADS threads that start at warp 0 (barrier 2); all of them take part below.
template <int THREADS>
__device__ __forceinline__ void join() {
  asm volatile("bar.sync 2, %0;" ::"n"(THREADS) : "memory");
}

// Fills in the table of tile `tile`, with the first THREADS threads of the CTA (at least
// kTile); `offsets` is a copy of the experts' in shared memory (null: one expert).
template <int THREADS>
__device__ __forceinline__ void build_table(Table& tb, const LoraArgs& p, const int* offsets, bool bad,
                                            int t, int tile) {
  const int64_t row0 = (int64_t)tile * kTile;
  const int rows = (int)min((int64_t)kTile, p.R - row0);
  join<THREADS>();  // (the last table is no longer read)
  int key = -2;
  if (t < kTile) {
    if (t < rows && !bad) {
      const int64_t row = row0 + t;
      const int l = p.ids[row];
      int e = 0;
      bool in = true;
      if (offsets) {
        int lo = 0, hi = p.E;  // the number of experts that end at or before the row
        while (lo < hi) {
          const int mid = (lo + hi) >> 1;
          if (offsets[mid + 1] <= row) lo = mid + 1;
          else hi = mid;
        }
        e = lo;
        in = e < p.E && row >= offsets[0];
      }
      if (in) {
        if (l < -1 || l >= p.L) mq::flag(p.status, MQ_DEV_BAD_ADAPTER_ID);
        key = l >= 0 && l < p.L ? l * p.E + e : -1;
      }
    }
    tb.key[t] = key;
    tb.blocks[t] = 0;
  }
  if (t == 0) {
    tb.rows = rows;
    tb.inside = 0;
  }
  join<THREADS>();
  int at = t;  // the first row of this row's group
  if (t < kTile) {
    if (key >= 0) {
      const int4* keys = reinterpret_cast<const int4*>(tb.key);
#pragma unroll 8
      for (int i = kTile / 4 - 1; i >= 0; --i) {
        const int4 k = keys[i];
        if (k.w == key) at = min(at, 4 * i + 3);
        if (k.z == key) at = min(at, 4 * i + 2);
        if (k.y == key) at = min(at, 4 * i + 1);
        if (k.x == key) at = min(at, 4 * i);
      }
    }
    const unsigned firsts = __ballot_sync(0xffffffffu, key >= 0 && at == t);
    const unsigned in = __ballot_sync(0xffffffffu, key != -2);
    if ((t & 31) == 0) {
      tb.first[t >> 5] = firsts;
      atomicAdd(&tb.inside, __popc(in));
    }
  }
  join<THREADS>();
  if (t < kTile) {
    int g = 0, n = 0;
#pragma unroll
    for (int w = 0; w < kTile / 32; ++w) {
      const unsigned f = tb.first[w];
      n += __popc(f);
      g += w < (at >> 5) ? __popc(f) : w == (at >> 5) ? __popc(f & ((1u << (at & 31)) - 1u)) : 0;
    }
    const int slot = key >= 0 ? g : key == -1 ? kNone : kOut;
    tb.slot[t] = (uint8_t)slot;
    if (key >= 0 && at == t) tb.group_key[g] = key;
    if (t == 0) tb.groups = n;
    const unsigned peers = __match_any_sync(0xffffffffu, slot);
    if (key >= 0 && (peers & ((1u << (t & 31)) - 1u)) == 0)
      atomicOr(&tb.blocks[g], ((peers & 0xffffu ? 1u : 0u) | (peers >> 16 ? 2u : 0u)) << (t >> 5) * 2);
  }
  join<THREADS>();
}

// The offsets' copy in shared memory; true where they fall or leave [0, R].
__device__ __forceinline__ bool copy_offsets(const LoraArgs& p, int* to) {
  bool bad = false;
  if (p.offsets)
    for (int i = threadIdx.x; i <= p.E; i += blockDim.x) {
      const int o = p.offsets[i];
      to[i] = o;
      bad |= o < 0 || o > p.R || (i < p.E && p.offsets[i + 1] < o);
    }
  bad = __syncthreads_or(bad);
  if (bad && threadIdx.x == 0 && blockIdx.x == 0) mq::flag(p.status, MQ_DEV_BAD_OFFSETS);
  return bad;
}

__device__ __forceinline__ int ceil16(int n) { return (n + 15) & -16; }

__device__ __forceinline__ int byte_of(const uint4& v, int i) {
  const uint32_t w = i < 4 ? v.x : i < 8 ? v.y : i < 12 ? v.z : v.w;
  return (int)(w >> (i & 3) * 8 & 0xff);
}

// ---- first launch: h = A x ----
constexpr int kDownThreads = 256;
constexpr int kDownSlots = 12;  // of 16 KB: a stage of x, or of an accumulator's groups
constexpr int kBatch = 4;       // accumulators at a time

struct DownCtl {
  uint64_t full[kDownSlots], empty[kDownSlots];
  uint64_t acc_full, acc_empty, drain;
  uint32_t tmem;
  volatile int abort_flag;
};
struct DownShared {
  DownCtl ctl;
  Table table;
  int offsets[kMaxE + 1];
};

__global__ void __launch_bounds__(kDownThreads, 1)
    lora_down(const __grid_constant__ CUtensorMap map_x, const __grid_constant__ CUtensorMap map_a,
              const LoraArgs p, int rp, int splits, int mparts) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* slots = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  DownShared* sh = reinterpret_cast<DownShared*>(slots + kDownSlots * kSlot);
  DownCtl* ctl = &sh->ctl;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    tma_prefetch_desc(&map_x);
    tma_prefetch_desc(&map_a);
    for (int i = 0; i < kDownSlots; ++i) {
      mbar_init(&ctl->full[i], 1);
      mbar_init(&ctl->empty[i], 1);
    }
    mbar_init(&ctl->acc_full, 1);
    mbar_init(&ctl->acc_empty, 4);
    mbar_init(&ctl->drain, 1);
    ctl->abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(&ctl->tmem, 512);
    tmem_relinquish();
  }
  mq::pdl_wait();
  mq::pdl_trigger();
  const bool bad = copy_offsets(p, sh->offsets);
  const int split = blockIdx.x % splits;
  const int mpart = blockIdx.x / splits % mparts;
  const int tile = blockIdx.x / (splits * mparts);
  build_table<kDownThreads>(sh->table, p, p.offsets ? sh->offsets : nullptr, bad, tid, tile);
  const Table& tb = sh->table;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ctl->tmem;
  const int64_t row0 = (int64_t)tile * kTile;
  const int per = kTile / rp;                          // groups of an accumulator
  const int accs = (tb.groups + per - 1) / per;        // accumulators of the tile
  const int mine = accs > mpart ? (accs - mpart + mparts - 1) / mparts : 0;
  const int nst = (p.K + 63) / 64;
  const int s0 = (int)((int64_t)nst * split / splits), s1 = (int)((int64_t)nst * (split + 1) / splits);

  if (warp == 0) {
    const bool el = elect_one();
    uint32_t it = 0;
    bool ok = true;
    auto take = [&]() -> uint8_t* {  // the next slot, once it is free
      const uint32_t s = it % kDownSlots;
      ok = warp_wait(&ctl->empty[s], ((it / kDownSlots) & 1) ^ 1, ctl, p.status);
      return slots + s * kSlot;
    };
    for (int b0 = 0; b0 < mine && ok; b0 += kBatch)
      for (int s = s0; s < s1 && ok; ++s) {
        uint8_t* dst = take();
        if (!ok) break;
        uint64_t* bar = &ctl->full[it % kDownSlots];
        if (el) {
          mbar_arrive_expect_tx(bar, kSlot);
          tma_load_2d(dst, &map_x, bar, s * 64, (int)row0);
        }
        ++it;
        for (int b = b0; b < min(b0 + kBatch, mine); ++b) {
          dst = take();
          if (!ok) break;
          bar = &ctl->full[it % kDownSlots];
          const int g0 = (mpart + b * mparts) * per, n = min(per, tb.groups - g0);
          if (el) {
            mbar_arrive_expect_tx(bar, n * rp * 128);
            for (int i = 0; i < n; ++i) tma_load_3d(dst + i * rp * 128, &map_a, bar, s * 64, 0, tb.group_key[g0 + i]);
          }
          ++it;
        }
      }
    if (ctl->abort_flag)
      for (uint32_t j = it < kDownSlots ? 0 : it - kDownSlots; j < it; ++j)
        wait_drain(&ctl->full[j % kDownSlots], (j / kDownSlots) & 1);
  } else if (warp == 1) {
    const bool el = elect_one();
    const uint32_t idesc = idesc_16(p.bf16, kTile, ceil16(tb.rows), false, false);
    uint32_t it = 0;
    bool ok = true;
    for (int b0 = 0, turn = 0; b0 < mine && ok; b0 += kBatch, ++turn) {
      ok = warp_wait(&ctl->acc_empty, (turn & 1) ^ 1, ctl, p.status);
      tc_fence_after();
      for (int s = s0; s < s1 && ok; ++s) {
        const uint32_t xs = it++ % kDownSlots;
        ok = warp_wait(&ctl->full[xs], ((it - 1) / kDownSlots) & 1, ctl, p.status);
        const uint64_t bd = smem_desc_k_sw128(smem_addr(slots + xs * kSlot));
        for (int b = b0; b < min(b0 + kBatch, mine) && ok; ++b) {
          const uint32_t as = it++ % kDownSlots;
          ok = warp_wait(&ctl->full[as], ((it - 1) / kDownSlots) & 1, ctl, p.status);
          if (!ok) break;
          tc_fence_after();
          if (el) {
            const uint64_t ad = smem_desc_k_sw128(smem_addr(slots + as * kSlot));
#pragma unroll
            for (int j = 0; j < 4; ++j)
              mma_ss<1>(tmem + (b - b0) * kTile, ad + j * 2, bd + j * 2, idesc, (s > s0) | j);
            mma_commit(&ctl->empty[as]);
          }
        }
        if (ok && el) mma_commit(&ctl->empty[xs]);
      }
      if (ok && el) mma_commit(&ctl->acc_full);
    }
    if (el) mma_commit(&ctl->drain);
    wait_drain(&ctl->drain, 0);
  } else if (warp >= 4) {
    // A lane is one rank of one of the accumulator's groups.
    const int quad = warp & 3;
    const int gl = (quad * 32 + lane) / rp, j = (quad * 32 + lane) % rp;
    bool ok = true;
    for (int b0 = 0, turn = 0; b0 < mine && ok; b0 += kBatch, ++turn) {
      ok = warp_wait(&ctl->acc_full, turn & 1, ctl, p.status);
      if (!ok) break;
      tc_fence_after();
      for (int b = b0; b < min(b0 + kBatch, mine); ++b) {
        const int g = (mpart + b * mparts) * per + gl;
        const bool live = g < tb.groups && j < p.r;
        const unsigned any = __reduce_or_sync(0xffffffffu, live ? tb.blocks[g] : 0u);
        float* dst = p.part + ((int64_t)split * p.R + row0) * p.r + j;
        for (int c = 0; c < kTile / 16; ++c) {
          if (!(any >> c & 1)) continue;
          uint32_t v[16];
          tmem_ld16_sync(tmem + (b - b0) * kTile + c * 16 + ((uint32_t)(quad * 32) << 16), v);
          const uint4 of = *reinterpret_cast<const uint4*>(tb.slot + c * 16);
#pragma unroll
          for (int i = 0; i < 16; ++i)
            if (live && byte_of(of, i) == g) dst[(c * 16 + i) * p.r] = __uint_as_float(v[i]);
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&ctl->acc_empty);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, 512);
}

// ---- second launch: out = base + B (s h) ----
// Warps 0 (B), 1 (MMAs) and 4-11 (epilogue) meet at each tile, warps 12 and up do not:
// warp 12 streams base.
constexpr int kUpThreads = 416;
constexpr int kUpJoined = 384;
constexpr int kIoWarp = 12;
constexpr int kUpBytes = 65536;    // of 128 outputs by up to 64 ranks of a group a slot
constexpr int kMaxUpSlots = 16;
constexpr int kUpEpi = 8;          // epilogue warps
constexpr int kIoBytes = kTile * kTile * 2;
constexpr int kMaxIo = 3;
constexpr int kAccs = 4;           // accumulators in flight, one group each

struct UpCtl {
  uint64_t full[kMaxUpSlots], empty[kMaxUpSlots];
  uint64_t acc_full[kAccs], acc_empty[kAccs];
  uint64_t io_full[kMaxIo], io_empty[kMaxIo];
  uint64_t drain;
  uint32_t tmem;
  volatile int abort_flag;
};
struct UpShared {
  UpCtl ctl;
  Table table;
  alignas(16) float row_scale[kTile];  // 2^m of each row
  int offsets[kMaxE + 1];
};

struct UpShape {
  int rp;      // r rounded up to 16, 32, 64 or 128
  int splits;  // partial sums of h
  int gparts;  // parts of a tile's groups
  int ntiles;  // of 128 outputs
  int units;   // (tile, part, 128 outputs)
  int nio;     // buffers of base and out; 0: read and written element by element
  int line;    // bytes of a slot's lines: min(64, rp) ranks
  int slots;   // kUpBytes / (128 * line)
};

__device__ __forceinline__ void epilogue_barrier() {
  asm volatile("bar.sync 1, %0;" ::"n"(kUpEpi * 32) : "memory");
}

__device__ __forceinline__ uint16_t to_half_bits(float v, bool bf16) {
  return bf16 ? __bfloat16_as_ushort(__float2bfloat16_rn(v)) : __half_as_ushort(__float2half_rn(v));
}
__device__ __forceinline__ float from_half_bits(uint16_t v, bool bf16) {
  return bf16 ? __uint_as_float((uint32_t)v << 16) : __half2float(__ushort_as_half(v));
}

// The magnitude of v, 0 where it is infinite or NaN.
__device__ __forceinline__ float finite(float v) { return isfinite(v) ? fabsf(v) : 0.0f; }

// The columns' operand: each row's s h in two 16-bit parts, side by side along k
// (ranks [0, rp) the high parts, [rp, 2 rp) the low ones), 128-byte swizzled lines in
// blocks of 64 k.  Eight lanes per row, four ranks a lane and turn.
__device__ __forceinline__ void build_rows(uint8_t* hs, UpShared* sh, const LoraArgs& p, const UpShape& u,
                                           int64_t row0) {
  const Table& tb = sh->table;
  constexpr int kPass = kUpJoined / 8;                   // rows at a time
  constexpr int kTurns = (kTile + kPass - 1) / kPass;
  const int sub = threadIdx.x & 7, first = threadIdx.x >> 3;
  for (int c0 = 0; c0 < u.rp; c0 += 64) {  // (128 ranks: in two halves, the largest of both first)
    float4 v[kTurns][2];
    float s[kTurns], most[kTurns];
    int key[kTurns];
#pragma unroll
    for (int q = 0; q < kTurns; ++q) {
      const int t = first + q * kPass;
      key[q] = t < kTile ? tb.key[t] : -1;
      s[q] = key[q] >= 0 && p.scaling ? p.scaling[key[q] / p.E] : 1.0f;
      most[q] = 0;
    }
    auto fetch = [&](int base) {
#pragma unroll
      for (int q = 0; q < kTurns; ++q)
#pragma unroll
        for (int c = 0; c < 2; ++c) v[q][c] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 2
      for (int k = 0; k < u.splits; ++k)
#pragma unroll
        for (int q = 0; q < kTurns; ++q)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const int j = base + c * 32 + sub * 4;
            if (key[q] < 0 || j >= p.r) continue;
            const float4 w = *reinterpret_cast<const float4*>(
                p.part + ((int64_t)k * p.R + row0 + first + q * kPass) * p.r + j);
            v[q][c].x += w.x;
            v[q][c].y += w.y;
            v[q][c].z += w.z;
            v[q][c].w += w.w;
          }
#pragma unroll
      for (int q = 0; q < kTurns; ++q)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          float4& w = v[q][c];
          w.x *= s[q];
          w.y *= s[q];
          w.z *= s[q];
          w.w *= s[q];
          most[q] = fmaxf(fmaxf(most[q], fmaxf(finite(w.x), finite(w.y))), fmaxf(finite(w.z), finite(w.w)));
        }
    };
    if (u.rp == 128) fetch(64 - c0);
    fetch(c0);
#pragma unroll
    for (int q = 0; q < kTurns; ++q) {
      const int t = first + q * kPass;
#pragma unroll
      for (int o = 4; o; o >>= 1) most[q] = fmaxf(most[q], __shfl_xor_sync(0xffffffffu, most[q], o));
      if (t >= kTile) continue;
      // 2^m with m the exponent of the largest, kept to where 2^m and 2^-m are normal
      const int e = min(max((int)(__float_as_uint(most[q]) >> 23), 1), 253);
      const float up = __uint_as_float((uint32_t)e << 23), down = __uint_as_float((uint32_t)(254 - e) << 23);
      if (sub == 0) sh->row_scale[t] = up;
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int j = c0 + c * 32 + sub * 4;
        if (j >= u.rp) continue;
        const float f[4] = {v[q][c].x * down, v[q][c].y * down, v[q][c].z * down, v[q][c].w * down};
        uint16_t hi[4], lo[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          hi[i] = to_half_bits(f[i], p.bf16);
          const float rest = f[i] - from_half_bits(hi[i], p.bf16);
          lo[i] = to_half_bits(isfinite(rest) ? rest : 0.0f, p.bf16);  // (infinity minus itself)
        }
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const uint16_t* h = half ? lo : hi;
          const int k = j + half * u.rp;
          const int chunk = ((k & 63) >> 3) ^ (t & 7);
          uint2* dst = reinterpret_cast<uint2*>(hs + (k >> 6) * kSlot + t * 128 + chunk * 16 + (k & 7) * 2);
          *dst = make_uint2(h[0] | (uint32_t)h[1] << 16, h[2] | (uint32_t)h[3] << 16);
        }
      }
    }
  }
}

__global__ void __launch_bounds__(kUpThreads, 1)
    lora_up(const __grid_constant__ CUtensorMap map_b, const __grid_constant__ CUtensorMap map_base,
            const __grid_constant__ CUtensorMap map_out, const LoraArgs p, const UpShape u) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* hs = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  uint8_t* slots = hs + ((2 * u.rp + 63) / 64) * kSlot;
  uint8_t* io = slots + kUpBytes;
  UpShared* sh = reinterpret_cast<UpShared*>(io + u.nio * kIoBytes);
  UpCtl* ctl = &sh->ctl;
  const Table& tb = sh->table;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    tma_prefetch_desc(&map_b);
    tma_prefetch_desc(&map_base);
    tma_prefetch_desc(&map_out);
    for (int i = 0; i < u.slots; ++i) {
      mbar_init(&ctl->full[i], 1);
      mbar_init(&ctl->empty[i], 1);
    }
    for (int i = 0; i < kAccs; ++i) {
      mbar_init(&ctl->acc_full[i], 1);
      mbar_init(&ctl->acc_empty[i], kUpEpi);
    }
    for (int i = 0; i < kMaxIo; ++i) {
      mbar_init(&ctl->io_full[i], 1);
      mbar_init(&ctl->io_empty[i], 1);
    }
    mbar_init(&ctl->drain, 1);
    ctl->abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(&ctl->tmem, 512);
    tmem_relinquish();
  }
  mq::pdl_wait();
  mq::pdl_trigger();
  const bool bad = copy_offsets(p, sh->offsets);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ctl->tmem;
  const int kblocks = (u.rp + 63) / 64;  // slots of a group's 128 outputs
  const int ksteps = (p.r + 15) / 16;
  const bool add = p.base != nullptr;

  // This CTA's units, one tile of rows after another.
  const int u0 = (int)((int64_t)u.units * blockIdx.x / gridDim.x);
  const int u1 = (int)((int64_t)u.units * (blockIdx.x + 1) / gridDim.x);
  const int per_part = u.ntiles, per_tile = u.ntiles * u.gparts;
  // each role's place in its rings
  uint32_t w_it = 0, acc_it = 0, io_it = 0;
  bool ok = true;
  if (warp == kIoWarp) {
    // ------------------------------------------------------------- base --
    // Runs ahead of the other warps, over the ends of tiles; so it finds out by itself
    // which tiles have nothing to do.
    const bool el = elect_one();
    for (int un = u0, tile = -1; u.nio && un < u1 && ok; ++un) {
      if (un / per_tile != tile) {
        tile = un / per_tile;
        bool some = false;
        for (int t = lane; t < kTile; t += 32) {
          const int64_t row = (int64_t)tile * kTile + t;
          if (bad || row >= p.R || (p.offsets && (row < sh->offsets[0] || row >= sh->offsets[p.E]))) continue;
          const int l = p.ids[row];
          some |= p.base != p.out || (l >= 0 && l < p.L);
        }
        if (!__any_sync(0xffffffffu, some)) {
          un = min(u1, (tile + 1) * per_tile) - 1;
          continue;
        }
      }
      const uint32_t s = io_it % u.nio;
      ok = warp_wait(&ctl->io_empty[s], ((io_it / u.nio) & 1) ^ 1, ctl, p.status);
      if (!ok) break;
      if (el) {
        if (add) {
          mbar_arrive_expect_tx(&ctl->io_full[s], kIoBytes);
          tma_load_2d(io + s * kIoBytes, &map_base, &ctl->io_full[s], un % per_part * kTile, tile * kTile);
        } else {
          mbar_arrive(&ctl->io_full[s]);
        }
      }
      ++io_it;
    }
    if (ctl->abort_flag)  // loads in flight land before the CTA goes
      for (uint32_t j = io_it < (uint32_t)u.nio ? 0 : io_it - u.nio; j < io_it; ++j)
        wait_drain(&ctl->io_full[j % u.nio], (j / u.nio) & 1);
  }
  for (int ua = u0, ub; ua < u1 && warp != kIoWarp; ua = ub) {
    const int tile = ua / per_tile;
    ub = min(u1, (tile + 1) * per_tile);
    const int64_t row0 = (int64_t)tile * kTile;
    build_table<kUpJoined>(sh->table, p, p.offsets ? sh->offsets : nullptr, bad, tid, tile);
    const bool nothing = tb.inside == 0 || (tb.groups == 0 && p.base == p.out);
    if (nothing) continue;
    build_rows(hs, sh, p, u, row0);
    fence_proxy_async_smem();
    join<kUpJoined>();
    const bool whole = tb.inside == tb.rows && u.gparts == 1;

    if (warp == 0) {
      // ------------------------------------------------------ groups' B --
      const bool el = elect_one();
      for (int un = ua; un < ub && ok; ++un) {
        const int n0 = un % per_part * kTile, part = un % per_tile / per_part;
        const int g0 = tb.groups * part / u.gparts, g1 = tb.groups * (part + 1) / u.gparts;
        for (int g = g0; g < g1 && ok; ++g)
          for (int k = 0; k < kblocks; ++k) {
            const uint32_t s = w_it % u.slots;
            ok = warp_wait(&ctl->empty[s], ((w_it / u.slots) & 1) ^ 1, ctl, p.status);
            if (!ok) break;
            if (el) {
              mbar_arrive_expect_tx(&ctl->full[s], kTile * u.line);
              tma_load_3d(slots + s * kTile * u.line, &map_b, &ctl->full[s], k * 64, n0, tb.group_key[g]);
            }
            ++w_it;
          }
      }
    } else if (warp == 1) {
      // ----------------------------------------------------------- MMAs --
      const bool el = elect_one();
      // Of the columns only those from a group's first block of rows to its last.
      const uint32_t idesc = idesc_16(p.bf16, kTile, 0, false, false);
      const uint32_t hb = smem_addr(hs);
      for (int un = ua; un < ub && ok; ++un) {
        const int part = un % per_tile / per_part;
        const int g0 = tb.groups * part / u.gparts, g1 = tb.groups * (part + 1) / u.gparts;
        for (int g = g0; g < g1 && ok; ++g, ++acc_it) {
          const uint32_t a = acc_it % kAccs;
          const int c0 = __ffs(tb.blocks[g]) - 1, c1 = 32 - __clz(tb.blocks[g]);
          ok = warp_wait(&ctl->acc_empty[a], ((acc_it / kAccs) & 1) ^ 1, ctl, p.status);
          tc_fence_after();
          for (int k = 0; k < kblocks && ok; ++k, ++w_it) {
            const uint32_t s = w_it % u.slots;
            ok = warp_wait(&ctl->full[s], (w_it / u.slots) & 1, ctl, p.status);
            if (!ok) break;
            if (el) {
              const uint64_t ad = smem_desc_k(smem_addr(slots + s * kTile * u.line), u.line);
              for (int j = k * 4; j < min(ksteps, k * 4 + 4); ++j)
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                  const int c = j + half * (u.rp / 16);  // the step's place among the columns' k
                  const uint64_t bd = smem_desc_k_sw128(hb + (c >> 2) * kSlot + c0 * 2048);
                  mma_ss<1>(tmem + a * kTile + c0 * 16, ad + (j & 3) * 2, bd + (c & 3) * 2,
                            idesc | (uint32_t)(c1 - c0) * 2 << 17, j | half);
                }
              mma_commit(&ctl->empty[s]);
            }
          }
          if (ok && el) mma_commit(&ctl->acc_full[a]);
        }
      }
    } else if (warp >= 4) {
      // ------------------------------------------------------- epilogue --
      // A lane is an output, the columns are the rows.
      const int quad = warp & 3, half = (warp - 4) >> 2;
      const bool bf = p.out_dtype == MQ_DTYPE_BF16;
      for (int un = ua; un < ub; ++un) {
        const int n0 = un % per_part * kTile, part = un % per_tile / per_part;
        const int g0 = tb.groups * part / u.gparts, g1 = tb.groups * (part + 1) / u.gparts;
        const int n = n0 + quad * 32 + lane;
        uint16_t* buf = nullptr;
        const uint32_t s = u.nio ? io_it % u.nio : 0;
        if (u.nio) {
          ok = ok && warp_wait(&ctl->io_full[s], (io_it / u.nio) & 1, ctl, p.status);
          buf = reinterpret_cast<uint16_t*>(io + s * kIoBytes) + quad * 32 + lane;
        }
        for (int g = g0; g < g1 && ok; ++g, ++acc_it) {
          const uint32_t a = acc_it % kAccs;
          ok = warp_wait(&ctl->acc_full[a], (acc_it / kAccs) & 1, ctl, p.status);
          if (!ok) break;
          tc_fence_after();
          const unsigned blocks = tb.blocks[g];
          for (int c = half; c < kTile / 16; c += 2) {
            if (!(blocks >> c & 1)) continue;
            uint32_t v[16];
            tmem_ld16_sync(tmem + a * kTile + c * 16 + ((uint32_t)(quad * 32) << 16), v);
            const uint4 of = *reinterpret_cast<const uint4*>(tb.slot + c * 16);
            const float4* up = reinterpret_cast<const float4*>(sh->row_scale + c * 16);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float4 f = up[i];
              v[4 * i] = __float_as_uint(__uint_as_float(v[4 * i]) * f.x);
              v[4 * i + 1] = __float_as_uint(__uint_as_float(v[4 * i + 1]) * f.y);
              v[4 * i + 2] = __float_as_uint(__uint_as_float(v[4 * i + 2]) * f.z);
              v[4 * i + 3] = __float_as_uint(__uint_as_float(v[4 * i + 3]) * f.w);
            }
            if (u.nio) {
              uint16_t* col = buf + c * 16 * kTile;
              uint16_t old[16];
#pragma unroll
              for (int i = 0; i < 16; ++i) old[i] = add ? col[i * kTile] : (uint16_t)0;
#pragma unroll
              for (int i = 0; i < 16; ++i)
                old[i] = to_half_bits(from_half_bits(old[i], bf) + __uint_as_float(v[i]), bf);
#pragma unroll
              for (int i = 0; i < 16; ++i)
                if (byte_of(of, i) == g) col[i * kTile] = old[i];
            } else if (n < p.N) {
#pragma unroll
              for (int i = 0; i < 16; ++i) {
                if (byte_of(of, i) != g) continue;
                const int64_t row = row0 + c * 16 + i;
                const float o = add ? load_as(p.base, p.out_dtype, row * p.base_stride + n) : 0.0f;
                store_out(p.out, p.out_dtype, row * p.out_stride + n, o + __uint_as_float(v[i]));
              }
            }
            __syncwarp();
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&ctl->acc_empty[a]);
        }
        // rows without an adapter: base as it is, or 0
        const bool copies = part == 0 && p.base != p.out;
        if (u.nio) {
          if (!add && part == 0)
            for (int t = half; t < tb.rows; t += 2)
              if (tb.slot[t] == kNone) buf[t * kTile] = 0;
          fence_proxy_async_smem();
          epilogue_barrier();
          if (whole) {
            if (warp == 4 && lane == 0) {
              if (ok) tma_store_2d(&map_out, io + s * kIoBytes, n0, (int)row0);
              bulk_commit();
              // the store before this one has read its buffer
              bulk_wait_read<1>();
              if (un > ua) mbar_arrive(&ctl->io_empty[(io_it - 1) % u.nio]);
            }
          } else {
            const int live = min(kTile, p.N - n0);  // (a multiple of 8)
            for (int t = warp - 4; t < tb.rows && ok; t += kUpEpi) {
              const int sl = tb.slot[t];
              const bool write = sl == kNone ? copies : sl != kOut && sl >= g0 && sl < g1;
              if (!write || lane * 4 >= live) continue;
              const uint2 q = *reinterpret_cast<const uint2*>(io + s * kIoBytes + t * kTile * 2 + lane * 8);
              *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.out) + (row0 + t) * p.out_stride + n0 + lane * 4) = q;
            }
            epilogue_barrier();
            if (warp == 4 && lane == 0) mbar_arrive(&ctl->io_empty[s]);
          }
          ++io_it;
        } else if (copies) {
          for (int t = half; t < tb.rows; t += 2)
            if (tb.slot[t] == kNone && n < p.N)
              copy_element(p.out, (row0 + t) * p.out_stride + n, p.base, (row0 + t) * p.base_stride + n,
                           p.out_dtype);
        }
      }
      if (u.nio && whole && warp == 4 && lane == 0) {
        bulk_wait_read<0>();
        mbar_arrive(&ctl->io_empty[(io_it - 1) % u.nio]);
      }
    }
    __syncwarp();
  }
  if (warp == 0 && ctl->abort_flag)  // loads in flight land before the CTA goes
    for (uint32_t j = w_it < (uint32_t)u.slots ? 0 : w_it - u.slots; j < w_it; ++j)
      wait_drain(&ctl->full[j % u.slots], (j / u.slots) & 1);
  if (warp == 1) {
    if (elect_one()) mma_commit(&ctl->drain);
    __syncwarp();
    wait_drain(&ctl->drain, 0);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, 512);
}

// ------------------------------------------------------------ host side --
int padded_rank(int r) { return r <= 16 ? 16 : r <= 32 ? 32 : r <= 64 ? 64 : 128; }

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

template <bool BF16>
cudaError_t launch_rows(const LoraArgs& g, cudaStream_t st) {
  const dim3 grid((unsigned)g.R * kCluster), block(kRowThreads);
  if (g.r <= 8) return launch_pdl_cluster(lora_rows<BF16, 1>, grid, block, kCluster, 0, st, g);
  if (g.r <= 16) return launch_pdl_cluster(lora_rows<BF16, 2>, grid, block, kCluster, 0, st, g);
  if (g.r <= 32) return launch_pdl_cluster(lora_rows<BF16, 4>, grid, block, kCluster, 0, st, g);
  if (g.r <= 64) return launch_pdl_cluster(lora_rows<BF16, 8>, grid, block, kCluster, 0, st, g);
  return launch_pdl_cluster(lora_rows<BF16, 16>, grid, block, kCluster, 0, st, g);
}

cudaError_t launch_down(const LoraArgs& g, const LoraPlan& pl, cudaStream_t st) {
  const CUtensorMapDataType dt = g.bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
  const int rp = padded_rank(g.r);
  CUtensorMap mx, ma;
  const cuuint64_t xd[2] = {(cuuint64_t)g.K, (cuuint64_t)g.R}, xs = 2 * (cuuint64_t)g.x_stride;
  const cuuint32_t xb[2] = {64, kTile};
  cudaError_t err = make_map(&mx, dt, 2, g.x, xd, &xs, xb);
  if (err != cudaSuccess) return err;
  const cuuint64_t ad[3] = {(cuuint64_t)g.K, (cuuint64_t)g.r, (cuuint64_t)g.L * g.E};
  const cuuint64_t as[2] = {2 * (cuuint64_t)g.K, 2 * (cuuint64_t)g.K * g.r};
  const cuuint32_t ab[3] = {64, (cuuint32_t)rp, 1};
  err = make_map(&ma, dt, 3, g.a, ad, as, ab);
  if (err != cudaSuccess) return err;
  constexpr size_t smem = 1024 + kDownSlots * kSlot + sizeof(DownShared);
  static_assert(smem <= kSmemMax, "shared memory");
  static std::atomic<uint64_t> ready{0};
  err = allow_smem(lora_down, smem, ready);
  if (err != cudaSuccess) return err;
  const int64_t tiles = (g.R + kTile - 1) / kTile;
  return launch_pdl(lora_down, dim3((unsigned)(tiles * pl.splits * pl.mparts)), dim3(kDownThreads), smem, st, mx,
                    ma, g, rp, pl.splits, pl.mparts);
}

cudaError_t launch_up(const LoraArgs& g, const LoraPlan& pl, cudaStream_t st) {
  const CUtensorMapDataType dt = g.bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
  UpShape u;
  u.rp = padded_rank(g.r);
  u.splits = pl.splits;
  u.gparts = pl.gparts;
  u.ntiles = (g.N + kTile - 1) / kTile;
  u.units = (int)((g.R + kTile - 1) / kTile) * u.ntiles * u.gparts;
  // base and out by TMA: 16 bits, rows on 16-byte boundaries
  const bool base_ok = !g.base || (g.base_stride % 8 == 0 && (reinterpret_cast<uintptr_t>(g.base) & 15u) == 0);
  const bool tma = g.out_dtype != MQ_DTYPE_F32 && base_ok && g.out_stride % 8 == 0 && g.N % 8 == 0 &&
                   (reinterpret_cast<uintptr_t>(g.out) & 15u) == 0;
  u.nio = !tma ? 0 : u.rp == 128 ? 2 : kMaxIo;
  u.line = std::min(u.rp, 64) * 2;
  u.slots = std::min(kMaxUpSlots, kUpBytes / (kTile * u.line));
  CUtensorMap mb, mbase, mout;
  const cuuint64_t bd[3] = {(cuuint64_t)g.r, (cuuint64_t)g.N, (cuuint64_t)g.L * g.E};
  const cuuint64_t bs[2] = {2 * (cuuint64_t)g.r, 2 * (cuuint64_t)g.r * g.N};
  const cuuint32_t bb[3] = {(cuuint32_t)u.line / 2, kTile, 1};
  cudaError_t err = make_map(&mb, dt, 3, g.b, bd, bs, bb,
                             u.line == 128  ? CU_TENSOR_MAP_SWIZZLE_128B
                             : u.line == 64 ? CU_TENSOR_MAP_SWIZZLE_64B
                                            : CU_TENSOR_MAP_SWIZZLE_32B);
  if (err != cudaSuccess) return err;
  mbase = mout = mb;
  if (tma) {
    const CUtensorMapDataType ot =
        g.out_dtype == MQ_DTYPE_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
    const cuuint64_t d[2] = {(cuuint64_t)g.N, (cuuint64_t)g.R};
    const cuuint64_t s0 = 2 * (cuuint64_t)g.base_stride, s1 = 2 * (cuuint64_t)g.out_stride;
    const cuuint32_t box[2] = {kTile, kTile};
    err = make_map(&mout, ot, 2, g.out, d, &s1, box, CU_TENSOR_MAP_SWIZZLE_NONE);
    if (err == cudaSuccess && g.base) err = make_map(&mbase, ot, 2, g.base, d, &s0, box, CU_TENSOR_MAP_SWIZZLE_NONE);
    if (err != cudaSuccess) return err;
  }
  constexpr size_t most = 1024 + 4 * kSlot + kUpBytes + 2 * kIoBytes + sizeof(UpShared);
  constexpr size_t most3 = 1024 + 2 * kSlot + kUpBytes + 3 * kIoBytes + sizeof(UpShared);
  static_assert(most <= kSmemMax && most3 <= kSmemMax, "shared memory");
  const size_t need = 1024 + (2 * u.rp + 63) / 64 * kSlot + kUpBytes + (size_t)u.nio * kIoBytes + sizeof(UpShared);
  const size_t smem = std::max<size_t>(need, 120 * 1024);  // one CTA per SM: each allocates all of tensor memory
  static std::atomic<uint64_t> ready{0};
  err = allow_smem(lora_up, kSmemMax, ready);
  if (err != cudaSuccess) return err;
  const int grid = std::min(u.units, tc_num_sms());
  return launch_pdl(lora_up, dim3(grid), dim3(kUpThreads), smem, st, mb, mbase, mout, g, u);
}

}  // namespace

LoraPlan lora_plan(int64_t R, int K, int N, int r, int L, int E) {
  LoraPlan pl = {};
  const int sms = tc_num_sms();
  const double adapter = 2.0 * r * ((double)K + N);                     // bytes
  const double groups = std::min<double>((double)R, (double)L * E);    // at most
  pl.splits = pl.mparts = pl.gparts = 1;
  pl.rows = R <= 1024 && R * adapter <= 48e6 + groups * adapter;
  if (pl.rows) return pl;
  const int64_t tiles = (R + kTile - 1) / kTile;
  const int per = kTile / padded_rank(r);
  const int tile_groups = (int)std::min<double>(kTile, groups);
  const int accs = (tile_groups + per - 1) / per;
  const int stages = (K + 63) / 64;
  pl.splits = (int)std::max<int64_t>(1, std::min<int64_t>({16, stages / 4, sms / tiles}));
  pl.mparts = (int)std::max<int64_t>(1, std::min<int64_t>(accs, sms / (tiles * pl.splits)));
  const int ntiles = (N + kTile - 1) / kTile;
  while (pl.gparts * 2 <= tile_groups && tiles * ntiles * pl.gparts * 2 <= sms) pl.gparts *= 2;
  return pl;
}

cudaError_t launch_lora(const LoraArgs& g, const LoraPlan& pl, int which, cudaStream_t st) {
  if (pl.rows) return g.bf16 ? launch_rows<true>(g, st) : launch_rows<false>(g, st);
  return which == 0 ? launch_down(g, pl, st) : launch_up(g, pl, st);
}
