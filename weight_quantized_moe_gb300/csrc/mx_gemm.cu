// Rows grouped by expert times 4-bit microscaled weights, on the block-scaled
// tensor-core instructions.
//
//   out[r, n] = sum_k A[r, k] * W[e(r), n, k]
//
// A: E4M3 or E2M1 rows, W: E2M1 [E, N, K], each with one E8M0 scale per 32
// consecutive k.  tcgen05.mma takes the codes and the scales as they are and
// accumulates in float32, so nothing is converted on the way.
//
// One persistent CTA per SM.  D[weight rows x rows of A]: the weights are the
// instruction's A operand (128 rows) and the token rows its B operand (as many
// columns as a chunk has rows, in steps of 16), so that a few rows cost a narrow
// instruction and no padding.  A unit is (expert, chunk of at most BN rows, 256
// weight rows, K split); when gated the 256 are 128 gate rows and their up rows.
//
// Two shapes (CG):
//   1  A CTA holds both 128-row tiles of a unit, BN <= 96.  For experts with few
//      rows: the weight stream bounds these (128 rows, E=8, K=4096, N=28672:
//      82 us, 91 % of the HBM's rate; 76 us, 99 %, with 4-bit rows).
//   2  A pair of CTAs (cta_group::2) holds the unit, 128 weight rows and half of
//      its 224 rows of A in each.  An instruction reads its operands from shared
//      memory at 64 bytes per cycle (measured: 64 cycles for 128 weight rows and
//      half a cycle per column), so a wide tile whose columns are split over two
//      SMs comes nearest the arithmetic rate.  8192 x 4096 x 28672: 595 us (3.2
//      PFLOP/s; at 1370 W the clock falls to 1.46 GHz, at 2.07 GHz it takes 525),
//      373 us (5.2 PFLOP/s) with 4-bit rows.
//
// Roles: warp 0 streams codes by TMA; warps 1-2 issue the MMAs (of a pair: warp 1
// of its first CTA); warps 3 and 12-14 bring the scales; warps 4-11 are the
// epilogue.
//   * Codes.  A stage holds 128 bytes of each row, 128-byte swizzled: 128 k of
//     E4M3 rows against 128 k of weights whose nibbles TMA spreads to 16-byte
//     groups (the operand form of the mixed 8/4-bit instruction), or 256 k of
//     both in 4 bits.  Four MMAs per stage and weight tile either way.
//   * Scales.  The instruction reads them from tensor memory, 4 scale bytes
//     (128 k, a "word") per row, row r in lane r % 32 and column r / 32.  The
//     scale warps read the rows' scale bytes (16 bytes = 512 k per row), and
//     write them to shared memory as that [32 lanes][4 columns] block for each
//     word; an MMA warp copies a block to tensor memory with one tcgen05.cp,
//     which the MMAs that follow it in the same thread see.
//   * Epilogue.  A thread is one weight row (tensor-memory lane) and walks the
//     columns, the rows of A.  32 lanes are 32 consecutive outputs: exactly
//     one block when the activations are requantised.  Two accumulator buffers:
//     the next unit's MMAs run meanwhile.
#include "mx.cuh"
#include "sm100_ptx.cuh"

#include <cudaTypedefs.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <mutex>

namespace {

using namespace mq::ptx;

constexpr int kTileM = 128;
constexpr int kABytes = kTileM * 128;  // one weight tile of a stage
constexpr int kThreads = 480;
constexpr int kSfWarps = 4;            // warps 3 and 12-14
constexpr int kEpiWarps = 8;
constexpr int kMaxStages = 12;
constexpr int kSfRing = 4;             // scale slots, 512 k each
// A slot is filled by one warp only: with more warps than slots one could be two
// turns ahead of the barrier's phase, which its parity cannot tell from none.
static_assert(kSfRing == kSfWarps, "one warp per scale slot");
constexpr int kMaxE = 1024;
constexpr int kPairRows = 224;         // rows per tile of a CTA pair
constexpr int kUnitList = 128;         // units of a CTA that are decoded at its start
constexpr int kGroup = 8;              // weight tiles that a chunk walk shares
constexpr unsigned long long kWaitNs = 1000000000ull;
constexpr size_t kSmemMax = 227 * 1024;

template <int BITS, int BN, int CG, int EPI>
struct Cfg {
  static constexpr int kTiles = CG == 2 ? 1 : 2;    // weight tiles of a unit, one MMA warp each
  static constexpr int kWords = BITS == 8 ? 1 : 2;  // 128-k scale words per stage
  static constexpr int kPerSb = 4 / kWords;         // stages per scale slot
  static constexpr int kBRows = BN / CG;            // rows of A (operand B) in each CTA
  static constexpr int kBBytes = kBRows * 128;
  static constexpr int kStageBytes = kTiles * kABytes + kBBytes;
  // bytes TMA reports for a stage's weights: those it reads, so half a tile
  // where it spreads the nibbles
  static constexpr int kTxWeights = kTiles * (BITS == 8 ? kABytes / 2 : kABytes);
  static constexpr int kBBlocks = (BN + 127) / 128;
  static constexpr int kSfWordBytes = (kTiles + kBBlocks) * 512;
  static constexpr int kSfSlotBytes = 4 * kSfWordBytes;
  // tensor-memory columns of one MMA warp's scales: its tile's and the rows'
  static constexpr int kSfCols = 4 * (1 + kBBlocks) * 4;
  static constexpr int kAccCols = kTiles * BN;
  static constexpr int kBufs = 2;
  static constexpr int kSfBase = kBufs * kAccCols;
  static_assert(kSfBase + kTiles * kSfCols <= 512, "tensor memory");
  // epilogue: where each column goes; gate and up values that change warps
  static constexpr int kDestBytes = EPI == MX_EPI_PART ? 2 * BN * 16 : 0;
  static constexpr int kSwapBytes = EPI == MX_EPI_GATED && CG == 2 ? 2 * kEpiWarps * 1024 : 0;
  static constexpr size_t kFixed = 1024 + (size_t)kSfRing * kSfSlotBytes + 1024 + kUnitList * 16 +
                                   kDestBytes + kSwapBytes + (kMaxE + 1) * 4;
  // 4-bit rows: a stage holds twice the weights, and four stages measured
  // faster than the five or six that fit (64 tokens, E=8: 137 -> 130 us; 8192
  // rows 386 -> 373)
  static constexpr int kFit = (int)((kSmemMax - kFixed) / kStageBytes);
  static constexpr int kWant = BITS == 4 && kFit > 4 ? 4 : kFit;
  static constexpr int kStages = kWant < kMaxStages ? kWant : kMaxStages;
  static_assert(kStages >= 2, "shared memory");
  // one CTA per SM: each allocates all of tensor memory
  static constexpr size_t kNeed = kFixed + (size_t)kStages * kStageBytes;
  static constexpr size_t kSmem = kNeed < 120 * 1024 ? 120 * 1024 : kNeed;
};

struct Ctl {
  uint64_t full[kMaxStages], empty[kMaxStages];
  uint64_t sf_full[kSfRing], sf_empty[kSfRing];
  uint64_t acc_full[2], acc_empty[2];
  uint64_t drain;
  uint32_t tmem;
  volatile int abort_flag;
};
static_assert(sizeof(Ctl) <= 1024, "control block");

struct Params {
  const uint8_t* w_scale;
  const uint8_t* a_scale;
  const int32_t* seg_start;
  const int32_t* seg_count;
  int E, K, N, R;
  int mrows;      // outputs of a unit
  int rank_rows;  // of them in each CTA of a pair
  int box_rows;   // weight rows of one load
  int up_row;     // weight row of a unit's second load, relative to its first
  int wrows;
  int mtiles, splits, words, sbs;
  bool evict_first;  // L2 policy of weights that are read once
  void* out;
  int out_dtype;
  float* part;
  int64_t part_rows;
  const int32_t* dest;
  const float* dest_w;
  uint8_t* act;
  uint8_t* act_scale;
  unsigned* status;
};

struct Unit {
  int e, row0, n, m, split;  // expert, first row, rows, first output, K split
  bool single;               // the expert has one chunk: its weights are read once
};

// Rows of expert e, kept inside [0, R) whatever the arrays hold; false where
// that took a correction.
__device__ __forceinline__ bool segment(const Params& p, int e, int& start, int& count) {
  if (!p.seg_start) {
    start = 0;
    count = p.R;
    return true;
  }
  const int s = p.seg_start[e];
  const int64_t end = p.seg_count ? (int64_t)s + p.seg_count[e] : p.seg_start[e + 1];
  start = min(max(s, 0), p.R);
  count = (int)(min(max(end, (int64_t)start), (int64_t)p.R) - start);
  return start == s && start + (int64_t)count == end;
}

// Unit u of the walk: expert by expert, groups of kGroup weight tiles, every
// chunk over a group before the next one (the CTAs at work share the group's
// weights and the chunks' rows in L2), K splits innermost.
template <int BN>
__device__ __forceinline__ Unit decode_unit(const Params& p, const int* chunk_start, uint32_t u) {
  const uint32_t per = p.mtiles * p.splits;
  const int g = (int)(u / per);  // a chunk's position in the walk locates its expert
  int lo = 0, hi = p.E;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (chunk_start[mid] <= g) lo = mid;
    else hi = mid;
  }
  Unit w;
  w.e = lo;
  const uint32_t nch = chunk_start[lo + 1] - chunk_start[lo];
  const uint32_t r = u - chunk_start[lo] * per;
  const uint32_t per_group = kGroup * nch * p.splits;
  const uint32_t grp = r / per_group;
  const uint32_t rem = r - grp * per_group;
  const uint32_t tiles = min(kGroup, p.mtiles - (int)grp * kGroup) * p.splits;
  const uint32_t c = rem / tiles;
  const uint32_t t = rem - c * tiles;
  w.m = (int)(grp * kGroup + t / p.splits) * p.mrows;
  w.split = (int)(t % p.splits);
  int start, count;
  segment(p, lo, start, count);
  w.row0 = start + (int)c * BN;
  w.n = min(BN, count - (int)c * BN);
  w.single = nch == 1;
  return w;
}

// The i-th unit of this CTA: from the list in shared memory (decoded once, by
// all threads at a time), past its end on the spot.
template <int BN, int CG>
__device__ __forceinline__ Unit unit_at(const Params& p, const int* chunk_start, const int4* list,
                                        uint32_t i) {
  if (i >= kUnitList) {
    Unit w = decode_unit<BN>(p, chunk_start, blockIdx.x / CG + i * (gridDim.x / CG));
    if (CG == 2) w.m += (int)cluster_rank() * p.rank_rows;
    return w;
  }
  const int4 v = list[i];
  Unit w;
  w.e = v.x & 0xffff;
  w.single = (v.x >> 16) & 1;
  w.split = v.x >> 17;
  w.row0 = v.y;
  w.n = v.z;
  w.m = v.w;
  return w;
}

template <int CG>
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
template <int CG = 1>
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

// Columns of the instruction for a chunk of n rows: n in steps of 16 for each
// CTA (32 for a pair), at most the tile's.
template <int CG>
__device__ __forceinline__ int columns(int n, int bn) {
  return min(bn, (n + 16 * CG - 1) & -(16 * CG));
}
// Rows of the boxes that load a partly filled chunk.
template <int CG>
constexpr int kPartRows = CG == 2 ? 16 : 32;

// After an abort: lets what is in flight land; bounded, ignores the flag.
__device__ __forceinline__ void wait_drain(uint64_t* bar, uint32_t parity) {
  const unsigned long long t0 = mq::global_timer_ns();
  while (!mbar_try_wait(bar, parity))
    if (mq::global_timer_ns() - t0 > kWaitNs) return;
}

// Four scale words (512 k) of one row from word w0 on; words past the row's
// end are 0 (their codes are 0 too).
__device__ __forceinline__ uint4 load_words(const uint8_t* row, int w0, int words) {
  const uint8_t* p = row + (int64_t)w0 * 4;
  if ((words & 3) == 0) return __ldg(reinterpret_cast<const uint4*>(p));
  uint4 v = make_uint4(0, 0, 0, 0);
  if ((words & 1) == 0) {
    if (w0 < words) {
      const uint2 a = __ldg(reinterpret_cast<const uint2*>(p));
      v.x = a.x;
      v.y = a.y;
    }
    if (w0 + 2 < words) {
      const uint2 a = __ldg(reinterpret_cast<const uint2*>(p) + 1);
      v.z = a.x;
      v.w = a.y;
    }
    return v;
  }
  const uint32_t* q = reinterpret_cast<const uint32_t*>(p);
  if (w0 < words) v.x = __ldg(q);
  if (w0 + 1 < words) v.y = __ldg(q + 1);
  if (w0 + 2 < words) v.z = __ldg(q + 2);
  if (w0 + 3 < words) v.w = __ldg(q + 3);
  return v;
}

// Joins the epilogue warps.
__device__ __forceinline__ void epilogue_barrier() {
  asm volatile("bar.sync 1, %0;" ::"n"(kEpiWarps * 32) : "memory");
}

// Joins the gate warp and the up warp of one pair of lane quarters.
__device__ __forceinline__ void swap_barrier(int pair) {
  asm volatile("bar.sync %0, 64;" ::"r"(2 + pair) : "memory");
}

__device__ __forceinline__ void store_out(void* out, int dtype, int64_t i, float v) {
  if (dtype == MQ_DTYPE_BF16) static_cast<__nv_bfloat16*>(out)[i] = __float2bfloat16_rn(v);
  else if (dtype == MQ_DTYPE_F16) static_cast<__half*>(out)[i] = __float2half_rn(v);
  else static_cast<float*>(out)[i] = v;
}

template <int BITS, int BN, int EPI, int CG>
__global__ void __launch_bounds__(kThreads, 1)
    mx_gemm(const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_a,
            const __grid_constant__ CUtensorMap map_part, const Params p) {
  using C = Cfg<BITS, BN, CG, EPI>;
  constexpr int kTiles = C::kTiles;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  uint8_t* stages = smem;
  uint8_t* sf = stages + (size_t)C::kStages * C::kStageBytes;
  Ctl* ctl = reinterpret_cast<Ctl*>(sf + (size_t)kSfRing * C::kSfSlotBytes);
  int4* list = reinterpret_cast<int4*>(reinterpret_cast<uint8_t*>(ctl) + 1024);
  int4* dest_table = list + kUnitList;  // [2][BN]
  float* swap = reinterpret_cast<float*>(reinterpret_cast<uint8_t*>(dest_table) + C::kDestBytes);  // [2][kEpiWarps][8][32]
  int* chunk_start = reinterpret_cast<int*>(reinterpret_cast<uint8_t*>(swap) + C::kSwapBytes);
  const int tid = threadIdx.x;
  const int warp = tid >> 5;
  const int lane = tid & 31;
  const uint32_t rank = CG == 2 ? cluster_rank() : 0;  // 0 issues the pair's MMAs
  const uint32_t worker = blockIdx.x / CG, workers = gridDim.x / CG;

  if (tid == 0) {
    tma_prefetch_desc(&map_w);
    tma_prefetch_desc(&map_a);
    tma_prefetch_desc(&map_part);
    for (int i = 0; i < C::kStages; ++i) {
      mbar_init(&ctl->full[i], 1);
      mbar_init(&ctl->empty[i], kTiles);
    }
    for (int i = 0; i < kSfRing; ++i) {
      mbar_init(&ctl->sf_full[i], CG);
      mbar_init(&ctl->sf_empty[i], kTiles);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&ctl->acc_full[i], kTiles);
      mbar_init(&ctl->acc_empty[i], CG * kEpiWarps);
    }
    mbar_init(&ctl->drain, kTiles);
    ctl->abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    if (CG == 2) {
      tmem_alloc_pair(&ctl->tmem, 512);
      tmem_relinquish_pair();
    } else {
      tmem_alloc(&ctl->tmem, 512);
      tmem_relinquish();
    }
  }
  mq::pdl_wait();
  mq::pdl_trigger();
  // Chunks of each expert, scanned; then this CTA's units.
  bool fine = true;
  for (int e = tid; e < p.E; e += kThreads) {
    int start, count;
    fine &= segment(p, e, start, count);
    chunk_start[e] = (count + BN - 1) / BN;
  }
  // offsets that fall or leave [0, R]: nothing is computed
  const bool bad = __syncthreads_or(!fine);
  if (bad && tid == 0 && blockIdx.x == 0) mq::flag(p.status, MQ_DEV_BAD_OFFSETS);
  if (warp == 0) {
    int run = 0;
    for (int e0 = 0; e0 < p.E; e0 += 32) {
      const int e = e0 + lane;
      const int mine = e < p.E ? chunk_start[e] : 0;
      int incl = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int t = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += t;
      }
      if (e < p.E) chunk_start[e] = run + incl - mine;
      run += __shfl_sync(0xffffffffu, incl, 31);
    }
    if (lane == 0) chunk_start[p.E] = run;
  }
  __syncthreads();
  const uint32_t total = bad ? 0 : (uint32_t)chunk_start[p.E] * p.mtiles * p.splits;
  const uint32_t units = worker < total ? (total - worker + workers - 1) / workers : 0;
  if (tid < kUnitList && tid < units) {
    const Unit w = decode_unit<BN>(p, chunk_start, worker + tid * workers);
    list[tid] = make_int4(w.e | (w.single ? 1 << 16 : 0) | w.split << 17, w.row0, w.n,
                          w.m + (int)rank * p.rank_rows);
  }
  tc_fence_before();
  if (CG == 2) cluster_sync();  // (the barriers are set up in both)
  else __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ctl->tmem;

  if (warp == 0) {
    // ---------------------------------------------------------- codes --
    const bool el = elect_one();
    const uint64_t pol_once = l2_policy_evict_first();
    uint32_t it = 0;
    bool ok = true;
    for (uint32_t u = 0; u < units && ok; ++u) {
      const Unit w = unit_at<BN, CG>(p, chunk_start, list, u);
      const int sb0 = (int)((int64_t)p.sbs * w.split / p.splits);
      const int sb1 = (int)((int64_t)p.sbs * (w.split + 1) / p.splits);
      // a partly filled chunk: as many boxes of kPartRows rows as its columns
      // (CG = 2: each CTA brings its half of them)
      const int n_cols = columns<CG>(w.n, BN);
      const int rows = n_cols == BN ? C::kBRows : (n_cols / CG + kPartRows<CG> - 1) / kPartRows<CG> * kPartRows<CG>;
      const int row0 = w.row0 + (int)rank * (n_cols / CG);
      const int st0 = sb0 * C::kPerSb;
      const int st1 = min(sb1 * C::kPerSb, (p.words + C::kWords - 1) / C::kWords);
      for (int s = st0; s < st1; ++s, ++it) {
        const uint32_t slot = it % C::kStages;
        if (!warp_wait(&ctl->empty[slot], ((it / C::kStages) & 1) ^ 1, ctl, p.status)) {
          ok = false;
          break;
        }
        uint8_t* dst = stages + (size_t)slot * C::kStageBytes;
        uint8_t* dst_a = dst + kTiles * kABytes;
        if (el) {
          if (rank == 0) mbar_arrive_expect_tx(&ctl->full[slot], CG * (C::kTxWeights + rows * 128));
          if constexpr (CG == 2) {
            const uint32_t bar = map_rank(&ctl->full[slot], 0);
            tma_load_3d_pair(dst, &map_w, bar, s * 128, w.m, w.e);
            if (EPI == MX_EPI_GATED)  // 64 gate rows and their 64 up rows
              tma_load_3d_pair(dst + kABytes / 2, &map_w, bar, s * 128, w.m + p.up_row, w.e);
            if (n_cols == BN) {
              tma_load_2d_pair(dst_a, &map_a, bar, s * 128, row0);
            } else {
              for (int r = 0; r < rows; r += kPartRows<CG>)
                tma_load_2d_pair(dst_a + r * 128, &map_part, bar, s * 128, row0 + r);
            }
          } else {
#pragma unroll
            for (int a = 0; a < kTiles; ++a) {
              const int row = w.m + a * p.up_row;
              if (w.single && p.evict_first)
                tma_load_3d_hint(dst + a * kABytes, &map_w, &ctl->full[slot], s * 128, row, w.e, pol_once);
              else
                tma_load_3d(dst + a * kABytes, &map_w, &ctl->full[slot], s * 128, row, w.e);
            }
            if (n_cols == BN) {
              tma_load_2d(dst_a, &map_a, &ctl->full[slot], s * 128, row0);
            } else {
              for (int r = 0; r < rows; r += kPartRows<CG>)
                tma_load_2d(dst_a + r * 128, &map_part, &ctl->full[slot], s * 128, row0 + r);
            }
          }
        }
      }
    }
    if (ctl->abort_flag && rank == 0) {  // loads in flight land before the CTA goes
      for (uint32_t j = it < (uint32_t)C::kStages ? 0 : it - C::kStages; j < it; ++j)
        wait_drain(&ctl->full[j % C::kStages], (j / C::kStages) & 1);
    }
  } else if (warp <= kTiles && rank == 0) {
    // ----------------------------------------------------------- MMAs --
    // Bound by operand reads (64 bytes per cycle) where rows are many, else by
    // the weight stream.  One warp per weight tile: an instruction takes about 90 cycles to issue
    // whatever its width, two warps issue at once.  The warp walks the loop
    // together and one elected lane issues, so that the descriptors stay in
    // uniform registers (a lone lane takes three times as long).
    const int tile = warp - 1;
    const bool el = elect_one();
    const int nst = (p.words + C::kWords - 1) / C::kWords;
    const uint32_t sfc = tmem + C::kSfBase + tile * C::kSfCols;  // [word][tile, rows] x 4 columns
    uint32_t it = 0, sb_it = 0;
    bool ok = true;
    for (uint32_t t = 0; t < units && ok; ++t) {
      const Unit w = unit_at<BN, CG>(p, chunk_start, list, t);
      const int sb0 = (int)((int64_t)p.sbs * w.split / p.splits);
      const int sb1 = (int)((int64_t)p.sbs * (w.split + 1) / p.splits);
      const uint32_t buf = t % C::kBufs;
      ok = warp_wait<CG>(&ctl->acc_empty[buf], ((t / C::kBufs) & 1) ^ 1, ctl, p.status);
      tc_fence_after();
      const uint32_t acc = tmem + buf * C::kAccCols + tile * BN;
      const uint32_t idesc = idesc_mx<BITS>(CG * kTileM, columns<CG>(w.n, BN), 0);
      uint32_t accumulate = 0;
      for (int sb = sb0; sb < sb1 && ok; ++sb, ++sb_it) {
        const uint32_t ss = sb_it % kSfRing;
        ok = warp_wait<CG>(&ctl->sf_full[ss], (sb_it / kSfRing) & 1, ctl, p.status);
        if (!ok) break;
        if (el) {
          const uint32_t slot = smem_addr(sf + (size_t)ss * C::kSfSlotBytes);
#pragma unroll
          for (int wd = 0; wd < 4; ++wd) {
            const uint32_t blk = slot + wd * C::kSfWordBytes;
            const uint32_t col = sfc + wd * (1 + C::kBBlocks) * 4;
            tmem_cp_scales<CG>(col, smem_desc_scales(blk + tile * 512));
#pragma unroll
            for (int b = 0; b < C::kBBlocks; ++b)
              tmem_cp_scales<CG>(col + 4 + b * 4, smem_desc_scales(blk + (kTiles + b) * 512));
          }
        }
        const int last = min((sb + 1) * C::kPerSb, nst);
        for (int s = sb * C::kPerSb; s < last; ++s, ++it) {
          const uint32_t slot = it % C::kStages;
          ok = warp_wait(&ctl->full[slot], (it / C::kStages) & 1, ctl, p.status);
          if (!ok) break;
          if (el) {
            const uint32_t base = smem_addr(stages + (size_t)slot * C::kStageBytes);
            const uint64_t ad = smem_desc_k_sw128(base + tile * kABytes);
            const uint64_t bd = smem_desc_k_sw128(base + kTiles * kABytes);
            const int word0 = (s % C::kPerSb) * C::kWords;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const int word = word0 + (BITS == 8 ? 0 : j / 2);
              const uint32_t id = BITS == 8 ? j : (j & 1) * 2;
              const uint32_t sfw = sfc + word * (1 + C::kBBlocks) * 4;
              mma_mx<BITS, CG>(acc, ad + j * 2, bd + j * 2, idesc | id << 4 | id << 29, sfw, sfw + 4,
                           accumulate | j);
            }
            commit<CG>(&ctl->empty[slot]);
          }
          accumulate = 1;
        }
        if (ok && el) commit<CG>(&ctl->sf_empty[ss]);
      }
      if (ok && el) commit<CG>(&ctl->acc_full[buf]);
    }
    // nothing these warps issued may be in flight when the memory goes
    if (el) {
      if (CG == 2) mma_commit_pair_here(&ctl->drain);
      else mma_commit(&ctl->drain);
    }
    wait_drain(&ctl->drain, 0);
  } else if (warp == 3 || warp >= 12) {
    // ------------------------------------------------------------ scales --
    // A lane brings one row's 16 bytes of each 32-row group; the loads of a
    // warp's next slot are in flight while it waits for the slot to come free
    // (four warps: two left 8192 x 4096 x 28672 with 4-bit rows at 488 us
    // instead of 419).  Whole 32-byte sectors per load, or a prefetch of the
    // unit's scale rows into L2, changed nothing.
    const int lw = warp == 3 ? 0 : warp - 11;  // the slot of the ring it fills
    constexpr int kGroupsA = kTiles * 4, kGroupsB = (BN + 31) / 32;
    uint32_t sb_it = 0;
    bool ok = true;
    const int64_t row_bytes = (int64_t)p.words * 4;
    for (uint32_t u = 0; u < units && ok; ++u) {
      const Unit w = unit_at<BN, CG>(p, chunk_start, list, u);
      const int sb0 = (int)((int64_t)p.sbs * w.split / p.splits);
      const int sb1 = (int)((int64_t)p.sbs * (w.split + 1) / p.splits);
      for (int sb = sb0; sb < sb1; ++sb, ++sb_it) {
        if ((int)(sb_it % kSfWarps) != lw) continue;
        uint4 va[kGroupsA], vb[kGroupsB];
#pragma unroll
        for (int g = 0; g < kGroupsA; ++g) {
          const int r = g * 32 + lane, second = r >= p.box_rows;
          const int wr = w.m + (second ? p.up_row - p.box_rows : 0) + r;
          va[g] = make_uint4(0, 0, 0, 0);
          if (wr < p.wrows)
            va[g] = load_words(p.w_scale + ((int64_t)w.e * p.wrows + wr) * row_bytes, sb * 4, p.words);
        }
#pragma unroll
        for (int g = 0; g < kGroupsB; ++g) {
          const int r = w.row0 + g * 32 + lane;
          vb[g] = make_uint4(0, 0, 0, 0);
          if (g * 32 + lane < w.n)
            vb[g] = load_words(p.a_scale + (int64_t)r * row_bytes, sb * 4, p.words);
        }
        const uint32_t ss = sb_it % kSfRing;
        if (!warp_wait(&ctl->sf_empty[ss], ((sb_it / kSfRing) & 1) ^ 1, ctl, p.status)) {
          ok = false;
          break;
        }
        // block [word][32 lanes][4 groups]: a lane's words of four row groups
        // side by side, one 16-byte store each
        uint8_t* slot = sf + (size_t)ss * C::kSfSlotBytes + lane * 16;
#pragma unroll
        for (int b = 0; b < kTiles + C::kBBlocks; ++b) {
          uint4 g[4];
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            if (b < kTiles) g[c] = va[b < kTiles ? b * 4 + c : 0];
            else if ((b - kTiles) * 4 + c < kGroupsB) g[c] = vb[b < kTiles ? 0 : (b - kTiles) * 4 + c];
            else g[c] = make_uint4(0, 0, 0, 0);
          }
          uint4* d = reinterpret_cast<uint4*>(slot + b * 512);
          d[0 * (C::kSfWordBytes / 16)] = make_uint4(g[0].x, g[1].x, g[2].x, g[3].x);
          d[1 * (C::kSfWordBytes / 16)] = make_uint4(g[0].y, g[1].y, g[2].y, g[3].y);
          d[2 * (C::kSfWordBytes / 16)] = make_uint4(g[0].z, g[1].z, g[2].z, g[3].z);
          d[3 * (C::kSfWordBytes / 16)] = make_uint4(g[0].w, g[1].w, g[2].w, g[3].w);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) arrive<CG>(&ctl->sf_full[ss]);
      }
    }
  } else if (warp >= 4 && warp < 12) {
    // ---------------------------------------------------------- epilogue --
    const int quad = warp & 3;       // the tensor-memory lanes this warp may read
    const int half = (warp - 4) >> 2;  // which 16-column steps it takes
    // MX_EPI_PART: thread c of the epilogue looks up where column c of a unit
    // goes, one unit ahead, and passes it on through shared memory.
    const int col = tid - 128;
    int dest = 0;
    uint32_t swaps = 0;
    float factor = 1.0f;
    auto look_up = [&](uint32_t t) {
      if (t >= units || col >= BN) return;
      const Unit w = unit_at<BN, CG>(p, chunk_start, list, t);
      if (col >= w.n) return;
      dest = p.dest ? p.dest[w.row0 + col] : w.row0 + col;
      factor = p.dest_w ? p.dest_w[dest] : 1.0f;
    };
    if constexpr (EPI == MX_EPI_PART) look_up(0);
    bool ok = true;  // (a warp that gave up still meets the others at their barriers)
    for (uint32_t t = 0; t < units; ++t) {
      const Unit w = unit_at<BN, CG>(p, chunk_start, list, t);
      const uint32_t buf = t % C::kBufs;
      const int4* table = dest_table + (t & 1) * BN;
      if constexpr (EPI == MX_EPI_PART) {
        if (col < BN) {
          const int64_t at = (int64_t)dest * p.N;
          dest_table[(t & 1) * BN + col] =
              make_int4((int)(uint32_t)at, (int)(at >> 32), __float_as_int(factor), 0);
        }
        epilogue_barrier();
        look_up(t + 1);
      }
      ok = ok && warp_wait(&ctl->acc_full[buf], (t / C::kBufs) & 1, ctl, p.status);
      if (!ok) {
        if constexpr (CG == 2 && EPI == MX_EPI_GATED)
          for (int c0 = half * 16; c0 < w.n; c0 += 32) swap_barrier(half * 2 + (quad & 1));
        continue;
      }
      tc_fence_after();
      const uint32_t acc = tmem + buf * C::kAccCols + ((uint32_t)(quad * 32) << 16);
      if constexpr (EPI == MX_EPI_GATED) {
        // A lane's output: its weight row's, or with a pair's 64 + 64 rows the
        // gate row's (quarters 0-1 hold gate rows, 2-3 their up rows).
        const int n = w.m + (CG == 2 ? quad & 1 : quad) * 32 + lane;
        const bool live = n < p.N;  // (uniform: N is a multiple of 32)
        constexpr int kStep = CG == 2 ? 8 : 16;  // columns this warp finishes of 16
        const int mine0 = CG == 2 && quad >= 2 ? 8 : 0;
        for (int c0 = half * 16; c0 < w.n; c0 += 32) {
          uint32_t v0[16], v1[16];
          tmem_ld16_sync(acc + c0, v0);
          if constexpr (CG == 1) {
            tmem_ld16_sync(acc + BN + c0, v1);
          } else {
            // The gate warp finishes columns 0-7 of the step and the up warp
            // 8-15: each passes the other half on.
            float* out = swap + ((swaps & 1) * kEpiWarps + (warp - 4)) * 256 + lane;
            const float* in = swap + ((swaps & 1) * kEpiWarps + ((warp - 4) ^ 2)) * 256 + lane;
#pragma unroll
            for (int j = 0; j < 8; ++j)
              out[j * 32] = __uint_as_float(quad < 2 ? v0[8 + j] : v0[j]);
            swap_barrier(half * 2 + (quad & 1));
            ++swaps;  // (the buffer is written again only after the next barrier)
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const uint32_t got = __float_as_uint(in[j * 32]);
              v1[j] = quad < 2 ? got : v0[8 + j];  // up
              v0[j] = quad < 2 ? v0[j] : got;      // gate
            }
          }
          // One stage at a time over all columns, so that their latencies
          // overlap.
          float act[kStep];
          uint32_t code[kStep];
#pragma unroll
          for (int j = 0; j < kStep; ++j) {
            const float g = __uint_as_float(v0[j]);
            act[j] = __fdividef(g, 1.0f + __expf(-g)) * __uint_as_float(v1[j]);
          }
#pragma unroll
          for (int j = 0; j < kStep; ++j)
            code[j] = __reduce_max_sync(0xffffffffu, __float_as_uint(act[j]) & 0x7fffffffu);
          uint32_t codes = 0;  // lane j keeps column j's scale code
#pragma unroll
          for (int j = 0; j < kStep; ++j) {
            code[j] = mq::mx_scale_code<BITS>(code[j]);
            act[j] = mq::mx_scaled(act[j], mq::mx_inv_scale(code[j]));
            if (lane == j) codes = code[j];
          }
          // Two outputs of one column per lane: even lanes take the even
          // columns of their pair of outputs, odd lanes the odd ones.
          const int odd = lane & 1;
          uint8_t* dst = p.act + (((int64_t)(w.row0 + c0 + mine0 + odd) * p.N + (n & ~1)) * BITS >> 3);
          const int64_t two_rows = (int64_t)p.N * BITS >> 2;
#pragma unroll
          for (int j = 0; j < kStep; j += 2, dst += two_rows) {
            const float got = __shfl_xor_sync(0xffffffffu, odd ? act[j] : act[j + 1], 1);
            const float lo = odd ? got : act[j], hi = odd ? act[j + 1] : got;
            if (live && c0 + mine0 + j + odd < w.n) {
              if (BITS == 8) *reinterpret_cast<uint16_t*>(dst) = (uint16_t)mq::e4m3x2(lo, hi);
              else *dst = (uint8_t)mq::e2m1x2(lo, hi);
            }
          }
          const int c = c0 + mine0 + lane;
          if (live && lane < kStep && c < w.n)
            p.act_scale[(int64_t)(w.row0 + c) * (p.N >> 5) + ((n - lane) >> 5)] = (uint8_t)codes;
        }
      } else {
#pragma unroll
        for (int tile = 0; tile < kTiles; ++tile) {
          const int n = w.m + tile * p.up_row + quad * 32 + lane;  // this lane's output
          if (n - lane >= p.N) break;
          const bool live = n < p.N;
          for (int c0 = half * 16; c0 < w.n; c0 += 32) {
            uint32_t v[16];
            tmem_ld16_sync(acc + tile * BN + c0, v);
            if constexpr (EPI == MX_EPI_PART) {
              float* part = p.part + (int64_t)w.split * p.part_rows * p.N + n;
#pragma unroll
              for (int j = 0; j < 16; ++j) {
                const int4 d = table[c0 + j];
                const int64_t at = (int64_t)(uint32_t)d.x | (int64_t)d.y << 32;
                if (live && c0 + j < w.n)
                  part[at] = __uint_as_float(v[j]) * __int_as_float(d.z);
              }
            } else {
              const int64_t at = (int64_t)(w.row0 + c0) * p.N + n;
#pragma unroll
              for (int j = 0; j < 16; ++j)
                if (live && c0 + j < w.n)
                  store_out(p.out, p.out_dtype, at + (int64_t)j * p.N, __uint_as_float(v[j]));
            }
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) arrive<CG>(&ctl->acc_empty[buf]);
    }
  }
  tc_fence_before();
  __syncwarp();
  if (CG == 2) cluster_sync();  // (the other CTA's shared memory is in use until here)
  else __syncthreads();
  tc_fence_after();
  if (warp == 1) {
    if (CG == 2) tmem_dealloc_pair(tmem, 512);
    else tmem_dealloc(tmem, 512);
  }
}

// ------------------------------------------------------------ host side --
PFN_cuTensorMapEncodeTiled_v12000 g_encode = nullptr;
std::once_flag g_encode_once;

cudaError_t get_encoder() {
  std::call_once(g_encode_once, [] {
    void* fn = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault,
                                         &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      g_encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
  });
  return g_encode ? cudaSuccess : cudaErrorNotSupported;
}

cudaError_t make_map(CUtensorMap* map, CUtensorMapDataType dt, int rank, const void* base,
                     const cuuint64_t* dims, const cuuint64_t* strides, const cuuint32_t* box) {
  const cuuint32_t ones[3] = {1, 1, 1};
  const CUresult r = g_encode(map, dt, rank, const_cast<void*>(base), dims, strides, box, ones,
                              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                              CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

template <int BITS, int BN, int EPI, int CG>
cudaError_t launch_one(const CUtensorMap& mw, const CUtensorMap& ma, const CUtensorMap& mr, const Params& p,
                       int64_t units, cudaStream_t st) {
  constexpr size_t smem = Cfg<BITS, BN, CG, EPI>::kSmem;
  static_assert(smem <= kSmemMax, "shared memory");
  auto kern = mx_gemm<BITS, BN, EPI, CG>;
  static std::atomic<uint64_t> ready{0};  // devices whose attribute is set
  int dev = 0;
  cudaError_t err = cudaGetDevice(&dev);
  if (err != cudaSuccess) return err;
  const uint64_t bit = uint64_t(1) << (dev & 63);
  if (!(ready.load(std::memory_order_relaxed) & bit)) {
    err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (err != cudaSuccess) return err;
    ready.fetch_or(bit, std::memory_order_relaxed);
  }
  const int sms = tc_num_sms();
  const int workers = (int)std::min<int64_t>(units, sms / CG);
  return launch_pdl_cluster(kern, dim3(workers * CG), dim3(kThreads), CG, smem, st, mw, ma, mr, p);
}

template <int BITS, int EPI>
cudaError_t launch_bn(const MxPlan& pl, const CUtensorMap& mw, const CUtensorMap& ma,
                      const CUtensorMap& mr, const Params& p, int64_t units, cudaStream_t st) {
  if (pl.pair) return launch_one<BITS, kPairRows, EPI, 2>(mw, ma, mr, p, units, st);
  switch (pl.bn) {
    case 16: return launch_one<BITS, 16, EPI, 1>(mw, ma, mr, p, units, st);
    case 32: return launch_one<BITS, 32, EPI, 1>(mw, ma, mr, p, units, st);
    case 64: return launch_one<BITS, 64, EPI, 1>(mw, ma, mr, p, units, st);
    default: return launch_one<BITS, 96, EPI, 1>(mw, ma, mr, p, units, st);
  }
}

template <int BITS>
cudaError_t launch_epi(const MxGemm& g, const MxPlan& pl, const CUtensorMap& mw,
                       const CUtensorMap& ma, const CUtensorMap& mr, const Params& p, int64_t units, cudaStream_t st) {
  switch (g.epi) {
    case MX_EPI_OUT: return launch_bn<BITS, MX_EPI_OUT>(pl, mw, ma, mr, p, units, st);
    case MX_EPI_PART: return launch_bn<BITS, MX_EPI_PART>(pl, mw, ma, mr, p, units, st);
    default: return launch_bn<BITS, MX_EPI_GATED>(pl, mw, ma, mr, p, units, st);
  }
}

}  // namespace

// Rows per tile: as many as the fullest expert is likely to have, so that most
// experts are one chunk and their weights are read once; CTA pairs above 96 rows
// on average.  Of E random loads of average m the fullest is near m + sqrt(2 m ln
// E); half as much again covers routers that are less even.  A narrow tile leaves
// room for more stages, a wide one reads no weights twice.  Forwards in us with 32
// and 64 rows, 8-bit rows, the weights of three layers in turn; loads even / normal
// bias / Zipf:
//   E=8 k=2 H=4096 I=14336   m=16 137 146 / 132 143 / 121 129,  m=19 138 147 / 146
//     144 / 170 146,  m=24 150 147 / 173 148 / 154 141
//   E=40 k=4 H=2048 I=1408   m=13 51 54 / 48 49 / 38 38,  m=19 52 55 / 57 53 / 44 43
//   E=128 k=8 H=2048 I=768   m=10 75 79 / 67 66 / 45 44,  m=12 77 81 / 68 67 / 48 46,
//     m=16 80 83 / 74 73 / 56 50
// (4-bit rows have four stages with either: they differ only where the narrow tile
// reads weights twice.)  64 and 96 rows: m=24 to 40 within 1 % at an even load, up to
// 7 % for 96 with a bias; a skewed product of 256 rows, E=8, 54.9 and 44.7.  One
// expert, 24 rows, K=4096, N=28672: 15.6 with 32 rows, 18.2 with 64.
//
// K splits: the count with the least estimated time, in us.  The weights come
// in at the HBM's rate or, with few units, at what their SMs can take (70 GB/s
// each measured, or the instructions' time: 64 cycles and half a cycle per
// column); a unit costs 0.7 us more, partial sums their traffic and a launch.
// Measured against every count from 1 to 16: 128 rows, E=8, K=14336, N=4096
// 46.5 us unsplit, 50.9 with 7; 8 rows 35.3 and 32.8; one row, E=1, K=14336
// 32.4 and 12.7.
MxPlan mx_plan(int64_t S, int E, int K, int N, bool gated, int a_bits) {
  MxPlan pl;
  // experts with a row, if rows fall on experts at random
  const double live = std::max(1.0, E * (1.0 - std::pow(1.0 - 1.0 / E, (double)S)));
  const double avg = S / live;
  pl.pair = avg > 96;
  const double fullest = avg + 1.5 * std::sqrt(2 * avg * std::log((double)E));
  pl.bn = pl.pair ? kPairRows : S <= 16 ? 16 : fullest <= 32 || S <= 32 ? 32 : fullest <= 44 ? 64 : 96;
  pl.splits = 1;
  if (gated || S > 1024) return pl;  // (more rows: partial sums would cost more than idle SMs)
  const int sms = pl.pair ? tc_num_sms() / 2 : tc_num_sms();
  const int sbs = (K + 511) / 512;
  const double chunks = std::max(live, std::ceil((double)S / pl.bn));
  const double tiles = (N + 2 * kTileM - 1) / (2 * kTileM);
  const double row = a_bits / 8.0 + 1.0 / 32, wrow = 0.5 + 1.0 / 32;
  const double hbm = live * N * K * wrow / 6.6e6;
  double best = 0;
  for (int sp = 1; sp <= 16 && sp <= sbs; ++sp) {
    const double sb = std::ceil((double)sbs / sp);
    const double bytes = 512.0 * sb * (2 * kTileM * wrow + pl.bn * row) / (pl.pair ? 2 : 1);
    const double cycles = sb * (a_bits == 8 ? 32 : 16) * (64 + pl.bn / 2) / (pl.pair ? 2 : 1);
    const double waves = std::ceil(chunks * tiles * sp / sms);
    double us = std::max(hbm, waves * (std::max(bytes / 70e3, cycles / 2000) + 0.7));
    if (sp > 1) us += 3.0 + sp * (double)S * N * 8 / 5e6;
    if (best == 0 || us < best) {
      best = us;
      pl.splits = sp;
    }
  }
  return pl;
}

cudaError_t launch_mx_gemm(const MxGemm& g, const MxPlan& pl, cudaStream_t st) {
  cudaError_t err = get_encoder();
  if (err != cudaSuccess) return err;
  const bool gated = g.epi == MX_EPI_GATED;
  CUtensorMap mw, ma, mr;
  {
    // 8-bit rows: the weights' nibbles are spread to the mixed instruction's
    // operand form on the way; 4-bit rows: packed bytes, as both operands are
    const bool spread = g.a_bits == 8;
    const cuuint64_t kw = spread ? g.K : g.K / 2;
    const cuuint64_t dims[3] = {kw, (cuuint64_t)g.wrows, (cuuint64_t)g.E};
    const cuuint64_t strides[2] = {(cuuint64_t)g.K / 2, (cuuint64_t)g.K / 2 * g.wrows};
    const cuuint32_t box[3] = {128, (cuuint32_t)(gated && pl.pair ? kTileM / 2 : kTileM), 1};
    err = make_map(&mw, spread ? CU_TENSOR_MAP_DATA_TYPE_16U4_ALIGN16B : CU_TENSOR_MAP_DATA_TYPE_UINT8,
                   3, g.w, dims, strides, box);
    if (err != cudaSuccess) return err;
    const cuuint64_t row = (cuuint64_t)g.K * g.a_bits / 8;
    const cuuint64_t adims[2] = {row, (cuuint64_t)g.R};
    const cuuint32_t abox[2] = {128, (cuuint32_t)(pl.bn / (pl.pair ? 2 : 1))};
    err = make_map(&ma, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, g.a, adims, &row, abox);
    if (err != cudaSuccess) return err;
    const cuuint32_t rbox[2] = {128, pl.pair ? 16u : 32u};
    err = make_map(&mr, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, g.a, adims, &row, rbox);
    if (err != cudaSuccess) return err;
  }
  Params p = {};
  p.w_scale = g.w_scale;
  p.a_scale = g.a_scale;
  p.seg_start = g.seg_start;
  p.seg_count = g.seg_count;
  p.E = g.E;
  p.K = g.K;
  p.N = g.N;
  p.R = (int)g.R;
  // A unit is two weight tiles: gate and up of 128 outputs, or 256 outputs.
  // One CTA holds both; of a pair each CTA holds 128 rows of them.
  p.mrows = gated ? kTileM : 2 * kTileM;
  p.rank_rows = p.mrows / 2;
  p.box_rows = pl.pair ? p.rank_rows : kTileM;
  p.up_row = gated ? g.N : kTileM;
  p.wrows = g.wrows;
  p.mtiles = (g.N + p.mrows - 1) / p.mrows;
  p.splits = pl.splits;
  p.words = g.K / 128;
  // Weights that are read once leave L2 first, so that what the call reads again
  // (rows of A, scales, partial sums) stays.  Not so with 8-bit rows where a call
  // may read several times L2 (129 MB): a load takes 64 bytes of the 256 that L2
  // fetches, and in a long stream the rest may be gone before the next stages take
  // it.  Which of the two wins was measured with other weights streamed between any
  // two calls (us, normal and evict-first, 8-bit rows): forwards E=8 k=2 H=4096
  // I=14336 T=1 52.0 47.8, T=2 58.4 54.3, T=4 83.5 81.1, T=8 111 113, T=64 136 141,
  // T=256 158 156; E=128 k=8 H=2048 I=768 (288 MiB) T=8 45.6 42.3, T=64 72.9 70.6;
  // E=16 H=4096 I=6400 (600 MiB) T=64 130 132; products E=8 K=14336 N=4096 (224
  // MiB) 128 rows 46.8 48.5, 512 rows 53.6 51.6; E=16 K=4096 N=28672 (896 MiB) 128
  // rows 153 164.  The limit is where losses begin to outweigh gains, which either
  // way are a few percent near it.  With 4-bit rows evict-first was faster or equal at
  // all of these (E=8 T=64 131 127).
  p.evict_first = g.a_bits == 4 || g.weight_bytes < int64_t(400) << 20;
  p.sbs = (p.words + 3) / 4;
  p.out = g.out;
  p.out_dtype = g.out_dtype;
  p.part = g.part;
  p.part_rows = g.part_rows;
  p.dest = g.dest;
  p.dest_w = g.dest_w;
  p.act = g.act;
  p.act_scale = g.act_scale;
  p.status = g.status;
  const int64_t live = g.S < g.E ? g.S : g.E;
  const int64_t units = (live + g.S / pl.bn) * p.mtiles * p.splits;  // at most
  if (units <= 0) return cudaSuccess;
  return g.a_bits == 8 ? launch_epi<8>(g, pl, mw, ma, mr, p, units, st)
                       : launch_epi<4>(g, pl, mw, ma, mr, p, units, st);
}
