// Rows grouped by expert times 16-bit weights, and the gradients of that product,
// on tcgen05 (kind::f16, float32 accumulation):
//
//   GG_W_K   out[r, m] = sum_k A[r, k] * W[e(r), m, k]       W stored [E][M][K]
//   GG_W_M   the same with W stored [E][K][M]: the gradient of the rows, where W's
//            outputs are the contraction, or weights stored the other way round
//   GG_ROWS  out[e, m, n] = sum_{r in e} Y[r, m] * A[r, n]   the gradient of the weights
//
// One persistent CTA (or CTA pair) per SM (pair).  An accumulator tile has M in the
// tensor-memory lanes (128 per CTA) and BN columns.  In the first two forms the
// columns are rows of A, in steps of 16 (32 for a pair): an expert with a few rows
// costs a narrow instruction and no padding.
//
// Operands come by TMA in stages of 64 k.  A stage's bytes are the same whichever
// index is contiguous in memory: 128-byte swizzled lines of 64 elements, along k, or
// along m (n) in blocks of 64 by 64, and the instruction's descriptors say which.  So
// nothing is transposed on the way.
//
// GG_ROWS: an expert's rows end anywhere.  The rows behind them that the last stage
// brings are another expert's, and may hold infinities or NaN: one warp of each CTA
// overwrites both operands' lines with zeros up to the next step of 16 before the MMAs
// see them, and the steps after that are not issued.
//
// Roles: warp 0 streams both operands; warp 1 issues the MMAs (of a pair: in its
// first CTA); warp 2 clears the tail of GG_ROWS; warp 3 zeroes rows of no expert;
// warps 4-11 are the epilogue.  Two accumulator buffers: the next unit's MMAs run
// while the epilogue stores.
//
// What bounds it: with few rows per expert the weights (128 rows, 8 experts, 4096 x 28672:
// 273 us, 6.9 TB/s); with many the tensor pipe, and with it power (8192 rows there: 1245 us,
// 1.55 PFLOP/s in a loop at 1.45 GHz; there a CTA pair holds 256 by 256, which halves the
// operand reads of two CTAs by themselves).  The gradient of the weights writes more than
// it reads where experts have few rows, and writes alone go at little more than half the
// rate of a copy, so both gradients then run side by side in one launch: 16 experts, 517 rows,
// 1408 x 2048, float32: 66 us one after the other, 55 together.
#include "grouped.cuh"
#include "pipe.cuh"

#include <algorithm>
#include <cmath>
#include <type_traits>

namespace {

using namespace mq::pipe;

constexpr int kTileM = 128;
constexpr int kStageK = 64;                    // 128 bytes of k
constexpr int kABytes = kTileM * 128;
constexpr int kBlockBytes = kStageK * 128;     // 64 by 64 elements
constexpr int kThreads = 384;
constexpr int kEpiWarps = 8;
constexpr int kMaxStages = 12;
constexpr int kMaxE = 1024;
constexpr int kUnitList = 256;  // units of a CTA that are decoded at its start
constexpr int kGroup = 8;       // M tiles that a walk over the columns shares
constexpr int kPartRows = 16;   // rows of the boxes that load a partly filled chunk
constexpr size_t kSmemMax = 227 * 1024;

// Stages whose sum stays in tensor memory; longer sums are made of such segments, which the
// epilogue adds up in registers, to nearest.  The tensor core's additions round towards
// zero, four of them a stage, so that an error grows with their number: K 2056, 2.3e-6 of
// the values in one go, 2.6e-7 in segments of four stages.  Four for float32 results: 3001
// rows of 64 experts, 2056 x 2817, 128 us in one go and 132.  16 for results of 16 bits: what
// is cut off stays below a 250th of f16's half step however long the sum is (in one go a
// ninth at 28672).  us in one go and in segments of 16, 12, 8 and 4 stages: 8192 rows of 8
// experts, 4096 x 28672, 1221, 1245, 1259, 1306, 1363, both gradients there 2607, 2636, 2658,
// 2669, 2739 (storing 256 columns takes longer than the two short segments that the
// accumulators hold meanwhile).
constexpr int kSegment = 4;
constexpr int kSegment16 = 16;

constexpr int kChunkBytes = 32 * 64;  // an epilogue warp's 32 lanes by 64 bytes of columns

template <int FORM, int BN, int CG>
struct Cfg {
  static constexpr int kBRows = BN / CG;  // columns whose operand each CTA holds
  static constexpr int kStageBytes = kABytes + kBRows * 128;
  static constexpr int kBufs = 2;
  static_assert(kBufs * BN <= 512, "tensor memory");
  static constexpr size_t kOutBytes = FORM == GG_ROWS ? kEpiWarps * kChunkBytes : 0;
  static constexpr size_t kFixed = 1024 + kOutBytes + 1024 + kUnitList * 16 + (kMaxE + 1) * 4;
  static constexpr int kFit = (int)((kSmemMax - kFixed) / kStageBytes);
  static constexpr int kStages = kFit < kMaxStages ? kFit : kMaxStages;
  static_assert(kStages >= 3, "shared memory");
  // one CTA per SM: each allocates all of tensor memory
  static constexpr size_t kNeed = kFixed + (size_t)kStages * kStageBytes;
  static constexpr size_t kSmem = kNeed < 120 * 1024 ? 120 * 1024 : kNeed;
  static_assert(kSmem <= kSmemMax, "shared memory");
};

struct Ctl {
  uint64_t full[kMaxStages], empty[kMaxStages];
  uint64_t tail[kMaxStages];  // the last stage of an expert's rows has landed
  uint64_t acc_full[2], acc_empty[2];
  uint64_t drain;
  uint32_t tmem;
  volatile int abort_flag;
};
static_assert(sizeof(Ctl) <= 1024, "control block");

struct Params {
  const int32_t* offsets;
  int E, M, N, K, R;
  int mtiles, ntiles, splits;
  uint32_t idesc;  // without N
  bool listed;       // tiles are numbered in 16 bits: units fit the list
  bool tma_out;      // GG_ROWS: the result's rows start at 16-byte boundaries
  bool zero_outside;
  int segment;       // stages whose sum stays in tensor memory
  void* out;
  int out_dtype;
  float* part;
  unsigned* status;
};

// row0, n: first row and rows of a chunk; GG_ROWS: the first of the rows that are
// summed and their number, with col0 the first column.
struct Unit {
  int e, row0, n, m, split, col0;
  bool single;  // the expert has one chunk: its weights are read once
};

// Rows of expert e, kept inside [0, R) whatever the offsets hold; false where that
// took a correction.
__device__ __forceinline__ bool segment(const Params& p, int e, int& start, int& count) {
  if (!p.offsets) {
    start = 0;
    count = p.R;
    return true;
  }
  const int s = p.offsets[e], end = p.offsets[e + 1];
  start = min(max(s, 0), p.R);
  count = min(max(end, start), p.R) - start;
  return start == s && start + count == end;
}

// Unit u of the walk: expert by expert, groups of kGroup M tiles, every chunk of
// rows (GG_ROWS: column tile) over a group before the next group (the CTAs at work
// share the group's operands in L2), splits innermost.
template <int FORM, int BN, int CG>
__device__ __forceinline__ Unit decode_unit(const Params& p, const int* chunk_start, uint32_t u) {
  Unit w;
  const uint32_t per = p.mtiles * p.splits;
  uint32_t nch, r;
  if (FORM == GG_ROWS) {
    nch = p.ntiles;
    w.e = (int)(u / (per * nch));
    r = u - (uint32_t)w.e * per * nch;
  } else {
    const int g = (int)(u / per);  // a chunk's position in the walk locates its expert
    int lo = 0, hi = p.E;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (chunk_start[mid] <= g) lo = mid;
      else hi = mid;
    }
    w.e = lo;
    nch = chunk_start[lo + 1] - chunk_start[lo];
    r = u - chunk_start[lo] * per;
  }
  const uint32_t per_group = kGroup * nch * p.splits;
  const uint32_t grp = r / per_group;
  const uint32_t rem = r - grp * per_group;
  const uint32_t tiles = min(kGroup, p.mtiles - (int)grp * kGroup) * p.splits;
  const uint32_t c = rem / tiles;
  const uint32_t t = rem - c * tiles;
  w.m = (int)(grp * kGroup + t / p.splits) * (kTileM * CG);
  w.split = (int)(t % p.splits);
  int start, count;
  segment(p, w.e, start, count);
  if (FORM == GG_ROWS) {
    // the split's share of the expert's stages
    const int nst = (count + kStageK - 1) / kStageK;
    const int s0 = (int)((int64_t)nst * w.split / p.splits) * kStageK;
    const int s1 = (int)((int64_t)nst * (w.split + 1) / p.splits) * kStageK;
    w.row0 = start + s0;
    w.n = min(s1, count) - min(s0, count);
    w.col0 = (int)c * BN;
  } else {
    w.row0 = start + (int)c * BN;
    w.n = min(BN, count - (int)c * BN);
    w.col0 = 0;
  }
  w.single = nch == 1;
  return w;
}

// The i-th unit of this worker: from the list in shared memory (decoded once, by
// all threads at a time), past its end on the spot.  (Each role decoding each of its
// units cost GG_ROWS, whose units are short, more than their work: both gradients of 128 experts,
// 4096 rows, 1536 x 2048, 410 us that way and 372 with the list.)
template <int FORM, int BN, int CG>
__device__ __forceinline__ Unit unit_at(const Params& p, const int* chunk_start, const int4* list,
                                        uint32_t i, uint32_t worker, uint32_t workers) {
  if (i >= kUnitList || !p.listed)
    return decode_unit<FORM, BN, CG>(p, chunk_start, worker + i * workers);
  const int4 v = list[i];
  Unit w;
  w.e = v.x & 0xffff;
  w.single = (v.x >> 16) & 1;
  w.split = v.x >> 17;
  w.row0 = v.y;
  w.n = v.z;
  w.m = (int)((uint32_t)v.w & 0xffffu) * (kTileM * CG);
  w.col0 = (int)((uint32_t)v.w >> 16) * BN;
  return w;
}

// Stages of a unit: [first, last).
template <int FORM>
__device__ __forceinline__ void stages_of(const Params& p, const Unit& w, int& s0, int& s1) {
  if (FORM == GG_ROWS) {
    s0 = 0;
    s1 = (w.n + kStageK - 1) / kStageK;
  } else {
    const int nst = (p.K + kStageK - 1) / kStageK;
    s0 = (int)((int64_t)nst * w.split / p.splits);
    s1 = (int)((int64_t)nst * (w.split + 1) / p.splits);
  }
}

// Columns of the instruction: in steps of 16 for each CTA (32 for a pair), at most BN.
template <int FORM, int BN, int CG>
__device__ __forceinline__ int columns(const Params& p, const Unit& w) {
  const int n = FORM == GG_ROWS ? min(BN, p.N - w.col0) : w.n;
  return min(BN, (n + 16 * CG - 1) & -(16 * CG));
}

// Two float32 values rounded to a 16-bit type.
__device__ __forceinline__ uint32_t pack2(uint32_t lo, uint32_t hi, bool bf16) {
  const float a = __uint_as_float(lo), b = __uint_as_float(hi);
  if (bf16) {
    const __nv_bfloat162 t = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&t);
  }
  const __half2 t = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&t);
}

// 64 bytes of one lane's row of the result (16 float32 or 32 16-bit columns), into its
// line of the warp's buffer.
__device__ __forceinline__ void stage_line(uint8_t* chunk, int lane, const uint32_t (&w)[16]) {
#pragma unroll
  for (int j = 0; j < 4; ++j)
    *reinterpret_cast<uint4*>(chunk + lane * 64 + ((j ^ (lane >> 1 & 3)) << 4)) =
        make_uint4(w[4 * j], w[4 * j + 1], w[4 * j + 2], w[4 * j + 3]);
}

// One product, by the CTA `block` of `blocks` that work at it.  SEG: sums of p.segment
// stages leave tensor memory and are added up in the epilogue's registers.
template <int FORM, int BN, int CG, bool SEG>
__device__ __forceinline__ void gg_body(const CUtensorMap& map_w, const CUtensorMap& map_a,
                                        const CUtensorMap& map_part, const Params& p, uint32_t block,
                                        uint32_t blocks) {
  using C = Cfg<FORM, BN, CG>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  uint8_t* stages = smem;
  uint8_t* chunks_out = stages + (size_t)C::kStages * C::kStageBytes;  // GG_ROWS
  Ctl* ctl = reinterpret_cast<Ctl*>(chunks_out + C::kOutBytes);
  int4* list = reinterpret_cast<int4*>(reinterpret_cast<uint8_t*>(ctl) + 1024);
  int* chunk_start = reinterpret_cast<int*>(list + kUnitList);
  const int tid = threadIdx.x;
  const int warp = tid >> 5;
  const int lane = tid & 31;
  const uint32_t rank = CG == 2 ? cluster_rank() : 0;  // 0 issues the pair's MMAs
  const uint32_t worker = block / CG, workers = blocks / CG;

  if (tid == 0) {
    tma_prefetch_desc(&map_w);
    tma_prefetch_desc(&map_a);
    tma_prefetch_desc(&map_part);
    for (int i = 0; i < C::kStages; ++i) {
      mbar_init(&ctl->full[i], CG);
      mbar_init(&ctl->empty[i], 1);
      mbar_init(&ctl->tail[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&ctl->acc_full[i], 1);
      mbar_init(&ctl->acc_empty[i], CG * kEpiWarps);
    }
    mbar_init(&ctl->drain, 1);
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
  // Chunks of each expert, scanned; then this worker's units.
  bool fine = true, longer = FORM != GG_ROWS;  // (the others have one length: the kernel is chosen by it)
  for (int e = tid; e < p.E; e += kThreads) {
    int start, count;
    fine &= segment(p, e, start, count);
    chunk_start[e] = (count + BN - 1) / BN;
    longer |= count > p.segment * kStageK;
  }
  // offsets that fall or leave [0, R]: nothing is computed
  const bool bad = __syncthreads_or(!fine);
  if (bad && tid == 0 && block == 0) mq::flag(p.status, MQ_DEV_BAD_OFFSETS);
  const bool long_sums = SEG && __syncthreads_or(longer);  // some unit's sum has several segments
  if (FORM != GG_ROWS && warp == 0) {
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
  const uint32_t chunks = FORM == GG_ROWS ? (uint32_t)p.E * p.ntiles : (uint32_t)chunk_start[p.E];
  const uint32_t total = bad ? 0 : chunks * p.mtiles * p.splits;
  const uint32_t units = worker < total ? (total - worker + workers - 1) / workers : 0;
  if (p.listed && tid < kUnitList && tid < units) {
    const Unit w = decode_unit<FORM, BN, CG>(p, chunk_start, worker + tid * workers);
    list[tid] = make_int4(w.e | (w.single ? 1 << 16 : 0) | w.split << 17, w.row0, w.n,
                          w.m / (kTileM * CG) | (w.col0 / BN) << 16);
  }
  tc_fence_before();
  if (CG == 2) cluster_sync();  // (the barriers are set up in both)
  else __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ctl->tmem;

  if (warp == 0) {
    // ------------------------------------------------------- operands --
    const bool el = elect_one();
    const uint64_t pol_once = l2_policy_evict_first();
    uint32_t it = 0;
    uint32_t tail_last = 0, tail_parity = 0;  // by slot: its last load was a tail; tails so far, mod 2
    bool ok = true;
    for (uint32_t u = 0; u < units && ok; ++u) {
      const Unit w = unit_at<FORM, BN, CG>(p, chunk_start, list, u, worker, workers);
      int s0, s1;
      stages_of<FORM>(p, w, s0, s1);
      const int cols = columns<FORM, BN, CG>(p, w);
      const int m = w.m + (int)rank * kTileM;
      // this CTA's columns: their first, and how many TMA brings
      const int first = (int)rank * (cols / CG);
      const int brought = FORM == GG_ROWS ? (cols / CG + 63) & -64
                          : cols == BN    ? C::kBRows
                                          : cols / CG;
      const uint32_t bytes = kABytes + brought * 128;
      const bool once = FORM != GG_ROWS && w.single;
      for (int s = s0; s < s1; ++s, ++it) {
        const uint32_t slot = it % C::kStages;
        if (!warp_wait(&ctl->empty[slot], ((it / C::kStages) & 1) ^ 1, ctl, p.status)) {
          ok = false;
          break;
        }
        uint8_t* dst = stages + (size_t)slot * C::kStageBytes;
        uint8_t* dst_b = dst + kABytes;
        // the last stage of an expert's rows goes by way of warp 2
        const bool tail = FORM == GG_ROWS && s == s1 - 1 && (w.n & 15);
        tail_last = (tail_last & ~(1u << slot)) | (uint32_t)tail << slot;
        tail_parity ^= (uint32_t)tail << slot;
        if (el) {
          uint64_t* local = tail ? &ctl->tail[slot] : &ctl->full[slot];
          const uint32_t bar = CG == 2 && !tail ? map_rank(local, 0) : smem_addr(local);
          if (CG == 2) mbar_arrive_expect_tx_cluster(bar, bytes);
          else mbar_arrive_expect_tx(local, bytes);
          if constexpr (FORM == GG_ROWS) {
            const int row = w.row0 + s * kStageK;
#pragma unroll
            for (int b = 0; b < 2; ++b) {
              if (CG == 2) tma_load_2d_pair(dst + b * kBlockBytes, &map_w, bar, m + b * 64, row);
              else tma_load_2d(dst + b * kBlockBytes, &map_w, local, m + b * 64, row);
            }
            for (int b = 0; b < brought; b += 64) {
              if (CG == 2) tma_load_2d_pair(dst_b + b * 128, &map_a, bar, w.col0 + first + b, row);
              else tma_load_2d(dst_b + b * 128, &map_a, local, w.col0 + first + b, row);
            }
          } else {
            const int k = s * kStageK;
            if constexpr (FORM == GG_W_K) {
              if (CG == 2) tma_load_3d_pair(dst, &map_w, bar, k, m, w.e);
              else if (once) tma_load_3d_hint(dst, &map_w, local, k, m, w.e, pol_once);
              else tma_load_3d(dst, &map_w, local, k, m, w.e);
            } else {
#pragma unroll
              for (int b = 0; b < 2; ++b) {
                uint8_t* d = dst + b * kBlockBytes;
                if (CG == 2) tma_load_3d_pair(d, &map_w, bar, m + b * 64, k, w.e);
                else if (once) tma_load_3d_hint(d, &map_w, local, m + b * 64, k, w.e, pol_once);
                else tma_load_3d(d, &map_w, local, m + b * 64, k, w.e);
              }
            }
            const int row = w.row0 + first;
            if (cols == BN) {
              if (CG == 2) tma_load_2d_pair(dst_b, &map_a, bar, k, row);
              else tma_load_2d(dst_b, &map_a, local, k, row);
            } else {
              for (int r = 0; r < brought; r += kPartRows) {
                if (CG == 2) tma_load_2d_pair(dst_b + r * 128, &map_part, bar, k, row + r);
                else tma_load_2d(dst_b + r * 128, &map_part, local, k, row + r);
              }
            }
          }
        }
      }
    }
    if (ctl->abort_flag) {  // loads in flight land before the CTA goes
      for (uint32_t j = it < (uint32_t)C::kStages ? 0 : it - C::kStages; j < it; ++j) {
        const uint32_t slot = j % C::kStages;
        if (tail_last >> slot & 1) wait_drain(&ctl->tail[slot], (tail_parity >> slot & 1) ^ 1);
        else if (rank == 0) wait_drain(&ctl->full[slot], (j / C::kStages) & 1);
      }
    }
  } else if (warp == 1 && rank == 0) {
    // ----------------------------------------------------------- MMAs --
    // The warp walks the loop together and one elected lane issues, so that the
    // descriptors stay in uniform registers.
    const bool el = elect_one();
    uint32_t it = 0, done = 0;
    bool ok = true;
    for (uint32_t u = 0; u < units && ok; ++u) {
      const Unit w = unit_at<FORM, BN, CG>(p, chunk_start, list, u, worker, workers);
      int s0, s1;
      stages_of<FORM>(p, w, s0, s1);
      if (s0 == s1) continue;  // no rows: the epilogue stores zeros
      const uint32_t idesc = p.idesc | (uint32_t)(columns<FORM, BN, CG>(p, w) >> 3) << 17;
      for (int s = s0; s < s1 && ok;) {
        const int end = SEG ? min(s + p.segment, s1) : s1;
        const uint32_t buf = done & 1;
        ok = warp_wait<CG>(&ctl->acc_empty[buf], ((done >> 1) & 1) ^ 1, ctl, p.status);
        ++done;
        tc_fence_after();
        const uint32_t acc = tmem + buf * BN;
        uint32_t accumulate = 0;
        for (; s < end && ok; ++s, ++it) {
          const uint32_t slot = it % C::kStages;
          ok = warp_wait<CG>(&ctl->full[slot], (it / C::kStages) & 1, ctl, p.status);
          if (!ok) break;
          tc_fence_after();
          if (el) {
            const uint32_t base = smem_addr(stages + (size_t)slot * C::kStageBytes);
            const uint64_t ad = FORM == GG_W_K ? smem_desc_k_sw128(base)
                                               : smem_desc_mn_sw128(base, kBlockBytes);
            const uint64_t bd = FORM == GG_ROWS ? smem_desc_mn_sw128(base + kABytes, kBlockBytes)
                                                : smem_desc_k_sw128(base + kABytes);
            const int steps = FORM == GG_ROWS ? min(4, (w.n - s * kStageK + 15) >> 4) : 4;
#pragma unroll
            for (int j = 0; j < 4; ++j)
              if (FORM != GG_ROWS || j < steps)
                mma_ss<CG>(acc, ad + j * (FORM == GG_W_K ? 2 : 128), bd + j * (FORM == GG_ROWS ? 128 : 2),
                           idesc, accumulate | j);
            commit<CG>(&ctl->empty[slot]);
          }
          accumulate = 1;
        }
        if (ok && el) commit<CG>(&ctl->acc_full[buf]);
      }
    }
    // nothing this warp issued may be in flight when the memory goes
    if (el) {
      if (CG == 2) mma_commit_pair_here(&ctl->drain);
      else mma_commit(&ctl->drain);
    }
    wait_drain(&ctl->drain, 0);
  } else if (warp == 2 && FORM == GG_ROWS) {
    // ----------------------------------------------------------- tails --
    uint32_t it = 0, parity = 0;  // by slot: tails so far, mod 2
    bool ok = true;
    for (uint32_t u = 0; u < units && ok; ++u) {
      const Unit w = unit_at<FORM, BN, CG>(p, chunk_start, list, u, worker, workers);
      int s0, s1;
      stages_of<FORM>(p, w, s0, s1);
      it += s1 - s0;
      if (!(w.n & 15)) continue;
      const uint32_t slot = (it - 1) % C::kStages;
      ok = warp_wait(&ctl->tail[slot], parity >> slot & 1, ctl, p.status);
      parity ^= 1u << slot;
      if (!ok) break;
      const int live = w.n - (s1 - 1) * kStageK;  // rows of the stage that are the expert's
      uint8_t* dst = stages + (size_t)slot * C::kStageBytes;
      // line r of each 64 by 64 block; eight lanes cover its 128 bytes
      for (int r = live; r < ((live + 15) & -16); ++r)
        for (int b = lane >> 3; b < 2 + C::kBRows / 64; b += 4)
          *reinterpret_cast<uint4*>(dst + b * kBlockBytes + r * 128 + (lane & 7) * 16) =
              make_uint4(0, 0, 0, 0);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) arrive<CG>(&ctl->full[slot]);
    }
  } else if (warp == 3 && FORM != GG_ROWS) {
    // ------------------------------------------------ rows of no expert --
    if (p.zero_outside && p.offsets && !bad) {
      const int64_t lo = p.offsets[0], hi = p.offsets[p.E];
      const int64_t outside = lo + p.R - hi;
      for (int64_t i = block; i < outside; i += blocks) {
        const int64_t r = i < lo ? i : hi + i - lo;
        for (int m = lane; m < p.M; m += 32) store_out(p.out, p.out_dtype, r * p.M + m, 0.0f);
      }
    }
  } else if (warp >= 4) {
    // ---------------------------------------------------------- epilogue --
    const int quad = warp & 3;         // the tensor-memory lanes this warp may read
    const int half = (warp - 4) >> 2;  // which 16-column steps it takes
    uint32_t u = 0, done = 0;
    bool ok = true;
    // Units from u on: sums of one segment, or (kSegs) of several; where there are both
    // (kMixed), as long as they are of that kind.
    auto epilogue = [&](auto segs, auto mixed) {
      constexpr bool kSegs = decltype(segs)::value, kMixed = decltype(mixed)::value;
      for (; u < units && ok; ++u) {
        const Unit w = unit_at<FORM, BN, CG>(p, chunk_start, list, u, worker, workers);
        int s0, s1;
        stages_of<FORM>(p, w, s0, s1);
        if (kMixed && (s1 - s0 > p.segment) != kSegs) return;
        const int m = w.m + (int)rank * kTileM + quad * 32 + lane;  // this lane's output
        const int dtype = p.splits > 1 ? MQ_DTYPE_F32 : p.out_dtype;
        const bool empty = FORM == GG_ROWS && w.n == 0;
        const uint32_t lanes = (uint32_t)(quad * 32) << 16;
        auto sums_ready = [&]() -> bool {
          if (!warp_wait(&ctl->acc_full[done & 1], (done >> 1) & 1, ctl, p.status)) return false;
          tc_fence_after();
          return true;
        };
        auto sums_read = [&]() {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) {
            if (CG == 2) mbar_arrive_tmem_free(map_rank(&ctl->acc_empty[done & 1], 0));
            else mbar_arrive(&ctl->acc_empty[done & 1]);
          }
          ++done;
        };
        // Columns of a lane: a half of the tile in steps of 32 (GG_ROWS), or every other
        // step of 16.
        constexpr int kStep = FORM == GG_ROWS ? 32 : 16;
        constexpr int kSteps = BN / 2 / kStep;
        const int n = FORM == GG_ROWS ? min(BN, p.N - w.col0) : w.n;
        const int c1 = FORM == GG_ROWS ? min(n, (half + 1) * (BN / 2)) : n;
        auto column = [&](int i) { return FORM == GG_ROWS ? half * (BN / 2) + i * 32 : half * 16 + i * 32; };
        auto read = [&](int c0, uint32_t (&v)[kStep]) {
          const uint32_t at = tmem + (done & 1) * BN + lanes + c0;
          if constexpr (FORM == GG_ROWS) tmem_ld32_sync(at, v);
          else tmem_ld16_sync(at, v);
        };
        auto store = [&](int c0, const uint32_t (&v)[kStep]) {
          if constexpr (FORM == GG_ROWS) {
            // A lane is a row of the result: 64 bytes of it at a time go to shared memory
            // (swizzled) and from there by TMA, which leaves out what lies outside.  (Longer
            // lines would take a stage's place.)
            const bool f32 = dtype == MQ_DTYPE_F32;
            uint8_t* chunk = chunks_out + (warp - 4) * kChunkBytes;
            if (p.tma_out) {
              uint32_t line[16];
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                if (f32) {
#pragma unroll
                  for (int i = 0; i < 16; ++i) line[i] = v[16 * h + i];
                } else {
                  if (h) break;
#pragma unroll
                  for (int i = 0; i < 16; ++i) line[i] = pack2(v[2 * i], v[2 * i + 1], dtype == MQ_DTYPE_BF16);
                }
                if (lane == 0) bulk_wait_read<0>();  // what was there has been read
                __syncwarp();
                stage_line(chunk, lane, line);
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                  tma_store_3d(&map_part, chunk, w.col0 + c0 + 16 * h, m - lane, w.split * p.E + w.e);
                  bulk_commit();
                }
                if (f32 && c0 + 16 >= c1) break;
              }
            } else if (m < p.M) {
              void* out = p.splits > 1 ? p.part + (int64_t)w.split * p.E * p.M * p.N : p.out;
              const int64_t at = ((int64_t)w.e * p.M + m) * p.N + w.col0 + c0;
#pragma unroll
              for (int i = 0; i < 32; ++i)
                if (c0 + i < n) store_out(out, dtype, at + i, __uint_as_float(v[i]));
            }
          } else {
            void* out = p.out;
            if (p.splits > 1) out = p.part + (int64_t)w.split * p.R * p.M;
            const int64_t at = (int64_t)(w.row0 + c0) * p.M + m;
#pragma unroll
            for (int j = 0; j < 16; ++j)
              if (m < p.M && c0 + j < n) store_out(out, dtype, at + (int64_t)j * p.M, __uint_as_float(v[j]));
          }
        };
        if constexpr (!kSegs) {
          if (!empty) {
            ok = sums_ready();
            if (!ok) break;
          }
          if (m - lane < p.M) {
            for (int i = 0; column(i) < c1; ++i) {
              uint32_t v[kStep];
              if (empty) {
#pragma unroll
                for (int j = 0; j < kStep; ++j) v[j] = 0;
              } else {
                read(column(i), v);
              }
              store(column(i), v);
            }
          }
          if (!empty) sums_read();
        } else {
          uint32_t sum[kSteps][kStep];
#pragma unroll
          for (int i = 0; i < kSteps; ++i)
#pragma unroll
            for (int j = 0; j < kStep; ++j) sum[i][j] = 0;
          for (int s = s0; s < s1; s += p.segment) {
            ok = sums_ready();
            if (!ok) break;
            if (m - lane < p.M) {
#pragma unroll
              for (int i = 0; i < kSteps; ++i) {
                if (column(i) >= c1) continue;
#pragma unroll
                for (int h = 0; h < kStep; h += 16) {
                  uint32_t v[16];
                  tmem_ld16_sync(tmem + (done & 1) * BN + lanes + column(i) + h, v);
#pragma unroll
                  for (int j = 0; j < 16; ++j)
                    sum[i][h + j] = __float_as_uint(__uint_as_float(sum[i][h + j]) + __uint_as_float(v[j]));
                }
              }
            }
            sums_read();
          }
          if (!ok) break;
          if (m - lane < p.M) {
#pragma unroll
            for (int i = 0; i < kSteps; ++i)
              if (column(i) < c1) store(column(i), sum[i]);
          }
        }
      }
    };
    // (A choice for each unit costs where units are short: 128 experts, 4096 rows, 1536 x 2048,
    // whose sums are of one segment: 298 us with it, 364 as if all had several, 278 without.)
    constexpr std::true_type yes;
    constexpr std::false_type no;
    if constexpr (!SEG) {
      epilogue(no, no);
    } else if (!long_sums) {
      epilogue(no, no);
    } else if constexpr (FORM != GG_ROWS) {
      epilogue(yes, no);
    } else {
      while (u < units && ok) {
        epilogue(no, yes);
        epilogue(yes, yes);
      }
    }
  }
  if (FORM == GG_ROWS && warp >= 4 && lane == 0) bulk_wait_read<0>();
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

template <int FORM, int BN, int CG, bool SEG>
__global__ void __launch_bounds__(kThreads, 1)
    gg_gemm(const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_a,
            const __grid_constant__ CUtensorMap map_part, const Params p) {
  gg_body<FORM, BN, CG, SEG>(map_w, map_a, map_part, p, blockIdx.x, gridDim.x);
}

// Both gradients side by side: the first `rows_blocks` CTAs work at the rows', the others
// at the weights'.  For gradients that memory bounds: one reads the weights and the other
// writes as much, and HBM takes both at once at nearly twice the rate of writes alone (a
// fill runs at 3.84 TB/s, a copy at 6.69).
template <int FORM, bool SEG>
__global__ void __launch_bounds__(kThreads, 1)
    gg_both(const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_a,
            const __grid_constant__ CUtensorMap map_part, const __grid_constant__ CUtensorMap map_y,
            const __grid_constant__ CUtensorMap map_x, const __grid_constant__ CUtensorMap map_out,
            const Params rows, const Params weights, uint32_t rows_blocks) {
  if (blockIdx.x < rows_blocks)
    gg_body<FORM, 256, 2, SEG>(map_w, map_a, map_part, rows, blockIdx.x, rows_blocks);
  else
    gg_body<GG_ROWS, 256, 2, SEG>(map_y, map_x, map_out, weights, blockIdx.x - rows_blocks,
                             gridDim.x - rows_blocks);
}

// ------------------------------------------------------------ host side --
// Whether a sum may be longer than a segment (GG_ROWS: where an expert has most rows).
template <int FORM>
bool segmented(const Params& p) {
  const int64_t stages = ((int64_t)(FORM == GG_ROWS ? p.R : p.K) + kStageK - 1) / kStageK;
  return (stages + p.splits - 1) / p.splits > p.segment;
}

template <int FORM, int BN, int CG>
cudaError_t launch_one(const CUtensorMap& mw, const CUtensorMap& ma, const CUtensorMap& mr,
                       const Params& p, int64_t units, cudaStream_t st) {
  constexpr size_t smem = Cfg<FORM, BN, CG>::kSmem;
  const bool seg = segmented<FORM>(p);
  auto kern = seg ? gg_gemm<FORM, BN, CG, true> : gg_gemm<FORM, BN, CG, false>;
  static std::atomic<uint64_t> ready[2];
  const cudaError_t err = allow_smem(kern, smem, ready[seg]);
  if (err != cudaSuccess) return err;
  const int sms = tc_num_sms();
  const int workers = (int)std::max<int64_t>(1, std::min<int64_t>(units, sms / CG));
  return launch_pdl_cluster(kern, dim3(workers * CG), dim3(kThreads), CG, smem, st, mw, ma, mr, p);
}

template <int FORM>
cudaError_t launch_form(const GgPlan& pl, const CUtensorMap& mw, const CUtensorMap& ma,
                        const CUtensorMap& mr, const Params& p, int64_t units, cudaStream_t st) {
  if (pl.pair) return launch_one<FORM, 256, 2>(mw, ma, mr, p, units, st);
  if constexpr (FORM != GG_ROWS) {
    if (pl.bn == 64) return launch_one<FORM, 64, 1>(mw, ma, mr, p, units, st);
  }
  return launch_one<FORM, 128, 1>(mw, ma, mr, p, units, st);
}

}  // namespace

GgPlan gg_plan(GgForm form, int64_t R, int E, int M, int N, int K) {
  GgPlan pl = {};
  pl.splits = 1;
  // Few rows and weights: one launch (grouped_few.cu), where its estimated time is less: reads
  // in chunks of 2048 k (1.3 us each, one after the other) for as many turns as the CTAs take,
  // or the weights at 5.5 TB/s.  us there and here, K x N and rows: 4096 x 4096 1 7.8 10.2, 16
  // 8.6 10.5; 2048 x 1536 1 4.1 7.2, 16 4.6 7.6; 4096 x 256 1 5.4 7.7; of 8 experts, 2048 x 768
  // 4 5.2 7.8, 16 8.2 9.5; of 128, 768 x 2048 4 4.5 6.5, 16 14.0 10.0; of 13, 11096 x 79 1 11.4
  // 9.1; 4096 x 14336 (117 MB) 1 21.9 21.8, 8 27.2 21.8.
  if (form == GG_W_K && R <= kFewRows) {
    const double groups = (double)std::min<int64_t>(R, E);
    const double bytes = 2.0 * groups * M * K;
    const double turns = std::ceil(std::ceil(M / 16.0) / std::max(1.0, std::floor(2 * tc_num_sms() / groups)));
    const double chunks = std::ceil(K / 2048.0);
    const double few_us = std::max(2 + turns * (0.3 + 1.3 * chunks), 2 + bytes / 5.5e6);
    pl.few = bytes <= 64e6 && few_us <= 6.2 + bytes / 9e6;
  }
  if (pl.few) return pl;
  const int sms = tc_num_sms();
  if (form == GG_ROWS) {
    pl.pair = M > 128 && N > 128;
    pl.bn = pl.pair ? 256 : 128;
    // Splits while they leave a wave of units, by the estimated time: 0.27 us a stage, and for
    // the partial sums a second launch and their way to it at 8 TB/s.  us with 1, 2, 4, 8 and 16:
    // one expert, 512 x 512, 512 rows 8.4, 10.0, 10.5, 10.6, 11.4, 4096 rows 23.1, 17.5, 13.6,
    // 12.0, 12.8, 16384 rows 73.6, 42.9, 26.4, 18.8, 17.4; 2048 x 1024, 1024 rows 10.7, 13.6,
    // 16.1, 23.4, 50.6, 4096 rows 23.6, 20.6, 22.2, 31.2, 56.5; 1024 x 1024, 16384 rows, float32
    // 75.9, 45.5, 30.7, 37.7, 52.0; 8 experts, 512 x 512, 8192 rows 11.2, 14.4, 17.2, 24.1, 53.4.
    const double units = (double)E * ((M + pl.bn - 1) / pl.bn) * ((N + pl.bn - 1) / pl.bn);
    const double workers = pl.pair ? sms / 2 : sms;
    const double stages = std::ceil(R / 64.0 / E);
    double best = 0.27 * stages;
    for (int n = 2; n <= 16 && units * n <= workers; n *= 2) {
      const double t = 0.27 * stages / n + 3.5 + n * 8.0 * E * M * N / 8e6;
      if (t < best) best = t, pl.splits = n;
    }
    return pl;
  }
  const double live = std::max(1.0, E * (1.0 - std::pow(1.0 - 1.0 / E, (double)R)));
  // Columns of a tile: so many that a popular expert, with twice the average and 1.5
  // standard deviations of the fullest of E, is likely to fit.  Narrow tiles read a popular
  // expert's weights, from L2, for each of its chunks; wide ones cost little where the loads
  // are even, as the instructions are no wider than the rows.  us with 64, 128 and pairs'
  // 256 columns: 128 experts, 2048 x 1536, 16 rows each 124, 128, 130, 32 rows 126, 130, 132
  // (by Zipf's law 136, 129, 130), 64 rows 133, 138, 138 (156, 143, 136), 128 rows 178, 151,
  // 148 (206, 172, 154); 8 experts, 4096 x 14336, 16 rows 140, 142, 144, 64 rows 160, 147,
  // 149, 128 rows 191, 174, 154, 512 rows 632, 386, 294.  (16 and 32 columns save nothing
  // but the tail of an epilogue: 8 experts, 4096 x 28672, 16 rows 278 with 32, 270 with 64;
  // 1 row, 4096 x 28672, 40.9 with 16, 39.6 with 64.)
  const double likely = 2 * R / live;
  const double fullest = std::min<double>(R, likely + 1.5 * std::sqrt(2 * likely * std::log((double)E)));
  pl.pair = fullest > 128;
  pl.bn = pl.pair ? 256 : fullest > 64 ? 128 : 64;
  // K splits while they leave a wave of units and eight stages each (us unsplit, with 2, 4 and
  // 8): 4096 x 4096, 17 rows 15.5, 11.9, 10.7, 11.9, 256 rows 25.0, 19.4, 16.4, 19.2, 1024 rows
  // 26.1, 32.8, 42.4, 65.7; 8 experts, 14336 x 1024, 128 rows 48.3, 40.3, 41.0, 43.5; 16
  // experts, 2048 x 768, 128 rows 12.0, 14.6, 13.9, 14.9.  (As good with many rows: 8192 x
  // 512, 1500 rows 41.3 unsplit, 19.5 with two.)
  const double workers = pl.pair ? sms / 2 : sms;
  const double units = std::max(live, std::ceil((double)R / pl.bn)) * ((M + (pl.pair ? 255 : 127)) / (pl.pair ? 256 : 128));
  const int stages = (K + kStageK - 1) / kStageK;
  while (pl.splits < 16 && units * pl.splits * 2 <= workers && stages >= pl.splits * 8) pl.splits *= 2;
  return pl;
}

namespace {

// A product's tensor maps, parameters and (at most) units.
struct Prepared {
  CUtensorMap mw, ma, mr;
  Params p;
  int64_t units;
};

cudaError_t prepare(const GgGemm& g, const GgPlan& pl, Prepared& out) {
  const CUtensorMapDataType dt = g.bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
  const int cg = pl.pair ? 2 : 1;
  bool tma_out = false;
  CUtensorMap &mw = out.mw, &ma = out.ma, &mr = out.mr;
  cudaError_t err;
  const cuuint64_t ws = 2 * (cuuint64_t)g.w_stride, as = 2 * (cuuint64_t)g.a_stride;
  const cuuint32_t block[3] = {64, 64, 1};
  if (g.form == GG_ROWS) {
    const cuuint64_t wd[2] = {(cuuint64_t)g.M, (cuuint64_t)g.R};
    const cuuint64_t ad[2] = {(cuuint64_t)g.N, (cuuint64_t)g.R};
    err = make_map(&mw, dt, 2, g.w, wd, &ws, block);
    if (err == cudaSuccess) err = make_map(&ma, dt, 2, g.a, ad, &as, block);
    mr = ma;
    const bool f32 = pl.splits > 1 || g.out_dtype == MQ_DTYPE_F32;
    const void* result = pl.splits > 1 ? g.part : g.out;
    const cuuint64_t row = (cuuint64_t)g.N * (f32 ? 4 : 2);
    tma_out = row % 16 == 0 && (reinterpret_cast<uintptr_t>(result) & 15u) == 0 && row * g.M < cuuint64_t(1) << 40;
    if (err == cudaSuccess && tma_out) {
      const cuuint64_t od[3] = {(cuuint64_t)g.N, (cuuint64_t)g.M, (cuuint64_t)g.E * pl.splits};
      const cuuint64_t os[2] = {row, row * g.M};
      const cuuint32_t ob[3] = {f32 ? 16u : 32u, 32, 1};
      const CUtensorMapDataType ot = f32                               ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                                     : g.out_dtype == MQ_DTYPE_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                                                    : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
      err = make_map(&mr, ot, 3, result, od, os, ob, CU_TENSOR_MAP_SWIZZLE_64B);
    }
  } else {
    const bool by_k = g.form == GG_W_K;
    const cuuint64_t wd[3] = {(cuuint64_t)(by_k ? g.K : g.M), (cuuint64_t)(by_k ? g.M : g.K), (cuuint64_t)g.E};
    const cuuint64_t wst[2] = {ws, 2 * (cuuint64_t)g.w_expert};
    const cuuint32_t rows[3] = {64, kTileM, 1};
    err = make_map(&mw, dt, 3, g.w, wd, wst, by_k ? rows : block);
    const cuuint64_t ad[2] = {(cuuint64_t)g.K, (cuuint64_t)g.R};
    const cuuint32_t abox[2] = {64, (cuuint32_t)(pl.bn / cg)}, pbox[2] = {64, kPartRows};
    if (err == cudaSuccess) err = make_map(&ma, dt, 2, g.a, ad, &as, abox);
    if (err == cudaSuccess) err = make_map(&mr, dt, 2, g.a, ad, &as, pbox);
  }
  if (err != cudaSuccess) return err;
  Params& p = out.p;
  p = {};
  p.offsets = g.offsets;
  p.E = g.E;
  p.M = g.M;
  p.N = g.N;
  p.K = g.K;
  p.R = (int)g.R;
  p.mtiles = (g.M + kTileM * cg - 1) / (kTileM * cg);
  p.ntiles = g.form == GG_ROWS ? (g.N + pl.bn - 1) / pl.bn : 1;
  p.splits = pl.splits;
  p.idesc = idesc_16(g.bf16, kTileM * cg, 0, g.form != GG_W_K, g.form == GG_ROWS);
  p.listed = p.mtiles < 1 << 16 && p.ntiles < 1 << 16;
  p.zero_outside = g.zero_outside;
  p.segment = g.out_dtype == MQ_DTYPE_F32 ? kSegment : kSegment16;
  p.out = g.out;
  p.out_dtype = g.out_dtype;
  p.part = g.part;
  p.status = g.status;
  p.tma_out = tma_out;
  const int64_t live = std::min<int64_t>(g.R, g.E);
  out.units = (g.form == GG_ROWS ? (int64_t)g.E * p.ntiles : live + g.R / pl.bn) * p.mtiles * p.splits;
  return cudaSuccess;
}

}  // namespace

cudaError_t launch_gg(const GgGemm& g, const GgPlan& pl, cudaStream_t st) {
  if (pl.few) return launch_gg_few(g, st);
  Prepared q;
  const cudaError_t err = prepare(g, pl, q);
  if (err != cudaSuccess) return err;
  switch (g.form) {
    case GG_W_K: return launch_form<GG_W_K>(pl, q.mw, q.ma, q.mr, q.p, q.units, st);
    case GG_W_M: return launch_form<GG_W_M>(pl, q.mw, q.ma, q.mr, q.p, q.units, st);
    default: return launch_form<GG_ROWS>(pl, q.mw, q.ma, q.mr, q.p, q.units, st);
  }
}

// Side by side where memory bounds both and neither is split: the weights read and
// written at 6.6 and 3.8 TB/s, against the products at 1.5 PFLOP/s.  us one after the other
// and side by side: 16 experts, 1408 x 2048, 517 rows, float32, 66 and 55; 2 experts, 12792 x
// 2448, 353 rows 88 and 77; 128 experts, 2048 x 1536, 4096 rows (by Zipf's law) 281 and 286,
// 16384 rows 356 and 348; 8 experts, 4096 x 14336, 128 rows 310 and 321, 1024 rows 338 and 340,
// 1500 rows 382 and 386.  (Where the launches are long it makes little difference.)  Also where
// the rows' by itself would be gg_few's, which adds in another order: 4096 x 4096 stored [K, N],
// 1 row 24.9 and 19.4, 16 rows 31.5 and 19.4; 8 experts, 2048 x 768, 8 rows 22.3 and 14.7; 64
// experts there, 4 rows 41.5 and 44.4.
bool gg_side_by_side(const GgGemm& rows, const GgGemm& weights) {
  const int64_t n = (int64_t)rows.M * rows.K;
  const double live = (double)std::min<int64_t>(rows.R, rows.E);
  const double read = live * n * 2 / 6.6e6;
  const double write = (double)rows.E * n * (weights.out_dtype == MQ_DTYPE_F32 ? 4 : 2) / 3.8e6;
  const double flops = 4.0 * rows.R * n / 1.5e9;
  return rows.M > 128 && rows.K > 128 && read + write > 1.3 * flops &&
         gg_plan(rows.form, rows.R, rows.E, rows.M, rows.N, rows.K).splits == 1 &&
         gg_plan(GG_ROWS, weights.R, weights.E, weights.M, weights.N, weights.K).splits == 1;
}

cudaError_t launch_gg_both(const GgGemm& rows, const GgGemm& weights, cudaStream_t st) {
  const GgPlan pair = {false, 256, true, 1};
  Prepared r, w;
  cudaError_t err = prepare(rows, pair, r);
  if (err == cudaSuccess) err = prepare(weights, pair, w);
  if (err != cudaSuccess) return err;
  // SMs by what a pair of them reads and writes (102 and 85 GB/s measured), within the
  // shares that were tried, and more for the rows' side where an expert has many.  us with 30,
  // 35, 40, 45 and 50 % of them for it: 128 experts, 1536 x 2048, 4096 rows 340, 309, 287, 274,
  // 272; float32: 87 experts, 12528 x 344, 284 rows 449, 484, 531, 586, 637; 8 experts, 4096 x
  // 14336, 512 rows 491, 465, 480, 484, 533; 16 experts, 1408 x 2048, 517 rows 58, 54, 55, 56,
  // 62; 128 experts, 2048 x 1536, 16384 rows 455, 428, 409, 436, 480.
  const double read = (double)std::min<int64_t>(rows.R, rows.E) * 2 / 102;
  const double write = (double)rows.E * (weights.out_dtype == MQ_DTYPE_F32 ? 4 : 2) / 85;
  const int pairs = tc_num_sms() / 2;
  const double least = 0.3 + 0.1 * std::min(1.0, (double)rows.R / (128.0 * rows.E));
  int first = (int)(pairs * std::min(0.5, std::max(least, read / (read + write) + 0.05)));
  first = (int)std::max<int64_t>(1, std::min<int64_t>(first, r.units));
  const int second = (int)std::max<int64_t>(1, std::min<int64_t>(pairs - first, w.units));
  constexpr size_t smem = std::max({Cfg<GG_W_K, 256, 2>::kSmem, Cfg<GG_ROWS, 256, 2>::kSmem});
  const bool by_k = rows.form == GG_W_K;
  const bool seg = segmented<GG_W_K>(r.p) || segmented<GG_ROWS>(w.p);
  const auto kern = seg ? (by_k ? gg_both<GG_W_K, true> : gg_both<GG_W_M, true>)
                        : (by_k ? gg_both<GG_W_K, false> : gg_both<GG_W_M, false>);
  static std::atomic<uint64_t> ready[4];
  err = allow_smem(kern, smem, ready[seg * 2 + by_k]);
  if (err != cudaSuccess) return err;
  return launch_pdl_cluster(kern, dim3(2 * (first + second)), dim3(kThreads), 2, smem, st, r.mw, r.ma, r.mr, w.mw,
                            w.ma, w.mr, r.p, w.p, (uint32_t)(2 * first));
}
