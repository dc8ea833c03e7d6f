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
//          Nothing is masked, and what another request's adapter holds (infinities,
//          NaN) stays in the columns that are not kept.  x, base and out are never
//          gathered; only h, between the launches, has a tile's rows by group.
//
// Tiles, first launch (lora_down): h = A x in float32.  Groups are packed into the 128
// lanes of an accumulator (eight of rank 16, two of rank 64), x is the other operand; a
// cluster's CTAs take a share of K each and sum their h through distributed shared
// memory.  s h is written as the second product's operand, in two 16-bit parts: h = 2^m
// (hi + lo), m by the exponent of the row's largest |h|: 16 bits of precision for bf16 and
// 22 for f16, whose range it cannot leave either, for twice a small product; in three (24
// bits) where the result is float32.
// Second launch (lora_up): a group's product has the columns of its own rows only, so
// that groups in different blocks of 16 rows share an accumulator and a tile of several
// requests takes one turn of the epilogue, or a few.  base comes by TMA and goes back, with
// the sums added, the same way.
//
// Measured: rows, 4096 x 4096, rank 16: 1 row 5.5 to 6.1 us, 64 rows of 48 adapters 7.1 (a
// chain of dependent reads: ids, A, the exchange; B is on its way meanwhile).  Tiles: 4099
// rows of 16 adapters, rank 64, 38 us (67 MB of base and out beside two launches' ways in and
// out); 4096 rows of 64 experts, 2048 x 2816, rank 32, 16 groups in a tile, 70 us (short steps
// for each group and 128 outputs: DRAM at 30 %, the tensor pipe at 12 and 4 %).  Float32
// results, 2000 rows of 8 adapters, rank 16, 4096 x 4096: 52 us.
#include "lora.cuh"
#include "pipe.cuh"

#include <algorithm>
#include <cmath>
#include <type_traits>

namespace {

using namespace mq::pipe;

constexpr int kTile = 128;     // rows of a tile at most; outputs of an accumulator
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

__device__ __forceinline__ float as_float(float v) { return v; }
__device__ __forceinline__ float as_float(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float as_float(__half v) { return __half2float(v); }
template <typename T>
__device__ __forceinline__ T from_float(float v) {
  if constexpr (sizeof(T) == 4) return v;
  else if constexpr (std::is_same_v<T, __half>) return __float2half_rn(v);
  else return __float2bfloat16_rn(v);
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

  // A x over this CTA's vectors of eight; a warp takes two ranks at a time, with
  // two vectors of each and of x in flight.
  const int vecs = p.K / 8;
  const int v0 = (int)((int64_t)vecs * rank / kCluster), v1 = (int)((int64_t)vecs * (rank + 1) / kCluster);
  constexpr int kRanks = 2, kDeep = 2;
  bool met = false;
  for (int j0 = warp; j0 < p.r; j0 += 8 * kRanks) {
    float acc[kRanks] = {};
    for (int v = v0 + lane; v < v1; v += 32 * kDeep) {
      uint4 xv[kDeep], av[kDeep][kRanks];
#pragma unroll
      for (int d = 0; d < kDeep; ++d) {
        const int w = v + 32 * d;
        xv[d] = w < v1 ? __ldg(reinterpret_cast<const uint4*>(x) + w) : zero;
#pragma unroll
        for (int i = 0; i < kRanks; ++i)
          av[d][i] = w < v1 && j0 + 8 * i < p.r
                         ? __ldg(reinterpret_cast<const uint4*>(a + (int64_t)(j0 + 8 * i) * p.K) + w)
                         : zero;
      }
      float xf[8], af[8];
#pragma unroll
      for (int d = 0; d < kDeep; ++d) {
        unpack8(xv[d], BF16, xf);
#pragma unroll
        for (int i = 0; i < kRanks; ++i) {
          unpack8(av[d][i], BF16, af);
          acc[i] = dot8(xf, af, acc[i]);
        }
      }
    }
    if (!met) {
      // the first outputs' rows of B and base are on their way while the sums meet
#pragma unroll
      for (int i = 0; i < kAhead; ++i) fetch(first + i * kOuts, i);
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
constexpr int kNone = 255, kOut = 254;  // rows without an adapter; rows that are not written

// Groups of a tile's rows, as the first launch works them out.
struct Table {
  int key[kTile];                  // group of a row as an index into the adapters (l E + e); -1 none, -2 not written
  int group_key[kTile];            // key of each of the tile's groups, in order of their first rows
  unsigned blocks[kTile];          // the 16-row blocks that hold rows of a group
  alignas(16) uint8_t slot[kTile]; // a row's group; kNone, kOut
  unsigned first[kTile / 32];
  int groups, rows;
  int inside;                      // rows that are written
};

// What the second launch needs of it, in global memory.  It has the tile's rows in the
// order of their groups (then those without an adapter, then those that are not
// written): a row's place.  A group's accumulator has columns for the 16-row blocks of
// its places.  Groups whose blocks do not meet share one: each has a color, and colors 2 i
// and 2 i + 1 are round i.  (In the order that the rows come in, a group's range would reach
// from its first row to its last: 16 groups at random in a tile took 3.6 rounds, so 2.)
struct TileTable {
  alignas(16) uint8_t color[kTile];  // by place: color of the row's group; kNone, kOut
  alignas(16) uint8_t row[kTile];    // by place: the row
  float row_scale[kTile];            // by place: 2^m of the row
  int group_key[kTile];              // by round
  int group_range[kTile];            // first block | behind its last << 8 | color << 16
  int round_start[kTile / 2 + 4];    // first group of a round
  int groups, rounds, rows, inside;
};
static_assert(sizeof(TileTable) % 16 == 0, "copied in steps of 16 bytes");

// Fills in the table of the tile of `rows` rows from row0 on, with all threads of the CTA (at least kTile);
// `offsets` is a copy of the experts' in shared memory (null: one expert).
// `id`: thread t's row's adapter (any value behind the last row).
__device__ __forceinline__ void build_table(Table& tb, const LoraArgs& p, const int* offsets, bool bad,
                                            int64_t row0, int rows, int id) {
  const int t = threadIdx.x;
  int key = -2;
  if (t < kTile) {
    if (t < rows && !bad) {
      const int64_t row = row0 + t;
      const int l = id;
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
  __syncthreads();
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
  __syncthreads();
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
  __syncthreads();
}

// A tile's rows in the order of their groups.
struct Places {
  int begin[kTile + 2];    // first place of a group, of rows without an adapter (kTile), of others
  int fill[kTile + 2];     // while they are worked out: rows of each so far
  uint8_t of_row[kTile];
  uint8_t color[kTile];    // of a group
};

__device__ __forceinline__ int place_class(int slot) {
  return slot == kNone ? kTile : slot == kOut ? kTile + 1 : slot;
}

// By one warp.
__device__ __forceinline__ void sort_rows(Places& pl, const Table& tb, int lane) {
  constexpr int kClasses = kTile + 2;
  for (int i = lane; i < kClasses; i += 32) pl.fill[i] = 0;
  __syncwarp();
  unsigned peers[kTile / 32];
  int cls[kTile / 32], before[kTile / 32];
#pragma unroll
  for (int q = 0; q < kTile / 32; ++q) {
    cls[q] = place_class(tb.slot[q * 32 + lane]);
    peers[q] = __match_any_sync(0xffffffffu, cls[q]);
    const int rank = __popc(peers[q] & ((1u << lane) - 1u));
    const int so_far = pl.fill[cls[q]];
    before[q] = so_far + rank;
    __syncwarp();
    if (rank == 0) pl.fill[cls[q]] = so_far + __popc(peers[q]);
    __syncwarp();
  }
  int carry = 0;
  for (int i0 = 0; i0 < kClasses; i0 += 32) {
    const int n = i0 + lane < kClasses ? pl.fill[i0 + lane] : 0;
    int sum = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane >= o) sum += v;
    }
    if (i0 + lane < kClasses) pl.begin[i0 + lane] = carry + sum - n;
    carry += __shfl_sync(0xffffffffu, sum, 31);
  }
  __syncwarp();
#pragma unroll
  for (int q = 0; q < kTile / 32; ++q) pl.of_row[q * 32 + lane] = (uint8_t)(pl.begin[cls[q]] + before[q]);
  __syncwarp();
}

// The second launch's table of a tile, by one warp: colors in the order of the groups,
// each the least that no group of a meeting range has.
__device__ __forceinline__ void write_table(TileTable* to, const Table& tb, Places& pl, int lane) {
  auto first_block = [&](int g) { return pl.begin[g] >> 4; };
  auto end_block = [&](int g) { return (pl.begin[g] + pl.fill[g] + 15) >> 4; };
  unsigned used[4] = {};  // blocks taken, of colors lane, lane + 32, ...
  int colors = 0;
  for (int g = 0; g < tb.groups; ++g) {
    const unsigned range = (1u << end_block(g)) - (1u << first_block(g));
    bool placed = false;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      if (placed) continue;
      const unsigned free = __ballot_sync(0xffffffffu, (used[q] & range) == 0);
      if (!free) continue;
      const int l = __ffs(free) - 1;
      if (lane == l) used[q] |= range;
      if (lane == 0) pl.color[g] = (uint8_t)(q * 32 + l);
      colors = max(colors, q * 32 + l + 1);
      placed = true;
    }
  }
  __syncwarp();
  const int rounds = (colors + 1) / 2;
  int n = 0;
  for (int rd = 0; rd < rounds; ++rd) {
    if (lane == 0) to->round_start[rd] = n;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int g = q * 32 + lane;
      const bool here = g < tb.groups && pl.color[g] >> 1 == rd;
      const unsigned all = __ballot_sync(0xffffffffu, here);
      if (here) {
        const int at = n + __popc(all & ((1u << lane) - 1u));
        to->group_key[at] = tb.group_key[g];
        to->group_range[at] = first_block(g) | end_block(g) << 8 | pl.color[g] << 16;
      }
      n += __popc(all);
    }
  }
  for (int t = lane; t < kTile; t += 32) {
    const int s = tb.slot[t], place = pl.of_row[t];
    to->row[place] = (uint8_t)t;
    to->color[place] = s < kOut ? pl.color[s] : (uint8_t)s;
  }
  if (lane == 0) {
    to->round_start[rounds] = n;
    to->groups = tb.groups;
    to->rounds = rounds;
    to->rows = tb.rows;
    to->inside = tb.inside;
  }
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

// Two values rounded to 16 bits, the first in the low half.
template <bool BF16>
__device__ __forceinline__ uint32_t half_pair(float lo, float hi) {
  if constexpr (BF16) {
    const __nv_bfloat162 t = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&t);
  } else {
    const __half2 t = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&t);
  }
}
__device__ __forceinline__ float from_half_bits(uint16_t v, bool bf16) {
  return bf16 ? __uint_as_float((uint32_t)v << 16) : __half2float(__ushort_as_half(v));
}

// The magnitude of v, 0 where it is infinite or NaN.
__device__ __forceinline__ float finite(float v) { return isfinite(v) ? fabsf(v) : 0.0f; }

// f as the sum of two 16-bit values, both of its sign and neither zero: what an infinite
// factor makes of them then has the sign, and the kind, that it has with f.  The first is
// rounded towards zero, or, where that leaves nothing for the second, a unit lower.  (Of f16
// f has two units of 2^-24 at least.)
template <bool BF16>
__device__ __forceinline__ void two_parts(float f, float& hi, float& rest) {
  if constexpr (BF16) {
    hi = __uint_as_float(__float_as_uint(f) & 0xffff0000u);
    if (hi == f) hi = __uint_as_float(__float_as_uint(f) - 0x10000u);
  } else {
    const uint16_t h = __half_as_ushort(__float2half_rz(f));
    hi = from_half_bits(h, false);
    if (hi == f) hi = from_half_bits(h - 1, false);
  }
  rest = f - hi;
}

// v, or `least` of its sign.
__device__ __forceinline__ float raised(float v, float least) { return copysignf(fmaxf(fabsf(v), least), v); }

// v * down in PARTS parts (infinite or NaN, or zero, where v is).  Too small a value is
// raised, by at most 2^-36 of the row's largest.
template <bool BF16, int PARTS>
__device__ __forceinline__ void split_value(float v, float down, float (&part)[PARTS]) {
  constexpr float kUnit = BF16 ? 0.0f : 0x1p-24f;
  two_parts<BF16>(raised(copysignf(v * down, v), BF16 ? 0x1p-90f : 2 * kUnit), part[0], part[1]);
  if constexpr (PARTS == 3) two_parts<BF16>(raised(part[1], 2 * kUnit), part[1], part[2]);
  if constexpr (!BF16) part[PARTS - 1] = copysignf(fmaxf(fabsf(part[PARTS - 1]), kUnit), v);
  if (v == 0 || !isfinite(v))
#pragma unroll
    for (int i = 0; i < PARTS; ++i) part[i] = v;
}

// Four values' parts, `apart` elements from one another.
template <bool BF16, int PARTS>
__device__ __forceinline__ void store_parts(uint16_t* dst, int apart, const float4& v, float down) {
  float part[4][PARTS];
  split_value<BF16>(v.x, down, part[0]);
  split_value<BF16>(v.y, down, part[1]);
  split_value<BF16>(v.z, down, part[2]);
  split_value<BF16>(v.w, down, part[3]);
#pragma unroll
  for (int i = 0; i < PARTS; ++i)
    *reinterpret_cast<uint2*>(dst + i * apart) = make_uint2(half_pair<BF16>(part[0][i], part[1][i]), half_pair<BF16>(part[2][i], part[3][i]));
}

// ---- first launch: h = A x, its sum over the K splits, and s h in 16-bit parts ----
// A cluster holds the K splits of a tile (or of a part of its accumulators).
constexpr int kDownThreads = 256;
constexpr int kXSlots = 4, kASlots = 4;  // of 16 KB: a stage of x, of an accumulator's groups
constexpr int kBatch = 4;                // accumulators at a time
// Stages whose sum stays in tensor memory, whose additions round towards zero, for results
// of 32 and of 16 bits; longer sums are made of such segments, added up in shared memory, to
// nearest (as in grouped_gemm.cu).  Then two accumulators at a time, in two buffers.
constexpr int kSegment = 4, kSegment16 = 16;

struct DownCtl {
  uint64_t x_full[kXSlots], x_empty[kXSlots], a_full[kASlots], a_empty[kASlots];
  uint64_t acc_full[2], acc_empty[2], drain;
  uint32_t tmem;
  volatile int abort_flag;
};
struct DownShared {
  DownCtl ctl;
  Table table;
  int offsets[kMaxE + 1];
  Places places;
};
// floats between the rows of h in shared memory
__host__ __device__ constexpr int h_pitch(int rp) { return rp + 4; }
// s h is the sum of two 16-bit values, of three where the result is float32, which shows more
// of it: 16 bits for bf16 and 22 for f16, or 24.
constexpr int kMaxParts = 3;
int parts_of(int out_dtype) { return out_dtype == MQ_DTYPE_F32 ? 3 : 2; }
// 16-bit elements between the rows of the second product's operand
__host__ __device__ constexpr int h_row(int rp, int parts) { return (parts * rp + 63) / 64 * 64; }

struct DownShape {
  int height;  // rows of a tile
  int rp;      // r rounded up to 16, 32, 64 or 128
  int splits;  // K splits: CTAs of a cluster
  int mparts;  // clusters among which a tile's accumulators are divided
  int segment; // stages whose sum stays in tensor memory
  TileTable* tables;
  uint16_t* h;  // [tiles * height][h_row(rp, parts)], a tile's rows by place
};

// BF16: x and the adapters are.
template <bool BF16, int PARTS>
__global__ void __launch_bounds__(kDownThreads, 1)
    lora_down(const __grid_constant__ CUtensorMap map_x, const __grid_constant__ CUtensorMap map_a,
              const LoraArgs p, const DownShape d) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* xs = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  uint8_t* as = xs + kXSlots * kSlot;
  float* hs = reinterpret_cast<float*>(as + kASlots * kSlot);
  DownShared* sh = reinterpret_cast<DownShared*>(hs + kTile * h_pitch(d.rp));
  DownCtl* ctl = &sh->ctl;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    tma_prefetch_desc(&map_x);
    tma_prefetch_desc(&map_a);
    for (int i = 0; i < kXSlots; ++i) {
      mbar_init(&ctl->x_full[i], 1);
      mbar_init(&ctl->x_empty[i], 1);
    }
    for (int i = 0; i < kASlots; ++i) {
      mbar_init(&ctl->a_full[i], 1);
      mbar_init(&ctl->a_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&ctl->acc_full[i], 1);
      mbar_init(&ctl->acc_empty[i], 4);
    }
    mbar_init(&ctl->drain, 1);
    ctl->abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(&ctl->tmem, 512);
    tmem_relinquish();
  }
  const int split = blockIdx.x % d.splits;  // the rank in the cluster
  const int mpart = blockIdx.x / d.splits % d.mparts;
  const int tile = blockIdx.x / (d.splits * d.mparts);
  const int64_t row0 = (int64_t)tile * d.height;
  const int rows = (int)min((int64_t)d.height, p.R - row0);
  const int nst = (p.K + 63) / 64;
  const int s0 = (int)((int64_t)nst * split / d.splits), s1 = (int)((int64_t)nst * (split + 1) / d.splits);
  mq::pdl_wait();
  mq::pdl_trigger();
  const int id = tid < rows ? p.ids[row0 + tid] : -1;
  const bool bad = copy_offsets(p, sh->offsets);
  // the first stages of x are on their way while the groups are worked out
  const int early = min(kXSlots, s1 - s0);
  if (warp == 0 && elect_one())
    for (int i = 0; i < early; ++i) {
      mbar_arrive_expect_tx(&ctl->x_full[i], d.height * 128);
      tma_load_2d(xs + i * kSlot, &map_x, &ctl->x_full[i], (s0 + i) * 64, (int)row0);
    }
  __syncwarp();
  build_table(sh->table, p, p.offsets ? sh->offsets : nullptr, bad, row0, rows, id);
  const Table& tb = sh->table;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ctl->tmem;
  const int per = kTile / d.rp;                      // groups of an accumulator
  const int accs = (tb.groups + per - 1) / per;      // accumulators of the tile
  const int mine = accs > mpart ? (accs - mpart + d.mparts - 1) / d.mparts : 0;
  const int bufs = s1 - s0 > d.segment ? 2 : 1;      // of the accumulators
  const int batch = kBatch / bufs;
  // the scaling of this thread's (first) row of the last step, which is short
  const int row_share = kTile / d.splits, sub = tid & 7;
  auto scaling_of = [&](int i) {
    const int key = tb.key[split * row_share + i];
    return p.scaling && key >= 0 ? p.scaling[key / p.E] : 1.0f;
  };
  const float first_scaling = (tid >> 3) < row_share ? scaling_of(tid >> 3) : 1.0f;

  if (warp == 0) {
    const bool el = elect_one();
    uint32_t it = 0;
    bool ok = true;
    for (int b0 = 0; b0 < mine && ok; b0 += batch)
      for (int s = s0; s < s1; ++s, ++it) {
        if (it < (uint32_t)early) continue;
        const uint32_t slot = it % kXSlots;
        ok = warp_wait(&ctl->x_empty[slot], ((it / kXSlots) & 1) ^ 1, ctl, p.status);
        if (!ok) break;
        if (el) {
          mbar_arrive_expect_tx(&ctl->x_full[slot], d.height * 128);
          tma_load_2d(xs + slot * kSlot, &map_x, &ctl->x_full[slot], s * 64, (int)row0);
        }
      }
    it = max(it, (uint32_t)early);
    if (ctl->abort_flag || !mine)  // loads that nothing waits for land before the CTA goes
      for (uint32_t j = it < kXSlots ? 0 : it - kXSlots; j < it; ++j)
        wait_drain(&ctl->x_full[j % kXSlots], (j / kXSlots) & 1);
  } else if (warp == 2) {
    const bool el = elect_one();
    uint32_t it = 0;
    bool ok = true;
    for (int b0 = 0; b0 < mine && ok; b0 += batch)
      for (int s = s0; s < s1 && ok; ++s)
        for (int b = b0; b < min(b0 + batch, mine); ++b, ++it) {
          const uint32_t slot = it % kASlots;
          ok = warp_wait(&ctl->a_empty[slot], ((it / kASlots) & 1) ^ 1, ctl, p.status);
          if (!ok) break;
          const int g0 = (mpart + b * d.mparts) * per, n = min(per, tb.groups - g0);
          if (el) {
            mbar_arrive_expect_tx(&ctl->a_full[slot], n * d.rp * 128);
            for (int i = 0; i < n; ++i)
              tma_load_3d(as + slot * kSlot + i * d.rp * 128, &map_a, &ctl->a_full[slot], s * 64, 0,
                          tb.group_key[g0 + i]);
          }
        }
    if (ctl->abort_flag)
      for (uint32_t j = it < kASlots ? 0 : it - kASlots; j < it; ++j)
        wait_drain(&ctl->a_full[j % kASlots], (j / kASlots) & 1);
  } else if (warp == 1) {
    const bool el = elect_one();
    const uint32_t idesc = idesc_16(p.bf16, kTile, ceil16(tb.rows), false, false);
    uint32_t x_it = 0, a_it = 0;
    Ring ar;
    bool ok = true;
    for (int b0 = 0; b0 < mine && ok; b0 += batch) {
      const int b1 = min(b0 + batch, mine);
      for (int s = s0; s < s1 && ok;) {
        const int first = s, end = min(s + d.segment, s1);
        ok = warp_wait(&ctl->acc_empty[ar.slot], ar.turn ^ 1, ctl, p.status);
        tc_fence_after();
        const uint32_t acc = tmem + ar.slot * batch * kTile;
        for (; s < end && ok; ++s, ++x_it) {
          const uint32_t xslot = x_it % kXSlots;
          ok = warp_wait(&ctl->x_full[xslot], (x_it / kXSlots) & 1, ctl, p.status);
          const uint64_t bd = smem_desc_k_sw128(smem_addr(xs + xslot * kSlot));
          for (int b = b0; b < b1 && ok; ++b, ++a_it) {
            const uint32_t aslot = a_it % kASlots;
            ok = warp_wait(&ctl->a_full[aslot], (a_it / kASlots) & 1, ctl, p.status);
            if (!ok) break;
            tc_fence_after();
            if (el) {
              const uint64_t ad = smem_desc_k_sw128(smem_addr(as + aslot * kSlot));
#pragma unroll
              for (int j = 0; j < 4; ++j)
                mma_ss<1>(acc + (b - b0) * kTile, ad + j * 2, bd + j * 2, idesc, (s > first) | j);
              mma_commit(&ctl->a_empty[aslot]);
            }
          }
          if (ok && el) mma_commit(&ctl->x_empty[xslot]);
        }
        if (ok && el) mma_commit(&ctl->acc_full[ar.slot]);
        ar.next(bufs);
      }
    }
    if (el) mma_commit(&ctl->drain);
    wait_drain(&ctl->drain, 0);
  } else if (warp == 3) {
    sort_rows(sh->places, tb, lane);
    if (split == 0 && mpart == 0) write_table(d.tables + tile, tb, sh->places, lane);
  } else {
    // A lane is one rank of one of the accumulator's groups.
    const int quad = warp & 3;
    const int gl = (quad * 32 + lane) / d.rp, j = (quad * 32 + lane) % d.rp;
    Ring ar;
    // A segment's sums to shared memory, or onto those that are there.
    auto take = [&](int b0, auto onto) {
      if (!warp_wait(&ctl->acc_full[ar.slot], ar.turn, ctl, p.status)) return false;
      tc_fence_after();
      for (int b = b0; b < min(b0 + batch, mine); ++b) {
        const int g = (mpart + b * d.mparts) * per + gl;
        const bool live = g < tb.groups;
        const unsigned any = __reduce_or_sync(0xffffffffu, live ? tb.blocks[g] : 0u);
        for (int c = 0; c < kTile / 16; ++c) {
          if (!(any >> c & 1)) continue;
          uint32_t v[16];
          tmem_ld16_sync(tmem + (ar.slot * batch + b - b0) * kTile + c * 16 + ((uint32_t)(quad * 32) << 16), v);
          const uint4 of = *reinterpret_cast<const uint4*>(tb.slot + c * 16);
          float* const at = hs + c * 16 * h_pitch(d.rp) + j;
          if constexpr (decltype(onto)::value) {  // (all reads before the writes: one after the other took 2 us)
            float old[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) old[i] = live ? at[i * h_pitch(d.rp)] : 0.0f;
#pragma unroll
            for (int i = 0; i < 16; ++i) v[i] = __float_as_uint(old[i] + __uint_as_float(v[i]));
          }
#pragma unroll
          for (int i = 0; i < 16; ++i)
            if (live && byte_of(of, i) == g) at[i * h_pitch(d.rp)] = __uint_as_float(v[i]);
          __syncwarp();
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&ctl->acc_empty[ar.slot]);
      ar.next(bufs);
      return true;
    };
    bool ok = true;
    for (int b0 = 0; b0 < mine && ok; b0 += batch) {
      ok = take(b0, std::false_type());
      for (int s = s0 + d.segment; s < s1 && ok; s += d.segment) ok = take(b0, std::true_type());
    }
  }
  tc_fence_before();
  __syncwarp();
  cluster_sync();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, 512);
  // The sum over the splits, in their order, of this CTA's share of the rows; eight
  // lanes per row, four ranks a lane and turn.
  for (int i = tid >> 3; i < row_share; i += kDownThreads / 8) {
    const int t = split * row_share + i, g = tb.slot[t];
    const bool live = g < kOut && g / per % d.mparts == mpart;
    const float s = i < kDownThreads / 8 ? first_scaling : scaling_of(i);
    float4 v[4];
    float most = 0;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      v[q] = make_float4(0.f, 0.f, 0.f, 0.f);
      const int j = q * 32 + sub * 4;
      if (live && j < p.r) {  // (behind r: 0, whatever x holds)
        const float* row = hs + t * h_pitch(d.rp) + j;
#pragma unroll 4
        for (int c = 0; c < d.splits; ++c) {
          const float4 w = load_cluster(map_rank(row, c));
          v[q].x += w.x;
          v[q].y += w.y;
          v[q].z += w.z;
          v[q].w += w.w;
        }
        v[q].x *= s;
        v[q].y *= s;
        v[q].z *= s;
        v[q].w *= s;
        most = fmaxf(fmaxf(most, fmaxf(finite(v[q].x), finite(v[q].y))), fmaxf(finite(v[q].z), finite(v[q].w)));
      }
    }
#pragma unroll
    for (int o = 4; o; o >>= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
    if (!live) continue;
    // 2^m with m the exponent of the largest, for f16, which has less room below than above,
    // less 14; kept to where 2^m and 2^-m are normal
    constexpr int below = BF16 ? 0 : 14;
    const int e = min(max((int)(__float_as_uint(most) >> 23), 1 + below), 253) - below;
    const float up = __uint_as_float((uint32_t)e << 23), down = __uint_as_float((uint32_t)(254 - e) << 23);
    const int place = sh->places.of_row[t];
    if (sub == 0) d.tables[tile].row_scale[place] = up;
    uint16_t* dst = d.h + (row0 + place) * h_row(d.rp, PARTS);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int j = q * 32 + sub * 4;
      if (j >= d.rp) continue;
      store_parts<BF16, PARTS>(dst + j, d.rp, v[q], down);
    }
  }
  __syncwarp();
  cluster_sync();  // (the others read this CTA's h until here)
}

// ---- second launch: out = base + B (s h) ----
// Warps 0 (base), 1 (B), 2 and 12 (MMAs), 3 (out), 4-11 (epilogue).
constexpr int kUpEpi = 8;
constexpr int kUpMma = 2;
constexpr int kUpThreads = 128 + 32 * kUpEpi + 32;
constexpr int kMaxUpSlots = 16;
constexpr int kIoBytes = kTile * kTile * 2;
constexpr int kMaxIo = 4;
constexpr int kGroupBytes = 65536;  // of slots at ranks up to 32

struct UpCtl {
  uint64_t full[kMaxUpSlots], empty[kMaxUpSlots];
  uint64_t acc_full[2], acc_empty[2];
  uint64_t io_full[kMaxIo], io_done[kMaxIo], io_empty[kMaxIo];
  uint64_t tile_full, go;
  uint64_t drain;
  uint32_t tmem;
  volatile int abort_flag;
};
struct UpShared {
  TileTable table;
  UpCtl ctl;
};

struct UpShape {
  int height;  // rows of a tile
  int rp;      // r rounded up to 16, 32, 64 or 128
  int gparts;  // parts of a tile's rounds
  int ntiles;  // of 128 outputs
  int shares;  // CTAs of a tile, among which its (part, 128 outputs) are divided
  int nio;     // buffers of base and out; 0: read and written element by element
  int line;    // bytes of a slot's lines: min(64, rp) ranks
  int slots;   // of 128 outputs by up to 64 ranks of a group
  const TileTable* tables;
};

// base and out in shared memory: 128 rows of 64 outputs (128 bytes, swizzled) twice.
// Element (row t, 16-byte chunk c of 8 outputs, 0 <= c < 16) of the tile:
__device__ __forceinline__ uint32_t io_offset(int t, int c) {
  return (uint32_t)((c >> 3) * (kIoBytes / 2) + t * 128 + (((c & 7) ^ (t & 7)) << 4));
}

// Two outputs of a row pair, m from memory and the sums a and b of the rows' scales: one
// rounding, where `in` has the rows' bits.
template <bool BF16>
__device__ __forceinline__ uint32_t add_pair(uint32_t m, uint32_t a, uint32_t b, float2 scale, bool add, uint32_t in) {
  float lo = 0, hi = 0;
  if (add) {
    lo = from_half_bits((uint16_t)(m & 0xffffu), BF16);
    hi = BF16 ? __uint_as_float(m & 0xffff0000u) : from_half_bits((uint16_t)(m >> 16), BF16);
  }
  lo = fmaf(__uint_as_float(a), scale.x, lo);
  hi = fmaf(__uint_as_float(b), scale.y, hi);
  return (m & ~in) | (half_pair<BF16>(lo, hi) & in);
}

// 0xff in the bytes of v that, halved, are `rd`.
__device__ __forceinline__ uint4 rows_of_round(const uint4& v, int rd) {
  const uint32_t want = (uint32_t)rd * 0x01010101u, low = 0x7f7f7f7fu;
  return make_uint4(__vcmpeq4(v.x >> 1 & low, want), __vcmpeq4(v.y >> 1 & low, want),
                    __vcmpeq4(v.z >> 1 & low, want), __vcmpeq4(v.w >> 1 & low, want));
}

// A round's sums of a lane's output n added to base where rows move element by element, for
// the 16-row blocks of epilogue part `sub`.
template <typename T>
__device__ __forceinline__ void plain_blocks(const LoraArgs& p, const TileTable& tb, uint32_t acc, int rd, int sub,
                                             int row0, int n) {
  constexpr int kParts = kUpEpi / 4;
  const T* base = static_cast<const T*>(p.base) + (int64_t)row0 * p.base_stride + min(n, p.N - 1);
  T* out = static_cast<T*>(p.out) + (int64_t)row0 * p.out_stride + n;
#pragma unroll 1
  for (int c0 = sub; c0 < kTile / 16; c0 += 2 * kParts) {
    uint4 in[2];
    uint32_t any = 0, second = 0;
    T old[2][16];
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      const uint4 color = *reinterpret_cast<const uint4*>(tb.color + (c0 + b * kParts) * 16);
      in[b] = rows_of_round(color, rd);
      any |= in[b].x | in[b].y | in[b].z | in[b].w;
      second |= in[b].x & color.x | in[b].y & color.y | in[b].z & color.z | in[b].w & color.w;
    }
    if (!any) continue;
#pragma unroll
    for (int b = 0; b < 2; ++b)
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        // (the tile's first row for those of other rounds: no branch holds the reads up)
        const int row = byte_of(in[b], i) ? tb.row[(c0 + b * kParts) * 16 + i] : 0;
        old[b][i] = p.base ? base[row * p.base_stride] : T(0.0f);
      }
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      const int c = c0 + b * kParts;
      uint32_t v[16];
      __syncwarp();
      tmem_ld16_sync(acc + c * 16, v);
      if (second & 0x01010101u) {  // some of the second color
        const uint4 color = *reinterpret_cast<const uint4*>(tb.color + c * 16);
        uint32_t w[16];
        tmem_ld16_sync(acc + kTile + c * 16, w);
#pragma unroll
        for (int i = 0; i < 16; ++i) v[i] = byte_of(color, i) & 1 ? w[i] : v[i];
      }
#pragma unroll
      for (int i = 0; i < 16; ++i)
        if (byte_of(in[b], i) && n < p.N)
          out[tb.row[c * 16 + i] * p.out_stride] =
              from_float<T>(fmaf(__uint_as_float(v[i]), tb.row_scale[c * 16 + i], as_float(old[b][i])));
    }
    __syncwarp();
  }
}

// Rows without an adapter there: base as it is, or 0.
template <typename T>
__device__ __forceinline__ void plain_copies(const LoraArgs& p, const TileTable& tb, int sub, int row0, int n) {
  const T* base = static_cast<const T*>(p.base) + (int64_t)row0 * p.base_stride + min(n, p.N - 1);
  T* out = static_cast<T*>(p.out) + (int64_t)row0 * p.out_stride + n;
#pragma unroll 1
  for (int c = sub; c < kTile / 16; c += kUpEpi / 4) {
    const uint4 color = *reinterpret_cast<const uint4*>(tb.color + c * 16);
    T v[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const int row = byte_of(color, i) == kNone ? tb.row[c * 16 + i] : 0;
      v[i] = p.base ? base[row * p.base_stride] : T(0.0f);
    }
#pragma unroll
    for (int i = 0; i < 16; ++i)
      if (byte_of(color, i) == kNone && n < p.N) out[tb.row[c * 16 + i] * p.out_stride] = v[i];
  }
}

// BF16: out is bf16.  PARTS: 16-bit values of which s h is the sum.
template <bool BF16, int PARTS>
__global__ void __launch_bounds__(kUpThreads, 1)
    lora_up(const __grid_constant__ CUtensorMap map_b, const __grid_constant__ CUtensorMap map_h,
            const __grid_constant__ CUtensorMap map_base, const __grid_constant__ CUtensorMap map_out,
            const LoraArgs p, const UpShape u) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* hs = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  const int hblocks = h_row(u.rp, PARTS) / 64;
  uint8_t* slots = hs + hblocks * kSlot;
  uint8_t* io = slots + u.slots * kTile * u.line;
  UpShared* sh = reinterpret_cast<UpShared*>(io + u.nio * kIoBytes);
  UpCtl* ctl = &sh->ctl;
  const TileTable& tb = sh->table;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    tma_prefetch_desc(&map_b);
    tma_prefetch_desc(&map_h);
    tma_prefetch_desc(&map_base);
    tma_prefetch_desc(&map_out);
    for (int i = 0; i < u.slots; ++i) {
      mbar_init(&ctl->full[i], 1);
      mbar_init(&ctl->empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&ctl->acc_full[i], kUpMma);
      mbar_init(&ctl->acc_empty[i], kUpEpi);
    }
    for (int i = 0; i < kMaxIo; ++i) {
      mbar_init(&ctl->io_full[i], 1);
      mbar_init(&ctl->io_done[i], kUpEpi);
      mbar_init(&ctl->io_empty[i], 1);
    }
    mbar_init(&ctl->tile_full, 1);
    mbar_init(&ctl->go, 1);
    mbar_init(&ctl->drain, kUpMma);
    ctl->abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 2) {
    tmem_alloc(&ctl->tmem, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ctl->tmem;
  mq::pdl_wait();
  mq::pdl_trigger();
  const int kblocks = (u.rp + 63) / 64;  // slots of a group's 128 outputs
  const int ksteps = (p.r + 15) / 16;
  const bool add = p.base != nullptr;

  // This CTA's units: a share of one tile's.
  const int per_tile = u.ntiles * u.gparts;
  const int tile = blockIdx.x / u.shares, share = blockIdx.x % u.shares;
  const int u0 = (int)((int64_t)per_tile * share / u.shares), u1 = (int)((int64_t)per_tile * (share + 1) / u.shares);
  const int row0 = tile * u.height;
  const TileTable* const table = u.tables + tile;
  // nothing to write: no rows, or no groups and base in place
  const bool idle = table->inside == 0 || (table->groups == 0 && p.base == p.out);
  // Every role's walk over the units: on_unit(n0, part) returns whether to go on.
  auto walk = [&](auto on_unit) {
    if (idle) return;
    int part = u0 / u.ntiles, nt = u0 - part * u.ntiles;
    for (int un = u0; un < u1; ++un) {
      if (!on_unit(nt * kTile, part)) return;
      if (++nt == u.ntiles) {
        nt = 0;
        ++part;
      }
    }
  };
  auto first_round = [&](const TileTable& t, int part) {
    return u.gparts == 1 ? (part ? t.rounds : 0) : t.rounds * part / u.gparts;
  };

  if (warp == 0) {
    // ------------------------------------------------------------- base --
    // Behind the first groups' loads, which would else wait for all CTAs' buffers.
    const bool el = elect_one();
    Ring io_r;
    uint32_t it = 0;
    bool ok = u.nio && (idle || warp_wait(&ctl->go, 0, ctl, p.status));
    if (ok)
      walk([&](int n0, int) {
        const uint32_t s = io_r.slot;
        if (!warp_wait(&ctl->io_empty[s], io_r.turn ^ 1, ctl, p.status)) return false;
        if (el) {
          if (add) {
            mbar_arrive_expect_tx(&ctl->io_full[s], u.height * 256);
            // (the second half may lie behind the last output: nothing is read there)
            tma_load_2d(io + s * kIoBytes, &map_base, &ctl->io_full[s], n0, row0);
            tma_load_2d(io + s * kIoBytes + kIoBytes / 2, &map_base, &ctl->io_full[s], n0 + 64, row0);
          } else {
            mbar_arrive(&ctl->io_full[s]);
          }
        }
        io_r.next(u.nio);
        ++it;
        return true;
      });
    if (ctl->abort_flag)  // loads in flight land before the CTA goes
      for (uint32_t j = it < (uint32_t)u.nio ? 0 : it - u.nio; j < it; ++j)
        wait_drain(&ctl->io_full[j % u.nio], (j / u.nio) & 1);
  } else if (warp == 1) {
    // --------------------------------- the tile's table and rows; groups' B --
    // (The groups' keys from global memory: sooner than by way of the table's copy.)
    const bool el = elect_one();
    if (el) {
      mbar_arrive_expect_tx(&ctl->tile_full, sizeof(TileTable) + hblocks * u.height * 128);
      for (int b = 0; b < hblocks; ++b) tma_load_2d(hs + b * kSlot, &map_h, &ctl->tile_full, b * 64, row0);
      bulk_load(&sh->table, table, sizeof(TileTable), &ctl->tile_full);
    }
    int keys[kTile / 32];
#pragma unroll
    for (int q = 0; q < kTile / 32; ++q) keys[q] = q * 32 + lane < table->groups ? table->group_key[q * 32 + lane] : 0;
    Ring w;
    uint32_t it = 0;
    bool gone = false;
    auto go = [&] {
      if (el && !gone) mbar_arrive(&ctl->go);
      gone = true;
    };
    walk([&](int n0, int part) {
      const int g0 = u.gparts == 1 ? 0 : table->round_start[first_round(*table, part)];
      const int g1 = u.gparts == 1 ? table->groups : table->round_start[first_round(*table, part + 1)];
      for (int g = g0; g < g1; ++g) {
        int key = 0;
#pragma unroll
        for (int q = 0; q < kTile / 32; ++q) {
          const int v = __shfl_sync(0xffffffffu, keys[q], g & 31);
          if (g >> 5 == q) key = v;
        }
        for (int k = 0; k < kblocks; ++k) {
          if (it == (uint32_t)u.slots) go();
          if (!warp_wait(&ctl->empty[w.slot], w.turn ^ 1, ctl, p.status)) return false;
          if (el) {
            mbar_arrive_expect_tx(&ctl->full[w.slot], kTile * u.line);
            tma_load_3d(slots + w.slot * kTile * u.line, &map_b, &ctl->full[w.slot], k * 64, n0, key);
          }
          w.next(u.slots);
          ++it;
        }
      }
      go();
      return true;
    });
    // loads that nothing else may have waited for land before the CTA goes
    wait_drain(&ctl->tile_full, 0);
    if (ctl->abort_flag)
      for (uint32_t j = it < (uint32_t)u.slots ? 0 : it - u.slots; j < it; ++j)
        wait_drain(&ctl->full[j % u.slots], (j / u.slots) & 1);
  } else if (warp == 2 || warp == 12) {
    // ----------------------------------------------------------- MMAs --
    // Of the columns only those of a group's range.  Groups are small (their four to
    // eight instructions take less than the way to them): two warps take them in turn,
    // each with slots of its own.
    const bool second = warp == 12;
    bool odd = false;
    const bool el = elect_one();
    const uint32_t idesc = idesc_16(p.bf16, kTile, 0, false, false);
    const uint32_t hb = smem_addr(hs), sb = smem_addr(slots);
    const uint64_t desc = smem_desc_k(0, u.line);
    Ring w, ar;
    if (warp_wait(&ctl->tile_full, 0, ctl, p.status))
      walk([&](int, int part) {
           const int r1 = first_round(tb, part + 1);
           for (int rd = first_round(tb, part); rd < r1; ++rd) {
             if (!warp_wait(&ctl->acc_empty[ar.slot], ar.turn ^ 1, ctl, p.status)) return false;
             tc_fence_after();
             const int g1 = tb.round_start[rd + 1];
             for (int g = tb.round_start[rd]; g < g1; ++g, odd = !odd && kblocks == 1) {
               if (odd != second) {
                 for (int k = 0; k < kblocks; ++k) w.next(u.slots);
                 continue;
               }
               const int range = tb.group_range[g];
               const int c0 = range & 0xff, c1 = range >> 8 & 0xff;
               const uint32_t acc = tmem + (ar.slot * 2 + (range >> 16 & 1)) * kTile + c0 * 16;
               const uint32_t id = idesc | (uint32_t)(c1 - c0) * 2 << 17;
               for (int k = 0; k < kblocks; ++k) {
                 if (!warp_wait(&ctl->full[w.slot], w.turn, ctl, p.status)) return false;
                 if (el) {
                   const uint64_t ad = desc + ((sb + w.slot * kTile * u.line) >> 4);
#pragma unroll
                   for (int j = 0; j < 4; ++j) {
                     if (k * 4 + j >= ksteps) break;
#pragma unroll
                     for (int part = 0; part < PARTS; ++part) {
                       const int c = k * 4 + j + part * (u.rp / 16);  // the step's place among the columns' k
                       const uint64_t bd = smem_desc_k_sw128(hb + (c >> 2) * kSlot + c0 * 2048);
                       mma_ss<1>(acc, ad + j * 2, bd + (c & 3) * 2, id, k | j | part);
                     }
                   }
                   mma_commit(&ctl->empty[w.slot]);
                 }
                 w.next(u.slots);
               }
             }
             if (el) mma_commit(&ctl->acc_full[ar.slot]);
             ar.next(2);
           }
           return true;
         });
    if (el) mma_commit(&ctl->drain);
    wait_drain(&ctl->drain, 0);
  } else if (warp == 3) {
    // -------------------------------------------------------------- out --
    // Finished buffers to memory: whole tiles by TMA, of others the rows that the unit
    // writes.  Apart from the epilogue, so that a buffer is free for the next load as
    // soon as it has been read.
    Ring io_r;
    if (u.nio && warp_wait(&ctl->tile_full, 0, ctl, p.status))
      walk([&](int n0, int part) {
          const uint32_t s = io_r.slot;
          if (!warp_wait(&ctl->io_done[s], io_r.turn, ctl, p.status)) return false;
          if (tb.inside == tb.rows && u.gparts == 1) {
            if (lane == 0) {
              tma_store_2d(&map_out, io + s * kIoBytes, n0, row0);
              if (n0 + 64 < p.N) tma_store_2d(&map_out, io + s * kIoBytes + kIoBytes / 2, n0 + 64, row0);
              bulk_commit();
              bulk_wait_read<0>();
            }
          } else {
            const int r0 = first_round(tb, part), r1 = first_round(tb, part + 1);
            const int live = min(kTile, p.N - n0);  // (a multiple of 8)
            for (int t = 0; t < tb.rows; ++t) {
              const int color = tb.color[t];
              const bool write = color == kNone ? part == 0 && p.base != p.out
                                                : color != kOut && color >> 1 >= r0 && color >> 1 < r1;
              if (!write || lane * 4 >= live) continue;
              const int row = tb.row[t];
              const uint2 q = *reinterpret_cast<const uint2*>(io + s * kIoBytes + io_offset(row, lane >> 1) + (lane & 1) * 8);
              *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.out) + ((int64_t)row0 + row) * p.out_stride +
                                        n0 + lane * 4) = q;
            }
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(&ctl->io_empty[s]);
          io_r.next(u.nio);
          return true;
        });
  } else {
    // ------------------------------------------------------- epilogue --
    // A lane is an output, the columns are the rows.
    constexpr int kParts = kUpEpi / 4;
    const int quad = warp & 3, sub = (warp - 4) >> 2;  // lanes, and which blocks of 16 rows
    Ring ar, io_r;
    const bool ready = warp_wait(&ctl->tile_full, 0, ctl, p.status);
    // By this warp's blocks of 16 places: the rows of places lane % 8 (a byte each) and
    // eight on, and the colors of the four places of which this lane has sums.
    constexpr int kBlocks = kTile / 16 / kParts;
    static_assert(kBlocks == 4, "a byte each, two blocks at a time");
    uint32_t rows0 = 0, rows1 = 0, own[kBlocks];
#pragma unroll
    for (int i = 0; i < kBlocks; ++i) {
      const int at = (sub + i * kParts) * 16;
      rows0 |= (uint32_t)tb.row[at + (lane & 7)] << i * 8;
      rows1 |= (uint32_t)tb.row[at + 8 + (lane & 7)] << i * 8;
      const uint16_t* pair = reinterpret_cast<const uint16_t*>(tb.color + at);
      own[i] = pair[lane & 3] | (uint32_t)pair[4 + (lane & 3)] << 16;
    }
    if (ready)
      walk([&](int n0, int part) {
          const int n = n0 + quad * 32 + lane;
          const uint32_t buf = smem_addr(io) + io_r.slot * kIoBytes;
          if (u.nio && !warp_wait(&ctl->io_full[io_r.slot], io_r.turn, ctl, p.status)) return false;
          const int r1 = first_round(tb, part + 1);
          for (int rd = first_round(tb, part); rd < r1; ++rd) {
            if (!warp_wait(&ctl->acc_full[ar.slot], ar.turn, ctl, p.status)) return false;
            tc_fence_after();
            const uint32_t acc = tmem + ar.slot * 2 * kTile + ((uint32_t)(quad * 32) << 16);
            if (u.nio) {
              // Whole 16-byte chunks of a row move either way (two-byte accesses, 32 a warp,
              // bound this loop), for two blocks at a time.
#pragma unroll
              for (int i0 = 0; i0 < kBlocks; i0 += 2) {
                uint32_t in[2], odd[2];
                bool any[2];
#pragma unroll
                for (int b = 0; b < 2; ++b) {
                  in[b] = __vcmpeq4(own[i0 + b] >> 1 & 0x7f7f7f7fu, (uint32_t)rd * 0x01010101u);
                  odd[b] = in[b] & own[i0 + b] & 0x01010101u;  // of the second color
                  any[b] = __any_sync(0xffffffffu, in[b]);
                }
                if (!any[0] && !any[1]) continue;
                uint32_t at[2][2], m[2][2][4];
#pragma unroll
                for (int b = 0; b < 2; ++b)
#pragma unroll
                  for (int h = 0; h < 2; ++h) {
                    at[b][h] = buf + io_offset((h ? rows1 : rows0) >> (i0 + b) * 8 & 0xff, quad * 4 + (lane >> 3));
                    ldmatrix_x4_trans(at[b][h], m[b][h]);
                  }
                const uint32_t c0 = acc + (sub + i0 * kParts) * 16, c1 = c0 + kParts * 16;
                uint32_t v[2][2][8];
                tmem_ld_frag16_sync(c0, c1, v);
                if (__any_sync(0xffffffffu, odd[0] | odd[1])) {
                  uint32_t w[2][2][8];
                  tmem_ld_frag16_sync(c0 + kTile, c1 + kTile, w);
#pragma unroll
                  for (int b = 0; b < 2; ++b)
#pragma unroll
                    for (int h = 0; h < 2; ++h)
#pragma unroll
                      for (int k = 0; k < 2; ++k)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {  // rows 2 (lane % 4) + e % 2 of the eight
                          uint32_t& x = v[b][k][4 * h + e];
                          x = odd[b] >> (16 * h + 8 * (e & 1)) & 1 ? w[b][k][4 * h + e] : x;
                        }
                }
#pragma unroll
                for (int b = 0; b < 2; ++b) {
                  if (!any[b]) continue;
#pragma unroll
                  for (int h = 0; h < 2; ++h) {
                    const float2 scale = *reinterpret_cast<const float2*>(
                        tb.row_scale + (sub + (i0 + b) * kParts) * 16 + h * 8 + 2 * (lane & 3));
                    const uint32_t mask = __byte_perm(in[b], 0, h ? 0x3322 : 0x1100);
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                      const int e = 4 * h + 2 * (k & 1);
                      m[b][h][k] = add_pair<BF16>(m[b][h][k], v[b][k >> 1][e], v[b][k >> 1][e + 1], scale, add, mask);
                    }
                    stmatrix_x4_trans(at[b][h], m[b][h]);
                  }
                }
              }
            } else {
              // Element by element, two blocks' reads in flight together.
              if (p.out_dtype == MQ_DTYPE_F32) plain_blocks<float>(p, tb, acc, rd, sub, row0, n);
              else if (p.out_dtype == MQ_DTYPE_BF16) plain_blocks<__nv_bfloat16>(p, tb, acc, rd, sub, row0, n);
              else plain_blocks<__half>(p, tb, acc, rd, sub, row0, n);
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&ctl->acc_empty[ar.slot]);
            ar.next(2);
          }
          // rows without an adapter: base as it is, or 0
          if (u.nio) {
            // (each warp where it has added itself: a block of rows is read and written whole)
            if (!add && part == 0)
              for (int c = sub; c < kTile / 16; c += kParts)
                for (int t = c * 16; t < c * 16 + 16; ++t)
                  if (tb.color[t] == kNone && lane < 4)
                    *reinterpret_cast<uint4*>(io + io_r.slot * kIoBytes + io_offset(tb.row[t], quad * 4 + lane)) =
                        make_uint4(0, 0, 0, 0);
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&ctl->io_done[io_r.slot]);
            io_r.next(u.nio);
          } else if (part == 0 && p.base != p.out) {
            if (p.out_dtype == MQ_DTYPE_F32) plain_copies<float>(p, tb, sub, row0, n);
            else if (p.out_dtype == MQ_DTYPE_BF16) plain_copies<__nv_bfloat16>(p, tb, sub, row0, n);
            else plain_copies<__half>(p, tb, sub, row0, n);
          }
          __syncwarp();
          return true;
        });
  }
  tc_fence_before();
  __syncwarp();  // (the barrier and the deallocation are for whole warps)
  __syncthreads();
  tc_fence_after();
  if (warp == 2) tmem_dealloc(tmem, 512);
}

// ------------------------------------------------------------ host side --
int padded_rank(int r) { return r <= 16 ? 16 : r <= 32 ? 32 : r <= 64 ? 64 : 128; }

template <bool BF16>
cudaError_t launch_rows(const LoraArgs& g, cudaStream_t st) {
  const dim3 grid((unsigned)g.R * kCluster), block(kRowThreads);
  if (g.r <= 8) return launch_pdl_cluster(lora_rows<BF16, 1>, grid, block, kCluster, 0, st, g);
  if (g.r <= 16) return launch_pdl_cluster(lora_rows<BF16, 2>, grid, block, kCluster, 0, st, g);
  if (g.r <= 32) return launch_pdl_cluster(lora_rows<BF16, 4>, grid, block, kCluster, 0, st, g);
  if (g.r <= 64) return launch_pdl_cluster(lora_rows<BF16, 8>, grid, block, kCluster, 0, st, g);
  return launch_pdl_cluster(lora_rows<BF16, 16>, grid, block, kCluster, 0, st, g);
}

// The workspace: tables, then the second product's operand.
struct LoraLayout {
  int64_t tiles;
  size_t h, total;
};
LoraLayout lora_layout(const LoraPlan& pl, int64_t R, int r) {
  LoraLayout y;
  y.tiles = (R + pl.height - 1) / pl.height;
  y.h = ((size_t)y.tiles * sizeof(TileTable) + 255) & ~(size_t)255;
  y.total = y.h + (size_t)y.tiles * pl.height * h_row(padded_rank(r), kMaxParts) * 2;
  return y;
}

// CTAs of a tile in the second launch, and the launch's time in units of 128 rows by 128
// outputs: the way to a CTA's first unit takes about as long as three.
int up_shares(int64_t tiles, int height, int per_tile, double* time = nullptr) {
  const int sms = tc_num_sms();
  int shares = 1;
  double best = 0;
  for (int i = 1; i <= 4; ++i) {  // shares that fill i waves; one to four where a share each does
    const int n = (int)std::min<int64_t>(per_tile, tiles <= sms ? i * sms / tiles : i);
    const double t = (double)((tiles * n + sms - 1) / sms) * ((per_tile + n - 1) / n * (height / 128.0) + 3);
    if (i == 1 || t < best) best = t, shares = n;
  }
  if (time) *time = best;
  return shares;
}

cudaError_t launch_down(const LoraArgs& g, const LoraPlan& pl, cudaStream_t st) {
  const CUtensorMapDataType dt = g.bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
  const LoraLayout y = lora_layout(pl, g.R, g.r);
  DownShape d;
  d.height = pl.height;
  d.rp = padded_rank(g.r);
  d.splits = pl.splits;
  d.mparts = pl.mparts;
  d.segment = g.out_dtype == MQ_DTYPE_F32 ? kSegment : kSegment16;
  d.tables = reinterpret_cast<TileTable*>(g.workspace);
  d.h = reinterpret_cast<uint16_t*>(g.workspace + y.h);
  CUtensorMap mx, ma;
  const cuuint64_t xd[2] = {(cuuint64_t)g.K, (cuuint64_t)g.R}, xs = 2 * (cuuint64_t)g.x_stride;
  const cuuint32_t xb[2] = {64, (cuuint32_t)pl.height};
  cudaError_t err = make_map(&mx, dt, 2, g.x, xd, &xs, xb);
  if (err != cudaSuccess) return err;
  const cuuint64_t ad[3] = {(cuuint64_t)g.K, (cuuint64_t)g.r, (cuuint64_t)g.L * g.E};
  const cuuint64_t as[2] = {2 * (cuuint64_t)g.K, 2 * (cuuint64_t)g.K * g.r};
  const cuuint32_t ab[3] = {64, (cuuint32_t)d.rp, 1};
  err = make_map(&ma, dt, 3, g.a, ad, as, ab);
  if (err != cudaSuccess) return err;
  constexpr size_t fixed = 1024 + (kXSlots + kASlots) * kSlot + sizeof(DownShared);
  static_assert(fixed + sizeof(float) * kTile * h_pitch(kMaxRank) <= kSmemMax, "shared memory");
  static_assert(fixed >= 120 * 1024, "one CTA per SM: each allocates all of tensor memory");
  const size_t smem = fixed + sizeof(float) * kTile * h_pitch(d.rp);
  static std::atomic<uint64_t> ready[4];
  const bool wide = parts_of(g.out_dtype) == 3;
  const auto kern = wide ? (g.bf16 ? lora_down<true, 3> : lora_down<false, 3>)
                         : (g.bf16 ? lora_down<true, 2> : lora_down<false, 2>);
  err = allow_smem(kern, kSmemMax, ready[2 * wide + g.bf16]);
  if (err != cudaSuccess) return err;
  return launch_pdl_cluster(kern, dim3((unsigned)(y.tiles * pl.splits * pl.mparts)), dim3(kDownThreads),
                            pl.splits, smem, st, mx, ma, g, d);
}

cudaError_t launch_up(const LoraArgs& g, const LoraPlan& pl, cudaStream_t st) {
  const CUtensorMapDataType dt = g.bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
  const LoraLayout y = lora_layout(pl, g.R, g.r);
  UpShape u;
  u.height = pl.height;
  u.rp = padded_rank(g.r);
  const int parts = parts_of(g.out_dtype);
  u.gparts = pl.gparts;
  u.ntiles = (g.N + kTile - 1) / kTile;
  u.tables = reinterpret_cast<const TileTable*>(g.workspace);
  // base and out by TMA: 16 bits, rows on 16-byte boundaries
  const bool base_ok = !g.base || (g.base_stride % 8 == 0 && (reinterpret_cast<uintptr_t>(g.base) & 15u) == 0);
  const bool tma = g.out_dtype != MQ_DTYPE_F32 && base_ok && g.out_stride % 8 == 0 && g.N % 8 == 0 &&
                   (reinterpret_cast<uintptr_t>(g.out) & 15u) == 0;
  // In flight at a time: as many buffers of base, and as many groups, as fit beside the
  // rows.  Two warps consume the groups' slots in turn (one where a group has two slots),
  // so a slot has to belong to one of them for good, and their number is even: a warp
  // that came to a slot of which the other had the last turn could be a whole turn ahead
  // of its barrier, whose parity cannot tell that from none.
  u.nio = !tma ? 0 : u.rp == 128 ? 3 : 4;
  u.line = std::min(u.rp, 64) * 2;
  u.slots = u.rp >= 64 ? 2 : kGroupBytes / (kTile * u.line);
  CUtensorMap mb, mh, mbase, mout;
  const cuuint64_t bd[3] = {(cuuint64_t)g.r, (cuuint64_t)g.N, (cuuint64_t)g.L * g.E};
  const cuuint64_t bs[2] = {2 * (cuuint64_t)g.r, 2 * (cuuint64_t)g.r * g.N};
  const cuuint32_t bb[3] = {(cuuint32_t)u.line / 2, kTile, 1};
  cudaError_t err = make_map(&mb, dt, 3, g.b, bd, bs, bb,
                             u.line == 128  ? CU_TENSOR_MAP_SWIZZLE_128B
                             : u.line == 64 ? CU_TENSOR_MAP_SWIZZLE_64B
                                            : CU_TENSOR_MAP_SWIZZLE_32B);
  if (err != cudaSuccess) return err;
  const cuuint64_t hd[2] = {(cuuint64_t)h_row(u.rp, parts), (cuuint64_t)y.tiles * pl.height}, hst = 2 * hd[0];
  const cuuint32_t hb[2] = {64, (cuuint32_t)pl.height};
  err = make_map(&mh, dt, 2, g.workspace + y.h, hd, &hst, hb);
  if (err != cudaSuccess) return err;
  mbase = mout = mb;
  if (tma) {
    const CUtensorMapDataType ot =
        g.out_dtype == MQ_DTYPE_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
    const cuuint64_t d[2] = {(cuuint64_t)g.N, (cuuint64_t)g.R};
    const cuuint64_t t0 = 2 * (cuuint64_t)g.base_stride, t1 = 2 * (cuuint64_t)g.out_stride;
    const cuuint32_t box[2] = {kTile / 2, (cuuint32_t)pl.height};
    err = make_map(&mout, ot, 2, g.out, d, &t1, box);
    if (err == cudaSuccess && g.base) err = make_map(&mbase, ot, 2, g.base, d, &t0, box);
    if (err != cudaSuccess) return err;
  }
  const size_t need = 1024 + h_row(u.rp, parts) / 64 * kSlot + (size_t)u.slots * kTile * u.line + (size_t)u.nio * kIoBytes + sizeof(UpShared);
  static_assert(1024 + 4 * kSlot + 2 * kSlot + 3 * kIoBytes + sizeof(UpShared) <= kSmemMax &&
                    1024 + 2 * kSlot + 2 * kSlot + 4 * kIoBytes + sizeof(UpShared) <= kSmemMax &&
                    1024 + kSlot + kGroupBytes + 4 * kIoBytes + sizeof(UpShared) <= kSmemMax &&
                    1024 + 6 * kSlot + kGroupBytes + sizeof(UpShared) <= kSmemMax,
                "shared memory");
  static_assert(kGroupBytes / (kTile * 32) <= kMaxUpSlots && kGroupBytes / (kTile * 32) % 2 == 0 &&
                    kGroupBytes / (kTile * 64) % 2 == 0,
                "a slot belongs to one of the two MMA warps");
  const size_t smem = std::max<size_t>(need, 120 * 1024);  // one CTA per SM: each allocates all of tensor memory
  static std::atomic<uint64_t> ready[3];
  const bool bf = g.out_dtype == MQ_DTYPE_BF16;
  const auto kern = parts == 3 ? lora_up<false, 3> : bf ? lora_up<true, 2> : lora_up<false, 2>;
  err = allow_smem(kern, kSmemMax, ready[parts == 3 ? 2 : bf]);
  if (err != cudaSuccess) return err;
  u.shares = up_shares(y.tiles, pl.height, u.ntiles * u.gparts);
  const int64_t grid = y.tiles * u.shares;
  return launch_pdl(kern, dim3((unsigned)grid), dim3(kUpThreads), smem, st, mb, mh, mbase, mout, g, u);
}

}  // namespace

size_t lora_workspace(const LoraPlan& pl, int64_t R, int r) { return lora_layout(pl, R, r).total; }

LoraPlan lora_plan(int64_t R, int K, int N, int r, int L, int E) {
  LoraPlan pl = {};
  const int sms = tc_num_sms();
  const double adapter = 2.0 * r * ((double)K + N);                     // bytes
  const double groups = std::min<double>((double)R, (double)L * E);    // at most
  pl.splits = pl.mparts = pl.gparts = 1;
  // Rows or tiles, by their estimated times in us.  Rows: 64 at a time, each its adapter.
  // Tiles: the way through two launches, more with more groups in a tile; a mean over
  // adapters in runs and at random.  Measured, rows and tiles (at random / in runs), 4096 x
  // 4096: rank 16, 48 adapters, 64 rows 6.1 and 25 / 26, 256 rows 22.6 and 28 / 18, 512 rows
  // 48.6 and 46 / 19; of 4 adapters, 128 rows 11.0 and 21 / 22, 256 rows 20.7 and 15.9 /
  // 14.7; rank 32, 128 rows 20.5 and 29 / 24, 192 rows 30.6 and 28 / 18; rank 64, 1 row 9.7
  // and 13.0, 64 rows 16.7 and 22.7, 96 rows 35 and 27 / 25; rank 128, 1 row 17.0 and 14.0.
  // 1024 x 1024, rank 8: 256 rows 16.3 and 27.5 / 23.5, 512 rows 30.8 and 31.7 / 23.5.
  const double waves = R / 64.0, many = std::max(1.0, waves);
  const double rows_us = 3 * many + 7 * adapter * 1e-6 * (many + waves);
  const double tiles_us = 13.5 + 0.15 * std::min(64.0, 4 * groups);
  pl.rows = rows_us <= tiles_us;
  if (pl.rows) return pl;
  // Rows of a tile, and K splits (with the clusters of that many CTAs that the GPU holds at
  // a time, measured with 152 SMs): by the estimated time of both launches, in units of 128 x
  // 128 outputs of the second, 1.45 us.  A stage of the first takes a quarter of one, half of
  // it for the groups; the way in and out of it six.
  constexpr int kOf152[4] = {152, 76, 36, 15};
  int held[4];
  for (int i = 0; i < 4; ++i) held[i] = std::max(1, kOf152[i] * sms / 152);
  const int ntiles = (N + kTile - 1) / kTile, stages = (K + 63) / 64;
  double best = 0;
  for (int h = kTile; h >= 64; h -= 16) {
    const int64_t n = (R + h - 1) / h;
    double up, down = 0;
    int splits = 1;
    up_shares(n, h, ntiles, &up);
    for (int i = 0; i < 4 && (i == 0 || stages >= 8 << i); ++i) {
      const double t = (double)((n + held[i] - 1) / held[i]) * ((stages >> i) * (0.13 + 0.13 * h / 128) + 6);
      if (i == 0 || t < down) down = t, splits = 1 << i;
    }
    if (h == kTile || up + down < 0.97 * best) best = up + down, pl.height = h, pl.splits = splits;
  }
  const int64_t tiles = (R + pl.height - 1) / pl.height;
  const int per = kTile / padded_rank(r);
  const int tile_groups = (int)std::min<double>(pl.height, groups);
  const int accs = (tile_groups + per - 1) / per;
  const int clusters = held[pl.splits == 1 ? 0 : pl.splits == 2 ? 1 : pl.splits == 4 ? 2 : 3];
  pl.mparts = (int)std::max<int64_t>(1, std::min<int64_t>(accs, clusters / tiles));
  while (pl.gparts * 2 <= tile_groups && tiles * ntiles * pl.gparts * 2 <= sms) pl.gparts *= 2;
  return pl;
}

cudaError_t launch_lora(const LoraArgs& g, const LoraPlan& pl, int which, cudaStream_t st) {
  if (pl.rows) return g.bf16 ? launch_rows<true>(g, st) : launch_rows<false>(g, st);
  return which == 0 ? launch_down(g, pl, st) : launch_up(g, pl, st);
}
