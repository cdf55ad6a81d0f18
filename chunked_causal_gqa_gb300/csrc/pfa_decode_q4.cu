// pfa_decode_q4.cu -- attention of few tokens of a batch of sequences over
// their 4-bit caches, on the tensor cores.
//
// For each sequence and kv head the T * group query rows form tiles of 8, 16 or 24 rows,
// and for each tile
//   s_j = scale * <q, k_j>,  out = sum_j 2^(s_j log2 e - m) v_j / sum_j 2^(s_j log2 e - m)
// with the maximum, the sum and the output in fp32.  A cache byte is read once for all rows of a
// tile, so with few rows HBM's bytes are the floor: 144 a key of a head of 128, 24 a clock of an
// SM, which leaves a warp's scheduler some 24 issue slots a key.
//
// Products: mma.sync m16n8k16 on halves, transposed: S' = K Q' and O' = V' P', keys and channels
// in the 16 rows of a product and the query rows in its 8 columns, so that a tile of 8 rows wastes
// none of it (a product of 16 query rows would be half padding for a group of 8 or
// less).  A code times its e4m3 scale is exact in half; q is scaled to 2^13..2^14 by a power of
// two for each row, which makes bf16 q exact but for elements 2^27 below the row's largest; the
// weights are rounded to half.  For fp32, q and the weights are a high and a low half, each with
// products of its own.
//
// Fragments straight from the packed rows, as the order of a contraction is free:
//   K: lane (g, qd) has 16 bytes, 32 channels, of the keys g and g + 8 of a product; two bytes are
//      its part of a k16 step.  A byte converts to a half pair, one product with the scale follows.
//   V: lane g has the 16 channels of one scale, 8 bytes, of four keys.  The products want a channel
//      of two keys side by side: (a & 0f..) | (b & 0f..) << 4 is such pairs of codes, four in a word.
//   P: the scores' layout is that of O', and movmatrix turns it into the second operand.
// Keys stand in a product in the order 0 5 1 4 2 7 3 6, and the 16-byte pieces of every other
// pair of rows in shared memory are swapped in halves, so that the reads of both are free of
// bank conflicts.
//
// The exponent's base rises only when a score passes it by 2^4, so that most units need no
// maximum across lanes and no rescaling: a weight is 2^(s - base) 2^11, at most 2^15.
//
// Work split and join: pfa_decode.cuh.  Four warps take a run's units of 64 (or 32) keys in turn, each with
// its own ring of 128 keys filled by cp.async; head_dim 512: four warps share a unit, each with 128
// channels, and exchange partial scores.  Two blocks an SM: the unit's 64 keys want the registers.
//
// Accumulated weights: the join leaves each row's maximum and sum, and 2^(s - m) / l, added up over
// the rows of a key, follows beside the join or in a kernel behind it.  With few rows the scores go to the
// workspace as they are made (4 bytes a row and key beside the 144 of the cache; making them again would
// read K again, 72 bytes a key, where 16 are written and 16 read for four rows); with many they are made
// again (scores_again).
//
// Measured on GB300, all kernels of a call, one pass among others:
//   1 sequence of 131072 keys, 32/8 heads of 128, bf16 (151 MB)      32.1 us (floor 22.2): streaming at
//     7.1 TB/s (each further sequence takes 21.3 us), and 9 us of start, uneven ends and join
//   32 sequences up to 8192 keys with weights (144 MB)               39.9 us (floor 21.2): the same, 8 us
//     of which are the scores, written and read, and the third launch
//   32 tokens at 16384 keys with weights                             56 us (floor 4.4): eight tiles of rows
//     convert the codes anew, 38 us; the weights 16
//   4 sequences, 3 tokens, window 1024, 8/2 heads of 512, fp32       12.1 us: two launches and some ten
//     latencies (floor 0.6)
// Steps (the first two cases): units of 32 keys, three blocks an SM, each copy with its own addresses
// and bounds 38.6 / 49.1; running offsets, score factor and base in one fused multiply-add, units of 64
// keys and two blocks 32.2 / 39.4 (512 instructions for 32 keys of a warp, 715 before).  128 registers
// and four blocks with two stages lost (42.8 / 50.2), and so did making the next unit's scores beside this
// one's sum (33.0 / 40.8): it is HBM that streams, not the products that wait.  More than 8 rows (16 of 63488
// keys 28.4 -> 24.4 us in the kernel, issuing 40 -> 45 % of the cycles, the tensor pipe 34 %): second operands shared
// through shared memory, and the scores of all keys of a unit side by side.
#include "pfa_decode.cuh"
#include "pfa_q4.cuh"

#include "../../include/pfa.h"

#include <cmath>
#include <type_traits>

namespace pfa {
namespace {

constexpr int kBlocksPerSm = 2;
constexpr float kLag = 4.f, kUp = 11.f;        // powers of two: of a score above the base; of weights

struct Scores;
Divisor chunks_of(const Scores& p, int threads);

// What the accumulated weights need.
struct Scores : ListParams {
  float* scores;       // null, or [head][keys of whole units][row_pad]
  float* weights;      // [head][cap]
  int64_t score_head;  // floats of a head
  int row_pad, lanes;  // a multiple of 4; lanes to a key
  Divisor chunks;      // of a head's keys, blocks
  bool fused;          // weights are added beside the join
};

constexpr int kWeightThreads = 256, kMaxRows = PFA_DECODE_MAX_ROWS;
constexpr int kWeightKeys = 4, kWeightRounds = 2;   // keys of a thread in flight, rounds of them

// Largest score, 1 / sum and position of four rows each; rows behind the last see nothing.
struct RowSums {
  float4 m, inv;
  int4 pos;
};

// LANES lanes (0: p.lanes) take a key's rows four at a time and add up their weights: this block's keys of
// a head, chunk `chunk`, between rows lo and end.
template <int LANES>
__device__ __forceinline__ void add_weights(const Scores& p, int64_t bh, int chunk, int lo, int end,
                                            const RowSums* rows) {
  const int lanes = LANES > 0 ? LANES : p.lanes, sub = threadIdx.x & (lanes - 1), quads = p.row_pad / 4;
  const int step = blockDim.x / lanes, block = step * kWeightKeys * kWeightRounds;   // keys
  const float* const scores = p.scores + bh * p.score_head;
  float* const weights = p.weights + bh * p.cap;
#pragma unroll 1
  for (int64_t at = lo + (int64_t)chunk * block; at < end; at += (int64_t)p.chunks.by * block)
#pragma unroll 1
    for (int round = 0; round < kWeightRounds; ++round) {
      const int64_t j0 = at + round * (step * kWeightKeys) + threadIdx.x / lanes;
      float sum[kWeightKeys], was[kWeightKeys];
#pragma unroll
      for (int i = 0; i < kWeightKeys; ++i) {
        sum[i] = was[i] = 0.f;
        if (sub == 0 && j0 + i * step < end) was[i] = weights[j0 + i * step];
      }
#pragma unroll 1
      for (int q = sub; q < quads; q += lanes) {
        float4 v[kWeightKeys];
#pragma unroll
        for (int i = 0; i < kWeightKeys; ++i)
          if (j0 + i * step < end)
            v[i] = *reinterpret_cast<const float4*>(scores + (j0 + i * step) * p.row_pad + 4 * q);
        const RowSums r = rows[q];
#pragma unroll
        for (int i = 0; i < kWeightKeys; ++i) {
          const int64_t j = j0 + i * step;
          // (what a row does not see may not have been written)
          auto add = [&](float s, float m, float inv, int pos) {
            if (j <= pos && (p.window <= 0 || j > pos - p.window)) sum[i] += exp2_fast(s - m) * inv;
          };
          add(v[i].x, r.m.x, r.inv.x, r.pos.x);
          add(v[i].y, r.m.y, r.inv.y, r.pos.y);
          add(v[i].z, r.m.z, r.inv.z, r.pos.z);
          add(v[i].w, r.m.w, r.inv.w, r.pos.w);
        }
      }
#pragma unroll
      for (int i = 0; i < kWeightKeys; ++i) {
#pragma unroll
        for (int d = 1; d < lanes; d <<= 1) sum[i] += __shfl_xor_sync(0xffffffffu, sum[i], d);
        if (sub == 0 && j0 + i * step < end) weights[j0 + i * step] = was[i] + sum[i];
      }
    }
}

__device__ __forceinline__ void set_row(RowSums* rows, int r, float2 ml, int pos) {
  reinterpret_cast<float*>(&rows[r / 4].m)[r % 4] = ml.x;
  reinterpret_cast<float*>(&rows[r / 4].inv)[r % 4] = ml.y;
  reinterpret_cast<int*>(&rows[r / 4].pos)[r % 4] = pos;
}

// UNIT: keys of a unit, in products of 16.  A ring holds 128 keys a warp.
template <int UNIT>
struct Params : Scores {
  static constexpr int kUnit = UNIT, kHeadCost = 512 / UNIT;
  static constexpr bool kSums = true;
  const uint8_t *k4, *v4, *k_scale, *v_scale;

  int more_threads() const { return fused ? kWeightThreads : 0; }
  int64_t more_blocks(int threads) {
    if (!fused) return 0;
    chunks = chunks_of(*this, threads);
    return (int64_t)entries * Hkv * chunks.by;
  }
  // Weights beside the join, where a head's rows are one tile: their sums from the parts once more.
  template <int RM, int NW>
  __device__ __forceinline__ void more(int id, int blocks, int (*s_units)[2]) const {
    __shared__ RowSums s_rows[RM / 4];
    const int eh = id / chunks, chunk = id - eh * (int)chunks.by, e = eh / heads, h = eh - e * Hkv;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    asm volatile("griddepcontrol.launch_dependents;");
    const auto x = entry_of<RM, true>(*this, e);
    const Parts head = parts_of<RM, kWarps / NW>(*this, e, h, x, blocks, s_units);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int64_t bh = x.b * Hkv + h;
    if (head.n == 0 || x.lo + (int64_t)chunk * (blockDim.x / lanes * (kWeightKeys * kWeightRounds)) >= x.end) return;
    for (int r = warp; r < RM; r += warps) {
      float2 ml = make_float2(0.f, 0.f);
      if (r < x.nr && head.n == 1) {
        ml = sums[bh * rows + r];
      } else if (r < x.nr) {
        float m = -INFINITY, l = 0.f;
        for (int i = lane; i < head.n; i += 32) {
          const float2 v = *reinterpret_cast<const float2*>(part_at<RM, NW * 128>(*this, head, i) + RM * NW * 128 + 2 * r);
          const float to = fmaxf(m, v.x), base = to == -INFINITY ? 0.f : to;
          l = l * exp2_fast(m - base) + v.y * exp2_fast(v.x - base);
          m = to;
        }
        float most = m;
        for (int o = 16; o > 0; o >>= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
        l *= exp2_fast(m - (most == -INFINITY ? 0.f : most));
        for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
        ml = row_sums(most, l);
      }
      if (lane == 0) set_row(s_rows, r, ml, r < x.nr ? x.end - (int)T + r / group : -1);
    }
    __syncthreads();
    add_weights<0>(*this, bh, chunk, x.lo, x.end, s_rows);
  }
};

// Key of row i of a product, in its eight.
__device__ __forceinline__ int key_at(int i) { return i & 1 ? 4 + ((i >> 1) ^ 1) : i >> 1; }

// Where column d (a multiple of 4) of a row of the join area is: lanes hold 16 columns of every
// other row.
__device__ __forceinline__ int join_at(int d, int row) { return d ^ (((row >> 1) & 3) << 2); }

__device__ __forceinline__ void copy8(uint32_t dst, const void* src, bool on) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;"
               :: "r"(dst), "l"(src), "r"(on ? 8 : 0) : "memory");
}
__device__ __forceinline__ uint2 lds8(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
  return v;
}
__device__ __forceinline__ uint32_t lds2(uint32_t a) {
  uint16_t v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(a));
  return v;
}
__device__ __forceinline__ uint32_t lds1(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(a));
  return v;
}
__device__ __forceinline__ uint32_t mul2(uint32_t a, uint32_t b) {
  const __half2 h = __hmul2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
  return *reinterpret_cast<const uint32_t*>(&h);
}
// K's fragments of the k16 steps 2 w, 2 w + 1: words w of the two keys' 32 channels, their two scales each.
__device__ __forceinline__ void k_fragments(int w, uint32_t wa, uint32_t wc, uint32_t sa, uint32_t sc,
                                            uint32_t (&a)[4], uint32_t (&b)[4]) {
  const uint32_t fa = __byte_perm(sa, sa, w < 2 ? 0x1010 : 0x3232);
  const uint32_t fc = __byte_perm(sc, sc, w < 2 ? 0x1010 : 0x3232);
  a[0] = mul2(e2m1x2_to_half<0>(wa), fa);
  a[1] = mul2(e2m1x2_to_half<0>(wc), fc);
  a[2] = mul2(e2m1x2_to_half<1>(wa), fa);
  a[3] = mul2(e2m1x2_to_half<1>(wc), fc);
  b[0] = mul2(e2m1x2_to_half<2>(wa), fa);
  b[1] = mul2(e2m1x2_to_half<2>(wc), fc);
  b[2] = mul2(e2m1x2_to_half<3>(wa), fa);
  b[3] = mul2(e2m1x2_to_half<3>(wc), fc);
}
// The power of two that brings a row with this largest element to 2^13 .. 2^14.
__device__ __forceinline__ int row_exponent(float amax) {
  if (amax == 0.f || !(amax <= 3.402823466e38f)) return 0;
  return min(13 + 127 - (int)(__float_as_uint(amax) >> 23), 120);
}
__device__ __forceinline__ uint32_t transposed(uint32_t a) {
  uint32_t b;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(b) : "r"(a));
  return b;
}

// Whether the warps of a block share the second operands of the scores (see decode_kernel).
template <typename E, int NW, int NT>
constexpr bool kWide = NT > 1 && NW == 1 && sizeof(E) == 2;

template <int UNIT, int NT, bool WIDE>
struct Shared {
  static constexpr int kProducts = WIDE ? NT : 0;
  static constexpr int kStages = 128 / UNIT;
  static constexpr int kHalf = UNIT * 64;        // bytes of a warp's K (or V) codes of a stage
  static constexpr int kScales = UNIT * 8;       // and of its scales
  static constexpr int kStageBytes = 2 * (kHalf + kScales);
  // Joins: 8 row sums of 128 floats for each warp.  Score exchange: twice those of a unit and 16 rows.
  static constexpr int kJoinBytes = kWarps * UNIT * 128;
  alignas(128) uint8_t ring[kWarps][kStages][kStageBytes];
  alignas(16) uint8_t join[kJoinBytes];
  float2 ml[kWarps][8 * NT];                     // a warp's {m, l} of each row
  uint2 query[kProducts * 8 + 1][32];            // [product][k16 step][lane]
  float factor[kProducts * 8 + 2];               // of a row's scores
  ListShared list;
  static_assert(kJoinBytes >= kWarps * 8 * 128 * 4, "join area");
};
static_assert(kBlocksPerSm * (sizeof(Shared<64, 2, true>) + 1024) <= 228 * 1024, "shared memory of an SM");

// NW: warps of a unit (head_dim / 128).  NT: products a tile, tiles of 8 NT rows.
template <typename E, int NW, int NT, int UNIT>
__global__ void __launch_bounds__(kThreads, kBlocksPerSm) decode_kernel(const Params<UNIT> p) {
  // A team is a warp or the block, so that every barrier is the block's: it does not count
  // warps that have ended, and no lengths, not even changing ones, leave a warp waiting.
  static_assert(NW == 1 || NW == kWarps, "barriers are the block's");
  constexpr int D = NW * 128, TEAMS = kWarps / NW, RM = 8 * NT;
  constexpr bool F32 = sizeof(E) == 4;
  constexpr int SETS = F32 ? 2 : 1;   // high and low halves
  // More rows than a product's eight: the scores' second operands are in shared memory, each warp having
  // made those of one product, and what can be made anew is not held.  That leaves registers for
  // the products of all keys of a unit at once, NT * UNIT / 16 chains of them that do not wait for one another.
  constexpr bool WIDE = kWide<E, NW, NT>;
  static_assert(!WIDE || NT <= kWarps, "a warp for each product");
  using Sh = Shared<UNIT, NT, WIDE>;
  constexpr int kUnit = UNIT, kTiles = UNIT / 16, kStages = Sh::kStages;
  constexpr int kHalf = Sh::kHalf, kScales = Sh::kScales, kStageBytes = Sh::kStageBytes;
  static_assert(NW == 1 || Sh::kJoinBytes >= 2 * NW * kTiles * NT * 32 * 16, "score exchange");
  extern __shared__ __align__(128) uint8_t smem_raw[];
  Sh& sm = *reinterpret_cast<Sh*>(smem_raw);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, qd = lane & 3;
  const int team = warp / NW, part = warp % NW;

  // What ran before has written its results; only then may the join start (it reads the lengths
  // before its own wait).
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  int at, stop, first_entry, into;
  if (!run_start<RM, TEAMS>(p, sm.list, at, stop, first_entry, into)) return;

  Cursor<Params<UNIT>, RM, TEAMS> in, cu;   // copies, products
  in.start(p, at, stop, first_entry, into, team);
  cu = in;

  // Query rows of a piece as they are stored, this warp's columns: the lane's 32
  // elements of its rows.  Rows past the tile repeat its last.
  // They are asked for under the prologue or the join before, but for two fp32 rows, which
  // would need 64 registers across the join.  (WIDE: those of the product that is this warp's.)
  constexpr int RV = F32 ? 8 : 4;   // 16-byte vectors of a row
  constexpr bool EARLY = !WIDE && NT * RV <= 8;
  uint4 raw[EARLY ? NT * RV : RV];
  auto load_row = [&](int i) {
    const int r = cu.x.r0 + min(g + 8 * i, cu.x.nr - 1);
    const int t = r / p.group;   // its token
    const E* row = (const E*)p.q + (cu.x.b * p.T + t) * p.q_row +
                   (int64_t)(cu.h * (int)p.group.by + r - t * (int)p.group.by) * D + part * 128 + qd * 32;
#pragma unroll
    for (int j = 0; j < RV; ++j)
      raw[(EARLY ? i * RV : 0) + j] = *reinterpret_cast<const uint4*>(row + j * (16 / (int)sizeof(E)));
  };
  auto load_early = [&]() {
    if (cu.done()) return;
    if constexpr (EARLY) {
#pragma unroll
      for (int i = 0; i < NT; ++i) load_row(i);
    } else if constexpr (WIDE) {
      if (warp < NT) load_row(warp);
    }
  };
  load_early();

  const uint32_t ring = smem_u32(sm.ring[warp]);
  // Copies of a unit: K's codes and scales, then V's, each a group of its own: K's place is free
  // for a later unit when the scores are done, V's when its sum is.  Copy c of codes
  // is row 8 c + lane / 4, piece lane % 4; of scales, row 32 c + lane.
  // What moves from unit to unit is one offset of codes and one of scales, the same for K and V.
  const uint32_t dst = ring + (lane >> 2) * 64 + (((lane & 3) ^ ((lane >> 2) & 2)) << 4);
  const uint32_t dst_scales = ring + kHalf + lane * 8;
  struct Source {
    int64_t codes, scales;   // of this lane
    int lo, hi;              // rows [lo, hi] of the unit are copied
  } src = {};
  auto copy_half = [&](int stage_at, const uint8_t* codes, const uint8_t* scales) {
    const uint8_t* from = codes + src.codes;
    if (src.lo <= 0 && src.hi >= kUnit - 1) {   // all rows
#pragma unroll
      for (int c = 0; c < kUnit / 8; ++c) copy16(dst + stage_at + c * 512, from + c * 8 * (D / 2), true);
#pragma unroll
      for (int c = 0; c < kUnit / 32; ++c)
        copy8(dst_scales + stage_at + c * 256, scales + src.scales + c * 32 * (D / 16), true);
    } else {
#pragma unroll
      for (int c = 0; c < kUnit / 8; ++c) {
        const int row = 8 * c + (lane >> 2);
        const bool on = row >= src.lo && row <= src.hi;
        copy16(dst + stage_at + c * 512, on ? from + c * 8 * (D / 2) : codes, on);
      }
#pragma unroll
      for (int c = 0; c < kUnit / 32; ++c) {
        const int row = 32 * c + lane;
        const bool on = row >= src.lo && row <= src.hi;
        copy8(dst_scales + stage_at + c * 256, on ? scales + src.scales + c * 32 * (D / 16) : scales, on);
      }
    }
  };
  auto source = [&]() {   // of the first unit of a piece that is this team's
    const int64_t row = (in.x.b * p.Hkv + in.h) * p.cap + (int64_t)(in.x.u0 + in.k) * kUnit;
    src.codes = (row + (lane >> 2)) * (D / 2) + part * 64 + (lane & 3) * 16;
    src.scales = (row + lane) * (D / 16) + part * 8;
    src.lo = in.x.lo - (in.x.u0 + in.k) * kUnit;
    src.hi = in.x.hi - (in.x.u0 + in.k) * kUnit;
  };
  auto copy_k = [&](int stage) {
    if (!in.done() && in.k >= in.kend) {
#pragma unroll 1
      do in.next_piece(p, team);
      while (!in.done() && in.k >= in.kend);
      if (!in.done()) source();
    }
    if (!in.done()) copy_half(stage * kStageBytes, p.k4, p.k_scale);
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  // (after copy_k of the same unit: on to the team's next one)
  auto copy_v = [&](int stage) {
    if (!in.done()) {
      copy_half(stage * kStageBytes + kHalf + kScales, p.v4, p.v_scale);
      in.k += TEAMS;
      src.codes += TEAMS * kUnit * (D / 2);
      src.scales += TEAMS * kUnit * (D / 16);
      src.lo -= TEAMS * kUnit;
      src.hi -= TEAMS * kUnit;
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  // (a team may have nothing in its run's first piece)
  if (in.k < in.kend) source();
#pragma unroll 1
  for (int s = 0; s < kStages; ++s) {
    copy_k(s);
    copy_v(s);
  }

  // K: key g of a product; V: keys 2 qd and 2 qd + 1
  const uint32_t k_row = key_at(g), v_row0 = key_at(2 * qd), v_row1 = key_at(2 * qd + 1);
  const uint32_t k_at = k_row * 64 + ((qd ^ (k_row & 2)) << 4);
  const uint32_t v_at0 = v_row0 * 64 + (((g >> 1) ^ (v_row0 & 2)) << 4) + (g & 1) * 8;
  const uint32_t v_at1 = v_row1 * 64 + (((g >> 1) ^ (v_row1 & 2)) << 4) + (g & 1) * 8;
  int stage = 0, swap = 0;

  while (!cu.done()) {
    const auto x = cu.x;
    // ---- the piece's query rows, scaled by a power of two each (WIDE: one product's, for all warps)
    constexpr int QT = WIDE ? 1 : NT;
    uint32_t qf[QT][SETS][8][2];
    float srow[QT][2];     // rows 2 qd, 2 qd + 1 of each product
    int hi[QT][2], lo[QT][2];
    auto raw_at = [&](int i, int j) -> float {   // element j of the lane's 32 of row i
      const uint32_t* w = reinterpret_cast<const uint32_t*>(raw);
      if constexpr (F32) {
        return __uint_as_float(w[(EARLY ? i * 32 : 0) + j]);
      } else {
        const uint32_t v = w[i * 16 + j / 2];
        return __uint_as_float(j % 2 ? v & 0xffff0000u : v << 16);
      }
    };
    auto seen_to = [&](int r) { return x.end - (int)p.T + (x.r0 + min(r, x.nr - 1)) / p.group; };
    auto seen_from = [&](int to) { return p.window > 0 ? to - p.window + 1 : 0; };
#pragma unroll
    for (int i = 0; i < QT; ++i) {
      if constexpr (!EARLY && !WIDE) load_row(i);
      float amax = 0.f;
#pragma unroll
      for (int j = 0; j < 32; ++j) amax = fmaxf(amax, fabsf(raw_at(i, j)));
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
      if constexpr (NW > 1) {   // over the team's columns
        if (qd == 0) sm.ml[warp][g + 8 * i].x = amax;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < NW; ++w) amax = fmaxf(amax, sm.ml[team * NW + w][g + 8 * i].x);
      }
      const int ex = row_exponent(amax);
      const float up = pow2(ex), down = pow2(-ex) * p.scale_log2;
#pragma unroll
      for (int s = 0; s < 8; ++s)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const float w0 = raw_at(i, 4 * s + 2 * c) * up, w1 = raw_at(i, 4 * s + 2 * c + 1) * up;
          if constexpr (F32)
            split2(w0, w1, qf[i][0][s][c], qf[i][1][s][c]);
          else
            qf[i][0][s][c] = half2_of(w0, w1);
        }
      if constexpr (WIDE) {
        if (warp < NT) {
#pragma unroll
          for (int s = 0; s < 8; ++s) sm.query[warp * 8 + s][lane] = make_uint2(qf[0][0][s][0], qf[0][0][s][1]);
          if (qd == 0) sm.factor[warp * 8 + g] = down;
        }
        __syncthreads();   // (the join's last barrier is behind what used them before)
      } else {
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          srow[i][c] = __shfl_sync(0xffffffffu, down, (2 * qd + c) * 4);
          hi[i][c] = seen_to(8 * i + 2 * qd + c);
          lo[i][c] = seen_from(hi[i][c]);
        }
      }
    }
    // keys that every row of the tile sees need no mask
    const int all_hi = x.end - (int)p.T + x.r0 / p.group;
    const int all_lo = p.window > 0 ? x.hi - p.window + 1 : 0;
    float* const scores = p.scores ? p.scores + (x.b * p.Hkv + cu.h) * p.score_head : nullptr;

    // Channels 16 g + 2 t, + 1 of rows 2 qd, + 1: {channel, row} 00, 01, 10, 11 of product t.
    float o[NT][8][4];
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
      for (int t = 0; t < 8; ++t)
#pragma unroll
        for (int c = 0; c < 4; ++c) o[i][t][c] = 0.f;
    // Base, kUp - base (0 for none), this lane's part of the sum; what an exponent may be before
    // the bases are looked at.
    float m[NT][2], ups[QT][2], l[NT][2], limit = -INFINITY;
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
      for (int c = 0; c < 2; ++c) m[i][c] = -INFINITY, l[i][c] = 0.f;
#pragma unroll
    for (int i = 0; i < QT; ++i) ups[i][0] = ups[i][1] = 0.f;
    auto up = [&](int i, int c) {
      if constexpr (WIDE)
        return m[i][c] == -INFINITY ? 0.f : kUp - m[i][c];
      else
        return ups[i][c];
    };

#pragma unroll 1
    for (; cu.k < cu.kend; cu.k += TEAMS) {
      asm volatile("cp.async.wait_group %0;" :: "n"(2 * kStages - 1) : "memory");
      __syncwarp();
      const uint32_t kb = ring + stage * kStageBytes, vb = kb + kHalf + kScales;
      // ---- scores: [product of 16 keys][tile]{key g, row 2 qd, + 1; key g + 8, the same rows}
      float s[kTiles][NT][4];
      auto k_factors = [&](int h, uint32_t& sa, uint32_t& sc) {
        sa = e4m3x2_to_half(lds2(kb + kHalf + (h * 16 + k_row) * 8 + 2 * qd));
        sc = e4m3x2_to_half(lds2(kb + kHalf + (h * 16 + 8 + k_row) * 8 + 2 * qd));
      };
      if constexpr (WIDE) {
        uint4 ka[kTiles], kc[kTiles];
        uint32_t sa[kTiles], sc[kTiles];
#pragma unroll
        for (int h = 0; h < kTiles; ++h) {
          ka[h] = lds16(kb + h * 1024 + k_at);
          kc[h] = lds16(kb + h * 1024 + 512 + k_at);
          k_factors(h, sa[h], sc[h]);
#pragma unroll
          for (int i = 0; i < NT; ++i) s[h][i][0] = s[h][i][1] = s[h][i][2] = s[h][i][3] = 0.f;
        }
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          uint2 qw[NT][2];
#pragma unroll
          for (int i = 0; i < NT; ++i)
#pragma unroll
            for (int c = 0; c < 2; ++c) qw[i][c] = sm.query[i * 8 + 2 * w + c][lane];
#pragma unroll
          for (int h = 0; h < kTiles; ++h) {
            uint32_t a[2][4];
            k_fragments(w, reinterpret_cast<const uint32_t*>(&ka[h])[w], reinterpret_cast<const uint32_t*>(&kc[h])[w],
                        sa[h], sc[h], a[0], a[1]);
#pragma unroll
            for (int c = 0; c < 2; ++c)
#pragma unroll
              for (int i = 0; i < NT; ++i) mma(s[h][i], a[c], qw[i][c].x, qw[i][c].y);
          }
        }
      } else {
#pragma unroll
        for (int h = 0; h < kTiles; ++h) {
          float acc[NT][SETS][4];
#pragma unroll
          for (int i = 0; i < NT; ++i)
#pragma unroll
            for (int b = 0; b < SETS; ++b) acc[i][b][0] = acc[i][b][1] = acc[i][b][2] = acc[i][b][3] = 0.f;
          const uint4 ka = lds16(kb + h * 1024 + k_at), kc = lds16(kb + h * 1024 + 512 + k_at);
          uint32_t sa, sc;
          k_factors(h, sa, sc);
          const uint32_t wa[4] = {ka.x, ka.y, ka.z, ka.w}, wc[4] = {kc.x, kc.y, kc.z, kc.w};
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            uint32_t a[2][4];
            k_fragments(w, wa[w], wc[w], sa, sc, a[0], a[1]);
#pragma unroll
            for (int c = 0; c < 2; ++c)
#pragma unroll
              for (int i = 0; i < NT; ++i)
#pragma unroll
                for (int b = 0; b < SETS; ++b) mma(acc[i][b], a[c], qf[i][b][2 * w + c][0], qf[i][b][2 * w + c][1]);
          }
#pragma unroll
          for (int i = 0; i < NT; ++i)
#pragma unroll
            for (int c = 0; c < 4; ++c) s[h][i][c] = F32 ? acc[i][0][c] + acc[i][SETS - 1][c] : acc[i][0][c];
        }
      }
      __syncwarp();
      copy_k(stage);
      if constexpr (NW > 1) {
        // the team's partial scores, summed in the same order by each warp
        float4* ex = reinterpret_cast<float4*>(sm.join) + swap * (NW * kTiles * NT * 32);
#pragma unroll
        for (int h = 0; h < kTiles; ++h)
#pragma unroll
          for (int i = 0; i < NT; ++i)
            ex[(part * kTiles * NT + h * NT + i) * 32 + lane] =
                make_float4(s[h][i][0], s[h][i][1], s[h][i][2], s[h][i][3]);
        __syncthreads();
#pragma unroll
        for (int h = 0; h < kTiles; ++h)
#pragma unroll
          for (int i = 0; i < NT; ++i) {
            float4 t = ex[(h * NT + i) * 32 + lane];
#pragma unroll
            for (int w = 1; w < NW; ++w) {
              const float4 v = ex[(w * kTiles * NT + h * NT + i) * 32 + lane];
              t.x += v.x; t.y += v.y; t.z += v.z; t.w += v.w;
            }
            s[h][i][0] = t.x; s[h][i][1] = t.y; s[h][i][2] = t.z; s[h][i][3] = t.w;
          }
        swap ^= 1;
      }
      const int key0 = (x.u0 + cu.k) * kUnit;
      const bool masked = key0 < all_lo || key0 + kUnit - 1 > all_hi;
      // ---- scores become exponents over the base, up = kUp - base; hidden ones -infinity
#pragma unroll
      for (int i = 0; i < NT; ++i) {
        float2 f;
        if constexpr (WIDE)
          f = *reinterpret_cast<const float2*>(&sm.factor[8 * i + 2 * qd]);
        else
          f = make_float2(srow[i][0], srow[i][1]);
        const float u0 = up(i, 0), u1 = up(i, 1);
#pragma unroll
        for (int h = 0; h < kTiles; ++h)
#pragma unroll
          for (int c = 0; c < 4; ++c) s[h][i][c] = fmaf(s[h][i][c], c & 1 ? f.y : f.x, c & 1 ? u1 : u0);
      }
      if (masked) {
#pragma unroll
        for (int i = 0; i < NT; ++i) {
          int to[2], from[2];
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            if constexpr (WIDE)
              to[c] = seen_to(8 * i + 2 * qd + c), from[c] = seen_from(to[c]);
            else
              to[c] = hi[i][c], from[c] = lo[i][c];
          }
#pragma unroll
          for (int h = 0; h < kTiles; ++h)
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              const int key = key0 + h * 16 + (c >> 1) * 8 + (int)k_row;
              if (key < from[c & 1] || key > to[c & 1]) s[h][i][c] = -INFINITY;
            }
        }
      }
      if (scores && part == 0) {
#pragma unroll
        for (int i = 0; i < NT; ++i) {
          const int r = x.r0 + 8 * i + 2 * qd;
          if (r < p.rows) {
            float* to = scores + (int64_t)(key0 + (int)k_row) * p.row_pad + r;
#pragma unroll
            for (int h = 0; h < kTiles; ++h)
#pragma unroll
              for (int c = 0; c < 2; ++c)
                *reinterpret_cast<float2*>(to + (h * 16 + c * 8) * p.row_pad) =
                    make_float2(s[h][i][2 * c] - up(i, 0), s[h][i][2 * c + 1] - up(i, 1));
          }
        }
      }
      // ---- the base rises where a score is far above it
      auto largest = [&](int i, int c) {
        float mx = fmaxf(s[0][i][c], s[0][i][c + 2]);
#pragma unroll
        for (int h = 1; h < kTiles; ++h) mx = fmaxf(mx, fmaxf(s[h][i][c], s[h][i][c + 2]));
        return mx;
      };
      float most = -INFINITY;
#pragma unroll
      for (int i = 0; i < NT; ++i) most = fmaxf(most, fmaxf(largest(i, 0), largest(i, 1)));
      if (__any_sync(0xffffffffu, most > limit)) {
        limit = kUp + kLag;
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            float mx = largest(i, c);
#pragma unroll
            for (int d = 4; d < 32; d <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
            // (a row's own scores alone raise its base: its result does not depend on its tile's others)
            if (m[i][c] != -INFINITY && !(mx > kUp + kLag)) continue;
            mx = fmaxf(mx - up(i, c), m[i][c]);
            if (mx == -INFINITY) {   // nothing seen yet: the next unit asks again
              limit = -INFINITY;
              continue;
            }
            const float a = exp2_fast(m[i][c] - mx), by = kUp - mx - up(i, c);
            m[i][c] = mx;
            if constexpr (!WIDE) ups[i][c] = kUp - mx;
#pragma unroll
            for (int h = 0; h < kTiles; ++h) {
              s[h][i][c] += by;
              s[h][i][c + 2] += by;
            }
            l[i][c] *= a;
#pragma unroll
            for (int t = 0; t < 8; ++t) {
              o[i][t][c] *= a;
              o[i][t][c + 2] *= a;
            }
          }
      }
      // ---- weights and their sums; the weights as the second operand
      uint32_t pf[kTiles][NT][SETS][2];
#pragma unroll
      for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int h = 0; h < kTiles; ++h)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const float w0 = exp2_fast(s[h][i][2 * c]), w1 = exp2_fast(s[h][i][2 * c + 1]);
            l[i][0] += w0;
            l[i][1] += w1;
            if constexpr (F32) {
              uint32_t u, v;
              split2(w0, w1, u, v);
              pf[h][i][0][c] = transposed(u);
              pf[h][i][1][c] = transposed(v);
            } else {
              pf[h][i][0][c] = transposed(half2_of(w0, w1));
            }
          }
      // ---- weighted sum of V
      asm volatile("cp.async.wait_group %0;" :: "n"(2 * kStages - 1) : "memory");
      __syncwarp();
      // pairs of a channel of two keys, even channels and odd ones
      auto pairs = [&](uint32_t a, uint32_t b, uint32_t& even, uint32_t& odd) {
        even = (a & 0x0f0f0f0fu) | ((b << 4) & 0xf0f0f0f0u);
        odd = ((a >> 4) & 0x0f0f0f0fu) | (b & 0xf0f0f0f0u);
      };
      auto load_v = [&](int h, uint32_t (&w)[2][4], uint32_t (&f)[2]) {
        const uint32_t at = vb + h * 1024;
        const uint2 a = lds8(at + v_at0), b = lds8(at + v_at1);
        const uint2 c = lds8(at + 512 + v_at0), d = lds8(at + 512 + v_at1);
        pairs(a.x, b.x, w[0][0], w[0][1]);
        pairs(c.x, d.x, w[0][2], w[0][3]);
        pairs(a.y, b.y, w[1][0], w[1][1]);
        pairs(c.y, d.y, w[1][2], w[1][3]);
        const uint32_t sb = vb + kHalf + h * 128 + g;
        f[0] = e4m3x2_to_half(lds1(sb + v_row0 * 8) | lds1(sb + v_row1 * 8) << 8);
        f[1] = e4m3x2_to_half(lds1(sb + 64 + v_row0 * 8) | lds1(sb + 64 + v_row1 * 8) << 8);
      };
      auto fragment = [&](const uint32_t (&w)[4], const uint32_t (&f)[2], int i, uint32_t (&a)[4]) {
        switch (i) {
          case 0:
            a[0] = e2m1x2_to_half<0>(w[0]); a[1] = e2m1x2_to_half<0>(w[1]);
            a[2] = e2m1x2_to_half<0>(w[2]); a[3] = e2m1x2_to_half<0>(w[3]);
            break;
          case 1:
            a[0] = e2m1x2_to_half<1>(w[0]); a[1] = e2m1x2_to_half<1>(w[1]);
            a[2] = e2m1x2_to_half<1>(w[2]); a[3] = e2m1x2_to_half<1>(w[3]);
            break;
          case 2:
            a[0] = e2m1x2_to_half<2>(w[0]); a[1] = e2m1x2_to_half<2>(w[1]);
            a[2] = e2m1x2_to_half<2>(w[2]); a[3] = e2m1x2_to_half<2>(w[3]);
            break;
          default:
            a[0] = e2m1x2_to_half<3>(w[0]); a[1] = e2m1x2_to_half<3>(w[1]);
            a[2] = e2m1x2_to_half<3>(w[2]); a[3] = e2m1x2_to_half<3>(w[3]);
        }
        a[0] = mul2(a[0], f[0]); a[1] = mul2(a[1], f[0]);
        a[2] = mul2(a[2], f[1]); a[3] = mul2(a[3], f[1]);
      };
      if constexpr (F32) {
        // The tensor cores truncate as they accumulate: over thousands of keys that is a bias of
        // 1e-5 of the output.  So they add up 32 keys only, and rounding adds do the rest.
#pragma unroll
        for (int h = 0; h < kTiles; h += 2) {
          uint32_t w[2][2][4], f[2][2];
          load_v(h, w[0], f[0]);
          load_v(h + 1, w[1], f[1]);
#pragma unroll
          for (int t = 0; t < 8; ++t) {
            uint32_t a[2][4];
            fragment(w[0][t / 4], f[0], t % 4, a[0]);
            fragment(w[1][t / 4], f[1], t % 4, a[1]);
#pragma unroll
            for (int i = 0; i < NT; ++i) {
              float c[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
              for (int b = SETS - 1; b >= 0; --b) {
                mma(c, a[0], pf[h][i][b][0], pf[h][i][b][1]);
                mma(c, a[1], pf[h + 1][i][b][0], pf[h + 1][i][b][1]);
              }
#pragma unroll
              for (int k = 0; k < 4; ++k) o[i][t][k] += c[k];
            }
          }
        }
      } else {
#pragma unroll
        for (int h = 0; h < kTiles; ++h) {
          uint32_t w[2][4], f[2];
          load_v(h, w, f);
#pragma unroll
          for (int t = 0; t < 8; ++t) {
            uint32_t a[4];
            fragment(w[t / 4], f, t % 4, a);
#pragma unroll
            for (int i = 0; i < NT; ++i) mma(o[i][t], a, pf[h][i][0][0], pf[h][i][0][1]);
          }
        }
      }
      __syncwarp();
      copy_v(stage);
      stage = stage == kStages - 1 ? 0 : stage + 1;
    }

    // ---- join the block's teams, rows in rounds of eight
    const bool whole = cu.k0 == 0 && cu.kend == x.n;
    float* slot = p.parts + (int64_t)(2 * blockIdx.x + (cu.at == at ? 0 : 1)) * slot_floats<RM, D>();
    const int h = cu.h;
    cu.next_piece(p, team);
    load_early();   // arrives while the join runs
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) l[i][c] += __shfl_xor_sync(0xffffffffu, l[i][c], d);
        if (g == 0) sm.ml[warp][8 * i + 2 * qd + c] = make_float2(m[i][c], l[i][c]);
      }
    float* join = reinterpret_cast<float*>(sm.join);
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      if (8 * i >= x.nr) break;
      __syncthreads();   // ml is complete; what used the join area before is done
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int rr = 2 * qd + c, r = rr + 8 * i;
        if (r < x.nr) {
          float mx = -INFINITY;
          for (int w = 0; w < TEAMS; ++w) mx = fmaxf(mx, sm.ml[w * NW][r].x);
          const float f = exp2_fast(m[i][c] - (mx == -INFINITY ? 0.f : mx) - kUp);
          float* to = join + (team * 8 + rr) * D;
#pragma unroll
          for (int t = 0; t < 8; t += 2)
            *reinterpret_cast<float4*>(to + join_at(part * 128 + g * 16 + 2 * t, rr)) =
                make_float4(o[i][t][c] * f, o[i][t][c + 2] * f, o[i][t + 1][c] * f, o[i][t + 1][c + 2] * f);
        }
      }
      __syncthreads();
      const int rows = min(8, x.nr - 8 * i);
#pragma unroll 1
      for (int c = tid; c < rows * (D / 4); c += kThreads) {
        const int rr = c / (D / 4), d = c % (D / 4) * 4, r = rr + 8 * i;
        float4 sum = *reinterpret_cast<const float4*>(join + rr * D + join_at(d, rr));
        for (int w = 1; w < TEAMS; ++w) {
          const float4 v = *reinterpret_cast<const float4*>(join + (w * 8 + rr) * D + join_at(d, rr));
          sum.x += v.x; sum.y += v.y; sum.z += v.z; sum.w += v.w;
        }
        float mx = -INFINITY, ls = 0.f;
        for (int w = 0; w < TEAMS; ++w) mx = fmaxf(mx, sm.ml[w * NW][r].x);
        for (int w = 0; w < TEAMS; ++w)
          ls += sm.ml[w * NW][r].y * exp2_fast(sm.ml[w * NW][r].x - (mx == -INFINITY ? 0.f : mx) - kUp);
        if (whole) {
          const float n = ls == 0.f ? 0.f : p.unit / ls;
          const int q = x.r0 + r, t = q / p.group;
          E* to = (E*)p.out + (x.b * p.T + t) * p.out_row +
                  (int64_t)(h * (int)p.group.by + q - t * (int)p.group.by) * D + d;
          store_row4(to, make_float4(sum.x * n, sum.y * n, sum.z * n, sum.w * n));
          if (p.sums && d == 0) p.sums[(x.b * p.Hkv + h) * p.rows + q] = row_sums(mx, ls);
        } else {
          *reinterpret_cast<float4*>(slot + r * D + d) = sum;
          if (d == 0) *reinterpret_cast<float2*>(slot + RM * D + 2 * r) = make_float2(mx, ls);
        }
      }
    }
    __syncthreads();   // the join area and ml are free again
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
}

// Weights behind the join, from its row sums.
template <int LANES>
__global__ void __launch_bounds__(kWeightThreads) weights_kernel(const Scores p) {
  __shared__ RowSums s_rows[kMaxRows / 4];
  asm volatile("griddepcontrol.launch_dependents;");
  const int bh = blockIdx.x / p.chunks, chunk = blockIdx.x - bh * (int)p.chunks.by, b = bh / p.heads;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int64_t len = p.lengths[b];
  if (len < 0 || len > p.cap) return;
  const int end = (int)len, first = end - (int)p.T;
  const int lo = p.window > 0 ? max(0, max(first, 0) - p.window + 1) : 0;
  if (lo + (int64_t)chunk * (kWeightThreads / LANES * (kWeightKeys * kWeightRounds)) >= end) return;
  for (int r = threadIdx.x; r < p.row_pad; r += kWeightThreads)
    set_row(s_rows, r, r < p.rows ? p.sums[(int64_t)bh * p.rows + r] : make_float2(0.f, 0.f),
            r < p.rows ? first + r / p.group : -1);
  __syncthreads();
  add_weights<LANES>(p, bh, chunk, lo, end, s_rows);
}

// Blocks of `threads` for a head's keys.
Divisor chunks_of(const Scores& p, int threads) {
  const int64_t block = threads / p.lanes * kWeightKeys * kWeightRounds;
  const int64_t keys = p.window > 0 ? std::min<int64_t>(p.cap, p.window + p.T) : p.cap;
  return divisor((uint32_t)((keys + block - 1) / block));
}

int launch_weights(Scores p, int64_t heads, cudaStream_t stream) {
  p.chunks = chunks_of(p, kWeightThreads);
  if (heads * p.chunks.by > 0x7fffffff)   // (then each takes several)
    p.chunks = divisor((uint32_t)(0x7fffffff / heads));
  p.heads = divisor(p.Hkv);
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(heads * p.chunks.by));
  cfg.blockDim = dim3(kWeightThreads);
  cfg.stream = stream;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  auto* const kernel = p.lanes == 1 ? weights_kernel<1> : p.lanes == 2 ? weights_kernel<2>
                       : p.lanes == 4 ? weights_kernel<4> : weights_kernel<8>;
  if (cudaLaunchKernelEx(&cfg, kernel, p) == cudaSuccess) return kOk;
  cudaGetLastError();
  return kErrLaunch;
}

// Weights behind the join without stored scores: a warp converts 32 keys once and makes their scores with all
// rows again, 128 rows at a time, whose second operands the block's warps share; each lane has the sums of
// four keys over a quarter of the rows.  128 rows at 16384 keys: 16 us, where storing and reading 67 MB of
// scores took 25; 49 % of the tensor pipe, the rest the exponentials beside it and the start.  (Three blocks an SM
// 55.9 us for the whole call, two 54.0; four products at once 54.5.)
constexpr int kAgainRows = 128, kAgainBlocks = 2;

__global__ void __launch_bounds__(kThreads, kAgainBlocks) weights_again_kernel(const Params<64> p) {
  __shared__ uint2 s_query[kAgainRows / 8][8][32];   // [product][k16 step][lane]
  __shared__ float2 s_factor[kAgainRows / 2], s_minus[kAgainRows / 2], s_inv[kAgainRows / 2];   // two rows each
  __shared__ int2 s_pos[kAgainRows / 2];
  constexpr int D = 128;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, qd = lane & 3;
  asm volatile("griddepcontrol.launch_dependents;");
  const int bh = blockIdx.x / p.chunks, chunk = blockIdx.x - bh * (int)p.chunks.by;
  const int b = bh / p.heads, h = bh - b * p.Hkv;
  // (what the first kernel reads may be read before the wait, past this SM's own cache)
  const int64_t len = __ldcg((const long long*)p.lengths + b);
  const int end = len < 0 || len > p.cap ? 0 : (int)len, first = end - (int)p.T;
  const int lo = p.window > 0 ? max(0, max(first, 0) - p.window + 1) : 0;
  const int steps = (int)(((int64_t)end - lo + kThreads - 1) / kThreads);   // a key a thread
  if (chunk >= steps) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    return;
  }
  const uint8_t* const codes = p.k4 + (int64_t)bh * p.cap * (D / 2) + qd * 16;
  const uint8_t* const scales = p.k_scale + (int64_t)bh * p.cap * (D / 16) + qd * 2;
  float* const weights = p.weights + (int64_t)bh * p.cap;
  const int k_row = key_at(g);
  uint4 w[4];          // keys k_row, + 8, + 16, + 24: 32 channels each
  uint32_t scale[4];   // and their two scales
  auto load = [&](int step) {
    const int64_t key0 = lo + (int64_t)step * kThreads + warp * 32 + k_row;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const bool on = key0 + 8 * i < end;
      w[i] = on ? __ldcg(reinterpret_cast<const uint4*>(codes + (key0 + 8 * i) * (D / 2))) : make_uint4(0, 0, 0, 0);
      scale[i] = on ? __ldcg(reinterpret_cast<const unsigned short*>(scales + (key0 + 8 * i) * (D / 16))) : 0u;
    }
  };
#pragma unroll 1
  for (int r0 = 0; r0 < p.rows; r0 += kAgainRows) {
    const int nr = min(kAgainRows, p.rows - r0), products = (nr + 7) / 8;
    if (r0 > 0) __syncthreads();   // the rows before are done with
    load(chunk);
    uint4 x[kAgainRows / 8 / kWarps][4];   // this warp's rows, all asked for at once
#pragma unroll
    for (int n = 0; n < kAgainRows / 8 / kWarps; ++n) {
      const int i = warp + kWarps * n;
      if (i >= products) break;
      const int r = r0 + min(8 * i + g, nr - 1), t = r / p.group;
      const uint4* row = reinterpret_cast<const uint4*>(
          (const __nv_bfloat16*)p.q + (b * p.T + t) * p.q_row +
          (int64_t)(h * (int)p.group.by + r - t * (int)p.group.by) * D + qd * 32);
#pragma unroll
      for (int j = 0; j < 4; ++j) x[n][j] = __ldcg(row + j);
    }
#pragma unroll
    for (int n = 0; n < kAgainRows / 8 / kWarps; ++n) {
      const int i = warp + kWarps * n;
      if (i >= products) break;
      const uint32_t* const u = reinterpret_cast<const uint32_t*>(x[n]);
      float amax = 0.f;
#pragma unroll
      for (int j = 0; j < 16; ++j)
        amax = fmaxf(amax, fmaxf(fabsf(__uint_as_float(u[j] << 16)), fabsf(__uint_as_float(u[j] & 0xffff0000u))));
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
      const int ex = row_exponent(amax);
      const float up = pow2(ex);
#pragma unroll
      for (int s = 0; s < 8; ++s) {
        uint32_t f[2];
#pragma unroll
        for (int c = 0; c < 2; ++c)
          f[c] = half2_of(__uint_as_float(u[2 * s + c] << 16) * up, __uint_as_float(u[2 * s + c] & 0xffff0000u) * up);
        s_query[i][s][lane] = make_uint2(f[0], f[1]);
      }
      if (qd == 0) reinterpret_cast<float*>(s_factor)[8 * i + g] = pow2(-ex) * p.scale_log2;
    }
    if (r0 == 0) asm volatile("griddepcontrol.wait;" ::: "memory");
    for (int i = tid; i < 8 * products; i += kThreads) {
      const int r = r0 + min(i, nr - 1), pos = first + r / p.group;
      // (rows at negative positions may have no sums)
      const float2 ml = pos >= 0 ? p.sums[(int64_t)bh * p.rows + r] : make_float2(0.f, 0.f);
      reinterpret_cast<float*>(s_minus)[i] = -ml.x;
      reinterpret_cast<float*>(s_inv)[i] = i < nr ? ml.y : 0.f;
      reinterpret_cast<int*>(s_pos)[i] = pos;
    }
    __syncthreads();
    const int all_hi = first + r0 / p.group;   // keys that every row sees: up to here, and from
    const int all_lo = p.window > 0 ? first + (r0 + nr - 1) / p.group - p.window + 1 : 0;
#pragma unroll 1
    for (int step = chunk; step < steps; step += (int)p.chunks.by) {
      const int64_t key0 = lo + (int64_t)step * kThreads + warp * 32;
      uint32_t a[2][8][4];   // keys 16 h .. + 15
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint32_t sa = e4m3x2_to_half(scale[2 * i]), sc = e4m3x2_to_half(scale[2 * i + 1]);
        const uint32_t wa[4] = {w[2 * i].x, w[2 * i].y, w[2 * i].z, w[2 * i].w};
        const uint32_t wc[4] = {w[2 * i + 1].x, w[2 * i + 1].y, w[2 * i + 1].z, w[2 * i + 1].w};
#pragma unroll
        for (int j = 0; j < 4; ++j) k_fragments(j, wa[j], wc[j], sa, sc, a[i][2 * j], a[i][2 * j + 1]);
      }
      if (step + (int)p.chunks.by < steps) load(step + (int)p.chunks.by);
      if (key0 >= end) continue;
      const int64_t mine = key0 + k_row + 8 * qd;   // (four lanes have the same sums)
      const float was = mine < end ? weights[mine] : 0.f;
      float sum[4] = {0.f, 0.f, 0.f, 0.f};   // keys k_row, + 8, + 16, + 24
      // N products at once, N * 2 chains of eight
      auto add = [&](int i, auto count, auto masked) {
        constexpr int N = decltype(count)::value;
        float acc[N][2][4] = {};
#pragma unroll
        for (int s = 0; s < 8; ++s)
#pragma unroll
          for (int n = 0; n < N; ++n) {
            const uint2 q = s_query[i + n][s][lane];
            mma(acc[n][0], a[0][s], q.x, q.y);
            mma(acc[n][1], a[1][s], q.x, q.y);
          }
#pragma unroll
        for (int n = 0; n < N; ++n) {
          const int at = 4 * (i + n) + qd;
          const float2 f = s_factor[at], minus = s_minus[at], inv = s_inv[at];
          int2 pos;
          if constexpr (decltype(masked)::value) pos = s_pos[at];
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            if constexpr (decltype(masked)::value) {
              const int64_t key = key0 + k_row + 8 * (j / 2);
              const int to = j % 2 ? pos.y : pos.x;
              if (key > to || (p.window > 0 && key <= to - p.window)) continue;
            }
            sum[j / 2] = fmaf(exp2_fast(fmaf(acc[n][j / 4][j % 4], j % 2 ? f.y : f.x, j % 2 ? minus.y : minus.x)),
                              j % 2 ? inv.y : inv.x, sum[j / 2]);
          }
        }
      };
      int i = 0;
      if (key0 < all_lo || key0 + 31 > all_hi) {
#pragma unroll 1
        for (; i < products; ++i) add(i, std::integral_constant<int, 1>(), std::true_type());
      } else {
#pragma unroll 1
        for (; i + 2 <= products; i += 2) add(i, std::integral_constant<int, 2>(), std::false_type());
        if (i < products) add(i, std::integral_constant<int, 1>(), std::false_type());
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        sum[j] += __shfl_xor_sync(0xffffffffu, sum[j], 1);
        sum[j] += __shfl_xor_sync(0xffffffffu, sum[j], 2);
      }
      if (mine < end) weights[mine] = was + (qd & 2 ? (qd & 1 ? sum[3] : sum[2]) : qd & 1 ? sum[1] : sum[0]);
    }
  }
}

int launch_weights_again(Params<64> p, int64_t heads, int num_sms, cudaStream_t stream) {
  const int64_t keys = p.window > 0 ? std::min<int64_t>(p.cap, p.window + p.T) : p.cap;
  const int64_t slots = ((int64_t)num_sms * kAgainBlocks + heads - 1) / heads;   // of a head, at once
  p.chunks = divisor((uint32_t)std::min<int64_t>((keys + kThreads - 1) / kThreads, slots));
  p.heads = divisor(p.Hkv);
  if (heads * p.chunks.by > 0x7fffffff) return kErrShape;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(heads * p.chunks.by));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, weights_again_kernel, p) == cudaSuccess) return kOk;
  cudaGetLastError();
  return kErrLaunch;
}

template <typename E, int NW, int NT, int UNIT>
int launch(const Params<64>& all, const DecodeQ4Call& c) {
  using P = Params<UNIT>;
  P p;
  static_cast<Scores&>(p) = all;
  // Beside the join the weights save a launch, but each of their blocks finds its head's sums for
  // itself (us, beside / behind): 16 sequences of 1024 keys, 32/8 heads 13.8 / 15.4, one of 16384 12.9 / 14.0, of
  // 131072 42.8 / 41.2; 32 of up to 8192 42.2 / 38.9.
  p.fused = p.scores && p.rows <= 8 * NT &&
            c.span.B * p.Hkv * chunks_of(p, kWeightThreads).by <= (int64_t)2 * c.num_sms;
  p.k4 = all.k4; p.v4 = all.v4; p.k_scale = all.k_scale; p.v_scale = all.v_scale;
  static DeviceOnce once;
  const int rc = once.run(c.device, [] {
    return cudaFuncSetAttribute(decode_kernel<E, NW, NT, UNIT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                (int)sizeof(Shared<UNIT, NT, kWide<E, NW, NT>>)) == cudaSuccess ? kOk : kErrLaunch;
  });
  if (rc != kOk) return rc;
  const Kernels<P> k = {decode_kernel<E, NW, NT, UNIT>,
                        p.fused ? join_kernel<P, E, NW, 8 * NT, 8, true> : join_kernel<P, E, NW, 8 * NT, 8>,
                        p.fused ? join_kernel<P, E, NW, 8 * NT, 1, true> : join_kernel<P, E, NW, 8 * NT, 1>,
                        8 * NT, NW, kBlocksPerSm, sizeof(Shared<UNIT, NT, kWide<E, NW, NT>>)};
  const int r = launch_list(k, p, c.span.B, c.num_sms, c.stream);
  if (r != kOk || !c.weights || p.fused) return r;
  return p.scores ? launch_weights(p, c.span.B * p.Hkv, c.stream)
                  : launch_weights_again(all, c.span.B * p.Hkv, c.num_sms, c.stream);
}

// Whether accumulated weights come from scores that are made again, not stored: for many rows, as K's codes
// are converted once for all of them, and for few heads, whose blocks then have few keys each and wait little.
// bf16, head_dim 128 (us, again / stored): one sequence of 8 kv heads, 16384 keys, 16 / 24 / 32 / 128 rows
// 17.0 / 18.0, 20.6 / 23.4, 22.4 / 25.7, 54 / 63, 8 rows 14.6 / 14.0; 63488 keys, 32 / 256 rows 54 / 66, 325 / 384;
// 16 sequences of 2048 keys, 16 / 24 / 32 / 128 rows 29 / 27, 36 / 34, 41 / 42, 124 / 137.
bool scores_again(int64_t heads, int rows) { return rows > 24 || (rows > 8 && heads <= 16); }

// Partial sums, two slots a run.  (Slots for the most rows that a tile may have at this many rows or fewer.)
size_t parts_bytes(int rows, int D, int dtype, int num_sms) {
  const int rm = rows <= 8 ? 8 : D == 128 && dtype == PFA_BF16 ? 24 : 16;
  const size_t parts = 2 * (size_t)num_sms * kBlocksPerSm * (rm * D + rm * 2) * sizeof(float);
  return (parts + 255) & ~(size_t)255;
}

// Workspace: partial sums; with weights each row's sums and each score, where scores are stored.  `total` is the
// size that callers are told, `least` what a call makes do with: where scores can be made again, no call of fewer
// rows, sequences or keys needs more than a call that makes them again is told, so a workspace for the largest
// call holds every smaller one.
//
// Scores go by the capacity, whatever the sequences hold of it, so no more than kMaxScores bytes of them (or one
// sequence's) are kept: beyond that the sequences take turns, as many at a time as fit.  32 sequences of 32 fp32
// tokens, 32/8 heads, caches of 131072 rows (us, 4 GiB / all 17 GB): up to 8192 keys used 1120 / 1062, 65536 7285 / 7326;
// head_dim 512, bf16, 8192 used (4 GiB / 8.6 GB) 1285 / 1262.  (Making them again instead is no way out for few
// rows: 96 sequences of one token, 32/8 heads, up to 60000 keys, stored / again 971 / 1699.)
constexpr int64_t kMaxScores = (int64_t)1 << 32;
struct Layout {
  size_t sums, scores, total, least;
  int64_t score_head;
  int64_t at_once;     // sequences whose scores are kept at a time
  int row_pad;
};
Layout layout(int64_t B, int Hkv, int rows, int D, int dtype, int64_t cap, bool weights, int num_sms) {
  Layout w = {};
  const int64_t heads = B * Hkv;
  w.at_once = B;
  w.sums = parts_bytes(rows, D, dtype, num_sms);
  w.scores = w.total = w.least = w.sums;
  if (!weights) return w;
  const size_t sums = ((size_t)heads * rows * sizeof(float2) + 255) & ~(size_t)255;
  w.scores += sums;
  const bool again = D == 128 && dtype == PFA_BF16;
  w.total = w.least = parts_bytes(kMaxRows, D, dtype, num_sms) + sums;
  const int row_pad = (rows + 3) & ~3;
  const int64_t head = (cap + 63) / 64 * 64 * row_pad, sequence = Hkv * head * (int64_t)sizeof(float);
  const bool all = sequence <= kMaxScores / B;
  if (again && scores_again(heads, rows)) return w;
  w.row_pad = row_pad;
  w.score_head = head;
  if (!all) w.at_once = std::max<int64_t>(1, kMaxScores / sequence);
  // (the bound itself where sequences take turns: the size is not to fall as a sequence's grows)
  w.total = w.scores + (all ? B * sequence : std::max(sequence, kMaxScores));
  w.least = again ? std::min(w.total, w.least) : w.total;
  return w;
}

}  // namespace

DecodeQ4Sizes decode_q4_workspace(int64_t B, int64_t T, int H, int Hkv, int D, int dtype, int64_t cap,
                                  bool weights, int num_sms) {
  const Layout w = layout(B, Hkv, (int)std::min<int64_t>(T * (H / Hkv), 1 << 30), D, dtype, cap, weights, num_sms);
  return DecodeQ4Sizes{w.total, w.least};
}

int launch_decode_q4(const DecodeQ4Call& c) {
  Params<64> p;
  p.q = c.q; p.out = c.out;
  p.k4 = (const uint8_t*)c.cache.k4; p.v4 = (const uint8_t*)c.cache.v4;
  p.k_scale = (const uint8_t*)c.cache.k_scale; p.v_scale = (const uint8_t*)c.cache.v_scale;
  p.lengths = c.span.lengths;
  p.T = c.span.T; p.start_pos = c.span.start_pos;
  p.q_row = c.q_row; p.out_row = c.out_row;
  p.cap = (int)c.cache.max_seq_len;
  p.Hkv = c.Hkv; p.group = divisor(c.H / c.Hkv); p.window = c.window;
  if (p.T * (c.H / c.Hkv) > (1 << 30)) return kErrShape;
  p.rows = (int)p.T * (c.H / c.Hkv);
  p.scale_log2 = std::ldexp(c.scale * 1.4426950408889634f, c.cache.k_exp);
  p.unit = std::ldexp(1.f, c.cache.v_exp);
  p.err = c.err;
  const int64_t heads = c.span.B * c.Hkv;
  if (c.weights && heads > 0x7fffffff) return kErrShape;
  const Layout w = layout(c.span.B, c.Hkv, p.rows, c.D, c.dtype, p.cap, c.weights != nullptr, c.num_sms);
  const bool stored = w.score_head > 0 && c.ws_bytes >= w.total;
  if (stored && w.at_once < c.span.B) {   // (each call's first kernel waits for the one before it to end)
    const int64_t es = c.dtype == PFA_F32 ? 4 : 2, cache_rows = c.Hkv * c.cache.max_seq_len;
    for (int64_t b = 0; b < c.span.B; b += w.at_once) {
      DecodeQ4Call s = c;
      s.span.B = std::min(w.at_once, c.span.B - b);
      s.span.lengths += b;
      s.q = (const char*)c.q + b * c.span.T * c.q_row * es;
      s.out = (char*)c.out + b * c.span.T * c.out_row * es;
      s.weights += b * cache_rows;
      s.cache.k4 = (char*)c.cache.k4 + b * cache_rows * (c.D / 2);
      s.cache.v4 = (char*)c.cache.v4 + b * cache_rows * (c.D / 2);
      s.cache.k_scale = (char*)c.cache.k_scale + b * cache_rows * (c.D / 16);
      s.cache.v_scale = (char*)c.cache.v_scale + b * cache_rows * (c.D / 16);
      const int rc = launch_decode_q4(s);
      if (rc != kOk) return rc;
    }
    return kOk;
  }
  char* ws = static_cast<char*>(c.ws);
  p.parts = reinterpret_cast<float*>(ws);
  p.sums = c.weights ? reinterpret_cast<float2*>(ws + w.sums) : nullptr;
  p.scores = stored ? reinterpret_cast<float*>(ws + w.scores) : nullptr;
  p.score_head = w.score_head;
  p.row_pad = w.row_pad;
  p.weights = c.weights;
  // Lanes to a key: as many as it has four rows, or four or eight that take turns.
  const int quads = p.row_pad / 4;
  p.lanes = quads <= 1 ? 1 : quads <= 3 ? 2 : quads % 8 == 0 || quads >= 24 ? 8 : 4;
  // With tiles of 16 rows a converted code serves two products; with 8 there are twice as many units
  // to spread, and less code to fetch.  16 rows, bf16 (us, tiles of 8 / of 16):
  //   one sequence, 32/8 heads of 128, 1024 / 4096 / 16384 / 32768 keys   7.4 / 8.4   8.5 / 9.7   13.2 / 12.3   18.0 / 16.7
  //   16 sequences of 512 / 2048 keys                                     11.4 / 12.2   20.0 / 18.2
  //   8/2 heads of 512, 16 sequences of 2048, 4 of 32768 keys             26.3 / 31.6   65.9 / 53.7
  // fp32: 9.5 / 11.9 at 4096 keys, 23.2 / 23.8 at 32768, 8 sequences of 8192 keys 43.8 / 38.9.
  // 17 to 24 rows are one tile of 24 in place of two of 16 (24 rows, of 16 / of 24): one sequence, 32/8 heads,
  // 16384 / 63488 keys 16.4 / 15.1, 37.7 / 30.4, 16 of 2048 26.0 / 22.8; 8/1 heads, 131072 keys 19.3 / 20.0.  Two
  // or more such tiles are no faster than their rows in tiles of 16 (48 rows, 63488 keys 52.1 / 52.0), and
  // one of 32 spills (47 for 32 rows, 38 with two of 16).
  const int64_t rows = c.span.lengths ? p.cap : c.span.start_pos + p.T;   // most that a sequence can have
  const int64_t keys = p.window > 0 ? std::min<int64_t>(rows, p.window + p.T) : rows;
  const int64_t units = heads * ((p.rows + 7) / 8) * (keys / 64 + 1);
  const bool few = p.rows <= 8 || units < (int64_t)12 * c.num_sms * kBlocksPerSm;
  // Units of 64 keys need fewer instructions a key, units of 32 spread further and their code is fetched
  // sooner.  8 rows or less (us, 32 / 64 keys): one sequence, 32/8 heads of 128, 128 / 4096 / 16384 keys 4.8 / 5.4,
  // 7.2 / 7.8, 10.1 / 9.8, 32 sequences of 8192 59.7 / 54.4; 8/2 heads of 512, fp32, one sequence of 4096 keys
  // 9.7 / 10.8.  (16 fp32 rows and units of 64 keys need more registers than there are.)
  const bool small = units < (int64_t)2 * c.num_sms * kBlocksPerSm;
  if (c.dtype == PFA_BF16) {
    if (c.D == 128)
      return !few ? (p.rows > 16 && p.rows <= 24 ? launch<__nv_bfloat16, 1, 3, 32>(p, c)
                                                 : launch<__nv_bfloat16, 1, 2, 64>(p, c))
             : small ? launch<__nv_bfloat16, 1, 1, 32>(p, c) : launch<__nv_bfloat16, 1, 1, 64>(p, c);
    return !few ? launch<__nv_bfloat16, 4, 2, 64>(p, c)
           : small ? launch<__nv_bfloat16, 4, 1, 32>(p, c) : launch<__nv_bfloat16, 4, 1, 64>(p, c);
  }
  if (c.D == 128)
    return !few ? launch<float, 1, 2, 32>(p, c)
           : small ? launch<float, 1, 1, 32>(p, c) : launch<float, 1, 1, 64>(p, c);
  return !few ? launch<float, 4, 2, 32>(p, c)
         : small ? launch<float, 4, 1, 32>(p, c) : launch<float, 4, 1, 64>(p, c);
}

}  // namespace pfa
