// pfa_decode_q8.cu -- attention of few tokens of a batch of sequences over
// their 8-bit caches, on the tensor cores.
//
// For each sequence and kv head the T * group query rows form tiles of 16 rows
// (fp32: 16 or 8), and for each tile
//   s_j = scale * ks_j * <q, k8_j>,  out = sum_j 2^(s_j log2 e - m) vs_j v8_j / sum_j 2^(s_j log2 e - m)
// with the running maximum m, the sum and the output in fp32.  A cache byte is
// read once for all rows of a tile, so with up to 16 rows HBM's bytes bound it.
//
// Products: mma.sync m16n8k16 on halves.  e4m3 is exact in half; q is scaled
// to 2^13..2^14 by a power of two for each row, which makes bf16 q exact but for
// elements 2^27 below the row's largest; the weights, times their block's scale
// over the largest seen so far and 2^14, are rounded to half (2^-11, finer
// than the bf16 output).  For fp32, q and the weights are a high and a low half:
// rows 8-15 of a product hold the low halves of rows 0-7, so the same instructions
// give 21 bits.  tcgen05 would need 128 rows or K and V staged as its operands;
// the tensor work of these shapes is a third of the time of the bytes.
//
// Fragments straight from the rows: the contraction's order is free as long as
// both operands agree, so a lane reads 16-byte pieces of a K row and takes each
// word of four elements as its part of one k16 step; likewise output columns, so
// a lane reads 16 bytes of four V rows and pairs the rows' bytes with prmt.
//
// Work split: tiles of 32 keys ("units") of all row tiles, sequences and heads
// form one list, cut into equal runs, one for each block (two blocks an SM).
// Four warps take the run's units in turn, each with its own ring of three
// stages filled by cp.async (no barrier in the loop); their sums join in shared
// memory where a run leaves a head, while the SM's other block streams on.  What
// covers a head alone is stored as output, what covers part of it goes to the
// workspace, and a second kernel, launched so that its start overlaps, joins the
// parts in order.
//
// head_dim 512: four warps share a unit, each with 128 columns of K and V; the
// scores' four partial sums are exchanged through shared memory.  Covering the exchange
// with the next unit's scores gained nothing (16 sequences of 16384 keys, 8/2 heads: 101.9
// us against 101.7), and moving it in 16-byte pieces lost (99.4 against 93.1).
//
// Measured on GB300, both kernels, one pass among others:
//   1 sequence of 131072 keys, 32/8 heads of 128, bf16 (269 MB)   49.0 us, 5.5 TB/s (floor
//     39.5 us): 2 us to the first copies, 37 us of streaming at 7.2 TB/s, up to 4 us
//     more on the SMs whose part of the chip gets less of the bandwidth, 5 us for the join
//   32 sequences up to 8192 keys, 32/8 heads of 128 (243 MB)      45.4 us (floor 35.7 us)
//   4 sequences, 3 tokens, window 1024, 8/2 heads of 512, fp32    10.6 us: two launches and
//     a chain of some ten latencies (floor of the 7 MB: 1.1 us)
// Steps that carried it: one 8-warp block an SM 59.0 / 70.0 / 27.7 us (the three cases);
// two 4-warp blocks, so that one streams while the other starts or ends a head, and
// K's place refilled before V's is free, 53.4 / 62.2 / 21.9; the next head's query rows
// loaded under the join, a head's fixed cost counted in the split, launches
// overlapped, 51.4 / 49.9 / 12.5; 32-bit lists and divisions by products (code 94 ->
// 66 KB), 51.3 / 47.6 / 11.6; the join's warps by the parts to expect and its conflict-free
// area, 49.7 / 45.8 / 10.9.
// A long fp32 chunk is bound by instructions: 2048 tokens at 14336, 32/8 heads of 128, 3.5 ms
// (147 TFLOP/s; plain fp32 products run at 26).
#include "pfa_internal.h"
#include "pfa_ptx.cuh"
#include "pfa_q8.cuh"

#include "../../include/pfa.h"

#include <algorithm>
#include <cmath>

namespace pfa {
namespace {

constexpr int kWarps = 4, kThreads = kWarps * 32;
constexpr int kBlocksPerSm = 2;
constexpr int kUnit = 32;                      // keys of a unit
constexpr int kStages = 3;
constexpr int kHalf = kUnit * 128;             // bytes of a warp's K (or V) part of a stage
constexpr int kStageBytes = 2 * kHalf;
constexpr int kMaxEntries = 1 << 14;           // (sequence, row tile) pairs of one launch
constexpr int64_t kMaxUnits = 1 << 30;         // units that a launch can list
constexpr int kJoinBytes = kWarps * 8 * 128 * 4;  // joins: 8 row sums of 128 floats for each warp
// What the start and end of a head cost a block, in units: its query rows, the join.
constexpr int kHeadCost = 8;
constexpr float kWeightScale = 16384.f;

struct Params {
  const void* q;
  void* out;
  const uint8_t *k8, *v8;
  const float *k_scale, *v_scale;
  const int64_t* lengths;
  int64_t T, start_pos, q_row, out_row;
  int64_t b0;                 // first sequence and row tile of this launch
  int tile0;
  int cap, Hkv, window, block_shift;
  int rows, entries;          // T * group; entries of this launch
  Divisor group, seqs;        // H / Hkv; sequences in this launch
  Divisor heads, joined;      // Hkv, and the second kernel's blocks for a tile's rows
  float scale_log2;
  unsigned* err;
  float* parts;               // workspace: slots of partial sums
};

// A tile of rows of one sequence and the keys that they see.
struct Entry {
  int64_t b;
  int end, r0, nr;    // sequence length; first row of the tile, rows
  int lo, hi;         // keys [lo, hi] are seen by some row
  int u0, n;          // units u0 .. u0 + n - 1 hold them
  bool bad;
  // Units of a head in the list of all: its own and its start's cost.
  __device__ int listed() const { return n > 0 ? n + kHeadCost : 0; }
};

// L2: the length is read from there, past this SM's own cache.
template <int RM, bool L2 = false>
__device__ __forceinline__ Entry entry_of(const Params& p, int e) {
  Entry x;
  const int tile = e / p.seqs;
  x.b = p.b0 + e - tile * (int)p.seqs.by;
  x.r0 = (p.tile0 + tile) * RM;
  x.nr = min(RM, p.rows - x.r0);
  const int64_t end = !p.lengths ? p.start_pos + p.T
                      : L2       ? __ldcg((const long long*)p.lengths + x.b)
                                 : p.lengths[x.b];
  x.bad = end < 0 || end > p.cap;
  x.end = x.bad ? 0 : (int)end;
  const int first = x.end - (int)p.T;
  x.hi = first + (x.r0 + x.nr - 1) / p.group;
  x.lo = p.window > 0 ? max(0, first + x.r0 / p.group - p.window + 1) : 0;
  x.u0 = x.lo / kUnit;
  x.n = x.bad || x.hi < 0 ? 0 : x.hi / kUnit - x.u0 + 1;
  return x;
}

// Units of a run: those of all heads over the blocks, at least one for each of
// a block's teams.  Block c has the list's units [c * run, (c + 1) * run).
template <int TEAMS>
__device__ __forceinline__ int run_of(int total, int blocks) {
  return max((int)((uint32_t)(total + blocks - 1) / (uint32_t)blocks), TEAMS);
}

// Floats of a partial-sum slot: rows of output, then {m, l} of each row.
template <int RM, int D>
__host__ __device__ constexpr int slot_floats() { return RM * D + RM * 2; }

// Pieces of 16 bytes of a row are permuted by its place in a group of eight, so
// that K fragments (two rows, four pieces) and V fragments (every other row, two
// pieces) of eight lanes fall in distinct banks.
__device__ __forceinline__ int swizzle(int r) {
  return (((r ^ (r >> 1)) & 1) << 2) | ((r >> 1) & 2) | ((r >> 1) & 1);
}

// Where column d (a multiple of 4) of a row of the join area is: lanes hold runs of 16
// columns, 32 apart, and would all write to the same banks.
__device__ __forceinline__ int join_at(int d, int row) {
  return d ^ ((((d >> 5) & 3) | ((row & 1) << 2)) << 2);
}

__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool on) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;"
               :: "r"(dst), "l"(src), "r"(on ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copy4(uint32_t dst, const void* src, bool on) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;"
               :: "r"(dst), "l"(src), "r"(on ? 4 : 0) : "memory");
}
__device__ __forceinline__ uint4 lds16(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
  return v;
}
__device__ __forceinline__ void mma(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t half2_of(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
// a, b -> high halves and what they leave out.
__device__ __forceinline__ void split2(float a, float b, uint32_t& hi, uint32_t& lo) {
  const __half2 h = __floats2half2_rn(a, b);
  const float2 f = __half22float2(h);
  hi = *reinterpret_cast<const uint32_t*>(&h);
  lo = half2_of(a - f.x, b - f.y);
}
__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Walks the units of a run that belong to one team, piece by piece: the part of
// a head that lies in the run.  A head's list starts with kHeadCost units of no work.
template <int RM, int TEAMS>
struct Cursor {
  int at, stop;        // the run from the current piece on: [at, stop)
  int e, h;            // entry and kv head of the piece
  Entry x;
  int listed;          // listed units of the piece
  int k0, kend;        // the head's units k0 .. kend - 1 are in the piece
  int k;               // the team's current one
  __device__ __forceinline__ void start(const Params& p, int at_, int stop_, int e_, int into,
                                        int team) {
    at = at_;
    stop = stop_;
    e = e_;
    x = entry_of<RM>(p, e);
    // (the clamps matter only if the lengths change under the kernel)
    h = min((int)((uint32_t)into / (uint32_t)max(x.listed(), 1)), p.Hkv - 1);
    piece(min(into - h * x.listed(), x.listed()), team);
    if (kend <= k0) next_piece(p, team);
  }
  __device__ __forceinline__ void piece(int first, int team) {
    listed = min(stop - at, x.listed() - first);
    k0 = max(first - kHeadCost, 0);
    kend = first + listed - kHeadCost;
    k = k0 + team;
  }
  __device__ __forceinline__ bool done() const { return at >= stop; }
  __device__ __forceinline__ void next_piece(const Params& p, int team) {
#pragma unroll 1
    do {
      at += listed;
      if (at >= stop) return;
      if (++h == p.Hkv) {
        h = 0;
#pragma unroll 1
        do {
          if (++e >= p.entries) {  // only if the lengths changed under the kernel
            at = stop;
            return;
          }
          x = entry_of<RM>(p, e);
        } while (x.n == 0);
      }
      piece(0, team);
    } while (kend <= k0);
  }
};

template <typename E>
__device__ __forceinline__ void store_row4(E* o, float4 v) {
  if constexpr (sizeof(E) == 4) {
    *reinterpret_cast<float4*>(o) = v;
  } else {
    const __nv_bfloat162 a = __floats2bfloat162_rn(v.x, v.y), b = __floats2bfloat162_rn(v.z, v.w);
    *reinterpret_cast<uint2*>(o) = make_uint2(*reinterpret_cast<const uint32_t*>(&a),
                                              *reinterpret_cast<const uint32_t*>(&b));
  }
}

struct Shared {
  alignas(128) uint8_t ring[kWarps][kStages][kStageBytes];
  alignas(16) uint8_t join[kJoinBytes];   // also: score exchange
  float scales[kWarps][kStages][4];       // K and V scales of a unit's two halves
  float2 ml[kWarps][16];                  // a warp's {m, l} of each row
  float vref[kWarps];
  int sums[kWarps];
  int first_entry, into;
};

static_assert(kBlocksPerSm * (sizeof(Shared) + 1024) <= 228 * 1024, "shared memory of an SM");

// NW: warps of a unit (head_dim / 128).  NR: rows of a lane (g, g + 8), tiles of 8 NR
// rows.  bf16 has NR 2, one set of fragments for both; fp32 a set for each.
template <typename E, int NW, int NR>
__global__ void __launch_bounds__(kThreads, kBlocksPerSm) decode_kernel(const Params p) {
  // A team is a warp or the block, so that every barrier is the block's: it does not count
  // warps that have ended, and no lengths, not even changing ones, leave a warp waiting.
  static_assert(NW == 1 || NW == kWarps, "barriers are the block's");
  constexpr int D = NW * 128, TEAMS = kWarps / NW, RM = 8 * NR;
  constexpr bool F32 = sizeof(E) == 4;
  constexpr int SETS = F32 ? NR : 1;
  extern __shared__ __align__(128) uint8_t smem_raw[];
  Shared& sm = *reinterpret_cast<Shared*>(smem_raw);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, qd = lane & 3;
  const int team = warp / NW, part = warp % NW;

  // What ran before has written its results; only then may the join start (it reads the lengths
  // before its own wait).
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  // ---- the list of units, and where this block's run starts in it
  int at, stop, first_entry, into;
  if (p.entries <= 32) {   // each warp for itself, an entry a lane
    const Entry x = entry_of<RM>(p, min(lane, p.entries - 1));
    const int mine = lane < p.entries ? x.listed() * p.Hkv : 0;
    if (x.bad && blockIdx.x == 0 && warp == 0) atomicOr(p.err, kErrLengths);
    int up = mine;
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, up, o);
      if (lane >= o) up += v;
    }
    const int total = __shfl_sync(0xffffffffu, up, 31);
    const int run = run_of<TEAMS>(total, gridDim.x);
    at = blockIdx.x * run;
    stop = min(total, at + run);
    if (at >= total) return;
    first_entry = __ffs(__ballot_sync(0xffffffffu, at < up)) - 1;
    into = at - __shfl_sync(0xffffffffu, up - mine, first_entry);
  } else {   // thread i has the entries [i * per, (i + 1) * per)
    const int per = (p.entries + kThreads - 1) / kThreads;
    int mine = 0;
#pragma unroll 1
    for (int e = tid * per; e < min(p.entries, (tid + 1) * per); ++e) {
      const Entry x = entry_of<RM>(p, e);
      mine += x.listed() * p.Hkv;
      if (x.bad && blockIdx.x == 0) atomicOr(p.err, kErrLengths);
    }
    int up = mine;
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, up, o);
      if (lane >= o) up += v;
    }
    if (lane == 31) sm.sums[warp] = up;
    __syncthreads();
    int before = up - mine, total = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) before += sm.sums[w];
      total += sm.sums[w];
    }
    const int run = run_of<TEAMS>(total, gridDim.x);
    at = blockIdx.x * run;
    stop = min(total, at + run);
    if (at >= total) return;
    if (before <= at && at < before + mine) {   // one thread
      int e = tid * per, rest = at - before;
#pragma unroll 1
      for (;; ++e) {
        const int n = entry_of<RM>(p, e).listed() * p.Hkv;
        if (rest < n || e + 1 >= min(p.entries, (tid + 1) * per)) break;
        rest -= n;
      }
      sm.first_entry = e;
      sm.into = rest;
    }
    __syncthreads();
    first_entry = sm.first_entry;
    into = sm.into;
  }

  Cursor<RM, TEAMS> in, cu;   // copies, products
  in.start(p, at, stop, first_entry, into, team);
  cu = in;

  // Query rows of a piece as they are stored, this warp's columns: the lane's 32
  // elements of its rows.  Rows past the tile repeat its last.
  // They are asked for under the prologue or the join before, but for two fp32 rows, which
  // would need 64 registers across the join.
  constexpr int RV = F32 ? 8 : 4;   // 16-byte vectors of a row
  constexpr bool EARLY = NR * RV <= 8;
  uint4 raw[EARLY ? NR * RV : RV];
  auto load_row = [&](int i) {
    const int r = cu.x.r0 + min(g + 8 * i, cu.x.nr - 1);
    const int t = r / p.group;   // its token
    const E* row = (const E*)p.q + (cu.x.b * p.T + t) * p.q_row +
                   (int64_t)(cu.h * (int)p.group.by + r - t * (int)p.group.by) * D + part * 128 + qd * 16;
#pragma unroll
    for (int j = 0; j < RV; ++j)
      raw[(EARLY ? i * RV : 0) + j] = *reinterpret_cast<const uint4*>(
          row + (j >= RV / 2 ? 64 : 0) + j % (RV / 2) * (16 / (int)sizeof(E)));
  };
  auto load_early = [&]() {
    if constexpr (EARLY) {
      if (cu.done()) return;
#pragma unroll
      for (int i = 0; i < NR; ++i) load_row(i);
    }
  };
  load_early();

  const uint32_t ring = smem_u32(sm.ring[warp]);
  const uint32_t scales = smem_u32(sm.scales[warp]);
  // copy c of 8: row 4 c + lane / 8, piece lane % 8
  const uint32_t dst0 = (lane >> 3) * 128 + (((lane & 7) ^ swizzle(lane >> 3)) << 4);
  const uint32_t dst1 = (4 + (lane >> 3)) * 128 + (((lane & 7) ^ swizzle(4 + (lane >> 3))) << 4);
  // Copies come in halves of a unit, K then V, each a group of its own: K's place is
  // free for the unit after next but one when its scores are done, V's when its sum is.
  struct Source {
    const uint8_t* v;      // the V row of key0 (or of the first key seen), this lane's piece
    int key0, lo, hi;      // on: hi >= lo
    bool inner;            // all keys of the unit are seen by some row
  } src = {};
  auto copy_rows = [&](uint32_t dst, const uint8_t* from) {
    if (src.inner) {
#pragma unroll
      for (int c = 0; c < 8; ++c)
        copy16(dst + (c >> 1) * 1024 + (c & 1 ? dst1 : dst0), from + c * 4 * D, true);
    } else {
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        const int key = src.key0 + 4 * c + (lane >> 3);
        const bool on = key >= src.lo && key <= src.hi;
        copy16(dst + (c >> 1) * 1024 + (c & 1 ? dst1 : dst0), on ? from + c * 4 * D : p.k8, on);
      }
    }
  };
  auto copy_k = [&](int stage) {
    while (!in.done() && in.k >= in.kend) in.next_piece(p, team);
    src.lo = 0;
    src.hi = -1;
    if (!in.done()) {
      const Entry& x = in.x;
      src.key0 = (x.u0 + in.k) * kUnit;
      src.lo = x.lo;
      src.hi = x.hi;
      src.inner = src.key0 >= x.lo && src.key0 + kUnit - 1 <= x.hi;
      const int64_t head = x.b * p.Hkv + in.h;
      const int64_t off = (head * p.cap + src.key0 + (lane >> 3)) * D + part * 128 + (lane & 7) * 16;
      src.v = p.v8 + off;
      copy_rows(ring + stage * kStageBytes, p.k8 + off);
      if (lane < 4) {
        const int key = src.key0 + (lane & 1) * 16;
        const bool on = key + 15 >= x.lo && key <= x.hi;
        const int64_t at = head * (p.cap >> p.block_shift) + ((on ? key : x.lo) >> p.block_shift);
        copy4(scales + (stage * 4 + lane) * 4, (lane < 2 ? p.k_scale : p.v_scale) + at, on);
      }
      in.k += TEAMS;
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  auto copy_v = [&](int stage) {
    if (src.hi >= src.lo) copy_rows(ring + stage * kStageBytes + kHalf, src.v);
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
#pragma unroll 1
  for (int s = 0; s < kStages; ++s) {
    copy_k(s);
    copy_v(s);
  }

  const uint32_t k_at = g * 128 + ((qd ^ swizzle(g)) << 4);             // first piece; second: ^ 64
  const uint32_t v_at0 = (2 * qd) * 128 + ((g ^ swizzle(2 * qd)) << 4);
  const uint32_t v_at1 = (2 * qd + 1) * 128 + ((g ^ swizzle(2 * qd + 1)) << 4);
  int stage = 0, swap = 0;

  while (!cu.done()) {
    const Entry x = cu.x;
    // ---- the piece's query rows, scaled by a power of two each
    uint32_t qf[SETS][8][4];
    float srow[2];
    int hi[2], lo[2];
    auto raw_at = [&](int i, int j) -> float {   // element j of the lane's 32 of row i
      if constexpr (F32) {
        const uint32_t* w = reinterpret_cast<const uint32_t*>(raw);
        return __uint_as_float(w[(EARLY ? i * 32 : 0) + j]);
      } else {
        const uint32_t w = reinterpret_cast<const uint32_t*>(raw)[i * 16 + j / 2];
        return __uint_as_float(j % 2 ? w & 0xffff0000u : w << 16);
      }
    };
#pragma unroll
    for (int i = 0; i < NR; ++i) {
      if constexpr (!EARLY) load_row(i);
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
      int ex = 13 + 127 - (int)(__float_as_uint(amax) >> 23);
      if (amax == 0.f || !(amax <= 3.402823466e38f)) ex = 0;
      ex = min(ex, 120);
      const float up = __uint_as_float((uint32_t)(127 + ex) << 23);
      srow[i] = __uint_as_float((uint32_t)(127 - ex) << 23) * p.scale_log2;
#pragma unroll
      for (int s = 0; s < 8; ++s) {
        const float w0 = raw_at(i, 4 * s) * up, w1 = raw_at(i, 4 * s + 1) * up;
        const float w2 = raw_at(i, 4 * s + 2) * up, w3 = raw_at(i, 4 * s + 3) * up;
        if constexpr (F32) {
          split2(w0, w1, qf[i][s][0], qf[i][s][1]);
          split2(w2, w3, qf[i][s][2], qf[i][s][3]);
        } else {
          qf[0][s][i] = half2_of(w0, w1);
          qf[0][s][2 + i] = half2_of(w2, w3);
        }
      }
      const int r = x.r0 + min(g + 8 * i, x.nr - 1);
      hi[i] = x.end - (int)p.T + r / p.group;
      lo[i] = p.window > 0 ? hi[i] - p.window + 1 : 0;
    }
    // keys that every row of the tile sees need no mask
    const int all_hi = x.end - (int)p.T + x.r0 / p.group;
    const int all_lo = p.window > 0 ? x.hi - p.window + 1 : 0;

    // A lane's output columns, two to a row (fp32: the two halves' sum).
    constexpr int OC = 2 * NR;
    float o[16][OC];
#pragma unroll
    for (int i = 0; i < 16; ++i)
#pragma unroll
      for (int c = 0; c < OC; ++c) o[i][c] = 0.f;
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f}, vref = 0x1p-100f;

#pragma unroll 1
    for (; cu.k < cu.kend; cu.k += TEAMS) {
      asm volatile("cp.async.wait_group %0;" :: "n"(2 * kStages - 1) : "memory");
      __syncwarp();
      const uint32_t kb = ring + stage * kStageBytes, vb = kb + kHalf;
      const float4 sc = *reinterpret_cast<const float4*>(sm.scales[warp][stage]);
      // ---- scores
      float s[4][2 * NR];
#pragma unroll
      for (int nt = 0; nt < 4; ++nt) {
        float acc[SETS][4];
#pragma unroll
        for (int i = 0; i < SETS; ++i) acc[i][0] = acc[i][1] = acc[i][2] = acc[i][3] = 0.f;
        const uint4 a = lds16(kb + nt * 1024 + k_at), b = lds16(kb + nt * 1024 + (k_at ^ 64));
        const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          uint32_t b0, b1;
          e4m3x4_to_half(w[k], b0, b1);
#pragma unroll
          for (int i = 0; i < SETS; ++i) mma(acc[i], qf[i][k], b0, b1);
        }
        if constexpr (F32) {   // high and low halves
#pragma unroll
          for (int i = 0; i < NR; ++i) {
            s[nt][2 * i] = acc[i][0] + acc[i][2];
            s[nt][2 * i + 1] = acc[i][1] + acc[i][3];
          }
        } else {
#pragma unroll
          for (int c = 0; c < 4; ++c) s[nt][c] = acc[0][c];
        }
      }
      __syncwarp();
      copy_k(stage);
      if constexpr (NW > 1) {
        // the team's partial scores, summed in the same order by each warp
        float2* ex = reinterpret_cast<float2*>(sm.join) + (team * 2 + swap) * NW * 256;
#pragma unroll
        for (int nt = 0; nt < 4; ++nt)
#pragma unroll
          for (int i = 0; i < NR; ++i)
            ex[part * 256 + (nt * 2 + i) * 32 + lane] = make_float2(s[nt][2 * i], s[nt][2 * i + 1]);
        __syncthreads();
#pragma unroll
        for (int nt = 0; nt < 4; ++nt)
#pragma unroll
          for (int i = 0; i < NR; ++i) {
            float2 t = ex[(nt * 2 + i) * 32 + lane];
#pragma unroll
            for (int w = 1; w < NW; ++w) {
              const float2 v = ex[w * 256 + (nt * 2 + i) * 32 + lane];
              t.x += v.x; t.y += v.y;
            }
            s[nt][2 * i] = t.x;
            s[nt][2 * i + 1] = t.y;
          }
        swap ^= 1;
      }
      const float ksc[2] = {sc.x, sc.y};
#pragma unroll
      for (int i = 0; i < NR; ++i) {
        const float f0 = srow[i] * ksc[0], f1 = srow[i] * ksc[1];
#pragma unroll
        for (int nt = 0; nt < 4; ++nt) {
          s[nt][2 * i] *= nt < 2 ? f0 : f1;
          s[nt][2 * i + 1] *= nt < 2 ? f0 : f1;
        }
      }
      const int key0 = (x.u0 + cu.k) * kUnit;
      if (key0 < all_lo || key0 + kUnit - 1 > all_hi) {
#pragma unroll
        for (int i = 0; i < NR; ++i)
#pragma unroll
          for (int nt = 0; nt < 4; ++nt)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              const int key = key0 + nt * 8 + 2 * qd + c;
              if (key < lo[i] || key > hi[i]) s[nt][2 * i + c] = -INFINITY;
            }
      }
      // ---- running maximum, weights, sums
      const float nv = fmaxf(vref, fmaxf(sc.z, sc.w));
      const float inv = kWeightScale / nv;
      const float vf0 = sc.z * inv, vf1 = sc.w * inv;
      const float shrink = vref / nv;
      vref = nv;
      float alpha[2];
#pragma unroll
      for (int i = 0; i < NR; ++i) {
        float mx = fmaxf(s[0][2 * i], s[0][2 * i + 1]);
#pragma unroll
        for (int nt = 1; nt < 4; ++nt) mx = fmaxf(mx, fmaxf(s[nt][2 * i], s[nt][2 * i + 1]));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
        mx = fmaxf(mx, m[i]);
        const float base = mx == -INFINITY ? 0.f : mx;
        const float a = exp2_fast(m[i] - base);
        m[i] = mx;
        float sum = 0.f;
#pragma unroll
        for (int nt = 0; nt < 4; ++nt)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const float e = exp2_fast(s[nt][2 * i + c] - base);
            sum += e;
            s[nt][2 * i + c] = e * (nt < 2 ? vf0 : vf1);
          }
        l[i] = l[i] * a + sum;
        alpha[i] = a * shrink;
      }
      if (__any_sync(0xffffffffu, alpha[0] != 1.f || alpha[NR - 1] != 1.f)) {
#pragma unroll
        for (int i = 0; i < 16; ++i)
#pragma unroll
          for (int c = 0; c < OC; ++c) o[i][c] *= alpha[c / 2];
      }
      // ---- weighted sum of V
      asm volatile("cp.async.wait_group %0;" :: "n"(2 * kStages - 1) : "memory");
      __syncwarp();
      // V rows of k16 step j: 16 j + 2 qd, + 1 and 16 j + 8 + 2 qd, + 1
      auto load_v = [&](int j, uint4 (&r)[4]) {
        r[0] = lds16(vb + j * 2048 + v_at0);
        r[1] = lds16(vb + j * 2048 + v_at1);
        r[2] = lds16(vb + j * 2048 + 1024 + v_at0);
        r[3] = lds16(vb + j * 2048 + 1024 + v_at1);
      };
      // word w of those rows -> fragments of output tiles 4 w .. 4 w + 3
      auto fragments = [&](const uint4 (&r)[4], int w, uint32_t (&b)[8]) {
        uint32_t v[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) v[k] = w == 0 ? r[k].x : w == 1 ? r[k].y : w == 2 ? r[k].z : r[k].w;
        e4m3x4_to_half(__byte_perm(v[0], v[1], 0x5140), b[0], b[1]);
        e4m3x4_to_half(__byte_perm(v[0], v[1], 0x7362), b[2], b[3]);
        e4m3x4_to_half(__byte_perm(v[2], v[3], 0x5140), b[4], b[5]);
        e4m3x4_to_half(__byte_perm(v[2], v[3], 0x7362), b[6], b[7]);
      };
      if constexpr (F32) {
        // The tensor cores truncate as they accumulate: over thousands of keys that is a bias of
        // 1e-5 of the output.  So they add up one unit only, and rounding adds do the rest.
        uint32_t a[NR][2][4];
        uint4 r[2][4];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
#pragma unroll
          for (int k = 0; k < NR; ++k) {
            split2(s[2 * j][2 * k], s[2 * j][2 * k + 1], a[k][j][0], a[k][j][1]);
            split2(s[2 * j + 1][2 * k], s[2 * j + 1][2 * k + 1], a[k][j][2], a[k][j][3]);
          }
          load_v(j, r[j]);
        }
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          uint32_t b[2][8];
          fragments(r[0], w, b[0]);
          fragments(r[1], w, b[1]);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
#pragma unroll
            for (int k = 0; k < NR; ++k) {
              float c[4] = {0.f, 0.f, 0.f, 0.f};
              mma(c, a[k][0], b[0][i], b[0][4 + i]);
              mma(c, a[k][1], b[1][i], b[1][4 + i]);
              o[4 * w + i][2 * k] += c[0] + c[2];
              o[4 * w + i][2 * k + 1] += c[1] + c[3];
            }
          }
        }
      } else {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          uint32_t a[4];
          a[0] = half2_of(s[2 * j][0], s[2 * j][1]);
          a[1] = half2_of(s[2 * j][2], s[2 * j][3]);
          a[2] = half2_of(s[2 * j + 1][0], s[2 * j + 1][1]);
          a[3] = half2_of(s[2 * j + 1][2], s[2 * j + 1][3]);
          uint4 r[4];
          load_v(j, r);
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            uint32_t b[8];
            fragments(r, w, b);
#pragma unroll
            for (int i = 0; i < 4; ++i) mma(o[4 * w + i], a, b[i], b[4 + i]);
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
    for (int i = 0; i < NR; ++i) {
      l[i] += __shfl_xor_sync(0xffffffffu, l[i], 1);
      l[i] += __shfl_xor_sync(0xffffffffu, l[i], 2);
      if (qd == 0) sm.ml[warp][g + 8 * i] = make_float2(m[i], l[i]);
    }
    float* join = reinterpret_cast<float*>(sm.join);
#pragma unroll
    for (int i = 0; i < NR; ++i) {
      if (8 * i >= x.nr) break;
      __syncthreads();   // ml is complete; what used the join area before is done
      const bool on = g + 8 * i < x.nr;
      if (on) {
        float mx = -INFINITY;
        for (int w = 0; w < TEAMS; ++w) mx = fmaxf(mx, sm.ml[w * NW][g + 8 * i].x);
        const float f = exp2_fast(m[i] - (mx == -INFINITY ? 0.f : mx)) * vref / kWeightScale;
        float* to = join + (team * 8 + g) * D;
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
          for (int d = 0; d < 16; d += 4) {
            float v[4];
#pragma unroll
            for (int j = 0; j < 4; ++j)
              v[j] = o[d + j][2 * i + c] * f;
            *reinterpret_cast<float4*>(to + join_at(part * 128 + qd * 32 + c * 16 + d, g)) =
                make_float4(v[0], v[1], v[2], v[3]);
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
          ls += sm.ml[w * NW][r].y * exp2_fast(sm.ml[w * NW][r].x - (mx == -INFINITY ? 0.f : mx));
        if (whole) {
          const float n = ls == 0.f ? 0.f : 1.f / ls;
          const int q = x.r0 + r, t = q / p.group;
          E* to = (E*)p.out + (x.b * p.T + t) * p.out_row +
                  (int64_t)(h * (int)p.group.by + q - t * (int)p.group.by) * D + d;
          store_row4(to, make_float4(sum.x * n, sum.y * n, sum.z * n, sum.w * n));
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

// A block has 128 columns of one row (GROUPS warps that take the parts in turn, in the
// blocks' order, each with a running maximum) or, with GROUPS 1, of all rows of a
// tile, a warp each.  It joins the parts of its head, and writes the zeros of rows
// that see nothing.
template <typename E, int NW, int NR, int GROUPS>
__global__ void __launch_bounds__(512) join_kernel(const Params p, int blocks) {
  constexpr int D = NW * 128, TEAMS = kWarps / NW, RM = 8 * NR;
  __shared__ float4 s_sum[GROUPS > 1 ? GROUPS - 1 : 1][32];
  __shared__ float2 s_ml[GROUPS];
  __shared__ int s_units[16][2];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, warps = blockDim.x >> 5;
  const int grp = warp % GROUPS;
  const int id = blockIdx.x / NW, d = blockIdx.x % NW * 128 + lane * 4;
  const int eh = id / p.joined, r = id - eh * (int)p.joined.by + warp / GROUPS;
  const int e = eh / p.heads, h = eh - e * p.Hkv;
  asm volatile("griddepcontrol.launch_dependents;");
  // The list of units, as the first kernel counts it, while that one runs.  Its blocks let this
  // grid start behind their own wait: whatever wrote the lengths has ended, and its writes are in
  // L2.  (The first kernel's own results are read behind the wait below.)
  int before = 0, total = 0;
#pragma unroll 1
  for (int i = tid; i < p.entries; i += blockDim.x) {
    const int n = entry_of<RM, true>(p, i).listed() * p.Hkv;
    total += n;
    if (i < e) before += n;
  }
  for (int o = 16; o > 0; o >>= 1) {
    before += __shfl_xor_sync(0xffffffffu, before, o);
    total += __shfl_xor_sync(0xffffffffu, total, o);
  }
  if (lane == 0) {
    s_units[warp][0] = before;
    s_units[warp][1] = total;
  }
  __syncthreads();
  before = total = 0;
  for (int w = 0; w < warps; ++w) {
    before += s_units[w][0];
    total += s_units[w][1];
  }
  const Entry x = entry_of<RM, true>(p, e);
  const int run = run_of<TEAMS>(total, blocks);
  const int s0 = before + h * x.listed();
  int c0 = 0, n = 0, first = 0;
  if (x.n > 0) {
    c0 = (int)((uint32_t)(s0 + kHeadCost) / (uint32_t)run);
    n = (int)((uint32_t)(s0 + x.listed() - 1) / (uint32_t)run) - c0 + 1;
    // the first block's part is its run's last piece unless its run starts in this head
    first = c0 * run >= s0 ? 0 : 1;
  }
  // Every block waits, also one with nothing to do: this grid must not end before the first.
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (r >= x.nr || x.bad || n == 1) return;   // n 1: stored whole
  const int q = x.r0 + r, t = q / p.group;
  E* to = (E*)p.out + (x.b * p.T + t) * p.out_row +
          (int64_t)(h * (int)p.group.by + q - t * (int)p.group.by) * D + d;
  if (n == 0) {
    if (grp == 0) store_row4(to, make_float4(0.f, 0.f, 0.f, 0.f));
    return;
  }
  float mx = -INFINITY, l = 0.f;
  float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
  for (int i0 = grp; i0 < n; i0 += 6 * GROUPS) {
    float4 v[6];
    float2 ml[6];
#pragma unroll
    for (int j = 0; j < 6; ++j) {
      const int i = i0 + GROUPS * j;
      ml[j] = make_float2(-INFINITY, 0.f);
      v[j] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (i < n) {
        const float* slot =
            p.parts + (int64_t)(2 * (c0 + i) + (i == 0 ? first : 0)) * slot_floats<RM, D>();
        ml[j] = *reinterpret_cast<const float2*>(slot + RM * D + 2 * r);
        v[j] = *reinterpret_cast<const float4*>(slot + r * D + d);
      }
    }
    float m = mx;
#pragma unroll
    for (int j = 0; j < 6; ++j) m = fmaxf(m, ml[j].x);
    const float base = m == -INFINITY ? 0.f : m;
    const float a = exp2_fast(mx - base);
    mx = m;
    l *= a;
    sum.x *= a; sum.y *= a; sum.z *= a; sum.w *= a;
#pragma unroll
    for (int j = 0; j < 6; ++j) {
      const float f = exp2_fast(ml[j].x - base);
      l = fmaf(ml[j].y, f, l);
      sum.x = fmaf(v[j].x, f, sum.x); sum.y = fmaf(v[j].y, f, sum.y);
      sum.z = fmaf(v[j].z, f, sum.z); sum.w = fmaf(v[j].w, f, sum.w);
    }
  }
  if constexpr (GROUPS > 1) {
    if (grp > 0) s_sum[grp - 1][lane] = sum;
    if (lane == 0) s_ml[grp] = make_float2(mx, l);
    __syncthreads();   // the block has one row: no warp has returned
    if (grp > 0) return;
  }
  float m = mx;
#pragma unroll
  for (int w = 1; w < GROUPS; ++w) m = fmaxf(m, s_ml[w].x);
  const float base = m == -INFINITY ? 0.f : m;
  const float a = exp2_fast(mx - base);
  l *= a;
  sum.x *= a; sum.y *= a; sum.z *= a; sum.w *= a;
#pragma unroll
  for (int w = 1; w < GROUPS; ++w) {
    const float f = exp2_fast(s_ml[w].x - base);
    const float4 v = s_sum[w - 1][lane];
    l = fmaf(s_ml[w].y, f, l);
    sum.x = fmaf(v.x, f, sum.x); sum.y = fmaf(v.y, f, sum.y);
    sum.z = fmaf(v.z, f, sum.z); sum.w = fmaf(v.w, f, sum.w);
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
  store_row4(to, make_float4(sum.x * inv, sum.y * inv, sum.z * inv, sum.w * inv));
}

template <typename E, int NW, int NR>
int launch(Params p, const DecodeQ8Call& c, int64_t B) {
  constexpr int RM = 8 * NR;
  static DeviceOnce once;
  const int rc = once.run(c.device, [] {
    return cudaFuncSetAttribute(decode_kernel<E, NW, NR>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                (int)sizeof(Shared)) == cudaSuccess ? kOk : kErrLaunch;
  });
  if (rc != kOk) return rc;
  // A launch takes as many (sequence, row tile) entries as its list can count.
  const int64_t of_entry = (int64_t)p.Hkv * (p.cap / kUnit + 2 + kHeadCost);
  if (of_entry > kMaxUnits) return kErrShape;
  const int tiles = (p.rows + RM - 1) / RM;
  const int most = (int)std::min<int64_t>(kMaxEntries, kMaxUnits / of_entry);
  const int tiles_at_once = std::min(tiles, most);
  const int64_t at_once = tiles_at_once < tiles ? 1 : most / tiles;   // sequences
  p.parts = static_cast<float*>(c.ws);
  p.heads = divisor(p.Hkv);
  // The first kernel may be launched before what is in front of it has ended: it waits
  // (griddepcontrol) before it reads anything.  The second one starts when every block of the
  // first is past that wait, and waits for the first before it reads what that writes.
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.stream = c.stream;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  const int most_blocks = c.num_sms * kBlocksPerSm;
  for (int64_t b = 0; b < B; b += at_once)
    for (int tile = 0; tile < tiles; tile += tiles_at_once) {
      const int here = std::min(tiles_at_once, tiles - tile);
      p.b0 = b;
      p.tile0 = tile;
      const int seqs = (int)std::min(at_once, B - b);
      p.seqs = divisor(seqs);
      p.entries = seqs * here;
      // The list has all sequences' first row tiles, then all second ones: with a number of
      // blocks that the tiles divide, blocks far apart read the same keys at the same time and
      // the cache comes from HBM once (32 sequences of 8192 keys, 32/8 heads of 128, 8 / 12 / 20
      // tokens: 159 / 244 / 370 us; each sequence's tiles in a row 172 / 247 / -, tiles that
      // do not divide the blocks - / 254 / 407).
      const int blocks = here <= 16 ? most_blocks - most_blocks % here : most_blocks;
      // A head has about blocks / heads parts: for many of them eight warps to a row, for
      // few a warp (32 sequences of 8 heads: 49.7 us for both kernels with eight, 46.3 with one).
      const int rows = std::min(RM, p.rows);
      const bool many = (int64_t)p.entries * p.Hkv * 8 <= blocks;
      p.joined = divisor(many ? rows : 1);
      const int64_t joins = (int64_t)p.entries * p.Hkv * p.joined.by * NW;
      if (joins > 0x7fffffff) return kErrShape;
      cfg.gridDim = dim3((unsigned)blocks);
      cfg.blockDim = dim3(kThreads);
      cfg.dynamicSmemBytes = sizeof(Shared);
      cudaError_t err = cudaLaunchKernelEx(&cfg, decode_kernel<E, NW, NR>, (const Params)p);
      if (err == cudaSuccess) {
        cfg.gridDim = dim3((unsigned)joins);
        cfg.blockDim = dim3(many ? 256 : rows * 32);
        cfg.dynamicSmemBytes = 0;
        err = many ? cudaLaunchKernelEx(&cfg, join_kernel<E, NW, NR, 8>, (const Params)p, blocks)
                   : cudaLaunchKernelEx(&cfg, join_kernel<E, NW, NR, 1>, (const Params)p, blocks);
      }
      if (err != cudaSuccess) {
        cudaGetLastError();
        return kErrLaunch;
      }
    }
  return kOk;
}

}  // namespace

size_t decode_q8_workspace(int64_t T, int H, int Hkv, int D, int dtype, int num_sms) {
  const int rm = dtype == PFA_F32 && T * (H / Hkv) <= 8 ? 8 : 16;   // most rows of a tile
  return 2 * (size_t)num_sms * kBlocksPerSm * (rm * D + rm * 2) * sizeof(float);  // two slots a run
}

int launch_decode_q8(const DecodeQ8Call& c) {
  Params p;
  p.q = c.q; p.out = c.out;
  p.k8 = (const uint8_t*)c.cache.k8; p.v8 = (const uint8_t*)c.cache.v8;
  p.k_scale = c.cache.k_scale; p.v_scale = c.cache.v_scale;
  p.lengths = c.span.lengths;
  p.T = c.span.T; p.start_pos = c.span.start_pos;
  p.q_row = c.q_row; p.out_row = c.out_row;
  p.cap = (int)c.cache.max_seq_len;
  p.Hkv = c.Hkv; p.group = divisor(c.H / c.Hkv); p.window = c.window;
  p.block_shift = c.cache.block == 16 ? 4 : c.cache.block == 32 ? 5 : c.cache.block == 64 ? 6 : 7;
  if (p.T * (c.H / c.Hkv) > (1 << 30)) return kErrShape;
  p.rows = (int)p.T * (c.H / c.Hkv);
  p.scale_log2 = c.scale * 1.4426950408889634f;
  p.err = c.err;
  const int64_t B = c.span.B;
  if (c.dtype == PFA_BF16)
    return c.D == 128 ? launch<__nv_bfloat16, 1, 2>(p, c, B) : launch<__nv_bfloat16, 4, 2>(p, c, B);
  // fp32: with tiles of 16 rows each converted code serves two products, with 8 a unit is
  // through sooner.  2048 tokens at 14336, 32/8 heads of 128: 3514 us against 4183; 3 tokens of 4
  // sequences, window 1024, 8/2 heads of 512 (528 units of 8 rows): 12.6 against 10.8.
  const int64_t keys = p.window > 0 ? std::min<int64_t>(p.cap, p.window + p.T) : p.cap;
  const int64_t units = B * ((p.rows + 7) / 8) * p.Hkv * (keys / kUnit + 1);
  if (p.rows <= 8 || units < (int64_t)8 * c.num_sms * kBlocksPerSm)
    return c.D == 128 ? launch<float, 1, 1>(p, c, B) : launch<float, 4, 1>(p, c, B);
  return c.D == 128 ? launch<float, 1, 2>(p, c, B) : launch<float, 4, 2>(p, c, B);
}

}  // namespace pfa
