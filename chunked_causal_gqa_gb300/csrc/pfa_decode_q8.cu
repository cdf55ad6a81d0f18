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
#include "pfa_decode.cuh"

#include "../../include/pfa.h"

#include <cmath>

namespace pfa {
namespace {

constexpr int kBlocksPerSm = 2;
constexpr int kStages = 3;
constexpr int kUnit = 32;                      // keys of a unit
constexpr int kHalf = kUnit * 128;             // bytes of a warp's K (or V) part of a stage
constexpr int kStageBytes = 2 * kHalf;
constexpr int kJoinBytes = kWarps * 8 * 128 * 4;  // joins: 8 row sums of 128 floats for each warp
constexpr float kWeightScale = 16384.f;

struct Params : ListParams {
  static constexpr int kUnit = pfa::kUnit;
  static constexpr int kHeadCost = 8;
  static constexpr bool kSums = false;
  const uint8_t *k8, *v8;
  const float *k_scale, *v_scale;
  int block_shift;
};

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

struct Shared {
  alignas(128) uint8_t ring[kWarps][kStages][kStageBytes];
  alignas(16) uint8_t join[kJoinBytes];   // also: score exchange
  float scales[kWarps][kStages][4];       // K and V scales of a unit's two halves
  float2 ml[kWarps][16];                  // a warp's {m, l} of each row
  float vref[kWarps];
  ListShared list;
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

  int at, stop, first_entry, into;
  if (!run_start<RM, TEAMS>(p, sm.list, at, stop, first_entry, into)) return;

  Cursor<Params, RM, TEAMS> in, cu;   // copies, products
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
      const auto& x = in.x;
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
    const auto x = cu.x;
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

template <typename E, int NW, int NR>
int launch(const Params& p, const DecodeQ8Call& c) {
  static DeviceOnce once;
  const int rc = once.run(c.device, [] {
    return cudaFuncSetAttribute(decode_kernel<E, NW, NR>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                (int)sizeof(Shared)) == cudaSuccess ? kOk : kErrLaunch;
  });
  if (rc != kOk) return rc;
  const Kernels<Params> k = {decode_kernel<E, NW, NR>, join_kernel<Params, E, NW, 8 * NR, 8>,
                             join_kernel<Params, E, NW, 8 * NR, 1>, 8 * NR, NW, kBlocksPerSm,
                             sizeof(Shared)};
  return launch_list(k, p, c.span.B, c.num_sms, c.stream);
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
  p.unit = 1.f;
  p.err = c.err;
  p.parts = static_cast<float*>(c.ws);
  p.sums = nullptr;
  const int64_t B = c.span.B;
  if (c.dtype == PFA_BF16)
    return c.D == 128 ? launch<__nv_bfloat16, 1, 2>(p, c) : launch<__nv_bfloat16, 4, 2>(p, c);
  // fp32: with tiles of 16 rows each converted code serves two products, with 8 a unit is
  // through sooner.  2048 tokens at 14336, 32/8 heads of 128: 3514 us against 4183; 3 tokens of 4
  // sequences, window 1024, 8/2 heads of 512 (528 units of 8 rows): 12.6 against 10.8.
  const int64_t keys = p.window > 0 ? std::min<int64_t>(p.cap, p.window + p.T) : p.cap;
  const int64_t units = B * ((p.rows + 7) / 8) * p.Hkv * (keys / kUnit + 1);
  if (p.rows <= 8 || units < (int64_t)8 * c.num_sms * kBlocksPerSm)
    return c.D == 128 ? launch<float, 1, 1>(p, c) : launch<float, 4, 1>(p, c);
  return c.D == 128 ? launch<float, 1, 2>(p, c) : launch<float, 4, 2>(p, c);
}

}  // namespace pfa
