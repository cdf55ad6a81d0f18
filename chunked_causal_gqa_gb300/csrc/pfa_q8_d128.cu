// pfa_q8_d128.cu -- prefill attention of bf16 queries over an 8-bit cache,
// head_dim 128, on the sm_103a tensor cores, straight from the codes.
//
// The work of a block, its query tiles and its online softmax are those of
// pfa_bf16_d128.cu: a pair of 128-row tiles A and B of one kv head (row r of a tile:
// token r / group, head r % group) walks key tiles of 128, two softmax warpgroups
// (one row a thread) hide each other's products, and the pairs of the last
// partial wave are cut into key ranges that a second kernel merges.  What differs
// is how K and V reach the operand tiles: four converter warps read the codes
// (16 KB a tile, half of bf16's bytes), turn them into halves and write the
// 128-byte-swizzled layout that a TMA load of a 16-bit tile would leave.
//
// Arithmetic.  All operands are halves (one type for both sides of a product):
//   k: code * (its block's scale / the largest of the block's key range) * 2^7,
//   v: likewise.  Scales are powers of two, so a code is exact as long as its scale is
//      within 2^-22 of the largest (2^7 * 448 < 65504; e4m3's smallest step is 2^-9,
//      half's 2^-24); below that it is rounded to 2^-32 of the largest block's step.
//   q: times a power of two for each row that brings its largest element to 2^13 ..
//      2^14, exact but for elements 2^27 below it.
//   p = 2^(s - base + 7), rounded to 11 bits, small ones to 2^-25.  The base is at most 8 below
//      the row's running maximum, so p <= 2^15, and small weights are off by up to 2^-32 of the
//      row's largest (bf16 weights would keep 8 bits of each).  l has the same factor 2^7.
// The factors are undone in the scores' multiplier and in the final 1 / l.
//
// Conversion is 4 instructions for 4 codes (two cvt.rn.f16x2.e4m3x2, two
// products); through bf16 it would be 12 (no e4m3 -> bf16 conversion exists).
//
// Warps: 0-3 and 4-7 softmax of tiles A and B, 8-11 converters, 12 TMEM and MMA
// issue; 16 warps are launched with 128 registers a thread and split them
// 200 / 200 / 72 / 40 by warpgroup (512 = 4 * 128).
//
// Measured on GB300: 128 tokens at 63360, 32/8 heads, 124 us in a graph, 129 through Python
// (floor 69.5 us of tensor time; reading the cache back and running the 16-bit kernel takes
// 153 us, 60 of them for the 390 MB of the read-back).  A key tile of a pair takes 3600 cycles: 2200 of
// tensor work, 900 of waiting for tile A's weights (the softmax's chain, which the
// converters on the same schedulers lengthen: 2900 cycles a tile in pfa_bf16_d128.cu)
// and 350 for operand tiles.  From about 1000 rows a kv head on the read-back costs
// less than that, and pfa_prefill_attention_q8 takes it.
// Steps: bounds checks and lane order of the converters 171 -> 129 us; packed fp32 pairs
// and their registers 127.4; narrower merge blocks 126.3.  Tried: three converter warps
// with a tile each and twelve warps in all (164 us: too few loads in flight), registers
// 176 / 96 / 64 and 192 / 80 / 48 with scalar arithmetic (154, 139 us: spills).
#include "pfa_internal.h"
#include "pfa_ptx.cuh"
#include "pfa_q8.cuh"

#include "../../include/pfa.h"

#include <algorithm>
#include <climits>
#include <cmath>

namespace pfa {
namespace {

constexpr int kBM = 128, kBN = 128;             // rows of a query tile, keys of a key tile
constexpr int kHalfBytes = 128 * 128;           // 128 rows x 64 halves (one swizzle span)
constexpr int kTileBytes = 2 * kHalfBytes;
constexpr int kSlots = 5;                       // operand ring depth (tiles)
constexpr int kThreads = 512;
constexpr float kRescaleThreshold = 8.f;        // log2 units
constexpr float kOperandScale = 128.f;          // of k and v
constexpr float kWeightBits = 7.f;              // weights and their sum are times 2^7

constexpr int kSmemQ = 0;
constexpr int kSmemRing = 2 * kTileBytes;
constexpr int kSmemBars = kSmemRing + kSlots * kTileBytes;
constexpr int kSmemAlloc = kSmemBars + 512 + 1024;   // + alignment

constexpr int kBarQ = 0;                     // both Q tiles written (8 warps)
constexpr int kBarFull = 1;                  // kSlots: operand tile written (4 warps)
constexpr int kBarEmpty = kBarFull + kSlots; // kSlots
constexpr int kBarS = kBarEmpty + kSlots;    // 2 (A, B)
constexpr int kBarP = kBarS + 2;             // 2 (4 warps)
constexpr int kBarO = kBarP + 2;             // 2
constexpr int kBarDrain = kBarO + 2;
constexpr int kNumBars = kBarDrain + 1;
constexpr int kOffTmemSlot = kNumBars * 8, kOffAbort = kOffTmemSlot + 4, kOffRef = kOffAbort + 4;
static_assert(kOffRef + 32 * 8 + 8 <= 512, "barrier area");

// Instruction descriptors with half operands: the bf16 ones without the two type fields.
constexpr uint32_t kTypes = (1u << 7) | (1u << 10);
constexpr uint32_t kIdescQK = idesc_bf16_f32(kBM, kBN, false) & ~kTypes;
constexpr uint32_t kIdescPV = idesc_bf16_f32(kBM, 128, true) & ~kTypes;

constexpr int kPairRows = 2 * kBM;
constexpr size_t kSlotFloats = (size_t)kPairRows * 128 + 2 * kPairRows;  // O, base, sum

struct Params {
  const __nv_bfloat16* q;
  __nv_bfloat16* out;
  const uint8_t *k8, *v8;
  const float *k_scale, *v_scale;
  float* ws;
  int64_t row;                   // elements between tokens of q and of out
  int64_t cap;
  int T, start_pos, Hkv, tok_per_tile, window, units_per_head, block_shift;
  Divisor group;
  int p1, p2, parts;             // pairs run whole, pairs cut into parts
  float scale_log2;
  unsigned* err;
  uint64_t wait_limit_ns;
  int flags;
};

struct Unit {
  int kh, t0;        // kv head, first token of tile A (tile B: + tok_per_tile)
  int first, n;      // key tiles [first, first + n)
  int lo, hi;        // keys that some row sees
};
// Latest tokens (most keys) first.
__host__ __device__ inline Unit unit_of(int T, int start_pos, int Hkv, int tok_per_tile, int window,
                                        int units_per_head, int pair) {
  Unit u;
  u.kh = pair % Hkv;
  u.t0 = 2 * (units_per_head - 1 - pair / Hkv) * tok_per_tile;
  const int t_end = u.t0 + 2 * tok_per_tile < T ? u.t0 + 2 * tok_per_tile : T;
  u.hi = start_pos + t_end - 1;
  u.lo = 0;
  if (window > 0 && start_pos + u.t0 - window + 1 > 0) u.lo = start_pos + u.t0 - window + 1;
  u.first = u.lo / kBN;
  u.n = u.hi / kBN - u.first + 1;
  return u;
}

template <int N>
__device__ __forceinline__ void registers_up() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" :: "n"(N));
}
template <int N>
__device__ __forceinline__ void registers_down() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" :: "n"(N));
}
__device__ __forceinline__ uint32_t pack_half2(float a, float b) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
  return r;
}
__device__ __forceinline__ uint32_t mul_half2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// Two floats in a register pair, one instruction for both.
__device__ __forceinline__ uint64_t pair_of(float a, float b) {
  uint64_t v;
  asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(a), "f"(b));
  return v;
}
__device__ __forceinline__ void split_pair(uint64_t v, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ uint64_t fma_pair(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t v;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(v) : "l"(a), "l"(b), "l"(c));
  return v;
}
__device__ __forceinline__ uint64_t add_pair(uint64_t a, uint64_t b) {
  uint64_t v;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(v) : "l"(a), "l"(b));
  return v;
}

__global__ void __launch_bounds__(kThreads, 1)
q8_d128_kernel(const __grid_constant__ Params p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const uint32_t sbase = smem_u32(smem);
  const uint32_t bars = sbase + kSmemBars;
  auto bar = [&](int i) -> uint32_t { return bars + 8u * (uint32_t)i; };
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + kSmemBars + kOffTmemSlot);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + kSmemBars + kOffAbort);
  float2* refs = reinterpret_cast<float2*>(smem + kSmemBars + ((kOffRef + 7) & ~7));

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint64_t lim = p.wait_limit_ns;

  // ---- this block's pair and key tiles [kb, ke)
  int pair = blockIdx.x, kb = 0, slot = -1;
  if (pair >= p.p1) {
    slot = pair - p.p1;
    pair = p.p1 + slot % p.p2;
  }
  const Unit u = unit_of(p.T, p.start_pos, p.Hkv, p.tok_per_tile, p.window, p.units_per_head, pair);
  int ke = u.n;
  if (slot >= 0) {
    const int r = slot / p.p2;
    kb = (int)((int64_t)u.n * r / p.parts);
    ke = (int)((int64_t)u.n * (r + 1) / p.parts);
  }
  const int n = ke - kb;
  const int key_first = (u.first + kb) * kBN;
  const int lo = max(u.lo, key_first), hi = min(u.hi, key_first + n * kBN - 1);

  if (tid == 0) {
    for (int i = 0; i < kNumBars; ++i) {
      const bool four = (i >= kBarFull && i < kBarFull + kSlots) || i == kBarP || i == kBarP + 1;
      mbar_init(bar(i), i == kBarQ ? 8u : four ? 4u : 1u);
    }
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 12) {
    tmem_alloc(smem_u32(tmem_slot), 512);
    tmem_relinquish();
  }
  // the largest scales of the key range
  const int64_t scales = (int64_t)u.kh * (p.cap >> p.block_shift);
  {
    float a = 0x1p-100f, b = 0x1p-100f;
    for (int i = (lo >> p.block_shift) + tid; i <= hi >> p.block_shift; i += kThreads) {
      a = fmaxf(a, p.k_scale[scales + i]);
      b = fmaxf(b, p.v_scale[scales + i]);
    }
    for (int o = 16; o > 0; o >>= 1) {
      a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
      b = fmaxf(b, __shfl_xor_sync(0xffffffffu, b, o));
    }
    if (lane == 0) refs[warp] = make_float2(a, b);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  float kref = refs[0].x, vref = refs[0].y;
#pragma unroll
  for (int w = 1; w < kThreads / 32; ++w) {
    kref = fmaxf(kref, refs[w].x);
    vref = fmaxf(vref, refs[w].y);
  }

  if (warp >= 12) {
    registers_down<40>();
    if (warp == 12) {
      // ---------------------------------------------------------- MMA issue (whole warp)
      const uint32_t tSA = tmem + 0, tSB = tmem + 128, tOA = tmem + 256, tOB = tmem + 384;
      const uint64_t qdA = sdesc_sw128(sbase + kSmemQ, 16, 1024);
      const uint64_t qdB = sdesc_sw128(sbase + kSmemQ + kTileBytes, 16, 1024);
      uint32_t li = 0;  // ring index of the next K tile
      auto full = [&](uint32_t t) {
        return mbar_wait_warp(bar(kBarFull + (int)(t % kSlots)), (t / kSlots) & 1u, abort_flag,
                              p.err, lim);
      };
      auto pv = [&](uint32_t tO, uint32_t tP, uint32_t t, bool more) {
        const uint32_t at = sbase + kSmemRing + (t % kSlots) * kTileBytes;
        mma8_ts<2048 / 16>(tO, tP, sdesc_sw128(at, kHalfBytes, 1024), kIdescPV, more ? 1u : 0u);
      };
      bool ok = mbar_wait_warp(bar(kBarQ), 0, abort_flag, p.err, lim), issued = false;
      for (int i = 0; i < n && ok; ++i, li += 2) {
        if (!(ok = full(li))) break;
        tc_fence_after();
        const uint64_t kd = sdesc_sw128(sbase + kSmemRing + (li % kSlots) * kTileBytes, 16, 1024);
        mma8_ss_kmajor<kHalfBytes / 16>(tSA, qdA, kd, kIdescQK, 0);
        issued = true;
        tc_commit_elect(bar(kBarS + 0));
        if (i > 0) {
          if (!(ok = mbar_wait_warp(bar(kBarP + 1), (i - 1) & 1u, abort_flag, p.err, lim))) break;
          tc_fence_after();
          pv(tOB, tSB, li - 1, i > 1);
          tc_commit_elect(bar(kBarEmpty + (int)((li - 1) % kSlots)));
        }
        mma8_ss_kmajor<kHalfBytes / 16>(tSB, qdB, kd, kIdescQK, 0);
        tc_commit_elect(bar(kBarS + 1));
        tc_commit_elect(bar(kBarEmpty + (int)(li % kSlots)));
        if (!(ok = full(li + 1))) break;
        if (!(ok = mbar_wait_warp(bar(kBarP + 0), i & 1u, abort_flag, p.err, lim))) break;
        tc_fence_after();
        pv(tOA, tSA, li + 1, i > 0);
      }
      if (ok && (ok = mbar_wait_warp(bar(kBarP + 1), (n - 1) & 1u, abort_flag, p.err, lim))) {
        tc_fence_after();
        pv(tOB, tSB, li - 1, n > 1);
        tc_commit_elect(bar(kBarO + 0));
        tc_commit_elect(bar(kBarO + 1));
      }
      if (issued) {
        // everything issued must complete before TMEM is freed
        tc_commit_elect(bar(kBarDrain));
        mbar_wait_warp(bar(kBarDrain), 0, abort_flag, p.err, lim, true);
      }
    }
  } else if (warp >= 8) {
    // ------------------------------------------------------------ converters
    registers_down<72>();
    // A warp has 32 rows of the tile, eight at a time: lane l row l % 8 and, of the row's
    // eight pieces of 16 codes, piece l / 8 of the first half or of the second (load 2 g + half).
    // Eight lanes with eight rows and one chunk fill all chunks of the swizzle.
    const int r0 = (warp - 8) * 32 + (lane & 7), piece = lane >> 3;
    const uint32_t at = (uint32_t)r0 * 128 + (((uint32_t)piece * 2 ^ (uint32_t)(lane & 7)) << 4);
    const int64_t off0 = ((int64_t)u.kh * p.cap + r0) * 128 + piece * 16;
    const float unit_k = kOperandScale / kref, unit_v = kOperandScale / vref;
    uint4 code[8];
    float sc[4];
    // load i of the ring's tile t (K and V in turn); nothing of a key that no row sees
    auto load = [&](int t, int i) {
      const int key0 = key_first + (t >> 1) * kBN, key = key0 + r0 + 8 * (i >> 1);
      const uint8_t* src = (t & 1 ? p.v8 : p.k8) + off0 + (int64_t)key0 * 128 + (i >> 1) * 1024 +
                           (i & 1) * 64;
      const bool on = key >= lo && key <= hi;
      code[i] = on ? __ldg(reinterpret_cast<const uint4*>(src)) : make_uint4(0, 0, 0, 0);
      if (i % 2 == 0) {   // eight rows are in one block
        sc[i >> 1] = on ? __ldg((t & 1 ? p.v_scale : p.k_scale) + scales + (key >> p.block_shift)) : 0.f;
      }
    };
    auto load_inner = [&](int t, int i) {   // all keys of the tile are seen
      const int key0 = key_first + (t >> 1) * kBN, key = key0 + r0 + 8 * (i >> 1);
      const uint8_t* src = (t & 1 ? p.v8 : p.k8) + off0 + (int64_t)key0 * 128;
      code[i] = __ldg(reinterpret_cast<const uint4*>(src + (i >> 1) * 1024 + (i & 1) * 64));
      if (i % 2 == 0)
        sc[i >> 1] = __ldg((t & 1 ? p.v_scale : p.k_scale) + scales + (key >> p.block_shift));
    };
    auto convert = [&](int i, uint8_t* dst, float unit) {
      const uint32_t w[4] = {code[i].x, code[i].y, code[i].z, code[i].w};
      const float f = sc[i >> 1] * unit;
      const uint32_t ff = pack_half2(f, f);
      uint32_t h[8];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        e4m3x4_to_half(w[k], h[2 * k], h[2 * k + 1]);
        h[2 * k] = mul_half2(h[2 * k], ff);
        h[2 * k + 1] = mul_half2(h[2 * k + 1], ff);
      }
      uint8_t* to = dst + (i >> 1) * 1024 + (i & 1) * kHalfBytes;
      *reinterpret_cast<uint4*>(to + at) = make_uint4(h[0], h[1], h[2], h[3]);
      *reinterpret_cast<uint4*>(to + (at ^ 16u)) = make_uint4(h[4], h[5], h[6], h[7]);
    };
    bool ok = true;
#pragma unroll
    for (int i = 0; i < 8; ++i) load(0, i);
#pragma unroll 1
    for (int t = 0; t < 2 * n; ++t) {
      // the rows two key tiles on, into L2: one lane, one instruction
      const int ahead = key_first + ((t >> 1) + 2) * kBN;
      if (tid == 256 && ahead + kBN - 1 <= hi)
        asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;"
                     :: "l"((t & 1 ? p.v8 : p.k8) + ((int64_t)u.kh * p.cap + ahead) * 128),
                        "n"(kBN * 128) : "memory");
      const float unit = t & 1 ? unit_v : unit_k;
      const uint32_t e = (uint32_t)t % kSlots;
      ok = mbar_wait_warp(bar(kBarEmpty + (int)e), (((uint32_t)t / kSlots) & 1u) ^ 1u, abort_flag,
                          p.err, lim);
      if (!ok) break;
      uint8_t* dst = smem + kSmemRing + e * kTileBytes;
      const int next0 = key_first + ((t + 1) >> 1) * kBN;
      if (t + 1 < 2 * n && next0 >= lo && next0 + kBN - 1 <= hi) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          convert(i, dst, unit);
          if (i % 2) {
            load_inner(t + 1, i - 1);   // arrives while the ring is full
            load_inner(t + 1, i);
          }
        }
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) convert(i, dst, unit);
        if (t + 1 < 2 * n) {
#pragma unroll
          for (int i = 0; i < 8; ++i) load(t + 1, i);
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(kBarFull + (int)e));
    }
  } else {
    // ------------------------------------------------------------ softmax
    registers_up<200>();
    const int X = warp >> 2, wq = warp & 3, row = wq * 32 + lane;
    const int tok = row / p.group, hrow = row - tok * (int)p.group.by;
    const int t0 = u.t0 + X * p.tok_per_tile;
    const bool valid = tok < p.tok_per_tile && t0 + tok < p.T;
    const int64_t at = (int64_t)(t0 + tok) * p.row + (int64_t)(u.kh * (int)p.group.by + hrow) * 128;
    const uint32_t lane_off = (uint32_t)(wq * 32) << 16;
    const uint32_t tS = tmem + lane_off + (uint32_t)(X * 128);
    const uint32_t tO = tmem + lane_off + 256u + (uint32_t)(X * 128);

    // ---- the row as halves, its largest element at 2^13 .. 2^14
    float c;
    {
      uint4 w[16];
      float amax = 0.f;
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        w[i] = make_uint4(0, 0, 0, 0);
        if (valid) w[i] = __ldg(reinterpret_cast<const uint4*>(p.q + at) + i);
        const uint32_t v[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
        for (int k = 0; k < 4; ++k)
          amax = fmaxf(amax, fmaxf(fabsf(__uint_as_float(v[k] << 16)),
                                   fabsf(__uint_as_float(v[k] & 0xffff0000u))));
      }
      int ex = 13 + 127 - (int)(__float_as_uint(amax) >> 23);
      if (amax == 0.f || !(amax <= 3.402823466e38f)) ex = 0;
      ex = min(ex, 120);
      // a negative scale goes into the sign of q: the maximum is taken before the multiplier
      const float up = copysignf(__uint_as_float((uint32_t)(127 + ex) << 23), p.scale_log2);
      const float down = __uint_as_float((uint32_t)(127 - ex) << 23);
      // a multiplier of 0 would turn a masked score into NaN
      c = fmaxf(fabsf(p.scale_log2) * down * (kref / kOperandScale), 0x1p-126f);
      uint8_t* dst = smem + kSmemQ + X * kTileBytes + row * 128;
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const uint32_t v[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
        uint32_t h[4];
#pragma unroll
        for (int k = 0; k < 4; ++k)
          h[k] = pack_half2(__uint_as_float(v[k] << 16) * up, __uint_as_float(v[k] & 0xffff0000u) * up);
        *reinterpret_cast<uint4*>(dst + (i >> 3) * kHalfBytes + (((i & 7) ^ (row & 7)) << 4)) =
            make_uint4(h[0], h[1], h[2], h[3]);
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(kBarQ));
    }

    bool ok = true;
    if ((p.flags & kFlagForceTimeout) && X == 0) {
      // test hook: wait on a barrier nothing signals, so the limit expires
      ok = mbar_wait(bar(kBarDrain), 0, abort_flag, p.err, lim);
      ok = __all_sync(0xffffffffu, ok);
    }
    const int pos_first = p.start_pos + t0;
    int key_rel = key_first - (pos_first + tok);   // the tile's first key, from the row's position
    float m_run = -INFINITY, l = 0.f;
    for (int i = 0; i < n && ok; ++i, key_rel += kBN) {
      ok = mbar_wait(bar(kBarS + X), i & 1u, abort_flag, p.err, lim);
      if (!(ok = __all_sync(0xffffffffu, ok))) break;
      tc_fence_after();
      uint32_t r0[32], r1[32], r2[32], r3[32];
      tmem_ld32(tS + 0, r0);
      tmem_ld32(tS + 32, r1);
      tmem_ld32(tS + 64, r2);
      tmem_ld32(tS + 96, r3);
      tmem_wait_ld(r0);
      tmem_wait_ld(r1);
      tmem_wait_ld(r2);
      tmem_wait_ld(r3);
      float x[128];
#pragma unroll
      for (int k = 0; k < 32; ++k) {
        x[k] = __uint_as_float(r0[k]);
        x[32 + k] = __uint_as_float(r1[k]);
        x[64 + k] = __uint_as_float(r2[k]);
        x[96 + k] = __uint_as_float(r3[k]);
      }
      const int from_first = key_rel + tok;   // tile's first key - pos_first
      const bool all_visible = from_first + kBN - 1 <= 0 &&
                               (p.window <= 0 || from_first > p.tok_per_tile - 1 - p.window);
      if (!all_visible) {
        const int top = -key_rel, bottom = p.window > 0 ? -key_rel - p.window : -1;
#pragma unroll
        for (int k = 0; k < 128; ++k)
          if (k > top || k <= bottom) x[k] = -INFINITY;
      }
      float mx;
      {
        float m[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) m[k] = max3f(x[k], x[8 + k], x[16 + k]);
#pragma unroll
        for (int k = 24; k < 120; k += 16) {
#pragma unroll
          for (int q = 0; q < 8; ++q) m[q] = max3f(m[q], x[k + q], x[k + 8 + q]);
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) m[k] = fmaxf(m[k], x[120 + k]);
        mx = max3f(max3f(m[0], m[1], m[2]), max3f(m[3], m[4], m[5]), fmaxf(m[6], m[7])) * c;
      }
      float alpha = 1.f;
      bool rescale = false;
      if (mx > m_run + kRescaleThreshold) {
        alpha = ex2(m_run - mx);
        rescale = i > 0 && m_run != -INFINITY;
        m_run = mx;
      }
      const float base = m_run == -INFINITY ? 0.f : m_run;
      uint32_t pk0[32], pk1[32];
      const uint64_t cc = pair_of(c, c), bb = pair_of(kWeightBits - base, kWeightBits - base);
      uint64_t ls[4] = {0, 0, 0, 0};
#pragma unroll
      for (int k = 0; k < 64; ++k) {
        float a, b;
        split_pair(fma_pair(pair_of(x[2 * k], x[2 * k + 1]), cc, bb), a, b);
        a = ex2(a);
        b = ex2(b);
        const uint32_t w = pack_half2(a, b);
        if (k < 32) pk0[k] = w; else pk1[k - 32] = w;
        ls[k & 3] = add_pair(ls[k & 3], pair_of(a, b));
      }
      float s0, s1;
      split_pair(add_pair(add_pair(ls[0], ls[1]), add_pair(ls[2], ls[3])), s0, s1);
      l = l * alpha + (s0 + s1);
      // the commit that signalled these scores covers the last product into O
      if (__any_sync(0xffffffffu, rescale)) {
        const float f = rescale ? alpha : 1.f;
#pragma unroll 1
        for (int c0 = 0; c0 < 128; c0 += 32) {
          uint32_t o[32];
          tmem_ld32(tO + c0, o);
          tmem_wait_ld(o);
#pragma unroll
          for (int k = 0; k < 32; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * f);
          tmem_st32(tO + c0, o);
        }
      }
      tmem_st32(tS + 0, pk0);
      tmem_st32(tS + 32, pk1);
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(kBarP + X));
    }
    if (ok) {
      ok = mbar_wait(bar(kBarO + X), 0, abort_flag, p.err, lim);
      ok = __all_sync(0xffffffffu, ok);
    }
    if (ok) {
      tc_fence_after();
      const float undo = vref / kOperandScale;
      if (slot < 0) {
        const float inv = l > 0.f ? undo / l : (l == 0.f ? 0.f : l);   // NaN stays NaN
#pragma unroll 1
        for (int c0 = 0; c0 < 128; c0 += 32) {
          uint32_t o[32];
          tmem_ld32(tO + c0, o);
          tmem_wait_ld(o);
          uint32_t w[16];
#pragma unroll
          for (int k = 0; k < 16; ++k)
            w[k] = pack_bf16x2(__uint_as_float(o[2 * k]) * inv, __uint_as_float(o[2 * k + 1]) * inv);
          if (valid) {
            uint4* dst = reinterpret_cast<uint4*>(p.out + at + c0);
#pragma unroll
            for (int k = 0; k < 4; ++k)
              dst[k] = make_uint4(w[4 * k], w[4 * k + 1], w[4 * k + 2], w[4 * k + 3]);
          }
        }
      } else {
        // part of a pair: [column / 4][row][4], then exponent bases, then sums
        float* part = p.ws + (size_t)slot * kSlotFloats;
        const int R = X * kBM + row;
        float4* col = reinterpret_cast<float4*>(part) + R;
#pragma unroll 1
        for (int c0 = 0; c0 < 128; c0 += 32) {
          uint32_t o[32];
          tmem_ld32(tO + c0, o);
          tmem_wait_ld(o);
#pragma unroll
          for (int k = 0; k < 8; ++k)
            if (valid)
              col[(size_t)(c0 / 4 + k) * kPairRows] = make_float4(
                  __uint_as_float(o[4 * k]) * undo, __uint_as_float(o[4 * k + 1]) * undo,
                  __uint_as_float(o[4 * k + 2]) * undo, __uint_as_float(o[4 * k + 3]) * undo);
        }
        part[(size_t)kPairRows * 128 + R] = m_run;
        part[(size_t)kPairRows * 128 + kPairRows + R] = l;
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 12) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Joins the parts of a pair in key order: block (e, g) has pair p1 + e and columns
// 8 g .. 8 g + 7, thread R its row R.
constexpr int kMergeCols = 8, kMergeAhead = 8;
__global__ void __launch_bounds__(kPairRows) q8_merge_kernel(const __grid_constant__ Params p) {
  const int e = blockIdx.x, R = threadIdx.x, X = R / kBM, row = R % kBM;
  const Unit u = unit_of(p.T, p.start_pos, p.Hkv, p.tok_per_tile, p.window, p.units_per_head,
                         p.p1 + e);
  const int tok = row / p.group, t = u.t0 + X * p.tok_per_tile + tok;
  if (tok >= p.tok_per_tile || t >= p.T) return;
  const int cq = blockIdx.y * (kMergeCols / 4);
  const size_t off_m = (size_t)kPairRows * 128 + R;
  auto part = [&](int i) { return p.ws + (size_t)(i * p.p2 + e) * kSlotFloats; };
  float m = -INFINITY;
#pragma unroll 4
  for (int i = 0; i < p.parts; ++i) m = fmaxf(m, part(i)[off_m]);
  const float base = m == -INFINITY ? 0.f : m;
  float4 acc[kMergeCols / 4];
#pragma unroll
  for (int q = 0; q < kMergeCols / 4; ++q) acc[q] = make_float4(0.f, 0.f, 0.f, 0.f);
  float l = 0.f;
#pragma unroll kMergeAhead
  for (int i = 0; i < p.parts; ++i) {
    const float* s = part(i);
    const float w = ex2(s[off_m] - base);
    l = fmaf(w, s[off_m + kPairRows], l);
    const float4* col = reinterpret_cast<const float4*>(s) + R;
#pragma unroll
    for (int q = 0; q < kMergeCols / 4; ++q) {
      const float4 o = col[(size_t)(cq + q) * kPairRows];
      acc[q].x = fmaf(w, o.x, acc[q].x);
      acc[q].y = fmaf(w, o.y, acc[q].y);
      acc[q].z = fmaf(w, o.z, acc[q].z);
      acc[q].w = fmaf(w, o.w, acc[q].w);
    }
  }
  const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);
  uint32_t w[kMergeCols / 2];
#pragma unroll
  for (int q = 0; q < kMergeCols / 4; ++q) {
    w[2 * q] = pack_bf16x2(acc[q].x * inv, acc[q].y * inv);
    w[2 * q + 1] = pack_bf16x2(acc[q].z * inv, acc[q].w * inv);
  }
  const int h = u.kh * (int)p.group.by + row - tok * (int)p.group.by;
  uint4* dst = reinterpret_cast<uint4*>(p.out + (int64_t)t * p.row + (int64_t)h * 128 + cq * 4);
#pragma unroll
  for (int q = 0; q < kMergeCols / 8; ++q)
    dst[q] = make_uint4(w[4 * q], w[4 * q + 1], w[4 * q + 2], w[4 * q + 3]);
}

struct Plan {
  int tok_per_tile, units_per_head, pairs;
  int p1, p2, parts;
};
constexpr int kFixedTiles = 4;   // what a block costs beside its key tiles, in tiles

// Whole waves of pairs run whole; those of the last, partial wave are cut into
// the number of equal key ranges that ends soonest.
Plan plan_of(int T, int start_pos, int H, int Hkv, int window, int sms) {
  Plan s;
  s.tok_per_tile = kBM / (H / Hkv);
  s.units_per_head = ((T + s.tok_per_tile - 1) / s.tok_per_tile + 1) / 2;
  s.pairs = s.units_per_head * Hkv;
  s.p1 = s.pairs / sms * sms;
  s.p2 = s.pairs - s.p1;
  s.parts = 1;
  if (s.p2 > 0) {
    // every part of every pair has a key tile
    int least = INT_MAX, most = 0;
    for (int e = s.p1; e < s.pairs; ++e) {
      const int n = unit_of(T, start_pos, Hkv, s.tok_per_tile, window, s.units_per_head, e).n;
      least = std::min(least, n);
      most = std::max(most, n);
    }
    int64_t best = most + kFixedTiles;
    for (int parts = 2; parts <= std::min(least, s.p1 > 0 ? 8 : std::max(8, sms / s.p2)); ++parts) {
      const int64_t waves = ((int64_t)s.p2 * parts + sms - 1) / sms;
      const int64_t cost = waves * ((most + parts - 1) / parts + kFixedTiles) + kFixedTiles;  // + merge
      if (cost < best) {
        best = cost;
        s.parts = parts;
      }
    }
  }
  if (s.parts == 1) {
    s.p1 = s.pairs;
    s.p2 = 0;
  }
  return s;
}

}  // namespace

size_t q8_d128_workspace(int64_t T, int64_t start_pos, int H, int Hkv, int window, int num_sms) {
  const Plan s = plan_of((int)T, (int)start_pos, H, Hkv, window, num_sms);
  return (size_t)s.p2 * s.parts * kSlotFloats * sizeof(float);
}

int launch_q8_d128(const DecodeQ8Call& c) {
  const Plan s = plan_of((int)c.span.T, (int)c.span.start_pos, c.H, c.Hkv, c.window, c.num_sms);
  static DeviceOnce once;
  const int rc = once.run(c.device, [] {
    return cudaFuncSetAttribute(q8_d128_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                kSmemAlloc) == cudaSuccess ? kOk : kErrLaunch;
  });
  if (rc != kOk) return rc;
  Params p;
  p.q = (const __nv_bfloat16*)c.q;
  p.out = (__nv_bfloat16*)c.out;
  p.k8 = (const uint8_t*)c.cache.k8; p.v8 = (const uint8_t*)c.cache.v8;
  p.k_scale = c.cache.k_scale; p.v_scale = c.cache.v_scale;
  p.ws = (float*)c.ws;
  p.row = c.q_row;
  p.cap = c.cache.max_seq_len;
  p.T = (int)c.span.T; p.start_pos = (int)c.span.start_pos;
  p.Hkv = c.Hkv; p.tok_per_tile = s.tok_per_tile; p.window = c.window;
  p.units_per_head = s.units_per_head;
  p.block_shift = c.cache.block == 16 ? 4 : c.cache.block == 32 ? 5 : c.cache.block == 64 ? 6 : 7;
  p.group = divisor((uint32_t)(c.H / c.Hkv));
  p.p1 = s.p1; p.p2 = s.p2; p.parts = s.parts;
  p.scale_log2 = c.scale * 1.4426950408889634f;
  p.err = c.err;
  p.wait_limit_ns = c.wait_limit_ns;
  p.flags = c.flags;
  q8_d128_kernel<<<s.p1 + s.p2 * s.parts, kThreads, kSmemAlloc, c.stream>>>(p);
  if (cudaGetLastError() != cudaSuccess) return kErrLaunch;
  if (s.p2 > 0) {
    q8_merge_kernel<<<dim3(s.p2, 128 / kMergeCols), kPairRows, 0, c.stream>>>(p);
    if (cudaGetLastError() != cudaSuccess) return kErrLaunch;
  }
  return kOk;
}

}  // namespace pfa
