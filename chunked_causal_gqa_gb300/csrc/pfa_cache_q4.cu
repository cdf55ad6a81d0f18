// pfa_cache_q4.cu -- writing tokens into the 4-bit cache and reading rows back.
//
// Write: for each 16 channels of a new row, with y = x * 2^-exponent,
//   scale = e4m3(max |y| / 6),  code = e2m1(y / scale)
// and both roundings are those of the exact quotients, though these are rounded to a float in
// between: that could only move a quotient onto a border t between two codes (or scales).  The
// borders have at most five significant bits and the divisors s at most four, so s t is a
// float, and a y that differs from it does so by an ulp(y) at least; s being at most 1.875 * 2^e, the
// quotient is then 0.533 ulp(t) or more away from t, and the nearest float to it another one.
// y / s is y * (1 / s) with one correction by its residual y - q s, which is exact in a fused
// multiply-add: off by 2^-22 of a last place before its rounding, so exact where the quotient is a float
// (a border among them) and on the right side of every border elsewhere.
//
// Measured on GB300, one pass among others (GPU: in a graph):
//   write 1 token of 32 sequences, 8 heads of 128         3.9 to 4.2 us, the host's call (GPU 1.9)
//   write 2048 tokens of 8 heads of 128, bf16 (10.7 MB)   4.3 us (GPU 3.9; floor 1.6): one launch, position,
//     row and codes follow one another
//   read 63488 rows of 8 heads of 128 as bf16 (333 MB)    51.0 us, 6.5 TB/s (floor 49.1): HBM
//   read 3188 rows of 2 heads of 512 as fp32 (30 MB)      6.8 to 7.4 us, the host's call (GPU 5.6; floor 4.4)
// Reading back, a lane makes 16 output bytes at a time, so that both sides of a warp's pieces are contiguous.
#include "pfa_internal.h"
#include "pfa_ptx.cuh"
#include "pfa_q4.cuh"

#include "../../include/pfa.h"

#include <algorithm>
#include <cmath>

namespace pfa {
namespace {

constexpr int kThreads = 256;

struct WriteParams {
  const void *k, *v;
  uint8_t *k4, *v4, *k_scale, *v_scale;
  const int64_t* lengths;
  int64_t T, start_pos, cap, k_row, v_row, groups;   // groups: of K (and of V) in the call
  Divisor per_head, heads, tokens;                   // D / 16, Hkv, T
  float k_unit, v_unit;                              // 2^-exponent
  unsigned* err;
};

// A thread quantises 16 channels.
template <typename E>
__global__ void __launch_bounds__(kThreads) write_kernel(const WriteParams p) {
  asm volatile("griddepcontrol.launch_dependents;");
  const int64_t id = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  const bool isv = id >= p.groups;
  const int g = (int)(isv ? id - p.groups : id);
  if (id >= 2 * p.groups) return;
  const int hg = g / p.per_head, c = g - hg * (int)p.per_head.by;
  const int bt = hg / p.heads, h = hg - bt * (int)p.heads.by;
  const int b = bt / p.tokens, t = bt - b * (int)p.tokens.by;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int64_t end = p.lengths ? p.lengths[b] : p.start_pos + p.T;
  if (end < 0 || end > p.cap) {
    if (!isv && t == 0 && h == 0 && c == 0) atomicOr(p.err, kErrLengths);
    return;
  }
  const int64_t row = end - p.T + t;
  if (row < 0) return;
  const E* src = (isv ? (const E*)p.v : (const E*)p.k) + (int64_t)bt * (isv ? p.v_row : p.k_row) +
                 ((int64_t)h * p.per_head.by + c) * 16;
  const int64_t at = (((int64_t)b * p.heads.by + h) * p.cap + row) * p.per_head.by + c;
  float x[16];
  if constexpr (sizeof(E) == 4) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      *reinterpret_cast<float4*>(x + 4 * i) = reinterpret_cast<const float4*>(src)[i];
  } else {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint4 u = reinterpret_cast<const uint4*>(src)[i];
      const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        x[8 * i + 2 * j] = __uint_as_float(w[j] << 16);
        x[8 * i + 2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
      }
    }
  }
  const float unit = isv ? p.v_unit : p.k_unit;
  bool finite = true;
  float amax = 0.f;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    finite = finite && fabsf(x[i]) <= 3.402823466e38f;
    x[i] *= unit;
    amax = fmaxf(amax, fabsf(x[i]));
  }
  const uint8_t s = finite ? float_to_e4m3(__fdiv_rn(amax, 6.f)) : 0x7f;
  const float f = e4m3_to_float(s);
  uint2 w = make_uint2(0u, 0u);
  if (finite && f > 0.f) {
    const float r = __frcp_rn(f), most = 8.f * f;   // (beyond 8 the largest code, and no infinite product)
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const float y = fminf(fmaxf(x[i], -most), most), q = y * r;
      x[i] = copysignf(fmaf(fmaf(-q, f, y), r, q), y);   // (-0 stays -0)
    }
    w = make_uint2(float_to_e2m1x8(x), float_to_e2m1x8(x + 8));
  }
  reinterpret_cast<uint2*>(isv ? p.v4 : p.k4)[at] = w;
  (isv ? p.v_scale : p.k_scale)[at] = s;
}

struct ReadParams {
  const uint8_t *k4, *v4, *k_scale, *v_scale;
  void *k_out, *v_out;
  int64_t start, cap, out_head;
  Divisor chunks;   // blocks of threads for a head's rows
  int pieces;       // of 16 output bytes, of a head
  int D;
  float k_unit, v_unit;   // 2^exponent
};

// A thread makes kPieces pieces of 16 output bytes, all their codes asked for first.
constexpr int kPieces = 8;

template <typename E>
__global__ void __launch_bounds__(kThreads) read_kernel(const ReadParams p) {
  constexpr int N = 16 / sizeof(E);   // codes of a piece
  asm volatile("griddepcontrol.launch_dependents;");
  const int id = blockIdx.x / 2;
  const bool isv = blockIdx.x % 2;
  const int head = id / p.chunks, e0 = (id - head * (int)p.chunks.by) * (kThreads * kPieces);
  const int64_t row0 = (int64_t)head * p.cap + p.start;
  const uint8_t* src = (isv ? p.v4 : p.k4) + row0 * (p.D / 2);
  const uint8_t* scale = (isv ? p.v_scale : p.k_scale) + row0 * (p.D / 16);
  E* out = (isv ? (E*)p.v_out : (E*)p.k_out) + (int64_t)head * p.out_head;
  const float unit = isv ? p.v_unit : p.k_unit;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  uint32_t w[kPieces];
  uint8_t s[kPieces];
#pragma unroll
  for (int i = 0; i < kPieces; ++i) {
    const int e = e0 + i * kThreads + threadIdx.x;
    if (e >= p.pieces) break;
    if constexpr (N == 8)
      w[i] = reinterpret_cast<const uint32_t*>(src)[e];
    else
      w[i] = reinterpret_cast<const uint16_t*>(src)[e];
    s[i] = scale[e / (16 / N)];
  }
#pragma unroll
  for (int i = 0; i < kPieces; ++i) {
    const int e = e0 + i * kThreads + threadIdx.x;
    if (e >= p.pieces) break;
    const float f = e4m3_to_float(s[i]) * unit;
    float x[N];
    const uint32_t h[4] = {e2m1x2_to_half<0>(w[i]), e2m1x2_to_half<1>(w[i]),
                           e2m1x2_to_half<2>(w[i]), e2m1x2_to_half<3>(w[i])};
#pragma unroll
    for (int j = 0; j < N / 2; ++j) {
      const float2 y = __half22float2(*reinterpret_cast<const __half2*>(&h[j]));
      x[2 * j] = y.x * f;
      x[2 * j + 1] = y.y * f;
    }
    if constexpr (N == 8)
      store8(out + (int64_t)e * N, x);
    else
      *reinterpret_cast<float4*>(out + (int64_t)e * N) = make_float4(x[0], x[1], x[2], x[3]);
  }
}

// A launch that may start before what is in front of it has ended (it waits on the device).
template <typename P>
int launch(void (*kernel)(const P), int64_t grid, const P& p, cudaStream_t stream) {
  if (grid > 0x7fffffff) return kErrShape;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, kernel, p) == cudaSuccess) return kOk;
  cudaGetLastError();
  return kErrLaunch;
}

float power(int e) { return std::ldexp(1.f, e); }

}  // namespace

int launch_cache_write_q4(const WriteQ4Call& c) {
  WriteParams p;
  p.k = c.k; p.v = c.v;
  p.k4 = (uint8_t*)c.cache.k4; p.v4 = (uint8_t*)c.cache.v4;
  p.k_scale = (uint8_t*)c.cache.k_scale; p.v_scale = (uint8_t*)c.cache.v_scale;
  p.lengths = c.span.lengths;
  p.T = c.span.T; p.start_pos = c.span.start_pos;
  p.cap = c.cache.max_seq_len; p.k_row = c.k_row; p.v_row = c.v_row;
  const int per = c.D / 16;
  if (c.span.B * c.span.T > 0x7fffffff / ((int64_t)per * c.Hkv)) return kErrShape;
  p.groups = c.span.B * c.span.T * c.Hkv * per;
  p.per_head = divisor((uint32_t)per);
  p.heads = divisor((uint32_t)c.Hkv);
  p.tokens = divisor((uint32_t)c.span.T);
  p.k_unit = power(-c.cache.k_exp); p.v_unit = power(-c.cache.v_exp);
  p.err = c.err;
  const int64_t grid = (2 * p.groups + kThreads - 1) / kThreads;
  return c.dtype == PFA_F32 ? launch(write_kernel<float>, grid, p, c.stream)
                            : launch(write_kernel<__nv_bfloat16>, grid, p, c.stream);
}

int launch_cache_read_q4(const ReadQ4Call& c) {
  ReadParams p;
  p.D = c.D;
  p.cap = c.cache.max_seq_len;
  p.k4 = (const uint8_t*)c.cache.k4; p.v4 = (const uint8_t*)c.cache.v4;
  p.k_scale = (const uint8_t*)c.cache.k_scale; p.v_scale = (const uint8_t*)c.cache.v_scale;
  p.out_head = c.out_head;
  p.k_unit = power(c.cache.k_exp); p.v_unit = power(c.cache.v_exp);
  const int per_row = c.D / (c.dtype == PFA_F32 ? 4 : 8);
  const int64_t most = ((int64_t)1 << 30) / per_row;   // rows of a launch: pieces count in 31 bits
  for (int64_t at = 0; at < c.rows; at += most) {
    const int64_t rows = std::min(most, c.rows - at), es = c.dtype == PFA_F32 ? 4 : 2;
    p.start = c.start + at;
    p.k_out = (char*)c.k_out + at * c.D * es;
    p.v_out = (char*)c.v_out + at * c.D * es;
    p.pieces = (int)(rows * per_row);
    const int64_t chunks = (p.pieces + kThreads * kPieces - 1) / (kThreads * kPieces);
    p.chunks = divisor((uint32_t)chunks);
    const int64_t grid = c.heads * chunks * 2;
    const int rc = c.dtype == PFA_F32 ? launch(read_kernel<float>, grid, p, c.stream)
                                      : launch(read_kernel<__nv_bfloat16>, grid, p, c.stream);
    if (rc != kOk) return rc;
  }
  return kOk;
}

}  // namespace pfa
