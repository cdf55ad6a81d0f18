// pfa_norm_rope.cu -- RMS norm of every query and key head and the rotation
// of its position, one pass over the data.
//
//   y_d = x_d * rsqrt(mean_d x_d^2 + eps) * (w_d + offset)
//   (y_i, y_j) -> (y_i cos a - y_j sin a, y_i sin a + y_j cos a),  a = p * inv_freq_i
//
// with j = i + rot_dim / 2, or neighbouring pairs when interleaved.
//
// The angle is reduced in fixed point: inv_freq / 2 pi is held as a 64-bit
// fraction of a turn, so position times fraction, modulo 2^64, is the angle
// modulo one turn with an error of position * 2^-64 turns; only its top 32
// bits are then rounded to float.  (Doubles would do, but the chip runs two
// of their operations a clock and SM.)
#include "pfa_internal.h"
#include "pfa_q8.cuh"

#include "../../include/pfa.h"

namespace pfa {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxPairs = 256;  // rot_dim <= 512

struct Params {
  const void *q, *k;
  void *q_out, *k_out;
  const void *q_weight, *k_weight;
  const double* inv_freq;
  const int64_t* lengths;
  int64_t N, T, start_pos;
  int64_t q_row, k_row, q_out_row, k_out_row, k_out_head;
  int H, heads, D, rot, interleaved;  // heads = H + Hkv
  float eps, offset;
};

// f / (2 pi) modulo 1 as a 64-bit fraction, from the double's bits.
__device__ uint64_t turn_fraction(double f) {
  const uint64_t bits = (uint64_t)__double_as_longlong(f);
  const int ef = (int)((bits >> 52) & 0x7ff);
  const uint64_t m = (bits & 0xfffffffffffffull) | (ef ? 1ull << 52 : 0);
  // 1 / (2 pi) = c * 2^-66; f = m * 2^(e - 52)
  const uint64_t c = 0xa2f9836e4e44152aull;
  const uint64_t hi = __umul64hi(m, c), lo = m * c;
  const int sh = 54 - ((ef ? ef : 1) - 1023);  // fraction * 2^64 = (hi:lo) >> sh
  uint64_t r = 0;
  if (sh >= 128) r = 0;
  else if (sh >= 64) r = hi >> (sh - 64);
  else if (sh > 0) r = (lo >> sh) | (hi << (64 - sh));
  else if (sh > -64) r = lo << -sh;
  return (bits >> 63) ? 0 - r : r;
}

template <typename E>
__global__ void __launch_bounds__(kThreads) norm_rope_kernel(const Params p) {
  __shared__ float2 sCS[kMaxPairs];  // {cos, sin} of this token's pairs
  const int64_t n = blockIdx.x;
  const int64_t pos = p.lengths ? p.lengths[n / p.T] - p.T + n % p.T : p.start_pos + n;
  for (int i = threadIdx.x; i < p.rot / 2; i += kThreads) {
    const uint64_t turn = turn_fraction(p.inv_freq[i]) * (uint64_t)pos;
    float s, c;
    sincospif((float)(int32_t)(turn >> 32) * 0x1p-31f, &s, &c);
    sCS[i] = make_float2(c, s);
  }
  __syncthreads();
  // A lane owns two 8-element pieces of a head row: the two halves of eight
  // pairs, or sixteen neighbours.  `width` lanes (a power of two) share a row.
  const int pieces = p.D / 16, half = p.interleaved ? 0 : p.rot / 16;
  int width = 1;
  while (width < pieces) width *= 2;
  const int lane = threadIdx.x % width;
  for (int h0 = 0; h0 < p.heads; h0 += kThreads / width) {
    const int h = h0 + threadIdx.x / width;
    const bool on = h < p.heads && lane < pieces;
    const bool isq = h < p.H;
    const int a = lane < half ? 8 * lane : 16 * lane;
    const int b = lane < half ? a + 8 * half : a + 8;
    float x[16] = {};
    if (on) {
      const E* row = isq ? (const E*)p.q + n * p.q_row + (int64_t)h * p.D
                         : (const E*)p.k + n * p.k_row + (int64_t)(h - p.H) * p.D;
      load8(row + a, x);
      load8(row + b, x + 8);
    }
    const E* w = (const E*)(isq ? p.q_weight : p.k_weight);
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) ss = fmaf(x[i], x[i], ss);
    for (int o = width / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    if (!on) continue;
    if (w) {
      const float r = rsqrtf(ss / (float)p.D + p.eps);
      float g[16];
      load8(w + a, g);
      load8(w + b, g + 8);
#pragma unroll
      for (int i = 0; i < 16; ++i) x[i] = x[i] * r * (g[i] + p.offset);
    }
    if (p.interleaved) {
      if (a < p.rot) {
#pragma unroll
        for (int i = 0; i < 16; i += 2) {
          const float2 cs = sCS[a / 2 + i / 2];
          const float u = x[i], v = x[i + 1];
          x[i] = u * cs.x - v * cs.y;
          x[i + 1] = u * cs.y + v * cs.x;
        }
      }
    } else if (lane < half) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float2 cs = sCS[a + i];
        const float u = x[i], v = x[i + 8];
        x[i] = u * cs.x - v * cs.y;
        x[i + 8] = u * cs.y + v * cs.x;
      }
    }
    if (pos < 0) {  // padding in front of a short sequence
#pragma unroll
      for (int i = 0; i < 16; ++i) x[i] = 0.f;
    }
    E* o = isq ? (E*)p.q_out + n * p.q_out_row + (int64_t)h * p.D
               : (E*)p.k_out + n * p.k_out_row + (int64_t)(h - p.H) * p.k_out_head;
    store8(o + a, x);
    store8(o + b, x + 8);
  }
}

}  // namespace

int launch_norm_rope(const NormRopeCall& c) {
  Params p;
  p.q = c.q; p.k = c.k; p.q_out = c.q_out; p.k_out = c.k_out;
  p.q_weight = c.q_weight; p.k_weight = c.k_weight;
  p.inv_freq = c.inv_freq;
  p.lengths = c.span.lengths;
  p.N = c.span.B * c.span.T; p.T = c.span.T; p.start_pos = c.span.start_pos;
  p.q_row = c.q_row; p.k_row = c.k_row; p.q_out_row = c.q_out_row; p.k_out_row = c.k_out_row;
  p.k_out_head = c.k_out_head;
  p.H = c.H; p.heads = c.H + c.Hkv; p.D = c.D;
  p.rot = c.rot_dim; p.interleaved = c.interleaved;
  p.eps = c.eps; p.offset = c.weight_offset;
  if (c.dtype == PFA_F32)
    norm_rope_kernel<float><<<(unsigned)p.N, kThreads, 0, c.stream>>>(p);
  else
    norm_rope_kernel<__nv_bfloat16><<<(unsigned)p.N, kThreads, 0, c.stream>>>(p);
  return cudaGetLastError() == cudaSuccess ? kOk : kErrLaunch;
}

}  // namespace pfa
