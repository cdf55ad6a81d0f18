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

#include <algorithm>

namespace pfa {
namespace {

constexpr int kThreads = 256;
constexpr int kTableBytes = 32768;  // cosines and sines of a block's tokens

struct Params {
  const void *q, *k;
  void *q_out, *k_out;
  const void *q_weight, *k_weight;
  const double* inv_freq;
  const int64_t* lengths;
  int64_t start_pos;
  int64_t q_row, k_row, q_out_row, k_out_row, k_out_head;
  Divisor heads, T;        // H + Hkv
  int rows;                // tokens * heads
  int H, D, rot, interleaved, block_rows;
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

// Sixteen elements as they are stored.
template <typename E>
struct Raw {
  uint4 w[sizeof(E)];
  __device__ __forceinline__ void load(const E* a, const E* b) {
    constexpr int N = sizeof(E) / 2, V = 16 / sizeof(E);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      w[i] = *reinterpret_cast<const uint4*>(a + i * V);
      w[N + i] = *reinterpret_cast<const uint4*>(b + i * V);
    }
  }
  __device__ __forceinline__ float get(int i) const {
    const uint32_t* u = reinterpret_cast<const uint32_t*>(w);
    if (sizeof(E) == 4) return __uint_as_float(u[i]);
    return __uint_as_float(i % 2 ? u[i / 2] & 0xffff0000u : u[i / 2] << 16);
  }
};

// A block takes block_rows = ROWS * kThreads / width consecutive head rows (in the
// order of tokens, then query heads, then key heads).  `width` lanes, a power of two,
// share a row; a lane owns two pieces of 8 elements, the two halves of eight
// pairs or sixteen neighbours.  All of a block's rows are asked for before the
// cosines of its tokens are computed, once for all heads.
template <typename E, int ROWS>
__global__ void __launch_bounds__(kThreads) norm_rope_kernel(const Params p) {
  __shared__ __align__(16) float2 table[kTableBytes / sizeof(float2)];
  asm volatile("griddepcontrol.launch_dependents;");
  const int pieces = p.D / 16, half = p.interleaved ? 0 : p.rot / 16, turned = p.rot / 16;
  const int shift = pieces <= 1 ? 0 : 32 - __clz(pieces - 1);   // width = 1 << shift
  const int lane = threadIdx.x & ((1 << shift) - 1);
  const int a = lane < half ? 8 * lane : 16 * lane;
  const int b = lane < half ? a + 8 * half : a + 8;
  const int row0 = blockIdx.x * p.block_rows;
  const int row_end = min(p.rows, row0 + p.block_rows);
  const int n0 = row0 / p.heads, tokens = (row_end - 1) / p.heads - n0 + 1;
  asm volatile("griddepcontrol.wait;" ::: "memory");

  Raw<E> x[ROWS], wq, wk;
#pragma unroll
  for (int i = 0; i < ROWS; ++i) {
    const int row = row0 + i * (kThreads >> shift) + (threadIdx.x >> shift);
    if (row < row_end && lane < pieces) {
      const int n = row / p.heads, h = row - n * (int)p.heads.by;
      const E* src = h < p.H ? (const E*)p.q + n * p.q_row + h * p.D
                             : (const E*)p.k + n * p.k_row + (h - p.H) * p.D;
      x[i].load(src + a, src + b);
    } else {
      x[i] = {};
    }
  }
  if (lane < pieces) {
    if (p.q_weight) wq.load((const E*)p.q_weight + a, (const E*)p.q_weight + b);
    if (p.k_weight) wk.load((const E*)p.k_weight + a, (const E*)p.k_weight + b);
  }
  // pair 8 l + i of a token at [i / 2][l][i % 2]: the lanes of a row read side by side
  for (int j = threadIdx.x; j < tokens * (p.rot / 2); j += kThreads) {
    const int t = (uint32_t)j / (uint32_t)(p.rot / 2), pair = j - t * (p.rot / 2), n = n0 + t;
    const int s = n / p.T;
    const int64_t pos = p.lengths ? p.lengths[s] - (int)p.T.by + (n - s * (int)p.T.by)
                                  : p.start_pos + n;
    const uint64_t turn = turn_fraction(p.inv_freq[pair]) * (uint64_t)pos;
    float sn, cs;
    sincospif((float)(int32_t)(turn >> 32) * 0x1p-31f, &sn, &cs);
    table[t * (p.rot / 2) + ((pair % 8 / 2) * turned + pair / 8) * 2 + pair % 2] =
        make_float2(cs, sn);
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < ROWS; ++i) {
    const int row = row0 + i * (kThreads >> shift) + (threadIdx.x >> shift);
    float ss = 0.f;
#pragma unroll
    for (int j = 0; j < 16; ++j) ss = fmaf(x[i].get(j), x[i].get(j), ss);
    for (int o = (1 << shift) >> 1; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    if (row >= row_end || lane >= pieces) continue;
    const int n = row / p.heads, h = row - n * (int)p.heads.by;
    const bool isq = h < p.H;
    float y[16];
    if (isq ? p.q_weight != nullptr : p.k_weight != nullptr) {
      const float r = rsqrtf(ss / (float)p.D + p.eps);
#pragma unroll
      for (int j = 0; j < 16; ++j)
        y[j] = x[i].get(j) * r * ((isq ? wq.get(j) : wk.get(j)) + p.offset);
    } else {
#pragma unroll
      for (int j = 0; j < 16; ++j) y[j] = x[i].get(j);
    }
    if (lane < turned) {
      const float4* cs = reinterpret_cast<const float4*>(table + (n - n0) * (p.rot / 2)) + lane;
#pragma unroll
      for (int j = 0; j < 4; ++j) {   // pairs 2 j and 2 j + 1 of the lane
        const float4 c = cs[j * turned];
        if (p.interleaved) {
          const float u0 = y[4 * j], v0 = y[4 * j + 1], u1 = y[4 * j + 2], v1 = y[4 * j + 3];
          y[4 * j] = u0 * c.x - v0 * c.y;
          y[4 * j + 1] = u0 * c.y + v0 * c.x;
          y[4 * j + 2] = u1 * c.z - v1 * c.w;
          y[4 * j + 3] = u1 * c.w + v1 * c.z;
        } else {
          const float u0 = y[2 * j], v0 = y[2 * j + 8], u1 = y[2 * j + 1], v1 = y[2 * j + 9];
          y[2 * j] = u0 * c.x - v0 * c.y;
          y[2 * j + 8] = u0 * c.y + v0 * c.x;
          y[2 * j + 1] = u1 * c.z - v1 * c.w;
          y[2 * j + 9] = u1 * c.w + v1 * c.z;
        }
      }
    }
    if (p.lengths) {
      const int s = n / p.T;
      if (p.lengths[s] - (int)p.T.by + (n - s * (int)p.T.by) < 0) {  // padding in front
#pragma unroll
        for (int j = 0; j < 16; ++j) y[j] = 0.f;
      }
    }
    E* o = isq ? (E*)p.q_out + n * p.q_out_row + h * p.D
               : (E*)p.k_out + n * p.k_out_row + (h - p.H) * p.k_out_head;
    store8(o + a, y);
    store8(o + b, y + 8);
  }
}

template <typename E, int ROWS>
cudaError_t launch(Params p, int width, cudaStream_t stream) {
  p.block_rows = ROWS * kThreads / width;
  // the table holds the tokens that a block's rows can touch
  if (p.rot > 0) {
    const int most = kTableBytes / (p.rot / 2 * (int)sizeof(float2));
    p.block_rows = std::min<int64_t>(p.block_rows, (int64_t)(most - 1) * p.heads.by + 1);
  }
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((p.rows + p.block_rows - 1) / p.block_rows));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, norm_rope_kernel<E, ROWS>, (const Params)p);
}

}  // namespace

int launch_norm_rope(const NormRopeCall& c) {
  const int64_t tokens = c.span.B * c.span.T, rows = tokens * (c.H + c.Hkv);
  if (rows > 0x7fffffff - 65536) return kErrShape;
  Params p;
  p.q = c.q; p.k = c.k; p.q_out = c.q_out; p.k_out = c.k_out;
  p.q_weight = c.q_weight; p.k_weight = c.k_weight;
  p.inv_freq = c.inv_freq;
  p.lengths = c.span.lengths;
  p.start_pos = c.span.start_pos;
  p.q_row = c.q_row; p.k_row = c.k_row; p.q_out_row = c.q_out_row; p.k_out_row = c.k_out_row;
  p.k_out_head = c.k_out_head;
  p.heads = divisor(c.H + c.Hkv);
  p.T = divisor((uint32_t)c.span.T);
  p.rows = (int)rows;
  p.H = c.H; p.D = c.D;
  p.rot = c.rot_dim; p.interleaved = c.interleaved;
  p.eps = c.eps; p.offset = c.weight_offset;
  int width = 1;
  while (width < c.D / 16) width *= 2;
  // Few rows: one to a lane group, for the shortest chain; many: several in flight.
  const bool few = rows * width <= (int64_t)c.num_sms * kThreads * 4;
  cudaError_t e;
  if (c.dtype == PFA_F32)
    e = few ? launch<float, 1>(p, width, c.stream) : launch<float, 2>(p, width, c.stream);
  else
    e = few ? launch<__nv_bfloat16, 1>(p, width, c.stream) : launch<__nv_bfloat16, 4>(p, width, c.stream);
  if (e == cudaSuccess) return kOk;
  cudaGetLastError();
  return kErrLaunch;
}

}  // namespace pfa
