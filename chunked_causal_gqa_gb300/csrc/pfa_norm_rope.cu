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
//
// Bound by HBM's bytes, each element read and written once.  What costs beside them
// is the start: the first rows come after a launch and a DRAM latency, and the
// cosines (some 100 instructions a pair) are computed under that latency, once
// for all heads of a token.  Measured on GB300, one pass among others:
//   2048 tokens, 32/8 heads of 128, bf16 (42 MB)      10.1 us, 4.1 TB/s (floor 6.2 us)
//   1358 tokens, 8/2 heads of 512, fp32 (56 MB)       9.8 us, 5.7 TB/s (floor 8.2 us)
//   8 tokens, 32/8 heads of 128, bf16                 2.6 us: a launch and three latencies
// Tried: each lane's 16 elements contiguous (fp32 15.2 us: half of every 32-byte
// sector at a time); two rows ahead instead of one (11.0 / 11.4 us at 64 registers,
// 10.0 / 10.2 with three blocks an SM).
#include "pfa_internal.h"
#include "pfa_ptx.cuh"
#include "pfa_q8.cuh"

#include "../../include/pfa.h"

#include <algorithm>

namespace pfa {
namespace {

constexpr int kThreads = 256;
constexpr int kTableBytes = 32768;  // most of cosines and sines of a block's tokens

struct Side {               // the queries or the keys
  const void* in;
  void* out;
  const void* weight;
  int64_t in_row, out_row, out_head;
};
struct Params {
  Side q, k;
  const double* inv_freq;
  const int64_t* lengths;
  int64_t start_pos;
  Divisor heads, T;         // H + Hkv
  int H, rows, block_rows;  // tokens * heads; rows of a block
  int D, rot, interleaved;
  float eps, offset, inv_dim;   // 1 / D
  unsigned* err;
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

// Two floats in one register pair: one instruction for both.
struct F2 {
  float x, y;
};
__device__ __forceinline__ uint64_t bits(F2 a) {
  uint64_t v;
  asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(a.x), "f"(a.y));
  return v;
}
__device__ __forceinline__ F2 of_bits(uint64_t v) {
  F2 a;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a.x), "=f"(a.y) : "l"(v));
  return a;
}
__device__ __forceinline__ F2 mul(F2 a, F2 b) {
  uint64_t v;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(v) : "l"(bits(a)), "l"(bits(b)));
  return of_bits(v);
}
__device__ __forceinline__ F2 fma(F2 a, F2 b, F2 c) {
  uint64_t v;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(v) : "l"(bits(a)), "l"(bits(b)), "l"(bits(c)));
  return of_bits(v);
}

__device__ __forceinline__ float to_float(float x) { return x; }
__device__ __forceinline__ float to_float(__nv_bfloat16 x) { return __bfloat162float(x); }

// A lane's sixteen elements as they are stored: pieces of 16 bytes.
template <typename E>
struct Raw {
  static constexpr int V = 16 / sizeof(E), N = sizeof(E);   // elements of a piece, pieces
  uint4 w[N];
  __device__ __forceinline__ void load(const E* p, int stride) {
#pragma unroll
    for (int i = 0; i < N; ++i) w[i] = *reinterpret_cast<const uint4*>(p + i * stride);
  }
  __device__ __forceinline__ F2 pair(int i) const {   // elements 2 i and 2 i + 1
    const uint32_t* u = reinterpret_cast<const uint32_t*>(w);
    if (sizeof(E) == 4) return F2{__uint_as_float(u[2 * i]), __uint_as_float(u[2 * i + 1])};
    return F2{__uint_as_float(u[i] << 16), __uint_as_float(u[i] & 0xffff0000u)};
  }
};
__device__ __forceinline__ void store_pieces(float* p, int stride, const F2* y) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
    *reinterpret_cast<float4*>(p + i * stride) =
        make_float4(y[2 * i].x, y[2 * i].y, y[2 * i + 1].x, y[2 * i + 1].y);
}
__device__ __forceinline__ void store_pieces(__nv_bfloat16* p, int stride, const F2* y) {
  store8(p, reinterpret_cast<const float*>(y));
  store8(p + stride, reinterpret_cast<const float*>(y + 4));
}

// A block takes block_rows consecutive head rows (in the order of tokens, then query
// heads, then key heads), kThreads / width at a time, the next ones on their way.  `width`
// lanes, a power of two, share a row; a lane owns 16 elements, whose 16-byte pieces
// lie side by side with the other lanes'.  Of a head's rot / 16 lanes that rotate, lane l
// has the pieces l + m * rot / 16 of the first rot elements: for pairs (i, i + rot / 2) the
// second half of its pieces are the partners of the first.  A block's cosines are computed
// once for all heads of its tokens, while its first rows arrive.
// SHIFT: log2 of width where it is known (head_dim 128: 3, 512: 5), or -1.
// BATCH: positions come from lengths; a chunk's kernel is without their checks (2048 tokens, bf16,
// through Python: 10.2 us, 10.4 with them).
template <typename E, int SHIFT, bool NEIGHBOURS, bool BATCH>
__global__ void __launch_bounds__(kThreads, 4) norm_rope_kernel(const __grid_constant__ Params p) {
  extern __shared__ __align__(16) float smem[];
  float* gain = smem;                // weight + offset of q, then of k
  float* table = smem + 2 * p.D;
  asm volatile("griddepcontrol.launch_dependents;");
  constexpr int V = Raw<E>::V;
  const int lanes = SHIFT >= 0 ? 1 << SHIFT : p.D / 16, turned = p.rot / 16;
  const int shift = SHIFT >= 0 ? SHIFT : lanes <= 1 ? 0 : 32 - __clz(lanes - 1);
  const int lane = threadIdx.x & ((1 << shift) - 1);
  const int at = lane < turned ? V * lane : p.rot + V * (lane - turned);
  const int stride = V * (lane < turned ? turned : lanes - turned);
  const int row0 = blockIdx.x * p.block_rows;
  const int row_end = min(p.rows, row0 + p.block_rows);
  const int n0 = row0 / p.heads, tokens = (row_end - 1) / p.heads - n0 + 1;
  const int step = kThreads >> shift, mine = row0 + (threadIdx.x >> shift);
  const bool on = SHIFT >= 0 || lane < lanes;
  asm volatile("griddepcontrol.wait;" ::: "memory");

  Raw<E> next = {};
  auto load = [&](int row) {
    if (on && row < row_end) {
      const int n = row / p.heads, h = row - n * (int)p.heads.by;
      const E* src = h < p.H ? (const E*)p.q.in + n * p.q.in_row + h * p.D
                             : (const E*)p.k.in + n * p.k.in_row + (h - p.H) * p.D;
      next.load(src + at, stride);
    }
  };
  load(mine);
  auto position = [&](int n) -> int64_t {
    if (!BATCH) return p.start_pos + n;
    const int s = n / p.T;
    return p.lengths[s] - (int)p.T.by + (n - s * (int)p.T.by);
  };
  for (int i = threadIdx.x; i < 2 * p.D; i += kThreads) {
    const E* w = (const E*)(i < p.D ? p.q.weight : p.k.weight);
    gain[i] = w ? to_float(w[i < p.D ? i : i - p.D]) + p.offset : 1.f;
  }
  // a lane's pairs 2 i and 2 i + 1 at [i][lane]: {cos, cos, sin, sin}; a piece has `in` pairs
  constexpr int in = NEIGHBOURS ? V / 2 : V;
  const int pairs = p.rot / 2;
  if (pairs > 0) {   // a thread has one pair of every `apart`-th token
    const int apart = (int)((uint32_t)kThreads / (uint32_t)pairs);
    const int t0 = (int)((uint32_t)threadIdx.x / (uint32_t)pairs), pair = threadIdx.x - t0 * pairs;
    if (t0 < apart) {
      const uint64_t fraction = turn_fraction(p.inv_freq[pair]);
      const int piece = pair / in, m = (int)((uint32_t)piece / (uint32_t)turned);
      const int k = m * in + pair % in;
      float* to = table + ((k / 2) * turned + piece - m * turned) * 4 + k % 2;
      for (int t = t0; t < tokens; t += apart) {
        const uint64_t turn = fraction * (uint64_t)position(n0 + t);
        float sn, cs;
        sincospif((float)(int32_t)(turn >> 32) * 0x1p-31f, &sn, &cs);
        to[t * p.rot] = cs;
        to[t * p.rot + 2] = sn;
      }
    }
  }
  __syncthreads();
#pragma unroll 1
  for (int first = row0; first < row_end; first += step) {   // of the block's threads together
    const int row = first + (threadIdx.x >> shift);
    F2 y[8], sum = {0.f, 0.f};
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      y[j] = next.pair(j);
      sum = fma(y[j], y[j], sum);
    }
    load(row + step);
    float ss = sum.x + sum.y;
    if constexpr (SHIFT >= 0) {
#pragma unroll
      for (int o = (1 << SHIFT) >> 1; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    } else {
      for (int o = (1 << shift) >> 1; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    }
    if (on && row < row_end) {
      const int n = row / p.heads, h = row - n * (int)p.heads.by;
      const bool isq = h < p.H;
      if ((isq ? p.q.weight : p.k.weight) != nullptr) {
        const float r = rsqrtf(fmaf(ss, p.inv_dim, p.eps));
        const float4* g = reinterpret_cast<const float4*>(gain + (isq ? 0 : p.D) + at);
#pragma unroll
        for (int j = 0; j < 4; ++j) {   // four elements: V / 4 to a piece
          const float4 v = g[(j / (V / 4)) * (stride / 4) + j % (V / 4)];
          y[2 * j] = mul(mul(y[2 * j], F2{r, r}), F2{v.x, v.y});
          y[2 * j + 1] = mul(mul(y[2 * j + 1], F2{r, r}), F2{v.z, v.w});
        }
      }
      if (lane < turned) {
        const float4* cs = reinterpret_cast<const float4*>(table + (n - n0) * p.rot) + lane;
#pragma unroll
        for (int j = 0; j < 4; ++j) {   // pairs 2 j and 2 j + 1 of the lane
          const float4 t = cs[j * turned];
          const F2 c = {t.x, t.y}, s = {t.z, t.w}, ns = {-t.z, -t.w};
          if constexpr (NEIGHBOURS) {
            const F2 u = {y[2 * j].x, y[2 * j + 1].x}, v = {y[2 * j].y, y[2 * j + 1].y};
            const F2 re = fma(u, c, mul(v, ns)), im = fma(u, s, mul(v, c));
            y[2 * j] = {re.x, im.x};
            y[2 * j + 1] = {re.y, im.y};
          } else {
            const F2 u = y[j], v = y[j + 4];
            y[j] = fma(u, c, mul(v, ns));
            y[j + 4] = fma(u, s, mul(v, c));
          }
        }
      }
      if constexpr (BATCH) {
        const int s = n / p.T;
        const int64_t length = p.lengths[s];
        if (length < (s + 1) * (int64_t)p.T.by - n) {   // a negative position: padding in front
          if (length < 0) {
            if (h == 0 && lane == 0) atomicOr(p.err, kErrLengths);
            continue;
          }
#pragma unroll
          for (int j = 0; j < 8; ++j) y[j] = {0.f, 0.f};
        }
      }
      E* dst = isq ? (E*)p.q.out + n * p.q.out_row + h * p.D
                   : (E*)p.k.out + n * p.k.out_row + (h - p.H) * p.k.out_head;
      store_pieces(dst + at, stride, y);
    }
  }
}

template <typename E, int SHIFT, bool NEIGHBOURS>
cudaError_t launch(Params p, int num_sms, cudaStream_t stream) {
  int width = 1;
  while (width < p.D / 16) width *= 2;
  const int step = kThreads / width;
  // as many turns as bring all rows into one wave of four blocks an SM
  const int64_t turns = ((int64_t)p.rows + step - 1) / step, blocks = (int64_t)num_sms * 4;
  int64_t n = (turns + blocks - 1) / blocks * step;
  // the table holds the tokens that a block's rows can touch
  const int64_t heads = p.heads.by;
  if (p.rot > 0) n = std::min<int64_t>(n, (kTableBytes / (p.rot * (int64_t)sizeof(float)) - 1) * heads + 1);
  p.block_rows = (int)n;
  const int64_t tokens = (n - 1 + heads - 1) / heads + 1;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((p.rows + n - 1) / n));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = (size_t)(tokens * p.rot + 2 * p.D) * sizeof(float);
  cfg.stream = stream;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, p.lengths ? norm_rope_kernel<E, SHIFT, NEIGHBOURS, true>
                                            : norm_rope_kernel<E, SHIFT, NEIGHBOURS, false>,
                            (const Params)p);
}

template <typename E>
cudaError_t launch(const Params& p, int num_sms, cudaStream_t stream) {
  if (p.interleaved)
    return p.D == 128   ? launch<E, 3, true>(p, num_sms, stream)
           : p.D == 512 ? launch<E, 5, true>(p, num_sms, stream)
                        : launch<E, -1, true>(p, num_sms, stream);
  return p.D == 128   ? launch<E, 3, false>(p, num_sms, stream)
         : p.D == 512 ? launch<E, 5, false>(p, num_sms, stream)
                      : launch<E, -1, false>(p, num_sms, stream);
}

}  // namespace

int launch_norm_rope(const NormRopeCall& c) {
  const int64_t tokens = c.span.B * c.span.T, rows = tokens * (c.H + c.Hkv);
  if (rows > 0x7fffffff - (1 << 22)) return kErrShape;
  Params p;
  p.q = Side{c.q, c.q_out, c.q_weight, c.q_row, c.q_out_row, c.D};
  p.k = Side{c.k, c.k_out, c.k_weight, c.k_row, c.k_out_row, c.k_out_head};
  p.inv_freq = c.inv_freq;
  p.lengths = c.span.lengths;
  p.start_pos = c.span.start_pos;
  p.heads = divisor((uint32_t)(c.H + c.Hkv));
  p.T = divisor((uint32_t)c.span.T);
  p.H = c.H;
  p.rows = (int)rows;
  p.D = c.D;
  p.rot = c.rot_dim; p.interleaved = c.interleaved;
  p.eps = c.eps; p.offset = c.weight_offset; p.inv_dim = 1.f / (float)c.D;
  p.err = c.err;
  const cudaError_t e = c.dtype == PFA_F32 ? launch<float>(p, c.num_sms, c.stream)
                                           : launch<__nv_bfloat16>(p, c.num_sms, c.stream);
  if (e == cudaSuccess) return kOk;
  cudaGetLastError();
  return kErrLaunch;
}

}  // namespace pfa
