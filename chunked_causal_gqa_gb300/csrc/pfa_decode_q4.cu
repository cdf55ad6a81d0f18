// pfa_decode_q4.cu -- attention of few tokens of a batch of sequences over their 4-bit caches.
//
// For each sequence, token and query head
//   s_j = scale * <q, k_j>,  out = sum_j 2^(s_j log2 e - m) v_j / sum_j 2^(s_j log2 e - m)
// with the running maximum m, the sum and the output in fp32, and, where the caller keeps the
// keys' weights, weights[j] += the sum of 2^(s_j log2 e - m) / l over the tokens and heads of the kv head.
#include "pfa_internal.h"
#include "pfa_ptx.cuh"
#include "pfa_q4.cuh"

#include "../../include/pfa.h"

#include <algorithm>
#include <cmath>

namespace pfa {
namespace {

constexpr int kWarps = 4, kThreads = kWarps * 32;

struct Params {
  const void* q;
  void* out;
  float* weights;
  float2* sums;               // workspace: {m, l} of each row
  const uint8_t *k4, *v4, *k_scale, *v_scale;
  const int64_t* lengths;
  int64_t T, start_pos, q_row, out_row, cap;
  int Hkv, group, rows, window;
  float scale_log2, v_unit;
  unsigned* err;
};

struct Row {
  int64_t b;
  int h, r, t, lo, hi;     // keys [lo, hi] are seen
};
__device__ __forceinline__ bool row_of(const Params& p, int64_t bh, int r, Row& x) {
  x.b = bh / p.Hkv;
  x.h = (int)(bh - x.b * p.Hkv);
  x.r = r;
  x.t = r / p.group;
  const int64_t end = p.lengths ? p.lengths[x.b] : p.start_pos + p.T;
  if (end < 0 || end > p.cap) return false;
  x.hi = (int)(end - p.T) + x.t;
  x.lo = p.window > 0 ? max(0, x.hi - p.window + 1) : 0;
  return true;
}

template <typename E>
__device__ __forceinline__ float load(const E* p) {
  if constexpr (sizeof(E) == 4) return *p;
  else return __bfloat162float(*p);
}

// N consecutive values of a row.
template <int N>
__device__ __forceinline__ void values(const uint8_t* codes, const uint8_t* scales, int64_t row, int D, int d,
                                       float* x) {
  const float f = e4m3_to_float(scales[row * (D / 16) + d / 16]);
#pragma unroll
  for (int i = 0; i < N / 4; ++i) {
    const uint32_t w = *reinterpret_cast<const uint16_t*>(codes + row * (D / 2) + d / 2 + 2 * i);
    const uint32_t a = e2m1x2_to_half<0>(w), b = e2m1x2_to_half<1>(w);
    const float2 u = __half22float2(*reinterpret_cast<const __half2*>(&a));
    const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&b));
    x[4 * i] = u.x * f; x[4 * i + 1] = u.y * f; x[4 * i + 2] = v.x * f; x[4 * i + 3] = v.y * f;
  }
}

template <int N>
__device__ __forceinline__ float score(const float* q, const float* k) {
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < N; ++i) s = fmaf(q[i], k[i], s);
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  return s;
}

// A block for each row of queries: four warps take its keys in turn, a lane has D / 32 channels.
template <typename E, int D>
__global__ void __launch_bounds__(kThreads) decode_kernel(const Params p) {
  constexpr int N = D / 32;
  __shared__ float s_o[kWarps][D];
  __shared__ float2 s_ml[kWarps];
  asm volatile("griddepcontrol.launch_dependents;");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int64_t bh = blockIdx.x / p.rows;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, d = lane * N;
  Row x;
  if (!row_of(p, bh, (int)(blockIdx.x - bh * p.rows), x)) {
    if (threadIdx.x == 0) atomicOr(p.err, kErrLengths);
    return;
  }
  const int64_t head = (int64_t)x.h * p.group + x.r - x.t * p.group;
  const E* qr = (const E*)p.q + (x.b * p.T + x.t) * p.q_row + head * D + d;
  float q[N], o[N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    q[i] = load(qr + i) * p.scale_log2;
    o[i] = 0.f;
  }
  float m = -INFINITY, l = 0.f;
  for (int j = x.lo + warp; j <= x.hi; j += kWarps) {
    float k[N], v[N];
    values<N>(p.k4, p.k_scale, bh * p.cap + j, D, d, k);
    values<N>(p.v4, p.v_scale, bh * p.cap + j, D, d, v);
    const float s = score<N>(q, k), to = fmaxf(m, s);
    const float base = to == -INFINITY ? 0.f : to;
    const float a = exp2f(m - base), e = exp2f(s - base);
    m = to;
    l = l * a + e;
#pragma unroll
    for (int i = 0; i < N; ++i) o[i] = o[i] * a + e * v[i];
  }
#pragma unroll
  for (int i = 0; i < N; ++i) s_o[warp][d + i] = o[i];
  if (lane == 0) s_ml[warp] = make_float2(m, l);
  __syncthreads();
  m = -INFINITY;
  l = 0.f;
  for (int w = 0; w < kWarps; ++w) m = fmaxf(m, s_ml[w].x);
  const float base = m == -INFINITY ? 0.f : m;
  for (int w = 0; w < kWarps; ++w) l += s_ml[w].y * exp2f(s_ml[w].x - base);
  const float inv = l == 0.f ? 0.f : p.v_unit / l;
  E* to = (E*)p.out + (x.b * p.T + x.t) * p.out_row + head * D;
  for (int i = threadIdx.x; i < D; i += kThreads) {
    float sum = 0.f;
    for (int w = 0; w < kWarps; ++w) sum += s_o[w][i] * exp2f(s_ml[w].x - base);
    to[i] = (E)(sum * inv);
  }
  if (p.weights && threadIdx.x == 0) p.sums[bh * p.rows + x.r] = make_float2(base, l);
}

// A warp for each key of a head: the scores again, their weights added up over the rows.
template <typename E, int D>
__global__ void __launch_bounds__(kThreads) weights_kernel(const Params p, int chunks) {
  constexpr int N = D / 32;
  asm volatile("griddepcontrol.launch_dependents;");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int64_t bh = blockIdx.x / chunks;
  const int lane = threadIdx.x & 31, d = lane * N;
  const int first = (int)(blockIdx.x - bh * chunks) * kWarps + (threadIdx.x >> 5);
  Row x;
  if (!row_of(p, bh, 0, x)) return;
  Row last;
  row_of(p, bh, p.rows - 1, last);
  for (int j = x.lo + first; j <= last.hi; j += chunks * kWarps) {
    float k[N], sum = 0.f;
    values<N>(p.k4, p.k_scale, bh * p.cap + j, D, d, k);
    for (int r = 0; r < p.rows; ++r) {
      row_of(p, bh, r, x);
      if (j < x.lo || j > x.hi) continue;
      const E* qr = (const E*)p.q + (x.b * p.T + x.t) * p.q_row + ((int64_t)x.h * p.group + r - x.t * p.group) * D + d;
      float q[N];
#pragma unroll
      for (int i = 0; i < N; ++i) q[i] = load(qr + i) * p.scale_log2;
      const float2 ml = p.sums[bh * p.rows + r];
      sum += exp2f(score<N>(q, k) - ml.x) / ml.y;
    }
    if (lane == 0) p.weights[bh * p.cap + j] += sum;
  }
}

template <typename E, int D>
int launch(const Params& p, int64_t heads, cudaStream_t stream) {
  if (heads * p.rows > 0x7fffffff) return kErrShape;
  decode_kernel<E, D><<<(unsigned)(heads * p.rows), kThreads, 0, stream>>>(p);
  if (cudaGetLastError() != cudaSuccess) return kErrLaunch;
  if (!p.weights) return kOk;
  const int chunks = (int)std::min<int64_t>((p.cap + kWarps - 1) / kWarps, 0x7fffffff / heads);
  weights_kernel<E, D><<<(unsigned)(heads * chunks), kThreads, 0, stream>>>(p, chunks);
  return cudaGetLastError() == cudaSuccess ? kOk : kErrLaunch;
}

}  // namespace

size_t decode_q4_workspace(int64_t B, int64_t T, int H, int Hkv, int D, int dtype, int64_t cap,
                           bool weights, int num_sms) {
  return weights ? ((size_t)B * T * H * sizeof(float2) + 255) & ~(size_t)255 : 0;
}

int launch_decode_q4(const DecodeQ4Call& c) {
  Params p;
  p.q = c.q; p.out = c.out; p.weights = c.weights; p.sums = (float2*)c.ws;
  p.k4 = (const uint8_t*)c.cache.k4; p.v4 = (const uint8_t*)c.cache.v4;
  p.k_scale = (const uint8_t*)c.cache.k_scale; p.v_scale = (const uint8_t*)c.cache.v_scale;
  p.lengths = c.span.lengths;
  p.T = c.span.T; p.start_pos = c.span.start_pos;
  p.q_row = c.q_row; p.out_row = c.out_row;
  p.cap = c.cache.max_seq_len;
  p.Hkv = c.Hkv; p.group = c.H / c.Hkv; p.window = c.window;
  if (p.T * p.group > (1 << 30)) return kErrShape;
  p.rows = (int)p.T * p.group;
  p.scale_log2 = std::ldexp(c.scale * 1.4426950408889634f, c.cache.k_exp);
  p.v_unit = std::ldexp(1.f, c.cache.v_exp);
  p.err = c.err;
  const int64_t heads = c.span.B * c.Hkv;
  if (c.dtype == PFA_BF16)
    return c.D == 128 ? launch<__nv_bfloat16, 128>(p, heads, c.stream)
                      : launch<__nv_bfloat16, 512>(p, heads, c.stream);
  return c.D == 128 ? launch<float, 128>(p, heads, c.stream) : launch<float, 512>(p, heads, c.stream);
}

}  // namespace pfa
