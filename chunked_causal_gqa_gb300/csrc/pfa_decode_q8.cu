// pfa_decode_q8.cu -- attention of few tokens of a batch of sequences over
// their 8-bit caches.
//
// One block per (sequence, token, query head): tiles of 128 keys, a thread
// scores one key, the block takes the tile's maximum and sum, then each thread
// accumulates its columns of P.V (running maximum and sum, fp32).
#include "pfa_internal.h"
#include "pfa_ptx.cuh"
#include "pfa_q8.cuh"

#include "../../include/pfa.h"

#include <cmath>
#include <cuda_fp8.h>

namespace pfa {
namespace {

constexpr int kThreads = 128;
constexpr int kMaxD = 512;

struct Params {
  const void* q;
  void* out;
  const uint8_t *k8, *v8;
  const float *k_scale, *v_scale;
  const int64_t* lengths;
  int64_t B, T, start_pos, cap, q_row, out_row;
  int H, Hkv, D, window, block;
  float scale_log2;
  unsigned* err;
};

__device__ __forceinline__ float get(const float* p) { return *p; }
__device__ __forceinline__ float get(const __nv_bfloat16* p) { return __bfloat162float(*p); }
__device__ __forceinline__ void put(float* p, float x) { *p = x; }
__device__ __forceinline__ void put(__nv_bfloat16* p, float x) { *p = __float2bfloat16_rn(x); }

template <typename E>
__global__ void __launch_bounds__(kThreads) decode_kernel(const Params p) {
  __shared__ float sq[kMaxD], sp[kThreads], sr[kThreads / 32], ss[kThreads];
  const int h = blockIdx.x % p.H;
  const int64_t bt = blockIdx.x / p.H, b = bt / p.T, t = bt % p.T;
  const int64_t end = p.lengths ? p.lengths[b] : p.start_pos + p.T;
  if (end < 0 || end > p.cap) {
    if (t == 0 && h == 0 && threadIdx.x == 0) atomicOr(p.err, kErrLengths);
    return;
  }
  const int64_t pos = end - p.T + t;
  const int64_t lo = p.window > 0 ? max((int64_t)0, pos - p.window + 1) : 0;
  const int64_t head = b * p.Hkv + h / (p.H / p.Hkv);
  const uint8_t* k8 = p.k8 + head * p.cap * p.D;
  const uint8_t* v8 = p.v8 + head * p.cap * p.D;
  const float* ks = p.k_scale + head * (p.cap / p.block);
  const float* vs = p.v_scale + head * (p.cap / p.block);
  const int tid = threadIdx.x;
  for (int d = tid; d < p.D; d += kThreads)
    sq[d] = get((const E*)p.q + bt * p.q_row + (int64_t)h * p.D + d);
  float o[kMaxD / kThreads] = {};
  float m = -INFINITY, l = 0.f;
  for (int64_t j0 = lo; j0 <= pos; j0 += kThreads) {
    __syncthreads();
    const int64_t j = j0 + tid;
    float s = -INFINITY;
    if (j <= pos) {
      float acc = 0.f;
      for (int d = 0; d < p.D; d += 4) {
        float x[4];
        e4m3x4_to_float(*reinterpret_cast<const uint32_t*>(k8 + j * p.D + d), x);
#pragma unroll
        for (int i = 0; i < 4; ++i) acc = fmaf(x[i], sq[d + i], acc);
      }
      s = acc * ks[j / p.block] * p.scale_log2;
    }
    float tm = s;
    for (int w = 16; w > 0; w >>= 1) tm = fmaxf(tm, __shfl_xor_sync(0xffffffffu, tm, w));
    if (tid % 32 == 0) sr[tid / 32] = tm;
    __syncthreads();
    float nm = m;
    for (int w = 0; w < kThreads / 32; ++w) nm = fmaxf(nm, sr[w]);
    const float base = nm == -INFINITY ? 0.f : nm;
    const float e = exp2f(s - base), alpha = exp2f(m - base);
    m = nm;
    l = l * alpha + e;
    sp[tid] = j <= pos ? e * vs[j / p.block] : 0.f;
    __syncthreads();
    const int n = (int)min((int64_t)kThreads, pos + 1 - j0);
    for (int c = 0; c * kThreads + tid < p.D; ++c) {
      const int d = c * kThreads + tid;
      float acc = o[c] * alpha;
      for (int i = 0; i < n; ++i) {
        const __half_raw r = __nv_cvt_fp8_to_halfraw(v8[(j0 + i) * p.D + d], __NV_E4M3);
        acc = fmaf(sp[i], __half2float(__half(r)), acc);
      }
      o[c] = acc;
    }
  }
  ss[tid] = l;
  __syncthreads();
  float sum = 0.f;
  for (int i = 0; i < kThreads; ++i) sum += ss[i];
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  for (int c = 0; c * kThreads + tid < p.D; ++c)
    put((E*)p.out + bt * p.out_row + (int64_t)h * p.D + c * kThreads + tid, o[c] * inv);
}

}  // namespace

size_t decode_q8_workspace(int64_t, int64_t, int, int, int, int, int) { return 0; }

int launch_decode_q8(const DecodeQ8Call& c) {
  Params p;
  p.q = c.q; p.out = c.out;
  p.k8 = (const uint8_t*)c.cache.k8; p.v8 = (const uint8_t*)c.cache.v8;
  p.k_scale = c.cache.k_scale; p.v_scale = c.cache.v_scale;
  p.lengths = c.span.lengths;
  p.B = c.span.B; p.T = c.span.T; p.start_pos = c.span.start_pos;
  p.cap = c.cache.max_seq_len; p.q_row = c.q_row; p.out_row = c.out_row;
  p.H = c.H; p.Hkv = c.Hkv; p.D = c.D; p.window = c.window; p.block = c.cache.block;
  p.scale_log2 = c.scale * 1.4426950408889634f;
  p.err = c.err;
  const int64_t grid = p.B * p.T * p.H;
  if (grid > 0x7fffffff) return kErrShape;
  if (c.dtype == PFA_F32)
    decode_kernel<float><<<(unsigned)grid, kThreads, 0, c.stream>>>(p);
  else
    decode_kernel<__nv_bfloat16><<<(unsigned)grid, kThreads, 0, c.stream>>>(p);
  return cudaGetLastError() == cudaSuccess ? kOk : kErrLaunch;
}

}  // namespace pfa
