// pfa_cache_q8.cu -- writing tokens into the 8-bit cache and reading rows back.
//
// Write: for each head and block of `block` rows that the new rows touch,
//   s_old = the block's scale if it holds rows before the first new one, else 0
//   s_new = max(s_old, pow2_scale(max |x| over the block's new elements))
//   rows before the new ones: code <- e4m3(code * s_old / s_new)
//   new rows:                 code <- e4m3(x / s_new)
// Rows behind the last new one keep their codes.
#include "pfa_internal.h"
#include "pfa_ptx.cuh"
#include "pfa_q8.cuh"

#include "../../include/pfa.h"

namespace pfa {
namespace {

constexpr int kThreads = 128;

struct WriteParams {
  const void *k, *v;
  uint8_t *k8, *v8;
  float *k_scale, *v_scale;
  const int64_t* lengths;
  int64_t T, start_pos, cap, k_row, v_row;
  int Hkv, D, block, touched;  // touched: blocks that T rows can reach
  unsigned* err;
};

template <typename E>
__global__ void __launch_bounds__(kThreads) write_kernel(const WriteParams p) {
  __shared__ float s_max[kThreads / 32];
  int64_t id = blockIdx.x;
  const bool isv = id % 2;
  id /= 2;
  const int i = (int)(id % p.touched);
  id /= p.touched;
  const int h = (int)(id % p.Hkv);
  const int64_t b = id / p.Hkv;
  const int64_t end = p.lengths ? p.lengths[b] : p.start_pos + p.T;
  if (end < 0 || end > p.cap) {
    if (h == 0 && i == 0 && !isv && threadIdx.x == 0) atomicOr(p.err, kErrLengths);
    return;
  }
  const int64_t first = end - p.T, low = first > 0 ? first : 0;
  const int64_t c = low / p.block + i;
  const int64_t lo = max(low, c * p.block), hi = min(end, (c + 1) * p.block);
  if (lo >= hi) return;
  const int64_t head = b * p.Hkv + h;
  const E* src = isv ? (const E*)p.v + b * p.T * p.v_row : (const E*)p.k + b * p.T * p.k_row;
  const int64_t row = isv ? p.v_row : p.k_row;
  src += (int64_t)h * p.D;
  uint8_t* dst = (isv ? p.v8 : p.k8) + head * p.cap * p.D;
  float* scale = (isv ? p.v_scale : p.k_scale) + head * (p.cap / p.block) + c;
  const int per_row = p.D / 8, n = (int)(hi - lo) * per_row;
  float amax = 0.f;
  for (int e = threadIdx.x; e < n; e += kThreads) {
    float x[8];
    load8(src + (lo - first + e / per_row) * row + e % per_row * 8, x);
#pragma unroll
    for (int j = 0; j < 8; ++j) amax = fmaxf(amax, finite_abs(x[j]));
  }
  for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  if (threadIdx.x % 32 == 0) s_max[threadIdx.x / 32] = amax;
  const int old_rows = (int)(lo - c * p.block);
  const float s_old = old_rows > 0 ? *scale : 0.f;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) amax = fmaxf(amax, s_max[w]);
  const float s_new = fmaxf(s_old, pow2_scale(amax));
  const float inv = s_new > 0.f ? 1.f / s_new : 0.f;
  if (threadIdx.x == 0) *scale = s_new;
  if (s_new != s_old) {
    const float f = s_old * inv;
    for (int e = threadIdx.x; e < old_rows * per_row; e += kThreads) {
      uint2* at = reinterpret_cast<uint2*>(dst + c * p.block * p.D + (int64_t)e * 8);
      const uint2 w = *at;
      float x[8];
      e4m3x4_to_float(w.x, x);
      e4m3x4_to_float(w.y, x + 4);
      *at = make_uint2(float_to_e4m3x4(x[0] * f, x[1] * f, x[2] * f, x[3] * f),
                       float_to_e4m3x4(x[4] * f, x[5] * f, x[6] * f, x[7] * f));
    }
  }
  for (int e = threadIdx.x; e < n; e += kThreads) {
    float x[8];
    load8(src + (lo - first + e / per_row) * row + e % per_row * 8, x);
    *reinterpret_cast<uint2*>(dst + lo * p.D + (int64_t)e * 8) =
        make_uint2(float_to_e4m3x4(x[0] * inv, x[1] * inv, x[2] * inv, x[3] * inv),
                   float_to_e4m3x4(x[4] * inv, x[5] * inv, x[6] * inv, x[7] * inv));
  }
}

struct ReadParams {
  const uint8_t *k8, *v8;
  const float *k_scale, *v_scale;
  void *k_out, *v_out;
  int64_t heads, start, rows, cap, out_head;
  int D, block;
};

template <typename E>
__global__ void __launch_bounds__(kThreads) read_kernel(const ReadParams p) {
  const int per_row = p.D / 16;
  const int64_t n = p.heads * p.rows * per_row;
  for (int64_t e = blockIdx.x * (int64_t)kThreads + threadIdx.x; e < 2 * n;
       e += (int64_t)gridDim.x * kThreads) {
    const bool isv = e >= n;
    const int64_t at = isv ? e - n : e;
    const int64_t r = at / per_row, head = r / p.rows, row = p.start + r % p.rows;
    const int64_t d = at % per_row * 16;
    const uint4 w = *reinterpret_cast<const uint4*>((isv ? p.v8 : p.k8) +
                                                    (head * p.cap + row) * p.D + d);
    const float s = (isv ? p.v_scale : p.k_scale)[head * (p.cap / p.block) + row / p.block];
    float x[16];
    e4m3x4_to_float(w.x, x);
    e4m3x4_to_float(w.y, x + 4);
    e4m3x4_to_float(w.z, x + 8);
    e4m3x4_to_float(w.w, x + 12);
#pragma unroll
    for (int i = 0; i < 16; ++i) x[i] *= s;
    E* o = (E*)(isv ? p.v_out : p.k_out) + head * p.out_head + (row - p.start) * p.D + d;
    store8(o, x);
    store8(o + 8, x + 8);
  }
}

}  // namespace

int launch_cache_write_q8(const WriteQ8Call& c) {
  WriteParams p;
  p.k = c.k; p.v = c.v;
  p.k8 = (uint8_t*)c.cache.k8; p.v8 = (uint8_t*)c.cache.v8;
  p.k_scale = c.cache.k_scale; p.v_scale = c.cache.v_scale;
  p.lengths = c.span.lengths;
  p.T = c.span.T; p.start_pos = c.span.start_pos;
  p.cap = c.cache.max_seq_len; p.k_row = c.k_row; p.v_row = c.v_row;
  p.Hkv = c.Hkv; p.D = c.D; p.block = c.cache.block;
  p.touched = (int)((p.T + p.block - 2) / p.block + 1);
  p.err = c.err;
  const int64_t grid = c.span.B * c.Hkv * p.touched * 2;
  if (grid > 0x7fffffff) return kErrShape;
  if (c.dtype == PFA_F32)
    write_kernel<float><<<(unsigned)grid, kThreads, 0, c.stream>>>(p);
  else
    write_kernel<__nv_bfloat16><<<(unsigned)grid, kThreads, 0, c.stream>>>(p);
  return cudaGetLastError() == cudaSuccess ? kOk : kErrLaunch;
}

int launch_cache_read_q8(const ReadQ8Call& c) {
  ReadParams p;
  p.k8 = (const uint8_t*)c.cache.k8; p.v8 = (const uint8_t*)c.cache.v8;
  p.k_scale = c.cache.k_scale; p.v_scale = c.cache.v_scale;
  p.k_out = c.k_out; p.v_out = c.v_out;
  p.heads = c.heads; p.start = c.start; p.rows = c.rows; p.cap = c.cache.max_seq_len;
  p.out_head = c.out_head;
  p.D = c.D; p.block = c.cache.block;
  const int64_t n = 2 * p.heads * p.rows * (p.D / 16);
  const int64_t want = (n + kThreads - 1) / kThreads, most = (int64_t)c.num_sms * 64;
  const unsigned grid = (unsigned)(want < most ? want : most);
  if (c.dtype == PFA_F32)
    read_kernel<float><<<grid, kThreads, 0, c.stream>>>(p);
  else
    read_kernel<__nv_bfloat16><<<grid, kThreads, 0, c.stream>>>(p);
  return cudaGetLastError() == cudaSuccess ? kOk : kErrLaunch;
}

}  // namespace pfa
