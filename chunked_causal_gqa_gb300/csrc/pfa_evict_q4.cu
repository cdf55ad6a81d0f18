// pfa_evict_q4.cu -- cutting sequences of a 4-bit cache down to their newest and heaviest rows.
//
// For a sequence of n > keep rows, of each kv head: the `recent` newest rows stay, and the keep - recent
// largest of the others' weights (equal ones: the lower row).
//
// select_kernel, a block for each head: the key of a weight is its bits, turned so that unsigned order
// is the order of numbers.  Four passes over the candidates find the smallest key that
// is kept, eight bits at a time, from a histogram; a last pass lists the kept rows in
// order, counting equal keys, and moves their weights down.
//
// move_kernel, a block for each head and part of a row: kept rows move down in place.
// A row never moves up, so what is written in one round (rows 0 .. below the round's end) has no source
// left in a later one; a barrier stands between a round's reads and its writes.
#include "pfa_internal.h"
#include "pfa_ptx.cuh"
#include "pfa_q4.cuh"

namespace pfa {
namespace {

constexpr int kThreads = 512, kWarps = kThreads / 32;

struct Params {
  uint8_t* part[4];     // codes of K and V, scales of K and V
  int bytes[4];         // of a row
  float* weights;
  const int64_t* lengths;
  int64_t* lengths_out;
  int32_t* rows;
  int64_t cap;
  int keep, recent;
  int Hkv;
  unsigned* err;
};

// Unsigned order of the result is the order of the weights; NaN is the largest, -0 is 0.
__device__ __forceinline__ uint32_t key_of(float w) {
  const uint32_t u = __float_as_uint(w + 0.f);
  if (w != w) return 0xffffffffu;
  return u ^ (u >> 31 ? 0xffffffffu : 0x80000000u);
}

// Exclusive sum of x over the block's threads, and the total.
__device__ __forceinline__ int block_scan(int x, int* s_sum, int& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int up = x;
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, up, o);
    if (lane >= o) up += v;
  }
  __syncthreads();
  if (lane == 31) s_sum[warp] = up;
  __syncthreads();
  int before = up - x;
  total = 0;
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) before += s_sum[w];
    total += s_sum[w];
  }
  return before;
}

__global__ void __launch_bounds__(kThreads) select_kernel(const Params p) {
  __shared__ int hist[256];
  __shared__ int s_sum[kWarps];
  __shared__ uint32_t s_digit;
  __shared__ int s_left;
  asm volatile("griddepcontrol.launch_dependents;");
  const int64_t bh = blockIdx.x, b = bh / p.Hkv;
  const int tid = threadIdx.x;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int64_t len = p.lengths[b];
  const bool bad = len < 0 || len > p.cap;
  const int n = bad ? 0 : (int)len;
  int32_t* rows = p.rows + bh * p.keep;
  if (bad && tid == 0 && bh == b * p.Hkv) atomicOr(p.err, kErrLengths);
  if (n <= p.keep) {
    for (int i = tid; i < p.keep; i += kThreads) rows[i] = i < n ? i : -1;
    return;
  }
  float* w = p.weights + bh * p.cap;
  const int m = n - p.recent;          // candidates; more of them than places
  uint32_t key = 0, mask = 0;
  int left = p.keep - p.recent;        // of the candidates that agree with key so far
  for (int shift = 24; shift >= 0; shift -= 8) {
    for (int i = tid; i < 256; i += kThreads) hist[i] = 0;
    __syncthreads();
    for (int j = tid; j < m; j += kThreads) {
      const uint32_t k = key_of(w[j]);
      if ((k & mask) == key) atomicAdd(&hist[k >> shift & 255], 1);
    }
    __syncthreads();
    if (tid == 0) {
      int d = 255, rest = left;
      while (d > 0 && hist[d] < rest) rest -= hist[d--];
      s_digit = d;
      s_left = rest;
    }
    __syncthreads();
    key |= s_digit << shift;
    mask |= 255u << shift;
    left = s_left;
  }
  // left of the rows whose weight is the smallest kept one stay (none if nothing but the newest does)
  const bool any = p.keep > p.recent;
  int ties = 0, at = 0;
  for (int j0 = 0; j0 < n; j0 += kThreads) {
    const int j = j0 + tid;
    const float x = j < n ? w[j] : 0.f;
    const uint32_t k = key_of(x);
    const bool tie = j < m && any && k == key;
    int total;
    const int rank = ties + block_scan(tie, s_sum, total);
    ties += total;
    const bool kept = j < n && (j >= m || (any && k > key) || (tie && rank < left));
    const int to = at + block_scan(kept, s_sum, total);   // (its barriers: every w[j] has been read)
    at += total;
    if (kept) {
      rows[to] = j;
      w[to] = x;
    }
  }
  for (int j = p.keep + tid; j < n; j += kThreads) w[j] = 0.f;
}

__global__ void __launch_bounds__(kThreads) move_kernel(const Params p) {
  asm volatile("griddepcontrol.launch_dependents;");
  const int64_t bh = blockIdx.x >> 2, b = bh / p.Hkv;
  const int part = blockIdx.x & 3, tid = threadIdx.x;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (part == 0 && bh == b * p.Hkv && tid == 0) {
    const int64_t n = p.lengths[b];
    p.lengths_out[b] = n <= p.keep || n > p.cap ? n : p.keep;
  }
  const int32_t* rows = p.rows + bh * p.keep;
  if (rows[p.keep - 1] < p.keep) return;   // nothing moves
  const int width = part == 0 ? p.bytes[0] : part == 1 ? p.bytes[1] : part == 2 ? p.bytes[2] : p.bytes[3];
  uint8_t* base = (part == 0 ? p.part[0] : part == 1 ? p.part[1] : part == 2 ? p.part[2] : p.part[3]) +
                  bh * p.cap * width;
  const int64_t all = (int64_t)p.keep * width;
  for (int64_t e0 = 0; e0 < all; e0 += kThreads) {
    const int64_t e = e0 + tid;
    const int64_t r = e / width;
    uint8_t x = 0;
    if (e < all) x = base[(int64_t)rows[r] * width + (e - r * width)];
    __syncthreads();
    if (e < all) base[e] = x;
    __syncthreads();
  }
}

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

}  // namespace

int launch_cache_evict_q4(const EvictQ4Call& c) {
  Params p;
  p.part[0] = (uint8_t*)c.cache.k4; p.part[1] = (uint8_t*)c.cache.v4;
  p.part[2] = (uint8_t*)c.cache.k_scale; p.part[3] = (uint8_t*)c.cache.v_scale;
  p.bytes[0] = p.bytes[1] = c.D / 2;
  p.bytes[2] = p.bytes[3] = c.D / 16;
  p.weights = c.weights;
  p.lengths = c.lengths; p.lengths_out = c.lengths_out; p.rows = c.rows_out;
  p.cap = c.cache.max_seq_len;
  p.keep = (int)c.keep; p.recent = (int)c.recent;
  p.Hkv = c.Hkv;
  p.err = c.err;
  if (c.B * c.Hkv * 4 > 0x7fffffff) return kErrShape;
  const int rc = launch(select_kernel, c.B * c.Hkv, p, c.stream);
  return rc != kOk ? rc : launch(move_kernel, c.B * c.Hkv * 4, p, c.stream);
}

}  // namespace pfa
