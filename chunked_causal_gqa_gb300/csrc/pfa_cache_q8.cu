// pfa_cache_q8.cu -- writing tokens into the 8-bit cache and reading rows back.
//
// Write: for each head and block of `block` rows that the new rows touch,
//   s_old = the block's scale if it holds rows before the first new one, else 0
//   s_new = max(s_old, pow2_scale(max |x| over the block's new elements))
//   rows before the new ones: code <- e4m3(code * s_old / s_new)
//   new rows:                 code <- e4m3(x / s_new)
// Rows behind the last new one keep their codes.
//
// Both directions move bytes and nothing else.  Measured on GB300, one pass among others:
//   write 2048 tokens of 8 heads of 128, bf16 (12.6 MB)   4.8 us, 2.6 TB/s (floor 1.9 us:
//     a launch, the positions, the rows, a reduction and the codes follow one another)
//   write 1 token of 32 sequences, 8 heads of 128         2.6 us: the same chain
//   read 63488 rows of 8 heads of 128 as bf16 (390 MB)    57.9 us, 6.7 TB/s (floor 57.4 us)
//   read 3188 rows of 2 heads of 512 as fp32 (33 MB)      5.6 us, 5.8 TB/s (floor 4.8 us)
// A block of rows is read once: its elements wait in registers for the maximum (two
// passes over global memory took 8.5 us for the chunk).  Reading back, a lane makes 16
// output bytes at a time, so that both sides of a warp's pieces are contiguous (32
// bytes a lane: 66.0 and 9.3 us).
#include "pfa_internal.h"
#include "pfa_ptx.cuh"
#include "pfa_q8.cuh"

#include "../../include/pfa.h"

#include <algorithm>

namespace pfa {
namespace {

constexpr int kMaxThreads = 512;

struct WriteParams {
  const void *k, *v;
  uint8_t *k8, *v8;
  float *k_scale, *v_scale;
  const int64_t* lengths;
  int64_t T, start_pos, cap, k_row, v_row;
  Divisor touched, heads;  // blocks that T rows can reach; Hkv
  Divisor per_row;         // vectors of 8 elements in a row
  int D, block;
  unsigned* err;
};

// Eight elements as they are stored.
template <typename E>
struct Raw8 {
  uint4 w[sizeof(E) / 2];
  __device__ __forceinline__ void load(const E* p) {
#pragma unroll
    for (int i = 0; i < (int)sizeof(E) / 2; ++i) w[i] = reinterpret_cast<const uint4*>(p)[i];
  }
  __device__ __forceinline__ float get(int i) const {
    const uint32_t* u = reinterpret_cast<const uint32_t*>(w);
    if (sizeof(E) == 4) return __uint_as_float(u[i]);
    return __uint_as_float(i % 2 ? u[i / 2] & 0xffff0000u : u[i / 2] << 16);
  }
  __device__ __forceinline__ float amax() const {
    float a = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) a = fmaxf(a, finite_abs(get(i)));
    return a;
  }
  __device__ __forceinline__ uint2 codes(float f) const {
    return make_uint2(float_to_e4m3x4(get(0) * f, get(1) * f, get(2) * f, get(3) * f),
                      float_to_e4m3x4(get(4) * f, get(5) * f, get(6) * f, get(7) * f));
  }
};

// One block of threads for a block of rows of K or V of one head.  HELD vectors
// a thread stay in registers between the maximum and the codes, so that the new
// rows are read once (a block's elements beyond HELD * threads, which only
// 128 rows of wide heads have, are read again, from L2).
template <typename E, int HELD>
__global__ void __launch_bounds__(kMaxThreads) write_kernel(const WriteParams p) {
  __shared__ float s_max[kMaxThreads / 32];
  asm volatile("griddepcontrol.launch_dependents;");
  const int id = blockIdx.x / 2;
  const bool isv = blockIdx.x % 2;
  const int bh = id / p.touched, i = id - bh * (int)p.touched.by;
  const int64_t b = bh / p.heads;
  const int h = bh - (int)b * (int)p.heads.by;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int64_t end = p.lengths ? p.lengths[b] : p.start_pos + p.T;
  if (end < 0 || end > p.cap) {
    if (h == 0 && i == 0 && !isv && threadIdx.x == 0) atomicOr(p.err, kErrLengths);
    return;
  }
  const int first = (int)(end - p.T), low = max(first, 0);
  const int c = low / p.block + i, c0 = c * p.block;
  const int lo = max(low, c0), hi = min((int)end, c0 + p.block);
  if (lo >= hi) return;
  const int64_t row = isv ? p.v_row : p.k_row;
  const E* src = (isv ? (const E*)p.v : (const E*)p.k) + (b * p.T + lo - first) * row + (int64_t)h * p.D;
  uint8_t* dst = (isv ? p.v8 : p.k8) + ((int64_t)bh * p.cap + c0) * p.D;   // the block's rows
  float* scale = (isv ? p.v_scale : p.k_scale) + (int64_t)bh * (p.cap / p.block) + c;
  const int n = (hi - lo) * (int)p.per_row.by, old = (lo - c0) * (int)p.per_row.by;
  const int threads = blockDim.x, tid = threadIdx.x;
  auto at = [&](int e) {
    const int r = e / p.per_row;
    return src + r * row + (e - r * (int)p.per_row.by) * 8;
  };
  Raw8<E> x[HELD];
#pragma unroll
  for (int j = 0; j < HELD; ++j) {
    x[j] = {};
    if (tid + j * threads < n) x[j].load(at(tid + j * threads));
  }
  const float s_old = old > 0 ? *scale : 0.f;
  float amax = 0.f;
#pragma unroll
  for (int j = 0; j < HELD; ++j) amax = fmaxf(amax, x[j].amax());
#pragma unroll 1
  for (int e = tid + HELD * threads; e < n; e += threads) {
    Raw8<E> y;
    y.load(at(e));
    amax = fmaxf(amax, y.amax());
  }
  for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  if (threads > 32) {
    if (tid % 32 == 0) s_max[tid / 32] = amax;
    __syncthreads();
    for (int w = 0; w < threads / 32; ++w) amax = fmaxf(amax, s_max[w]);
  }
  const float s_new = fmaxf(s_old, pow2_scale(amax));
  const float inv = s_new > 0.f ? 1.f / s_new : 0.f;
  if (s_new != s_old) {
    if (tid == 0) *scale = s_new;   // every thread has read it: s_old went into s_new
    const float f = s_old * inv;
#pragma unroll 1
    for (int e = tid; e < old; e += threads) {
      uint2* const w = reinterpret_cast<uint2*>(dst + (int64_t)e * 8);
      const uint2 was = *w;
      float y[8];
      e4m3x4_to_float(was.x, y);
      e4m3x4_to_float(was.y, y + 4);
      *w = make_uint2(float_to_e4m3x4(y[0] * f, y[1] * f, y[2] * f, y[3] * f),
                      float_to_e4m3x4(y[4] * f, y[5] * f, y[6] * f, y[7] * f));
    }
  } else if (old == 0 && tid == 0) {
    *scale = s_new;                 // a new block of zeros
  }
  uint2* const to = reinterpret_cast<uint2*>(dst) + old;
#pragma unroll
  for (int j = 0; j < HELD; ++j)
    if (tid + j * threads < n) to[tid + j * threads] = x[j].codes(inv);
#pragma unroll 1
  for (int e = tid + HELD * threads; e < n; e += threads) {
    Raw8<E> y;
    y.load(at(e));
    to[e] = y.codes(inv);
  }
}

struct ReadParams {
  const uint8_t *k8, *v8;
  const float *k_scale, *v_scale;
  void *k_out, *v_out;
  int64_t start, cap, out_head;
  Divisor chunks;   // blocks of threads for a head's rows
  Divisor per_row;  // pieces of 16 output bytes in a row
  int pieces;       // of a head
  int D, block_shift;
};

// A thread makes kPieces pieces of 16 output bytes, all their codes asked for first.
constexpr int kReadThreads = 256, kPieces = 8;

template <typename E>
__global__ void __launch_bounds__(kReadThreads) read_kernel(const ReadParams p) {
  constexpr int N = 16 / sizeof(E);   // codes of a piece
  asm volatile("griddepcontrol.launch_dependents;");
  const int id = blockIdx.x / 2;
  const bool isv = blockIdx.x % 2;
  const int head = id / p.chunks, e0 = (id - head * (int)p.chunks.by) * (kReadThreads * kPieces);
  const uint8_t* src = (isv ? p.v8 : p.k8) + ((int64_t)head * p.cap + p.start) * p.D;
  const float* scale = (isv ? p.v_scale : p.k_scale) + (int64_t)head * (p.cap >> p.block_shift);
  E* out = (isv ? (E*)p.v_out : (E*)p.k_out) + (int64_t)head * p.out_head;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  uint32_t w[kPieces][N / 4];
  float s[kPieces];
#pragma unroll
  for (int i = 0; i < kPieces; ++i) {
    const int e = e0 + i * kReadThreads + threadIdx.x;
    if (e >= p.pieces) break;
    const int row = (int)p.start + e / p.per_row;
    const uint32_t* from = reinterpret_cast<const uint32_t*>(src + (int64_t)e * N);
    if constexpr (N == 8) {
      const uint2 v = *reinterpret_cast<const uint2*>(from);
      w[i][0] = v.x;
      w[i][1] = v.y;
    } else {
      w[i][0] = *from;
    }
    s[i] = scale[row >> p.block_shift];
  }
#pragma unroll
  for (int i = 0; i < kPieces; ++i) {
    const int e = e0 + i * kReadThreads + threadIdx.x;
    if (e >= p.pieces) break;
    float x[N];
#pragma unroll
    for (int j = 0; j < N / 4; ++j) e4m3x4_to_float(w[i][j], x + 4 * j);
#pragma unroll
    for (int j = 0; j < N; ++j) x[j] *= s[i];
    if constexpr (N == 8)
      store8(out + (int64_t)e * N, x);
    else
      *reinterpret_cast<float4*>(out + (int64_t)e * N) = make_float4(x[0], x[1], x[2], x[3]);
  }
}

int shift_of(int block) { return block == 16 ? 4 : block == 32 ? 5 : block == 64 ? 6 : 7; }

// A launch that may start before what is in front of it has ended (it waits on the device).
template <typename P>
int launch(void (*kernel)(const P), int64_t grid, int threads, const P& p, cudaStream_t stream) {
  if (grid > 0x7fffffff) return kErrShape;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3((unsigned)threads);
  cfg.stream = stream;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, kernel, p) == cudaSuccess) return kOk;
  cudaGetLastError();
  return kErrLaunch;
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
  p.D = c.D; p.block = c.cache.block;
  const int64_t touched = (p.T + p.block - 2) / p.block + 1;
  const int64_t grid = c.span.B * c.Hkv * touched * 2;
  if (grid > 0x7fffffff) return kErrShape;
  p.touched = divisor((uint32_t)touched);
  p.heads = divisor((uint32_t)c.Hkv);
  p.per_row = divisor((uint32_t)c.D / 8);
  p.err = c.err;
  // Threads for a block's rows at HELD vectors each; at least four warps, for
  // the rows of a block that a larger scale re-expresses.
  const bool f32 = c.dtype == PFA_F32;
  const int64_t vectors = std::min<int64_t>(p.T, p.block) * (c.D / 8), held = f32 ? 4 : 8;
  const int threads = (int)std::min<int64_t>(
      kMaxThreads, std::max<int64_t>(128, (vectors + held * 32 - 1) / (held * 32) * 32));
  if (vectors <= threads)   // decoding: one vector a thread, a third of the code to fetch
    return f32 ? launch(write_kernel<float, 1>, grid, threads, p, c.stream)
               : launch(write_kernel<__nv_bfloat16, 1>, grid, threads, p, c.stream);
  return f32 ? launch(write_kernel<float, 4>, grid, threads, p, c.stream)
             : launch(write_kernel<__nv_bfloat16, 8>, grid, threads, p, c.stream);
}

int launch_cache_read_q8(const ReadQ8Call& c) {
  ReadParams p;
  p.k8 = (const uint8_t*)c.cache.k8; p.v8 = (const uint8_t*)c.cache.v8;
  p.k_scale = c.cache.k_scale; p.v_scale = c.cache.v_scale;
  p.D = c.D; p.block_shift = shift_of(c.cache.block);
  p.cap = c.cache.max_seq_len;
  p.out_head = c.out_head;
  const int per_row = c.D / (c.dtype == PFA_F32 ? 4 : 8);
  p.per_row = divisor((uint32_t)per_row);
  // rows of a launch: pieces of a head count in 31 bits
  const int64_t most = (((int64_t)1 << 30) / per_row) & ~(int64_t)127;
  for (int64_t at = 0; at < c.rows; at += most) {
    const int64_t rows = std::min(most, c.rows - at), es = c.dtype == PFA_F32 ? 4 : 2;
    p.start = c.start + at;
    p.k_out = (char*)c.k_out + at * c.D * es;
    p.v_out = (char*)c.v_out + at * c.D * es;
    p.pieces = (int)(rows * per_row);
    const int64_t chunks = (p.pieces + kReadThreads * kPieces - 1) / (kReadThreads * kPieces);
    p.chunks = divisor((uint32_t)chunks);
    const int64_t grid = c.heads * chunks * 2;
    const int rc = c.dtype == PFA_F32
                       ? launch(read_kernel<float>, grid, kReadThreads, p, c.stream)
                       : launch(read_kernel<__nv_bfloat16>, grid, kReadThreads, p, c.stream);
    if (rc != kOk) return rc;
  }
  return kOk;
}

}  // namespace pfa
