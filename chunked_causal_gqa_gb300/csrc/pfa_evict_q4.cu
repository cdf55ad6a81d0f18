// pfa_evict_q4.cu -- cutting sequences of a 4-bit cache down to their newest and heaviest rows.
//
// For a sequence of n > keep rows, of each kv head: the `recent` newest rows stay, and the keep - recent
// largest of the others' weights (equal ones: the lower row).
//
// select_kernel, a cluster of up to eight blocks for each head, each with a run of its rows in registers:
// the key of a weight is its bits, turned so that unsigned order is the order of
// numbers.  Three passes over the candidates find the smallest key that is kept, 11, 11 and 10 bits at
// a time, from histograms that the blocks add up over distributed shared memory; then the kept rows
// are listed in order, each warp counting the kept rows in front of its own.
//
// Weights move and become zero there too: every block has read its own by then.
//
// move_kernel, a cluster for each head and array: kept rows move down in place.  A row never moves
// up, so what a round writes (rows 0 .. below its end) is no source of a later one; in a
// round, which takes up to half a megabyte, the cluster's barrier stands between the reads and the
// writes.
#include "pfa_internal.h"
#include "pfa_ptx.cuh"
#include "pfa_q4.cuh"

#include <algorithm>

namespace pfa {
namespace {

constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kBins = 4 * kThreads;
constexpr int kPieces = 8;       // of a thread in a round
constexpr int kMaxCluster = 8;

struct Params {
  uint8_t* part[4];     // codes of K and V, scales of K and V
  float* weights;
  const int64_t* lengths;
  int64_t* lengths_out;
  int32_t* rows;
  int64_t cap;
  int keep, recent;
  int Hkv, heads;       // of a sequence, in all
  int code_bytes, scale_bytes;   // of a row
  Divisor code_pieces, scale_pieces, one;   // of a row
  unsigned* err;
};

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}
// All threads of all blocks of the cluster; memory accesses before it come before those behind it.
__device__ __forceinline__ void cluster_barrier() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// Words of block `rank`'s shared memory.
__device__ __forceinline__ uint32_t remote_address(const void* p, uint32_t rank) {
  uint32_t a;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
  return a;
}
__device__ __forceinline__ int4 remote4(const int* p, uint32_t rank) {
  int4 v;
  asm volatile("ld.shared::cluster.v4.s32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(remote_address(p, rank)));
  return v;
}
__device__ __forceinline__ int2 remote2(const int* p, uint32_t rank) {
  int2 v;
  asm volatile("ld.shared::cluster.v2.s32 {%0, %1}, [%2];"
               : "=r"(v.x), "=r"(v.y) : "r"(remote_address(p, rank)));
  return v;
}

// Unsigned order of the result is the order of the weights; NaN is the largest, -0 is 0.
__device__ __forceinline__ uint32_t key_of(float w) {
  const uint32_t u = __float_as_uint(w + 0.f);
  if (w != w) return 0xffffffffu;
  return u ^ (u >> 31 ? 0xffffffffu : 0x80000000u);
}

__device__ __forceinline__ float weight_of(uint32_t key) {   // (a NaN, but not which; 0 for -0)
  return __uint_as_float(key ^ (key >> 31 ? 0x80000000u : 0xffffffffu));
}

__device__ __forceinline__ int warp_scan(int x) {   // inclusive
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += v;
  }
  return x;
}

// Rows `rows` of width.by pieces move to 0 .. keep - 1, in place.  `rank` of `size` blocks; barrier(): theirs.
template <typename T, typename B>
__device__ __forceinline__ void move_rows(T* base, const int32_t* rows, int keep, const Divisor& width, int rank,
                                          int size, B&& barrier) {
  const int w = (int)width.by, per_round = size * (kThreads * kPieces) / width;   // rows of a round
#pragma unroll 1
  for (int at = 0; at < keep;) {
    const int here = min(per_round, keep - at), pieces = here * w;
    // consecutive pieces for the threads of a block, runs of kThreads for the blocks in turn
    const int e0 = rank * kThreads + (int)threadIdx.x;
    T x[kPieces];
    int from[kPieces];
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      const int e = e0 + i * size * kThreads;
      if (e < pieces) from[i] = rows[at + e / width];
    }
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      const int e = e0 + i * size * kThreads;
      if (e < pieces) x[i] = base[(int64_t)from[i] * w + (e - e / width * w)];
    }
    barrier();
    T* const to = base + (int64_t)at * w;
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      const int e = e0 + i * size * kThreads;
      if (e < pieces) to[e] = x[i];
    }
    at += here;
  }
}

struct Select {
  alignas(16) int hist[3][kBins];    // a pass each: other blocks may still read the last one
  int sums[32];
  int sure[32], ties[32];            // rows of a warp that stay for sure, and at the border
  alignas(8) int total[2];           // and of the block
  int digit, left;
};

// R: rows of a lane that stay in registers, their keys; 0: none do, and weights are read in each pass.
template <int R>
__global__ void __launch_bounds__(kThreads, R == 32 ? 1 : 2) select_kernel(const Params p) {
  __shared__ Select sm;
  asm volatile("griddepcontrol.launch_dependents;");
  const uint32_t rank = cluster_rank(), size = cluster_size();
  const int bh = blockIdx.x / size, b = bh / p.Hkv;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  for (int i = tid; i < 3 * kBins; i += kThreads) sm.hist[0][i] = 0;
  if (tid < 32) sm.sums[tid] = sm.sure[tid] = sm.ties[tid] = 0;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int64_t len = p.lengths[b];
  const bool bad = len < 0 || len > p.cap;
  const int n = bad ? 0 : (int)len;
  int32_t* const rows = p.rows + (int64_t)bh * p.keep;
  if (bad && tid == 0 && rank == 0 && bh == b * p.Hkv) atomicOr(p.err, kErrLengths);
  if (n <= p.keep) {   // the same for the whole cluster
    for (int64_t i = rank * kThreads + tid; i < p.keep; i += size * kThreads) rows[i] = i < n ? (int)i : -1;
    return;
  }
  // The warp's rows [j0, j1), a whole number of them for each lane; row j0 + 32 i + lane is its i-th.
  const int per_lane = (int)(((int64_t)n + size * kThreads - 1) / (size * kThreads));
  const int64_t begin = ((int64_t)rank * kWarps + warp) * per_lane * 32;
  const int j0 = (int)min(begin, (int64_t)n), j1 = (int)min(begin + per_lane * 32, (int64_t)n);
  const int m = n - p.recent;          // candidates; more of them than places
  float* const w = p.weights + (int64_t)bh * p.cap;
  uint32_t held[R > 0 ? R : 1];
  if constexpr (R > 0) {
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const int j = j0 + 32 * i + lane;
      held[i] = j < j1 ? __float_as_uint(w[j]) : 0u;
    }
#pragma unroll
    for (int i = 0; i < R; ++i) held[i] = key_of(__uint_as_float(held[i]));
  }
  __syncthreads();
  // f(i, j, key) for each row of the warp's, whole warps at a time: j may be behind j1
  auto each = [&](auto&& f) {
    if constexpr (R > 0) {
#pragma unroll
      for (int i = 0; i < R; ++i)
        if (32 * i < j1 - j0) f(j0 + 32 * i + lane, held[i]);
    } else {
#pragma unroll 4
      for (int j = j0 + lane; j - lane < j1; j += 32) f(j, j < j1 ? key_of(w[j]) : 0u);
    }
  };

  uint32_t key = 0;
  int left = p.keep - p.recent;        // of the candidates that agree with key so far
  if (left > 0) {
    const int stop = min(j1, m);       // of the warp's candidates
#pragma unroll
    for (int pass = 0; pass < 3; ++pass) {
      const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, bits = pass == 2 ? 10 : 11;
      int* const hist = sm.hist[pass];
      each([&](int j, uint32_t k) {
        if (j < stop && (pass == 0 || (k ^ key) >> (shift + bits) == 0))
          atomicAdd(&hist[k >> shift & ((1 << bits) - 1)], 1);
      });
      cluster_barrier();
      // thread t has bins top - 3 .. top; larger digits are those of the threads below it
      const int top = kBins - 1 - 4 * tid;
      int4 v[kMaxCluster];
#pragma unroll
      for (uint32_t r = 0; r < kMaxCluster; ++r)
        v[r] = r < size ? remote4(&hist[top - 3], r) : make_int4(0, 0, 0, 0);
      int c[4] = {0, 0, 0, 0};
#pragma unroll
      for (int r = 0; r < kMaxCluster; ++r) c[0] += v[r].w, c[1] += v[r].z, c[2] += v[r].y, c[3] += v[r].x;
      const int mine = c[0] + c[1] + c[2] + c[3], up = warp_scan(mine);
      if (lane == 31) sm.sums[warp] = up;
      __syncthreads();
      int above = warp_scan(sm.sums[lane]) - sm.sums[lane];
      above = __shfl_sync(0xffffffffu, above, warp) + up - mine;
      if (above < left && left <= above + mine) {   // one thread
        int d = 0;
#pragma unroll
        for (int i = 0; i < 3; ++i)
          if (d == i && left > above + c[i]) above += c[i], ++d;
        sm.digit = top - d;
        sm.left = left - above;
      }
      __syncthreads();
      key |= (uint32_t)sm.digit << shift;
      left = sm.left;
    }
  }
  // Of the rows with that key the `left` lowest stay (with left 0: none), above it all.
  const bool any = left > 0;
  auto look = [&](int j, uint32_t k, uint32_t& sure, uint32_t& tie) {
    sure = __ballot_sync(0xffffffffu, j < j1 && (j >= m || (any && k > key)));
    tie = __ballot_sync(0xffffffffu, j < min(j1, m) && any && k == key);
  };
  int sure = 0, ties = 0;
  each([&](int j, uint32_t k) {
    uint32_t s, t;
    look(j, k, s, t);
    sure += __popc(s);
    ties += __popc(t);
  });
  if (lane == 0) {
    sm.sure[warp] = sure;
    sm.ties[warp] = ties;
  }
  __syncthreads();
  int s_before = warp_scan(sm.sure[lane]), t_before = warp_scan(sm.ties[lane]);
  if (tid == 31) {
    sm.total[0] = s_before;
    sm.total[1] = t_before;
  }
  s_before = __shfl_sync(0xffffffffu, s_before - sm.sure[lane], warp);
  t_before = __shfl_sync(0xffffffffu, t_before - sm.ties[lane], warp);
  cluster_barrier();
#pragma unroll
  for (uint32_t r = 0; r < kMaxCluster; ++r) {
    const int2 v = r < rank ? remote2(sm.total, r) : make_int2(0, 0);
    s_before += v.x;
    t_before += v.y;
  }
  const uint32_t below = (1u << lane) - 1;
  each([&](int j, uint32_t k) {
    uint32_t s, t;
    look(j, k, s, t);
    const int rank_t = t_before + __popc(t & below);
    if ((s >> lane & 1) || ((t >> lane & 1) && rank_t < left)) {
      const int to = s_before + __popc(s & below) + min(rank_t, left);
      rows[to] = j;
      // Weights in registers go to their places at once: no block reads its own from memory any more.
      if (R > 0) w[to] = weight_of(k);
    }
    s_before += __popc(s);
    t_before += __popc(t);
  });
  cluster_barrier();   // the others have read this block's totals, and written their part of the list
  if (R == 0) move_rows(w, rows, p.keep, p.one, (int)rank, (int)size, [] { cluster_barrier(); });
  for (int64_t j = p.keep + (int64_t)rank * kThreads + tid; j < n; j += size * kThreads)
    w[j] = 0.f;
}

__global__ void __launch_bounds__(kThreads, 2) move_kernel(const Params p) {
  asm volatile("griddepcontrol.launch_dependents;");
  const int rank = (int)cluster_rank(), size = (int)cluster_size();
  const int id = blockIdx.x / size, part = id / p.heads;
  const int64_t bh = id - part * p.heads, b = bh / p.Hkv;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (part == 0 && bh == b * p.Hkv && rank == 0 && threadIdx.x == 0) {   // lengths_out may be lengths
    const int64_t n = p.lengths[b];
    p.lengths_out[b] = n > p.keep && n <= p.cap ? p.keep : n;
  }
  const int32_t* const rows = p.rows + bh * p.keep;
  if (rows[p.keep - 1] < p.keep) return;   // nothing moves (the same for the whole cluster)
  const int bytes = part < 2 ? p.code_bytes : p.scale_bytes;
  uint8_t* const base = (part == 0 ? p.part[0] : part == 1 ? p.part[1] : part == 2 ? p.part[2] : p.part[3]) +
                        bh * p.cap * bytes;
  const Divisor& pieces = part < 2 ? p.code_pieces : p.scale_pieces;
  auto barrier = [] { cluster_barrier(); };
  switch (bytes / (int)pieces.by) {
    case 16: move_rows(reinterpret_cast<uint4*>(base), rows, p.keep, pieces, rank, size, barrier); break;
    case 8: move_rows(reinterpret_cast<uint2*>(base), rows, p.keep, pieces, rank, size, barrier); break;
    case 4: move_rows(reinterpret_cast<uint32_t*>(base), rows, p.keep, pieces, rank, size, barrier); break;
    case 2: move_rows(reinterpret_cast<uint16_t*>(base), rows, p.keep, pieces, rank, size, barrier); break;
    default: move_rows(base, rows, p.keep, pieces, rank, size, barrier);
  }
}

int launch(void (*kernel)(const Params), int64_t clusters, int size, const Params& p, cudaStream_t stream) {
  if (clusters * size > 0x7fffffff) return kErrShape;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)size;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(clusters * size));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  if (cudaLaunchKernelEx(&cfg, kernel, p) == cudaSuccess) return kOk;
  cudaGetLastError();
  return kErrLaunch;
}

// The smallest power of two of blocks, up to a cluster's, that leaves each at most `most` of n.
int blocks_for(int64_t n, int64_t most) {
  int c = 1;
  while (c < kMaxCluster && n > most * c) c *= 2;
  return c;
}

// Pieces of a row of n bytes, as large as its alignment lets them be, up to 16 bytes.
Divisor pieces_of(int n) {
  int size = 16;
  while (n % size) size /= 2;
  return divisor((uint32_t)(n / size));
}

}  // namespace

int launch_cache_evict_q4(const EvictQ4Call& c) {
  Params p;
  p.part[0] = (uint8_t*)c.cache.k4; p.part[1] = (uint8_t*)c.cache.v4;
  p.part[2] = (uint8_t*)c.cache.k_scale; p.part[3] = (uint8_t*)c.cache.v_scale;
  p.code_bytes = c.D / 2; p.scale_bytes = c.D / 16;
  p.code_pieces = pieces_of(p.code_bytes); p.scale_pieces = pieces_of(p.scale_bytes);
  p.one = divisor(1);
  p.weights = c.weights;
  p.lengths = c.lengths; p.lengths_out = c.lengths_out; p.rows = c.rows_out;
  p.cap = c.cache.max_seq_len;
  p.keep = (int)c.keep; p.recent = (int)c.recent;
  p.Hkv = c.Hkv;
  p.err = c.err;
  const int64_t heads = c.B * c.Hkv;
  if (4 * heads * kMaxCluster > 0x7fffffff) return kErrShape;
  p.heads = (int)heads;
  // Rows of a block by registers: 16 a lane, 32 where a cluster's eight blocks do not suffice, else none.
  const int sel = blocks_for(p.cap, 16 * kThreads);
  const int64_t per_lane = (p.cap + (int64_t)sel * kThreads - 1) / ((int64_t)sel * kThreads);
  const int rc = launch(per_lane <= 16 ? select_kernel<16> : per_lane <= 32 ? select_kernel<32> : select_kernel<0>,
                        heads, sel, p, c.stream);
  if (rc != kOk) return rc;
  const int mov = blocks_for(c.keep * p.code_bytes, (int64_t)kThreads * kPieces * 16);
  return launch(move_kernel, 4 * heads, mov, p, c.stream);
}

}  // namespace pfa
