// pfa_evict_q4.cu -- cutting sequences of a 4-bit cache down to their newest and heaviest rows.
//
// For a sequence of n > keep rows, of each kv head: the `recent` newest rows stay, and the keep - recent
// largest of the others' weights (equal ones: the lower row).
//
// select_kernel, a cluster of up to eight blocks for each head, each with a run of its rows in registers:
// the key of a weight is its bits, turned so that unsigned order is the order of
// numbers.  Up to four passes over the candidates find the smallest key that is kept, eight bits at
// a time, from histograms that the blocks add up over distributed shared memory; then the kept rows
// are listed in order, each lane counting the kept rows in front of its own.  Weights move and become
// zero there too: every block has read its own by then.
//
// move_kernel, a cluster for each head and array: kept rows move down in place.  A row never moves
// up, so what a round writes (rows 0 .. below its end) is no source of a later one; in a
// round, which takes up to half a megabyte, the cluster's barrier stands between the reads and the
// writes.
//
// Measured on GB300, one pass among others:
//   63488 -> 16384 rows of 8 heads of 128 (42 MB)               23.9 us (floor 6.2): 11 us of selection, a
//     chain of some fifteen latencies in each of four passes and a list; 9 us for two rounds of moving
//   32 sequences of up to 8192 rows -> 2048, 8 heads (119 MB)   39.0 us (floor 17.6): moving reads 94 MB (rows
//     of scales are a quarter of a 32-byte sector) in 27 us
// Steps (the two cases): one block a head 1387 / 317; clusters 46.3 / 65.8; weights moved where they are
// selected 44.2 / 55.2; in registers 41.3 / 47.4; eight bits a pass (the blocks exchange 8 KB and not 64), a lane's
// rows side by side and the list through shared memory 23.9 / 40.7; moving blocks of 256 threads - / 39.0.
#include "pfa_internal.h"
#include "pfa_ptx.cuh"
#include "pfa_q4.cuh"

#include <algorithm>

namespace pfa {
namespace {

constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kBins = 256;
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
__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// A word of block `rank`'s shared memory.
__device__ __forceinline__ uint32_t remote_address(const void* p, uint32_t rank) {
  uint32_t a;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
  return a;
}
__device__ __forceinline__ int remote(const int* p, uint32_t rank) {
  int v;
  asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(remote_address(p, rank)));
  return v;
}
__device__ __forceinline__ int64_t remote(const int64_t* p, uint32_t rank) {
  int64_t v;
  asm volatile("ld.shared::cluster.s64 %0, [%1];" : "=l"(v) : "r"(remote_address(p, rank)));
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

template <typename T>
__device__ __forceinline__ T warp_scan(T x) {   // inclusive
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const T v = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += v;
  }
  return x;
}
// Exclusive sum over the block's threads, and the total; sums is zero behind the block's warps.
__device__ __forceinline__ int64_t block_scan(int64_t x, int64_t* sums, int64_t& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t up = warp_scan(x);
  __syncthreads();
  if (lane == 31) sums[warp] = up;
  __syncthreads();
  const int64_t all = warp_scan(sums[lane]);
  total = __shfl_sync(0xffffffffu, all, 31);
  return __shfl_sync(0xffffffffu, all - sums[lane], warp) + up - x;
}

// Rows `rows` of width.by pieces move to 0 .. keep - 1, in place, each piece x as as(x).  `rank` of `size` blocks;
// barrier(): theirs.
template <int THREADS, typename T, typename B, typename F>
__device__ __forceinline__ void move_rows(T* base, const int32_t* rows, int keep, const Divisor& width, int rank,
                                          int size, B&& barrier, F&& as) {
  const int w = (int)width.by, per_round = size * (THREADS * kPieces) / width;   // rows of a round
#pragma unroll 1
  for (int at = 0; at < keep;) {
    const int here = min(per_round, keep - at), pieces = here * w;
    // consecutive pieces for the threads of a block, runs of THREADS for the blocks in turn
    const int e0 = rank * THREADS + (int)threadIdx.x;
    T x[kPieces];
    int from[kPieces];
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      const int e = e0 + i * size * THREADS;
      if (e < pieces) from[i] = rows[at + e / width];
    }
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      const int e = e0 + i * size * THREADS;
      if (e < pieces) x[i] = base[(int64_t)from[i] * w + (e - e / width * w)];
    }
    barrier();
    T* const to = base + (int64_t)at * w;
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      const int e = e0 + i * size * THREADS;
      if (e < pieces) to[e] = as(x[i]);
    }
    at += here;
  }
}

template <int LANE>
struct Select {
  int hist[4][kBins];                // a pass each: other blocks may still read the last one
  int sums[32];                      // of the warps; zero behind the last
  int64_t pairs[32], total;          // rows that stay for sure, and 2^32 times those at the border
  int digit, count, left;
  uint32_t keys[kWarps][32][LANE + 1];   // a lane's rows, one word apart from the next lane's
  uint16_t kept[kWarps][32 * LANE];      // of a warp, in order
};

// LANE: rows of a lane at a time.
template <int LANE>
__global__ void __launch_bounds__(kThreads, 2) select_kernel(const Params p) {
  constexpr int kLane = LANE, kTile = kThreads * LANE;
  extern __shared__ __align__(16) uint8_t smem_raw[];
  Select<LANE>& sm = *reinterpret_cast<Select<LANE>*>(smem_raw);
  asm volatile("griddepcontrol.launch_dependents;");
  const uint32_t rank = cluster_rank(), size = cluster_size();
  const int bh = blockIdx.x / size, b = bh / p.Hkv;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  for (int i = tid; i < 4 * kBins; i += kThreads) sm.hist[0][i] = 0;
  if (tid < 32) sm.sums[tid] = 0, sm.pairs[tid] = 0;
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
  // The block's rows come in tiles; a lane has kLane consecutive rows of each, in registers.  With one
  // tile, which is the rule, they are read once.
  const int tiles = (int)(((int64_t)n + (int64_t)size * kTile - 1) / ((int64_t)size * kTile));
  const int m = n - p.recent;          // candidates; more of them than places
  float* const w = p.weights + (int64_t)bh * p.cap;
  uint32_t keys[kLane];
  int64_t j0;                          // this lane's first row of the tile
  auto load = [&](int tile) {
    const int64_t first = ((int64_t)rank * tiles + tile) * kTile + warp * (32 * kLane);   // the warp's
    j0 = first + lane * kLane;
    float x[kLane];
#pragma unroll
    for (int i = 0; i < kLane; ++i) x[i] = first + 32 * i + lane < n ? w[first + 32 * i + lane] : 0.f;
    __syncwarp();
#pragma unroll
    for (int i = 0; i < kLane; ++i) sm.keys[warp][(32 * i + lane) / kLane][lane % kLane] = key_of(x[i]);
    __syncwarp();
#pragma unroll
    for (int i = 0; i < kLane; ++i) keys[i] = sm.keys[warp][lane][i];
  };
  auto lane_rows = [&](int end) { return (int)max((int64_t)0, min((int64_t)kLane, end - j0)); };
  load(0);
  __syncthreads();

  uint32_t key = 0;
  bool inclusive = false;              // rows with a key above `key` stay, or not below it
  int left = p.keep - p.recent;        // of the candidates that agree with key so far
  if (left > 0) {
#pragma unroll 1
    for (int pass = 0; pass < 4 && !inclusive; ++pass) {
      const int shift = 24 - 8 * pass;
      int* const hist = sm.hist[pass];
#pragma unroll 1
      for (int tile = 0; tile < tiles; ++tile) {
        if (tiles > 1) load(tile);
        const int here = lane_rows(m);
        const uint32_t agree = pass == 0 ? 0u : 0xffffffffu << (shift + 8);
#pragma unroll
        for (int i = 0; i < kLane; ++i)
          if (i < here && ((keys[i] ^ key) & agree) == 0) atomicAdd(&hist[keys[i] >> shift & 255], 1);
      }
      cluster_barrier();
      // thread t has bin 255 - t; larger digits are those of the threads below it
      int v[kMaxCluster];
#pragma unroll
      for (uint32_t r = 0; r < kMaxCluster; ++r)
        v[r] = tid < kBins && r < size ? remote(&hist[kBins - 1 - tid], r) : 0;
      int mine = 0;
#pragma unroll
      for (int r = 0; r < kMaxCluster; ++r) mine += v[r];
      const int up = warp_scan(mine);
      if (lane == 31) sm.sums[warp] = up;
      __syncthreads();
      int above = warp_scan(sm.sums[lane]) - sm.sums[lane];
      above = __shfl_sync(0xffffffffu, above, warp) + up - mine;
      if (above < left && left <= above + mine) {   // one thread
        sm.digit = kBins - 1 - tid;
        sm.count = mine;
        sm.left = left - above;
      }
      __syncthreads();
      key |= (uint32_t)sm.digit << shift;
      left = sm.left;
      inclusive = sm.count == left;   // all that agree so far stay: the digits behind do not matter
    }
    if (inclusive) left = 0;
  }
  const bool any = p.keep > p.recent;
  // Of the rows with that key the `left` lowest stay, above it all.  Bits of this lane's rows:
  auto look = [&](uint32_t& sure, uint32_t& tie) {
    const uint32_t rows = (1u << lane_rows(n)) - 1, candidates = (1u << lane_rows(m)) - 1;
    uint32_t least = 0, equal = 0;
#pragma unroll
    for (int i = 0; i < kLane; ++i) {
      least |= keys[i] >= key ? 1u << i : 0u;
      equal |= keys[i] == key ? 1u << i : 0u;
    }
    sure = (any ? candidates & (inclusive ? least : least & ~equal) : 0u) | (rows & ~candidates);
    tie = any && !inclusive ? candidates & equal : 0u;
  };
  auto counts = [&](uint32_t sure, uint32_t tie) { return (int64_t)__popc(sure) | (int64_t)__popc(tie) << 32; };
  uint32_t sure, tie;
  int64_t mine = 0, total;
#pragma unroll 1
  for (int tile = 0; tile < tiles; ++tile) {
    if (tiles > 1) load(tile);
    look(sure, tie);
    mine += counts(sure, tie);
  }
  int64_t before = block_scan(mine, sm.pairs, total);
  if (tid == 0) sm.total = total;
  cluster_barrier();
  int64_t base = 0;
#pragma unroll
  for (uint32_t r = 0; r < kMaxCluster; ++r)
    if (r < rank) base += remote(&sm.total, r);
  cluster_arrive();   // this block has read the others' totals
#pragma unroll 1
  for (int tile = 0; tile < tiles; ++tile) {
    if (tiles > 1) {
      load(tile);
      look(sure, tie);
      before = block_scan(counts(sure, tie), sm.pairs, total);
    }
    const int ties = (int)((base + before) >> 32);
    int at = (int)(base + before) + min(ties, left);
#pragma unroll 1
    while (ties + __popc(tie) > left && tie != 0) tie &= ~(0x80000000u >> __clz(tie));
    const uint32_t kept = sure | tie;
    // through shared memory, so that a warp writes its part of the list in one piece
    const int warp_at = __shfl_sync(0xffffffffu, at, 0);
    int to = at - warp_at;
#pragma unroll
    for (int i = 0; i < kLane; ++i)
      if (kept >> i & 1) sm.kept[warp][to++] = (uint16_t)(lane * kLane + i);
    const int count = __shfl_sync(0xffffffffu, to, 31);
    const int first = (int)__shfl_sync(0xffffffffu, j0, 0);
    __syncwarp();
#pragma unroll 4
    for (int t = lane; t < count; t += 32) {
      const int i = sm.kept[warp][t];
      rows[warp_at + t] = first + i;
      // No block reads weights from memory any more, where there is one tile: they move at once.
      if (tiles == 1) w[warp_at + t] = weight_of(sm.keys[warp][i / kLane][i % kLane]);
    }
    __syncwarp();
    base += total;
  }
  cluster_wait();
  if (tiles > 1) {
    cluster_barrier();   // the list is whole
    // (as what its key stands for, as with one tile)
    move_rows<kThreads>(w, rows, p.keep, p.one, (int)rank, (int)size, [] { cluster_barrier(); },
                        [](float x) { return weight_of(key_of(x)); });
  }
  for (int64_t j = p.keep + (int64_t)rank * kThreads + tid; j < n; j += size * kThreads)
    w[j] = 0.f;
}

template <int THREADS>
__global__ void __launch_bounds__(THREADS, 1024 / THREADS) move_kernel(const Params p) {
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
  auto as = [](auto x) { return x; };
  switch (bytes / (int)pieces.by) {
    case 16: move_rows<THREADS>(reinterpret_cast<uint4*>(base), rows, p.keep, pieces, rank, size, barrier, as); break;
    case 8: move_rows<THREADS>(reinterpret_cast<uint2*>(base), rows, p.keep, pieces, rank, size, barrier, as); break;
    case 4: move_rows<THREADS>(reinterpret_cast<uint32_t*>(base), rows, p.keep, pieces, rank, size, barrier, as); break;
    case 2: move_rows<THREADS>(reinterpret_cast<uint16_t*>(base), rows, p.keep, pieces, rank, size, barrier, as); break;
    default: move_rows<THREADS>(base, rows, p.keep, pieces, rank, size, barrier, as);
  }
}

int launch(void (*kernel)(const Params), int64_t clusters, int size, int threads, size_t smem, const Params& p,
           cudaStream_t stream) {
  if (clusters * size > 0x7fffffff) return kErrShape;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)size;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(clusters * size));
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = smem;
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

// Threads of a moving block.  Blocks of 256, four to an SM, are in different phases of their rounds; where
// the heads are too few to fill the SMs with them, larger ones take fewer rounds.  Whole call, us,
// 256 / 512 threads: 63488 -> 16384 rows of 8 heads of 128 27.3 / 23.2, 120000 -> 65536 90.8 / 67.2; 32768 ->
// 16384 rows of 32 heads 37.5 / 41.6, 16384 -> 8192 of 64 39.6 / 49.8, 8192 -> 6000 of 256 127 / 170.  (1024
// threads, one block an SM: 27.3, 68.3, 60.1, 53.9, 184.)
int move_threads(int64_t heads, int num_sms) {
  return heads * 2 * kMaxCluster < (int64_t)2 * num_sms ? 512 : 256;
}

template <int LANE>
int launch_select(const Params& p, const EvictQ4Call& c) {
  static DeviceOnce once;
  const int rc = once.run(c.device, [] {
    return cudaFuncSetAttribute(select_kernel<LANE>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                (int)sizeof(Select<LANE>)) == cudaSuccess ? kOk : kErrLaunch;
  });
  if (rc != kOk) return rc;
  return launch(select_kernel<LANE>, p.heads, blocks_for(p.cap, kThreads * LANE), kThreads, sizeof(Select<LANE>), p,
                c.stream);
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
  // With 4 rows a lane a pass is shorter and a head has more blocks: gains where they are all there at once
  // (16 / 4 rows, us: 16000 rows of 8 heads 17 / 15, 8000 of 16 17 / 15; 8192 of 256 48 / 60, 1000 of 256 23 / 21).
  const bool thin = p.cap <= 4 * kThreads ||
                    (p.cap <= 4 * kThreads * kMaxCluster &&
                     heads * blocks_for(p.cap, 4 * kThreads) <= (int64_t)2 * c.num_sms);
  const int rc = thin ? launch_select<4>(p, c) : launch_select<16>(p, c);
  if (rc != kOk) return rc;
  const int64_t bytes = c.keep * p.code_bytes;
  const int threads = move_threads(heads, c.num_sms);
  return launch(threads == 512 ? move_kernel<512> : move_kernel<256>, 4 * heads,
                blocks_for(bytes, (int64_t)threads * kPieces * 16), threads, 0, p, c.stream);
}

}  // namespace pfa
