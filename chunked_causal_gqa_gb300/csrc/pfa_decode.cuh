// pfa_decode.cuh -- what the decode kernels over the 8-bit and the 4-bit cache share: the list
// of work and its split over the blocks, and the kernel that joins partial sums.
//
// Work split: tiles of P::kUnit keys ("units") of all row tiles, sequences and heads form one
// list, cut into equal runs, one for each block.  What covers a head alone is stored as
// output by the block, what covers part of it goes to the workspace, and a second kernel,
// launched so that its start overlaps, joins the parts in order.
#pragma once
#include "pfa_internal.h"
#include "pfa_ptx.cuh"
#include "pfa_q8.cuh"

#include <cuda_bf16.h>

#include <algorithm>

namespace pfa {
namespace {

constexpr int kWarps = 4, kThreads = kWarps * 32;
constexpr int kMaxEntries = 1 << 14;           // (sequence, row tile) pairs of one launch
constexpr int64_t kMaxUnits = 1 << 30;         // units that a launch can list

// What the list and the join need of a launch.  A kernel's own parameters derive from it and
// say P::kUnit, P::kHeadCost, what the start and end of a head cost a block, in units (its query rows, the
// join), and P::kSums, whether row sums can be asked for (then also more_blocks() and, with
// MORE, more(): blocks behind those of the join for other work that waits for the first kernel).
struct ListParams {
  const void* q;
  void* out;
  const int64_t* lengths;
  int64_t T, start_pos, q_row, out_row;
  int64_t b0;                 // first sequence and row tile of this launch
  int tile0;
  int cap, Hkv, window;
  int rows, entries;          // T * group; entries of this launch
  Divisor group, seqs;        // H / Hkv; sequences in this launch
  Divisor heads, joined;      // Hkv, and the second kernel's blocks for a tile's rows
  int joins;                  // the second kernel's blocks that join
  float scale_log2, unit;     // of the scores, in powers of two; of the output
  unsigned* err;
  float* parts;               // workspace: slots of partial sums
  float2* sums;               // null, or {largest score, 1 / sum} of each row of each head
};

// A tile of rows of one sequence and the keys that they see.
template <int COST>
struct Entry {
  int64_t b;
  int end, r0, nr;    // sequence length; first row of the tile, rows
  int lo, hi;         // keys [lo, hi] are seen by some row
  int u0, n;          // units u0 .. u0 + n - 1 hold them
  bool bad;
  // Units of a head in the list of all: its own and its start's cost.
  __device__ int listed() const { return n > 0 ? n + COST : 0; }
};

// L2: the length is read from there, past this SM's own cache.
template <int RM, bool L2 = false, typename P>
__device__ __forceinline__ Entry<P::kHeadCost> entry_of(const P& p, int e) {
  Entry<P::kHeadCost> x;
  const int tile = e / p.seqs;
  x.b = p.b0 + e - tile * (int)p.seqs.by;
  x.r0 = (p.tile0 + tile) * RM;
  x.nr = min(RM, p.rows - x.r0);
  const int64_t end = !p.lengths ? p.start_pos + p.T
                      : L2       ? __ldcg((const long long*)p.lengths + x.b)
                                 : p.lengths[x.b];
  x.bad = end < 0 || end > p.cap;
  x.end = x.bad ? 0 : (int)end;
  const int first = x.end - (int)p.T;
  x.hi = first + (x.r0 + x.nr - 1) / p.group;
  x.lo = p.window > 0 ? max(0, first + x.r0 / p.group - p.window + 1) : 0;
  x.u0 = x.lo / P::kUnit;
  x.n = x.bad || x.hi < 0 ? 0 : x.hi / P::kUnit - x.u0 + 1;
  return x;
}

// Units of a run: those of all heads over the blocks, at least one for each of
// a block's teams.  Block c has the list's units [c * run, (c + 1) * run).
template <int TEAMS>
__device__ __forceinline__ int run_of(int total, int blocks) {
  return max((int)((uint32_t)(total + blocks - 1) / (uint32_t)blocks), TEAMS);
}

// Floats of a partial-sum slot: rows of output, then {m, l} of each row.
template <int RM, int D>
__host__ __device__ constexpr int slot_floats() { return RM * D + RM * 2; }

__device__ __forceinline__ float2 row_sums(float m, float l) {
  return make_float2(m == -INFINITY ? 0.f : m, l == 0.f ? 0.f : 1.f / l);
}

__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool on) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;"
               :: "r"(dst), "l"(src), "r"(on ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copy4(uint32_t dst, const void* src, bool on) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;"
               :: "r"(dst), "l"(src), "r"(on ? 4 : 0) : "memory");
}
__device__ __forceinline__ uint4 lds16(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
  return v;
}
__device__ __forceinline__ void mma(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t half2_of(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
// a, b -> high halves and what they leave out.
__device__ __forceinline__ void split2(float a, float b, uint32_t& hi, uint32_t& lo) {
  const __half2 h = __floats2half2_rn(a, b);
  const float2 f = __half22float2(h);
  hi = *reinterpret_cast<const uint32_t*>(&h);
  lo = half2_of(a - f.x, b - f.y);
}
__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Walks the units of a run that belong to one team, piece by piece: the part of
// a head that lies in the run.  A head's list starts with P::kHeadCost units of no work.
template <typename P, int RM, int TEAMS>
struct Cursor {
  static constexpr int kHeadCost = P::kHeadCost;
  int at, stop;        // the run from the current piece on: [at, stop)
  int e, h;            // entry and kv head of the piece
  Entry<kHeadCost> x;
  int listed;          // listed units of the piece
  int k0, kend;        // the head's units k0 .. kend - 1 are in the piece
  int k;               // the team's current one
  __device__ __forceinline__ void start(const P& p, int at_, int stop_, int e_, int into,
                                        int team) {
    at = at_;
    stop = stop_;
    e = e_;
    x = entry_of<RM>(p, e);
    // (the clamps matter only if the lengths change under the kernel)
    h = min((int)((uint32_t)into / (uint32_t)max(x.listed(), 1)), p.Hkv - 1);
    piece(min(into - h * x.listed(), x.listed()), team);
    if (kend <= k0) next_piece(p, team);
  }
  __device__ __forceinline__ void piece(int first, int team) {
    listed = min(stop - at, x.listed() - first);
    k0 = max(first - kHeadCost, 0);
    kend = first + listed - kHeadCost;
    k = k0 + team;
  }
  __device__ __forceinline__ bool done() const { return at >= stop; }
  __device__ __forceinline__ void next_piece(const P& p, int team) {
#pragma unroll 1
    do {
      at += listed;
      if (at >= stop) return;
      if (++h == p.Hkv) {
        h = 0;
#pragma unroll 1
        do {
          if (++e >= p.entries) {  // only if the lengths changed under the kernel
            at = stop;
            return;
          }
          x = entry_of<RM>(p, e);
        } while (x.n == 0);
      }
      piece(0, team);
    } while (kend <= k0);
  }
};

template <typename E>
__device__ __forceinline__ void store_row4(E* o, float4 v) {
  if constexpr (sizeof(E) == 4) {
    *reinterpret_cast<float4*>(o) = v;
  } else {
    const __nv_bfloat162 a = __floats2bfloat162_rn(v.x, v.y), b = __floats2bfloat162_rn(v.z, v.w);
    *reinterpret_cast<uint2*>(o) = make_uint2(*reinterpret_cast<const uint32_t*>(&a),
                                              *reinterpret_cast<const uint32_t*>(&b));
  }
}

struct ListShared {
  int sums[kWarps];
  int first_entry, into;
};

// The list of units, and where this block's run [at, stop) starts in it: `into` units into
// those of first_entry.  False: the block has none.
template <int RM, int TEAMS, typename P>
__device__ __forceinline__ bool run_start(const P& p, ListShared& sh, int& at, int& stop,
                                          int& first_entry, int& into) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (p.entries <= 32) {   // each warp for itself, an entry a lane
    const auto x = entry_of<RM>(p, min(lane, p.entries - 1));
    const int mine = lane < p.entries ? x.listed() * p.Hkv : 0;
    if (x.bad && blockIdx.x == 0 && warp == 0) atomicOr(p.err, kErrLengths);
    int up = mine;
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, up, o);
      if (lane >= o) up += v;
    }
    const int total = __shfl_sync(0xffffffffu, up, 31);
    const int run = run_of<TEAMS>(total, gridDim.x);
    at = blockIdx.x * run;
    stop = min(total, at + run);
    if (at >= total) return false;
    first_entry = __ffs(__ballot_sync(0xffffffffu, at < up)) - 1;
    into = at - __shfl_sync(0xffffffffu, up - mine, first_entry);
  } else {   // thread i has the entries [i * per, (i + 1) * per)
    const int per = (p.entries + kThreads - 1) / kThreads;
    int mine = 0;
#pragma unroll 1
    for (int e = tid * per; e < min(p.entries, (tid + 1) * per); ++e) {
      const auto x = entry_of<RM>(p, e);
      mine += x.listed() * p.Hkv;
      if (x.bad && blockIdx.x == 0) atomicOr(p.err, kErrLengths);
    }
    int up = mine;
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, up, o);
      if (lane >= o) up += v;
    }
    if (lane == 31) sh.sums[warp] = up;
    __syncthreads();
    int before = up - mine, total = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) before += sh.sums[w];
      total += sh.sums[w];
    }
    const int run = run_of<TEAMS>(total, gridDim.x);
    at = blockIdx.x * run;
    stop = min(total, at + run);
    if (at >= total) return false;
    if (before <= at && at < before + mine) {   // one thread
      int e = tid * per, rest = at - before;
#pragma unroll 1
      for (;; ++e) {
        const int n = entry_of<RM>(p, e).listed() * p.Hkv;
        if (rest < n || e + 1 >= min(p.entries, (tid + 1) * per)) break;
        rest -= n;
      }
      sh.first_entry = e;
      sh.into = rest;
    }
    __syncthreads();
    first_entry = sh.first_entry;
    into = sh.into;
  }
  return true;
}

// The parts of a head: blocks c0 .. c0 + n - 1 have one each, the first of them in its slot `first`.  None
// (n 0): nothing is seen.  One: the block has stored the output.
struct Parts {
  int c0, n, first;
};

// The list of units, as the first kernel counts it, while that one runs.  Its blocks let this
// grid start behind their own wait: whatever wrote the lengths has ended, and its writes are in
// L2.  (The first kernel's own results are read behind a wait of the caller's.)
template <int RM, int TEAMS, typename P>
__device__ __forceinline__ Parts parts_of(const P& p, int e, int h, const Entry<P::kHeadCost>& x,
                                          int blocks, int (*s_units)[2]) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, warps = blockDim.x >> 5;
  int before = 0, total = 0;
#pragma unroll 1
  for (int i = tid; i < p.entries; i += blockDim.x) {
    const int n = entry_of<RM, true>(p, i).listed() * p.Hkv;
    total += n;
    if (i < e) before += n;
  }
  for (int o = 16; o > 0; o >>= 1) {
    before += __shfl_xor_sync(0xffffffffu, before, o);
    total += __shfl_xor_sync(0xffffffffu, total, o);
  }
  if (lane == 0) {
    s_units[warp][0] = before;
    s_units[warp][1] = total;
  }
  __syncthreads();
  before = total = 0;
  for (int w = 0; w < warps; ++w) {
    before += s_units[w][0];
    total += s_units[w][1];
  }
  const int run = run_of<TEAMS>(total, blocks);
  const int s0 = before + h * x.listed();
  Parts y = {};
  if (x.n > 0) {
    y.c0 = (int)((uint32_t)(s0 + P::kHeadCost) / (uint32_t)run);
    y.n = (int)((uint32_t)(s0 + x.listed() - 1) / (uint32_t)run) - y.c0 + 1;
    // the first block's part is its run's last piece unless its run starts in this head
    y.first = y.c0 * run >= s0 ? 0 : 1;
  }
  return y;
}

// Where part i of a head is.
template <int RM, int D, typename P>
__device__ __forceinline__ const float* part_at(const P& p, const Parts& y, int i) {
  return p.parts + (int64_t)(2 * (y.c0 + i) + (i == 0 ? y.first : 0)) * slot_floats<RM, D>();
}

// A block has 128 columns of one row (GROUPS warps that take the parts in turn, in the
// blocks' order, each with a running maximum) or, with GROUPS 1, of up to 16 rows of a
// tile, a warp each.  It joins the parts of its head, and writes the zeros of rows
// that see nothing.
template <typename P, typename E, int NW, int RM, int GROUPS, bool MORE = false>
__global__ void __launch_bounds__(512) join_kernel(const P p, int blocks) {
  constexpr int D = NW * 128, TEAMS = kWarps / NW;
  __shared__ float4 s_sum[GROUPS > 1 ? GROUPS - 1 : 1][32];
  __shared__ float2 s_ml[GROUPS];
  __shared__ int s_units[16][2];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int grp = warp % GROUPS;
  if constexpr (MORE)
    if ((int)blockIdx.x >= p.joins) {
      p.template more<RM, NW>((int)blockIdx.x - p.joins, blocks, s_units);
      return;
    }
  const int id = blockIdx.x / NW, d = blockIdx.x % NW * 128 + lane * 4;
  const int eh = id / p.joined;
  const int r = (id - eh * (int)p.joined.by) * ((int)(blockDim.x >> 5) / GROUPS) + warp / GROUPS;
  const int e = eh / p.heads, h = eh - e * p.Hkv;
  asm volatile("griddepcontrol.launch_dependents;");
  const auto x = entry_of<RM, true>(p, e);
  const Parts head = parts_of<RM, TEAMS>(p, e, h, x, blocks, s_units);
  const int n = head.n;
  // Every block waits, also one with nothing to do: this grid must not end before the first.
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (r >= x.nr || x.bad || n == 1) return;   // n 1: stored whole
  const int q = x.r0 + r, t = q / p.group;
  E* to = (E*)p.out + (x.b * p.T + t) * p.out_row +
          (int64_t)(h * (int)p.group.by + q - t * (int)p.group.by) * D + d;
  if (n == 0) {
    if (grp == 0) store_row4(to, make_float4(0.f, 0.f, 0.f, 0.f));
    return;
  }
  float mx = -INFINITY, l = 0.f;
  float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
  for (int i0 = grp; i0 < n; i0 += 6 * GROUPS) {
    float4 v[6];
    float2 ml[6];
#pragma unroll
    for (int j = 0; j < 6; ++j) {
      const int i = i0 + GROUPS * j;
      ml[j] = make_float2(-INFINITY, 0.f);
      v[j] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (i < n) {
        const float* slot = part_at<RM, D>(p, head, i);
        ml[j] = *reinterpret_cast<const float2*>(slot + RM * D + 2 * r);
        v[j] = *reinterpret_cast<const float4*>(slot + r * D + d);
      }
    }
    float m = mx;
#pragma unroll
    for (int j = 0; j < 6; ++j) m = fmaxf(m, ml[j].x);
    const float base = m == -INFINITY ? 0.f : m;
    const float a = exp2_fast(mx - base);
    mx = m;
    l *= a;
    sum.x *= a; sum.y *= a; sum.z *= a; sum.w *= a;
#pragma unroll
    for (int j = 0; j < 6; ++j) {
      const float f = exp2_fast(ml[j].x - base);
      l = fmaf(ml[j].y, f, l);
      sum.x = fmaf(v[j].x, f, sum.x); sum.y = fmaf(v[j].y, f, sum.y);
      sum.z = fmaf(v[j].z, f, sum.z); sum.w = fmaf(v[j].w, f, sum.w);
    }
  }
  if constexpr (GROUPS > 1) {
    if (grp > 0) s_sum[grp - 1][lane] = sum;
    if (lane == 0) s_ml[grp] = make_float2(mx, l);
    __syncthreads();   // the block has one row: no warp has returned
    if (grp > 0) return;
  }
  float m = mx;
#pragma unroll
  for (int w = 1; w < GROUPS; ++w) m = fmaxf(m, s_ml[w].x);
  const float base = m == -INFINITY ? 0.f : m;
  const float a = exp2_fast(mx - base);
  l *= a;
  sum.x *= a; sum.y *= a; sum.z *= a; sum.w *= a;
#pragma unroll
  for (int w = 1; w < GROUPS; ++w) {
    const float f = exp2_fast(s_ml[w].x - base);
    const float4 v = s_sum[w - 1][lane];
    l = fmaf(s_ml[w].y, f, l);
    sum.x = fmaf(v.x, f, sum.x); sum.y = fmaf(v.y, f, sum.y);
    sum.z = fmaf(v.z, f, sum.z); sum.w = fmaf(v.w, f, sum.w);
  }
  if (P::kSums && p.sums && d == 0) p.sums[(x.b * p.Hkv + h) * p.rows + q] = row_sums(m, l);
  const float inv = l == 0.f ? 0.f : p.unit / l;
  store_row4(to, make_float4(sum.x * inv, sum.y * inv, sum.z * inv, sum.w * inv));
}

// The kernels of a launch and what they need.
template <typename P>
struct Kernels {
  void (*decode)(const P);
  void (*join_many)(const P, int);   // eight warps a row
  void (*join_few)(const P, int);    // a warp a row, up to 16 rows of a tile
  int rm, nw, blocks_per_sm;         // rows of a tile, head_dim / 128
  size_t smem;
};

// Both kernels over all sequences and row tiles, as many (sequence, row tile) entries a launch as
// its list can count.
template <typename P>
int launch_list(const Kernels<P>& k, P p, int64_t B, int num_sms, cudaStream_t stream) {
  const int64_t of_entry = (int64_t)p.Hkv * (p.cap / P::kUnit + 2 + P::kHeadCost);
  if (of_entry > kMaxUnits) return kErrShape;
  const int tiles = (p.rows + k.rm - 1) / k.rm;
  const int most = (int)std::min<int64_t>(kMaxEntries, kMaxUnits / of_entry);
  const int tiles_at_once = std::min(tiles, most);
  const int64_t at_once = tiles_at_once < tiles ? 1 : most / tiles;   // sequences
  p.heads = divisor(p.Hkv);
  // The first kernel may be launched before what is in front of it has ended: it waits
  // (griddepcontrol) before it reads anything.  The second one starts when every block of the
  // first is past that wait, and waits for the first before it reads what that writes.
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.stream = stream;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  const int most_blocks = num_sms * k.blocks_per_sm;
  for (int64_t b = 0; b < B; b += at_once)
    for (int tile = 0; tile < tiles; tile += tiles_at_once) {
      const int here = std::min(tiles_at_once, tiles - tile);
      p.b0 = b;
      p.tile0 = tile;
      const int seqs = (int)std::min(at_once, B - b);
      p.seqs = divisor(seqs);
      p.entries = seqs * here;
      // The list has all sequences' first row tiles, then all second ones: with a number of
      // blocks that the tiles divide, blocks far apart read the same keys at the same time and
      // the cache comes from HBM once (32 sequences of 8192 keys, 32/8 heads of 128, 8 / 12 / 20
      // tokens: 159 / 244 / 370 us; each sequence's tiles in a row 172 / 247 / -, tiles that
      // do not divide the blocks - / 254 / 407).
      const int blocks = here <= 16 ? most_blocks - most_blocks % here : most_blocks;
      // A head has about blocks / heads parts: for many of them eight warps to a row, for
      // few a warp (32 sequences of 8 heads: 49.7 us for both kernels with eight, 46.3 with one).
      const int rows = std::min(k.rm, p.rows);
      const bool many = (int64_t)p.entries * p.Hkv * 8 <= blocks;
      int threads = many ? 256 : std::min(rows, 16) * 32;
      int64_t more = 0;
      if constexpr (P::kSums) {
        threads = std::max(threads, p.more_threads());
        more = p.more_blocks(threads);
      }
      const int block_rows = many ? 1 : threads / 32;
      p.joined = divisor((rows + block_rows - 1) / block_rows);
      const int64_t joins = (int64_t)p.entries * p.Hkv * p.joined.by * k.nw;
      if (joins + more > 0x7fffffff) return kErrShape;
      p.joins = (int)joins;
      cfg.gridDim = dim3((unsigned)blocks);
      cfg.blockDim = dim3(kThreads);
      cfg.dynamicSmemBytes = k.smem;
      cudaError_t err = cudaLaunchKernelEx(&cfg, k.decode, p);
      if (err == cudaSuccess) {
        cfg.gridDim = dim3((unsigned)(joins + more));
        cfg.blockDim = dim3((unsigned)threads);
        cfg.dynamicSmemBytes = 0;
        err = cudaLaunchKernelEx(&cfg, many ? k.join_many : k.join_few, p, blocks);
      }
      if (err != cudaSuccess) {
        cudaGetLastError();
        return kErrLaunch;
      }
    }
  return kOk;
}

}  // namespace
}  // namespace pfa
