// pfa_q4_api.cu -- the C entry points of the operators around the 4-bit cache
// (declared in include/pfa.h): argument checks and dispatch.  Checks that need
// no device come first, so that a bad call is refused on any machine.
#include "pfa_checks.h"

#include <algorithm>
#include <cmath>

namespace pfa {
namespace {

constexpr int kMaxExp = 64;

// The shape of a 4-bit cache of `heads` blocks of rows.
int check_cache(int64_t heads, int head_dim, int64_t cap, int k_exp, int v_exp) {
  if (heads < 0 || head_dim <= 0 || head_dim > 512 || head_dim % 16 != 0) return PFA_ERR_SHAPE;
  if (cap <= 0 || cap > kMaxLen) return PFA_ERR_SHAPE;
  // sizes in bytes and work counts stay far inside 64 bits
  if (heads > ((int64_t)1 << 50) / (cap * head_dim)) return PFA_ERR_SHAPE;
  if (k_exp < -kMaxExp || k_exp > kMaxExp || v_exp < -kMaxExp || v_exp > kMaxExp) return PFA_ERR_VALUE;
  return PFA_OK;
}
// Rows are read up to 16 bytes at a time: what the largest power of two in head_dim / 16 leaves.
size_t scale_alignment(int head_dim) {
  const size_t n = (size_t)head_dim / 16, two = n & (~n + 1);
  return std::min<size_t>(two, 16);
}
int check_cache_pointers(const CacheQ4& c, int head_dim) {
  if (!c.k4 || !c.v4 || !c.k_scale || !c.v_scale) return PFA_ERR_NULL;
  const size_t a = scale_alignment(head_dim), codes = std::min<size_t>(8 * a, 16);
  if (misaligned(c.k4, codes) || misaligned(c.v4, codes) || misaligned(c.k_scale, a) ||
      misaligned(c.v_scale, a))
    return PFA_ERR_ALIGNMENT;
  return PFA_OK;
}
bool cache_shares(const CacheQ4& c, int64_t heads, int head_dim, const void* p, size_t n) {
  const size_t codes = (size_t)heads * c.max_seq_len * (head_dim / 2), scales = codes / 8;
  return overlaps(p, n, c.k4, codes) || overlaps(p, n, c.v4, codes) ||
         overlaps(p, n, c.k_scale, scales) || overlaps(p, n, c.v_scale, scales);
}
// Whether parts of a cache that is written lie over one another.
bool cache_overlaps_itself(const CacheQ4& c, int64_t heads, int head_dim) {
  const size_t codes = (size_t)heads * c.max_seq_len * (head_dim / 2), scales = codes / 8;
  return overlaps(c.k4, codes, c.v4, codes) || overlaps(c.k4, codes, c.k_scale, scales) ||
         overlaps(c.k4, codes, c.v_scale, scales) || overlaps(c.v4, codes, c.k_scale, scales) ||
         overlaps(c.v4, codes, c.v_scale, scales) ||
         overlaps(c.k_scale, scales, c.v_scale, scales);
}
bool accessible(const CacheQ4& c, int dev) {
  return device_accessible(c.k4, dev) && device_accessible(c.v4, dev) &&
         device_accessible(c.k_scale, dev) && device_accessible(c.v_scale, dev);
}
CacheQ4 cache_of(const void* k4, const void* v4, const void* k_scale, const void* v_scale,
                 int64_t cap, int k_exp, int v_exp) {
  return CacheQ4{const_cast<void*>(k4), const_cast<void*>(v4), const_cast<void*>(k_scale),
                 const_cast<void*>(v_scale), cap, k_exp, v_exp};
}

// The scores' factor with K's exponent has to be a float.
int check_scale(float scale, int k_exp) {
  return std::isfinite(std::ldexp(scale * 1.4426950408889634f, k_exp)) ? PFA_OK : PFA_ERR_VALUE;
}

// How a chunk of one sequence runs: few rows, and all of fp32, by the decode kernel; else the
// visible cache rows are read back into the workspace and the bf16 kernels run on them.
struct PrefillPlan {
  bool decode;
  int window;             // 0: none
  size_t total, least;    // workspace: what callers are told; what the call needs
  int64_t lo, rows;       // read back: cache rows [lo, lo + rows) are visible
  size_t v_at, ws_at;
  Call call;              // on the read-back rows
};

// Which is faster.  The decode kernel takes some 11 us and, at head_dim 128, 1.7e-6 us for each row, kv
// head and key; the other reads the cache back (656 bytes a key and kv head) and walks the keys with
// 128-row tiles: some 20 us (less below 1000 keys) and (0.1e-3 Hkv + 0.8e-3) us a key.  The constants are those of
// the least time lost over 669 shapes (256 to 63488 keys, 1 to 16 kv heads, groups of 1 to 8): 0.1 % on average, 11 %
// at most.  Measured on GB300 (us, decode / read back, the rule's last rows of decode and the next):
//   8 kv heads,  4096 keys, rows 192 / 256     21.5 / 25.3   26.7 / 25.5
//               16384 keys, rows 128 / 160     38.9 / 43.6   48.6 / 44.0
//               63488 keys, rows 112 / 128      112 / 114     123 / 114
//   2 kv heads,  4096 keys, rows 768 / 1024    22.8 / 22.9   26.8 / 23.4
//               16384 keys, rows 384 / 512     33.1 / 35.7   39.8 / 36.4
//               63488 keys, rows 256 / 384     67.0 / 67.2   94.9 / 61.3
//   1 kv head,  16384 keys, rows 768 / 1024    34.6 / 39.3   40.6 / 34.9
// head_dim 512: some 14 us and 1.1e-5 us for each row, kv head and key, against 11 us and 13e-3 us a key in each wave
// of the other's tiles; below some 500 keys it is the launches that count (438 shapes: 0.2 % and 17 %, at 64 keys)
//   2 kv heads,  1024 keys, rows 256 / 320     20.5 / 24.0   23.0 / 22.9
//                4096 keys, rows 512 / 640     61.9 / 64.2   73.5 / 63.4
//               16384 keys, rows 512 / 640      188 / 224     233 / 223
// fp32 always runs the decode kernel: the bf16 parts of the fp32 kernel would leave some 6e-5 of the
// output, and at head_dim 512 that attention runs on the CUDA cores.
constexpr int64_t kWave512 = 1300, kKeys512 = 650000;
int64_t waves_512(int64_t rows, int Hkv, int num_sms) {
  return ((rows + 255) / 256 * 4 * Hkv + num_sms - 1) / num_sms;
}
bool prefill_by_decode(int64_t T, int64_t keys, int H, int Hkv, int D, int dtype, int num_sms) {
  if (dtype == PFA_F32) return true;
  const int64_t rows = T * (H / Hkv);
  if (D == 128) return rows * Hkv <= std::min<int64_t>(4250000 / keys, 2100) + 60 * Hkv + 450;
  return rows * Hkv <= std::max(kWave512 * waves_512(rows, Hkv, num_sms) - kKeys512 / keys, 60000 / keys + 400);
}
// The most keys, up to `keys`, at which T tokens or fewer may be read back.
int64_t most_read_back(int64_t T, int64_t keys, int H, int Hkv, int D, int dtype, int num_sms) {
  if (!prefill_by_decode(T, keys, H, Hkv, D, dtype, num_sms)) return keys;
  if (dtype == PFA_F32 || D == 128) return 0;   // fewer rows and fewer keys run the decode kernel all the more
  const int64_t rows = T * (H / Hkv), more = kWave512 * waves_512(rows, Hkv, num_sms) - rows * Hkv;
  return rows * Hkv <= 400 ? 0 : more > 0 ? std::min(keys, kKeys512 / more + 1) : keys;
}

int prefill_plan(int64_t T, int64_t start_pos, int H, int Hkv, int D, int window, float scale,
                 int dtype, int64_t qkv_dim, int num_sms, void* stream, PrefillPlan* p) {
  // a window of all keys is none, and the kernels' 32-bit positions stay in range
  if (window < 0 || window >= start_pos + T) window = 0;
  p->window = window;
  const int64_t keys = window > 0 ? std::min<int64_t>(start_pos + T, window + T) : start_pos + T;
  p->decode = prefill_by_decode(T, keys, H, Hkv, D, dtype, num_sms);
  // (the decode kernel's slots grow with the rows: those of T hold any shorter chunk's)
  const size_t parts = decode_q4_workspace(1, T, H, Hkv, D, dtype, start_pos + T, false, num_sms).total;
  if (p->decode) {
    p->least = parts;
    // (an earlier start may read back where this one does not)
    const int64_t back = most_read_back(T, keys, H, Hkv, D, dtype, num_sms);
    p->total = std::max(parts, 2 * round256((size_t)Hkv * back * D * elem(PFA_BF16)));
    return PFA_OK;
  }
  p->lo = window > 0 ? std::max<int64_t>(0, start_pos - window + 1) : 0;
  p->rows = start_pos + T - p->lo;
  const size_t kv = round256((size_t)Hkv * p->rows * D * elem(PFA_BF16));
  // causal and window masks depend on differences of positions only
  const int rc = prepare_layout(nullptr, nullptr, nullptr, nullptr, T, start_pos - p->lo, H, Hkv,
                                D, window, scale, PFA_BF16, qkv_dim, p->rows, 0, stream, false,
                                &p->call);
  if (rc != PFA_OK) return rc;
  p->v_at = kv;
  p->ws_at = 2 * kv;
  p->least = p->ws_at;   // without more the plain schedule runs
  p->total = std::max(parts, p->ws_at + round256(workspace_bytes_bf16(p->call)));
  return PFA_OK;
}

}  // namespace
}  // namespace pfa

using namespace pfa;

extern "C" {

int pfa_cache_write_q4(const void* k, const void* v, void* k4, void* v4, void* k_scale,
                       void* v_scale, int64_t B, int64_t T, int64_t start_pos,
                       const int64_t* lengths, int num_kv_heads, int head_dim,
                       int64_t max_seq_len, int k_exp, int v_exp, int dtype, int64_t k_stride,
                       int64_t v_stride, void* stream) {
  if (dtype != PFA_F32 && dtype != PFA_BF16) return PFA_ERR_DTYPE;
  if (num_kv_heads <= 0 || num_kv_heads > 65536) return PFA_ERR_SHAPE;
  int rc = check_span(B, T, start_pos, lengths);
  if (rc != PFA_OK) return rc;
  if ((rc = check_cache(B * num_kv_heads, head_dim, max_seq_len, k_exp, v_exp)) != PFA_OK) return rc;
  if (T > max_seq_len || (!lengths && start_pos + T > max_seq_len)) return PFA_ERR_SHAPE;
  if (B == 0 || T == 0) return PFA_OK;
  if (!k || !v) return PFA_ERR_NULL;
  WriteQ4Call c;
  c.cache = cache_of(k4, v4, k_scale, v_scale, max_seq_len, k_exp, v_exp);
  if ((rc = check_cache_pointers(c.cache, head_dim)) != PFA_OK) return rc;
  const int64_t es = (int64_t)elem(dtype), width = (int64_t)num_kv_heads * head_dim;
  if (k_stride < width || v_stride < width) return PFA_ERR_SHAPE;
  if ((k_stride * es) % 16 || (v_stride * es) % 16 || misaligned(k, 16) || misaligned(v, 16))
    return PFA_ERR_ALIGNMENT;
  const int64_t heads = B * num_kv_heads;
  const Rows rk{k, B * T, (size_t)(k_stride * es), (size_t)(width * es)};
  const Rows rv{v, B * T, (size_t)(v_stride * es), (size_t)(width * es)};
  if (cache_shares(c.cache, heads, head_dim, k, rk.span()) ||
      cache_shares(c.cache, heads, head_dim, v, rv.span()) ||
      cache_overlaps_itself(c.cache, heads, head_dim) ||
      (lengths && cache_shares(c.cache, heads, head_dim, lengths, (size_t)B * 8)))
    return PFA_ERR_ALIAS;
  DeviceInfo d;
  if ((rc = current_device(&d)) != kOk) return rc;
  if (!device_accessible(k, d.device) || !device_accessible(v, d.device) ||
      !accessible(c.cache, d.device) || (lengths && !device_accessible(lengths, d.device)))
    return PFA_ERR_DEVICE;
  c.k = k; c.v = v;
  c.span = Span{B, T, start_pos, lengths};
  c.Hkv = num_kv_heads; c.D = head_dim; c.dtype = dtype;
  c.k_row = k_stride; c.v_row = v_stride;
  c.err = d.err;
  c.stream = static_cast<cudaStream_t>(stream);
  return launch_cache_write_q4(c);
}

int pfa_cache_read_q4(const void* k4, const void* v4, const void* k_scale, const void* v_scale,
                      void* k_out, void* v_out, int64_t heads, int64_t start, int64_t rows,
                      int head_dim, int64_t max_seq_len, int k_exp, int v_exp, int dtype,
                      int64_t out_head_stride, void* stream) {
  if (dtype != PFA_F32 && dtype != PFA_BF16) return PFA_ERR_DTYPE;
  int rc = check_cache(heads, head_dim, max_seq_len, k_exp, v_exp);
  if (rc != PFA_OK) return rc;
  if (heads > kMaxLen || start < 0 || rows < 0 || start > max_seq_len ||
      rows > max_seq_len - start)
    return PFA_ERR_SHAPE;
  if (heads == 0 || rows == 0) return PFA_OK;
  ReadQ4Call c;
  c.cache = cache_of(k4, v4, k_scale, v_scale, max_seq_len, k_exp, v_exp);
  if ((rc = check_cache_pointers(c.cache, head_dim)) != PFA_OK) return rc;
  if (!k_out || !v_out) return PFA_ERR_NULL;
  const int64_t es = (int64_t)elem(dtype), width = rows * head_dim;
  if (out_head_stride < width) return PFA_ERR_SHAPE;
  if ((out_head_stride * es) % 16 || misaligned(k_out, 16) || misaligned(v_out, 16))
    return PFA_ERR_ALIGNMENT;
  const Rows ok{k_out, heads, (size_t)(out_head_stride * es), (size_t)(width * es)};
  const Rows ov{v_out, heads, (size_t)(out_head_stride * es), (size_t)(width * es)};
  if (share(ok, ov) || cache_shares(c.cache, heads, head_dim, k_out, ok.span()) ||
      cache_shares(c.cache, heads, head_dim, v_out, ov.span()))
    return PFA_ERR_ALIAS;
  DeviceInfo d;
  if ((rc = current_device(&d)) != kOk) return rc;
  if (!accessible(c.cache, d.device) || !device_accessible(k_out, d.device) ||
      !device_accessible(v_out, d.device))
    return PFA_ERR_DEVICE;
  c.k_out = k_out; c.v_out = v_out;
  c.heads = heads; c.start = start; c.rows = rows; c.out_head = out_head_stride;
  c.D = head_dim; c.dtype = dtype;
  c.stream = static_cast<cudaStream_t>(stream);
  return launch_cache_read_q4(c);
}

int pfa_decode_workspace_bytes_q4(int64_t B, int64_t T, int num_heads, int num_kv_heads,
                                  int head_dim, int dtype, int64_t max_seq_len, int weights,
                                  size_t* bytes) {
  if (!bytes) return PFA_ERR_NULL;
  *bytes = 0;
  int rc = check_attention(B, T, num_heads, num_kv_heads, head_dim, 1.f, dtype);
  if (rc != PFA_OK) return rc;
  if (B > kMaxLen || T > kMaxLen || T * (num_heads / num_kv_heads) > PFA_DECODE_MAX_ROWS)
    return PFA_ERR_SHAPE;
  if ((rc = check_cache(B * num_kv_heads, head_dim, max_seq_len, 0, 0)) != PFA_OK) return rc;
  if (B == 0 || T == 0) return PFA_OK;
  DeviceInfo d;
  if ((rc = current_device(&d)) != kOk) return rc;
  *bytes = decode_q4_workspace(B, T, num_heads, num_kv_heads, head_dim, dtype, max_seq_len,
                               weights != 0, d.num_sms).total;
  return PFA_OK;
}

int pfa_decode_attention_q4(const void* q, const void* k4, const void* v4, const void* k_scale,
                            const void* v_scale, void* out, float* weights, int64_t B, int64_t T,
                            const int64_t* lengths, int num_heads, int num_kv_heads, int head_dim,
                            int window, float scale, int dtype, int64_t q_stride,
                            int64_t out_stride, int64_t max_seq_len, int k_exp, int v_exp,
                            void* workspace, size_t workspace_bytes, void* stream) {
  int rc = check_attention(B, T, num_heads, num_kv_heads, head_dim, scale, dtype);
  if (rc != PFA_OK) return rc;
  if (B > kMaxLen || T > kMaxLen || T * (num_heads / num_kv_heads) > PFA_DECODE_MAX_ROWS)
    return PFA_ERR_SHAPE;
  if ((rc = check_cache(B * num_kv_heads, head_dim, max_seq_len, k_exp, v_exp)) != PFA_OK) return rc;
  if ((rc = check_scale(scale, k_exp)) != PFA_OK) return rc;
  if (B == 0 || T == 0) return PFA_OK;
  if (!lengths) return PFA_ERR_NULL;
  if ((rc = check_span(B, T, 0, lengths)) != PFA_OK) return rc;
  DecodeQ4Call c;
  c.cache = cache_of(k4, v4, k_scale, v_scale, max_seq_len, k_exp, v_exp);
  if ((rc = check_cache_pointers(c.cache, head_dim)) != PFA_OK) return rc;
  if (!q || !out) return PFA_ERR_NULL;
  const int64_t es = (int64_t)elem(dtype), width = (int64_t)num_heads * head_dim;
  if (q_stride < width || out_stride < width) return PFA_ERR_SHAPE;
  if ((q_stride * es) % 16 || (out_stride * es) % 16 || misaligned(q, 16) || misaligned(out, 16) ||
      misaligned(weights, 4) || misaligned(workspace, 256))
    return PFA_ERR_ALIGNMENT;
  const int64_t heads = B * num_kv_heads;
  const Rows rq{q, B * T, (size_t)(q_stride * es), (size_t)(width * es)};
  const Rows ro{out, B * T, (size_t)(out_stride * es), (size_t)(width * es)};
  const size_t wbytes = weights ? (size_t)heads * max_seq_len * sizeof(float) : 0;
  if (share(ro, rq) || cache_shares(c.cache, heads, head_dim, out, ro.span()) ||
      overlaps(out, ro.span(), lengths, (size_t)B * 8))
    return PFA_ERR_ALIAS;
  if (weights &&
      (cache_shares(c.cache, heads, head_dim, weights, wbytes) ||
       overlaps(weights, wbytes, q, rq.span()) || overlaps(weights, wbytes, out, ro.span()) ||
       overlaps(weights, wbytes, lengths, (size_t)B * 8)))
    return PFA_ERR_ALIAS;
  DeviceInfo d;
  if ((rc = current_device(&d)) != kOk) return rc;
  const DecodeQ4Sizes need = decode_q4_workspace(B, T, num_heads, num_kv_heads, head_dim, dtype,
                                                 max_seq_len, weights != nullptr, d.num_sms);
  if (!workspace || workspace_bytes < need.least) return PFA_ERR_SCRATCH;
  const size_t used = std::min(workspace_bytes, need.total);
  if (overlaps(workspace, used, q, rq.span()) || overlaps(workspace, used, out, ro.span()) ||
      overlaps(workspace, used, lengths, (size_t)B * 8) ||
      (weights && overlaps(workspace, used, weights, wbytes)) ||
      cache_shares(c.cache, heads, head_dim, workspace, used))
    return PFA_ERR_ALIAS;
  if (!device_accessible(workspace, d.device)) return PFA_ERR_DEVICE;
  if (!device_accessible(q, d.device) || !device_accessible(out, d.device) ||
      !device_accessible(lengths, d.device) || !accessible(c.cache, d.device) ||
      (weights && !device_accessible(weights, d.device)))
    return PFA_ERR_DEVICE;
  c.q = q; c.out = out; c.weights = weights;
  c.span = Span{B, T, 0, lengths};
  c.H = num_heads; c.Hkv = num_kv_heads; c.D = head_dim;
  // (a window of the whole cache is none, and the kernels' 32-bit positions stay in range)
  c.window = window > 0 && window < max_seq_len ? window : 0;
  c.dtype = dtype; c.scale = scale;
  c.q_row = q_stride; c.out_row = out_stride;
  c.err = d.err; c.num_sms = d.num_sms; c.device = d.device;
  c.ws = workspace; c.ws_bytes = workspace_bytes;
  c.stream = static_cast<cudaStream_t>(stream);
  return launch_decode_q4(c);
}

int pfa_prefill_workspace_bytes_q4(int64_t T, int64_t start_pos, int num_heads, int num_kv_heads,
                                   int head_dim, int window, int dtype, size_t* bytes) {
  if (!bytes) return PFA_ERR_NULL;
  *bytes = 0;
  int rc = check_attention(1, T, num_heads, num_kv_heads, head_dim, 1.f, dtype);
  if (rc != PFA_OK) return rc;
  if ((rc = check_span(1, T, start_pos, nullptr)) != PFA_OK) return rc;
  if (T == 0) return PFA_OK;
  DeviceInfo d;
  if ((rc = current_device(&d)) != kOk) return rc;
  PrefillPlan plan;
  rc = prefill_plan(T, start_pos, num_heads, num_kv_heads, head_dim, window, 1.f, dtype,
                    (int64_t)num_heads * head_dim, d.num_sms, nullptr, &plan);
  if (rc == PFA_OK) *bytes = plan.total;
  return rc;
}

int pfa_prefill_attention_q4(const void* q, const void* k4, const void* v4, const void* k_scale,
                             const void* v_scale, void* out, int64_t T, int64_t start_pos,
                             int num_heads, int num_kv_heads, int head_dim, int window,
                             float scale, int dtype, int64_t qkv_dim, int64_t max_seq_len,
                             int k_exp, int v_exp, void* workspace, size_t workspace_bytes,
                             void* stream) {
  int rc = check_attention(1, T, num_heads, num_kv_heads, head_dim, scale, dtype);
  if (rc != PFA_OK) return rc;
  if ((rc = check_span(1, T, start_pos, nullptr)) != PFA_OK) return rc;
  if ((rc = check_cache(num_kv_heads, head_dim, max_seq_len, k_exp, v_exp)) != PFA_OK) return rc;
  if ((rc = check_scale(scale, k_exp)) != PFA_OK) return rc;
  if (start_pos + T > max_seq_len) return PFA_ERR_SHAPE;
  if (T == 0) return PFA_OK;
  const CacheQ4 cache = cache_of(k4, v4, k_scale, v_scale, max_seq_len, k_exp, v_exp);
  if ((rc = check_cache_pointers(cache, head_dim)) != PFA_OK) return rc;
  if (!q || !out) return PFA_ERR_NULL;
  const int64_t es = (int64_t)elem(dtype), width = (int64_t)num_heads * head_dim;
  if (qkv_dim < width) return PFA_ERR_SHAPE;
  if ((qkv_dim * es) % 16 || misaligned(q, 16) || misaligned(out, 16) ||
      misaligned(workspace, 256))
    return PFA_ERR_ALIGNMENT;
  const Rows rq{q, T, (size_t)(qkv_dim * es), (size_t)(width * es)};
  const Rows ro{out, T, (size_t)(qkv_dim * es), (size_t)(width * es)};
  if (share(ro, rq) || cache_shares(cache, num_kv_heads, head_dim, out, ro.span()))
    return PFA_ERR_ALIAS;
  DeviceInfo d;
  if ((rc = current_device(&d)) != kOk) return rc;
  PrefillPlan plan;
  rc = prefill_plan(T, start_pos, num_heads, num_kv_heads, head_dim, window, scale, dtype, qkv_dim,
                    d.num_sms, stream, &plan);
  if (rc != PFA_OK) return rc;
  if (!workspace || workspace_bytes < plan.least) return PFA_ERR_SCRATCH;
  const size_t used = std::min(workspace_bytes, plan.total);
  if (overlaps(workspace, used, q, rq.span()) || overlaps(workspace, used, out, ro.span()) ||
      cache_shares(cache, num_kv_heads, head_dim, workspace, used))
    return PFA_ERR_ALIAS;
  if (!device_accessible(workspace, d.device)) return PFA_ERR_DEVICE;
  if (!device_accessible(q, d.device) || !device_accessible(out, d.device) ||
      !accessible(cache, d.device))
    return PFA_ERR_DEVICE;
  if (plan.decode) {
    DecodeQ4Call c;
    c.q = q; c.out = out; c.weights = nullptr; c.cache = cache;
    c.span = Span{1, T, start_pos, nullptr};
    c.H = num_heads; c.Hkv = num_kv_heads; c.D = head_dim;
    c.window = plan.window; c.dtype = dtype; c.scale = scale;
    c.q_row = qkv_dim; c.out_row = qkv_dim;
    c.err = d.err; c.num_sms = d.num_sms; c.device = d.device;
    c.ws = workspace; c.ws_bytes = workspace_bytes;
    c.stream = static_cast<cudaStream_t>(stream);
    return launch_decode_q4(c);
  }
  char* base = static_cast<char*>(workspace);
  ReadQ4Call r;
  r.cache = cache;
  r.k_out = base; r.v_out = base + plan.v_at;
  r.heads = num_kv_heads; r.start = plan.lo; r.rows = plan.rows;
  r.out_head = plan.rows * head_dim;
  r.D = head_dim; r.dtype = PFA_BF16;
  r.stream = static_cast<cudaStream_t>(stream);
  if ((rc = launch_cache_read_q4(r)) != kOk) return rc;
  plan.call.q = q; plan.call.out = out;
  plan.call.k = r.k_out; plan.call.v = r.v_out;
  plan.call.ws_bytes = used - plan.ws_at;
  plan.call.ws = plan.call.ws_bytes ? base + plan.ws_at : nullptr;
  return dispatch(plan.call, PFA_BF16);
}

int pfa_cache_evict_q4(void* k4, void* v4, void* k_scale, void* v_scale, float* weights, int64_t B,
                       const int64_t* lengths, int num_kv_heads, int head_dim, int64_t max_seq_len,
                       int64_t keep, int64_t recent, int64_t* lengths_out, int32_t* rows_out,
                       void* stream) {
  if (B < 0 || B > kMaxLen || num_kv_heads <= 0 || num_kv_heads > 65536) return PFA_ERR_SHAPE;
  int rc = check_cache(B * num_kv_heads, head_dim, max_seq_len, 0, 0);
  if (rc != PFA_OK) return rc;
  if (keep < 1 || keep > max_seq_len || recent < 0 || recent > keep) return PFA_ERR_SHAPE;
  if (B == 0) return PFA_OK;
  if (!weights || !lengths || !lengths_out || !rows_out) return PFA_ERR_NULL;
  EvictQ4Call c;
  c.cache = cache_of(k4, v4, k_scale, v_scale, max_seq_len, 0, 0);
  if ((rc = check_cache_pointers(c.cache, head_dim)) != PFA_OK) return rc;
  if (misaligned(weights, 4) || misaligned(lengths, 8) || misaligned(lengths_out, 8) ||
      misaligned(rows_out, 4))
    return PFA_ERR_ALIGNMENT;
  const int64_t heads = B * num_kv_heads;
  const size_t wbytes = (size_t)heads * max_seq_len * sizeof(float), nbytes = (size_t)B * 8;
  const size_t rbytes = (size_t)heads * keep * sizeof(int32_t);
  if (cache_overlaps_itself(c.cache, heads, head_dim) ||
      cache_shares(c.cache, heads, head_dim, weights, wbytes) ||
      cache_shares(c.cache, heads, head_dim, lengths, nbytes) ||
      cache_shares(c.cache, heads, head_dim, lengths_out, nbytes) ||
      cache_shares(c.cache, heads, head_dim, rows_out, rbytes) ||
      overlaps(weights, wbytes, lengths, nbytes) || overlaps(weights, wbytes, lengths_out, nbytes) ||
      overlaps(weights, wbytes, rows_out, rbytes) || overlaps(rows_out, rbytes, lengths, nbytes) ||
      overlaps(rows_out, rbytes, lengths_out, nbytes) ||
      (lengths_out != lengths && overlaps(lengths_out, nbytes, lengths, nbytes)))
    return PFA_ERR_ALIAS;
  DeviceInfo d;
  if ((rc = current_device(&d)) != kOk) return rc;
  if (!accessible(c.cache, d.device) || !device_accessible(weights, d.device) ||
      !device_accessible(lengths, d.device) || !device_accessible(lengths_out, d.device) ||
      !device_accessible(rows_out, d.device))
    return PFA_ERR_DEVICE;
  c.weights = weights;
  c.B = B; c.lengths = lengths;
  c.Hkv = num_kv_heads; c.D = head_dim;
  c.keep = keep; c.recent = recent;
  c.lengths_out = lengths_out; c.rows_out = rows_out;
  c.err = d.err; c.num_sms = d.num_sms; c.device = d.device;
  c.stream = static_cast<cudaStream_t>(stream);
  return launch_cache_evict_q4(c);
}

}  // extern "C"
