// pfa_q8_api.cu -- the C entry points of the operators around the 8-bit cache
// (declared in include/pfa.h): argument checks and dispatch.  Checks that need
// no device come first, so that a bad call is refused on any machine.
#include "pfa_checks.h"

#include <algorithm>
#include <cmath>

namespace pfa {
namespace {

// The shape of an 8-bit cache of `heads` blocks of rows.
int check_cache(int64_t heads, int head_dim, int64_t cap, int block) {
  if (heads < 0 || head_dim <= 0 || head_dim > 512 || head_dim % 16 != 0) return PFA_ERR_SHAPE;
  if (block != 16 && block != 32 && block != 64 && block != 128) return PFA_ERR_SHAPE;
  if (cap <= 0 || cap > kMaxLen || cap % block != 0) return PFA_ERR_SHAPE;
  // sizes in bytes and work counts stay far inside 64 bits
  if (heads > ((int64_t)1 << 50) / (cap * head_dim)) return PFA_ERR_SHAPE;
  return PFA_OK;
}
int check_cache_pointers(const CacheQ8& c) {
  if (!c.k8 || !c.v8 || !c.k_scale || !c.v_scale) return PFA_ERR_NULL;
  if (misaligned(c.k8, 16) || misaligned(c.v8, 16) || misaligned(c.k_scale, 4) ||
      misaligned(c.v_scale, 4))
    return PFA_ERR_ALIGNMENT;
  return PFA_OK;
}
bool cache_shares(const CacheQ8& c, int64_t heads, int head_dim, const void* p, size_t n) {
  const size_t codes = (size_t)heads * c.max_seq_len * head_dim;
  const size_t scales = (size_t)heads * (c.max_seq_len / c.block) * sizeof(float);
  return overlaps(p, n, c.k8, codes) || overlaps(p, n, c.v8, codes) ||
         overlaps(p, n, c.k_scale, scales) || overlaps(p, n, c.v_scale, scales);
}
bool accessible(const CacheQ8& c, int dev) {
  return device_accessible(c.k8, dev) && device_accessible(c.v8, dev) &&
         device_accessible(c.k_scale, dev) && device_accessible(c.v_scale, dev);
}

CacheQ8 cache_of(const void* k8, const void* v8, const float* k_scale, const float* v_scale,
                 int64_t cap, int block) {
  return CacheQ8{const_cast<void*>(k8), const_cast<void*>(v8), const_cast<float*>(k_scale),
                 const_cast<float*>(v_scale), cap, block};
}

// How a chunk of one sequence runs: few rows, and all of fp32, by the decode kernel; the
// tiles of a bf16 chunk of head_dim 128 from the codes; or the visible cache rows read
// back into the workspace and the bf16 kernels on them.
enum class How { kDecode, kCodes, kReadBack };
struct PrefillPlan {
  How how;
  int window;             // 0: none
  size_t total;           // workspace
  int64_t lo, rows;       // kReadBack: cache rows [lo, lo + rows) are visible
  size_t v_at, ws_at;
  Call call;              // on the read-back rows
};

// Which of them is fastest, by what bounds it.  The decode kernel's time grows with rows *
// kv heads (it takes 16 rows at a time, 8 of fp32); the others walk the keys with
// 128-row tiles in waves of the SMs.  Measured on GB300 (us):
//   bf16, head_dim 128, 32/8 heads, rows = T * 4:      decode  codes  read back
//     63488 keys, rows 32 / 64 / 128                 50 / 82 / 144   71 / 70 / 72   120
//     63488 keys, rows 512 / 768 / 1024 / 2048        123 / 171 / 244 / 434 (codes), 153 / 191 / 235 / 398 (read back)
//     4096 keys, rows 32 / 128 / 256 / 384           15 / 21 / 33 / 43   21 / 22 / 25 / 26   26 / 25 / 26 / 24
//   The thresholds of head_dim 128 are those of 8 kv heads (8/8 heads within 4% of 32/8).  With
//   few kv heads the decode kernel would be the faster one for longer, up to some 400 rows *
//   kv heads, which this rule leaves unused (decode / codes / read back):
//     1 kv head, 16384 keys, rows 64 / 256 / 512     11 / 50 / 45   16 / 55 / 47   26 / 38 / 49
//     1 kv head, 63488 keys, rows 64 / 256 / 512     18 / 56 / 89   42 / 61 / 91   76 / 52 / 61
//     2 kv heads, 16384 keys, rows 64 / 256 / 512    12 / 34 / 51   26 / 39 / 51   44 / 32 / 38
//     2 kv heads, 63488 keys, rows 64 / 256 / 512    26 / 46 / 69   77 / 52 / 68   144 / 52 / 64
//   bf16, head_dim 512, 16384 keys (decode / read back), the rule's last rows of decode and the next:
//     1 kv head, rows 1024 / 1536      195 / 219   290 / 219
//     2 kv heads, rows 512 / 768       196 / 225   292 / 225
//     4 kv heads, rows 256 / 512       197 / 240   385 / 240
//     (4096 keys: 56 / 63 and 83 / 63, 58 / 65 and 85 / 65, 58 / 67 and 109 / 67)
// fp32 always runs the decode kernel: pfa_f32x3_d128.cu on rows read back is faster from
// some 600 rows on (16384 keys, 32/8 heads, 768 rows: 360 us against 398), but its split
// into bf16 parts and its long sums leave up to 6e-5 of the output, six times what a
// plain fp32 computation does; with head_dim 512 that attention runs on the CUDA cores
// (8192 keys, 8/2 heads, 256 / 1024 rows: 3456 / 6847 us against 101 / 366).
How prefill_how(int64_t T, int64_t keys, int H, int Hkv, int D, int dtype, int num_sms) {
  const int64_t rows = T * (H / Hkv);
  if (dtype == PFA_F32) return How::kDecode;
  if (D == 128) {
    if (rows <= 48) return How::kDecode;
    return rows <= 256 || (rows <= 768 && keys >= 16384) ? How::kCodes : How::kReadBack;
  }
  // A wave of tiles costs what the decode kernel takes for this many rows of one kv head.
  const int64_t blocks = (rows + 255) / 256 * 4 * Hkv;
  return rows * Hkv <= 1150 * ((blocks + num_sms - 1) / num_sms) ? How::kDecode : How::kReadBack;
}

int prefill_plan(int64_t T, int64_t start_pos, int H, int Hkv, int D, int window, float scale,
                 int dtype, int64_t qkv_dim, int num_sms, void* stream, PrefillPlan* p) {
  // a window of all keys is none, and the kernels' 32-bit positions stay in range
  if (window < 0 || window >= start_pos + T) window = 0;
  p->window = window;
  p->how = prefill_how(T, window > 0 ? std::min<int64_t>(start_pos + T, window + T) : start_pos + T,
                       H, Hkv, D, dtype, num_sms);
  if (p->how == How::kDecode) {
    p->total = decode_q8_workspace(T, H, Hkv, D, dtype, num_sms);
    return PFA_OK;
  }
  if (p->how == How::kCodes) {
    if (T * H >= (int64_t)1 << 30) return PFA_ERR_SHAPE;   // 32-bit rows; its q takes 256 GB
    p->total = q8_d128_workspace(T, start_pos, H, Hkv, window, num_sms);
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
  p->call.ws_bytes = workspace_bytes_bf16(p->call);
  p->total = p->ws_at + round256(p->call.ws_bytes);
  return PFA_OK;
}

}  // namespace
}  // namespace pfa

using namespace pfa;

extern "C" {

int pfa_qk_norm_rope(const void* q, const void* k, void* q_out, void* k_out, int64_t B, int64_t T,
                     int64_t start_pos, const int64_t* lengths, int num_heads, int num_kv_heads,
                     int head_dim, const void* q_weight, const void* k_weight, float eps,
                     float weight_offset, const double* inv_freq, int rot_dim, int interleaved,
                     int dtype, int64_t q_stride, int64_t k_stride, int64_t q_out_stride,
                     int64_t k_out_stride, int64_t k_out_head_stride, void* stream) {
  if (dtype != PFA_F32 && dtype != PFA_BF16) return PFA_ERR_DTYPE;
  if (num_heads <= 0 || num_kv_heads <= 0 || num_heads > 65536 || num_kv_heads > 65536)
    return PFA_ERR_SHAPE;
  if (head_dim <= 0 || head_dim > 512 || head_dim % 16 != 0) return PFA_ERR_SHAPE;
  if (rot_dim < 0 || rot_dim > head_dim || rot_dim % 16 != 0) return PFA_ERR_SHAPE;
  int rc = check_span(B, T, start_pos, lengths);
  if (rc != PFA_OK) return rc;
  if (!std::isfinite(eps) || eps < 0.f || !std::isfinite(weight_offset)) return PFA_ERR_VALUE;
  if (B == 0 || T == 0) return PFA_OK;
  if (!q || !k || !q_out || !k_out || (rot_dim > 0 && !inv_freq)) return PFA_ERR_NULL;
  const int64_t n = B * T, es = (int64_t)elem(dtype), D = head_dim;
  const int64_t wq = num_heads * D, wk = num_kv_heads * D;
  if (q_stride < wq || k_stride < wk || q_out_stride < wq || k_out_head_stride < D)
    return PFA_ERR_SHAPE;
  // k_out: heads inside a token's row, or tokens inside a head's rows (a cache)
  const bool k_token_major = k_out_stride >= (num_kv_heads - 1) * k_out_head_stride + D;
  const bool k_head_major = k_out_stride >= D && k_out_head_stride >= (n - 1) * k_out_stride + D;
  if (!k_token_major && !k_head_major) return PFA_ERR_SHAPE;
  if ((q_stride * es) % 16 || (k_stride * es) % 16 || (q_out_stride * es) % 16 ||
      (k_out_stride * es) % 16 || (k_out_head_stride * es) % 16)
    return PFA_ERR_ALIGNMENT;
  if (misaligned(q, 16) || misaligned(k, 16) || misaligned(q_out, 16) || misaligned(k_out, 16) ||
      misaligned(q_weight, 16) || misaligned(k_weight, 16) || misaligned(inv_freq, 8))
    return PFA_ERR_ALIGNMENT;
  const Rows rq{q, n, (size_t)(q_stride * es), (size_t)(wq * es)};
  const Rows rk{k, n, (size_t)(k_stride * es), (size_t)(wk * es)};
  const Rows oq{q_out, n, (size_t)(q_out_stride * es), (size_t)(wq * es)};
  Rows ok{k_out, n, (size_t)(k_out_stride * es), (size_t)(wk * es)};
  const bool k_rows = k_out_head_stride == D && k_token_major;
  if (!k_rows) {  // one span over all of it
    ok.n = 1;
    ok.width = (size_t)(((num_kv_heads - 1) * k_out_head_stride + (n - 1) * k_out_stride + D) * es);
    ok.pitch = ok.width;
  }
  const bool q_in_place = q_out == q && q_out_stride == q_stride;
  const bool k_in_place = k_out == k && k_rows && k_out_stride == k_stride;
  if ((!q_in_place && share(oq, rq)) || share(oq, rk) || share(oq, ok) ||
      (!k_in_place && share(ok, rk)) || share(ok, rq))
    return PFA_ERR_ALIAS;
  const size_t wbytes = (size_t)(D * es), fbytes = (size_t)rot_dim / 2 * sizeof(double);
  const Rows outs[] = {oq, ok};
  for (const Rows& o : outs)
    if ((q_weight && overlaps(o.p, o.span(), q_weight, wbytes)) ||
        (k_weight && overlaps(o.p, o.span(), k_weight, wbytes)) ||
        (rot_dim && overlaps(o.p, o.span(), inv_freq, fbytes)) ||
        (lengths && overlaps(o.p, o.span(), lengths, (size_t)B * 8)))
      return PFA_ERR_ALIAS;
  DeviceInfo d;
  if ((rc = current_device(&d)) != kOk) return rc;
  const void* used[] = {q, k, q_out, k_out, q_weight, k_weight, rot_dim ? inv_freq : nullptr,
                        lengths};
  for (const void* p : used)
    if (p && !device_accessible(p, d.device)) return PFA_ERR_DEVICE;
  NormRopeCall c;
  c.q = q; c.k = k; c.q_out = q_out; c.k_out = k_out;
  c.span = Span{B, T, start_pos, lengths};
  c.H = num_heads; c.Hkv = num_kv_heads; c.D = head_dim;
  c.q_weight = q_weight; c.k_weight = k_weight;
  c.eps = eps; c.weight_offset = weight_offset;
  c.inv_freq = inv_freq; c.rot_dim = rot_dim; c.interleaved = interleaved ? 1 : 0;
  c.dtype = dtype;
  c.q_row = q_stride; c.k_row = k_stride; c.q_out_row = q_out_stride;
  c.k_out_row = k_out_stride; c.k_out_head = k_out_head_stride;
  c.err = d.err;
  c.num_sms = d.num_sms;
  c.stream = static_cast<cudaStream_t>(stream);
  return launch_norm_rope(c);
}

int pfa_cache_write_q8(const void* k, const void* v, void* k8, void* v8, float* k_scale,
                       float* v_scale, int64_t B, int64_t T, int64_t start_pos,
                       const int64_t* lengths, int num_kv_heads, int head_dim,
                       int64_t max_seq_len, int block, int dtype, int64_t k_stride,
                       int64_t v_stride, void* stream) {
  if (dtype != PFA_F32 && dtype != PFA_BF16) return PFA_ERR_DTYPE;
  if (num_kv_heads <= 0 || num_kv_heads > 65536) return PFA_ERR_SHAPE;
  int rc = check_span(B, T, start_pos, lengths);
  if (rc != PFA_OK) return rc;
  if ((rc = check_cache(B * num_kv_heads, head_dim, max_seq_len, block)) != PFA_OK) return rc;
  if (T > max_seq_len || (!lengths && start_pos + T > max_seq_len)) return PFA_ERR_SHAPE;
  if (B == 0 || T == 0) return PFA_OK;
  if (!k || !v) return PFA_ERR_NULL;
  WriteQ8Call c;
  c.cache = CacheQ8{k8, v8, k_scale, v_scale, max_seq_len, block};
  if ((rc = check_cache_pointers(c.cache)) != PFA_OK) return rc;
  const int64_t es = (int64_t)elem(dtype), width = (int64_t)num_kv_heads * head_dim;
  if (k_stride < width || v_stride < width) return PFA_ERR_SHAPE;
  if ((k_stride * es) % 16 || (v_stride * es) % 16 || misaligned(k, 16) || misaligned(v, 16))
    return PFA_ERR_ALIGNMENT;
  const int64_t heads = B * num_kv_heads;
  const size_t codes = (size_t)heads * max_seq_len * head_dim;
  const size_t scales = (size_t)heads * (max_seq_len / block) * sizeof(float);
  const Rows rk{k, B * T, (size_t)(k_stride * es), (size_t)(width * es)};
  const Rows rv{v, B * T, (size_t)(v_stride * es), (size_t)(width * es)};
  if (cache_shares(c.cache, heads, head_dim, k, rk.span()) ||
      cache_shares(c.cache, heads, head_dim, v, rv.span()) || overlaps(k8, codes, v8, codes) ||
      overlaps(k8, codes, k_scale, scales) || overlaps(k8, codes, v_scale, scales) ||
      overlaps(v8, codes, k_scale, scales) || overlaps(v8, codes, v_scale, scales) ||
      overlaps(k_scale, scales, v_scale, scales) ||
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
  return launch_cache_write_q8(c);
}

int pfa_cache_read_q8(const void* k8, const void* v8, const float* k_scale, const float* v_scale,
                      void* k_out, void* v_out, int64_t heads, int64_t start, int64_t rows,
                      int head_dim, int64_t max_seq_len, int block, int dtype,
                      int64_t out_head_stride, void* stream) {
  if (dtype != PFA_F32 && dtype != PFA_BF16) return PFA_ERR_DTYPE;
  int rc = check_cache(heads, head_dim, max_seq_len, block);
  if (rc != PFA_OK) return rc;
  if (heads > kMaxLen || start < 0 || rows < 0 || start > max_seq_len ||
      rows > max_seq_len - start)
    return PFA_ERR_SHAPE;
  if (heads == 0 || rows == 0) return PFA_OK;
  ReadQ8Call c;
  c.cache = cache_of(k8, v8, k_scale, v_scale, max_seq_len, block);
  if ((rc = check_cache_pointers(c.cache)) != PFA_OK) return rc;
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
  return launch_cache_read_q8(c);
}

int pfa_decode_workspace_bytes_q8(int64_t B, int64_t T, int num_heads, int num_kv_heads,
                                  int head_dim, int dtype, size_t* bytes) {
  if (!bytes) return PFA_ERR_NULL;
  *bytes = 0;
  int rc = check_attention(B, T, num_heads, num_kv_heads, head_dim, 1.f, dtype);
  if (rc != PFA_OK) return rc;
  if (B > kMaxLen || T > kMaxLen || T * (num_heads / num_kv_heads) > PFA_DECODE_MAX_ROWS)
    return PFA_ERR_SHAPE;
  if (B == 0 || T == 0) return PFA_OK;
  DeviceInfo d;
  if ((rc = current_device(&d)) != kOk) return rc;
  *bytes = decode_q8_workspace(T, num_heads, num_kv_heads, head_dim, dtype, d.num_sms);
  return PFA_OK;
}

int pfa_decode_attention_q8(const void* q, const void* k8, const void* v8, const float* k_scale,
                            const float* v_scale, void* out, int64_t B, int64_t T,
                            const int64_t* lengths, int num_heads, int num_kv_heads, int head_dim,
                            int window, float scale, int dtype, int64_t q_stride,
                            int64_t out_stride, int64_t max_seq_len, int block, void* workspace,
                            size_t workspace_bytes, void* stream) {
  int rc = check_attention(B, T, num_heads, num_kv_heads, head_dim, scale, dtype);
  if (rc != PFA_OK) return rc;
  if (B > kMaxLen || T > kMaxLen || T * (num_heads / num_kv_heads) > PFA_DECODE_MAX_ROWS)
    return PFA_ERR_SHAPE;
  if ((rc = check_cache(B * num_kv_heads, head_dim, max_seq_len, block)) != PFA_OK) return rc;
  if (B == 0 || T == 0) return PFA_OK;
  if (!lengths) return PFA_ERR_NULL;
  if ((rc = check_span(B, T, 0, lengths)) != PFA_OK) return rc;
  DecodeQ8Call c;
  c.cache = cache_of(k8, v8, k_scale, v_scale, max_seq_len, block);
  if ((rc = check_cache_pointers(c.cache)) != PFA_OK) return rc;
  if (!q || !out) return PFA_ERR_NULL;
  const int64_t es = (int64_t)elem(dtype), width = (int64_t)num_heads * head_dim;
  if (q_stride < width || out_stride < width) return PFA_ERR_SHAPE;
  if ((q_stride * es) % 16 || (out_stride * es) % 16 || misaligned(q, 16) || misaligned(out, 16) ||
      misaligned(workspace, 256))
    return PFA_ERR_ALIGNMENT;
  const int64_t heads = B * num_kv_heads;
  const Rows rq{q, B * T, (size_t)(q_stride * es), (size_t)(width * es)};
  const Rows ro{out, B * T, (size_t)(out_stride * es), (size_t)(width * es)};
  if (share(ro, rq) || cache_shares(c.cache, heads, head_dim, out, ro.span()) ||
      overlaps(out, ro.span(), lengths, (size_t)B * 8))
    return PFA_ERR_ALIAS;
  DeviceInfo d;
  if ((rc = current_device(&d)) != kOk) return rc;
  const size_t need =
      decode_q8_workspace(T, num_heads, num_kv_heads, head_dim, dtype, d.num_sms);
  if (need > 0) {
    if (!workspace || workspace_bytes < need) return PFA_ERR_SCRATCH;
    if (overlaps(workspace, need, q, rq.span()) || overlaps(workspace, need, out, ro.span()) ||
        overlaps(workspace, need, lengths, (size_t)B * 8) ||
        cache_shares(c.cache, heads, head_dim, workspace, need))
      return PFA_ERR_ALIAS;
    if (!device_accessible(workspace, d.device)) return PFA_ERR_DEVICE;
  }
  if (!device_accessible(q, d.device) || !device_accessible(out, d.device) ||
      !device_accessible(lengths, d.device) || !accessible(c.cache, d.device))
    return PFA_ERR_DEVICE;
  c.q = q; c.out = out;
  c.span = Span{B, T, 0, lengths};
  c.H = num_heads; c.Hkv = num_kv_heads; c.D = head_dim;
  // (a window of the whole cache is none, and the kernels' 32-bit positions stay in range)
  c.window = window > 0 && window < max_seq_len ? window : 0;
  c.dtype = dtype; c.scale = scale;
  c.q_row = q_stride; c.out_row = out_stride;
  c.err = d.err; c.num_sms = d.num_sms; c.device = d.device;
  c.wait_limit_ns = d.wait_limit_ns; c.flags = d.flags;
  c.ws = workspace;
  c.stream = static_cast<cudaStream_t>(stream);
  return launch_decode_q8(c);
}

int pfa_prefill_workspace_bytes_q8(int64_t T, int64_t start_pos, int num_heads, int num_kv_heads,
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

int pfa_prefill_attention_q8(const void* q, const void* k8, const void* v8, const float* k_scale,
                             const float* v_scale, void* out, int64_t T, int64_t start_pos,
                             int num_heads, int num_kv_heads, int head_dim, int window,
                             float scale, int dtype, int64_t qkv_dim, int64_t max_seq_len,
                             int block, void* workspace, size_t workspace_bytes, void* stream) {
  int rc = check_attention(1, T, num_heads, num_kv_heads, head_dim, scale, dtype);
  if (rc != PFA_OK) return rc;
  if ((rc = check_span(1, T, start_pos, nullptr)) != PFA_OK) return rc;
  if ((rc = check_cache(num_kv_heads, head_dim, max_seq_len, block)) != PFA_OK) return rc;
  if (start_pos + T > max_seq_len) return PFA_ERR_SHAPE;
  if (T == 0) return PFA_OK;
  const CacheQ8 cache = cache_of(k8, v8, k_scale, v_scale, max_seq_len, block);
  if ((rc = check_cache_pointers(cache)) != PFA_OK) return rc;
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
  if (plan.total > 0) {
    if (!workspace || workspace_bytes < plan.total) return PFA_ERR_SCRATCH;
    if (overlaps(workspace, plan.total, q, rq.span()) ||
        overlaps(workspace, plan.total, out, ro.span()) ||
        cache_shares(cache, num_kv_heads, head_dim, workspace, plan.total))
      return PFA_ERR_ALIAS;
    if (!device_accessible(workspace, d.device)) return PFA_ERR_DEVICE;
  }
  if (!device_accessible(q, d.device) || !device_accessible(out, d.device) ||
      !accessible(cache, d.device))
    return PFA_ERR_DEVICE;
  if (plan.how != How::kReadBack) {
    DecodeQ8Call c;
    c.q = q; c.out = out; c.cache = cache;
    c.span = Span{1, T, start_pos, nullptr};
    c.H = num_heads; c.Hkv = num_kv_heads; c.D = head_dim;
    c.window = plan.window; c.dtype = dtype; c.scale = scale;
    c.q_row = qkv_dim; c.out_row = qkv_dim;
    c.err = d.err; c.num_sms = d.num_sms; c.device = d.device;
    c.wait_limit_ns = d.wait_limit_ns; c.flags = d.flags;
    c.ws = workspace;
    c.stream = static_cast<cudaStream_t>(stream);
    return plan.how == How::kDecode ? launch_decode_q8(c) : launch_q8_d128(c);
  }
  char* base = static_cast<char*>(workspace);
  ReadQ8Call r;
  r.cache = cache;
  r.k_out = base; r.v_out = base + plan.v_at;
  r.heads = num_kv_heads; r.start = plan.lo; r.rows = plan.rows;
  r.out_head = plan.rows * head_dim;
  r.D = head_dim; r.dtype = PFA_BF16;
  r.stream = static_cast<cudaStream_t>(stream);
  if ((rc = launch_cache_read_q8(r)) != kOk) return rc;
  plan.call.q = q; plan.call.out = out;
  plan.call.k = r.k_out; plan.call.v = r.v_out;
  plan.call.ws = plan.call.ws_bytes ? base + plan.ws_at : nullptr;
  return dispatch(plan.call, PFA_BF16);
}

}  // extern "C"
