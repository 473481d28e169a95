// dense_api.cu — the C ABI of the dense stage's attention (lh_attn_*): validation, sizes, workspace layout and the
// launch sequences.  Semantics are documented in include/lh.h.
#include <math.h>
#include <string.h>

#include "dense.cuh"

namespace lh {
namespace {

constexpr float kMinCap = 0x1p-80f, kMaxCap = 0x1p80f;
constexpr size_t kAlign = 256;
inline size_t align_up(size_t x) { return (x + kAlign - 1) & ~(kAlign - 1); }
inline bool aligned16(const void* p) { return p && ((uintptr_t)p & 15u) == 0; }
inline bool aligned4(const void* p) { return ((uintptr_t)p & 3u) == 0; }

int validate(const lh_attn_params* P) {
  if (!P) return LH_ERR_INVALID_ARG;
  if (P->B < 1 || P->Hq < 1 || P->Hkv < 1 || P->Sq < 1 || P->Skv < 1 || P->d < 1 || P->Hq % P->Hkv)
    return LH_ERR_INVALID_ARG;
  if ((P->dtype != LH_BF16 && P->dtype != LH_FP16) || (P->causal & ~1) || (P->bidirectional & ~1))
    return LH_ERR_INVALID_ARG;
  if (!(P->scale > 0.f) || !(P->softcap >= 0.f) || isinf(P->scale) || isinf(P->softcap)) return LH_ERR_INVALID_ARG;
  if (P->buckets) {
    if (P->buckets < 2 || P->buckets > LH_MAX_BUCKETS) return LH_ERR_INVALID_ARG;
    if (P->bidirectional && (P->buckets < 4 || P->buckets % 2)) return LH_ERR_INVALID_ARG;
    const int n = P->bidirectional ? P->buckets / 2 : P->buckets;
    if (P->max_distance <= n / 2) return LH_ERR_INVALID_ARG;
  }
  if (P->d != 64 && P->d != 128) return LH_ERR_UNSUPPORTED;
  if ((int64_t)P->B * P->Hq > 65535 || P->Skv > kMaxDenseKeys) return LH_ERR_UNSUPPORTED;
  if ((int64_t)P->B * P->Hq * P->Sq > INT32_MAX) return LH_ERR_UNSUPPORTED;
  return LH_OK;
}

// First sizes of the buckets.  The border of bucket b is e (D / e)^((b - e) / (n - e)); in 64-bit mantissas its error is
// far below the distance of a border that is not whole from the next whole number, so one within 1e-15 of a whole
// number is that number.
void bucket_starts(const lh_attn_params& P, BucketStarts* s) {
  memset(s, 0, sizeof(*s));
  if (!P.buckets) return;
  s->both = P.bidirectional;
  s->n = P.bidirectional ? P.buckets / 2 : P.buckets;
  const int e = s->n / 2;
  for (int b = 0; b < s->n; ++b) {
    if (b < e) { s->start[b] = b; continue; }
    const long double x = e * powl((long double)P.max_distance / e, (long double)(b - e) / (s->n - e));
    const long double near = roundl(x);
    s->start[b] = (int)(fabsl(x - near) <= 1e-15L * x ? near : ceill(x));
  }
}

// The sizes that the launches and the workspace go by.
void dense_sizes(const lh_attn_params& P, DenseDims* a, BucketStarts* bs) {
  memset(a, 0, sizeof(*a));
  a->B = P.B; a->Hq = P.Hq; a->Hkv = P.Hkv; a->G = P.Hq / P.Hkv; a->Sq = P.Sq; a->Skv = P.Skv; a->d = P.d;
  a->buckets = P.buckets;
  bucket_starts(P, bs);
  if (P.buckets) {  // beyond the last bucket's first size, and beyond the longest distance, nothing changes
    const int64_t longest = (int64_t)P.Skv + P.Sq;
    a->near = bs->start[bs->n - 1];
    if (a->near > longest) a->near = (int)longest;
  }
}

int make_dense(const lh_attn_params* P, const lh_attn_mods* M, DenseDims* a, BucketStarts* bs) {
  const int rc = validate(P);
  if (rc) return rc;
  static const lh_attn_mods none = {};
  if (!M) M = &none;
  dense_sizes(*P, a, bs);
  a->f16 = P->dtype == LH_FP16;
  a->causal = P->causal;
  a->scale = P->scale;
  // scale / cap and cap log2(e) stay normal numbers; scores near or beyond either bound do not tell them from the cap itself
  a->cap = P->softcap > 0.f ? fminf(fmaxf(P->softcap, kMinCap), kMaxCap) : 0.f;
  a->cap_in = a->cap > 0.f ? (float)fmin((double)P->scale / a->cap, (double)kMaxCapIn) : 0.f;
  if ((P->buckets > 0) != (M->table != nullptr) || (M->slopes && M->table)) return LH_ERR_INVALID_ARG;
  if (M->prefix && !P->causal) return LH_ERR_INVALID_ARG;
  if (!aligned4(M->slopes) || !aligned4(M->docs) || !aligned4(M->prefix) || !aligned4(M->kv_len) ||
      ((uintptr_t)M->table & 1u))
    return LH_ERR_INVALID_ARG;
  a->slopes = M->slopes; a->table = M->table; a->docs = M->docs; a->prefix = M->prefix; a->kv_len = M->kv_len;
  return LH_OK;
}

// Checks a tensor and takes its strides (a dimension of one gets those of a contiguous tensor).
bool take(const lh_tensor* t, int B, int H, int S, int d, DenseTensor* out) {
  if (!t || !aligned16(t->ptr)) return false;
  const int64_t lim = int64_t(1) << 38;  // the tensor map's strides are below 2^40 bytes
  const int64_t st[3] = {B > 1 ? t->stride_b : (int64_t)d, H > 1 ? t->stride_h : (int64_t)d, S > 1 ? t->stride_s : (int64_t)d};
  for (int64_t v : st)
    if (v <= 0 || v % 8 || v > lim) return false;
  out->p = t->ptr;
  out->st = Strides{st[0], st[1], st[2]};
  return true;
}

struct DenseWs {
  size_t kdoc, part_o, part_lse, fwd_total;
  size_t qdoc, stats, amax, dqacc, dkv, bias, bucket, range, dtpart, bwd_total;
};
DenseWs dense_ws(const DenseDims& a) {
  DenseWs w;
  const size_t nk = (a.Skv + kKeyTile - 1) / kKeyTile, bhq = (size_t)a.B * a.Hq, bhk = (size_t)a.B * a.Hkv;
  const DenseFwdPlan f = dense_fwd_plan(a);
  const size_t rows = f.nsplit > 1 ? f.nsplit * bhq * a.Sq : 0;
  size_t o = 0;
  auto take = [&](size_t bytes) {
    const size_t at = o;
    o = align_up(o + bytes);
    return at;
  };
  w.kdoc = take(a.B * nk * sizeof(int2));
  w.part_o = take(rows * a.d * 4);
  w.part_lse = take(rows * 4);
  w.fwd_total = o;
  o = w.part_o;
  w.qdoc = take(a.B * (((size_t)a.Sq + 63) / 64) * sizeof(int2));
  w.stats = take(2 * bhq * (((size_t)a.Sq + 3) & ~(size_t)3) * 4);
  w.amax = take(bhk * 8);
  w.dqacc = take(bhq * a.Sq * a.d * 4);
  const int shares = dense_bwd_shares(a);
  w.dkv = take(shares > 1 ? 2 * shares * bhk * a.Skv * a.d * 4 : 0);
  const size_t wide = a.buckets ? 2 * (size_t)a.near + 1 : 0;
  w.bias = take(a.Hq * wide * 4);
  w.bucket = take(wide);
  w.range = take(a.buckets * sizeof(int2));
  w.dtpart = take(bhk * nk * a.G * 8 * a.buckets * 4);
  w.bwd_total = o;
  return w;
}

}  // namespace
}  // namespace lh

using namespace lh;

#define LH_TRY(expr)        \
  do {                      \
    const int rc_ = (expr); \
    if (rc_) return rc_;    \
  } while (0)

extern "C" {

int lh_attn_validate(const lh_attn_params* P) { return validate(P); }

size_t lh_attn_workspace_bytes(const lh_attn_params* P, int backward) {
  if (validate(P)) return 0;
  DenseDims a;
  BucketStarts bs;
  dense_sizes(*P, &a, &bs);
  const DenseWs w = dense_ws(a);
  return backward && w.bwd_total > w.fwd_total ? w.bwd_total : w.fwd_total;
}

int lh_attn_bucket_starts(const lh_attn_params* P, int32_t* starts) {
  if (validate(P) || !P->buckets || !starts) return -1;
  BucketStarts s;
  bucket_starts(*P, &s);
  memcpy(starts, s.start, s.n * sizeof(int32_t));
  return s.n;
}

int lh_attn_forward(const lh_attn_params* P, const lh_attn_mods* M, const lh_tensor* q, const lh_tensor* k,
                    const lh_tensor* v, const lh_tensor* o, const lh_tensor* low, float* lse, void* ws, size_t ws_bytes,
                    void* stream) {
  DenseDims a;
  BucketStarts bs;
  LH_TRY(make_dense(P, M, &a, &bs));
  DenseTensor tq, tk, tv, to, tl = {nullptr, {0, 0, 0}};
  if (!take(q, a.B, a.Hq, a.Sq, a.d, &tq) || !take(k, a.B, a.Hkv, a.Skv, a.d, &tk) ||
      !take(v, a.B, a.Hkv, a.Skv, a.d, &tv) || !take(o, a.B, a.Hq, a.Sq, a.d, &to) ||
      (low && !take(low, a.B, a.Hq, a.Sq, a.d, &tl)) || !lse || !aligned4(lse))
    return LH_ERR_INVALID_ARG;
  const DenseWs w = dense_ws(a);
  if (!aligned16(ws) || ws_bytes < w.fwd_total) return ws ? LH_ERR_WORKSPACE : LH_ERR_INVALID_ARG;
  LH_TRY(device_status(&a.status));
  uint8_t* wsb = static_cast<uint8_t*>(ws);
  cudaStream_t st = (cudaStream_t)stream;
  int2* kdoc = reinterpret_cast<int2*>(wsb + w.kdoc);
  if (a.docs && (a.Skv + kKeyTile - 1) / kKeyTile > kOwnDocTiles) LH_TRY(launch_dense_doc_ranges(a, kdoc, st));
  return launch_dense_fwd(a, bs, tq, tk, tv, to, tl, lse, kdoc,
                          reinterpret_cast<float*>(wsb + w.part_o), reinterpret_cast<float*>(wsb + w.part_lse), st);
}

int lh_attn_backward(const lh_attn_params* P, const lh_attn_mods* M, const lh_tensor* q, const lh_tensor* k,
                     const lh_tensor* v, const lh_tensor* o, const lh_tensor* low, const float* lse,
                     const lh_tensor* dout, const lh_tensor* dq, const lh_tensor* dk, const lh_tensor* dv, void* dtable, void* ws,
                     size_t ws_bytes, void* stream) {
  DenseDims a;
  BucketStarts bs;
  LH_TRY(make_dense(P, M, &a, &bs));
  DenseTensor tq, tk, tv, to, tl = {nullptr, {0, 0, 0}}, tdo, tdq, tdk, tdv;
  if (!take(q, a.B, a.Hq, a.Sq, a.d, &tq) || !take(k, a.B, a.Hkv, a.Skv, a.d, &tk) ||
      !take(v, a.B, a.Hkv, a.Skv, a.d, &tv) || !take(o, a.B, a.Hq, a.Sq, a.d, &to) ||
      (low && !take(low, a.B, a.Hq, a.Sq, a.d, &tl)) || !lse || !aligned4(lse) ||
      !take(dout, a.B, a.Hq, a.Sq, a.d, &tdo) || !take(dq, a.B, a.Hq, a.Sq, a.d, &tdq) ||
      !take(dk, a.B, a.Hkv, a.Skv, a.d, &tdk) || !take(dv, a.B, a.Hkv, a.Skv, a.d, &tdv) ||
      (a.table && (!dtable || ((uintptr_t)dtable & 1u))))
    return LH_ERR_INVALID_ARG;
  const DenseWs w = dense_ws(a);
  if (!aligned16(ws) || ws_bytes < w.bwd_total) return ws ? LH_ERR_WORKSPACE : LH_ERR_INVALID_ARG;
  LH_TRY(device_status(&a.status));
  uint8_t* wsb = static_cast<uint8_t*>(ws);
  cudaStream_t st = (cudaStream_t)stream;
  DenseBwdBuf buf;
  int2 *kdoc = reinterpret_cast<int2*>(wsb + w.kdoc), *qdoc = reinterpret_cast<int2*>(wsb + w.qdoc);
  buf.stats = reinterpret_cast<float*>(wsb + w.stats);
  buf.amax = reinterpret_cast<unsigned int*>(wsb + w.amax);
  buf.dqacc = reinterpret_cast<float*>(wsb + w.dqacc);
  buf.dkv = reinterpret_cast<float*>(wsb + w.dkv);
  buf.kdoc = kdoc;
  buf.qdoc = qdoc;
  buf.bias = reinterpret_cast<float*>(wsb + w.bias);
  buf.bucket = wsb + w.bucket;
  buf.range = reinterpret_cast<int2*>(wsb + w.range);
  buf.dtpart = reinterpret_cast<float*>(wsb + w.dtpart);
  LH_TRY(launch_dense_bwd_prep(a, bs, to, tl, tdo, tv, lse, buf, kdoc, qdoc, st));
  LH_TRY(launch_dense_bwd(a, tq, tk, tv, tdo, tdk, tdv, buf, st));
  return launch_dense_bwd_out(a, tdq, tdk, tdv, dtable, buf, st);
}

}  // extern "C"
