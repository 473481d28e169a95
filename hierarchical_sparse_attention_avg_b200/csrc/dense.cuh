// dense.cuh — sizes, masks and distance buckets shared by the dense stage's attention kernels (lh_attn_*).
//
// Row i of a batch entry sits at position x = len - Sq + i behind its len valid keys; key j at position j.  A row sees
// the keys j < len with j <= x (causal) or j < prefix, of its own document; a row with x < 0 or a negative document
// id, and a key with j >= len or a negative id, take part in no pair (they are "dead": whatever memory holds there
// reaches no result).
#pragma once

#include "internal.h"

namespace lh {

constexpr int kMaxBuckets = 128;       // columns of the bias table
constexpr int kMaxDenseKeys = 1 << 20; // keys per head (one flag byte per 128-key tile in shared memory)
constexpr int kKeyTile = 128;

// First distance of every bucket of one direction: buckets 0 .. n/2 - 1 hold one distance each, the rest grow
// logarithmically up to `distance`, the last one holds everything beyond.
struct BucketStarts {
  int n;     // buckets of one direction
  int both;  // keys after the row have n further buckets of their own
  int start[kMaxBuckets];
};

// Bucket of the distance delta = x - j (the last bucket whose first distance is <= its size).
__host__ __device__ __forceinline__ int bucket_of(const BucketStarts& s, int delta) {
  const int size = s.both ? (delta < 0 ? -delta : delta) : (delta < 0 ? 0 : delta);
  int lo = 0, hi = s.n;  // start[lo] <= size < start[hi]
  while (hi - lo > 1) {
    const int m = (lo + hi) >> 1;
    if (s.start[m] <= size) lo = m; else hi = m;
  }
  return s.both && delta < 0 ? lo + s.n : lo;
}

struct Strides {
  int64_t b, h, s;  // elements
};

// One call, by value to the kernels.
struct DenseDims {
  int B, Hq, Hkv, G, Sq, Skv, d;
  int f16;  // operands fp16 (else bf16)
  int causal;
  int buckets, near;  // table columns; distances of magnitude >= near share the end buckets
  float scale, cap;
  const float* slopes;
  const void* table;
  const int32_t* docs;
  const int32_t* prefix;
  const int32_t* kv_len;
  int* status;
};

__device__ __forceinline__ int dense_len(const DenseDims& a, int b) {
  return a.kv_len ? min(max(__ldg(a.kv_len + b), 0), a.Skv) : a.Skv;
}
__device__ __forceinline__ int dense_prefix(const DenseDims& a, int b, int len) {
  return a.prefix ? min(__ldg(a.prefix + b), len) : 0;
}
// Last key position that a row at x may see (-1: none); its own document apart.
__device__ __forceinline__ int last_key(const DenseDims& a, int x, int len, int prefix) {
  if (x < 0) return -1;
  return a.causal ? min(max(x, prefix - 1), len - 1) : len - 1;
}
// Document of position x; -1 where there is no valid position.
__device__ __forceinline__ int doc_at(const DenseDims& a, int b, int x, int len) {
  if (x < 0 || x >= len) return -1;
  return a.docs ? __ldg(a.docs + (int64_t)b * a.Skv + x) : 0;
}
// Whether two ranges of ids can have a common document, and whether both are one and the same document.
__device__ __forceinline__ bool docs_meet(int2 p, int2 q) { return p.x <= q.y && q.x <= p.y && p.y >= 0 && q.y >= 0; }
__device__ __forceinline__ bool docs_one(int2 p, int2 q) { return p.x == p.y && q.x == q.y && p.x == q.x && p.x >= 0; }

// tanh from one exponential and one reciprocal: |error| <= about 2e-7, where the hardware's tanh has 5e-4 (times a cap
// of 50: a score off by 0.02, more than the operands' own rounding gives).
__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

template <bool F16>
__device__ __forceinline__ uint32_t pack2_rn(float lo, float hi) {
  return F16 ? pack_half2_rn(lo, hi) : pack_bf16x2_rn(lo, hi);
}
template <bool F16>
__device__ __forceinline__ float2 unpack2(uint32_t w) {
  if (F16) return __half22float2(*reinterpret_cast<const __half2*>(&w));
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}
template <bool F16>
__device__ __forceinline__ float table_at(const void* t, int64_t i) {
  const uint32_t w = __ldg(static_cast<const unsigned short*>(t) + i);
  return F16 ? __half2float(__ushort_as_half((unsigned short)w)) : __uint_as_float(w << 16);
}
// Bits set where one of the two 16-bit values of w is not finite.
template <bool F16>
__device__ __forceinline__ uint32_t nonfinite2(uint32_t w) {
  return F16 ? (((w & 0x7C007C00u) + 0x04000400u) & 0x80008000u) : (((w & 0x7F807F80u) + 0x00800080u) & 0x80008000u);
}

// o's 16-bit row chunk of 8 features, and what its rounding dropped (low may be null).
template <bool F16>
__device__ __forceinline__ void store8(uint16_t* o, uint16_t* low, const float* v) {
  uint32_t w[4], r[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    w[i] = pack2_rn<F16>(v[2 * i], v[2 * i + 1]);
    const float2 u = unpack2<F16>(w[i]);
    r[i] = pack2_rn<F16>(v[2 * i] - u.x, v[2 * i + 1] - u.y);
  }
  st16(o, make_uint4(w[0], w[1], w[2], w[3]));
  if (low) st16(low, make_uint4(r[0], r[1], r[2], r[3]));
}

// ---- launches (each in the file it names) ----------------------------------------------------------------
// A [B,H,S,d] tensor with unit feature stride.
struct DenseTensor {
  const void* p;
  Strides st;
};
struct DenseFwdPlan {
  int pack;    // query heads of one key head that share a query tile (a divisor of G)
  int tok;     // tokens of a 128-row query tile
  int ntile;   // query tiles per (batch, head group)
  int dual;    // one query tile per block, its keys in two interleaved streams
  int nsplit;  // blocks that share one query tile's keys
};
DenseFwdPlan dense_fwd_plan(const DenseDims& a);
// dense_prep.cu: ids' range (min, max) of every key tile: kdoc [B][ceil(Skv / 128)]; with qdoc, of every 64-row
// sub-tile of the queries too: qdoc [B][ceil(Sq / 64)].
int launch_dense_doc_ranges(const DenseDims& a, int2* kdoc, int2* qdoc, cudaStream_t st);
// dense_fwd.cu: low.p may be null; part_o / part_lse: nsplit > 1 only.
int launch_dense_fwd(const DenseDims& a, const BucketStarts& bs, const DenseTensor& q, const DenseTensor& k,
                     const DenseTensor& v, const DenseTensor& o, const DenseTensor& low, float* lse, const int2* kdoc,
                     float* part_o, float* part_lse, cudaStream_t st);

// Backward: workspace buffers.
struct DenseBwdBuf {
  float* stats;         // [2][B Hq][Sq rounded up to 4]: -LSE log2(e) (fp16: + 12; -inf for a dead row), -D
  unsigned int* amax;   // [B Hkv][2] bits of the largest |dO_i| and |V_j| (fp16 only; zeroed by the caller)
  float* dqacc;         // fp32 [B Hq][Sq][d]
  float* dkv;           // fp32 [shares][dV, dK][B Hkv][Skv][d], where the query heads of a key head are shared out
  const int2 *kdoc, *qdoc;
  float* bias;          // [Hq][2 near + 1] log2(e) table[h][bucket(delta)], delta = -near .. near
  uint8_t* bucket;      // [2 near + 1]
  int2* range;          // [buckets] first and last delta of each bucket
  float* dtpart;        // [B Hkv][key tiles][G][8 warps][buckets]
};
// Blocks that the query heads of one key head are shared out over (dense_bwd.cu).
int dense_bwd_shares(const DenseDims& a);
int launch_dense_bwd(const DenseDims& a, const DenseTensor& q, const DenseTensor& k, const DenseTensor& v,
                     const DenseTensor& dout, const DenseTensor& dk, const DenseTensor& dv, const DenseBwdBuf& w,
                     cudaStream_t st);
// dense_prep.cu: the rows' statistics, dqacc = 0 and (fp16) the largest norms; the bias by distance; the results.
int launch_dense_bwd_rows(const DenseDims& a, const DenseTensor& o, const DenseTensor& low, const DenseTensor& dout,
                          const DenseTensor& v, const float* lse, const DenseBwdBuf& w, cudaStream_t st);
int launch_dense_bias(const DenseDims& a, const BucketStarts& bs, const DenseBwdBuf& w, cudaStream_t st);
int launch_dense_bwd_out(const DenseDims& a, const DenseTensor& dq, const DenseTensor& dk, const DenseTensor& dv,
                         void* dtable, const DenseBwdBuf& w, cudaStream_t st);
// Device status word of the current device (api.cu).
int device_status(int** out);
// 16-bit tensor map over a strided [B,H,S,d] tensor: box {64, pack, rows, 1, 1} of (d, pack, S, H / pack, B).
int make_tmap_dense(CUtensorMap* map, const DenseTensor& t, int d, int S, int H, int B, int pack, int box_rows);

}  // namespace lh
