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
constexpr float kMaxCapIn = 0x1p100f;  // (a score of zero times it is zero, any other one is at the cap)
// Up to this many key tiles the forward's blocks take the ids' ranges of the tiles themselves (a few loads a warp);
// beyond it they come from a launch of their own.
constexpr int kOwnDocTiles = 32;

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
  float scale, cap, cap_in;  // cap_in: scale / cap, at most kMaxCapIn
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
  return a.prefix ? min(max(__ldg(a.prefix + b), 0), len) : 0;
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
// Ids of a run of positions: x the smallest and y the largest (-1: none) among its live ones; x is complemented (and so
// negative) where some position is dead.
__device__ __forceinline__ int2 id_range(int lo, int hi, bool dead) { return make_int2(dead ? ~lo : lo, hi); }
// That of positions x0 .. x0 + n - 1, in every lane of a warp.
__device__ __forceinline__ int2 warp_doc_range(const DenseDims& a, int b, int x0, int n, int len, int lane) {
  int lo = INT32_MAX, hi = -1;
  bool dead = false;
  for (int i = lane; i < n; i += 32) {
    const int id = doc_at(a, b, x0 + i, len);
    if (id < 0) dead = true;
    else lo = min(lo, id), hi = max(hi, id);
  }
  return id_range(__reduce_min_sync(0xffffffffu, lo), __reduce_max_sync(0xffffffffu, hi),
                  __any_sync(0xffffffffu, dead));
}
// Whether two runs can have a common document, and whether both are wholly of one and the same document.
__device__ __forceinline__ bool docs_meet(int2 p, int2 q) {
  return (p.x < 0 ? ~p.x : p.x) <= q.y && (q.x < 0 ? ~q.x : q.x) <= p.y;
}
__device__ __forceinline__ bool docs_one(int2 p, int2 q) { return p.x == p.y && q.x == q.y && p.x == q.x; }
// Bit i: position of lane i has this lane's document (`other` and `mine`: their ids; one document after the other).
__device__ __forceinline__ uint32_t same_doc(int other, int mine) {
  uint32_t todo = __ballot_sync(0xffffffffu, mine >= 0), same = 0;
#pragma unroll 1
  while (todo) {
    const int doc = __shfl_sync(0xffffffffu, mine, __ffs(todo) - 1);
    const uint32_t m = __ballot_sync(0xffffffffu, other == doc);
    if (mine == doc) same = m;
    todo &= ~__ballot_sync(0xffffffffu, mine == doc);
  }
  return same;
}

// tanh with an error that goes by its own value (about 1e-6 of it), so that a score's does not go by the cap (the
// hardware's tanh has 5e-4 absolute: times a cap of 50 a score off by 0.02, more than the operands' own rounding gives).
// Small arguments take an odd polynomial x p(x^2), p fitted to tanh(x) / x for the least relative error (weighted least
// squares, the weights raised where the error was large): 3 coefficients on [0, 1/4] 5.0e-7, 4 on [0, 1/2] 6.2e-7, 8 on
// [0, 5/4] 1.8e-7, rounding included.  Beyond 1/4 the form by the exponential, some 1e-7 off, is as good; below it that
// form's difference from 1 loses digits: 1e-2 of a score at a cap of 1e5, and 1.3e-5 at most up to a cap of 64, where the
// forward does without the second form (Careful false; 617 against 827 us at 16 heads of 8,192 keys with many scores beyond
// a cap of 20).  Where a warp's arguments are all small (scores below the cap, nearly always), the polynomials run on pairs:
// 6 or 10 packed FMAs, against two exponentials and two reciprocals, whose pipe the softmax itself fills.
__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
constexpr float kCarefulCap = 64.f;
template <bool Careful>
__device__ __forceinline__ float tanh_any(float x) {
  const float far = fmaf(-2.f, rcp_approx(1.f + ex2(x * (2.f * 1.4426950408889634f))), 1.f);
  if (!Careful) return far;
  const float u = x * x, near = x * fmaf(fmaf(0.128416136f, u, -0.333219081f), u, 0.999999583f);
  return fabsf(x) < 0.25f ? near : far;
}
template <bool Half>
struct TanhPoly {  // f * tanh
  static constexpr int N = Half ? 4 : 8;
  uint64_t c[N];
  __device__ __forceinline__ explicit TanhPoly(float f) {
    const float k4[4] = {0.999999464f, -0.333263189f, 0.131902963f, -0.0444022231f};
    const float k8[8] = {0.99999994f, -0.333326995f, 0.133245066f, -0.0534903407f, 0.0205571726f, -0.00679615559f,
                         0.0015881143f, -0.000182598116f};
#pragma unroll
    for (int i = 0; i < N; ++i) c[i] = f2pack((Half ? k4[i % 4] : k8[i]) * f, (Half ? k4[i % 4] : k8[i]) * f);
  }
};
// f tanh(in v) of 32 values, all of magnitude <= 1/2 (Half) or 5/4 after the scaling.
template <bool Half>
__device__ __forceinline__ void tanh32(float (&v)[32], float in, float f) {
  const TanhPoly<Half> poly(f);
  const uint64_t in2 = f2pack(in, in);
#pragma unroll
  for (int i = 0; i < 32; i += 16) {  // eight pairs side by side: a chain alone would wait for each of its steps
    uint64_t x[8], u[8], y[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = mul_f32x2(f2pack(v[i + 2 * e], v[i + 2 * e + 1]), in2);
#pragma unroll
    for (int e = 0; e < 8; ++e) u[e] = mul_f32x2(x[e], x[e]);
#pragma unroll
    for (int e = 0; e < 8; ++e) y[e] = fma_f32x2(poly.c[TanhPoly<Half>::N - 1], u[e], poly.c[TanhPoly<Half>::N - 2]);
#pragma unroll
    for (int k = TanhPoly<Half>::N - 3; k >= 0; --k)
#pragma unroll
      for (int e = 0; e < 8; ++e) y[e] = fma_f32x2(y[e], u[e], poly.c[k]);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const uint64_t t = mul_f32x2(y[e], x[e]);
      v[i + 2 * e] = f2lo(t);
      v[i + 2 * e + 1] = f2hi(t);
    }
  }
}
// The smaller one; NaN if either is.
__device__ __forceinline__ float min_nan(float a, float b) {
  float r;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
// Largest magnitude of 32 values against m.
__device__ __forceinline__ float absmax32(const float (&v)[32], float m) {
  float a = m, b = 0.f, c = 0.f, d = 0.f;
#pragma unroll
  for (int i = 0; i < 32; i += 8) {
    a = fmax3(a, fabsf(v[i]), fabsf(v[i + 1]));
    b = fmax3(b, fabsf(v[i + 2]), fabsf(v[i + 3]));
    c = fmax3(c, fabsf(v[i + 4]), fabsf(v[i + 5]));
    d = fmax3(d, fabsf(v[i + 6]), fabsf(v[i + 7]));
  }
  return fmaxf(fmaxf(a, b), fmaxf(c, d));
}

// 5-D tiled TMA load (no multicast) into shared memory, completion counted on `bar`.
__device__ __forceinline__ void tma_load_5d(uint32_t dst, const CUtensorMap* map, uint32_t bar, int c0, int c1,
                                            int c2, int c3, int c4) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5, %6, %7}], "
      "[%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(c4)
      : "memory");
}

// 5-D tiled TMA store of a shared-memory box; completion tracked by bulk groups.
__device__ __forceinline__ void tma_store_5d(const CUtensorMap* map, uint32_t src, int c0, int c1, int c2, int c3, int c4) {
  asm volatile(
      "cp.async.bulk.tensor.5d.global.shared::cta.bulk_group [%0, {%2, %3, %4, %5, %6}], [%1];" ::"l"(
          reinterpret_cast<uint64_t>(map)),
      "r"(src), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(c4)
      : "memory");
}

__device__ __forceinline__ uint64_t add_f32x2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
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
// The larger magnitude of each of two 16-bit values (signs as they come), NaN if either is: nonfinite2 of it tells whether one
// of them is not finite, at one instruction a word.
template <bool F16>
__device__ __forceinline__ uint32_t absmax2(uint32_t a, uint32_t b) {
  uint32_t r;
  if (F16) asm("max.NaN.xorsign.abs.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  else asm("max.NaN.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// 8 features as 16-bit values, and what the rounding dropped.
template <bool F16>
__device__ __forceinline__ uint4 round8(const float* v, uint4* low) {
  uint32_t w[4], r[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    w[i] = pack2_rn<F16>(v[2 * i], v[2 * i + 1]);
    const float2 u = unpack2<F16>(w[i]);
    r[i] = pack2_rn<F16>(v[2 * i] - u.x, v[2 * i + 1] - u.y);
  }
  *low = make_uint4(r[0], r[1], r[2], r[3]);
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// A warp's 32 result rows on their way out, 128 bytes of each at a time, through 4 KB of shared memory: a thread has a row,
// and storing it from there writes 32 rows at 16 bytes apiece (15,000 cycles for a 128 x 128 tile and its low half); out of
// shared memory eight lanes write 128 bytes of one row.
struct RowStage {
  uint8_t* buf;
  __device__ __forceinline__ uint4* at(int row, int chunk) const {
    return reinterpret_cast<uint4*>(buf + row * 128 + ((chunk ^ (row & 7)) << 4));
  }
  // The rows in `valid` go to dst, each lane's own row's place.
  __device__ __forceinline__ void flush(uint32_t valid, void* dst, int lane) const {
    __syncwarp();
#pragma unroll 4
    for (int r = 0; r < 32; r += 4) {
      const int row = r + (lane >> 3), c = lane & 7;
      uint8_t* p = reinterpret_cast<uint8_t*>(__shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(dst), row));
      if (valid >> row & 1) st16(p + 16 * c, *at(row, c));
    }
    __syncwarp();
  }
};

// Tensor-core instructions of a converged issuer warp: every lane runs the issuing code with the same values, so that
// descriptors stay in uniform registers, and the one lane with `leader` set issues.
__device__ __forceinline__ uint32_t elect_one() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
  return r;
}
__device__ __forceinline__ void umma_ss_by(uint32_t leader, uint32_t d_tmem, uint64_t a, uint64_t b, uint32_t idesc,
                                           uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, l;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 l, %5, 0;\n\t"
      "@l tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate), "r"(leader)
      : "memory");
}
__device__ __forceinline__ void umma_ts_by(uint32_t leader, uint32_t d_tmem, uint32_t a, uint64_t b, uint32_t idesc,
                                           uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, l;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 l, %5, 0;\n\t"
      "@l tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a), "l"(b), "r"(idesc), "r"(accumulate), "r"(leader)
      : "memory");
}
__device__ __forceinline__ void umma_commit_by(uint32_t leader, uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred l;\n\tsetp.ne.b32 l, %1, 0;\n\t"
      "@l tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar), "r"(leader)
      : "memory");
}

// Registers of a warpgroup (four warps), given back or taken from those the block was launched with.
template <int N>
__device__ __forceinline__ void set_regs_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void set_regs_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}

// ---- launches (each in the file it names) ----------------------------------------------------------------
// A [B,H,S,d] tensor with unit feature stride.
struct DenseTensor {
  const void* p;
  Strides st;
};
struct DenseFwdPlan {
  int pack;    // query heads of one key head that share a query tile (a divisor of G)
  int rep;     // copies of the queries in a tile: 4 where they take at most 32 rows, else 1
  int tok;     // tokens of a query tile
  int ntile;   // query tiles per (batch, head group)
  int dual;    // one query tile per block, its keys in two interleaved streams
  int nsplit;  // blocks that share one query tile's keys
};
DenseFwdPlan dense_fwd_plan(const DenseDims& a);
// dense_prep.cu: ids' range (as id_range has it) of every key tile: kdoc [B][ceil(Skv / 128)].
int launch_dense_doc_ranges(const DenseDims& a, int2* kdoc, cudaStream_t st);
// dense_fwd.cu: low.p may be null; part_o / part_lse: nsplit > 1 only.
int launch_dense_fwd(const DenseDims& a, const BucketStarts& bs, const DenseTensor& q, const DenseTensor& k,
                     const DenseTensor& v, const DenseTensor& o, const DenseTensor& low, float* lse, const int2* kdoc,
                     float* part_o, float* part_lse, cudaStream_t st);

// Backward: workspace buffers.
struct DenseBwdBuf {
  float* stats;         // [2][B Hq][Sq rounded up to 4]: -LSE log2(e) (fp16: + 12; slopes: - slope (i mod 64) log2(e);
                        // -inf for a dead row), -D
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
// dense_prep.cu: before the main kernel (the rows' statistics, dqacc = 0, fp16: the largest norms, the ids' ranges, the
// bias by distance) and after it (the results' last sums and roundings).
int launch_dense_bwd_prep(const DenseDims& a, const BucketStarts& bs, const DenseTensor& o, const DenseTensor& low,
                          const DenseTensor& dout, const DenseTensor& v, const float* lse, const DenseBwdBuf& w,
                          int2* kdoc, int2* qdoc, cudaStream_t st);
int launch_dense_bwd_out(const DenseDims& a, const DenseTensor& dq, const DenseTensor& dk, const DenseTensor& dv,
                         void* dtable, const DenseBwdBuf& w, cudaStream_t st);
// Device status word of the current device (api.cu).
int device_status(int** out);
// 16-bit tensor map over a strided [B,H,S,d] tensor: box {64, pack, rows, 1, 1} of (d, pack, S, H / pack, B).
int make_tmap_dense(CUtensorMap* map, const DenseTensor& t, int d, int S, int H, int B, int pack, int box_rows);

}  // namespace lh
