// dense_fwd.cu — host side of the dense stage's forward: how a call is cut into blocks, and the join of split keys.
#include "dense_fwd.cuh"

namespace lh {
namespace fwd {

#define LH_DENSE_FWD(D, F16)                                                                                         \
  extern template int launch<D, F16>(const FwdMaps&, const FwdArgs&, const BucketStarts&, int, cudaStream_t);
LH_DENSE_FWD(64, false)
LH_DENSE_FWD(64, true)
LH_DENSE_FWD(128, false)
LH_DENSE_FWD(128, true)
#undef LH_DENSE_FWD

// Joins the splits of a row: W warps a row over its splits (one where they are few, so that many rows are in flight), then
// over shared memory.  Reads nsplit (d + 1) floats a row; latency-bound (tens of rows per SM).
template <int D, bool F16, int W>
__global__ void __launch_bounds__(128) join_kernel(const float* __restrict__ part_o, const float* __restrict__ part_lse,
                                                   DenseTensor o, DenseTensor low, float* __restrict__ lse, int nsplit,
                                                   int64_t rows, int Hq, int Sq) {
  const int slot = threadIdx.x / (32 * W), w = threadIdx.x / 32 % W, lane = threadIdx.x % 32;
  const int64_t row = min((int64_t)blockIdx.x * (4 / W) + slot, rows - 1);  // (a last block's spare warps repeat a row)
  constexpr int E = D / 32;
  __shared__ float s_acc[4][D], s_l[4];
  float m = -INFINITY;
  for (int s = lane; s < nsplit; s += 32) m = fmaxf(m, part_lse[s * rows + row]);
#pragma unroll
  for (int i = 16; i; i >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, i));
  const float mm = m == -INFINITY ? 0.f : m;
  float acc[E] = {}, l = 0.f;
#pragma unroll 4
  for (int s = w; s < nsplit; s += W) {
    const float ls = part_lse[s * rows + row], c = ex2(ls - mm);
    const float* src = part_o + (s * rows + row) * D + lane * E;
    float v[E];
    if (E == 4) *reinterpret_cast<float4*>(v) = *reinterpret_cast<const float4*>(src);
    else *reinterpret_cast<float2*>(v) = *reinterpret_cast<const float2*>(src);
    if (ls != -INFINITY) {  // (a split without a visible key adds nothing)
      l += c;
#pragma unroll
      for (int i = 0; i < E; ++i) acc[i] = fmaf(v[i], c, acc[i]);
    }
  }
#pragma unroll
  for (int i = 0; i < E; ++i) s_acc[slot * W + w][lane * E + i] = acc[i];
  if (lane == 0) s_l[slot * W + w] = l;
  __syncthreads();
  float lt = 0.f;
#pragma unroll
  for (int e = 0; e < W; ++e) lt += s_l[slot * W + e];
  const float inv = lt == 0.f ? 0.f : 1.0f / lt;
  const int64_t tk = row % Sq, bh = row / Sq, h = bh % Hq, b = bh / Hq;
  auto at = [&](const DenseTensor& t) {
    return static_cast<uint16_t*>(const_cast<void*>(t.p)) + b * t.st.b + h * t.st.h + tk * t.st.s;
  };
  const int i = (threadIdx.x % (32 * W)) * 8;
  if (i < D) {
    float v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      float x = 0.f;
#pragma unroll
      for (int u = 0; u < W; ++u) x += s_acc[slot * W + u][i + e];
      v[e] = x * inv;
    }
    uint4 lo;
    st16(at(o) + i, round8<F16>(v, &lo));
    if (low.p) st16(at(low) + i, lo);
  }
  if (threadIdx.x % (32 * W) == 0) lse[row] = lt == 0.f ? -INFINITY : (m + __log2f(lt)) * kLn2;
}

}  // namespace fwd

using namespace fwd;

DenseFwdPlan dense_fwd_plan(const DenseDims& a) {
  DenseFwdPlan f;
  // The query heads of a key head share query tiles where that takes fewer of them than tiles of one head each (few
  // tokens): a divisor of the group, so that a tile belongs to one key head, of at most 16, so that the bias windows of a
  // tile's heads leave the ring its place (one rule with and without a table).  A group whose divisors are larger, as 17,
  // reads its keys once for each head.
  f.pack = 1;
  int64_t least = a.G * (((int64_t)a.Sq + kTile - 1) / kTile);
  for (int g = 2; g <= 16 && g <= a.G; ++g) {
    const int tok = kTile / g;
    const int64_t tiles = a.G / g * (((int64_t)a.Sq + tok - 1) / tok);
    if (a.G % g == 0 && tiles < least) {
      least = tiles;
      f.pack = g;
    }
  }
  f.rep = a.Sq * f.pack <= kTile / 4 ? 4 : 1;
  f.tok = kTile / f.rep / f.pack;
  f.ntile = (int)(((int64_t)a.Sq + f.tok - 1) / f.tok);
  f.dual = f.ntile == 1;
  const int npair = f.dual ? 1 : (f.ntile + 1) / 2;
  const int64_t blocks = (int64_t)a.B * (a.Hq / f.pack) * npair;
  const int nk = (a.Skv + kTile - 1) / kTile;
  // Fewer blocks than SMs: the shares of the keys that are through first, counted in key tiles: rounds of blocks times a
  // block's tiles and about four for its start and end, and two for the join (5 pairs of 128-row tiles over 128 key tiles,
  // 8 head groups: 107 us in one round of 120 blocks, 103 in two of 280).
  f.nsplit = 1;
  int64_t best = nk + 4;
  for (int rounds = 1; blocks < kSms && rounds <= 2; ++rounds) {
    const int n = (int)(rounds * kSms / blocks) < nk / 4 ? (int)(rounds * kSms / blocks) : nk / 4;
    const int64_t cost = n > 1 ? (blocks * n + kSms - 1) / kSms * ((nk + n - 1) / n + 4) + 2 : INT64_MAX;
    if (cost < best) {
      best = cost;
      f.nsplit = n;
    }
  }
  return f;
}

int launch_dense_fwd(const DenseDims& a, const BucketStarts& bs, const DenseTensor& q, const DenseTensor& k,
                     const DenseTensor& v, const DenseTensor& o, const DenseTensor& low, float* lse, const int2* kdoc,
                     float* part_o, float* part_lse, cudaStream_t st) {
  const DenseFwdPlan f = dense_fwd_plan(a);
  FwdMaps m;
  if (make_tmap_dense(&m.q, q, a.d, a.Sq, a.Hq, a.B, f.pack, f.tok) ||
      make_tmap_dense(&m.k, k, a.d, a.Skv, a.Hkv, a.B, 1, kTile) ||
      make_tmap_dense(&m.v, v, a.d, a.Skv, a.Hkv, a.B, 1, kTile))
    return LH_ERR_CUDA;
  // whole result tiles leave by TMA (few rows, and the parts of split keys, by plain stores: the maps are not used)
  m.o = m.low = m.q;
  if (f.rep == 1 && f.nsplit == 1 &&
      (make_tmap_dense(&m.o, o, a.d, a.Sq, a.Hq, a.B, f.pack, f.tok) ||
       (low.p && make_tmap_dense(&m.low, low, a.d, a.Sq, a.Hq, a.B, f.pack, f.tok))))
    return LH_ERR_CUDA;
  fwd::FwdArgs p;
  p.a = a;
  p.pack = f.pack;
  p.tok = f.tok;
  p.rep = f.rep;
  p.ntile = f.ntile;
  p.dual = f.dual;
  p.npair = f.dual ? 1 : (f.ntile + 1) / 2;
  p.nsplit = f.nsplit;
  p.head_fast = p.npair < kHeadFastBelow;
  // key and value tiles in flight: what shared memory holds
  const uint32_t tile = kTile * a.d * 2, queries = (f.dual ? 1 : 2) * tile;
  const int nk = (a.Skv + kTile - 1) / kTile, per = (nk + f.nsplit - 1) / f.nsplit;
  p.win = a.table ? f.pack * (f.tok + kTile - 1) : 0;
  const uint32_t fixed = queries + kNBar * 8 + 2 * p.win * 4 + ((per + 3) & ~3);
  int slots = (int)((kSmemLimit - 1024 - fixed) / tile);
  if (slots > kMaxSlots) slots = kMaxSlots;
  p.slots = f.dual ? slots / 2 : slots;
  if (f.dual) slots = 2 * p.slots;
  p.off_kv = queries;
  p.off_bar = p.off_kv + slots * tile;
  p.off_win = p.off_bar + kNBar * 8;
  p.off_flags = p.off_win + 2 * p.win * 4;
  p.v = v;
  p.o = o;
  p.low = low;
  p.lse = lse;
  p.kdoc = kdoc;
  p.part_o = part_o;
  p.part_lse = part_lse;
  int smem = (int)p.off_flags + ((per + 3) & ~3) + 1024;
  if (smem < 120 * 1024) smem = 120 * 1024;  // one block (and its 512 tensor-memory columns) per SM
  int rc;
  {
    KernelTimer timer("dense_fwd", st);
    rc = a.d == 64 ? (a.f16 ? fwd::launch<64, true>(m, p, bs, smem, st) : fwd::launch<64, false>(m, p, bs, smem, st))
                   : (a.f16 ? fwd::launch<128, true>(m, p, bs, smem, st) : fwd::launch<128, false>(m, p, bs, smem, st));
  }
  if (rc || f.nsplit == 1) return rc;
  KernelTimer timer("dense_join", st);
  const int64_t rows = (int64_t)a.B * a.Hq * a.Sq;
  const bool few = f.nsplit <= 8;
  auto join = a.d == 64 ? (a.f16 ? (few ? join_kernel<64, true, 1> : join_kernel<64, true, 4>)
                                 : (few ? join_kernel<64, false, 1> : join_kernel<64, false, 4>))
                        : (a.f16 ? (few ? join_kernel<128, true, 1> : join_kernel<128, true, 4>)
                                 : (few ? join_kernel<128, false, 1> : join_kernel<128, false, 4>));
  const int64_t grid = few ? (rows + 3) / 4 : rows;
  join<<<(unsigned)grid, 128, 0, st>>>(part_o, part_lse, o, low, lse, f.nsplit, rows, a.Hq, a.Sq);
  return check_launch();
}

}  // namespace lh
