// dense_bwd.cuh — the dense stage's attention, backward, on the tcgen05 tensor cores.
//
// With P = exp(Z - LSE) recomputed, dV = P^T dO, dP = dO V^T, D = rowsum(dO o O), dZ = P o (dP - D), dtable[h, b] = the
// sum of dZ over the pairs of bucket b, dS = dZ (1 - tanh^2), dQ = scale dS K, dK = scale dS^T Q.
//
// One block per (batch, key head, 128-key tile, share of the query heads); the visible 64-row query sub-tiles of its
// heads stream past the resident K and V, so the gradients of a shared key head are one sum in tensor memory.  Warp
// roles and products as in the gathered attention's backward:
//   warp 0      TMA producer: K, V once; Q, dO and the rows' statistics into a three-stage ring;
//   warp 1      MMA issuer: S^T = K Q^T and dP^T = V dO^T, then for the sub-tile before dV += P^T dO, dK += dS^T Q and
//               dQ^T = K^T dS^T;
//   warps 4-11  one key row per thread, 32 of the sub-tile's 64 rows per warp: P^T and dS^T (16-bit) to tensor memory
//               over S^T and dP^T, dS^T to shared memory too (the B operand of dQ^T);
//   warps 12-15 dQ^T out of tensor memory, through a shared tile, to the fp32 accumulator with TMA reduce-add.
//
// The bias's gradient: nearly every 32 x 32 block of pairs lies inside one bucket (distances beyond a few hundred share
// few buckets): its sum goes to one number per warp.  A block across buckets is summed along its diagonals by rotating
// partial sums through the warp (lane r adds the pair (c, r) at step c; its sum came from lane r - 1), and lane b takes
// bucket b's run of diagonals as a difference of prefix sums.  No atomics: a warp's 32-bit sums go to its own place and
// are added in a fixed order.
//
// fp16: dZ can be as small as 1 / Skv of a small gradient.  P is carried times 2^12, and dS times a power of two from
// the largest row norms, 2 max|dO_i| max|V_j| 2^e < 2^15 (|dZ| <= 2 |dO_i| |V_j|), so it neither overflows nor drowns.
// P and dS are rounded once to the operands' type, the other operand of their products having it.
//
// dQ is accumulated with fp32 reduce-adds whose order is not fixed; dK, dV and dtable are bitwise reproducible.
#pragma once

#include <atomic>
#include <type_traits>

#include "dense.cuh"

namespace lh {
namespace bwd {

constexpr int kThreads = 512;
// Registers a thread of the issuing, computing and draining warps: 128 (48 + 2 * 184 + 96) = 512 * 128.
constexpr int kRegsIssue = 48, kRegsCompute = 184, kRegsDrain = 96;
constexpr int kQTile = 64;
constexpr int kStages = 3;
constexpr float kLog2e = 1.4426950408889634f;
constexpr int kBarCompute = 1, kBarDrain = 2;
constexpr int kHeadFastBelow = 148;
// LSE is rounded to a step of its size, and so is each term of the exponent: from this magnitude (of log2) on a P of 1 could
// come out as more than 2^(3/16), and at scores of 2^25 as 2^8.
constexpr float kFarTerm = 1048576.f;
constexpr float kShift16 = 4096.f;  // fp16: P is carried times this

template <int D>
struct BwdLayout {
  static constexpr uint32_t KT = kKeyTile * D * 2;
  static constexpr uint32_t QT = kQTile * D * 2;
  static constexpr uint32_t PT = kKeyTile * kQTile * 2;
  static constexpr uint32_t K = 0;
  static constexpr uint32_t V = KT;
  static constexpr uint32_t Q = 2 * KT;
  static constexpr uint32_t DO = Q + kStages * QT;
  static constexpr uint32_t DS = DO + kStages * QT;
  static constexpr uint32_t DQ = DS + 2 * PT;  // [d/32][64 rows][32 features] fp32
  static constexpr uint32_t ST = 2 * kQTile * 4;
  static constexpr uint32_t STAT = DQ + kQTile * D * 4;
  static constexpr uint32_t BAR = STAT + kStages * ST;
  static constexpr uint32_t B_KV = 0, B_QF = 1, B_QE = 1 + kStages, B_SF = 1 + 2 * kStages, B_DSF = B_SF + 2,
                            B_MM = B_DSF + 2, B_DQF = B_MM + 2, B_FIN = B_DQF + 2, B_DRAIN = B_FIN + 1,
                            NBAR = B_DRAIN + 1;
  static constexpr uint32_t BYTES = BAR + NBAR * 8;
};

struct BwdArgs {
  DenseDims a;
  int nkt, heads, head_fast;  // key tiles; query heads of one block (a divisor of G)
  DenseBwdBuf w;
};

template <int D, bool F16, bool CAP, int BIAS>
__global__ void __launch_bounds__(kThreads, 1)
    dense_bwd_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                     const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CUtensorMap tmDO,
                     const __grid_constant__ CUtensorMap tmDQ, const __grid_constant__ CUtensorMap tmST,
                     const __grid_constant__ CUtensorMap tmDK, const __grid_constant__ CUtensorMap tmDV,
                     const __grid_constant__ BwdArgs p) {
  using Lay = BwdLayout<D>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint32_t s_tmem;
  __shared__ WaitCtl s_wait;
  __shared__ int s_ilo, s_ihi, s_klo, s_khi;
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sb = smem_u32(smem);
  auto bar = [&](uint32_t i) { return sb + Lay::BAR + 8u * i; };
  const DenseDims& a = p.a;
  int* status = a.status;

  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int kt = p.head_fast ? blockIdx.y : blockIdx.x;
  const int bh = p.head_fast ? blockIdx.x : blockIdx.y;
  const int b = bh / a.Hkv, kvh = bh % a.Hkv;
  const int h0 = kvh * a.G + (int)blockIdx.z * p.heads;  // first query head of this block
  const int len = dense_len(a, b), prefix = dense_prefix(a, b, len), off = len - a.Sq;
  const int k0 = kt * kKeyTile;
  const int nq = (a.Sq + kQTile - 1) / kQTile;

  if (threadIdx.x == 0) {
    wait_ctl_init(&s_wait, status);
    mbar_init(bar(Lay::B_KV), 1);
    for (int s = 0; s < kStages; ++s) {
      mbar_init(bar(Lay::B_QF + s), 1);
      mbar_init(bar(Lay::B_QE + s), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(Lay::B_SF + i), 1);
      mbar_init(bar(Lay::B_DSF + i), 256);
      mbar_init(bar(Lay::B_MM + i), 1);
      mbar_init(bar(Lay::B_DQF + i), 128);
    }
    mbar_init(bar(Lay::B_FIN), 1);
    mbar_init(bar(Lay::B_DRAIN), 1);
    fence_mbar_init();
    s_ilo = INT32_MAX;
    s_ihi = -1;
    s_klo = INT32_MAX;
    s_khi = -1;
    prefetch_tmap(&tmQ);
    prefetch_tmap(&tmK);
    prefetch_tmap(&tmV);
    prefetch_tmap(&tmDO);
    prefetch_tmap(&tmDQ);
    prefetch_tmap(&tmST);
  }
  if (warp == 1) tmem_alloc(smem_u32(&s_tmem), 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s_tmem;
  // columns: S^T buffer i at 128 i, dP^T buffer i at 128 i + 64; dV at 256; dK at 256 + D
  const uint32_t tDV = tmem + 256, tDK = tmem + 256 + D;

  // the run of sub-tiles with a visible pair (ids in no order may leave invisible ones inside it; they add nothing)
  const int2 kd = a.docs ? __ldg(p.w.kdoc + (int64_t)b * p.nkt + kt) : make_int2(0, 0);
  const int2* qdoc = p.w.qdoc + (int64_t)b * nq;
  for (int i = threadIdx.x; i < nq; i += kThreads) {
    const int xb = off + min((i + 1) * kQTile, a.Sq) - 1;
    if (k0 > last_key(a, xb, len, prefix)) continue;
    if (a.docs && !docs_meet(kd, __ldg(qdoc + i))) continue;
    atomicMin(&s_ilo, i);
    atomicMax(&s_ihi, i);
  }
  __syncthreads();
  const int ilo = s_ilo, n1 = max(0, s_ihi - ilo + 1);  // sub-tiles per head (ilo is read only where n1 > 0)
  const int nit = n1 * p.heads;
  float fs = 1.f;  // fp16: the power of two that dS is carried times, over kShift16
  if (F16) {
    const float top = 2.f * __uint_as_float(__ldg(p.w.amax + 2 * bh)) * __uint_as_float(__ldg(p.w.amax + 2 * bh + 1));
    int e = 0;
    if (top > 0.f && top < 3e38f) e = min(max(14 - (int)floorf(__log2f(top)) - 1, -100), 100);
    fs = exp2f((float)(e - 12));
  }
  const float q_out = F16 ? a.scale / (fs * kShift16) : a.scale;  // brings dQ and dK to scale

  if (warp < 4) {
    set_regs_dec<kRegsIssue>();
    if (warp == 0) {
      // ---------------------------------------------------------------- TMA producer
      if (lane == 0 && nit > 0) {
        bool ok = true;
        int issued = 0;
        mbar_arrive_expect_tx(bar(Lay::B_KV), 2 * Lay::KT);
        for (int db = 0; db < D / 64; ++db) {
          tma_load_5d(sb + Lay::K + db * 16384, &tmK, bar(Lay::B_KV), db * 64, 0, k0, kvh, b);
          tma_load_5d(sb + Lay::V + db * 16384, &tmV, bar(Lay::B_KV), db * 64, 0, k0, kvh, b);
        }
        for (int it = 0; it < nit && ok; ++it) {
          const int s = it % kStages;
          if (it >= kStages) ok = mbar_wait(bar(Lay::B_QE + s), ((it / kStages) - 1) & 1, &s_wait, status);
          if (!ok) break;
          const int h = h0 + it / n1, row = (ilo + it % n1) * kQTile;
          mbar_arrive_expect_tx(bar(Lay::B_QF + s), 2 * Lay::QT + Lay::ST);
          for (int db = 0; db < D / 64; ++db) {
            tma_load_5d(sb + Lay::Q + s * Lay::QT + db * 8192, &tmQ, bar(Lay::B_QF + s), db * 64, 0, row, h, b);
            tma_load_5d(sb + Lay::DO + s * Lay::QT + db * 8192, &tmDO, bar(Lay::B_QF + s), db * 64, 0, row, h, b);
          }
          tma_load_3d(sb + Lay::STAT + s * Lay::ST, &tmST, bar(Lay::B_QF + s), row, b * a.Hq + h, 0);  // both planes
          issued = it + 1;
        }
        // every copy has landed before the block lets go of its memory, whoever gave up
        mbar_wait_teardown(bar(Lay::B_KV), 0);
        for (int it = issued >= kStages ? issued - kStages : 0; it < issued; ++it)
          mbar_wait_teardown(bar(Lay::B_QF + it % kStages), (it / kStages) & 1);
      }
    } else if (warp == 1) {
      // ---------------------------------------------------------------- MMA issuer (the whole warp, one lane issuing)
      if (nit > 0) {
        constexpr int fmt = F16 ? kFmtF16 : kFmtBF16;
        constexpr uint32_t idesc_s = idesc_f32acc(fmt, 128, kQTile, 0, 0);   // K-major x K-major
        constexpr uint32_t idesc_acc = idesc_f32acc(fmt, 128, D, 0, 1);      // K-major x MN-major
        constexpr uint32_t idesc_dq = idesc_f32acc(fmt, 128, kQTile, 1, 1);  // MN-major x MN-major
        const uint32_t leader = elect_one();
        const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
        const uint64_t dK = sdesc_sw128(sb + Lay::K, 16, 1024), dV = sdesc_sw128(sb + Lay::V, 16, 1024);
        const uint64_t dQ = sdesc_sw128(sb + Lay::Q, 16, 1024), dDO = sdesc_sw128(sb + Lay::DO, 16, 1024);
        const uint64_t tK = sdesc_sw128(sb + Lay::K, 16384, 1024), tDS = sdesc_sw128(sb + Lay::DS, 8192, 1024);  // MN-major
        const uint64_t tQ = sdesc_sw128(sb + Lay::Q, 8192, 1024), tDO = sdesc_sw128(sb + Lay::DO, 8192, 1024);
        auto wait = [&](uint32_t i, uint32_t ph) {
          return __all_sync(0xffffffffu, mbar_wait(bar(i), ph, &s_wait, status)) != 0;
        };
        bool ok = wait(Lay::B_KV, 0);
        auto products = [&](int jt, int s) {  // dV, dK, dQ^T of sub-tile jt, in stage s
          const int i = jt & 1;
          if (!wait(Lay::B_DSF + i, (jt >> 1) & 1)) return false;
          tc_fence_after();
          const uint64_t bQ = tQ + s * (Lay::QT >> 4), bDO = tDO + s * (Lay::QT >> 4), bDS = tDS + i * (Lay::PT >> 4);
          const uint32_t aP = tm + 128 * i, aDS = tm + 128 * i + 64;
#pragma unroll
          for (int kk = 0; kk < kQTile / 16; ++kk) {  // reduction over the 64 queries
            const uint32_t acc = (jt > 0 || kk > 0) ? 1u : 0u;
            const uint32_t pc = (kk >> 1) * 32 + (kk & 1) * 8;  // column half kk/2 packed at 32 (kk/2)
            umma_ts_by(leader, tm + 256, aP + pc, bDO + kk * (2048 >> 4), idesc_acc, acc);
            umma_ts_by(leader, tm + 256 + D, aDS + pc, bQ + kk * (2048 >> 4), idesc_acc, acc);
          }
#pragma unroll
          for (int kk = 0; kk < kKeyTile / 16; ++kk)  // reduction over the 128 keys
            umma_ss_by(leader, tm + 128 * i, tK + kk * (2048 >> 4), bDS + kk * (2048 >> 4), idesc_dq, kk > 0 ? 1u : 0u);
          umma_commit_by(leader, bar(Lay::B_MM + i));
          umma_commit_by(leader, bar(Lay::B_QE + s));
          return true;
        };
        int s = 0, ph = 0, before = 0;  // stage and phase of sub-tile it, stage of the one before
        for (int it = 0; it < nit && ok; ++it) {
          const int i = it & 1;
          ok = wait(Lay::B_QF + s, ph);
          // buffer pair i: its dQ^T of sub-tile it-2 has been read out of tensor memory
          if (ok && it >= 2) ok = wait(Lay::B_DQF + i, ((it >> 1) - 1) & 1);
          if (!ok) break;
          tc_fence_after();
          const uint64_t bQ = dQ + s * (Lay::QT >> 4), bDO = dDO + s * (Lay::QT >> 4);
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint32_t ko = ((kk >> 2) * 16384 + (kk & 3) * 32) >> 4, qo = ((kk >> 2) * 8192 + (kk & 3) * 32) >> 4;
            umma_ss_by(leader, tm + 128 * i, dK + ko, bQ + qo, idesc_s, kk > 0 ? 1u : 0u);
            umma_ss_by(leader, tm + 128 * i + 64, dV + ko, bDO + qo, idesc_s, kk > 0 ? 1u : 0u);
          }
          umma_commit_by(leader, bar(Lay::B_SF + i));
          if (it >= 1) ok = products(it - 1, before);
          before = s;
          if (++s == kStages) s = 0, ph ^= 1;
        }
        if (ok) ok = products(nit - 1, before);
        umma_commit_by(leader, bar(Lay::B_FIN));  // dV, dK final once every product above has completed
        umma_commit_by(leader, bar(Lay::B_DRAIN));
        mbar_wait_teardown(bar(Lay::B_DRAIN), 0);
      }
    }
  } else if (warp < 12) {
    // ---------------------------------------------------------------- compute: P^T and dS^T
    set_regs_inc<kRegsCompute>();
    const int quarter = warp & 3, hc = (warp - 4) >> 2;
    const int r = quarter * 32 + lane;  // key row inside the tile = TMEM lane
    const int tid = threadIdx.x - 128;
    const uint32_t lane_base = (uint32_t)(quarter * 32) << 16;
    const int key = k0 + r, kw = k0 + quarter * 32;  // this thread's key, the warp's first
    const int kid = doc_at(a, b, key, len);
    const bool kdead = kid < 0;
    const float mul = CAP ? a.cap * kLog2e : a.scale * kLog2e;
    const float cap_in = a.cap_in;
    const uint64_t mul2 = f2pack(mul, mul);
    const int E = a.near, wide = 2 * E + 1;
    float bacc[4] = {0.f, 0.f, 0.f, 0.f};  // lane l: dtable sums of buckets l, l + 32, ...
    float run = 0.f;                       // this thread's sum of dZ in bucket `run_b`
    int run_b = -1;
    auto flush = [&]() {
      if (run_b < 0) return;
      float t = run;
#pragma unroll
      for (int o = 16; o; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
#pragma unroll
      for (int m = 0; m < 4; ++m)
        if (run_b == lane + 32 * m) bacc[m] += t;
      run = 0.f;
      run_b = -1;
    };
    bool ok = true;
    int it = 0;
    for (int g = 0; g < p.heads; ++g) {
      const float slope2 = BIAS == 1 ? -__ldg(a.slopes + h0 + g) * kLog2e : 0.f;
      const float* bias = BIAS == 2 ? p.w.bias + (int64_t)(h0 + g) * wide + E : nullptr;
      for (int n = 0; n < n1 && ok; ++n, ++it) {
        const int i = it & 1, s = it % kStages, sub = ilo + n;
        const int row0 = sub * kQTile + 32 * hc, x0 = off + row0;  // this warp's first query row and its position
        int2 qd = make_int2(0, 0);
        if (a.docs) qd = __ldg(qdoc + sub);
        const bool whole = row0 + 31 < a.Sq && k0 + kKeyTile - 1 <= last_key(a, x0, len, prefix) &&
                           (!a.docs || docs_one(kd, qd));
        const bool qdead = off + sub * kQTile < 0 || (a.docs && qd.x < 0);
        bool near = false;
        float badd = 0.f;
        int bucket = 0;
        const int d0 = x0 - key;  // distance of column 0
        if (BIAS == 1) {
          near = x0 - (kw + 31) < 0;
          // a tile on one side of the slopes: the statistics hold the columns' share, this is the key's and the tile's
          if (!near) badd = slope2 * (float)(d0 - 32 * hc);
        }
        if (BIAS == 2) {
          const int lo = min(max(x0 - (kw + 31), -E), E), hi = min(max(x0 + 31 - kw, -E), E);
          bucket = __ldg(p.w.bucket + E + hi);
          near = bucket != __ldg(p.w.bucket + E + lo);
          badd = __ldg(bias + hi);
        }
        ok = __all_sync(0xffffffffu, mbar_wait(bar(Lay::B_SF + i), (it >> 1) & 1, &s_wait, status));
        if (ok) ok = __all_sync(0xffffffffu, mbar_wait(bar(Lay::B_QF + s), (it / kStages) & 1, &s_wait, status));
        if (!ok) break;
        float sv[32], dp[32];
        tc_fence_after();
        tmem_ld32(tmem + 128 * i + lane_base + 32 * hc, sv);
        tmem_ld32(tmem + 128 * i + 64 + lane_base + 32 * hc, dp);
        bool far = false;
        if (BIAS == 1) {
          const float nlse = reinterpret_cast<const float*>(smem + Lay::STAT + s * Lay::ST)[32 * hc + lane];
          far = __any_sync(0xffffffffu, (fabsf(nlse) > kFarTerm && nlse != -INFINITY) || fabsf(badd) > kFarTerm);
        }
        tmem_ld_wait();
        if (CAP) {
          const float big = absmax32(sv, 0.f) * cap_in;
          if (__all_sync(0xffffffffu, big <= 0.5f)) {
            tanh32<true>(sv, cap_in, 1.f);
          } else if (__all_sync(0xffffffffu, big <= 1.25f)) {
            tanh32<false>(sv, cap_in, 1.f);
          } else {
#pragma unroll
            for (int c = 0; c < 32; ++c) sv[c] = tanh_any<true>(sv[c] * cap_in);
          }
        }
        uint32_t vis = 0xffffffffu;  // bit c: the pair (row0 + c, key) is visible
        if (!whole) {
          const int lo = max(max(key < prefix || !a.causal ? 0 : key - x0, -x0), 0), hi = min(a.Sq - row0, 32);
          vis = kdead || lo >= hi ? 0u : (0xffffffffu >> (32 - hi)) & (0xffffffffu << lo);  // rows [lo, hi)
          if (a.docs) vis &= same_doc(doc_at(a, b, x0 + lane, len), kid);
        }
        uint32_t pk[16], dk[16];
        const ulonglong2* nl4 = reinterpret_cast<const ulonglong2*>(smem + Lay::STAT + s * Lay::ST) + 8 * hc;
        const ulonglong2* nd4 = reinterpret_cast<const ulonglong2*>(smem + Lay::STAT + s * Lay::ST + kQTile * 4) + 8 * hc;
        const uint64_t badd2 = f2pack(badd, badd);
        uint64_t sum2 = 0ull;
        // P and dS of the 32 columns; Near: the bias differs from pair to pair.  P is kept at 1 at most; with slopes only
        // where the exponent's terms are large, in the form for any pair (16,384 rows, backward 1420 us; kept there for every
        // pair too 1487; the other kernels pay up to 1 % for it, and up to 13 % for a second form of the loop)
        constexpr float top = F16 ? 12.f : 0.f;
        auto columns = [&](auto tag) {
          constexpr bool Near = decltype(tag)::value;
#pragma unroll
          for (int c = 0; c < 32; c += 4) {
            const ulonglong2 nl = nl4[c >> 2], nd = nd4[c >> 2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const int cc = c + 2 * h;
              uint64_t arg = fma_f32x2(f2pack(sv[cc], sv[cc + 1]), mul2, h ? nl.y : nl.x);
              if (BIAS != 0 && !Near) arg = add_f32x2(arg, badd2);
              if (BIAS == 1 && Near) {  // (also right on one side)
                auto bb = [&](int e) { return slope2 * (fabsf((float)(d0 + e)) - (float)(32 * hc + e)); };
                arg = add_f32x2(arg, f2pack(bb(cc), bb(cc + 1)));
              }
              if (BIAS == 2 && Near)
                arg = add_f32x2(arg, f2pack(__ldg(bias + min(max(d0 + cc, -E), E)), __ldg(bias + min(max(d0 + cc + 1, -E), E))));
              float a0 = f2lo(arg), a1 = f2hi(arg);
              if (Near || BIAS != 1) a0 = min_nan(a0, top), a1 = min_nan(a1, top);
              const float p0 = ex2(a0), p1 = ex2(a1);
              uint64_t z2 = mul_f32x2(f2pack(p0, p1), add_f32x2(f2pack(dp[cc], dp[cc + 1]), h ? nd.y : nd.x));
              pk[cc / 2] = pack2_rn<F16>(p0, p1);
              if (BIAS == 2) {
                sum2 = add_f32x2(sum2, z2);
                dp[cc] = f2lo(z2);
                dp[cc + 1] = f2hi(z2);
              }
              if (CAP) {
                const uint64_t t2 = f2pack(sv[cc], sv[cc + 1]), nt2 = f2pack(-sv[cc], -sv[cc + 1]);
                z2 = mul_f32x2(z2, fma_f32x2(t2, nt2, f2pack(1.f, 1.f)));
              }
              if (F16) z2 = mul_f32x2(z2, f2pack(fs, fs));
              dk[cc / 2] = pack2_rn<F16>(f2lo(z2), f2hi(z2));
            }
          }
        };
        if (BIAS != 0 && (near || far)) columns(std::true_type{});
        else columns(std::false_type{});
        if (!whole) {  // masked pairs are nothing, whatever came out
          sum2 = 0ull;
#pragma unroll
          for (int c = 0; c < 32; c += 2) {
            const uint32_t m = (vis >> c & 1 ? 0xffffu : 0u) | (vis >> (c + 1) & 1 ? 0xffff0000u : 0u);
            pk[c / 2] &= m;
            dk[c / 2] &= m;
            if (BIAS == 2) {
              dp[c] = vis >> c & 1 ? dp[c] : 0.f;
              dp[c + 1] = vis >> (c + 1) & 1 ? dp[c + 1] : 0.f;
              sum2 = add_f32x2(sum2, f2pack(dp[c], dp[c + 1]));
            }
          }
        }
        if (it >= 2) ok = __all_sync(0xffffffffu, mbar_wait(bar(Lay::B_MM + i), ((it >> 1) - 1) & 1, &s_wait, status));
        if (!ok) break;
        tmem_st16(tmem + 128 * i + lane_base + 32 * hc, pk);
        tmem_st16(tmem + 128 * i + 64 + lane_base + 32 * hc, dk);
        uint8_t* sDS = smem + Lay::DS + i * Lay::PT;
#pragma unroll
        for (int ch = 0; ch < 4; ++ch) {
          const uint32_t o = sw128_offset(r, 4 * hc + ch);
          *reinterpret_cast<uint4*>(sDS + o) = make_uint4(dk[4 * ch], dk[4 * ch + 1], dk[4 * ch + 2], dk[4 * ch + 3]);
        }
        // dead rows and keys: whatever they hold would meet a zero of P or dS in the products
        if (qdead && (tid >> 7) < D / 64) {
          const int c = tid & 63;
          if (doc_at(a, b, off + sub * kQTile + c, len) < 0) {
            uint8_t* t = smem + ((tid >> 6) & 1 ? Lay::DO : Lay::Q) + s * Lay::QT + (tid >> 7) * 8192 + c * 128;
#pragma unroll
            for (int e = 0; e < 8; ++e) *reinterpret_cast<uint4*>(t + (((e + c) & 7) << 4)) = make_uint4(0, 0, 0, 0);
          }
        }
        if (it == 0 && kdead && hc < D / 64) {
          uint8_t* t = smem + Lay::K + hc * 16384 + r * 128;
#pragma unroll
          for (int e = 0; e < 8; ++e) *reinterpret_cast<uint4*>(t + (((e + r) & 7) << 4)) = make_uint4(0, 0, 0, 0);
        }
        fence_proxy_async_smem();
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(bar(Lay::B_DSF + i));
        if (BIAS == 2) {
          if (!near) {
            if (bucket != run_b) flush();
            run_b = bucket;
            run += f2lo(sum2) + f2hi(sum2);
          } else {
            // diagonals: after step c lane r holds, of distance base + ((c - r) mod 32), `up`, and of 32 less, `dn`; four
            // runs of eight columns side by side, each brought to the last one's place at the end
            float ups[4] = {}, dns[4] = {};
#pragma unroll
            for (int e = 0; e < 8; ++e)
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                const int c = 8 * k + e;
                if (e > 0) {
                  ups[k] = __shfl_sync(0xffffffffu, ups[k], (lane + 31) & 31);
                  dns[k] = __shfl_sync(0xffffffffu, dns[k], (lane + 31) & 31);
                }
                if (lane <= c) ups[k] += dp[c]; else dns[k] += dp[c];
              }
            float up = ups[3], dn = dns[3];
#pragma unroll
            for (int k = 0; k < 3; ++k) {
              up += __shfl_sync(0xffffffffu, ups[k], (lane + 8 * k + 8) & 31);
              dn += __shfl_sync(0xffffffffu, dns[k], (lane + 8 * k + 8) & 31);
            }
            // lane r: up is distance base + 31 - r, dn base - 1 - r; sums over the lanes from r on are prefixes
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
              const float u = __shfl_down_sync(0xffffffffu, up, o), d = __shfl_down_sync(0xffffffffu, dn, o);
              if (lane + o < 32) up += u, dn += d;
            }
            const float all_dn = __shfl_sync(0xffffffffu, dn, 0);
            const int first = x0 - kw - 32;  // place u holds distance first + u, 0 <= u < 64
            auto prefix_to = [&](int u) {
              const float vd = __shfl_sync(0xffffffffu, dn, 31 - min(max(u, 0), 31));
              const float vu = __shfl_sync(0xffffffffu, up, 63 - min(max(u, 32), 63));
              return u < 0 ? 0.f : u < 32 ? vd : all_dn + vu;
            };
#pragma unroll
            for (int m = 0; m < 4; ++m) {
              if (32 * m >= a.buckets) break;
              const int bk = lane + 32 * m;
              const int2 rg = bk < a.buckets ? __ldg(p.w.range + bk) : make_int2(1, 0);
              const int ulo = max(rg.x - first, 0), uhi = min(rg.y - first, 63);
              const float vh = prefix_to(uhi), vl = prefix_to(ulo - 1);
              if (ulo <= uhi) bacc[m] += vh - vl;
            }
          }
        }
      }
      if (BIAS == 2) {
        flush();
        float* out = p.w.dtpart +
                     ((((int64_t)bh * p.nkt + kt) * a.G + (h0 - kvh * a.G + g)) * 8 + (warp - 4)) * a.buckets;
#pragma unroll
        for (int m = 0; m < 4; ++m) {
          if (lane + 32 * m < a.buckets) out[lane + 32 * m] = F16 ? bacc[m] / kShift16 : bacc[m];
          bacc[m] = 0.f;
        }
      }
    }
    // epilogue: dV (half 0's warps) or dK (half 1's) rows of this key tile, final after B_FIN
    ok = named_barrier_and(kBarCompute, 256, ok);
    if (ok && nit > 0) ok = __all_sync(0xffffffffu, mbar_wait(bar(Lay::B_FIN), 0, &s_wait, status));
    if (ok) {
      tc_fence_after();
      const uint32_t tacc = hc == 0 ? tDV : tDK;
      const float f = hc == 0 ? (F16 ? 1.f / kShift16 : 1.f) : q_out;
      uint8_t* tile = smem + (hc == 0 ? Lay::K : Lay::V);  // (K and V are consumed)
      auto result = [&](int c, float (&v)[32]) {
        if (nit > 0) {
          tmem_ld32(tacc + lane_base + c * 32, v);
          tmem_ld_wait();
        }
#pragma unroll
        for (int e = 0; e < 32; ++e) v[e] = nit > 0 ? v[e] * f : 0.f;
      };
      if (p.w.dkv) {  // query heads shared out: fp32 sums [share][dV, dK][B Hkv][Skv][d], added by another kernel
        float* part = p.w.dkv + ((((int64_t)blockIdx.z * 2 + hc) * a.B * a.Hkv + bh) * a.Skv + key) * D;
        const RowStage stage{tile + quarter * 4096};
        const uint32_t rows = __ballot_sync(0xffffffffu, key < a.Skv);
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
          float v[32];
          result(c, v);
#pragma unroll
          for (int e = 0; e < 8; ++e)
            *reinterpret_cast<float4*>(stage.at(lane, e)) = make_float4(v[4 * e], v[4 * e + 1], v[4 * e + 2], v[4 * e + 3]);
          stage.flush(rows, part + 32 * c, lane);
        }
      } else {  // the whole tile in the layout K and V came in, by TMA (rows at or beyond Skv are outside its tensor)
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
          const RowStage stage{tile + (c >> 1) * 16384 + quarter * 4096};
          float v[32];
          result(c, v);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            uint4 lo;
            *stage.at(lane, 4 * (c & 1) + e) = round8<F16>(v + 8 * e, &lo);
          }
        }
        fence_proxy_async_smem();
        named_barrier_and(3 + hc, 128, true);
        if (r == 0) {
          for (int db = 0; db < D / 64; ++db)
            tma_store_5d(hc == 0 ? &tmDV : &tmDK, smem_u32(tile + db * 16384), db * 64, 0, k0, kvh, b);
          bulk_commit_group();
          bulk_wait_group0();
        }
      }
    }
  } else {
    // ---------------------------------------------------------------- drain: dQ^T -> shared tile -> TMA reduce-add
    set_regs_dec<kRegsDrain>();
    const int quarter = warp & 3;
    const int f = quarter * 32 + lane;  // feature = TMEM lane of dQ^T
    const int dt = threadIdx.x - 384;
    const uint32_t lane_base = (uint32_t)(quarter * 32) << 16;
    float* stage = reinterpret_cast<float*>(smem + Lay::DQ);
    bool ok = true;
    for (int it = 0; it < nit; ++it) {
      const int i = it & 1;
      ok = __all_sync(0xffffffffu, ok && mbar_wait(bar(Lay::B_MM + i), (it >> 1) & 1, &s_wait, status));
      float v[64];
      if (ok) {
        tc_fence_after();
        tmem_ld32(tmem + 128 * i + lane_base, *reinterpret_cast<float(*)[32]>(&v[0]));
        tmem_ld32(tmem + 128 * i + lane_base + 32, *reinterpret_cast<float(*)[32]>(&v[32]));
        tmem_ld_wait();
        tc_fence_before();
        mbar_arrive(bar(Lay::B_DQF + i));  // buffer pair i may take the next S^T
      }
      // the previous reduce must have finished reading the staging tile before it is overwritten
      if (dt == 0) bulk_wait_group_read0();
      ok = named_barrier_and(kBarDrain, 128, ok);
      if (!ok) break;
      if (f < D) {
        float* col = stage + (f >> 5) * (kQTile * 32) + (f & 31);
#pragma unroll
        for (int c = 0; c < kQTile; ++c) col[c * 32] = v[c] * q_out;
      }
      fence_proxy_async_smem();
      named_barrier_and(kBarDrain, 128, true);
      if (dt == 0) {
        const int h = h0 + it / n1, row = (ilo + it % n1) * kQTile;
        for (int fb = 0; fb < D / 32; ++fb)
          tma_reduce_add_3d(&tmDQ, smem_u32(stage + fb * kQTile * 32), fb * 32, row, b * a.Hq + h);
        bulk_commit_group();
      }
    }
    if (dt == 0) bulk_wait_group0();
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <int D, bool F16, bool CAP, int BIAS>
int launch_t(const CUtensorMap (&m)[8], const BwdArgs& p, cudaStream_t st) {
  auto kernel = dense_bwd_kernel<D, F16, CAP, BIAS>;
  const int smem = BwdLayout<D>::BYTES + 1024;
  static std::atomic<uint64_t> ready{0};  // devices on which the kernel's shared-memory limit is set
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return LH_ERR_CUDA;
  if (!(ready.load(std::memory_order_acquire) >> (dev & 63) & 1)) {
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
      return LH_ERR_CUDA;
    ready.fetch_or(uint64_t(1) << (dev & 63), std::memory_order_release);
  }
  const int nbh = p.a.B * p.a.Hkv, nz = p.a.G / p.heads;
  const dim3 grid = p.head_fast ? dim3(nbh, p.nkt, nz) : dim3(p.nkt, nbh, nz);
  kernel<<<grid, kThreads, smem, st>>>(m[0], m[1], m[2], m[3], m[4], m[5], m[6], m[7], p);
  return check_launch();
}
// Instantiated for each width and type in a file of its own.
template <int D, bool F16>
int launch(const CUtensorMap (&m)[8], const BwdArgs& p, cudaStream_t st) {
  const int bias = p.a.slopes ? 1 : p.a.table ? 2 : 0;
  const bool cap = p.a.cap > 0.f;
  if (bias == 0) return cap ? launch_t<D, F16, true, 0>(m, p, st) : launch_t<D, F16, false, 0>(m, p, st);
  if (bias == 1) return cap ? launch_t<D, F16, true, 1>(m, p, st) : launch_t<D, F16, false, 1>(m, p, st);
  return cap ? launch_t<D, F16, true, 2>(m, p, st) : launch_t<D, F16, false, 2>(m, p, st);
}

}  // namespace bwd
}  // namespace lh
