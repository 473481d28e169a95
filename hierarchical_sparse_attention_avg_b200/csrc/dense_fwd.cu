// dense_fwd.cu — the dense stage's attention, forward, on the tcgen05 tensor cores.
//
//   O = softmax(Z + mask) V,  Z = cap tanh(scale Q K^T / cap) + bias(h, x - j),  LSE = log sum exp Z
//
// in one pass over the keys with a running maximum and sum per row.  One block per (batch, head group, pair of 128-row
// query tiles, share of the keys), warp roles as in the gathered attention: warp 0 TMA producer, warp 1 MMA issuer,
// warps 2-5 and 6-9 the softmax of "stream" 0 and 1, one query row (= TMEM lane) per thread.  A stream has its own
// scores S (128 fp32 TMEM columns, the probabilities written over them as the A operand of the next product) and its
// own accumulator O, so the tensor core works for one stream while the other's exponentials run.
//
// - Long queries: the two streams are two query tiles over the same keys.
// - At most one query tile per head group (single tokens, short chunks): both streams take the same queries, stream 0
//   the even and stream 1 the odd key tiles of the block (`dual`), and are joined through shared memory at the end; the
//   query heads of one key head share the 128 rows (`pack`), so the cache is read once for all of them; and where the
//   blocks are fewer than the SMs, `nsplit` blocks share the keys, each writes its normalised fp32 rows and their LSE,
//   and join_kernel adds them with weights exp(LSE - max LSE).
//
// The block first classes its key tiles for each stream (invisible / partly masked / distances of several buckets), one
// byte each in shared memory, from the lengths and the ids' ranges of the tiles; every role walks the visible ones.
// Scores are formed in the log2 domain.  A tile inside one bucket adds one constant per row; a tile across buckets
// reads the bias from a window of distances in shared memory; slopes are one packed FMA on top.
//
// Masked places: a masked score is overwritten after it is computed, whatever it was.  A value row that is not finite
// would still reach other rows through 0 * inf, so in tiles with masked pairs the softmax threads clear such rows of V
// in shared memory before the product (dead rows for good; others are added to the rows that see them at the end).
//
// Precision: Q, K, V enter as they are, scores and statistics fp32; the probabilities are rounded once to the operands'
// type (2^-9 bf16, 2^-12 fp16 relative) as both operands of one tensor-core product must share it, and lie in
// [0, 2^8] against a reference maximum that moves only when exceeded by more than 2^8.
#include "dense.cuh"

namespace lh {

namespace {

constexpr int kThreads = 320;
constexpr int kTile = 128;
constexpr int kMaxStages = 4;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kSlack = 8.0f;
constexpr int kHeadFastBelow = 512;  // as in the gathered attention: heads fastest, heaviest tiles first, below this
constexpr int kSms = 148;

// flag byte of a key tile: bit q visible to stream q, 2 + q some pair masked, 4 + q distances of several buckets (or
// signs, with slopes), 6 + q some value row not finite (set by the softmax threads)
constexpr int kSees = 1, kMasked = 4, kNear = 16, kBad = 64;

enum { kBQ = 0, kBKF = 1, kBKE = 5, kBVF = 9, kBVE = 13, kBSF = 17, kBPF = 19, kBOD = 21, kBDrain = 23, kNBar = 24 };

struct FwdArgs {
  DenseDims a;
  int pack, tok, ntile, npair, nsplit, dual, head_fast, nst;
  uint32_t off_k, off_v, off_bar, off_ids, off_win, off_flags;
  int win;  // floats of one stream's bias window
  DenseTensor v;
  DenseTensor o, low;
  float* lse;
  const int2* kdoc;
  float *part_o, *part_lse;
};

template <int D, bool F16, bool CAP, int BIAS>
__global__ void __launch_bounds__(kThreads, 1)
    dense_fwd_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                     const __grid_constant__ CUtensorMap tmV, const __grid_constant__ FwdArgs p,
                     const __grid_constant__ BucketStarts starts) {
  constexpr uint32_t TILE = kTile * D * 2;
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint32_t s_tmem;
  __shared__ WaitCtl s_wait;
  __shared__ BucketStarts s_bs;
  __shared__ int s_first, s_last, s_qlo[2], s_qhi[2];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sb = smem_u32(smem);
  auto bar = [&](int i) { return sb + p.off_bar + 8u * i; };
  uint8_t* flags = smem + p.off_flags;
  const DenseDims& a = p.a;
  int* status = a.status;

  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int pt = p.npair - 1 - (int)(p.head_fast ? blockIdx.y : blockIdx.x);  // heaviest first
  const int bh = p.head_fast ? blockIdx.x : blockIdx.y;
  const int split = blockIdx.z;
  const int nhp = a.Hq / p.pack;
  const int b = bh / nhp, hp = bh % nhp, kvh = hp * p.pack / a.G;
  const int len = dense_len(a, b), prefix = dense_prefix(a, b, len), off = len - a.Sq;
  const int tile0 = p.dual ? pt : 2 * pt;
  const int nstream = p.dual || tile0 + 1 < p.ntile ? 2 : 1;
  auto tok0 = [&](int q) { return (p.dual ? tile0 : tile0 + q) * p.tok; };
  const int nk = (len + kTile - 1) / kTile, per = (nk + p.nsplit - 1) / p.nsplit;
  const int ks = split * per, ke = min(nk, ks + per);  // key tiles of this block

  if (threadIdx.x == 0) {
    wait_ctl_init(&s_wait, status);
    mbar_init(bar(kBQ), 1);
    for (int i = 0; i < p.nst; ++i) {
      mbar_init(bar(kBKF + i), 1);
      mbar_init(bar(kBKE + i), 1);
      mbar_init(bar(kBVF + i), 1);
      mbar_init(bar(kBVE + i), 1);
    }
    for (int q = 0; q < 2; ++q) {
      mbar_init(bar(kBSF + q), 1);
      mbar_init(bar(kBPF + q), kTile);
      mbar_init(bar(kBOD + q), 1);
      s_qlo[q] = INT32_MAX;
      s_qhi[q] = -1;
    }
    mbar_init(bar(kBDrain), 1);
    fence_mbar_init();
    s_first = INT32_MAX;
    s_last = -1;
    prefetch_tmap(&tmQ);
    prefetch_tmap(&tmK);
    prefetch_tmap(&tmV);
  }
  if (warp == 1) tmem_alloc(smem_u32(&s_tmem), 512);
  if (BIAS == 2)
    for (int i = threadIdx.x; i < kMaxBuckets + 2; i += kThreads)
      reinterpret_cast<int*>(&s_bs)[i] = reinterpret_cast<const int*>(&starts)[i];
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s_tmem;  // columns: S/P of stream q at 128 q, O at 256 + 128 q

  // Class every key tile for both streams.
  if (a.docs) {
    for (int i = threadIdx.x; i < 2 * p.tok; i += kThreads) {
      const int q = i / p.tok, t = tok0(q) + i % p.tok;
      if (q < nstream && t < a.Sq) {
        const int id = max(doc_at(a, b, off + t, len), -1);
        atomicMin(&s_qlo[q], id);
        atomicMax(&s_qhi[q], id);
      }
    }
    __syncthreads();
  }
  for (int t = ks + threadIdx.x; t < ke; t += kThreads) {
    const int j0 = t * kTile;
    int f = 0;
    for (int q = 0; q < nstream; ++q) {
      if (p.dual && ((t - ks) & 1) != q) continue;
      const int xa = off + tok0(q), xb = off + min(tok0(q) + p.tok, a.Sq) - 1;
      if (j0 > last_key(a, xb, len, prefix)) continue;
      bool whole = j0 + kTile - 1 <= last_key(a, xa, len, prefix);
      if (a.docs) {
        const int2 kd = __ldg(p.kdoc + (int64_t)b * ((a.Skv + kTile - 1) / kTile) + t), qd = make_int2(s_qlo[q], s_qhi[q]);
        if (!docs_meet(kd, qd)) continue;
        whole = whole && docs_one(kd, qd);
      }
      f |= kSees << q;
      if (!whole) f |= kMasked << q;
      const int dmin = xa - (j0 + kTile - 1), dmax = xb - j0;
      if (BIAS == 1 && dmin < 0) f |= kNear << q;
      if (BIAS == 2 && bucket_of(s_bs, dmin) != bucket_of(s_bs, dmax)) f |= kNear << q;
    }
    flags[t - ks] = (uint8_t)f;
    if (f) {
      atomicMin(&s_first, t);
      atomicMax(&s_last, t);
    }
  }
  __syncthreads();
  const int last = s_last;
  auto next = [&](int t) {  // the next visible tile after t (> last: none)
    for (++t; t <= last && !(flags[t - ks] & 3); ++t) {}
    return t;
  };
  const int first = last >= 0 ? s_first : 1;  // first > last when there is none
  struct Ring {  // stage and phase of the n-th tile
    int s = 0, ph = 0;
    __device__ void step(int nst) {
      if (++s == nst) s = 0, ph ^= 1;
    }
  };

  if (warp == 0) {
    // ---------------------------------------------------------------- TMA producer
    if (lane == 0 && first <= last) {
      bool ok = true;
      const int nqt = p.dual ? 1 : nstream;
      mbar_arrive_expect_tx(bar(kBQ), nqt * p.pack * p.tok * D * 2);
      for (int q = 0; q < nqt; ++q)
        for (int db = 0; db < D / 64; ++db)
          tma_load_5d(sb + q * TILE + db * 16384, &tmQ, bar(kBQ), db * 64, 0, tok0(q), hp, b);
      int n = 0;
      Ring r;
      for (int t = first; t <= last; t = next(t), ++n, r.step(p.nst)) {
        const uint32_t free_ph = r.ph ^ 1;
        if (n >= p.nst) ok = mbar_wait(bar(kBKE + r.s), free_ph, &s_wait, status);
        if (!ok) break;
        mbar_arrive_expect_tx(bar(kBKF + r.s), TILE);
        for (int db = 0; db < D / 64; ++db)
          tma_load_5d(sb + p.off_k + r.s * TILE + db * 16384, &tmK, bar(kBKF + r.s), db * 64, 0, t * kTile, kvh, b);
        if (n >= p.nst) ok = mbar_wait(bar(kBVE + r.s), free_ph, &s_wait, status);
        if (!ok) {
          mbar_wait_teardown(bar(kBKF + r.s), r.ph);
          break;
        }
        mbar_arrive_expect_tx(bar(kBVF + r.s), TILE);
        for (int db = 0; db < D / 64; ++db)
          tma_load_5d(sb + p.off_v + r.s * TILE + db * 16384, &tmV, bar(kBVF + r.s), db * 64, 0, t * kTile, kvh, b);
      }
      if (!ok) {  // drain the copies this thread issued before leaving
        mbar_wait_teardown(bar(kBQ), 0);
        for (int m = n > p.nst ? n - p.nst : 0; m < n; ++m) {
          mbar_wait_teardown(bar(kBKF + m % p.nst), (m / p.nst) & 1);
          mbar_wait_teardown(bar(kBVF + m % p.nst), (m / p.nst) & 1);
        }
      }
    }
  } else if (warp == 1) {
    // ---------------------------------------------------------------- MMA issuer
    if (lane == 0 && first <= last) {
      constexpr int fmt = F16 ? kFmtF16 : kFmtBF16;
      constexpr uint32_t idesc_qk = idesc_f32acc(fmt, 128, 128, 0, 0);
      constexpr uint32_t idesc_pv = idesc_f32acc(fmt, 128, D, 0, 1);
      auto mma_s = [&](int q, int stage) {  // S_q = Q_q K^T
        const uint32_t sQ = sb + (p.dual ? 0 : q) * TILE, sK = sb + p.off_k + stage * TILE;
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t ko = (kk >> 2) * 16384 + (kk & 3) * 32;
          umma_ss(tmem + 128 * q, sdesc_sw128(sQ + ko, 16, 1024), sdesc_sw128(sK + ko, 16, 1024), idesc_qk,
                  kk > 0 ? 1u : 0u);
        }
        umma_commit(bar(kBSF + q));
      };
      auto mma_pv = [&](int q, int stage, bool add) {  // O_q (+)= P_q V
        const uint32_t sV = sb + p.off_v + stage * TILE;
#pragma unroll
        for (int kk = 0; kk < kTile / 16; ++kk)
          umma_ts(tmem + 256 + 128 * q, tmem + 128 * q + kk * 8, sdesc_sw128(sV + kk * 2048, 16384, 1024), idesc_pv,
                  (add || kk > 0) ? 1u : 0u);
      };
      // the scores of a stream's next tile are issued right behind its product: one tile ahead, or, when the tiles
      // alternate between the streams, two
      const int ahead = p.dual ? 2 : 1;
      int ta = first;
      Ring ra, r;
      bool ok = mbar_wait(bar(kBQ), 0, &s_wait, status);
      for (int i = 0; i < ahead && ta <= last && ok; ++i) {
        ok = mbar_wait(bar(kBKF + ra.s), ra.ph, &s_wait, status);
        if (!ok) break;
        tc_fence_after();
        const int f = flags[ta - ks];
        for (int q = 0; q < 2; ++q)
          if (f >> q & 1) mma_s(q, ra.s);
        umma_commit(bar(kBKE + ra.s));
        ta = next(ta);
        ra.step(p.nst);
      }
      int cnt[2] = {0, 0};
      for (int t = first; t <= last && ok; t = next(t), r.step(p.nst)) {
        const int f = flags[t - ks], fa = ta <= last ? flags[ta - ks] : 0;
        ok = mbar_wait(bar(kBVF + r.s), r.ph, &s_wait, status);
        bool k_here = false;
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          if (ok && (f >> q & 1)) {
            ok = mbar_wait(bar(kBPF + q), cnt[q] & 1, &s_wait, status);
            if (ok) {
              tc_fence_after();
              mma_pv(q, r.s, cnt[q] > 0);
              ++cnt[q];
            }
          }
          if (ok && (fa >> q & 1)) {
            if (!k_here) ok = mbar_wait(bar(kBKF + ra.s), ra.ph, &s_wait, status);
            k_here = true;
            if (ok) {
              tc_fence_after();
              mma_s(q, ra.s);
            }
          }
        }
        if (!ok) break;
        umma_commit(bar(kBVE + r.s));
        if (ta <= last) {
          umma_commit(bar(kBKE + ra.s));
          ta = next(ta);
          ra.step(p.nst);
        }
      }
      umma_commit(bar(kBOD + 0));
      umma_commit(bar(kBOD + 1));
      umma_commit(bar(kBDrain));  // every product issued above completes before the block releases its memory
      mbar_wait_teardown(bar(kBDrain), 0);
    }
  } else {
    // ---------------------------------------------------------------- softmax (warps 2..5: stream 0, 6..9: stream 1)
    const int q = (warp - 2) >> 2;
    if (q < nstream) {
      const int quarter = warp & 3;  // TMEM lane quarter this warp may access
      const int row = quarter * 32 + lane;
      const uint32_t lane_base = (uint32_t)(quarter * 32) << 16;
      const uint32_t tS = tmem + 128 * q + lane_base, tO = tmem + 256 + 128 * q + lane_base;
      const int tl = row / p.pack, g = row - tl * p.pack, tk = tok0(q) + tl;
      const bool valid = tl < p.tok && tk < a.Sq;
      const bool active = __any_sync(0xffffffffu, valid);  // a warp without a row only keeps the hand-offs going
      const int x = off + tk, h = hp * p.pack + g;
      const int jlast = valid ? last_key(a, x, len, prefix) : -1;
      const int mydoc = valid ? doc_at(a, b, x, len) : -1;
      const float mul0 = CAP ? a.cap * kLog2e : a.scale * kLog2e;
      const float cap_in = 2.f * kLog2e * a.scale / (CAP ? a.cap : 1.f);
      const float slope2 = BIAS == 1 ? -__ldg(a.slopes + h) * kLog2e : 0.f;
      const int64_t trow = (int64_t)h * a.buckets;
      int* ids = reinterpret_cast<int*>(smem + p.off_ids) + q * kTile;
      float* win = reinterpret_cast<float*>(smem + p.off_win) + q * p.win;
      float m_run = -INFINITY, l_run = 0.f;
      bool ok = true;
      int cnt = 0;
      Ring r;
      for (int t = first; t <= last; t = next(t), r.step(p.nst)) {
        const int f = flags[t - ks];
        if (!(f >> q & 1)) continue;
        const bool masked = f & (kMasked << q), near = BIAS && (f & (kNear << q));
        const int j0 = t * kTile;
        bool dead = false;
        float cadd = 0.f;
        // what the tile needs besides its scores, fetched before they are waited for
        if ((masked && a.docs) || (BIAS == 2 && near)) {
          ok = named_barrier_and(1 + q, kTile, ok);  // the last tile's ids and window are done with
          if (masked && a.docs) {
            const int id = doc_at(a, b, j0 + row, len);
            ids[row] = id < 0 ? -2 : id;
            dead = id < 0;
          }
          if (BIAS == 2 && near) {  // distances of the tile's rows and keys, one run of tok + 127 per head
            const int w = p.tok + kTile - 1, d0 = off + tok0(q) - j0 - (kTile - 1);
            for (int i = row; i < p.pack * w; i += kTile) {
              const int gi = i / w;
              win[i] = kLog2e * table_at<F16>(a.table, (int64_t)(hp * p.pack + gi) * a.buckets +
                                                           bucket_of(s_bs, d0 + i - gi * w));
            }
          }
          ok = named_barrier_and(1 + q, kTile, ok);
        }
        if (masked && j0 + row >= len) dead = true;
        if (BIAS == 2 && !near && active) cadd = kLog2e * table_at<F16>(a.table, trow + bucket_of(s_bs, x - j0));
        if (ok) ok = __all_sync(0xffffffffu, mbar_wait(bar(kBSF + q), cnt & 1, &s_wait, status));
        if (!ok) continue;  // (the group's later barriers still count this warp)
        tc_fence_after();
        if (active) {
          float s[4][32];
#pragma unroll
          for (int c = 0; c < 4; ++c) tmem_ld32(tS + c * 32, s[c]);
          tmem_ld_wait();
          float mul = mul0;
          if (CAP) {
#pragma unroll
            for (int c = 0; c < 4; ++c)
#pragma unroll
              for (int i = 0; i < 32; ++i) s[c][i] = fmaf(-2.f, rcp_approx(1.f + ex2(s[c][i] * cap_in)), 1.f);
          }
          if (BIAS == 1) {
            if (near) {
#pragma unroll
              for (int c = 0; c < 4; ++c)
#pragma unroll
                for (int i = 0; i < 32; ++i)
                  s[c][i] = fmaf(s[c][i], mul, slope2 * fabsf((float)(x - j0 - (c * 32 + i))));
            } else {
              const float base = slope2 * (float)(x - j0);
              const uint64_t mul2 = f2pack(mul, mul), ns2 = f2pack(-slope2, -slope2), base2 = f2pack(base, base);
#pragma unroll
              for (int c = 0; c < 4; ++c)
#pragma unroll
                for (int i = 0; i < 32; i += 2) {
                  const uint64_t bb = fma_f32x2(f2pack((float)(c * 32 + i), (float)(c * 32 + i + 1)), ns2, base2);
                  const uint64_t v = fma_f32x2(f2pack(s[c][i], s[c][i + 1]), mul2, bb);
                  s[c][i] = f2lo(v);
                  s[c][i + 1] = f2hi(v);
                }
            }
            mul = 1.f;
          }
          if (BIAS == 2 && near) {
            const float* wr = win + g * (p.tok + kTile - 1) + min(tl, p.tok - 1) + kTile - 1;
#pragma unroll
            for (int c = 0; c < 4; ++c)
#pragma unroll
              for (int i = 0; i < 32; ++i) s[c][i] = fmaf(s[c][i], mul, wr[-(c * 32 + i)]);
            mul = 1.f;
          }
          if (masked) {
            const int jl = jlast - j0;
#pragma unroll
            for (int c = 0; c < 4; ++c)
#pragma unroll
              for (int i = 0; i < 32; ++i)
                if (c * 32 + i > jl) s[c][i] = -INFINITY;
            if (a.docs) {
#pragma unroll
              for (int c = 0; c < 4; ++c)
#pragma unroll
                for (int i = 0; i < 32; i += 4) {
                  const int4 kd = *reinterpret_cast<const int4*>(ids + c * 32 + i);
                  if (kd.x != mydoc) s[c][i] = -INFINITY;
                  if (kd.y != mydoc) s[c][i + 1] = -INFINITY;
                  if (kd.z != mydoc) s[c][i + 2] = -INFINITY;
                  if (kd.w != mydoc) s[c][i + 3] = -INFINITY;
                }
            }
          }
          // row max as 8 independent chains of three-input maxima
          auto col = [&](int i) { return s[i >> 5][i & 31]; };
          float mx8[8];
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            float m = fmax3(col(k), col(k + 8), col(k + 16));
#pragma unroll
            for (int i = 3; i + 1 < 16; i += 2) m = fmax3(m, col(k + 8 * i), col(k + 8 * i + 8));
            mx8[k] = fmaxf(m, col(k + 120));
          }
          const float mx = fmaf(fmax3(fmax3(mx8[0], mx8[1], mx8[2]), fmax3(mx8[3], mx8[4], mx8[5]),
                                      fmaxf(mx8[6], mx8[7])), mul, cadd);
          float alpha = 1.0f;
          const bool move = __any_sync(0xffffffffu, mx > m_run + kSlack);
          if (move) {
            const float m_new = fmaxf(m_run, mx);
            alpha = m_run == -INFINITY ? 0.f : ex2(m_run - m_new);
            l_run *= alpha;
            m_run = m_new;
          }
          // P over the first 64 columns of S, and its row sum; a row that has seen no key yet keeps P = 0
          const float sub = cadd - (m_run == -INFINITY ? 0.f : m_run);
          uint64_t rs2[4] = {0ull, 0ull, 0ull, 0ull};
          const uint64_t mul2 = f2pack(mul, mul), sub2 = f2pack(sub, sub), one2 = f2pack(1.f, 1.f);
#pragma unroll
          for (int hh = 0; hh < 2; ++hh) {
            float pk[32];
#pragma unroll
            for (int c = 2 * hh; c < 2 * hh + 2; ++c)
#pragma unroll
              for (int i = 0; i < 32; i += 2) {
                const uint64_t arg = fma_f32x2(f2pack(s[c][i], s[c][i + 1]), mul2, sub2);
                const float p0 = ex2(f2lo(arg)), p1 = ex2(f2hi(arg));
                rs2[(i >> 1) & 3] = fma_f32x2(f2pack(p0, p1), one2, rs2[(i >> 1) & 3]);
                pk[(c & 1) * 16 + i / 2] = __uint_as_float(pack2_rn<F16>(p0, p1));
              }
            tmem_st32(tS + 32 * hh, pk);
          }
          // O_q's last product has completed (it was issued before these scores): bring O_q to the new maximum
          if (cnt > 0 && move) {
#pragma unroll
            for (int c = 0; c < D / 32; ++c) {
              float o[32];
              tmem_ld32(tO + c * 32, o);
              tmem_ld_wait();
#pragma unroll
              for (int i = 0; i < 32; ++i) o[i] *= alpha;
              tmem_st32(tO + c * 32, o);
            }
          }
          tmem_st_wait();
          float rs[8] = {f2lo(rs2[0]), f2hi(rs2[0]), f2lo(rs2[1]), f2hi(rs2[1]),
                         f2lo(rs2[2]), f2hi(rs2[2]), f2lo(rs2[3]), f2hi(rs2[3])};
          l_run += ((rs[0] + rs[1]) + (rs[2] + rs[3])) + ((rs[4] + rs[5]) + (rs[6] + rs[7]));
        }
        if (masked) {  // value rows that may meet a probability of zero: clear what is not finite (thread = row)
          ok = __all_sync(0xffffffffu, mbar_wait(bar(kBVF + r.s), r.ph, &s_wait, status));
          if (!ok) continue;
          uint8_t* vr = smem + p.off_v + r.s * TILE + row * 128;
          uint32_t bad = 0;
          if (!dead) {
#pragma unroll
            for (int i = 0; i < D / 8; ++i) {
              const uint4 w = *reinterpret_cast<const uint4*>(vr + (i >> 3) * 16384 + (((i + lane) & 7) << 4));
              bad |= nonfinite2<F16>(w.x) | nonfinite2<F16>(w.y) | nonfinite2<F16>(w.z) | nonfinite2<F16>(w.w);
            }
          }
          if (dead) {
#pragma unroll
            for (int i = 0; i < D / 8; ++i)
              *reinterpret_cast<uint4*>(vr + (i >> 3) * 16384 + (((i + lane) & 7) << 4)) = make_uint4(0, 0, 0, 0);
          } else if (bad) {
            for (int i = 0; i < D; ++i) {
              unsigned short* e = reinterpret_cast<unsigned short*>(vr + (i >> 6) * 16384) + (i & 63);
              if (nonfinite2<F16>(*e)) *e = 0;
            }
            atomicOr(reinterpret_cast<unsigned int*>(flags) + ((t - ks) >> 2), (unsigned)(kBad << q) << (8 * ((t - ks) & 3)));
          }
          fence_proxy_async_smem();
        }
        tc_fence_before();
        mbar_arrive(bar(kBPF + q));
        ++cnt;
      }

      // ---- epilogue: the last product, the join of the streams, the rows
      if (ok && first <= last) ok = mbar_wait(bar(kBOD + q), 0, &s_wait, status);
      ok = __all_sync(0xffffffffu, ok);
      tc_fence_after();
      float l1 = 0.f, a0 = 1.f, a1 = 0.f;
      float* so = reinterpret_cast<float*>(smem + p.off_k);  // [D][128] of stream 1 (the keys are consumed)
      float* sm = reinterpret_cast<float*>(smem + p.off_v);  // [2][128] its maxima and sums
      if (p.dual) {
        if (q == 1 && ok && active) {
          sm[row] = m_run;
          sm[kTile + row] = l_run;
          if (cnt > 0) {
#pragma unroll
            for (int c = 0; c < D / 32; ++c) {
              float o[32];
              tmem_ld32(tO + c * 32, o);
              tmem_ld_wait();
#pragma unroll
              for (int i = 0; i < 32; ++i) so[(c * 32 + i) * kTile + row] = o[i];
            }
          }
        }
        ok = named_barrier_and(3, 2 * kTile, ok);
        if (q == 0 && ok && active) {
          const float m1 = sm[row], m = fmaxf(m_run, m1);
          l1 = sm[kTile + row];
          if (m != -INFINITY) {
            a0 = m_run == -INFINITY ? 0.f : ex2(m_run - m);
            a1 = m1 == -INFINITY ? 0.f : ex2(m1 - m);
          }
          l_run = l_run * a0 + l1 * a1;
          m_run = m;
        }
      } else {
        ok = named_barrier_and(1 + q, kTile, ok);  // the group's flags of tiles with values that are not finite
      }
      if (ok && active && (q == 0 || !p.dual)) {
        const float inv = l_run == 0.f ? 0.f : 1.0f / l_run;
        const int64_t ri = ((int64_t)b * a.Hq + h) * a.Sq + tk;
        const bool part = p.nsplit > 1;
        const int64_t pi = (int64_t)split * a.B * a.Hq * a.Sq + ri;
        auto at = [&](const DenseTensor& t) {
          return static_cast<uint16_t*>(const_cast<void*>(t.p)) + b * t.st.b + h * t.st.h + (int64_t)tk * t.st.s;
        };
        uint16_t *orow = at(p.o), *lrow = p.low.p ? at(p.low) : nullptr;
        float* prow = part ? p.part_o + pi * D : nullptr;
        const bool use1 = p.dual && a1 != 0.f;
        const float c0 = cnt > 0 ? a0 * inv : 0.f, c1 = a1 * inv;
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
          float o[32];
          if (cnt > 0) {
            tmem_ld32(tO + c * 32, o);
            tmem_ld_wait();
          }
#pragma unroll
          for (int i = 0; i < 32; ++i) o[i] = inv == 0.f || cnt == 0 ? 0.f : o[i] * c0;
          if (use1 && inv != 0.f) {
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] = fmaf(so[(c * 32 + i) * kTile + row], c1, o[i]);
          }
          if (valid) {
            if (part) {
#pragma unroll
              for (int i = 0; i < 32; i += 4)
                *reinterpret_cast<float4*>(prow + c * 32 + i) = make_float4(o[i], o[i + 1], o[i + 2], o[i + 3]);
            } else {
#pragma unroll
              for (int i = 0; i < 32; i += 8)
                store8<F16>(orow + c * 32 + i, lrow ? lrow + c * 32 + i : nullptr, o + i);
            }
          }
        }
        if (valid) {
          const float l2 = l_run == 0.f ? -INFINITY : m_run + __log2f(l_run);
          if (part) p.part_lse[pi] = l2;
          else p.lse[ri] = l2 * kLn2;
          // values that are not finite, added to the rows that see them (rare)
          for (int t = first; t <= last; ++t) {
            if (!(flags[t - ks] & (p.dual ? 3 * kBad : kBad << q))) continue;
            for (int j = t * kTile; j < min((t + 1) * kTile, jlast + 1); ++j) {
              if (a.docs && (mydoc < 0 || doc_at(a, b, j, len) != mydoc)) continue;
              const uint16_t* vr = static_cast<const uint16_t*>(p.v.p) + b * p.v.st.b + kvh * p.v.st.h + j * p.v.st.s;
              for (int i = 0; i < D; ++i) {
                const uint32_t w = vr[i];
                if (!nonfinite2<F16>(w)) continue;
                const float vv = unpack2<F16>(w).x;
                if (part) prow[i] += vv;
                else orow[i] = (uint16_t)pack2_rn<F16>(unpack2<F16>(orow[i]).x + vv, 0.f);
              }
            }
          }
        }
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Joins the splits of a row: one block per row, its warps over the splits, then over shared memory.  Reads
// nsplit (d + 1) floats a row; latency-bound (a few rows per SM).
template <int D, bool F16>
__global__ void __launch_bounds__(128) join_kernel(const float* __restrict__ part_o, const float* __restrict__ part_lse,
                                                   DenseTensor o, DenseTensor low, float* __restrict__ lse, int nsplit,
                                                   int64_t rows, int Hq, int Sq) {
  const int64_t row = blockIdx.x;
  const int w = threadIdx.x / 32, lane = threadIdx.x % 32;
  constexpr int E = D / 32;
  __shared__ float s_acc[4][D], s_l[4];
  float m = -INFINITY;
  for (int s = lane; s < nsplit; s += 32) m = fmaxf(m, part_lse[s * rows + row]);
#pragma unroll
  for (int i = 16; i; i >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, i));
  const float mm = m == -INFINITY ? 0.f : m;
  float acc[E] = {}, l = 0.f;
#pragma unroll 4
  for (int s = w; s < nsplit; s += 4) {
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
  for (int i = 0; i < E; ++i) s_acc[w][lane * E + i] = acc[i];
  if (lane == 0) s_l[w] = l;
  __syncthreads();
  const float lt = (s_l[0] + s_l[1]) + (s_l[2] + s_l[3]), inv = lt == 0.f ? 0.f : 1.0f / lt;
  const int64_t tk = row % Sq, bh = row / Sq, h = bh % Hq, b = bh / Hq;
  auto at = [&](const DenseTensor& t) {
    return static_cast<uint16_t*>(const_cast<void*>(t.p)) + b * t.st.b + h * t.st.h + tk * t.st.s;
  };
  const int i = threadIdx.x * 8;
  if (i < D) {
    float v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e)
      v[e] = ((s_acc[0][i + e] + s_acc[1][i + e]) + (s_acc[2][i + e] + s_acc[3][i + e])) * inv;
    store8<F16>(at(o) + i, low.p ? at(low) + i : nullptr, v);
  }
  if (threadIdx.x == 0) lse[row] = lt == 0.f ? -INFINITY : (m + __log2f(lt)) * kLn2;
}

template <int D, bool F16, bool CAP, int BIAS>
int launch_t(const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mv, const FwdArgs& p,
             const BucketStarts& bs, int smem, cudaStream_t st) {
  auto kernel = dense_fwd_kernel<D, F16, CAP, BIAS>;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
    return LH_ERR_CUDA;
  const int nbh = p.a.B * (p.a.Hq / p.pack);
  const dim3 grid = p.head_fast ? dim3(nbh, p.npair, p.nsplit) : dim3(p.npair, nbh, p.nsplit);
  kernel<<<grid, kThreads, smem, st>>>(mq, mk, mv, p, bs);
  return check_launch();
}
template <int D, bool F16>
int launch_d(const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mv, const FwdArgs& p,
             const BucketStarts& bs, int smem, cudaStream_t st) {
  const int bias = p.a.slopes ? 1 : p.a.table ? 2 : 0;
  const bool cap = p.a.cap > 0.f;
  if (bias == 0) return cap ? launch_t<D, F16, true, 0>(mq, mk, mv, p, bs, smem, st)
                            : launch_t<D, F16, false, 0>(mq, mk, mv, p, bs, smem, st);
  if (bias == 1) return cap ? launch_t<D, F16, true, 1>(mq, mk, mv, p, bs, smem, st)
                            : launch_t<D, F16, false, 1>(mq, mk, mv, p, bs, smem, st);
  return cap ? launch_t<D, F16, true, 2>(mq, mk, mv, p, bs, smem, st)
             : launch_t<D, F16, false, 2>(mq, mk, mv, p, bs, smem, st);
}

}  // namespace

DenseFwdPlan dense_fwd_plan(const DenseDims& a) {
  DenseFwdPlan f;
  // Fewer tokens than a query tile has rows: the query heads of a key head share tiles (at most 16 of them, so that
  // the bias windows of a tile's heads stay small).
  f.pack = 1;
  if (a.Sq < kTile)
    for (int g = 1; g <= 16 && g <= a.G; ++g)
      if (a.G % g == 0) f.pack = g;
  f.tok = kTile / f.pack;
  f.ntile = (a.Sq + f.tok - 1) / f.tok;
  f.dual = f.ntile == 1;
  const int npair = f.dual ? 1 : (f.ntile + 1) / 2;
  const int64_t blocks = (int64_t)a.B * (a.Hq / f.pack) * npair;
  const int nk = (a.Skv + kTile - 1) / kTile;
  // Too few blocks for the SMs: as many shares of the keys as fill them once, of four tiles at least.
  f.nsplit = 1;
  if (blocks <= kSms / 2) {
    f.nsplit = (int)(kSms / blocks);
    if (f.nsplit > (nk + 3) / 4) f.nsplit = (nk + 3) / 4;
    if (f.nsplit < 1) f.nsplit = 1;
  }
  return f;
}

int launch_dense_fwd(const DenseDims& a, const BucketStarts& bs, const DenseTensor& q, const DenseTensor& k,
                     const DenseTensor& v, const DenseTensor& o, const DenseTensor& low, float* lse, const int2* kdoc,
                     float* part_o, float* part_lse, cudaStream_t st) {
  const DenseFwdPlan f = dense_fwd_plan(a);
  CUtensorMap mq, mk, mv;
  if (make_tmap_dense(&mq, q, a.d, a.Sq, a.Hq, a.B, f.pack, f.tok) ||
      make_tmap_dense(&mk, k, a.d, a.Skv, a.Hkv, a.B, 1, kTile) ||
      make_tmap_dense(&mv, v, a.d, a.Skv, a.Hkv, a.B, 1, kTile))
    return LH_ERR_CUDA;
  FwdArgs p;
  p.a = a;
  p.pack = f.pack;
  p.tok = f.tok;
  p.ntile = f.ntile;
  p.dual = f.dual;
  p.npair = f.dual ? 1 : (f.ntile + 1) / 2;
  p.nsplit = f.nsplit;
  p.head_fast = p.npair < kHeadFastBelow;
  p.nst = a.d == 64 ? 4 : 2;
  const uint32_t tile = kTile * a.d * 2;
  p.off_k = (f.dual ? 1 : 2) * tile;
  p.off_v = p.off_k + p.nst * tile;
  p.off_bar = p.off_v + p.nst * tile;
  p.off_ids = p.off_bar + kNBar * 8;
  p.off_win = p.off_ids + 2 * kTile * 4;
  p.win = a.table ? f.pack * (f.tok + kTile - 1) : 0;
  p.off_flags = p.off_win + 2 * p.win * 4;
  p.v = v;
  p.o = o;
  p.low = low;
  p.lse = lse;
  p.kdoc = kdoc;
  p.part_o = part_o;
  p.part_lse = part_lse;
  const int nk = (a.Skv + kTile - 1) / kTile;
  int smem = (int)p.off_flags + ((nk + 3) & ~3) + 1024;
  if (smem < 120 * 1024) smem = 120 * 1024;  // one block (and its 512 tensor-memory columns) per SM
  int rc;
  {
    KernelTimer timer("dense_fwd", st);
    rc = a.d == 64 ? (a.f16 ? launch_d<64, true>(mq, mk, mv, p, bs, smem, st) : launch_d<64, false>(mq, mk, mv, p, bs, smem, st))
                   : (a.f16 ? launch_d<128, true>(mq, mk, mv, p, bs, smem, st) : launch_d<128, false>(mq, mk, mv, p, bs, smem, st));
  }
  if (rc || f.nsplit == 1) return rc;
  KernelTimer timer("dense_join", st);
  const int64_t rows = (int64_t)a.B * a.Hq * a.Sq;
  auto join = a.d == 64 ? (a.f16 ? join_kernel<64, true> : join_kernel<64, false>)
                        : (a.f16 ? join_kernel<128, true> : join_kernel<128, false>);
  join<<<(unsigned)rows, 128, 0, st>>>(part_o, part_lse, o, low, lse, f.nsplit, rows, a.Hq, a.Sq);
  return check_launch();
}

}  // namespace lh
