// dense_fwd.cuh — the dense stage's attention, forward, on the tcgen05 tensor cores.
//
//   O = softmax(Z + mask) V,  Z = cap tanh(scale Q K^T / cap) + bias(h, x - j),  LSE = log sum exp Z
//
// in one pass over the keys with a running maximum and sum per row.  One block per (batch, head group, pair of 128-row
// query tiles, share of the keys) with two "streams".  A stream has its own scores S (128 fp32 TMEM columns, the
// probabilities written over them as the A operand of the next product), its own accumulator O and four softmax warps, one
// query row (= TMEM lane) per thread, so the tensor core works for one stream while the other's exponentials run.  Warps 0
// and 3 are TMA producers, 1 and 2 MMA issuers, 4-7 and 8-11 the streams' softmax; the first four give registers to the
// others (224 a thread: the 128 scores of a row and tile stay in registers).
//
// - Long queries: the two streams are two query tiles over the same keys, from one producer, and one issuer alternates
//   their products.
// - At most one query tile per head group (single tokens, short chunks): both streams take the same queries, stream 0
//   the even and stream 1 the odd key tiles of the block (`dual`), and are joined through shared memory at the end; the
//   query heads of one key head share the 128 rows (`pack`), so the cache is read once for all of them; and where the
//   blocks are fewer than the SMs, `nsplit` blocks share the keys, each writes its normalised fp32 rows and their LSE,
//   and join_kernel adds them with weights exp(LSE - max LSE).  Each stream has a producer, an issuer and a ring of its own.
//   With at most 32 rows (`REP` = 4) the queries stand four times in the tile, once in each lane quarter, and a warp takes
//   the 32 columns of its quarter: the exponentials of a key tile are spread over all four schedulers instead of one
//   (each copy keeps its own maximum, sum and accumulator, with zeros for the other columns' probabilities).
//
// The block first classes its key tiles for each stream (invisible / partly masked / distances of several buckets), one
// byte each in shared memory, from the lengths and the ids' ranges of the tiles; every role walks the visible ones.
// Scores are formed in the log2 domain.  A tile inside one bucket adds one constant per row; a tile across buckets
// reads the bias from a window of distances in shared memory; slopes are one FMA more.
//
// Masked places: a masked score is overwritten after it is computed, whatever it was.  A value row that is not finite
// would still reach other rows through 0 * inf, so in key tiles with masked pairs for either query tile of the block the
// softmax threads of both clear such rows of V in shared memory before their product (dead rows for good; others are added
// to the rows that see them at the end).
//
// Precision: Q, K, V enter as they are, scores and statistics fp32; the probabilities are rounded once to the operands'
// type (by at most 2^-8 bf16, 2^-11 fp16 relative), as both operands of one tensor-core product must share it.  They are taken
// against the running maximum itself, so that a row's largest one is 1 up to fp32 rounding: with a maximum that only moves when exceeded by
// 2^8 the accumulator is rescaled more rarely (269 us instead of 275 at 16 heads of 8,192 causal keys), but <dO, O>, which
// the backward subtracts from nearly equal numbers, then makes bf16 dQ and dK 2.8e-3 off instead of 2.4e-3.
// fp16 probabilities are carried times 2^14, so that the many small ones of a long row beside one large key do not vanish.
#pragma once

#include <atomic>
#include <type_traits>

#include "dense.cuh"

namespace lh {
namespace fwd {

constexpr int kThreads = 384;
constexpr int kTile = 128;
constexpr int kMaxSlots = 12;  // key and value tiles in shared memory
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kLog2e = 1.4426950408889634f;
constexpr int kHeadFastBelow = 512;  // as in the gathered attention: heads fastest, heaviest tiles first, below this
constexpr int kSms = 148;
constexpr uint32_t kSmemLimit = 226 * 1024;  // dynamic shared memory of a block, beside at most 1 KB of static

// flag byte of a key tile: bit q visible to stream q, 2 + q some pair masked, 4 + q distances of several buckets (or
// signs, with slopes), 6 a value row that is not finite was cleared
constexpr int kSees = 1, kMasked = 4, kNear = 16, kBad = 64;

// An exponent is one FMA, score * mul + (shift - maximum), with the second term rounded to a step of the maximum.  Beyond
// this magnitude (of log2) the largest probability would be more than 2^(1/16) off 1, overflow fp16 from 2^25 on, and
// vanish or overflow fp32 from 2^31 on: there the score is rounded before the maximum is taken off.  (The test for it costs
// 1 %, with slopes 2 %: 16,384 rows 569 -> 582 us; a cap of at most 64 without a bias does without.)
constexpr float kFarMax = 1048576.f;

// Registers a thread: 128 * 56 + 256 * 224 = 384 * 168, what the block is launched with.
constexpr int kRegsIssue = 56, kRegsSoftmax = 224;

enum { kBQ = 0, kBFull = 1, kBFree = kBFull + kMaxSlots, kBSF = kBFree + kMaxSlots, kBPF = kBSF + 2, kBOD = kBPF + 4,
       kBDrain = kBOD + 2, kNBar = kBDrain + 2 };

struct FwdMaps {
  CUtensorMap q, k, v, o, low;
};
struct FwdArgs {
  DenseDims a;
  int pack, tok, rep, ntile, npair, nsplit, dual, head_fast, slots;
  uint32_t off_kv, off_bar, off_win, off_flags;
  int win;  // floats of one stream's bias window
  DenseTensor v, o, low;
  float* lse;
  const int2* kdoc;
  float *part_o, *part_lse;
};

// CAP: 0 none, 1 up to kCarefulCap, 2 beyond it; BIAS: 0 none, 1 slopes, 2 table; REP: copies of the queries.
template <int D, bool F16, int CAP, int BIAS, int REP>
__global__ void __launch_bounds__(kThreads, 1)
    dense_fwd_kernel(const __grid_constant__ FwdMaps m, const __grid_constant__ FwdArgs p,
                     const __grid_constant__ BucketStarts starts) {
  constexpr uint32_t TILE = kTile * D * 2;
  constexpr float kShift = F16 ? 14.f : 0.f;  // log2 of what the probabilities are carried times
  constexpr int ROWS = kTile / REP, CH = 4 / REP;  // rows of a copy of the queries; 32-column runs of a thread
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint32_t s_tmem;
  __shared__ WaitCtl s_wait;
  __shared__ BucketStarts s_bs;
  __shared__ int s_first, s_last, s_qlo[2], s_qhi[2], s_qdead[2], s_bad;
  __shared__ int2 s_kdoc[kOwnDocTiles];
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

  auto load = [&](const CUtensorMap* map, int slot, int t) {  // a key or value tile
    mbar_arrive_expect_tx(bar(kBFull + slot), TILE);
    for (int db = 0; db < D / 64; ++db)
      tma_load_5d(sb + p.off_kv + slot * TILE + db * 16384, map, bar(kBFull + slot), db * 64, 0, t * kTile, kvh, b);
  };
  auto load_q = [&]() {
    const int nqt = p.dual ? 1 : nstream;
    mbar_arrive_expect_tx(bar(kBQ), nqt * REP * p.pack * p.tok * D * 2);
    for (int q = 0; q < nqt; ++q)
      for (int db = 0; db < D / 64; ++db)
        for (int c = 0; c < REP; ++c)
          tma_load_5d(sb + q * TILE + db * 16384 + c * ROWS * 128, &m.q, bar(kBQ), db * 64, 0, tok0(q), hp, b);
  };

  if (threadIdx.x == 0) {
    wait_ctl_init(&s_wait, status);
    mbar_init(bar(kBQ), 1);
    for (int i = 0; i < kMaxSlots; ++i) {
      mbar_init(bar(kBFull + i), 1);
      mbar_init(bar(kBFree + i), 1);
    }
    for (int q = 0; q < 2; ++q) {
      mbar_init(bar(kBSF + q), 1);
      mbar_init(bar(kBPF + q), kTile);
      mbar_init(bar(kBPF + 2 + q), kTile);
      mbar_init(bar(kBOD + q), 1);
      s_qlo[q] = INT32_MAX;
      s_qhi[q] = -1;
      s_qdead[q] = 0;
    }
    mbar_init(bar(kBDrain), 1);
    mbar_init(bar(kBDrain + 1), 1);
    fence_mbar_init();
    fence_proxy_async_smem();  // (the first copies may be this thread's)
    s_first = INT32_MAX;
    s_last = -1;
    s_bad = 0;
    if (!a.docs) {  // the last visible tile is known without its flags: its copies go out before anything else
      const int lk = last_key(a, off + min(tok0(nstream - 1) + p.tok, a.Sq) - 1, len, prefix);
      const int t = lk < 0 ? -1 : min(lk / kTile, ke - 1);
      if (t >= ks) {
        load_q();
        const int e = p.dual ? (t - ks) & 1 : 0;
        load(&m.k, e * p.slots, t);
        load(&m.v, e * p.slots + 1, t);
      }
    } else {
      prefetch_tmap(&m.q);
      prefetch_tmap(&m.k);
      prefetch_tmap(&m.v);
    }
  }
  if (warp == 1) tmem_alloc(smem_u32(&s_tmem), 512);
  if (BIAS == 2)
    for (int i = threadIdx.x; i < kMaxBuckets + 2; i += kThreads)
      reinterpret_cast<int*>(&s_bs)[i] = reinterpret_cast<const int*>(&starts)[i];
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s_tmem;  // columns: S/P of stream q at 128 q, O at 256 + 128 q

  // Class every key tile for both streams.  (Ids' ranges of few tiles are taken here: kOwnDocTiles.)
  const int nkt = (a.Skv + kTile - 1) / kTile;
  const bool own_docs = nkt <= kOwnDocTiles;
  if (a.docs) {
    for (int i = threadIdx.x; i < 2 * p.tok; i += kThreads) {
      const int q = i / p.tok, t = tok0(q) + i % p.tok;
      if (q < nstream && t < a.Sq) {
        const int id = doc_at(a, b, off + t, len);
        if (id < 0) {
          s_qdead[q] = 1;
        } else {
          atomicMin(&s_qlo[q], id);
          atomicMax(&s_qhi[q], id);
        }
      }
    }
    if (own_docs)
      for (int t = ks + warp; t < ke; t += kThreads / 32) {
        const int2 r = warp_doc_range(a, b, t * kTile, min(kTile, a.Skv - t * kTile), len, lane);
        if (lane == 0) s_kdoc[t] = r;
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
        const int2 kd = own_docs ? s_kdoc[t] : __ldg(p.kdoc + (int64_t)b * nkt + t), qd = id_range(s_qlo[q], s_qhi[q], s_qdead[q]);
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
  // Tiles are taken from the last to the first: a causal row's own neighbourhood, where slopes and learned biases are
  // largest, comes first, and the maximum seldom moves afterwards.
  const int first = s_first, last = s_last;  // first > last: none
  auto next = [&](int t, int mask) {  // the next tile below t that a stream of `mask` sees (< first: none)
    for (--t; t >= first && !(flags[t - ks] & mask); --t) {}
    return t;
  };
  // Ring e of `slots` tiles carries K, V, K, V, ... of its tiles in that order; in dual blocks stream e has ring e.
  struct Ring {
    int s = 0, ph = 0;
    __device__ __forceinline__ void step(int n) {
      if (++s == n) s = 0, ph ^= 1;
    }
  };

  if (warp < 4) {
    set_regs_dec<kRegsIssue>();
    if (warp == 0 || warp == 3) {
      // ---------------------------------------------------------------- TMA producer of ring e
      const int e = warp == 0 ? 0 : 1, mask = p.dual ? 1 << e : 3;  // of the streams it feeds
      if (lane == 0 && first <= last && (e == 0 || p.dual)) {
        bool ok = true;
        if (e == 0 && a.docs) load_q();
        int n = 0;  // loads
        Ring r;
        for (int t = next(last + 1, mask); t >= first && ok; t = next(t, mask))
          for (int kv = 0; kv < 2; ++kv) {
            const int slot = e * p.slots + r.s;
            if (n >= p.slots) ok = mbar_wait(bar(kBFree + slot), r.ph ^ 1, &s_wait, status);
            if (!ok) break;
            if (a.docs || t != last) load(kv ? &m.v : &m.k, slot, t);  // (else it is on its way)
            ++n;
            r.step(p.slots);
          }
        // every copy has landed before the block lets go of its memory, whoever gave up
        if (e == 0) mbar_wait_teardown(bar(kBQ), 0);
        for (int i = n > p.slots ? n - p.slots : 0; i < n; ++i)
          mbar_wait_teardown(bar(kBFull + e * p.slots + i % p.slots), (i / p.slots) & 1);
      }
    } else {
      // ---------------------------------------------------------------- MMA issuers (whole warps, one lane issuing)
      const int me = warp == 1 ? 0 : 1;
      if (first <= last && (me == 0 || p.dual)) {
        constexpr int fmt = F16 ? kFmtF16 : kFmtBF16;
        constexpr uint32_t idesc_qk = idesc_f32acc(fmt, 128, 128, 0, 0);
        constexpr uint32_t idesc_pv = idesc_f32acc(fmt, 128, D, 0, 1);
        const uint32_t leader = elect_one();
        const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
        const uint64_t dQ = sdesc_sw128(sb, 16, 1024);
        const uint64_t dK = sdesc_sw128(sb + p.off_kv, 16, 1024), dV = sdesc_sw128(sb + p.off_kv, 16384, 1024);
        auto wait = [&](int i, uint32_t ph) {
          return __all_sync(0xffffffffu, mbar_wait(bar(i), ph, &s_wait, status)) != 0;
        };
        auto scores = [&](int q, int slot) {  // S_q = Q_q K^T
          const uint64_t q0 = dQ + (p.dual ? 0 : q) * (TILE >> 4), k0 = dK + slot * (TILE >> 4);
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint32_t ko = ((kk >> 2) * 16384 + (kk & 3) * 32) >> 4;
            umma_ss_by(leader, tm + 128 * q, q0 + ko, k0 + ko, idesc_qk, kk > 0 ? 1u : 0u);
          }
          umma_commit_by(leader, bar(kBSF + q));
        };
        // O_q (+)= P_q V, the keys of each half of the tile as soon as their probabilities are there
        auto values = [&](int q, int slot, bool add, uint32_t ph) {
          const uint64_t v0 = dV + slot * (TILE >> 4);
#pragma unroll
          for (int hh = 0; hh < 2; ++hh) {
            if (!wait(kBPF + 2 * hh + q, ph)) return false;
            tc_fence_after();
#pragma unroll
            for (int kk = 4 * hh; kk < 4 * hh + 4; ++kk)
              umma_ts_by(leader, tm + 256 + 128 * q, tm + 128 * q + kk * 8, v0 + kk * (2048 >> 4), idesc_pv,
                         (add || kk > 0) ? 1u : 0u);
          }
          return true;
        };
        // A stream's next scores are issued right behind its product: they overwrite P once the product has read it, and
        // their commit tells the softmax that the product is done.
        bool ok = wait(kBQ, 0);
        Ring r;
        if (p.dual) {  // an issuer per stream: one alone would be busy for longer than the tensor core
          const int mask = 1 << me, s0 = me * p.slots;
          int t = next(last + 1, mask);
          if (ok && t >= first) {
            ok = wait(kBFull + s0, 0);
            if (ok) {
              tc_fence_after();
              scores(me, s0);
              umma_commit_by(leader, bar(kBFree + s0));
              r.step(p.slots);
            }
          }
          for (int n = 0; t >= first && ok; ++n) {
            // while the softmax works: the tile's values, and the next tile's keys
            const int sv = s0 + r.s, tn = next(t, mask);
            ok = wait(kBFull + sv, r.ph);
            r.step(p.slots);
            const int sk = s0 + r.s;
            if (ok && tn >= first) ok = wait(kBFull + sk, r.ph);
            if (ok) ok = values(me, sv, n > 0, n & 1);
            if (!ok) break;
            if (tn >= first) {
              scores(me, sk);
              umma_commit_by(leader, bar(kBFree + sv));
              umma_commit_by(leader, bar(kBFree + sk));
              r.step(p.slots);
            }
            t = tn;
          }
          umma_commit_by(leader, bar(kBOD + me));
        } else {
          // both streams see the same tiles: one issuer alternates them, O_0 += P_0 V | S_0 next | O_1 += P_1 V | S_1 next,
          // so that one stream's products run under the other's softmax
          ok = ok && wait(kBFull, 0);
          int t = last;
          if (ok) {
            tc_fence_after();
            const int f = flags[t - ks];
            if (f & 1) scores(0, 0);
            if (f & 2) scores(1, 0);
            umma_commit_by(leader, bar(kBFree));
            r.step(p.slots);
          }
          int cnt[2] = {0, 0};
          while (t >= first && ok) {
            const int ta = next(t, 3), f = flags[t - ks], fa = ta >= first ? flags[ta - ks] : 0;
            const int sv = r.s;
            ok = wait(kBFull + sv, r.ph);
            r.step(p.slots);
            if (ok && fa) ok = wait(kBFull + r.s, r.ph);  // the next keys too, while the softmax works
#pragma unroll
            for (int q = 0; q < 2; ++q) {
              if (ok && (f >> q & 1)) {
                ok = values(q, sv, cnt[q] > 0, cnt[q] & 1);
                ++cnt[q];
              }
              if (ok && (fa >> q & 1)) scores(q, r.s);
            }
            if (!ok) break;
            umma_commit_by(leader, bar(kBFree + sv));
            if (ta >= first) {
              umma_commit_by(leader, bar(kBFree + r.s));
              r.step(p.slots);
            }
            t = ta;
          }
          umma_commit_by(leader, bar(kBOD + 0));
          umma_commit_by(leader, bar(kBOD + 1));
        }
        umma_commit_by(leader, bar(kBDrain + me));  // every product issued above completes before the block lets go
        mbar_wait_teardown(bar(kBDrain + me), 0);
      }
    }
  } else {
    set_regs_inc<kRegsSoftmax>();
    // ---------------------------------------------------------------- softmax (warps 4..7: stream 0, 8..11: stream 1)
    const int q = (warp - 4) >> 2;
    if (q < nstream) {
      const int quarter = warp & 3;  // TMEM lane quarter this warp may access
      const int row = quarter * 32 + lane;
      const uint32_t lane_base = (uint32_t)(quarter * 32) << 16;
      const uint32_t tS = tmem + 128 * q + lane_base, tO = tmem + 256 + 128 * q + lane_base;
      const int col0 = REP == 1 ? 0 : quarter * 32;  // this thread's columns of a tile: col0 .. col0 + 32 CH - 1
      const int tl = row % ROWS / p.pack, g = row % ROWS - tl * p.pack, tk = tok0(q) + tl;
      const bool valid = tl < p.tok && tk < a.Sq;
      const bool active = __any_sync(0xffffffffu, valid);  // a warp without a row only keeps the hand-offs going
      const int x = off + tk, h = hp * p.pack + g;
      const int jlast = valid ? last_key(a, x, len, prefix) : -1;
      const int mydoc = valid ? doc_at(a, b, x, len) : -1;
      const float mul0 = CAP ? a.cap * kLog2e : a.scale * kLog2e;
      // (a.cap_in as a constant operand of the loop is slower here: chunk 110 us against 103; the backward gains by it)
      const float cap_in = CAP ? fminf(a.scale / a.cap, kMaxCapIn) : 0.f;
      const float slope2 = BIAS == 1 ? -__ldg(a.slopes + h) * kLog2e : 0.f;
      const int64_t trow = (int64_t)h * a.buckets;
      float* win = reinterpret_cast<float*>(smem + p.off_win) + q * p.win;
      float m_run = -INFINITY, l_run = 0.f;
      constexpr bool kMayBeFar = CAP != 1 || BIAS != 0;  // (no score is beyond kCarefulCap else)
      bool far = false;                                  // some row's maximum is beyond kFarMax
      bool ok = true;
      int cnt = 0;
      const int ring = p.dual ? q * p.slots : 0, mask = p.dual ? 1 << q : 3;
      Ring r;  // of the tile's values
      r.step(p.slots);
      for (int t = next(last + 1, mask); t >= first; t = next(t, mask), r.step(p.slots), r.step(p.slots)) {
        const int f = flags[t - ks];
        if (!(f >> q & 1)) continue;
        const bool masked = f & (kMasked << q), near = BIAS && (f & (kNear << q));
        const int j0 = t * kTile;
        bool dead = false;
        float cadd = 0.f;
        // what the tile needs besides its scores, fetched before they are waited for
        int kid[4];  // ids of keys j0 + 32 c + lane
        if (masked && a.docs) {
#pragma unroll
          for (int c = 0; c < 4; ++c) kid[c] = doc_at(a, b, j0 + 32 * c + lane, len);
          dead = (quarter == 0 ? kid[0] : quarter == 1 ? kid[1] : quarter == 2 ? kid[2] : kid[3]) < 0;
        }
        if (BIAS == 2 && near) {
          ok = named_barrier_and(1 + q, kTile, ok);  // the last tile's window is done with
          // distances of the tile's rows and keys, one run of tok + 127 per head
          const int w = p.tok + kTile - 1, d0 = off + tok0(q) - j0 - (kTile - 1);
          for (int i = row; i < p.pack * w; i += kTile) {
            const int gi = i / w;
            win[i] = kLog2e * table_at<F16>(a.table, (int64_t)(hp * p.pack + gi) * a.buckets +
                                                         bucket_of(s_bs, d0 + i - gi * w));
          }
          ok = named_barrier_and(1 + q, kTile, ok);
        }
        if (masked && j0 + row >= len) dead = true;
        if (BIAS == 2 && !near && active) cadd = kLog2e * table_at<F16>(a.table, trow + bucket_of(s_bs, x - j0));
        if (ok) ok = __all_sync(0xffffffffu, mbar_wait(bar(kBSF + q), cnt & 1, &s_wait, status));
        if (!ok) continue;  // (the group's later barriers still count this warp)
        tc_fence_after();
        // Value rows that may meet a probability of zero: clear what is not finite (thread = row).  Both tiles of a block do so
        // where one has masked pairs, each ahead of its own product: V is theirs together, and whether the other's clearing
        // comes first must not show.
        if (f & (3 * kMasked)) {
          ok = __all_sync(0xffffffffu, mbar_wait(bar(kBFull + ring + r.s), r.ph, &s_wait, status));
          if (!ok) continue;  // (the group's later barriers still count this warp)
          uint8_t* vr = smem + p.off_kv + (ring + r.s) * TILE + row * 128;
          uint32_t bad = 0;
          if (!dead) {
            uint4 most = make_uint4(0, 0, 0, 0);
#pragma unroll
            for (int i = 0; i < D / 8; ++i) {
              const uint4 w = *reinterpret_cast<const uint4*>(vr + (i >> 3) * 16384 + (((i + lane) & 7) << 4));
              most.x = absmax2<F16>(most.x, w.x);
              most.y = absmax2<F16>(most.y, w.y);
              most.z = absmax2<F16>(most.z, w.z);
              most.w = absmax2<F16>(most.w, w.w);
            }
            bad = nonfinite2<F16>(absmax2<F16>(absmax2<F16>(most.x, most.y), absmax2<F16>(most.z, most.w)));
          }
          if (dead) {
#pragma unroll
            for (int i = 0; i < D / 8; ++i)
              *reinterpret_cast<uint4*>(vr + (i >> 3) * 16384 + (((i + lane) & 7) << 4)) = make_uint4(0, 0, 0, 0);
          } else if (bad) {  // (the flag first: the other stream's product may find the cleared row)
            atomicOr(reinterpret_cast<unsigned int*>(flags) + ((t - ks) >> 2), (unsigned)kBad << (8 * ((t - ks) & 3)));
            *static_cast<volatile int*>(&s_bad) = 1;
            __threadfence_block();
#pragma unroll 1
            for (int i = 0; i < D; ++i) {
              unsigned short* e = reinterpret_cast<unsigned short*>(vr + (i >> 6) * 16384) + (i & 63);
              if (nonfinite2<F16>(*e)) *e = 0;
            }
          }
          fence_proxy_async_smem();
        }
        if (active) {
          float s[CH][32];
#pragma unroll
          for (int c = 0; c < CH; ++c) tmem_ld32(tS + col0 + c * 32, s[c]);
          tmem_ld_wait();
          float mul = mul0;
          if (CAP) {
            constexpr bool kPoly = REP == 1 || CAP == 2;  // (few rows are bound by memory: the short code serves them)
            float big = 0.f;
            if constexpr (kPoly) {
#pragma unroll
              for (int c = 0; c < CH; ++c) big = absmax32(s[c], big);
            }
            big *= cap_in;
            if (kPoly && __all_sync(0xffffffffu, !valid || big <= 1.25f)) {
#pragma unroll
              for (int c = 0; c < CH; ++c) tanh32<false>(s[c], cap_in, mul0);
              mul = 1.f;
            } else {
#pragma unroll
              for (int c = 0; c < CH; ++c)
#pragma unroll
                for (int i = 0; i < 32; ++i) s[c][i] = tanh_any<CAP == 2>(s[c][i] * cap_in);
            }
          }
          if (BIAS == 1) {
            if (near) {
#pragma unroll
              for (int c = 0; c < CH; ++c)
#pragma unroll
                for (int i = 0; i < 32; ++i)
                  s[c][i] = fmaf(s[c][i], mul, slope2 * fabsf((float)(x - j0 - col0 - (c * 32 + i))));
            } else {
              const float base = slope2 * (float)(x - j0 - col0);
#pragma unroll
              for (int c = 0; c < CH; ++c)
#pragma unroll
                for (int i = 0; i < 32; ++i) s[c][i] = fmaf(s[c][i], mul, fmaf((float)(c * 32 + i), -slope2, base));
            }
            mul = 1.f;
          }
          if (BIAS == 2 && near) {
            const float* wr = win + g * (p.tok + kTile - 1) + min(tl, p.tok - 1) + kTile - 1 - col0;
#pragma unroll
            for (int c = 0; c < CH; ++c)
#pragma unroll
              for (int i = 0; i < 32; ++i) s[c][i] = fmaf(s[c][i], mul, wr[-(c * 32 + i)]);
            mul = 1.f;
          }
          if (masked) {
            uint32_t vis[CH];  // visible columns as bits
            const int jl = jlast - j0 - col0;  // last one by position
#pragma unroll
            for (int c = 0; c < CH; ++c) {
              const int n = min(max(jl + 1 - 32 * c, 0), 32);
              vis[c] = n == 0 ? 0u : 0xffffffffu >> (32 - n);
            }
            if (a.docs) {  // one document of the warp's rows after the other: its keys by ballots
              uint32_t todo = __ballot_sync(0xffffffffu, mydoc >= 0), same[CH] = {};
#pragma unroll 1
              while (todo) {
                const int doc = __shfl_sync(0xffffffffu, mydoc, __ffs(todo) - 1);
                const bool mine = mydoc == doc;
#pragma unroll
                for (int c = 0; c < CH; ++c) {
                  const int id = REP == 1 ? kid[c] : quarter == 0 ? kid[0] : quarter == 1 ? kid[1] : quarter == 2 ? kid[2] : kid[3];
                  const uint32_t m = __ballot_sync(0xffffffffu, id == doc);
                  same[c] = mine ? m : same[c];
                }
                todo &= ~__ballot_sync(0xffffffffu, mine);
              }
#pragma unroll
              for (int c = 0; c < CH; ++c) vis[c] &= same[c];
            }
#pragma unroll
            for (int c = 0; c < CH; ++c)
#pragma unroll
              for (int i = 0; i < 32; ++i) s[c][i] = vis[c] >> i & 1 ? s[c][i] : -INFINITY;
          }
          // row max as 4 chains of three-input maxima per 32 columns
          float mx8[8];
#pragma unroll
          for (int k = 0; k < 8; ++k) mx8[k] = fmaxf(s[0][k], s[0][k + 8]);
#pragma unroll
          for (int c = 0; c < CH; ++c)
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              if (c > 0) mx8[k] = fmax3(mx8[k], s[c][k], s[c][k + 8]);
              mx8[k] = fmax3(mx8[k], s[c][k + 16], s[c][k + 24]);
            }
          const float mx = fmaf(fmax3(fmax3(mx8[0], mx8[1], mx8[2]), fmax3(mx8[3], mx8[4], mx8[5]),
                                      fmaxf(mx8[6], mx8[7])), mul, cadd);
          float alpha = 1.0f;
          const bool move = __any_sync(0xffffffffu, valid && mx > m_run);
          if (move) {
            const float m_new = fmaxf(m_run, mx);
            alpha = m_run == -INFINITY ? 0.f : ex2(m_run - m_new);
            l_run *= alpha;
            m_run = m_new;
            if (kMayBeFar) far = __any_sync(0xffffffffu, valid && m_run != -INFINITY && fabsf(m_run) > kFarMax);
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
          // P over the first 64 columns of S, and its row sum; a row that has seen no key yet keeps P = 0
          float sub = cadd + kShift - (m_run == -INFINITY ? 0.f : m_run);
          if (kMayBeFar && __builtin_expect(far, 0)) {  // the score rounded first, then the difference, exact near the maximum
            const float top = m_run == -INFINITY ? 0.f : m_run;
            const uint64_t mul2 = f2pack(mul, mul), cadd2 = f2pack(cadd, cadd), top2 = f2pack(-top, -top);
#pragma unroll
            for (int c = 0; c < CH; ++c)
#pragma unroll
              for (int i = 0; i < 32; i += 2) {
                const uint64_t z = add_f32x2(fma_f32x2(f2pack(s[c][i], s[c][i + 1]), mul2, cadd2), top2);
                s[c][i] = f2lo(z);
                s[c][i + 1] = f2hi(z);
              }
            mul = 1.f;
            sub = kShift;
          }
          uint64_t rs2[4] = {0ull, 0ull, 0ull, 0ull};
          const uint64_t mul2 = f2pack(mul, mul), sub2 = f2pack(sub, sub), one2 = f2pack(1.f, 1.f);
          auto pair = [&](int c, int i) {  // the probabilities of columns i, i + 1 of run c, packed
            const uint64_t arg = fma_f32x2(f2pack(s[c][i], s[c][i + 1]), mul2, sub2);
            const float p0 = ex2(f2lo(arg)), p1 = ex2(f2hi(arg));
            rs2[(i >> 1) & 3] = fma_f32x2(f2pack(p0, p1), one2, rs2[(i >> 1) & 3]);
            return pack2_rn<F16>(p0, p1);
          };
          if constexpr (REP == 1) {
#pragma unroll
            for (int hh = 0; hh < 2; ++hh) {
              float pk[32];
#pragma unroll
              for (int i = 0; i < 64; i += 2) pk[i / 2] = __uint_as_float(pair(2 * hh + i / 32, i % 32));
              tmem_st32(tS + 32 * hh, pk);
              if (hh == 0) {  // the product may start on the first 64 keys
                tmem_st_wait();
                tc_fence_before();
                mbar_arrive(bar(kBPF + q));
              }
            }
          } else {  // the other copies' columns are theirs: zeros here
            uint32_t pk[16];
            const uint32_t zero[16] = {};
#pragma unroll
            for (int i = 0; i < 32; i += 2) pk[i / 2] = pair(0, i);
#pragma unroll
            for (int e = 0; e < REP; ++e)
              if (e != quarter) tmem_st16(tS + 16 * e, zero);
            tmem_st16(tS + 16 * quarter, pk);
          }
          tmem_st_wait();
          tc_fence_before();
          if (REP != 1) mbar_arrive(bar(kBPF + q));
          mbar_arrive(bar(kBPF + 2 + q));
          float rs[8] = {f2lo(rs2[0]), f2hi(rs2[0]), f2lo(rs2[1]), f2hi(rs2[1]),
                         f2lo(rs2[2]), f2hi(rs2[2]), f2lo(rs2[3]), f2hi(rs2[3])};
          l_run += ((rs[0] + rs[1]) + (rs[2] + rs[3])) + ((rs[4] + rs[5]) + (rs[6] + rs[7]));
        }
        if (!active) {
          tc_fence_before();
          mbar_arrive(bar(kBPF + q));
          mbar_arrive(bar(kBPF + 2 + q));
        }
        ++cnt;
      }

      // ---- epilogue: the last product, the join of the streams (and copies), the rows
      if (ok && first <= last) ok = mbar_wait(bar(kBOD + q), 0, &s_wait, status);
      // joined streams pass their rows through the memory of the tiles: the other one must be done with them too
      if (ok && first <= last && p.dual) ok = mbar_wait(bar(kBOD + 1 - q), 0, &s_wait, status);
      ok = __all_sync(0xffffffffu, ok);
      tc_fence_after();
      const bool part = p.nsplit > 1;
      auto out = [&](const DenseTensor& t, int hh, int tt) {  // a row's place in o or low
        return t.p ? static_cast<uint16_t*>(const_cast<void*>(t.p)) + b * t.st.b + hh * t.st.h + (int64_t)tt * t.st.s
                   : nullptr;
      };
      const int64_t pbase = (int64_t)split * a.B * a.Hq * a.Sq;  // rows of the splits before this one
      // values that are not finite, of the keys that the row sees (rare): v's features [f0, f0 + n) with them added
      auto add_bad = [&](int jl, int doc, int f0, int n, float* v) {
        if (!*static_cast<volatile int*>(&s_bad)) return;
#pragma unroll 1
        for (int t = first; t <= last; ++t) {
          if (!(flags[t - ks] & kBad)) continue;
#pragma unroll 1
          for (int j = t * kTile; j < min((t + 1) * kTile, jl + 1); ++j) {
            if (a.docs && (doc < 0 || doc_at(a, b, j, len) != doc)) continue;
            const uint16_t* vr = static_cast<const uint16_t*>(p.v.p) + b * p.v.st.b + kvh * p.v.st.h + j * p.v.st.s + f0;
#pragma unroll
            for (int i = 0; i < n; ++i) v[i] += nonfinite2<F16>(vr[i]) ? unpack2<F16>(vr[i]).x : 0.f;
          }
        }
      };
      auto stats = [&](int64_t ri, float m, float l) {
        const float l2 = l == 0.f ? -INFINITY : m - kShift + __log2f(l);
        if (part) p.part_lse[pbase + ri] = l2;
        else p.lse[ri] = l2 * kLn2;
      };
      if constexpr (REP == 1) {
        float a0 = 1.f, a1 = 0.f;
        float* so = reinterpret_cast<float*>(smem + p.off_kv);  // [D][128] of stream 1 (keys and values are consumed)
        float* sm = so + D * kTile;                             // [2][128] its maxima and sums
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
            if (m != -INFINITY) {
              a0 = m_run == -INFINITY ? 0.f : ex2(m_run - m);
              a1 = m1 == -INFINITY ? 0.f : ex2(m1 - m);
            }
            l_run = l_run * a0 + sm[kTile + row] * a1;
            m_run = m;
          }
        } else {
          ok = named_barrier_and(1 + q, kTile, ok);  // the group's flags of tiles with values that are not finite
        }
        if (ok && (q == 0 || !p.dual)) {
          const float inv = l_run == 0.f ? 0.f : 1.0f / l_run;
          const int64_t ri = ((int64_t)b * a.Hq + h) * a.Sq + tk;
          const bool use0 = cnt > 0 && inv != 0.f, use1 = p.dual && a1 != 0.f && inv != 0.f;
          // features [32 c, 32 c + 32) of this row
          auto result = [&](int c, float (&o)[32]) {
            if (cnt > 0) {
              tmem_ld32(tO + c * 32, o);
              tmem_ld_wait();
            }
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] = use0 ? o[i] * (a0 * inv) : 0.f;
            if (use1) {
#pragma unroll
              for (int i = 0; i < 32; ++i) o[i] = fmaf(so[(c * 32 + i) * kTile + row], a1 * inv, o[i]);
            }
            if (valid) add_bad(jlast, mydoc, c * 32, 32, o);
          };
          uint8_t* tile = smem + (p.dual ? 0 : q) * TILE;  // the queries' place, consumed
          if (part) {
            const uint32_t rows = __ballot_sync(0xffffffffu, valid);
            const RowStage stage{tile + quarter * 4096};
            float* prow = p.part_o + (pbase + ri) * D;
            if (active) {
#pragma unroll
              for (int c = 0; c < D / 32; ++c) {
                float o[32];
                result(c, o);
#pragma unroll
                for (int i = 0; i < 8; ++i)
                  *reinterpret_cast<float4*>(stage.at(lane, i)) = make_float4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
                stage.flush(rows, prow + 32 * c, lane);
              }
            }
          } else {
            // 64 features of all rows at a time, in the layout the queries came in, leave by one TMA store (rows at or
            // beyond Sq are outside its tensor); at d = 128 the low halves have the tile's second block, else its turn
            const RowStage stage{tile + quarter * 4096}, stage2{tile + (D == 128 ? 16384 : 0) + quarter * 4096};
            const bool chief = row == 0;
            auto send = [&](const CUtensorMap* map, const RowStage& from, int half) {
              tma_store_5d(map, smem_u32(from.buf), half * 64, 0, tok0(q), hp, b);
              bulk_commit_group();
            };
#pragma unroll
            for (int half = 0; half < D / 64; ++half) {
              uint4 lo[8];
              if (active) {
#pragma unroll
                for (int cc = 0; cc < 2; ++cc) {
                  float o[32];
                  result(2 * half + cc, o);
#pragma unroll
                  for (int i = 0; i < 4; ++i) {
                    *stage.at(lane, 4 * cc + i) = round8<F16>(o + 8 * i, lo + 4 * cc + i);
                    if (D == 128 && p.low.p) *stage2.at(lane, 4 * cc + i) = lo[4 * cc + i];
                  }
                }
              }
              fence_proxy_async_smem();
              named_barrier_and(1 + q, kTile, true);
              if (chief) {
                send(&m.o, stage, half);
                if (D == 128 && p.low.p) send(&m.low, stage2, half);
              }
              if (half + 1 < D / 64 || (D == 64 && p.low.p)) {  // the block is written again
                if (chief) bulk_wait_group_read0();
                named_barrier_and(1 + q, kTile, true);
              }
              if (D == 64 && p.low.p) {
#pragma unroll
                for (int i = 0; i < 8; ++i) *stage2.at(lane, i) = lo[i];
                fence_proxy_async_smem();
                named_barrier_and(1 + q, kTile, true);
                if (chief) send(&m.low, stage2, half);
              }
            }
            if (chief) bulk_wait_group0();
          }
          if (valid) stats(ri, m_run, l_run);
        }
      } else {
        // 2 REP partial results of each row: all in shared memory, then a thread for 16 (8 at d = 64) features of a row
        float* so = reinterpret_cast<float*>(smem + p.off_kv);  // [2 REP][D][ROWS] (keys and values are consumed)
        float* sm = reinterpret_cast<float*>(smem);            // [2 REP][2][ROWS] (the queries too)
        const int me = q * REP + quarter;
        if (ok) {
          sm[(2 * me) * ROWS + lane] = m_run;
          sm[(2 * me + 1) * ROWS + lane] = l_run;
          if (cnt > 0) {
#pragma unroll
            for (int c = 0; c < D / 32; ++c) {
              float o[32];
              tmem_ld32(tO + c * 32, o);
              tmem_ld_wait();
#pragma unroll
              for (int i = 0; i < 32; ++i) so[(me * D + c * 32 + i) * ROWS + lane] = o[i];
            }
          }
        }
        ok = named_barrier_and(3, 2 * kTile, ok);
        if (ok && valid) {
          constexpr int N = D / 8;
          float m = -INFINITY, l = 0.f, wgt[2 * REP], o[N];
#pragma unroll
          for (int e = 0; e < 2 * REP; ++e) m = fmaxf(m, sm[2 * e * ROWS + lane]);
#pragma unroll
          for (int e = 0; e < 2 * REP; ++e) {
            const float me_m = sm[2 * e * ROWS + lane];
            wgt[e] = me_m == -INFINITY ? 0.f : ex2(me_m - m);
            l = fmaf(sm[(2 * e + 1) * ROWS + lane], wgt[e], l);
          }
          const float inv = l == 0.f ? 0.f : 1.0f / l;
#pragma unroll
          for (int i = 0; i < N; ++i) o[i] = 0.f;
#pragma unroll
          for (int e = 0; e < 2 * REP; ++e)
            if (wgt[e] != 0.f && inv != 0.f) {
#pragma unroll
              for (int i = 0; i < N; ++i) o[i] = fmaf(so[(e * D + me * N + i) * ROWS + lane], wgt[e] * inv, o[i]);
            }
          const int64_t ri = ((int64_t)b * a.Hq + h) * a.Sq + tk;
          add_bad(jlast, mydoc, me * N, N, o);
          if (part) {
            float* dst = p.part_o + (pbase + ri) * D + me * N;
#pragma unroll
            for (int i = 0; i < N; i += 4) *reinterpret_cast<float4*>(dst + i) = make_float4(o[i], o[i + 1], o[i + 2], o[i + 3]);
          } else {
            uint16_t *od = out(p.o, h, tk) + me * N, *ld = out(p.low, h, tk);
#pragma unroll
            for (int i = 0; i < N; i += 8) {
              uint4 lo;
              st16(od + i, round8<F16>(o + i, &lo));
              if (ld) st16(ld + me * N + i, lo);
            }
          }
          if (me == 0) stats(ri, m, l);
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

template <int D, bool F16, int CAP, int BIAS, int REP>
int launch_r(const FwdMaps& m, const FwdArgs& p, const BucketStarts& bs, int smem, cudaStream_t st) {
  auto kernel = dense_fwd_kernel<D, F16, CAP, BIAS, REP>;
  static std::atomic<uint64_t> ready{0};  // devices on which the kernel's shared-memory limit is set
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return LH_ERR_CUDA;
  if (!(ready.load(std::memory_order_acquire) >> (dev & 63) & 1)) {
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemLimit) != cudaSuccess)
      return LH_ERR_CUDA;
    ready.fetch_or(uint64_t(1) << (dev & 63), std::memory_order_release);
  }
  const int nbh = p.a.B * (p.a.Hq / p.pack);
  const dim3 grid = p.head_fast ? dim3(nbh, p.npair, p.nsplit) : dim3(p.npair, nbh, p.nsplit);
  kernel<<<grid, kThreads, smem, st>>>(m, p, bs);
  return check_launch();
}
template <int D, bool F16, int CAP, int BIAS>
int launch_t(const FwdMaps& m, const FwdArgs& p, const BucketStarts& bs, int smem, cudaStream_t st) {
  return p.rep == 4 ? launch_r<D, F16, CAP, BIAS, 4>(m, p, bs, smem, st)
                    : launch_r<D, F16, CAP, BIAS, 1>(m, p, bs, smem, st);
}
// Instantiated for each width and type in a file of its own.
template <int D, bool F16>
int launch(const FwdMaps& m, const FwdArgs& p, const BucketStarts& bs, int smem, cudaStream_t st) {
  const int bias = p.a.slopes ? 1 : p.a.table ? 2 : 0;
  auto with = [&](auto tag) {
    constexpr int C = decltype(tag)::value;
    return bias == 0 ? launch_t<D, F16, C, 0>(m, p, bs, smem, st)
                     : bias == 1 ? launch_t<D, F16, C, 1>(m, p, bs, smem, st) : launch_t<D, F16, C, 2>(m, p, bs, smem, st);
  };
  if (p.a.cap > kCarefulCap) return with(std::integral_constant<int, 2>{});
  return p.a.cap > 0.f ? with(std::integral_constant<int, 1>{}) : with(std::integral_constant<int, 0>{});
}

}  // namespace fwd
}  // namespace lh
