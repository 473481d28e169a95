// dense_prep.cu — the small kernels around the dense stage's attention: the documents' ranges of the tiles, the
// backward's row statistics and bias by distance, and the results' last sums and roundings.  All are bound by memory or
// by their launch.
#include "dense.cuh"

namespace lh {

namespace {

// The ids' range of tile w (its live positions' least and largest id, the least one complemented where a position is dead:
// id_range): key tiles first, then 64-row query sub-tiles.  One warp each.
__device__ __forceinline__ void doc_range(const DenseDims& a, int b, int w, int lane, int nk, int2* kdoc, int2* qdoc,
                                          int nq) {
  const int len = dense_len(a, b);
  const bool key = w < nk;
  const int x0 = key ? w * kKeyTile : len - a.Sq + (w - nk) * 64;
  const int n = key ? min(kKeyTile, a.Skv - x0) : min(64, a.Sq - (w - nk) * 64);
  const int2 r = warp_doc_range(a, b, x0, n, len, lane);
  if (lane == 0) (key ? kdoc[(int64_t)b * nk + w] : qdoc[(int64_t)b * nq + w - nk]) = r;
}

__global__ void __launch_bounds__(256) doc_ranges_kernel(const DenseDims a, int2* __restrict__ kdoc, int nk) {
  const int w = blockIdx.x * 8 + threadIdx.x / 32;
  if (w < nk) doc_range(a, blockIdx.y, w, threadIdx.x % 32, nk, kdoc, nullptr, 0);
}

// One group of d / 8 lanes per query row, 16-byte loads: D = <dO, O>, the statistics, the zeroed dQ accumulator, and for
// fp16 the largest |dO_i| of the key head's rows (one atomicMax of a bit pattern per block: order-free).
template <int D, bool F16>
__device__ __forceinline__ void bwd_row(const DenseDims& a, const DenseTensor& o, const DenseTensor& low,
                                        const DenseTensor& dout, const float* __restrict__ lse, const DenseBwdBuf& w,
                                        int blk, int bh) {
  constexpr int L = D / 8, ROWS = 256 / L;
  const int b = bh / a.Hq, h = bh % a.Hq;
  const int i = blk * ROWS + threadIdx.x / L, f = (threadIdx.x % L) * 8;
  const bool in = i < a.Sq;
  auto at = [&](const DenseTensor& t) {
    return ld16(static_cast<const uint16_t*>(t.p) + b * t.st.b + h * t.st.h + (int64_t)i * t.st.s + f);
  };
  float dot = 0.f, norm = 0.f;
  if (in) {
    const uint4 x = at(o), y = at(dout), z = low.p ? at(low) : make_uint4(0, 0, 0, 0);
    const uint32_t xw[4] = {x.x, x.y, x.z, x.w}, yw[4] = {y.x, y.y, y.z, y.w}, zw[4] = {z.x, z.y, z.z, z.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float2 u = unpack2<F16>(xw[e]), v = unpack2<F16>(yw[e]), r = unpack2<F16>(zw[e]);
      dot = fmaf(u.x + r.x, v.x, fmaf(u.y + r.y, v.y, dot));
      norm = fmaf(v.x, v.x, fmaf(v.y, v.y, norm));
    }
    float4* acc = reinterpret_cast<float4*>(w.dqacc + ((int64_t)bh * a.Sq + i) * D + f);
    acc[0] = acc[1] = make_float4(0.f, 0.f, 0.f, 0.f);
  }
#pragma unroll
  for (int s = L / 2; s; s >>= 1) {
    dot += __shfl_xor_sync(0xffffffffu, dot, s);
    norm += __shfl_xor_sync(0xffffffffu, norm, s);
  }
  bool dead = true;
  if (in) {
    const int len = dense_len(a, b);
    const float l = lse[(int64_t)bh * a.Sq + i];
    dead = l == -INFINITY || doc_at(a, b, len - a.Sq + i, len) < 0;
    if (f == 0) {
      const int64_t pitch = (a.Sq + 3) & ~3, at = bh * pitch + i;
      // -LSE log2(e); with slopes also the share of the row's place in its 64-row sub-tile, - slope (i mod 64) log2(e)
      const float nl = fmaf(l, -1.4426950408889634f, F16 ? 12.f : 0.f);
      const float sl = a.slopes ? -1.4426950408889634f * __ldg(a.slopes + h) * (float)(i & 63) : 0.f;
      w.stats[at] = dead ? -INFINITY : nl + sl;
      w.stats[(int64_t)a.B * a.Hq * pitch + at] = dead ? 0.f : -dot;
    }
  }
  if (F16) {
    __shared__ unsigned int s_max;
    if (threadIdx.x == 0) s_max = 0;
    __syncthreads();
    if (!dead && f == 0) atomicMax(&s_max, __float_as_uint(sqrtf(norm)));
    __syncthreads();
    if (threadIdx.x == 0) atomicMax(w.amax + 2 * (b * a.Hkv + h / a.G), s_max);
  }
}

// fp16: the largest |V_j| of a key head.
template <int D>
__device__ __forceinline__ void v_norm(const DenseDims& a, const DenseTensor& v, unsigned int* __restrict__ amax, int blk,
                                       int bh) {
  constexpr int L = D / 8, ROWS = 256 / L;
  const int b = bh / a.Hkv, h = bh % a.Hkv, len = dense_len(a, b);
  const int f = (threadIdx.x % L) * 8;
  __shared__ unsigned int s_max;
  if (threadIdx.x == 0) s_max = 0;
  __syncthreads();
  for (int k = 0; k < 8; ++k) {
    const int j = (blk * 8 + k) * ROWS + threadIdx.x / L;
    float norm = 0.f;
    const bool live = j < len && doc_at(a, b, j, len) >= 0;
    if (live) {
      const uint4 y = ld16(static_cast<const uint16_t*>(v.p) + b * v.st.b + h * v.st.h + (int64_t)j * v.st.s + f);
      const uint32_t yw[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 u = unpack2<true>(yw[e]);
        norm = fmaf(u.x, u.x, fmaf(u.y, u.y, norm));
      }
    }
#pragma unroll
    for (int s = L / 2; s; s >>= 1) norm += __shfl_xor_sync(0xffffffffu, norm, s);
    if (live && f == 0) atomicMax(&s_max, __float_as_uint(sqrtf(norm)));
  }
  __syncthreads();
  if (threadIdx.x == 0) atomicMax(amax + 2 * bh + 1, s_max);
}

// The bias by distance of head h; head 0 also writes the buckets by distance and their ranges.
template <bool F16>
__device__ __forceinline__ void bias_by_distance(const DenseDims& a, const BucketStarts& bs, const DenseBwdBuf& w, int blk,
                                                 int h) {
  const int wide = 2 * a.near + 1, i = blk * 256 + threadIdx.x;
  if (i < wide) {
    const int k = bucket_of(bs, i - a.near);
    w.bias[(int64_t)h * wide + i] = 1.4426950408889634f * table_at<F16>(a.table, (int64_t)h * a.buckets + k);
    if (h == 0) w.bucket[i] = (uint8_t)k;
  }
  const int k = threadIdx.x;
  if (h == 0 && blk == 0 && k < a.buckets) {
    const int m = k % bs.n;
    const int lo = bs.start[m], hi = m + 1 < bs.n ? bs.start[m + 1] - 1 : 1 << 29;  // sizes lo .. hi
    int2 r;
    if (!bs.both) r = make_int2(m == 0 ? -(1 << 29) : lo, hi);
    else r = k < bs.n ? make_int2(lo, hi) : make_int2(-hi, min(-lo, -1));
    w.range[k] = r;
  }
}

// Everything the backward needs before its main kernel, in one launch: blocks [0, e0) row statistics, [e0, e1) value
// norms, [e1, e2) ids' ranges, [e2, end) bias.
struct PrepArgs {
  DenseDims a;
  BucketStarts bs;
  DenseTensor o, low, dout, v;
  const float* lse;
  DenseBwdBuf w;
  int2 *kdoc, *qdoc;
  int row_blocks, v_blocks, doc_blocks, bias_blocks;  // per head, head, batch entry, head
  int64_t e0, e1, e2;
};
template <int D, bool F16>
__global__ void __launch_bounds__(256) bwd_prep_kernel(const __grid_constant__ PrepArgs p) {
  const int64_t x = blockIdx.x;
  if (x < p.e0) {
    bwd_row<D, F16>(p.a, p.o, p.low, p.dout, p.lse, p.w, (int)(x % p.row_blocks), (int)(x / p.row_blocks));
  } else if (x < p.e1) {
    if (F16) v_norm<D>(p.a, p.v, p.w.amax, (int)((x - p.e0) % p.v_blocks), (int)((x - p.e0) / p.v_blocks));
  } else if (x < p.e2) {
    const int nk = (p.a.Skv + kKeyTile - 1) / kKeyTile, nq = (p.a.Sq + 63) / 64;
    const int w = (int)((x - p.e1) % p.doc_blocks) * 8 + threadIdx.x / 32;
    if (w < nk + nq)
      doc_range(p.a, (int)((x - p.e1) / p.doc_blocks), w, threadIdx.x % 32, nk, p.kdoc, p.qdoc, nq);
  } else {
    bias_by_distance<F16>(p.a, p.bs, p.w, (int)((x - p.e2) % p.bias_blocks), (int)((x - p.e2) / p.bias_blocks));
  }
}

// dQ: the accumulator rounded once; dV, dK: the shares' sums rounded once.  Eight features a thread.
template <int D, bool F16>
__device__ __forceinline__ void round_rows(const float* __restrict__ src, int64_t plane, int n, int heads, int rows,
                                           const DenseTensor& out, int64_t total, int64_t blk) {
  const int64_t e = (blk * 256 + threadIdx.x) * 8;
  if (e >= total) return;
  float v[8] = {};
  for (int s = 0; s < n; ++s) {
    const float4 x = *reinterpret_cast<const float4*>(src + s * plane + e);
    const float4 y = *reinterpret_cast<const float4*>(src + s * plane + e + 4);
    v[0] += x.x; v[1] += x.y; v[2] += x.z; v[3] += x.w;
    v[4] += y.x; v[5] += y.y; v[6] += y.z; v[7] += y.w;
  }
  const int64_t row = e / D, i = row % rows, bh = row / rows;
  uint16_t* dst = static_cast<uint16_t*>(const_cast<void*>(out.p)) + (bh / heads) * out.st.b + (bh % heads) * out.st.h +
                  i * out.st.s + e % D;
  st16(dst, make_uint4(pack2_rn<F16>(v[0], v[1]), pack2_rn<F16>(v[2], v[3]), pack2_rn<F16>(v[4], v[5]),
                       pack2_rn<F16>(v[6], v[7])));
}

// dtable[h][k]: the warps' sums of every batch entry and key tile, in a fixed order; 64-bit, as a far bucket's sum is the
// small rest of large ones.
template <bool F16>
__device__ __forceinline__ void dtable_rows(const DenseDims& a, const float* __restrict__ part, int nkt, void* dtable,
                                            int h, int k0) {
  const int kvh = h / a.G, g = h % a.G, k = k0 + threadIdx.x % 32, w = threadIdx.x / 32;
  __shared__ double s_sum[8][32];
  double sum = 0.0;
  if (k < a.buckets) {
    const int64_t step = (int64_t)a.G * 8 * a.buckets, jump = (int64_t)(a.Hkv - 1) * nkt * step;
    const float* src = part + (((int64_t)kvh * nkt * a.G + g) * 8 + w) * a.buckets + k;
    const int total = a.B * nkt;
    int kt = 0;
#pragma unroll 8
    for (int t = 0; t < total; ++t) {
      sum += *src;
      src += step;
      if (++kt == nkt) kt = 0, src += jump;  // the next batch entry
    }
  }
  s_sum[w][threadIdx.x % 32] = sum;
  __syncthreads();
  if (w == 0 && k < a.buckets) {
    for (int i = 1; i < 8; ++i) sum += s_sum[i][threadIdx.x];
    // the differences of prefix sums leave up to 2^-20 of the neighbours' |dZ|: nothing of that for a masked bucket
    if (1.4426950408889634f * table_at<F16>(a.table, (int64_t)h * a.buckets + k) == -INFINITY) sum = 0.0;
    static_cast<uint16_t*>(dtable)[(int64_t)h * a.buckets + k] = (uint16_t)pack2_rn<F16>((float)sum, 0.f);
  }
}

// The results, in one launch: blocks [0, e0) dtable (the longest first), [e0, e1) dQ, then, with shared query heads,
// dV and dK.
struct OutArgs {
  DenseDims a;
  DenseTensor dq, dk, dv;
  void* dtable;
  DenseBwdBuf w;
  int nkt, shares;
  int64_t e0, e1, kv_blocks;
};
template <int D, bool F16>
__global__ void __launch_bounds__(256) bwd_out_kernel(const __grid_constant__ OutArgs p) {
  const DenseDims& a = p.a;
  const int64_t x = blockIdx.x, one = (int64_t)a.B * a.Hkv * a.Skv * D;
  if (x < p.e0) {
    const int n = (a.buckets + 31) / 32;
    dtable_rows<F16>(a, p.w.dtpart, p.nkt, p.dtable, (int)(x / n), (int)(x % n) * 32);
  } else if (x < p.e1) {
    round_rows<D, F16>(p.w.dqacc, 0, 1, a.Hq, a.Sq, p.dq, (int64_t)a.B * a.Hq * a.Sq * D, x - p.e0);
  } else if (x < p.e1 + p.kv_blocks) {
    round_rows<D, F16>(p.w.dkv, 2 * one, p.shares, a.Hkv, a.Skv, p.dv, one, x - p.e1);
  } else {
    round_rows<D, F16>(p.w.dkv + one, 2 * one, p.shares, a.Hkv, a.Skv, p.dk, one, x - p.e1 - p.kv_blocks);
  }
}

}  // namespace

int launch_dense_bwd_prep(const DenseDims& a, const BucketStarts& bs, const DenseTensor& o, const DenseTensor& low,
                          const DenseTensor& dout, const DenseTensor& v, const float* lse, const DenseBwdBuf& w,
                          int2* kdoc, int2* qdoc, cudaStream_t st) {
  PrepArgs p;
  p.a = a; p.bs = bs; p.o = o; p.low = low; p.dout = dout; p.v = v; p.lse = lse; p.w = w; p.kdoc = kdoc; p.qdoc = qdoc;
  const int rows = 256 / (a.d / 8), nk = (a.Skv + kKeyTile - 1) / kKeyTile, nq = (a.Sq + 63) / 64;
  p.row_blocks = (a.Sq + rows - 1) / rows;
  p.v_blocks = a.f16 ? (a.Skv + 8 * rows - 1) / (8 * rows) : 0;
  p.doc_blocks = a.docs ? (nk + nq + 7) / 8 : 0;
  p.bias_blocks = a.table ? (2 * a.near + 1 + 255) / 256 : 0;
  p.e0 = (int64_t)p.row_blocks * a.B * a.Hq;
  p.e1 = p.e0 + (int64_t)p.v_blocks * a.B * a.Hkv;
  p.e2 = p.e1 + (int64_t)p.doc_blocks * a.B;
  const int64_t blocks = p.e2 + (int64_t)p.bias_blocks * a.Hq;
  if (blocks > INT32_MAX) return LH_ERR_UNSUPPORTED;
  KernelTimer timer("dense_bwd_prep", st);
  if (a.f16 && cudaMemsetAsync(w.amax, 0, (size_t)a.B * a.Hkv * 8, st) != cudaSuccess) return LH_ERR_CUDA;
  auto kernel = a.d == 64 ? (a.f16 ? bwd_prep_kernel<64, true> : bwd_prep_kernel<64, false>)
                          : (a.f16 ? bwd_prep_kernel<128, true> : bwd_prep_kernel<128, false>);
  kernel<<<(unsigned)blocks, 256, 0, st>>>(p);
  return check_launch();
}

int launch_dense_bwd_out(const DenseDims& a, const DenseTensor& dq, const DenseTensor& dk, const DenseTensor& dv,
                         void* dtable, const DenseBwdBuf& w, cudaStream_t st) {
  OutArgs p;
  p.a = a; p.dq = dq; p.dk = dk; p.dv = dv; p.dtable = dtable; p.w = w;
  p.nkt = (a.Skv + kKeyTile - 1) / kKeyTile;
  p.shares = dense_bwd_shares(a);
  auto blocks_of = [&](int64_t rows) { return (rows * (a.d / 8) + 255) / 256; };
  p.e0 = a.table ? (int64_t)a.Hq * ((a.buckets + 31) / 32) : 0;
  p.e1 = p.e0 + blocks_of((int64_t)a.B * a.Hq * a.Sq);
  p.kv_blocks = p.shares > 1 ? blocks_of((int64_t)a.B * a.Hkv * a.Skv) : 0;
  const int64_t blocks = p.e1 + 2 * p.kv_blocks;
  if (blocks > INT32_MAX) return LH_ERR_UNSUPPORTED;
  KernelTimer timer("dense_bwd_out", st);
  auto kernel = a.d == 64 ? (a.f16 ? bwd_out_kernel<64, true> : bwd_out_kernel<64, false>)
                          : (a.f16 ? bwd_out_kernel<128, true> : bwd_out_kernel<128, false>);
  kernel<<<(unsigned)blocks, 256, 0, st>>>(p);
  return check_launch();
}

int launch_dense_doc_ranges(const DenseDims& a, int2* kdoc, cudaStream_t st) {
  const int nk = (a.Skv + kKeyTile - 1) / kKeyTile;
  KernelTimer timer("dense_doc_ranges", st);
  doc_ranges_kernel<<<dim3((nk + 7) / 8, a.B), 256, 0, st>>>(a, kdoc, nk);
  return check_launch();
}

}  // namespace lh
