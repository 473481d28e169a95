// dense_prep.cu — the small kernels around the dense stage's attention: the documents' ranges of the tiles, the
// backward's row statistics and bias by distance, and the results' last sums and roundings.  All are bound by memory or
// by their launch.
#include "dense.cuh"

namespace lh {

namespace {

// One warp per 64 positions: the smallest and largest id among them (a dead position counts as -1).  Key tiles take
// two such halves.  Reads each id once; launch-bound.
__global__ void doc_ranges_kernel(const DenseDims a, int2* __restrict__ kdoc, int2* __restrict__ qdoc, int nk, int nq) {
  const int w = blockIdx.x * (blockDim.x / 32) + threadIdx.x / 32, lane = threadIdx.x % 32, b = blockIdx.y;
  if (w >= nk + nq) return;
  const int len = dense_len(a, b);
  const bool key = w < nk;
  const int x0 = key ? w * kKeyTile : len - a.Sq + (w - nk) * 64;
  const int n = key ? min(kKeyTile, a.Skv - x0) : min(64, a.Sq - (w - nk) * 64);
  int lo = INT32_MAX, hi = -1;
  for (int i = lane; i < n; i += 32) {
    const int id = max(doc_at(a, b, x0 + i, len), -1);
    lo = min(lo, id);
    hi = max(hi, id);
  }
  lo = __reduce_min_sync(0xffffffffu, lo);
  hi = __reduce_max_sync(0xffffffffu, hi);
  if (lane == 0) (key ? kdoc[(int64_t)b * nk + w] : qdoc[(int64_t)b * nq + w - nk]) = make_int2(lo, hi);
}

// One group of d / 8 lanes per query row, 16-byte loads: D = <dO, O>, the statistics, the zeroed dQ accumulator, and for
// fp16 the largest |dO_i| of the key head's rows (one atomicMax of a bit pattern per block: order-free).
template <int D, bool F16>
__global__ void __launch_bounds__(256)
    bwd_rows_kernel(const DenseDims a, const uint16_t* __restrict__ o, Strides os, const uint16_t* __restrict__ low,
                    Strides ls, const uint16_t* __restrict__ dout, Strides ds, const float* __restrict__ lse, float* __restrict__ stats, float* __restrict__ dqacc,
                    unsigned int* __restrict__ amax) {
  constexpr int L = D / 8, ROWS = 256 / L;
  const int bh = blockIdx.y, b = bh / a.Hq, h = bh % a.Hq;
  const int i = blockIdx.x * ROWS + threadIdx.x / L, f = (threadIdx.x % L) * 8;
  const bool in = i < a.Sq;
  float dot = 0.f, norm = 0.f;
  if (in) {
    const uint4 x = ld16(o + b * os.b + h * os.h + (int64_t)i * os.s + f);
    const uint4 y = ld16(dout + b * ds.b + h * ds.h + (int64_t)i * ds.s + f);
    const uint4 z = low ? ld16(low + b * ls.b + h * ls.h + (int64_t)i * ls.s + f) : make_uint4(0, 0, 0, 0);
    const uint32_t xw[4] = {x.x, x.y, x.z, x.w}, yw[4] = {y.x, y.y, y.z, y.w}, zw[4] = {z.x, z.y, z.z, z.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float2 u = unpack2<F16>(xw[e]), w = unpack2<F16>(yw[e]), r = unpack2<F16>(zw[e]);
      dot = fmaf(u.x + r.x, w.x, fmaf(u.y + r.y, w.y, dot));
      norm = fmaf(w.x, w.x, fmaf(w.y, w.y, norm));
    }
    float4* acc = reinterpret_cast<float4*>(dqacc + ((int64_t)bh * a.Sq + i) * D + f);
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
      stats[at] = dead ? -INFINITY : fmaf(l, -1.4426950408889634f, F16 ? 12.f : 0.f);
      stats[(int64_t)a.B * a.Hq * pitch + at] = dead ? 0.f : -dot;
    }
  }
  if (F16) {
    __shared__ unsigned int s_max;
    if (threadIdx.x == 0) s_max = 0;
    __syncthreads();
    if (!dead && f == 0) atomicMax(&s_max, __float_as_uint(sqrtf(norm)));
    __syncthreads();
    if (threadIdx.x == 0) atomicMax(amax + 2 * (b * a.Hkv + h / a.G), s_max);
  }
}

// fp16: the largest |V_j| of a key head.
template <int D>
__global__ void __launch_bounds__(256) v_norm_kernel(const DenseDims a, const uint16_t* __restrict__ v, Strides vs,
                                                     unsigned int* __restrict__ amax) {
  constexpr int L = D / 8, ROWS = 256 / L;
  const int bh = blockIdx.y, b = bh / a.Hkv, h = bh % a.Hkv, len = dense_len(a, b);
  const int f = (threadIdx.x % L) * 8;
  __shared__ unsigned int s_max;
  if (threadIdx.x == 0) s_max = 0;
  __syncthreads();
  for (int k = 0; k < 8; ++k) {
    const int j = (blockIdx.x * 8 + k) * ROWS + threadIdx.x / L;
    float norm = 0.f;
    const bool live = j < len && doc_at(a, b, j, len) >= 0;
    if (live) {
      const uint4 y = ld16(v + b * vs.b + h * vs.h + (int64_t)j * vs.s + f);
      const uint32_t yw[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 w = unpack2<true>(yw[e]);
        norm = fmaf(w.x, w.x, fmaf(w.y, w.y, norm));
      }
    }
#pragma unroll
    for (int s = L / 2; s; s >>= 1) norm += __shfl_xor_sync(0xffffffffu, norm, s);
    if (live && f == 0) atomicMax(&s_max, __float_as_uint(sqrtf(norm)));
  }
  __syncthreads();
  if (threadIdx.x == 0) atomicMax(amax + 2 * bh + 1, s_max);
}

// The bias by distance, for every head; block row 0 also writes the buckets by distance and their ranges.
template <bool F16>
__global__ void bias_kernel(const DenseDims a, const __grid_constant__ BucketStarts bs, float* __restrict__ bias,
                            uint8_t* __restrict__ bucket, int2* __restrict__ range) {
  const int wide = 2 * a.near + 1, h = blockIdx.y;
  for (int i = blockIdx.x * blockDim.x + threadIdx.x; i < wide; i += gridDim.x * blockDim.x) {
    const int k = bucket_of(bs, i - a.near);
    bias[(int64_t)h * wide + i] = 1.4426950408889634f * table_at<F16>(a.table, (int64_t)h * a.buckets + k);
    if (h == 0) bucket[i] = (uint8_t)k;
  }
  const int k = threadIdx.x;
  if (h == 0 && blockIdx.x == 0 && k < a.buckets) {
    const int m = k % bs.n;
    const int lo = bs.start[m], hi = m + 1 < bs.n ? bs.start[m + 1] - 1 : 1 << 29;  // sizes lo .. hi
    int2 r;
    if (!bs.both) r = make_int2(m == 0 ? -(1 << 29) : lo, hi);
    else r = k < bs.n ? make_int2(lo, hi) : make_int2(-hi, min(-lo, -1));
    range[k] = r;
  }
}

// dQ: the accumulator rounded once; dV, dK: the shares' sums rounded once.  Eight features a thread.
template <int D, bool F16>
__global__ void __launch_bounds__(256) bwd_out_kernel(const float* __restrict__ src, int64_t plane, int n, int heads,
                                                      int rows, void* __restrict__ out, Strides st, int64_t total) {
  const int64_t e = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 8;
  if (e >= total) return;
  float v[8] = {};
  for (int s = 0; s < n; ++s) {
    const float4 x = *reinterpret_cast<const float4*>(src + s * plane + e);
    const float4 y = *reinterpret_cast<const float4*>(src + s * plane + e + 4);
    v[0] += x.x; v[1] += x.y; v[2] += x.z; v[3] += x.w;
    v[4] += y.x; v[5] += y.y; v[6] += y.z; v[7] += y.w;
  }
  const int64_t row = e / D, i = row % rows, bh = row / rows;
  uint16_t* dst = static_cast<uint16_t*>(out) + (bh / heads) * st.b + (bh % heads) * st.h + i * st.s + e % D;
  st16(dst, make_uint4(pack2_rn<F16>(v[0], v[1]), pack2_rn<F16>(v[2], v[3]), pack2_rn<F16>(v[4], v[5]),
                       pack2_rn<F16>(v[6], v[7])));
}

// dtable[h][k]: the warps' sums of every batch entry and key tile, in a fixed order; 64-bit, as a far bucket's sum is the
// small rest of large ones.
template <bool F16>
__global__ void __launch_bounds__(256) dtable_kernel(const DenseDims a, const float* __restrict__ part, int nkt,
                                                     void* __restrict__ dtable) {
  const int h = blockIdx.x, kvh = h / a.G, g = h % a.G, k = blockIdx.y * 32 + threadIdx.x % 32, w = threadIdx.x / 32;
  __shared__ double s_sum[8][32];
  double sum = 0.0;
  if (k < a.buckets)
    for (int64_t t = 0; t < (int64_t)a.B * nkt; ++t) {
      const int64_t b = t / nkt, kt = t % nkt;
      sum += part[((((b * a.Hkv + kvh) * nkt + kt) * a.G + g) * 8 + w) * a.buckets + k];
    }
  s_sum[w][threadIdx.x % 32] = sum;
  __syncthreads();
  if (w == 0 && k < a.buckets) {
    for (int i = 1; i < 8; ++i) sum += s_sum[i][threadIdx.x];
    static_cast<uint16_t*>(dtable)[(int64_t)h * a.buckets + k] = (uint16_t)pack2_rn<F16>((float)sum, 0.f);
  }
}

template <int D, bool F16>
int rows_t(const DenseDims& a, const DenseTensor& o, const DenseTensor& low, const DenseTensor& dout, const DenseTensor& v, const float* lse,
           const DenseBwdBuf& w, cudaStream_t st) {
  constexpr int ROWS = 256 / (D / 8);
  KernelTimer timer("dense_bwd_rows", st);
  if (F16 && cudaMemsetAsync(w.amax, 0, (size_t)a.B * a.Hkv * 8, st) != cudaSuccess) return LH_ERR_CUDA;
  bwd_rows_kernel<D, F16><<<dim3((a.Sq + ROWS - 1) / ROWS, a.B * a.Hq), 256, 0, st>>>(
      a, static_cast<const uint16_t*>(o.p), o.st, static_cast<const uint16_t*>(low.p), low.st,
      static_cast<const uint16_t*>(dout.p), dout.st, lse, w.stats, w.dqacc,
      w.amax);
  if (F16)
    v_norm_kernel<D><<<dim3((a.Skv + 8 * ROWS - 1) / (8 * ROWS), a.B * a.Hkv), 256, 0, st>>>(
        a, static_cast<const uint16_t*>(v.p), v.st, w.amax);
  return check_launch();
}

template <int D, bool F16>
int out_t(const DenseDims& a, const DenseTensor& dq, const DenseTensor& dk, const DenseTensor& dv, void* dtable,
          const DenseBwdBuf& w, cudaStream_t st) {
  KernelTimer timer("dense_bwd_out", st);
  auto run = [&](const float* src, int64_t plane, int n, int heads, int rows, const DenseTensor& t) {
    const int64_t total = (int64_t)a.B * heads * rows * D;
    bwd_out_kernel<D, F16><<<(unsigned)((total / 8 + 255) / 256), 256, 0, st>>>(src, plane, n, heads, rows,
                                                                               const_cast<void*>(t.p), t.st, total);
  };
  run(w.dqacc, 0, 1, a.Hq, a.Sq, dq);
  const int shares = dense_bwd_shares(a);
  if (shares > 1) {
    const int64_t one = (int64_t)a.B * a.Hkv * a.Skv * D;
    run(w.dkv, 2 * one, shares, a.Hkv, a.Skv, dv);
    run(w.dkv + one, 2 * one, shares, a.Hkv, a.Skv, dk);
  }
  if (a.table)
    dtable_kernel<F16><<<dim3(a.Hq, (a.buckets + 31) / 32), 256, 0, st>>>(a, w.dtpart, (a.Skv + kKeyTile - 1) / kKeyTile,
                                                                         dtable);
  return check_launch();
}

}  // namespace

int launch_dense_bwd_rows(const DenseDims& a, const DenseTensor& o, const DenseTensor& low, const DenseTensor& dout,
                          const DenseTensor& v, const float* lse, const DenseBwdBuf& w, cudaStream_t st) {
  auto run = a.d == 64 ? (a.f16 ? rows_t<64, true> : rows_t<64, false>) : (a.f16 ? rows_t<128, true> : rows_t<128, false>);
  return run(a, o, low, dout, v, lse, w, st);
}

int launch_dense_bias(const DenseDims& a, const BucketStarts& bs, const DenseBwdBuf& w, cudaStream_t st) {
  KernelTimer timer("dense_bias", st);
  const int blocks = (2 * a.near + 1 + 255) / 256;
  const dim3 grid(blocks < 64 ? blocks : 64, a.Hq);
  if (a.f16) bias_kernel<true><<<grid, 256, 0, st>>>(a, bs, w.bias, w.bucket, w.range);
  else bias_kernel<false><<<grid, 256, 0, st>>>(a, bs, w.bias, w.bucket, w.range);
  return check_launch();
}

int launch_dense_bwd_out(const DenseDims& a, const DenseTensor& dq, const DenseTensor& dk, const DenseTensor& dv,
                         void* dtable, const DenseBwdBuf& w, cudaStream_t st) {
  return a.d == 64 ? (a.f16 ? out_t<64, true>(a, dq, dk, dv, dtable, w, st) : out_t<64, false>(a, dq, dk, dv, dtable, w, st))
                   : (a.f16 ? out_t<128, true>(a, dq, dk, dv, dtable, w, st)
                            : out_t<128, false>(a, dq, dk, dv, dtable, w, st));
}

int launch_dense_doc_ranges(const DenseDims& a, int2* kdoc, int2* qdoc, cudaStream_t st) {
  const int nk = (a.Skv + kKeyTile - 1) / kKeyTile, nq = qdoc ? (a.Sq + 63) / 64 : 0;
  KernelTimer timer("dense_doc_ranges", st);
  doc_ranges_kernel<<<dim3((nk + nq + 7) / 8, a.B), 256, 0, st>>>(a, kdoc, qdoc, nk, nq);
  return check_launch();
}

}  // namespace lh
