// dense_prep.cu — the small kernels around the dense stage's attention: the documents' ranges of the tiles.
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

}  // namespace

int launch_dense_doc_ranges(const DenseDims& a, int2* kdoc, int2* qdoc, cudaStream_t st) {
  const int nk = (a.Skv + kKeyTile - 1) / kKeyTile, nq = qdoc ? (a.Sq + 63) / 64 : 0;
  KernelTimer timer("dense_doc_ranges", st);
  doc_ranges_kernel<<<dim3((nk + nq + 7) / 8, a.B), 256, 0, st>>>(a, kdoc, qdoc, nk, nq);
  return check_launch();
}

}  // namespace lh
