// dense_bwd.cu — host side of the dense stage's backward.
#include "dense_bwd.cuh"

namespace lh {
namespace bwd {

extern template int launch<64, false>(const CUtensorMap (&)[8], const BwdArgs&, cudaStream_t);
extern template int launch<64, true>(const CUtensorMap (&)[8], const BwdArgs&, cudaStream_t);
extern template int launch<128, false>(const CUtensorMap (&)[8], const BwdArgs&, cudaStream_t);
extern template int launch<128, true>(const CUtensorMap (&)[8], const BwdArgs&, cudaStream_t);

}  // namespace bwd

int dense_bwd_shares(const DenseDims& a) {
  // Query heads of one key head in as many blocks as it takes to give every SM two blocks.
  const int64_t blocks = (int64_t)a.B * a.Hkv * ((a.Skv + kKeyTile - 1) / kKeyTile);
  for (int n = 1; n < a.G; ++n)
    if (a.G % n == 0 && blocks * n >= 2 * 148) return n;
  return a.G;
}

int launch_dense_bwd(const DenseDims& a, const DenseTensor& q, const DenseTensor& k, const DenseTensor& v,
                     const DenseTensor& dout, const DenseTensor& dk, const DenseTensor& dv, const DenseBwdBuf& w,
                     cudaStream_t st) {
  CUtensorMap m[8];
  if (make_tmap_dense(&m[0], q, a.d, a.Sq, a.Hq, a.B, 1, bwd::kQTile) ||
      make_tmap_dense(&m[1], k, a.d, a.Skv, a.Hkv, a.B, 1, kKeyTile) ||
      make_tmap_dense(&m[2], v, a.d, a.Skv, a.Hkv, a.B, 1, kKeyTile) ||
      make_tmap_dense(&m[3], dout, a.d, a.Sq, a.Hq, a.B, 1, bwd::kQTile) ||
      make_tmap_f32_3d(&m[4], w.dqacc, a.d, a.Sq, a.B * a.Hq, 32, bwd::kQTile) ||
      make_tmap_stats(&m[5], w.stats, a.Sq, a.B * a.Hq, bwd::kQTile) ||
      make_tmap_dense(&m[6], dk, a.d, a.Skv, a.Hkv, a.B, 1, kKeyTile) ||
      make_tmap_dense(&m[7], dv, a.d, a.Skv, a.Hkv, a.B, 1, kKeyTile))
    return LH_ERR_CUDA;
  bwd::BwdArgs p;
  p.a = a;
  p.nkt = (a.Skv + kKeyTile - 1) / kKeyTile;
  p.heads = a.G / dense_bwd_shares(a);
  p.head_fast = p.nkt < bwd::kHeadFastBelow;
  p.w = w;
  if (p.heads == a.G) p.w.dkv = nullptr;
  KernelTimer timer("dense_bwd", st);
  return a.d == 64 ? (a.f16 ? bwd::launch<64, true>(m, p, st) : bwd::launch<64, false>(m, p, st))
                   : (a.f16 ? bwd::launch<128, true>(m, p, st) : bwd::launch<128, false>(m, p, st));
}

}  // namespace lh
