// dense_bwd_fp16_64.cu — the dense stage's backward kernels for fp16 rows of 64 features.
#include "dense_bwd.cuh"

namespace lh {
namespace bwd {
template int launch<64, true>(const CUtensorMap (&)[8], const BwdArgs&, cudaStream_t);
}  // namespace bwd
}  // namespace lh
