// dense_bwd_fp16_128.cu — the dense stage's backward kernels for fp16 rows of 128 features.
#include "dense_bwd.cuh"

namespace lh {
namespace bwd {
template int launch<128, true>(const CUtensorMap (&)[8], const BwdArgs&, cudaStream_t);
}  // namespace bwd
}  // namespace lh
