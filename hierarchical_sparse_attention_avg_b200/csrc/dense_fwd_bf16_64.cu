// dense_fwd_bf16_64.cu — the dense stage's forward kernels for bf16 rows of 64 features.
#include "dense_fwd.cuh"

namespace lh {
namespace fwd {
template int launch<64, false>(const FwdMaps&, const FwdArgs&, const BucketStarts&, int, cudaStream_t);
}  // namespace fwd
}  // namespace lh
