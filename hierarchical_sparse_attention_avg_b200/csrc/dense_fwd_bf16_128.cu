// dense_fwd_bf16_128.cu — the dense stage's forward kernels for bf16 rows of 128 features.
#include "dense_fwd.cuh"

namespace lh {
namespace fwd {
template int launch<128, false>(const FwdMaps&, const FwdArgs&, const BucketStarts&, int, cudaStream_t);
}  // namespace fwd
}  // namespace lh
