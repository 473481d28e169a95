// dense_fwd_fp16_128.cu — the dense stage's forward kernels for fp16 rows of 128 features.
#include "dense_fwd.cuh"

namespace lh {
namespace fwd {
template int launch<128, true>(const FwdMaps&, const FwdArgs&, const BucketStarts&, int, cudaStream_t);
}  // namespace fwd
}  // namespace lh
