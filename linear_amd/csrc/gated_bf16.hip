// The gated block's streaming kernels for bfloat16 words.
#include "gemm_impl.h"

namespace lin {

template hipError_t launch_gated_stream_t<kBF16>(int cfg, const LinearArgs& a, hipStream_t stream);

}  // namespace lin
