// The gated block's streaming kernels for binary16 words.
#include "gemm_impl.h"

namespace lin {

template hipError_t launch_gated_stream_t<kF16>(int cfg, const LinearArgs& a, hipStream_t stream);

}  // namespace lin
