// The gradients' streaming kernels for bfloat16 words.
#include "outer_impl.h"

namespace lin {

template hipError_t launch_grad_stream_t<kBF16>(int, bool, int, const StreamProduct&, hipStream_t);
template hipError_t launch_outer_t<kBF16>(int, const StreamProduct&, hipStream_t);
template hipError_t launch_grad_pair_t<kBF16>(bool, const StreamProduct&, const StreamProduct&, hipStream_t);

}  // namespace lin
