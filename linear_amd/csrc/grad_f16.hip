// The gradients' streaming kernels for binary16 words.
#include "grad_impl.h"

namespace lin {

template hipError_t launch_grad_stream_t<kF16>(int, bool, int, const StreamProduct&, hipStream_t);
template hipError_t launch_grad_pair_t<kF16>(bool, const StreamProduct&, const StreamProduct&, hipStream_t);

}  // namespace lin
