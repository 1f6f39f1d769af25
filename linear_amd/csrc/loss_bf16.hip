// The cross entropy's streaming kernels for bfloat16 words.
#include "loss_impl.h"

namespace lin {

template hipError_t launch_loss_stream_t<kBF16>(int cfg, int mode, const LossArgs& a, hipStream_t stream);

}  // namespace lin
