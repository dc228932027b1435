// loss_f16.cu -- the losses' kernels for logits of type fp16 (sources are compiled in
// parallel, one type to each).
#include "loss.cuh"

namespace kfac {
namespace loss {
KFAC_LOSS_LAUNCHES(, KFAC_F16)
}  // namespace loss
}  // namespace kfac
