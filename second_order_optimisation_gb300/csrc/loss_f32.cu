// loss_f32.cu -- the losses' kernels for logits of type fp32 (sources are compiled in
// parallel, one type to each).
#include "loss.cuh"

namespace kfac {
namespace loss {
KFAC_LOSS_LAUNCHES(, KFAC_F32)
}  // namespace loss
}  // namespace kfac
