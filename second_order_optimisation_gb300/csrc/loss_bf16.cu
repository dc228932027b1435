// loss_bf16.cu -- the losses' kernels for logits of type bf16 (sources are compiled in
// parallel, one type to each).
#include "loss.cuh"

namespace kfac {
namespace loss {
KFAC_LOSS_LAUNCHES(, KFAC_BF16)
}  // namespace loss
}  // namespace kfac
