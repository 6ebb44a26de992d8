// Logits: bf16 storage.
#include "logits.cuh"
namespace mt {
MT_DEFINE_LOGITS(__nv_bfloat16, bf16)
}  // namespace mt
