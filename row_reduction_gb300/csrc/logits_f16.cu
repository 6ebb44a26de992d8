// Logits: f16 storage.
#include "logits.cuh"
namespace mt {
MT_DEFINE_LOGITS(__half, f16)
}  // namespace mt
