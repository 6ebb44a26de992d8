// Norms around a block: bf16 storage.
#include "block_norm.cuh"
namespace mt {
MT_DEFINE_BLOCK_NORM(__nv_bfloat16, bf16)
}  // namespace mt
