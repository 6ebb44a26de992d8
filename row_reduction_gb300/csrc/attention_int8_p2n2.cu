// Attention over the cache: int8 codes, FP16 and FP32 queries, 16 columns.
#include "attention_mma.cuh"
namespace mt {
MT_DEFINE_ATTENTION(launch_attention_int8_p2n2, true, 2, 2)
}  // namespace mt
