// Attention over the cache: e4m3 codes, FP16 and FP32 queries, 16 columns.
#include "attention_mma.cuh"
namespace mt {
MT_DEFINE_ATTENTION(launch_attention_e4m3_p2n2, false, 2, 2)
}  // namespace mt
