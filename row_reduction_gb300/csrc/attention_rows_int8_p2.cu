// Attention over the cache, many rows: int8 codes, FP16 and FP32 queries.
#include "attention_rows.cuh"
namespace mt {
MT_DEFINE_ATTENTION_ROWS(launch_attention_rows_int8_p2, true, 2)
}  // namespace mt
