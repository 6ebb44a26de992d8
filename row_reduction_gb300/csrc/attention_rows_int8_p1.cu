// Attention over the cache, many rows: int8 codes, BF16 queries.
#include "attention_rows.cuh"
namespace mt {
MT_DEFINE_ATTENTION_ROWS(launch_attention_rows_int8_p1, true, 1)
}  // namespace mt
