/* Between libtq.so and the torch module alone. */
#pragma once

#include "tq.h"

#ifdef __cplusplus
extern "C" {
#endif

/* tq_kv8_attention; zero_behind: the rows of d_out behind the last entry's become 0
 * (an output that nobody has written yet) instead of staying as they were. */
TQ_API int tq_kv8_attention_rows(const tq_kv8_t *c, int layer, int ns, const int32_t *d_slots,
                                 const int32_t *d_cu, int64_t total_q, int max_q, int heads_q,
                                 const void *d_q, int q_dtype, int64_t q_ts, int64_t q_hs, float scale,
                                 int causal, int window, void *d_out, int zero_behind, float *d_lse,
                                 void *d_ws, size_t ws_bytes, void *stream);

#ifdef __cplusplus
}
#endif
