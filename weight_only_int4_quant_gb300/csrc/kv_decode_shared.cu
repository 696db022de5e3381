// The kernel of kv_decode.cu for a batch that shares a prefix: the same source,
// compiled as a translation unit of its own so that the two build in parallel.
#define TLQ_KV_SHARED_UNIT 1
#include "kv_decode.cu"
