#include "kvd_internal.h"
extern "C" kvd_status kvd_sample_filtered(const float*, int64_t, int32_t, int32_t, const float*, const int32_t*, const float*, const float*, const float*, int32_t*, float*, int32_t*, uint32_t, int32_t*, kvd_stream_t) { return KVD_ERR_UNSUPPORTED; }
