// The library is one translation unit: the weight quantizers, then the
// key/value cache, which uses their device check and error record.
#include "fp8bq.hip"

#include "kv.hip"
