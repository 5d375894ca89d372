// The library is one translation unit: the weight quantizers, then the
// key/value cache, which uses their device check and error record, then the
// latent cache, which uses the key/value cache's batches, and both caches' pages.
#include "fp8bq.hip"

#include "kv.hip"

#include "latent.hip"

#include "pages.hip"
