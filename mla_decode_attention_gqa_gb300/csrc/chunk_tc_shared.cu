// The tensor-core attention kernel's variants for the passes of a shared prefix.
#define SKV_CHUNK_SHARED
#include "chunk_tc.cu"
