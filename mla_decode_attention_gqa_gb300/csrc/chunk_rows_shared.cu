// The variants of the attention kernel for few rows for the passes of a shared prefix.
#define SKV_CHUNK_SHARED
#include "chunk_rows.cu"
