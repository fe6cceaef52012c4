// attn_rows.cu -- attention of few new tokens per sequence, each with what it sees: the kernels of attn_decode.cu, built for
// columns of several tokens.
#define K3_AD_SINKS 2
#include "attn_decode.cu"
