// attn_sinks.cu -- attention of at most one new token per sequence, with the first tokens that stay visible: the kernels of
// attn_decode.cu, built for rows found by offsets.  A translation unit of its own, so that both are compiled at the same
// time and the calls without offsets keep the code they had.
#define K3_AD_SINKS 1
#include "attn_decode.cu"
