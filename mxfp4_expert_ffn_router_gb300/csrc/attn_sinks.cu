// attn_sinks.cu -- attention of at most one new token per sequence over its window and the first tokens that stay
// visible: the kernels of attn_decode.cu, built for rows found by offsets.  They are a translation unit of their own so that
// both are compiled at the same time, and the calls without sinks keep the code they had.
#define K3_AD_SINKS 1
#include "attn_decode.cu"
