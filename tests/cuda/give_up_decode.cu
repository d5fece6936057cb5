// The decode attention with a wait that gives up on demand.
#include "give_up.cuh"

#include "gdn_attn_decode.cu"
#include "gdn_paged.cu"

extern "C" unsigned give_up_flags() { return gdn::read_and_clear_watchdog_attn_decode(nullptr); }
