// Host-side pieces of libmoe_block.so.
#include "moe_block.h"

extern "C" int moe_block_abi_version(void) { return 1; }
