// Status reporting of libmoe_block.so (C ABI in block/moe_block.h).
#include "block_host.h"

namespace block {

namespace {
thread_local int g_last_hip = 0;
}

block_status_t fail_hip(hipError_t e)
{
    g_last_hip = (int)e;
    return BLOCK_ERR_HIP;
}

}  // namespace block

extern "C" {

const char *moe_block_status_string(block_status_t status)
{
    switch (status) {
    case BLOCK_OK: return "ok";
    case BLOCK_ERR_INVALID_ARG: return "invalid argument";
    case BLOCK_ERR_ALIGNMENT: return "misaligned pointer, or a width that is not a multiple of 8";
    case BLOCK_ERR_HIP: return "HIP launch failed";
    }
    return "unknown status";
}

int moe_block_last_hip_error(void) { return block::g_last_hip; }

int moe_block_abi_version(void) { return MOE_BLOCK_ABI_VERSION; }

}  // extern "C"
