// placeholder
#include "ssd_delta.cuh"
#include "ssd_internal.h"
extern "C" SSD_API size_t ssd_delta_bwd_workspace_size(const ssd_delta_bwd_args*) { return 0; }
extern "C" SSD_API ssd_status ssd_delta_bwd(const ssd_delta_bwd_args*, void*) { return SSD_ERR_UNSUPPORTED; }
