// device_context.h -- what ltxattn_create sets up for the current device, for the host files
// that launch attention kernels (internal; defined in ltxattn.cu).
#pragma once

#include <atomic>

#include "host_common.h"

namespace ltx {

struct DeviceContext {
  EncodeTiledFn encode;  // cuTensorMapEncodeTiled
  int num_sms;
  int* d_status;         // device status word
  std::atomic<uint64_t>* masked_limits;  // bit i: masked kernel i has its shared-memory limit
};

// The current device's context: LTXATTN_OK, LTXATTN_ERR_NOT_INITIALIZED without
// ltxattn_create, or LTXATTN_ERR_CUDA.
int device_context(DeviceContext* out);

}  // namespace ltx
