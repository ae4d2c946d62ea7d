// What the host sides of the C ABI share: the set-up of the current device.
#pragma once

#include <cudaTypedefs.h>

namespace attn {

struct HostDevice {
  int dev, n_sm;
  int* err;              // the device's error word
  long long wait_limit;  // cycles, for every bounded wait
  int fault;             // host-injected (attn_debug_inject)
  PFN_cuTensorMapEncodeTiled_v12000 encode;
};
// Checks the current device on its first use; an attn_status.
int host_setup(HostDevice* out);

}  // namespace attn
