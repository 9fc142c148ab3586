// host.cuh -- what the translation units of libovc share on the host: the
// per-device state and the tensor-map encoder, both defined in ovc.cu.
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>

#include "ovc.h"

namespace ovc {

struct DeviceState {
  bool init = false;
  bool supported = false;
  int index = 0;                    // the device's ordinal
  int sms = 0;
  unsigned int* status = nullptr;   // the device's status word
};

// State of the current device, set up on its first use; OVC_ERR_UNSUPPORTED
// unless it is an sm_103 device.
ovc_status device_state(DeviceState** out);

// cuTensorMapEncodeTiled, or nullptr.
PFN_cuTensorMapEncodeTiled_v12000 encode_fn();

// Bits of the device status word (kStatusTimeout, for expired waits, is 1).
constexpr unsigned kStatusBadIndex = 2u;

}  // namespace ovc
