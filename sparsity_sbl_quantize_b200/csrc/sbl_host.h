// sbl_host.h -- what the library's translation units share on the host: the
// current device as sbl_api.cu probed it.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "sbl.h"

namespace sbl {

constexpr int kMaxDevices = 64;
constexpr int64_t kMaxDim = 65536;

typedef CUresult (*EncodeTiledFn)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *,
                                  const cuuint64_t *, const cuuint64_t *, const cuuint32_t *,
                                  const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                                  CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

struct HostDevice {
    int index;             // device number
    int num_sms;
    uint32_t *err;         // the device error word
    EncodeTiledFn encode;  // cuTensorMapEncodeTiled
};

// SBL_ERR_DEVICE unless an sm_100 device is current.
sbl_status host_device(HostDevice *out);

}  // namespace sbl
