// api_internal.h -- host helpers shared by the files that hold the C ABI.
#pragma once

#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

#include "../../include/longspec_hta.h"

namespace hta_api {

struct DeviceInfo {
    bool probed = false;
    bool supported = false;
    int num_sms = 0;
};
// The current device; LONGSPEC_HTA_ERR_UNSUPPORTED_DEVICE unless sm_100.
int current_device(DeviceInfo *out);

typedef CUresult (*EncodeTiledFn)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *,
                                  const cuuint64_t *, const cuuint64_t *, const cuuint32_t *,
                                  const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                                  CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeTiledFn encode_fn();

inline bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline bool aligned4(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
inline size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

int check_dims(const longspec_hta_dims *d);
float scale_of(const longspec_hta_dims *d);

}  // namespace hta_api
