// What the kernels of libgba_moe share.
#pragma once

#include "../experts/gx_common.hpp"

namespace gbm {

using namespace gba;
using gbx::launch;

enum { DTYPE_F32 = 2 };   // beside DT_F16 and DT_BF16

// LDS that this wave's lanes wrote may be read by its other lanes.
__device__ __forceinline__ void wave_sync() {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

}  // namespace gbm
