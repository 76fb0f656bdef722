// host.cuh — host-side helpers shared by the translation units of the entry
// points: error reporting, device facts, programmatic-dependent launches and
// the tensor-map encoder.  Defined in qmoe.cu unless inline here.
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "../../include/qmoe.h"
#include "ptx.cuh"

namespace qmoe {

// Records the message qmoe_last_error returns on this thread; returns `st`.
__attribute__((format(printf, 2, 3))) qmoe_status fail(qmoe_status st, const char* fmt, ...);
qmoe_status cuda_fail(cudaError_t e, const char* what);
void clear_error();

inline bool aligned(const void* p, uintptr_t a) {
    return (reinterpret_cast<uintptr_t>(p) % a) == 0;
}

struct DevInfo {
    bool init = false;
    bool supported = false;
    int dev = 0;
    int sms = 0;
    int smem_optin = 0;
    int smem_pair = 0;  // dynamic shared memory per CTA that lets two CTAs share an SM
    DevCtl* err = nullptr;
    int cc_major = 0, cc_minor = 0;
};

// Facts of the current device; UNSUPPORTED unless it is sm_103.
qmoe_status device_info(DevInfo** out);

template <typename Kern, typename... Args>
static cudaError_t launch_pdl(Kern kern, dim3 grid, dim3 block, size_t smem, cudaStream_t st,
                              Args... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, args...);
}

// cuTensorMapEncodeTiled, looked up once through the runtime (no link
// against the driver library); null if the driver lacks it.
using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                   const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                   const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                   CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeTiledFn encode_tiled();

}  // namespace qmoe
