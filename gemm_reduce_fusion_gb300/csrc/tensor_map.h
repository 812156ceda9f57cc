// The driver's tensor-map encoder, looked up once (tp_fused.cu).
#pragma once
#include <cuda.h>
#include <cudaTypedefs.h>

namespace tpf {
PFN_cuTensorMapEncodeTiled_v12000 encode_fn();
}
