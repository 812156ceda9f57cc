// Internal interface of the 4-bit sharded Linear (w4.cu).
#pragma once
#include <cstddef>
#include <cstdint>

namespace tpf {

// Workspace of the 4-bit forward calls: the status word and fp32 partials.
size_t w4_workspace(bool row, int p, int64_t M, int64_t N, int64_t K);

}  // namespace tpf
