// Shared-prefix attention over coded caches with 32 channels per code (shared_mma.cuh, shared_rows.cuh).
#include "shared_launch.cuh"

namespace loopvq {

LQ_DEFINE_CODED(32)

}  // namespace loopvq
