// Shared-prefix attention over coded caches with 8 channels per code (shared_mma.cuh, shared_rows.cuh).
#include "shared_launch.cuh"

namespace loopvq {

LQ_DEFINE_CODED(8)

}  // namespace loopvq
