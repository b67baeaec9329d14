// Attention of decode steps over q4 keys and f16 values.
#include "attend_step.cuh"

namespace tria {

cudaError_t launch_attend_step_q4_f16(const AttendArgs& A, int cols, int workers, cudaStream_t st) {
  return launch_attend_step_kv<TRIA_Q4_0, TRIA_F16>(A, cols, workers, st);
}

}  // namespace tria
