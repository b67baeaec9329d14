// Attention of decode steps over q8 keys and q4 values.
#include "attend_step.cuh"

namespace tria {

cudaError_t launch_attend_step_q8_q4(const AttendArgs& A, int cols, int workers, cudaStream_t st) {
  return launch_attend_step_kv<TRIA_Q8_0, TRIA_Q4_0>(A, cols, workers, st);
}

}  // namespace tria
