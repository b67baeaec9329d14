// Attention of prompts over q4 keys and f16 values.
#include "attend_prompt.cuh"

namespace tria {

cudaError_t launch_attend_prompt_q4_f16(const AttendArgs& A, cudaStream_t st) {
  return launch_attend_prompt_kv<TRIA_Q4_0, TRIA_F16>(A, st);
}

}  // namespace tria
