// Attention of prompts over q8 keys and q4 values.
#include "attend_prompt.cuh"

namespace tria {

cudaError_t launch_attend_prompt_q8_q4(const AttendArgs& A, cudaStream_t st) {
  return launch_attend_prompt_kv<TRIA_Q8_0, TRIA_Q4_0>(A, st);
}

}  // namespace tria
