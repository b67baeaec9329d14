// Attention of prompts over q8 keys and q8 values.
#include "attend_prompt.cuh"

namespace tria {

cudaError_t launch_attend_prompt_q8_q8(const AttendArgs& A, cudaStream_t st) {
  return launch_attend_prompt_kv<TRIA_Q8_0, TRIA_Q8_0>(A, st);
}

}  // namespace tria
