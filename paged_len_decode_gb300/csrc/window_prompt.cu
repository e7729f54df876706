// window_prompt.cu -- the prompt attention's kernels (window_prompt.cuh).
#include "window_prompt.cuh"

namespace vh {

cudaError_t prepare_window_prompt(int (&clusters)[5]) { return prepare_prompt<false>(clusters); }
cudaError_t launch_window_prompt(const PromptParams& p, cudaStream_t stream) { return launch_prompt<false>(p, stream); }

}  // namespace vh
