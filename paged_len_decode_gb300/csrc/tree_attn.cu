// tree_attn.cu -- attention of drafted tokens that form a tree: the prompt
// attention's kernels (window_prompt.cuh) with a mask of ancestors.
//
// Operation: a row's n drafted tokens lie in the slots from base = L - n on; token i sees
//   {j < base: at_i - j < W or j < S}, the drafted tokens k < i of its mask, and itself,
// at_i = base + popcount(mask_i & (2^i - 1)): its position, which its window counts back from.
// All that is seen lies before the token's own slot, so the lists of key tiles are the prompt's
// (windows begin at the root's place), and only what a row sees of a tile differs: the bits of
// 32 keys come from two words of its mask, in the one or two tiles that hold drafted tokens.
#include "window_prompt.cuh"

namespace vh {

cudaError_t prepare_tree_attn(int (&clusters)[5]) { return prepare_prompt<true>(clusters); }
cudaError_t launch_tree_attn(const PromptParams& p, cudaStream_t stream) { return launch_prompt<true>(p, stream); }

}  // namespace vh
