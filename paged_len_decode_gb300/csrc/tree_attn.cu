// tree_attn.cu -- attention of drafted tokens that form a tree: the prompt
// attention's kernels (window_prompt.cuh) with a mask of ancestors.
//
// Operation: a row's n drafted tokens lie in the slots from base = L - n on; token i sees
//   {j < base: at_i - j < W or j < S}, the drafted tokens k < i of its mask, and itself,
// at_i = base + popcount(mask_i & (2^i - 1)): its position, which its window counts back from.
// (Masks without the ancestors that a window hides keep this right: the W - 1 that are left put at_i at
// base + W - 1, where the window ends behind the context.)
// All that is seen lies before the token's own slot, so the lists of key tiles are the prompt's
// (windows begin at the root's place), and only what a row sees of a tile differs: the bits of
// 32 keys come from two words of its mask, in the one or two tiles that hold drafted tokens.
//
// Bound by HBM for small trees (2 D bytes of a key and value against 4 D G n flops), by HBM and
// the tensor cores alike for 64 tokens of 4 q heads a kv head: 256 rows over 180,000 keys
// (745 MB, 188 GFLOP), which need 110 and 100 us, take 168.  What they lose is balance: every
// (request, kv head) has a cluster of two, 128 CTAs on 152 SMs, and the longest of the eight requests
// has 1.25 times the mean's keys: 0.84 x 0.80 of the machine is 0.67, which is 110 / 168.  Equal
// shares of every block through memory (2 to 8 units of the same counter, joined by a second kernel)
// filled every SM, kept the shares of the long requests long, paid a start each, and took
// 174-191; one CTA a block 286, two blocks of 128 rows a request 177.  32 ragged trees of
// up to 59 tokens (head_dim 64, window 1024) take 25 us, 16 tokens over 5000 14.5: start 4.5,
// five key tiles 4.5, outputs and the cluster's join 5.
#include "window_prompt.cuh"

namespace vh {

cudaError_t prepare_tree_attn(int (&clusters)[5]) { return prepare_prompt<true>(clusters); }
cudaError_t launch_tree_attn(const PromptParams& p, cudaStream_t stream) { return launch_prompt<true>(p, stream); }

}  // namespace vh
