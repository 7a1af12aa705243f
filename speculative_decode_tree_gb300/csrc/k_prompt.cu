// The prompt attention: which items go row by row (all of them).
#include "prompt_list.cuh"

namespace ddtree {
namespace {

__global__ void __launch_bounds__(128) prompt_all_kernel(const __grid_constant__ PromptArgs a) {
  __shared__ int scratch[12];
  await_grid();
  PromptItem it;
  const int got = find_prompt_item<128>(a, blockIdx.x / a.n_kv_heads, scratch, it);
  if (threadIdx.x == 0) a.words[blockIdx.x] = got == 2 ? DDTREE_ST_BAD_LENGTH : got == 0 ? kPromptAgain : 0;
}

}  // namespace

int prompt_tile_tokens(int group, int head_dim) { return 128 / group * (head_dim == 256 ? 1 : 2); }

cudaError_t launch_prompt(const PromptArgs& a, int num_sms, cudaStream_t stream) {
  const cudaError_t e = launch_early(prompt_all_kernel, a.max_items, 128, 0, stream, a);
  return e != cudaSuccess ? e : launch_prompt_rows(a, num_sms, stream);
}

}  // namespace ddtree
