// Attention of drafted tokens (tree_attn.h), bf16 queries.
#include "tree_attn.h"

namespace tcm {

hipError_t launch_tree_attention_bf16(const TreeArgs& a, bool e4m3, hipStream_t st) { return launch_tree<__bf16>(a, e4m3, st); }

}  // namespace tcm
