// Attention of drafted tokens (tree_attn.h), f16 queries.
#include "tree_attn.h"

namespace tcm {

hipError_t launch_tree_attention_f16(const TreeArgs& a, bool e4m3, hipStream_t st) { return launch_tree<_Float16>(a, e4m3, st); }

}  // namespace tcm
