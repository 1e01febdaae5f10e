// attn_window_decode.hip -- attention of new tokens with a sliding window and
// sinks over a paged cache, gfx950: the kernel of attn_tree.hip over the
// positions that the window and the sinks leave.
//
// The token at position p sees position x <= p if x > p - window or x < sinks.
// A row tile (16 to 128 tokens x grouped heads) walks the sinks and the
// positions from its first token's window to its last token, numbered without
// the gap between them; tiles of 32 keys that hold the end of the sinks, a
// window's beginning for some of the tokens, or the tokens themselves are
// masked.  What lies in the gap is not read: however long the context, a
// sequence costs its window and sinks once per key head, and the step is
// bound by HBM as that of the whole context is (256 sequences, 32/8 heads of
// 128, window 1024: 181 us, 4.6 TB/s; 64 with a window of 8192: 384 us, 5.6
// TB/s).  One sequence of 16k: two launches one after the other, 8.4 and 4.5 us.
#include "attn_tree.hpp"

namespace kda {

hipError_t launch_attn_window_decode(const TreeArgs& a, const TreePlan& p) {
    return a.T_q == 0 ? hipSuccess : launch_tree<TreeMode::kWindow>(a, p);
}

}  // namespace kda
