// What the plans of vocab_api.hip say, for calling them as host code.
#include "vocab_internal.h"

extern "C" {

// Numbers that the loss's one workgroup turns into G, zeros behind the rows
// included; 0 where a kernel of its own does it.
int64_t rules_turned_with_loss(int64_t count, int64_t vocab, int64_t width, int bf16, int64_t piece) {
    zk::HeadArgs a = {};
    a.bf16 = bf16;
    a.count = count;
    a.vocab = vocab;
    a.width = width;
    a.grad_hidden = a.grad_table = &a;
    const zk::HeadPlan p = zk::plan_head(a, piece);
    return p.turn_with_loss ? p.piece_p * p.vocab_p : 0;
}

// Workgroups of the sort, and ids of each.
int64_t rules_sort_groups(int64_t count, int64_t rows, int *ids) {
    const zk::EmbedGradPlan p = zk::plan_embed_grad(count, rows, 8);
    *ids = p.ids_per_group;
    return (int64_t)1 << p.sort_groups_log2;
}

}
