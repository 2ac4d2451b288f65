// Stand-ins for the launchers of the vocabulary operators, for running
// vocab_api.hip as host code: a launch is counted and the last arguments kept.
#include "vocab_internal.h"

namespace {

int launches;
zk::Drop drop;
zk::HeadPlan head;

hipError_t launched() {
    ++launches;
    return hipSuccess;
}

}  // namespace

extern "C" {

int double_vocab_launches() { return launches; }
uint32_t double_drop_limit() { return drop.limit; }
float double_drop_scale() { return drop.scale; }
int64_t double_head_bytes() { return head.bytes; }
int64_t double_head_pieces() { return head.pieces; }
int double_head_parts(int steps, int k, int *per) {
    const zk::HeadParts h = zk::head_parts(steps, k);
    *per = h.per;
    return h.parts;
}

}

namespace zk {

hipError_t launch_embed(const EmbedArgs &a, hipStream_t) {
    drop = a.drop;
    return launched();
}
hipError_t launch_embed_grad(const EmbedGradArgs &a, const EmbedGradPlan &, hipStream_t) {
    drop = a.drop;
    return launched();
}
hipError_t launch_dropout(const DropoutArgs &a, hipStream_t) {
    drop = a.drop;
    return launched();
}
hipError_t launch_head(const HeadArgs &, const HeadPlan &p, hipStream_t) {
    head = p;
    return launched();
}

}  // namespace zk
