// The gate's arguments and checks, shared by its entry points (moe_gate.hip) and by the router
// that runs it on its own logits (moe_layer.hip).
#ifndef MBE_GATE_H
#define MBE_GATE_H

#include "block_host.h"

namespace block {

constexpr int kGateExperts = 1024, kGateSlots = 64, kGateGroups = 64;

// How experts are chosen and weighted.
struct GateRule {
    int top_k, scores, groups, top_groups, group_top, renormalize;
    float scale;
};

struct GateArgs {
    const void *logits;  // [tokens][experts], or the router's partial sums [parts][tokens][experts] in fp64
    const float *bias;
    int *ids;
    float *probs;
    const int *valid;
    int tokens, experts, parts;
    GateRule rule;
};

inline bool good_gate_scores(int scores, float scale)
{
    return (scores == BLOCK_SCORES_SOFTMAX || scores == BLOCK_SCORES_SIGMOID) && scale - scale == 0.0f;
}

inline bool good_gate(const GateRule &r, int experts)
{
    return experts >= 1 && experts <= kGateExperts && good_gate_scores(r.scores, r.scale) && r.groups >= 1 &&
           r.groups <= kGateGroups && experts % r.groups == 0 && r.top_groups >= 1 && r.top_groups <= r.groups &&
           r.group_top >= 1 && r.group_top <= 2 && (r.groups == 1 || r.group_top <= experts / r.groups) &&
           r.top_k >= 1 && r.top_k <= kGateSlots && r.top_k <= r.top_groups * (experts / r.groups);
}

// The gate over the router's partial sums (defined in moe_gate.hip).
block_status_t gate_of_parts(const GateArgs &a, hipStream_t stream);

}  // namespace block

#endif  // MBE_GATE_H
