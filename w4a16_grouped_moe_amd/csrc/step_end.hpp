// Declarations of the operators at the end of a serving step (not part of the
// ABI): the few-token W4A16 product, the rules on logits, the sampler with them.
#pragma once

#include "dgw4_internal.hpp"

#include "dgw4.h"

namespace dgw4 {

// The dense W4A16 product for few tokens (w4_few.hip): at most kW4FewTokens.
constexpr int kW4FewTokens = 64;

struct W4FewArgs {
    const void *x;              // [T, K] of x_type (DGW4_F16, DGW4_BF16), rows ldx apart
    const uint8_t *q;           // one packed matrix [N, K/2], canonical or tiled
    const uint16_t *s, *z;      // [N, K/g]
    void *y;                    // [T, N] of y_type, rows ldy apart
    long long ldx, ldy;         // in elements
    int T, K, N;
    int x_type, y_type, tiled;
};

hipError_t launch_w4_few(const W4FewArgs &a, int g, hipStream_t stream);

// A batch of requests' rules on its logits (logit_rules.hip), on their own and
// inside the sampler's pass; any output of the latter may be null.
struct LogitArgs {
    dgw4_logit_rules rules;
    const void *logits;         // [R, V] of type, rows ld apart
    void *out;                  // adjust: [R, V] of out_type, rows ld_out apart
    void *parts;                // sample: the partials (workspace)
    float *entropy;
    int32_t *sample, *argmax;
    long long ld, ld_out;
    int R, V, type, out_type;
    uint32_t k0, k1;            // the noise's key
};

hipError_t launch_adjust_logits(const LogitArgs &a, hipStream_t stream);
size_t sample_adjusted_workspace_bytes(int R, int V);
hipError_t launch_sample_adjusted(const LogitArgs &a, hipStream_t stream);

}  // namespace dgw4
