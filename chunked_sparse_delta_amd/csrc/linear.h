// Linear attention with a decay for each head: what its kernels and host entry points share.
#pragma once

#include "delta_tile.h"

namespace sdm {

// Tokens of a segment: its sum of k v is one product of the state kernel, and inside it pairs of tokens meet
// directly. At most the threads of a workgroup (a token's gate each), a multiple of the attending kernel's query tiles.
constexpr int kLinSegMax = 256;

// Log-decays [P, T, Hv] (strides T * Hv, Hv) or [Hv] (strides 0, 0).
struct LinGates {
    const float *g;
    int64_t sp, st;
};

struct LinArgs {
    Rows q, k, v;
    LinGates gates;
    const float *state;      // [P, Hv, K, V] or null
    float *state_out;        // or null
    const int32_t *valid;    // [P] or null
    void *out;               // [P, T, Hv, V]
    int32_t P, T, Hk, Hv, K, V;
    float scale;
};

// ph = stream * Hv + value head; segments of `tokens` tokens.
struct LinWs {
    float *S;          // [ph][segs + 1][K][V]: each segment's sum, then its start state; the end state last
    float *decay;      // [ph][segs]: exp of a segment's summed log-decays
    float *dS;         // [ph][segs][K][V]: the same for the state's gradient: a segment's end (backward)
    float *dots;       // [ph][segs][lin_dot_parts]: <end state, its gradient> by wavefronts (backward)
    float *rows, *cols;  // [slices][ph][T]: the gates' shares through dq and dk, a slice of K each (backward)
    double *sums;      // [ph][segs]: a segment's sum of log-decay gradients (backward, a decay for each head)
    int32_t segs, tokens;
};

struct LinGrads {
    Rows go;                 // [P, T, Hv, V]
    const float *gstate;     // [P, Hv, K, V] or null
    void *q, *k, *v;
    float *g;                // as the log-decays, or null
    float *state;            // or null
};

inline int lin_width(int n) { return n <= 64 ? 64 : n <= 128 ? 128 : 256; }   // padded depth of scores
inline int lin_slice(int n) { return n <= 64 ? 64 : 128; }                    // columns of a workgroup
inline int lin_slices(int n) { return (n + lin_slice(n) - 1) / lin_slice(n); }
int lin_dot_parts(int K, int V);

hipError_t linear_prepare();
// keep: the start states and decays stay in ws for the backward.
hipError_t launch_linear_fwd(const LinArgs &a, const LinWs &ws, bool is_bf16, bool keep, hipStream_t st);
// kept: ws holds them already.
hipError_t launch_linear_bwd(const LinArgs &a, const LinWs &ws, const LinGrads &g, bool is_bf16, bool kept, hipStream_t st);

}  // namespace sdm
