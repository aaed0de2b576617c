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

// Tokens of a segment of a sequence of T. Longer ones have fewer states to write and read, shorter ones fewer pairs of tokens: of
// bfloat16 rows 256 took 170 us where 128 took 185 (4 x 16 heads of up to 4096 tokens of 128 x 128), of float32 rows, whose products cost
// twice as much, 128 took 78 us where 256 took 101 and 64, with twice the states, 75 (2 x 10 heads of 1500 tokens of 72 x 200).
// A sequence of at most half as much again takes halves, not a whole and a rest (training 32 x 16 heads of 128 x 128: 380 bfloat16
// tokens 579 us, whole ones 672; 160 float32 ones 489 and 594; readings of 4 x 8 heads: 300 bfloat16 tokens 39 and 46).
// The streams have no part in it: a stream's bits do not depend on the others.
inline int lin_seg_tokens(bool is_bf16, int T) {
    const int most = is_bf16 ? kLinSegMax : 128;
    if (T <= most) return T > 128 ? (T + 127) / 128 * 128 : 128;
    return T <= most / 2 * 3 ? most / 2 : most;
}

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
    float *dots;       // [ph][segs + 1][lin_dot_parts]: <state, its gradient> at each segment's start and at the end, by wavefronts (backward)
    float *rows, *cols;  // [slices][ph][T]: the gates' shares through dq and, negative, through dk, a slice of K each (backward)
    float *rest;       // dq's and dk's sums between the value heads that share a key head, lin_rest_floats each (backward)
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
__host__ __device__ constexpr int lin_slice(int n) { return n <= 64 ? 64 : 128; }                    // columns of a workgroup
inline int lin_slices(int n) { return (n + lin_slice(n) - 1) / lin_slice(n); }
// Over how many XCDs units of workgroups that share their operands are dealt; the grid is padded to as many.
__host__ __device__ inline int lin_xcds(int64_t units) { return units % kXcds == 0 || units >= 8 * kXcds ? kXcds : 1; }
inline size_t lin_rest_floats(int P, int Hk, int K, int segs, int seg_tokens) {
    return size_t(P) * size_t(segs) * size_t(Hk) * size_t(seg_tokens) * size_t(lin_slices(K) * lin_slice(K));
}
int lin_dot_parts(int K, int V);

hipError_t linear_prepare();
// keep: the start states and decays stay in ws for the backward.
hipError_t launch_linear_fwd(const LinArgs &a, const LinWs &ws, bool is_bf16, bool keep, hipStream_t st);
// kept: ws holds them already.
hipError_t launch_linear_bwd(const LinArgs &a, const LinWs &ws, const LinGrads &g, bool is_bf16, bool kept, hipStream_t st);

}  // namespace sdm
