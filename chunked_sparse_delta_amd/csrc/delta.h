// The dense gated delta rule: what its kernels and host entry points share.
#pragma once

#include "common.h"

namespace sdm {

// A [P, T, heads, width] view (strides in elements).
struct Rows {
    const void *data;
    int64_t sp, st, sh;
    int32_t width;
};
constexpr int64_t kCus = 256;                  // MI355X
// Of tokens that the chunked kernels take as they are: a chunk's offsets fit 32 bits (those of copies: check_delta).
constexpr int64_t kDeltaMaxStride = 1 << 24;

// q or k as the chunked kernels take them: rows of the padded head_dim in bfloat16, `plane` elements
// between the pieces of a float32 input (see delta_tile.h), every row 16-byte aligned. They are
// the caller's rows where these are so, and copies otherwise; so with v (rows of a multiple of eight elements).
struct KeyRows {
    const bf16 *data;
    int64_t plane, sp, st, sh;
};

struct DeltaArgs {
    Rows q, k, v;
    KeyRows kk, qq;              // chunked kernels only; v is then regular too
    const float *beta, *g;       // [P, T, Hv]
    const float *state;          // [.., Hv, K, V] or null
    float *state_out;            // or null
    const int32_t *valid;        // [P] or null
    const int32_t *ids;          // [P] or null (step)
    int64_t slots;               // states (step)
    int64_t g_stream, g_token;   // g's strides (linear attention's step)
    void *out;                   // [P, T, Hv, V]
    int32_t P, T, Hk, Hv, K, V;
    float scale;
};

__device__ __forceinline__ int delta_valid(const DeltaArgs &a, int p) {
    return a.valid ? max(0, min(a.valid[p], a.T)) : a.T;
}

// The chunked kernels' workspace: chunk n = (stream * Hv + head) * Nt + chunk. U, Y, S and dS are
// kept as the accumulators hold them: [n][16-column group of V][32-row block][lane][8 rows].
struct DeltaWs {
    unsigned char *mats;   // [n] ChunkMem
    float *U, *Y;          // rows: the chunk's tokens (backward)
    float *S, *dS;         // rows: the padded head_dim; start states, gradients of the end states (backward)
    // A sequence may be walked in `segs` segments of seg_chunks chunks at once (delta_segments): their start states (the first's
    // too) [seg][stream * Hv + head][KP][VP] and the maps from a segment's start state to its end state [seg][..][KP][KP].
    float *seg_state, *seg_map;
    int32_t Nt, segs, seg_chunks;
    bool backward;         // X is computed for the backward (delta_beta_safe)
};

// Segments of Nt chunks for `heads` states walked by `slices` workgroups each.
int delta_segments(int64_t heads, int slices, int K, int Nt);

struct DeltaGrads {
    Rows go;                 // [P, T, Hv, V]
    const float *gstate;     // [P, Hv, K, V] or null
    void *q, *k, *v;
    float *beta, *g, *state; // state or null
};

// Padded head_dim of the chunked kernels, and tokens of a chunk.
inline int delta_kp(int K) { return K <= 64 ? 64 : K <= 128 ? 128 : 256; }
inline int delta_chunk(int K, bool is_bf16) { return is_bf16 && K <= 128 ? 64 : 32; }

hipError_t delta_prepare();
hipError_t delta_bwd_prepare();
// `results`: the readings and the final state are wanted (else, with ws.backward, only what the backward takes).
hipError_t launch_delta_fwd(const DeltaArgs &a, const DeltaWs &ws, bool is_bf16, bool results, hipStream_t st);
// Whether the chunked kernels can take the rows as they are, and the copies where they cannot (at `to`).
bool delta_regular_keys(const Rows &r, bool is_bf16);
bool delta_regular_values(const Rows &r, bool is_bf16);
// (`there`: they are at `to` already.)
hipError_t launch_delta_copy_keys(const Rows &r, KeyRows *k, void *to, int P, int T, int H, bool is_bf16, bool there, hipStream_t st);
hipError_t launch_delta_copy_values(Rows *r, void *to, int P, int T, int H, bool is_bf16, bool there, hipStream_t st);
size_t delta_mats_bytes(int K, bool is_bf16);   // of a chunk
hipError_t launch_delta_bwd(const DeltaArgs &a, const DeltaWs &ws, const DeltaGrads &g, bool is_bf16, bool kept, hipStream_t st);
hipError_t launch_delta_step(const DeltaArgs &a, bool is_bf16, int cus, hipStream_t st);
hipError_t launch_linear_step(const DeltaArgs &a, bool is_bf16, int cus, hipStream_t st);   // without beta

}  // namespace sdm
