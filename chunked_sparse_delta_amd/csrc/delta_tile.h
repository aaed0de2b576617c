// Tiles of the chunked gated delta rule: 16 x 16 blocks on v_mfma_f32_16x16x4f32.
//
// An accumulator block holds, in lane l, column l & 15 of rows 4 (l >> 4) + r, r = 0..3. The
// instruction's k index is l >> 4, so step r of a 16-deep product may take k = 4 (l >> 4) + r:
// an accumulator block is then a B operand as it is, register by register.
#pragma once

#include "delta.h"

namespace sdm {

typedef float dt4 __attribute__((ext_vector_type(4)));

// Row-operand of rows r0.. and depth k0..: lane l holds m[r0 + (l & 15)][k0 + 4 (l >> 4) + r]
// (an A operand, or the B operand of a product with the transpose). ld a multiple of 4.
__device__ __forceinline__ dt4 tile_row(const float *m, int ld, int r0, int k0) {
    const int lane = threadIdx.x & 63;
    return *reinterpret_cast<const dt4 *>(m + (r0 + (lane & 15)) * ld + k0 + 4 * (lane >> 4));
}
// Column-operand: lane l holds m[k0 + 4 (l >> 4) + r][c0 + (l & 15)].
__device__ __forceinline__ dt4 tile_col(const float *m, int ld, int k0, int c0) {
    const int lane = threadIdx.x & 63;
    const float *p = m + (k0 + 4 * (lane >> 4)) * ld + c0 + (lane & 15);
    return dt4{p[0], p[ld], p[2 * ld], p[3 * ld]};
}
__device__ __forceinline__ dt4 tile_mma(dt4 a, dt4 b, dt4 acc) {
#pragma unroll
    for (int r = 0; r < 4; ++r) acc = __builtin_amdgcn_mfma_f32_16x16x4f32(a[r], b[r], acc, 0, 0, 0);
    return acc;
}
// Stores an accumulator block at rows r0.., columns c0...
__device__ __forceinline__ void tile_put(float *m, int ld, int r0, int c0, dt4 x) {
    const int lane = threadIdx.x & 63;
    float *p = m + (r0 + 4 * (lane >> 4)) * ld + c0 + (lane & 15);
#pragma unroll
    for (int r = 0; r < 4; ++r) p[r * ld] = x[r];
}

// A chunk's gates. G is the running sum of the log-decays, in 64 bits: differences of it are
// as exact as the log-decays themselves however large the sum grew, and a log-decay below
// -1e4 (-inf among them: it clears the state) counts as -1e4, whose exponential is 0 too.
template <int C> struct Gates {
    double G[C];
    float beta[C], eG[C], eL[C];   // exp(G), exp(G_last - G)
    float last;                    // exp(G_last)
};

// Fills them for the `live` first tokens (at least one) from token t0 on: the others have beta 0 and decay 1. By the
// first wavefront; the caller's barrier follows.
template <int C> __device__ __forceinline__ void load_gates(const DeltaArgs &a, int p, int h, int t0, int live, Gates<C> &s) {
    if (threadIdx.x >= 64) return;
    const int t = threadIdx.x;
    const int64_t at = (int64_t(p) * a.T + t0 + t) * a.Hv + h;
    const bool in = t < C && t < live;
    float g = in ? a.g[at] : 0.0f;
    if (g < -1e4f) g = -1e4f;
    double G = double(g);
#pragma unroll
    for (int d = 1; d < C; d <<= 1) {
        const double o = __shfl_up(G, d, 64);
        if (t >= d) G += o;
    }
    const double GL = __shfl(G, C - 1, 64);
    if (t < C) {
        s.G[t] = G;
        s.beta[t] = in ? a.beta[at] : 0.0f;
        s.eG[t] = expf(float(G));
        s.eL[t] = expf(float(GL - G));
    }
    if (t == 0) s.last = expf(float(GL));
}

// Rows of `width` elements of `live` tokens into tile [C][LD] (columns up to KP), zeros elsewhere.
template <typename T, int C, int KP, int LD>
__device__ __forceinline__ void load_tile(const Rows &r, int p, int h, int t0, int live, int width, float *m) {
    const T *src = static_cast<const T *>(r.data) + p * r.sp + h * r.sh + t0 * r.st;
    for (int i = threadIdx.x; i < C * KP; i += blockDim.x) {
        const int t = i / KP, c = i % KP;
        m[t * LD + c] = t < live && c < width ? to_f32(src[t * r.st + c]) : 0.0f;
    }
}
template <int R, int N, int LD> __device__ __forceinline__ void load_mat(const float *src, float *m) {
    for (int i = threadIdx.x; i < R * N / 4; i += blockDim.x) {
        const int r = i / (N / 4), c = i % (N / 4) * 4;
        *reinterpret_cast<dt4 *>(m + r * LD + c) = *reinterpret_cast<const dt4 *>(src + r * N + c);
    }
}

// The beta that the backward computes U with: its U / beta is the write error for every beta.
__device__ __forceinline__ float delta_beta_safe(float b) { return fabsf(b) < 1e-20f ? 1e-20f : b; }

// Tokens of a chunk and padded head_dim of a shape.
inline int delta_kp(int K) { return K <= 64 ? 64 : K <= 128 ? 128 : 256; }
inline int delta_chunk(int K) { return K <= 128 ? 64 : 32; }

}  // namespace sdm
