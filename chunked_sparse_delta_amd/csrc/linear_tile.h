// What linear attention's kernels share: rows brought from memory to LDS blocks, and a segment's gates.
#pragma once

#include <type_traits>

#include "linear.h"

namespace sdm {

// Eight neighbours of a row, as loaded.
template <typename T> struct Eight;
template <> struct Eight<bf16> {
    du4 w;
};
template <> struct Eight<float> {
    dt4 a, b;
};
__device__ __forceinline__ void eight_load(const bf16 *p, Eight<bf16> &o) {
    typedef uint32_t raw __attribute__((ext_vector_type(4), aligned(2)));
    o.w = *reinterpret_cast<const raw *>(p);
}
__device__ __forceinline__ void eight_load(const float *p, Eight<float> &o) {
    typedef float raw __attribute__((ext_vector_type(4), aligned(4)));
    o.a = *reinterpret_cast<const raw *>(p);
    o.b = *reinterpret_cast<const raw *>(p + 4);
}
__device__ __forceinline__ void eight_part(const bf16 *p, int left, Eight<bf16> &o) {
#pragma unroll
    for (int j = 0; j < 4; ++j)
        o.w[j] = (2 * j < left ? uint32_t(p[2 * j].bits) : 0u) | (2 * j + 1 < left ? uint32_t(p[2 * j + 1].bits) << 16 : 0u);
}
__device__ __forceinline__ void eight_part(const float *p, int left, Eight<float> &o) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        o.a[j] = j < left ? p[j] : 0.0f;
        o.b[j] = 4 + j < left ? p[4 + j] : 0.0f;
    }
}
__device__ __forceinline__ void eight_clear(Eight<bf16> &o) { o.w = du4{}; }
__device__ __forceinline__ void eight_clear(Eight<float> &o) { o.a = o.b = dt4{}; }
// The elements p[0 .. 8) of which `left` are there (zeros after them; <= 0: none, and p is not read).
template <typename T> __device__ __forceinline__ Eight<T> eight(const T *p, int left) {
    Eight<T> o;
    if (left >= 8) eight_load(p, o);
    else if (left > 0) eight_part(p, left, o);
    else eight_clear(o);
    return o;
}
__device__ __forceinline__ void eight_values(const Eight<bf16> &x, dt4 &a, dt4 &b) {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        a[2 * j] = __uint_as_float(x.w[j] << 16);
        a[2 * j + 1] = __uint_as_float(x.w[j] & 0xFFFF0000u);
        b[2 * j] = __uint_as_float(x.w[2 + j] << 16);
        b[2 * j + 1] = __uint_as_float(x.w[2 + j] & 0xFFFF0000u);
    }
}
__device__ __forceinline__ void eight_values(const Eight<float> &x, dt4 &a, dt4 &b) {
    a = x.a;
    b = x.b;
}
__device__ __forceinline__ Frag<1> pieces(const Eight<bf16> &x) { return {{__builtin_bit_cast(db8, x.w)}}; }
__device__ __forceinline__ Frag<3> pieces(const Eight<float> &x) { return split<3>(x.a, x.b); }

// a and b, rounded, to p[0 .. 8) of which `left` are there.
__device__ __forceinline__ void eight_store(bf16 *p, int left, dt4 a, dt4 b) {
    typedef uint32_t raw __attribute__((ext_vector_type(4), aligned(2)));
    const raw w = {f32x2_to_bf16x2(a[0], a[1]), f32x2_to_bf16x2(a[2], a[3]), f32x2_to_bf16x2(b[0], b[1]), f32x2_to_bf16x2(b[2], b[3])};
    if (left >= 8) *reinterpret_cast<raw *>(p) = w;
    else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (j < left) p[j].bits = uint16_t(w[j / 2] >> (j & 1 ? 16 : 0));
    }
}
__device__ __forceinline__ void eight_store(float *p, int left, dt4 a, dt4 b) {
    typedef float raw __attribute__((ext_vector_type(4), aligned(4)));
    if (left >= 8) {
        *reinterpret_cast<raw *>(p) = raw{a[0], a[1], a[2], a[3]};
        *reinterpret_cast<raw *>(p + 4) = raw{b[0], b[1], b[2], b[3]};
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (j < left) p[j] = j < 4 ? a[j & 3] : b[j & 3];
    }
}

// A tile of ROWS tokens (a multiple of 32) and W columns from column c0 of `width`, brought by the 256 threads of a workgroup and
// kept in LDS as [piece][32 rows][32 columns] blocks. Rows outside [0, live) and columns past the width are zeros.
template <typename T, int ROWS, int W> struct Tile {
    static constexpr int N = ROWS * W / 2048, WB = W / 32, kPlane = ROWS / 32 * WB * kBlk;   // eights of a thread
    static_assert(ROWS * W % 2048 == 0, "whole eights for every thread");
    Eight<T> x[N];
    // rows: of the tile's first token; st: a token's stride
    __device__ __forceinline__ void load(const T *rows, int64_t st, int live, int c0, int width) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int slot = int(threadIdx.x) + 256 * i, blk = slot / 128, r = blk / WB * 32 + slot % 128 / 4;
            const int c = c0 + blk % WB * 32 + slot % 4 * 8;
            x[i] = eight(rows + r * st + c, r < live ? width - c : 0);
        }
    }
    __device__ __forceinline__ void store(unsigned char *lds) const {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int slot = int(threadIdx.x) + 256 * i, at = slot / 128 * kBlk + block_at(slot % 128 / 4, slot % 4);
            const auto f = pieces(x[i]);
#pragma unroll
            for (int n = 0; n < kPieces<T>; ++n) *reinterpret_cast<db8 *>(lds + n * kPlane + at) = f.p[n];
        }
    }
    // ... each row times its weight, in three pieces.
    __device__ __forceinline__ void store_weighted(unsigned char *lds, const float *w) const {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int slot = int(threadIdx.x) + 256 * i, blk = slot / 128, at = blk * kBlk + block_at(slot % 128 / 4, slot % 4);
            const float f = w[blk / WB * 32 + slot % 128 / 4];
            dt4 a, b;
            eight_values(x[i], a, b);
            const Frag<3> s = split<3>(a * f, b * f);
#pragma unroll
            for (int n = 0; n < 3; ++n) *reinterpret_cast<db8 *>(lds + n * kPlane + at) = s.p[n];
        }
    }
};

// The running sums of a segment's log-decays over log 2 (chunk_G) of its `live` <= 256 tokens from row `s0` on, a token per thread;
// tokens after them repeat the last sum. Returns the thread's own sum; all of them are in G after the next barrier.
__device__ __forceinline__ void segment_gates(const LinGates &gates, int p, int h, int s0, int live, double *G, double *total) {
    const int tid = threadIdx.x, wv = tid >> 6, lane = tid & 63;
    const float g = tid < live ? gates.g[p * gates.sp + (s0 + tid) * gates.st + h] : 0.0f;
    double x = chunk_G<64>(g);
    if (lane == 63) total[wv] = x;
    lds_barrier();
    for (int w = 0; w < wv; ++w) x += total[w];
    G[tid] = x;
}

// A or B operand of the block's transpose with its columns in order: columns 16 a .. 16 a + 15 as rows, its rows as depth.
template <int N> __device__ __forceinline__ Frag<N> read_cols_in_order(const unsigned char *blk, int stride, int a) {
    const int lane = threadIdx.x & 63, g = lane >> 4, i = lane & 15;
    Frag<N> f;
#pragma unroll
    for (int n = 0; n < N; ++n) {
        ds4 h[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const unsigned char *p = blk + n * stride + block_at(g * 8 + e * 4 + (i >> 2), 2 * a + (i >> 1 & 1)) + (i & 1) * 8;
            h[e] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) ds4 *)(p));
        }
        f.p[n] = __builtin_bit_cast(db8, __builtin_shufflevector(h[0], h[1], 0, 1, 2, 3, 4, 5, 6, 7));
    }
    return f;
}

__device__ __forceinline__ int lin_valid(const int32_t *valid, int p, int T) { return valid ? max(0, min(valid[p], T)) : T; }

}  // namespace sdm
