// What linear attention's kernels share: rows brought from memory to LDS blocks, and a segment's gates.
#pragma once

#include <limits.h>

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
// Eight elements from column c on of a row of `width` at p. Past its end there may be anything, until eight_mask. EVEN: the width is a
// multiple of 16 bytes, so that every load is one whole vector and none is behind a branch; else the vector across the end goes by elements.
template <bool EVEN> __device__ __forceinline__ Eight<bf16> eight_load(const bf16 *p, int c, int width) {
    typedef uint32_t raw __attribute__((ext_vector_type(4), aligned(2)));
    Eight<bf16> o;
    const bool whole = EVEN ? c < width : c + 8 <= width;
    if (EVEN || width >= 8) o.w = *reinterpret_cast<const raw *>(p + (whole ? c : 0));
    if (!EVEN && !whole && c < width) {
        uint32_t h[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) h[j] = p[min(c + j, width - 1)].bits;
#pragma unroll
        for (int j = 0; j < 4; ++j) o.w[j] = (c + 2 * j < width ? h[2 * j] : 0u) | (c + 2 * j + 1 < width ? h[2 * j + 1] << 16 : 0u);
    }
    return o;
}
template <bool EVEN> __device__ __forceinline__ Eight<float> eight_load(const float *p, int c, int width) {
    typedef float raw __attribute__((ext_vector_type(4), aligned(4)));
    Eight<float> o;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        const int at = c + 4 * e;
        const bool whole = EVEN ? at < width : at + 4 <= width;
        dt4 x = {};
        if (EVEN || width >= 4) x = *reinterpret_cast<const raw *>(p + (whole ? at : 0));
        if (!EVEN && !whole && at < width) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float h = p[min(at + j, width - 1)];
                x[j] = at + j < width ? h : 0.0f;
            }
        }
        (e ? o.b : o.a) = x;
    }
    return o;
}
// Zeros past the row's end and, where the row is not `live`, in its place. (Apart from the load, since it waits for it.)
__device__ __forceinline__ void eight_mask(Eight<bf16> &o, int c, int width, bool live) {
    const bool in = live && c < width;
#pragma unroll
    for (int j = 0; j < 4; ++j) o.w[j] = in ? o.w[j] : 0u;
}
__device__ __forceinline__ void eight_mask(Eight<float> &o, int c, int width, bool live) {
    const bool in = live && c < width, more = live && c + 4 < width;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        o.a[j] = in ? o.a[j] : 0.0f;
        o.b[j] = more ? o.b[j] : 0.0f;
    }
}
__device__ __forceinline__ void eight_negate(Eight<bf16> &o) { o.w ^= 0x80008000u; }
__device__ __forceinline__ void eight_negate(Eight<float> &o) {
    o.a = -o.a;
    o.b = -o.b;
}
template <bool EVEN, typename T> __device__ __forceinline__ Eight<T> eight(const T *p, int c, int width, bool live) {
    Eight<T> o = eight_load<EVEN>(p, c, width);
    eight_mask(o, c, width, live);
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
// NaN where an infinity or NaN is among the eight, else 0: a sum of them times 0.
__device__ __forceinline__ float eight_seen(const Eight<bf16> &x) {
    float seen = 0.0f;
    typedef __bf16 b2 __attribute__((ext_vector_type(2)));
#pragma unroll
    for (int j = 0; j < 4; ++j) seen = __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(b2, uint32_t(x.w[j])), b2{}, seen, false);
    return seen;
}
__device__ __forceinline__ float eight_seen(const Eight<float> &x) {
    float seen = 0.0f;
#pragma unroll
    for (int j = 0; j < 4; ++j) seen = fmaf(x.b[j], 0.0f, fmaf(x.a[j], 0.0f, seen));
    return seen;
}
// Infinities and NaN to zeros, f(j) for each of them.
template <typename F> __device__ __forceinline__ void eight_sift(Eight<bf16> &x, F f) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const uint32_t bits = 0x7F80u << (j & 1 ? 16 : 0), all = j & 1 ? 0xFFFF0000u : 0xFFFFu;
        if ((x.w[j / 2] & bits) == bits) {
            x.w[j / 2] &= ~all;
            f(j);
        }
    }
}
template <typename F> __device__ __forceinline__ void eight_sift(Eight<float> &x, F f) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        float y = j < 4 ? x.a[j % 4] : x.b[j % 4];
        if ((__float_as_uint(y) & 0x7F800000u) == 0x7F800000u) {
            (j < 4 ? x.a : x.b)[j % 4] = 0.0f;
            f(j);
        }
    }
}
// split<3>, each value on its own: there an infinity or NaN would reach the other value of its pair, here another column.
__device__ __forceinline__ Frag<3> split_apart(dt4 a, dt4 b) {
    Frag<3> f;
    float x[8] = {a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        du4 w;
#pragma unroll
        for (int j = 0; j < 4; ++j) w[j] = __builtin_amdgcn_perm(__float_as_uint(x[2 * j + 1]), __float_as_uint(x[2 * j]), 0x07060302);
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] -= __uint_as_float(__float_as_uint(x[j]) & 0xFFFF0000u);
        f.p[i] = __builtin_bit_cast(db8, w);
    }
    du4 w;
#pragma unroll
    for (int j = 0; j < 4; ++j) w[j] = f32x2_to_bf16x2(x[2 * j], x[2 * j + 1]);
    f.p[2] = __builtin_bit_cast(db8, w);
    return f;
}
__device__ __forceinline__ Frag<1> pieces(const Eight<bf16> &x) { return {{__builtin_bit_cast(db8, x.w)}}; }
__device__ __forceinline__ Frag<3> pieces(const Eight<float> &x) { return split_apart(x.a, x.b); }

// a and b, rounded, to p[0 .. 8) of which `left` are there (EVEN: all, or none, or for float32 four).
template <bool EVEN> __device__ __forceinline__ void eight_store(bf16 *p, int left, dt4 a, dt4 b) {
    typedef uint32_t raw __attribute__((ext_vector_type(4), aligned(2)));
    const raw w = {f32x2_to_bf16x2(a[0], a[1]), f32x2_to_bf16x2(a[2], a[3]), f32x2_to_bf16x2(b[0], b[1]), f32x2_to_bf16x2(b[2], b[3])};
    if (EVEN ? left > 0 : left >= 8) *reinterpret_cast<raw *>(p) = w;
    else if (!EVEN) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (j < left) p[j].bits = uint16_t(w[j / 2] >> (j & 1 ? 16 : 0));
    }
}
template <bool EVEN> __device__ __forceinline__ void eight_store(float *p, int left, dt4 a, dt4 b) {
    typedef float raw __attribute__((ext_vector_type(4), aligned(4)));
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        const dt4 x = e ? b : a;
        if (EVEN ? left > 4 * e : left >= 4 * e + 4) *reinterpret_cast<raw *>(p + 4 * e) = raw{x[0], x[1], x[2], x[3]};
        else if (!EVEN) {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (4 * e + j < left) p[4 * e + j] = x[j];
        }
    }
}

// A tile of ROWS rows (a multiple of 32) and W columns from column c0 of `width`, brought by the 256 threads of a workgroup and
// (tid: a thread's number) kept in LDS as [piece][32 rows][32 columns] blocks. Rows from `live` >= 1 on and columns past the width are zeros.
template <typename T, int ROWS, int W, bool EVEN> struct Tile {
    static constexpr int N = ROWS * W / 2048, WB = W / 32, kPlane = ROWS / 32 * WB * kBlk;   // eights of a thread
    static_assert(ROWS * W % 2048 == 0, "whole eights for every thread");
    Eight<T> x[N];
    int live, c0, width;
    static __device__ __forceinline__ int row_of(int slot) { return slot / 128 / WB * 32 + slot % 128 / 4; }
    static __device__ __forceinline__ int col_of(int slot) { return slot / 128 % WB * 32 + slot % 4 * 8; }
    // rows: the tile's first row; st: a row's stride
    __device__ __forceinline__ void load(const T *rows, int64_t st, int live_, int c0_, int width_, int tid) {
        live = live_;
        c0 = c0_;
        width = width_;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int slot = tid + 256 * i;
            x[i] = eight_load<EVEN>(rows + min(row_of(slot), live - 1) * st, c0 + col_of(slot), width);
        }
    }
    // Infinities and NaN to zeros; `first` (LDS) keeps the least row, counted from `row0`, with one in each of the W columns, behind them in any.
    __device__ __forceinline__ void sift(int tid, int row0, int *first) {
        float seen = 0.0f;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int slot = tid + 256 * i;
            if (live < ROWS || c0 + W > width) eight_mask(x[i], c0 + col_of(slot), width, row_of(slot) < live);
            seen += eight_seen(x[i]);
        }
        if (seen == seen) return;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int slot = tid + 256 * i, row = row0 + row_of(slot), col = col_of(slot);
            eight_sift(x[i], [&](int j) {
                atomicMin(first + col + j, row);
                atomicMin(first + W, row);
            });
        }
    }
    template <int NP, typename F> __device__ __forceinline__ void put(unsigned char *lds, int tid, F cut) {
        const bool whole = live >= ROWS && c0 + W <= width;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int slot = tid + 256 * i, at = slot / 128 * kBlk + block_at(slot % 128 / 4, slot % 4);
            if (!whole) eight_mask(x[i], c0 + col_of(slot), width, row_of(slot) < live);
            const Frag<NP> f = cut(x[i], row_of(slot));
#pragma unroll
            for (int n = 0; n < NP; ++n) *reinterpret_cast<db8 *>(lds + n * kPlane + at) = f.p[n];
        }
    }
    __device__ __forceinline__ void store(unsigned char *lds, int tid) {
        put<kPieces<T>>(lds, tid, [](const Eight<T> &e, int) { return pieces(e); });
    }
    // ... each row times its weight, in three pieces.
    __device__ __forceinline__ void store_weighted(unsigned char *lds, const float *w, int tid) {
        put<3>(lds, tid, [w](const Eight<T> &e, int row) {
            dt4 a, b;
            eight_values(e, a, b);
            return split_apart(a * w[row], b * w[row]);
        });
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
