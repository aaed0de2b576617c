// Tiles of the chunked gated delta rule: 32-deep products on v_mfma_f32_16x16x32_bf16, with
// float32 quantities as sums of bfloat16 pieces.
//
// Pieces. A float32 x is hi + mid + lo, each piece 8 bits of it: cutting x after its first 8
// bits, and what is left after the next 8, leaves nothing out. A product of pieces is exact and is
// accumulated in float32; of x y the products of pieces i and j with i + j <= 2 keep it to 2^-23.
// Three pieces against a bfloat16 operand are 3 instructions of 16 cycles for a 16 x 16 x 32
// block, two split operands 6; the float32 instruction takes 256 cycles for it.
//
// Layout. The instruction wants in lane l, with m = l & 15 and g = l >> 4, row m of A (column m
// of B) at depths 8 g + j, j = 0..7; its result holds column m of rows 4 g + r, r = 0..3. The rows of
// a 32-row block are dealt to two result tiles a = 0, 1 so that row 8 g + 4 a + r lands in element r of
// tile a: the eight values a lane then holds are rows 8 g .. 8 g + 7, a B operand as they stand. (So
// row m of tile a is row block_row(m, a), which only the A operand's address has to know.)
//
// Matrices in LDS (and in the workspace) are 32 x 32 blocks of 2 KB: 32 rows of four 16-byte
// chunks, chunk c of row r at place c ^ ((r >> 3) & 3), so that the sixteen rows of an operand read
// (16 bytes per lane) meet all banks once.
#pragma once

#include "delta.h"

namespace sdm {

typedef float dt4 __attribute__((ext_vector_type(4)));
typedef uint32_t du4 __attribute__((ext_vector_type(4)));
typedef __bf16 db8 __attribute__((ext_vector_type(8)));
typedef short ds4 __attribute__((ext_vector_type(4)));

constexpr int kBlk = 2048;    // bytes of a 32 x 32 block

__device__ __forceinline__ int block_row(int m, int a) { return (m >> 2) * 8 + a * 4 + (m & 3); }
// Byte offset of chunk c of row r in a block.
__device__ __forceinline__ int block_at(int r, int c) { return r * 64 + ((c ^ ((r >> 3) & 3)) << 4); }

template <int N> struct Frag {
    db8 p[N];
};

// Eight float32 values as N pieces.
template <int N> __device__ __forceinline__ Frag<N> split(dt4 a, dt4 b) {
    Frag<N> f;
    float x[8] = {a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
#pragma unroll
    for (int i = 0; i < N; ++i) {
        du4 w;
        if (i == N - 1) {   // the last piece is rounded
#pragma unroll
            for (int j = 0; j < 4; ++j) w[j] = f32x2_to_bf16x2(x[2 * j], x[2 * j + 1]);
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const uint32_t u = __float_as_uint(x[2 * j]), v = __float_as_uint(x[2 * j + 1]);
                w[j] = __builtin_amdgcn_perm(v, u, 0x07060302);   // the high halves, u's low
                x[2 * j] -= __uint_as_float(u & 0xFFFF0000u);
                x[2 * j + 1] -= __uint_as_float(v & 0xFFFF0000u);
            }
        }
        f.p[i] = __builtin_bit_cast(db8, w);
    }
    return f;
}

// acc += A B over the products of pieces whose indexes sum to less than ORD.
template <int ORD, int NA, int NB> __device__ __forceinline__ dt4 mma(const Frag<NA> &a, const Frag<NB> &b, dt4 acc) {
#pragma unroll
    for (int i = NA - 1; i >= 0; --i)
#pragma unroll
        for (int j = NB - 1; j >= 0; --j)
            if (i + j < ORD) acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a.p[i], b.p[j], acc, 0, 0, 0);
    return acc;
}

// A operand: the rows of tile a of the block at `blk`; N pieces `stride` bytes apart.
template <int N> __device__ __forceinline__ Frag<N> read_rows(const unsigned char *blk, int stride, int a) {
    const int lane = threadIdx.x & 63, at = block_at(block_row(lane & 15, a), lane >> 4);
    Frag<N> f;
#pragma unroll
    for (int i = 0; i < N; ++i) f.p[i] = *reinterpret_cast<const db8 *>(blk + i * stride + at);
    return f;
}
// A operand of the block's transpose: columns block_row(., a) as rows, its rows as depth. Each 16 lanes
// read 4 rows x 16 columns of 16-bit elements, transposed on the way.
template <int N> __device__ __forceinline__ Frag<N> read_cols(const unsigned char *blk, int stride, int a) {
    const int lane = threadIdx.x & 63, g = lane >> 4, i = lane & 15;
    Frag<N> f;
#pragma unroll
    for (int n = 0; n < N; ++n) {
        ds4 h[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const unsigned char *p = blk + n * stride + block_at(g * 8 + e * 4 + (i >> 2), i & 3) + a * 8;
            h[e] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) ds4 *)(p));
        }
        f.p[n] = __builtin_bit_cast(db8, __builtin_shufflevector(h[0], h[1], 0, 1, 2, 3, 4, 5, 6, 7));
    }
    return f;
}

// Eight elements of a row of `width` from column c on, zeros past its end, as one 16-byte load
// (two for float32) at any element address: where the row ends inside it, the load starts at the row's last eight
// elements and is shifted. The caller gives in = false for rows that are not there (p then has to be readable all the
// same). Only rows narrower than eight elements are read one by one.
template <typename T> struct Eight;
template <> struct Eight<bf16> {
    du4 x;
    __device__ __forceinline__ void load(const bf16 *p, int c, int width) {
        typedef uint32_t raw __attribute__((ext_vector_type(4), aligned(2)));
        if (width >= 8) {
            const raw y = *reinterpret_cast<const raw *>(p + min(c, width - 8));
            x = du4{y[0], y[1], y[2], y[3]};
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const uint32_t lo = c + 2 * j < width ? p[c + 2 * j].bits : 0u;
                const uint32_t hi = c + 2 * j + 1 < width ? p[c + 2 * j + 1].bits : 0u;
                x[j] = lo | hi << 16;
            }
        }
    }
    // After the load: the shift, and zeros where there is nothing.
    __device__ __forceinline__ void fix(int c, int width, bool in) {
        if (width & 7) {
            if (width >= 8) {
                const int s = max(c - (width - 8), 0);       // elements to shift out
                uint64_t lo = uint64_t(x[1]) << 32 | x[0], hi = uint64_t(x[3]) << 32 | x[2];
                if (s >= 4) {
                    lo = hi;
                    hi = 0;
                }
                const int b = (s & 3) * 16;
                if (b) {
                    lo = lo >> b | hi << (64 - b);
                    hi >>= b;
                }
                x = du4{uint32_t(lo), uint32_t(lo >> 32), uint32_t(hi), uint32_t(hi >> 32)};
            }
        }
        if (!in || c >= width) x = du4{0, 0, 0, 0};
    }
    __device__ __forceinline__ Frag<1> pieces() const { return {{__builtin_bit_cast(db8, x)}}; }
    __device__ __forceinline__ void floats(dt4 &a, dt4 &b) const {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float l = __uint_as_float(x[j] << 16), h = __uint_as_float(x[j] & 0xFFFF0000u);
            if (j < 2) {
                a[2 * j] = l;
                a[2 * j + 1] = h;
            } else {
                b[2 * j - 4] = l;
                b[2 * j - 3] = h;
            }
        }
    }
};
template <> struct Eight<float> {
    dt4 a, b;
    __device__ __forceinline__ void load(const float *p, int c, int width) {
        typedef float raw __attribute__((ext_vector_type(4), aligned(4)));
        if (width >= 8) {
            const float *s = p + min(c, width - 8);
            const raw y = *reinterpret_cast<const raw *>(s), z = *reinterpret_cast<const raw *>(s + 4);
            a = dt4{y[0], y[1], y[2], y[3]};
            b = dt4{z[0], z[1], z[2], z[3]};
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float v = c + j < width ? p[c + j] : 0.0f;
                if (j < 4) a[j] = v;
                else b[j - 4] = v;
            }
        }
    }
    __device__ __forceinline__ void fix(int c, int width, bool in) {
        if ((width & 7) && width >= 8) {
            int s = max(c - (width - 8), 0);
#pragma unroll
            for (int bit = 4; bit; bit >>= 1)
                if (s & bit) {
                    float v[8] = {a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const float y = j + bit < 8 ? v[j + bit] : 0.0f;
                        if (j < 4) a[j] = y;
                        else b[j - 4] = y;
                    }
                }
        }
        if (!in || c >= width) a = b = dt4{0.0f, 0.0f, 0.0f, 0.0f};
    }
    __device__ __forceinline__ Frag<3> pieces() const { return split<3>(a, b); }
    __device__ __forceinline__ void floats(dt4 &x, dt4 &y) const {
        x = a;
        y = b;
    }
};
// Eight neighbours of an output row of which `left` are inside it: one 16-byte store (two for float32) at any element
// address where all are.
__device__ __forceinline__ void put_eight(bf16 *p, int left, dt4 a, dt4 b) {
    typedef uint32_t raw __attribute__((ext_vector_type(4), aligned(2)));
    const raw x = {f32x2_to_bf16x2(a[0], a[1]), f32x2_to_bf16x2(a[2], a[3]), f32x2_to_bf16x2(b[0], b[1]), f32x2_to_bf16x2(b[2], b[3])};
    if (left >= 8) *reinterpret_cast<raw *>(p) = x;
    else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (j < left) p[j].bits = uint16_t(x[j / 2] >> (j & 1 ? 16 : 0));
    }
}
__device__ __forceinline__ void put_eight(float *p, int left, dt4 a, dt4 b) {
    typedef float raw __attribute__((ext_vector_type(4), aligned(4)));
    if (left >= 8) {
        *reinterpret_cast<raw *>(p) = raw{a[0], a[1], a[2], a[3]};
        *reinterpret_cast<raw *>(p + 4) = raw{b[0], b[1], b[2], b[3]};
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (j < left) p[j] = j < 4 ? a[j] : b[j - 4];
    }
}
// Pieces of an input element.
template <typename T> constexpr int kPieces = sizeof(T) == 2 ? 1 : 3;

// The beta that the backward computes U with: its U / beta is the write error for every beta.
__device__ __forceinline__ float delta_beta_safe(float b) { return fabsf(b) < 1e-20f ? 1e-20f : b; }

// A chunk's gates, as delta_prep_kernel leaves them: beta, exp(G), exp(G_last - G) of every token, exp(G_last).
template <int C> struct Gates {
    float beta[C], eG[C], eL[C], last, pad[C == 64 ? 63 : 31];
};

// What the prep kernel leaves of a chunk for the kernels that walk it: the lower 32 x 32
// blocks of X and P in pieces (LDS images), and the gates.
template <int C> constexpr int kTri = C == 64 ? 3 : 1;     // blocks (0, 0), (1, 0), (1, 1)
template <int C, int NP> struct ChunkMats {
    unsigned char X[3][kTri<C>][kBlk];
    unsigned char P[NP][kTri<C>][kBlk];
    Gates<C> g;
};
// Pieces of P: the forward's readings are all that P goes into there, and two are enough for those in bfloat16.
template <typename T> constexpr int kPPieces(bool backward) { return backward || sizeof(T) == 4 ? 3 : 2; }

}  // namespace sdm
