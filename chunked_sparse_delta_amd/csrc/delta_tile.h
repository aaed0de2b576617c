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

// A workgroup barrier that orders LDS only: nothing waits for loads or stores of memory on their way.
__device__ __forceinline__ void lds_barrier() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

// LDS accesses keep their side of this point (other instructions may cross): the operands of the
// products to come are read before the products at hand, whose 16 cycles each hide the way to LDS.
__device__ __forceinline__ void lds_point() { __builtin_amdgcn_sched_barrier(0x7F); }

// x less its first 8 bits, for both halves of a pair `w` of such cuts, as one instruction each: w . (-1, 0) + x and
// w . (0, -1) + x, which are exact. (The constants stay in registers: as an inline constant -1.0 the second one
// would be taken for a pair of another type.)
struct CutRest {
    uint32_t lo, hi;
    __device__ __forceinline__ CutRest() {
        asm("s_mov_b32 %0, 0xbf80" : "=s"(lo));
        asm("s_mov_b32 %0, 0xbf800000" : "=s"(hi));
    }
    __device__ __forceinline__ float operator()(uint32_t w, uint32_t which, float x) const {
        typedef __bf16 b2 __attribute__((ext_vector_type(2)));
        return __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(b2, w), __builtin_bit_cast(b2, which), x, false);
    }
};

// Eight float32 values as N pieces.
template <int N> __device__ __forceinline__ Frag<N> split(dt4 a, dt4 b) {
    Frag<N> f;
    float x[8] = {a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
    const CutRest rest;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        du4 w;
        if (i == N - 1) {   // the last piece is rounded
#pragma unroll
            for (int j = 0; j < 4; ++j) w[j] = f32x2_to_bf16x2(x[2 * j], x[2 * j + 1]);
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                w[j] = __builtin_amdgcn_perm(__float_as_uint(x[2 * j + 1]), __float_as_uint(x[2 * j]), 0x07060302);   // the high halves
                x[2 * j] = rest(w[j], rest.lo, x[2 * j]);
                x[2 * j + 1] = rest(w[j], rest.hi, x[2 * j + 1]);
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

__device__ __forceinline__ dt4 mma1(db8 a, db8 b, dt4 acc) { return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, acc, 0, 0, 0); }
// The same products, the smallest first, each for all the caller's blocks in turn (neighbouring instructions then do not
// wait for each other).
template <int ORD, int NA, int NB, typename F> __device__ __forceinline__ void each_product(F f) {
#pragma unroll
    for (int i = NA - 1; i >= 0; --i)
#pragma unroll
        for (int j = NB - 1; j >= 0; --j)
            if (i + j < ORD) f(i, j);
}

// The lane's number, as a value of its own: addresses made from it stay in the part of the program that makes it. (Where a loop
// reads many blocks, all their addresses are worth keeping to the compiler, in registers that it then spills.)
__device__ __forceinline__ int fresh_lane() {
    int lane = threadIdx.x & 63;
    asm volatile("" : "+v"(lane));
    return lane;
}

// A operand: the rows of tile a of the block at `blk`; N pieces `stride` bytes apart.
template <int N> __device__ __forceinline__ Frag<N> read_rows(const unsigned char *blk, int stride, int a, int lane = threadIdx.x & 63) {
    const int at = block_at(block_row(lane & 15, a), lane >> 4);
    Frag<N> f;
#pragma unroll
    for (int i = 0; i < N; ++i) f.p[i] = *reinterpret_cast<const db8 *>(blk + i * stride + at);
    return f;
}
// A operand of the block's transpose: columns block_row(., a) as rows, its rows as depth. Each 16 lanes
// read 4 rows x 16 columns of 16-bit elements, transposed on the way.
template <int N> __device__ __forceinline__ Frag<N> read_cols(const unsigned char *blk, int stride, int a, int lane = threadIdx.x & 63) {
    const int g = lane >> 4, i = lane & 15;
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

// Eight elements of a row of q or k.
template <int N> __device__ __forceinline__ Frag<N> load_keys(const bf16 *p, int64_t plane) {
    Frag<N> f;
#pragma unroll
    for (int i = 0; i < N; ++i) f.p[i] = *reinterpret_cast<const db8 *>(p + i * plane);
    return f;
}
template <int N> __device__ __forceinline__ void clear(Frag<N> &f) {
#pragma unroll
    for (int i = 0; i < N; ++i) f.p[i] = __builtin_bit_cast(db8, du4{0, 0, 0, 0});
}

// Pieces of an input element.
template <typename T> constexpr int kPieces = sizeof(T) == 2 ? 1 : 3;
// Tokens of a chunk where head_dim is at most 128 (32 above it): two chunks' operands in LDS at once.
template <typename T> constexpr int kChunk = sizeof(T) == 2 ? 64 : 32;

// The beta that the backward computes U with: its U / beta is the write error for every beta.
__device__ __forceinline__ float delta_beta_safe(float b) { return fabsf(b) < 1e-20f ? 1e-20f : b; }

// The running sum of a chunk's log-decays, over log 2 (so that exp2_of of a difference is the decay between two tokens), by one
// wavefront: a token per lane (g: its log-decay, 0 for padding). In 64 bits: differences are as exact as the log-decays themselves however large the sum
// grew. A log-decay below -1e4 (-inf among them: it clears the state) counts as -1e4, whose exponential is 0 too.
template <int C> __device__ __forceinline__ double chunk_G(float g) {
    const int lane = threadIdx.x & 63;
    if (g < -1e4f) g = -1e4f;
    double G = double(g) * 1.4426950408889634;
#pragma unroll
    for (int d = 1; d < C; d <<= 1) {
        const double o = __shfl_up(G, d, 64);
        if (lane >= d) G += o;
    }
    return G;
}
__device__ __forceinline__ float exp2_of(double x) { return __builtin_amdgcn_exp2f(float(x)); }

// A chunk's gates, as delta_prep_kernel leaves them: beta, exp(G), exp(G_last - G) of every token (0 for padding tokens,
// whose rows the kernels then need not clear), exp(G_last).
template <int C> struct Gates {
    float beta[C], eG[C], eL[C], last, pad[255 - 3 * C];
};

// Slice and head of a block. The slices of a head, and the heads that share a key head, read the same q and k: they go to one
// XCD (blocks are dealt to the eight in turn), where the key heads divide among them.
struct BlockAt {
    int slice, ph;
    __device__ __forceinline__ BlockAt(int b, int slices, int heads, int group) {
        const bool even = heads / group % kXcds == 0;
        const int i = even ? b / kXcds : b, head = i / slices;
        slice = i % slices;
        ph = even ? (head / group * kXcds + b % kXcds) * group + head % group : head;
    }
};

// What the prep kernel leaves of a chunk for the kernels that walk it: the lower 32 x 32 blocks of X and P, rows of 32, and the
// gates.
template <int C> constexpr int kTri = C == 64 ? 3 : 1;     // blocks (0, 0), (1, 0), (1, 1)
template <int C> struct ChunkMem {
    float X[kTri<C>][32][32], P[kTri<C>][32][32];
    Gates<C> g;
};
// ... and as these have it in LDS: blocks in pieces.
template <int C> struct ChunkMats {
    unsigned char X[3][kTri<C>][kBlk];
    unsigned char P[3][kTri<C>][kBlk];
    Gates<C> g;
};
}  // namespace sdm
