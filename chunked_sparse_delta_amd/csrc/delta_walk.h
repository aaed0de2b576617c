// What the kernels that walk a sequence's chunks share: the chunk's operands in LDS, copied there a
// chunk ahead, and the state in accumulators.
#pragma once

#include "delta_tile.h"

namespace sdm {

constexpr size_t kDeltaMaxLds = 160 * 1024 - 256;

// A wavefront's 1 KB from per-lane addresses to consecutive LDS, without a register between. Written out, since the
// compiler makes any later LDS read wait for its own form of it: Walk::arrive waits for these. (It has no result register,
// and what the compiler waits for by count comes no later for more being on its way.)
__device__ __forceinline__ void copy_to_lds(const void *src, const void *dst) {
    const uint32_t at = uint32_t(reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) const void *)(dst)));
    asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, off"
                 :: "v"(src), "s"(__builtin_amdgcn_readfirstlane(at)) : "memory");
}

// T: the inputs' type; NP: pieces of P; Q: q is wanted too.
template <typename T, int C, int KP, int NP, bool Q> struct Walk {
    static constexpr int NI = kPieces<T>, KB = KP / 32, TB = C / 32;
    static constexpr int kStride = TB * KB * kBlk;              // between the pieces of k (and of q)
    static constexpr int KS = kStride / 1024 / 4;               // kilobytes of a piece of k per wavefront
    static constexpr int MS = (sizeof(ChunkMats<C, NP>) / 1024 + 3) / 4;
    static constexpr int RS = 16 * sizeof(T) / 16;              // 16-byte pieces of a row of v's 16 columns
    static constexpr int VS = C * RS / 64;
    struct Lds {
        unsigned char k[NI][TB][KB][kBlk];
        unsigned char q[Q ? NI : 0][TB][KB][kBlk];
        ChunkMats<C, NP> m;
        T v[4][C][16];
    };
    static constexpr int kBufs = 2 * sizeof(Lds) <= kDeltaMaxLds ? 2 : 1;
    static constexpr size_t kLds = kBufs * sizeof(Lds);
    const bf16 *kp, *qp;
    const T *vp;
    const unsigned char *mats;
    int64_t kplane, qplane, ks, qs, vs;
    int col0, n, Nc;

    // Rows of `val` (v, or what takes its place) head vh; cg: the wavefront's group of 16 columns.
    __device__ Walk(const DeltaArgs &a, const DeltaWs &ws, int p, int h, int hk, int ph, int cg, const Rows &val, int tokens)
        : kp(a.kk.data + p * a.kk.sp + hk * a.kk.sh), qp(a.qq.data + p * a.qq.sp + hk * a.qq.sh),
          vp(static_cast<const T *>(val.data) + p * val.sp + h * val.sh),
          mats(ws.mats + int64_t(ph) * ws.Nt * sizeof(ChunkMats<C, NP>)), kplane(a.kk.plane), qplane(a.qq.plane), ks(a.kk.st),
          qs(a.qq.st), vs(val.st), n(tokens), Nc((tokens + C - 1) / C) {
        // columns past the row's end are read from its last ones: nothing that they reach is kept
        const int piece = int(threadIdx.x) % RS * (16 / int(sizeof(T)));
        col0 = min(cg * 16 + piece, val.width - 16 / int(sizeof(T)));
    }

    // Chunk c's operands, on their way to `s`. Rows past the last valid token are that token's: finite where it is, and met by
    // gates of 0 everywhere.
    __device__ __forceinline__ void load(Lds &s, int c) const {
        const int t0 = c * C, top = n - 1 - t0, lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
        const bf16 *kc = kp + t0 * ks, *qc = qp + t0 * qs;
        const T *vc = vp + t0 * vs;
#pragma unroll
        for (int i = 0; i < KS; ++i) {
            const int slot = i * 256 + wv * 64 + lane, blk = slot / 128, r = slot % 128 / 4;
            const int row = min(blk / KB * 32 + r, top), d = blk % KB * 32 + ((slot ^ (r >> 3)) & 3) * 8;
            unsigned char *dk = &s.k[0][0][0][0] + (i * 256 + wv * 64) * 16;
#pragma unroll
            for (int e = 0; e < NI; ++e) copy_to_lds(kc + e * kplane + (row * int(ks) + d), dk + e * kStride);
            if constexpr (Q) {
                unsigned char *dq = &s.q[0][0][0][0] + (i * 256 + wv * 64) * 16;
#pragma unroll
                for (int e = 0; e < NI; ++e) copy_to_lds(qc + e * qplane + (row * int(qs) + d), dq + e * kStride);
            }
        }
#pragma unroll
        for (int i = 0; i < VS; ++i)
            copy_to_lds(vc + (min((lane + 64 * i) / RS, top) * int(vs) + col0), reinterpret_cast<unsigned char *>(&s.v[wv][0][0]) + i * 1024);
        const unsigned char *src = mats + int64_t(c) * sizeof(ChunkMats<C, NP>) + lane * 16;
#pragma unroll
        for (int i = 0; i < MS; ++i) {
            const int kb = wv + 4 * i;
            if (kb < int(sizeof(ChunkMats<C, NP>) / 1024)) copy_to_lds(src + kb * 1024, reinterpret_cast<unsigned char *>(&s.m) + kb * 1024);
        }
    }
    __device__ __forceinline__ bool has(int c) const { return c >= 0 && c < Nc; }
    static __device__ __forceinline__ void arrive() {   // everything on its way is there, for every wavefront
        __builtin_amdgcn_s_waitcnt(0x0F70);   // vmcnt(0)
        __syncthreads();
    }
    // LDS holds the current chunk's operands. With two buffers the next chunk's are on their way to the other one meanwhile.
    __device__ __forceinline__ void begin(Lds *bufs, int c) const {
        if (!has(c)) return;
        load(bufs[0], c);
        arrive();
    }
    // At the start of the i-th chunk taken: `next` is the chunk after it.
    __device__ __forceinline__ void ahead(Lds *bufs, int i, int next) const {
        if constexpr (kBufs == 2)
            if (has(next)) load(bufs[(i + 1) & 1], next);
    }
    // At its end.
    __device__ __forceinline__ void turn(Lds *bufs, int next) const {
        if constexpr (kBufs == 1) {
            __syncthreads();
            if (has(next)) load(bufs[0], next);
        }
        arrive();
    }
    __device__ __forceinline__ dt4 value(const Lds &s, int tb, int e) const {
        const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6, g = lane >> 4, i = lane & 15, t = tb * 32 + g * 8 + e * 4;
        dt4 x;
        if constexpr (sizeof(T) == 2) {
            const ds4 y = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                (__attribute__((address_space(3))) ds4 *)(&s.v[wv][t + (i >> 2)][(i & 3) * 4]));
#pragma unroll
            for (int j = 0; j < 4; ++j) x[j] = __uint_as_float(uint32_t(uint16_t(y[j])) << 16);
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) x[j] = s.v[wv][t + j][i];
        }
        return x;
    }
};

// Column `lane & 15` of the wavefront's 16 columns of a chunk's rows t0.. of `out` (token stride os), of which `live` are there.
template <typename T, int TB>
__device__ __forceinline__ void put_columns(T *out, int64_t os, int live, bool in, const dt4 (&y)[TB][2]) {
    const int lg = (threadIdx.x & 63) >> 4;
    if (!in) return;
#pragma unroll
    for (int tb = 0; tb < TB; ++tb)
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int t = tb * 32 + lg * 8 + e * 4 + i;
                if (t < live) out[t * os] = from_f32<T>(y[tb][e][i]);
            }
}
// Four neighbours of an output row of which `left` are inside it.
__device__ __forceinline__ void put_four(bf16 *p, int left, dt4 x) {
    typedef uint32_t raw __attribute__((ext_vector_type(2), aligned(2)));
    const raw w = {f32x2_to_bf16x2(x[0], x[1]), f32x2_to_bf16x2(x[2], x[3])};
    if (left >= 4) *reinterpret_cast<raw *>(p) = w;
    else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (j < left) p[j].bits = uint16_t(w[j / 2] >> (j & 1 ? 16 : 0));
    }
}
__device__ __forceinline__ void put_four(float *p, int left, dt4 x) {
    typedef float raw __attribute__((ext_vector_type(4), aligned(4)));
    if (left >= 4) *reinterpret_cast<raw *>(p) = raw{x[0], x[1], x[2], x[3]};
    else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (j < left) p[j] = x[j];
    }
}

// The wavefront's 16 columns of a [K, V] state, zeros past its ends and where there is none.
template <int KB> __device__ __forceinline__ void load_state(dt4 (&S)[KB][2], const float *state, int ph, int K, int V, int col) {
    const int lg = (threadIdx.x & 63) >> 4;
    const float *src = state + int64_t(ph) * K * V + col;
#pragma unroll
    for (int kb = 0; kb < KB; ++kb)
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int row = kb * 32 + lg * 8 + e * 4 + r;
                S[kb][e][r] = state && col < V && row < K ? src[int64_t(row) * V] : 0.0f;
            }
}
template <int KB> __device__ __forceinline__ void store_state(const dt4 (&S)[KB][2], float *state, int ph, int K, int V, int col) {
    if (!state || col >= V) return;
    const int lg = (threadIdx.x & 63) >> 4;
    float *dst = state + int64_t(ph) * K * V + col;
#pragma unroll
    for (int kb = 0; kb < KB; ++kb)
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int row = kb * 32 + lg * 8 + e * 4 + r;
                if (row < K) dst[int64_t(row) * V] = S[kb][e][r];
            }
}
// B row blocks of the wavefront's column group in the workspace's layout (see DeltaWs).
template <int B> __device__ __forceinline__ float *blocks_at(float *m, int64_t n, int VG, int cg) {
    return m + ((n * VG + cg) * B * 64 + (threadIdx.x & 63)) * 8;
}
template <int B> __device__ __forceinline__ void save_blocks(float *m, int64_t n, int VG, int cg, const dt4 (&x)[B][2]) {
    if (cg >= VG) return;
    float *p = blocks_at<B>(m, n, VG, cg);
#pragma unroll
    for (int b = 0; b < B; ++b)
#pragma unroll
        for (int e = 0; e < 2; ++e) *reinterpret_cast<dt4 *>(p + b * 512 + e * 4) = x[b][e];
}

}  // namespace sdm
