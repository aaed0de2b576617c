// What the kernels that walk a sequence's chunks share: the chunk's operands in LDS, loaded into
// registers a chunk ahead, and the state in accumulators.
#pragma once

#include "delta_tile.h"

namespace sdm {

constexpr size_t kDeltaMaxLds = 160 * 1024 - 256;

// T: the inputs' type; NP: pieces of P; Q: q is wanted too.
template <typename T, int C, int KP, int NP, bool Q> struct Walk {
    static constexpr int NI = kPieces<T>, KB = KP / 32, TB = C / 32;
    static constexpr int kStride = TB * KB * kBlk;              // between the pieces of k (and of q)
    static constexpr int KS = C * KP / 8 / 256;                 // eights of k per thread
    static constexpr int MS = (sizeof(ChunkMats<C, NP>) / 16 + 255) / 256;
    static constexpr int VS = C * 2 / 64;                       // eights of the wavefront's 16 columns of v per lane
    struct Lds {
        unsigned char k[NI][TB][KB][kBlk];
        unsigned char q[Q ? NI : 0][TB][KB][kBlk];
        ChunkMats<C, NP> m;
        T v[4][C][16];
    };
    const T *kp, *qp, *vp;
    const unsigned char *mats;
    int64_t ks, qs, vs;
    int K, V, col0;
    Eight<T> k[KS], q[Q ? KS : 1], v[VS];
    du4 m[MS];

    // Rows of `val` (v, or what takes its place) head vh; cg: the wavefront's group of 16 columns.
    __device__ Walk(const DeltaArgs &a, const DeltaWs &ws, int p, int h, int hk, int ph, int cg, const Rows &val, int vh)
        : kp(static_cast<const T *>(a.k.data) + p * a.k.sp + hk * a.k.sh),
          qp(static_cast<const T *>(a.q.data) + p * a.q.sp + hk * a.q.sh),
          vp(static_cast<const T *>(val.data) + p * val.sp + vh * val.sh),
          mats(ws.mats + int64_t(ph) * ws.Nt * sizeof(ChunkMats<C, NP>)), ks(a.k.st), qs(a.q.st), vs(val.st), K(a.K), V(a.V),
          col0(cg * 16) {}

    // Rows past the last valid token are read from that token's place and put down as zeros.
    __device__ __forceinline__ void load(int c, int n) {
        const int t0 = c * C, top = n - 1 - t0, tid = threadIdx.x, lane = tid & 63;
#pragma unroll
        for (int i = 0; i < KS; ++i) {
            const int slot = tid + 256 * i, b = slot / 128, row = b / KB * 32 + slot % 128 / 4, d = b % KB * 32 + slot % 4 * 8;
            const int64_t t = t0 + min(row, top);
            k[i].load(kp + t * ks, d, K);
            if constexpr (Q) q[i].load(qp + t * qs, d, K);
        }
#pragma unroll
        for (int i = 0; i < VS; ++i) {
            const int slot = lane + 64 * i;
            v[i].load(vp + (t0 + min(slot / 2, top)) * vs, min(col0 + slot % 2 * 8, V - 1), V);
        }
        const unsigned char *src = mats + int64_t(c) * sizeof(ChunkMats<C, NP>);
#pragma unroll
        for (int i = 0; i < MS; ++i)
            m[i] = *reinterpret_cast<const du4 *>(src + min(tid + 256 * i, int(sizeof(ChunkMats<C, NP>) / 16) - 1) * 16);
    }
    __device__ __forceinline__ void store(Lds &s, int c, int n) {
        const int top = n - 1 - c * C, tid = threadIdx.x, lane = tid & 63, wv = tid >> 6;
#pragma unroll
        for (int i = 0; i < KS; ++i) {
            const int slot = tid + 256 * i, b = slot / 128, r = slot % 128 / 4, d = b % KB * 32 + slot % 4 * 8;
            const bool in = b / KB * 32 + r <= top;
            const int at = b * kBlk + block_at(r, slot % 4);
            k[i].fix(d, K, in);
            const Frag<NI> f = k[i].pieces();
#pragma unroll
            for (int e = 0; e < NI; ++e) *reinterpret_cast<db8 *>(&s.k[0][0][0][0] + e * kStride + at) = f.p[e];
            if constexpr (Q) {
                q[i].fix(d, K, in);
                const Frag<NI> fq = q[i].pieces();
#pragma unroll
                for (int e = 0; e < NI; ++e) *reinterpret_cast<db8 *>(&s.q[0][0][0][0] + e * kStride + at) = fq.p[e];
            }
        }
#pragma unroll
        for (int i = 0; i < VS; ++i) {
            const int slot = lane + 64 * i, d = col0 + slot % 2 * 8;
            // the load was made at min(d, V - 1): a chunk that starts past the row's end holds nothing
            v[i].fix(min(d, V - 1), V, slot / 2 <= top && d < V);
            T *at = &s.v[wv][slot / 2][slot % 2 * 8];
            if constexpr (sizeof(T) == 2) *reinterpret_cast<du4 *>(at) = v[i].x;
            else {
                *reinterpret_cast<dt4 *>(at) = v[i].a;
                *reinterpret_cast<dt4 *>(at + 4) = v[i].b;
            }
        }
#pragma unroll
        for (int i = 0; i < MS; ++i) {
            const int slot = tid + 256 * i;
            if (slot < int(sizeof(ChunkMats<C, NP>) / 16)) reinterpret_cast<du4 *>(&s.m)[slot] = m[i];
        }
    }
    // Rows tb * 32 + 8 g + 4 e + i, i = 0..3, of the wavefront's columns of v, column lane & 15.
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
