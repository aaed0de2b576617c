// What the kernels that walk a sequence's chunks share: the chunk's operands in LDS, and the state in
// accumulators.
#pragma once

#include "delta_tile.h"

namespace sdm {

constexpr size_t kDeltaMaxLds = 160 * 1024 - 256;

// A pointer that all lanes share, in scalar registers.
template <typename T> __device__ __forceinline__ const T *uniform(const T *p) {
    const uint64_t u = reinterpret_cast<uint64_t>(p);
    const uint32_t lo = __builtin_amdgcn_readfirstlane(uint32_t(u)), hi = __builtin_amdgcn_readfirstlane(uint32_t(u >> 32));
    return reinterpret_cast<const T *>(uint64_t(hi) << 32 | lo);
}

// Workgroups of eight wavefronts: four that compute, 16 columns of the state each, and four that
// bring the chunks' operands from memory to LDS through their registers, a chunk ahead in LDS and another on its way. (The
// computing ones have no registers for that, and the copy past the registers, global_load_lds, took 25 bytes a
// cycle of a compute unit and LDS reads waited for it: 0.55 us of a chunk's 3.9.)
constexpr int kWalkThreads = 512;

// T: the inputs' type; Q: q and P are wanted too.
template <typename T, int C, int KP, bool Q> struct Walk {
    static constexpr int NI = kPieces<T>, KB = KP / 32, TB = C / 32;
    static constexpr int kStride = TB * KB * kBlk;              // between the pieces of k (and of q)
    static constexpr int KS = kStride / 4096;                   // 16-byte eights of a piece of k per thread
    using Mem = ChunkMem<C>;
    static constexpr int NE = kTri<C> * 128, ES = (NE + 255) / 256;   // eights of X (and of P), and those of a thread
    static constexpr int RS = sizeof(T);                        // 16-byte pieces of a row of v's 16 columns
    static constexpr int VS = C * RS / 64;
    struct Lds {
        unsigned char k[NI][TB][KB][kBlk];
        unsigned char q[Q ? NI : 0][TB][KB][kBlk];
        ChunkMats<C> m;
        T v[4][C][16];
    };
    static constexpr int kBufs = 2 * sizeof(Lds) <= kDeltaMaxLds ? 2 : 1;
    static constexpr size_t kLds = kBufs * sizeof(Lds);

    // The computing wavefronts' side: the i-th chunk taken is in buffer i & (kBufs - 1) after begin() and i times turn().
    static __device__ __forceinline__ void begin() { lds_barrier(); }
    static __device__ __forceinline__ void turn() {
        lds_barrier();
        if constexpr (kBufs == 1) lds_barrier();
    }

    // The other side. val: v, or what takes its place; cg: the column group of the wavefront four before this one.
    struct Bring {
        const bf16 *kp, *qp;
        const T *vp;
        const Mem *mats;
        int64_t kplane, qplane, ks, qs, vs;
        int col0, n;
        du4 k[NI][KS], q[Q ? NI : 1][Q ? KS : 1], v[VS], x[ES][2], pp[Q ? ES : 1][2], g;

        __device__ Bring(const DeltaArgs &a, const DeltaWs &ws, int p, int h, int hk, int ph, int cg, const Rows &val, int tokens)
            : kp(uniform(a.kk.data + p * a.kk.sp + hk * a.kk.sh)), qp(uniform(a.qq.data + p * a.qq.sp + hk * a.qq.sh)),
              vp(uniform(static_cast<const T *>(val.data) + p * val.sp + h * val.sh)),
              mats(uniform(reinterpret_cast<const Mem *>(ws.mats) + int64_t(ph) * ws.Nt)), kplane(a.kk.plane), qplane(a.qq.plane),
              ks(a.kk.st), qs(a.qq.st), vs(val.st), n(tokens) {
            // columns past the row's end are read from its last ones: nothing that they reach is kept
            col0 = min(cg * 16 + int(threadIdx.x) % RS * (16 / int(sizeof(T))), val.width - 16 / int(sizeof(T)));
        }
        // Rows past the last valid token are read as that token's: finite where it is, and met by gates of 0 everywhere.
        __device__ __forceinline__ void load(int c) {
            const int top = n - 1 - c * C, tid = threadIdx.x & 255, lane = tid & 63;
            const int64_t t0 = int64_t(c) * C;
            const bf16 *kc = kp + t0 * ks, *qc = qp + t0 * qs;
            const T *vc = vp + t0 * vs;
#pragma unroll
            for (int i = 0; i < KS; ++i) {
                const int slot = tid + 256 * i, row = min(slot / 128 / KB * 32 + slot % 128 / 4, top);
                const int d = slot / 128 % KB * 32 + slot % 4 * 8;
#pragma unroll
                for (int e = 0; e < NI; ++e) {
                    k[e][i] = *reinterpret_cast<const du4 *>(kc + e * kplane + uint32_t(row * int(ks) + d));
                    if constexpr (Q) q[e][i] = *reinterpret_cast<const du4 *>(qc + e * qplane + uint32_t(row * int(qs) + d));
                }
            }
#pragma unroll
            for (int i = 0; i < VS; ++i)
                v[i] = *reinterpret_cast<const du4 *>(vc + uint32_t(min((lane + 64 * i) / RS, top) * int(vs) + col0));
            const Mem &mem = mats[c];
#pragma unroll
            for (int i = 0; i < ES; ++i) {
                const int e = min(tid + 256 * i, NE - 1);
                const du4 *px = reinterpret_cast<const du4 *>(&mem.X[0][0][0]), *from = reinterpret_cast<const du4 *>(&mem.P[0][0][0]);
#pragma unroll
                for (int w = 0; w < 2; ++w) {
                    x[i][w] = px[e * 2 + w];
                    if constexpr (Q) pp[i][w] = from[e * 2 + w];
                }
            }
            g = reinterpret_cast<const du4 *>(&mem.g)[lane];
        }
        __device__ __forceinline__ void store(Lds &s) const {
            const int tid = threadIdx.x & 255, lane = tid & 63, wv = tid >> 6;
#pragma unroll
            for (int i = 0; i < KS; ++i) {
                const int slot = tid + 256 * i, at = slot / 128 * kBlk + block_at(slot % 128 / 4, slot % 4);
#pragma unroll
                for (int e = 0; e < NI; ++e) {
                    *reinterpret_cast<du4 *>(&s.k[0][0][0][0] + e * kStride + at) = k[e][i];
                    if constexpr (Q) *reinterpret_cast<du4 *>(&s.q[0][0][0][0] + e * kStride + at) = q[e][i];
                }
            }
#pragma unroll
            for (int i = 0; i < VS; ++i) reinterpret_cast<du4 *>(&s.v[wv][0][0])[lane + 64 * i] = v[i];
#pragma unroll
            for (int i = 0; i < ES; ++i) {
                const int e = tid + 256 * i;
                if (NE % 256 && e >= NE) break;
                const int at = block_at(e % 128 / 4, e % 4);
                const Frag<3> fx = split<3>(__builtin_bit_cast(dt4, x[i][0]), __builtin_bit_cast(dt4, x[i][1]));
#pragma unroll
                for (int n = 0; n < 3; ++n) *reinterpret_cast<db8 *>(s.m.X[n][e / 128] + at) = fx.p[n];
                if constexpr (Q) {
                    const Frag<3> fp = split<3>(__builtin_bit_cast(dt4, pp[i][0]), __builtin_bit_cast(dt4, pp[i][1]));
#pragma unroll
                    for (int n = 0; n < 3; ++n) *reinterpret_cast<db8 *>(s.m.P[n][e / 128] + at) = fp.p[n];
                }
            }
            if (wv == 0) reinterpret_cast<du4 *>(&s.m.g)[lane] = g;
        }
        // Chunks c0, c0 + dir, ..., `count` of them.
        __device__ __forceinline__ void run(Lds *bufs, int c0, int dir, int count) {
            if (count > 0) {
                load(c0);
                store(bufs[0]);
            }
            if (count > 1) load(c0 + dir);
            lds_barrier();
            for (int i = 0; i < count; ++i) {
                if constexpr (kBufs == 1) lds_barrier();
                if (i + 1 < count) store(bufs[(i + 1) & (kBufs - 1)]);
                if (i + 2 < count) load(c0 + (i + 2) * dir);
                lds_barrier();
            }
        }
    };
    static __device__ __forceinline__ dt4 value(const Lds &s, int tb, int e) {
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
template <int KB> __device__ __forceinline__ void load_state(dt4 (&S)[KB][2], const float *state, int64_t ph, int K, int V, int col) {
    const int lg = (threadIdx.x & 63) >> 4;
    const float *src = state + ph * K * V + col;
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
template <int KB> __device__ __forceinline__ void store_state(const dt4 (&S)[KB][2], float *state, int64_t ph, int K, int V, int col) {
    if (!state || col >= V) return;
    const int lg = (threadIdx.x & 63) >> 4;
    float *dst = state + ph * K * V + col;
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
