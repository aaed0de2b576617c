// Linear attention with a decay for each head: the sum of decayed products k v over a segment (and of q and the readings' gradient).
//
// Bound by memory: 16 heads of 16384 tokens of 128 x 128, bfloat16, in segments of 256 tokens: 50 us for 101 MB read and 85 written, 67 of
// them the sums, stored 64 bytes in a row (at a copy's rate 36 us; its matrix instructions 10, the others 13). The product's accumulators are the sum, a wavefront's ZW / 4 columns of it,
// so that nothing is added up across wavefronts.
#pragma once

#include "linear_tile.h"

namespace sdm {

struct StateArgs {
    Rows y, z;               // widths K and V
    LinGates gates;
    const int32_t *valid;
    float *S;                // [ph][slots][K][V]
    float *decay;            // [ph][segs] or null
    const float *base;       // `final`: [ph][K][V] or null
    int32_t P, T, Hk, Hv, K, V, segs, slots, seg_tokens;
    float scale;
    bool back, final;        // back: weights scale e^{G_t}; final: the one segment's end state, from base
};

template <typename T, int KP, int ZW, bool EVEN> struct StateCfg {
    static constexpr int NI = kPieces<T>, KT = NI == 1 && KP <= 128 ? 64 : 32;
    using Y = Tile<T, KT, KP, EVEN>;
    using Z = Tile<T, KT, ZW, EVEN>;
    static constexpr size_t kTiles = size_t(NI) * Y::kPlane + 3 * size_t(Z::kPlane);
    static constexpr size_t kLds = kTiles + kLinSegMax * sizeof(float) + (kLinSegMax + 4) * sizeof(double);
};

// sum_t w_t y_t z_t over one segment: all of y's columns and ZW of z's. A wavefront takes ZW / 4 columns; z is weighted and cut into
// pieces on its way to LDS.
template <typename T, int KP, int ZW, bool EVEN> __device__ __forceinline__ void lin_state(const StateArgs &a, const int block) {
    using C = StateCfg<T, KP, ZW, EVEN>;
    constexpr int NI = C::NI, KT = C::KT, KB = KP / 32, ZB = ZW / 32, TB = KT / 32, NC = ZW / 64;
    using Y = typename C::Y;
    using Z = typename C::Z;
    extern __shared__ __align__(16) unsigned char lds[];
    unsigned char *ly = lds, *lz = lds + NI * Y::kPlane;
    double *G = reinterpret_cast<double *>(lds + C::kTiles), *total_of = G + kLinSegMax;
    float *w = reinterpret_cast<float *>(total_of + 4);
    const int slices = (a.V + ZW - 1) / ZW, slice = block % slices, seg = block / slices % a.segs, ph = block / slices / a.segs;
    const int h = ph % a.Hv, p = ph / a.Hv, hk = h / (a.Hv / a.Hk), z0 = slice * ZW;
    const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lc = lane & 15, lg = lane >> 4;
    const int s0 = seg * a.seg_tokens, live = min(a.seg_tokens, lin_valid(a.valid, p, a.T) - s0);
    if (live <= 0 && !a.final) return;
    const T *yr = static_cast<const T *>(a.y.data) + p * a.y.sp + hk * a.y.sh + s0 * a.y.st;
    const T *zr = static_cast<const T *>(a.z.data) + p * a.z.sp + h * a.z.sh + s0 * a.z.st;
    Y ty;
    Z tz;
    auto bring = [&](int t0) {
        ty.load(yr + t0 * a.y.st, a.y.st, live - t0, 0, a.K, threadIdx.x);
        tz.load(zr + t0 * a.z.st, a.z.st, live - t0, z0, a.V, threadIdx.x);
    };
    if (live > 0) bring(0);
    segment_gates(a.gates, p, h, s0, live, G, total_of);
    lds_barrier();
    const double end = live > 0 ? G[live - 1] : 0.0;
    w[threadIdx.x] = a.back ? a.scale * exp2_of(G[threadIdx.x]) : exp2_of(end - G[threadIdx.x]);
    if (a.decay && slice == 0 && threadIdx.x == 0) a.decay[int64_t(ph) * a.segs + seg] = exp2_of(end);
    dt4 acc[KB][2][NC];
#pragma unroll
    for (int kb = 0; kb < KB; ++kb)
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
            for (int c = 0; c < NC; ++c) acc[kb][e][c] = dt4{};
    for (int t0 = 0; t0 < live; t0 += KT) {
        lds_barrier();
        ty.store(ly, threadIdx.x);
        tz.store_weighted(lz, w + t0, threadIdx.x);
        lds_barrier();
        if (t0 + KT < live) bring(t0 + KT);
#pragma unroll
        for (int tb = 0; tb < TB; ++tb) {
            Frag<3> fz[NC];
#pragma unroll
            for (int c = 0; c < NC; ++c) {
                const int ct = wv * NC + c;
                fz[c] = read_cols_in_order<3>(lz + (tb * ZB + ct / 2) * kBlk, Z::kPlane, ct & 1);
            }
#pragma unroll
            for (int kb = 0; kb < KB; ++kb) {
                Frag<NI> f[2];
#pragma unroll
                for (int e = 0; e < 2; ++e) f[e] = read_cols<NI>(ly + (tb * KB + kb) * kBlk, Y::kPlane, e);
                each_product<3, NI, 3>([&](int m, int l) {
#pragma unroll
                    for (int e = 0; e < 2; ++e)
#pragma unroll
                        for (int c = 0; c < NC; ++c) acc[kb][e][c] = mma1(f[e].p[m], fz[c].p[l], acc[kb][e][c]);
                });
            }
        }
    }
    const int64_t KV = int64_t(a.K) * a.V;
    float *dst = a.S + (int64_t(ph) * a.slots + (a.final ? 0 : seg)) * KV;
    const float *base = a.final && a.base ? a.base + ph * KV : nullptr;
    const float decay = exp2_of(end);
#pragma unroll
    for (int c = 0; c < NC; ++c) {
        const int col = z0 + (wv * NC + c) * 16 + lc;
        if (col >= a.V) continue;
#pragma unroll
        for (int kb = 0; kb < KB; ++kb)
#pragma unroll
            for (int e = 0; e < 2; ++e)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int row = kb * 32 + lg * 8 + e * 4 + r;
                    if (row >= a.K) continue;
                    const int64_t at = int64_t(row) * a.V + col;
                    dst[at] = base ? fmaf(decay, base[at], acc[kb][e][c][r]) : acc[kb][e][c][r];
                }
    }
}
template <typename T, int KP, int ZW, bool EVEN> __global__ __launch_bounds__(256, 2) void lin_state_kernel(StateArgs a) {
    lin_state<T, KP, ZW, EVEN>(a, blockIdx.x);
}

template <typename T, int KP, int ZW, bool EVEN> hipError_t state_go(const StateArgs &a, hipStream_t st) {
    const int64_t slices = (a.V + ZW - 1) / ZW;
    hipLaunchKernelGGL((lin_state_kernel<T, KP, ZW, EVEN>), dim3(unsigned(slices * a.segs * a.P * a.Hv)), dim3(256), (StateCfg<T, KP, ZW, EVEN>::kLds), st, a);
    return hipGetLastError();
}
template <typename T, int KP, int ZW> hipError_t state_even(const StateArgs &a, hipStream_t st) {
    constexpr int vec = 16 / sizeof(T);
    return a.K % vec == 0 && a.V % vec == 0 ? state_go<T, KP, ZW, true>(a, st) : state_go<T, KP, ZW, false>(a, st);
}
template <typename T, int KP> hipError_t state_slices(const StateArgs &a, hipStream_t st) {
    return lin_slice(a.V) == 64 ? state_even<T, KP, 64>(a, st) : state_even<T, KP, 128>(a, st);
}
template <typename T> hipError_t state_pick(const StateArgs &a, hipStream_t st) {
    switch (lin_width(a.K)) {
        case 64: return state_slices<T, 64>(a, st);
        case 128: return state_slices<T, 128>(a, st);
        default: return state_slices<T, 256>(a, st);
    }
}
}  // namespace sdm
