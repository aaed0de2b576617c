// Linear attention with a decay for each head: the kernel that makes the readings and the gradients of q, k and v. All four
// are decayed products of pairs of tokens beside a product with a state:
//     out_a = a0 e^{w_a} M x_a + a1 sum over b of e^{|G_a - G_b|} (x_a . y_b) z_b
// over the b of a's segment at or before it (readings, dq) or at or after it (dk, dv), G the running sum of log-decays:
//     readings: x, y, z = q, k, v      M = S^T, the segment's start state     w = G_a
//     dq:       x, y, z = do, v, k     M = S                                  w = G_a
//     dk:       x, y, z = v, do, q     M = dS, the end state's gradient       w = G_end - G_a
//     dv:       x, y, z = k, q, do     M = dS^T                               w = G_end - G_a
// KEYS: dq and dk, which sum over the value heads of a key head and also give each head's share of the log-decays' gradient
// (linear_bwd.hip): the row's own q or k times the sum above without b = a.
//
// A workgroup takes 64 NQ tokens a, 16 NQ to a wavefront, and ZW columns. Scores are computed transposed: with y as the A operand a lane's
// accumulators are eight neighbouring b of one a, a B operand as they stand (delta_tile.h), so decayed scores go from registers
// into the product with z. The outcome is transposed too: a lane holds eight neighbouring columns of its token. LDS holds a tile of y and z, or
// 32 rows of M, while the next one is on its way through registers.
#pragma once

#include "linear_tile.h"

namespace sdm {

struct AttendSide {
    Rows x, y, z, own;       // own: KEYS
    const float *M;          // [ph][..] + a segment's, [K][V], or null
    int64_t M_head, M_seg;
    void *out;               // dense [P, T, heads, width of z]
    float *dot;              // KEYS: [slices][ph][T], or null
    float a0, a1;
    bool back;               // b at or after a
};
struct AttendArgs {
    AttendSide side[2];      // blockIdx.y
    LinGates gates;
    const int32_t *valid;
    int32_t P, T, Hk, Hv, K, V, seg_tokens;
};

template <typename T, int XP, int ZW, bool KEYS> struct AttendCfg {
    static constexpr int NI = kPieces<T>;
    // Tokens of a wavefront in sixteens: two share every operand read from LDS, where the registers hold them.
    static constexpr int NQ = NI == 1 && XP <= 128 ? 2 : 1;
    static constexpr int QT = 64 * NQ, KT = NI == 1 && XP <= 128 ? 64 : 32;
    using Y = Tile<T, KT, XP>;
    using Z = Tile<T, KT, ZW>;
    using S = Tile<float, KEYS ? ZW : 32, KEYS ? 32 : ZW>;
    static constexpr size_t kTiles = size_t(NI) * (Y::kPlane + Z::kPlane), kState = 3 * size_t(S::kPlane);
    static constexpr size_t kLds = (kTiles > kState ? kTiles : kState) + (kLinSegMax + 4) * sizeof(double);
    static_assert(kLinSegMax % QT == 0, "a query tile lies in one segment");
};

template <typename T, int XP, int ZW, bool KEYS>
__global__ __launch_bounds__(256, 2) void lin_attend_kernel(AttendArgs a) {
    using C = AttendCfg<T, XP, ZW, KEYS>;
    constexpr int NI = C::NI, NQ = C::NQ, QT = C::QT, KT = C::KT, XB = XP / 32, ZB = ZW / 32, TB = KT / 32;
    using Y = typename C::Y;
    using Z = typename C::Z;
    extern __shared__ __align__(16) unsigned char lds[];
    unsigned char *ly = lds, *lz = lds + NI * Y::kPlane;
    double *G = reinterpret_cast<double *>(lds + C::kLds) - (kLinSegMax + 4), *total_of = G + kLinSegMax;
    const AttendSide &s = a.side[blockIdx.y];
    const bool back = s.back;
    const int heads = KEYS ? a.Hk : a.Hv, group = a.Hv / a.Hk, X = s.x.width, Zw = s.z.width;
    const int slices = (Zw + ZW - 1) / ZW, tiles = (a.T + QT - 1) / QT;
    const int slice = blockIdx.x % slices, tile = blockIdx.x / slices % tiles;
    const int oh = blockIdx.x / slices / tiles % heads, p = blockIdx.x / slices / tiles / heads;
    const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lc = lane & 15, lg = lane >> 4;
    const int z0 = slice * ZW, q0 = tile * QT, n = lin_valid(a.valid, p, a.T);
    const int seg = q0 / a.seg_tokens, s0 = seg * a.seg_tokens, s1 = min(s0 + a.seg_tokens, n);
    const int qw = q0 + wv * 16 * NQ, diag = qw & ~31;     // the wavefront's first token; the 32 tokens that it lies in
    T *out = static_cast<T *>(s.out) + (int64_t(p) * a.T * heads + oh) * Zw + z0;
    const int64_t os = int64_t(heads) * Zw;
    auto put = [&](int t, int zb, dt4 lo, dt4 hi) {
        if (t < a.T) eight_store(out + t * os + zb * 32 + lg * 8, Zw - z0 - zb * 32 - lg * 8, lo, hi);
    };
    if (q0 >= n) {
#pragma unroll
        for (int nq = 0; nq < NQ; ++nq)
#pragma unroll
            for (int zb = 0; zb < ZB; ++zb) put(qw + nq * 16 + lc, zb, dt4{}, dt4{});
        return;
    }
    dt4 sum[KEYS ? ZB : 1][2][NQ];
    if constexpr (KEYS) {
#pragma unroll
        for (int zb = 0; zb < ZB; ++zb)
#pragma unroll
            for (int e = 0; e < 2; ++e)
#pragma unroll
                for (int nq = 0; nq < NQ; ++nq) sum[zb][e][nq] = dt4{};
    }
    dt4 acc[ZB][2][NQ];
    auto rows = [&](const Rows &r, int head) { return static_cast<const T *>(r.data) + p * r.sp + head * r.sh; };
    const int first = KEYS ? oh * group : oh, count = KEYS ? group : 1;
    for (int h = first; h < first + count; ++h) {
        const int hk = h / group;
        // x and y are of one kind (keys or values), z of the other
        const T *xr = rows(s.x, KEYS ? h : hk), *yr = rows(s.y, KEYS ? h : hk), *zr = rows(s.z, KEYS ? hk : h);
        segment_gates(a.gates, p, h, s0, s1 - s0, G, total_of);
        Frag<NI> fx[NQ][XB];
#pragma unroll
        for (int nq = 0; nq < NQ; ++nq) {
            const int t = qw + nq * 16 + lc;
            const T *row = xr + int64_t(t) * s.x.st;
#pragma unroll
            for (int d = 0; d < XB; ++d) fx[nq][d] = pieces(eight(row + d * 32 + lg * 8, t < n ? X - d * 32 - lg * 8 : 0));
        }
#pragma unroll
        for (int zb = 0; zb < ZB; ++zb)
#pragma unroll
            for (int e = 0; e < 2; ++e)
#pragma unroll
                for (int nq = 0; nq < NQ; ++nq) acc[zb][e][nq] = dt4{};
        // the product with the state
        if (s.M) {
            const float *M = s.M + (int64_t(p) * a.Hv + h) * s.M_head + seg * s.M_seg;
            const int V = a.V;
            typename C::S t;
            auto bring = [&](int d) {
                if constexpr (KEYS) t.load(M + int64_t(z0) * V, V, Zw - z0, d * 32, V);
                else t.load(M + int64_t(d * 32) * V, V, X - d * 32, z0, V);
            };
            bring(0);
#pragma unroll
            for (int d = 0; d < XB; ++d) {
                lds_barrier();
                t.store(lds);
                lds_barrier();
                if (d + 1 < XB) bring(d + 1);
#pragma unroll
                for (int zb = 0; zb < ZB; ++zb) {
                    Frag<3> f[2];
#pragma unroll
                    for (int e = 0; e < 2; ++e)
                        f[e] = KEYS ? read_rows<3>(lds + zb * kBlk, C::S::kPlane, e) : read_cols<3>(lds + zb * kBlk, C::S::kPlane, e);
                    each_product<3, 3, NI>([&](int m, int l) {
#pragma unroll
                        for (int e = 0; e < 2; ++e)
#pragma unroll
                            for (int nq = 0; nq < NQ; ++nq) acc[zb][e][nq] = mma1(f[e].p[m], fx[nq][d].p[l], acc[zb][e][nq]);
                    });
                }
            }
        } else {
            lds_barrier();
        }
        // Decays are taken relative to a border of the wavefront's tokens until the pairs within its 32: e^{ref - H_b} before it
        // and e^{H_a - ref} after, both at most 1 where the log-decays are (H: G, or -G where b follows a).
        const double sign = back ? -1.0 : 1.0;
        const int border = back ? min(qw + 16 * NQ, s1) - 1 - s0 : qw - 1 - s0;
        const double ref = border >= 0 && border < kLinSegMax ? sign * G[border] : 0.0;
        const float ws = s.a0 * exp2_of(ref + (back ? G[s1 - 1 - s0] : 0.0));
        double Ha[NQ];
#pragma unroll
        for (int nq = 0; nq < NQ; ++nq) Ha[nq] = sign * G[min(qw + nq * 16 + lc - s0, kLinSegMax - 1)];
#pragma unroll
        for (int zb = 0; zb < ZB; ++zb)
#pragma unroll
            for (int e = 0; e < 2; ++e)
#pragma unroll
                for (int nq = 0; nq < NQ; ++nq) acc[zb][e][nq] *= ws;
        float self[NQ] = {};     // a1 (x_a . y_a), in the lanes that come upon it
        // tiles of the segment, from its far end to the wavefront's own tokens
        const int k0 = back ? (s1 - 1 - s0) / KT : 0, k1 = back ? (q0 - s0) / KT : (min(q0 + QT, s1) - 1 - s0) / KT, step = back ? -1 : 1;
        Y ty;
        Z tz;
        auto bring = [&](int kt) {
            const int t0 = s0 + kt * KT;
            ty.load(yr + int64_t(t0) * s.y.st, s.y.st, s1 - t0, 0, X);
            tz.load(zr + int64_t(t0) * s.z.st, s.z.st, s1 - t0, z0, Zw);
        };
        bring(k0);
        for (int kt = k0;; kt += step) {
            lds_barrier();
            ty.store(ly);
            tz.store(lz);
            lds_barrier();
            if (kt != k1) bring(kt + step);
            for (int i = 0; i < TB; ++i) {
                const int tb = back ? TB - 1 - i : i, b0 = s0 + kt * KT + tb * 32;
                if (qw >= s1 || b0 >= s1 || (back ? b0 < diag : b0 > diag)) continue;
                dt4 st[2][NQ] = {};
#pragma unroll
                for (int d = 0; d < XB; ++d) {
                    Frag<NI> f[2];
#pragma unroll
                    for (int e = 0; e < 2; ++e) f[e] = read_rows<NI>(ly + (tb * XB + d) * kBlk, Y::kPlane, e);
                    each_product<3, NI, NI>([&](int m, int l) {
#pragma unroll
                        for (int e = 0; e < 2; ++e)
#pragma unroll
                            for (int nq = 0; nq < NQ; ++nq) st[e][nq] = mma1(f[e].p[m], fx[nq][d].p[l], st[e][nq]);
                    });
                }
                const double *Gb = G + (b0 - s0) + lg * 8;
                if (b0 != diag) {
#pragma unroll
                    for (int e = 0; e < 2; ++e)
#pragma unroll
                        for (int r = 0; r < 4; ++r) {
                            const float w = s.a1 * exp2_of(ref - sign * Gb[e * 4 + r]);
#pragma unroll
                            for (int nq = 0; nq < NQ; ++nq) st[e][nq][r] *= w;
                        }
                } else {
#pragma unroll
                    for (int nq = 0; nq < NQ; ++nq) {
                        const float w = exp2_of(Ha[nq] - ref);
#pragma unroll
                        for (int zb = 0; zb < ZB; ++zb)
#pragma unroll
                            for (int e = 0; e < 2; ++e) acc[zb][e][nq] *= w;
                        const int at = qw + nq * 16 + lc - diag;      // of 32
#pragma unroll
                        for (int e = 0; e < 2; ++e)
#pragma unroll
                            for (int r = 0; r < 4; ++r) {
                                const int b = lg * 8 + e * 4 + r;
                                const float x = s.a1 * st[e][nq][r];
                                if (KEYS && b == at) self[nq] = x;
                                const bool in = KEYS ? (back ? b > at : b < at) : (back ? b >= at : b <= at);
                                st[e][nq][r] = in ? x * exp2_of(Ha[nq] - sign * Gb[e * 4 + r]) : 0.0f;
                            }
                    }
                }
                Frag<3> fp[NQ];
#pragma unroll
                for (int nq = 0; nq < NQ; ++nq) fp[nq] = split<3>(st[0][nq], st[1][nq]);
#pragma unroll
                for (int zb = 0; zb < ZB; ++zb) {
                    Frag<NI> f[2];
#pragma unroll
                    for (int e = 0; e < 2; ++e) f[e] = read_cols<NI>(lz + (tb * ZB + zb) * kBlk, Z::kPlane, e);
                    each_product<3, NI, 3>([&](int m, int l) {
#pragma unroll
                        for (int e = 0; e < 2; ++e)
#pragma unroll
                            for (int nq = 0; nq < NQ; ++nq) acc[zb][e][nq] = mma1(f[e].p[m], fp[nq].p[l], acc[zb][e][nq]);
                    });
                }
            }
            if (kt == k1) break;
        }
        if constexpr (KEYS) {
            const T *mine = rows(s.own, oh) + z0, *other = zr + z0;
#pragma unroll
            for (int nq = 0; nq < NQ; ++nq) {
                const int t = qw + nq * 16 + lc, at = (t - diag) & 31;
                const float w = __shfl(self[nq], at / 8 * 16 + lc, 64);
                float dot = 0.0f;
#pragma unroll
                for (int zb = 0; zb < ZB; ++zb) {
                    const int left = t < n ? Zw - z0 - zb * 32 - lg * 8 : 0;
                    dt4 m[2], o[2];
                    eight_values(eight(mine + int64_t(t) * s.own.st + zb * 32 + lg * 8, left), m[0], m[1]);
                    eight_values(eight(other + int64_t(t) * s.z.st + zb * 32 + lg * 8, left), o[0], o[1]);
#pragma unroll
                    for (int e = 0; e < 2; ++e)
#pragma unroll
                        for (int r = 0; r < 4; ++r) {
                            const float x = acc[zb][e][nq][r];
                            dot = fmaf(m[e][r], x, dot);
                            sum[zb][e][nq][r] += fmaf(w, o[e][r], x);
                        }
                }
                dot += __shfl_xor(dot, 16, 64);
                dot += __shfl_xor(dot, 32, 64);
                if (s.dot && lg == 0 && t < n) s.dot[((int64_t(slice) * a.P + p) * a.Hv + h) * a.T + t] = dot;
            }
            lds_barrier();       // G and the tiles are free
        }
    }
#pragma unroll
    for (int nq = 0; nq < NQ; ++nq) {
        const int t = qw + nq * 16 + lc;
#pragma unroll
        for (int zb = 0; zb < ZB; ++zb) {
            dt4 o[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) o[e] = t < n ? (KEYS ? sum[KEYS ? zb : 0][e][nq] : acc[zb][e][nq]) : dt4{};
            put(t, zb, o[0], o[1]);
        }
    }
}

template <typename T, int XP, int ZW, bool KEYS> hipError_t attend_go(const AttendArgs &a, int sides, hipStream_t st) {
    using C = AttendCfg<T, XP, ZW, KEYS>;
    const int64_t tiles = (int64_t(a.T) + C::QT - 1) / C::QT, slices = (a.side[0].z.width + ZW - 1) / ZW;
    hipLaunchKernelGGL((lin_attend_kernel<T, XP, ZW, KEYS>), dim3(unsigned(tiles * slices * a.P * (KEYS ? a.Hk : a.Hv)), unsigned(sides)), dim3(256),
                       C::kLds, st, a);
    return hipGetLastError();
}
template <typename T, int XP, bool KEYS> hipError_t attend_slices(const AttendArgs &a, int sides, hipStream_t st) {
    return lin_slice(a.side[0].z.width) == 64 ? attend_go<T, XP, 64, KEYS>(a, sides, st) : attend_go<T, XP, 128, KEYS>(a, sides, st);
}
template <typename T, bool KEYS> hipError_t attend(const AttendArgs &a, int sides, hipStream_t st) {
    switch (lin_width(a.side[0].x.width)) {
        case 64: return attend_slices<T, 64, KEYS>(a, sides, st);
        case 128: return attend_slices<T, 128, KEYS>(a, sides, st);
        default: return attend_slices<T, 256, KEYS>(a, sides, st);
    }
}
template <typename T, int XP, int ZW, bool KEYS> hipError_t attend_attr() {
    static_assert(AttendCfg<T, XP, ZW, KEYS>::kLds <= 80 * 1024, "two workgroups to a compute unit");
    return hipFuncSetAttribute(reinterpret_cast<const void *>(&lin_attend_kernel<T, XP, ZW, KEYS>), hipFuncAttributeMaxDynamicSharedMemorySize,
                               int(AttendCfg<T, XP, ZW, KEYS>::kLds));
}
template <typename T, bool KEYS> hipError_t attend_prepare() {
    hipError_t e = attend_attr<T, 64, 64, KEYS>();
    if (e == hipSuccess) e = attend_attr<T, 64, 128, KEYS>();
    if (e == hipSuccess) e = attend_attr<T, 128, 64, KEYS>();
    if (e == hipSuccess) e = attend_attr<T, 128, 128, KEYS>();
    if (e == hipSuccess) e = attend_attr<T, 256, 64, KEYS>();
    if (e == hipSuccess) e = attend_attr<T, 256, 128, KEYS>();
    return e;
}

// One translation unit for each element type and kind (linear_attend_*.hip).
hipError_t attend_values_bf16(const AttendArgs &a, hipStream_t st);
hipError_t attend_values_f32(const AttendArgs &a, hipStream_t st);
hipError_t attend_keys_bf16(const AttendArgs &a, hipStream_t st);
hipError_t attend_keys_f32(const AttendArgs &a, hipStream_t st);
hipError_t attend_prepare_values_bf16();
hipError_t attend_prepare_values_f32();
hipError_t attend_prepare_keys_bf16();
hipError_t attend_prepare_keys_f32();

}  // namespace sdm
