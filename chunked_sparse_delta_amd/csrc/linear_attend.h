// Linear attention with a decay for each head: the kernel that makes the readings and the gradients of q, k and v. All four
// are decayed products of pairs of tokens beside a product with a state:
//     out_a = a0 e^{w_a} M x_a + a1 sum over b of e^{|G_a - G_b|} (x_a . y_b) z_b
// over the b of a's segment at or before it (readings, dq) or at or after it (dk, dv), G the running sum of log-decays:
//     readings: x, y, z = q, k, v      M = S^T, the segment's start state     w = G_a
//     dq:       x, y, z = do, v, k     M = S                                  w = G_a
//     dk:       x, y, z = v, do, q     M = dS, the end state's gradient       w = G_end - G_a
//     dv:       x, y, z = k, q, do     M = dS^T                               w = G_end - G_a
// KEYS: dq and dk, which sum over the value heads of a key head and also give each head's share of the log-decays' gradient
// (linear.hip): the row's own q or k times the sum above without b = a.
//
// CAUSAL, the readings: no infinity or NaN in a z behind a reaches it, though a's scores with the 32 tokens around it are zeros in a product
// with all of their z. Tiles that may lie behind some of the a are sifted on their way to LDS: such values go in as zeros, and the a at or behind
// the first one of a column read NaN there. (1 % of the time: 16384 tokens of 16 heads 180.5 us of all kernels, 178.5 without.)
//
// A workgroup takes 64 NQ tokens a, 16 NQ to a wavefront, and ZW columns. Scores are computed transposed: with y as the A operand a lane's
// accumulators are eight neighbouring b of one a, a B operand as they stand (delta_tile.h), so decayed scores go from registers
// into the product with z. The outcome is transposed too: a lane holds eight neighbouring columns of its token. LDS holds a tile of y and z, or
// 32 rows of M, while the next one is on its way through registers; two workgroups share a compute unit.
// dk is summed with its sign turned. The matrix instruction's sums come out low on average, whatever their sign, and so did a token's shares
// as query and as key, in which q and k of one sign are common: their difference, summed over a segment, was off by as much in all heads. So
// the one is low and the other high, by as much for every token together, which the correction at the segment's ends takes out (a head's
// log-decay gradient, 2 x 128 float32 tokens of 64 x 64: 7.1e-7 off on average, now 2.0e-7; a token's 3.6e-7 and 1.9e-7).
// Precision: sums are float32, G float64. M, decayed scores and float32 rows are three bfloat16 pieces each, so that products keep
// float32's 24 bits; results are rounded once.
// Measured (bfloat16, 128 x 128, 256 tokens to a segment): the readings of 16 heads of 16384 tokens 109 us; dq, dk and dv of 4 x 16 heads
// of 2048 tokens, keys shared by two, 199 (of 147 and 55 one after the other). Of the 109: matrix instructions alone would take 26 (62.9 M cycles on
// 1024 SIMDs at 2.4 GHz), the other vector instructions about 32, a copy of as many bytes 74 (319 MB read, 67 written). None hides
// the others well. Of the 199: 38, 55 and 154 (655 MB read, 143 written): a workgroup takes one tile and reads its segment's rows and state again, and
// sums over sharing heads go through memory. A form that took 120 us took 84 without its matrix instructions and 57 with nothing but the tiles' way through
// LDS; a workgroup with one tile takes 7. Without effect on that form (2 % at most): tiles or M another step ahead in registers or in a
// second LDS buffer, operands read from LDS ahead of the products before, 32 tokens of y and z at a time, wavefronts' priorities; eight
// wavefronts that share a whole segment's tiles, two LDS buffers of them, took 119. With effect: one XCD for what reads
// the same rows, all tiles of a segment in one workgroup in turn, loads without branches around them.
#pragma once

#include "linear_state.h"

namespace sdm {

struct AttendSide {
    Rows x, y, z, own;       // own: KEYS
    const float *M;          // [ph][..] + a segment's, [K][V], or null
    int64_t M_head, M_seg;
    void *out;               // dense [P, T, heads, width of z]
    float *dot;              // KEYS: [slices][ph][T], or null (dk: negative)
    float *rest;             // KEYS with shared key heads: lin_rest_floats
    float a0, a1;
    bool back;               // b at or after a (not CAUSAL)
};
struct AttendArgs {
    AttendSide side[3];      // the readings; or dq, dk and dv
    LinGates gates;
    const int32_t *valid;
    int32_t P, T, Hk, Hv, K, V, segs, seg_tokens;
    bool whole;
};

template <typename T, int XP, int ZW, bool KEYS, bool EVEN> struct AttendCfg {
    static constexpr int NI = kPieces<T>;
    // Tokens of a wavefront in sixteens: two share every operand read from LDS, where the registers hold them (one, with
    // twice the wavefronts, took 126 us where two took 120).
    static constexpr int NQ = NI == 1 && XP <= 128 ? 2 : 1;
    static constexpr int QT = 64 * NQ, KT = NI == 1 && XP <= 128 ? 64 : 32;
    using Y = Tile<T, KT, XP, EVEN>;
    using Z = Tile<T, KT, ZW, EVEN>;
    using S = Tile<float, KEYS ? ZW : 32, KEYS ? 32 : ZW, EVEN>;
    static constexpr size_t kTiles = size_t(NI) * (Y::kPlane + Z::kPlane), kState = 3 * size_t(S::kPlane);
    static constexpr size_t kGates = (kLinSegMax + 4) * sizeof(double) + kLinSegMax * sizeof(float) + (ZW + 4) * sizeof(int);
    static constexpr size_t kLds = (kTiles > kState ? kTiles : kState) + kGates;
    static_assert(kLinSegMax % QT == 0, "a query tile lies in one segment");
};

template <typename T, int XP, int ZW, bool KEYS, bool EVEN, bool CAUSAL>
__device__ __forceinline__ void lin_attend(const AttendArgs &a, const AttendSide &s, const int block) {
    using C = AttendCfg<T, XP, ZW, KEYS, EVEN>;
    constexpr int NI = C::NI, NQ = C::NQ, QT = C::QT, KT = C::KT, XB = XP / 32, ZB = ZW / 32, TB = KT / 32;
    using Y = typename C::Y;
    using Z = typename C::Z;
    extern __shared__ __align__(16) unsigned char lds[];
    unsigned char *ly = lds, *lz = lds + NI * Y::kPlane;
    double *total_of = reinterpret_cast<double *>(lds + C::kLds) - 4, *G = total_of - kLinSegMax;
    float *local = reinterpret_cast<float *>(G) - kLinSegMax;     // a token's decay to the edge of its 32 on the side of the a
    int *first = reinterpret_cast<int *>(local) - (ZW + 4);       // CAUSAL: see Tile::sift
    if (CAUSAL && threadIdx.x <= ZW) first[threadIdx.x] = INT_MAX;
    const bool back = s.back;
    const int heads = KEYS ? a.Hk : a.Hv, group = a.Hv / a.Hk, X = s.x.width, Zw = s.z.width;
    const int slices = (Zw + ZW - 1) / ZW, seg_tiles = a.seg_tokens / QT;
    // What reads the same keys, values and states goes to one XCD (blocks are dealt to the eight in turn), where there is enough for
    // all of them: the tiles and slices of a segment, of the value heads that share a key head.
    // A workgroup takes one tile, or (`whole`, not KEYS) all of a segment's in turn.
    const int tiles = !KEYS && a.whole ? 1 : seg_tiles;
    const int unit = slices * tiles * (KEYS ? 1 : group), units = a.P * a.Hk * a.segs, xcds = lin_xcds(units);
    const int at_xcd = block / xcds, u = at_xcd / unit * xcds + int(block) % xcds, in_unit = at_xcd % unit;
    if (u >= units) return;
    const int seg = u % a.segs, khead = u / a.segs % a.Hk, p = u / a.segs / a.Hk;
    const int slice = in_unit % slices, oh = KEYS ? khead : khead * group + in_unit / slices / tiles;
    const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int s0 = seg * a.seg_tokens, n = lin_valid(a.valid, p, a.T), s1 = min(s0 + a.seg_tokens, n), z0 = slice * ZW;
    T *out = static_cast<T *>(s.out) + (int64_t(p) * a.T * heads + oh) * Zw + z0;
    const int64_t os = int64_t(heads) * Zw;
    dt4 acc[ZB][2][NQ];
    auto rows = [&](const Rows &r, int head) { return static_cast<const T *>(r.data) + p * r.sp + head * r.sh; };
    // KEYS: the value heads in turn; else tiles, those that see most of their segment first
    bool gated = false;
    const int turns = KEYS ? group : seg_tiles / tiles;
    for (int turn = 0; turn < turns; ++turn) {
        const int h = KEYS ? oh * group + turn : oh, hk = h / group;
        const int tile = in_unit / slices % tiles + (KEYS ? 0 : turn), q0 = s0 + (back ? tile : seg_tiles - 1 - tile) * QT;
        if (q0 >= a.T) continue;
        const int qw = q0 + wv * 16 * NQ, diag = qw & ~31;     // the wavefront's first token; the 32 tokens that it lies in
        const bool x_whole = qw + 16 * NQ <= n && XP <= X;
        // The thread's number as a value of its own: addresses made from it stay in this turn of the loop, where the compiler
        // would keep them all in registers through it.
        int tid = threadIdx.x;
        asm volatile("" : "+v"(tid));
        const int lane = tid & 63, lc = lane & 15, lg = lane >> 4;
        auto put = [&](int t, int zb, dt4 lo, dt4 hi) {
            if (t < a.T) eight_store<EVEN>(out + t * os + zb * 32 + lg * 8, Zw - z0 - zb * 32 - lg * 8, lo, hi);
        };
        if (q0 >= n) {
            if (KEYS && turn > 0) break;
#pragma unroll
            for (int nq = 0; nq < NQ; ++nq)
#pragma unroll
                for (int zb = 0; zb < ZB; ++zb) put(qw + nq * 16 + lc, zb, dt4{}, dt4{});
            continue;
        }
        // x and y are of one kind (keys or values), z of the other
        const T *xr = rows(s.x, KEYS ? h : hk), *yr = rows(s.y, KEYS ? h : hk), *zr = rows(s.z, KEYS ? hk : h);
        const float *M = s.M ? s.M + (int64_t(p) * a.Hv + h) * s.M_head + seg * s.M_seg : nullptr;
        typename C::S tm;
        auto bring_state = [&](int d) {
            const int V = a.V;
            if constexpr (KEYS) tm.load(M + int64_t(z0) * V, V, Zw - z0, d * 32, V, tid);
            else tm.load(M + int64_t(min(d * 32, X - 1)) * V, V, max(X - d * 32, 1), z0, V, tid);     // no rows left: x is 0 there
        };
        if (M) bring_state(0);
        // tiles of the segment, from its far end to the wavefront's own tokens
        const int k0 = back ? (s1 - 1 - s0) / KT : 0, k1 = back ? (q0 - s0) / KT : (min(q0 + QT, s1) - 1 - s0) / KT, step = back ? -1 : 1;
        Y ty;
        Z tz;
        auto bring = [&](int kt) {
            const int t0 = s0 + kt * KT;
            ty.load(yr + int64_t(t0) * s.y.st, s.y.st, s1 - t0, 0, X, tid);
            tz.load(zr + int64_t(t0) * s.z.st, s.z.st, s1 - t0, z0, Zw, tid);
        };
        const bool new_gates = KEYS || !gated;
        gated = true;
        if (new_gates) segment_gates(a.gates, p, h, s0, s1 - s0, G, total_of);
        Eight<T> ex[NQ][XB];
#pragma unroll
        for (int nq = 0; nq < NQ; ++nq) {
            const T *row = xr + int64_t(min(qw + nq * 16 + lc, n - 1)) * s.x.st;
#pragma unroll
            for (int d = 0; d < XB; ++d) ex[nq][d] = eight_load<EVEN>(row, d * 32 + lg * 8, X);
        }
        Frag<NI> fx[NQ][XB];
#pragma unroll
        for (int nq = 0; nq < NQ; ++nq)
#pragma unroll
            for (int d = 0; d < XB; ++d) {
                if (!x_whole) eight_mask(ex[nq][d], d * 32 + lg * 8, X, qw + nq * 16 + lc < n);
                if (KEYS && back) eight_negate(ex[nq][d]);
                fx[nq][d] = pieces(ex[nq][d]);
            }
#pragma unroll
        for (int zb = 0; zb < ZB; ++zb)
#pragma unroll
            for (int e = 0; e < 2; ++e)
#pragma unroll
                for (int nq = 0; nq < NQ; ++nq) acc[zb][e][nq] = dt4{};
        // the product with the state, 32 of its rows (KEYS: columns) at a time
        if (M) {
#pragma unroll
            for (int d = 0; d < XB; ++d) {
                lds_barrier();
                tm.store(lds, tid);
                lds_barrier();
                if (d + 1 < XB) bring_state(d + 1);
#pragma unroll
                for (int zb = 0; zb < ZB; ++zb) {
                    Frag<3> f[2];
#pragma unroll
                    for (int e = 0; e < 2; ++e)
                        f[e] = KEYS ? read_rows<3>(lds + zb * kBlk, C::S::kPlane, e, lane) : read_cols<3>(lds + zb * kBlk, C::S::kPlane, e, lane);
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
        const double sign = back ? -1.0 : 1.0;
        auto edge_of = [&](int b) { return back ? (b > 0 ? G[b - 1] : 0.0) : G[b + 31]; };    // of the 32 tokens from b on
        if (new_gates) local[threadIdx.x] = exp2_of(sign * (edge_of(threadIdx.x & ~31) - G[threadIdx.x]));
        // Decays are taken relative to a border of the wavefront's tokens until the pairs within its 32: e^{ref - H_b} before it
        // and e^{H_a - ref} after, both at most 1 where the log-decays are (H: G, or -G where b follows a).
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
        bring(k0);
        for (int kt = k0;; kt += step) {
            lds_barrier();
            ty.store(ly, tid);
            if (CAUSAL && s0 + (kt + 1) * KT > q0) tz.sift(tid, kt * KT, first);      // (what lies before all of the a reaches them all)
            tz.store(lz, tid);
            lds_barrier();
            if (kt != k1) bring(kt + step);
            for (int j = 0; j < TB; ++j) {
                const int tb = back ? TB - 1 - j : j, b0 = s0 + kt * KT + tb * 32;
                if (qw >= s1 || b0 >= s1 || (back ? b0 < diag : b0 > diag)) continue;
                dt4 st[2][NQ] = {};
#pragma unroll
                for (int d = 0; d < XB; ++d) {
                    Frag<NI> f[2];
#pragma unroll
                    for (int e = 0; e < 2; ++e) f[e] = read_rows<NI>(ly + (tb * XB + d) * kBlk, Y::kPlane, e, lane);
                    each_product<3, NI, NI>([&](int m, int l) {
#pragma unroll
                        for (int e = 0; e < 2; ++e)
#pragma unroll
                            for (int nq = 0; nq < NQ; ++nq) st[e][nq] = mma1(f[e].p[m], fx[nq][d].p[l], st[e][nq]);
                    });
                }
                const double *Gb = G + (b0 - s0) + lg * 8;
                if (b0 != diag) {
                    const float w = s.a1 * exp2_of(ref - sign * edge_of(b0 - s0));
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const dt4 d = w * *reinterpret_cast<const dt4 *>(local + (b0 - s0) + lg * 8 + e * 4);
#pragma unroll
                        for (int nq = 0; nq < NQ; ++nq) st[e][nq] *= d;
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
                    for (int e = 0; e < 2; ++e) f[e] = read_cols<NI>(lz + (tb * ZB + zb) * kBlk, Z::kPlane, e, lane);
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
            // The sum over the value heads that share the key head waits in memory for the next one: registers hold one head's alone.
            const bool begins = turn == 0, ends = turn + 1 == turns;
            dt4 *rest = reinterpret_cast<dt4 *>(s.rest) +
                        ((((int64_t(p) * a.segs + seg) * a.Hk + oh) * seg_tiles + (q0 - s0) / QT) * slices + slice) * (2 * ZB * NQ * 256) + tid;
            const T *mine = rows(s.own, oh);
#pragma unroll
            for (int nq = 0; nq < NQ; ++nq) {
                const int t = qw + nq * 16 + lc, at = (t - diag) & 31, row = min(t, n - 1);
                const float w = __shfl(self[nq], at / 8 * 16 + lc, 64);
                float dot = 0.0f;
#pragma unroll
                for (int zb = 0; zb < ZB; ++zb) {
                    __builtin_amdgcn_sched_barrier(0);      // not all the rows' loads at once: registers
                    const int c = z0 + zb * 32 + lg * 8;
                    dt4 m[2], o[2];
                    eight_values(eight<EVEN>(mine + row * s.own.st, c, Zw, t < n), m[0], m[1]);
                    eight_values(eight<EVEN>(zr + row * s.z.st, c, Zw, t < n), o[0], o[1]);
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        dt4 &x = acc[zb][e][nq];
                        dt4 *r = rest + ((zb * 2 + e) * NQ + nq) * 256;
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            dot = fmaf(m[e][i], x[i], dot);
                            x[i] = fmaf(w, o[e][i], x[i]);
                        }
                        if (!begins) x += *r;
                        if (!ends) *r = x;
                    }
                }
                dot += __shfl_xor(dot, 16, 64);
                dot += __shfl_xor(dot, 32, 64);
                if (s.dot && lg == 0 && t < n) s.dot[((int64_t(slice) * a.P + p) * a.Hv + h) * a.T + t] = dot;
            }
            lds_barrier();       // G and the tiles are free
            if (!ends) continue;
        }
        if (CAUSAL && __builtin_amdgcn_readfirstlane(first[ZW]) < qw + 16 * NQ - s0) {
#pragma unroll
            for (int zb = 0; zb < ZB; ++zb)
#pragma unroll
                for (int e = 0; e < 2; ++e)
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const int from = first[zb * 32 + lg * 8 + e * 4 + r];
#pragma unroll
                        for (int nq = 0; nq < NQ; ++nq)
                            if (qw - s0 + nq * 16 + lc >= from) acc[zb][e][nq][r] = __builtin_nanf("");
                    }
        }
#pragma unroll
        for (int nq = 0; nq < NQ; ++nq) {
            const int t = qw + nq * 16 + lc;
#pragma unroll
            for (int zb = 0; zb < ZB; ++zb) {
                if (KEYS && back) {
                    acc[zb][0][nq] = -acc[zb][0][nq];
                    acc[zb][1][nq] = -acc[zb][1][nq];
                }
                put(t, zb, t < n ? acc[zb][0][nq] : dt4{}, t < n ? acc[zb][1][nq] : dt4{});
            }
        }
    }
}

template <typename T, int XP, int ZW, bool EVEN> __global__ __launch_bounds__(256, 2) void lin_attend_kernel(AttendArgs a) {
    lin_attend<T, XP, ZW, false, EVEN, true>(a, a.side[0], blockIdx.x);
}
// A sequence of one segment: its readings and, by the workgroups from `attends` on, its end state. (One launch for two: of 200
// tokens of 4 heads of 64 x 64, 13.6 us and 9 one after the other.)
template <typename T, int XP, int ZW, bool EVEN> __global__ __launch_bounds__(256, 2) void lin_single_kernel(AttendArgs a, StateArgs s, int attends) {
    if (int(blockIdx.x) < attends) lin_attend<T, XP, ZW, false, EVEN, true>(a, a.side[0], blockIdx.x);
    else lin_state<T, XP, ZW, EVEN>(s, int(blockIdx.x) - attends);
}
// dq, dk and dv: `keys` workgroups for each of the first two, then those of dv, which fill the device where the others leave it (of
// 3 x 6 heads of 301 float32 tokens of 40 x 72: 36 us in one launch, 34 and 16 in two). The
// launch begins with workgroup `first`.
template <typename T, int KP, int VP, bool EVEN> __global__ __launch_bounds__(256, 2) void lin_grads_kernel(AttendArgs a, int keys, int first) {
    const int b = int(blockIdx.x) + first;
    if (b < 2 * keys) lin_attend<T, VP, lin_slice(KP), true, EVEN, false>(a, a.side[b < keys ? 0 : 1], b < keys ? b : b - keys);
    else lin_attend<T, KP, lin_slice(VP), false, EVEN, false>(a, a.side[2], b - 2 * keys);
}

// Workgroups of a side; sets `whole`.
template <typename C, bool KEYS> int64_t attend_blocks(AttendArgs &a, const AttendSide &s, int ZW) {
    // All tiles of a segment in one workgroup where that leaves two to a compute unit: it meets the segment's gates and the kernel's
    // arguments once (16 heads of 16384 tokens of 128 x 128, bfloat16: 120 us tile by tile, 111 so; 64 heads of 2048: 61 and 56).
    const int64_t slices = (s.z.width + ZW - 1) / ZW;
    if (!KEYS) a.whole = int64_t(a.P) * a.Hv * a.segs * slices >= 2 * kCus;
    const int64_t unit = slices * (!KEYS && a.whole ? 1 : a.seg_tokens / C::QT) * (KEYS ? 1 : a.Hv / a.Hk);
    const int64_t units = int64_t(a.P) * a.Hk * a.segs, xcds = lin_xcds(units);
    return (units + xcds - 1) / xcds * xcds * unit;
}
// single: the end states that go with the readings of one segment, or null.
template <typename T, int XP, int ZW, bool EVEN> hipError_t attend_go(const AttendArgs &a, const StateArgs *single, hipStream_t st) {
    using C = AttendCfg<T, XP, ZW, false, EVEN>;
    AttendArgs b = a;
    const int64_t blocks = attend_blocks<C, false>(b, a.side[0], ZW);
    if (single) {
        constexpr size_t other = StateCfg<T, XP, ZW, EVEN>::kLds;
        const int64_t states = (a.V + ZW - 1) / ZW * a.P * a.Hv;
        hipLaunchKernelGGL((lin_single_kernel<T, XP, ZW, EVEN>), dim3(unsigned(blocks + states)), dim3(256), C::kLds > other ? C::kLds : other, st, b, *single,
                           int(blocks));
    } else {
        hipLaunchKernelGGL((lin_attend_kernel<T, XP, ZW, EVEN>), dim3(unsigned(blocks)), dim3(256), C::kLds, st, b);
    }
    return hipGetLastError();
}
template <typename T, int KP, int VP, bool EVEN> constexpr size_t grads_lds() {
    constexpr size_t keys = AttendCfg<T, VP, lin_slice(KP), true, EVEN>::kLds, values = AttendCfg<T, KP, lin_slice(VP), false, EVEN>::kLds;
    static_assert(keys <= 80 * 1024 && values <= 80 * 1024, "two workgroups to a compute unit");
    return keys > values ? keys : values;
}
template <typename T, int KP, int VP, bool EVEN> hipError_t grads_go(const AttendArgs &a, hipStream_t st) {
    AttendArgs b = a;
    const int64_t keys = attend_blocks<AttendCfg<T, VP, lin_slice(KP), true, EVEN>, true>(b, a.side[0], lin_slice(KP));
    const int64_t values = attend_blocks<AttendCfg<T, KP, lin_slice(VP), false, EVEN>, false>(b, a.side[2], lin_slice(VP));
    const int64_t all = 2 * keys + values, most = 1 << 23;      // 2^32 threads to a launch
    for (int64_t first = 0; first < all; first += most)
        hipLaunchKernelGGL((lin_grads_kernel<T, KP, VP, EVEN>), dim3(unsigned(all - first < most ? all - first : most)), dim3(256),
                           (grads_lds<T, KP, VP, EVEN>()), st, b, int(keys), int(first));
    return hipGetLastError();
}

template <typename T> bool lin_even(int K, int V) { return K % int(16 / sizeof(T)) == 0 && V % int(16 / sizeof(T)) == 0; }
// f(KP or XP, VP or ZW, EVEN as constants) for the padded widths.
template <typename F> hipError_t for_width(int width, F f) {
    switch (width) {
        case 64: return f(std::integral_constant<int, 64>{});
        case 128: return f(std::integral_constant<int, 128>{});
        default: return f(std::integral_constant<int, 256>{});
    }
}
template <typename T> hipError_t attend(const AttendArgs &a, const StateArgs *single, hipStream_t st) {
    return for_width(lin_width(a.side[0].x.width), [&](auto xp) {
        constexpr int XP = decltype(xp)::value;
        const bool even = lin_even<T>(a.K, a.V);
        if (lin_slice(a.side[0].z.width) == 64) return even ? attend_go<T, XP, 64, true>(a, single, st) : attend_go<T, XP, 64, false>(a, single, st);
        return even ? attend_go<T, XP, 128, true>(a, single, st) : attend_go<T, XP, 128, false>(a, single, st);
    });
}
template <typename T> hipError_t attend_grads(const AttendArgs &a, hipStream_t st) {
    return for_width(lin_width(a.K), [&](auto kp) {
        return for_width(lin_width(a.V), [&](auto vp) {
            constexpr int KP = decltype(kp)::value, VP = decltype(vp)::value;
            return lin_even<T>(a.K, a.V) ? grads_go<T, KP, VP, true>(a, st) : grads_go<T, KP, VP, false>(a, st);
        });
    });
}

template <typename F> hipError_t set_lds(F kernel, size_t bytes) {
    return hipFuncSetAttribute(reinterpret_cast<const void *>(kernel), hipFuncAttributeMaxDynamicSharedMemorySize, int(bytes));
}
template <typename T, int XP, int ZW> hipError_t attend_attr() {
    constexpr size_t bytes = AttendCfg<T, XP, ZW, false, true>::kLds, other = StateCfg<T, XP, ZW, true>::kLds, both = bytes > other ? bytes : other;
    static_assert(both <= 80 * 1024, "two workgroups to a compute unit");
    hipError_t e = set_lds(&lin_attend_kernel<T, XP, ZW, true>, bytes);
    if (e == hipSuccess) e = set_lds(&lin_attend_kernel<T, XP, ZW, false>, bytes);
    if (e == hipSuccess) e = set_lds(&lin_single_kernel<T, XP, ZW, true>, both);
    return e == hipSuccess ? set_lds(&lin_single_kernel<T, XP, ZW, false>, both) : e;
}
template <typename T> hipError_t attend_prepare() {
    hipError_t e = hipSuccess;
    for (int width : {64, 128, 256})
        if (e == hipSuccess)
            e = for_width(width, [](auto xp) {
                const hipError_t r = attend_attr<T, decltype(xp)::value, 64>();
                return r == hipSuccess ? attend_attr<T, decltype(xp)::value, 128>() : r;
            });
    return e;
}
template <typename T> hipError_t grads_prepare() {
    hipError_t e = hipSuccess;
    for (int k : {64, 128, 256})
        for (int v : {64, 128, 256})
            if (e == hipSuccess)
                e = for_width(k, [&](auto kp) {
                    return for_width(v, [&](auto vp) {
                        constexpr int KP = decltype(kp)::value, VP = decltype(vp)::value;
                        const hipError_t r = set_lds(&lin_grads_kernel<T, KP, VP, true>, grads_lds<T, KP, VP, true>());
                        return r == hipSuccess ? set_lds(&lin_grads_kernel<T, KP, VP, false>, grads_lds<T, KP, VP, false>()) : r;
                    });
                });
    return e;
}

// One translation unit for each element type and kind (linear_attend_*.hip).
hipError_t attend_bf16(const AttendArgs &a, const StateArgs *single, hipStream_t st);
hipError_t attend_f32(const AttendArgs &a, const StateArgs *single, hipStream_t st);
hipError_t attend_grads_bf16(const AttendArgs &a, hipStream_t st);
hipError_t attend_grads_f32(const AttendArgs &a, hipStream_t st);
hipError_t attend_prepare_bf16();
hipError_t attend_prepare_f32();
hipError_t grads_prepare_bf16();
hipError_t grads_prepare_f32();

}  // namespace sdm
