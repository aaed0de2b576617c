// The chunked gated delta rule, backward.
//
// The forward's chunk quantities are computed again, or were kept (delta.hip: X, P, U and every chunk's
// start state S0). With dS1 the gradient of a chunk's end state:
//     dU = P^T do + e^{G_C - G} k dS1,   Y = X^T dU
//     dv = beta Y,   dbeta = Y . U / beta,   dA = -(beta Y) U^T,   dP = do U^T
//     dS0 = e^{G_C} dS1 + (scale e^G q)^T do - (e^G k)^T (beta Y)
//     dq = scale e^G (do S0^T) + (scale D dP) k
//     dk = -e^G (beta Y S0^T) + e^{G_C - G} (U dS1^T) + (scale D dP)^T q + (D dA) k + (D dA)^T k
// delta_back_kernel walks the chunks from the last, 16 columns of dS per wavefront, and keeps Y
// and dS1; delta_grad_kernel then does every chunk at once, a key head's value heads in order.
//
// The gradient of log-decay m gathers every product that exp(g_m) is a factor of: those of
// tokens i >= m with the start state (a_i), of the end state with tokens j < m (b_j), of the
// two states (c) and of pairs i >= m > j (M_ij = dP_ij P_ij + dA_ij A_ij):
//     dg_m = sum_{i >= m} a_i + sum_{j < m} b_j + c + sum_{i >= m > j} M_ij
// The last sum follows from row and column sums of M; these run in 64 bits, since they cancel.
//
// U / beta is the write error; where beta is (nearly) 0 the backward's own X and U are computed
// with beta 1e-20 instead, which changes no other result, so that it still is.
#include <type_traits>

#include "delta_walk.h"

namespace sdm {

namespace {

// dS from the last chunk to the first, as delta_state_kernel walks S. Bound like it by the one computing wavefront of a SIMD: 198
// matrix instructions (1.3 us) of a chunk's 5.3 (64 tokens of 128 x 128, bfloat16; 4 x 16 heads of 2048 tokens: 173 us); beside
// the walk's chain it writes dS1, Y and dv, 56 KB a chunk. Its 256 registers do not hold it all: 15 vector registers of that variant
// are spilled, 71 of float32's with head_dim above 128 (2 x 8 heads of 1024 tokens of 200 x 200: 299 us).
template <typename T, int C, int KP>
__global__ __launch_bounds__(kWalkThreads) void delta_back_kernel(DeltaArgs a, DeltaWs ws, DeltaGrads d) {
    constexpr int NI = kPieces<T>, KB = KP / 32, TB = C / 32, NTR = kTri<C>;
    using W = Walk<T, C, KP, true>;
    extern __shared__ __align__(16) unsigned char raw[];
    typename W::Lds *bufs = reinterpret_cast<typename W::Lds *>(raw);
    const int slices = (a.V + 63) / 64, VG = (a.V + 15) / 16;
    const int slice = BlockAt(blockIdx.x, slices, a.P * a.Hv, a.Hv / a.Hk).slice, ph = BlockAt(blockIdx.x, slices, a.P * a.Hv, a.Hv / a.Hk).ph;
    const int h = ph % a.Hv, p = ph / a.Hv, hk = h / (a.Hv / a.Hk);
    const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lc = lane & 15, lg = lane >> 4;
    const int cg = slice * 4 + (wv & 3), col = cg * 16 + lc;
    const bool in = col < a.V;
    const int n = delta_valid(a, p), Nc = (n + C - 1) / C;
    if (wv >= 4) {
        typename W::Bring w(a, ws, p, h, hk, ph, cg, d.go, n);
        w.run(bufs, Nc - 1, -1, Nc);
        return;
    }
    T *dv = static_cast<T *>(d.v) + (int64_t(p) * a.T * a.Hv + h) * a.V + col;
    const int64_t os = int64_t(a.Hv) * a.V;
    dt4 S[KB][2];
    load_state<KB>(S, d.gstate, ph, a.K, a.V, col);
    W::begin();
    Frag<3> fs[KB];
#pragma unroll
    for (int kb = 0; kb < KB; ++kb) fs[kb] = split<3>(S[kb][0], S[kb][1]);
    for (int c = Nc - 1, turn = 0; c >= 0; --c, ++turn) {
        const typename W::Lds &s = bufs[turn & (W::kBufs - 1)];
        const int t0 = c * C;
        const int64_t nc = int64_t(ph) * ws.Nt + c;
        save_blocks<KB>(ws.dS, nc, VG, cg, S);
        const Gates<C> &g = s.m.g;
        const int ln = fresh_lane();
        // The products in this order, each group's operands read ahead of the group before it: P^T do, k dS, half of
        // q^T do, X^T dU, the other half, k^T Y; the halves stand where dU and Y are being put together.
        Frag<3> ft[2][2];            // a block of P^T or X^T
        auto tri_of = [&](Frag<3>(&f)[2], const unsigned char *m) {
#pragma unroll
            for (int e = 0; e < 2; ++e) f[e] = read_cols<3>(m, NTR * kBlk, e, ln);
        };
        Frag<NI> A[2][TB][2];        // a column block of k
        auto rows_of = [&](Frag<NI>(&f)[TB][2], const unsigned char *m) {
#pragma unroll
            for (int tb = 0; tb < TB; ++tb)
#pragma unroll
                for (int e = 0; e < 2; ++e) f[tb][e] = read_rows<NI>(m + tb * KB * kBlk, W::kStride, e, ln);
        };
        Frag<NI> fk[2][KB];          // half of a row block of k^T or q^T
        auto cols_of = [&](Frag<NI>(&f)[KB], const unsigned char *m, int i) {
#pragma unroll
            for (int x = 0; x < KB; ++x) f[x] = read_cols<NI>(m + (i / 2 * KB + i % 2 * (KB / 2) + x / 2) * kBlk, W::kStride, x & 1, ln);
        };
        tri_of(ft[0], s.m.P[0][0]);
        dt4 o[TB][2], b[TB][2], eG[TB][2], eL[TB][2];
#pragma unroll
        for (int tb = 0; tb < TB; ++tb)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int t = tb * 32 + lg * 8 + e * 4;
                o[tb][e] = W::value(s, tb, e);
                if (!in) o[tb][e] = dt4{};
                b[tb][e] = *reinterpret_cast<const dt4 *>(g.beta + t);
                eG[tb][e] = *reinterpret_cast<const dt4 *>(g.eG + t);
                eL[tb][e] = *reinterpret_cast<const dt4 *>(g.eL + t);
            }
        const float last = g.last;
        Frag<NI> fo[TB];
#pragma unroll
        for (int tb = 0; tb < TB; ++tb) fo[tb] = split<NI>(o[tb][0], o[tb][1]);
        dt4 z[TB][2] = {}, x[TB][2] = {};
#pragma unroll
        for (int i = 0; i < NTR; ++i) {
            if (i + 1 < NTR) tri_of(ft[(i + 1) & 1], s.m.P[0][i + 1]);
            else rows_of(A[0], s.k[0][0][0]);
            lds_point();
            each_product<3, 3, NI>([&](int m, int l) {
#pragma unroll
                for (int e = 0; e < 2; ++e) z[i == 2][e] = mma1(ft[i & 1][e].p[m], fo[i > 0].p[l], z[i == 2][e]);
            });
            lds_point();
        }
#pragma unroll
        for (int i = 0; i < KB; ++i) {
            if (i + 1 < KB) rows_of(A[(i + 1) & 1], s.k[0][0][i + 1]);
            else cols_of(fk[0], s.q[0][0][0], 0);
            lds_point();
            each_product<3, NI, 3>([&](int m, int l) {
#pragma unroll
                for (int tb = 0; tb < TB; ++tb)
#pragma unroll
                    for (int e = 0; e < 2; ++e) x[tb][e] = mma1(A[i & 1][tb][e].p[m], fs[i].p[l], x[tb][e]);
            });
            lds_point();
        }
        Frag<3> fu[TB], fq[TB];
#pragma unroll
        for (int tb = 0; tb < TB; ++tb) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                x[tb][e] = eL[tb][e] * x[tb][e] + z[tb][e];
                o[tb][e] *= a.scale * eG[tb][e];
            }
            fu[tb] = split<3>(x[tb][0], x[tb][1]);
            fq[tb] = split<3>(o[tb][0], o[tb][1]);
        }
#pragma unroll
        for (int kb = 0; kb < KB; ++kb)
#pragma unroll
            for (int e = 0; e < 2; ++e) S[kb][e] *= last;
        auto add = [&](const Frag<NI>(&f)[KB], const Frag<3> &u, int i) {
            each_product<3, NI, 3>([&](int m, int l) {
#pragma unroll
                for (int x = 0; x < KB; ++x) {
                    dt4 &d = S[i % 2 * (KB / 2) + x / 2][x & 1];
                    d = mma1(f[x].p[m], u.p[l], d);
                }
            });
        };
        dt4 Y[TB][2] = {};
#pragma unroll
        for (int i = 0; i < TB; ++i) {
            if (i + 1 < TB) cols_of(fk[(i + 1) & 1], s.q[0][0][0], i + 1);
            else tri_of(ft[0], s.m.X[0][0]);
            lds_point();
            add(fk[i & 1], fq[i / 2], i);
            lds_point();
        }
#pragma unroll
        for (int i = 0; i < NTR; ++i) {
            if (i + 1 < NTR) tri_of(ft[(i + 1) & 1], s.m.X[0][i + 1]);
            else cols_of(fk[0], s.q[0][0][0], TB);
            lds_point();
            each_product<3, 3, 3>([&](int m, int l) {
#pragma unroll
                for (int e = 0; e < 2; ++e) Y[i == 2][e] = mma1(ft[i & 1][e].p[m], fu[i > 0].p[l], Y[i == 2][e]);
            });
            lds_point();
        }
        dt4 v[TB][2];
        Frag<3> fy[TB];
#pragma unroll
        for (int tb = 0; tb < TB; ++tb) {
            dt4 y[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                v[tb][e] = b[tb][e] * Y[tb][e];
                y[e] = -eG[tb][e] * v[tb][e];
            }
            fy[tb] = split<3>(y[0], y[1]);
        }
#pragma unroll
        for (int i = 0; i < TB; ++i) {
            if (i + 1 < TB) cols_of(fk[(i + 1) & 1], s.q[0][0][0], TB + i + 1);
            else cols_of(fk[(i + 1) & 1], s.k[0][0][0], 0);
            lds_point();
            add(fk[i & 1], fq[(TB + i) / 2], TB + i);
            lds_point();
        }
        save_blocks<TB>(ws.Y, nc, VG, cg, Y);
        put_columns<T, TB>(dv + t0 * os, os, n - t0, in, v);
#pragma unroll
        for (int i = 0; i < 2 * TB; ++i) {
            if (i + 1 < 2 * TB) cols_of(fk[(TB + i + 1) & 1], s.k[0][0][0], i + 1);
            lds_point();
            add(fk[(TB + i) & 1], fy[i / 2], i);
            lds_point();
        }
#pragma unroll
        for (int kb = 0; kb < KB; ++kb) fs[kb] = split<3>(S[kb][0], S[kb][1]);
        W::turn();
    }
    for (int t = n + lg; t < a.T; t += 4)
        if (in) dv[t * os] = from_f32<T>(0.0f);
    store_state<KB>(S, d.state, ph, a.K, a.V, col);
}

// Every chunk of a key head at once, its value heads in order. The gradients of q and k are computed transposed (rows:
// head_dim, columns: tokens), so that a lane's accumulators are neighbours of an output row; U, Y, S and dS lie in
// LDS transposed too (rows: columns of V, as the workspace holds them). A head goes by in stages: V, 32 columns at a time,
// then q and k. Four wavefronts bring a stage's operands, cut into pieces, from memory to LDS while eight work on the stage before:
// 16 tokens by a share of head_dim each.
constexpr int kGradThreads = 768;

template <typename T, int C, int KP> struct GradLds {
    static constexpr int NI = kPieces<T>, KB = KP / 32, TB = C / 32, KG = 8 / (C / 16);
    union Stage {
        struct {
            unsigned char go[NI][TB][kBlk], U[3][TB][kBlk], Y[3][TB][kBlk], S[3][KB][kBlk], dS[3][KB][kBlk];
        };
        struct {
            unsigned char k[NI][TB][KB][kBlk], q[NI][TB][KB][kBlk];
            unsigned char Mq[3][kTri<C>][kBlk], Ma[3][kTri<C>][kBlk];   // scale D dP and D dA, rows: token i
        };
    };
    struct Small {
        float ai[KG][C], bj[KG][C], ub[2][C];   // a_i, b_j, Y . U, in parts
        double row[TB][C], col[2 * TB][C];      // sums of M = dP P + dA A below the diagonal, by blocks of columns and tiles of rows
        double G[C];
        double cs[4];
        Gates<C> g;
    };
    static constexpr int kBufs = 2 * sizeof(Stage) + sizeof(Small) <= kDeltaMaxLds ? 2 : 1;
    Stage stage[kBufs];
    Small small;
};

// A workgroup's way through its chunks of key heads: stage vb of value head hh of chunk `task`, vb = nb for q and k. Chunks
// without a valid token have no stages.
template <int C> struct GradAt {
    const DeltaArgs &a;
    int Nt, group, nb, tasks, task, p, hk, c, live, hh, vb;
    __device__ __forceinline__ GradAt(const DeltaArgs &a, const DeltaWs &ws)
        : a(a), Nt(ws.Nt), group(a.Hv / a.Hk), nb(((a.V + 15) / 16 + 1) / 2), tasks(a.P * a.Hk * ws.Nt) {
        enter(blockIdx.x);
    }
    __device__ __forceinline__ void enter(int t) {
        hh = vb = 0;
        for (task = t; task < tasks; task += gridDim.x) {
            const int ph = task / Nt;
            c = task % Nt, hk = ph % a.Hk, p = ph / a.Hk;
            live = min(C, delta_valid(a, p) - c * C);
            if (live > 0) break;
        }
    }
    __device__ __forceinline__ bool more() const { return task < tasks; }
    __device__ __forceinline__ bool keys() const { return vb == nb; }
    __device__ __forceinline__ void next() {
        if (++vb <= nb) return;
        vb = 0;
        if (++hh == group) enter(task + gridDim.x);
    }
};

// The wavefronts that bring the operands.
template <typename T, int C, int KP> struct GradBring {
    using Lds = GradLds<T, C, KP>;
    using Stage = typename Lds::Stage;
    using At = GradAt<C>;
    static constexpr int NI = Lds::NI, KB = Lds::KB, TB = Lds::TB, kBufs = Lds::kBufs;
    static constexpr int OS = (C * 4 + 255) / 256, US = (TB * 128 + 255) / 256, SS = KB * 128 / 256, QS = C * KP / 8 / 256;
    const DeltaArgs &a;
    const DeltaWs &ws;
    const Rows &gr;
    int VG;
    // A stage on its way, as it was loaded: do, U, Y, S and dS, or k and q.
    static constexpr int OW = NI == 1 ? 1 : 2, U0 = OS * OW, Y0 = U0 + 2 * US, X0 = Y0 + 2 * US, Z0 = X0 + 2 * SS, RV = Z0 + 2 * SS;
    static constexpr int Q0 = QS * NI, RK = 2 * Q0;
    du4 r[RV > RK ? RV : RK];
    du4 gates;
    float g, ub[8];
    double cc;

    __device__ GradBring(const DeltaArgs &a, const DeltaWs &ws, const Rows &gr) : a(a), ws(ws), gr(gr), VG((a.V + 15) / 16) {}

    __device__ __forceinline__ void load(const At &w) {
        const int tid = threadIdx.x & 255, lane = tid & 63, p = w.p, hk = w.hk, h = hk * w.group + w.hh, live = w.live;
        const int64_t t0 = int64_t(w.c) * C, nc = (int64_t(p) * a.Hv + h) * ws.Nt + w.c;
        if (!w.keys()) {
            const int vg = w.vb * 2;
            const T *go = static_cast<const T *>(gr.data) + p * gr.sp + t0 * gr.st + h * gr.sh;
            // columns past V's end are read from its last ones, rows past the last valid token from that one: store clears them
#pragma unroll
            for (int j = 0; j < OS; ++j) {
                const int s = tid + 256 * j, e = vg * 16 + s % 4 * 8;
                const du4 *from = reinterpret_cast<const du4 *>(go + (min(s / 4, live - 1) * int(gr.st) + min(e, gr.width - 8)));
#pragma unroll
                for (int n = 0; n < OW; ++n) r[j * OW + n] = from[n];
            }
#pragma unroll
            for (int j = 0; j < US; ++j) {
                const int s = tid + 256 * j, cg = min(vg + s / (TB * 64), VG - 1), b = s / 64 % TB;
                const int64_t from = (((nc * VG + cg) * TB + b) * 64 + lane) * 8;
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    r[U0 + j * 2 + e] = *reinterpret_cast<const du4 *>(ws.U + from + e * 4);
                    r[Y0 + j * 2 + e] = *reinterpret_cast<const du4 *>(ws.Y + from + e * 4);
                }
            }
#pragma unroll
            for (int j = 0; j < SS; ++j) {
                const int s = tid + 256 * j, cg = min(vg + s / (KB * 64), VG - 1), b = s / 64 % KB;
                const int64_t from = (((nc * VG + cg) * KB + b) * 64 + lane) * 8;
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    r[X0 + j * 2 + e] = *reinterpret_cast<const du4 *>(ws.S + from + e * 4);
                    r[Z0 + j * 2 + e] = *reinterpret_cast<const du4 *>(ws.dS + from + e * 4);
                }
            }
        } else {
            const bf16 *kp = a.kk.data + p * a.kk.sp + hk * a.kk.sh + t0 * a.kk.st;
            const bf16 *qp = a.qq.data + p * a.qq.sp + hk * a.qq.sh + t0 * a.qq.st;
#pragma unroll
            for (int j = 0; j < QS; ++j) {
                const int s = tid + 256 * j, b = s / 128, t = min(b / KB * 32 + s % 128 / 4, live - 1), e = b % KB * 32 + s % 4 * 8;
#pragma unroll
                for (int n = 0; n < NI; ++n) {
                    r[j * NI + n] = *reinterpret_cast<const du4 *>(kp + n * a.kk.plane + (t * int(a.kk.st) + e));
                    r[Q0 + j * NI + n] = *reinterpret_cast<const du4 *>(qp + n * a.qq.plane + (t * int(a.qq.st) + e));
                }
            }
            g = lane < live && lane < C ? a.g[(p * int64_t(a.T) + t0 + lane) * a.Hv + h] : 0.0f;
            gates = reinterpret_cast<const du4 *>(&(reinterpret_cast<const ChunkMem<C> *>(ws.mats) + nc)->g)[lane];
        }
    }
    static __device__ __forceinline__ dt4 kept(du4 x, bool in) { return in ? __builtin_bit_cast(dt4, x) : dt4{}; }
    __device__ __forceinline__ void store(Lds &l, const At &w, int i) {
        const int tid = threadIdx.x & 255, lane = tid & 63, lc = lane & 15, lg = lane >> 4, wv = tid >> 6;
        Stage &s = l.stage[i & (kBufs - 1)];
        if (!w.keys()) {
            if (w.vb == 0) {
                cc = 0.0;
#pragma unroll
                for (int e = 0; e < 8; ++e) ub[e] = 0.0f;
            }
            const int vg = w.vb * 2;
#pragma unroll
            for (int j = 0; j < OS; ++j) {
                const int at = tid + 256 * j, t = at / 4, e = vg * 16 + at % 4 * 8;
                if (C * 4 % 256 && at >= C * 4) break;
                Frag<NI> f;
                if constexpr (NI == 1) f.p[0] = __builtin_bit_cast(db8, r[j]);
                else f = split<NI>(__builtin_bit_cast(dt4, r[j * 2]), __builtin_bit_cast(dt4, r[j * 2 + 1]));
                if (t >= w.live || e >= gr.width) clear(f);
#pragma unroll
                for (int n = 0; n < NI; ++n) *reinterpret_cast<db8 *>(s.go[n][t / 32] + block_at(t % 32, at % 4)) = f.p[n];
            }
#pragma unroll
            for (int j = 0; j < US; ++j) {       // US = 1: a thread keeps its tokens through all stages
                const int at = tid + 256 * j, cg = at / (TB * 64), b = at / 64 % TB, row = cg * 16 + lc;
                if (TB * 128 % 256 && at >= TB * 128) break;
                const bool in = vg + cg < VG;
                const dt4 u[2] = {kept(r[U0 + j * 2], in), kept(r[U0 + j * 2 + 1], in)}, y[2] = {kept(r[Y0 + j * 2], in), kept(r[Y0 + j * 2 + 1], in)};
#pragma unroll
                for (int e = 0; e < 8; ++e) ub[e] = fmaf(u[e / 4][e % 4], y[e / 4][e % 4], ub[e]);
                const Frag<3> fu = split<3>(u[0], u[1]), fy = split<3>(y[0], y[1]);
#pragma unroll
                for (int n = 0; n < 3; ++n) {
                    *reinterpret_cast<db8 *>(s.U[n][b] + block_at(row, lg)) = fu.p[n];
                    *reinterpret_cast<db8 *>(s.Y[n][b] + block_at(row, lg)) = fy.p[n];
                }
            }
#pragma unroll
            for (int j = 0; j < SS; ++j) {
                const int at = tid + 256 * j, cg = at / (KB * 64), b = at / 64 % KB, row = cg * 16 + lc;
                const bool in = vg + cg < VG;
                const dt4 x[2] = {kept(r[X0 + j * 2], in), kept(r[X0 + j * 2 + 1], in)}, z[2] = {kept(r[Z0 + j * 2], in), kept(r[Z0 + j * 2 + 1], in)};
                float m = 0.0f;
#pragma unroll
                for (int e = 0; e < 8; ++e) m = fmaf(x[e / 4][e % 4], z[e / 4][e % 4], m);
                cc += double(m);
                const Frag<3> fx = split<3>(x[0], x[1]), fz = split<3>(z[0], z[1]);
#pragma unroll
                for (int n = 0; n < 3; ++n) {
                    *reinterpret_cast<db8 *>(s.S[n][b] + block_at(row, lg)) = fx.p[n];
                    *reinterpret_cast<db8 *>(s.dS[n][b] + block_at(row, lg)) = fz.p[n];
                }
            }
            return;
        }
#pragma unroll
        for (int j = 0; j < QS; ++j) {
            const int at = tid + 256 * j, to = at / 128 * kBlk + block_at(at % 128 / 4, at % 4);
            const bool in = at / 128 / KB * 32 + at % 128 / 4 < w.live;
#pragma unroll
            for (int n = 0; n < NI; ++n) {
                *reinterpret_cast<du4 *>(&s.k[n][0][0][0] + to) = in ? r[j * NI + n] : du4{};
                *reinterpret_cast<du4 *>(&s.q[n][0][0][0] + to) = in ? r[Q0 + j * NI + n] : du4{};
            }
        }
        // Y . U of each token: over the 16 columns of a lane group, in two column groups; S . dS
        if (tid < TB * 128) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
#pragma unroll
                for (int m = 8; m > 0; m >>= 1) ub[e] += __shfl_xor(ub[e], m, 64);
                if (lc == 0) l.small.ub[tid / (TB * 64)][tid / 64 % TB * 32 + lg * 8 + e] = ub[e];
            }
        }
#pragma unroll
        for (int m = 32; m > 0; m >>= 1) cc += __shfl_xor(cc, m, 64);
        if (lane == 0) l.small.cs[wv] = cc;
        if (wv == 0) {
            const double G = chunk_G<C>(g);
            if (lane < C) l.small.G[lane] = G;
        }
        if (wv == 1) reinterpret_cast<du4 *>(&l.small.g)[lane] = gates;
    }
    __device__ __forceinline__ void run(Lds &l) {
        At at(a, ws), sent = at, put = at;      // the stage being worked on, and the next to load and to store
        if (!at.more()) return;
        load(sent);
        sent.next();
        store(l, put, 0);
        put.next();
        if (sent.more()) {
            load(sent);
            sent.next();
        }
        lds_barrier();
        auto ahead = [&](int i) {
            if (put.more()) {
                store(l, put, i + 1);
                put.next();
            }
            if (sent.more()) {
                load(sent);
                sent.next();
            }
        };
        for (int i = 0; at.more(); ++i, at.next()) {
            if constexpr (kBufs == 2) ahead(i);
            if (at.keys()) lds_barrier();    // the working wavefronts' own
            lds_barrier();
            if constexpr (kBufs == 1) {
                ahead(i);
                lds_barrier();
            }
        }
    }
};

// Sum over the 16 lanes of a row, by moves within the row.
__device__ __forceinline__ double lanes16(double x) {
    auto add = [&](auto ctrl) {
        const uint64_t u = __builtin_bit_cast(uint64_t, x);
        const uint32_t lo = __builtin_amdgcn_update_dpp(0u, uint32_t(u), decltype(ctrl)::value, 0xF, 0xF, false);
        const uint32_t hi = __builtin_amdgcn_update_dpp(0u, uint32_t(u >> 32), decltype(ctrl)::value, 0xF, 0xF, false);
        x += __builtin_bit_cast(double, uint64_t(hi) << 32 | lo);
    };
    add(std::integral_constant<int, 0xB1>{});    // quad_perm 1, 0, 3, 2
    add(std::integral_constant<int, 0x4E>{});    // quad_perm 2, 3, 0, 1
    add(std::integral_constant<int, 0x141>{});   // row_half_mirror
    add(std::integral_constant<int, 0x140>{});   // row_mirror
    return x;
}

// The value heads' shares of dq and dk meet in accumulators: no atomics, one rounding. One workgroup per compute unit walks its
// share of the chunks. Bound by the memory it reads, S0, dS1, U and Y in float32: 0.51 GB in and 0.06 out (by counters) for 4 x 16
// heads of 2048 tokens of 128 x 128 in 215 us, 2.7 TB/s on the whole: near the copy's rate while a chunk's states come in, well under
// it through the products with q and k between them.
template <typename T, int C, int KP>
__global__ __launch_bounds__(kGradThreads) void delta_grad_kernel(DeltaArgs a, DeltaWs ws, DeltaGrads d) {
    using Lds = GradLds<T, C, KP>;
    constexpr int NI = kPieces<T>, KB = KP / 32, TB = C / 32, NT = C / 16;
    constexpr int KG = Lds::KG, KW = KB * 2 / KG;   // wavefronts on the same tokens, their share of head_dim in 16-row tiles
    constexpr int kStride = TB * KB * kBlk;
    extern __shared__ __align__(16) unsigned char raw[];
    Lds &l = *reinterpret_cast<Lds *>(raw);
    typename Lds::Small &sm = l.small;
    const int tid = threadIdx.x, lane = tid & 63, wv = __builtin_amdgcn_readfirstlane(tid >> 6);
    if (wv >= 8) {
        GradBring<T, C, KP> bring(a, ws, d.go);
        bring.run(l);
        return;
    }
    const int tile = wv % NT, tb = tile / 2, ta = tile % 2, part = wv / NT, kt0 = part * KW;   // this wavefront's tokens and tiles of dq, dk
    dt4 aq[KW] = {}, ak[KW] = {};
    int stage = 0;
    auto turn = [&]() {
        lds_barrier();
        if constexpr (Lds::kBufs == 1) lds_barrier();
        ++stage;
    };
    GradAt<C> at(a, ws);
    if (at.more()) lds_barrier();
    const int nb = at.nb;
    while (at.more()) {
        const int ln = fresh_lane();
        const int p = at.p, hk = at.hk, t0 = at.c * C, live = at.live, h = hk * at.group + at.hh;
        // dP and dA (transposed: columns i, rows j): tile pe of the columns of row block bi, both row tiles of column block bj
        const int pb = wv / 2, pe = wv & 1, bi = pb > 0, bj = pb == 2;
        const bool pairs = pb < kTri<C>;
        dt4 dP[2] = {}, dA[2] = {}, oS[KW] = {}, yS[KW] = {}, uS[KW] = {};
        for (int vb = 0; vb < nb; ++vb) {
            const typename Lds::Stage &s = l.stage[stage & (Lds::kBufs - 1)];
            Frag<3> fs, fd;     // a tile of S, a tile of dS: one is read while the other's products run
            const Frag<NI> fo = read_rows<NI>(s.go[0][tb], TB * kBlk, ta, ln);
            const Frag<3> fy = read_cols<3>(s.Y[0][tb], TB * kBlk, ta, ln);
            fs = read_cols<3>(s.S[0][kt0 / 2], KB * kBlk, kt0 & 1, ln);
            const Frag<3> fu = read_cols<3>(s.U[0][tb], TB * kBlk, ta, ln);
#pragma unroll
            for (int j = 0; j < KW; ++j) {
                const int t = kt0 + j;
                fd = read_cols<3>(s.dS[0][t / 2], KB * kBlk, t & 1, ln);
                lds_point();
                oS[j] = mma<3>(fs, fo, oS[j]);
                yS[j] = mma<3>(fs, fy, yS[j]);
                lds_point();
                if (j + 1 < KW) fs = read_cols<3>(s.S[0][(t + 1) / 2], KB * kBlk, (t + 1) & 1, ln);
                lds_point();
                uS[j] = mma<3>(fd, fu, uS[j]);
                lds_point();
            }
            if (pairs) {
                const Frag<NI> po = read_rows<NI>(s.go[0][bi], TB * kBlk, pe, ln);
                const Frag<3> py = read_cols<3>(s.Y[0][bi], TB * kBlk, pe, ln);
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    const Frag<3> pu = read_cols<3>(s.U[0][bj], TB * kBlk, x, ln);
                    dP[x] = mma<3>(pu, po, dP[x]);
                    dA[x] = mma<3>(pu, py, dA[x]);
                }
            }
            turn();
        }
        typename Lds::Stage &s = l.stage[stage & (Lds::kBufs - 1)];
        const int lp = fresh_lane(), lc = lp & 15, lg = lp >> 4, tok = tb * 32 + block_row(lc, ta);    // the lane's token
        // D, P and A again, and the weights of k and q in the gradients (accumulators: rows j, columns i)
        if (pairs) {
            dt4 kk[2] = {}, qk[2] = {};
#pragma unroll
            for (int x = 0; x < KB; ++x) {
                const Frag<NI> fk = read_rows<NI>(s.k[0][bi][x], kStride, pe, lp), fq = read_rows<NI>(s.q[0][bi][x], kStride, pe, lp);
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                    const Frag<NI> f = read_rows<NI>(s.k[0][bj][x], kStride, y, lp);
                    kk[y] = mma<3>(f, fk, kk[y]);
                    qk[y] = mma<3>(f, fq, qk[y]);
                }
            }
            const int i = bi * 32 + block_row(lc, pe);
            const double Gi = sm.G[i];
            const float beta = sm.g.beta[i];
            dt4 wq[2], wa[2];
            double row = 0.0, cols[8];
#pragma unroll
            for (int y = 0; y < 2; ++y)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int jj = bj * 32 + lg * 8 + y * 4 + r;
                    const float D = i >= jj ? exp2_of(Gi - sm.G[jj]) : 0.0f;
                    wq[y][r] = i >= jj ? a.scale * (D * dP[y][r]) : 0.0f;
                    wa[y][r] = i > jj ? -beta * (D * dA[y][r]) : 0.0f;
                    const double m = i > jj ? double(fmaf(wq[y][r], qk[y][r], wa[y][r] * kk[y][r])) : 0.0;
                    row += m;
                    cols[y * 4 + r] = m;
                }
            row += __shfl_xor(row, 16, 64);
            row += __shfl_xor(row, 32, 64);
            if (lg == 0) sm.row[bj][i] = row;
#pragma unroll
            for (int r = 0; r < 8; ++r) cols[r] = lanes16(cols[r]);
            if (lc == 0) {
#pragma unroll
                for (int r = 0; r < 8; ++r) sm.col[bi * 2 + pe][bj * 32 + lg * 8 + r] = cols[r];
            }
            // a lane holds eight neighbours j of row i
            const Frag<3> fq = split<3>(wq[0], wq[1]), fa = split<3>(wa[0], wa[1]);
#pragma unroll
            for (int n = 0; n < 3; ++n) {
                *reinterpret_cast<db8 *>(s.Mq[n][pb] + block_at(block_row(lc, pe), lg)) = fq.p[n];
                *reinterpret_cast<db8 *>(s.Ma[n][pb] + block_at(block_row(lc, pe), lg)) = fa.p[n];
            }
        }
        // the states' part of dq and dk, and its products with q and k
        {
            const float eG = sm.g.eG[tok], eL = sm.g.eL[tok], xo = a.scale * eG, xy = -(sm.g.beta[tok] * eG);
            float ai = 0.0f, bj_ = 0.0f;
#pragma unroll
            for (int j = 0; j < KW; ++j) {
                const int t = kt0 + j;
                dt4 k{}, q{};
#pragma unroll
                for (int n = NI - 1; n >= 0; --n) {
                    const int at = n * kStride + (tb * KB + t / 2) * kBlk + block_at(tok % 32, lg) + (t & 1) * 8;
                    typedef uint32_t u2 __attribute__((ext_vector_type(2)));
                    const u2 kw = *reinterpret_cast<const u2 *>(&s.k[0][0][0][0] + at), qw = *reinterpret_cast<const u2 *>(&s.q[0][0][0][0] + at);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int sh = e & 1 ? 0 : 16;
                        k[e] += __uint_as_float((kw[e / 2] << sh) & 0xFFFF0000u);
                        q[e] += __uint_as_float((qw[e / 2] << sh) & 0xFFFF0000u);
                    }
                }
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const float x = xo * oS[j][r], y = xy * yS[j][r], z = eL * uS[j][r];
                    ai += fmaf(x, q[r], y * k[r]);
                    bj_ = fmaf(z, k[r], bj_);
                    aq[j][r] += x;
                    ak[j][r] += y + z;
                }
            }
            ai += __shfl_xor(ai, 16, 64);
            bj_ += __shfl_xor(bj_, 16, 64);
            ai += __shfl_xor(ai, 32, 64);
            bj_ += __shfl_xor(bj_, 32, 64);
            if (lg == 0) {
                sm.ai[part][tok] = ai;
                sm.bj[part][tok] = bj_;
            }
        }
        lds_barrier();
        // the pairs' part: the tokens as i (depth j up to them) and as j (depth i from them on)
#pragma unroll
        for (int x = 0; x < TB; ++x) {
            if (x <= tb) {
                const Frag<3> mq = read_rows<3>(s.Mq[0][tb + x], kTri<C> * kBlk, ta, lp), ma = read_rows<3>(s.Ma[0][tb + x], kTri<C> * kBlk, ta, lp);
#pragma unroll
                for (int j = 0; j < KW; ++j) {
                    const int t = kt0 + j;
                    const Frag<NI> k = read_cols<NI>(s.k[0][x][t / 2], kStride, t & 1, lp);
                    aq[j] = mma<3>(k, mq, aq[j]);
                    ak[j] = mma<3>(k, ma, ak[j]);
                }
            }
            if (x >= tb) {
                const Frag<3> mq = read_cols<3>(s.Mq[0][tb + x], kTri<C> * kBlk, ta, lp), ma = read_cols<3>(s.Ma[0][tb + x], kTri<C> * kBlk, ta, lp);
#pragma unroll
                for (int j = 0; j < KW; ++j) {
                    const int t = kt0 + j;
                    ak[j] = mma<3>(read_cols<NI>(s.q[0][x][t / 2], kStride, t & 1, lp), mq, ak[j]);
                    ak[j] = mma<3>(read_cols<NI>(s.k[0][x][t / 2], kStride, t & 1, lp), ma, ak[j]);
                }
            }
        }
        // dg: suffix sums of a_i, prefix sums of b_j and of the pairs begun less those ended, a token per lane
        if (wv == 0) {
            double suf = 0.0, pre = 0.0;
            if (lane < C) {
#pragma unroll
                for (int n = 0; n < KG; ++n) {
                    suf += double(sm.ai[n][lane]);
                    pre += double(sm.bj[n][lane]);
                }
#pragma unroll
                for (int n = 0; n < TB; ++n)
                    if (n <= lane / 32) pre -= sm.row[n][lane];
#pragma unroll
                for (int n = 0; n < 2 * TB; ++n)
                    if (n / 2 >= lane / 32) pre += sm.col[n][lane];
            }
            const double own = pre;
#pragma unroll
            for (int m = 1; m < C; m <<= 1) {
                const double x = __shfl_down(suf, m, 64), y = __shfl_up(pre, m, 64);
                if (lane + m < C) suf += x;
                if (lane >= m) pre += y;
            }
            if (lane < live) {
                const double x = double(sm.g.last) * (sm.cs[0] + sm.cs[1] + sm.cs[2] + sm.cs[3]) + suf + (pre - own);
                const int64_t at = (int64_t(p) * a.T + t0 + lane) * a.Hv + h;
                d.g[at] = float(x);
                d.beta[at] = (sm.ub[0][lane] + sm.ub[1][lane]) / delta_beta_safe(sm.g.beta[lane]);
            }
        }
        const bool last = at.hh + 1 == at.group;
        at.vb = nb;
        at.next();
        if (last) {
            if (tok < live) {
#pragma unroll
                for (int j = 0; j < KW; ++j) {
                    const int t = kt0 + j, e0 = t / 2 * 32 + lg * 8 + (t & 1) * 4;
                    if (e0 >= a.K) continue;
                    const int64_t to = ((int64_t(p) * a.T + t0 + tok) * a.Hk + hk) * a.K + e0;
                    put_four(static_cast<T *>(d.q) + to, a.K - e0, aq[j]);
                    put_four(static_cast<T *>(d.k) + to, a.K - e0, ak[j]);
                }
            }
#pragma unroll
            for (int j = 0; j < KW; ++j) aq[j] = ak[j] = dt4{};
        }
        turn();
    }
    // padding tokens have gradients of 0
    const int tasks = a.P * a.Hk * ws.Nt, group = a.Hv / a.Hk;
    for (int task = blockIdx.x; task < tasks; task += gridDim.x) {
        const int ph = task / ws.Nt, t0 = task % ws.Nt * C, hk = ph % a.Hk, p = ph / a.Hk;
        const int from = max(0, min(C, delta_valid(a, p) - t0)), rows = min(C, a.T - t0);
        for (int i = from * group + tid; i < rows * group; i += 512) {
            const int64_t to = (int64_t(p) * a.T + t0 + i / group) * a.Hv + hk * group + i % group;
            d.g[to] = d.beta[to] = 0.0f;
        }
        for (int i = from * a.K + tid; i < rows * a.K; i += 512) {
            const int64_t to = ((int64_t(p) * a.T + t0 + i / a.K) * a.Hk + hk) * a.K + i % a.K;
            static_cast<T *>(d.q)[to] = static_cast<T *>(d.k)[to] = from_f32<T>(0.0f);
        }
    }
}

template <typename T, int C, int KP>
hipError_t bwd_go(const DeltaArgs &a, const DeltaWs &ws, const DeltaGrads &d, hipStream_t st) {
    hipLaunchKernelGGL((delta_back_kernel<T, C, KP>), dim3(unsigned(int64_t(a.P) * a.Hv * ((a.V + 63) / 64))), dim3(kWalkThreads),
                       (Walk<T, C, KP, true>::kLds), st, a, ws, d);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || ws.Nt == 0) return e;
    const int64_t tasks = int64_t(a.P) * a.Hk * ws.Nt;   // a compute unit holds one workgroup: more would start cold
    hipLaunchKernelGGL((delta_grad_kernel<T, C, KP>), dim3(unsigned(tasks < kCus ? tasks : kCus)), dim3(kGradThreads),
                       sizeof(GradLds<T, C, KP>), st, a, ws, d);
    return hipGetLastError();
}
template <typename T>
hipError_t bwd_pick(const DeltaArgs &a, const DeltaWs &ws, const DeltaGrads &d, hipStream_t st) {
    switch (delta_kp(a.K)) {
        case 64: return bwd_go<T, kChunk<T>, 64>(a, ws, d, st);
        case 128: return bwd_go<T, kChunk<T>, 128>(a, ws, d, st);
        default: return bwd_go<T, 32, 256>(a, ws, d, st);
    }
}
template <typename T, int C, int KP> hipError_t bwd_attr() {
    constexpr size_t lw = Walk<T, C, KP, true>::kLds, lg = sizeof(GradLds<T, C, KP>);
    static_assert(lw <= kDeltaMaxLds && lg <= kDeltaMaxLds, "LDS of a workgroup");
    const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void *>(&delta_back_kernel<T, C, KP>),
                                             hipFuncAttributeMaxDynamicSharedMemorySize, lw);
    return e != hipSuccess ? e : hipFuncSetAttribute(reinterpret_cast<const void *>(&delta_grad_kernel<T, C, KP>),
                                                     hipFuncAttributeMaxDynamicSharedMemorySize, lg);
}
template <typename T> hipError_t bwd_attrs() {
    hipError_t e = bwd_attr<T, kChunk<T>, 64>();
    if (e == hipSuccess) e = bwd_attr<T, kChunk<T>, 128>();
    if (e == hipSuccess) e = bwd_attr<T, 32, 256>();
    return e;
}

}  // namespace

hipError_t delta_bwd_prepare() {
    const hipError_t e = bwd_attrs<float>();
    return e == hipSuccess ? bwd_attrs<bf16>() : e;
}

hipError_t launch_delta_bwd(const DeltaArgs &a, const DeltaWs &ws, const DeltaGrads &d, bool is_bf16, bool kept, hipStream_t st) {
    if (!kept) {
        const hipError_t e = launch_delta_fwd(a, ws, is_bf16, false, st);
        if (e != hipSuccess) return e;
    }
    return is_bf16 ? bwd_pick<bf16>(a, ws, d, st) : bwd_pick<float>(a, ws, d, st);
}

}  // namespace sdm
