// The chunked gated delta rule, backward.
//
// The forward's chunk quantities are computed again (delta.hip keeps U and every chunk's start
// state S0). With dS1 the gradient of a chunk's end state:
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
#include "delta_walk.h"

namespace sdm {

namespace {

template <typename T, int C, int KP>
__global__ __launch_bounds__(kWalkThreads) void delta_back_kernel(DeltaArgs a, DeltaWs ws, DeltaGrads d) {
    constexpr int NI = kPieces<T>, KB = KP / 32, TB = C / 32, NTR = kTri<C>;
    using W = Walk<T, C, KP, 3, true>;
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
        // The products in this order, each group's operands read ahead of the group before it: P^T do, k dS, half of
        // q^T do, X^T dU, the other half, k^T Y; the halves stand where dU and Y are being put together.
        Frag<3> ft[2][2];            // a block of P^T or X^T
        auto tri_of = [&](Frag<3>(&f)[2], const unsigned char *m) {
#pragma unroll
            for (int e = 0; e < 2; ++e) f[e] = read_cols<3>(m, NTR * kBlk, e);
        };
        Frag<NI> A[2][TB][2];        // a column block of k
        auto rows_of = [&](Frag<NI>(&f)[TB][2], const unsigned char *m) {
#pragma unroll
            for (int tb = 0; tb < TB; ++tb)
#pragma unroll
                for (int e = 0; e < 2; ++e) f[tb][e] = read_rows<NI>(m + tb * KB * kBlk, W::kStride, e);
        };
        Frag<NI> fk[2][KB];          // half of a row block of k^T or q^T
        auto cols_of = [&](Frag<NI>(&f)[KB], const unsigned char *m, int i) {
#pragma unroll
            for (int x = 0; x < KB; ++x) f[x] = read_cols<NI>(m + (i / 2 * KB + i % 2 * (KB / 2) + x / 2) * kBlk, W::kStride, x & 1);
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

// Every chunk of a key head at once. The gradients of q and k are computed transposed (rows:
// head_dim, columns: tokens), so that a lane's accumulators are eight neighbours of an output row;
// U, Y, S and dS lie in LDS transposed too (rows: columns of V, as the workspace holds them). V is
// taken 32 columns at a time.
template <typename T, int C, int KP> struct GradLds {
    static constexpr int NI = kPieces<T>, KB = KP / 32, TB = C / 32, NM = NI == 1 ? 2 : 3;
    union {
        struct {
            unsigned char go[NI][TB][kBlk], U[3][TB][kBlk], Y[3][TB][kBlk], S[3][KB][kBlk], dS[3][KB][kBlk];
        };
        struct {
            unsigned char k[NI][TB][KB][kBlk], q[NI][TB][KB][kBlk];
            unsigned char Mq[NM][kTri<C>][kBlk], Ma[NM][kTri<C>][kBlk];   // scale D dP and D dA, rows: token i
            float M[C * (C + 1)];                                        // dP P + dA A below the diagonal
        };
    };
    float ai[2][C], bj[2][C], ub[2][C];   // a_i, b_j, Y . U, in two parts
    double row[C], colm[C], G[C];
    double cs[4];
    Gates<C> g;
};

template <typename T, int C, int KP>
__global__ __launch_bounds__(256) void delta_grad_kernel(DeltaArgs a, DeltaWs ws, DeltaGrads d) {
    using Lds = GradLds<T, C, KP>;
    constexpr int NI = kPieces<T>, KB = KP / 32, TB = C / 32, NT = C / 16, NM = Lds::NM;
    constexpr int KG = 4 / NT, KW = KB / KG;        // wavefronts on the same tokens, their share of head_dim's blocks
    constexpr int NJ = (kTri<C> * 2 + 3) / 4;       // tiles of pairs per wavefront
    constexpr int kStride = TB * KB * kBlk;
    extern __shared__ __align__(16) unsigned char raw[];
    Lds &s = *reinterpret_cast<Lds *>(raw);
    const int group = a.Hv / a.Hk, VG = (a.V + 15) / 16;
    const int c = int(blockIdx.x % ws.Nt), ph = int(blockIdx.x / ws.Nt), hk = ph % a.Hk, p = ph / a.Hk;
    const int t0 = c * C, live = max(0, min(C, delta_valid(a, p) - t0));
    const int tid = threadIdx.x, lane = tid & 63, wv = tid >> 6, lc = lane & 15, lg = lane >> 4;
    const int tb = wv % NT / 2, ta = wv % 2, kb0 = wv / NT * KW;     // this wavefront's tokens and blocks of dq, dk
    const int tok = tb * 32 + block_row(lc, ta);                    // the lane's token
    const Rows &gr = d.go;
    dt4 aq[KW][2] = {}, ak[KW][2] = {};
    for (int hh = 0; live > 0 && hh < group; ++hh) {
        const int h = hk * group + hh;
        const int64_t nc = (int64_t(p) * a.Hv + h) * ws.Nt + c;
        const T *go = static_cast<const T *>(gr.data) + p * gr.sp + t0 * gr.st + h * gr.sh;
        const ChunkMem<C, 3> *mats = reinterpret_cast<const ChunkMem<C, 3> *>(ws.mats) + nc;
        if (tid < int(sizeof(Gates<C>) / 4)) reinterpret_cast<float *>(&s.g)[tid] = reinterpret_cast<const float *>(&mats->g)[tid];
        if (wv == 3) {
            const double G = chunk_G<C>(a, p, h, t0, live);
            if (lane < C) s.G[lane] = G;
        }
        // over V: dP, dA (transposed: columns i, rows j), S do^T, S Y^T, dS U^T
        dt4 dP[NJ][2] = {}, dA[NJ][2] = {}, oS[KW][2] = {}, yS[KW][2] = {}, uS[KW][2] = {};
        double cc = 0.0;
        float ub[8] = {};
        for (int vg = 0; vg < VG; vg += 2) {
            for (int i = tid; i < C * 4; i += 256) {      // eights of do
                const int t = i / 4, e = vg * 16 + i % 4 * 8;
                Frag<NI> f = load_pieces(go + min(t, live - 1) * gr.st + min(e, gr.width - 8));
                if (t >= live || e >= gr.width) clear(f);
#pragma unroll
                for (int n = 0; n < NI; ++n) *reinterpret_cast<db8 *>(s.go[n][t / 32] + block_at(t % 32, i % 4)) = f.p[n];
            }
            for (int i = tid; i < TB * 128; i += 256) {   // eights of tokens of U and Y: one per thread
                const int cg = i / (TB * 64), b = i / 64 % TB, row = cg * 16 + lc;
                dt4 u[2] = {}, y[2] = {};
                if (vg + cg < VG) {
                    const int64_t at = (((nc * VG + vg + cg) * TB + b) * 64 + lane) * 8;
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        u[e] = *reinterpret_cast<const dt4 *>(ws.U + at + e * 4);
                        y[e] = *reinterpret_cast<const dt4 *>(ws.Y + at + e * 4);
                    }
                }
#pragma unroll
                for (int e = 0; e < 8; ++e) ub[e] = fmaf(u[e / 4][e % 4], y[e / 4][e % 4], ub[e]);
                const Frag<3> fu = split<3>(u[0], u[1]), fy = split<3>(y[0], y[1]);
#pragma unroll
                for (int n = 0; n < 3; ++n) {
                    *reinterpret_cast<db8 *>(s.U[n][b] + block_at(row, lg)) = fu.p[n];
                    *reinterpret_cast<db8 *>(s.Y[n][b] + block_at(row, lg)) = fy.p[n];
                }
            }
            for (int i = tid; i < KB * 128; i += 256) {   // eights of head_dim of S and dS
                const int cg = i / (KB * 64), b = i / 64 % KB, row = cg * 16 + lc;
                dt4 x[2] = {}, y[2] = {};
                if (vg + cg < VG) {
                    const int64_t at = (((nc * VG + vg + cg) * KB + b) * 64 + lane) * 8;
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        x[e] = *reinterpret_cast<const dt4 *>(ws.S + at + e * 4);
                        y[e] = *reinterpret_cast<const dt4 *>(ws.dS + at + e * 4);
                    }
                }
                float m = 0.0f;
#pragma unroll
                for (int e = 0; e < 8; ++e) m = fmaf(x[e / 4][e % 4], y[e / 4][e % 4], m);
                cc += double(m);
                const Frag<3> fx = split<3>(x[0], x[1]), fy = split<3>(y[0], y[1]);
#pragma unroll
                for (int n = 0; n < 3; ++n) {
                    *reinterpret_cast<db8 *>(s.S[n][b] + block_at(row, lg)) = fx.p[n];
                    *reinterpret_cast<db8 *>(s.dS[n][b] + block_at(row, lg)) = fy.p[n];
                }
            }
            lds_barrier();
#pragma unroll
            for (int j = 0; j < NJ; ++j) {    // tile e of the columns i, both tiles of the rows j
                const int m = wv + 4 * j, b = m / 2, e = m & 1, bi = b > 0, bj = b == 2;
                if (b >= kTri<C>) break;
                const Frag<NI> fo = read_rows<NI>(s.go[0][bi], TB * kBlk, e);
                const Frag<3> fy = read_cols<3>(s.Y[0][bi], TB * kBlk, e);
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    const Frag<3> fu = read_cols<3>(s.U[0][bj], TB * kBlk, x);
                    dP[j][x] = mma<3>(fu, fo, dP[j][x]);
                    dA[j][x] = mma<3>(fu, fy, dA[j][x]);
                }
            }
            const Frag<NI> fo = read_rows<NI>(s.go[0][tb], TB * kBlk, ta);
            const Frag<3> fu = read_cols<3>(s.U[0][tb], TB * kBlk, ta), fy = read_cols<3>(s.Y[0][tb], TB * kBlk, ta);
#pragma unroll
            for (int b = 0; b < KW; ++b)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const Frag<3> fs = read_cols<3>(s.S[0][kb0 + b], KB * kBlk, e);
                    oS[b][e] = mma<3>(fs, fo, oS[b][e]);
                    yS[b][e] = mma<3>(fs, fy, yS[b][e]);
                    uS[b][e] = mma<3>(read_cols<3>(s.dS[0][kb0 + b], KB * kBlk, e), fu, uS[b][e]);
                }
            lds_barrier();
        }
        // Y . U of each token: over the 16 columns of a lane group, then the two column groups
        if (tid < TB * 128) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
#pragma unroll
                for (int m = 8; m > 0; m >>= 1) ub[e] += __shfl_xor(ub[e], m, 64);
                if (lc == 0) s.ub[tid / (TB * 64)][tid / 64 % TB * 32 + lg * 8 + e] = ub[e];
            }
        }
#pragma unroll
        for (int m = 32; m > 0; m >>= 1) cc += __shfl_xor(cc, m, 64);
        if (lane == 0) s.cs[wv] = cc;
        {
            const bf16 *kp = a.kk.data + p * a.kk.sp + hk * a.kk.sh + t0 * a.kk.st;
            const bf16 *qp = a.qq.data + p * a.qq.sp + hk * a.qq.sh + t0 * a.qq.st;
#pragma unroll
            for (int i = tid; i < C * KP / 8; i += 256) {
                const int b = i / 128, r = i % 128 / 4, t = b / KB * 32 + r, e = b % KB * 32 + i % 4 * 8, at = b * kBlk + block_at(r, i % 4);
                Frag<NI> fk = load_keys<NI>(kp + (min(t, live - 1) * int(a.kk.st) + e), a.kk.plane);
                Frag<NI> fq = load_keys<NI>(qp + (min(t, live - 1) * int(a.qq.st) + e), a.qq.plane);
                if (t >= live) {
                    clear(fk);
                    clear(fq);
                }
#pragma unroll
                for (int n = 0; n < NI; ++n) {
                    *reinterpret_cast<db8 *>(&s.k[n][0][0][0] + at) = fk.p[n];
                    *reinterpret_cast<db8 *>(&s.q[n][0][0][0] + at) = fq.p[n];
                }
            }
        }
        lds_barrier();
        // D, P and A again, and the weights of k and q in the gradients (accumulators: rows j, columns i)
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
            const int m = wv + 4 * j, b = m / 2, e = m & 1, bi = b > 0, bj = b == 2;
            if (b >= kTri<C>) break;
            dt4 kk[2] = {}, qk[2] = {};
#pragma unroll
            for (int x = 0; x < KB; ++x) {
                const Frag<NI> fk = read_rows<NI>(s.k[0][bi][x], kStride, e), fq = read_rows<NI>(s.q[0][bi][x], kStride, e);
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                    const Frag<NI> f = read_rows<NI>(s.k[0][bj][x], kStride, y);
                    kk[y] = mma<3>(f, fk, kk[y]);
                    qk[y] = mma<3>(f, fq, qk[y]);
                }
            }
            const int i = bi * 32 + block_row(lc, e);
            const double Gi = s.G[i];
            const float beta = s.g.beta[i];
            dt4 wq[2], wa[2];
#pragma unroll
            for (int y = 0; y < 2; ++y)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int jj = bj * 32 + lg * 8 + y * 4 + r;
                    const float D = i >= jj ? exp2_of(Gi - s.G[jj]) : 0.0f;
                    wq[y][r] = i >= jj ? a.scale * (D * dP[j][y][r]) : 0.0f;
                    wa[y][r] = i > jj ? -beta * (D * dA[j][y][r]) : 0.0f;
                    s.M[i * (C + 1) + jj] = i > jj ? fmaf(wq[y][r], qk[y][r], wa[y][r] * kk[y][r]) : 0.0f;
                }
            // a lane holds eight neighbours j of row i
            const Frag<NM> fq = split<NM>(wq[0], wq[1]), fa = split<NM>(wa[0], wa[1]);
#pragma unroll
            for (int n = 0; n < NM; ++n) {
                *reinterpret_cast<db8 *>(s.Mq[n][b] + block_at(block_row(lc, e), lg)) = fq.p[n];
                *reinterpret_cast<db8 *>(s.Ma[n][b] + block_at(block_row(lc, e), lg)) = fa.p[n];
            }
        }
        // the states' part of dq and dk, and its products with q and k
        {
            const float eG = s.g.eG[tok], eL = s.g.eL[tok], xo = a.scale * eG, xy = -(s.g.beta[tok] * eG);
            float ai = 0.0f, bj = 0.0f;
#pragma unroll
            for (int b = 0; b < KW; ++b) {
                dt4 k[2] = {}, q[2] = {};
#pragma unroll
                for (int n = NI - 1; n >= 0; --n) {
                    const int at = n * kStride + (tb * KB + kb0 + b) * kBlk + block_at(tok % 32, lg);
                    const du4 kw = *reinterpret_cast<const du4 *>(&s.k[0][0][0][0] + at);
                    const du4 qw = *reinterpret_cast<const du4 *>(&s.q[0][0][0][0] + at);
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const int sh = e & 1 ? 0 : 16;
                        k[e / 4][e % 4] += __uint_as_float((kw[e / 2] << sh) & 0xFFFF0000u);
                        q[e / 4][e % 4] += __uint_as_float((qw[e / 2] << sh) & 0xFFFF0000u);
                    }
                }
#pragma unroll
                for (int e = 0; e < 2; ++e)
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const float x = xo * oS[b][e][r], y = xy * yS[b][e][r], z = eL * uS[b][e][r];
                        ai += fmaf(x, q[e][r], y * k[e][r]);
                        bj = fmaf(z, k[e][r], bj);
                        aq[b][e][r] += x;
                        ak[b][e][r] += y + z;
                    }
            }
            ai += __shfl_xor(ai, 16, 64);
            bj += __shfl_xor(bj, 16, 64);
            ai += __shfl_xor(ai, 32, 64);
            bj += __shfl_xor(bj, 32, 64);
            if (lg == 0) {
                s.ai[wv / NT][tok] = ai;
                s.bj[wv / NT][tok] = bj;
            }
        }
        lds_barrier();
        // the pairs' part: the tokens as i (depth j up to them) and as j (depth i from them on)
#pragma unroll
        for (int x = 0; x < TB; ++x) {
            if (x <= tb) {
                const Frag<NM> mq = read_rows<NM>(s.Mq[0][tb + x], kTri<C> * kBlk, ta), ma = read_rows<NM>(s.Ma[0][tb + x], kTri<C> * kBlk, ta);
#pragma unroll
                for (int b = 0; b < KW; ++b)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const Frag<NI> k = read_cols<NI>(s.k[0][x][kb0 + b], kStride, e);
                        aq[b][e] = mma<NM>(k, mq, aq[b][e]);
                        ak[b][e] = mma<NM>(k, ma, ak[b][e]);
                    }
            }
            if (x >= tb) {
                const Frag<NM> mq = read_cols<NM>(s.Mq[0][tb + x], kTri<C> * kBlk, ta), ma = read_cols<NM>(s.Ma[0][tb + x], kTri<C> * kBlk, ta);
#pragma unroll
                for (int b = 0; b < KW; ++b)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        ak[b][e] = mma<NM>(read_cols<NI>(s.q[0][x][kb0 + b], kStride, e), mq, ak[b][e]);
                        ak[b][e] = mma<NM>(read_cols<NI>(s.k[0][x][kb0 + b], kStride, e), ma, ak[b][e]);
                    }
            }
        }
        if (tid < C) {
            double x = 0.0;
            for (int j = 0; j < tid; ++j) x += double(s.M[tid * (C + 1) + j]);
            s.row[tid] = x;
        } else if (tid >= 128 && tid < 128 + C) {
            const int j = tid - 128;
            double x = 0.0;
            for (int i = j + 1; i < C; ++i) x += double(s.M[i * (C + 1) + j]);
            s.colm[j] = x;
        }
        lds_barrier();
        if (tid < live) {
            const int m = tid;
            double x = double(s.g.last) * (s.cs[0] + s.cs[1] + s.cs[2] + s.cs[3]);
            for (int i = 0; i < C; ++i) {
                float y = i >= m ? s.ai[0][i] : s.bj[0][i];
                if constexpr (KG > 1) y += i >= m ? s.ai[1][i] : s.bj[1][i];
                x += double(y);
            }
            for (int i = 0; i < m; ++i) x += s.colm[i] - s.row[i];   // pairs i >= m > j: those begun and not ended
            const int64_t at = (int64_t(p) * a.T + t0 + m) * a.Hv + h;
            d.g[at] = float(x);
            d.beta[at] = (s.ub[0][m] + s.ub[1][m]) / delta_beta_safe(s.g.beta[m]);
        }
        lds_barrier();
    }
    const int rows = min(C, a.T - t0);
    for (int i = tid; i < rows * group; i += 256) {
        const int t = i / group, h = hk * group + i % group;
        const int64_t at = (int64_t(p) * a.T + t0 + t) * a.Hv + h;
        if (t >= live) d.g[at] = d.beta[at] = 0.0f;
    }
    if (tok >= rows) return;
#pragma unroll
    for (int b = 0; b < KW; ++b) {
        const int e0 = (kb0 + b) * 32 + lg * 8;
        const int64_t at = ((int64_t(p) * a.T + t0 + tok) * a.Hk + hk) * a.K + e0;
        put_eight(static_cast<T *>(d.q) + at, a.K - e0, aq[b][0], aq[b][1]);
        put_eight(static_cast<T *>(d.k) + at, a.K - e0, ak[b][0], ak[b][1]);
    }
}

template <typename T, int C, int KP>
hipError_t bwd_go(const DeltaArgs &a, const DeltaWs &ws, const DeltaGrads &d, hipStream_t st) {
    hipLaunchKernelGGL((delta_back_kernel<T, C, KP>), dim3(unsigned(int64_t(a.P) * a.Hv * ((a.V + 63) / 64))), dim3(kWalkThreads),
                       (Walk<T, C, KP, 3, true>::kLds), st, a, ws, d);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || ws.Nt == 0) return e;
    hipLaunchKernelGGL((delta_grad_kernel<T, C, KP>), dim3(unsigned(int64_t(a.P) * a.Hk * ws.Nt)), dim3(256),
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
    constexpr size_t lw = Walk<T, C, KP, 3, true>::kLds, lg = sizeof(GradLds<T, C, KP>);
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

hipError_t launch_delta_bwd(const DeltaArgs &a, const DeltaWs &ws, const DeltaGrads &d, bool is_bf16, hipStream_t st) {
    const hipError_t e = launch_delta_fwd(a, ws, is_bf16, st);
    if (e != hipSuccess) return e;
    return is_bf16 ? bwd_pick<bf16>(a, ws, d, st) : bwd_pick<float>(a, ws, d, st);
}

}  // namespace sdm
