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
#include "delta_tile.h"

namespace sdm {

namespace {

template <int C, int KP> struct BackLds {
    static constexpr int LK = KP + 4, LC = C + 4;
    float k[C * LK], q[C * LK], X[C * LC], P[C * LC];
    Gates<C> g;
};

template <typename T, int C, int KP>
__global__ __launch_bounds__(256) void delta_back_kernel(DeltaArgs a, DeltaWs ws, DeltaGrads d) {
    using Lds = BackLds<C, KP>;
    constexpr int LK = Lds::LK, LC = Lds::LC, NT = C / 16, KT = KP / 16;
    extern __shared__ __align__(16) unsigned char raw[];
    Lds &s = *reinterpret_cast<Lds *>(raw);
    const int slices = (a.V + 63) / 64;
    const int slice = blockIdx.x % slices, ph = blockIdx.x / slices, h = ph % a.Hv, p = ph / a.Hv, hk = h / (a.Hv / a.Hk);
    const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6, lc = lane & 15, lg = lane >> 4;
    const int col = slice * 64 + wv * 16 + lc;
    const bool in = col < a.V;
    const int n = delta_valid(a, p);
    const int64_t so = int64_t(ph) * a.K * a.V + col;
    const int64_t os = int64_t(a.Hv) * a.V, oo = (int64_t(p) * a.T * a.Hv + h) * a.V + col;
    const T *go = static_cast<const T *>(d.go) + oo;
    T *dv = static_cast<T *>(d.v) + oo;
    dt4 S[KT];
#pragma unroll
    for (int i = 0; i < KT; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int row = i * 16 + 4 * lg + r;
            S[i][r] = in && row < a.K && d.gstate ? d.gstate[so + int64_t(row) * a.V] : 0.0f;
        }
    for (int c = (n + C - 1) / C - 1; c >= 0; --c) {
        const int t0 = c * C, live = min(C, n - t0);
        const int64_t nc = int64_t(ph) * ws.Nt + c;
        load_tile<T, C, KP, LK>(a.k, p, hk, t0, live, a.K, s.k);
        load_tile<T, C, KP, LK>(a.q, p, hk, t0, live, a.K, s.q);
        load_mat<C, C, LC>(ws.X + nc * C * C, s.X);
        load_mat<C, C, LC>(ws.Pm + nc * C * C, s.P);
        load_gates<C>(a, p, h, t0, live, s.g);
        __syncthreads();
#pragma unroll
        for (int i = 0; i < KT; ++i)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int row = i * 16 + 4 * lg + r;
                if (in && row < a.K) ws.dS[nc * a.K * a.V + int64_t(row) * a.V + col] = S[i][r];
            }
        dt4 O[NT], U[NT], Y[NT];
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int row = t * 16 + 4 * lg + r;
                O[t][r] = in && row < live ? to_f32(go[(t0 + row) * os]) : 0.0f;
            }
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            dt4 x{};
#pragma unroll
            for (int i = 0; i < KT; ++i) x = tile_mma(tile_row(s.k, LK, t * 16, i * 16), S[i], x);
#pragma unroll
            for (int r = 0; r < 4; ++r) x[r] *= s.g.eL[t * 16 + 4 * lg + r];
#pragma unroll
            for (int i = t; i < NT; ++i) x = tile_mma(tile_col(s.P, LC, i * 16, t * 16), O[i], x);
            U[t] = x;
        }
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            Y[t] = dt4{};
#pragma unroll
            for (int i = t; i < NT; ++i) Y[t] = tile_mma(tile_col(s.X, LC, i * 16, t * 16), U[i], Y[t]);
        }
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int row = t * 16 + 4 * lg + r;
                if (in) ws.Y[(nc * C + row) * a.V + col] = Y[t][r];
                const float y = s.g.beta[row] * Y[t][r];
                if (in && row < live) dv[(t0 + row) * os] = from_f32<T>(y);
                O[t][r] *= a.scale * s.g.eG[row];
                Y[t][r] = -s.g.eG[row] * y;
            }
#pragma unroll
        for (int i = 0; i < KT; ++i) {
#pragma unroll
            for (int r = 0; r < 4; ++r) S[i][r] *= s.g.last;
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                S[i] = tile_mma(tile_col(s.q, LK, t * 16, i * 16), O[t], S[i]);
                S[i] = tile_mma(tile_col(s.k, LK, t * 16, i * 16), Y[t], S[i]);
            }
        }
        __syncthreads();
    }
    for (int t = n + lg; t < a.T; t += 4)
        if (in) dv[t * os] = from_f32<T>(0.0f);
    if (d.state) {
#pragma unroll
        for (int i = 0; i < KT; ++i)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int row = i * 16 + 4 * lg + r;
                if (in && row < a.K) d.state[so + int64_t(row) * a.V] = S[i][r];
            }
    }
}

// V columns of the state, the readings' gradient, U and Y are taken VB at a time.
constexpr int VB = 32, LV = VB + 4;

template <int C, int KP> struct GradLds {
    static constexpr int LK = KP + 4, LC = C + 4;
    union {
        struct {
            float go[C * LV], U[C * LV], Y[C * LV], S[KP * LV], dS[KP * LV];
        };
        struct {
            float k[C * LK], q[C * LK];
        };
    };
    float Mq[C * LC], Ma[C * LC];     // scale D dP and D dA
    float M[C * (C + 1)];             // dP P + dA A below the diagonal
    float ai[C], bj[C], ub[C];        // a_i, b_j, Y . U
    double row[C], colm[C];           // sums of M
    double cs[4];
    Gates<C> g;
};

// Sum over the 16 lanes of a row of accumulator blocks.
__device__ __forceinline__ float lanes16(float x) {
#pragma unroll
    for (int m = 8; m > 0; m >>= 1) x += __shfl_xor(x, m, 64);
    return x;
}

template <typename T, int C, int KP>
__global__ __launch_bounds__(256) void delta_grad_kernel(DeltaArgs a, DeltaWs ws, DeltaGrads d) {
    using Lds = GradLds<C, KP>;
    constexpr int LK = Lds::LK, LC = Lds::LC, NT = C / 16, KT = KP / 16;
    constexpr int CG = 4 / NT, CT = KT / CG;      // wavefronts side by side on a row of blocks, blocks of each
    extern __shared__ __align__(16) unsigned char raw[];
    Lds &s = *reinterpret_cast<Lds *>(raw);
    const int group = a.Hv / a.Hk;
    const int c = int(blockIdx.x % ws.Nt), ph = int(blockIdx.x / ws.Nt), hk = ph % a.Hk, p = ph / a.Hk;
    const int t0 = c * C, live = max(0, min(C, delta_valid(a, p) - t0));
    const int tid = threadIdx.x, lane = tid & 63, wv = tid >> 6, lc = lane & 15, lg = lane >> 4;
    const int rt = wv % NT, ct0 = wv / NT * CT;   // this wavefront's rows and first column block of dq, dk
    T *dq = static_cast<T *>(d.q), *dk = static_cast<T *>(d.k);
    dt4 aq[CT] = {}, ak[CT] = {};
    for (int hh = 0; live > 0 && hh < group; ++hh) {
        const int h = hk * group + hh;
        const int64_t nc = (int64_t(p) * a.Hv + h) * ws.Nt + c;
        const T *go = static_cast<const T *>(d.go) + (int64_t(p) * a.T + t0) * a.Hv * a.V + int64_t(h) * a.V;
        load_gates<C>(a, p, h, t0, live, s.g);
        // over V: dP, dA (blocks dealt to the wavefronts), do S0^T, Y S0^T, U dS1^T
        constexpr int NP = (NT * (NT + 1) / 2 + 3) / 4;
        dt4 dP[NP] = {}, dA[NP] = {}, oS[CT] = {}, yS[CT] = {}, uS[CT] = {};
        double cc = 0.0;
        float ub = 0.0f;
        for (int v0 = 0; v0 < a.V; v0 += VB) {
            for (int i = tid; i < C * VB; i += 256) {
                const int t = i / VB, v = i % VB;
                const bool in = v0 + v < a.V;
                s.go[t * LV + v] = in && t < live ? to_f32(go[int64_t(t) * a.Hv * a.V + v0 + v]) : 0.0f;
                s.U[t * LV + v] = in ? ws.U[(nc * C + t) * a.V + v0 + v] : 0.0f;
                s.Y[t * LV + v] = in ? ws.Y[(nc * C + t) * a.V + v0 + v] : 0.0f;
            }
            for (int i = tid; i < KP * VB; i += 256) {
                const int r = i / VB, v = i % VB;
                const bool in = v0 + v < a.V && r < a.K;
                const int64_t at = nc * a.K * a.V + int64_t(r) * a.V + v0 + v;
                const float x = in ? ws.S[at] : 0.0f, y = in ? ws.dS[at] : 0.0f;
                s.S[r * LV + v] = x;
                s.dS[r * LV + v] = y;
                cc += double(x * y);
            }
            __syncthreads();
#pragma unroll
            for (int j = 0; j < NP; ++j) {
                const int i = wv + 4 * j;
                if (i >= NT * (NT + 1) / 2) break;
                int r = 0, q = i;
                while (q > r) q -= ++r;
#pragma unroll
                for (int v = 0; v < VB; v += 16) {
                    const dt4 u = tile_row(s.U, LV, q * 16, v);
                    dP[j] = tile_mma(tile_row(s.go, LV, r * 16, v), u, dP[j]);
                    dA[j] = tile_mma(tile_row(s.Y, LV, r * 16, v), u, dA[j]);
                }
            }
#pragma unroll
            for (int v = 0; v < VB; v += 16) {
                const dt4 o = tile_row(s.go, LV, rt * 16, v), y = tile_row(s.Y, LV, rt * 16, v),
                          u = tile_row(s.U, LV, rt * 16, v);
#pragma unroll
                for (int j = 0; j < CT; ++j) {
                    const dt4 S = tile_row(s.S, LV, (ct0 + j) * 16, v), dS = tile_row(s.dS, LV, (ct0 + j) * 16, v);
                    oS[j] = tile_mma(o, S, oS[j]);
                    yS[j] = tile_mma(y, S, yS[j]);
                    uS[j] = tile_mma(u, dS, uS[j]);
                }
            }
            if (tid < C) {
#pragma unroll
                for (int v = 0; v < VB; ++v) ub = fmaf(s.Y[tid * LV + v], s.U[tid * LV + v], ub);
            }
            __syncthreads();
        }
        if (tid < C) s.ub[tid] = ub;
#pragma unroll
        for (int m = 32; m > 0; m >>= 1) cc += __shfl_xor(cc, m, 64);
        if (lane == 0) s.cs[wv] = cc;
        load_tile<T, C, KP, LK>(a.k, p, hk, t0, live, a.K, s.k);
        load_tile<T, C, KP, LK>(a.q, p, hk, t0, live, a.K, s.q);
        for (int i = tid; i < C * LC; i += 256) s.Mq[i] = s.Ma[i] = 0.0f;
        for (int i = tid; i < C; i += 256) s.ai[i] = s.bj[i] = 0.0f;
        __syncthreads();
        // D, P and A again, and the weights of k and q in the gradients
#pragma unroll
        for (int j = 0; j < NP; ++j) {
            const int i = wv + 4 * j;
            if (i >= NT * (NT + 1) / 2) break;
            int r = 0, q = i;
            while (q > r) q -= ++r;
            dt4 kk{}, qk{};
            for (int x = 0; x < KP; x += 16) {
                const dt4 b = tile_row(s.k, LK, q * 16, x);
                kk = tile_mma(tile_row(s.k, LK, r * 16, x), b, kk);
                qk = tile_mma(tile_row(s.q, LK, r * 16, x), b, qk);
            }
            const int col = q * 16 + lc;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int row = r * 16 + 4 * lg + e;
                const float D = row >= col ? expf(float(s.g.G[row] - s.g.G[col])) : 0.0f;
                const float wq = row >= col ? a.scale * (D * dP[j][e]) : 0.0f;
                const float wa = row > col ? -s.g.beta[row] * (D * dA[j][e]) : 0.0f;
                s.Mq[row * LC + col] = wq;
                s.Ma[row * LC + col] = wa;
                s.M[row * (C + 1) + col] = row > col ? fmaf(wq, qk[e], wa * kk[e]) : 0.0f;
            }
        }
        __syncthreads();
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int row = rt * 16 + 4 * lg + r;
            const float eG = s.g.eG[row], eL = s.g.eL[row], b = s.g.beta[row];
            float ai = 0.0f, bj = 0.0f;
#pragma unroll
            for (int j = 0; j < CT; ++j) {
                const int col = (ct0 + j) * 16 + lc;
                const float k = s.k[row * LK + col], q = s.q[row * LK + col];
                const float x = a.scale * (eG * oS[j][r]), y = -(b * eG) * yS[j][r], z = eL * uS[j][r];
                ai += fmaf(x, q, y * k);
                bj = fmaf(z, k, bj);
                aq[j][r] += x;
                ak[j][r] += y + z;
            }
            ai = lanes16(ai);
            bj = lanes16(bj);
            if constexpr (CG == 1) {
                if (lc == 0) {
                    s.ai[row] = ai;
                    s.bj[row] = bj;
                }
            } else if (lc == 0) {   // two wavefronts per row: the sum of two terms has one value
                atomicAdd(&s.ai[row], ai);
                atomicAdd(&s.bj[row], bj);
            }
        }
#pragma unroll
        for (int j = 0; j < CT; ++j) {
            const int c0 = (ct0 + j) * 16;
            for (int t = 0; t < NT; ++t) {
                const dt4 kt = tile_col(s.k, LK, t * 16, c0);
                if (t <= rt) {
                    aq[j] = tile_mma(tile_row(s.Mq, LC, rt * 16, t * 16), kt, aq[j]);
                    ak[j] = tile_mma(tile_row(s.Ma, LC, rt * 16, t * 16), kt, ak[j]);
                }
                if (t >= rt) {
                    ak[j] = tile_mma(tile_col(s.Ma, LC, t * 16, rt * 16), kt, ak[j]);
                    ak[j] = tile_mma(tile_col(s.Mq, LC, t * 16, rt * 16), tile_col(s.q, LK, t * 16, c0), ak[j]);
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
        __syncthreads();
        if (tid < live) {
            const int m = tid;
            double x = double(s.g.last) * (s.cs[0] + s.cs[1] + s.cs[2] + s.cs[3]);
            for (int i = 0; i < C; ++i) x += i >= m ? double(s.ai[i]) : double(s.bj[i]);
            for (int i = 0; i < m; ++i) x += s.colm[i] - s.row[i];   // pairs i >= m > j: those begun and not ended
            const int64_t at = (int64_t(p) * a.T + t0 + m) * a.Hv + h;
            d.g[at] = float(x);
            d.beta[at] = s.ub[m] / delta_beta_safe(s.g.beta[m]);
        }
        __syncthreads();
    }
    if (c * C >= a.T) return;
    const int rows = min(C, a.T - t0);
    for (int i = tid; i < rows * group; i += 256) {
        const int t = i / group, h = hk * group + i % group;
        const int64_t at = (int64_t(p) * a.T + t0 + t) * a.Hv + h;
        if (t >= live) d.g[at] = d.beta[at] = 0.0f;
    }
#pragma unroll
    for (int j = 0; j < CT; ++j)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int row = rt * 16 + 4 * lg + r, col = (ct0 + j) * 16 + lc;
            if (row >= rows || col >= a.K) continue;
            const int64_t at = ((int64_t(p) * a.T + t0 + row) * a.Hk + hk) * a.K + col;
            dq[at] = from_f32<T>(row < live ? aq[j][r] : 0.0f);
            dk[at] = from_f32<T>(row < live ? ak[j][r] : 0.0f);
        }
}

template <typename T, int C, int KP>
hipError_t bwd_go(const DeltaArgs &a, const DeltaWs &ws, const DeltaGrads &d, hipStream_t st) {
    hipLaunchKernelGGL((delta_back_kernel<T, C, KP>), dim3(unsigned(int64_t(a.P) * a.Hv * ((a.V + 63) / 64))), dim3(256),
                       sizeof(BackLds<C, KP>), st, a, ws, d);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || ws.Nt == 0) return e;
    hipLaunchKernelGGL((delta_grad_kernel<T, C, KP>), dim3(unsigned(int64_t(a.P) * a.Hk * ws.Nt)), dim3(256),
                       sizeof(GradLds<C, KP>), st, a, ws, d);
    return hipGetLastError();
}
template <typename T>
hipError_t bwd_pick(const DeltaArgs &a, const DeltaWs &ws, const DeltaGrads &d, hipStream_t st) {
    switch (delta_kp(a.K)) {
        case 64: return bwd_go<T, 64, 64>(a, ws, d, st);
        case 128: return bwd_go<T, 64, 128>(a, ws, d, st);
        default: return bwd_go<T, 32, 256>(a, ws, d, st);
    }
}
template <typename T, int C, int KP> hipError_t bwd_attr() {
    hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void *>(&delta_back_kernel<T, C, KP>),
                                       hipFuncAttributeMaxDynamicSharedMemorySize, sizeof(BackLds<C, KP>));
    if (e == hipSuccess)
        e = hipFuncSetAttribute(reinterpret_cast<const void *>(&delta_grad_kernel<T, C, KP>),
                                hipFuncAttributeMaxDynamicSharedMemorySize, sizeof(GradLds<C, KP>));
    static_assert(sizeof(GradLds<C, KP>) <= 160 * 1024 && sizeof(BackLds<C, KP>) <= 160 * 1024, "LDS of a workgroup");
    return e;
}
template <typename T> hipError_t bwd_attrs() {
    hipError_t e = bwd_attr<T, 64, 64>();
    if (e == hipSuccess) e = bwd_attr<T, 64, 128>();
    if (e == hipSuccess) e = bwd_attr<T, 32, 256>();
    return e;
}

}  // namespace

hipError_t delta_bwd_prepare() {
    const hipError_t e = bwd_attrs<float>();
    return e == hipSuccess ? bwd_attrs<bf16>() : e;
}

hipError_t launch_delta_bwd(const DeltaArgs &a, const DeltaWs &ws, const DeltaGrads &d, bool is_bf16, hipStream_t st) {
    const hipError_t e = launch_delta_fwd(a, ws, is_bf16, true, st);
    if (e != hipSuccess) return e;
    return is_bf16 ? bwd_pick<bf16>(a, ws, d, st) : bwd_pick<float>(a, ws, d, st);
}

}  // namespace sdm
