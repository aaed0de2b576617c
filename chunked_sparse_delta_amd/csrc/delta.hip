// The chunked gated delta rule, forward.
//
// In a chunk of C tokens with G the running sum of the log-decays, D_ij = exp(G_i - G_j) and
// S0 the state before it:
//     A = tril(D kk^T, -1),  X = (I + beta A)^-1,  P = scale tril(D qk^T)
//     U = X beta (v - e^G k S0),  out = scale e^G q S0 + P U,  S1 = e^{G_C} S0 + (e^{G_C - G} k)^T U
// delta_prep_kernel computes X and P of every chunk at once; delta_state_kernel walks the
// chunks of a stream's head in order. Every column of the state evolves on its own: a
// wavefront keeps 16 columns of S in accumulators through the whole sequence, and the four
// wavefronts of a workgroup share the chunk's k, q, X and P in LDS.
#include "delta_tile.h"

namespace sdm {

namespace {

template <int C, int KP> struct PrepLds {
    static constexpr int LK = KP + 4, LC = C + 4;
    float k[C * LK], q[C * LK], L[C * LC], X[C * LC];
    Gates<C> g;
};

template <typename T, int C, int KP> __global__ __launch_bounds__(256) void delta_prep_kernel(DeltaArgs a, DeltaWs ws) {
    using Lds = PrepLds<C, KP>;
    constexpr int LK = Lds::LK, LC = Lds::LC, NT = C / 16;
    extern __shared__ __align__(16) unsigned char raw[];
    Lds &s = *reinterpret_cast<Lds *>(raw);
    const int64_t n = blockIdx.x;
    const int c = int(n % ws.Nt), h = int(n / ws.Nt % a.Hv), p = int(n / ws.Nt / a.Hv), hk = h / (a.Hv / a.Hk);
    const int t0 = c * C, live = min(C, delta_valid(a, p) - t0);
    if (live <= 0) return;
    const int tid = threadIdx.x, lane = tid & 63, wv = tid >> 6, lc = lane & 15, lg = lane >> 4;
    load_tile<T, C, KP, LK>(a.k, p, hk, t0, live, a.K, s.k);
    load_tile<T, C, KP, LK>(a.q, p, hk, t0, live, a.K, s.q);
    load_gates<C>(a, p, h, t0, live, s.g);
    for (int i = tid; i < C * LC; i += 256) s.L[i] = s.X[i] = 0.0f;
    __syncthreads();
    float *P = ws.Pm + n * C * C;
    for (int i = wv; i < NT * NT; i += 4) {
        const int rt = i / NT, ct = i % NT;
        dt4 kk{}, qk{};
        if (ct <= rt) {
#pragma unroll 4
            for (int d = 0; d < KP; d += 16) {
                const dt4 b = tile_row(s.k, LK, ct * 16, d);
                kk = tile_mma(tile_row(s.k, LK, rt * 16, d), b, kk);
                qk = tile_mma(tile_row(s.q, LK, rt * 16, d), b, qk);
            }
        }
        const int col = ct * 16 + lc;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int row = rt * 16 + 4 * lg + r;
            const float D = row >= col ? expf(float(s.g.G[row] - s.g.G[col])) : 0.0f;
            P[row * C + col] = row >= col ? a.scale * (D * qk[r]) : 0.0f;
            if (row > col) {
                const float b = ws.backward ? delta_beta_safe(s.g.beta[row]) : s.g.beta[row];
                s.L[row * LC + col] = b * (D * kk[r]);
            }
        }
    }
    __syncthreads();
    // the inverse of I + L: the 16 x 16 diagonal blocks by substitution, one column per lane
    if (wv < NT && lane < 16) {
        const float *L = s.L + wv * 16 * (LC + 1);
        float x[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            float v = i == lane ? 1.0f : 0.0f;
#pragma unroll
            for (int j = 0; j < i; ++j) v = fmaf(-L[i * LC + j], x[j], v);
            x[i] = v;
            s.X[(wv * 16 + i) * LC + wv * 16 + lane] = v;
        }
    }
    __syncthreads();
    // ... then [A 0; B D]^-1 = [A^-1 0; -D^-1 B A^-1 D^-1] of blocks of 16 and 32; B A^-1 takes B's place in L
#pragma unroll
    for (int b = 1; b < NT; b *= 2) {
        const int per = b * b, work = NT / (2 * b) * per;
        for (int pass = 0; pass < 2; ++pass) {
            dt4 acc[2] = {};
            int m = 0;
            for (int i = wv; i < work; i += 4, ++m) {
                const int pair = i / per, rt = pair * 2 * b + b + i % per / b, ct = pair * 2 * b + i % per % b;
                const int k0 = pair * 2 * b + (pass ? b : 0);
                for (int kb = k0; kb < k0 + b; ++kb)
                    acc[m] = pass ? tile_mma(tile_row(s.X, LC, rt * 16, kb * 16), tile_col(s.L, LC, kb * 16, ct * 16), acc[m])
                                  : tile_mma(tile_row(s.L, LC, rt * 16, kb * 16), tile_col(s.X, LC, kb * 16, ct * 16), acc[m]);
            }
            __syncthreads();
            m = 0;
            for (int i = wv; i < work; i += 4, ++m) {
                const int pair = i / per, rt = pair * 2 * b + b + i % per / b, ct = pair * 2 * b + i % per % b;
                tile_put(pass ? s.X : s.L, LC, rt * 16, ct * 16, pass ? -acc[m] : acc[m]);
            }
            __syncthreads();
        }
    }
    float *X = ws.X + n * C * C;
    for (int i = tid; i < C * C; i += 256) X[i] = s.X[i / C * LC + i % C];
}

template <int C, int KP> struct StateLds {
    static constexpr int LK = KP + 4, LC = C + 4;
    float k[C * LK], q[C * LK], X[C * LC], P[C * LC];
    Gates<C> g;
};

// SAVE: keeps U and each chunk's start state for the backward, and gives no output.
template <typename T, int C, int KP, bool SAVE>
__global__ __launch_bounds__(256) void delta_state_kernel(DeltaArgs a, DeltaWs ws) {
    using Lds = StateLds<C, KP>;
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
    T *out = static_cast<T *>(a.out) + (int64_t(p) * a.T * a.Hv + h) * a.V + col;
    const int64_t os = int64_t(a.Hv) * a.V;
    const T *v = static_cast<const T *>(a.v.data) + p * a.v.sp + h * a.v.sh + col;
    dt4 S[KT];
#pragma unroll
    for (int i = 0; i < KT; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int row = i * 16 + 4 * lg + r;
            S[i][r] = in && row < a.K && a.state ? a.state[so + int64_t(row) * a.V] : 0.0f;
        }
    for (int c = 0; c * C < n; ++c) {
        const int t0 = c * C, live = min(C, n - t0);
        const int64_t nc = int64_t(ph) * ws.Nt + c;
        load_tile<T, C, KP, LK>(a.k, p, hk, t0, live, a.K, s.k);
        if constexpr (!SAVE) load_tile<T, C, KP, LK>(a.q, p, hk, t0, live, a.K, s.q);
        load_mat<C, C, LC>(ws.X + nc * C * C, s.X);
        if constexpr (!SAVE) load_mat<C, C, LC>(ws.Pm + nc * C * C, s.P);
        load_gates<C>(a, p, h, t0, live, s.g);
        __syncthreads();
        if constexpr (SAVE) {
#pragma unroll
            for (int i = 0; i < KT; ++i)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int row = i * 16 + 4 * lg + r;
                    if (in && row < a.K) ws.S[nc * a.K * a.V + int64_t(row) * a.V + col] = S[i][r];
                }
        }
        dt4 R[NT], U[NT], O[NT];
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            dt4 x{}, y{};
#pragma unroll
            for (int d = 0; d < KT; ++d) {
                x = tile_mma(tile_row(s.k, LK, t * 16, d * 16), S[d], x);
                if constexpr (!SAVE) y = tile_mma(tile_row(s.q, LK, t * 16, d * 16), S[d], y);
            }
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int row = t * 16 + 4 * lg + r;
                const float vv = in && row < live ? to_f32(v[(t0 + row) * a.v.st]) : 0.0f;
                R[t][r] = (SAVE ? delta_beta_safe(s.g.beta[row]) : s.g.beta[row]) * (vv - s.g.eG[row] * x[r]);
                O[t][r] = a.scale * (s.g.eG[row] * y[r]);
            }
        }
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            U[t] = dt4{};
#pragma unroll
            for (int d = 0; d <= t; ++d) U[t] = tile_mma(tile_row(s.X, LC, t * 16, d * 16), R[d], U[t]);
        }
        if constexpr (SAVE) {
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    if (in) ws.U[(nc * C + t * 16 + 4 * lg + r) * a.V + col] = U[t][r];
        } else {
#pragma unroll
            for (int t = 0; t < NT; ++t) {
#pragma unroll
                for (int d = 0; d <= t; ++d) O[t] = tile_mma(tile_row(s.P, LC, t * 16, d * 16), U[d], O[t]);
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int row = t * 16 + 4 * lg + r;
                    if (in && row < live) out[(t0 + row) * os] = from_f32<T>(O[t][r]);
                }
            }
        }
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int r = 0; r < 4; ++r) U[t][r] *= s.g.eL[t * 16 + 4 * lg + r];
#pragma unroll
        for (int i = 0; i < KT; ++i) {
#pragma unroll
            for (int r = 0; r < 4; ++r) S[i][r] *= s.g.last;
#pragma unroll
            for (int t = 0; t < NT; ++t) S[i] = tile_mma(tile_col(s.k, LK, t * 16, i * 16), U[t], S[i]);
        }
        __syncthreads();
    }
    if constexpr (!SAVE) {
        for (int t = n + lg; t < a.T; t += 4)
            if (in) out[t * os] = from_f32<T>(0.0f);
        if (a.state_out) {
#pragma unroll
            for (int i = 0; i < KT; ++i)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int row = i * 16 + 4 * lg + r;
                    if (in && row < a.K) a.state_out[so + int64_t(row) * a.V] = S[i][r];
                }
        }
    }
}

template <typename T, int C, int KP> hipError_t fwd_go(const DeltaArgs &a, const DeltaWs &ws, bool save, hipStream_t st) {
    if (ws.Nt > 0) {
        hipLaunchKernelGGL((delta_prep_kernel<T, C, KP>), dim3(unsigned(int64_t(a.P) * a.Hv * ws.Nt)), dim3(256),
                           sizeof(PrepLds<C, KP>), st, a, ws);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    const dim3 grid(unsigned(int64_t(a.P) * a.Hv * ((a.V + 63) / 64)));
    if (save)
        hipLaunchKernelGGL((delta_state_kernel<T, C, KP, true>), grid, dim3(256), sizeof(StateLds<C, KP>), st, a, ws);
    else
        hipLaunchKernelGGL((delta_state_kernel<T, C, KP, false>), grid, dim3(256), sizeof(StateLds<C, KP>), st, a, ws);
    return hipGetLastError();
}
template <typename T> hipError_t fwd_pick(const DeltaArgs &a, const DeltaWs &ws, bool save, hipStream_t st) {
    switch (delta_kp(a.K)) {
        case 64: return fwd_go<T, 64, 64>(a, ws, save, st);
        case 128: return fwd_go<T, 64, 128>(a, ws, save, st);
        default: return fwd_go<T, 32, 256>(a, ws, save, st);
    }
}

template <typename T, int C, int KP> hipError_t fwd_attr() {
    hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void *>(&delta_prep_kernel<T, C, KP>),
                                       hipFuncAttributeMaxDynamicSharedMemorySize, sizeof(PrepLds<C, KP>));
    for (auto k : {&delta_state_kernel<T, C, KP, false>, &delta_state_kernel<T, C, KP, true>})
        if (e == hipSuccess)
            e = hipFuncSetAttribute(reinterpret_cast<const void *>(k), hipFuncAttributeMaxDynamicSharedMemorySize,
                                    sizeof(StateLds<C, KP>));
    return e;
}
template <typename T> hipError_t fwd_attrs() {
    hipError_t e = fwd_attr<T, 64, 64>();
    if (e == hipSuccess) e = fwd_attr<T, 64, 128>();
    if (e == hipSuccess) e = fwd_attr<T, 32, 256>();
    return e;
}

}  // namespace

hipError_t delta_prepare() {
    const hipError_t e = fwd_attrs<float>();
    return e == hipSuccess ? fwd_attrs<bf16>() : e;
}

hipError_t launch_delta_fwd(const DeltaArgs &a, const DeltaWs &ws, bool is_bf16, bool save, hipStream_t st) {
    return is_bf16 ? fwd_pick<bf16>(a, ws, save, st) : fwd_pick<float>(a, ws, save, st);
}

}  // namespace sdm
