// The chunked gated delta rule, forward.
//
// In a chunk of C tokens with G the running sum of the log-decays, D_ij = exp(G_i - G_j) and
// S0 the state before it:
//     A = tril(D kk^T, -1),  X = (I + beta A)^-1,  P = scale tril(D qk^T)
//     U = X beta (v - e^G k S0),  out = scale e^G q S0 + P U,  S1 = e^{G_C} S0 + (e^{G_C - G} k)^T U
// delta_prep_kernel computes X and P of every chunk at once; delta_state_kernel walks the
// chunks of a stream's head in order.
#include "delta_walk.h"

namespace sdm {

namespace {

template <int C> struct PrepLds {
    static constexpr int LC = C + 4;
    float L[C * LC], X[C * LC];     // X holds P first
    double G[C];
    Gates<C> g;
};

// float32 16 x 16 blocks of row-major LDS matrices on v_mfma_f32_16x16x4_f32 (step r takes depth
// 4 (lane >> 4) + r): the inverse is too small a part to be worth splitting.
__device__ __forceinline__ dt4 f32_mma(const float *A, const float *B, int ld, dt4 acc) {
    const int lane = threadIdx.x & 63;
    const dt4 a = *reinterpret_cast<const dt4 *>(A + (lane & 15) * ld + 4 * (lane >> 4));
    const float *b = B + 4 * (lane >> 4) * ld + (lane & 15);
#pragma unroll
    for (int r = 0; r < 4; ++r) acc = __builtin_amdgcn_mfma_f32_16x16x4f32(a[r], b[r * ld], acc, 0, 0, 0);
    return acc;
}

// The lower 32 x 32 blocks of the row-major m as NP pieces, block images NP * kTri apart.
template <int C, int NP> __device__ __forceinline__ void put_pieces(const float *m, unsigned char *out) {
    constexpr int LC = PrepLds<C>::LC;
    for (int i = threadIdx.x; i < kTri<C> * 128; i += 256) {
        const int b = i / 128, r = i % 128 / 4, c = i % 4, br = b > 0, bc = b == 2;
        const float *src = m + (br * 32 + r) * LC + bc * 32 + c * 8;
        const Frag<NP> f = split<NP>(*reinterpret_cast<const dt4 *>(src), *reinterpret_cast<const dt4 *>(src + 4));
#pragma unroll
        for (int n = 0; n < NP; ++n)
            *reinterpret_cast<db8 *>(out + (n * kTri<C> + b) * kBlk + block_at(r, c)) = f.p[n];
    }
}

template <typename T, int C, int KP, int NP>
__global__ __launch_bounds__(256) void delta_prep_kernel(DeltaArgs a, DeltaWs ws) {
    constexpr int LC = PrepLds<C>::LC, NT = C / 16, NI = kPieces<T>;
    __shared__ PrepLds<C> s;
    const int64_t n = blockIdx.x;
    const int c = int(n % ws.Nt), h = int(n / ws.Nt % a.Hv), p = int(n / ws.Nt / a.Hv), hk = h / (a.Hv / a.Hk);
    const int t0 = c * C, live = min(C, delta_valid(a, p) - t0);
    if (live <= 0) return;
    const int tid = threadIdx.x, lane = tid & 63, wv = tid >> 6, lc = lane & 15, lg = lane >> 4;
    if (wv == 3) {
        // G in 64 bits: its differences are as exact as the log-decays themselves however large it grew. A log-decay
        // below -1e4 (-inf among them: it clears the state) counts as -1e4, whose exponential is 0 too.
        const int64_t at = (int64_t(p) * a.T + t0 + lane) * a.Hv + h;
        const bool in = lane < C && lane < live;
        float g = in ? a.g[at] : 0.0f;
        if (g < -1e4f) g = -1e4f;
        double G = double(g);
#pragma unroll
        for (int d = 1; d < C; d <<= 1) {
            const double o = __shfl_up(G, d, 64);
            if (lane >= d) G += o;
        }
        const double GL = __shfl(G, C - 1, 64);
        if (lane < C) {
            s.G[lane] = G;
            s.g.beta[lane] = in ? a.beta[at] : 0.0f;
            s.g.eG[lane] = expf(float(G));
            s.g.eL[lane] = expf(float(GL - G));
        }
        if (lane == 0) s.g.last = expf(float(GL));
    }
    dt4 kk[NT] = {}, qk[NT] = {};
    if (wv < NT) {
        const T *k = static_cast<const T *>(a.k.data) + p * a.k.sp + hk * a.k.sh + t0 * a.k.st;
        const T *q = static_cast<const T *>(a.q.data) + p * a.q.sp + hk * a.q.sh + t0 * a.q.st;
#pragma unroll
        for (int kb = 0; kb < KP / 32; ++kb) {
            const int d = kb * 32 + lg * 8;
            Eight<T> x[NT], y;
#pragma unroll
            for (int ct = 0; ct < NT; ++ct)
                if (ct <= wv) x[ct].load(k + min(ct * 16 + lc, live - 1) * a.k.st, d, a.K);
            y.load(q + min(wv * 16 + lc, live - 1) * a.q.st, d, a.K);
            y.fix(d, a.K, wv * 16 + lc < live);
            Frag<NI> fk[NT];
            const Frag<NI> fq = y.pieces();
#pragma unroll
            for (int ct = 0; ct < NT; ++ct)
                if (ct <= wv) {
                    x[ct].fix(d, a.K, ct * 16 + lc < live);
                    fk[ct] = x[ct].pieces();
                }
            Frag<NI> fa;      // this wavefront's own rows of k
#pragma unroll
            for (int ct = 0; ct < NT; ++ct)
                if (ct == wv) fa = fk[ct];
#pragma unroll
            for (int ct = 0; ct < NT; ++ct)
                if (ct <= wv) {
                    kk[ct] = mma<3>(fa, fk[ct], kk[ct]);
                    qk[ct] = mma<3>(fq, fk[ct], qk[ct]);
                }
        }
    }
    __syncthreads();
    if (wv < NT) {
#pragma unroll
        for (int ct = 0; ct < NT; ++ct)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int row = wv * 16 + 4 * lg + r, col = ct * 16 + lc;
                const float D = row >= col ? expf(float(s.G[row] - s.G[col])) : 0.0f;
                const float b = ws.backward ? delta_beta_safe(s.g.beta[row]) : s.g.beta[row];
                s.L[row * LC + col] = row > col ? b * (D * kk[ct][r]) : 0.0f;
                s.X[row * LC + col] = row >= col ? a.scale * (D * qk[ct][r]) : 0.0f;
            }
    }
    __syncthreads();
    ChunkMats<C, NP> *out = reinterpret_cast<ChunkMats<C, NP> *>(ws.mats) + n;
    put_pieces<C, NP>(s.X, &out->P[0][0][0]);
    if (tid < int(sizeof(Gates<C>) / 4)) reinterpret_cast<float *>(&out->g)[tid] = reinterpret_cast<const float *>(&s.g)[tid];
    __syncthreads();
    for (int i = tid; i < C * LC; i += 256) s.X[i] = 0.0f;
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
        const int per = b * b, work = NT / (2 * b) * per;     // at most 4 blocks, one per wavefront
        const int pair = wv / per, rt = pair * 2 * b + b + wv % per / b, ct = pair * 2 * b + wv % per % b;
#pragma unroll
        for (int pass = 0; pass < 2; ++pass) {
            dt4 acc{};
            if (wv < work)
                for (int i = 0; i < b; ++i) {
                    const int kb = pair * 2 * b + (pass ? b : 0) + i;
                    acc = f32_mma((pass ? s.X : s.L) + rt * 16 * LC + kb * 16, (pass ? s.L : s.X) + kb * 16 * LC + ct * 16, LC, acc);
                }
            __syncthreads();
            if (wv < work) {
                float *d = (pass ? s.X : s.L) + (rt * 16 + 4 * lg) * LC + ct * 16 + lc;
#pragma unroll
                for (int r = 0; r < 4; ++r) d[r * LC] = pass ? -acc[r] : acc[r];
            }
            __syncthreads();
        }
    }
    put_pieces<C, 3>(s.X, &out->X[0][0][0]);
}

// Every column of the state evolves on its own: a wavefront keeps 16 columns of S in
// accumulators through the whole sequence, and the four wavefronts of a workgroup share the
// chunk's k, q, X and P in LDS. The next chunk's are loaded into registers under this one's products.
// SAVE: keeps U and each chunk's start state for the backward, and gives no output.
template <typename T, int C, int KP, bool SAVE>
__global__ __launch_bounds__(256) void delta_state_kernel(DeltaArgs a, DeltaWs ws) {
    constexpr int NI = kPieces<T>, NP = kPPieces<T>(SAVE), KB = KP / 32, TB = C / 32;
    constexpr int NS = NI == 1 ? 2 : 3;    // pieces of S and U that reach the readings only
    using W = Walk<T, C, KP, NP, !SAVE>;
    extern __shared__ __align__(16) unsigned char raw[];
    typename W::Lds &s = *reinterpret_cast<typename W::Lds *>(raw);
    const int slices = (a.V + 63) / 64, VG = (a.V + 15) / 16;
    const int slice = blockIdx.x % slices, ph = blockIdx.x / slices, h = ph % a.Hv, p = ph / a.Hv, hk = h / (a.Hv / a.Hk);
    const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6, lc = lane & 15, lg = lane >> 4;
    const int cg = slice * 4 + wv, col = cg * 16 + lc;
    const bool in = col < a.V;
    const int n = delta_valid(a, p), Nc = (n + C - 1) / C;
    T *out = static_cast<T *>(a.out) + (int64_t(p) * a.T * a.Hv + h) * a.V + col;
    const int64_t os = int64_t(a.Hv) * a.V;
    dt4 S[KB][2];
    load_state<KB>(S, a.state, ph, a.K, a.V, col);
    W w(a, ws, p, h, hk, ph, cg, a.v, h);
    if (Nc > 0) {
        w.load(0, n);
        w.store(s, 0, n);
        __syncthreads();
    }
    for (int c = 0; c < Nc; ++c) {
        const int t0 = c * C;
        if (c + 1 < Nc) w.load(c + 1, n);
        const int64_t nc = int64_t(ph) * ws.Nt + c;
        if constexpr (SAVE) save_blocks<KB>(ws.S, nc, VG, cg, S);
        const Gates<C> &g = s.m.g;
        dt4 x[TB][2] = {}, y[TB][2] = {};
#pragma unroll
        for (int kb = 0; kb < KB; ++kb) {
            const Frag<3> fs = split<3>(S[kb][0], S[kb][1]);
#pragma unroll
            for (int tb = 0; tb < TB; ++tb)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    x[tb][e] = mma<3>(read_rows<NI>(s.k[0][tb][kb], W::kStride, e), fs, x[tb][e]);
                    if constexpr (!SAVE) y[tb][e] = mma<NS>(read_rows<NI>(s.q[0][tb][kb], W::kStride, e), fs, y[tb][e]);
                }
        }
        Frag<3> fr[TB];
#pragma unroll
        for (int tb = 0; tb < TB; ++tb) {
            dt4 r[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int t = tb * 32 + lg * 8 + e * 4;
                const dt4 b = *reinterpret_cast<const dt4 *>(g.beta + t), eG = *reinterpret_cast<const dt4 *>(g.eG + t);
                const dt4 v = w.value(s, tb, e);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    r[e][i] = (SAVE ? delta_beta_safe(b[i]) : b[i]) * (v[i] - eG[i] * x[tb][e][i]);
                    y[tb][e][i] *= a.scale * eG[i];
                }
            }
            fr[tb] = split<3>(r[0], r[1]);
        }
        dt4 U[TB][2];
#pragma unroll
        for (int tb = 0; tb < TB; ++tb)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                U[tb][e] = dt4{};
#pragma unroll
                for (int d = 0; d <= tb; ++d)
                    U[tb][e] = mma<3>(read_rows<3>(s.m.X[0][tb + d], kTri<C> * kBlk, e), fr[d], U[tb][e]);
            }
        if constexpr (SAVE) save_blocks<TB>(ws.U, nc, VG, cg, U);
        else {
#pragma unroll
            for (int d = 0; d < TB; ++d) {
                const Frag<NS> fu = split<NS>(U[d][0], U[d][1]);
#pragma unroll
                for (int tb = d; tb < TB; ++tb)
#pragma unroll
                    for (int e = 0; e < 2; ++e)
                        y[tb][e] = mma<NS>(read_rows<NP>(s.m.P[0][tb + d], kTri<C> * kBlk, e), fu, y[tb][e]);
            }
#pragma unroll
            for (int tb = 0; tb < TB; ++tb)
#pragma unroll
                for (int e = 0; e < 2; ++e)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int t = t0 + tb * 32 + lg * 8 + e * 4 + i;
                        if (in && t < n) out[t * os] = from_f32<T>(y[tb][e][i]);
                    }
        }
        const float last = g.last;
#pragma unroll
        for (int kb = 0; kb < KB; ++kb)
#pragma unroll
            for (int e = 0; e < 2; ++e) S[kb][e] *= last;
#pragma unroll
        for (int tb = 0; tb < TB; ++tb) {
#pragma unroll
            for (int e = 0; e < 2; ++e) U[tb][e] *= *reinterpret_cast<const dt4 *>(g.eL + tb * 32 + lg * 8 + e * 4);
            const Frag<3> fu = split<3>(U[tb][0], U[tb][1]);
#pragma unroll
            for (int kb = 0; kb < KB; ++kb)
#pragma unroll
                for (int e = 0; e < 2; ++e) S[kb][e] = mma<3>(read_cols<NI>(s.k[0][tb][kb], W::kStride, e), fu, S[kb][e]);
        }
        if (c + 1 < Nc) {
            __syncthreads();
            w.store(s, c + 1, n);
            __syncthreads();
        }
    }
    if constexpr (!SAVE) {
        for (int t = n + lg; t < a.T; t += 4)
            if (in) out[t * os] = from_f32<T>(0.0f);
        store_state<KB>(S, a.state_out, ph, a.K, a.V, col);
    }
}

template <typename T, int C, int KP> hipError_t fwd_go(const DeltaArgs &a, const DeltaWs &ws, hipStream_t st) {
    const dim3 chunks(unsigned(int64_t(a.P) * a.Hv * ws.Nt)), grid(unsigned(int64_t(a.P) * a.Hv * ((a.V + 63) / 64)));
    constexpr int N0 = kPPieces<T>(false), N1 = kPPieces<T>(true);
    if (ws.Nt > 0) {
        if (ws.backward) hipLaunchKernelGGL((delta_prep_kernel<T, C, KP, N1>), chunks, dim3(256), 0, st, a, ws);
        else hipLaunchKernelGGL((delta_prep_kernel<T, C, KP, N0>), chunks, dim3(256), 0, st, a, ws);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    if (ws.backward)
        hipLaunchKernelGGL((delta_state_kernel<T, C, KP, true>), grid, dim3(256), sizeof(typename Walk<T, C, KP, N1, false>::Lds), st, a, ws);
    else
        hipLaunchKernelGGL((delta_state_kernel<T, C, KP, false>), grid, dim3(256), sizeof(typename Walk<T, C, KP, N0, true>::Lds), st, a, ws);
    return hipGetLastError();
}
template <typename T> hipError_t fwd_pick(const DeltaArgs &a, const DeltaWs &ws, hipStream_t st) {
    switch (delta_kp(a.K)) {
        case 64: return fwd_go<T, 64, 64>(a, ws, st);
        case 128: return fwd_go<T, 64, 128>(a, ws, st);
        default: return fwd_go<T, 32, 256>(a, ws, st);
    }
}

template <typename T, int C, int KP> hipError_t fwd_attr() {
    constexpr int N0 = kPPieces<T>(false), N1 = kPPieces<T>(true);
    constexpr size_t l0 = sizeof(typename Walk<T, C, KP, N0, true>::Lds), l1 = sizeof(typename Walk<T, C, KP, N1, false>::Lds);
    static_assert(l0 <= kDeltaMaxLds && l1 <= kDeltaMaxLds, "LDS of a workgroup");
    const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void *>(&delta_state_kernel<T, C, KP, false>),
                                             hipFuncAttributeMaxDynamicSharedMemorySize, l0);
    return e != hipSuccess ? e : hipFuncSetAttribute(reinterpret_cast<const void *>(&delta_state_kernel<T, C, KP, true>),
                                                     hipFuncAttributeMaxDynamicSharedMemorySize, l1);
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

hipError_t launch_delta_fwd(const DeltaArgs &a, const DeltaWs &ws, bool is_bf16, hipStream_t st) {
    return is_bf16 ? fwd_pick<bf16>(a, ws, st) : fwd_pick<float>(a, ws, st);
}

size_t delta_mats_bytes(int K, bool is_bf16, bool backward) {
    const bool three = backward || !is_bf16;
    if (delta_chunk(K) == 64) return three ? sizeof(ChunkMats<64, 3>) : sizeof(ChunkMats<64, 2>);
    return three ? sizeof(ChunkMats<32, 3>) : sizeof(ChunkMats<32, 2>);
}

}  // namespace sdm
