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

// The lower 32 x 32 blocks of the row-major m.
template <int C> __device__ __forceinline__ void put_blocks(const float *m, float (*out)[32][32]) {
    constexpr int LC = PrepLds<C>::LC;
    for (int i = threadIdx.x; i < kTri<C> * 256; i += 256) {
        const int b = i / 256, r = i % 256 / 8, c = i % 8, br = b > 0, bc = b == 2;
        reinterpret_cast<dt4 *>(out)[i] = *reinterpret_cast<const dt4 *>(m + (br * 32 + r) * LC + bc * 32 + c * 4);
    }
}

// X, P and the gates of one chunk per workgroup. A wavefront takes 16 rows of both products, with all its operands on their way
// before the first one; the inverse is substitution within blocks of 16 and products between them, in float32.
// Measured: 56 us for the 4096 chunks of 16 heads of 16384 tokens (head_dim 128, bfloat16), four workgroups on a compute unit (61
// with three, whose registers the compiler takes if it may); 170 MB in and out are 33 us at a copy's 5.1 TB/s. The rest is
// its chain of phases: the operands' way from memory, 16 dependent steps of substitution, the two joins.
template <typename T, int C, int KP>
__global__ __launch_bounds__(256, sizeof(T) == 2 ? 4 : 1) void delta_prep_kernel(DeltaArgs a, DeltaWs ws) {
    constexpr int LC = PrepLds<C>::LC, NT = C / 16, NI = kPieces<T>;
    __shared__ PrepLds<C> s;
    const int64_t n = blockIdx.x;
    const int c = int(n % ws.Nt), h = int(n / ws.Nt % a.Hv), p = int(n / ws.Nt / a.Hv), hk = h / (a.Hv / a.Hk);
    const int t0 = c * C, live = min(C, delta_valid(a, p) - t0);
    if (live <= 0) return;
    const int tid = threadIdx.x, lane = tid & 63, wv = tid >> 6, lc = lane & 15, lg = lane >> 4;
    // every operand is on its way before the first product: row tile wv of q and row tiles 0 .. wv of k
    const int row = wv * 16 + lc;
    constexpr int KB = KP / 32;
    Frag<NI> fk[NT][KB], fq[KB];
    if (wv < NT) {
        const bf16 *k = a.kk.data + p * a.kk.sp + hk * a.kk.sh + t0 * a.kk.st;
        const bf16 *q = a.qq.data + p * a.qq.sp + hk * a.qq.sh + t0 * a.qq.st;
#pragma unroll
        for (int kb = 0; kb < KB; ++kb) {
            const int d = kb * 32 + lg * 8;
            fq[kb] = load_keys<NI>(q + (min(row, live - 1) * int(a.qq.st) + d), a.qq.plane);
#pragma unroll
            for (int ct = 0; ct < NT; ++ct)
                if (ct <= wv) fk[ct][kb] = load_keys<NI>(k + (min(ct * 16 + lc, live - 1) * int(a.kk.st) + d), a.kk.plane);
        }
    }
    if (wv == (NT == 4 ? 0 : 3)) {      // the wavefront with the fewest products
        const bool in = lane < C && lane < live;
        const double G = chunk_G<C>(in ? a.g[(int64_t(p) * a.T + t0 + lane) * a.Hv + h] : 0.0f), GL = __shfl(G, C - 1, 64);
        if (lane < C) {
            s.G[lane] = G;
            s.g.beta[lane] = in ? a.beta[(int64_t(p) * a.T + t0 + lane) * a.Hv + h] : 0.0f;
            s.g.eG[lane] = in ? exp2_of(G) : 0.0f;
            s.g.eL[lane] = in ? exp2_of(GL - G) : 0.0f;
        }
        if (lane == 0) s.g.last = exp2_of(GL);
    }
    dt4 kk[NT] = {}, qk[NT] = {};
    if (wv < NT) {
        // rows past the last valid token are cleared: their columns of X and P, and rows of P, are then 0
#pragma unroll
        for (int kb = 0; kb < KB; ++kb) {
            if (row >= live) clear(fq[kb]);
            Frag<NI> fa;
#pragma unroll
            for (int ct = 0; ct < NT; ++ct)
                if (ct <= wv) {
                    if (ct * 16 + lc >= live) clear(fk[ct][kb]);
                    if (ct == wv) fa = fk[ct][kb];
                }
#pragma unroll
            for (int ct = 0; ct < NT; ++ct)
                if (ct <= wv) {
                    kk[ct] = mma<3>(fa, fk[ct][kb], kk[ct]);
                    qk[ct] = mma<3>(fq[kb], fk[ct][kb], qk[ct]);
                }
        }
    }
    lds_barrier();
    if (wv < NT) {
        double Gr[4];
        float b[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int row = wv * 16 + 4 * lg + r;
            Gr[r] = s.G[row];
            b[r] = ws.backward ? delta_beta_safe(s.g.beta[row]) : s.g.beta[row];
        }
#pragma unroll
        for (int ct = 0; ct < NT; ++ct) {
            const int col = ct * 16 + lc;
            const double Gc = ct <= wv ? s.G[col] : 0.0;
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int row = wv * 16 + 4 * lg + r;
                float l = 0.0f, x = 0.0f;
                if (ct <= wv) {
                    const float D = exp2_of(Gr[r] - Gc);
                    l = row > col ? b[r] * (D * kk[ct][r]) : 0.0f;
                    x = row >= col ? a.scale * (D * qk[ct][r]) : 0.0f;
                }
                s.L[row * LC + col] = l;
                s.X[row * LC + col] = x;
            }
        }
    }
    lds_barrier();
    ChunkMem<C> *out = reinterpret_cast<ChunkMem<C> *>(ws.mats) + n;
    put_blocks<C>(s.X, out->P);
    if (tid < int(sizeof(Gates<C>) / 4)) reinterpret_cast<float *>(&out->g)[tid] = reinterpret_cast<const float *>(&s.g)[tid];
    lds_barrier();     // X's blocks above the diagonal stay the zeros that P has there
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
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) s.X[(wv * 16 + i) * LC + wv * 16 + lane] = x[i];
    }
    lds_barrier();
    // ... then [A 0; B D]^-1 = [A^-1 0; -D^-1 B A^-1 D^-1]: of blocks of 16, a wavefront each with B A^-1 in B's place,
    auto put = [&](float *d, float sign, dt4 x) {
#pragma unroll
        for (int r = 0; r < 4; ++r) d[(4 * lg + r) * LC + lc] = sign * x[r];
    };
    if (wv < NT / 2) {
        const int at = (wv * 32 + 16) * LC + wv * 32;
        put(s.L + at, 1.0f, f32_mma(s.L + at, s.X + wv * 32 * (LC + 1), LC, dt4{}));
        __builtin_amdgcn_wave_barrier();
        put(s.X + at, -1.0f, f32_mma(s.X + at + 16, s.L + at, LC, dt4{}));
    }
    lds_barrier();
    // ... and of blocks of 32, a 16 x 16 tile per wavefront, with B A^-1 in the block above the diagonal, which nobody reads.
    if constexpr (C == 64) {
        const int r0 = wv / 2 * 16, c0 = wv % 2 * 16;
        dt4 x{};
#pragma unroll
        for (int kb = 0; kb < 32; kb += 16) x = f32_mma(s.L + (32 + r0) * LC + kb, s.X + kb * LC + c0, LC, x);
        put(s.X + r0 * LC + 32 + c0, 1.0f, x);
        lds_barrier();
        x = dt4{};
#pragma unroll
        for (int kb = 0; kb < 32; kb += 16) x = f32_mma(s.X + (32 + r0) * LC + 32 + kb, s.X + kb * LC + 32 + c0, LC, x);
        put(s.X + (32 + r0) * LC + c0, -1.0f, x);
        lds_barrier();
    }
    put_blocks<C>(s.X, out->X);
}

// Every column of the state evolves on its own: a wavefront keeps 16 columns of S in
// accumulators through the whole sequence, and the four wavefronts of a workgroup share the
// chunk's k, q, X and P in LDS. One wavefront per SIMD has nothing beside it to hide its waits: the
// operands of each group of products are read from LDS before the group ahead of it.
// Precision: S, U, X and P are three bfloat16 pieces each wherever they go, so that products keep float32's bits (2^-23); the readings
// are rounded once. (Two pieces of S, U and P where they reach bfloat16 readings took 222 us where this takes 249 for 4 x 16 heads of
// 4096 tokens of 128 x 128, but terms of a reading that cancel then had 16 bits.)
// Bound by that one wavefront's chain: a chunk of 64 tokens of 128 x 128 (bfloat16) takes 3.9 us with half of the compute units
// at work, 5.0 with all: of the 8700 cycles of the first, 3456 in 216 matrix instructions (by counters), the rest splits,
// gates and the way from one group of products through LDS or a split to the next.
// kRead gives the readings (4 x 16 heads of up to 4096 tokens: 235 us). kSave keeps U and each chunk's start state for the
// backward instead, kBoth does both (4 x 16 heads of 2048 tokens: 160 us). kMap, for sequences walked in segments at once: the
// segment's end state from a start state of zeros (the first's: from the caller's) and, in workgroups of their own, what it
// makes of the columns of the identity, with v = 0: the two give a segment's end state from any start state
// (delta_join_kernel); 2.6 us a chunk.
enum { kRead, kSave, kBoth, kMap };
template <typename T, int C, int KP, int MODE>
__global__ __launch_bounds__(kWalkThreads) void delta_state_kernel(DeltaArgs a, DeltaWs ws) {
    constexpr bool SAVE = MODE == kSave || MODE == kBoth, READ = MODE == kRead || MODE == kBoth;
    constexpr int NI = kPieces<T>, KB = KP / 32, TB = C / 32, NTR = kTri<C>;
    using W = Walk<T, C, KP, READ>;
    extern __shared__ __align__(16) unsigned char raw[];
    typename W::Lds *bufs = reinterpret_cast<typename W::Lds *>(raw);
    const int vslices = (a.V + 63) / 64, VG = (a.V + 15) / 16, VP = VG * 16, heads = a.P * a.Hv;
    const int slices = MODE == kMap ? vslices + KP / 64 : vslices, seg = blockIdx.x / (heads * slices);
    const int block = blockIdx.x % (heads * slices), slice = BlockAt(block, slices, heads, a.Hv / a.Hk).slice;
    const int ph = BlockAt(block, slices, heads, a.Hv / a.Hk).ph, h = ph % a.Hv, p = ph / a.Hv, hk = h / (a.Hv / a.Hk);
    const bool map = MODE == kMap && slice >= vslices;     // columns of the identity
    if (map && seg == 0) return;
    const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lc = lane & 15, lg = lane >> 4;
    const int cg = (map ? slice - vslices : slice) * 4 + (wv & 3), col = cg * 16 + lc;
    const bool in = !map && col < a.V;
    const int n = delta_valid(a, p), Nc = (n + C - 1) / C, c0 = seg * ws.seg_chunks, c1 = min(c0 + ws.seg_chunks, Nc);
    if (wv >= 4) {
        typename W::Bring w(a, ws, p, h, hk, ph, cg, a.v, n);
        w.run(bufs, c0, 1, c1 - c0);
        return;
    }
    float *seg_state = ws.seg_state + int64_t(seg) * heads * KP * VP;
    const int oc = cg * 16 + lg * 4;   // readings come transposed: a lane holds four columns of the tokens block_row(lc, .)
    T *out = static_cast<T *>(a.out) + (int64_t(p) * a.T * a.Hv + h) * a.V;
    const int os = a.Hv * a.V;
    dt4 S[KB][2];
    // Walked in segments, the readings' launch writes the final state in one workgroup while others begin: it reads start states from
    // the workspace alone, the first segment's too, since the caller's state may be advanced in place.
    if (MODE == kRead && ws.segs > 1) load_state<KB>(S, seg_state, ph, KP, VP, col);
    else if (seg == 0) load_state<KB>(S, a.state, ph, a.K, a.V, col);
    else {
#pragma unroll
        for (int kb = 0; kb < KB; ++kb)
#pragma unroll
            for (int e = 0; e < 2; ++e)
#pragma unroll
                for (int r = 0; r < 4; ++r) S[kb][e][r] = map && kb * 32 + lg * 8 + e * 4 + r == col ? 1.0f : 0.0f;
    }
    if (MODE == kMap && seg == 0) store_state<KB>(S, seg_state, ph, KP, VP, col);
    W::begin();
    dt4 y[TB][2] = {};
    const int left = a.V - oc;
    auto put = [&](int c) {
        T *o = out + int64_t(c) * C * os;
        const int live = n - c * C;
        if (live >= C) {
            if (left >= 4) {
#pragma unroll
                for (int tb = 0; tb < TB; ++tb)
#pragma unroll
                    for (int e = 0; e < 2; ++e) put_four(o + ((tb * 32 + block_row(lc, e)) * os + oc), 4, y[tb][e]);
                return;
            }
        }
#pragma unroll
        for (int tb = 0; tb < TB; ++tb)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int t = tb * 32 + block_row(lc, e);
                if (t < live && left > 0) put_four(o + (t * os + oc), left, y[tb][e]);
            }
    };
    Frag<3> fs[KB];
#pragma unroll
    for (int kb = 0; kb < KB; ++kb) fs[kb] = split<3>(S[kb][0], S[kb][1]);
    for (int c = c0; c < c1; ++c) {
        const typename W::Lds &s = bufs[(c - c0) & (W::kBufs - 1)];
        const Gates<C> &g = s.m.g;
        const int ln = NI == 1 ? fresh_lane() : lane;     // float32 inputs spill more with addresses of each chunk's own
        if (READ && c > c0) put(c - 1);
        // k S and q S
        Frag<NI> A[2][TB][2];
        auto rows_of = [&](Frag<NI>(&f)[TB][2], const unsigned char *m) {
#pragma unroll
            for (int tb = 0; tb < TB; ++tb)
#pragma unroll
                for (int e = 0; e < 2; ++e) f[tb][e] = read_rows<NI>(m + tb * KB * kBlk, W::kStride, e, ln);
        };
        rows_of(A[0], s.k[0][0][0]);
        dt4 v[TB][2], b[TB][2], eG[TB][2];
        float et[TB][2];             // exp(G) of the lane's tokens in the transposed readings
#pragma unroll
        for (int tb = 0; tb < TB; ++tb)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int t = tb * 32 + lg * 8 + e * 4;
                v[tb][e] = W::value(s, tb, e);
                if (MODE != kRead && !in) v[tb][e] = dt4{};
                b[tb][e] = *reinterpret_cast<const dt4 *>(g.beta + t);
                eG[tb][e] = *reinterpret_cast<const dt4 *>(g.eG + t);
                et[tb][e] = g.eG[tb * 32 + block_row(lc, e)];
            }
        const int64_t nc = int64_t(ph) * ws.Nt + c;
        if constexpr (SAVE) save_blocks<KB>(ws.S, nc, VG, cg, S);
        dt4 x[TB][2] = {};
#pragma unroll
        for (int tb = 0; tb < TB; ++tb) y[tb][0] = y[tb][1] = dt4{};
        constexpr int KQ = READ ? 2 * KB : KB;
        Frag<3> fx[2][2], fr[TB];    // X's blocks, a step ahead
        auto x_of = [&](Frag<3>(&f)[2], int i) {
#pragma unroll
            for (int e = 0; e < 2; ++e) f[e] = read_rows<3>(s.m.X[0][i], NTR * kBlk, e, ln);
        };
#pragma unroll
        for (int i = 0; i < KQ; ++i) {
            if (i + 1 < KB) rows_of(A[(i + 1) & 1], s.k[0][0][i + 1]);
            else if (i + 1 < KQ) rows_of(A[(i + 1) & 1], s.q[0][0][i + 1 - KB]);
            else x_of(fx[0], 0);
            lds_point();
            if (i < KB) {
                each_product<3, NI, 3>([&](int m, int l) {
#pragma unroll
                    for (int tb = 0; tb < TB; ++tb)
#pragma unroll
                        for (int e = 0; e < 2; ++e) x[tb][e] = mma1(A[i & 1][tb][e].p[m], fs[i % KB].p[l], x[tb][e]);
                });
            } else {
                each_product<3, NI, 3>([&](int m, int l) {
#pragma unroll
                    for (int tb = 0; tb < TB; ++tb)
#pragma unroll
                        for (int e = 0; e < 2; ++e) y[tb][e] = mma1(fs[i % KB].p[l], A[i & 1][tb][e].p[m], y[tb][e]);
                });
            }
            if (i == KB - 1) {
#pragma unroll
                for (int tb = 0; tb < TB; ++tb) {
                    dt4 r[2];
#pragma unroll
                    for (int e = 0; e < 2; ++e)
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            r[e][j] = (SAVE ? delta_beta_safe(b[tb][e][j]) : b[tb][e][j]) * (v[tb][e][j] - eG[tb][e][j] * x[tb][e][j]);
                    fr[tb] = split<3>(r[0], r[1]);
                }
            }
            lds_point();
        }
        // U = X r, then P U; block i of the lower triangle is row block i > 0, column block i == 2
        dt4 U[TB][2] = {};
        Frag<3> fp[2][2];
        auto p_of = [&](Frag<3>(&f)[2], int i) {
#pragma unroll
            for (int e = 0; e < 2; ++e) f[e] = read_rows<3>(s.m.P[0][i], NTR * kBlk, e, ln);
        };
        Frag<NI> fk[2][KB];          // blocks of k^T, half of a row block of them at a time (the halves of all row blocks in turn)
        auto kt_of = [&](Frag<NI>(&f)[KB], int i) {
#pragma unroll
            for (int m = 0; m < KB; ++m) {
                const int kb = i / TB * (KB / 2) + m / 2;
                f[m] = read_cols<NI>(s.k[0][i % TB][kb], W::kStride, m & 1, ln);
            }
        };
#pragma unroll
        for (int i = 0; i < NTR; ++i) {
            if (i + 1 < NTR) x_of(fx[(i + 1) & 1], i + 1);
            else if constexpr (READ) p_of(fp[0], 0);
            else kt_of(fk[0], 0);
            lds_point();
            each_product<3, 3, 3>([&](int m, int l) {
#pragma unroll
                for (int e = 0; e < 2; ++e) U[i > 0][e] = mma1(fx[i & 1][e].p[m], fr[i == 2].p[l], U[i > 0][e]);
            });
            lds_point();
        }
        Frag<3> fu[TB];
        dt4 eL[TB][2];
#pragma unroll
        for (int tb = 0; tb < TB; ++tb)
#pragma unroll
            for (int e = 0; e < 2; ++e) eL[tb][e] = *reinterpret_cast<const dt4 *>(g.eL + tb * 32 + lg * 8 + e * 4);
        const float last = g.last;
        if constexpr (SAVE) save_blocks<TB>(ws.U, nc, VG, cg, U);
        if constexpr (READ) {
            Frag<3> fv[TB];
#pragma unroll
            for (int tb = 0; tb < TB; ++tb) {
                fv[tb] = split<3>(U[tb][0], U[tb][1]);
#pragma unroll
                for (int e = 0; e < 2; ++e) y[tb][e] *= a.scale * et[tb][e];
            }
#pragma unroll
            for (int i = 0; i < NTR; ++i) {
                if (i + 1 < NTR) p_of(fp[(i + 1) & 1], i + 1);
                else kt_of(fk[0], 0);
                lds_point();
                each_product<3, 3, 3>([&](int m, int l) {
#pragma unroll
                    for (int e = 0; e < 2; ++e) y[i > 0][e] = mma1(fv[i == 2].p[l], fp[i & 1][e].p[m], y[i > 0][e]);
                });
                lds_point();
            }
        }
        // S = e^{G_C} S + k^T (e^{G_C - G} U)
#pragma unroll
        for (int tb = 0; tb < TB; ++tb) {
#pragma unroll
            for (int e = 0; e < 2; ++e) U[tb][e] *= eL[tb][e];
            fu[tb] = split<3>(U[tb][0], U[tb][1]);
        }
#pragma unroll
        for (int kb = 0; kb < KB; ++kb)
#pragma unroll
            for (int e = 0; e < 2; ++e) S[kb][e] *= last;
#pragma unroll
        for (int i = 0; i < 2 * TB; ++i) {
            if (i + 1 < 2 * TB) kt_of(fk[(i + 1) & 1], i + 1);
            lds_point();
            each_product<3, NI, 3>([&](int x, int l) {
#pragma unroll
                for (int m = 0; m < KB; ++m) {
                    const int kb = i / TB * (KB / 2) + m / 2;
                    S[kb][m & 1] = mma1(fk[i & 1][m].p[x], fu[i % TB].p[l], S[kb][m & 1]);
                }
            });
            lds_point();
            if (i % TB == TB - 1) {      // half of the rows are there
#pragma unroll
                for (int kb = i / TB * (KB / 2); kb < (i / TB + 1) * (KB / 2); ++kb) fs[kb] = split<3>(S[kb][0], S[kb][1]);
            }
        }
        W::turn();
    }
    if constexpr (READ) {
        if (c1 > c0) put(c1 - 1);
        const int end = seg + 1 < ws.segs ? min(a.T, (c0 + ws.seg_chunks) * C) : a.T;
        for (int t = max(n, c0 * C) + lc; t < end; t += 16)
            if (left > 0) put_four(out + (int64_t(t) * os + oc), left, dt4{});
        // the segment with the last chunk; the first one where there is none
        if (seg == (Nc > 0 ? (Nc - 1) / ws.seg_chunks : 0)) store_state<KB>(S, a.state_out, ph, a.K, a.V, col);
    }
    if constexpr (MODE == kMap) {
        if (map) store_state<KB>(S, ws.seg_map + int64_t(seg) * heads * KP * KP, ph, KP, KP, col);
        else store_state<KB>(S, seg_state + int64_t(heads) * KP * VP, ph, KP, VP, col);
    }
}

// The segments' start states from their maps M and their end states from zeros N, in order: S_{i + 1} = M_i S_i + N_i. A
// workgroup takes 16 columns, its four wavefronts a quarter of the rows each, which meet in LDS between the steps; the next step's
// M is on its way under the products. (A wavefront for all the rows of 16 columns, splitting all of M by itself, took
// 38 us for three steps of 16 heads of 128 x 128; this takes 13.5.)
template <int KP> __global__ __launch_bounds__(256, 1) void delta_join_kernel(DeltaWs ws, int heads, int VP) {
    constexpr int KB = KP / 32, TILES = KB / 2, BUF = KP <= 128 ? 2 : 1;     // TILES of a wavefront, 16 rows each
    __shared__ dt4 shared[2][2 * KB][64];
    const int VG = VP / 16, ph = blockIdx.x / VG, lane = threadIdx.x & 63, lc = lane & 15, lg = lane >> 4;
    const int col = int(blockIdx.x) % VG * 16 + lc, t0 = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) * TILES;
    auto at = [&](int i, int t) { return (int64_t(i) * heads + ph) * KP * VP + int64_t(t / 2 * 32 + lg * 8 + t % 2 * 4) * VP + col; };
    auto tile_of = [&](int i, int t) {
        dt4 x;
#pragma unroll
        for (int r = 0; r < 4; ++r) x[r] = ws.seg_state[at(i, t) + r * VP];
        return x;
    };
    struct Next {
        dt4 m[TILES][KB][2], n[TILES];
    } next[BUF];
    auto load = [&](Next &x, int i) {
        const float *M = ws.seg_map + (int64_t(i) * heads + ph) * KP * KP + lg * 8;
#pragma unroll
        for (int j = 0; j < TILES; ++j) {
            const float *row = M + ((t0 + j) / 2 * 32 + block_row(lc, (t0 + j) & 1)) * KP;
#pragma unroll
            for (int kb = 0; kb < KB; ++kb)
#pragma unroll
                for (int e = 0; e < 2; ++e) x.m[j][kb][e] = *reinterpret_cast<const dt4 *>(row + kb * 32 + e * 4);
            x.n[j] = tile_of(i + 1, t0 + j);
        }
    };
    const int last = ws.segs - 2;
#pragma unroll
    for (int j = 0; j < TILES; ++j) shared[1][t0 + j][lane] = tile_of(1, t0 + j);
    if (last > 0) load(next[0], 1);
    lds_barrier();
    auto step = [&](int i, Next &now, Next &then) {
        Frag<3> fs[KB];
#pragma unroll
        for (int kb = 0; kb < KB; ++kb) fs[kb] = split<3>(shared[i & 1][2 * kb][lane], shared[i & 1][2 * kb + 1][lane]);
        if (BUF == 2 && i < last) load(then, i + 1);
#pragma unroll
        for (int j = 0; j < TILES; ++j) {
            dt4 x[2] = {now.n[j], dt4{}};
#pragma unroll
            for (int kb = 0; kb < KB; ++kb) x[kb & 1] = mma<3>(split<3>(now.m[j][kb][0], now.m[j][kb][1]), fs[kb], x[kb & 1]);
            x[0] += x[1];
            shared[~i & 1][t0 + j][lane] = x[0];
#pragma unroll
            for (int r = 0; r < 4; ++r) ws.seg_state[at(i + 1, t0 + j) + r * VP] = x[0][r];
        }
        if (BUF == 1 && i < last) load(then, i + 1);
        lds_barrier();
    };
    for (int i = 1; i <= last; i += 2) {
        step(i, next[0], next[BUF - 1]);
        if (i < last) step(i + 1, next[BUF - 1], next[0]);
    }
}

// Rows of q or k as dense rows of KP elements, padded with zeros, a plane per piece: eight elements per thread. Only rows that the
// walking kernels cannot load by 16 bytes (see delta_regular_keys) and float32 ones, whose pieces are made once here, come
// this way: 3.8 us for 903 tokens of 3 heads of 40 (a launch; 2.6 MB).
template <typename T> __global__ __launch_bounds__(256) void delta_copy_keys_kernel(Rows r, bf16 *out, int64_t rows, int tokens, int heads, int KP) {
    const T *src = static_cast<const T *>(r.data);
    const int per = KP / 8;
    for (int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x; i < rows * per; i += int64_t(gridDim.x) * 256) {
        const int64_t row = i / per, t = row / heads % tokens, p = row / heads / tokens;
        const int c = int(i % per) * 8, h = int(row % heads);
        const T *x = src + p * r.sp + t * r.st + h * r.sh;
        dt4 v[2];
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j / 4][j % 4] = c + j < r.width ? to_f32(x[c + j]) : 0.0f;
        const Frag<kPieces<T>> f = split<kPieces<T>>(v[0], v[1]);
#pragma unroll
        for (int n = 0; n < kPieces<T>; ++n) *reinterpret_cast<db8 *>(out + n * rows * KP + row * KP + c) = f.p[n];
    }
}
// Rows of v, or of the readings' gradient, as dense rows of VP elements, padded with zeros.
template <typename T> __global__ __launch_bounds__(256) void delta_copy_values_kernel(Rows r, T *out, int64_t rows, int tokens, int heads, int VP) {
    const T *src = static_cast<const T *>(r.data);
    for (int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x; i < rows * VP; i += int64_t(gridDim.x) * 256) {
        const int64_t row = i / VP, t = row / heads % tokens, p = row / heads / tokens;
        const int c = int(i % VP), h = int(row % heads);
        out[i] = c < r.width ? src[p * r.sp + t * r.st + h * r.sh + c] : from_f32<T>(0.0f);
    }
}

template <typename T, int C, int KP> hipError_t fwd_go(const DeltaArgs &a, const DeltaWs &ws, bool results, hipStream_t st) {
    const dim3 chunks(unsigned(int64_t(a.P) * a.Hv * ws.Nt));
    if (ws.Nt > 0) {
        hipLaunchKernelGGL((delta_prep_kernel<T, C, KP>), chunks, dim3(256), 0, st, a, ws);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    const unsigned heads = unsigned(a.P) * unsigned(a.Hv), slices = unsigned(a.V + 63) / 64;
    if (ws.backward) {
        if (results)     // a call without tokens has no `out`, but a final state
            hipLaunchKernelGGL((delta_state_kernel<T, C, KP, kBoth>), dim3(heads * slices), dim3(kWalkThreads), (Walk<T, C, KP, true>::kLds), st, a, ws);
        else
            hipLaunchKernelGGL((delta_state_kernel<T, C, KP, kSave>), dim3(heads * slices), dim3(kWalkThreads), (Walk<T, C, KP, false>::kLds), st, a, ws);
        return hipGetLastError();
    }
    if (ws.segs > 1) {
        hipLaunchKernelGGL((delta_state_kernel<T, C, KP, kMap>), dim3(heads * (slices + KP / 64) * unsigned(ws.segs - 1)), dim3(kWalkThreads),
                           (Walk<T, C, KP, false>::kLds), st, a, ws);
        hipLaunchKernelGGL(delta_join_kernel<KP>, dim3(heads * (unsigned(a.V + 15) / 16)), dim3(256), 0, st, ws, int(heads), (a.V + 15) / 16 * 16);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    hipLaunchKernelGGL((delta_state_kernel<T, C, KP, kRead>), dim3(heads * slices * unsigned(ws.segs)), dim3(kWalkThreads), (Walk<T, C, KP, true>::kLds), st, a, ws);
    return hipGetLastError();
}
template <typename T> hipError_t fwd_pick(const DeltaArgs &a, const DeltaWs &ws, bool results, hipStream_t st) {
    switch (delta_kp(a.K)) {
        case 64: return fwd_go<T, kChunk<T>, 64>(a, ws, results, st);
        case 128: return fwd_go<T, kChunk<T>, 128>(a, ws, results, st);
        default: return fwd_go<T, 32, 256>(a, ws, results, st);
    }
}

template <typename T, int C, int KP> hipError_t fwd_attr() {
    constexpr size_t l0 = Walk<T, C, KP, true>::kLds, l1 = Walk<T, C, KP, false>::kLds;
    static_assert(l0 <= kDeltaMaxLds && l1 <= kDeltaMaxLds, "LDS of a workgroup");
    auto set = [](auto kernel, size_t bytes) {
        return hipFuncSetAttribute(reinterpret_cast<const void *>(kernel), hipFuncAttributeMaxDynamicSharedMemorySize, int(bytes));
    };
    hipError_t e = set(&delta_state_kernel<T, C, KP, kRead>, l0);
    if (e == hipSuccess) e = set(&delta_state_kernel<T, C, KP, kSave>, l1);
    if (e == hipSuccess) e = set(&delta_state_kernel<T, C, KP, kBoth>, l0);
    return e == hipSuccess ? set(&delta_state_kernel<T, C, KP, kMap>, l1) : e;
}
template <typename T> hipError_t fwd_attrs() {
    hipError_t e = fwd_attr<T, kChunk<T>, 64>();
    if (e == hipSuccess) e = fwd_attr<T, kChunk<T>, 128>();
    if (e == hipSuccess) e = fwd_attr<T, 32, 256>();
    return e;
}

}  // namespace

hipError_t delta_prepare() {
    const hipError_t e = fwd_attrs<float>();
    return e == hipSuccess ? fwd_attrs<bf16>() : e;
}

hipError_t launch_delta_fwd(const DeltaArgs &a, const DeltaWs &ws, bool is_bf16, bool results, hipStream_t st) {
    return is_bf16 ? fwd_pick<bf16>(a, ws, results, st) : fwd_pick<float>(a, ws, results, st);
}

static bool rows_aligned(const Rows &r, int elements) {
    return reinterpret_cast<uintptr_t>(r.data) % 16 == 0 && r.sp % elements == 0 && r.st % elements == 0 && r.sh % elements == 0 &&
           r.st < kDeltaMaxStride;
}
bool delta_regular_keys(const Rows &r, bool is_bf16) { return is_bf16 && r.width == delta_kp(r.width) && rows_aligned(r, 8); }
bool delta_regular_values(const Rows &r, bool is_bf16) { return r.width % 8 == 0 && rows_aligned(r, is_bf16 ? 8 : 4); }

static unsigned copy_grid(int64_t threads) { return unsigned(threads / 256 + 1 < 8192 ? threads / 256 + 1 : 8192); }

hipError_t launch_delta_copy_keys(const Rows &r, KeyRows *k, void *to, int P, int T, int H, bool is_bf16, bool there, hipStream_t st) {
    const int KP = delta_kp(r.width);
    const int64_t rows = int64_t(P) * T * H;
    bf16 *out = static_cast<bf16 *>(to);
    const dim3 grid(copy_grid(rows * (KP / 8)));
    *k = {out, rows * KP, int64_t(T) * H * KP, int64_t(H) * KP, KP};
    if (there) return hipSuccess;
    if (is_bf16) hipLaunchKernelGGL(delta_copy_keys_kernel<bf16>, grid, dim3(256), 0, st, r, out, rows, T, H, KP);
    else hipLaunchKernelGGL(delta_copy_keys_kernel<float>, grid, dim3(256), 0, st, r, out, rows, T, H, KP);
    return hipGetLastError();
}

hipError_t launch_delta_copy_values(Rows *r, void *to, int P, int T, int H, bool is_bf16, bool there, hipStream_t st) {
    const int VP = (r->width + 7) / 8 * 8;
    const int64_t rows = int64_t(P) * T * H;
    const dim3 grid(copy_grid(rows * VP));
    const Rows from = *r;
    *r = {to, int64_t(T) * H * VP, int64_t(H) * VP, VP, VP};
    if (there) return hipSuccess;
    if (is_bf16) hipLaunchKernelGGL(delta_copy_values_kernel<bf16>, grid, dim3(256), 0, st, from, static_cast<bf16 *>(to), rows, T, H, VP);
    else hipLaunchKernelGGL(delta_copy_values_kernel<float>, grid, dim3(256), 0, st, from, static_cast<float *>(to), rows, T, H, VP);
    return hipGetLastError();
}

// A workgroup walks a sequence's chunks one after the other, at a pace that hardly depends on the others: few states leave
// most of the device idle. Walking segments at once costs the readings' walk again, once for the columns of the state and once
// for those of the map, a third cheaper (no readings), and a join of about a chunk's time per segment; a launch's workgroups beyond
// a compute unit each come in turns. Times below are in chunks of the readings' walk, and segments have to gain a tenth.
// Measured, whole call, one walk / the segments taken (us): bfloat16, 16 heads of 16384 tokens of 128 x 128 872 / 357 (5; with 8 335, with
// 3 527); 8 of 8192 of 200 x 200 773 / 343 (5); 64 of 2048 of 64 x 64 121 / 93 (3; with 8 115); float32, 16 of 4096 of 128 x 128 405 / 200
// (5; with 6 226); 8 of 16384 of 64 x 64 1011 / 205 (15); 4 of 4096 of 256 x 256 1007 / 315 (8). Four heads of 1344 tokens of 72 x 40,
// bfloat16, stay at one walk (89) where five segments would take 66.
int delta_segments(int64_t heads, int slices, int K, int Nt) {
    const int64_t wgs = heads * slices, maps = heads * (slices + delta_kp(K) / 64);
    int best = 1;
    double least = double(Nt);
    if (wgs * 2 > kCus) return 1;
    for (int g = 3; g <= 32 && Nt / g >= 4; ++g) {
        const int64_t len = (Nt + g - 1) / g;
        const int64_t a = (wgs + (g - 2) * maps + kCus - 1) / kCus, b = (wgs * g + kCus - 1) / kCus;
        const double t = double(len) * (0.7 * double(a) + double(b)) + 1.0 * double(g) + 6.0;
        if (t < 0.9 * least) {
            least = t;
            best = g;
        }
    }
    return best;
}

size_t delta_mats_bytes(int K, bool is_bf16) { return delta_chunk(K, is_bf16) == 64 ? sizeof(ChunkMem<64>) : sizeof(ChunkMem<32>); }

}  // namespace sdm
