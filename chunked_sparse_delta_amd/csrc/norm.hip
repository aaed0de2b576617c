// Layer norm over the last axis, forward and backward.
//
//   mean = sum(x) / N, var = sum((x - mean)^2) / N, rstd = 1 / sqrt(var + eps)
//   y = (x - mean) rstd w + b
// and with h = dy w, xh = (x - mean) rstd:
//   dx = rstd (h - sum(h) / N - xh sum(h xh) / N),  dw = sum over rows (dy xh),  db = sum over rows (dy)
//
// Both passes are bound by memory: each row is read once into registers (16 bytes per lane
// and load) and its sums run there in float32, so the variance is that of the differences
// from the mean. A row belongs to L lanes (8 to 1024, the fewest that can hold it,
// norm_max_items), several rows to a wavefront where they are short; rows of more columns than 1024 lanes hold are walked
// in memory. Rows need no alignment beyond their element's: a vector load or store
// takes any element address, and the columns left over after the whole vectors go one by one.
//
// The backward's sums over rows have a fixed order: workgroup g of G takes the row groups g, g + G, ...,
// keeps its columns' sums in registers and writes them once; a second kernel adds the G
// partial rows in order.
//
// Measured, 16384 rows of 4096 bfloat16 columns: forward 47 us (5.7 TB/s; 59 in the middle of a training step), backward 82 to 91
// us (402 MB, 4.4 to 4.9 TB/s) and 4 for the sums over workgroups; a large copy: 5.1 TB/s. 64 rows: 5 us, a launch and two ways
// to memory. 1001 rows of 1537 float32 columns: 7.8 and 10.7 + 4.3 us.
#include "norm_vec.h"
#include "host.h"

namespace sdm {

namespace {

// Vectors of a row that one of its L lanes may hold: as many as the registers take without costing the wavefronts that
// hide each other's loads (the backward holds seven arrays of that size: 8192 bfloat16 columns took 130 us
// with four vectors in 256 lanes and 85 us with one in 1024, 8192 rows). Fewer than 64 lanes hold one each.
constexpr int norm_max_items(int L, int V, bool bwd) {
    const int elems = L < 64 ? V : bwd || L == 64 ? 16 : L == 256 ? 64 : 32;
    return elems / V < 8 ? elems / V : 8;
}

// Sums of a and b over the row's L lanes (each gets them). `buf` holds two floats per wavefront of a row of more than one
// and is used by one sum at a time: two buffers taken in turn need one barrier each.
template <int L> __device__ __forceinline__ float2 row_sum(float a, float b, float *buf) {
#pragma unroll
    for (int m = (L < 64 ? L : 64) / 2; m > 0; m >>= 1) {
        a += __shfl_xor(a, m, 64);
        b += __shfl_xor(b, m, 64);
    }
    if constexpr (L > 64) {
        const int w = threadIdx.x >> 6;
        if ((threadIdx.x & 63) == 0) {
            buf[2 * w] = a;
            buf[2 * w + 1] = b;
        }
        // orders LDS only: the next row's loads stay on their way
        __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
        __builtin_amdgcn_s_barrier();
        __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
        a = b = 0.0f;
#pragma unroll
        for (int i = 0; i < L / 64; ++i) {
            a += buf[2 * i];
            b += buf[2 * i + 1];
        }
    }
    return make_float2(a, b);
}

struct NormArgs {
    const void *x, *weight, *bias, *dy;
    const float *mean_in, *rstd_in;
    void *y, *dx;
    float *mean, *rstd, *part;   // part: [2][groups][cols]
    int64_t rows;
    int32_t cols;
    float eps;
};

// Threads of a workgroup: 256 / L rows at a time, or one. ITEMS = 0: the row stays in memory.
template <int L> constexpr int norm_block = L < 256 ? 256 : L;

template <typename T, typename TW, int L, int ITEMS>
__global__ __launch_bounds__(norm_block<L>) void norm_fwd_kernel(NormArgs a) {
    constexpr int V = NormVec<T>::V;
    __shared__ float buf[2][2 * (L > 64 ? L / 64 : 1)];
    const int t = threadIdx.x % L, n = a.cols;
    const int64_t row = int64_t(blockIdx.x) * (norm_block<L> / L) + threadIdx.x / L;
    if (row >= a.rows) return;   // all lanes of a row; rows of more than a wavefront have the workgroup to themselves
    const T *x = static_cast<const T *>(a.x) + row * n;
    T *y = static_cast<T *>(a.y) + row * n;
    const TW *w = static_cast<const TW *>(a.weight), *b = static_cast<const TW *>(a.bias);
    const float inv_n = 1.0f / float(n);
    const int nv = (n + V - 1) / V;
    constexpr int R = ITEMS > 0 ? ITEMS : 1;
    float v[R][V];
    float s = 0.0f;
    if constexpr (ITEMS > 0) {
#pragma unroll
        for (int i = 0; i < R; ++i) {
#pragma unroll
            for (int j = 0; j < V; ++j) v[i][j] = 0.0f;
            if (t + i * L < nv) norm_get<T, V>(x, t + i * L, n, 0.0f, v[i]);
        }
#pragma unroll
        for (int i = 0; i < R; ++i)
#pragma unroll
            for (int j = 0; j < V; ++j) s += v[i][j];
    } else {
        for (int i = t; i < nv; i += L) {
            norm_get<T, V>(x, i, n, 0.0f, v[0]);
#pragma unroll
            for (int j = 0; j < V; ++j) s += v[0][j];
        }
    }
    // The sum's rounding grows with the mean's size: the differences from it are summed again
    // beside their squares, and what is left of them is the mean's correction.
    const float m0 = row_sum<L>(s, 0.0f, buf[0]).x * inv_n;
    float q = 0.0f, e = 0.0f;
    auto add_squares = [&](int i, const float (&o)[V]) {
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const float d = i * V + j < n ? o[j] - m0 : 0.0f;
            e += d;
            q = fmaf(d, d, q);
        }
    };
    if constexpr (ITEMS > 0) {
#pragma unroll
        for (int i = 0; i < R; ++i) add_squares(t + i * L, v[i]);
    } else {
        for (int i = t; i < nv; i += L) {
            norm_get<T, V>(x, i, n, 0.0f, v[0]);
            add_squares(i, v[0]);
        }
    }
    const float2 sums = row_sum<L>(q, e, buf[1]);
    const float off = sums.y * inv_n;
    const float v2 = fmaf(-off, off, sums.x * inv_n), var = v2 < 0.0f ? 0.0f : v2;   // a NaN stays one
    const float rstd = 1.0f / sqrtf(var + a.eps);
    auto emit = [&](int i, const float (&o)[V]) {
        float g[V], c[V], r[V];
        if (w) norm_get<TW, V>(w, i, n, 0.0f, g);
        if (b) norm_get<TW, V>(b, i, n, 0.0f, c);
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const float h = ((o[j] - m0) - off) * rstd;
            r[j] = fmaf(h, w ? g[j] : 1.0f, b ? c[j] : 0.0f);
        }
        norm_put<T, V>(y, i, n, r);
    };
    if constexpr (ITEMS > 0) {
#pragma unroll
        for (int i = 0; i < R; ++i)
            if (t + i * L < nv) emit(t + i * L, v[i]);
    } else {
        for (int i = t; i < nv; i += L) {
            norm_get<T, V>(x, i, n, 0.0f, v[0]);
            emit(i, v[0]);
        }
    }
    if (t == 0) {
        a.mean[row] = m0 + off;
        a.rstd[row] = rstd;
    }
}

// dx of every row, and each workgroup's sums of dy xh and dy over its rows: in registers, or
// (ITEMS = 0) in its own rows of the workspace, each column in one thread's care.
template <typename T, typename TW, int L, int ITEMS>
__global__ __launch_bounds__(norm_block<L>) void norm_bwd_kernel(NormArgs a) {
    constexpr int V = NormVec<T>::V;
    constexpr int RPG = norm_block<L> / L;       // rows of a workgroup at a time
    constexpr int R = ITEMS > 0 ? ITEMS : 1;
    __shared__ float buf[2][2 * (L > 64 ? L / 64 : 1)];
    const int t = threadIdx.x % L, n = a.cols, mine = threadIdx.x / L;
    const TW *w = static_cast<const TW *>(a.weight);
    const float inv_n = 1.0f / float(n);
    const int nv = (n + V - 1) / V;
    const int64_t G = gridDim.x;
    float *pw = a.part ? a.part + int64_t(blockIdx.x) * n : nullptr;
    float *pb = a.part ? a.part + (G + blockIdx.x) * n : nullptr;
    float sw[R][V], sb[R][V], g[R][V];
#pragma unroll
    for (int i = 0; i < R; ++i) {
#pragma unroll
        for (int j = 0; j < V; ++j) {
            sw[i][j] = sb[i][j] = 0.0f;
            g[i][j] = 1.0f;
        }
        if constexpr (ITEMS > 0)
            if (w && t + i * L < nv) norm_get<TW, V>(w, t + i * L, n, 0.0f, g[i]);
    }
    if constexpr (ITEMS == 0) {
        if (a.part)
            for (int i = t; i < nv; i += L)
                for (int c = i * V; c < min(n, i * V + V); ++c) pw[c] = pb[c] = 0.0f;
    }
    int turn = 0;
    // the next row is on its way while this one's sums are made
    typename NormVec<T>::raw xr[R], dr[R];
    float mean_r = 0.0f, rstd_r = 0.0f;
    auto bring = [&](int64_t row) {
        if (row >= a.rows) return;
        const T *x = static_cast<const T *>(a.x) + row * n, *dy = static_cast<const T *>(a.dy) + row * n;
        mean_r = a.mean_in[row];
        rstd_r = a.rstd_in[row];
        if constexpr (ITEMS > 0) {
#pragma unroll
            for (int i = 0; i < R; ++i) {
                const int c = (t + i * L) * V;
                if (c + V <= n) {
                    xr[i] = *reinterpret_cast<const typename NormVec<T>::raw *>(x + c);
                    dr[i] = *reinterpret_cast<const typename NormVec<T>::raw *>(dy + c);
                } else if (c < n) {
                    xr[i] = NormVec<T>::part(x + c, n - c);
                    dr[i] = NormVec<T>::part(dy + c, n - c);
                }
            }
        }
    };
    bring(int64_t(blockIdx.x) * RPG + mine);
    for (int64_t r0 = int64_t(blockIdx.x) * RPG; r0 < a.rows; r0 += G * RPG) {
        const int64_t row = r0 + mine;
        if (RPG > 1 && row >= a.rows) break;   // nothing waits for a row's lanes here
        const T *x = static_cast<const T *>(a.x) + row * n, *dy = static_cast<const T *>(a.dy) + row * n;
        T *dx = a.dx ? static_cast<T *>(a.dx) + row * n : nullptr;
        const float mean = mean_r, rstd = rstd_r;
        float xv[R][V], dv[R][V];
        float c1 = 0.0f, c2 = 0.0f;
        auto fetch = [&](int i, float (&xo)[V], float (&d)[V]) {   // xh and dy of vector i, zeros past the row
            norm_get<T, V>(x, i, n, mean, xo);
            norm_get<T, V>(dy, i, n, 0.0f, d);
        };
        auto sums = [&](float (&xo)[V], const float (&d)[V], const float (&gw)[V]) {
#pragma unroll
            for (int j = 0; j < V; ++j) {
                xo[j] = (xo[j] - mean) * rstd;
                const float h = d[j] * gw[j];
                c1 += h;
                c2 = fmaf(h, xo[j], c2);
            }
        };
        if constexpr (ITEMS > 0) {
#pragma unroll
            for (int i = 0; i < R; ++i) {
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    xv[i][j] = mean;
                    dv[i][j] = 0.0f;
                }
                if (t + i * L < nv) {
                    NormVec<T>::unpack(xr[i], xv[i]);
                    NormVec<T>::unpack(dr[i], dv[i]);
                    if ((t + i * L) * V + V > n) {
#pragma unroll
                        for (int j = 0; j < V; ++j)
                            if ((t + i * L) * V + j >= n) xv[i][j] = mean;
                    }
                }
            }
            bring(row + G * RPG);
#pragma unroll
            for (int i = 0; i < R; ++i) sums(xv[i], dv[i], g[i]);
        } else {
            for (int i = t; i < nv; i += L) {
                fetch(i, xv[0], dv[0]);
                if (w) norm_get<TW, V>(w, i, n, 0.0f, g[0]);
                sums(xv[0], dv[0], g[0]);
            }
            bring(row + G * RPG);
        }
        const float2 c = row_sum<L>(c1, c2, buf[turn]);
        turn ^= 1;
        const float m1 = c.x * inv_n, m2 = c.y * inv_n;
        auto emit = [&](int i, const float (&xh)[V], const float (&d)[V], const float (&gw)[V], float (&aw)[V],
                        float (&ab)[V]) {
            float o[V];
#pragma unroll
            for (int j = 0; j < V; ++j) {
                o[j] = rstd * (d[j] * gw[j] - m1 - xh[j] * m2);
                aw[j] = fmaf(d[j], xh[j], aw[j]);
                ab[j] += d[j];
            }
            if (dx) norm_put<T, V>(dx, i, n, o);
        };
        if constexpr (ITEMS > 0) {
#pragma unroll
            for (int i = 0; i < R; ++i)
                if (t + i * L < nv) emit(t + i * L, xv[i], dv[i], g[i], sw[i], sb[i]);
        } else {
            for (int i = t; i < nv; i += L) {
                fetch(i, xv[0], dv[0]);
                if (w) norm_get<TW, V>(w, i, n, 0.0f, g[0]);
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    xv[0][j] = (xv[0][j] - mean) * rstd;
                    sw[0][j] = sb[0][j] = 0.0f;
                }
                emit(i, xv[0], dv[0], g[0], sw[0], sb[0]);
                if (a.part) {
#pragma unroll
                    for (int j = 0; j < V; ++j)
                        if (i * V + j < n) {
                            pw[i * V + j] += sw[0][j];
                            pb[i * V + j] += sb[0][j];
                        }
                }
            }
        }
    }
    if constexpr (ITEMS > 0) {
        if (!a.part) return;
        if constexpr (RPG > 1) {   // the sums of the workgroup's other rows, added in order
            __shared__ float all[RPG - 1][ITEMS * L * V];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                float(&s)[R][V] = k ? sb : sw;
                if (k) __syncthreads();
                if (mine > 0) {
#pragma unroll
                    for (int i = 0; i < R; ++i)
#pragma unroll
                        for (int j = 0; j < V; ++j) all[mine - 1][(i * V + j) * L + t] = s[i][j];
                }
                __syncthreads();
                if (mine == 0) {
                    for (int m = 0; m < RPG - 1; ++m)
#pragma unroll
                        for (int i = 0; i < R; ++i)
#pragma unroll
                            for (int j = 0; j < V; ++j) s[i][j] += all[m][(i * V + j) * L + t];
                }
            }
            if (mine > 0) return;
        }
#pragma unroll
        for (int i = 0; i < R; ++i)
            if (t + i * L < nv) {
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    const int c = (t + i * L) * V + j;
                    if (c < n) {
                        pw[c] = sw[i][j];
                        pb[c] = sb[i][j];
                    }
                }
            }
    }
}

// Column sums of the partial rows [groups][cols] of the weight (blockIdx.y = 0) and the bias
// (1): 16 wavefronts take a share of the rows each for the same 64 columns.
template <typename TW>
__global__ __launch_bounds__(1024) void norm_reduce_kernel(const float *part, int groups, int n, TW *dw, TW *db) {
    __shared__ float buf[16][64];
    const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
    const int c = blockIdx.x * 64 + lane;
    TW *out = blockIdx.y ? db : dw;
    if (!out) return;
    const float *p = part + int64_t(blockIdx.y) * groups * n;
    const int share = (groups + 15) / 16, g1 = min(groups, (wv + 1) * share);
    float s = 0.0f;
    if (c < n) {
#pragma unroll 8
        for (int g = wv * share; g < g1; ++g) s += p[int64_t(g) * n + c];
    }
    buf[wv][lane] = s;
    __syncthreads();
    if (wv == 0 && c < n) {
#pragma unroll
        for (int i = 1; i < 16; ++i) s += buf[i][lane];
        out[c] = from_f32<TW>(s);
    }
}

struct NormPlan {
    int L, items;
};
NormPlan norm_plan(int32_t cols, int V, bool bwd) {
    const int64_t nv = (int64_t(cols) + V - 1) / V;
    for (int L : {8, 16, 32, 64, 256, 1024}) {
        const int64_t items = (nv + L - 1) / L;
        if (items <= norm_max_items(L, V, bwd)) return {L, items <= 1 ? 1 : items <= 2 ? 2 : items <= 4 ? 4 : 8};
    }
    return {1024, 0};
}

template <bool BWD, typename T, typename TW, int L, int ITEMS>
hipError_t norm_go(const NormArgs &a, unsigned grid, hipStream_t st) {
    if constexpr (ITEMS <= norm_max_items(L, NormVec<T>::V, BWD) && (ITEMS > 0 || L == 1024)) {
        if constexpr (BWD)
            hipLaunchKernelGGL((norm_bwd_kernel<T, TW, L, ITEMS>), dim3(grid), dim3(norm_block<L>), 0, st, a);
        else
            hipLaunchKernelGGL((norm_fwd_kernel<T, TW, L, ITEMS>), dim3(grid), dim3(norm_block<L>), 0, st, a);
        return hipGetLastError();
    } else {
        return hipErrorInvalidValue;   // norm_plan gives no such plan
    }
}
template <bool BWD, typename T, typename TW, int L>
hipError_t norm_items(const NormArgs &a, const NormPlan &p, unsigned grid, hipStream_t st) {
    switch (p.items) {
        case 0: return norm_go<BWD, T, TW, L, 0>(a, grid, st);
        case 1: return norm_go<BWD, T, TW, L, 1>(a, grid, st);
        case 2: return norm_go<BWD, T, TW, L, 2>(a, grid, st);
        case 4: return norm_go<BWD, T, TW, L, 4>(a, grid, st);
        default: return norm_go<BWD, T, TW, L, 8>(a, grid, st);
    }
}
template <bool BWD, typename T, typename TW>
hipError_t norm_pick(const NormArgs &a, const NormPlan &p, unsigned grid, hipStream_t st) {
    switch (p.L) {
        case 8: return norm_items<BWD, T, TW, 8>(a, p, grid, st);
        case 16: return norm_items<BWD, T, TW, 16>(a, p, grid, st);
        case 32: return norm_items<BWD, T, TW, 32>(a, p, grid, st);
        case 64: return norm_items<BWD, T, TW, 64>(a, p, grid, st);
        case 256: return norm_items<BWD, T, TW, 256>(a, p, grid, st);
        default: return norm_items<BWD, T, TW, 1024>(a, p, grid, st);
    }
}
template <bool BWD>
hipError_t norm_launch(const NormArgs &a, int32_t dtype, int32_t wdtype, const NormPlan &p, unsigned grid,
                       hipStream_t st) {
    if (dtype == SDM_F32) return norm_pick<BWD, float, float>(a, p, grid, st);
    if (wdtype == SDM_F32) return norm_pick<BWD, bf16, float>(a, p, grid, st);
    return norm_pick<BWD, bf16, bf16>(a, p, grid, st);
}

// Workgroups of the backward: as many as keep the device full, each with enough rows that its sums cost little.
int norm_groups(int64_t rows, const NormPlan &p) {
    const int64_t want = p.L == 1024 ? 256 : 512, at_once = p.L < 256 ? 256 / p.L : 1;
    const int64_t most = (rows + at_once - 1) / at_once;
    return int(most < want ? (most < 1 ? 1 : most) : want);
}

int norm_check(int64_t rows, int32_t cols, int32_t dtype, int32_t wdtype, const sdm_exec *exec) {
    if (!exec) return fail(SDM_ERR_NULL, "exec must not be NULL");
    if (rows < 0 || cols < 1) return fail(SDM_ERR_SHAPE, "rows must be >= 0 and cols >= 1, got %lld and %d", (long long)rows, cols);
    if (rows > int64_t(0x7fffffff) || cols > (1 << 24))
        return fail(SDM_ERR_RANGE, "at most 2^31 - 1 rows of 2^24 columns, got %lld of %d", (long long)rows, cols);
    if ((dtype != SDM_F32 && dtype != SDM_BF16) || (wdtype != SDM_F32 && wdtype != SDM_BF16))
        return fail(SDM_ERR_DTYPE, "dtype and weight_dtype must be SDM_F32 or SDM_BF16, got %d and %d", dtype, wdtype);
    if (dtype == SDM_F32 && wdtype != SDM_F32)
        return fail(SDM_ERR_DTYPE, "float32 rows take float32 parameters");
    return SDM_OK;
}

int norm_align(const void *const *p, int n, int32_t dtype, const char *what) {
    for (int i = 0; i < n; ++i)
        if (p[i] && !aligned(p[i], dtype == SDM_BF16 ? 2 : 4))
            return fail(SDM_ERR_ALIGN, "%s must be aligned to their element size", what);
    return SDM_OK;
}

}  // namespace

}  // namespace sdm

using namespace sdm;

extern "C" {

int sdm_layer_norm_fwd(int64_t rows, int32_t cols, const void *x, int32_t dtype, const void *weight, const void *bias,
                       int32_t weight_dtype, float eps, void *y, float *mean, float *rstd, const sdm_exec *exec) {
    g_err[0] = 0;
    int rc = norm_check(rows, cols, dtype, weight_dtype, exec);
    if (rc) return rc;
    if (!(eps >= 0.0f)) return fail(SDM_ERR_RANGE, "eps must be >= 0, got %g", double(eps));
    if (rows == 0) return SDM_OK;
    if (!x || !y || !mean || !rstd) return fail(SDM_ERR_NULL, "x, y, mean and rstd must not be NULL");
    const void *d[] = {x, y}, *w[] = {weight, bias}, *f[] = {mean, rstd};
    if ((rc = norm_align(d, 2, dtype, "x and y")) || (rc = norm_align(w, 2, weight_dtype, "weight and bias")) ||
        (rc = norm_align(f, 2, SDM_F32, "mean and rstd")))
        return rc;
    NormArgs a{};
    a.x = x; a.weight = weight; a.bias = bias; a.y = y; a.mean = mean; a.rstd = rstd;
    a.rows = rows; a.cols = cols; a.eps = eps;
    const NormPlan p = norm_plan(cols, dtype == SDM_BF16 ? 8 : 4, false);
    // A launch holds less than 2^32 threads, L to a row: more rows go in several.
    const int64_t at_once = p.L < 256 ? 256 / p.L : 1, most = int64_t(1) << 31;
    const size_t row_bytes = size_t(cols) * (dtype == SDM_BF16 ? 2 : 4);
    for (int64_t left = rows; left > 0; left -= a.rows) {
        a.rows = left < most / p.L ? left : most / p.L;
        const unsigned grid = unsigned((a.rows + at_once - 1) / at_once);
        const hipError_t e = norm_launch<false>(a, dtype, weight_dtype, p, grid, static_cast<hipStream_t>(exec->stream));
        if (e != hipSuccess) return hip_fail(e, "layer norm launch");
        a.x = static_cast<const char *>(a.x) + size_t(a.rows) * row_bytes;
        a.y = static_cast<char *>(a.y) + size_t(a.rows) * row_bytes;
        a.mean += a.rows;
        a.rstd += a.rows;
    }
    return SDM_OK;
}

size_t sdm_layer_norm_bwd_workspace_bytes(int64_t rows, int32_t cols, int32_t dtype) {
    if (rows < 0 || cols < 1 || (dtype != SDM_F32 && dtype != SDM_BF16)) return 0;
    return align256(size_t(norm_groups(rows, norm_plan(cols, dtype == SDM_BF16 ? 8 : 4, true))) * size_t(cols) * 8);
}

int sdm_layer_norm_bwd(int64_t rows, int32_t cols, const void *grad_out, const void *x, int32_t dtype,
                       const void *weight, int32_t weight_dtype, const float *mean, const float *rstd, void *grad_x,
                       void *grad_weight, void *grad_bias, const sdm_exec *exec) {
    g_err[0] = 0;
    int rc = norm_check(rows, cols, dtype, weight_dtype, exec);
    if (rc) return rc;
    if (!grad_x && !grad_weight && !grad_bias) return SDM_OK;
    if (rows > 0 && (!grad_out || !x || !mean || !rstd))
        return fail(SDM_ERR_NULL, "grad_out, x, mean and rstd must not be NULL");
    const void *d[] = {grad_out, x, grad_x}, *w[] = {weight, grad_weight, grad_bias}, *f[] = {mean, rstd};
    if ((rc = norm_align(d, 3, dtype, "grad_out, x and grad_x")) ||
        (rc = norm_align(w, 3, weight_dtype, "weight and its gradients")) ||
        (rc = norm_align(f, 2, SDM_F32, "mean and rstd")))
        return rc;
    const bool sums = grad_weight || grad_bias;
    const size_t need = sdm_layer_norm_bwd_workspace_bytes(rows, cols, dtype);
    if (sums && (!exec->workspace || exec->workspace_bytes < need))
        return fail(SDM_ERR_WORKSPACE, "workspace of %zu bytes is below the %zu bytes the gradients need",
                    exec->workspace ? exec->workspace_bytes : size_t(0), need);
    if (sums && !aligned(exec->workspace, 256)) return fail(SDM_ERR_ALIGN, "workspace must be 256-byte aligned");
    NormArgs a{};
    a.x = x; a.dy = grad_out; a.weight = weight; a.dx = grad_x; a.mean_in = mean; a.rstd_in = rstd;
    a.part = sums ? static_cast<float *>(exec->workspace) : nullptr;
    a.rows = rows; a.cols = cols;
    const NormPlan p = norm_plan(cols, dtype == SDM_BF16 ? 8 : 4, true);
    const int groups = norm_groups(rows, p);
    const hipStream_t st = static_cast<hipStream_t>(exec->stream);
    hipError_t e = norm_launch<true>(a, dtype, weight_dtype, p, unsigned(groups), st);
    if (e != hipSuccess) return hip_fail(e, "layer norm backward launch");
    if (!sums) return SDM_OK;
    const dim3 grid(unsigned((cols + 63) / 64), 2);
    if (weight_dtype == SDM_F32)
        hipLaunchKernelGGL(norm_reduce_kernel<float>, grid, dim3(1024), 0, st, a.part, groups, cols,
                           static_cast<float *>(grad_weight), static_cast<float *>(grad_bias));
    else
        hipLaunchKernelGGL(norm_reduce_kernel<bf16>, grid, dim3(1024), 0, st, a.part, groups, cols,
                           static_cast<bf16 *>(grad_weight), static_cast<bf16 *>(grad_bias));
    e = hipGetLastError();
    return e == hipSuccess ? SDM_OK : hip_fail(e, "layer norm reduction launch");
}

}  // extern "C"
