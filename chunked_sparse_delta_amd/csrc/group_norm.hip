// Group norm with an activation, channels last, forward and backward.
//
// x [samples, rows, channels], G groups of D neighbouring channels; per sample and group, over its m = rows D elements:
//     mean = sum(x) / m, var = sum((x - mean)^2) / m, rstd = 1 / sqrt(var + eps)
//     xh = (x - mean) rstd, z = xh w + b, y = act(z)
// and with dz = dy act'(z), h = dz w:
//     dx = rstd (h - sum(h) / m - xh sum(h xh) / m),  dw = sum over samples and rows (dz xh),  db = the same of dz
//
// Bound by memory where samples are long, by the issue of instructions where they are short and many. A thread owns a vector of 16 bytes
// of channels and takes rows of it; neighbouring threads take neighbouring vectors, so that rows are read whole whatever the groups. A workgroup takes a tile: whole groups side by side.
//  - Resident: where a tile's rows fit the registers of a workgroup each element is read once. Several samples share a workgroup
//    where they are short; their sums meet by shuffles where a group is 1, 2, 4, ... lanes of one wavefront, through LDS elsewhere.
//  - Split: longer samples are cut into blocks of rows; one kernel leaves each block's sums, the next joins them and reads the rows again.
// Measured: 8192 tokens of 4096 channels in 32 groups, bfloat16, silu: forward 37 us (134 MB, 26 us at a copy's rate; 17.6 M vector
// instructions, 29 us at four cycles each on 1024 SIMDs at 2.4 GHz), backward 53 (201 MB, 39; 22.9 M, 37) and 4 for the sums over workgroups; 64
// tokens: 4.4. Split, 8 x 4096 rows of 512 channels: statistics 12 to 13, their join 4, values 13.5 (67 MB, 5.0 TB/s); sums 20 (67 MB),
// their join 5, gradients 19 (101 MB, 5.3 TB/s), the parameters' sums 4. A large copy: 5.2 TB/s.
// Statistics: a thread's mean and sum of squared differences from it, joined with their counts. Split: sums of differences from the first
// of at most kGnRun rows and of their squares, less the square of the sum, joined likewise.
// All sums run in float32 in a fixed order: results are the same from run to run.
#include <type_traits>

#include "host.h"
#include "norm_vec.h"

namespace sdm {

namespace {

enum { kShuffle, kVectors, kChannels };     // how a tile's threads meet: see GnPlan

struct GnPlan {
    int mode;        // kShuffle: groups of 2^k lanes, one thread row to a sample; kVectors: D a multiple of the vector; kChannels: any D
    int threads;     // of a workgroup
    int items;       // rows of a thread held in registers; 0: split
    int gt, tiles;   // groups of a tile; tiles of a row (pieces of a group where one exceeds a workgroup: gt 0)
    int cv;          // vectors of a tile's row
    int rt;          // rows at once
    int rs, spw;     // thread rows of a sample, samples of a workgroup (resident)
    int lanes;       // that join a group's sums
    int blocks, block_rows;   // of a sample (split)
};

struct GnArgs {
    const void *x, *weight, *bias, *dy;
    void *y, *dx;
    float *mean, *rstd;          // [samples][G]
    const int32_t *valid;        // [samples] or null
    float *part;
    int64_t N, L, x_sample, x_row;
    int32_t C, G, D, act;
    bool w_f32;
    float eps;
    GnPlan p;
};

__device__ __forceinline__ int64_t gn_valid(const GnArgs &a, int64_t n) {
    if (!a.valid) return a.L;
    const int64_t v = a.valid[n];
    return v < 0 ? 0 : v < a.L ? v : a.L;
}

// V parameters from channel c on, of which `left` are there.
template <int V> __device__ __forceinline__ void gn_params(const void *p, bool f32, int c, int left, float none, float (&o)[V]) {
#pragma unroll
    for (int j = 0; j < V; ++j) o[j] = none;
    if (!p || left <= 0) return;
    if constexpr (V == NormVec<bf16>::V) {     // float32 rows take float32 parameters
        if (!f32) {
            norm_get<bf16, V>(static_cast<const bf16 *>(p) + c, 0, left, none, o);
            return;
        }
    }
    norm_get<float, V>(static_cast<const float *>(p) + c, 0, left, none, o);
}

// 1 / (1 + 2^(-z / log 2)): the exponent's rounding, 2^-24 of it, is |z| 2^-24 of a value that falls as e^z: at most 2^-24 in z sigmoid(z).
// (With expf and joins by division in each group's lanes the forward of 8192 x 4096 took 56 us; now 36.)
__device__ __forceinline__ float gn_sigmoid(float z) { return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-1.44269504f * z)); }
__device__ __forceinline__ float gn_phi(float z) { return 0.5f * erfcf(-0.70710678f * z); }

template <int V> __device__ __forceinline__ void gn_act(int act, float (&z)[V]) {
    if (act == SDM_ACT_SILU) {
#pragma unroll
        for (int j = 0; j < V; ++j) z[j] *= gn_sigmoid(z[j]);
    } else if (act == SDM_ACT_GELU) {
#pragma unroll
        for (int j = 0; j < V; ++j) z[j] *= gn_phi(z[j]);
    }
}
// d times the activation's slope at z.
template <int V> __device__ __forceinline__ void gn_slope(int act, const float (&z)[V], float (&d)[V]) {
    if (act == SDM_ACT_SILU) {
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const float s = gn_sigmoid(z[j]);
            d[j] *= s * fmaf(z[j], 1.0f - s, 1.0f);
        }
    } else if (act == SDM_ACT_GELU) {
#pragma unroll
        for (int j = 0; j < V; ++j) d[j] *= fmaf(z[j], 0.3989422804f * expf(-0.5f * z[j] * z[j]), gn_phi(z[j]));
    }
}

// A thread's place: vector `col` of the tile's row, thread row `tr`.
struct GnAt {
    int tile, g0, c0, width, col, tr, c, left;    // g0: first group; c: the thread's first channel, `left` of the tile's from it
    __device__ __forceinline__ GnAt(const GnArgs &a, int tile_, int V) : tile(tile_) {
        if (a.p.gt > 0) {
            g0 = tile * a.p.gt;
            c0 = g0 * a.D;
            width = min(a.p.gt, a.G - g0) * a.D;
        } else {      // a piece of a group
            const int pieces = a.p.tiles / a.G, piece = tile % pieces, most = a.p.cv * V;
            g0 = tile / pieces;
            c0 = g0 * a.D + piece * most;
            width = min(most, a.D - piece * most);
        }
        col = int(threadIdx.x) % a.p.cv;
        tr = int(threadIdx.x) / a.p.cv;
        c = c0 + col * V;
        left = tr < a.p.rt ? width - col * V : 0;
    }
    // The tile's groups (or the one that it is a piece of).
    __device__ __forceinline__ int groups(const GnArgs &a) const { return a.p.gt > 0 ? width / a.D : 1; }
};

template <typename T, int V> __device__ __forceinline__ typename NormVec<T>::raw gn_load(const T *p, int left) {
    typename NormVec<T>::raw r = {};
    if (left >= V) r = *reinterpret_cast<const typename NormVec<T>::raw *>(p);
    else if (left > 0) r = NormVec<T>::part(p, left);
    return r;
}

// Joins (count, mean, sum of squared differences) of two sets.
struct GnStat {
    float n, mean, m2;
    __device__ __forceinline__ void add(const GnStat &o) {
        const float all = n + o.n, d = o.mean - mean, f = all > 0.0f ? o.n / all : 0.0f, w = n * f;
        mean = fmaf(d, f, mean);
        m2 += w > 0.0f ? fmaf(d * d, w, o.m2) : o.m2;      // beside an empty set d is a mean, whose square may be infinite
        n = all;
    }
};
__device__ __forceinline__ GnStat gn_shuffle(const GnStat &s, int m) { return {__shfl_xor(s.n, m, 64), __shfl_xor(s.mean, m, 64), __shfl_xor(s.m2, m, 64)}; }

// The sum over `lanes` (a power of two) neighbouring lanes, for each of them: within rows of 16 by register moves, then by
// swapped halves.
__device__ __forceinline__ float gn_lanes_sum(float x, int lanes) {
    auto moved = [](float y, auto ctrl) {
        return __uint_as_float(__builtin_amdgcn_update_dpp(0u, __float_as_uint(y), decltype(ctrl)::value, 0xF, 0xF, false));
    };
    if (lanes >= 2) x += moved(x, std::integral_constant<int, 0xB1>{});      // lane ^ 1
    if (lanes >= 4) x += moved(x, std::integral_constant<int, 0x4E>{});      // lane ^ 2
    if (lanes >= 8) x += moved(x, std::integral_constant<int, 0x141>{});     // the other four of eight
    if (lanes >= 16) x += moved(x, std::integral_constant<int, 0x140>{});    // the other eight of a row
    if (lanes >= 32) {
        const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
        x = __uint_as_float(r[0]) + __uint_as_float(r[1]);
    }
    if (lanes >= 64) {
        const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
        x = __uint_as_float(r[0]) + __uint_as_float(r[1]);
    }
    return x;
}

// ---- resident --------------------------------------------------------------------------------------------------------

// LDS of the joins: per thread (kVectors) or per channel and thread row (kChannels), and per group of every sample.
template <int MODE, int NT, int V> struct GnLds {
    static constexpr int N = MODE == kChannels ? NT * V : NT;
    float a[N], b[N], n[NT], ga[N], gb[N];
};

template <typename T, int NT, int ITEMS, int MODE> __global__ __launch_bounds__(NT) void gn_fwd_kernel(GnArgs a) {
    constexpr int V = NormVec<T>::V;
    using raw = typename NormVec<T>::raw;
    const GnAt at(a, blockIdx.y, V);
    const int D = a.D, rs = a.p.rs, spw = a.p.spw, slot = at.tr / rs, rb = at.tr % rs;
    const bool mine = at.left > 0 && slot < spw;
    const int left = mine ? at.left : 0;
    float w[V], b[V];
    gn_params<V>(a.weight, a.w_f32, at.c, left, 1.0f, w);
    gn_params<V>(a.bias, a.w_f32, at.c, left, 0.0f, b);
    raw r[ITEMS];
    int64_t nv = 0;
    auto bring = [&](int64_t block) {
        const int64_t n = block * spw + slot;
        nv = mine && n < a.N ? gn_valid(a, n) : 0;
        const T *x = static_cast<const T *>(a.x) + n * a.x_sample + at.c;
#pragma unroll
        for (int i = 0; i < ITEMS; ++i) r[i] = gn_load<T, V>(x + (rb + rs * i) * a.x_row, rb + rs * i < nv ? left : 0);
    };
    const int64_t blocks = (a.N + spw - 1) / spw;
    bring(blockIdx.x);
    for (int64_t block = blockIdx.x; block < blocks; block += gridDim.x) {
        const int64_t n = block * spw + slot;
        const int live = rb < nv ? min(ITEMS, int((nv - rb + rs - 1) / rs)) : 0;
        float x[ITEMS][V];
#pragma unroll
        for (int i = 0; i < ITEMS; ++i) NormVec<T>::unpack(r[i], x[i]);
        if (block + gridDim.x < blocks) bring(block + gridDim.x);
        // the thread's own statistics, of all its channels or of each
        float mean[V], rstd[V];
        if constexpr (MODE != kChannels) {
            float s = 0.0f;
#pragma unroll
            for (int i = 0; i < ITEMS; ++i)
#pragma unroll
                for (int j = 0; j < V; ++j) s += x[i][j];
            // kShuffle: a group's lanes hold equally many rows, so that plain sums over them do
            const int count = MODE == kShuffle ? live * D : live * V;
            if (MODE == kShuffle) s = gn_lanes_sum(s, a.p.lanes);
            GnStat t{float(count), count > 0 ? s / float(count) : 0.0f, 0.0f};
#pragma unroll
            for (int i = 0; i < ITEMS; ++i)
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    const float d = x[i][j] - t.mean;
                    if (i < live) t.m2 = fmaf(d, d, t.m2);
                }
            if constexpr (MODE == kShuffle) {
                t.m2 = gn_lanes_sum(t.m2, a.p.lanes);
            } else {
                __shared__ GnLds<MODE, NT, V> s;
                s.a[threadIdx.x] = t.mean;
                s.b[threadIdx.x] = t.m2;
                s.n[threadIdx.x] = t.n;
                __syncthreads();
                const int vecs = D / V, gt = at.groups(a), all = spw * gt, lane = threadIdx.x % a.p.lanes;
                for (int g = threadIdx.x / a.p.lanes; g < all; g += NT / a.p.lanes) {
                    const int first = g / gt * rs * a.p.cv + g % gt * vecs;
                    GnStat u{0.0f, 0.0f, 0.0f};
                    for (int i = lane; i < rs * vecs; i += a.p.lanes) {
                        const int from = first + i / vecs * a.p.cv + i % vecs;
                        u.add({s.n[from], s.a[from], s.b[from]});
                    }
                    for (int m = a.p.lanes / 2; m > 0; m >>= 1) u.add(gn_shuffle(u, m));
                    if (lane == 0) {
                        s.ga[g] = u.mean;
                        s.gb[g] = u.n > 0.0f ? u.m2 / u.n : 0.0f;
                    }
                }
                __syncthreads();
                const int g = mine ? slot * gt + at.col * V / D : 0;
                t.mean = s.ga[g];
                t.m2 = s.gb[g];
                t.n = 1.0f;
            }
            const float q = 1.0f / sqrtf((t.n > 0.0f ? t.m2 / t.n : 0.0f) + a.eps);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                mean[j] = t.mean;
                rstd[j] = q;
            }
            const int vec = at.col * V;
            if (mine && n < a.N && rb == 0 && vec % D == 0) {
                a.mean[n * a.G + at.g0 + vec / D] = t.mean;
                a.rstd[n * a.G + at.g0 + vec / D] = q;
            }
        } else {
            __shared__ GnLds<MODE, NT, V> s;
            const int cw = a.p.cv * V;
            if (mine) {
                s.n[at.tr] = float(live);
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    float t = 0.0f, q = 0.0f;
#pragma unroll
                    for (int i = 0; i < ITEMS; ++i) t += x[i][j];
                    if (live > 0) t /= float(live);
#pragma unroll
                    for (int i = 0; i < ITEMS; ++i) {
                        const float d = x[i][j] - t;
                        if (i < live) q = fmaf(d, d, q);
                    }
                    s.a[at.tr * cw + at.col * V + j] = t;
                    s.b[at.tr * cw + at.col * V + j] = q;
                }
            }
            __syncthreads();
            const int gt = at.groups(a), all = spw * gt, lane = threadIdx.x % a.p.lanes;
            for (int g = threadIdx.x / a.p.lanes; g < all; g += NT / a.p.lanes) {
                const int row = g / gt * rs, first = g % gt * D;
                GnStat u{0.0f, 0.0f, 0.0f};
                for (int i = lane; i < rs * D; i += a.p.lanes) {
                    const int from = (row + i / D) * cw + first + i % D;
                    u.add({s.n[row + i / D], s.a[from], s.b[from]});
                }
                for (int m = a.p.lanes / 2; m > 0; m >>= 1) u.add(gn_shuffle(u, m));
                if (lane == 0) {
                    const float q = 1.0f / sqrtf((u.n > 0.0f ? u.m2 / u.n : 0.0f) + a.eps);
                    s.ga[g] = u.mean;
                    s.gb[g] = q;
                    const int64_t to = block * spw + g / gt;
                    if (to < a.N) {
                        a.mean[to * a.G + at.g0 + g % gt] = u.mean;
                        a.rstd[to * a.G + at.g0 + g % gt] = q;
                    }
                }
            }
            __syncthreads();
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const int g = j < left ? slot * gt + (at.col * V + j) / D : 0;
                mean[j] = s.ga[g];
                rstd[j] = s.gb[g];
            }
        }
        if (left > 0 && n < a.N) {
            T *y = static_cast<T *>(a.y) + n * a.L * a.C + at.c;
#pragma unroll
            for (int i = 0; i < ITEMS; ++i) {
                const int row = rb + rs * i;
                if (row >= a.L) break;
                float z[V];
#pragma unroll
                for (int j = 0; j < V; ++j) z[j] = fmaf((x[i][j] - mean[j]) * rstd[j], w[j], b[j]);
                gn_act<V>(a.act, z);
#pragma unroll
                for (int j = 0; j < V; ++j) z[j] = i < live ? z[j] : 0.0f;
                norm_put<T, V>(y + int64_t(row) * a.C, 0, left, z);
            }
        }
        if constexpr (MODE != kShuffle) __syncthreads();      // the joins' memory is free
    }
}

// part: [2][gridDim.x][C], or null: sums of dz xh and dz over the workgroup's samples.
template <typename T, int NT, int ITEMS, int MODE> __global__ __launch_bounds__(NT) void gn_bwd_kernel(GnArgs a) {
    constexpr int V = NormVec<T>::V;
    using raw = typename NormVec<T>::raw;
    __shared__ GnLds<MODE, NT, V> s;
    const GnAt at(a, blockIdx.y, V);
    const int D = a.D, rs = a.p.rs, spw = a.p.spw, slot = at.tr / rs, rb = at.tr % rs, cw = a.p.cv * V, gt = at.groups(a);
    const bool mine = at.left > 0 && slot < spw;
    const int left = mine ? at.left : 0;
    float w[V], b[V], dw[V] = {}, db[V] = {};
    gn_params<V>(a.weight, a.w_f32, at.c, left, 1.0f, w);
    gn_params<V>(a.bias, a.w_f32, at.c, left, 0.0f, b);
    raw rx[ITEMS], rd[ITEMS];
    int64_t nv = 0;
    float mr[MODE == kChannels ? V : 1], qr[MODE == kChannels ? V : 1];
    auto bring = [&](int64_t block) {
        const int64_t n = block * spw + slot;
        const bool in = mine && n < a.N;
        nv = in ? gn_valid(a, n) : 0;
        const T *x = static_cast<const T *>(a.x) + n * a.x_sample + at.c, *d = static_cast<const T *>(a.dy) + n * a.L * a.C + at.c;
#pragma unroll
        for (int i = 0; i < ITEMS; ++i) {
            const int row = rb + rs * i, l = row < nv ? left : 0;
            rx[i] = gn_load<T, V>(x + row * a.x_row, l);
            rd[i] = gn_load<T, V>(d + int64_t(row) * a.C, l);
        }
#pragma unroll
        for (int j = 0; j < (MODE == kChannels ? V : 1); ++j) {
            const bool on = in && j < left;
            const int64_t g = on ? n * a.G + at.g0 + (at.col * V + j) / D : 0;
            mr[j] = on ? a.mean[g] : 0.0f;
            qr[j] = on ? a.rstd[g] : 0.0f;
        }
    };
    const int64_t blocks = (a.N + spw - 1) / spw;
    bring(blockIdx.x);
    for (int64_t block = blockIdx.x; block < blocks; block += gridDim.x) {
        const int64_t n = block * spw + slot;
        const int live = rb < nv ? min(ITEMS, int((nv - rb + rs - 1) / rs)) : 0;
        const float inv = nv > 0 ? 1.0f / (float(nv) * float(D)) : 0.0f;
        float xh[ITEMS][V], dz[ITEMS][V], q[V];
#pragma unroll
        for (int j = 0; j < V; ++j) q[j] = qr[MODE == kChannels ? j : 0];
        float c1[V] = {}, c2[V] = {};
#pragma unroll
        for (int i = 0; i < ITEMS; ++i) {
            float z[V];
            NormVec<T>::unpack(rx[i], xh[i]);
            NormVec<T>::unpack(rd[i], dz[i]);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                xh[i][j] = (xh[i][j] - mr[MODE == kChannels ? j : 0]) * q[j];
                z[j] = fmaf(xh[i][j], w[j], b[j]);
            }
            gn_slope<V>(a.act, z, dz[i]);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const bool in = i < live && j < left;
                dz[i][j] = in ? dz[i][j] : 0.0f;
                xh[i][j] = in ? xh[i][j] : 0.0f;
                c1[j] += dz[i][j];
                c2[j] = fmaf(dz[i][j], xh[i][j], c2[j]);
            }
        }
        if (block + gridDim.x < blocks) bring(block + gridDim.x);
        float s1[V], s2[V];
#pragma unroll
        for (int j = 0; j < V; ++j) {
            db[j] += c1[j];
            dw[j] += c2[j];
            c1[j] *= w[j];
            c2[j] *= w[j];
        }
        if constexpr (MODE != kChannels) {
            float t1 = 0.0f, t2 = 0.0f;
#pragma unroll
            for (int j = 0; j < V; ++j) {
                t1 += c1[j];
                t2 += c2[j];
            }
            if constexpr (MODE == kShuffle) {
                t1 = gn_lanes_sum(t1, a.p.lanes);
                t2 = gn_lanes_sum(t2, a.p.lanes);
            } else {
                s.a[threadIdx.x] = t1;
                s.b[threadIdx.x] = t2;
            }
#pragma unroll
            for (int j = 0; j < V; ++j) {
                s1[j] = t1;
                s2[j] = t2;
            }
        } else if (mine) {
#pragma unroll
            for (int j = 0; j < V; ++j) {
                s.a[at.tr * cw + at.col * V + j] = c1[j];
                s.b[at.tr * cw + at.col * V + j] = c2[j];
            }
        }
        if constexpr (MODE != kShuffle) {
            __syncthreads();
            const int each = MODE == kChannels ? D : D / V, step = MODE == kChannels ? cw : a.p.cv, lane = threadIdx.x % a.p.lanes;
            for (int g = threadIdx.x / a.p.lanes; g < spw * gt; g += NT / a.p.lanes) {
                const int first = g / gt * rs * step + g % gt * each;
                float t1 = 0.0f, t2 = 0.0f;
                for (int i = lane; i < rs * each; i += a.p.lanes) {
                    const int from = first + i / each * step + i % each;
                    t1 += s.a[from];
                    t2 += s.b[from];
                }
                t1 = gn_lanes_sum(t1, a.p.lanes);
                t2 = gn_lanes_sum(t2, a.p.lanes);
                if (lane == 0) {
                    s.ga[g] = t1;
                    s.gb[g] = t2;
                }
            }
            __syncthreads();
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const int g = j < left ? slot * gt + (at.col * V + j) / D : 0;
                s1[j] = s.ga[g];
                s2[j] = s.gb[g];
            }
        }
        if (left > 0 && n < a.N && a.dx) {
            T *dx = static_cast<T *>(a.dx) + n * a.L * a.C + at.c;
#pragma unroll
            for (int i = 0; i < ITEMS; ++i) {
                const int row = rb + rs * i;
                if (row >= a.L) break;
                float o[V];
#pragma unroll
                for (int j = 0; j < V; ++j) o[j] = i < live ? q[j] * (dz[i][j] * w[j] - inv * fmaf(xh[i][j], s2[j], s1[j])) : 0.0f;
                norm_put<T, V>(dx + int64_t(row) * a.C, 0, left, o);
            }
        }
        if constexpr (MODE != kShuffle) __syncthreads();
    }
    if (!a.part) return;
    // the thread rows' sums of each channel, in order
    __shared__ float all[NT * V];
    for (int k = 0; k < 2; ++k) {
        __syncthreads();
        if (mine) {
#pragma unroll
            for (int j = 0; j < V; ++j) all[at.tr * cw + at.col * V + j] = k ? db[j] : dw[j];
        }
        __syncthreads();
        for (int c = threadIdx.x; c < at.width; c += NT) {
            float t = 0.0f;
            for (int r = 0; r < rs * spw; ++r) t += all[r * cw + c];
            a.part[(int64_t(k) * gridDim.x + blockIdx.x) * a.C + at.c0 + c] = t;
        }
    }
}

// ---- split -----------------------------------------------------------------------------------------------------------

constexpr int kGnThreads = 256;
// Rows of a run of the statistics. What cancels between a run's squares and the square of its sum grows with its length: 165 of
// 2^-24 of the variance at most for 8 rows of which the first lies far off; one run of the 128 rows that a thread had of 2048 x 16384 x 8
// was off by 4700. (8 rows are a thread's share where blocks are not long.)
constexpr int kGnRun = 8;
// Rows of a thread on their way at once (one after another the sums of 8 x 4096 x 512 bfloat16 took 21 us, so 19; the gradients' kernel, short of
// registers, the other way round 19 and 23).
constexpr int kGnAhead = 4;

// The statistics of the groups of one block of rows: part[sample][block][tile's groups or pieces] as (mean, sum of squares).
template <typename T> __global__ __launch_bounds__(kGnThreads) void gn_stats_kernel(GnArgs a) {
    constexpr int V = NormVec<T>::V;
    __shared__ float sm[kGnThreads * V], sq[kGnThreads * V], sn[kGnThreads];
    const GnAt at(a, blockIdx.y, V);
    const int64_t n = blockIdx.x / a.p.blocks;
    const int block = blockIdx.x % a.p.blocks;
    const int64_t nv = gn_valid(a, n), r0 = int64_t(block) * a.p.block_rows, r1 = min(r0 + a.p.block_rows, nv);
    const int cw = a.p.cv * V;
    if (at.left > 0) {
        // runs of up to kGnRun rows: sums of differences from the run's first one, joined with their counts
        const T *x = static_cast<const T *>(a.x) + n * a.x_sample + at.c;
        float mean[V] = {}, m2[V] = {};
        int count = 0;
        for (int64_t r = r0 + at.tr; r < r1;) {
            float first[V], s[V] = {}, q[V] = {};
            const int64_t end = min(r1, r + kGnRun * a.p.rt);
            NormVec<T>::unpack(gn_load<T, V>(x + r * a.x_row, at.left), first);
            int rows = 0;
            constexpr int U = 4;
            for (; r + (U - 1) * a.p.rt < end; r += U * a.p.rt) {
                typename NormVec<T>::raw w[U];
#pragma unroll
                for (int u = 0; u < U; ++u) w[u] = gn_load<T, V>(x + (r + u * a.p.rt) * a.x_row, at.left);
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    float v[V];
                    NormVec<T>::unpack(w[u], v);
#pragma unroll
                    for (int j = 0; j < V; ++j) {
                        const float d = v[j] - first[j];
                        s[j] += d;
                        q[j] = fmaf(d, d, q[j]);
                    }
                }
                rows += U;
            }
            for (; r < end; r += a.p.rt, ++rows) {
                float v[V];
                NormVec<T>::unpack(gn_load<T, V>(x + r * a.x_row, at.left), v);
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    const float d = v[j] - first[j];
                    s[j] += d;
                    q[j] = fmaf(d, d, q[j]);
                }
            }
            const float inv = 1.0f / float(rows);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float left = fmaf(-s[j] * inv, s[j], q[j]);
                GnStat t{float(count), mean[j], m2[j]};
                t.add({float(rows), fmaf(s[j], inv, first[j]), left < 0.0f ? 0.0f : left});
                mean[j] = t.mean;
                m2[j] = t.m2;
            }
            count += rows;
        }
        sn[at.tr] = float(count);
#pragma unroll
        for (int j = 0; j < V; ++j) {
            sm[at.tr * cw + at.col * V + j] = mean[j];
            sq[at.tr * cw + at.col * V + j] = m2[j];
        }
    }
    __syncthreads();
    const int gt = at.groups(a), D = a.p.gt > 0 ? a.D : at.width, lane = threadIdx.x % a.p.lanes;
    float *part = a.part + (int64_t(blockIdx.x) * (a.p.gt > 0 ? a.G : a.p.tiles) + (a.p.gt > 0 ? at.g0 : at.tile)) * 2;
    for (int g = threadIdx.x / a.p.lanes; g < gt; g += kGnThreads / a.p.lanes) {
        GnStat u{0.0f, 0.0f, 0.0f};
        for (int i = lane; i < a.p.rt * D; i += a.p.lanes) {
            const int row = i / D, from = row * cw + g * D + i % D;
            u.add({sn[row], sm[from], sq[from]});
        }
        for (int m = a.p.lanes / 2; m > 0; m >>= 1) u.add(gn_shuffle(u, m));
        if (lane == 0) {
            part[2 * g] = u.mean;
            part[2 * g + 1] = u.m2;
        }
    }
}

// The statistics of every sample and group from its blocks' (a wavefront each).
__global__ __launch_bounds__(64) void gn_join_kernel(GnArgs a, int V) {
    const int pieces = a.p.gt > 0 ? 1 : a.p.tiles / a.G, stride = a.p.gt > 0 ? a.G : a.p.tiles;
    for (int64_t to = blockIdx.x; to < a.N * a.G; to += gridDim.x) {
        const int64_t n = to / a.G, nv = gn_valid(a, n);
        const int g = int(to % a.G);
        GnStat u{0.0f, 0.0f, 0.0f};
        for (int i = threadIdx.x; i < a.p.blocks * pieces; i += 64) {
            const int block = i / pieces, piece = i % pieces;
            const int64_t rows = min(int64_t(a.p.block_rows), nv - int64_t(block) * a.p.block_rows);
            if (rows <= 0) continue;
            const int most = a.p.cv * V, width = a.p.gt > 0 ? a.D : min(most, a.D - piece * most);
            const float *p = a.part + ((n * a.p.blocks + block) * stride + g * pieces + piece) * 2;
            u.add({float(rows) * float(width), p[0], p[1]});
        }
#pragma unroll
        for (int m = 32; m > 0; m >>= 1) u.add(gn_shuffle(u, m));
        if (threadIdx.x == 0) {
            a.mean[to] = u.mean;
            a.rstd[to] = 1.0f / sqrtf((u.n > 0.0f ? u.m2 / u.n : 0.0f) + a.eps);
        }
    }
}

// The groups of a thread's channels, 0 for those that are not there.
template <int V> __device__ __forceinline__ void gn_groups(const GnArgs &a, const GnAt &at, int (&g)[V]) {
    int q = at.c / a.D, r = at.c - q * a.D;
#pragma unroll
    for (int j = 0; j < V; ++j) {
        g[j] = j < at.left ? q : 0;
        const bool ends = ++r == a.D;
        q += ends;
        r = ends ? 0 : r;
    }
}
// A thread's channels' mean and rstd.
template <int V> __device__ __forceinline__ void gn_thread_stats(const GnArgs &a, const int (&g)[V], int64_t n, float (&mean)[V], float (&rstd)[V]) {
#pragma unroll
    for (int j = 0; j < V; ++j) {
        mean[j] = a.mean[n * a.G + g[j]];
        rstd[j] = a.rstd[n * a.G + g[j]];
    }
}

template <typename T> __global__ __launch_bounds__(kGnThreads) void gn_apply_kernel(GnArgs a) {
    constexpr int V = NormVec<T>::V;
    const GnAt at(a, blockIdx.y, V);
    if (at.left <= 0) return;
    const int64_t n = blockIdx.x / a.p.blocks, nv = gn_valid(a, n), r0 = int64_t(blockIdx.x % a.p.blocks) * a.p.block_rows, r1 = min(r0 + a.p.block_rows, a.L);
    float w[V], b[V], mean[V], rstd[V];
    gn_params<V>(a.weight, a.w_f32, at.c, at.left, 1.0f, w);
    gn_params<V>(a.bias, a.w_f32, at.c, at.left, 0.0f, b);
    int g[V];
    gn_groups<V>(a, at, g);
    gn_thread_stats<V>(a, g, n, mean, rstd);
    const T *x = static_cast<const T *>(a.x) + n * a.x_sample + at.c;
    T *y = static_cast<T *>(a.y) + n * a.L * a.C + at.c;
    for (int64_t r0t = r0 + at.tr; r0t < r1; r0t += kGnAhead * a.p.rt) {
        typename NormVec<T>::raw rx[kGnAhead];
#pragma unroll
        for (int u = 0; u < kGnAhead; ++u) {
            const int64_t r = r0t + u * a.p.rt;
            rx[u] = gn_load<T, V>(x + r * a.x_row, r < r1 && r < nv ? at.left : 0);
        }
#pragma unroll
        for (int u = 0; u < kGnAhead; ++u) {
            const int64_t r = r0t + u * a.p.rt;
            if (r >= r1) break;
            float z[V] = {};
            if (r < nv) {
                float v[V];
                NormVec<T>::unpack(rx[u], v);
#pragma unroll
                for (int j = 0; j < V; ++j) z[j] = fmaf((v[j] - mean[j]) * rstd[j], w[j], b[j]);
                gn_act<V>(a.act, z);
            }
            norm_put<T, V>(y + r * a.C, 0, at.left, z);
        }
    }
}

// Sums of dz xh and dz of each channel of a block's rows: part[sample][block][2][C].
template <typename T> __global__ __launch_bounds__(kGnThreads) void gn_bwd_sums_kernel(GnArgs a) {
    constexpr int V = NormVec<T>::V;
    __shared__ float s1[kGnThreads * V], s2[kGnThreads * V];
    const GnAt at(a, blockIdx.y, V);
    const int64_t n = blockIdx.x / a.p.blocks, nv = gn_valid(a, n), r0 = int64_t(blockIdx.x % a.p.blocks) * a.p.block_rows, r1 = min(r0 + a.p.block_rows, nv);
    const int cw = a.p.cv * V;
    if (at.left > 0) {
        float w[V], b[V], mean[V], rstd[V], c1[V] = {}, c2[V] = {};
        gn_params<V>(a.weight, a.w_f32, at.c, at.left, 1.0f, w);
        gn_params<V>(a.bias, a.w_f32, at.c, at.left, 0.0f, b);
        int g[V];
        gn_groups<V>(a, at, g);
        gn_thread_stats<V>(a, g, n, mean, rstd);
        const T *x = static_cast<const T *>(a.x) + n * a.x_sample + at.c, *dy = static_cast<const T *>(a.dy) + n * a.L * a.C + at.c;
        for (int64_t r0t = r0 + at.tr; r0t < r1; r0t += kGnAhead * a.p.rt) {
            typename NormVec<T>::raw rx[kGnAhead], rd[kGnAhead];
#pragma unroll
            for (int u = 0; u < kGnAhead; ++u) {
                const int64_t r = r0t + u * a.p.rt;
                rx[u] = gn_load<T, V>(x + r * a.x_row, r < r1 ? at.left : 0);
                rd[u] = gn_load<T, V>(dy + r * a.C, r < r1 ? at.left : 0);
            }
#pragma unroll
            for (int u = 0; u < kGnAhead; ++u) {
                if (r0t + u * a.p.rt >= r1) break;
                float v[V], d[V], z[V];
                NormVec<T>::unpack(rx[u], v);
                NormVec<T>::unpack(rd[u], d);
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    v[j] = (v[j] - mean[j]) * rstd[j];
                    z[j] = fmaf(v[j], w[j], b[j]);
                }
                gn_slope<V>(a.act, z, d);
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    c1[j] += d[j];
                    c2[j] = fmaf(d[j], v[j], c2[j]);
                }
            }
        }
#pragma unroll
        for (int j = 0; j < V; ++j) {
            s1[at.tr * cw + at.col * V + j] = c2[j];
            s2[at.tr * cw + at.col * V + j] = c1[j];
        }
    }
    __syncthreads();
    float *part = a.part + int64_t(blockIdx.x) * 2 * a.C + at.c0;
    for (int c = threadIdx.x; c < at.width; c += kGnThreads) {
        float t1 = 0.0f, t2 = 0.0f;
        for (int r = 0; r < a.p.rt; ++r) {
            t1 += s1[r * cw + c];
            t2 += s2[r * cw + c];
        }
        part[c] = t1;
        part[a.C + c] = t2;
    }
}

// A sample's sums of each channel (into its first block's place) and, weighted, of each group: sums[sample][G][2]. A workgroup per
// group: its threads share the group's channels, up to 256 at a time, and the blocks.
__global__ __launch_bounds__(256) void gn_bwd_join_kernel(GnArgs a, float *sums) {
    __shared__ float s1[256], s2[256];
    const int at_once = min(a.D, 256), shares = 256 / at_once, mine = int(threadIdx.x) / at_once, i0 = int(threadIdx.x) % at_once;
    for (int64_t to = blockIdx.x; to < a.N * a.G; to += gridDim.x) {
        const int64_t n = to / a.G;
        const int g = int(to % a.G);
        float t1 = 0.0f, t2 = 0.0f;
        for (int i = i0; i < a.D + i0; i += at_once) {      // every thread as often
            const int c = g * a.D + min(i, a.D - 1);
            float *p = a.part + n * a.p.blocks * 2 * a.C + c;
            float u2 = 0.0f, u1 = 0.0f;
            if (mine < shares) {
#pragma unroll 4
                for (int k = mine; k < a.p.blocks; k += shares) {
                    u2 += p[int64_t(k) * 2 * a.C];
                    u1 += p[int64_t(k) * 2 * a.C + a.C];
                }
            }
            __syncthreads();
            s1[threadIdx.x] = u1;
            s2[threadIdx.x] = u2;
            __syncthreads();
            if (mine == 0 && i < a.D) {
                for (int m = 1; m < shares; ++m) {
                    u1 += s1[m * at_once + i0];
                    u2 += s2[m * at_once + i0];
                }
                p[0] = u2;
                p[a.C] = u1;
                const float w = !a.weight ? 1.0f : a.w_f32 ? static_cast<const float *>(a.weight)[c] : to_f32(static_cast<const bf16 *>(a.weight)[c]);
                t1 = fmaf(w, u1, t1);
                t2 = fmaf(w, u2, t2);
            }
        }
        __syncthreads();
        s1[threadIdx.x] = t1;
        s2[threadIdx.x] = t2;
        for (int m = 128; m > 0; m >>= 1) {
            __syncthreads();
            if (int(threadIdx.x) < m) {
                s1[threadIdx.x] += s1[threadIdx.x + m];
                s2[threadIdx.x] += s2[threadIdx.x + m];
            }
        }
        if (threadIdx.x == 0) {
            sums[to * 2] = s1[0];
            sums[to * 2 + 1] = s2[0];
        }
    }
}

template <typename T> __global__ __launch_bounds__(kGnThreads) void gn_bwd_apply_kernel(GnArgs a, const float *sums) {
    constexpr int V = NormVec<T>::V;
    const GnAt at(a, blockIdx.y, V);
    if (at.left <= 0) return;
    const int64_t n = blockIdx.x / a.p.blocks, nv = gn_valid(a, n), r0 = int64_t(blockIdx.x % a.p.blocks) * a.p.block_rows, r1 = min(r0 + a.p.block_rows, a.L);
    const float inv = nv > 0 ? 1.0f / (float(nv) * float(a.D)) : 0.0f;
    float w[V], b[V], mean[V], rstd[V], m1[V], m2[V];
    gn_params<V>(a.weight, a.w_f32, at.c, at.left, 1.0f, w);
    gn_params<V>(a.bias, a.w_f32, at.c, at.left, 0.0f, b);
    int g[V];
    gn_groups<V>(a, at, g);
    gn_thread_stats<V>(a, g, n, mean, rstd);
#pragma unroll
    for (int j = 0; j < V; ++j) {
        m1[j] = sums[(n * a.G + g[j]) * 2] * inv;
        m2[j] = sums[(n * a.G + g[j]) * 2 + 1] * inv;
    }
    const T *x = static_cast<const T *>(a.x) + n * a.x_sample + at.c, *dy = static_cast<const T *>(a.dy) + n * a.L * a.C + at.c;
    T *dx = static_cast<T *>(a.dx) + n * a.L * a.C + at.c;
#pragma unroll 4
    for (int64_t r = r0 + at.tr; r < r1; r += a.p.rt) {
        float o[V] = {};
        if (r < nv) {
            float v[V], d[V], z[V];
            NormVec<T>::unpack(gn_load<T, V>(x + r * a.x_row, at.left), v);
            NormVec<T>::unpack(gn_load<T, V>(dy + r * a.C, at.left), d);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                v[j] = (v[j] - mean[j]) * rstd[j];
                z[j] = fmaf(v[j], w[j], b[j]);
            }
            gn_slope<V>(a.act, z, d);
#pragma unroll
            for (int j = 0; j < V; ++j) o[j] = rstd[j] * (d[j] * w[j] - fmaf(v[j], m2[j], m1[j]));
        }
        norm_put<T, V>(dx + r * a.C, 0, at.left, o);
    }
}

// Column sums of `count` partial rows [.][C], `stride` floats apart, at part (the weight's: blockIdx.y = 0) and part + second (the
// bias's): 16 wavefronts take a share of the rows each for the same 64 columns.
template <typename TW>
__global__ __launch_bounds__(1024) void gn_reduce_kernel(const float *part, int64_t second, int64_t stride, int64_t count, int C, TW *dw, TW *db) {
    __shared__ float buf[16][64];
    const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6, c = blockIdx.x * 64 + lane;
    TW *out = blockIdx.y ? db : dw;
    if (!out) return;
    const float *p = part + (blockIdx.y ? second : 0) + c;
    const int64_t share = (count + 15) / 16, g1 = min(count, (wv + 1) * share);
    float s = 0.0f;
    if (c < C) {
#pragma unroll 8
        for (int64_t g = wv * share; g < g1; ++g) s += p[g * stride];
    }
    buf[wv][lane] = s;
    __syncthreads();
    if (wv == 0 && c < C) {
#pragma unroll
        for (int i = 1; i < 16; ++i) s += buf[i][lane];
        out[c] = from_f32<TW>(s);
    }
}

// ---- host ------------------------------------------------------------------------------------------------------------

int pow2_at_most(int64_t n) {
    int p = 1;
    while (p * 2 <= n) p *= 2;
    return p;
}

// bwd: rows held by a thread cost three times the registers.
GnPlan gn_plan(int64_t N, int64_t L, int C, int G, int V, bool bwd) {
    const int D = C / G;
    if (L < 1) L = 1;
    GnPlan p{};
    // Resident: rows of the tile at least 512 bytes (or whole) if they fit so, else 128, with as few rows to a thread as fit.
    for (int run : {32, 8}) {
        for (int threads : {256, 1024}) {
            if (threads == 1024 && (D <= 256 * V || D % V)) continue;     // groups wider than 256 threads
            for (int items : {1, 2, 4, 8}) {
                if ((bwd && items > 4) || (threads == 1024 && items > (bwd ? 1 : 2)) || L > int64_t(threads) * items) continue;
                const int rs = int((L + items - 1) / items);
                const int64_t most = int64_t(threads / rs) * V;     // channels of a tile
                if (D > most) continue;
                int gt = int(most / D < G ? most / D : G);
                if (gt < G && gt * D < run * V) continue;
                const int tiles = (G + gt - 1) / gt;
                gt = (G + tiles - 1) / tiles;
                p.threads = threads;
                p.items = items;
                p.gt = gt;
                p.tiles = (G + gt - 1) / gt;
                p.cv = (gt * D + V - 1) / V;
                p.rt = threads / p.cv;
                p.rs = rs;
                p.spw = p.rt / rs;
                const int vecs = D / V;
                p.mode = D % V ? kChannels : rs == 1 && vecs <= 64 && (vecs & (vecs - 1)) == 0 ? kShuffle : kVectors;
                const int64_t per = int64_t(rs) * (D % V ? D : vecs), all = int64_t(p.spw) * gt;
                p.lanes = p.mode == kShuffle ? vecs : pow2_at_most(per < 64 ? per : 64);
                while (p.mode != kShuffle && p.lanes > 1 && all * p.lanes > threads) p.lanes /= 2;
                return p;
            }
        }
    }
    const int most = kGnThreads * V;
    p.threads = kGnThreads;
    if (D <= most) {
        p.gt = most / D < G ? most / D : G;
        p.tiles = (G + p.gt - 1) / p.gt;
        p.gt = (G + p.tiles - 1) / p.tiles;
        p.tiles = (G + p.gt - 1) / p.gt;
        p.cv = (p.gt * D + V - 1) / V;
    } else {
        const int pieces = (D + most - 1) / most;
        p.tiles = pieces * G;
        p.cv = ((D + pieces - 1) / pieces + V - 1) / V;
    }
    p.rt = kGnThreads / p.cv;
    p.lanes = pow2_at_most(kGnThreads / (p.gt > 0 ? p.gt : 1) < 64 ? kGnThreads / (p.gt > 0 ? p.gt : 1) : 64);
    // Blocks of eight rows to a thread, or of four where eight leave the device half empty (8 x 4096 x 512 bfloat16, training, in a form
    // that took 83 us with eight: four 93, sixteen 81; 5 x 1001 x 320 float32: 51, 46 and 71), at most 2048 workgroups.
    const int64_t eight = (L + p.rt * 8 - 1) / (p.rt * 8), four = (L + p.rt * 4 - 1) / (p.rt * 4), most_blocks = 2048 / (N * p.tiles < 2048 ? N * p.tiles : 2048);
    const int64_t fit = N * p.tiles * eight >= 512 ? eight : four, blocks = fit < most_blocks ? fit : most_blocks;
    p.block_rows = int((L + blocks - 1) / blocks);
    p.blocks = int((L + p.block_rows - 1) / p.block_rows);
    return p;
}
// Workgroups of a resident tile: each takes samples in turn. The backward's, half as many as fill the device, leave a row of
// sums each (8192 x 4096 bfloat16: 2048 took 57 + 6 us, 1024 52 + 4, 512 61 + 4).
unsigned gn_grid(const GnPlan &p, int64_t N, bool bwd) {
    const int64_t blocks = (N + p.spw - 1) / p.spw, want = (p.threads == 256 ? (bwd ? 1024 : 2048) : 512) / p.tiles;
    return unsigned(blocks < want ? blocks : want < 1 ? 1 : want);
}

template <bool BWD, typename T, int NT, int ITEMS, int MODE> hipError_t gn_go(const GnArgs &a, hipStream_t st) {
    const dim3 grid(gn_grid(a.p, a.N, BWD), unsigned(a.p.tiles));
    if constexpr (BWD) hipLaunchKernelGGL((gn_bwd_kernel<T, NT, ITEMS, MODE>), grid, dim3(NT), 0, st, a);
    else hipLaunchKernelGGL((gn_fwd_kernel<T, NT, ITEMS, MODE>), grid, dim3(NT), 0, st, a);
    return hipGetLastError();
}
template <bool BWD, typename T, int ITEMS> hipError_t gn_mode(const GnArgs &a, hipStream_t st) {
    if (a.p.threads == 1024) {
        if constexpr (ITEMS <= (BWD ? 1 : 2)) return gn_go<BWD, T, 1024, ITEMS, kVectors>(a, st);
        return hipErrorInvalidValue;      // gn_plan gives no such plan
    }
    switch (a.p.mode) {
        case kShuffle: return gn_go<BWD, T, 256, ITEMS, kShuffle>(a, st);
        case kVectors: return gn_go<BWD, T, 256, ITEMS, kVectors>(a, st);
        default: return gn_go<BWD, T, 256, ITEMS, kChannels>(a, st);
    }
}
template <bool BWD, typename T> hipError_t gn_resident(const GnArgs &a, hipStream_t st) {
    switch (a.p.items) {
        case 1: return gn_mode<BWD, T, 1>(a, st);
        case 2: return gn_mode<BWD, T, 2>(a, st);
        case 4: return gn_mode<BWD, T, 4>(a, st);
        default:
            if constexpr (!BWD) return gn_mode<BWD, T, 8>(a, st);
            return hipErrorInvalidValue;
    }
}

size_t gn_floats(int64_t N, int C, int G, const GnPlan &p, bool bwd) {
    if (p.items > 0) return bwd ? size_t(gn_grid(p, N, true)) * size_t(C) * 2 : 0;
    if (!bwd) return size_t(N) * size_t(p.blocks) * size_t(p.gt > 0 ? G : p.tiles) * 2;
    return size_t(N) * (size_t(p.blocks) * size_t(C) * 2 + size_t(G) * 2);
}

// Workgroups of 256 threads stay below 2^24 in a launch (a resident plan's always do).
bool gn_launches(const GnPlan &p, int64_t N) { return p.items > 0 || N * p.blocks * p.tiles < int64_t(1) << 24; }
dim3 gn_join_grid(const GnArgs &a) { return dim3(unsigned(a.N * a.G < 65536 ? a.N * a.G : 65536)); }

template <typename T> hipError_t gn_fwd(const GnArgs &a, hipStream_t st) {
    if (a.p.items > 0) return gn_resident<false, T>(a, st);
    const dim3 grid(unsigned(a.N * a.p.blocks), unsigned(a.p.tiles));
    hipLaunchKernelGGL(gn_stats_kernel<T>, grid, dim3(kGnThreads), 0, st, a);
    hipLaunchKernelGGL(gn_join_kernel, gn_join_grid(a), dim3(64), 0, st, a, NormVec<T>::V);
    hipLaunchKernelGGL(gn_apply_kernel<T>, grid, dim3(kGnThreads), 0, st, a);
    return hipGetLastError();
}
template <typename T> hipError_t gn_bwd(const GnArgs &a, bool sums, void *dw, void *db, hipStream_t st) {
    int64_t second = 0, stride = 0, count = 0;
    hipError_t e;
    if (a.N == 0) {     // no rows: the reductions write zeros
    } else if (a.p.items > 0) {
        if ((e = gn_resident<true, T>(a, st)) != hipSuccess) return e;
        count = gn_grid(a.p, a.N, true);
        stride = a.C;
        second = count * a.C;
    } else {
        const dim3 grid(unsigned(a.N * a.p.blocks), unsigned(a.p.tiles));
        float *groups = a.part + size_t(a.N) * size_t(a.p.blocks) * size_t(a.C) * 2;
        hipLaunchKernelGGL(gn_bwd_sums_kernel<T>, grid, dim3(kGnThreads), 0, st, a);
        hipLaunchKernelGGL(gn_bwd_join_kernel, gn_join_grid(a), dim3(256), 0, st, a, groups);
        if (a.dx) hipLaunchKernelGGL(gn_bwd_apply_kernel<T>, grid, dim3(kGnThreads), 0, st, a, groups);
        if ((e = hipGetLastError()) != hipSuccess) return e;
        count = a.N;
        stride = int64_t(a.p.blocks) * 2 * a.C;
        second = a.C;
    }
    if (!sums) return hipSuccess;
    const dim3 grid(unsigned((a.C + 63) / 64), 2);
    if (a.w_f32)
        hipLaunchKernelGGL(gn_reduce_kernel<float>, grid, dim3(1024), 0, st, a.part, second, stride, count, a.C, static_cast<float *>(dw), static_cast<float *>(db));
    else
        hipLaunchKernelGGL(gn_reduce_kernel<bf16>, grid, dim3(1024), 0, st, a.part, second, stride, count, a.C, static_cast<bf16 *>(dw), static_cast<bf16 *>(db));
    return hipGetLastError();
}

int gn_check(const sdm_group_shape *s) {
    if (!s) return fail(SDM_ERR_NULL, "shape must not be NULL");
    if ((s->dtype != SDM_F32 && s->dtype != SDM_BF16) || (s->weight_dtype != SDM_F32 && s->weight_dtype != SDM_BF16))
        return fail(SDM_ERR_DTYPE, "dtype and weight_dtype must be SDM_F32 or SDM_BF16, got %d and %d", s->dtype, s->weight_dtype);
    if (s->dtype == SDM_F32 && s->weight_dtype != SDM_F32) return fail(SDM_ERR_DTYPE, "float32 rows take float32 parameters");
    if (s->samples < 0 || s->rows < 0 || s->channels < 1 || s->groups < 1)
        return fail(SDM_ERR_SHAPE, "samples and rows must be >= 0, channels and groups >= 1, got %lld, %lld, %d and %d", (long long)s->samples,
                    (long long)s->rows, s->channels, s->groups);
    if (s->channels % s->groups) return fail(SDM_ERR_SHAPE, "channels (%d) must be a multiple of groups (%d)", s->channels, s->groups);
    if (s->activation < SDM_ACT_NONE || s->activation > SDM_ACT_GELU)
        return fail(SDM_ERR_RANGE, "activation must be one of SDM_ACT_*, got %d", s->activation);
    if (!(s->eps >= 0.0f)) return fail(SDM_ERR_RANGE, "eps must be >= 0, got %g", double(s->eps));
    if (s->samples > 0x7fffffff || s->rows > 0x7fffffff || s->channels > 1 << 20)
        return fail(SDM_ERR_RANGE, "at most 2^31 - 1 samples and rows of 2^20 channels, got %lld, %lld and %d", (long long)s->samples,
                    (long long)s->rows, s->channels);
    return SDM_OK;
}

// The arguments without their outputs; `bwd`: whose plan.
int gn_args(const sdm_group_shape *s, bool bwd, const void *x, int64_t x_sample, int64_t x_row, const void *weight, const void *bias,
            const int32_t *valid, const sdm_exec *exec, GnArgs *a) {
    if (!exec) return fail(SDM_ERR_NULL, "exec must not be NULL");
    if (x_sample < 0 || x_row < 0) return fail(SDM_ERR_SHAPE, "x: strides must be >= 0");
    if (!aligned(x, s->dtype == SDM_BF16 ? 2 : 4)) return fail(SDM_ERR_ALIGN, "x must be aligned to its element size");
    const size_t ws = s->weight_dtype == SDM_BF16 ? 2 : 4;
    if (!aligned(weight, ws) || !aligned(bias, ws)) return fail(SDM_ERR_ALIGN, "weight and bias must be aligned to their element size");
    if (!aligned(valid, 4)) return fail(SDM_ERR_ALIGN, "valid_rows must be 4-byte aligned");
    a->x = x; a->weight = weight; a->bias = bias; a->valid = valid;
    a->N = s->samples; a->L = s->rows; a->x_sample = x_sample; a->x_row = x_row;
    a->C = s->channels; a->G = s->groups; a->D = s->channels / s->groups;
    a->act = s->activation; a->w_f32 = s->weight_dtype == SDM_F32; a->eps = s->eps;
    a->p = gn_plan(s->samples > 0 ? s->samples : 1, s->rows, s->channels, s->groups, s->dtype == SDM_BF16 ? 8 : 4, bwd);
    if (!gn_launches(a->p, a->N))
        return fail(SDM_ERR_RANGE, "%lld samples of %lld rows are too many for a launch", (long long)a->N, (long long)a->L);
    return SDM_OK;
}

// Whether an output of n bytes at p (null: not wanted) meets an input. `in_place`: it may be x, where that is dense, or grad_out, whose
// elements the thread that writes the output's reads before, and no other.
bool gn_meets(const sdm_group_shape *s, const GnArgs &a, const void *p, size_t n, bool in_place) {
    if (!p) return false;
    const int es = s->dtype == SDM_BF16 ? 2 : 4;
    const Extent x{a.x, {{1, 0}, {a.N, a.x_sample}, {a.L, a.x_row}}, a.C, es};
    const size_t params = size_t(a.C) * (a.w_f32 ? 4 : 2), groups = a.dy ? size_t(a.N) * size_t(a.G) * 4 : 0;
    auto dense = [&](const void *q, size_t m) { return q && overlap(p, n, q, m); };
    return (!(in_place && p == a.x && x.dense()) && x.meets(p, n)) ||
           (!(in_place && p == a.dy) && dense(a.dy, size_t(a.N) * size_t(a.L) * size_t(a.C) * size_t(es))) || dense(a.weight, params) ||
           dense(a.bias, params) || dense(a.valid, size_t(a.N) * 4) || dense(a.mean, groups) || dense(a.rstd, groups);
}

int gn_workspace(const sdm_exec *exec, size_t need, GnArgs *a) {
    if (need == 0) return SDM_OK;
    if (!exec->workspace || exec->workspace_bytes < need)
        return fail(SDM_ERR_WORKSPACE, "workspace of %zu bytes is below the %zu bytes needed", exec->workspace ? exec->workspace_bytes : size_t(0), need);
    if (!aligned(exec->workspace, 256)) return fail(SDM_ERR_ALIGN, "workspace must be 256-byte aligned");
    a->part = static_cast<float *>(exec->workspace);
    return SDM_OK;
}

}  // namespace

}  // namespace sdm

using namespace sdm;

extern "C" {

size_t sdm_group_norm_workspace_bytes(const sdm_group_shape *s, int32_t backward) {
    if (gn_check(s) != SDM_OK || s->samples == 0) return 0;
    const GnPlan p = gn_plan(s->samples, s->rows, s->channels, s->groups, s->dtype == SDM_BF16 ? 8 : 4, backward != 0);
    return gn_launches(p, s->samples) ? align256(gn_floats(s->samples, s->channels, s->groups, p, backward != 0) * 4) : 0;
}

int sdm_group_norm_fwd(const sdm_group_shape *s, const void *x, int64_t x_sample, int64_t x_row, const void *weight, const void *bias,
                       const int32_t *valid, void *y, float *mean, float *rstd, const sdm_exec *exec) {
    g_err[0] = 0;
    GnArgs a{};
    int rc = gn_check(s);
    if (rc || (rc = gn_args(s, false, x, x_sample, x_row, weight, bias, valid, exec, &a))) return rc;
    if (s->samples == 0) return SDM_OK;
    if (!mean || !rstd || (s->rows > 0 && (!x || !y))) return fail(SDM_ERR_NULL, "x, y, mean and rstd must not be NULL");
    if (!aligned(y, s->dtype == SDM_BF16 ? 2 : 4) || !aligned(mean, 4) || !aligned(rstd, 4))
        return fail(SDM_ERR_ALIGN, "y, mean and rstd must be aligned to their element size");
    const size_t groups = size_t(a.N) * size_t(a.G) * 4;
    if (gn_meets(s, a, y, size_t(a.N) * size_t(a.L) * size_t(a.C) * (s->dtype == SDM_BF16 ? 2 : 4), true) || gn_meets(s, a, mean, groups, false) ||
        gn_meets(s, a, rstd, groups, false))
        return fail(SDM_ERR_SHAPE, "y, mean or rstd overlaps an input (y may be a dense x)");
    if ((rc = gn_workspace(exec, sdm_group_norm_workspace_bytes(s, 0), &a))) return rc;
    a.y = y; a.mean = mean; a.rstd = rstd;
    const hipStream_t st = static_cast<hipStream_t>(exec->stream);
    const hipError_t e = s->dtype == SDM_BF16 ? gn_fwd<bf16>(a, st) : gn_fwd<float>(a, st);
    return e == hipSuccess ? SDM_OK : hip_fail(e, "group norm launch");
}

int sdm_group_norm_bwd(const sdm_group_shape *s, const void *grad_out, const void *x, int64_t x_sample, int64_t x_row, const void *weight,
                       const void *bias, const int32_t *valid, const float *mean, const float *rstd, void *grad_x, void *grad_weight,
                       void *grad_bias, const sdm_exec *exec) {
    g_err[0] = 0;
    GnArgs a{};
    int rc = gn_check(s);
    if (rc || (rc = gn_args(s, true, x, x_sample, x_row, weight, bias, valid, exec, &a))) return rc;
    if (!grad_x && !grad_weight && !grad_bias) return SDM_OK;
    const size_t es = s->dtype == SDM_BF16 ? 2 : 4, ws = s->weight_dtype == SDM_BF16 ? 2 : 4;
    if (!aligned(grad_out, es) || !aligned(grad_x, es) || !aligned(grad_weight, ws) || !aligned(grad_bias, ws) || !aligned(mean, 4) || !aligned(rstd, 4))
        return fail(SDM_ERR_ALIGN, "the gradients, mean and rstd must be aligned to their element size");
    if (s->samples > 0 && (!mean || !rstd || (s->rows > 0 && (!grad_out || !x))))
        return fail(SDM_ERR_NULL, "grad_out, x, mean and rstd must not be NULL");
    a.dy = grad_out;
    a.mean = const_cast<float *>(mean); a.rstd = const_cast<float *>(rstd);
    if (gn_meets(s, a, grad_x, size_t(a.N) * size_t(a.L) * size_t(a.C) * es, true) || gn_meets(s, a, grad_weight, size_t(a.C) * ws, false) ||
        gn_meets(s, a, grad_bias, size_t(a.C) * ws, false))
        return fail(SDM_ERR_SHAPE, "a gradient overlaps an input (grad_x may be grad_out, or a dense x)");
    const bool sums = grad_weight || grad_bias;
    const bool split = a.p.items == 0;
    if ((sums || split) && (rc = gn_workspace(exec, sdm_group_norm_workspace_bytes(s, 1), &a))) return rc;
    a.dx = grad_x;
    const hipStream_t st = static_cast<hipStream_t>(exec->stream);
    const hipError_t e = s->dtype == SDM_BF16 ? gn_bwd<bf16>(a, sums, grad_weight, grad_bias, st) : gn_bwd<float>(a, sums, grad_weight, grad_bias, st);
    return e == hipSuccess ? SDM_OK : hip_fail(e, "group norm backward launch");
}

}  // extern "C"
