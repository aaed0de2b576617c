// The gated delta rule token by token, for single tokens and a few at once.
//
// With r = k S and s = q S of the state before the token, a = exp(g) and c = q k:
//     u = beta (v - a r),   out = scale (a s + c u),   S = a S + k u
// so both products and c need the old state only and share one reduction.
//
// Bound by memory: a state is 4 K V bytes read and written once per call, against 2 (2 K + 2 V)
// of bfloat16 rows. A wavefront owns CW columns of one state and keeps them in registers
// through all tokens: CW / VW lanes side by side hold VW columns each of a row, and
// RG = 64 VW / CW such groups of lanes a share of the rows each, so a load instruction fetches RG row pieces of CW columns
// and the reduction over the rows is RG-way across lanes. Wavefronts share nothing.
// Measured: 64 streams x 32 heads of 128 x 128: 46 us, 5.8 TB/s (a large copy: 5.1); one stream of 16 heads: 5.7 us, a launch
// and the way to memory and back; 7 x 10 heads of 72 x 200, float32: 6.2 us, three tokens 8.6. Every load of a row is one
// instruction in the lanes that have it whole, and one branch in the others: with a branch per element the first figure was 56.
#include <type_traits>

#include "delta.h"

namespace sdm {

namespace {

// Sum over the lanes whose index differs in the bits from LOW (4 or 8) up, the same bits in all of them: rotations within rows of
// 16 lanes, then the halves of pairs of rows and of the wavefront, swapped. (With four shuffles through LDS a further token of 128 x
// 128 took 1.1 us, this way 0.87.)
template <int LOW> __device__ __forceinline__ float rows_sum(float x) {
    auto rotated = [](float y, auto ctrl) {
        return __uint_as_float(__builtin_amdgcn_update_dpp(0u, __float_as_uint(y), decltype(ctrl)::value, 0xF, 0xF, false));
    };
    x += rotated(x, std::integral_constant<int, 0x128>{});                            // by 8
    if constexpr (LOW == 4) x += rotated(x, std::integral_constant<int, 0x124>{});    // by 4
    const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    x = __uint_as_float(r[0]) + __uint_as_float(r[1]);
    const auto h = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return __uint_as_float(h[0]) + __uint_as_float(h[1]);
}

// The lane's VW columns of a state row of which `cols` are left: one load or store at any element address where all are.
constexpr int VW = 4;
typedef float f4u __attribute__((ext_vector_type(4), aligned(4)));
__device__ __forceinline__ void cols_load(const float *p, int cols, float (&o)[VW]) {
    if (cols >= VW) {
        const f4u x = *reinterpret_cast<const f4u *>(p);
#pragma unroll
        for (int j = 0; j < VW; ++j) o[j] = x[j];
    } else {
#pragma unroll
        for (int j = 0; j < VW; ++j) o[j] = 0.0f;
        if (cols > 0) {     // one branch for the lanes past the end
#pragma unroll
            for (int j = 0; j < VW; ++j)
                if (j < cols) o[j] = p[j];
        }
    }
}
__device__ __forceinline__ void cols_store(float *p, int cols, const float (&o)[VW]) {
    if (cols >= VW) *reinterpret_cast<f4u *>(p) = f4u{o[0], o[1], o[2], o[3]};
    else {
#pragma unroll
        for (int j = 0; j < VW; ++j)
            if (j < cols) p[j] = o[j];
    }
}

// N neighbours of a row of q or k of which `left` are there, zeros after them: 16 bytes (four elements: 8 or 16) per load at any
// element address.
__device__ __forceinline__ void row_load(const float *p, float (&o)[4]) {
    const f4u x = *reinterpret_cast<const f4u *>(p);
#pragma unroll
    for (int j = 0; j < 4; ++j) o[j] = x[j];
}
template <int N> __device__ __forceinline__ void row_load(const bf16 *p, float (&o)[N]) {
    typedef uint32_t raw __attribute__((ext_vector_type(N / 2), aligned(2)));
    const raw x = *reinterpret_cast<const raw *>(p);
#pragma unroll
    for (int j = 0; j < N / 2; ++j) {
        o[2 * j] = __uint_as_float(x[j] << 16);
        o[2 * j + 1] = __uint_as_float(x[j] & 0xFFFF0000u);
    }
}
template <typename T, int N> __device__ __forceinline__ void rows_load(const T *p, int left, float (&o)[N]) {
    constexpr int S = sizeof(T) == 4 || N < 8 ? 4 : 8;
#pragma unroll
    for (int i = 0; i < N; i += S) {
        float x[S];
        if (left >= i + S) row_load(p + i, x);
        else {
#pragma unroll
            for (int j = 0; j < S; ++j) x[j] = 0.0f;
            if (left > i) {     // one branch for the lanes past the end
#pragma unroll
                for (int j = 0; j < S; ++j)
                    if (i + j < left) x[j] = to_f32(p[i + j]);
            }
        }
#pragma unroll
        for (int j = 0; j < S; ++j) o[i + j] = x[j];
    }
}

__device__ __forceinline__ void out_store(float *p, int cols, const float (&o)[VW]) { cols_store(p, cols, o); }
__device__ __forceinline__ void out_store(bf16 *p, int cols, const float (&o)[VW]) {
    typedef uint32_t raw __attribute__((ext_vector_type(2), aligned(2)));
    if (cols >= VW) *reinterpret_cast<raw *>(p) = raw{f32x2_to_bf16x2(o[0], o[1]), f32x2_to_bf16x2(o[2], o[3])};
    else {
#pragma unroll
        for (int j = 0; j < VW; ++j)
            if (j < cols) p[j] = from_f32<bf16>(o[j]);
    }
}

template <typename T, int CW, int RPL>
__global__ __launch_bounds__(256) void delta_step_kernel(DeltaArgs a) {
    constexpr int LPR = CW / VW;                     // lanes per row piece
    const int lane = threadIdx.x & 63;
    const int slices = (a.V + CW - 1) / CW;
    const int64_t wave = int64_t(blockIdx.x) * 4 + (threadIdx.x >> 6);
    if (wave >= int64_t(a.P) * a.Hv * slices) return;
    const int slice = int(wave % slices);
    const int h = int(wave / slices % a.Hv), p = int(wave / slices / a.Hv);
    const int hk = h / (a.Hv / a.Hk);
    const int rg = lane / LPR, c0 = slice * CW + lane % LPR * VW;
    const int cols = a.V - c0;                       // left from c0 on, <= 0 for lanes past the state
    T *out = static_cast<T *>(a.out) + (int64_t(p) * a.T * a.Hv + h) * a.V + c0;
    const int64_t so = int64_t(a.Hv) * a.V;
    const int64_t slot = a.ids ? int64_t(a.ids[p]) : p;
    const bool idle = slot < 0 || slot >= a.slots;
    const int n = idle ? 0 : delta_valid(a, p);
    auto put = [&](int t, const float (&o)[VW]) {
        if (rg == 0) out_store(out + t * so, cols, o);
    };
    const float zero[VW] = {};
    for (int t = n; t < a.T; ++t) put(t, zero);
    if (idle || (n == 0 && a.state == a.state_out)) return;

    const int64_t s0 = (slot * a.Hv + h) * a.K * a.V + c0;
    float S[RPL][VW];
    const int row0 = rg * RPL;                       // a lane's rows are neighbours: so are its elements of q and k
#pragma unroll
    for (int i = 0; i < RPL; ++i) {
        const int row = row0 + i;
#pragma unroll
        for (int j = 0; j < VW; ++j) S[i][j] = 0.0f;
        if (row < a.K) cols_load(a.state + s0 + int64_t(row) * a.V, cols, S[i]);
    }
    const T *kp = static_cast<const T *>(a.k.data) + p * a.k.sp + hk * a.k.sh;
    const T *qp = static_cast<const T *>(a.q.data) + p * a.q.sp + hk * a.q.sh;
    const T *vp = static_cast<const T *>(a.v.data) + p * a.v.sp + h * a.v.sh + c0;
    const float *bp = a.beta + int64_t(p) * a.T * a.Hv + h, *gp = a.g + int64_t(p) * a.T * a.Hv + h;
    for (int t = 0; t < n; ++t) {
        float kk[RPL], qq[RPL], r[VW] = {}, s[VW] = {}, c = 0.0f, v[VW];
        rows_load(kp + t * a.k.st + row0, a.K - row0, kk);
        rows_load(qp + t * a.q.st + row0, a.K - row0, qq);
        rows_load(vp + t * a.v.st, cols, v);
        const float beta = bp[int64_t(t) * a.Hv], decay = expf(gp[int64_t(t) * a.Hv]);
#pragma unroll
        for (int i = 0; i < RPL; ++i) {
            c = fmaf(qq[i], kk[i], c);
#pragma unroll
            for (int j = 0; j < VW; ++j) {
                r[j] = fmaf(kk[i], S[i][j], r[j]);
                s[j] = fmaf(qq[i], S[i][j], s[j]);
            }
        }
        c = rows_sum<LPR>(c);
        float u[VW], o[VW];
#pragma unroll
        for (int j = 0; j < VW; ++j) {
            r[j] = rows_sum<LPR>(r[j]);
            s[j] = rows_sum<LPR>(s[j]);
            u[j] = beta * (v[j] - decay * r[j]);
            o[j] = a.scale * fmaf(c, u[j], decay * s[j]);
        }
        put(t, o);
#pragma unroll
        for (int i = 0; i < RPL; ++i)
#pragma unroll
            for (int j = 0; j < VW; ++j) S[i][j] = fmaf(kk[i], u[j], decay * S[i][j]);
    }
#pragma unroll
    for (int i = 0; i < RPL; ++i) {
        const int row = row0 + i;
        if (row < a.K) cols_store(a.state_out + s0 + int64_t(row) * a.V, cols, S[i]);
    }
}

template <typename T, int CW, int RPL> hipError_t step_go(const DeltaArgs &a, hipStream_t st) {
    const int64_t waves = int64_t(a.P) * a.Hv * ((a.V + CW - 1) / CW);
    hipLaunchKernelGGL((delta_step_kernel<T, CW, RPL>), dim3(unsigned((waves + 3) / 4)), dim3(256), 0, st, a);
    return hipGetLastError();
}
// The fewest rows per lane that hold K.
template <typename T, int CW> hipError_t step_rows(const DeltaArgs &a, hipStream_t st) {
    constexpr int RG = 64 * VW / CW;
    if (a.K <= 64) return step_go<T, CW, 64 / RG>(a, st);
    if constexpr (CW == 16) {
        if (a.K <= 128) return step_go<T, CW, 128 / RG>(a, st);
        return step_go<T, CW, 256 / RG>(a, st);
    }
    return hipErrorInvalidValue;   // step_pick takes wide slices for K <= 64 only
}
template <typename T> hipError_t step_pick(const DeltaArgs &a, int cus, hipStream_t st) {
    // Eight rows of four columns per lane keep enough loads on their way: with K = 128, 16 columns took 55 us where 32 (sixteen
    // rows) took 60 (64 streams x 32 heads x 128 x 128; 46 since); with K = 64, 32 columns take 15.7 us where 16 take 18.6 (128 x
    // 16 x 64 x 64). Few states take the narrow slices for the wavefronts they give.
    if (a.K <= 64 && int64_t(a.P) * a.Hv * ((a.V + 31) / 32) >= 8 * cus) return step_rows<T, 32>(a, st);
    return step_rows<T, 16>(a, st);
}

}  // namespace

hipError_t launch_delta_step(const DeltaArgs &a, bool is_bf16, int cus, hipStream_t st) {
    return is_bf16 ? step_pick<bf16>(a, cus, st) : step_pick<float>(a, cus, st);
}

}  // namespace sdm
