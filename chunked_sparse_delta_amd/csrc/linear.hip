// Linear attention with a decay for each head: segments' states, the scans over them, the log-decays' gradient, and the launches.
//
// With G the running sum of a segment's log-decays, in a segment of tokens with the start state S0:
//     S1 = e^{G_end} S0 + sum_t e^{G_end - G_t} k_t v_t,   o_t = scale (e^{G_t} q_t S0 + sum_{j <= t} e^{G_t - G_j} (q_t . k_j) v_j)
// Nothing in the sum of S1 depends on S0, so all segments' sums are made at once (lin_state_kernel), then scanned
// (lin_scan_kernel), then all readings are made at once (linear_attend.h). The gradient of the states runs the same way backwards:
//     dS0 = e^{G_end} dS1 + scale sum_t e^{G_t} q_t do_t
//
// The scan is bound by memory: 134 MB of the sums of 16 heads of 16384 tokens in 32 us (4.2 TB/s).
//
// The gradient of the log-decays. e^{G_i - G_j} is a factor of the pairs (i, j), e^{G_i} of the readings of the start state and
// e^{G_end - G_j} of the tokens' part in the end state. With r_i the readings' share of token i but its own pair (i, i), c_j the
// same of j as a key (both from linear_attend.h), dG_i = r_i - c_i and dG_end has <S1, dS1> besides, so
//     dg_m = sum_{i >= m} (r_i - c_i) + <S1, dS1>
// over the segment: the sums that cancel span one segment, in 64 bits, and leave out what any decay leaves alone. At the segment's
// start this has to be <S0, dS0>: what it misses, the roundings of all the shares, is spread over the segment, which halves it.
// Where e^{g_m} is 0 in float32 nothing before m counts after it, and dg_m = e^{g_m} <S, dS> is 0: there the shares cancel, and the 0 is
// written instead of what their roundings leave (1e-5 of a log-decay of -inf among 400 tokens).
#include "linear_attend.h"
#include "linear_state.h"

namespace sdm {

namespace {

struct ScanArgs {
    float *S;                // [ph][slots][KV]: sums in, states out
    const float *decay;      // [ph][segs]
    const float *first;      // [ph][KV]: the state it begins with, or null
    float *last;             // [ph][KV]: the state it ends with, or null
    const float *with;       // backward: the forward's states [ph][segs + 1][KV], or null
    float *dots;             // backward: [ph][segs + 1][parts]
    const int32_t *valid;
    int32_t T, Hv, KV, segs, slots, seg_tokens, parts;
};

// Segments' sums to segments' start states (and the end state behind them) in place, every element on its own: N neighbours to
// a thread, eight segments' loads on their way at once. BACK: from the last segment to the first, to the
// gradients of their end states; with the products of these and the end states, summed over the wavefront, for the log-decays.
template <int N, bool BACK> __global__ __launch_bounds__(256) void lin_scan_kernel(ScanArgs a) {
    typedef float raw __attribute__((ext_vector_type(N), aligned(4)));
    constexpr int AHEAD = 8;
    const int blocks = (a.KV + 256 * N - 1) / (256 * N), ph = blockIdx.x / blocks;
    const int i = (blockIdx.x % blocks * 256 + threadIdx.x) * N;
    const bool in = i < a.KV;
    const int n = lin_valid(a.valid, ph / a.Hv, a.T), live = (n + a.seg_tokens - 1) / a.seg_tokens;
    float *S = a.S + int64_t(ph) * a.slots * a.KV + i;
    const float *with = BACK && a.with ? a.with + (int64_t(ph) * (a.segs + 1) + 1) * a.KV + i : nullptr;
    const float *decay = a.decay + int64_t(ph) * a.segs;
    // <x, y> of the wavefront's elements at the start of segment m
    auto put_dot = [&](int m, raw x, raw y) {
        float dot = 0.0f;
        if (in) {
#pragma unroll
            for (int e = 0; e < N; ++e) dot = fmaf(x[e], y[e], dot);
        }
#pragma unroll
        for (int d = 32; d > 0; d >>= 1) dot += __shfl_xor(dot, d, 64);
        if ((threadIdx.x & 63) == 0)
            a.dots[(int64_t(ph) * (a.segs + 1) + m) * a.parts + blockIdx.x % blocks * 4 + (threadIdx.x >> 6)] = dot;
    };
    raw s = {};
    if (in && a.first) s = *reinterpret_cast<const raw *>(a.first + int64_t(ph) * a.KV + i);
    for (int m0 = 0; m0 < live; m0 += AHEAD) {
        raw u[AHEAD], o[AHEAD];
#pragma unroll
        for (int j = 0; j < AHEAD; ++j) {
            const int m = BACK ? live - 1 - m0 - j : m0 + j;
            if (in && m0 + j < live) {
                u[j] = *reinterpret_cast<const raw *>(S + int64_t(m) * a.KV);
                if (BACK && with) o[j] = *reinterpret_cast<const raw *>(with + int64_t(m) * a.KV);
            }
        }
#pragma unroll
        for (int j = 0; j < AHEAD; ++j) {
            const int m = BACK ? live - 1 - m0 - j : m0 + j;
            if (m0 + j >= live) break;
            if (BACK && with) put_dot(m + 1, o[j], s);
            if (in) {
                *reinterpret_cast<raw *>(S + int64_t(m) * a.KV) = s;
                const float d = decay[m];
#pragma unroll
                for (int e = 0; e < N; ++e) s[e] = fmaf(d, s[e], u[j][e]);
            }
        }
    }
    if (BACK && with && live > 0) {
        raw x = {};
        if (in) x = *reinterpret_cast<const raw *>(with - a.KV);
        put_dot(0, x, s);
    }
    if (!in) return;
    if (!BACK) *reinterpret_cast<raw *>(S + int64_t(live) * a.KV) = s;
    if (a.last) *reinterpret_cast<raw *>(a.last + int64_t(ph) * a.KV + i) = s;
}

struct GateGradArgs {
    LinGates gates;
    const float *rows, *cols, *dots;
    const int32_t *valid;
    float *g;                // [P, T, Hv], or null:
    double *sums;            // [ph][segs]
    int32_t P, T, Hv, segs, seg_tokens, parts, slices;
};

// Sum over the workgroup's 256 threads, each gets it.
__device__ __forceinline__ double block_sum(double x, double *buf) {
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) x += __shfl_xor(x, d, 64);
    __syncthreads();
    if ((threadIdx.x & 63) == 0) buf[threadIdx.x >> 6] = x;
    __syncthreads();
    return (buf[0] + buf[1]) + (buf[2] + buf[3]);
}

// dg of one segment, a token per thread.
__global__ __launch_bounds__(256) void lin_gate_grad_kernel(GateGradArgs a) {
    __shared__ double buf[4];
    const int seg = blockIdx.x % a.segs, ph = blockIdx.x / a.segs, h = ph % a.Hv, p = ph / a.Hv, tid = threadIdx.x;
    const int s0 = seg * a.seg_tokens, live = min(a.seg_tokens, lin_valid(a.valid, p, a.T) - s0), t = s0 + tid;
    const bool counts = tid < live && expf(a.gates.g[p * a.gates.sp + t * a.gates.st + h]) != 0.0f;
    double head = 0.0, tail = 0.0, d = 0.0;     // at the segment's start and end
    if (live > 0)
        for (int i = tid; i < a.parts; i += 256) {
            const float *at = a.dots + (int64_t(ph) * (a.segs + 1) + seg) * a.parts + i;
            head += at[0];
            tail += at[a.parts];
        }
    if (tid < live)
        for (int s = 0; s < a.slices; ++s) {
            const int64_t at = (int64_t(s) * a.P * a.Hv + ph) * a.T + t;
            d += double(a.rows[at]) + double(a.cols[at]);
        }
    head = block_sum(head, buf);
    tail = block_sum(tail, buf);
    const double all = block_sum(d, buf);
    double before = d;       // the sum up to this token
#pragma unroll
    for (int e = 1; e < 64; e <<= 1) {
        const double o = __shfl_up(before, e, 64);
        if ((tid & 63) >= e) before += o;
    }
    __syncthreads();
    if ((tid & 63) == 63) buf[tid >> 6] = before;
    __syncthreads();
    for (int w = 0; w < tid >> 6; ++w) before += buf[w];
    const double g = counts ? tail + (all - before + d) + (head - (tail + all)) * double(live - tid) / double(live) : 0.0;
    if (a.g) {
        if (tid < a.seg_tokens && t < a.T) a.g[(int64_t(p) * a.T + t) * a.Hv + h] = float(g);
    } else {
        const double s = block_sum(g, buf);
        if (tid == 0) a.sums[int64_t(ph) * a.segs + seg] = s;
    }
}

// A head's log-decay gradient: its streams' segments' sums, by one wavefront.
__global__ __launch_bounds__(64) void lin_gate_sum_kernel(const double *sums, float *g, int P, int Hv, int segs) {
    const int h = blockIdx.x;
    double s = 0.0;
    for (int64_t i = threadIdx.x; i < int64_t(P) * segs; i += 64) s += sums[(i / segs * Hv + h) * segs + i % segs];
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) s += __shfl_xor(s, d, 64);
    if (threadIdx.x == 0) g[h] = float(s);
}

hipError_t launch_state(const StateArgs &a, bool is_bf16, hipStream_t st) { return is_bf16 ? state_pick<bf16>(a, st) : state_pick<float>(a, st); }

template <bool BACK> hipError_t launch_scan(const ScanArgs &a, int heads, hipStream_t st) {
    if (a.KV % 4 == 0)
        hipLaunchKernelGGL((lin_scan_kernel<4, BACK>), dim3(unsigned(heads) * unsigned((a.KV + 1023) / 1024)), dim3(256), 0, st, a);
    else
        hipLaunchKernelGGL((lin_scan_kernel<1, BACK>), dim3(unsigned(heads) * unsigned((a.KV + 255) / 256)), dim3(256), 0, st, a);
    return hipGetLastError();
}

template <typename T, int KP, int ZW> hipError_t state_attr() {
    constexpr size_t bytes = StateCfg<T, KP, ZW, true>::kLds;
    static_assert(bytes <= 80 * 1024, "two workgroups to a compute unit");
    auto set = [](auto kernel) { return hipFuncSetAttribute(reinterpret_cast<const void *>(kernel), hipFuncAttributeMaxDynamicSharedMemorySize, int(bytes)); };
    const hipError_t e = set(&lin_state_kernel<T, KP, ZW, true>);
    return e == hipSuccess ? set(&lin_state_kernel<T, KP, ZW, false>) : e;
}
template <typename T> hipError_t state_prepare() {
    hipError_t e = state_attr<T, 64, 64>();
    if (e == hipSuccess) e = state_attr<T, 64, 128>();
    if (e == hipSuccess) e = state_attr<T, 128, 64>();
    if (e == hipSuccess) e = state_attr<T, 128, 128>();
    if (e == hipSuccess) e = state_attr<T, 256, 64>();
    if (e == hipSuccess) e = state_attr<T, 256, 128>();
    return e;
}

StateArgs state_args(const LinArgs &a, const LinWs &ws) {
    StateArgs s{};
    s.gates = a.gates;
    s.valid = a.valid;
    s.decay = ws.decay;
    s.P = a.P; s.T = a.T; s.Hk = a.Hk; s.Hv = a.Hv; s.K = a.K; s.V = a.V;
    s.segs = ws.segs; s.seg_tokens = ws.tokens;
    return s;
}
AttendArgs attend_args(const LinArgs &a, const LinWs &ws) {
    AttendArgs t{};
    t.gates = a.gates;
    t.valid = a.valid;
    t.P = a.P; t.T = a.T; t.Hk = a.Hk; t.Hv = a.Hv; t.K = a.K; t.V = a.V;
    t.segs = ws.segs;
    t.seg_tokens = ws.tokens;
    return t;
}

// The segments' sums and their scan: ws.S and ws.decay; the end state to `last` (may be null).
hipError_t make_states(const LinArgs &a, const LinWs &ws, float *last, bool is_bf16, hipStream_t st) {
    StateArgs s = state_args(a, ws);
    s.y = a.k;
    s.z = a.v;
    s.S = ws.S;
    s.slots = ws.segs + 1;
    const hipError_t e = launch_state(s, is_bf16, st);
    if (e != hipSuccess) return e;
    ScanArgs c{};
    c.S = ws.S; c.decay = ws.decay; c.first = a.state; c.last = last; c.valid = a.valid;
    c.T = a.T; c.Hv = a.Hv; c.KV = a.K * a.V; c.segs = ws.segs; c.slots = ws.segs + 1; c.seg_tokens = ws.tokens;
    return launch_scan<false>(c, a.P * a.Hv, st);
}

}  // namespace

int lin_dot_parts(int K, int V) { return (K * V + (K * V % 4 ? 255 : 1023)) / (K * V % 4 ? 256 : 1024) * 4; }

hipError_t linear_prepare() {
    hipError_t e = state_prepare<bf16>();
    if (e == hipSuccess) e = state_prepare<float>();
    if (e == hipSuccess) e = attend_prepare_bf16();
    if (e == hipSuccess) e = attend_prepare_f32();
    if (e == hipSuccess) e = grads_prepare_bf16();
    if (e == hipSuccess) e = grads_prepare_f32();
    return e;
}

hipError_t launch_linear_fwd(const LinArgs &a, const LinWs &ws, bool is_bf16, bool keep, hipStream_t st) {
    const int64_t KV = int64_t(a.K) * a.V;
    const bool scan = keep || ws.segs > 1;
    hipError_t e = hipSuccess;
    if (scan && (e = make_states(a, ws, a.state_out, is_bf16, st)) != hipSuccess) return e;
    // one segment: its end state from the start state, after the readings where it goes in the start state's place
    StateArgs s = state_args(a, ws);
    s.y = a.k; s.z = a.v;
    s.S = a.state_out; s.base = a.state; s.decay = nullptr;
    s.slots = 1; s.final = true;
    if (a.T > 0) {
        AttendArgs t = attend_args(a, ws);
        AttendSide &r = t.side[0];
        r.x = a.q; r.y = a.k; r.z = a.v;
        r.M = scan ? ws.S : a.state;
        r.M_head = scan ? (ws.segs + 1) * KV : KV;
        r.M_seg = scan ? KV : 0;
        r.out = a.out;
        r.a0 = r.a1 = a.scale;
        const bool both = !scan && a.state_out && a.state_out != a.state;
        e = is_bf16 ? attend_bf16(t, both ? &s : nullptr, st) : attend_f32(t, both ? &s : nullptr, st);
        if (e != hipSuccess || both) return e;
    }
    if (scan || !a.state_out) return hipSuccess;
    return launch_state(s, is_bf16, st);
}

hipError_t launch_linear_bwd(const LinArgs &a, const LinWs &ws, const LinGrads &g, bool is_bf16, bool kept, hipStream_t st) {
    const int64_t KV = int64_t(a.K) * a.V;
    hipError_t e = hipSuccess;
    if (!kept && (e = make_states(a, ws, nullptr, is_bf16, st)) != hipSuccess) return e;
    StateArgs s = state_args(a, ws);
    s.y = a.q; s.z = g.go;
    s.S = ws.dS; s.decay = nullptr;
    s.slots = ws.segs; s.scale = a.scale; s.back = true;
    if ((e = launch_state(s, is_bf16, st)) != hipSuccess) return e;
    ScanArgs c{};
    c.S = ws.dS; c.decay = ws.decay; c.first = g.gstate; c.last = g.state; c.valid = a.valid;
    c.with = g.g ? ws.S : nullptr; c.dots = ws.dots; c.parts = lin_dot_parts(a.K, a.V);
    c.T = a.T; c.Hv = a.Hv; c.KV = a.K * a.V; c.segs = ws.segs; c.slots = ws.segs; c.seg_tokens = ws.tokens;
    if ((e = launch_scan<true>(c, a.P * a.Hv, st)) != hipSuccess) return e;
    if (a.T > 0) {
        AttendArgs t = attend_args(a, ws);
        AttendSide &q = t.side[0], &k = t.side[1], &v = t.side[2];
        q.x = g.go; q.y = a.v; q.z = a.k; q.own = a.q;
        q.M = ws.S; q.M_head = (ws.segs + 1) * KV; q.M_seg = KV;
        q.out = g.q; q.dot = g.g ? ws.rows : nullptr;
        q.a0 = q.a1 = a.scale;
        q.rest = ws.rest;
        k.x = a.v; k.y = g.go; k.z = a.q; k.own = a.k;
        k.M = ws.dS; k.M_head = ws.segs * KV; k.M_seg = KV;
        k.out = g.k; k.dot = g.g ? ws.cols : nullptr;
        k.a0 = 1.0f; k.a1 = a.scale; k.back = true;
        k.rest = ws.rest + lin_rest_floats(a.P, a.Hk, a.K, ws.segs, ws.tokens);
        v = k;
        v.x = a.k; v.y = a.q; v.z = g.go;
        v.out = g.v; v.dot = nullptr;
        if ((e = is_bf16 ? attend_grads_bf16(t, st) : attend_grads_f32(t, st)) != hipSuccess) return e;
    }
    if (!g.g) return hipSuccess;
    GateGradArgs d{};
    const bool per_token = a.gates.st != 0;
    d.gates = a.gates;
    d.rows = ws.rows; d.cols = ws.cols; d.dots = ws.dots; d.valid = a.valid;
    d.g = per_token ? g.g : nullptr; d.sums = ws.sums;
    d.P = a.P; d.T = a.T; d.Hv = a.Hv; d.segs = ws.segs; d.seg_tokens = ws.tokens;
    d.parts = c.parts; d.slices = lin_slices(a.K);
    hipLaunchKernelGGL(lin_gate_grad_kernel, dim3(unsigned(a.P) * unsigned(a.Hv) * unsigned(ws.segs)), dim3(256), 0, st, d);
    if ((e = hipGetLastError()) != hipSuccess || per_token) return e;
    hipLaunchKernelGGL(lin_gate_sum_kernel, dim3(unsigned(a.Hv)), dim3(64), 0, st, ws.sums, g.g, a.P, a.Hv, ws.segs);
    return hipGetLastError();
}

}  // namespace sdm
