// Layer norm over the channels of each row, with the residual join before it:
//   u = x + residual,  y = gamma (u - mean) rstd + beta,
//   backward: h = (u - mean) rstd, w = gamma dy,
//   du = rstd (w - mean(w) - h mean(w h)) (+ dtotal),
//   dgamma = sum dy h, dbeta = sum dy over the rows.
// A row lies in the registers of 2 to 64 lanes, eight channels a lane and
// step, so every tensor is read once; what bounds large calls is memory.  266,426 x
// 128 bf16: forward with the residual 50 us (5.4 TB/s), backward onto a later
// gradient 62 us (4.4 TB/s), whose rows wait for three sums each; the sums of
// the workgroups' parts 4.7 us.  Small calls are their launches: 2,000 x 16
// fp32 3.6 us.
//
// Differences are taken from the rounded mean and their own mean, near 0, is
// taken out again: a row far from 0 next to its spread keeps the precision
// that its values have.  The backward does the same from the saved mean.
#include "rows.h"

namespace spc {
namespace {

constexpr int LT = 256;          // threads per workgroup
constexpr int LN_C_MAX = 4096;   // channels that one wave holds: 8 steps of 512

// v of the lane that differs from this one by a step of the row's sum: within
// 16 lanes by lane moves of the vector unit (once the quads' lanes agree, any
// lane of the other quad serves), above by swaps of 16 and 32 lanes; no LDS.
template <int M>
__device__ __forceinline__ float other(float v) {
    const int i = __float_as_int(v);
    if constexpr (M == 1) return __int_as_float(__builtin_amdgcn_mov_dpp(i, 0xB1, 0xf, 0xf, true));        // 1 0 3 2
    else if constexpr (M == 2) return __int_as_float(__builtin_amdgcn_mov_dpp(i, 0x4E, 0xf, 0xf, true));   // 2 3 0 1
    else if constexpr (M == 4) return __int_as_float(__builtin_amdgcn_mov_dpp(i, 0x141, 0xf, 0xf, true));  // mirror of 8
    else return __int_as_float(__builtin_amdgcn_mov_dpp(i, 0x140, 0xf, 0xf, true));                        // mirror of 16
}
__device__ __forceinline__ float sum_rows16(float v) {
    const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}
__device__ __forceinline__ float sum_rows32(float v) {
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

// Sums of K values over the lanes of a row (lanes a power of two from 2 on, aligned).
template <int K>
__device__ __forceinline__ void row_sums(float (&v)[K], int lanes) {
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] += other<1>(v[k]);
    if (lanes < 4) return;
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] += other<2>(v[k]);
    if (lanes < 8) return;
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] += other<4>(v[k]);
    if (lanes < 16) return;
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] += other<8>(v[k]);
    if (lanes < 32) return;
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] = sum_rows16(v[k]);
    if (lanes < 64) return;
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] = sum_rows32(v[k]);
}

__device__ __forceinline__ float sum8(const f32x8_t& v) { return ((v[0] + v[1]) + (v[2] + v[3])) + ((v[4] + v[5]) + (v[6] + v[7])); }

__device__ __forceinline__ f32x8_t ldf8(const float* p) { return widen<F32>(ld8<F32>(p)); }

// V steps of 512 channels (lanes = 64), or one step of `lanes` lanes.
template <typename TT, int V, bool RES>
__global__ __launch_bounds__(LT) void k_ln_fwd(const void* x_, const void* res_, int64_t n, int C, int lanes, float inv_c,
                                               const float* gamma, const float* beta, float eps, void* y_, void* total_,
                                               float2* stats) {
    using S = typename TT::storage;
    const S *x = static_cast<const S*>(x_), *res = static_cast<const S*>(res_);
    S *y = static_cast<S*>(y_), *total = static_cast<S*>(total_);
    const int rl = int(threadIdx.x) / lanes, c0 = (int(threadIdx.x) % lanes) * 8, per = LT / lanes;
    const int64_t r = int64_t(blockIdx.x) * per + rl;
    f32x8_t u[V];
    float s[1] = {0.f};
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int c = c0 + 512 * v;
        u[v] = 0.f;
        if (r < n && c < C) {
            u[v] = widen<TT>(ld8<TT>(x + r * C + c));
            if constexpr (RES) {
                const Raw8<TT> t = narrow<TT>(u[v] + widen<TT>(ld8<TT>(res + r * C + c)));
                st8<TT>(total + r * C + c, t);
                u[v] = widen<TT>(t);      // the sum as it is stored, so that the backward sees the same
            }
        }
        s[0] += sum8(u[v]);
    }
    row_sums(s, lanes);
    const float mean = s[0] * inv_c;
    float q[2] = {0.f, 0.f};
#pragma unroll
    for (int v = 0; v < V; ++v) {
        if (c0 + 512 * v < C) u[v] -= mean;
        q[0] += sum8(u[v]);
        q[1] += sum8(u[v] * u[v]);
    }
    row_sums(q, lanes);
    const float md = q[0] * inv_c, rstd = rsqrtf(fmaxf(fmaf(-md, md, q[1] * inv_c), 0.f) + eps);
    if (r >= n) return;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int c = c0 + 512 * v;
        if (c >= C) continue;
        f32x8_t h = (u[v] - md) * rstd;
        if (gamma) h *= ldf8(gamma + c);
        if (beta) h += ldf8(beta + c);
        st8<TT>(y + r * C + c, narrow<TT>(h));
    }
    if (c0 == 0) stats[r] = float2{mean + md, rstd};
}

// Sums over the rows: every workgroup's part goes to the workspace, and a second
// launch adds the parts up in double, so that results repeat, as atomics' would not.
// A workgroup takes `iters` (at most 16) rows of each of its row groups, keeps
// its channels' two sums in fp32 over them, and adds up the groups in double:
// part[workgroup][C] (dgamma, dbeta), or the results where there is one.
template <typename TT, int V, bool AFFINE, bool JOIN>
__global__ __launch_bounds__(LT) void k_ln_bwd(const void* dy_, const void* x_, int64_t n, int C, int lanes, int iters, float inv_c,
                                               const float* gamma, const float2* stats, const void* dtotal_, void* dx_,
                                               float2* part, float* dgamma, float* dbeta) {
    using S = typename TT::storage;
    const S *dy = static_cast<const S*>(dy_), *x = static_cast<const S*>(x_), *dtotal = static_cast<const S*>(dtotal_);
    S* dx = static_cast<S*>(dx_);
    __shared__ float2 lds[AFFINE ? LT * 8 : 1];
    const int rl = int(threadIdx.x) / lanes, c0 = (int(threadIdx.x) % lanes) * 8, per = LT / lanes;
    f32x8_t sg[V], sb[V];
#pragma unroll
    for (int v = 0; v < V; ++v) sg[v] = 0.f, sb[v] = 0.f;
    // One round's rows as stored; the next round's are in flight while one is
    // worked on (up to 1,024 channels: above, the registers hold one).
    constexpr bool TWO = V <= 2;
    Raw8<TT> xs[V], gs[V], ts[V];
    float2 st;
    auto row = [&](int it) { return (int64_t(blockIdx.x) * iters + it) * per + rl; };
    auto load = [&](int it) {
        const int64_t r = row(it) < n ? row(it) : n - 1;
        st = stats[r];
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int c = c0 + 512 * v < C ? c0 + 512 * v : 0;
            xs[v] = ld8<TT>(x + r * C + c);
            gs[v] = ld8<TT>(dy + r * C + c);
            if constexpr (JOIN) ts[v] = ld8<TT>(dtotal + r * C + c);
        }
    };
    if (TWO) load(0);
    for (int it = 0; it < iters; ++it) {
        const int64_t r = row(it);
        if (!TWO) load(it);
        f32x8_t d[V], g[V], t[JOIN ? V : 1];
        const float rstd = st.y;
        float s[3] = {0.f, 0.f, 0.f};
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const bool in = c0 + 512 * v < C;
            d[v] = in ? widen<TT>(xs[v]) - st.x : f32x8_t(0.f);
            g[v] = in ? widen<TT>(gs[v]) : f32x8_t(0.f);
            if constexpr (JOIN) t[v] = widen<TT>(ts[v]);
        }
        if (TWO && it + 1 < iters) load(it + 1);
#pragma unroll
        for (int v = 0; v < V; ++v) {
            f32x8_t w = g[v];
            if (gamma && c0 + 512 * v < C) w *= ldf8(gamma + c0 + 512 * v);
            s[0] += sum8(d[v]);
            s[1] += sum8(w);
            s[2] += sum8(w * d[v]);
        }
        row_sums(s, lanes);
        const float md = s[0] * inv_c, m1 = s[1] * inv_c, m2 = rstd * fmaf(-md, s[1], s[2]) * inv_c;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int c = c0 + 512 * v;
            if (r >= n || c >= C) continue;
            const f32x8_t h = (d[v] - md) * rstd;
            f32x8_t w = g[v];
            if (gamma) w *= ldf8(gamma + c);
            w = (w - m1 - h * m2) * rstd;
            if constexpr (JOIN) w += t[v];
            st8<TT>(dx + r * C + c, narrow<TT>(w));
            if constexpr (AFFINE) sg[v] += g[v] * h, sb[v] += g[v];
        }
    }
    if constexpr (AFFINE) {
        const int cw = lanes * 8;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            __syncthreads();
#pragma unroll
            for (int e = 0; e < 8; ++e) lds[rl * cw + c0 + e] = float2{sg[v][e], sb[v][e]};
            __syncthreads();
            for (int i = int(threadIdx.x); i < cw; i += LT) {
                const int c = i + 512 * v;
                if (c >= C) continue;
                double a = 0.0, b = 0.0;
                for (int k = 0; k < per; ++k) a += lds[k * cw + i].x, b += lds[k * cw + i].y;
                if (part) {
                    part[int64_t(blockIdx.x) * C + c] = float2{float(a), float(b)};
                } else {
                    if (dgamma) dgamma[c] = float(a);
                    if (dbeta) dbeta[c] = float(b);
                }
            }
        }
    }
}

// Sums of the workgroups' parts in double, four channels to a workgroup.
__global__ __launch_bounds__(LT) void k_ln_sums(const float2* part, int64_t parts, int C, float* dgamma, float* dbeta) {
    __shared__ double2 lds[LT];
    const int e = int(threadIdx.x) & 3, c = int(blockIdx.x) * 4 + e;
    double a = 0.0, b = 0.0;
#pragma unroll 8
    for (int64_t k = threadIdx.x >> 2; k < parts; k += LT / 4) {
        const float2 t = part[k * C + c];
        a += t.x, b += t.y;
    }
    lds[threadIdx.x] = double2{a, b};
    for (int m = LT / 2; m >= 4; m >>= 1) {
        __syncthreads();
        if (int(threadIdx.x) < m) lds[threadIdx.x].x += lds[threadIdx.x + m].x, lds[threadIdx.x].y += lds[threadIdx.x + m].y;
    }
    if (threadIdx.x < 4) {
        if (dgamma) dgamma[c] = float(lds[e].x);
        if (dbeta) dbeta[c] = float(lds[e].y);
    }
}

struct LnCut {
    int lanes, per;          // lanes of a row, rows of a workgroup at a time
    int iters;               // the backward's rounds
    int64_t parts;           // its workgroups
    size_t bytes;
};

spc_status check_sizes(int64_t n, int32_t C, LnCut& k) {
    if (n < 0 || n >= ROWS_END) return fail(SPC_ERR_ARG, "n=%lld is out of range", (long long)n);
    if (C <= 0 || C % 16) return fail(SPC_ERR_UNSUPPORTED, "C=%d: channels must be a positive multiple of 16", C);
    if (C > LN_C_MAX) return fail(SPC_ERR_UNSUPPORTED, "C=%d: at most %d channels", C, LN_C_MAX);
    k.lanes = 2;
    while (k.lanes < 64 && k.lanes * 8 < C) k.lanes *= 2;
    k.per = LT / k.lanes;
    // rounds for about 1,024 workgroups: fewer rounds cost parts to add up, more leave compute units idle
    const int64_t want = ceil_div(n, int64_t(k.per) * 1024);
    k.iters = int(want < 1 ? 1 : want > 16 ? 16 : want);
    k.parts = ceil_div(n, int64_t(k.per) * k.iters);
    k.bytes = k.parts > 1 ? size_t(k.parts) * size_t(C) * 8 : 0;
    if (!launchable(k.parts, LT) || !launchable(ceil_div(n, k.per), LT))
        return fail(SPC_ERR_UNSUPPORTED, "%lld rows of %d channels exceed one launch", (long long)n, C);
    return SPC_OK;
}

Rows dense(spc_dtype dtype, const void* p, int64_t n, int32_t C, const char* name) {
    const int64_t w = int64_t(C) * dtype_size(dtype);
    return Rows{p, n, w, w, name};
}

template <typename TT, int V>
spc_status launch_fwd(const void* x, const void* res, int64_t n, int C, const LnCut& k, const float* gamma, const float* beta,
                      float eps, void* y, void* total, float2* stats, hipStream_t stream) {
    const dim3 grid(unsigned(ceil_div(n, k.per)));
    const float inv = 1.f / float(C);
    if (res) hipLaunchKernelGGL((k_ln_fwd<TT, V, true>), grid, dim3(LT), 0, stream, x, res, n, C, k.lanes, inv, gamma, beta, eps, y, total, stats);
    else hipLaunchKernelGGL((k_ln_fwd<TT, V, false>), grid, dim3(LT), 0, stream, x, res, n, C, k.lanes, inv, gamma, beta, eps, y, total, stats);
    SPC_LAUNCHED("k_ln_fwd");
    return SPC_OK;
}

template <typename TT>
spc_status dispatch_fwd(const void* x, const void* res, int64_t n, int C, const LnCut& k, const float* gamma, const float* beta,
                        float eps, void* y, void* total, float2* stats, hipStream_t stream) {
    if (C <= 512) return launch_fwd<TT, 1>(x, res, n, C, k, gamma, beta, eps, y, total, stats, stream);
    if (C <= 1024) return launch_fwd<TT, 2>(x, res, n, C, k, gamma, beta, eps, y, total, stats, stream);
    if (C <= 2048) return launch_fwd<TT, 4>(x, res, n, C, k, gamma, beta, eps, y, total, stats, stream);
    return launch_fwd<TT, 8>(x, res, n, C, k, gamma, beta, eps, y, total, stats, stream);
}

template <typename TT, int V>
spc_status launch_bwd(const void* dy, const void* x, int64_t n, int C, const LnCut& k, const float* gamma, const float2* stats,
                      const void* dtotal, void* dx, float* dgamma, float* dbeta, float2* part, hipStream_t stream) {
    const dim3 grid(unsigned(k.parts));
    const float inv = 1.f / float(C);
    if (k.parts <= 1) part = nullptr;
#define LN_BWD(AFFINE, JOIN)                                                                                              \
    hipLaunchKernelGGL((k_ln_bwd<TT, V, AFFINE, JOIN>), grid, dim3(LT), 0, stream, dy, x, n, C, k.lanes, k.iters, inv, gamma, \
                       stats, dtotal, dx, part, dgamma, dbeta)
    const bool affine = dgamma || dbeta;
    if (k.parts) {
        if (affine && dtotal) LN_BWD(true, true);
        else if (affine) LN_BWD(true, false);
        else if (dtotal) LN_BWD(false, true);
        else LN_BWD(false, false);
        SPC_LAUNCHED("k_ln_bwd");
    }
#undef LN_BWD
    if (!affine) return SPC_OK;
    if (k.parts != 1) {
        hipLaunchKernelGGL(k_ln_sums, dim3(unsigned(C / 4)), dim3(LT), 0, stream, part, k.parts, C, dgamma, dbeta);
        SPC_LAUNCHED("k_ln_sums");
    }
    return SPC_OK;
}

template <typename TT>
spc_status dispatch_bwd(const void* dy, const void* x, int64_t n, int C, const LnCut& k, const float* gamma, const float2* stats,
                        const void* dtotal, void* dx, float* dgamma, float* dbeta, float2* part, hipStream_t stream) {
    if (n == 0 && !dgamma && !dbeta) return SPC_OK;
    if (C <= 512) return launch_bwd<TT, 1>(dy, x, n, C, k, gamma, stats, dtotal, dx, dgamma, dbeta, part, stream);
    if (C <= 1024) return launch_bwd<TT, 2>(dy, x, n, C, k, gamma, stats, dtotal, dx, dgamma, dbeta, part, stream);
    if (C <= 2048) return launch_bwd<TT, 4>(dy, x, n, C, k, gamma, stats, dtotal, dx, dgamma, dbeta, part, stream);
    return launch_bwd<TT, 8>(dy, x, n, C, k, gamma, stats, dtotal, dx, dgamma, dbeta, part, stream);
}

}  // namespace
}  // namespace spc

using namespace spc;

extern "C" spc_status spc_layer_norm_workspace(int64_t n, int32_t C, size_t* bytes) {
    clear_error();
    if (!bytes) return fail(SPC_ERR_ARG, "bytes is NULL");
    LnCut k;
    const spc_status st = check_sizes(n, C, k);
    if (st == SPC_OK) *bytes = k.bytes;
    return st;
}

extern "C" spc_status spc_layer_norm_fwd(spc_dtype dtype, const void* x, const void* residual, int64_t n, int32_t C,
                                         const float* gamma, const float* beta, float eps, void* y, void* total, float* stats,
                                         hipStream_t stream) {
    clear_error();
    LnCut k;
    if (dtype != SPC_F32 && dtype != SPC_F16 && dtype != SPC_BF16) return fail(SPC_ERR_ARG, "unknown dtype %d", int(dtype));
    spc_status st = check_sizes(n, C, k);
    if (st != SPC_OK) return st;
    if (!(eps > 0.f)) return fail(SPC_ERR_ARG, "eps=%g must be positive", double(eps));
    if (!residual != !total) return fail(SPC_ERR_ARG, "residual and total: give both or neither");
    for (const void* q : {x, residual, (const void*)gamma, (const void*)beta, (const void*)y, (const void*)total, (const void*)stats})
        if (q && !aligned16(q)) return fail(SPC_ERR_ARG, "device pointers must be 16-byte aligned");
    if (n == 0) return SPC_OK;
    if (!x || !y || !stats) return fail(SPC_ERR_ARG, "x, y or stats is NULL");
    const Rows rx = dense(dtype, x, n, C, "x"), rr = dense(dtype, residual, n, C, "residual"), ry = dense(dtype, y, n, C, "y"),
               rt = dense(dtype, total, n, C, "total");
    for (const Rows* in : {&rx, &rr})
        for (const Rows* o : {&ry, &rt})
            if ((st = check_overlap(*o, *in, true)) != SPC_OK) return st;
    if ((st = check_overlap(ry, rt)) != SPC_OK) return st;
    float2* so = reinterpret_cast<float2*>(stats);
    switch (dtype) {
        case SPC_F32: return dispatch_fwd<F32>(x, residual, n, C, k, gamma, beta, eps, y, total, so, stream);
        case SPC_F16: return dispatch_fwd<F16>(x, residual, n, C, k, gamma, beta, eps, y, total, so, stream);
        case SPC_BF16: return dispatch_fwd<BF16>(x, residual, n, C, k, gamma, beta, eps, y, total, so, stream);
    }
    return fail(SPC_ERR_ARG, "unknown dtype %d", int(dtype));
}

extern "C" spc_status spc_layer_norm_bwd(spc_dtype dtype, const void* dout, const void* x, int64_t n, int32_t C, const float* gamma,
                                         const float* stats, const void* dtotal, void* dx, float* dgamma, float* dbeta, void* ws,
                                         size_t ws_bytes, hipStream_t stream) {
    clear_error();
    LnCut k;
    if (dtype != SPC_F32 && dtype != SPC_F16 && dtype != SPC_BF16) return fail(SPC_ERR_ARG, "unknown dtype %d", int(dtype));
    spc_status st = check_sizes(n, C, k);
    if (st != SPC_OK) return st;
    for (const void* q : {dout, x, (const void*)gamma, (const void*)stats, dtotal, (const void*)dx, (const void*)dgamma, (const void*)dbeta, (const void*)ws})
        if (q && !aligned16(q)) return fail(SPC_ERR_ARG, "device pointers must be 16-byte aligned");
    if (n > 0 && (!dout || !x || !stats || !dx)) return fail(SPC_ERR_ARG, "dout, x, stats or dx is NULL");
    const size_t need = dgamma || dbeta ? k.bytes : 0;
    if (need && !ws) return fail(SPC_ERR_ARG, "ws is NULL");
    if (ws_bytes < need) return fail(SPC_ERR_WORKSPACE, "ws_bytes=%zu, need %zu", ws_bytes, need);
    const Rows rx = dense(dtype, x, n, C, "x"), rd = dense(dtype, dout, n, C, "dout"), rt = dense(dtype, dtotal, n, C, "dtotal"),
               ro = dense(dtype, dx, n, C, "dx");
    for (const Rows* in : {&rd, &rt})
        if ((st = check_overlap(ro, *in, true)) != SPC_OK) return st;
    if ((st = check_overlap(ro, rx)) != SPC_OK) return st;
    const float2* si = reinterpret_cast<const float2*>(stats);
    float2* part = static_cast<float2*>(ws);
    switch (dtype) {
        case SPC_F32: return dispatch_bwd<F32>(dout, x, n, C, k, gamma, si, dtotal, dx, dgamma, dbeta, part, stream);
        case SPC_F16: return dispatch_bwd<F16>(dout, x, n, C, k, gamma, si, dtotal, dx, dgamma, dbeta, part, stream);
        case SPC_BF16: return dispatch_bwd<BF16>(dout, x, n, C, k, gamma, si, dtotal, dx, dgamma, dbeta, part, stream);
    }
    return fail(SPC_ERR_ARG, "unknown dtype %d", int(dtype));
}
