// Gated linear recurrence over the rows of ragged samples, per channel:
//   a_t = sigmoid(gate_t),  h_t = a_t h_{t-1} + (1 - a_t) x_t,  h_{-1} = h0
// and backward, D_t = dh_t + a_{t+1} D_{t+1} (D_last = dh_last + dh):
//   dx_t = (1 - a_t) D_t,  dgate_t = a_t (1 - a_t) (h_{t-1} - x_t) D_t,  dh0 = a_0 D_0
//
// One lane walks one channel of one sample: right for every case, and bound
// by the latency of its row loads.
#include "rows.h"

namespace spc {
namespace {

struct LrArgs {
    Segs segs;
    int32_t C, reverse;
    int64_t ld;            // row stride of gate and x (and of their gradients: ldg)
    int64_t ldg;
    const int32_t* order;  // row of each position, NULL: the identity

    // Row of the t-th step of the sample [a, b), -1 where the order names none.
    __device__ __forceinline__ int row(int a, int b, int t) const {
        const int q = reverse ? b - 1 - t : a + t;
        if (!order) return q;
        const int r = order[q];
        return unsigned(r) < unsigned(segs.n) ? r : -1;
    }
};

template <typename TT>
__device__ __forceinline__ float get1(const void* p, int64_t i);
template <>
__device__ __forceinline__ float get1<F32>(const void* p, int64_t i) { return static_cast<const float*>(p)[i]; }
template <>
__device__ __forceinline__ float get1<F16>(const void* p, int64_t i) { return float(static_cast<const _Float16*>(p)[i]); }
template <>
__device__ __forceinline__ float get1<BF16>(const void* p, int64_t i) {
    return __uint_as_float(uint32_t(static_cast<const uint16_t*>(p)[i]) << 16);
}
template <typename TT>
__device__ __forceinline__ void put1(void* p, int64_t i, float v);
template <>
__device__ __forceinline__ void put1<F32>(void* p, int64_t i, float v) { static_cast<float*>(p)[i] = v; }
template <>
__device__ __forceinline__ void put1<F16>(void* p, int64_t i, float v) { static_cast<_Float16*>(p)[i] = _Float16(v); }
template <>
__device__ __forceinline__ void put1<BF16>(void* p, int64_t i, float v) { static_cast<uint16_t*>(p)[i] = f32_to_bf16_rne(v); }

// a = sigmoid(g) and na = 1 - a = sigmoid(-g), each to full relative precision.
__device__ __forceinline__ void gates(float g, float& a, float& na) {
    const float e = __expf(-fabsf(g)), big = 1.f / (1.f + e), small = e * big;
    a = g >= 0.f ? big : small;
    na = g >= 0.f ? small : big;
    if (g != g) a = na = g;
}

template <typename TT>
__global__ __launch_bounds__(WAVE) void k_lr_fwd(const void* gate, const void* x, LrArgs p, const float* h0, void* out,
                                                 float* h_last, float* carry) {
    const int s = blockIdx.x, c = blockIdx.y * WAVE + threadIdx.x;
    if (c >= p.C) return;
    const int a0 = p.segs.at(s), b0 = p.segs.at(s + 1);
    float h = h0 ? h0[int64_t(s) * p.C + c] : 0.f;
    for (int t = 0; t < b0 - a0; ++t) {
        const int r = p.row(a0, b0, t);
        if (r < 0) continue;
        float a, na;
        gates(get1<TT>(gate, r * p.ld + c), a, na);
        if (carry) carry[int64_t(r) * p.C + c] = h;
        h = a * h + na * get1<TT>(x, r * p.ld + c);
        put1<TT>(out, int64_t(r) * p.C + c, h);
    }
    if (h_last) h_last[int64_t(s) * p.C + c] = h;
}

template <typename TT>
__global__ __launch_bounds__(WAVE) void k_lr_bwd(const void* dh, const void* gate, const void* x, LrArgs p,
                                                 const float* carry, const float* dh_last, void* dgate, void* dx,
                                                 float* dh0) {
    const int s = blockIdx.x, c = blockIdx.y * WAVE + threadIdx.x;
    if (c >= p.C) return;
    const int a0 = p.segs.at(s), b0 = p.segs.at(s + 1);
    float d = dh_last ? dh_last[int64_t(s) * p.C + c] : 0.f;
    for (int t = b0 - a0 - 1; t >= 0; --t) {
        const int r = p.row(a0, b0, t);
        if (r < 0) continue;
        float a, na;
        gates(get1<TT>(gate, r * p.ld + c), a, na);
        d += get1<TT>(dh, int64_t(r) * p.C + c);
        put1<TT>(dx, r * p.ldg + c, na * d);
        put1<TT>(dgate, r * p.ldg + c, a * na * (carry[int64_t(r) * p.C + c] - get1<TT>(x, r * p.ld + c)) * d);
        d *= a;
    }
    if (dh0) dh0[int64_t(s) * p.C + c] = d;
}

// One row of each of n running sequences: state is read, replaced and rounded to out.
template <typename TT>
__global__ __launch_bounds__(256) void k_lr_step(const void* gate, const void* x, int64_t ld, int64_t n, int32_t C,
                                                 const float* state, float* new_state, void* out) {
    const int64_t i = (int64_t(blockIdx.x) * 256 + threadIdx.x) * 8;
    if (i >= n * C) return;
    using S = typename TT::storage;
    const int64_t r = i / C, o = r * ld + (i - r * C);
    const f32x8_t g = widen<TT>(ld8<TT>(static_cast<const S*>(gate) + o)), v = widen<TT>(ld8<TT>(static_cast<const S*>(x) + o));
    f32x8_t h = widen<F32>(ld8<F32>(state + i));
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        float a, na;
        gates(g[j], a, na);
        h[j] = a * h[j] + na * v[j];
    }
    st8<F32>(new_state + i, narrow<F32>(h));
    st8<TT>(static_cast<S*>(out) + i, narrow<TT>(h));
}

spc_status check_sizes(spc_dtype dtype, int64_t n, int32_t C, int64_t n_seg) {
    if (dtype != SPC_F32 && dtype != SPC_F16 && dtype != SPC_BF16) return fail(SPC_ERR_ARG, "unknown dtype %d", int(dtype));
    if (n < 0 || n >= (int64_t(1) << 31) - 4096) return fail(SPC_ERR_ARG, "n=%lld is out of range", (long long)n);
    if (n_seg < 1 || n_seg >= (int64_t(1) << 31) - 1) return fail(SPC_ERR_ARG, "n_seg=%lld is out of range", (long long)n_seg);
    if (C <= 0 || C % 16) return fail(SPC_ERR_UNSUPPORTED, "C=%d: channels must be a positive multiple of 16", C);
    if (ceil_div(C, WAVE) > 65535) return fail(SPC_ERR_UNSUPPORTED, "C=%d is beyond one launch", C);
    return SPC_OK;
}

// A row stride holds a whole row and keeps every row 16-byte aligned.
spc_status check_stride(spc_dtype dtype, int64_t ld, int32_t C, const char* name) {
    if (ld < C || (ld * dtype_size(dtype)) % 16 || ld >= (int64_t(1) << 31))
        return fail(SPC_ERR_ARG, "%s=%lld: a row stride is at least C=%d and a multiple of 16 bytes", name, (long long)ld, C);
    return SPC_OK;
}

size_t carry_bytes(int64_t n, int32_t C) { return size_t(n) * C * 4; }
size_t ws_need(int64_t, int32_t) { return 16; }

spc_status check_call(spc_dtype dtype, int64_t n, int32_t C, int64_t ld, const int32_t* seg_ptr, int64_t n_seg,
                      const int32_t* order, int32_t reverse, const void* ws, size_t ws_bytes, LrArgs& p) {
    spc_status st = check_sizes(dtype, n, C, n_seg);
    if (st == SPC_OK) st = check_stride(dtype, ld, C, "ld");
    if (st != SPC_OK) return st;
    if (!seg_ptr && n_seg != 1) return fail(SPC_ERR_ARG, "seg_ptr is NULL with n_seg=%lld", (long long)n_seg);
    if (!ws) return fail(SPC_ERR_ARG, "ws is NULL");
    for (const void* q : {(const void*)seg_ptr, (const void*)order, ws})
        if (q && !aligned16(q)) return fail(SPC_ERR_ARG, "device pointers must be 16-byte aligned");
    if (ws_bytes < ws_need(n, C)) return fail(SPC_ERR_WORKSPACE, "ws_bytes=%zu, need %zu", ws_bytes, ws_need(n, C));
    p.segs = Segs{seg_ptr, int32_t(n_seg), int32_t(n)};
    p.C = C, p.reverse = reverse != 0, p.ld = ld, p.ldg = C, p.order = order;
    return SPC_OK;
}

}  // namespace
}  // namespace spc

using namespace spc;

#define LR_DISPATCH(name, grid, block, ...)                                                                       \
    do {                                                                                                          \
        if (dtype == SPC_F32) hipLaunchKernelGGL(name<F32>, grid, block, 0, stream, __VA_ARGS__);                 \
        if (dtype == SPC_F16) hipLaunchKernelGGL(name<F16>, grid, block, 0, stream, __VA_ARGS__);                 \
        if (dtype == SPC_BF16) hipLaunchKernelGGL(name<BF16>, grid, block, 0, stream, __VA_ARGS__);               \
        SPC_LAUNCHED(#name);                                                                                      \
    } while (0)

extern "C" spc_status spc_linear_recurrence_workspace(spc_dtype dtype, int64_t n, int32_t C, int64_t n_seg, size_t* ws,
                                                      size_t* carry) {
    clear_error();
    if (!ws || !carry) return fail(SPC_ERR_ARG, "ws or carry is NULL");
    const spc_status st = check_sizes(dtype, n, C, n_seg);
    if (st == SPC_OK) *ws = ws_need(n, C), *carry = carry_bytes(n, C);
    return st;
}

extern "C" spc_status spc_linear_recurrence_fwd(spc_dtype dtype, const void* gate, const void* x, int64_t ld, int64_t n,
                                                int32_t C, const int32_t* seg_ptr, int64_t n_seg, const int32_t* order,
                                                int32_t reverse, const float* h0, void* out, float* h_last, float* carry,
                                                void* ws, size_t ws_bytes, hipStream_t stream) {
    clear_error();
    LrArgs p;
    const spc_status st = check_call(dtype, n, C, ld, seg_ptr, n_seg, order, reverse, ws, ws_bytes, p);
    if (st != SPC_OK) return st;
    if (n > 0 && (!gate || !x || !out)) return fail(SPC_ERR_ARG, "gate, x or out is NULL");
    for (const void* q : {gate, x, (const void*)h0, (const void*)out, (const void*)h_last, (const void*)carry})
        if (q && !aligned16(q)) return fail(SPC_ERR_ARG, "device pointers must be 16-byte aligned");
    const dim3 grid(unsigned(n_seg), unsigned(ceil_div(C, WAVE)));
    LR_DISPATCH(k_lr_fwd, grid, dim3(WAVE), gate, x, p, h0, out, h_last, carry);
    return SPC_OK;
}

extern "C" spc_status spc_linear_recurrence_bwd(spc_dtype dtype, const void* dout, const void* gate, const void* x,
                                                int64_t ld, int64_t n, int32_t C, const int32_t* seg_ptr, int64_t n_seg,
                                                const int32_t* order, int32_t reverse, const float* h0, const float* carry,
                                                const float* dh_last, void* dgate, void* dx, int64_t ldg, float* dh0,
                                                void* ws, size_t ws_bytes, hipStream_t stream) {
    clear_error();
    LrArgs p;
    spc_status st = check_call(dtype, n, C, ld, seg_ptr, n_seg, order, reverse, ws, ws_bytes, p);
    if (st == SPC_OK) st = check_stride(dtype, ldg, C, "ldg");
    if (st != SPC_OK) return st;
    if (n > 0 && (!dout || !gate || !x || !carry || !dgate || !dx))
        return fail(SPC_ERR_ARG, "dout, gate, x, carry, dgate or dx is NULL");
    for (const void* q : {dout, gate, x, (const void*)h0, (const void*)carry, (const void*)dh_last, (const void*)dgate,
                          (const void*)dx, (const void*)dh0})
        if (q && !aligned16(q)) return fail(SPC_ERR_ARG, "device pointers must be 16-byte aligned");
    p.ldg = ldg;
    const dim3 grid(unsigned(n_seg), unsigned(ceil_div(C, WAVE)));
    LR_DISPATCH(k_lr_bwd, grid, dim3(WAVE), dout, gate, x, p, carry, dh_last, dgate, dx, dh0);
    return SPC_OK;
}

extern "C" spc_status spc_linear_recurrence_step(spc_dtype dtype, const void* gate, const void* x, int64_t ld, int64_t n,
                                                 int32_t C, const float* state, float* new_state, void* out,
                                                 hipStream_t stream) {
    clear_error();
    spc_status st = check_sizes(dtype, n, C, 1);
    if (st == SPC_OK) st = check_stride(dtype, ld, C, "ld");
    if (st != SPC_OK) return st;
    if (n == 0) return SPC_OK;
    if (!gate || !x || !state || !new_state || !out) return fail(SPC_ERR_ARG, "gate, x, state, new_state or out is NULL");
    for (const void* q : {gate, x, (const void*)state, (const void*)new_state, (const void*)out})
        if (!aligned16(q)) return fail(SPC_ERR_ARG, "device pointers must be 16-byte aligned");
    const int64_t blocks = ceil_div(n * C, 8 * 256);
    if (blocks >= (int64_t(1) << 31)) return fail(SPC_ERR_UNSUPPORTED, "%lld rows of %d channels exceed one launch", (long long)n, C);
    LR_DISPATCH(k_lr_step, dim3(unsigned(blocks)), dim3(256), gate, x, ld, n, C, state, new_state, out);
    return SPC_OK;
}
