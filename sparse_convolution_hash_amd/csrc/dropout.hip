// Dropout whose mask is drawn from a counter and never stored:
//   forward   out[i] = residual[i] + (keep(i) ? x[i] * scale : 0)
//   backward  din[i] = keep(i) ? dout[i] * scale : 0
// keep(i) is a function of (seed, offset, layer, i) alone (rows.h), so the
// backward draws the forward's mask again instead of reading one: 2 tensors
// of traffic (3 with a residual), no mask bytes.  One thread takes the eight
// elements of one Philox counter, the whole of its 128 bits, so the generator
// costs 7 instructions an element and hides behind the memory: 266,426 x 128
// bf16 with a residual 36 us (5.7 TB/s), without 23 us (5.9 TB/s), the rate of a
// copy of that size.
#include "rows.h"

namespace spc {
namespace {

constexpr int DT = 256;  // threads per workgroup

template <typename TT, bool RES>
__global__ __launch_bounds__(DT) void k_dropout(const void* x_, const void* res_, int64_t numel, Drop d, void* out_) {
    using S = typename TT::storage;
    const S* x = static_cast<const S*>(x_);
    const S* res = static_cast<const S*>(res_);
    S* out = static_cast<S*>(out_);
    const uint64_t seed = d.rng[0], offset = d.rng[1];
    const int64_t step = int64_t(gridDim.x) * DT;
    for (int64_t g = int64_t(blockIdx.x) * DT + threadIdx.x; g * 8 < numel; g += step) {
        const int64_t i = g * 8;
        const u32x4 bits = philox(seed, offset + uint64_t(g), d.layer);
        if (i + 8 <= numel) {
            f32x8_t v = drop8(widen<TT>(ld8<TT>(x + i)) * d.scale, bits, d.thr);
            if constexpr (RES) v += widen<TT>(ld8<TT>(res + i));
            st8<TT>(out + i, narrow<TT>(v));
        } else {  // the last, short group, element by element
            const int m = int(numel - i);
            Raw8<TT> rx{}, rr{};
#pragma unroll
            for (int j = 0; j < 7; ++j) {
                if (j >= m) continue;
                reinterpret_cast<S*>(&rx)[j] = x[i + j];
                if constexpr (RES) reinterpret_cast<S*>(&rr)[j] = res[i + j];
            }
            f32x8_t v = drop8(widen<TT>(rx) * d.scale, bits, d.thr);
            if constexpr (RES) v += widen<TT>(rr);
            const Raw8<TT> ro = narrow<TT>(v);
#pragma unroll
            for (int j = 0; j < 7; ++j)
                if (j < m) out[i + j] = reinterpret_cast<const S*>(&ro)[j];
        }
    }
}

template <typename TT>
spc_status launch(const void* x, const void* res, int64_t numel, const Drop& d, void* out, hipStream_t stream) {
    const int64_t blocks = ceil_div(ceil_div(numel, 8), DT);
    const unsigned grid = unsigned(blocks < 65536 * 4 ? blocks : 65536 * 4);
    if (res)
        hipLaunchKernelGGL((k_dropout<TT, true>), dim3(grid), dim3(DT), 0, stream, x, res, numel, d, out);
    else
        hipLaunchKernelGGL((k_dropout<TT, false>), dim3(grid), dim3(DT), 0, stream, x, res, numel, d, out);
    SPC_LAUNCHED("k_dropout");
    return SPC_OK;
}

spc_status dropout(spc_dtype dtype, const void* x, int64_t numel, const void* res, const spc_dropout* drop, void* out,
                   hipStream_t stream) {
    if (dtype != SPC_F32 && dtype != SPC_F16 && dtype != SPC_BF16) return fail(SPC_ERR_ARG, "unknown dtype %d", int(dtype));
    if (numel < 0) return fail(SPC_ERR_ARG, "numel=%lld is negative", (long long)numel);
    if (!drop) return fail(SPC_ERR_ARG, "drop is NULL");
    Drop d;
    const spc_status st = make_drop(drop, d);
    if (st != SPC_OK) return st;
    if (numel == 0) return SPC_OK;
    if (!x || !out) return fail(SPC_ERR_ARG, "input or output is NULL");
    for (const void* p : {x, res, (const void*)out})
        if (p && !aligned16(p)) return fail(SPC_ERR_ARG, "device pointers must be 16-byte aligned");
    switch (dtype) {
        case SPC_F32: return launch<F32>(x, res, numel, d, out, stream);
        case SPC_F16: return launch<F16>(x, res, numel, d, out, stream);
        case SPC_BF16: return launch<BF16>(x, res, numel, d, out, stream);
    }
    return fail(SPC_ERR_ARG, "unknown dtype %d", int(dtype));
}

}  // namespace
}  // namespace spc

using namespace spc;

extern "C" spc_status spc_dropout_fwd(spc_dtype dtype, const void* x, int64_t numel, const void* residual,
                                      const spc_dropout* drop, void* out, hipStream_t stream) {
    clear_error();
    return dropout(dtype, x, numel, residual, drop, out, stream);
}

extern "C" spc_status spc_dropout_bwd(spc_dtype dtype, const void* dout, int64_t numel, const spc_dropout* drop,
                                      void* din, hipStream_t stream) {
    clear_error();
    return dropout(dtype, dout, numel, nullptr, drop, din, stream);
}
