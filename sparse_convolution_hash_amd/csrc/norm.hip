// Group norm with an activation (and optional dropout) on channels-last
// features with ragged samples.  Per sample s and group of C / G channels:
//   mean, var over the sample's rows and the group's channels
//   xhat = (x - mean) * rstd,  rstd = (var + eps)^-1/2,  z = gamma * xhat + beta
//   y = dropout(act(z))
// and backward, with dz = act'(z) * dropout'(dy):
//   dbeta = sum dz,  dgamma = sum dz * xhat  (over all rows of all samples)
//   dx = rstd * (gamma dz - mean_g(gamma dz) - xhat * mean_g(gamma dz xhat))
//
// Rows are cut into tiles of R rows; a tile's rows of one sample are a run.
// Run (tile t, sample s) owns slot t + s: t and s never fall from one run to
// the next and one of them rises, so slots are distinct, there are at most
// tiles + samples of them, and a sample's runs lie side by side.  Three
// launches each way: per-channel sums of every run, their reduction to group
// (and channel) values, the elementwise pass.  All sums are fp32 within a run
// and double across runs, in a fixed order (no atomics).
#include "rows.h"

namespace spc {
namespace {

constexpr int NT = 256;   // threads per workgroup
constexpr int CPR = 8;    // threads per row: 8 x 8 = 64 channels per workgroup
constexpr int RL = NT / CPR;  // rows in flight per workgroup step
constexpr int R = 128;    // rows per tile

struct NormArgs {
    Segs segs;
    int32_t C, G;
    float eps;
    Drop drop;
};

// v summed over the lanes of a wave that share threadIdx.x % CPR.
__device__ __forceinline__ float sum_rows(float v) {
#pragma unroll
    for (int o = CPR; o < WAVE; o <<= 1) v += __shfl_xor(v, o);
    return v;
}

// Sums over the rows of a workgroup of two 8-channel values per thread; the
// result is valid in the threads of the first row (threadIdx.x < CPR).
__device__ __forceinline__ void reduce_rows(f32x8_t& a, f32x8_t& b, float (*lds)[CPR][16]) {
    const int oct = threadIdx.x % CPR, wave = threadIdx.x / WAVE;
#pragma unroll
    for (int j = 0; j < 8; ++j) a[j] = sum_rows(a[j]), b[j] = sum_rows(b[j]);
    if (threadIdx.x % WAVE < CPR)
#pragma unroll
        for (int j = 0; j < 8; ++j) lds[wave][oct][j] = a[j], lds[wave][oct][8 + j] = b[j];
    __syncthreads();
    if (threadIdx.x < CPR)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            a[j] = lds[0][oct][j], b[j] = lds[0][oct][8 + j];
#pragma unroll
            for (int w = 1; w < NT / WAVE; ++w) a[j] += lds[w][oct][j], b[j] += lds[w][oct][8 + j];
        }
    __syncthreads();
}

// Calls f(sample, first row, end row) for every run of tile t.
template <typename F>
__device__ __forceinline__ void for_runs(const Segs& g, int t, F f) {
    const int r0 = t * R, r1 = r0 + R < g.n ? r0 + R : g.n;
    for (int s = g.find(r0); s < g.n_seg; ++s) {
        int a = g.at(s), b = g.at(s + 1);
        if (a >= r1) break;
        a = a > r0 ? a : r0;
        b = b < r1 ? b : r1;
        if (a < b) f(s, a, b);
    }
}

// Mean and sum of squared differences of every run, per channel.  The sums
// are taken of differences from the run's first row, which lies within the
// data: sum (x - k)^2 is then at most rows + 1 times the spread around the
// mean, and the subtraction below costs at most that factor in precision.
template <typename TT>
__global__ __launch_bounds__(NT) void k_norm_stats(const void* __restrict__ x_, NormArgs p, float2* __restrict__ part) {
    using S = typename TT::storage;
    __shared__ float lds[NT / WAVE][CPR][16];
    const S* x = static_cast<const S*>(x_);
    const int oct = blockIdx.y * CPR + threadIdx.x % CPR, rl = threadIdx.x / CPR;
    const bool on = oct * 8 < p.C;
    const int ch = on ? oct * 8 : 0;
    for_runs(p.segs, blockIdx.x, [&](int s, int a, int b) {
        const f32x8_t k = widen<TT>(ld8<TT>(x + int64_t(a) * p.C + ch));
        f32x8_t s1 = 0.f, s2 = 0.f;
        for (int r = a + rl; r < b; r += RL) {
            const f32x8_t d = widen<TT>(ld8<TT>(x + int64_t(r) * p.C + ch)) - k;
            s1 += d;
            s2 += d * d;
        }
        reduce_rows(s1, s2, lds);
        if (rl == 0 && on) {
            float2* o = part + int64_t(blockIdx.x + s) * p.C + ch;
            const float inv = 1.f / float(b - a);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float m = s1[j] * inv, m2 = s2[j] - s1[j] * m;
                o[j] = float2{k[j] + m, m2 > 0.f || m2 != m2 ? m2 : 0.f};
            }
        }
    });
}

// Sum of a double over a workgroup, in every thread.
__device__ __forceinline__ double sum_block(double v, double* lds) {
#pragma unroll
    for (int o = 1; o < WAVE; o <<= 1) v += __shfl_xor(v, o);
    if (threadIdx.x % WAVE == 0) lds[threadIdx.x / WAVE] = v;
    __syncthreads();
    double t = lds[0];
#pragma unroll
    for (int w = 1; w < NT / WAVE; ++w) t += lds[w];
    __syncthreads();
    return t;
}

// Calls f(slot, rows, channel) for the runs and channels of (sample, group).
template <typename F>
__device__ __forceinline__ void for_parts(const NormArgs& p, int s, int g, F f) {
    const int a = p.segs.at(s), b = p.segs.at(s + 1), cg = p.C / p.G;
    if (a >= b) return;
    const int t0 = a / R, nt = (b - 1) / R - t0 + 1;
    for (int64_t i = threadIdx.x; i < int64_t(nt) * cg; i += NT) {
        const int q = int(i / cg), t = t0 + q;
        const int ra = a > t * R ? a : t * R, rb = b < (t + 1) * R ? b : (t + 1) * R;
        f(int64_t(t) + s, rb - ra, g * cg + int(i - int64_t(q) * cg));
    }
}

// Group mean and reciprocal deviation from the runs' means and spreads; an
// empty sample gets mean 0 and variance 0.
__global__ __launch_bounds__(NT) void k_norm_group(NormArgs p, const float2* __restrict__ part, float2* __restrict__ stats) {
    __shared__ double lds[NT / WAVE];
    const int s = blockIdx.x, g = blockIdx.y;
    double sum = 0, cnt = 0;
    for_parts(p, s, g, [&](int64_t slot, int rows, int c) {
        sum += double(rows) * part[slot * p.C + c].x;
        cnt += rows;
    });
    sum = sum_block(sum, lds);
    cnt = sum_block(cnt, lds);
    const double mean = cnt > 0 ? sum / cnt : 0.0;
    double m2 = 0;
    for_parts(p, s, g, [&](int64_t slot, int rows, int c) {
        const float2 v = part[slot * p.C + c];
        const double d = double(v.x) - mean;
        m2 += double(v.y) + double(rows) * d * d;
    });
    m2 = sum_block(m2, lds);
    if (threadIdx.x == 0)
        stats[int64_t(s) * p.G + g] = float2{float(mean), float(1.0 / sqrt((cnt > 0 ? m2 / cnt : 0.0) + double(p.eps)))};
}

// act(z), and act'(z) in the second form.
__device__ __forceinline__ float act_f(float z, int act) {
    if (act == SPC_ACT_RELU) return z < 0.f ? 0.f : z;
    if (act == SPC_ACT_SILU) return z / (1.f + __expf(-z));
    return z;
}
__device__ __forceinline__ float act_d(float z, int act) {
    if (act == SPC_ACT_RELU) return z > 0.f ? 1.f : 0.f;
    if (act == SPC_ACT_SILU) {
        const float s = 1.f / (1.f + __expf(-z));
        return s * (1.f + z * (1.f - s));
    }
    return 1.f;
}

// One run's constants of a thread's eight channels.
struct Chan8 {
    f32x8_t mean, rstd, gamma, beta;
    __device__ __forceinline__ void affine(const float* g, const float* b, int ch) {
#pragma unroll
        for (int j = 0; j < 8; ++j) gamma[j] = g ? g[ch + j] : 1.f, beta[j] = b ? b[ch + j] : 0.f;
    }
    __device__ __forceinline__ void stats(const float2* st, int s, int G, int cg, int ch) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float2 v = st[int64_t(s) * G + (ch + j) / cg];
            mean[j] = v.x, rstd[j] = v.y;
        }
    }
};

template <typename TT>
__global__ __launch_bounds__(NT) void k_norm_apply(const void* x_, NormArgs p, const float* __restrict__ gamma,
                                                   const float* __restrict__ beta, const float2* __restrict__ stats, int act,
                                                   void* y_) {
    using S = typename TT::storage;
    const S* x = static_cast<const S*>(x_);
    S* y = static_cast<S*>(y_);
    const int oct = blockIdx.y * CPR + threadIdx.x % CPR, rl = threadIdx.x / CPR;
    const bool on = oct * 8 < p.C;
    const int ch = on ? oct * 8 : 0;
    const uint64_t seed = p.drop.rng ? p.drop.rng[0] : 0, offset = p.drop.rng ? p.drop.rng[1] : 0;
    Chan8 c;
    c.affine(gamma, beta, ch);
    for_runs(p.segs, blockIdx.x, [&](int s, int a, int b) {
        c.stats(stats, s, p.G, p.C / p.G, ch);
        for (int r = a + rl; r < b && on; r += RL) {
            const int64_t i = int64_t(r) * p.C + ch;
            f32x8_t z = (widen<TT>(ld8<TT>(x + i)) - c.mean) * c.rstd * c.gamma + c.beta;
#pragma unroll
            for (int j = 0; j < 8; ++j) z[j] = act_f(z[j], act);
            if (p.drop.rng) z = drop8(z, philox(seed, offset + uint64_t(i / 8), p.drop.layer), p.drop.thr, p.drop.scale);
            st8<TT>(y + i, narrow<TT>(z));
        }
    });
}

// xhat and dz of eight elements.
template <typename TT>
__device__ __forceinline__ void grad8(const void* x, const void* dy, const Chan8& c, const NormArgs& p, uint64_t seed,
                                      uint64_t offset, int64_t i, int act, f32x8_t& xhat, f32x8_t& dz) {
    using S = typename TT::storage;
    xhat = (widen<TT>(ld8<TT>(static_cast<const S*>(x) + i)) - c.mean) * c.rstd;
    dz = widen<TT>(ld8<TT>(static_cast<const S*>(dy) + i));
    if (p.drop.rng) dz = drop8(dz, philox(seed, offset + uint64_t(i / 8), p.drop.layer), p.drop.thr, p.drop.scale);
    const f32x8_t z = xhat * c.gamma + c.beta;
#pragma unroll
    for (int j = 0; j < 8; ++j) dz[j] *= act_d(z[j], act);
}

// Sums of dz and dz * xhat of every run, per channel.
template <typename TT>
__global__ __launch_bounds__(NT) void k_norm_bwd_sums(const void* __restrict__ x, const void* __restrict__ dy, NormArgs p,
                                                      const float* __restrict__ gamma, const float* __restrict__ beta,
                                                      const float2* __restrict__ stats, int act, float2* __restrict__ part) {
    __shared__ float lds[NT / WAVE][CPR][16];
    const int oct = blockIdx.y * CPR + threadIdx.x % CPR, rl = threadIdx.x / CPR;
    const bool on = oct * 8 < p.C;
    const int ch = on ? oct * 8 : 0;
    const uint64_t seed = p.drop.rng ? p.drop.rng[0] : 0, offset = p.drop.rng ? p.drop.rng[1] : 0;
    Chan8 c;
    c.affine(gamma, beta, ch);
    for_runs(p.segs, blockIdx.x, [&](int s, int a, int b) {
        c.stats(stats, s, p.G, p.C / p.G, ch);
        f32x8_t s1 = 0.f, s2 = 0.f;
        for (int r = a + rl; r < b; r += RL) {
            f32x8_t xhat, dz;
            grad8<TT>(x, dy, c, p, seed, offset, int64_t(r) * p.C + ch, act, xhat, dz);
            s1 += dz;
            s2 += dz * xhat;
        }
        reduce_rows(s1, s2, lds);
        if (rl == 0 && on) {
            float2* o = part + int64_t(blockIdx.x + s) * p.C + ch;
#pragma unroll
            for (int j = 0; j < 8; ++j) o[j] = float2{s1[j], s2[j]};
        }
    });
}

// Workgroups [0, samples * G): the group's means of gamma dz and gamma dz
// xhat.  Workgroups after them: one channel's dbeta and dgamma each.
__global__ __launch_bounds__(NT) void k_norm_bwd_group(NormArgs p, const float* __restrict__ gamma,
                                                       const float2* __restrict__ part, float2* __restrict__ means,
                                                       float* __restrict__ dgamma, float* __restrict__ dbeta) {
    __shared__ double lds[NT / WAVE];
    const int64_t groups = int64_t(p.segs.n_seg) * p.G;
    double a = 0, b = 0, cnt = 0;
    if (int64_t(blockIdx.x) < groups) {
        const int s = int(blockIdx.x / p.G), g = int(blockIdx.x % p.G);
        for_parts(p, s, g, [&](int64_t slot, int rows, int c) {
            const float2 v = part[slot * p.C + c];
            const double w = gamma ? gamma[c] : 1.f;
            a += w * v.x;
            b += w * v.y;
            cnt += rows;
        });
        a = sum_block(a, lds);
        b = sum_block(b, lds);
        cnt = sum_block(cnt, lds);
        if (threadIdx.x == 0) means[blockIdx.x] = cnt > 0 ? float2{float(a / cnt), float(b / cnt)} : float2{0.f, 0.f};
        return;
    }
    const int c = int(blockIdx.x - groups);
    for (int s = 0; s < p.segs.n_seg; ++s) {
        const int ra = p.segs.at(s), rb = p.segs.at(s + 1);
        if (ra >= rb) continue;
        for (int t = ra / R + int(threadIdx.x); t <= (rb - 1) / R; t += NT) {
            const float2 v = part[(int64_t(t) + s) * p.C + c];
            a += v.x;
            b += v.y;
        }
    }
    a = sum_block(a, lds);
    b = sum_block(b, lds);
    if (threadIdx.x == 0) {
        if (dbeta) dbeta[c] = float(a);
        if (dgamma) dgamma[c] = float(b);
    }
}

template <typename TT>
__global__ __launch_bounds__(NT) void k_norm_bwd_apply(const void* __restrict__ x, const void* dy, NormArgs p,
                                                       const float* __restrict__ gamma, const float* __restrict__ beta,
                                                       const float2* __restrict__ stats, const float2* __restrict__ means,
                                                       int act, void* dx_) {
    using S = typename TT::storage;
    S* dx = static_cast<S*>(dx_);
    const int oct = blockIdx.y * CPR + threadIdx.x % CPR, rl = threadIdx.x / CPR;
    const bool on = oct * 8 < p.C;
    const int ch = on ? oct * 8 : 0, cg = p.C / p.G;
    const uint64_t seed = p.drop.rng ? p.drop.rng[0] : 0, offset = p.drop.rng ? p.drop.rng[1] : 0;
    Chan8 c;
    c.affine(gamma, beta, ch);
    for_runs(p.segs, blockIdx.x, [&](int s, int a, int b) {
        c.stats(stats, s, p.G, cg, ch);
        f32x8_t m1, m2;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float2 v = means[int64_t(s) * p.G + (ch + j) / cg];
            m1[j] = v.x, m2[j] = v.y;
        }
        for (int r = a + rl; r < b && on; r += RL) {
            const int64_t i = int64_t(r) * p.C + ch;
            f32x8_t xhat, dz;
            grad8<TT>(x, dy, c, p, seed, offset, i, act, xhat, dz);
            st8<TT>(dx + i, narrow<TT>((dz * c.gamma - m1 - xhat * m2) * c.rstd));
        }
    });
}

struct NormWs {
    int64_t tiles, part, stats;  // counts: row tiles, float2 of the partial sums, float2 of the group values
    size_t bytes() const { return align_up(size_t(part) * 8, 256) + size_t(stats) * 8; }
};

spc_status check_sizes(int64_t n, int32_t C, int32_t G, int64_t n_seg, NormWs& w) {
    if (n < 0 || n >= (int64_t(1) << 31) - R) return fail(SPC_ERR_ARG, "n=%lld is out of range", (long long)n);
    if (n_seg < 1 || n_seg >= (int64_t(1) << 31) - 1) return fail(SPC_ERR_ARG, "n_seg=%lld is out of range", (long long)n_seg);
    if (C <= 0 || C % 16) return fail(SPC_ERR_UNSUPPORTED, "C=%d: channels must be a positive multiple of 16", C);
    if (G < 1 || C % G) return fail(SPC_ERR_ARG, "groups=%d does not divide C=%d", G, C);
    if (ceil_div(C, 64) > 65535 || G > 65535) return fail(SPC_ERR_UNSUPPORTED, "C=%d is beyond one launch", C);
    w.tiles = ceil_div(n, R);
    w.part = (w.tiles + n_seg) * C;
    w.stats = n_seg * G;
    if (w.stats + C >= (int64_t(1) << 31)) return fail(SPC_ERR_UNSUPPORTED, "%lld groups are beyond one launch", (long long)w.stats);
    return SPC_OK;
}

spc_status check_call(spc_dtype dtype, int64_t n, int32_t C, int32_t G, const int32_t* seg_ptr, int64_t n_seg, int32_t act,
                      const spc_dropout* drop, const void* ws, size_t ws_bytes, NormWs& w, NormArgs& p) {
    if (dtype != SPC_F32 && dtype != SPC_F16 && dtype != SPC_BF16) return fail(SPC_ERR_ARG, "unknown dtype %d", int(dtype));
    spc_status st = check_sizes(n, C, G, n_seg, w);
    if (st != SPC_OK) return st;
    if (act != SPC_ACT_NONE && act != SPC_ACT_RELU && act != SPC_ACT_SILU) return fail(SPC_ERR_ARG, "unknown activation %d", act);
    if (!seg_ptr && n_seg != 1) return fail(SPC_ERR_ARG, "seg_ptr is NULL with n_seg=%lld", (long long)n_seg);
    if (seg_ptr && !aligned16(seg_ptr)) return fail(SPC_ERR_ARG, "device pointers must be 16-byte aligned");
    if (!ws || !aligned16(ws)) return fail(SPC_ERR_ARG, "ws is NULL or not 16-byte aligned");
    if (ws_bytes < w.bytes()) return fail(SPC_ERR_WORKSPACE, "ws_bytes=%zu, need %zu", ws_bytes, w.bytes());
    p.segs = Segs{seg_ptr, int32_t(n_seg), int32_t(n)};
    p.C = C, p.G = G, p.eps = 0.f;
    return make_drop(drop, p.drop);
}

template <typename TT>
spc_status launch_fwd(const void* x, const NormArgs& p, const NormWs& w, const float* gamma, const float* beta, int act,
                      void* y, float2* stats, void* ws, hipStream_t stream) {
    float2* part = static_cast<float2*>(ws);
    const dim3 grid(unsigned(w.tiles), unsigned(ceil_div(p.C, 8 * CPR)));
    if (w.tiles) {
        hipLaunchKernelGGL(k_norm_stats<TT>, grid, dim3(NT), 0, stream, x, p, part);
        SPC_LAUNCHED("k_norm_stats");
    }
    hipLaunchKernelGGL(k_norm_group, dim3(unsigned(p.segs.n_seg), unsigned(p.G)), dim3(NT), 0, stream, p, part, stats);
    SPC_LAUNCHED("k_norm_group");
    if (w.tiles) {
        hipLaunchKernelGGL(k_norm_apply<TT>, grid, dim3(NT), 0, stream, x, p, gamma, beta, stats, act, y);
        SPC_LAUNCHED("k_norm_apply");
    }
    return SPC_OK;
}

template <typename TT>
spc_status launch_bwd(const void* dy, const void* x, const NormArgs& p, const NormWs& w, const float* gamma,
                      const float* beta, const float2* stats, int act, void* dx, float* dgamma, float* dbeta, void* ws,
                      hipStream_t stream) {
    float2* part = static_cast<float2*>(ws);
    float2* means = reinterpret_cast<float2*>(static_cast<char*>(ws) + align_up(size_t(w.part) * 8, 256));
    const dim3 grid(unsigned(w.tiles), unsigned(ceil_div(p.C, 8 * CPR)));
    if (w.tiles) {
        hipLaunchKernelGGL(k_norm_bwd_sums<TT>, grid, dim3(NT), 0, stream, x, dy, p, gamma, beta, stats, act, part);
        SPC_LAUNCHED("k_norm_bwd_sums");
    }
    const int64_t blocks = w.stats + (dgamma || dbeta ? p.C : 0);
    hipLaunchKernelGGL(k_norm_bwd_group, dim3(unsigned(blocks)), dim3(NT), 0, stream, p, gamma, part, means, dgamma, dbeta);
    SPC_LAUNCHED("k_norm_bwd_group");
    if (w.tiles) {
        hipLaunchKernelGGL(k_norm_bwd_apply<TT>, grid, dim3(NT), 0, stream, x, dy, p, gamma, beta, stats, means, act, dx);
        SPC_LAUNCHED("k_norm_bwd_apply");
    }
    return SPC_OK;
}

}  // namespace
}  // namespace spc

using namespace spc;

extern "C" spc_status spc_group_norm_workspace(int64_t n, int32_t C, int32_t groups, int64_t n_seg, size_t* bytes) {
    clear_error();
    if (!bytes) return fail(SPC_ERR_ARG, "bytes is NULL");
    NormWs w;
    const spc_status st = check_sizes(n, C, groups, n_seg, w);
    if (st == SPC_OK) *bytes = w.bytes();
    return st;
}

extern "C" spc_status spc_group_norm_fwd(spc_dtype dtype, const void* x, int64_t n, int32_t C, int32_t groups,
                                         const int32_t* seg_ptr, int64_t n_seg, const float* gamma, const float* beta,
                                         float eps, int32_t act, const spc_dropout* drop, void* y, float* stats, void* ws,
                                         size_t ws_bytes, hipStream_t stream) {
    clear_error();
    NormWs w;
    NormArgs p;
    const spc_status st = check_call(dtype, n, C, groups, seg_ptr, n_seg, act, drop, ws, ws_bytes, w, p);
    if (st != SPC_OK) return st;
    if (!(eps > 0.f)) return fail(SPC_ERR_ARG, "eps=%g must be positive", double(eps));
    if (!stats || (n > 0 && (!x || !y))) return fail(SPC_ERR_ARG, "x, y or stats is NULL");
    for (const void* q : {x, (const void*)gamma, (const void*)beta, (const void*)y, (const void*)stats})
        if (q && !aligned16(q)) return fail(SPC_ERR_ARG, "device pointers must be 16-byte aligned");
    p.eps = eps;
    float2* so = reinterpret_cast<float2*>(stats);
    switch (dtype) {
        case SPC_F32: return launch_fwd<F32>(x, p, w, gamma, beta, act, y, so, ws, stream);
        case SPC_F16: return launch_fwd<F16>(x, p, w, gamma, beta, act, y, so, ws, stream);
        case SPC_BF16: return launch_fwd<BF16>(x, p, w, gamma, beta, act, y, so, ws, stream);
    }
    return fail(SPC_ERR_ARG, "unknown dtype %d", int(dtype));
}

extern "C" spc_status spc_group_norm_bwd(spc_dtype dtype, const void* dout, const void* x, int64_t n, int32_t C,
                                         int32_t groups, const int32_t* seg_ptr, int64_t n_seg, const float* gamma,
                                         const float* beta, const float* stats, int32_t act, const spc_dropout* drop,
                                         void* dx, float* dgamma, float* dbeta, void* ws, size_t ws_bytes,
                                         hipStream_t stream) {
    clear_error();
    NormWs w;
    NormArgs p;
    const spc_status st = check_call(dtype, n, C, groups, seg_ptr, n_seg, act, drop, ws, ws_bytes, w, p);
    if (st != SPC_OK) return st;
    if (!stats || (n > 0 && (!dout || !x || !dx))) return fail(SPC_ERR_ARG, "dout, x, stats or dx is NULL");
    for (const void* q : {dout, x, (const void*)gamma, (const void*)beta, (const void*)stats, (const void*)dx,
                          (const void*)dgamma, (const void*)dbeta})
        if (q && !aligned16(q)) return fail(SPC_ERR_ARG, "device pointers must be 16-byte aligned");
    const float2* si = reinterpret_cast<const float2*>(stats);
    switch (dtype) {
        case SPC_F32: return launch_bwd<F32>(dout, x, p, w, gamma, beta, si, act, dx, dgamma, dbeta, ws, stream);
        case SPC_F16: return launch_bwd<F16>(dout, x, p, w, gamma, beta, si, act, dx, dgamma, dbeta, ws, stream);
        case SPC_BF16: return launch_bwd<BF16>(dout, x, p, w, gamma, beta, si, act, dx, dgamma, dbeta, ws, stream);
    }
    return fail(SPC_ERR_ARG, "unknown dtype %d", int(dtype));
}
