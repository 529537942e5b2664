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
// (and channel) values, the elementwise pass.  A thread's sums are fp32, over
// at most 16 rows; all above are double, in a fixed order (no atomics), with one
// rounding to fp32 where a run's pair is stored for the next launch (half the
// bytes; it is off by half a unit, next to a thread's 16 roundings).
//
// What bounds it: x is read twice forward, x and dy twice backward, the second
// time mostly from the 256 MB cache, so on 266,426 x 128 bf16 (68 MB a tensor)
// the passes over memory would take 14 + 22 and 27 + 35 us.  Statistics: 14 us
// (4.9 TB/s).  The other three are held by the vector units next to that:
// with silu and dropout an element costs 20 to 28 instructions, a third of them
// the generator's, which each pass draws anew: 27 us (apply), 35 (sums), 38
// (backward apply).  Forward and backward with all launches: 135 us.
#include "rows.h"

namespace spc {
namespace {

constexpr int NT = 256;      // threads per workgroup
constexpr int OPR = 8;       // most lanes (of 8 channels) per row: slabs of up to 64 channels
constexpr int U = 4;         // rows that a thread loads at a time (2: 120,000 x 64 fp16 forward 22 -> 28 us)

// How [n, C] is cut: slabs of CW channels, CPR lanes to a row, RL rows side by
// side, tiles of R rows.  Workgroup y of Y takes every Y-th run of its tile.
struct Cut {
    int32_t nslab, CPR, CW, RL, R;
    int32_t tiles, Y;
    unsigned blocks() const { return unsigned(tiles) * unsigned(Y) * unsigned(nslab); }
};

inline Cut cut_of(int64_t n, int32_t C, int64_t n_seg) {
    Cut k;
    k.nslab = int32_t(ceil_div(C / 8, OPR));
    k.CPR = int32_t(ceil_div(C / 8, k.nslab));
    k.CW = 8 * k.CPR;
    k.RL = NT / k.CPR;
    // the longest tiles that still give every CU 8 workgroups (266,426 x 128 both
    // ways: 145 us; with 4 151, with 16 158)
    k.R = k.RL * U;
    while (k.R < k.RL * U * 4 && ceil_div(n, 2 * k.R) * k.nslab >= 8 * 256) k.R *= 2;
    k.tiles = int32_t(ceil_div(n, k.R));
    // a run takes a round trip to memory and three barriers, 2 us: two go side by
    // side where CUs are idle (20,011 x 48 fp32 in 37 samples, both ways: 42 -> 37 us
    // with Y = 2, 37 with 4, 47 with 8, whose workgroups mostly find nothing to do)
    k.Y = n_seg > 1 && int64_t(k.tiles) * k.nslab <= 2 * 256 ? 2 : 1;
    return k;
}

struct NormArgs {
    Segs segs;
    int32_t C, G;
    float eps;
    Drop drop;
    Cut k;
};

// A thread's place: 8 channels from ch, rows rl, rl + RL, ... of a run.
struct Place {
    int tile, y, slab, rl, ch, c;   // c: ch within the slab
    bool on;
    __device__ __forceinline__ explicit Place(const NormArgs& p) {
        tile = int(blockIdx.x) / p.k.nslab;
        slab = int(blockIdx.x) - tile * p.k.nslab;
        y = tile % p.k.Y;
        tile /= p.k.Y;
        rl = int(threadIdx.x) / p.k.CPR;
        c = (int(threadIdx.x) - rl * p.k.CPR) * 8;
        ch = slab * p.k.CW + c;
        on = rl < p.k.RL && ch < p.C;
        if (!on) ch = 0;
    }
};

// Calls f(sample, first row, end row) for the workgroup's runs.  Lane i of
// every wave reads the offset of sample s0 + i: one load, with up to 62
// samples, instead of a search and a walk.
template <typename F>
__device__ __forceinline__ void for_runs(const NormArgs& p, const Place& q, F f) {
    const Segs& g = p.segs;
    const int r0 = q.tile * p.k.R, r1 = p.k.R < g.n - r0 ? r0 + p.k.R : g.n;
    int s = g.n_seg < WAVE - 1 ? 0 : g.find(r0), turn = 0;
    while (s < g.n_seg) {
        const int i = s + int(threadIdx.x) % WAVE;
        const int off = g.at(i < g.n_seg ? i : g.n_seg);
        // the first sample that reaches past r0
        const uint64_t ends = __ballot(off > r0) >> 1;
        const int skip = ends ? __builtin_ctzll(ends) : WAVE - 1;
        s += skip;
        for (int j = skip; j < WAVE - 1 && s < g.n_seg; ++j, ++s) {
            int a = __builtin_amdgcn_readlane(off, j), b = __builtin_amdgcn_readlane(off, j + 1);
            if (a >= r1) return;
            a = a > r0 ? a : r0;
            b = b < r1 ? b : r1;
            if (a >= b) continue;
            if (turn == q.y) f(s, a, b);
            turn = turn + 1 == p.k.Y ? 0 : turn + 1;
        }
    }
}

// Sums in double over the RL rows of a workgroup of THREADS of two values per channel
// (of CW, a thread's eight from c): f(channel, sum of a, sum of b) in one
// thread per channel, side by side over the first CW threads.
template <int THREADS, typename F>
__device__ __forceinline__ void reduce_rows(int CW, int RL, int rl, int c8, const f32x8_t& a, const f32x8_t& b, float2* lds, double2* part,
                                            F f) {
    const int parts = THREADS / CW, per = (RL + parts - 1) / parts;   // 8 or 9 rows
    if (rl < RL) {
        f32x4_t* o = reinterpret_cast<f32x4_t*>(lds + rl * CW + c8);
#pragma unroll
        for (int j = 0; j < 4; ++j) o[j] = f32x4_t{a[2 * j], b[2 * j], a[2 * j + 1], b[2 * j + 1]};
    }
    __syncthreads();
    const int i = int(threadIdx.x) / CW, c = int(threadIdx.x) - i * CW;
    if (i < parts) {
        double2 t{0., 0.};
        const int end = (i + 1) * per < RL ? (i + 1) * per : RL;
#pragma unroll 8
        for (int r = i * per; r < end; ++r) t.x += lds[r * CW + c].x, t.y += lds[r * CW + c].y;
        part[i * CW + c] = t;
    }
    __syncthreads();
    if (i == 0) {
        double2 t{0., 0.};
#pragma unroll 8
        for (int r = 0; r < parts; ++r) t.x += part[r * CW + c].x, t.y += part[r * CW + c].y;
        f(c, t.x, t.y);
    }
    __syncthreads();
}

// A value within rows [a, b) for sums of differences and their squares, per
// channel: the median of the first, the middle and the last row.  The roundings of
// (x - k)^2 count by 1 + (k - mean)^2 / variance, about twice for any ordinary
// row; one far from all others would make it the count of rows (first tokens and
// borders often are: on 1,000 constant rows after such a one the variance was off
// by 430 units of 2^-24, with the median it is within 6), and the median takes it only
// if two of the three are.  Each run or sample takes one: two loads more, side by side.
template <typename TT>
__device__ __forceinline__ f32x8_t middle_of(const typename TT::storage* x, int a, int b, const NormArgs& p, int ch) {
    const f32x8_t u = widen<TT>(ld8<TT>(x + int64_t(a) * p.C + ch)), v = widen<TT>(ld8<TT>(x + int64_t(a + (b - a) / 2) * p.C + ch)),
                  w = widen<TT>(ld8<TT>(x + int64_t(b - 1) * p.C + ch));
    f32x8_t k;
#pragma unroll
    for (int j = 0; j < 8; ++j) k[j] = __builtin_amdgcn_fmed3f(u[j], v[j], w[j]);
    return k;
}

// Mean and sum of squared differences of every run, per channel.
template <typename TT>
__global__ __launch_bounds__(NT) void k_norm_stats(const void* __restrict__ x_, NormArgs p, float2* __restrict__ part) {
    using S = typename TT::storage;
    __shared__ float2 lds[NT * 8];
    __shared__ double2 sums[NT];
    __shared__ float base[8 * OPR];
    const S* x = static_cast<const S*>(x_);
    const Place q(p);
    for_runs(p, q, [&](int s, int a, int b) {
        const f32x8_t k = middle_of<TT>(x, a, b, p, q.ch);
        if (q.rl == 0)
#pragma unroll
            for (int j = 0; j < 8; ++j) base[q.c + j] = k[j];
        f32x8_t s1 = 0.f, s2 = 0.f;
        for (int r = a + q.rl; r < b && q.on; r += p.k.RL * U) {
            Raw8<TT> v[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {   // beyond the end: the last row once more, not counted
                const int ru = r + u * p.k.RL;
                v[u] = ld8<TT>(x + int64_t(ru < b ? ru : b - 1) * p.C + q.ch);
            }
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (r + u * p.k.RL < b) {
                    const f32x8_t d = widen<TT>(v[u]) - k;
                    s1 += d;
                    s2 += d * d;
                }
        }
        reduce_rows<NT>(p.k.CW, p.k.RL, q.rl, q.c, s1, s2, lds, sums, [&](int c, double t1, double t2) {
            if (q.slab * p.k.CW + c >= p.C) return;
            // in double: t1 m is (base - mean)^2 / variance times what is left of t2
            const double m = t1 / double(b - a), m2 = t2 - t1 * m;
            part[int64_t(q.tile + s) * p.C + q.slab * p.k.CW + c] = float2{float(double(base[c]) + m), m2 > 0. || m2 != m2 ? float(m2) : 0.f};
        });
    });
}

// Sums of two doubles over a workgroup, in every thread.
constexpr int NG = 512;   // threads of the reductions across runs
__device__ __forceinline__ void sum_block(double& a, double& b, double2* lds) {
#pragma unroll
    for (int o = 1; o < WAVE; o <<= 1) a += __shfl_xor(a, o), b += __shfl_xor(b, o);
    if (threadIdx.x % WAVE == 0) lds[threadIdx.x / WAVE] = double2{a, b};
    __syncthreads();
    a = lds[0].x, b = lds[0].y;
#pragma unroll
    for (int w = 1; w < NG / WAVE; ++w) a += lds[w].x, b += lds[w].y;
}

// Calls f(slot, rows, channel) for the runs and channels of (sample, group),
// a workgroup's threads side by side over the channels, then over the runs.
template <typename F>
__device__ __forceinline__ void for_parts(const NormArgs& p, int s, int g, F f) {
    const int a = p.segs.at(s), b = p.segs.at(s + 1), cg = p.C / p.G, R = p.k.R;
    if (a >= b) return;
    const int w = cg < NG ? cg : NG, i = int(threadIdx.x) / w, step = NG / w;
    if (i >= step) return;
    for (int c = int(threadIdx.x) - i * w; c < cg; c += w)
        for (int t = a / R + i; t <= (b - 1) / R; t += step) {
            const int ra = a > t * R ? a : t * R, rb = b - t * R < R ? b : (t + 1) * R;
            f(int64_t(t) + s, rb - ra, g * cg + c);
        }
}

// The reductions across runs take a workgroup for each of `jobs` things, up to
// a grid that one launch holds; beyond it the workgroups go round again.
constexpr unsigned JOBS = unsigned(((int64_t(1) << 32) - 1) / NG / 2);
inline dim3 job_grid(int64_t jobs) { return dim3(jobs < JOBS ? unsigned(jobs) : JOBS); }
template <typename F>
__device__ __forceinline__ void for_jobs(unsigned jobs, F f) {
    for (unsigned i = blockIdx.x; i < jobs; i += gridDim.x) {
        f(i);
        __syncthreads();   // the LDS is free again
    }
}

// Group mean and reciprocal deviation from the runs' means and spreads, whose
// squares are taken around the first of the means; an empty sample gets mean 0
// and variance 0.
__global__ __launch_bounds__(NG) void k_norm_group(NormArgs p, unsigned groups, const float2* __restrict__ part, float2* __restrict__ stats) {
    __shared__ double2 lds[NG / WAVE];
    for_jobs(groups, [&](unsigned job) {
        const int s = int(job / p.G), g = int(job % p.G);
        const int a = p.segs.at(s), b = p.segs.at(s + 1);
        double mean = 0, var = 0;
        if (a < b) {
            const double k = part[(int64_t(a / p.k.R) + s) * p.C + g * (p.C / p.G)].x;
            double s1 = 0, s2 = 0;
            for_parts(p, s, g, [&](int64_t slot, int rows, int c) {
                const float2 v = part[slot * p.C + c];
                const double d = double(v.x) - k;
                s1 += double(rows) * d;
                s2 += double(v.y) + double(rows) * d * d;
            });
            sum_block(s1, s2, lds);
            const double cnt = double(b - a) * (p.C / p.G), m = s1 / cnt;
            mean = k + m;
            var = s2 / cnt - m * m;
            var = var > 0 || var != var ? var : 0;
        }
        if (threadIdx.x == 0) stats[job] = float2{float(mean), float(1.0 / sqrt(var + double(p.eps)))};
    });
}

// v sigmoid(z), v = 1 / inv.  Rounding log2(e) z and its constant moves it by up to
// 1.23 |z| 2^-24 of its value where z is far below 0, which in z sigmoid(z) is
// never above 2^-24.  It is not corrected: these kernels are held by the vector units.
__device__ __forceinline__ float sigmoid(float z, float inv) {
    const float e = __builtin_amdgcn_exp2f(-1.44269504f * z);
    return __builtin_amdgcn_rcpf(fmaf(e, inv, inv));
}
// act(z) / inv of an activation that scales with its argument (z comes
// multiplied) or of silu, and act'(z) in the second form.
template <int ACT>
__device__ __forceinline__ float act_f(float z, float inv) {
    if (ACT == SPC_ACT_RELU) return z < 0.f ? 0.f : z;
    if (ACT == SPC_ACT_SILU) return z * sigmoid(z, inv);
    return z;
}
template <int ACT>
__device__ __forceinline__ float act_d(float z) {
    if (ACT == SPC_ACT_RELU) return z > 0.f ? 1.f : 0.f;
    if (ACT == SPC_ACT_SILU) {
        const float s = sigmoid(z, 1.f);
        return s * fmaf(z, 1.f - s, 1.f);
    }
    return 1.f;
}

// The constants of a thread's eight channels: a run's mean and rstd (of the
// channel's group), and z = scale (x - mean) + beta.
struct Chan8 {
    f32x8_t gamma, beta, mean, rstd, scale;
    int cg, g0, first;   // channels per group, the first channel's group, and its place there
    __device__ __forceinline__ Chan8(const NormArgs& p, const float* g, const float* b, int ch) {
        gamma = 1.f, beta = 0.f;
        if (g) gamma = widen<F32>(ld8<F32>(g + ch));
        if (b) beta = widen<F32>(ld8<F32>(b + ch));
        cg = p.C / p.G;
        g0 = ch / cg;
        first = ch - g0 * cg;
    }
    // v[j] = the pair of channel j's group
    template <typename F>
    __device__ __forceinline__ void groups(const float2* row, F f) const {
        if (cg % 8 == 0) {
            const float2 v = row[g0];
#pragma unroll
            for (int j = 0; j < 8; ++j) f(j, v);
        } else {
            int g = g0, i = first;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                f(j, row[g]);
                if (++i == cg) i = 0, ++g;
            }
        }
    }
    __device__ __forceinline__ void run(const float2* stats, int s, int G) {
        groups(stats + int64_t(s) * G, [&](int j, const float2& v) { mean[j] = v.x, rstd[j] = v.y, scale[j] = v.y * gamma[j]; });
    }
};

template <typename TT, int ACT, bool DROP>
__global__ __launch_bounds__(NT) void k_norm_apply(const void* x_, NormArgs p, const float* __restrict__ gamma,
                                                   const float* __restrict__ beta, const float2* __restrict__ stats, void* y_) {
    using S = typename TT::storage;
    const S* x = static_cast<const S*>(x_);
    S* y = static_cast<S*>(y_);
    const Place q(p);
    const uint64_t seed = DROP ? p.drop.rng[0] : 0, offset = DROP ? p.drop.rng[1] : 0;
    Chan8 c(p, gamma, beta, q.ch);
    // dropout's factor goes into the affine step, silu's into its division
    if (DROP && ACT != SPC_ACT_SILU) c.gamma *= p.drop.scale, c.beta *= p.drop.scale;
    for_runs(p, q, [&](int s, int a, int b) {
        c.run(stats, s, p.G);
        for (int r = a + q.rl; r < b && q.on; r += p.k.RL * U) {
            Raw8<TT> v[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int ru = r + u * p.k.RL;
                v[u] = ld8<TT>(x + int64_t(ru < b ? ru : b - 1) * p.C + q.ch);
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int64_t i = int64_t(r + u * p.k.RL) * p.C + q.ch;
                if (r + u * p.k.RL >= b) break;
                f32x8_t z = widen<TT>(v[u]) - c.mean;
#pragma unroll
                for (int j = 0; j < 8; ++j) z[j] = act_f<ACT>(fmaf(z[j], c.scale[j], c.beta[j]), DROP ? p.drop.inv : 1.f);
                if (DROP) z = drop8(z, philox(seed, offset + uint64_t(i / 8), p.drop.layer), p.drop.thr);
                st8<TT>(y + i, narrow<TT>(z));
            }
        }
    });
}

// d = x - mean and dz / (dropout's factor) of eight elements.
template <typename TT, int ACT, bool DROP>
__device__ __forceinline__ void grad8(const Raw8<TT>& x, const Raw8<TT>& dy, const Chan8& c, const NormArgs& p, uint64_t seed,
                                      uint64_t offset, int64_t i, f32x8_t& d, f32x8_t& dz) {
    d = widen<TT>(x) - c.mean;
    dz = widen<TT>(dy);
    if (DROP) dz = drop8(dz, philox(seed, offset + uint64_t(i / 8), p.drop.layer), p.drop.thr);
#pragma unroll
    for (int j = 0; j < 8; ++j) dz[j] *= act_d<ACT>(fmaf(d[j], c.scale[j], c.beta[j]));
}

// Sums of dz and dz * xhat of every run, and (tot, NULL ok) of the workgroup's runs, per channel.
template <typename TT, int ACT, bool DROP>
__global__ __launch_bounds__(NT) void k_norm_bwd_sums(const void* __restrict__ x_, const void* __restrict__ dy_, NormArgs p,
                                                      const float* __restrict__ gamma, const float* __restrict__ beta,
                                                      const float2* __restrict__ stats, float2* __restrict__ part,
                                                      float2* __restrict__ tot) {
    using S = typename TT::storage;
    __shared__ float2 lds[NT * 8];
    __shared__ double2 sums[NT];
    const S *x = static_cast<const S*>(x_), *dy = static_cast<const S*>(dy_);
    const Place q(p);
    const uint64_t seed = DROP ? p.drop.rng[0] : 0, offset = DROP ? p.drop.rng[1] : 0;
    Chan8 c(p, gamma, beta, q.ch);
    double2 t{0., 0.};
    for_runs(p, q, [&](int s, int a, int b) {
        c.run(stats, s, p.G);
        f32x8_t s1 = 0.f, s2 = 0.f;
        for (int r = a + q.rl; r < b && q.on; r += p.k.RL * U) {
            Raw8<TT> v[U], w[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int ru = r + u * p.k.RL;
                const int64_t i = int64_t(ru < b ? ru : b - 1) * p.C + q.ch;
                v[u] = ld8<TT>(x + i);
                w[u] = ld8<TT>(dy + i);
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (r + u * p.k.RL >= b) break;
                f32x8_t d, dz;
                grad8<TT, ACT, DROP>(v[u], w[u], c, p, seed, offset, int64_t(r + u * p.k.RL) * p.C + q.ch, d, dz);
                s1 += dz;
                s2 += dz * d;
            }
        }
        s1 *= p.drop.scale;
        s2 *= c.rstd * p.drop.scale;
        reduce_rows<NT>(p.k.CW, p.k.RL, q.rl, q.c, s1, s2, lds, sums, [&](int k, double t1, double t2) {
            if (q.slab * p.k.CW + k >= p.C) return;
            part[int64_t(q.tile + s) * p.C + q.slab * p.k.CW + k] = float2{float(t1), float(t2)};
            t.x += t1, t.y += t2;
        });
    });
    if (tot && int(threadIdx.x) < p.k.CW && q.slab * p.k.CW + int(threadIdx.x) < p.C)
        tot[(int64_t(q.tile) * p.k.Y + q.y) * p.C + q.slab * p.k.CW + threadIdx.x] = float2{float(t.x), float(t.y)};
}

// Jobs [0, groups), groups = samples * G: the group's means of gamma dz and
// gamma dz xhat.  Jobs after them: dbeta and dgamma of 8 channels each, from
// ntot rows of tot.
__global__ __launch_bounds__(NG) void k_norm_bwd_group(NormArgs p, unsigned jobs, unsigned groups, const float* __restrict__ gamma,
                                                       const float2* __restrict__ part, const float2* __restrict__ tot,
                                                       int ntot, float2* __restrict__ means, float* __restrict__ dgamma,
                                                       float* __restrict__ dbeta) {
    __shared__ double2 lds[NG / WAVE];
    __shared__ double2 ch[NG / WAVE][8];
    for_jobs(jobs, [&](unsigned job) {
        double a = 0, b = 0;
        if (job < groups) {
            const int s = int(job / p.G), g = int(job % p.G);
            for_parts(p, s, g, [&](int64_t slot, int, int c) {
                const float2 v = part[slot * p.C + c];
                const double w = gamma ? gamma[c] : 1.f;
                a += w * v.x;
                b += w * v.y;
            });
            sum_block(a, b, lds);
            const double cnt = double(p.segs.at(s + 1) - p.segs.at(s)) * (p.C / p.G);
            if (threadIdx.x == 0) means[job] = cnt > 0 ? float2{float(a / cnt), float(b / cnt)} : float2{0.f, 0.f};
            return;
        }
        const int c = int(job - groups) * 8 + int(threadIdx.x) % 8;
#pragma unroll 4
        for (int t = int(threadIdx.x) / 8; t < ntot; t += NG / 8) {
            const float2 v = tot[int64_t(t) * p.C + c];
            a += v.x;
            b += v.y;
        }
        // 8 channels side by side: over the lanes 8 apart, then over the waves
#pragma unroll
        for (int o = 8; o < WAVE; o <<= 1) a += __shfl_xor(a, o), b += __shfl_xor(b, o);
        if (threadIdx.x % WAVE < 8) ch[threadIdx.x / WAVE][threadIdx.x % WAVE] = double2{a, b};
        __syncthreads();
        if (threadIdx.x < 8) {
            a = b = 0;
#pragma unroll
            for (int w = 0; w < NG / WAVE; ++w) a += ch[w][threadIdx.x].x, b += ch[w][threadIdx.x].y;
            if (dbeta) dbeta[c] = float(a);
            if (dgamma) dgamma[c] = float(b);
        }
    });
}

template <typename TT, int ACT, bool DROP>
__global__ __launch_bounds__(NT) void k_norm_bwd_apply(const void* __restrict__ x_, const void* dy_, NormArgs p,
                                                       const float* __restrict__ gamma, const float* __restrict__ beta,
                                                       const float2* __restrict__ stats, const float2* __restrict__ means,
                                                       void* dx_) {
    using S = typename TT::storage;
    const S *x = static_cast<const S*>(x_), *dy = static_cast<const S*>(dy_);
    S* dx = static_cast<S*>(dx_);
    const Place q(p);
    const uint64_t seed = DROP ? p.drop.rng[0] : 0, offset = DROP ? p.drop.rng[1] : 0;
    Chan8 c(p, gamma, beta, q.ch);
    for_runs(p, q, [&](int s, int a, int b) {
        c.run(stats, s, p.G);
        // dx = scale dz - (rstd m1 + rstd^2 m2 (x - mean))
        f32x8_t k1, k2;
        const f32x8_t k0 = c.scale * p.drop.scale;
        c.groups(means + int64_t(s) * p.G, [&](int j, const float2& v) { k1[j] = c.rstd[j] * v.x, k2[j] = c.rstd[j] * c.rstd[j] * v.y; });
        for (int r = a + q.rl; r < b && q.on; r += p.k.RL * U) {
            Raw8<TT> v[U], w[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int ru = r + u * p.k.RL;
                const int64_t i = int64_t(ru < b ? ru : b - 1) * p.C + q.ch;
                v[u] = ld8<TT>(x + i);
                w[u] = ld8<TT>(dy + i);
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (r + u * p.k.RL >= b) break;
                const int64_t i = int64_t(r + u * p.k.RL) * p.C + q.ch;
                f32x8_t d, dz;
                grad8<TT, ACT, DROP>(v[u], w[u], c, p, seed, offset, i, d, dz);
#pragma unroll
                for (int j = 0; j < 8; ++j) dz[j] = fmaf(k0[j], dz[j], -fmaf(k2[j], d[j], k1[j]));
                st8<TT>(dx + i, narrow<TT>(dz));
            }
        }
    });
}

// ------------------------------------------------------------ small inputs

// One launch (and one for dgamma and dbeta) does it all: a workgroup takes one
// sample and CW channels, the fewest that are whole groups and whole loads, and
// goes over its rows twice (the second time from the cache).  The three
// launches above take 11 us (backward 13 to 15) at the least; this takes 6 (6) for
// 500 elements of a workgroup, 7 (7 to 8) for 4,000, 7 to 13 (9 to 17) for 16,000
// (and 4 us of the host's time less), 15 to 34 (26 to 86) for 64,000.  Eight
// samples of 2,000 elements each: 7 (9).  So it takes
// calls with SMALL elements at most in the channels of a workgroup, or SMALL_MAX
// if the samples have SMALL_MEAN on average, whatever their lengths.
constexpr int NS = 512;
constexpr int64_t SMALL = 16384, SMALL_MEAN = 8192, SMALL_MAX = 32768;

inline int small_width(int32_t C, int32_t G) {
    int w = C / G;
    while (w % 8) w *= 2;
    return w;
}

// A thread's place in such a workgroup.
struct Corner {
    int s, a, b, CW, CPR, RL, rl, c, ch;
    bool on;
    __device__ __forceinline__ Corner(const NormArgs& p, int CW_) : CW(CW_) {
        const int n = p.C / CW;
        s = int(blockIdx.x) / n;
        a = p.segs.at(s), b = p.segs.at(s + 1);
        CPR = CW / 8;
        RL = NS / CPR;
        rl = int(threadIdx.x) / CPR;
        c = (int(threadIdx.x) - rl * CPR) * 8;
        on = rl < RL;
        ch = (int(blockIdx.x) - s * n) * CW + c;
    }
    __device__ __forceinline__ int c0() const { return ch - c; }
};

// Adds up v(channel) over each group of a workgroup's channels, one wave a
// group, in double: f(group in the workgroup, sums of the pair).
template <typename V, typename F>
__device__ __forceinline__ void sum_groups(int CW, int cg, V v, F f) {
    for (int g = int(threadIdx.x) / WAVE; g < CW / cg; g += NS / WAVE) {
        double a = 0, b = 0;
        for (int c = int(threadIdx.x) % WAVE; c < cg; c += WAVE) {
            const double2 t = v(g, g * cg + c);
            a += t.x, b += t.y;
        }
#pragma unroll
        for (int o = 1; o < WAVE; o <<= 1) a += __shfl_xor(a, o), b += __shfl_xor(b, o);
        if (threadIdx.x % WAVE == 0) f(g, a, b);
    }
    __syncthreads();
}

template <typename TT, int ACT, bool DROP>
__global__ __launch_bounds__(NS) void k_norm_small(const void* x_, NormArgs p, int CW, const float* __restrict__ gamma,
                                                   const float* __restrict__ beta, float2* __restrict__ stats, void* y_) {
    using S = typename TT::storage;
    __shared__ float2 lds[NS * 8];
    __shared__ double2 sums[NS], chan[NS];   // chan: a channel's sums around base
    __shared__ float base[NS];
    const S* x = static_cast<const S*>(x_);
    S* y = static_cast<S*>(y_);
    const Corner q(p, CW);
    const int cg = p.C / p.G, g0 = q.c0() / cg;
    float2* row = stats + int64_t(q.s) * p.G;
    if (q.a >= q.b) {
        for (int g = threadIdx.x; g < CW / cg; g += NS) row[g0 + g] = float2{0.f, float(1.0 / sqrt(double(p.eps)))};
        return;
    }
    const uint64_t seed = DROP ? p.drop.rng[0] : 0, offset = DROP ? p.drop.rng[1] : 0;
    Chan8 c(p, gamma, beta, q.ch);
    if (DROP && ACT != SPC_ACT_SILU) c.gamma *= p.drop.scale, c.beta *= p.drop.scale;
    const f32x8_t k = middle_of<TT>(x, q.a, q.b, p, q.ch);
    if (q.rl == 0)
#pragma unroll
        for (int j = 0; j < 8; ++j) base[q.c + j] = k[j];
    f32x8_t s1 = 0.f, s2 = 0.f;
#pragma unroll 4
    for (int r = q.a + q.rl; r < q.b && q.on; r += q.RL) {
        const f32x8_t d = widen<TT>(ld8<TT>(x + int64_t(r) * p.C + q.ch)) - k;
        s1 += d;
        s2 += d * d;
    }
    reduce_rows<NS>(CW, q.RL, q.rl, q.c, s1, s2, lds, sums, [&](int i, double t1, double t2) { chan[i] = double2{t1, t2}; });
    float2* const group = lds;   // free again
    // around the base of the group's first channel k: sum (x - k) and its square
    const double rows = double(q.b - q.a), cnt = rows * cg;
    sum_groups(CW, cg,
               [&](int g, int i) {
                   const double o = double(base[i]) - double(base[g * cg]), t1 = chan[i].x, t2 = chan[i].y;
                   return double2{t1 + rows * o, t2 + o * (2 * t1 + rows * o)};
               },
               [&](int g, double t1, double t2) {
                   const double m = t1 / cnt, v = t2 / cnt - m * m;
                   group[g] = float2{float(double(base[g * cg]) + m), float(1.0 / sqrt((v > 0 || v != v ? v : 0) + double(p.eps)))};
                   row[g0 + g] = group[g];
               });
    c.g0 -= g0;
    c.run(group, 0, 0);
#pragma unroll 4
    for (int r = q.a + q.rl; r < q.b && q.on; r += q.RL) {
        const int64_t i = int64_t(r) * p.C + q.ch;
        f32x8_t z = widen<TT>(ld8<TT>(x + i)) - c.mean;
#pragma unroll
        for (int j = 0; j < 8; ++j) z[j] = act_f<ACT>(fmaf(z[j], c.scale[j], c.beta[j]), DROP ? p.drop.inv : 1.f);
        if (DROP) z = drop8(z, philox(seed, offset + uint64_t(i / 8), p.drop.layer), p.drop.thr);
        st8<TT>(y + i, narrow<TT>(z));
    }
}

// tot (NULL ok): every sample's sums of dz and dz * xhat, per channel; dgamma
// and dbeta (NULL ok) directly, where there is one sample.
template <typename TT, int ACT, bool DROP>
__global__ __launch_bounds__(NS) void k_norm_bwd_small(const void* __restrict__ x_, const void* dy_, NormArgs p, int CW,
                                                       const float* __restrict__ gamma, const float* __restrict__ beta,
                                                       const float2* __restrict__ stats, float2* __restrict__ tot,
                                                       float* __restrict__ dgamma, float* __restrict__ dbeta, void* dx_) {
    using S = typename TT::storage;
    __shared__ float2 lds[NS * 8];
    __shared__ double2 sums[NS], chan[NS];
    const S *x = static_cast<const S*>(x_), *dy = static_cast<const S*>(dy_);
    S* dx = static_cast<S*>(dx_);
    const Corner q(p, CW);
    const int cg = p.C / p.G;
    if (q.a >= q.b) {
        for (int i = threadIdx.x; i < CW; i += NS) {
            if (tot) tot[int64_t(q.s) * p.C + q.c0() + i] = float2{0.f, 0.f};
            if (dgamma) dgamma[q.c0() + i] = 0.f;
            if (dbeta) dbeta[q.c0() + i] = 0.f;
        }
        return;
    }
    const uint64_t seed = DROP ? p.drop.rng[0] : 0, offset = DROP ? p.drop.rng[1] : 0;
    Chan8 c(p, gamma, beta, q.ch);
    c.run(stats, q.s, p.G);
    f32x8_t s1 = 0.f, s2 = 0.f;
#pragma unroll 2
    for (int r = q.a + q.rl; r < q.b && q.on; r += q.RL) {
        const int64_t i = int64_t(r) * p.C + q.ch;
        f32x8_t d, dz;
        grad8<TT, ACT, DROP>(ld8<TT>(x + i), ld8<TT>(dy + i), c, p, seed, offset, i, d, dz);
        s1 += dz;
        s2 += dz * d;
    }
    s1 *= p.drop.scale;
    s2 *= c.rstd * p.drop.scale;
    reduce_rows<NS>(CW, q.RL, q.rl, q.c, s1, s2, lds, sums, [&](int i, double t1, double t2) {
        chan[i] = double2{t1, t2};
        if (tot) tot[int64_t(q.s) * p.C + q.c0() + i] = float2{float(t1), float(t2)};
        if (dgamma) dgamma[q.c0() + i] = float(t2);
        if (dbeta) dbeta[q.c0() + i] = float(t1);
    });
    const double cnt = double(q.b - q.a) * cg;
    float2* const group = lds;   // free again
    const float* ga = gamma ? gamma + q.c0() : nullptr;
    sum_groups(CW, cg,
               [&](int, int i) {
                   const double w = ga ? ga[i] : 1.f;
                   return double2{w * chan[i].x, w * chan[i].y};
               },
               [&](int g, double t1, double t2) { group[g] = float2{float(t1 / cnt), float(t2 / cnt)}; });
    c.g0 -= q.c0() / cg;
    f32x8_t k1, k2;
    const f32x8_t k0 = c.scale * p.drop.scale;
    c.groups(group, [&](int j, const float2& v) { k1[j] = c.rstd[j] * v.x, k2[j] = c.rstd[j] * c.rstd[j] * v.y; });
#pragma unroll 2
    for (int r = q.a + q.rl; r < q.b && q.on; r += q.RL) {
        const int64_t i = int64_t(r) * p.C + q.ch;
        f32x8_t d, dz;
        grad8<TT, ACT, DROP>(ld8<TT>(x + i), ld8<TT>(dy + i), c, p, seed, offset, i, d, dz);
#pragma unroll
        for (int j = 0; j < 8; ++j) dz[j] = fmaf(k0[j], dz[j], -fmaf(k2[j], d[j], k1[j]));
        st8<TT>(dx + i, narrow<TT>(dz));
    }
}

struct NormWs {
    Cut k;
    int32_t CW;                // one launch does: its channels to a workgroup; 0: it does not
    int64_t part, tot, stats;  // counts of float2: the runs' sums, the workgroups' sums, the group values
    size_t bytes() const { return CW ? size_t(part) * 8 : align_up(size_t(part) * 8, 256) + align_up(size_t(tot) * 8, 256) + size_t(stats) * 8; }
    float2* tot_of(void* ws) const { return reinterpret_cast<float2*>(static_cast<char*>(ws) + align_up(size_t(part) * 8, 256)); }
    float2* means_of(void* ws) const {
        return reinterpret_cast<float2*>(reinterpret_cast<char*>(tot_of(ws)) + align_up(size_t(tot) * 8, 256));
    }
};

spc_status check_sizes(int64_t n, int32_t C, int32_t G, int64_t n_seg, NormWs& w) {
    if (n < 0 || n >= ROWS_END) return fail(SPC_ERR_ARG, "n=%lld is out of range", (long long)n);
    if (n_seg < 1 || n_seg >= ROWS_END) return fail(SPC_ERR_ARG, "n_seg=%lld is out of range", (long long)n_seg);
    if (C <= 0 || C % 16) return fail(SPC_ERR_UNSUPPORTED, "C=%d: channels must be a positive multiple of 16", C);
    if (G < 1 || C % G) return fail(SPC_ERR_ARG, "groups=%d does not divide C=%d", G, C);
    if (C > C_MAX) return fail(SPC_ERR_UNSUPPORTED, "C=%d: at most %d channels", C, C_MAX);
    w.k = cut_of(n, C, n_seg);
    w.part = (w.k.tiles + n_seg) * C;
    w.tot = int64_t(w.k.tiles) * w.k.Y * C;
    w.stats = n_seg * G;
    w.CW = small_width(C, G);
    const int64_t all = n * w.CW;
    if (!(w.CW <= NS && (all <= SMALL || (all <= SMALL_MAX && all <= SMALL_MEAN * n_seg)) && launchable(n_seg * (C / w.CW), NS))) w.CW = 0;
    if (w.CW) w.part = n_seg > 1 ? n_seg * C : 0, w.tot = 0;      // the samples' sums of the backward
    if (!launchable(int64_t(w.k.tiles) * w.k.Y * w.k.nslab, NT)) return fail(SPC_ERR_UNSUPPORTED, "%lld rows of %d channels exceed one launch", (long long)n, C);
    if (w.stats + C >= (int64_t(1) << 31)) return fail(SPC_ERR_UNSUPPORTED, "%lld groups are too many", (long long)w.stats);
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
    if ((!ws && w.bytes()) || !aligned16(ws)) return fail(SPC_ERR_ARG, "ws is NULL or not 16-byte aligned");
    if (ws_bytes < w.bytes()) return fail(SPC_ERR_WORKSPACE, "ws_bytes=%zu, need %zu", ws_bytes, w.bytes());
    p.segs = Segs{seg_ptr, int32_t(n_seg), int32_t(n)};
    p.C = C, p.G = G, p.eps = 0.f, p.k = w.k;
    return make_drop(drop, p.drop);
}

// One kernel of the activations' and dropout's variants.
#define NORM_VARIANT(name, grid, NT, ...)                                                                    \
    do {                                                                                                      \
        if (p.drop.rng) {                                                                                     \
            if (act == SPC_ACT_RELU) hipLaunchKernelGGL((name<TT, SPC_ACT_RELU, true>), grid, dim3(NT), 0, stream, __VA_ARGS__);  \
            else if (act == SPC_ACT_SILU) hipLaunchKernelGGL((name<TT, SPC_ACT_SILU, true>), grid, dim3(NT), 0, stream, __VA_ARGS__); \
            else hipLaunchKernelGGL((name<TT, SPC_ACT_NONE, true>), grid, dim3(NT), 0, stream, __VA_ARGS__);  \
        } else {                                                                                              \
            if (act == SPC_ACT_RELU) hipLaunchKernelGGL((name<TT, SPC_ACT_RELU, false>), grid, dim3(NT), 0, stream, __VA_ARGS__); \
            else if (act == SPC_ACT_SILU) hipLaunchKernelGGL((name<TT, SPC_ACT_SILU, false>), grid, dim3(NT), 0, stream, __VA_ARGS__); \
            else hipLaunchKernelGGL((name<TT, SPC_ACT_NONE, false>), grid, dim3(NT), 0, stream, __VA_ARGS__); \
        }                                                                                                     \
        SPC_LAUNCHED(#name);                                                                                  \
    } while (0)

template <typename TT>
spc_status launch_fwd(const void* x, const NormArgs& p, const NormWs& w, const float* gamma, const float* beta, int act,
                      void* y, float2* stats, void* ws, hipStream_t stream) {
    if (const int CW = w.CW) {
        NORM_VARIANT(k_norm_small, dim3(unsigned(p.segs.n_seg) * unsigned(p.C / CW)), NS, x, p, CW, gamma, beta, stats, y);
        return SPC_OK;
    }
    float2* part = static_cast<float2*>(ws);
    const dim3 grid(p.k.blocks());
    if (p.k.tiles) {
        hipLaunchKernelGGL(k_norm_stats<TT>, grid, dim3(NT), 0, stream, x, p, part);
        SPC_LAUNCHED("k_norm_stats");
    }
    hipLaunchKernelGGL(k_norm_group, job_grid(w.stats), dim3(NG), 0, stream, p, unsigned(w.stats), part, stats);
    SPC_LAUNCHED("k_norm_group");
    if (p.k.tiles) NORM_VARIANT(k_norm_apply, grid, NT, x, p, gamma, beta, stats, y);
    return SPC_OK;
}

template <typename TT>
spc_status launch_bwd(const void* dy, const void* x, const NormArgs& p, const NormWs& w, const float* gamma,
                      const float* beta, const float2* stats, int act, void* dx, float* dgamma, float* dbeta, void* ws,
                      hipStream_t stream) {
    const bool affine = dgamma || dbeta;
    float2 *part = static_cast<float2*>(ws), *tot = affine ? w.tot_of(ws) : nullptr, *means = w.means_of(ws);
    if (const int CW = w.CW) {
        const bool one = p.segs.n_seg == 1;
        tot = affine && !one ? part : nullptr;
        NORM_VARIANT(k_norm_bwd_small, dim3(unsigned(p.segs.n_seg) * unsigned(p.C / CW)), NS, x, dy, p, CW, gamma, beta, stats, tot,
                     one ? dgamma : nullptr, one ? dbeta : nullptr, dx);
        if (tot) {
            hipLaunchKernelGGL(k_norm_bwd_group, job_grid(p.C / 8), dim3(NG), 0, stream, p, unsigned(p.C / 8), 0u, gamma, part, tot,
                               p.segs.n_seg, means, dgamma, dbeta);
            SPC_LAUNCHED("k_norm_bwd_group");
        }
        return SPC_OK;
    }
    const dim3 grid(p.k.blocks());
    if (p.k.tiles) NORM_VARIANT(k_norm_bwd_sums, grid, NT, x, dy, p, gamma, beta, stats, part, tot);
    const int64_t jobs = w.stats + (affine ? p.C / 8 : 0);
    hipLaunchKernelGGL(k_norm_bwd_group, job_grid(jobs), dim3(NG), 0, stream, p, unsigned(jobs), unsigned(w.stats), gamma, part, tot,
                       p.k.tiles * p.k.Y, means, dgamma, dbeta);
    SPC_LAUNCHED("k_norm_bwd_group");
    if (p.k.tiles) NORM_VARIANT(k_norm_bwd_apply, grid, NT, x, dy, p, gamma, beta, stats, means, dx);
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
