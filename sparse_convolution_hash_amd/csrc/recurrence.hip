// Gated linear recurrence over the rows of ragged samples, per channel:
//   a_t = sigmoid(gate_t),  h_t = a_t h_{t-1} + (1 - a_t) x_t,  h_{-1} = h0
// and backward, D_t = dh_t + a_{t+1} D_{t+1} (D_last = dh_last + dh):
//   dx_t = (1 - a_t) D_t,  dgate_t = a_t (1 - a_t) (h_{t-1} - x_t) D_t,  dh0 = a_0 D_0
//
// Both directions are scans of maps h -> A h + B, which compose as
//   (A2, B2) o (A1, B1) = (A2 A1, A2 B1 + B2).
// A sample's first step forgets what came before: its map is (reset, B), with
// A = -0 as the mark.  (A sigmoid is never negative, and -0 times it stays -0.)
// So samples need no structure of their own, and tiles of rows are cut evenly
// whatever the lengths.  Backward, with E_t = a_t D_t, the map is
// E -> a_t (dh_t + E), over the rows in the opposite order.
//
// One pass over the data.  A thread holds a chunk of T rows x 4 channels in
// registers and folds them to one map per channel; the chunks of a workgroup
// (its tile) are folded in LDS; tiles are joined across workgroups by
// look-back over published maps, in a tree of radix 16: word i of level l is
// the map of tiles [i 16^l, (i + 1) 16^l), and a tile folds at most 15 words a
// level.  The tree is fixed by the tile numbers, so the result does not depend
// on timing.  A word is one 64-bit atomic (A, B) and is its own flag: all ones
// (a NaN that is never published as A) until written.
// Waits end: tiles are numbered by a ticket taken when a workgroup starts, a
// tile waits only for lower tickets, and those have started.
#include "rows.h"

namespace spc {
namespace {

constexpr int NT = 256;     // threads per workgroup
constexpr int QPR = 16;     // most lanes (of 4 channels) per row: slabs of up to 64 channels
constexpr int RADIX = 16;   // tiles per group of the look-back tree

// Rows per chunk: 16-bit types hold twice the rows in the same registers.
template <typename TT>
struct ChunkRows {
    static constexpr int T = TT::E == 8 ? 16 : 8;
};
inline int chunk_rows(spc_dtype t) { return t == SPC_F32 ? 8 : 16; }

// How [n, C] is cut: slabs of CW channels, CPR lanes to a row, NCH chunks to a tile.
struct Cut {
    int32_t nslab, CPR, CW, NCH, rows;
    int32_t tiles;
};

inline Cut cut_of(spc_dtype dtype, int64_t n, int32_t C) {
    Cut k;
    k.nslab = int32_t(ceil_div(C / 4, QPR));
    k.CPR = int32_t(ceil_div(C / 4, k.nslab));
    k.CW = 4 * k.CPR;
    k.NCH = NT / k.CPR;
    k.rows = k.NCH * chunk_rows(dtype);
    k.tiles = int32_t(ceil_div(n, k.rows));
    return k;
}

struct LrArgs {
    Segs segs;
    int32_t C, reverse;
    int64_t ld;             // row stride of gate and x (and of their gradients: ldg)
    int64_t ldg;
    const int32_t* order;   // row of each position, NULL: the identity
    Cut k;
    uint32_t* ticket;       // NULL with one tile
    uint64_t* words;
};

// ---------------------------------------------------------------- elements

// Four channels as stored.
template <typename TT>
struct Raw4 {
    uint32_t v[16 / TT::E];
};
template <typename TT>
__device__ __forceinline__ Raw4<TT> ldr(const void* p);
template <>
__device__ __forceinline__ Raw4<F32> ldr<F32>(const void* p) { return __builtin_bit_cast(Raw4<F32>, ld16(p)); }
template <>
__device__ __forceinline__ Raw4<F16> ldr<F16>(const void* p) { return __builtin_bit_cast(Raw4<F16>, *static_cast<const uint2*>(p)); }
template <>
__device__ __forceinline__ Raw4<BF16> ldr<BF16>(const void* p) { return __builtin_bit_cast(Raw4<BF16>, *static_cast<const uint2*>(p)); }

template <typename TT>
__device__ __forceinline__ float elem(const Raw4<TT>& r, int j);
template <>
__device__ __forceinline__ float elem<F32>(const Raw4<F32>& r, int j) { return __uint_as_float(r.v[j]); }
template <>
__device__ __forceinline__ float elem<F16>(const Raw4<F16>& r, int j) {
    return float(__builtin_bit_cast(_Float16, uint16_t(j & 1 ? r.v[j / 2] >> 16 : r.v[j / 2])));
}
template <>
__device__ __forceinline__ float elem<BF16>(const Raw4<BF16>& r, int j) {
    return __uint_as_float(j & 1 ? r.v[j / 2] & 0xffff0000u : r.v[j / 2] << 16);
}

// Four values rounded once (nearest even) and stored.
template <typename TT>
__device__ __forceinline__ void str(void* p, const f32x4_t& f);
template <>
__device__ __forceinline__ void str<F32>(void* p, const f32x4_t& f) { *static_cast<f32x4_t*>(p) = f; }
typedef _Float16 f16x4v_t __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x4v_t __attribute__((ext_vector_type(4)));
template <>
__device__ __forceinline__ void str<F16>(void* p, const f32x4_t& f) {
    *static_cast<uint2*>(p) = __builtin_bit_cast(uint2, __builtin_convertvector(f, f16x4v_t));
}
template <>
__device__ __forceinline__ void str<BF16>(void* p, const f32x4_t& f) {
    *static_cast<uint2*>(p) = __builtin_bit_cast(uint2, __builtin_convertvector(f, bf16x4v_t));
}

// The smaller of sigmoid(g) and sigmoid(-g) to full relative precision (2 and
// 1 units of exp and rcp), and the larger as its complement to 1.
__device__ __forceinline__ float gate_small(float g, float& big) {
    const float e = __builtin_amdgcn_exp2f(-1.44269504f * fabsf(g));
    big = __builtin_amdgcn_rcpf(1.f + e);
    return e * big;
}
// a = sigmoid(g) and na = 1 - a = sigmoid(-g), each to full relative precision.
__device__ __forceinline__ void gates(float g, float& a, float& na) {
    float big;
    const float small = gate_small(g, big);
    a = g >= 0.f ? big : small;
    na = g >= 0.f ? small : big;
}

// -------------------------------------------------------------------- maps

struct Map {
    float A, B;
};
__device__ __forceinline__ bool is_reset(float A) { return __float_as_int(A) < 0; }

// s after f.
__device__ __forceinline__ Map after(const Map& s, const Map& f) {
    const bool r = is_reset(s.A);
    return Map{r ? s.A : s.A * f.A, r ? s.B : fmaf(s.A, f.B, s.B)};
}
__device__ __forceinline__ float apply(const Map& m, float h) { return is_reset(m.A) ? m.B : fmaf(m.A, h, m.B); }

constexpr uint64_t EMPTY = ~uint64_t(0);
__device__ __forceinline__ void publish(uint64_t* p, Map m) {
    if (m.A != m.A) m.A = __uint_as_float(0x7fc00000u);
    __hip_atomic_store(p, uint64_t(__float_as_uint(m.A)) | uint64_t(__float_as_uint(m.B)) << 32, __ATOMIC_RELAXED,
                       __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ uint64_t peek(const uint64_t* p) {
    return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ bool there(uint64_t w) { return uint32_t(w) != 0xffffffffu; }

// A wait that has lasted this many polls (a good part of a second) can only mean a workspace
// that another call is using at the same time: the missing maps become NaN
// and the kernel ends.
constexpr int MAX_POLLS = 1 << 18;

// The map of all tiles before tile t, whose own map is own, for the channel of
// this lane; called by one wave (lanes from CW on take part in its votes only).
__device__ __forceinline__ Map look_back(const LrArgs& p, int t, int slab, int c, bool on, Map own) {
    const Cut& k = p.k;
    const int64_t stride = int64_t(k.nslab) * k.CW;
    uint64_t* w = p.words + int64_t(slab) * k.CW + c;
    Map before{1.f, 0.f}, all = own;
    if (on) publish(w + t * stride, own);
    bool full = true;
    for (int i = t, count = k.tiles;;) {
        const int m = i % RADIX;
        if (!__all(!on || is_reset(before.A))) {
            const uint64_t* q = w + (i - m) * stride;
            uint64_t v[RADIX - 1];
            for (int polls = 0;; ++polls) {
                bool ready = true;
#pragma unroll
                for (int j = 0; j < RADIX - 1; ++j) v[j] = j < m && on ? peek(q + j * stride) : 0;
#pragma unroll
                for (int j = 0; j < RADIX - 1; ++j) ready = ready && there(v[j]);
                if (__all(ready) || polls == MAX_POLLS) break;
                __builtin_amdgcn_s_sleep(1);
            }
            Map f{1.f, 0.f};
#pragma unroll
            for (int j = 0; j < RADIX - 1; ++j)
                if (j < m) f = after(Map{__uint_as_float(uint32_t(v[j])), __uint_as_float(uint32_t(v[j] >> 32))}, f);
            before = after(before, f);
            all = after(all, f);
        }
        w += count * stride;
        full = full && m == RADIX - 1;
        i /= RADIX;
        count /= RADIX;
        if (full && on && i < count) publish(w + i * stride, all);
        if (i == 0 || (!full && __all(!on || is_reset(before.A)))) return before;
    }
}

// Words of the look-back tree.
inline int64_t tree_words(const Cut& k) {
    int64_t w = 0;
    for (int64_t c = k.tiles; c > 0; c /= RADIX) w += c;
    return w * k.nslab * k.CW;
}

// ------------------------------------------------------------------- tiles

// What a workgroup shares.
struct Shared {
    float2 map[NT * 4];       // [chunk][channel]: a chunk's map
    float2 part[NT];          // [part][channel]: the map of a part's chunks
    float in[NT * 4];         // [chunk][channel]: the state a chunk starts from
    int32_t sample[NT * 4];   // of a marked row (NT / 4 chunks at most, of 16 rows)
    uint32_t first[NT / 8], last[NT / 8];   // marks: a sample's first and last row
    int32_t tile;
};

// Takes the next tile; returns tile and slab (slabs of one tile are neighbours).
__device__ __forceinline__ void take(const LrArgs& p, Shared& sh, int& tile, int& slab) {
    int id = blockIdx.x;
    if (p.ticket) {
        if (threadIdx.x == 0) sh.tile = int(atomicAdd(p.ticket, 1u));
        __syncthreads();
        id = sh.tile;
    }
    tile = id / p.k.nslab;
    slab = id - tile * p.k.nslab;
}

// Marks the first and last rows of the samples that lie in positions
// [p0, p0 + rows) of the walk, and leaves the rows' own numbers in rowno
// (ORDERED: -1 where there is none).
template <bool ORDERED>
__device__ __forceinline__ void mark(const LrArgs& p, Shared& sh, int32_t* rowno, int p0) {
    const int n = p.segs.n, rows = p.k.rows;
    if (threadIdx.x < NT / 8) sh.first[threadIdx.x] = sh.last[threadIdx.x] = 0;
    const int f0 = p0 > 0 ? p0 : 0, f1 = p0 + rows < n ? p0 + rows : n;      // within the walk
    const int qa = p.reverse ? n - f1 : f0, qb = p.reverse ? n - f0 : f1;    // as positions of the samples
    if constexpr (ORDERED) {
        const int lo = p.segs.at(0), hi = p.segs.at(p.segs.n_seg);
        for (int i = threadIdx.x; i < rows; i += NT) {
            const int f = p0 + i, q = p.reverse ? n - 1 - f : f;
            int r = -1;
            if (q >= qa && q < qb && q >= lo && q < hi) r = p.order[q];
            rowno[i] = unsigned(r) < unsigned(n) ? r : -1;
        }
    }
    const int s0 = p.segs.find(qa);
    __syncthreads();
    for (int s = s0 + int(threadIdx.x); s < p.segs.n_seg; s += NT) {
        const int a = p.segs.at(s), b = p.segs.at(s + 1);
        if (a >= qb) break;
        if (a >= b) continue;
        const int i0 = (p.reverse ? n - b : a) - p0, i1 = (p.reverse ? n - 1 - a : b - 1) - p0;
        if (unsigned(i0) < unsigned(rows)) {
            sh.sample[i0] = s;
            atomicOr(&sh.first[i0 / 32], 1u << (i0 % 32));
        }
        if (unsigned(i1) < unsigned(rows)) {
            sh.sample[i1] = s;
            atomicOr(&sh.last[i1 / 32], 1u << (i1 % 32));
        }
    }
    __syncthreads();
}

// The state that each chunk starts from, given the chunks' maps in sh.map in
// the order of the walk.  All threads call it.
__device__ __forceinline__ void join(const LrArgs& p, Shared& sh, int tile, int slab) {
    const int CW = p.k.CW, NCH = p.k.NCH, parts = NT / CW;
    const int per = (NCH + parts - 1) / parts;   // 4 or 5 chunks
    const int part = int(threadIdx.x) / CW, c = int(threadIdx.x) - part * CW;
    const int k0 = part * per, k1 = part < parts ? (k0 + per < NCH ? k0 + per : NCH) : 0;
    __syncthreads();
    Map m{1.f, 0.f};
    for (int k = k0; k < k1; ++k) {
        const float2 v = sh.map[k * CW + c];
        m = after(Map{v.x, v.y}, m);
    }
    if (part < parts) sh.part[part * CW + c] = float2{m.A, m.B};
    __syncthreads();
    if (threadIdx.x < WAVE) {
        const bool on = int(threadIdx.x) < CW;
        float h = 0.f;
        if (p.ticket) {
            Map own{1.f, 0.f};
            if (on)
                for (int i = 0; i < parts; ++i) {
                    const float2 v = sh.part[i * CW + threadIdx.x];
                    own = after(Map{v.x, v.y}, own);
                }
            h = apply(look_back(p, tile, slab, on ? int(threadIdx.x) : 0, on, own), 0.f);
        }
        if (on)
            for (int i = 0; i < parts; ++i) {
                const float2 v = sh.part[i * CW + threadIdx.x];
                sh.part[i * CW + threadIdx.x].x = h;
                h = apply(Map{v.x, v.y}, h);
            }
    }
    __syncthreads();
    if (part < parts) {
        float h = sh.part[part * CW + c].x;
        for (int k = k0; k < k1; ++k) {
            const float2 v = sh.map[k * CW + c];
            sh.in[k * CW + c] = h;
            h = apply(Map{v.x, v.y}, h);
        }
    }
    __syncthreads();
}

// States of the samples without rows.
__device__ __forceinline__ void pass_empty(const LrArgs& p, const float* from, float* to, int64_t first, int64_t step) {
    if (!to) return;
    for (int64_t s = first; s < p.segs.n_seg; s += step)
        if (p.segs.at(int(s)) >= p.segs.at(int(s) + 1))
            for (int c = 0; c < p.C; c += 4) {
                const int64_t i = s * p.C + c;
                *reinterpret_cast<f32x4_t*>(to + i) = from ? *reinterpret_cast<const f32x4_t*>(from + i) : f32x4_t{0, 0, 0, 0};
            }
}

// Before a scan of several tiles: its words and ticket, and the samples without rows.
__global__ __launch_bounds__(NT) void k_lr_clear(LrArgs p, int64_t words, const float* from, float* to) {
    const int64_t i = int64_t(blockIdx.x) * NT + threadIdx.x, step = int64_t(gridDim.x) * NT;
    if (p.ticket) {
        if (i == 0) *p.ticket = 0;
        for (int64_t j = i; 2 * j < words; j += step) st16(p.words + 2 * j, u32x4{~0u, ~0u, ~0u, ~0u});
    }
    pass_empty(p, from, to, i, step);
}

// A thread's chunk.
template <typename TT, bool ORDERED, bool BACK>
struct Chunk {
    static constexpr int T = ChunkRows<TT>::T;
    const LrArgs& p;
    const int32_t* rowno;
    int ch;          // number within the tile, in the order of the scan
    int i0;          // its first row within the tile
    int pos;         // position in the walk of its first row
    int lo, hi;      // positions [lo, hi) lie in samples
    int c;           // first channel
    bool on;
    uint32_t first, last;   // marks
    bool plain;      // the wave's chunks have no marks and all their rows

    __device__ __forceinline__ Chunk(const LrArgs& a, Shared& sh, const int32_t* rn, int tile, int slab) : p(a), rowno(rn) {
        const int CPR = p.k.CPR, n = p.segs.n;
        ch = int(threadIdx.x) / CPR;
        const int quad = int(threadIdx.x) - ch * CPR;
        c = (slab * CPR + quad) * 4;
        on = ch < p.k.NCH && c < p.C;
        i0 = (BACK ? p.k.NCH - 1 - ch : ch) * T;
        if (!on) i0 = 0;
        pos = base(p, tile) + i0;
        const int a0 = p.segs.at(0), b0 = p.segs.at(p.segs.n_seg);
        lo = p.reverse ? n - b0 : a0;
        hi = p.reverse ? n - a0 : b0;
        const uint32_t mask = (1u << T) - 1;
        first = on ? sh.first[i0 / 32] >> (i0 % 32) & mask : 0;
        last = on ? sh.last[i0 / 32] >> (i0 % 32) & mask : 0;
        bool whole = pos >= lo && pos + T <= hi;
        if constexpr (ORDERED)
#pragma unroll
            for (int t = 0; t < T; ++t) whole = whole && rowno[i0 + t] >= 0;
        plain = __all(!on || (whole && !(first | last)));
    }

    // Position of a tile's first row: the backward's tiles are numbered from
    // the end, and cut at the same chunks as the forward's.
    static __device__ __forceinline__ int base(const LrArgs& p, int tile) {
        if (!BACK) return tile * p.k.rows;
        const int chunks = (p.segs.n + T - 1) / T;
        return (chunks - (tile + 1) * p.k.NCH) * T;
    }

    __device__ __forceinline__ int row(int t) const {
        if constexpr (ORDERED) return rowno[i0 + t];
        const int f = pos + t;
        return f >= lo && f < hi ? (p.reverse ? p.segs.n - 1 - f : f) : -1;
    }
    // The row of a plain chunk.
    __device__ __forceinline__ int64_t prow(int t) const {
        if constexpr (ORDERED) return rowno[i0 + t];
        return p.reverse ? p.segs.n - 1 - pos - t : pos + t;
    }
};

template <typename TT, bool ORDERED>
__global__ __launch_bounds__(NT, 2) void k_lr_fwd(const void* __restrict__ gate_, const void* __restrict__ x_, LrArgs p,
                                                  const float* __restrict__ h0, void* __restrict__ out_,
                                                  float* __restrict__ h_last, float* __restrict__ carry) {
    constexpr int T = ChunkRows<TT>::T;
    using S = typename TT::storage;
    const S *gate = static_cast<const S*>(gate_), *x = static_cast<const S*>(x_);
    S* out = static_cast<S*>(out_);
    __shared__ Shared sh;
    __shared__ int32_t rowno[ORDERED ? NT * 4 : 1];
    int tile, slab;
    take(p, sh, tile, slab);
    if (tile >= p.k.tiles) return;
    mark<ORDERED>(p, sh, rowno, Chunk<TT, ORDERED, false>::base(p, tile));
    const Chunk<TT, ORDERED, false> k(p, sh, rowno, tile, slab);

    f32x4_t a[T], b[T];
    f32x4_t A = 1.f, B = 0.f;
    if (k.plain) {
        if (k.on) {
            Raw4<TT> g[T], v[T];
#pragma unroll
            for (int t = 0; t < T; ++t) {
                const int64_t o = k.prow(t) * p.ld + k.c;
                g[t] = ldr<TT>(gate + o);
                v[t] = ldr<TT>(x + o);
            }
#pragma unroll
            for (int t = 0; t < T; ++t)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    float aj, na;
                    gates(elem<TT>(g[t], j), aj, na);
                    a[t][j] = aj;
                    b[t][j] = na * elem<TT>(v[t], j);
                    A[j] *= a[t][j];
                    B[j] = fmaf(a[t][j], B[j], b[t][j]);
                }
        }
    } else if (k.on) {
        Raw4<TT> g[T], v[T];
#pragma unroll
        for (int t = 0; t < T; ++t) {
            const int r = k.row(t);
            const int64_t o = (r < 0 ? 0 : r) * p.ld + k.c;
            g[t] = ldr<TT>(gate + o);
            v[t] = ldr<TT>(x + o);
        }
#pragma unroll
        for (int t = 0; t < T; ++t) {
            const bool ok = k.row(t) >= 0, start = k.first >> t & 1;
            f32x4_t h = 0.f;
            if (start && h0) h = *reinterpret_cast<const f32x4_t*>(h0 + int64_t(sh.sample[k.i0 + t]) * p.C + k.c);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                float aj, na;
                gates(elem<TT>(g[t], j), aj, na);
                a[t][j] = aj;
                b[t][j] = na * elem<TT>(v[t], j);
                if (!ok) a[t][j] = 1.f, b[t][j] = 0.f;
                if (start) b[t][j] = fmaf(a[t][j], h[j], b[t][j]), a[t][j] = -0.f;
                const Map m = after(Map{a[t][j], b[t][j]}, Map{A[j], B[j]});
                A[j] = m.A, B[j] = m.B;
            }
        }
    }
    const int at = k.ch * p.k.CW + k.c - slab * p.k.CW;
    if (k.ch < p.k.NCH) {
        f32x4_t* q = reinterpret_cast<f32x4_t*>(&sh.map[at]);
        q[0] = f32x4_t{A[0], B[0], A[1], B[1]};
        q[1] = f32x4_t{A[2], B[2], A[3], B[3]};
    }
    join(p, sh, tile, slab);
    if (!k.on) return;
    f32x4_t h = *reinterpret_cast<const f32x4_t*>(&sh.in[at]);
    if (carry && k.pos < p.segs.n)
        *reinterpret_cast<f32x4_t*>(carry + int64_t(tile * p.k.NCH + k.ch) * p.C + k.c) = h;
    if (k.plain) {
#pragma unroll
        for (int t = 0; t < T; ++t) {
#pragma unroll
            for (int j = 0; j < 4; ++j) h[j] = fmaf(a[t][j], h[j], b[t][j]);
            str<TT>(out + k.prow(t) * p.C + k.c, h);
        }
    } else {
#pragma unroll
        for (int t = 0; t < T; ++t) {
#pragma unroll
            for (int j = 0; j < 4; ++j) h[j] = apply(Map{a[t][j], b[t][j]}, h[j]);
            const int r = k.row(t);
            if (r >= 0) str<TT>(out + int64_t(r) * p.C + k.c, h);
            if ((k.last >> t & 1) && h_last)
                *reinterpret_cast<f32x4_t*>(h_last + int64_t(sh.sample[k.i0 + t]) * p.C + k.c) = h;
        }
    }
}

template <typename TT, bool ORDERED>
__global__ __launch_bounds__(NT, 2) void k_lr_bwd(const void* __restrict__ dout_, const void* __restrict__ gate_,
                                                  const void* __restrict__ x_, LrArgs p, const float* __restrict__ h0,
                                                  const float* __restrict__ carry, const float* __restrict__ dh_last,
                                                  void* __restrict__ dgate_, void* __restrict__ dx_, float* __restrict__ dh0) {
    constexpr int T = ChunkRows<TT>::T;
    using S = typename TT::storage;
    const S *gate = static_cast<const S*>(gate_), *x = static_cast<const S*>(x_), *dout = static_cast<const S*>(dout_);
    S *dgate = static_cast<S*>(dgate_), *dx = static_cast<S*>(dx_);
    __shared__ Shared sh;
    __shared__ int32_t rowno[ORDERED ? NT * 4 : 1];
    int tile, slab;
    take(p, sh, tile, slab);
    if (tile >= p.k.tiles) return;
    mark<ORDERED>(p, sh, rowno, Chunk<TT, ORDERED, true>::base(p, tile));
    const Chunk<TT, ORDERED, true> k(p, sh, rowno, tile, slab);
    const bool on = k.on && k.pos >= 0;      // the last tile reaches past the walk's start

    // Kept of every element: sm, the smaller of a and 1 - a, with the gate's
    // sign; u = h_{t-1} - x_t; and dout as it is.
    f32x4_t sm[T], u[T];
    Raw4<TT> d[T];
    f32x4_t A = 1.f, B = 0.f;
    const auto a_of = [](float s, float& na) {
        const float m = fabsf(s);
        const bool pos = !(__float_as_int(s) < 0);
        na = pos ? m : 1.f - m;
        return pos ? 1.f - m : m;
    };
    if (on) {
        Raw4<TT> g[T], v[T];
        f32x4_t h = *reinterpret_cast<const f32x4_t*>(carry + int64_t(k.pos / T) * p.C + k.c);
#pragma unroll
        for (int t = 0; t < T; ++t) {
            const int64_t r = k.plain ? k.prow(t) : (k.row(t) < 0 ? 0 : k.row(t));
            g[t] = ldr<TT>(gate + r * p.ld + k.c);
            v[t] = ldr<TT>(x + r * p.ld + k.c);
            d[t] = ldr<TT>(dout + r * p.C + k.c);
        }
#pragma unroll
        for (int t = 0; t < T; ++t) {
            bool ok = true;
            if (!k.plain) {
                ok = k.row(t) >= 0;
                if (k.first >> t & 1)
                    h = h0 ? *reinterpret_cast<const f32x4_t*>(h0 + int64_t(sh.sample[k.i0 + t]) * p.C + k.c) : f32x4_t{0, 0, 0, 0};
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float gj = elem<TT>(g[t], j), xj = elem<TT>(v[t], j);
                float big;
                const float small = gate_small(gj, big);
                sm[t][j] = __builtin_copysignf(small, gj);
                u[t][j] = h[j] - xj;
                const float a = gj >= 0.f ? big : small, na = gj >= 0.f ? small : big;
                const float next = fmaf(a, h[j], na * xj);
                h[j] = ok ? next : h[j];
            }
        }
#pragma unroll
        for (int t = T - 1; t >= 0; --t) {
            if (!k.plain) {
                if (k.last >> t & 1) {
                    A = -0.f;
                    B = dh_last ? *reinterpret_cast<const f32x4_t*>(dh_last + int64_t(sh.sample[k.i0 + t]) * p.C + k.c)
                                : f32x4_t{0, 0, 0, 0};
                }
                if (k.row(t) < 0) continue;
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                float na;
                const float a = a_of(sm[t][j], na);
                A[j] *= a;
                B[j] = a * (elem<TT>(d[t], j) + B[j]);
            }
        }
    }
    const int at = k.ch * p.k.CW + k.c - slab * p.k.CW;
    if (k.ch < p.k.NCH) {
        f32x4_t* q = reinterpret_cast<f32x4_t*>(&sh.map[at]);
        q[0] = f32x4_t{A[0], B[0], A[1], B[1]};
        q[1] = f32x4_t{A[2], B[2], A[3], B[3]};
    }
    join(p, sh, tile, slab);
    if (!on) return;
    f32x4_t E = *reinterpret_cast<const f32x4_t*>(&sh.in[at]);
#pragma unroll
    for (int t = T - 1; t >= 0; --t) {
        int64_t r = 0;
        if (k.plain) {
            r = k.prow(t);
        } else {
            r = k.row(t);
            if (k.last >> t & 1)
                E = dh_last ? *reinterpret_cast<const f32x4_t*>(dh_last + int64_t(sh.sample[k.i0 + t]) * p.C + k.c)
                            : f32x4_t{0, 0, 0, 0};
        }
        if (k.plain || r >= 0) {
            f32x4_t gx, gg;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                float na;
                const float a = a_of(sm[t][j], na), D = elem<TT>(d[t], j) + E[j];
                gx[j] = na * D;
                E[j] = a * D;
                gg[j] = na * u[t][j] * E[j];
            }
            str<TT>(dx + r * p.ldg + k.c, gx);
            str<TT>(dgate + r * p.ldg + k.c, gg);
        }
        if (!k.plain && (k.first >> t & 1) && dh0)
            *reinterpret_cast<f32x4_t*>(dh0 + int64_t(sh.sample[k.i0 + t]) * p.C + k.c) = E;
    }
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

// The states that the chunks start from.
size_t carry_bytes(spc_dtype dtype, int64_t n, int32_t C) { return size_t(ceil_div(n, chunk_rows(dtype))) * C * 4; }
// The ticket and the look-back tree; a scan of one tile needs neither.
size_t ws_need(spc_dtype dtype, int64_t n, int32_t C) {
    const Cut k = cut_of(dtype, n, C);
    return 256 + (k.tiles > 1 ? size_t(tree_words(k)) * 8 : 0);
}

spc_status check_call(spc_dtype dtype, int64_t n, int32_t C, int64_t ld, const int32_t* seg_ptr, int64_t n_seg,
                      const int32_t* order, int32_t reverse, void* ws, size_t ws_bytes, LrArgs& p) {
    spc_status st = check_sizes(dtype, n, C, n_seg);
    if (st == SPC_OK) st = check_stride(dtype, ld, C, "ld");
    if (st != SPC_OK) return st;
    if (!seg_ptr && n_seg != 1) return fail(SPC_ERR_ARG, "seg_ptr is NULL with n_seg=%lld", (long long)n_seg);
    if (!ws) return fail(SPC_ERR_ARG, "ws is NULL");
    for (const void* q : {(const void*)seg_ptr, (const void*)order, (const void*)ws})
        if (q && !aligned16(q)) return fail(SPC_ERR_ARG, "device pointers must be 16-byte aligned");
    if (ws_bytes < ws_need(dtype, n, C))
        return fail(SPC_ERR_WORKSPACE, "ws_bytes=%zu, need %zu", ws_bytes, ws_need(dtype, n, C));
    p.segs = Segs{seg_ptr, int32_t(n_seg), int32_t(n)};
    p.C = C, p.reverse = reverse != 0, p.ld = ld, p.ldg = C, p.order = order;
    p.k = cut_of(dtype, n, C);
    if (int64_t(p.k.tiles) * p.k.nslab >= (int64_t(1) << 31)) return fail(SPC_ERR_UNSUPPORTED, "%lld rows of %d channels exceed one launch", (long long)n, C);
    const bool many = p.k.tiles > 1;
    p.ticket = many ? static_cast<uint32_t*>(ws) : nullptr;
    p.words = many ? reinterpret_cast<uint64_t*>(static_cast<char*>(ws) + 256) : nullptr;
    return SPC_OK;
}

// The launch before a scan; a single tile of a single sample with rows needs none.
spc_status clear(const LrArgs& p, const float* from, float* to, hipStream_t stream) {
    const int64_t words = p.ticket ? tree_words(p.k) : 0;
    if (!p.ticket && !(to && (p.segs.ptr || p.segs.n == 0))) return SPC_OK;
    const int64_t work = ceil_div(words / 2 > p.segs.n_seg ? words / 2 : p.segs.n_seg, NT);
    hipLaunchKernelGGL(k_lr_clear, dim3(unsigned(work < 4096 ? work : 4096)), dim3(NT), 0, stream, p, words, from, to);
    SPC_LAUNCHED("k_lr_clear");
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

#define LR_DISPATCH2(name, flag, grid, block, ...)                                                                \
    do {                                                                                                          \
        if (dtype == SPC_F32) hipLaunchKernelGGL((name<F32, flag>), grid, block, 0, stream, __VA_ARGS__);         \
        if (dtype == SPC_F16) hipLaunchKernelGGL((name<F16, flag>), grid, block, 0, stream, __VA_ARGS__);         \
        if (dtype == SPC_BF16) hipLaunchKernelGGL((name<BF16, flag>), grid, block, 0, stream, __VA_ARGS__);       \
        SPC_LAUNCHED(#name);                                                                                      \
    } while (0)

extern "C" spc_status spc_linear_recurrence_workspace(spc_dtype dtype, int64_t n, int32_t C, int64_t n_seg, size_t* ws,
                                                      size_t* carry) {
    clear_error();
    if (!ws || !carry) return fail(SPC_ERR_ARG, "ws or carry is NULL");
    const spc_status st = check_sizes(dtype, n, C, n_seg);
    if (st == SPC_OK) *ws = ws_need(dtype, n, C), *carry = carry_bytes(dtype, n, C);
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
    const spc_status cs = clear(p, h0, h_last, stream);
    if (cs != SPC_OK || n == 0) return cs;
    const dim3 grid(unsigned(p.k.tiles) * unsigned(p.k.nslab));
    if (order) LR_DISPATCH2(k_lr_fwd, true, grid, dim3(NT), gate, x, p, h0, out, h_last, carry);
    else LR_DISPATCH2(k_lr_fwd, false, grid, dim3(NT), gate, x, p, h0, out, h_last, carry);
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
    st = clear(p, dh_last, dh0, stream);
    if (st != SPC_OK || n == 0) return st;
    const dim3 grid(unsigned(p.k.tiles) * unsigned(p.k.nslab));
    if (order) LR_DISPATCH2(k_lr_bwd, true, grid, dim3(NT), dout, gate, x, p, h0, carry, dh_last, dgate, dx, dh0);
    else LR_DISPATCH2(k_lr_bwd, false, grid, dim3(NT), dout, gate, x, p, h0, carry, dh_last, dgate, dx, dh0);
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
