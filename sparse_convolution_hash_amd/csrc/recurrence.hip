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
// A thread walks a strip of L rows x 4 channels.  Launches: the strips' maps,
// folded within each workgroup's tile of strips (k_lr_reduce); the tiles'
// maps to the states they start from (k_lr_tiles); the walk again from its
// start state, with the outputs (k_lr_fwd, k_lr_bwd).  Up to FEW tiles the walk folds
// the tiles before its own itself, and a single tile takes one launch.  The
// order of all folds is fixed by the sizes, so results do not depend on timing.
//
// What bounds it: memory.  Gate and value are read twice (backward gate and
// dout), the second time from the 256 MB cache as far as they fit.  266,426 x 128
// bf16 along an order: reduce 29 us (136 MB read, 17 MB written, 5.3 TB/s),
// tiles 6, walk 40 (5.6 TB/s with the states kept for the backward); backward
// 30 + 6 + 75 (5.0 TB/s).  1,000,003 x 64 bf16 forward: 54 + 7 + 70, 142 us with
// the gaps between launches.  A single pass whose workgroups wait for the maps of
// the tiles before theirs reads once, and measured 123 us there and 184 for the
// 194 us of training above.  Two forms of it were built: with waits that rest on the
// order in which workgroups start (those figures), and with the order taken from one
// counter, which costs 11 ns a workgroup (151 and 221 us).  Here no workgroup waits
// for another one.  A grid of workgroups that are all resident, and long sequences in
// pieces whose second read stays in the cache, have not been measured.
#include "rows.h"

namespace spc {
namespace {

constexpr int NT = 256;      // threads per workgroup
constexpr int QPR = 16;      // most lanes (of 4 channels) per row: slabs of up to 64 channels
constexpr int T = 8;         // rows loaded at a time
constexpr int LMAX = 32;     // most rows of a strip
constexpr int RMAX = NT / 4 * LMAX;   // most rows of a tile
// Tiles that a walk folds itself: 200 to 1,000 rows of 64 channels 11 us instead
// of 13.5 (backward 12.5 instead of 15), the same from 2,000 to 4,000 rows on; with
// 64 tiles 18 instead of 13.5.
constexpr int FEW = 16;

// How [n, C] is cut: slabs of CW channels, CPR lanes to a row, NCH strips of L rows to a tile.
struct Cut {
    int32_t nslab, CPR, CW, NCH, L, rows;
    int32_t tiles;
};

inline Cut cut_of(int64_t n, int32_t C) {
    Cut k;
    k.nslab = int32_t(ceil_div(C / 4, QPR));
    k.CPR = int32_t(ceil_div(C / 4, k.nslab));
    k.CW = 4 * k.CPR;
    k.NCH = NT / k.CPR;
    // the longest strips that still leave 6 waves to each SIMD (half and twice as
    // many: 194 us of training on 266,426 x 128 become 202 and 210); LMAX 16: 147 us
    // forward on 1,000,003 x 64 become 165
    k.L = T;   // longer ones never leave a single tile
    while (k.L < LMAX && n > k.NCH * k.L * 2 && n * (C / 4) / (2 * k.L) >= 6 * 1024 * WAVE) k.L *= 2;
    k.rows = k.NCH * k.L;
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
    float2* strip;          // [tile * NCH + strip][C]: map of the strips before it in its tile
    float2* tile;           // [tile][C]: its map
    float* start;           // [tile][C]: the state it starts from (more than FEW tiles)
};

// ---------------------------------------------------------------- elements

// The compiler takes v for a new value from here on.
__device__ __forceinline__ void hide(float& v) { asm volatile("" : "+v"(v)); }

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

// The smaller of sigmoid(g) and sigmoid(-g): e / (1 + e) with e = exp(-|g|),
// which is 0 below the smallest normal number.  exp2 and rcp are off by a unit in
// the last place each and three roundings come on top, 4 units together.  Rounding
// t = log2(e) |g| and its constant would move e by up to 0.6 |g| units more.  For
// fp32 gates e is corrected by what they lost (beyond 128 e is 0 all the same, and
// an infinite g would lose inf - inf): 30,011 x 48 training 44.6 -> 45.7 us.  A
// 16-bit gate was rounded itself, which moved its e by up to |g| 2^-8 or 2^-11 of its
// value, 6,000 times as much and more: there the correction would only cost time
// (266,426 x 128 bf16 training 194 -> 197 to 199 us, 120,000 x 64 fp16 forward 26.3
// -> 27.2 to 27.9).
template <typename TT>
__device__ __forceinline__ float gate_small(float g) {
    if constexpr (TT::E == 4) {
        const float m = __builtin_elementwise_minimum(fabsf(g), 128.f);   // a NaN stays
        const float t = -1.44269504f * m;
        const float lost = fmaf(fmaf(-1.44269504f, m, -t), 0.693147182f, -1.33497581e-8f * m);
        const float e0 = __builtin_amdgcn_exp2f(t), e = fmaf(e0, lost, e0);
        return e * __builtin_amdgcn_rcpf(1.f + e);
    } else {
        const float e = __builtin_amdgcn_exp2f(-1.44269504f * fabsf(g));
        return e * __builtin_amdgcn_rcpf(1.f + e);
    }
}
// a = sigmoid(g) and na = 1 - a = sigmoid(-g).  The larger is 1 less the
// smaller, half a unit off where that is near 1: there products of thousands of
// gates add up their errors, and rcp(1 + e) would be off by three times as much.
template <typename TT>
__device__ __forceinline__ void gates(float g, float& a, float& na) {
    const float small = gate_small<TT>(g), big = 1.f - small;
    a = g >= 0.f ? big : small;
    na = g >= 0.f ? small : big;
}
// Both from the smaller one with the gate's sign, which is what a chunk keeps
// of its gates: half the registers of the two, and no second exp and rcp.
template <typename TT>
__device__ __forceinline__ float keep(float g) {
    return __builtin_copysignf(gate_small<TT>(g), g);
}
__device__ __forceinline__ void gates_of(float kept, float& a, float& na) {
    const float small = fabsf(kept), big = 1.f - small;
    const bool neg = __float_as_int(kept) < 0;
    a = neg ? small : big;
    na = neg ? big : small;
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

// ------------------------------------------------------------------- tiles

// What a workgroup shares.
struct Shared {
    float2 map[NT * 4];       // [strip][channel]
    float2 part[NT];          // [part][channel]: the map of a part's strips
    int32_t sample[RMAX];     // of a marked row
    uint32_t first[RMAX / 32], last[RMAX / 32];   // marks: a sample's first and last row
};

// The samples around a tile, read once: lane i of every wave holds the offset
// of sample s0 + i.  With up to 63 samples that is all of them and takes one
// load, whose latency the tile's own loads hide.
struct Window {
    int s0, off, lo, hi;   // positions [lo, hi) of the walk lie in samples
};

// Positions of a tile, in the walk [f0, f1) and among the samples [qa, qb).
struct Span {
    int p0, f0, f1, qa, qb;
    __device__ __forceinline__ Span(const LrArgs& p, int tile) {
        const int n = p.segs.n;
        f0 = p0 = tile * p.k.rows;
        f1 = p.k.rows < n - p0 ? p0 + p.k.rows : n;
        qa = p.reverse ? n - f1 : f0;
        qb = p.reverse ? n - f0 : f1;
    }
};

__device__ __forceinline__ Window open_window(const LrArgs& p, const Span& r) {
    const Segs& g = p.segs;
    Window w;
    w.s0 = g.n_seg < WAVE ? 0 : g.find(r.qa);
    const int s = w.s0 + int(threadIdx.x) % WAVE;
    w.off = g.at(s < g.n_seg ? s : g.n_seg);
    const int a = g.at(0), b = g.at(g.n_seg);
    w.lo = p.reverse ? g.n - b : a;
    w.hi = p.reverse ? g.n - a : b;
    return w;
}

// Marks the first and last rows of the samples that lie in the tile; returns
// false, and leaves the marks alone, if there are none.
__device__ __forceinline__ bool mark(const LrArgs& p, Shared& sh, const Span& r, const Window& w) {
    const int n = p.segs.n, rows = p.k.rows;
    // a sample's first or last row is in the tile only if an offset is in [qa, qb]
    const bool past = __any(w.off >= r.qb || w.s0 + int(threadIdx.x) % WAVE >= p.segs.n_seg);
    if (past && !__any(w.off >= r.qa && w.off <= r.qb)) return false;
    for (int i = threadIdx.x; i * 32 < rows; i += NT) sh.first[i] = sh.last[i] = 0;
    __syncthreads();
    for (int s = w.s0 + int(threadIdx.x); s < p.segs.n_seg; s += NT) {
        const int a = p.segs.at(s), b = p.segs.at(s + 1);
        if (a >= r.qb) break;
        if (a >= b) continue;
        const int i0 = (p.reverse ? n - b : a) - r.p0, i1 = (p.reverse ? n - 1 - a : b - 1) - r.p0;
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
    return true;
}

// A thread's strip.
struct Strip {
    int ch;      // number within the tile, in the order of the scan
    int i0;      // its first row within the tile
    int pos;     // position in the walk of its first row
    int c;       // first channel
    int at;      // of its channels in [strip][channel]
    bool on;     // has rows and channels
    __device__ __forceinline__ Strip(const LrArgs& p, const Span& r, int slab, bool back) {
        const int CPR = p.k.CPR;
        ch = int(threadIdx.x) / CPR;
        const int quad = int(threadIdx.x) - ch * CPR;
        c = (slab * CPR + quad) * 4;
        at = ch * p.k.CW + quad * 4;
        i0 = (back ? p.k.NCH - 1 - ch : ch) * p.k.L;
        pos = r.p0 + i0;
        on = ch < p.k.NCH && c < p.C && pos < p.segs.n;
    }
};

// T rows of a strip: their numbers (-1 where there is none) and marks.
template <bool ORDERED>
struct Rows {
    int r[T];
    uint32_t first, last;
    bool simple;     // no marks and all rows, for the whole wave
    __device__ __forceinline__ void numbers(const LrArgs& p, const Window& w, int pos) {
        const int n = p.segs.n;
#pragma unroll
        for (int t = 0; t < T; ++t) {
            const int f = pos + t, q = p.reverse ? n - 1 - f : f;
            r[t] = f >= w.lo && f < w.hi ? (ORDERED ? p.order[q] : q) : -1;
        }
        if constexpr (ORDERED)
#pragma unroll
            for (int t = 0; t < T; ++t) r[t] = unsigned(r[t]) < unsigned(n) ? r[t] : -1;
    }
    __device__ __forceinline__ void marks(const Shared& sh, bool marked, int i) {
        first = marked ? sh.first[i / 32] >> (i % 32) & ((1u << T) - 1) : 0;
        last = marked ? sh.last[i / 32] >> (i % 32) & ((1u << T) - 1) : 0;
        bool all = !(first | last);
#pragma unroll
        for (int t = 0; t < T; ++t) all = all && r[t] >= 0;
        simple = __all(all);
    }
    // A row to load for step t: its own, or any if it has none.
    __device__ __forceinline__ int64_t any(int t) const { return r[t] < 0 ? 0 : r[t]; }
};

__device__ __forceinline__ f32x4_t ld4(const float* p) { return *reinterpret_cast<const f32x4_t*>(p); }
__device__ __forceinline__ void st4(float* p, const f32x4_t& v) { *reinterpret_cast<f32x4_t*>(p) = v; }

// A marked row's sample's state in an optional array [n_seg, C].
__device__ __forceinline__ f32x4_t state_of(const float* a, const LrArgs& p, const Shared& sh, int i, int c) {
    return a ? ld4(a + int64_t(sh.sample[i]) * p.C + c) : f32x4_t{0, 0, 0, 0};
}

// T rows of gate and x, or (BACK) of gate and dout.
template <typename TT, bool ORDERED>
struct Pair {
    Rows<ORDERED> rows;
    Raw4<TT> g[T], x[T];
    __device__ __forceinline__ void load(const LrArgs& p, const Window& w, const void* gate, const void* v, int64_t ldv, int pos, int c) {
        using S = typename TT::storage;
        rows.numbers(p, w, pos);
#pragma unroll
        for (int t = 0; t < T; ++t) {
            g[t] = ldr<TT>(static_cast<const S*>(gate) + rows.any(t) * p.ld + c);
            x[t] = ldr<TT>(static_cast<const S*>(v) + rows.any(t) * ldv + c);
        }
    }
};

// T rows onto a strip's map, from row i of it.  from: h0, or dh_last.
template <typename TT, bool ORDERED, bool BACK>
__device__ __forceinline__ void fold(const Rows<ORDERED>& rows, const Raw4<TT> (&g)[T], const Raw4<TT> (&x)[T], const float* from,
                                     const LrArgs& p, const Shared& sh, const Strip& k, int i, f32x4_t& A, f32x4_t& B) {
    const auto step = [&](int t) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            float a, na;
            gates<TT>(elem<TT>(g[t], j), a, na);
            A[j] *= a;
            B[j] = BACK ? a * (elem<TT>(x[t], j) + B[j]) : fmaf(a, B[j], na * elem<TT>(x[t], j));
        }
    };
    if (rows.simple) {
#pragma unroll
        for (int t = 0; t < T; ++t) step(BACK ? T - 1 - t : t);
    } else {
#pragma unroll
        for (int u = 0; u < T; ++u) {
            const int t = BACK ? T - 1 - u : u;
            if ((BACK ? rows.last : rows.first) >> t & 1) A = -0.f, B = state_of(from, p, sh, k.i0 + i + t, k.c);
            if (rows.r[t] >= 0) step(t);
        }
    }
}

// The map of a strip.
template <typename TT, bool ORDERED, bool BACK>
__device__ __forceinline__ void reduce(const void* gate, const void* v, const float* from, const LrArgs& p, const Shared& sh,
                                       const Window& w, bool marked, const Strip& k, f32x4_t& A, f32x4_t& B) {
    A = 1.f, B = 0.f;
    if (!k.on) return;
    for (int o = 0; o < p.k.L; o += T) {
        const int i = BACK ? p.k.L - T - o : o;
        Pair<TT, ORDERED> b;
        b.load(p, w, gate, v, BACK ? p.C : p.ld, k.pos + i, k.c);
        b.rows.marks(sh, marked, k.i0 + i);
        fold<TT, ORDERED, BACK>(b.rows, b.g, b.x, from, p, sh, k, i, A, B);
    }
}

// Joins the strips' maps of a workgroup in the order of the scan: the map of
// those before each strip goes to out(strip, channel, map), that of all of
// them to all(channel, map).
template <typename F, typename G>
__device__ __forceinline__ void join(const LrArgs& p, Shared& sh, const Strip& k, const f32x4_t& A, const f32x4_t& B, F out, G all) {
    const int CW = p.k.CW, NCH = p.k.NCH, parts = NT / CW;
    const int per = (NCH + parts - 1) / parts;   // 4 or 5 strips
    const int part = int(threadIdx.x) / CW, c = int(threadIdx.x) - part * CW;
    const int k0 = part * per, k1 = part < parts ? (k0 + per < NCH ? k0 + per : NCH) : 0;
    if (k.ch < NCH) {   // a strip without rows: the identity
        f32x4_t* q = reinterpret_cast<f32x4_t*>(&sh.map[k.at]);
        q[0] = f32x4_t{A[0], B[0], A[1], B[1]};
        q[1] = f32x4_t{A[2], B[2], A[3], B[3]};
    }
    __syncthreads();
    Map m{1.f, 0.f};
#pragma unroll 4
    for (int i = k0; i < k1; ++i) {
        const float2 v = sh.map[i * CW + c];
        m = after(Map{v.x, v.y}, m);
    }
    if (part < parts) sh.part[part * CW + c] = float2{m.A, m.B};
    __syncthreads();
    if (part < parts) {
        m = Map{1.f, 0.f};
#pragma unroll 4
        for (int i = 0; i < part; ++i) {
            const float2 v = sh.part[i * CW + c];
            m = after(Map{v.x, v.y}, m);
        }
#pragma unroll 4
        for (int i = k0; i < k1; ++i) {
            const float2 v = sh.map[i * CW + c];
            out(i, c, m);
            m = after(Map{v.x, v.y}, m);
        }
        if (part == parts - 1) all(c, m);
    }
}

template <typename TT, bool ORDERED, bool BACK>
__global__ __launch_bounds__(NT, TT::E == 8 ? 5 : 4) void k_lr_reduce(const void* __restrict__ gate, const void* __restrict__ v,
                                                                             LrArgs p, const float* __restrict__ from) {
    __shared__ Shared sh;
    const int tile = int(blockIdx.x) / p.k.nslab, slab = int(blockIdx.x) - tile * p.k.nslab;
    const Span span(p, tile);
    const Strip k(p, span, slab, BACK);
    const Window w = open_window(p, span);
    const bool marked = mark(p, sh, span, w);
    f32x4_t A, B;
    reduce<TT, ORDERED, BACK>(gate, v, from, p, sh, w, marked, k, A, B);
    const int c0 = slab * p.k.CW;
    join(p, sh, k, A, B,
         [&](int i, int c, const Map& m) {
             if (c0 + c < p.C) p.strip[int64_t(tile * p.k.NCH + i) * p.C + c0 + c] = float2{m.A, m.B};
         },
         [&](int c, const Map& m) {
             if (c0 + c < p.C) p.tile[int64_t(tile) * p.C + c0 + c] = float2{m.A, m.B};
         });
}

// The states that the tiles start from.  A workgroup takes 4 channels; part i
// of 256 folds TP tiles, the parts are joined in their wave by shuffles and
// across the 16 waves in LDS.  More tiles than that go round again.
constexpr int TN = 1024, TP = 8, TR = TN / 4 * TP;
__global__ __launch_bounds__(TN) void k_lr_tiles(LrArgs p, bool back) {
    __shared__ float2 wave[TN / WAVE][4];
    const int c = int(threadIdx.x) % 4, part = int(threadIdx.x) / 4, lane = int(threadIdx.x) % WAVE;
    const int ch = int(blockIdx.x) * 4 + c, tiles = p.k.tiles;
    float h = 0.f;   // before this round's tiles
    for (int base = 0; base < tiles; base += TR) {
        const int count = tiles - base < TR ? tiles - base : TR, per = (count + TN / 4 - 1) / (TN / 4);
        const int i0 = base + part * per;
        Map v[TP], m{1.f, 0.f};
#pragma unroll
        for (int j = 0; j < TP; ++j) {
            const int i = i0 + j;
            v[j] = Map{1.f, 0.f};
            if (j < per && i < tiles) {
                const float2 q = p.tile[int64_t(back ? tiles - 1 - i : i) * p.C + ch];
                v[j] = Map{q.x, q.y};
            }
        }
#pragma unroll
        for (int j = 0; j < TP; ++j) m = after(v[j], m);
        for (int o = 4; o < WAVE; o <<= 1) {
            const Map f{__shfl_up(m.A, o), __shfl_up(m.B, o)};
            if (lane >= o) m = after(m, f);
        }
        if (lane >= WAVE - 4) wave[threadIdx.x / WAVE][c] = float2{m.A, m.B};
        Map before{__shfl_up(m.A, 4), __shfl_up(m.B, 4)};
        if (lane < 4) before = Map{1.f, 0.f};
        __syncthreads();
        float g = h;
#pragma unroll
        for (int i = 0; i < TN / WAVE; ++i) {
            if (i == int(threadIdx.x) / WAVE) h = g;
            g = apply(Map{wave[i][c].x, wave[i][c].y}, g);
        }
        h = apply(before, h);
#pragma unroll
        for (int j = 0; j < TP; ++j) {
            const int i = i0 + j;
            if (j < per && i < tiles) p.start[int64_t(back ? tiles - 1 - i : i) * p.C + ch] = h;
            h = apply(v[j], h);
        }
        h = g;
        __syncthreads();
    }
}

// The state that strip k of a tile starts from, after k_lr_reduce.
template <bool BACK>
__device__ __forceinline__ f32x4_t start_of(const LrArgs& p, int tile, const Strip& k) {
    f32x4_t h = 0.f;
    const auto through = [&](const float2* q) {
        const f32x4_t u = ld4(&q->x), v = ld4(&q[2].x);
        h = f32x4_t{apply(Map{u[0], u[1]}, h[0]), apply(Map{u[2], u[3]}, h[1]), apply(Map{v[0], v[1]}, h[2]), apply(Map{v[2], v[3]}, h[3])};
    };
    if (p.k.tiles > FEW) {
        h = ld4(p.start + int64_t(tile) * p.C + k.c);
    } else {
#pragma unroll 2
        for (int i = BACK ? p.k.tiles - 1 : 0; i != tile; i += BACK ? -1 : 1) through(p.tile + int64_t(i) * p.C + k.c);
    }
    through(p.strip + int64_t(tile * p.k.NCH + k.ch) * p.C + k.c);
    return h;
}

// The samples without rows pass their state on.
__device__ __forceinline__ void pass_empty(const LrArgs& p, const float* from, float* to) {
    if (!to) return;
    for (int64_t s = int64_t(blockIdx.x) * NT + threadIdx.x; s < p.segs.n_seg; s += int64_t(gridDim.x) * NT)
        if (p.segs.at(int(s)) >= p.segs.at(int(s) + 1))
            for (int c = 0; c < p.C; c += 4) st4(to + s * p.C + c, from ? ld4(from + s * p.C + c) : f32x4_t{0, 0, 0, 0});
}
__global__ __launch_bounds__(NT) void k_lr_empty(LrArgs p, const float* from, float* to) { pass_empty(p, from, to); }

// The walk takes the tiles from the last to the first: what the reduction read
// last is still in the cache (1 to 4% on 122 to 977 MiB of gates and values,
// nothing on less).
__device__ __forceinline__ void walk_tile(const LrArgs& p, int& tile, int& slab) {
    const int turn = int(blockIdx.x) / p.k.nslab;
    tile = p.k.tiles - 1 - turn;
    slab = int(blockIdx.x) - turn * p.k.nslab;
}

// ONE: a single tile, whose strips are reduced and joined here.
template <typename TT, bool ORDERED, bool ONE>
__global__ __launch_bounds__(NT, TT::E == 8 ? 5 : 4) void k_lr_fwd(const void* __restrict__ gate, const void* __restrict__ x, LrArgs p,
                                                                          const float* __restrict__ h0, void* __restrict__ out_,
                                                                          float* __restrict__ h_last, float* __restrict__ carry) {
    typename TT::storage* out = static_cast<typename TT::storage*>(out_);
    __shared__ Shared sh;
    __shared__ float in[ONE ? NT * 4 : 4];
    int tile, slab;
    walk_tile(p, tile, slab);
    const Span span(p, tile);
    const Strip k(p, span, slab, false);
    const Window w = open_window(p, span);
    const bool marked = mark(p, sh, span, w);
    f32x4_t h = 0.f;
    Pair<TT, ORDERED> b;
    if constexpr (ONE) {   // L = T: the strip stays in registers
        f32x4_t A = 1.f, B = 0.f;
        if (k.on) {
            b.load(p, w, gate, x, p.ld, k.pos, k.c);
            b.rows.marks(sh, marked, k.i0);
            fold<TT, ORDERED, false>(b.rows, b.g, b.x, h0, p, sh, k, 0, A, B);
        }
        join(p, sh, k, A, B, [&](int i, int c, const Map& m) { in[i * p.k.CW + c] = apply(m, 0.f); }, [](int, const Map&) {});
        __syncthreads();
        if (k.on) h = ld4(&in[k.at]);
    } else if (k.on) {
        h = start_of<false>(p, tile, k);
    }
    if (k.on)
        for (int i = 0; i < (ONE ? T : p.k.L); i += T) {
            if (!ONE) {
                b.load(p, w, gate, x, p.ld, k.pos + i, k.c);
                b.rows.marks(sh, marked, k.i0 + i);
            }
            if (carry && k.pos + i < p.segs.n) st4(carry + int64_t((k.pos + i) / T) * p.C + k.c, h);
            const auto step = [&](int t) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    float a, na;
                    gates<TT>(elem<TT>(b.g[t], j), a, na);
                    h[j] = fmaf(a, h[j], na * elem<TT>(b.x[t], j));
                }
                str<TT>(out + int64_t(b.rows.r[t]) * p.C + k.c, h);
            };
            if (b.rows.simple) {
#pragma unroll
                for (int t = 0; t < T; ++t) step(t);
            } else {
#pragma unroll
                for (int t = 0; t < T; ++t) {
                    if (b.rows.first >> t & 1) h = state_of(h0, p, sh, k.i0 + i + t, k.c);
                    if (b.rows.r[t] >= 0) step(t);
                    if ((b.rows.last >> t & 1) && h_last) st4(h_last + int64_t(sh.sample[k.i0 + i + t]) * p.C + k.c, h);
                }
            }
        }
    pass_empty(p, h0, h_last);
}

// T rows of the backward's walk, and the state ahead of them.
template <typename TT, bool ORDERED>
struct Triple {
    Rows<ORDERED> rows;
    Raw4<TT> g[T], v[T], d[T];
    f32x4_t h;
    __device__ __forceinline__ void load(const LrArgs& p, const Window& w, const void* gate, const void* x, const void* dout,
                                         const float* carry, int pos, int c) {
        using S = typename TT::storage;
        rows.numbers(p, w, pos);
        h = ld4(carry + int64_t(pos / T) * p.C + c);
#pragma unroll
        for (int t = 0; t < T; ++t) {
            g[t] = ldr<TT>(static_cast<const S*>(gate) + rows.any(t) * p.ld + c);
            v[t] = ldr<TT>(static_cast<const S*>(x) + rows.any(t) * p.ld + c);
            d[t] = ldr<TT>(static_cast<const S*>(dout) + rows.any(t) * p.C + c);
        }
    }
};

// Keeps of every element the gate and h_{t-1} - x_t in fp32 between the way
// ahead through T rows and the way back, which sets its registers: 153, three
// waves to a SIMD (four would spill).
template <typename TT, bool ORDERED, bool ONE>
__global__ __launch_bounds__(NT, TT::E == 8 ? 3 : 2) void k_lr_bwd(const void* __restrict__ dout, const void* __restrict__ gate,
                                               const void* __restrict__ x, LrArgs p, const float* __restrict__ h0,
                                               const float* __restrict__ carry, const float* __restrict__ dh_last,
                                               void* __restrict__ dgate_, void* __restrict__ dx_, float* __restrict__ dh0) {
    using S = typename TT::storage;
    S *dgate = static_cast<S*>(dgate_), *dx = static_cast<S*>(dx_);
    __shared__ Shared sh;
    __shared__ float in[ONE ? NT * 4 : 4];
    int tile, slab;
    walk_tile(p, tile, slab);
    const Span span(p, tile);
    const Strip k(p, span, slab, true);
    const Window w = open_window(p, span);
    const bool marked = mark(p, sh, span, w);
    f32x4_t E = 0.f;
    Triple<TT, ORDERED> b;
    if constexpr (ONE) {
        f32x4_t A = 1.f, B = 0.f;
        if (k.on) {
            b.load(p, w, gate, x, dout, carry, k.pos, k.c);
            b.rows.marks(sh, marked, k.i0);
            fold<TT, ORDERED, true>(b.rows, b.g, b.d, dh_last, p, sh, k, 0, A, B);
        }
        join(p, sh, k, A, B, [&](int i, int c, const Map& m) { in[i * p.k.CW + c] = apply(m, 0.f); }, [](int, const Map&) {});
        __syncthreads();
        if (k.on) E = ld4(&in[k.at]);
    } else if (k.on) {
        E = start_of<true>(p, tile, k);
    }
    if (k.on)
        for (int i = ONE ? 0 : p.k.L - T; i >= 0; i -= T) {
            if (k.pos + i >= p.segs.n) continue;
            if (!ONE) {
                b.load(p, w, gate, x, dout, carry, k.pos + i, k.c);
                b.rows.marks(sh, marked, k.i0 + i);
            }
            const auto& rows = b.rows;
            f32x4_t h = b.h;
            f32x4_t a[T], u[T];   // the gates as kept, and h_{t-1} - x_t
#pragma unroll
            for (int t = 0; t < T; ++t) {
                if (!rows.simple && (rows.first >> t & 1)) h = state_of(h0, p, sh, k.i0 + i + t, k.c);
                const bool ok = rows.simple || rows.r[t] >= 0;
                float kept[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float xj = elem<TT>(b.v[t], j);
                    float aj, na;
                    kept[j] = keep<TT>(elem<TT>(b.g[t], j));
                    gates_of(kept[j], aj, na);
                    u[t][j] = h[j] - xj;
                    const float next = fmaf(aj, h[j], na * xj);
                    h[j] = ok ? next : h[j];
                }
                // the compiler would otherwise keep both gates of all elements, in twice the registers
#pragma unroll
                for (int j = 0; j < 4; ++j) hide(kept[j]);
                a[t] = f32x4_t{kept[0], kept[1], kept[2], kept[3]};
            }
#pragma unroll
            for (int t = T - 1; t >= 0; --t) {
                if (!rows.simple && (rows.last >> t & 1)) E = state_of(dh_last, p, sh, k.i0 + i + t, k.c);
                if (rows.simple || rows.r[t] >= 0) {
                    f32x4_t gx, gg;
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        float aj, na;
                        gates_of(a[t][j], aj, na);
                        const float D = elem<TT>(b.d[t], j) + E[j];
                        gx[j] = na * D;
                        E[j] = aj * D;
                        gg[j] = na * u[t][j] * E[j];
                    }
                    str<TT>(dx + int64_t(rows.r[t]) * p.ldg + k.c, gx);
                    str<TT>(dgate + int64_t(rows.r[t]) * p.ldg + k.c, gg);
                }
                if (!rows.simple && (rows.first >> t & 1) && dh0) st4(dh0 + int64_t(sh.sample[k.i0 + i + t]) * p.C + k.c, E);
            }
        }
    pass_empty(p, dh_last, dh0);
}

// One row of each of n running sequences: state is read, replaced and rounded
// to out.  Bound by its launch: 1.3 us for 7 x 64 bf16.
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
        gates<TT>(g[j], a, na);
        h[j] = a * h[j] + na * v[j];
    }
    st8<F32>(new_state + i, narrow<F32>(h));
    st8<TT>(static_cast<S*>(out) + i, narrow<TT>(h));
}

spc_status check_sizes(spc_dtype dtype, int64_t n, int32_t C, int64_t n_seg) {
    if (dtype != SPC_F32 && dtype != SPC_F16 && dtype != SPC_BF16) return fail(SPC_ERR_ARG, "unknown dtype %d", int(dtype));
    if (n < 0 || n >= ROWS_END) return fail(SPC_ERR_ARG, "n=%lld is out of range", (long long)n);
    if (n_seg < 1 || n_seg >= ROWS_END) return fail(SPC_ERR_ARG, "n_seg=%lld is out of range", (long long)n_seg);
    if (C <= 0 || C % 16) return fail(SPC_ERR_UNSUPPORTED, "C=%d: channels must be a positive multiple of 16", C);
    if (C > C_MAX) return fail(SPC_ERR_UNSUPPORTED, "C=%d: at most %d channels", C, C_MAX);
    const Cut k = cut_of(n, C);
    if (!launchable(int64_t(k.tiles) * k.nslab, NT))
        return fail(SPC_ERR_UNSUPPORTED, "%lld rows of %d channels exceed one launch", (long long)n, C);
    return SPC_OK;
}

// A row stride holds a whole row and keeps every row 16-byte aligned.
spc_status check_stride(spc_dtype dtype, int64_t ld, int32_t C, const char* name) {
    if (ld < C || (ld * dtype_size(dtype)) % 16 || ld >= (int64_t(1) << 31))
        return fail(SPC_ERR_ARG, "%s=%lld: a row stride is at least C=%d and a multiple of 16 bytes", name, (long long)ld, C);
    return SPC_OK;
}

// The states that the chunks start from.
size_t carry_bytes(int64_t n, int32_t C) { return size_t(ceil_div(n, T)) * C * 4; }
// The strips', the tiles' maps and the states that the tiles start from.
size_t ws_need(int64_t n, int32_t C) {
    const Cut k = cut_of(n, C);
    return k.tiles > 1 ? size_t(k.tiles) * C * (8 * size_t(k.NCH) + 8 + 4) : 16;
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
    if (ws_bytes < ws_need(n, C))
        return fail(SPC_ERR_WORKSPACE, "ws_bytes=%zu, need %zu", ws_bytes, ws_need(n, C));
    p.segs = Segs{seg_ptr, int32_t(n_seg), int32_t(n)};
    p.C = C, p.reverse = reverse != 0, p.ld = ld, p.ldg = C, p.order = order;
    p.k = cut_of(n, C);
    p.strip = static_cast<float2*>(ws);
    p.tile = p.strip + int64_t(p.k.tiles) * p.k.NCH * C;
    p.start = reinterpret_cast<float*>(p.tile + int64_t(p.k.tiles) * C);
    return SPC_OK;
}

// The launches of a scan: ahead of the walk, which is apply(one tile).
template <typename TT, bool ORDERED, bool BACK>
spc_status launch_reduce(const void* gate, const void* v, const LrArgs& p, const float* from, hipStream_t stream) {
    hipLaunchKernelGGL((k_lr_reduce<TT, ORDERED, BACK>), dim3(unsigned(p.k.tiles) * unsigned(p.k.nslab)), dim3(NT), 0, stream, gate, v,
                       p, from);
    SPC_LAUNCHED("k_lr_reduce");
    if (p.k.tiles > FEW) {
        hipLaunchKernelGGL(k_lr_tiles, dim3(unsigned(p.C / 4)), dim3(TN), 0, stream, p, BACK);
        SPC_LAUNCHED("k_lr_tiles");
    }
    return SPC_OK;
}

spc_status launch_empty(const LrArgs& p, const float* from, float* to, hipStream_t stream) {
    if (!to) return SPC_OK;
    const int64_t blocks = ceil_div(p.segs.n_seg, NT);
    hipLaunchKernelGGL(k_lr_empty, dim3(unsigned(blocks < 4096 ? blocks : 4096)), dim3(NT), 0, stream, p, from, to);
    SPC_LAUNCHED("k_lr_empty");
    return SPC_OK;
}

template <typename TT, bool ORDERED>
spc_status launch_fwd(const void* gate, const void* x, const LrArgs& p, const float* h0, void* out, float* h_last, float* carry,
                      hipStream_t stream) {
    const dim3 grid(unsigned(p.k.tiles) * unsigned(p.k.nslab));
    if (p.k.tiles == 1) {
        hipLaunchKernelGGL((k_lr_fwd<TT, ORDERED, true>), grid, dim3(NT), 0, stream, gate, x, p, h0, out, h_last, carry);
    } else {
        const spc_status st = launch_reduce<TT, ORDERED, false>(gate, x, p, h0, stream);
        if (st != SPC_OK) return st;
        hipLaunchKernelGGL((k_lr_fwd<TT, ORDERED, false>), grid, dim3(NT), 0, stream, gate, x, p, h0, out, h_last, carry);
    }
    SPC_LAUNCHED("k_lr_fwd");
    return SPC_OK;
}

template <typename TT, bool ORDERED>
spc_status launch_bwd(const void* dout, const void* gate, const void* x, const LrArgs& p, const float* h0, const float* carry,
                      const float* dh_last, void* dgate, void* dx, float* dh0, hipStream_t stream) {
    const dim3 grid(unsigned(p.k.tiles) * unsigned(p.k.nslab));
    if (p.k.tiles == 1) {
        hipLaunchKernelGGL((k_lr_bwd<TT, ORDERED, true>), grid, dim3(NT), 0, stream, dout, gate, x, p, h0, carry, dh_last, dgate, dx, dh0);
    } else {
        const spc_status st = launch_reduce<TT, ORDERED, true>(gate, dout, p, dh_last, stream);
        if (st != SPC_OK) return st;
        hipLaunchKernelGGL((k_lr_bwd<TT, ORDERED, false>), grid, dim3(NT), 0, stream, dout, gate, x, p, h0, carry, dh_last, dgate, dx, dh0);
    }
    SPC_LAUNCHED("k_lr_bwd");
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

#define LR_ORDERED(fn, ...)                                                                                        \
    switch (dtype) {                                                                                              \
        case SPC_F32: return order ? fn<F32, true>(__VA_ARGS__) : fn<F32, false>(__VA_ARGS__);                    \
        case SPC_F16: return order ? fn<F16, true>(__VA_ARGS__) : fn<F16, false>(__VA_ARGS__);                    \
        case SPC_BF16: return order ? fn<BF16, true>(__VA_ARGS__) : fn<BF16, false>(__VA_ARGS__);                 \
    }                                                                                                             \
    return fail(SPC_ERR_ARG, "unknown dtype %d", int(dtype))

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
    if (n == 0) return launch_empty(p, h0, h_last, stream);
    LR_ORDERED(launch_fwd, gate, x, p, h0, out, h_last, carry, stream);
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
    if (n == 0) return launch_empty(p, dh_last, dh0, stream);
    LR_ORDERED(launch_bwd, dout, gate, x, p, h0, carry, dh_last, dgate, dx, dh0, stream);
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
    if (!launchable(blocks, 256)) return fail(SPC_ERR_UNSUPPORTED, "%lld rows of %d channels exceed one launch", (long long)n, C);
    LR_DISPATCH(k_lr_step, dim3(unsigned(blocks)), dim3(256), gate, x, ld, n, C, state, new_state, out);
    return SPC_OK;
}
