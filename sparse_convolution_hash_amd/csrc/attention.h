// Attention over ragged samples: the kernels, compiled per dtype in
// attention_{f32,f16,bf16}.hip; entry points and launch rules in attention.hip.
//
//   forward    s_ij = scale q_i . k_j,  p = softmax_j s,  o_i = sum_j p_ij v_j
//   backward   p_ij = 2^(c q_i . k_j - m_i) / l_i from the forward's m and l,
//              ds_ij = p_ij (do_i . v_j - do_i . o_i),
//              dq_i = scale sum_j ds_ij k_j,  dk_j = scale sum_i ds_ij q_i,
//              dv_j = sum_i p_ij do_i
//
// Scores never leave the registers.  A wave owns 32 columns (queries, or keys
// in k_attn_dkv) and walks the other side in tiles that its workgroup stages
// in LDS.  v_mfma_f32_32x32 gives a tile of scores with its column in lane % 32
// and 16 rows in registers, so a column's maximum and sum cost one exchange
// between the wave's halves, its rescaling no exchange at all, and the tile is
// at once the right operand of the second product: the contraction may run
// over the rows in the order in which the registers hold them, as long as the
// left operand comes in the same one, and the transposing LDS read
// (ds_read_b64_tr_b16) gives it so from rows as they were stored.
//
// Windows of 1,024 on 266,426 x 4 x 32 bf16, where the exponentials and the
// packing keep the vector unit busy and not memory: forward 315 us (140 GFLOP
// in the two products, 440 TFLOP/s), backward 850 (k_attn_dq three products, 210
// GFLOP, k_attn_dkv four, 279 GFLOP; 353, 487 and 526 us under the tracer).  Causal
// 16,411 x 8 heads over 2 x 128 bf16: forward 720 us, 552 GFLOP, 770 TFLOP/s (matrix
// unit busy for 32% of its cycles, vector unit for 45%, two waves a SIMD to cover
// each other's waits).  fp32, 5,003 x 6 x 48 ragged and causal: 129, 154 and 246
// us, one wave a SIMD, the matrix unit busy for half of its cycles.
#pragma once

#include <type_traits>

#include "rows.h"

namespace spc {
namespace attn {

typedef float f32x16_t __attribute__((ext_vector_type(16)));
typedef short i16x4_t __attribute__((ext_vector_type(4)));

struct Args {
    const char *q, *k, *v, *o, *dout;       // o: the forward's output, read by the backward
    char *out, *dq, *dk, *dv;
    char* rest;                             // [n_q, heads, D], what rounding left of the output (NULL: not kept)
    int64_t ldq, ldk, ldv, ldo, lddo, lddq, lddk, lddv;   // bytes between rows
    const int32_t *q_order, *kv_order;
    Segs qs, ks;
    int32_t g, hk, D, causal;               // query heads to a key head, key heads, head dimension
    uint32_t inv_g;                         // 2^32 / g, rounded up (g > 1)
    float c, scale;                         // c = scale log2(e)
    float2* stats;                          // [heads, n_q] (m, l)
    float* delta;                           // [heads, n_q] do . o
    float* part;                            // partial results of the splits
    int32_t splits, slots;
    unsigned group, total;                  // workgroups that an XCD takes in a row, of all
};

__device__ __forceinline__ f32x16_t all16(float v) {
    f32x16_t z;
#pragma unroll
    for (int r = 0; r < 16; ++r) z[r] = v;
    return z;
}
__device__ __forceinline__ f32x16_t zero16() { return all16(0.f); }

// One 32x32 tile step over 32 bytes of contraction: lane l supplies row
// (column) l % 32 and the 16 bytes of half l / 32.
template <typename TT>
__device__ __forceinline__ f32x16_t mfma32(const u32x4& a, const u32x4& b, f32x16_t c);
template <>
__device__ __forceinline__ f32x16_t mfma32<BF16>(const u32x4& a, const u32x4& b, f32x16_t c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8_t, a), __builtin_bit_cast(bf16x8_t, b), c, 0, 0, 0);
}
template <>
__device__ __forceinline__ f32x16_t mfma32<F16>(const u32x4& a, const u32x4& b, f32x16_t c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8_t, a), __builtin_bit_cast(f16x8_t, b), c, 0, 0, 0);
}
template <>
__device__ __forceinline__ f32x16_t mfma32<F32>(const u32x4& a, const u32x4& b, f32x16_t c) {
    const float fa[4] = {__uint_as_float(a.x), __uint_as_float(a.y), __uint_as_float(a.z), __uint_as_float(a.w)};
    const float fb[4] = {__uint_as_float(b.x), __uint_as_float(b.y), __uint_as_float(b.z), __uint_as_float(b.w)};
#pragma unroll
    for (int i = 0; i < 4; ++i) c = __builtin_amdgcn_mfma_f32_32x32x2f32(fa[i], fb[i], c, 0, 0, 0);
    return c;
}

// The value of the wave's other half, next to this one's.
__device__ __forceinline__ float2 halves(float v) {
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return float2{__uint_as_float(r[0]), __uint_as_float(r[1])};
}
__device__ __forceinline__ float sum_halves(float v) {
    const float2 t = halves(v);
    return t.x + t.y;
}

__device__ __forceinline__ float exp2_(float v) { return __builtin_amdgcn_exp2f(v); }

// Four results of one row, rounded once and stored.
template <typename TT>
__device__ __forceinline__ void put4(char* p, f32x4_t v) {
    if constexpr (TT::id == SPC_BF16) {
        typedef __bf16 b4 __attribute__((ext_vector_type(4)));
        *reinterpret_cast<uint2*>(p) = __builtin_bit_cast(uint2, __builtin_convertvector(v, b4));
    } else if constexpr (TT::id == SPC_F16) {
        typedef _Float16 h4 __attribute__((ext_vector_type(4)));
        *reinterpret_cast<uint2*>(p) = __builtin_bit_cast(uint2, __builtin_convertvector(v, h4));
    } else {
        *reinterpret_cast<f32x4_t*>(p) = v;
    }
}

// What that rounding left of v, to be rounded itself; times 2^11 for fp16, where
// it comes to at most v and does not end among the type's smallest numbers.
template <typename TT>
constexpr float REST_UP = TT::id == SPC_F16 ? 2048.f : 1.f;
template <typename TT>
__device__ __forceinline__ f32x4_t left_of(f32x4_t v) {
    if constexpr (TT::id == SPC_BF16) {
        typedef __bf16 b4 __attribute__((ext_vector_type(4)));
        return v - __builtin_convertvector(__builtin_convertvector(v, b4), f32x4_t);
    } else if constexpr (TT::id == SPC_F16) {
        typedef _Float16 h4 __attribute__((ext_vector_type(4)));
        return (v - __builtin_convertvector(__builtin_convertvector(v, h4), f32x4_t)) * REST_UP<TT>;
    } else {
        return f32x4_t{0.f, 0.f, 0.f, 0.f};
    }
}

// Row of a tile register: register r of a lane in half h holds row
// 8 (r / 4) + 4 h + r % 4; bit_of(r) is the row of h = 0.
constexpr int bit_of(int r) { return 8 * (r / 4) + r % 4; }

// Tile of `rows` rows of DP elements in LDS, in 16-byte chunks.  The chunk
// number is XORed with bits of the row so that what one access takes lies spread
// over 128 bytes of banks: 8 consecutive rows of one chunk (row reads), and two
// chunks of 4 consecutive rows (transposing reads).  M chunks a row: rows repeat
// their banks every 1, 2 or 4 rows when M is a multiple of 8, 4 or 2.  The banks
// are 256 bytes wide, and the counters still show conflicts, of LDS's busy cycles
// 40% in the forward of 128 elements, 25, 33 and 17% in the forward, k_attn_dq and
// k_attn_dkv of 32 (bf16), 11 to 19% for fp32.
template <typename TT, int DP>
struct Tile {
    static constexpr int ES = sizeof(typename TT::storage);
    static constexpr int PITCH = DP * ES, M = PITCH / 16;
    static constexpr int NS = PITCH / 32;                 // steps of a product over DP
    static constexpr int NB = (DP + 31) / 32;             // 32-row blocks of a result over DP
    static __device__ __forceinline__ int swz(int row) {
        if constexpr (M % 8 == 0) return ((row & 3) << 1) | ((row >> 2) & 1);
        else if constexpr (M % 4 == 0) return (row & 2) | ((row >> 2) & 1);
        else return (row >> 2) & 1;
    }
    static __device__ __forceinline__ int at(int row, int chunk) { return row * PITCH + ((chunk ^ swz(row)) << 4); }
    static __device__ __forceinline__ u32x4 row16(const char* t, int row, int chunk) { return ld16(t + at(row, chunk)); }
};

// ------------------------------------------------- second kind of product

// acc[db][rows d, cols] += sum over the tile's 32 rows j of X[j][d] w[j][col],
// X a tile in LDS, w in the registers as a score tile is.
template <typename TT, int DP>
struct Second {
    using T = Tile<TT, DP>;
    static constexpr int STEPS = TT::E == 8 ? 2 : 16;     // contraction steps of a 32-row tile
    static constexpr int PER = 16 / STEPS;                // registers (rows of each half) to a step

    // Left operand of step t, block db: PER elements of this lane's d.
    static __device__ __forceinline__ u32x4 left(const char* x, int row0, int t, int db, int lane) {
        u32x4 f = zero4();
        const bool narrow_block = DP % 32 != 0 && db == T::NB - 1;     // 16 of 32 rows exist; the others repeat them
        if constexpr (TT::E == 8) {
            const int i = lane & 15, h = lane >> 5, odd = narrow_block ? 0 : (lane >> 4) & 1;
            const int row = row0 + 16 * t + 4 * h + (i >> 2);
            const int chunk = 4 * db + 2 * odd + ((i >> 1) & 1);
            const i16x4_t a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) i16x4_t*)(x + T::at(row, chunk) + 8 * (i & 1)));
            const i16x4_t b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) i16x4_t*)(x + T::at(row + 8, chunk) + 8 * (i & 1)));
            const uint2 ua = __builtin_bit_cast(uint2, a), ub = __builtin_bit_cast(uint2, b);
            f = u32x4{ua.x, ua.y, ub.x, ub.y};
        } else {
            const int h = lane >> 5, d = 32 * db + (narrow_block ? lane & 15 : lane & 31);
            f.x = *reinterpret_cast<const uint32_t*>(x + T::at(row0 + bit_of(t) + 4 * h, d >> 2) + 4 * (d & 3));
        }
        return f;
    }

    static __device__ __forceinline__ u32x4 pack(const float* w) {
        u32x4 f = zero4();
        if constexpr (TT::E == 8) {
            f32x8_t v;
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = w[e];
            f = narrow<TT>(v).v[0];
        } else {
            f.x = __float_as_uint(w[0]);
        }
        return f;
    }

    static __device__ __forceinline__ f32x16_t step(const u32x4& a, const u32x4& b, f32x16_t c) {
        if constexpr (TT::E == 8) return mfma32<TT>(a, b, c);
        else return __builtin_amdgcn_mfma_f32_32x32x2f32(__uint_as_float(a.x), __uint_as_float(b.x), c, 0, 0, 0);
    }

    // The weights as the right operands of all steps, rounded to the type.
    struct Packed {
        u32x4 b[STEPS];
        __device__ __forceinline__ Packed() {}
        __device__ __forceinline__ explicit Packed(const f32x16_t& w) {
#pragma unroll
            for (int t = 0; t < STEPS; ++t) {
                float wt[PER];
#pragma unroll
                for (int e = 0; e < PER; ++e) wt[e] = w[t * PER + e];
                b[t] = pack(wt);
            }
        }
    };

    // As sums of two numbers of the type, for twice the products: for dq of
    // narrow heads, whose matrix unit has room for it (ds sums to 0 over a row, so
    // its rounding counts for more than that of p: windows of 1,024 on 266,426 x 4
    // x 32 bf16 trained in 1,170 us with a relative error of dq below 2.4e-3, in
    // 1,095 us with 2.6e-3 where ds is rounded once), and for the forward's p
    // where few rows meet many keys.
    struct Two {
        Packed hi, lo;
        __device__ __forceinline__ Two() {}
        __device__ __forceinline__ explicit Two(const f32x16_t& w) : hi(w) {
#pragma unroll
            for (int t = 0; t < STEPS; ++t) {
                Raw8<TT> r;
                r.v[0] = hi.b[t];
                const f32x8_t f = widen<TT>(r);
                f32x8_t v;
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] = w[t * PER + e] - f[e];
                lo.b[t] = narrow<TT>(v).v[0];
            }
        }
    };

    static __device__ __forceinline__ f32x16_t step(const u32x4& a, const Packed& w, int t, f32x16_t c) { return step(a, w.b[t], c); }
    static __device__ __forceinline__ f32x16_t step(const u32x4& a, const Two& w, int t, f32x16_t c) {
        return step(a, w.lo.b[t], step(a, w.hi.b[t], c));
    }

    template <typename W>
    static __device__ __forceinline__ void add(f32x16_t (&acc)[T::NB], const char* x, int row0, const W& w, int lane) {
#pragma unroll
        for (int t = 0; t < STEPS; ++t)
#pragma unroll
            for (int db = 0; db < T::NB; ++db) acc[db] = step(left(x, row0, t, db, lane), w, t, acc[db]);
    }

    // The finite elements of a left operand, the others 0.
    static __device__ __forceinline__ u32x4 finite(const u32x4& a) {
        uint32_t w[4] = {a.x, a.y, a.z, a.w};
        if constexpr (TT::E == 4) {
            w[0] = (w[0] & 0x7f800000u) == 0x7f800000u ? 0u : w[0];
        } else {
            constexpr uint32_t INF = TT::id == SPC_BF16 ? 0x7f80u : 0x7c00u;
#pragma unroll
            for (int i = 0; i < 4; ++i) w[i] &= ((w[i] & INF) == INF ? 0u : 0xffffu) | ((w[i] >> 16 & INF) == INF ? 0u : 0xffff0000u);
        }
        return u32x4{w[0], w[1], w[2], w[3]};
    }
    // Elements that are infinity (kind 0), minus infinity (1) or NaN (2), as 1.
    static __device__ __forceinline__ u32x4 only(const u32x4& a, int kind) {
        uint32_t w[4] = {a.x, a.y, a.z, a.w};
        constexpr bool W = TT::E == 4;
        constexpr uint32_t INF = W ? 0x7f800000u : TT::id == SPC_BF16 ? 0x7f80u : 0x7c00u;
        constexpr uint32_t ONE = W ? 0x3f800000u : TT::id == SPC_BF16 ? 0x3f80u : 0x3c00u;
        constexpr uint32_t SIGN = W ? 0x80000000u : 0x8000u;
        auto one = [&](uint32_t u) { return (kind == 2 ? (u & (SIGN - 1)) > INF : u == (kind ? INF | SIGN : INF)) ? ONE : 0u; };
#pragma unroll
        for (int i = 0; i < (W ? 1 : 4); ++i) w[i] = W ? one(w[i]) : one(w[i] & 0xffffu) | one(w[i] >> 16) << 16;
        return u32x4{w[0], w[1], w[2], w[3]};
    }

    // The same where a mask hides pairs (bit bit_of(r) of vis is 0, and w is 0).
    // Hidden pairs are not in the sum, so an infinite or NaN X[j][d] must not
    // reach the columns that do not see row j, as 0 * inf would: the finite
    // values are summed.  With OTHERS (w are probabilities, positive), an
    // infinite or NaN value reaches the columns that see its row: counted
    // apart.  Without, it has made w itself NaN in those columns.
    template <bool OTHERS, typename W>
    static __device__ __forceinline__ void add_masked(f32x16_t (&acc)[T::NB], const char* x, int row0, const W& w,
                                                      uint32_t vis, int lane) {
        bool odd = false;
#pragma unroll
        for (int t = 0; t < STEPS; ++t) {
#pragma unroll
            for (int db = 0; db < T::NB; ++db) {
                const u32x4 a = left(x, row0, t, db, lane), f = finite(a);
                if constexpr (OTHERS) odd |= a.x != f.x || a.y != f.y || a.z != f.z || a.w != f.w;
                acc[db] = step(f, w, t, acc[db]);
            }
        }
        if constexpr (OTHERS) {
            if (!__any(odd)) return;
#pragma unroll
            for (int db = 0; db < T::NB; ++db)
#pragma unroll 1
                for (int kind = 0; kind < 3; ++kind) {
                    asm volatile("" : "+v"(lane), "+v"(vis));      // nothing of this part is computed ahead of it
                    f32x16_t n = zero16();
#pragma unroll
                    for (int t = 0; t < STEPS; ++t) {
                        float see[PER];
#pragma unroll
                        for (int e = 0; e < PER; ++e) see[e] = (vis >> bit_of(t * PER + e)) & 1u ? 1.f : 0.f;
                        n = step(only(left(x, row0, t, db, lane), kind), pack(see), n);
                    }
                    const float v = kind == 0 ? INFINITY : kind == 1 ? -INFINITY : NAN;
#pragma unroll
                    for (int r = 0; r < 16; ++r) acc[db][r] += n[r] > 0.f ? v : 0.f;
                }
        }
    }
};

// ------------------------------------------------------------------ jobs

// A workgroup's part: rows [r0, r0 + BM) of one sample, counted over the
// positions and, for queries, the heads that share keys (row = position * mult
// + head).  Sample s owns the slots from floor(at(s) mult / BM) + s on, at
// least as many as it has tiles, so no table of tiles is needed; the slots left
// over end at once.  Workgroups go round the 8 XCDs in launch order: an XCD
// takes groups of neighbours in (split, slot, head), which read the same keys
// through its L2, and the groups go round the XCDs, so that long samples, and
// the late rows of a causal one, spread over all of them.
struct Job {
    int s, head, split, r0, a, len;    // sample, key head, split, first row, first position of the sample, its positions
};

template <int BM>
__device__ __forceinline__ bool job_of(const Args& p, const Segs& segs, int mult, bool reverse, Job& j) {
    const unsigned x = blockIdx.x & 7u, i = blockIdx.x >> 3;
    unsigned l = (i / p.group * 8u + x) * p.group + i % p.group;
    if (l >= p.total) return false;
    j.head = int(l % unsigned(p.hk));
    l /= unsigned(p.hk);
    int slot = int(l % unsigned(p.slots));
    j.split = int(l / unsigned(p.slots));
    if (reverse) slot = p.slots - 1 - slot;
    const int lane = int(threadIdx.x) & (WAVE - 1);
    auto first = [&](int s) { return int(unsigned(segs.at(s)) * unsigned(mult) / unsigned(BM)) + s; };
    int lo = 0, hi = segs.n_seg;       // the count of samples that begin at or before the slot is in [lo, hi]
    while (lo < hi) {
        const int step = (hi - lo + WAVE - 1) / WAVE;
        const int t = lo + lane * step;
        const int k = __popcll(__ballot(t < hi && first(t < hi ? t : lo) <= slot));
        if (k == 0) break;
        if (step == 1) {
            lo += k;
            break;
        }
        const int nlo = lo + (k - 1) * step + 1, nhi = lo + k * step;
        lo = nlo;
        hi = nhi < hi ? nhi : hi;
    }
    j.s = lo > 0 ? lo - 1 : 0;
    j.s = __builtin_amdgcn_readfirstlane(j.s);
    j.a = __builtin_amdgcn_readfirstlane(segs.at(j.s));
    const int b = __builtin_amdgcn_readfirstlane(segs.at(j.s + 1));
    j.len = b > j.a ? b - j.a : 0;
    const int t = slot - (int(unsigned(j.a) * unsigned(mult) / unsigned(BM)) + j.s);
    if (t < 0 || int64_t(t) * BM >= int64_t(j.len) * mult) return false;
    j.r0 = t * BM;
    return true;
}

// Position pos of a sample that begins at a: its row, or -1 where an order
// names none.
__device__ __forceinline__ int row_of(const int32_t* order, int a, int pos, int n) {
    const int r = order ? order[a + pos] : a + pos;
    return r >= 0 && r < n ? r : -1;
}

// A query of the walk: row index rq counts (position, head within its group).
struct Query {
    int pos, head, row;      // row -1: there is none
};
__device__ __forceinline__ Query place_of(const Args& p, const Job& j, int rq) {
    Query q{rq, j.head, -1};
    if (p.g > 1) {
        // rq times the rounded-up 2^32 / g: the quotient, or one more
        q.pos = int(__umulhi(unsigned(rq), p.inv_g));
        q.pos -= unsigned(q.pos) * unsigned(p.g) > unsigned(rq);
        q.head = j.head * p.g + (rq - q.pos * p.g);
    }
    return q;
}
__device__ __forceinline__ Query query_of(const Args& p, const Job& j, int qa, int rq, int rows) {
    Query q = place_of(p, j, rq);
    if (rq < rows) q.row = row_of(p.q_order, qa, q.pos, p.qs.n);
    return q;
}

// Bits of the first cnt of 64 rows.
__device__ __forceinline__ uint64_t first_bits(int cnt) { return cnt >= 64 ? ~0ull : cnt <= 0 ? 0ull : (1ull << cnt) - 1; }

// Fragments of one row of DP elements (zeros past D, or for no row), as the
// column operand of the first product.
template <typename TT, int DP>
__device__ __forceinline__ void load_frags(u32x4* f, const char* row, bool there, int D, int h) {
    using T = Tile<TT, DP>;
#pragma unroll
    for (int s = 0; s < T::NS; ++s) f[s] = there && (2 * s + h) * 16 < D * T::ES ? ld16(row + (2 * s + h) * 16) : zero4();
}

// Narrow heads of 16-bit types spend their time in the vector unit, a score's
// multiplication by c and subtraction of m among it, and leave the matrix unit
// idle.  For bf16 the column operand is multiplied by c once, kept as the sum of
// two numbers of the type (off by 2^-18 of itself), and the product starts from
// -m, so that the matrix unit hands over the exponent itself.  Wider heads would
// pay more in the matrix unit (a second product over DP) than they save: 64
// cycles for DP / 16 products of 32 on each tile.  fp16 has not the range: the
// second number is below its smallest, 2^-24, as soon as the factor is below
// 2^-3, and the product above its largest where c is above 1.
// An infinite key meets both numbers, and inf - inf is NaN where the plain
// product gives minus infinity.
template <typename TT, int DP>
constexpr bool SPLIT = TT::id == SPC_BF16 && DP <= 32;

// Where dq takes ds as two numbers of the type.
template <typename TT, int DP>
constexpr bool TWO_DS = TT::E == 8 && DP <= 32;

// f times c as f + lo (lo has entries where the product is split).
template <typename TT, int DP>
__device__ __forceinline__ void split_frags(u32x4* f, u32x4* lo, float c) {
    if constexpr (SPLIT<TT, DP>) {
#pragma unroll
        for (int s = 0; s < Tile<TT, DP>::NS; ++s) {
            Raw8<TT> x;
            x.v[0] = f[s];
            const f32x8_t t = widen<TT>(x) * c;
            x = narrow<TT>(t);
            f[s] = x.v[0];
            lo[s] = narrow<TT>(t - widen<TT>(x)).v[0];
        }
    }
}

// Staging of tiles of BN rows from two tensors: what a thread moves.
template <typename TT, int DP, int BN, int NT>
struct Stage {
    using T = Tile<TT, DP>;
    static constexpr int CH = BN * T::M, PT = (CH + NT - 1) / NT;
    static __device__ __forceinline__ bool mine(int i) { return CH % NT == 0 || int(threadIdx.x) + i * NT < CH; }
    static __device__ __forceinline__ int row(int i) { return (int(threadIdx.x) + i * NT) / T::M; }
    static __device__ __forceinline__ int chunk(int i) { return (int(threadIdx.x) + i * NT) % T::M; }

    u32x4 ra[PT], rb[PT];
    bool whole;          // every element of the tile is there (the same for all threads)
    uint32_t there;      // bit i: this thread's part i is

    // Rows that lie ld bytes apart from `a` and `b` on, the first cnt > 0 of
    // them there, `width` bytes of each.  Loads are unconditional, so that
    // nothing waits for them before put(): absent parts load a part that is
    // there, and put() writes zeros for them.
    __device__ __forceinline__ void load(const char* a, int64_t lda, const char* b, int64_t ldb, int cnt, int width) {
        whole = cnt >= BN && width == T::PITCH;
        there = ~0u;
        int64_t oa[PT], ob[PT];
#pragma unroll
        for (int i = 0; i < PT; ++i) oa[i] = row(i) * lda + chunk(i) * 16, ob[i] = row(i) * ldb + chunk(i) * 16;
        if (!whole) {
            there = 0;
#pragma unroll
            for (int i = 0; i < PT; ++i) {
                const int r = row(i) < cnt ? row(i) : cnt - 1, c = chunk(i) * 16 < width ? chunk(i) * 16 : 0;
                there |= uint32_t(row(i) < cnt && chunk(i) * 16 < width) << i;
                oa[i] = r * lda + c, ob[i] = r * ldb + c;
            }
        }
#pragma unroll
        for (int i = 0; i < PT; ++i)
            if (mine(i)) ra[i] = ld16(a + oa[i]), rb[i] = ld16(b + ob[i]);
    }
    // Part i of this thread from the row at `a` and `b` plus the offsets; call
    // begin_parts() first.
    __device__ __forceinline__ void begin_parts() { whole = false, there = 0; }
    __device__ __forceinline__ void load_part(int i, bool is, const char* a, const char* b, int width) {
        const bool in = chunk(i) * 16 < width;
        there |= uint32_t(is && in) << i;
        const int c = in ? chunk(i) * 16 : 0;
        if (mine(i)) ra[i] = ld16(a + c), rb[i] = ld16(b + c);
    }
    __device__ __forceinline__ void put(char* ta, char* tb) {
        if (!whole) {
#pragma unroll
            for (int i = 0; i < PT; ++i)
                if (!((there >> i) & 1u)) ra[i] = zero4(), rb[i] = zero4();
        }
#pragma unroll
        for (int i = 0; i < PT; ++i)
            if (mine(i)) {
                st16(ta + T::at(row(i), chunk(i)), ra[i]);
                st16(tb + T::at(row(i), chunk(i)), rb[i]);
            }
    }
};

// Keys of a sample, tile by tile: rows in place come from one base; entries of
// an order are read one tile ahead of the rows that they name, and looked at
// when those are fetched.
template <typename TT, int DP, int BN, int NT>
struct KeyStage : Stage<TT, DP, BN, NT> {
    using S = Stage<TT, DP, BN, NT>;
    const char *k, *v;
    int ka, lk, width;
    int at[S::PT], mark;
    uint64_t live;           // keys of the fetched tile that are there, as bits

    __device__ __forceinline__ void begin(const Args& p, const Job& j, int a, int len) {
        width = p.D * S::T::ES;
        const int64_t in = int64_t(j.head) * width;
        k = p.k + in, v = p.v + in;
        ka = a, lk = len;
    }
    __device__ __forceinline__ void find(const Args& p, int t) {
        if (!p.kv_order) return;
        const int32_t* o = p.kv_order + ka;
        mark = o[min(t * BN + (int(threadIdx.x) & (WAVE - 1)), lk - 1)];
#pragma unroll
        for (int i = 0; i < S::PT; ++i) at[i] = o[min(t * BN + S::row(i), lk - 1)];
    }
    __device__ __forceinline__ void fetch(const Args& p, int t) {
        const int cnt = lk - t * BN;
        if (!p.kv_order) {
            const int64_t row = ka + t * BN;
            live = first_bits(cnt < BN ? cnt : BN);
            S::load(k + row * p.ldk, p.ldk, v + row * p.ldv, p.ldv, cnt, width);
        } else {
            const int l = int(threadIdx.x) & (WAVE - 1);
            live = __ballot(l < BN && l < cnt && unsigned(mark) < unsigned(p.ks.n));
            S::begin_parts();
#pragma unroll
            for (int i = 0; i < S::PT; ++i) {
                const bool is = S::row(i) < cnt && unsigned(at[i]) < unsigned(p.ks.n);
                const int64_t r = is ? at[i] : 0;
                S::load_part(i, is, k + r * p.ldk, v + r * p.ldv, width);
            }
        }
    }
};

// ----------------------------------------------------------- forward

// 32-key blocks of a staged tile: 64 keys for the wide workgroups of 16-bit
// types, 32 else (LDS and registers of the staging).
template <typename TT, int NW>
constexpr int KT_OF = TT::E == 8 && NW > 1 ? 2 : 1;

// The forward's: workgroups of four waves take 2 up to heads of 96, and of 128
// where nothing is masked (one sample of 16,384 x 8 x 128: 1,270 us with 2, 1,311
// with 1; windows of 1,024 on 100,000 x 2 x 128: 196 and 222; causal 16,411 x 8
// over 2 x 128 spills with 2: 1,064 and 737; causal 30,000 x 8 x 96 in 20 ragged
// samples: 471 and 603, without the mask 829 and 789; windows of 1,024 on 60,000 x
// 4 x 80: 180 and 185, causal 136 and 173).
template <typename TT, int DP, int NW, bool CAUSAL>
constexpr int KT_FWD = DP <= 64 || (NW == 4 && (DP <= 96 || !CAUSAL)) ? KT_OF<TT, NW> : 1;

// Waves that a SIMD is to hold at least, which bounds the registers.  Most kernels
// fit without spills; k_attn_dkv of causal 16-bit heads, and their forward of 128 in
// two waves, keep up to 40 registers in scratch, fp32's k_attn_dkv of heads from 96
// on up to 185 at one wave already.
template <typename TT, int DP, bool CAUSAL>
constexpr int FWD_WAVES = TT::E == 4 ? 1 : DP <= 32 ? 4 - CAUSAL : DP <= 64 ? 3 - CAUSAL : 2;
template <typename TT, int DP>
constexpr int BWD_WAVES = TT::E == 4 ? 1 : DP <= 32 ? 3 : DP <= 64 ? 2 : 1;

// Probabilities that are rounded to fp16 are held times a power of two, since
// below 2^-14 the type keeps no more than its smallest number, 2^-24: where a key
// outweighs many others by 2^20, their sum was off by 1%.  The forward's (relative
// to a maximum that may be LAZY below the row's own) have 5 binades above it, the
// backward's, at most 1, have 15; sums (and l) carry the power along.
template <typename TT>
constexpr float FWD_UP = TT::id == SPC_F16 ? 5.f : 0.f;
template <typename TT>
constexpr float BWD_UP = TT::id == SPC_F16 ? 15.f : 0.f;

// The sum of a tile's probabilities (of half a column) from which a new maximum
// is taken: 1,024 times the maximum's own, below fp16's largest, 65,504, which a
// single one may not pass.
template <typename TT>
constexpr float LAZY = TT::id == SPC_F16 ? 32768.f : 1024.f;

// TWO: p as two numbers of the type.
template <typename TT, int DP, int NW, bool CAUSAL, bool TWO>
__device__ __forceinline__ void attn_fwd(const Args& p) {
    constexpr int BM = 32 * NW, KT = KT_FWD<TT, DP, NW, CAUSAL>, BN = 32 * KT, NT = 64 * NW;
    constexpr bool SP = SPLIT<TT, DP>;
    using T = Tile<TT, DP>;
    __shared__ __attribute__((aligned(16))) char lds[2][2][BN * T::PITCH];
    Job j;
    if (!job_of<BM>(p, p.qs, p.g, CAUSAL, j)) return;
    const int lane = int(threadIdx.x) & 63, wave = int(threadIdx.x) >> 6, h = lane >> 5, col = lane & 31;
    const int ka = __builtin_amdgcn_readfirstlane(p.ks.at(j.s)), kb = __builtin_amdgcn_readfirstlane(p.ks.at(j.s + 1));
    const int lk = kb > ka ? kb - ka : 0, rows = j.len * p.g, off = lk - j.len;
    const int rw = __builtin_amdgcn_readfirstlane(j.r0 + 32 * wave);          // the wave's first row
    const Query q = query_of(p, j, j.a, rw + col, rows);
    u32x4 qf[T::NS], ql[SP ? T::NS : 1];
    load_frags<TT, DP>(qf, p.q + int64_t(q.row) * p.ldq + int64_t(q.head) * p.D * T::ES, q.row >= 0, p.D, h);
    split_frags<TT, DP>(qf, ql, p.c);
    // keys that the workgroup's last row, the wave's first and its last see
    auto limit = [&](int r) { return !CAUSAL ? lk : max(0, min(lk, (r < rows ? r : rows - 1) / p.g + 1 + off)); };
    const int nk = limit(j.r0 + BM - 1), seen_first = rw < rows ? limit(rw) : 0, seen_last = rw < rows ? limit(rw + 31) : 0;
    const int mine = CAUSAL ? q.pos + 1 + off : lk;        // keys [0, mine) of this lane's query
    const int tiles = (nk + BN - 1) / BN, per = (tiles + p.splits - 1) / p.splits;
    const int t0 = j.split * per, t1 = min(tiles, t0 + per);

    KeyStage<TT, DP, BN, NT> stage;
    stage.begin(p, j, ka, lk);
    f32x16_t acc[T::NB], from = zero16();                  // from: -m for the split product
#pragma unroll
    for (int db = 0; db < T::NB; ++db) acc[db] = zero16();
    float m = -INFINITY, l = 0.f;                          // m in units of log2: p = 2^(c s - m)
    uint32_t seen = 0;

    if (t0 < t1) {
        stage.find(p, t0);
        stage.fetch(p, t0);
        if (t0 + 1 < t1) stage.find(p, t0 + 1);
        stage.put(lds[0][0], lds[0][1]);
    }
    lds_barrier();
    for (int t = t0; t < t1; ++t) {
        const int buf = (t - t0) & 1, p0 = t * BN;
        const bool more = t + 1 < t1;
        const uint64_t live = stage.live;
        if (more) {
            stage.fetch(p, t + 1);
            if (t + 2 < t1) stage.find(p, t + 2);
        }
        if (p0 < seen_last) {          // else none of the wave's rows sees the tile
            const char *kt = lds[buf][0], *vt = lds[buf][1];
            const bool edge = p0 + BN > seen_first || live != first_bits(BN);
            uint32_t vis[KT];
            if (edge) {
#pragma unroll
                for (int u = 0; u < KT; ++u) {
                    const int n = mine - (p0 + 32 * u);
                    vis[u] = (uint32_t(live >> (32 * u)) & uint32_t(first_bits(n < 32 ? n : 32))) >> (4 * h);
                    seen |= vis[u] & 0x0f0f0f0fu;
                }
            } else {
                seen = 1;
            }
            // Scores are exponentiated against the maximum so far.  Their sum
            // tells whether it still serves: where a column's part of the tile
            // sums to more than LAZY, the scores are computed once more (the
            // tile is still there) for a new maximum.  A column without one
            // (the first tile, or hidden keys and scores of minus infinity so
            // far, as a query with an infinity may have along the whole walk)
            // takes it before anything is exponentiated.  Columns next to such a
            // one may still need the second round.
            using X = Second<TT, DP>;
            f32x16_t s[KT];
            std::conditional_t<TWO, typename X::Two, typename X::Packed> w[KT];
            float sum = 0.f;
            bool fresh = __any(m == -INFINITY && l == 0.f), last = false;    // (l is NaN where a query is)
            for (;;) {
                int c = col;
                asm volatile("" : "+v"(c));    // the second round reads the tile again: nothing is kept for it
#pragma unroll
                for (int u = 0; u < KT; ++u) {
                    s[u] = SP ? from : zero16();
#pragma unroll
                    for (int st = 0; st < T::NS; ++st) {
                        const u32x4 a = T::row16(kt, 32 * u + c, 2 * st + h);
                        s[u] = mfma32<TT>(a, qf[st], s[u]);
                        if constexpr (SP) s[u] = mfma32<TT>(a, ql[st], s[u]);
                    }
                }
                if (edge) {
#pragma unroll
                    for (int u = 0; u < KT; ++u) {
                        asm volatile("" : "+v"(vis[u]));
#pragma unroll
                        for (int r = 0; r < 16; ++r) s[u][r] = (vis[u] >> bit_of(r)) & 1u ? s[u][r] : -INFINITY;
                    }
                }
                if (fresh) {
                    float top = s[0][0];
#pragma unroll
                    for (int u = 0; u < KT; ++u)
#pragma unroll
                        for (int r = 0; r < 16; ++r) top = fmaxf(top, s[u][r]);
                    const float2 both = halves(top), sums = halves(sum);
                    top = fmaxf(both.x, both.y);
                    // the other columns keep their sums to the bit
                    const bool none = m == -INFINITY, grew = top > -INFINITY && (none || sums.x > LAZY<TT> || sums.y > LAZY<TT>);
                    float a = 1.f;
                    if constexpr (SP) {    // s is c s - m already
                        const float d = grew ? top : 0.f;
                        a = !grew ? 1.f : none ? 0.f : exp2_(-top);
#pragma unroll
                        for (int u = 0; u < KT; ++u) s[u] -= d;
                        m = !grew ? m : none ? top : m + top;
                        from = all16(m == -INFINITY ? 0.f : -m);
                    } else if (grew) {
                        const float was = m;
                        m = top * p.c - FWD_UP<TT>;
                        a = none ? 0.f : exp2_(was - m);
                    }
                    l *= a;
#pragma unroll
                    for (int db = 0; db < T::NB; ++db) acc[db] *= a;
                }
                const float base = m == -INFINITY ? 0.f : m;
                float part[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int u = 0; u < KT; ++u) {
#pragma unroll
                    for (int r = 0; r < 16; ++r) {
                        s[u][r] = exp2_(SP ? s[u][r] : fmaf(s[u][r], p.c, -base));
                        part[r & 3] += s[u][r];
                    }
                    w[u] = std::remove_reference_t<decltype(w[u])>(s[u]);
                }
                sum = (part[0] + part[1]) + (part[2] + part[3]);
                if (last || !__any(sum > LAZY<TT>)) break;
                last = fresh = true;
            }
            l += sum;
#pragma unroll
            for (int u = 0; u < KT; ++u) {
                if (CAUSAL && edge) X::template add_masked<true>(acc, vt, 32 * u, w[u], vis[u], lane);
                else X::add(acc, vt, 32 * u, w[u], lane);
            }
        }
        if (more) stage.put(lds[buf ^ 1][0], lds[buf ^ 1][1]);
        lds_barrier();
    }
    l = sum_halves(l);
    seen |= uint32_t(__shfl_xor(int(seen), 32));
    if (q.row < 0) return;
    const int64_t id = int64_t(q.head) * p.qs.n + q.row;
    if (p.splits > 1) {
        float* part = p.part + (int64_t(j.split) * p.qs.n * (int64_t(p.g) * p.hk) + id) * (p.D + 4);
#pragma unroll
        for (int db = 0; db < T::NB; ++db)
#pragma unroll
            for (int b = 0; b < 4; ++b) {
                const int d = 32 * db + 8 * b + 4 * h;
                if (d < p.D) *reinterpret_cast<f32x4_t*>(part + d) = f32x4_t{acc[db][4 * b], acc[db][4 * b + 1], acc[db][4 * b + 2], acc[db][4 * b + 3]};
            }
        if (h == 0) *reinterpret_cast<f32x4_t*>(part + p.D) = f32x4_t{m, l, seen ? 1.f : 0.f, 0.f};
        return;
    }
    if (seen && l == 0.f) l = NAN;     // keys are seen, and every score is minus infinity
    const float inv = l == 0.f ? 0.f : 1.f / l;
    char* out = p.out + int64_t(q.row) * p.ldo + int64_t(q.head) * p.D * T::ES;
    char* rest = p.rest + (int64_t(q.row) * (int64_t(p.g) * p.hk) + q.head) * p.D * T::ES;
#pragma unroll
    for (int db = 0; db < T::NB; ++db)
#pragma unroll
        for (int b = 0; b < 4; ++b) {
            const int d = 32 * db + 8 * b + 4 * h;
            if (d >= p.D) continue;
            const f32x4_t o = f32x4_t{acc[db][4 * b], acc[db][4 * b + 1], acc[db][4 * b + 2], acc[db][4 * b + 3]} * inv;
            put4<TT>(out + d * T::ES, o);
            if (TT::E == 8 && p.rest) put4<TT>(rest + d * T::ES, left_of<TT>(o));
        }
    if (p.stats && h == 0) p.stats[id] = float2{m, l};
}

template <typename TT, int DP, int NW, bool CAUSAL>
__global__ __launch_bounds__(64 * NW, (FWD_WAVES<TT, DP, CAUSAL>)) void k_attn_fwd(const Args p) {
    attn_fwd<TT, DP, NW, CAUSAL, false>(p);
}

// For few rows against many keys: where a sample's rows fit one wave and its keys
// are split, a staged tile meets one tile of products and the walk waits for
// memory, so that p as two numbers costs nothing (a query to each of 4 samples of
// 266,426 x 8 x 16 bf16 in all: 47.5 us with a relative error of out of 1.6e-3, the
// rounding of out itself, and 47.3 with 2.4e-3).  Others would pay: causal 8,000 x
// 4 over 2 x 48 124 us, 109 with one number; windows of 1,024 on 266,426 x 4 x 32
// 413 and 315; causal 16,411 x 8 over 2 x 128 883 and 729.
// One wave less to a SIMD where that leaves the registers for it.
template <typename TT, int DP, int NW, bool CAUSAL>
__global__ __launch_bounds__(64 * NW, (FWD_WAVES<TT, DP, CAUSAL> - (DP == (CAUSAL ? 128 : 32)))) void k_attn_fwd_few(const Args p) {
    attn_fwd<TT, DP, NW, CAUSAL, true>(p);
}

// How the joining kernels lay a workgroup of 256 threads out over rows, splits
// (up to 8 to a thread, all in flight) and quads of elements: powers of two,
// the quads fastest.
struct JoinLayout {
    int quads, splits, rows;
    __device__ __forceinline__ JoinLayout(int q, int s) {
        quads = splits = 1;
        while (quads < q) quads *= 2;
        while (splits * 8 < s && quads * splits < 256) splits *= 2;
        rows = 256 / (quads * splits);
    }
};

// Joins the splits of the forward: the parts of a row are read side by side
// and added up in a tree.
template <typename TT>
__global__ __launch_bounds__(256) void k_attn_join(const Args p) {
    constexpr int BM = 32, ES = sizeof(typename TT::storage);
    __shared__ __attribute__((aligned(16))) f32x4_t sum_o[256];
    __shared__ __attribute__((aligned(16))) f32x4_t sum_ml[256];      // m, l, whether keys are seen
    Job j;
    if (!job_of<BM>(p, p.qs, p.g, false, j)) return;
    const JoinLayout w(p.D / 4, p.splits);
    const int tid = int(threadIdx.x), d = (tid % w.quads) * 4, s0 = tid / w.quads % w.splits, rl = tid / (w.quads * w.splits);
    const int rows = min(j.len * p.g, j.r0 + BM);
    const int64_t step = int64_t(p.qs.n) * (int64_t(p.g) * p.hk) * (p.D + 4);
    for (int r = j.r0; r < rows; r += w.rows) {
        const Query q = query_of(p, j, j.a, r + rl, rows);
        const int64_t id = int64_t(q.head) * p.qs.n + q.row;
        float m = -INFINITY, l = 0.f, seen = 0.f;
        f32x4_t o = {0.f, 0.f, 0.f, 0.f};
        auto add = [&](const f32x4_t& ml, const f32x4_t& o2) {
            const float m2 = ml[0], top = fmaxf(m, m2), base = top == -INFINITY ? 0.f : top;
            const float a = exp2_(m - base), b = exp2_(m2 - base);
            l = l * a + ml[1] * b;                         // a part without keys: m = -inf, l and o are 0
            seen += ml[2];
            o = o * a + o2 * b;
            m = top;
        };
        if (q.row >= 0 && d < p.D)
#pragma unroll 4
            for (int s = s0; s < p.splits; s += w.splits) {
                const float* part = p.part + id * (p.D + 4) + s * step;
                add(*reinterpret_cast<const f32x4_t*>(part + p.D), *reinterpret_cast<const f32x4_t*>(part + d));
            }
        for (int n = w.splits / 2; n > 0; n /= 2) {
            __syncthreads();
            sum_o[tid] = o, sum_ml[tid] = f32x4_t{m, l, seen, 0.f};
            __syncthreads();
            if (s0 < n) add(sum_ml[tid + n * w.quads], sum_o[tid + n * w.quads]);
        }
        if (s0 > 0 || q.row < 0 || d >= p.D) continue;
        if (seen > 0.f && l == 0.f) l = NAN;
        const float inv = l == 0.f ? 0.f : 1.f / l;
        o *= inv;
        put4<TT>(p.out + int64_t(q.row) * p.ldo + (int64_t(q.head) * p.D + d) * ES, o);
        if (TT::E == 8 && p.rest) put4<TT>(p.rest + ((int64_t(q.row) * (int64_t(p.g) * p.hk) + q.head) * p.D + d) * ES, left_of<TT>(o));
        if (p.stats && d == 0) p.stats[id] = float2{m, l};
    }
}

// ---------------------------------------------------------- backward

// What a row's probabilities are computed from: p = 2^(c s + x) * y.
// 16-bit types fold the sum into x (m + log2 l is off by up to 2^-24 of its
// size, far below the rounding of p that follows); fp32 multiplies by 1 / l,
// so that a large m costs no precision.
template <typename TT>
__device__ __forceinline__ float2 from_stats(float2 ml) {
    if (ml.y == 0.f) return float2{-INFINITY, 0.f};        // a row that sees no key: 2^-inf
    if constexpr (TT::E == 8) return float2{-(ml.x + __log2f(ml.y)), 1.f};
    else return float2{-ml.x, 1.f / ml.y};
}

// ds is rounded to the type for its products.  fp16 has 40 binades, and ds more:
// the probabilities' of a long row times the gradients' of any training.  There a
// column holds ds times a power of two, which its sums lose at the end.  It
// begins where any ds that counts passes TOP, and is cut so that the largest
// comes to 2^10 whenever one does: what is below half of fp16's smallest number
// then is below 2^-35 of the column's largest, and nothing passes fp16's largest.
// 266,426 x 4 x 32 in windows of 1,024: backward 906 us, 835 at ds' own size, which
// had an error of 2% in dq at gradients of 10^-4 and infinite rows at 10^4.
template <typename TT>
constexpr bool RANGED = TT::id == SPC_F16;
constexpr float DS_FACTOR = 18446744073709551616.f;        // 2^64; ds itself is below 2^48
constexpr float DS_TOP = 32768.f;

// Brings w (ds times f) of the lanes' columns below TOP, with the sums so far.
template <int NB>
__device__ __forceinline__ void into_range(f32x16_t& w, f32x16_t (&acc)[NB], float& f) {
    float top = 0.f;
#pragma unroll
    for (int r = 0; r < 16; ++r) top = fmaxf(top, fabsf(w[r]));
    if (!__any(top > DS_TOP)) return;
    const float2 both = halves(top);
    top = fmaxf(both.x, both.y);
    const float a = top > DS_TOP && top < INFINITY ? ldexpf(1.f, 10 - __builtin_amdgcn_frexp_expf(top)) : 1.f;
    f *= a;
    w *= a;
#pragma unroll
    for (int db = 0; db < NB; ++db) acc[db] *= a;
}

// dq and delta: as the forward, a wave of 32 queries walks the keys.
template <typename TT, int DP, int NW, bool CAUSAL>
__global__ __launch_bounds__(64 * NW, (BWD_WAVES<TT, DP>)) void k_attn_dq(const Args p) {
    constexpr int BM = 32 * NW, KT = KT_OF<TT, NW>, BN = 32 * KT, NT = 64 * NW;
    constexpr bool SP = SPLIT<TT, DP>;
    using T = Tile<TT, DP>;
    __shared__ __attribute__((aligned(16))) char lds[2][2][BN * T::PITCH];
    Job j;
    if (!job_of<BM>(p, p.qs, p.g, CAUSAL, j)) return;
    const int lane = int(threadIdx.x) & 63, wave = int(threadIdx.x) >> 6, h = lane >> 5, col = lane & 31;
    const int ka = __builtin_amdgcn_readfirstlane(p.ks.at(j.s)), kb = __builtin_amdgcn_readfirstlane(p.ks.at(j.s + 1));
    const int lk = kb > ka ? kb - ka : 0, rows = j.len * p.g, off = lk - j.len;
    const int rw = __builtin_amdgcn_readfirstlane(j.r0 + 32 * wave);
    const Query q = query_of(p, j, j.a, rw + col, rows);
    const int64_t id = int64_t(q.head) * p.qs.n + q.row, in = int64_t(q.head) * p.D * T::ES;
    u32x4 qf[T::NS], ql[SP ? T::NS : 1], gf[T::NS];
    load_frags<TT, DP>(gf, p.dout + int64_t(q.row) * p.lddo + in, q.row >= 0, p.D, h);
    float delta = 0.f;
    {
        u32x4 of[T::NS], ol[T::NS];
        load_frags<TT, DP>(of, p.o + int64_t(q.row) * p.ldo + in, q.row >= 0, p.D, h);
        // the output as it was before its rounding: where one key outweighs the
        // others, do . v_j - delta is a small difference of large numbers
        const bool kept = TT::E == 8 && p.rest;
        load_frags<TT, DP>(ol, p.rest + (int64_t(q.row) * (int64_t(p.g) * p.hk) + q.head) * p.D * T::ES, kept && q.row >= 0, p.D, h);
#pragma unroll
        for (int s = 0; s < T::NS; ++s) {
            if constexpr (TT::E == 8) {
                Raw8<TT> x, y, z;
                x.v[0] = of[s], y.v[0] = gf[s], z.v[0] = ol[s];
                const f32x8_t a = widen<TT>(x) + widen<TT>(z) * (1.f / REST_UP<TT>), b = widen<TT>(y);
#pragma unroll
                for (int e = 0; e < 8; ++e) delta = fmaf(a[e], b[e], delta);
            } else {
                delta = fmaf(__uint_as_float(of[s].x), __uint_as_float(gf[s].x), delta);
                delta = fmaf(__uint_as_float(of[s].y), __uint_as_float(gf[s].y), delta);
                delta = fmaf(__uint_as_float(of[s].z), __uint_as_float(gf[s].z), delta);
                delta = fmaf(__uint_as_float(of[s].w), __uint_as_float(gf[s].w), delta);
            }
        }
        delta = sum_halves(delta);
    }
    load_frags<TT, DP>(qf, p.q + int64_t(q.row) * p.ldq + in, q.row >= 0, p.D, h);
    split_frags<TT, DP>(qf, ql, p.c);
    if (q.row >= 0 && h == 0 && j.split == 0) p.delta[id] = delta;
    const float2 mf = from_stats<TT>(q.row >= 0 ? p.stats[id] : float2{0.f, 0.f});
    auto limit = [&](int r) { return !CAUSAL ? lk : max(0, min(lk, (r < rows ? r : rows - 1) / p.g + 1 + off)); };
    const int nk = limit(j.r0 + BM - 1), seen_first = rw < rows ? limit(rw) : 0, seen_last = rw < rows ? limit(rw + 31) : 0;
    const int mine = CAUSAL ? q.pos + 1 + off : lk;
    const int tiles = (nk + BN - 1) / BN, per = (tiles + p.splits - 1) / p.splits;
    const int t0 = j.split * per, t1 = min(tiles, t0 + per);

    KeyStage<TT, DP, BN, NT> stage;
    stage.begin(p, j, ka, lk);
    const f32x16_t from_s = SP ? all16(mf.x) : zero16(), from_d = all16(-delta);   // what the products start from
    float f = DS_FACTOR;                                   // what ds is held times (RANGED)
    f32x16_t acc[T::NB];
#pragma unroll
    for (int db = 0; db < T::NB; ++db) acc[db] = zero16();
    if (t0 < t1) {
        stage.find(p, t0);
        stage.fetch(p, t0);
        if (t0 + 1 < t1) stage.find(p, t0 + 1);
        stage.put(lds[0][0], lds[0][1]);
    }
    lds_barrier();
    for (int t = t0; t < t1; ++t) {
        const int buf = (t - t0) & 1, p0 = t * BN;
        const bool more = t + 1 < t1;
        const uint64_t live = stage.live;
        if (more) {
            stage.fetch(p, t + 1);
            if (t + 2 < t1) stage.find(p, t + 2);
        }
        if (p0 < seen_last) {
            const char *kt = lds[buf][0], *vt = lds[buf][1];
            const bool edge = p0 + BN > seen_first || live != first_bits(BN);
#pragma unroll
            for (int u = 0; u < KT; ++u) {
                using X = Second<TT, DP>;
                f32x16_t s = from_s, d = from_d;
#pragma unroll
                for (int st = 0; st < T::NS; ++st) {
                    const u32x4 a = T::row16(kt, 32 * u + col, 2 * st + h);
                    s = mfma32<TT>(a, qf[st], s);
                    if constexpr (SP) s = mfma32<TT>(a, ql[st], s);
                }
#pragma unroll
                for (int st = 0; st < T::NS; ++st) d = mfma32<TT>(T::row16(vt, 32 * u + col, 2 * st + h), gf[st], d);
#pragma unroll
                for (int r = 0; r < 16; ++r) {
                    float w = exp2_(SP ? s[r] : fmaf(s[r], p.c, mf.x));
                    if constexpr (TT::E == 4) w *= mf.y;
                    if constexpr (RANGED<TT>) w *= f;
                    s[r] = w * d[r];
                }
                uint32_t vis = 0;
                if (edge) {
                    const int n = mine - (p0 + 32 * u);
                    vis = (uint32_t(live >> (32 * u)) & uint32_t(first_bits(n < 32 ? n : 32))) >> (4 * h);
#pragma unroll
                    for (int r = 0; r < 16; ++r) s[r] = (vis >> bit_of(r)) & 1u ? s[r] : 0.f;
                }
                if constexpr (RANGED<TT>) into_range(s, acc, f);
                const std::conditional_t<TWO_DS<TT, DP>, typename X::Two, typename X::Packed> w(s);
                if (CAUSAL && edge) X::template add_masked<false>(acc, kt, 32 * u, w, vis, lane);
                else X::add(acc, kt, 32 * u, w, lane);
            }
        }
        if (more) stage.put(lds[buf ^ 1][0], lds[buf ^ 1][1]);
        lds_barrier();
    }
    if (q.row < 0) return;
    if constexpr (RANGED<TT>) {
#pragma unroll
        for (int db = 0; db < T::NB; ++db) acc[db] *= 1.f / f;
    }
    if (p.splits > 1) {
        float* part = p.part + (int64_t(j.split) * p.qs.n * (int64_t(p.g) * p.hk) + id) * p.D;
#pragma unroll
        for (int db = 0; db < T::NB; ++db)
#pragma unroll
            for (int b = 0; b < 4; ++b) {
                const int d = 32 * db + 8 * b + 4 * h;
                if (d < p.D) *reinterpret_cast<f32x4_t*>(part + d) = f32x4_t{acc[db][4 * b], acc[db][4 * b + 1], acc[db][4 * b + 2], acc[db][4 * b + 3]};
            }
        return;
    }
    char* out = p.dq + int64_t(q.row) * p.lddq + in;
#pragma unroll
    for (int db = 0; db < T::NB; ++db)
#pragma unroll
        for (int b = 0; b < 4; ++b) {
            const int d = 32 * db + 8 * b + 4 * h;
            if (d < p.D)
                put4<TT>(out + d * T::ES, f32x4_t{acc[db][4 * b], acc[db][4 * b + 1], acc[db][4 * b + 2], acc[db][4 * b + 3]} * p.scale);
        }
}

// dk and dv: a wave of 32 keys walks the queries of all heads that share them,
// which sums their gradients without an atomic.
template <typename TT, int DP, int NW, bool CAUSAL>
__global__ __launch_bounds__(64 * NW, (BWD_WAVES<TT, DP>)) void k_attn_dkv(const Args p) {
    constexpr int BM = 32 * NW, KT = DP <= 64 ? KT_OF<TT, NW> : 1, BN = 32 * KT, NT = 64 * NW;
    constexpr bool SP = SPLIT<TT, DP>;
    using T = Tile<TT, DP>;
    using S = Stage<TT, DP, BN, NT>;
    __shared__ __attribute__((aligned(16))) char lds[2][2][BN * T::PITCH];
    __shared__ __attribute__((aligned(16))) float row_m[2][BN], row_f[2][BN], row_d[2][BN];
    Job j;
    if (!job_of<BM>(p, p.ks, 1, false, j)) return;
    const int lane = int(threadIdx.x) & 63, wave = int(threadIdx.x) >> 6, h = lane >> 5, col = lane & 31;
    const int qa = __builtin_amdgcn_readfirstlane(p.qs.at(j.s)), qb = __builtin_amdgcn_readfirstlane(p.qs.at(j.s + 1));
    const int lq = qb > qa ? qb - qa : 0, rows = lq * p.g, off = j.len - lq;
    const int kw = __builtin_amdgcn_readfirstlane(j.r0 + 32 * wave), key = kw + col;   // the wave's first key, this lane's
    const int krow = key < j.len ? row_of(p.kv_order, j.a, key, p.ks.n) : -1;
    const int64_t in = int64_t(j.head) * p.D * T::ES;
    u32x4 kf[T::NS], kl[SP ? T::NS : 1], vf[T::NS];
    load_frags<TT, DP>(kf, p.k + int64_t(krow) * p.ldk + in, krow >= 0, p.D, h);
    load_frags<TT, DP>(vf, p.v + int64_t(krow) * p.ldv + in, krow >= 0, p.D, h);
    split_frags<TT, DP>(kf, kl, p.c);
    // the first row that sees a key: of the workgroup's first, the wave's first and last, this lane's
    auto begin = [&](int k) { return !CAUSAL ? 0 : min(lq, max(0, k - off)) * p.g; };
    const int first = begin(j.r0), first_lo = begin(kw), first_hi = begin(kw + 31), mine = begin(key);
    const int tb = first / BN, tiles = (rows + BN - 1) / BN - tb, per = (tiles + p.splits - 1) / p.splits;
    const int t0 = tb + j.split * per, t1 = min(tb + tiles, t0 + per);

    const bool in_place = p.g == 1 && !p.q_order;
    S stage;
    int mark = 0, row = -1;        // of this lane's row of the tile: its order entry, its row
    uint64_t live = 0;             // rows of the fetched tile that are there, as bits
    float2 own_ml = {0.f, 0.f};
    float own_d = 0.f;
    auto find = [&](int t) {
        if (p.q_order) mark = p.q_order[qa + min(place_of(p, j, t * BN + lane).pos, lq - 1)];
    };
    auto fetch = [&](int t) {
        const int cnt = rows - t * BN;
        const Query q = place_of(p, j, t * BN + lane);
        const int w = p.q_order ? mark : qa + q.pos;
        row = lane < BN && lane < cnt && unsigned(w) < unsigned(p.qs.n) ? w : -1;
        live = __ballot(row >= 0);
        if (in_place) {
            const int64_t at = qa + t * BN;
            stage.load(p.q + at * p.ldq + in, p.ldq, p.dout + at * p.lddo + in, p.lddo, cnt, p.D * T::ES);
        } else {                   // every row's place from the lane that has it
            stage.begin_parts();
#pragma unroll
            for (int i = 0; i < S::PT; ++i) {
                const int e = S::mine(i) ? S::row(i) : 0, r = __shfl(row, e), hd = p.g > 1 ? __shfl(q.head, e) : j.head;
                const int64_t at = r < 0 ? 0 : r, o = int64_t(hd) * p.D * T::ES;
                stage.load_part(i, r >= 0, p.q + at * p.ldq + o, p.dout + at * p.lddo + o, p.D * T::ES);
            }
        }
        if (wave == 0) {
            const int64_t id = row < 0 ? 0 : int64_t(q.head) * p.qs.n + row;
            own_ml = p.stats[id], own_d = p.delta[id];
        }
    };
    auto put = [&](int buf) {
        stage.put(lds[buf][0], lds[buf][1]);
        if (int(threadIdx.x) < BN) {
            const float2 mf = from_stats<TT>(row >= 0 ? own_ml : float2{0.f, 0.f});
            row_m[buf][threadIdx.x] = mf.x + BWD_UP<TT>;
            if constexpr (TT::E == 4) row_f[buf][threadIdx.x] = mf.y;
            row_d[buf][threadIdx.x] = row >= 0 ? -own_d : 0.f;
        }
    };

    constexpr float P_FACTOR = TT::id == SPC_F16 ? 32768.f : 1.f;     // 2^BWD_UP, what p is held times
    float fk = DS_FACTOR / P_FACTOR;       // what ds is held times beside it (RANGED)
    f32x16_t dk[T::NB], dv[T::NB];
#pragma unroll
    for (int db = 0; db < T::NB; ++db) dk[db] = zero16(), dv[db] = zero16();
    if (t0 < t1) {
        find(t0);
        fetch(t0);
        put(0);
        if (t0 + 1 < t1) find(t0 + 1);
    }
    lds_barrier();
    for (int t = t0; t < t1; ++t) {
        const int buf = (t - t0) & 1, p0 = t * BN;
        const bool more = t + 1 < t1;
        const uint64_t here = live;
        if (more) {
            fetch(t + 1);
            if (t + 2 < t1) find(t + 2);
        }
        if (p0 + BN > first_lo && kw < j.len) {
            const char *qt = lds[buf][0], *gt = lds[buf][1];
            const bool edge = here != first_bits(BN) || p0 < first_hi;
#pragma unroll
            for (int u = 0; u < KT; ++u) {
                using X = Second<TT, DP>;
                // the products start from the rows' -m and -delta
                f32x16_t s = zero16(), d;
#pragma unroll
                for (int b = 0; b < 4; ++b) {
                    const int r0 = 32 * u + 8 * b + 4 * h;
                    const f32x4_t d4 = *reinterpret_cast<const f32x4_t*>(&row_d[buf][r0]);
                    f32x4_t m4;
                    if constexpr (SP) m4 = *reinterpret_cast<const f32x4_t*>(&row_m[buf][r0]);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        d[4 * b + e] = d4[e];
                        if constexpr (SP) s[4 * b + e] = m4[e];
                    }
                }
#pragma unroll
                for (int st = 0; st < T::NS; ++st) {
                    const u32x4 a = T::row16(qt, 32 * u + col, 2 * st + h);
                    s = mfma32<TT>(a, kf[st], s);
                    if constexpr (SP) s = mfma32<TT>(a, kl[st], s);
                }
#pragma unroll
                for (int st = 0; st < T::NS; ++st) d = mfma32<TT>(T::row16(gt, 32 * u + col, 2 * st + h), vf[st], d);
#pragma unroll
                for (int b = 0; b < 4; ++b) {
                    const int r0 = 32 * u + 8 * b + 4 * h;
                    f32x4_t m4, f4;
                    if constexpr (!SP) m4 = *reinterpret_cast<const f32x4_t*>(&row_m[buf][r0]);
                    if constexpr (TT::E == 4) f4 = *reinterpret_cast<const f32x4_t*>(&row_f[buf][r0]);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int r = 4 * b + e;
                        float w = exp2_(SP ? s[r] : fmaf(s[r], p.c, m4[e]));
                        if constexpr (TT::E == 4) w *= f4[e];
                        s[r] = w;
                        if constexpr (RANGED<TT>) w *= fk;
                        d[r] *= w;
                    }
                }
                uint32_t vis = 0;
                if (edge) {
                    const int n = mine - (p0 + 32 * u);    // rows before this lane's first are hidden
                    vis = (uint32_t(here >> (32 * u)) & ~uint32_t(first_bits(n < 32 ? n : 32))) >> (4 * h);
#pragma unroll
                    for (int r = 0; r < 16; ++r) {
                        const bool see = (vis >> bit_of(r)) & 1u;
                        s[r] = see ? s[r] : 0.f, d[r] = see ? d[r] : 0.f;
                    }
                }
                if constexpr (RANGED<TT>) into_range(d, dk, fk);
                if (edge) {
                    if constexpr (CAUSAL) {
                        X::template add_masked<true>(dv, gt, 32 * u, typename X::Packed(s), vis, lane);
                        X::template add_masked<false>(dk, qt, 32 * u, typename X::Packed(d), vis, lane);
                        continue;
                    }
                }
                X::add(dv, gt, 32 * u, typename X::Packed(s), lane);
                X::add(dk, qt, 32 * u, typename X::Packed(d), lane);
            }
        }
        if (more) put(buf ^ 1);
        lds_barrier();
    }
    if (krow < 0) return;
    if constexpr (RANGED<TT>) {
#pragma unroll
        for (int db = 0; db < T::NB; ++db) dk[db] *= 1.f / (fk * P_FACTOR), dv[db] *= 1.f / P_FACTOR;
    }
    if (p.splits > 1) {
        float* part = p.part + (int64_t(j.split) * p.ks.n * p.hk + int64_t(j.head) * p.ks.n + krow) * (2 * p.D);
#pragma unroll
        for (int db = 0; db < T::NB; ++db)
#pragma unroll
            for (int b = 0; b < 4; ++b) {
                const int d = 32 * db + 8 * b + 4 * h;
                if (d >= p.D) continue;
                *reinterpret_cast<f32x4_t*>(part + d) = f32x4_t{dk[db][4 * b], dk[db][4 * b + 1], dk[db][4 * b + 2], dk[db][4 * b + 3]};
                *reinterpret_cast<f32x4_t*>(part + p.D + d) = f32x4_t{dv[db][4 * b], dv[db][4 * b + 1], dv[db][4 * b + 2], dv[db][4 * b + 3]};
            }
        return;
    }
    char *ok = p.dk + int64_t(krow) * p.lddk + in, *ov = p.dv + int64_t(krow) * p.lddv + in;
#pragma unroll
    for (int db = 0; db < T::NB; ++db)
#pragma unroll
        for (int b = 0; b < 4; ++b) {
            const int d = 32 * db + 8 * b + 4 * h;
            if (d >= p.D) continue;
            put4<TT>(ok + d * T::ES, f32x4_t{dk[db][4 * b], dk[db][4 * b + 1], dk[db][4 * b + 2], dk[db][4 * b + 3]} * p.scale);
            put4<TT>(ov + d * T::ES, f32x4_t{dv[db][4 * b], dv[db][4 * b + 1], dv[db][4 * b + 2], dv[db][4 * b + 3]});
        }
}

// Sums the splits of a gradient, in a tree: of dq (KEYS false), or of dk and dv.
template <typename TT, bool KEYS>
__global__ __launch_bounds__(256) void k_attn_sum(const Args p) {
    constexpr int BM = 32, ES = sizeof(typename TT::storage);
    __shared__ __attribute__((aligned(16))) f32x4_t sum[256];
    Job j;
    const int mult = KEYS ? 1 : p.g;
    if (!job_of<BM>(p, KEYS ? p.ks : p.qs, mult, false, j)) return;
    const int width = KEYS ? 2 * p.D : p.D;
    const JoinLayout w(width / 4, p.splits);
    const int tid = int(threadIdx.x), d = (tid % w.quads) * 4, s0 = tid / w.quads % w.splits, rl = tid / (w.quads * w.splits);
    const int rows = min(j.len * mult, j.r0 + BM);
    const int64_t n = KEYS ? p.ks.n : p.qs.n, heads = KEYS ? int64_t(p.hk) : int64_t(p.g) * p.hk;
    for (int r = j.r0; r < rows; r += w.rows) {
        int row = -1, head = j.head;
        if constexpr (KEYS) {
            if (r + rl < rows) row = row_of(p.kv_order, j.a, r + rl, p.ks.n);
        } else {
            const Query q = query_of(p, j, j.a, r + rl, rows);
            row = q.row, head = q.head;
        }
        f32x4_t t = {0.f, 0.f, 0.f, 0.f};
        if (row >= 0 && d < width) {
            const float* part = p.part + (int64_t(head) * n + row) * width + d;
#pragma unroll 8
            for (int s = s0; s < p.splits; s += w.splits) t += *reinterpret_cast<const f32x4_t*>(part + s * (n * heads * width));
        }
        for (int k = w.splits / 2; k > 0; k /= 2) {
            __syncthreads();
            sum[tid] = t;
            __syncthreads();
            if (s0 < k) t += sum[tid + k * w.quads];
        }
        if (s0 > 0 || row < 0 || d >= width) continue;
        if constexpr (KEYS) {
            if (d < p.D) put4<TT>(p.dk + int64_t(row) * p.lddk + (int64_t(head) * p.D + d) * ES, t * p.scale);
            else put4<TT>(p.dv + int64_t(row) * p.lddv + (int64_t(head) * p.D + d - p.D) * ES, t);
        } else {
            put4<TT>(p.dq + int64_t(row) * p.lddq + (int64_t(head) * p.D + d) * ES, t * p.scale);
        }
    }
}

// ------------------------------------------------------------- launches

// How a walk is cut: waves to a workgroup, splits of the other side.
struct Cut {
    int32_t nw, splits;
    int64_t slots, blocks;     // of BM = 32 nw rows; workgroups of all splits and heads
};

spc_status launch_fwd_f32(const Args& p, const Cut& c, hipStream_t stream);
spc_status launch_fwd_f16(const Args& p, const Cut& c, hipStream_t stream);
spc_status launch_fwd_bf16(const Args& p, const Cut& c, hipStream_t stream);
spc_status launch_bwd_f32(const Args& p, const Cut& q, const Cut& k, hipStream_t stream);
spc_status launch_bwd_f16(const Args& p, const Cut& q, const Cut& k, hipStream_t stream);
spc_status launch_bwd_bf16(const Args& p, const Cut& q, const Cut& k, hipStream_t stream);

inline int64_t slots_of(int64_t rows, int64_t n_seg, int bm) { return rows / bm + n_seg + 1; }

// Sets the grid of a walk; its workgroups.  A group is 1,024 rows of all heads
// where there are many, a slot where the work of neighbours differs (causal) or
// there are few.  Forward and backward in us, with groups of one slot, of 1,024
// rows and of an eighth of the call: windows of 1,024 on 266,426 x 4 x 32 bf16 342 +
// 900, 323 + 872 and 325 + 867, of 500 on 120,000 x 8 x 16 139 + 352, 138 + 351 and
// 133 + 347, of 2,048 on 60,000 x 8 over 2 x 64 341 + 1,069, 341 + 1,068 and 339 +
// 1,066; causal 16,411 x 8 over 2 x 128 forward 736 with one slot and 1,554 with
// eighths, 8,000 x 4 over 2 x 64 fp32 407 + 1,377 and 583 + 1,467, 20 ragged samples
// of 30,000 x 8 x 64 in all 378 + 1,000 and 789 + 1,957.
inline unsigned set_grid(Args& p, int64_t slots, int splits, int rows_of_slot, bool even) {
    p.slots = int32_t(slots), p.splits = splits;
    p.total = unsigned(slots * splits * p.hk);
    const int64_t g = 1024 / rows_of_slot;
    p.group = unsigned(p.hk) * unsigned(even && slots * splits >= 64 * g ? g : 1);
    return unsigned(ceil_div(int64_t(p.total), int64_t(p.group) * 8)) * p.group * 8u;
}

#define ATTN_WIDTH(name, dp, nw, grid, p)                                                                                     \
    do {                                                                                                                      \
        if (p.causal) hipLaunchKernelGGL((name<TT, dp, nw, true>), dim3(grid), dim3(64 * nw), 0, stream, p);                  \
        else hipLaunchKernelGGL((name<TT, dp, nw, false>), dim3(grid), dim3(64 * nw), 0, stream, p);                          \
    } while (0)

// Workgroups of four waves, or of the fewest: one, and two where heads are so
// wide that one wave's share of the staging would not fit its registers.
constexpr int few_waves(int D) { return D <= 64 ? 1 : 2; }

// Heads of every multiple of 16 up to 96 have kernels of their own width, in every
// type: work, LDS and registers go with it.  Padded to 64 and 128 they took
// (40,000 x 4 heads in windows of 1,024, training, us; then one causal sample of
// 8,000 x 4):
//         48 own, as 64        80 own, as 128       96 own, as 128
//   fp32  1,729, 1,782         2,854, 3,937         2,858, 3,977
//         1,590, 1,907         2,308, 4,450         2,518, 4,489
//   bf16  309, 306             472, 737             662, 756
//         421, 638             641, 860             646, 870
// Heads of 112 have as many 32-row blocks as 128 and gain nothing: bf16 839 us in a
// width of their own, 797 as 128; causal 936 and 885.
#define ATTN_WIDTHS(name, nw, grid, p)                                                                                        \
    do {                                                                                                                      \
        constexpr int NW = nw, NW2 = nw == 1 ? few_waves(128) : nw;                                                           \
        switch (p.D / 16) {                                                                                                   \
            case 1: ATTN_WIDTH(name, 16, NW, grid, p); break;                                                                 \
            case 2: ATTN_WIDTH(name, 32, NW, grid, p); break;                                                                 \
            case 3: ATTN_WIDTH(name, 48, NW, grid, p); break;                                                                 \
            case 4: ATTN_WIDTH(name, 64, NW, grid, p); break;                                                                 \
            case 5: ATTN_WIDTH(name, 80, NW2, grid, p); break;                                                                \
            case 6: ATTN_WIDTH(name, 96, NW2, grid, p); break;                                                                \
            default: ATTN_WIDTH(name, 128, NW2, grid, p);                                                                     \
        }                                                                                                                     \
        SPC_LAUNCHED(#name);                                                                                                  \
    } while (0)

template <typename TT>
spc_status launch_fwd(Args p, const Cut& c, hipStream_t stream) {
    const unsigned grid = set_grid(p, c.slots, c.splits, 32 * c.nw, !p.causal);
    const bool few = TT::E == 8 && c.splits > 1 && int64_t(p.qs.n) * p.g <= int64_t(32) * p.qs.n_seg;
    if (c.nw == 4) ATTN_WIDTHS(k_attn_fwd, 4, grid, p);
    else if (!few) ATTN_WIDTHS(k_attn_fwd, 1, grid, p);
    else if constexpr (TT::E == 8) ATTN_WIDTHS(k_attn_fwd_few, 1, grid, p);
    if (c.splits > 1) {
        const int splits = p.splits;
        const unsigned rows = set_grid(p, slots_of(int64_t(p.qs.n) * p.g, p.qs.n_seg, 32), 1, 32, false);
        p.splits = splits;
        hipLaunchKernelGGL(k_attn_join<TT>, dim3(rows), dim3(256), 0, stream, p);
        SPC_LAUNCHED("k_attn_join");
    }
    return SPC_OK;
}

template <typename TT>
spc_status launch_bwd(Args p, const Cut& cq, const Cut& ck, hipStream_t stream) {
    if (p.qs.n) {
        unsigned grid = set_grid(p, cq.slots, cq.splits, 32 * cq.nw, !p.causal);
        if (cq.nw == 4) ATTN_WIDTHS(k_attn_dq, 4, grid, p);
        else ATTN_WIDTHS(k_attn_dq, 1, grid, p);
        if (cq.splits > 1) {
            grid = set_grid(p, slots_of(int64_t(p.qs.n) * p.g, p.qs.n_seg, 32), 1, 32, false);
            p.splits = cq.splits;
            hipLaunchKernelGGL((k_attn_sum<TT, false>), dim3(grid), dim3(256), 0, stream, p);
            SPC_LAUNCHED("k_attn_sum");
        }
    }
    if (p.ks.n) {
        unsigned grid = set_grid(p, ck.slots, ck.splits, 32 * ck.nw, !p.causal);
        if (ck.nw == 4) ATTN_WIDTHS(k_attn_dkv, 4, grid, p);
        else ATTN_WIDTHS(k_attn_dkv, 1, grid, p);
        if (ck.splits > 1) {
            grid = set_grid(p, slots_of(p.ks.n, p.ks.n_seg, 32), 1, 32, false);
            p.splits = ck.splits;
            hipLaunchKernelGGL((k_attn_sum<TT, true>), dim3(grid), dim3(256), 0, stream, p);
            SPC_LAUNCHED("k_attn_sum");
        }
    }
    return SPC_OK;
}

}  // namespace attn
}  // namespace spc
