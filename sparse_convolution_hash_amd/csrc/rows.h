// Helpers of the row operators (norm.hip, dropout.hip, recurrence.hip): eight
// channels per thread, ragged samples by row offsets, and the dropout
// generator.  Not part of the ABI.
#pragma once

#include "common.h"

namespace spc {

// ------------------------------------------------------- eight channels

typedef float f32x8_t __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8v_t __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8v_t __attribute__((ext_vector_type(8)));

// Eight consecutive elements as stored: one 16-byte word of a 16-bit type,
// two of fp32.  Loads and arithmetic are separate so that a thread can keep
// several rows in flight in half the registers.
template <typename TT>
struct Raw8 {
    u32x4 v[8 / TT::E];
};

template <typename TT>
__device__ __forceinline__ Raw8<TT> ld8(const void* p) {
    Raw8<TT> r;
#pragma unroll
    for (int i = 0; i < 8 / TT::E; ++i) r.v[i] = ld16(static_cast<const char*>(p) + 16 * i);
    return r;
}

template <typename TT>
__device__ __forceinline__ void st8(void* p, const Raw8<TT>& r) {
#pragma unroll
    for (int i = 0; i < 8 / TT::E; ++i) st16(static_cast<char*>(p) + 16 * i, r.v[i]);
}

template <typename TT>
__device__ __forceinline__ f32x8_t widen(const Raw8<TT>& r);
template <>
__device__ __forceinline__ f32x8_t widen<F32>(const Raw8<F32>& r) {
    return __builtin_bit_cast(f32x8_t, r);
}
template <>
__device__ __forceinline__ f32x8_t widen<F16>(const Raw8<F16>& r) {
    return __builtin_convertvector(__builtin_bit_cast(f16x8v_t, r), f32x8_t);
}
template <>
__device__ __forceinline__ f32x8_t widen<BF16>(const Raw8<BF16>& r) {
    const uint32_t w[4] = {r.v[0].x, r.v[0].y, r.v[0].z, r.v[0].w};
    f32x8_t f;
#pragma unroll
    for (int i = 0; i < 4; ++i) f[2 * i] = __uint_as_float(w[i] << 16), f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    return f;
}

// The one rounding to the storage type (nearest even; a NaN stays a NaN).
template <typename TT>
__device__ __forceinline__ Raw8<TT> narrow(const f32x8_t& f);
template <>
__device__ __forceinline__ Raw8<F32> narrow<F32>(const f32x8_t& f) {
    return __builtin_bit_cast(Raw8<F32>, f);
}
template <>
__device__ __forceinline__ Raw8<F16> narrow<F16>(const f32x8_t& f) {
    return __builtin_bit_cast(Raw8<F16>, __builtin_convertvector(f, f16x8v_t));
}
template <>
__device__ __forceinline__ Raw8<BF16> narrow<BF16>(const f32x8_t& f) {
    return __builtin_bit_cast(Raw8<BF16>, __builtin_convertvector(f, bf16x8v_t));
}

// --------------------------------------------------------- ragged samples

// What the host checks hold every call to: n and n_seg below ROWS_END, so that
// rounded up to tiles and waves they are still ints, and at most C_MAX channels.
constexpr int64_t ROWS_END = (int64_t(1) << 31) - 4096;
constexpr int32_t C_MAX = 64 * 65535;

// Whether one launch can have that many workgroups: it holds fewer than 2^32
// threads, and of a larger grid the runtime starts a part without an error.
inline bool launchable(int64_t blocks, int threads) { return blocks * threads < (int64_t(1) << 32); }

// Sample s owns the rows [at(s), at(s + 1)).  ptr NULL is one sample of all n
// rows.  The offsets come from device memory unchecked, so each is clamped to
// [0, n]: whatever they hold, no row outside the arrays is touched.
struct Segs {
    const int32_t* ptr;
    int32_t n_seg, n;

    __device__ __forceinline__ int at(int s) const {
        const int v = ptr ? ptr[s] : (s ? n : 0);
        return v < 0 ? 0 : v > n ? n : v;
    }

    // The last sample whose offset is <= row (0 if there is none).  Called by
    // whole waves with one row: 64 offsets per step.
    __device__ __forceinline__ int find(int row) const {
        const int lane = int(threadIdx.x) & (WAVE - 1);
        int lo = 0, hi = n_seg;  // the count of offsets <= row is in [lo, hi]
        while (lo < hi) {
            const int step = (hi - lo + WAVE - 1) / WAVE;
            const int p = lo + lane * step;
            const int k = __popcll(__ballot(p < hi && at(p < hi ? p : lo) <= row));
            if (k == 0) break;
            if (step == 1) {
                lo += k;
                break;
            }
            const int nlo = lo + (k - 1) * step + 1, nhi = lo + k * step;
            lo = nlo;
            hi = nhi < hi ? nhi : hi;
        }
        return lo > 0 ? lo - 1 : 0;
    }
};

// ------------------------------------------------- where tensors overlap

// Rows of `width` bytes, `ld` bytes apart.
struct Rows {
    const void* p;
    int64_t n, width, ld;
    const char* name;
};

// Whether two tensors share a byte.  Columns of one wider tensor do not: rows of
// the same stride are compared by their distance, others row by row (of the one
// with fewer), where their ranges meet at all.
inline bool overlap(Rows a, Rows b) {
    if (!a.p || !b.p || a.n <= 0 || b.n <= 0 || a.width <= 0 || b.width <= 0) return false;
    using I = __int128;                // rows times strides may pass 64 bits
    I d = I(reinterpret_cast<intptr_t>(b.p)) - reinterpret_cast<intptr_t>(a.p);                 // where b begins, from a
    if (a.n > b.n) {
        const Rows t = a;
        a = b, b = t, d = -d;
    }
    if (d >= I(a.n - 1) * a.ld + a.width || -d >= I(b.n - 1) * b.ld + b.width) return false;
    // One row of width w that begins `at` bytes past b's first: b's row j meets it iff -b.width < j ld - at < w.
    auto meets = [&](I at, int64_t w, int64_t lo, int64_t hi) {
        const I x = at - b.width + 1, q = x / b.ld, j = q + (x > q * b.ld ? 1 : 0);             // the first row past the left bound
        const I first = j > lo ? j : I(lo);
        return first <= hi && first * b.ld - at < w;
    };
    // rows i of a and j of b lie (j - i) ld + d apart
    if (a.ld == b.ld || a.n == 1) return meets(-d, a.width, 1 - a.n, b.n - 1);
    for (int64_t i = 0; i < a.n; ++i)
        if (meets(I(i) * a.ld - d, a.width, 0, b.n - 1)) return true;
    return false;
}

// Refuses an output that overlaps another tensor; with `same`, it may be that
// tensor.
inline spc_status check_overlap(const Rows& out, const Rows& other, bool same = false) {
    if (same && out.p == other.p && (out.n <= 1 || out.ld == other.ld)) return SPC_OK;
    if (overlap(out, other)) return fail(SPC_ERR_ARG, "%s and %s overlap", out.name, other.name);
    return SPC_OK;
}

// ---------------------------------------------------------------- dropout

// Philox4x32-10 (Salmon, Moraes, Dror and Shaw, "Parallel random numbers: as
// easy as 1, 2, 3", SC 2011), key = seed, counter = (ctr, layer, 0).  Its 128
// bits are eight 16-bit uniforms, one per element: element i of a tensor
// takes half-word i % 8 (low half of a word first) of counter offset + i / 8.
struct Drop {
    const uint64_t* rng;  // device {seed, offset}; NULL: no dropout
    uint32_t layer;
    uint32_t thr;         // an element is dropped iff its 16 bits are below thr
    float scale;          // of the kept ones: 65536 / (65536 - thr)
    float inv;            // its reciprocal, exact
};

// a ^ b ^ c in one instruction.
__device__ __forceinline__ uint32_t xor3(uint32_t a, uint32_t b, uint32_t c) { return __builtin_amdgcn_bitop3_b32(a, b, c, 0x96); }

__device__ __forceinline__ u32x4 philox(uint64_t seed, uint64_t ctr, uint32_t layer) {
    uint32_t c0 = uint32_t(ctr), c1 = uint32_t(ctr >> 32), c2 = layer, c3 = 0;
    uint32_t k0 = uint32_t(seed), k1 = uint32_t(seed >> 32);
#pragma unroll
    for (int r = 0; r < 10; ++r) {
        const uint64_t p0 = uint64_t(c0) * 0xD2511F53u, p1 = uint64_t(c2) * 0xCD9E8D57u;
        c0 = xor3(uint32_t(p1 >> 32), c1, k0);
        c1 = uint32_t(p1);
        c2 = xor3(uint32_t(p0 >> 32), c3, k1);
        c3 = uint32_t(p0);
        k0 += 0x9E3779B9u;
        k1 += 0xBB67AE85u;
    }
    return u32x4{c0, c1, c2, c3};
}

// v[j] where the element stays, 0 where it is dropped (also for an infinite
// or NaN v[j]).
__device__ __forceinline__ f32x8_t drop8(f32x8_t v, const u32x4& bits, uint32_t thr) {
    const uint32_t w[4] = {bits.x, bits.y, bits.z, bits.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = (w[i] & 0xffffu) >= thr ? v[2 * i] : 0.f;
        v[2 * i + 1] = (w[i] >> 16) >= thr ? v[2 * i + 1] : 0.f;
    }
    return v;
}

// Host: checks a dropout descriptor (NULL: none) and turns it into kernel
// arguments.
inline spc_status make_drop(const spc_dropout* d, Drop& out) {
    out = Drop{nullptr, 0, 0, 1.f, 1.f};
    if (!d) return SPC_OK;
    if (!(d->p >= 0.f && d->p <= 1.f)) return fail(SPC_ERR_ARG, "dropout p=%g is outside [0, 1]", double(d->p));
    if (!d->rng || !aligned16(d->rng)) return fail(SPC_ERR_ARG, "dropout rng is NULL or not 16-byte aligned");
    out.rng = d->rng;
    out.layer = d->layer;
    out.thr = uint32_t(d->p * 65536.f + 0.5f);
    // p = 1 drops everything: no element is left to scale
    out.scale = out.thr < 65536u ? 65536.f / float(65536u - out.thr) : 0.f;
    out.inv = float(65536u - out.thr) / 65536.f;
    return SPC_OK;
}

}  // namespace spc
