// Rotary positions of several axes: pair j of a head, elements 2j and 2j + 1,
// belongs to one axis of the row's position and is rotated by the angle
// position * freq[j]; pairs past the axes' are copied as they are stored (a
// rotation by 0 would multiply infinities by 0).
//
// A workgroup computes the sines and cosines of its rows once into LDS, for
// all heads, and then walks the rows' chunks of 8 elements in memory order,
// reading and writing every line once.  Angles: the product of the int32
// position and the fp32 frequency, and its quarter turns, are taken as sums of
// two doubles, so that a position of 2^31 loses nothing (one double would leave
// 10^-6 radians there); what is left of whole quarter turns, at most an eighth of
// a turn, goes to fp32.
//
// Bound by memory: 266,426 x 8 x 32 bf16 63 us with inputs from memory (4.4 TB/s; 61
// without the second doubles of the angles and the copies), 120,000 x 8 x 16 fp16 13 us.
// Four chunks of a thread are in flight (one: 67 us where four took 53).
#include "rows.h"

namespace spc {
namespace {

constexpr int RT = 256;           // threads per workgroup
constexpr int TABLE = 2048;       // pairs a workgroup has room for (16 KB)
constexpr int AXES = 8;
constexpr int ROT_D_MAX = 2 * TABLE;

struct RotArgs {
    const char* x;
    char* out;
    int64_t ldx, ldo;             // bytes between rows
    const int32_t* pos;
    int64_t ldp;                  // elements between positions
    const float* freq;
    int64_t n;
    int heads, D, rows;           // rows of a workgroup
    int axes, pairs;              // rotated pairs of a head
    int end[AXES];                // pairs of the axes up to and with each
    float sign;                   // -1: the rotation back
};

// Whole quarter turns (mod 4) of the angle pos * freq, and what is left of one.
__device__ __forceinline__ int quarter_turns(int pos, float freq, float& rest) {
#pragma clang fp contract(off)        // the products below are rounded where they stand
    constexpr double TURN = 0x1.45f306dc9c883p-1, TURN_LEFT = -0x1.6b01ec5417056p-55;   // 2 / pi, what rounding left of it
    const double a = pos, b = freq, t = a * b, t2 = fma(a, b, -t);
    const double q = t * TURN, q2 = fma(t2, TURN, fma(t, TURN_LEFT, fma(t, TURN, -q)));
    const double r = fma(-4.0, rint(q * 0.25), q) + q2, whole = rint(r);      // the fma is exact
    rest = float(r - whole);
    return int(whole) & 3;
}

constexpr float COPIED = 2.f;     // the cosine of a pair past the axes in the table

// Those pairs of a chunk as they were in x.
template <typename TT>
__device__ __forceinline__ void keep_pairs(Raw8<TT>& y, const Raw8<TT>& x, const float2* t) {
    constexpr int W = 8 / TT::E;      // words of a pair
    uint32_t a[4 * W], b[4 * W];
    __builtin_memcpy(a, &y, sizeof(a));
    __builtin_memcpy(b, &x, sizeof(b));
#pragma unroll
    for (int i = 0; i < 4 * W; ++i) a[i] = t[i / W].x == COPIED ? b[i] : a[i];
    __builtin_memcpy(&y, a, sizeof(a));
}

template <typename TT>
__global__ __launch_bounds__(RT) void k_rotary(const RotArgs p) {
    __shared__ __attribute__((aligned(16))) float2 table[TABLE];
    constexpr int ES = sizeof(typename TT::storage);
    const int64_t row0 = int64_t(blockIdx.x) * p.rows;
    const int rows = int(p.n - row0 < p.rows ? p.n - row0 : p.rows), half = p.D / 2;
    for (int e = int(threadIdx.x); e < rows * half; e += RT) {
        const int r = e / half, j = e - r * half;
        float2 cs = {COPIED, 0.f};
        if (j < p.pairs) {
            int axis = 0;
            while (j >= p.end[axis]) ++axis;
            float s, c, rest;
            const int k = quarter_turns(p.pos[(row0 + r) * p.ldp + axis], p.freq[j], rest);
            sincospif(rest * 0.5f, &s, &c);
            cs.x = k == 0 ? c : k == 1 ? -s : k == 2 ? -c : s;
            cs.y = (k == 0 ? s : k == 1 ? c : k == 2 ? -s : -c) * p.sign;
        }
        table[e] = cs;
    }
    __syncthreads();
    // four chunks of a thread in flight
    const int per = p.D / 8, width = p.heads * per, chunks = rows * width;
    for (int e0 = int(threadIdx.x); e0 < chunks; e0 += 4 * RT) {
        Raw8<TT> x[4];
        int at[4];
        int64_t to[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int e = e0 + k * RT < chunks ? e0 + k * RT : e0;
            const int r = e / width, c = e - r * width;
            at[k] = r * half + (c % per) * 4;
            to[k] = (row0 + r) * p.ldo + int64_t(c) * 8 * ES;
            x[k] = ld8<TT>(p.x + (row0 + r) * p.ldx + int64_t(c) * 8 * ES);
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            if (e0 + k * RT >= chunks) continue;
            f32x8_t v = widen<TT>(x[k]);
            const float2* t = table + at[k];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 cs = t[i];
                const float a = v[2 * i], b = v[2 * i + 1];
                v[2 * i] = fmaf(a, cs.x, -(b * cs.y));
                v[2 * i + 1] = fmaf(a, cs.y, b * cs.x);
            }
            Raw8<TT> y = narrow<TT>(v);
            if (p.pairs < half) keep_pairs<TT>(y, x[k], t);
            st8<TT>(p.out + to[k], y);
        }
    }
}

}  // namespace
}  // namespace spc

using namespace spc;

extern "C" spc_status spc_rotary(spc_dtype dtype, const void* x, int64_t ldx, int64_t n, int32_t heads, int32_t head_dim,
                                 const int32_t* pos, int64_t ldp, int32_t n_axes, const int32_t* pairs, const float* freq,
                                 int32_t inverse, void* out, int64_t ldo, hipStream_t stream) {
    clear_error();
    if (dtype != SPC_F32 && dtype != SPC_F16 && dtype != SPC_BF16) return fail(SPC_ERR_ARG, "unknown dtype %d", int(dtype));
    if (n < 0 || n >= ROWS_END) return fail(SPC_ERR_ARG, "n=%lld is out of range", (long long)n);
    if (heads < 1) return fail(SPC_ERR_ARG, "heads=%d must be positive", heads);
    if (head_dim < 1 || head_dim % 16 || head_dim > ROT_D_MAX)
        return fail(SPC_ERR_UNSUPPORTED, "head_dim=%d: a multiple of 16 up to %d", head_dim, ROT_D_MAX);
    if (int64_t(heads) * head_dim > C_MAX) return fail(SPC_ERR_UNSUPPORTED, "%d heads of %d are too many", heads, head_dim);
    if (n_axes < 1 || n_axes > AXES || !pairs) return fail(SPC_ERR_ARG, "n_axes=%d: 1 to %d, with their pairs", n_axes, AXES);
    const int64_t e = dtype_size(dtype), width = int64_t(heads) * head_dim;
    for (const int64_t ld : {ldx, ldo})
        if (ld < width || ld * e % 16 || ld >= (int64_t(1) << 31))
            return fail(SPC_ERR_ARG, "row stride %lld: at least heads x head_dim, a multiple of 16 bytes, below 2^31", (long long)ld);
    if (ldp < n_axes || ldp >= (int64_t(1) << 31)) return fail(SPC_ERR_ARG, "ldp=%lld is not between n_axes=%d and 2^31", (long long)ldp, n_axes);
    RotArgs p{};
    int64_t sum = 0;
    for (int a = 0; a < n_axes; ++a) {
        if (pairs[a] < 0) return fail(SPC_ERR_ARG, "pairs[%d]=%d is negative", a, pairs[a]);
        sum += pairs[a];
        if (sum > head_dim / 2) return fail(SPC_ERR_ARG, "%lld pairs exceed half of head_dim=%d", (long long)sum, head_dim);
        p.end[a] = int(sum);
    }
    if (n == 0) return SPC_OK;
    if (!x || !out || !pos || (sum && !freq)) return fail(SPC_ERR_ARG, "x, out, pos or freq is NULL");
    for (const void* q : {x, (const void*)out})
        if (!aligned16(q)) return fail(SPC_ERR_ARG, "device pointers must be 16-byte aligned");
    const spc_status st = check_overlap(Rows{out, n, width * e, ldo * e, "out"}, Rows{x, n, width * e, ldx * e, "x"}, true);
    if (st != SPC_OK) return st;
    // positions may be columns of the coordinates: aligned as their type
    for (const void* q : {(const void*)pos, (const void*)freq})
        if (reinterpret_cast<uintptr_t>(q) & 3u) return fail(SPC_ERR_ARG, "pos and freq must be aligned to 4 bytes");
    p.x = static_cast<const char*>(x), p.out = static_cast<char*>(out);
    p.ldx = ldx * e, p.ldo = ldo * e, p.ldp = ldp, p.pos = pos, p.freq = freq;
    p.n = n, p.heads = heads, p.D = head_dim, p.axes = n_axes, p.pairs = int(sum), p.sign = inverse ? -1.f : 1.f;
    // as many rows as the table holds, fewer where that leaves compute units without work
    const int64_t room = TABLE / (head_dim / 2), fill = ceil_div(n, 1024);
    p.rows = int(fill < room ? fill : room);
    const int64_t blocks = ceil_div(n, p.rows);
    if (!launchable(blocks, RT)) return fail(SPC_ERR_UNSUPPORTED, "%lld rows of %d elements exceed one launch", (long long)n, head_dim);
    switch (dtype) {
        case SPC_F32: hipLaunchKernelGGL(k_rotary<F32>, dim3(unsigned(blocks)), dim3(RT), 0, stream, p); break;
        case SPC_F16: hipLaunchKernelGGL(k_rotary<F16>, dim3(unsigned(blocks)), dim3(RT), 0, stream, p); break;
        case SPC_BF16: hipLaunchKernelGGL(k_rotary<BF16>, dim3(unsigned(blocks)), dim3(RT), 0, stream, p); break;
    }
    SPC_LAUNCHED("k_rotary");
    return SPC_OK;
}
