// Lists of tensors: the AdamW step with states in 32 bits or in 8, the
// gradients' sum of squares, and the conversion of states, with their host
// side.  Written for gfx950 (CDNA4, wave64).
//
// All are streams bounded by HBM: per element a step reads W gradients, the
// weights and the states and writes weights and states back (28 bytes with
// bf16 gradients of one rank, a master and fp32 states; 16 with 8-bit states;
// 10 with 8-bit states and no master).  Measured on MI355X over 218 M elements
// in nine tensors (124 M in 148 with the master), of 8 TB/s:
//   fp32 states, W = 1: bf16 weights 6.7 TB/s, fp32 weights and gradients 6.7,
//     a master 6.5; W = 2, 3, 4, 5, 8 with a master 6.6, 6.6, 6.6, 6.5, 6.6
//     (rows of gradients at multiples of 256 bytes; at multiples of 16 every
//     load takes a line more: 6.5, 6.3, 6.5, 6.2, 6.2)
//   8-bit states: 6.3 (a master), 6.2 (bf16 weights), 6.7 (fp32)
//   to 8 bits 6.8, to 32 bits 6.3, sum of squares 6.2 (both launches)
// Large streams of the same mixes reach 6.8 here.
//
// Work decomposition.  A list's tensors are cut into pieces of kPiece
// elements, each taken by one to four one-wave workgroups, so one launch takes
// any number of tensors of any sizes.  A workgroup finds its tensor in the
// list's table in device memory: the tensor's number for each piece, then the
// tensor's record, both wave-uniform scalar loads.  A tensor's own pieces, one
// for each kPiece elements, lie together; where a step's units start later than
// the tensor it may need one more, and those lie behind all tensors' own, so
// that the sum of squares, which has no need to start late, takes the same
// elements in the same order wherever the arrays lie.  As in zs_step.hip every
// load or store of a wave covers one contiguous run, all loads of a part are
// issued before its arithmetic, loads are non-temporal and aligned stores
// stream to HBM with system scope.

#include <hip/hip_runtime.h>

#include <algorithm>
#include <cfloat>
#include <cmath>
#include <cstdint>
#include <new>
#include <type_traits>
#include <vector>

#include "zs_codes.h"
#include "zs_device.h"
#include "zs_internal.h"
#include "zs_tensors.h"

namespace {

typedef unsigned int u32x2 __attribute__((ext_vector_type(2)));
typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
// the same at any element's address; the hardware takes vector accesses at
// such addresses whole
typedef u32x2 u32x2_2 __attribute__((aligned(2)));
typedef f32x4 f32x4_4 __attribute__((aligned(4)));
typedef u32x4 u32x4_2 __attribute__((aligned(2)));
typedef u32x4 u32x4_4 __attribute__((aligned(4)));

constexpr int kWave = 64;
constexpr int kBlock = ZS_STATE8_BLOCK;
static_assert(kBlock == 4 * kWave, "a wave's unit is one block");
constexpr int kPiece = 4 * kBlock;
// Pieces that one launch takes: HIP launches fewer than 2^32 work-items along
// x, and a piece is four workgroups at most.
constexpr int64_t kLaunchPieces = (int64_t(1) << 24) - 1;
constexpr int64_t kMaxPieces = (int64_t(1) << 28) - 1;
// Units of kBlock elements to a workgroup.  One keeps what is in flight most
// compact: the 124 M step with fp32 states 537 us, 559 with two, 627 with four.
// With 8-bit states two share the reductions and the division (bf16 weights
// 351 us, 391 with one, 380 with four); where those cost little it is even
// (with a master 318 us, 316 with one).
constexpr int kStep32Units = 1, kStep8Units = 2;
// Parts that an XCD takes in a run where the 8-bit step's weights are fp32: 64
// blocks, whose scales are two lines.  218 M elements in fp32 524 us, 539 with
// the parts in turn, 24 M with a master 59.4 and 61; with bf16 weights alone
// 359 and 355, so those go in turn.  With fp32 states and in conversions runs
// of 2 to 256 parts are 1 to 6 % slower.
constexpr int kStep8Run = 32;
// To 8 bits 326 us (two units 340); to 32 bits 348 us with four at 8
// workgroups per CU (10: 358, 12: 351, 16: 382), with two at 22 353 and as many
// as fit 380, with one 382.
constexpr int kPackUnits = 1, kUnpackUnits = 4;
constexpr int kUnpackResidency = 8;
constexpr int64_t kMaxReach = int64_t(1) << 46;
constexpr int64_t kMaxSlices = int64_t(1) << 22;

// One tensor in the table.
struct Rec {
    const void* grad;
    int64_t gstride;
    void* param;
    float* master;
    void* m;
    void* v;
    float* ms;
    float* vs;
    int64_t numel;
    int32_t piece0;     // its first piece
    int32_t group;
    int32_t pre;        // places before its first element in a step's units
    int32_t flags;
};
// Four elements from a unit's start on are aligned; so are lines of all ranks'
// gradients.
constexpr int32_t kRecFours = 1, kRecLines = 2;
static_assert(sizeof(Rec) == 88, "the header states it");

struct Hp {
    float b1, b2, omb1, omb2;   // beta1, beta2, 1-beta1, 1-beta2
    float ss;                   // lr / (1 - beta1^t)
    float bc2s, ibc2s;          // sqrt(1 - beta2^t) and its reciprocal
    float dec;                  // 1 - lr*wd
    float eps;
};

struct Table {
    const Rec* recs;
    const int32_t* tensor;      // of each piece
    int32_t own;                // the tensors' own pieces; more lie behind
    int32_t first;              // a launch's first piece
};

// Of W ranks' gradients.
struct Ranks {
    int32_t W;
    float fw, invw;     // W and 1/W
    int32_t pow2;       // W is a power of two (1/W exact)
};

struct StepArgs {
    Table t;
    const double* sumsq;        // nullable
    float max_norm;
    Ranks ranks;
    Hp hp[ZS_TENSORS_MAX_GROUPS];
};

// ---- device side -------------------------------------------------------------

__device__ __forceinline__ float bf16_lo(uint32_t u)
{
    return __uint_as_float(u << 16);
}

__device__ __forceinline__ float bf16_hi(uint32_t u)
{
    return __uint_as_float(u & 0xffff0000u);
}

// A pointer to device memory.  Pointers that come from the table are generic
// to the compiler, and accesses through them would be flat ones.
template <class T>
using Global = __attribute__((address_space(1))) T*;

template <class T, class P>
__device__ __forceinline__ Global<T> global(P* p)
{
    return (Global<T>)p;
}

struct V4 {
    float x[4];
};

// What a workgroup works on: U units of kBlock places, a part of a piece.  The
// tensor's elements are those of its places lo .. n-1.
template <int U>
struct Part {
    int64_t off;        // the first place's element of the tensor, or below 0
    int lo, n;
    bool whole;
};

// Which of a launch's parts this workgroup has: with RUN > 1, each XCD (they
// take workgroups in turn) has runs of RUN parts.  Those that do not fill
// eight runs are in order.
template <int RUN>
__device__ __forceinline__ uint32_t part_index()
{
    const uint32_t b = blockIdx.x;
    constexpr uint32_t kAll = 8 * RUN;
    if (RUN == 1 || b >= gridDim.x / kAll * kAll)
        return b;
    return b / kAll * kAll + b % 8 * RUN + b % kAll / 8;
}

// Part i of a launch is number i % (4 / U) of its piece.
template <int U>
__device__ __forceinline__ int32_t record_of(const Table& t, uint32_t i)
{
    return t.tensor[t.first + (int32_t)(i / (4 / U))];
}

// LATE: units may start later than their tensor, as those of lists with fp32
// states do.
template <int U, bool LATE>
__device__ __forceinline__ Part<U> part_of(const Table& t, const Rec& r,
                                           uint32_t i)
{
    const int32_t p = t.first + (int32_t)(i / (4 / U));
    int64_t piece = p - r.piece0;
    if (LATE && p >= t.own)     // the one behind the tensor's own
        piece = (r.numel + kPiece - 1) / kPiece;
    Part<U> q;
    q.off = piece * kPiece + (int)(i % (4 / U)) * (U * kBlock) - r.pre;
    const int64_t left = r.numel - q.off;
    q.lo = q.off < 0 ? (int)-q.off : 0;
    q.n = left < U * kBlock ? (int)left : U * kBlock;
    q.whole = q.lo == 0 && q.n == U * kBlock;
    return q;
}

// How a part is accessed.  kAligned: all its elements exist, at addresses
// aligned to four of them; kLines: and so do the ranks' gradients, at lines of
// 128 bytes.  kWhole: all exist, at any addresses.  kEdge: those of lo .. n-1
// exist.
constexpr int kLines = 0, kAligned = 1, kWhole = 2, kEdge = 3;

// Four elements as they lie in memory.  Kept so until all loads of a part are
// on their way: a conversion waits for its load.
template <class T>
struct Raw;
template <>
struct Raw<float> {
    f32x4 x;
};
template <>
struct Raw<uint16_t> {
    u32x2 x;
};

__device__ __forceinline__ V4 wide(const Raw<float>& r)
{
    return {r.x.x, r.x.y, r.x.z, r.x.w};
}

__device__ __forceinline__ V4 wide(const Raw<uint16_t>& r)
{
    return {bf16_lo(r.x.x), bf16_hi(r.x.x), bf16_lo(r.x.y), bf16_hi(r.x.y)};
}

// A part's places lo .. n-1.
struct Places {
    int lo, n;
    // whether place i, or places i .. i+3, are of it
    __device__ __forceinline__ bool has(int i) const
    {
        return i >= lo && i < n;
    }
    __device__ __forceinline__ bool has4(int i) const
    {
        return i >= lo && i + 4 <= n;
    }
};

// Elements at places i .. i+3 of p; 0 where there is none.  NT: non-temporal.
template <int MODE, bool NT = true>
__device__ __forceinline__ Raw<float> load4(Global<const float> p, int i,
                                            Places q)
{
    const auto a = (Global<const f32x4>)(p + i);
    const auto u = (Global<const f32x4_4>)(p + i);
    if constexpr (MODE <= kAligned)
        return {NT ? __builtin_nontemporal_load(a) : *a};
    if (MODE == kWhole || q.has4(i))
        return {NT ? __builtin_nontemporal_load(u) : *u};
    Raw<float> r = {{0, 0, 0, 0}};
#pragma unroll
    for (int j = 0; j < 4; ++j)
        if (q.has(i + j))
            r.x[j] = p[i + j];
    return r;
}

template <int MODE, bool NT = true>
__device__ __forceinline__ Raw<uint16_t> load4(Global<const uint16_t> p,
                                               int i, Places q)
{
    const auto a = (Global<const u32x2>)(p + i);
    const auto u = (Global<const u32x2_2>)(p + i);
    if constexpr (MODE <= kAligned)
        return {NT ? __builtin_nontemporal_load(a) : *a};
    if (MODE == kWhole || q.has4(i))
        return {NT ? __builtin_nontemporal_load(u) : *u};
    Raw<uint16_t> r = {{0, 0}};
#pragma unroll
    for (int j = 0; j < 4; ++j)
        if (q.has(i + j))
            r.x[j / 2] |= (uint32_t)p[i + j] << (16 * (j % 2));
    return r;
}

// Stores of a part whose first place is at p (wave-uniform): streamed on to
// HBM where they are aligned.
template <int MODE>
__device__ __forceinline__ void store4(Global<float> p, int i, Places q,
                                       const V4& r)
{
    const f32x4 x = {r.x[0], r.x[1], r.x[2], r.x[3]};
    if constexpr (MODE <= kAligned) {
        zsdev::stream_store((void*)p, (uint32_t)q.n * 4u, (uint32_t)i * 4u,
                            x);
        return;
    }
    if (MODE == kWhole || q.has4(i)) {
        __builtin_nontemporal_store(x, (Global<f32x4_4>)(p + i));
        return;
    }
#pragma unroll
    for (int j = 0; j < 4; ++j)
        if (q.has(i + j))
            p[i + j] = r.x[j];
}

template <int MODE>
__device__ __forceinline__ void store4(Global<uint16_t> p, int i, Places q,
                                       const V4& r)
{
    const u32x2 x = {to_bf16(r.x[0], r.x[1]), to_bf16(r.x[2], r.x[3])};
    if constexpr (MODE <= kAligned) {
        zsdev::stream_store((void*)p, (uint32_t)q.n * 2u, (uint32_t)i * 2u,
                            x);
        return;
    }
    if (MODE == kWhole || q.has4(i)) {
        __builtin_nontemporal_store(x, (Global<u32x2_2>)(p + i));
        return;
    }
#pragma unroll
    for (int j = 0; j < 4; ++j)
        if (q.has(i + j))
            p[i + j] = (uint16_t)(x[j / 2] >> (16 * (j % 2)));
}

// Four codes in a word (codes are always aligned to four, and none lies before
// a part's first place).
template <int MODE>
__device__ __forceinline__ uint32_t load_codes(Global<const uint8_t> p, int i,
                                               Places q)
{
    if (MODE != kEdge || q.has4(i))
        return __builtin_nontemporal_load((Global<const uint32_t>)(p + i));
    uint32_t r = 0;
#pragma unroll
    for (int j = 0; j < 3; ++j)
        if (q.has(i + j))
            r |= (uint32_t)p[i + j] << (8 * j);
    return r;
}

template <int MODE>
__device__ __forceinline__ void store_codes(Global<uint8_t> p, int i,
                                            Places q, uint32_t x)
{
    if constexpr (MODE != kEdge) {
        zsdev::stream_store((void*)p, (uint32_t)q.n, (uint32_t)i, x);
        return;
    }
    if (q.has4(i)) {
        *(Global<uint32_t>)(p + i) = x;
        return;
    }
#pragma unroll
    for (int j = 0; j < 3; ++j)
        if (q.has(i + j))
            p[i + j] = (uint8_t)(x >> (8 * j));
}

// Elements of a part's gradients from the ranks, WT of them at compile time
// (0: as many as there are, eight at a time; at a tensor's ends two): all
// loads, then the sum in rank order from the first (so that the sign of a zero
// sum is its own) and the mean.
//
// Gradients of one rank, and rows that do not start at lines, so that every
// load shares a line with its neighbours', are loaded with the caches' usual
// policy: W = 1 with bf16 weights 709 us against 717 non-temporal, W = 8 with
// rows at multiples of 16 bytes 1481 against 1511 (8-bit states 1026 against
// 1085).  Rows of several ranks that start at lines are non-temporal: W = 8
// 1390 against 1447, W = 5 1198 against 1242.
//
// SEEN: the bits of all ranks' gradients are kept, for blank().
template <int MODE, int U, int WT, class T, bool SEEN = false>
struct Gradients {
    static constexpr bool kAll = WT == 1 || (WT > 0 && MODE != kEdge);
    static constexpr int NB = kAll ? WT : MODE == kEdge ? 2 : 8;
    Raw<T> x[NB][U];
    using Words = std::conditional_t<sizeof(T) == 2, u32x2, u32x4>;
    Words seen[U];

    __device__ __forceinline__ void load(const Rec& r, int64_t off, int s0,
                                         int W, Places q)
    {
        const Global<const T> g0 = global<const T>(r.grad) + off;
#pragma unroll
        for (int s = 0; s < NB; ++s)
            if (kAll || s0 + s < W)
#pragma unroll
                for (int k = 0; k < U; ++k)
                    x[s][k] = load4<MODE, MODE == kLines>(
                        g0 + (int64_t)(s0 + s) * r.gstride,
                        4 * (k * kWave + (int)threadIdx.x), q);
    }

    __device__ __forceinline__ void add(int s0, int W, V4 (&g)[U])
    {
#pragma unroll
        for (int s = 0; s < NB; ++s)
            if (kAll || s0 + s < W)
#pragma unroll
                for (int k = 0; k < U; ++k) {
                    const V4 y = wide(x[s][k]);
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        g[k].x[j] =
                            s0 + s == 0 ? y.x[j] : g[k].x[j] + y.x[j];
                    if constexpr (SEEN && !kAll) {
                        const Words w = __builtin_bit_cast(Words, x[s][k]);
                        seen[k] = s0 + s == 0 ? w : seen[k] | w;
                    }
                }
    }

    // Bit 4 k + j: element j of unit k is zero, of either sign, on every rank,
    // though another of its block is not.  g: the mean, which has to be zero
    // for that, so that the ranks' bits are looked at in few waves only.
    __device__ __forceinline__ uint32_t blank(const V4 (&g)[U]) const
    {
        float least = INFINITY;
#pragma unroll
        for (int k = 0; k < U; ++k)
#pragma unroll
            for (int j = 0; j < 4; ++j)     // the smaller of both
                least = __builtin_amdgcn_fmed3f(least, fabsf(g[k].x[j]),
                                                0.0f);
        if (__builtin_expect(!__any(least == 0.0f), 1))
            return 0;
        uint32_t r = 0;
#pragma unroll
        for (int k = 0; k < U; ++k) {
            Words w;
            if constexpr (kAll) {
                w = __builtin_bit_cast(Words, x[0][k]);
#pragma unroll
                for (int s = 1; s < NB; ++s)
                    w |= __builtin_bit_cast(Words, x[s][k]);
            } else {
                w = seen[k];
            }
            uint32_t b = 0;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const uint32_t y = sizeof(T) == 4 ? w[j] & 0x7fffffffu
                    : w[j / 2] & (j % 2 ? 0x7fff0000u : 0x7fffu);
                b |= (uint32_t)(y == 0) << j;
            }
            if (__any(b != 15))
                r |= b << (4 * k);
        }
        return r;
    }

    // The mean, the first slices loaded by load(rec, off, 0, W, q).
    __device__ __forceinline__ void mean(const Rec& rec, int64_t off,
                                         const Ranks& r, Places q,
                                         V4 (&g)[U])
    {
        add(0, r.W, g);
        if constexpr (!kAll)
            for (int s0 = NB; s0 < r.W; s0 += NB) {
                load(rec, off, s0, r.W, q);
                add(s0, r.W, g);
            }
        if constexpr (WT == 1)
            return;
#pragma unroll
        for (int k = 0; k < U; ++k)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (WT > 0 ? (WT & (WT - 1)) == 0 : r.pow2 != 0)
                    g[k].x[j] = g[k].x[j] * r.invw;
                else
                    g[k].x[j] = g[k].x[j] / r.fw;
    }
};

// ---- codes

__device__ __forceinline__ uint32_t abs_bits(float x)
{
    return __float_as_uint(x) & 0x7fffffffu;
}

template <int CTRL>
__device__ __forceinline__ uint32_t max_dpp(uint32_t x)
{
    const uint32_t y = (uint32_t)__builtin_amdgcn_update_dpp(
        0, (int)x, CTRL, 0xf, 0xf, true);
    return max(x, y);
}
constexpr int kRor1 = 0x121, kRor2 = 0x122, kRor4 = 0x124, kRor8 = 0x128;

// a's upper 32 lanes change places with b's lower ones; the larger of each.
__device__ __forceinline__ uint32_t max_halves(uint32_t a, uint32_t b)
{
    const auto p = __builtin_amdgcn_permlane32_swap(a, b, false, false);
    return max(p[0], p[1]);
}

// a's rows 1 and 3 (of 16 lanes) change places with b's rows 0 and 2; the
// larger of each.
__device__ __forceinline__ uint32_t max_rows(uint32_t a, uint32_t b)
{
    const auto p = __builtin_amdgcn_permlane16_swap(a, b, false, false);
    return max(p[0], p[1]);
}

// The largest of each unit's m and r over the wave, as bits: those of |x|
// order as |x| does, with infinity above all numbers and NaN above infinity.
// The 2 U reductions go together, m in the lower and r in the upper lanes: of
// unit k, m's largest is in lane 16 k and r's in lane 32 + 16 k (and their
// neighbours).
template <int U>
__device__ __forceinline__ uint32_t wave_max(const uint32_t (&m)[U],
                                             const uint32_t (&r)[U])
{
    static_assert(U == 1 || U == 2, "a row of 16 lanes to each of m and r");
    uint32_t x[U];
#pragma unroll
    for (int k = 0; k < U; ++k)
        x[k] = max_halves(m[k], r[k]);
    uint32_t y = max_rows(x[0], x[U - 1]);
    y = max_dpp<kRor4>(max_dpp<kRor8>(y));
    return max_dpp<kRor1>(max_dpp<kRor2>(y));
}

// The roots of U units, correctly rounded; 0, smaller and larger values take
// the compiler's form.
template <int U>
__device__ __forceinline__ void roots(const float (&x)[U][4],
                                      float (&r)[U][4])
{
    float lo = INFINITY;
    uint32_t hi = 0;
#pragma unroll
    for (int k = 0; k < U; ++k)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            lo = fminf(lo, x[k][j]);
            hi = max(hi, __float_as_uint(x[k][j]));
        }
    if (__builtin_expect(__any(lo < 0x1p-96f || hi >= 0x7f800000u), 0)) {
#pragma unroll
        for (int k = 0; k < U; ++k)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                r[k][j] = sqrtf(x[k][j]);
        return;
    }
#pragma unroll
    for (int k = 0; k < U; ++k)
#pragma unroll
        for (int j = 0; j < 4; ++j)
            r[k][j] = root_of(x[k][j]);
}

// Codes of four m, those up to kFade that `blank` has a bit for rounded towards
// zero.  A step takes a tenth of m away at a beta1 of 0.9, less than half a
// step of the codes up to 9: to the nearest they would stay for ever, and the
// weight of an element that has no gradient any more would go on moving, by a
// third of lr a step.  Larger codes go down by themselves, and where elements
// are without a gradient now and then their roundings have to be right on
// average (all towards zero took 5 to 12 % off what such weights move, those
// up to 9 nothing).  Looking for zeros costs 0 to 1 % (bf16 weights, 218 M
// elements: 358 us of 356), gradients with many of them 3 to 11 % (392 of 359).
constexpr float kFade = 9.0f;

__device__ __forceinline__ uint32_t faded(const float (&m)[4], float im,
                                          uint32_t c, uint32_t blank)
{
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int q = (int8_t)(c >> (8 * j));
        const float a = fabsf((float)q);
        if ((blank >> j & 1) && a <= kFade && a * a > fabsf(m[j]) * im)
            c = (c & ~(0xffu << (8 * j))) |
                (uint32_t)(uint8_t)(q < 0 ? q + 1 : q - 1) << (8 * j);
    }
    return c;
}

// Holds U units' m and roots of v: codes, and scales in the lanes that
// wave_max() has them in.  blank: as Gradients has it.
template <int U>
__device__ __forceinline__ void hold(const float (&m)[U][4],
                                     const float (&r)[U][4], uint32_t blank,
                                     uint32_t (&cm)[U], uint32_t (&cr)[U],
                                     float& S)
{
    uint32_t am[U], ar[U];
#pragma unroll
    for (int k = 0; k < U; ++k) {
        am[k] = max(max(abs_bits(m[k][0]), abs_bits(m[k][1])),
                    max(abs_bits(m[k][2]), abs_bits(m[k][3])));
        ar[k] = max(max(abs_bits(r[k][0]), abs_bits(r[k][1])),
                    max(abs_bits(r[k][2]), abs_bits(r[k][3])));
    }
    const uint32_t a = wave_max<U>(am, ar);
    const float A = __uint_as_float(a);
    const bool upper = threadIdx.x >= 32;
    const float top = upper ? kTopR : kTopM;
    S = A * (upper ? (float)(1.0 / 65025.0) : (float)(1.0 / 16129.0));
    float inv = quotient_of(top, A);
    const bool odd = __any(a - 0x0d800000u >= 0x7e800000u - 0x0d800000u);
    if (__builtin_expect(odd, 0)) {
        inv = top / A;
        if (a < 0x0d800000u)            // below 2^-100
            S = inv = 0.0f;
        if (a >= 0x7f800000u)           // an infinity or a NaN
            S = __uint_as_float(0x7fc00000u);
    }
    auto lane = [](float x, int i) {
        return __uint_as_float((uint32_t)__builtin_amdgcn_readlane(
            (int)__float_as_uint(x), i));
    };
#pragma unroll
    for (int k = 0; k < U; ++k)
        codes(m[k], r[k], lane(inv, 16 * k), lane(inv, 16 * k + 32), cm[k],
              cr[k]);
    if (__builtin_expect(__any(blank != 0), 0)) {
#pragma unroll
        for (int k = 0; k < U; ++k)
            cm[k] = faded(m[k], lane(inv, 16 * k), cm[k], blank >> (4 * k));
    }
    if (__builtin_expect(odd, 0)) {
#pragma unroll
        for (int k = 0; k < U; ++k) {
            const float sm = lane(S, 16 * k), sr = lane(S, 16 * k + 32);
            cm[k] = sm == sm ? cm[k] : 0;
            cr[k] = sr == sr ? cr[k] : 0;
        }
    }
}

// Writes what hold() gave for a part.
template <int MODE, int U>
__device__ __forceinline__ void store_held(Global<uint8_t> mp,
                                           Global<uint8_t> vp,
                                           Global<float> msp,
                                           Global<float> vsp, Places q,
                                           const uint32_t (&cm)[U],
                                           const uint32_t (&cr)[U], float S)
{
    const int lane = (int)threadIdx.x;
#pragma unroll
    for (int k = 0; k < U; ++k) {
        if (MODE == kEdge && k * kBlock >= q.n)
            break;
        store_codes<MODE>(mp, 4 * (k * kWave + lane), q, cm[k]);
        store_codes<MODE>(vp, 4 * (k * kWave + lane), q, cr[k]);
    }
    const int k = lane % 32 / 16;
    if (lane % 16 == 0 && k < U && (MODE != kEdge || k * kBlock < q.n))
        (lane < 32 ? msp : vsp)[k] = S;
}

// ---- the step

// The factor of the gradients; false for no step at all: *sumsq negative or
// not finite.
__device__ __forceinline__ bool clip_of(const double* sumsq, float max_norm,
                                        float& c)
{
    c = 1.0f;
    if (!sumsq)
        return true;
    const double s = *sumsq;
    const double norm = sqrt(s);
    if (norm > (double)max_norm)
        c = (float)((double)max_norm / norm);
    return norm - norm == 0.0;
}

// Kinds of weights.
constexpr int kMaster = 0, kBf16 = 1, kF32 = 2;

template <int MODE, int U, int WM>
struct Weights {
    using T = std::conditional_t<WM == kBf16, uint16_t, float>;
    Raw<T> x[U];

    __device__ __forceinline__ void load(const Rec& r, int64_t off, Places q)
    {
        const Global<const T> p =
            global<const T>(WM == kMaster ? r.master : r.param) + off;
#pragma unroll
        for (int k = 0; k < U; ++k)
            x[k] = load4<MODE>(p, 4 * (k * kWave + (int)threadIdx.x), q);
    }
};

template <int MODE, int WM>
__device__ __forceinline__ void store_weights(const Rec& r, int64_t off,
                                              int i, Places q, const V4& w)
{
    if constexpr (WM == kMaster)
        store4<MODE>(global<float>(r.master) + off, i, q, w);
    using T = std::conditional_t<WM == kF32, float, uint16_t>;
    store4<MODE>(global<T>(r.param) + off, i, q, w);
}

template <int MODE, int U, int WM, int WT, class G>
__device__ __forceinline__ void step32_part(const StepArgs& a, const Rec& r,
                                            int64_t off, Places q)
{
    const Global<float> mp = global<float>(r.m) + off;
    const Global<float> vp = global<float>(r.v) + off;
    const int lane = (int)threadIdx.x;
    Weights<MODE, U, WM> wx;
    Raw<float> mx[U], vx[U];
    Gradients<MODE, U, WT, G> gx;
    wx.load(r, off, q);
#pragma unroll
    for (int k = 0; k < U; ++k) {
        mx[k] = load4<MODE>(mp, 4 * (k * kWave + lane), q);
        vx[k] = load4<MODE>(vp, 4 * (k * kWave + lane), q);
    }
    gx.load(r, off, 0, a.ranks.W, q);
    const Hp h = a.hp[r.group];
    float c;
    if (!clip_of(a.sumsq, a.max_norm, c))
        return;
    V4 g[U];
    gx.mean(r, off, a.ranks, q, g);
#pragma unroll
    for (int k = 0; k < U; ++k) {
        V4 w = wide(wx.x[k]), m = wide(mx[k]), v = wide(vx[k]);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float gi = g[k].x[j] * c;
            m.x[j] = h.b1 * m.x[j] + h.omb1 * gi;
            v.x[j] = h.b2 * v.x[j] + h.omb2 * (gi * gi);
            const float den = sqrtf(v.x[j]) / h.bc2s + h.eps;
            w.x[j] = w.x[j] * h.dec - h.ss * (m.x[j] / den);
        }
        const int i = 4 * (k * kWave + lane);
        store_weights<MODE, WM>(r, off, i, q, w);
        store4<MODE>(mp, i, q, m);
        store4<MODE>(vp, i, q, v);
    }
}

template <int MODE, int U, int WM, int WT, class G>
__device__ __forceinline__ void step8_part(const StepArgs& a, const Rec& r,
                                           int64_t off, Places q)
{
    const Global<uint8_t> mp = global<uint8_t>(r.m) + off;
    const Global<uint8_t> vp = global<uint8_t>(r.v) + off;
    const Global<float> msp = global<float>(r.ms) + off / kBlock;
    const Global<float> vsp = global<float>(r.vs) + off / kBlock;
    const int lane = (int)threadIdx.x;
    Weights<MODE, U, WM> wx;
    uint32_t mq[U], vq[U];
    float ms[U], vs[U];
    Gradients<MODE, U, WT, G, true> gx;
    wx.load(r, off, q);
#pragma unroll
    for (int k = 0; k < U; ++k) {
        mq[k] = load_codes<MODE>(mp, 4 * (k * kWave + lane), q);
        vq[k] = load_codes<MODE>(vp, 4 * (k * kWave + lane), q);
        const bool there = MODE != kEdge || k * kBlock < q.n;
        ms[k] = there ? msp[k] : 0.0f;
        vs[k] = there ? vsp[k] : 0.0f;
    }
    gx.load(r, off, 0, a.ranks.W, q);
    const Hp h = a.hp[r.group];
    float c = 1.0f;
    if (!clip_of(a.sumsq, a.max_norm, c))
        return;
    V4 g[U];
    gx.mean(r, off, a.ranks, q, g);
    const uint32_t blank = gx.blank(g);
    if (a.sumsq) {
#pragma unroll
        for (int k = 0; k < U; ++k)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                g[k].x[j] *= c;
    }
    // elements behind the tensor's last are 0 here: gradients and codes were
    // loaded as 0
    float m[U][4], v[U][4], root[U][4];
#pragma unroll
    for (int k = 0; k < U; ++k)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float qm = (float)(int8_t)(mq[k] >> (8 * j));
            const float qv = (float)(uint8_t)(vq[k] >> (8 * j));
            const float r0 = (qv * qv) * vs[k];
            const float gi = g[k].x[j];
            m[k][j] = h.b1 * ((qm * fabsf(qm)) * ms[k]) + h.omb1 * gi;
            v[k][j] = h.b2 * (r0 * r0) + h.omb2 * (gi * gi);
        }
    roots<U>(v, root);
#pragma unroll
    for (int k = 0; k < U; ++k) {
        if (MODE == kEdge && k * kBlock >= q.n)
            break;
        V4 w = wide(wx.x[k]);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float rden = __builtin_amdgcn_rcpf(
                __builtin_fmaf(root[k][j], h.ibc2s, h.eps));
            w.x[j] = __builtin_fmaf(-h.ss, m[k][j] * rden, w.x[j] * h.dec);
        }
        store_weights<MODE, WM>(r, off, 4 * (k * kWave + lane), q, w);
    }
    uint32_t cm[U], cr[U];
    float S;
    hold<U>(m, root, blank, cm, cr, S);
    store_held<MODE, U>(mp, vp, msp, vsp, q, cm, cr, S);
}

template <int BITS, int MODE, int U, int WM, int WT, class G>
__device__ __forceinline__ void step_part(const StepArgs& a, const Rec& r,
                                          int64_t off, Places q)
{
    if constexpr (BITS == 32)
        step32_part<MODE, U, WM, WT, G>(a, r, off, q);
    else
        step8_part<MODE, U, WM, WT, G>(a, r, off, q);
}

template <int BITS, int WM>
constexpr int step_run()
{
    return BITS == 32 || WM == kBf16 ? 1 : kStep8Run;
}

template <int BITS, int U, int WM, int WT, class G>
__global__ __launch_bounds__(kWave) void step_kernel(StepArgs a)
{
    const uint32_t part = part_index<step_run<BITS, WM>()>();
    const Rec r = a.t.recs[record_of<U>(a.t, part)];
    const Part<U> q = part_of<U, BITS == 32>(a.t, r, part);
    if (q.n <= 0)
        return;
    if constexpr (WT != 1)
        if (q.whole && r.flags == (kRecFours | kRecLines)) {
            step_part<BITS, kLines, U, WM, WT, G>(a, r, q.off,
                                                  {0, U * kBlock});
            return;
        }
    if (q.whole && r.flags & kRecFours)
        step_part<BITS, kAligned, U, WM, WT, G>(a, r, q.off,
                                                {0, U * kBlock});
    else if (q.whole)
        step_part<BITS, kWhole, U, WM, WT, G>(a, r, q.off, {0, U * kBlock});
    else
        step_part<BITS, kEdge, U, WM, WT, G>(a, r, q.off, {q.lo, q.n});
}

// ---- the sum of squares

// Squares and sums are fp64, whose fused multiply-add runs at fp32's rate
// here, so no gradient's square overflows or is lost.  Each wave takes a run
// of consecutive pieces (32 waves to a CU), workgroups leave one partial sum
// each, and a second launch adds those: 70 us over 218 M bf16 elements, 5 of
// them the second launch; 154, 295 and 575 us for two, four and eight ranks
// (5.7 to 6.1 TB/s, 6.1 with fp32 gradients), 1 % more with rows off lines.
constexpr int kSumThreads = 256;
constexpr int kSumWaves = kSumThreads / kWave;
constexpr int kSumMaxGroups = 2048;     // workgroups, and so partial sums
constexpr int64_t kSumOne = 32;         // pieces that one workgroup takes alone

struct SumArgs {
    Table t;
    int32_t per_wave;           // consecutive pieces of a wave
    Ranks ranks;
    double* out;                // one per workgroup
};

template <int MODE, int WT, class G>
__device__ __forceinline__ double sum_piece(const SumArgs& a, const Rec& r,
                                            int64_t off, Places q)
{
    constexpr int U = 4;
    Gradients<MODE, U, WT, G> gx;
    gx.load(r, off, 0, a.ranks.W, q);
    V4 g[U];
    gx.mean(r, off, a.ranks, q, g);
    double s = 0.0;
#pragma unroll
    for (int k = 0; k < U; ++k)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const double x = g[k].x[j];
            s = __builtin_fma(x, x, s);
        }
    return s;
}

// The sum over a workgroup's threads, in a fixed order, in thread 0.
__device__ __forceinline__ double group_sum(double s, double* lds, int waves)
{
#pragma unroll
    for (int d = kWave / 2; d > 0; d >>= 1)
        s += __shfl_down(s, d, kWave);
    const int tid = (int)(threadIdx.x + threadIdx.y * blockDim.x);
    if ((tid & (kWave - 1)) == 0)
        lds[tid / kWave] = s;
    __syncthreads();
    s = 0.0;
    if (tid == 0)
        for (int i = 0; i < waves; ++i)
            s += lds[i];
    return s;
}

// The sum over n whole pieces from p on, one rank's: sixteen bytes of a lane to
// a load, and while a batch of kSumBatch loads is added the next is on its way
// (70 us; piece by piece with a lookup and a wait each 75).
constexpr int kSumBatch = 4;

template <class G>
__device__ __forceinline__ double square_sum(u32x4 x)
{
    double s = 0.0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const double lo = sizeof(G) == 4 ? __uint_as_float(x[j])
                                         : bf16_lo(x[j]);
        s = __builtin_fma(lo, lo, s);
        if constexpr (sizeof(G) == 2) {
            const double hi = bf16_hi(x[j]);
            s = __builtin_fma(hi, hi, s);
        }
    }
    return s;
}

template <class G>
__device__ __forceinline__ double sum_run(Global<const G> p, int n)
{
    constexpr int kStep = 16 / sizeof(G) * kWave;       // elements of a load
    constexpr int kLoads = kPiece / kStep;              // of a piece
    static_assert(kSumBatch % kLoads == 0, "batches of whole pieces");
    using Load = std::conditional_t<sizeof(G) == 2, u32x4_2, u32x4_4>;
    p += (int)threadIdx.x * (16 / (int)sizeof(G));
    const int loads = n * kLoads;
    u32x4 x[kSumBatch], y[kSumBatch];
#pragma unroll
    for (int k = 0; k < kSumBatch; ++k)
        if (k < loads)
            x[k] = __builtin_nontemporal_load(
                (Global<const Load>)(p + k * kStep));
    double s[kSumBatch] = {};
    for (int i = 0; i < loads; i += kSumBatch) {
        p += kSumBatch * kStep;
#pragma unroll
        for (int k = 0; k < kSumBatch; ++k)
            if (i + kSumBatch + k < loads)
                y[k] = __builtin_nontemporal_load(
                    (Global<const Load>)(p + k * kStep));
#pragma unroll
        for (int k = 0; k < kSumBatch; ++k)
            if (i + k < loads)
                s[k] += square_sum<G>(x[k]);
#pragma unroll
        for (int k = 0; k < kSumBatch; ++k)
            x[k] = y[k];
    }
    double t = 0.0;
#pragma unroll
    for (int k = 0; k < kSumBatch; ++k)
        t += s[k];
    return t;
}

// threadIdx.x: lane, threadIdx.y: wave of the workgroup.
template <int WT, class G>
__global__ __launch_bounds__(kSumThreads) void sumsq_kernel(SumArgs a)
{
    __shared__ double lds[kSumWaves];
    const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.y);
    const int64_t first =
        ((int64_t)blockIdx.x * kSumWaves + wave) * a.per_wave;
    const int64_t end = min(first + a.per_wave, (int64_t)a.t.own);
    double s = 0.0;
    for (int64_t p = first; p < end;) {
        const Rec r = a.t.recs[a.t.tensor[p]];
        const int64_t off = (p - r.piece0) * kPiece;
        const int64_t left = r.numel - off;
        if (left < kPiece) {
            s += sum_piece<kEdge, WT, G>(a, r, off, {0, (int)left});
            ++p;
        } else if constexpr (WT == 1) {
            const int n = (int)min(left / kPiece, end - p);
            s += sum_run<G>(global<const G>(r.grad) + off, n);
            p += n;
        } else {
            // the flag is of where a step's units start
            s += r.flags & kRecFours && r.pre % 4 == 0
                     ? sum_piece<kAligned, WT, G>(a, r, off, {0, kPiece})
                     : sum_piece<kWhole, WT, G>(a, r, off, {0, kPiece});
            ++p;
        }
    }
    s = group_sum(s, lds, kSumWaves);
    if (threadIdx.x == 0 && threadIdx.y == 0)
        a.out[blockIdx.x] = s;
}

// The partial sums of `count` workgroups, to one.
constexpr int kLastThreads = 1024;
__global__ __launch_bounds__(kLastThreads) void sumsq_last_kernel(
    const double* part, int32_t count, double* out)
{
    __shared__ double lds[kLastThreads / kWave];
    double s = 0.0;
    for (int i = (int)threadIdx.x; i < count; i += kLastThreads)
        s += part[i];
    s = group_sum(s, lds, kLastThreads / kWave);
    if (threadIdx.x == 0)
        *out = s;
}

// ---- conversions

struct ConvertArgs {
    Table from, to;
};

template <int MODE, int U>
__device__ __forceinline__ void pack_part(const Rec& f, const Rec& t,
                                          int64_t off, Places q)
{
    const Global<const float> mp = global<const float>(f.m) + off;
    const Global<const float> vp = global<const float>(f.v) + off;
    const int lane = (int)threadIdx.x;
    Raw<float> mx[U], vx[U];
#pragma unroll
    for (int k = 0; k < U; ++k) {
        mx[k] = load4<MODE>(mp, 4 * (k * kWave + lane), q);
        vx[k] = load4<MODE>(vp, 4 * (k * kWave + lane), q);
    }
    float m[U][4], v[U][4], root[U][4];
#pragma unroll
    for (int k = 0; k < U; ++k)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            m[k][j] = mx[k].x[j];
            v[k][j] = vx[k].x[j];
        }
    roots<U>(v, root);
    uint32_t cm[U], cr[U];
    float S;
    hold<U>(m, root, 0, cm, cr, S);
    store_held<MODE, U>(global<uint8_t>(t.m) + off, global<uint8_t>(t.v) + off,
                        global<float>(t.ms) + off / kBlock,
                        global<float>(t.vs) + off / kBlock, q, cm, cr, S);
}

template <int MODE, int U>
__device__ __forceinline__ void unpack_part(const Rec& f, const Rec& t,
                                            int64_t off, Places q)
{
    const Global<const uint8_t> mp = global<const uint8_t>(f.m) + off;
    const Global<const uint8_t> vp = global<const uint8_t>(f.v) + off;
    const Global<const float> msp = global<const float>(f.ms) + off / kBlock;
    const Global<const float> vsp = global<const float>(f.vs) + off / kBlock;
    const int lane = (int)threadIdx.x;
    uint32_t mq[U], vq[U];
    float ms[U], vs[U];
#pragma unroll
    for (int k = 0; k < U; ++k) {
        mq[k] = load_codes<MODE>(mp, 4 * (k * kWave + lane), q);
        vq[k] = load_codes<MODE>(vp, 4 * (k * kWave + lane), q);
        const bool there = MODE != kEdge || k * kBlock < q.n;
        ms[k] = there ? msp[k] : 0.0f;
        vs[k] = there ? vsp[k] : 0.0f;
    }
#pragma unroll
    for (int k = 0; k < U; ++k) {
        V4 m, v;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float qm = (float)(int8_t)(mq[k] >> (8 * j));
            const float qv = (float)(uint8_t)(vq[k] >> (8 * j));
            const float r0 = (qv * qv) * vs[k];
            m.x[j] = (qm * fabsf(qm)) * ms[k];
            v.x[j] = r0 * r0;
        }
        store4<MODE>(global<float>(t.m) + off, 4 * (k * kWave + lane), q, m);
        store4<MODE>(global<float>(t.v) + off, 4 * (k * kWave + lane), q, v);
    }
}

template <bool PACK, int MODE, int U>
__device__ __forceinline__ void convert_part(const Rec& f, const Rec& t,
                                             int64_t off, Places q)
{
    if constexpr (PACK)
        pack_part<MODE, U>(f, t, off, q);
    else
        unpack_part<MODE, U>(f, t, off, q);
}

// Whether a record's fp32 states are aligned to four elements (its flags are of
// its own units).
__device__ __forceinline__ bool aligned16(const Rec& r)
{
    return (((uintptr_t)r.m | (uintptr_t)r.v) & 15) == 0;
}

template <bool PACK, int U>
__global__ __launch_bounds__(kWave) void convert_kernel(ConvertArgs a)
{
    // the pieces of the list in 8 bits, whose units are its blocks
    const Table& held = PACK ? a.to : a.from;
    const int32_t i = record_of<U>(held, blockIdx.x);
    const Rec f = a.from.recs[i];
    const Rec t = a.to.recs[i];
    const Part<U> q = part_of<U, false>(held, PACK ? t : f, blockIdx.x);
    if (q.n <= 0)
        return;
    if (q.whole && aligned16(PACK ? f : t))
        convert_part<PACK, kAligned, U>(f, t, q.off, {0, U * kBlock});
    else if (q.whole)
        convert_part<PACK, kWhole, U>(f, t, q.off, {0, U * kBlock});
    else
        convert_part<PACK, kEdge, U>(f, t, q.off, {0, q.n});
}

}  // namespace

// ---- host side ---------------------------------------------------------------

namespace {

// A stretch of device memory that a step reads or writes.
struct Span {
    uintptr_t lo, hi;
    bool written;
};

}  // namespace

struct zs_tensors {
    int32_t world = 1, grad_type = ZS_BF16, param_type = ZS_BF16;
    int32_t state = ZS_STATE_NONE;
    bool grads = false, params = false, master = false;
    int32_t max_group = 0;
    std::vector<int64_t> numel;         // of every tensor, empty ones too
    std::vector<Rec> recs;              // of those with elements
    std::vector<int32_t> tensor;        // record of each piece
    int32_t own = 0;                    // the tensors' own pieces
    std::vector<Span> states;           // m, v and scales, in order
    Table table = {nullptr, nullptr, 0, 0};
    int device = -1;
};

namespace {

using zs::fail;

bool aligned(const void* p, uintptr_t to)
{
    return reinterpret_cast<uintptr_t>(p) % to == 0;
}

int64_t recs_bytes(const zs_tensors* L)
{
    return ((int64_t)(L->recs.size() * sizeof(Rec)) + 15) / 16 * 16;
}

bool before(const Span& a, const Span& b)
{
    return a.lo < b.lo;
}

// Whether something written shares bytes with something else.
bool overlap(std::vector<Span>& s)
{
    std::sort(s.begin(), s.end(), before);
    uintptr_t any = 0, written = 0;     // ends of what began before
    for (const Span& x : s) {
        if (x.lo < (x.written ? any : written))
            return true;
        any = std::max(any, x.hi);
        if (x.written)
            written = std::max(written, x.hi);
    }
    return false;
}

void add_span(std::vector<Span>& s, const void* p, int64_t bytes,
              bool written)
{
    const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
    if (p && bytes > 0)
        s.push_back({lo, lo + (uintptr_t)bytes, written});
}

void state_spans(const zs_tensors* L, const Rec& r, std::vector<Span>& s)
{
    const int64_t per = L->state == ZS_STATE_8 ? 1 : 4;
    const int64_t blocks = (r.numel + kBlock - 1) / kBlock;
    add_span(s, r.m, r.numel * per, true);
    add_span(s, r.v, r.numel * per, true);
    add_span(s, r.ms, blocks * 4, true);
    add_span(s, r.vs, blocks * 4, true);
}

// Whether two lists, each in order and without overlaps, share bytes.
bool shared(const std::vector<Span>& a, const std::vector<Span>& b)
{
    for (size_t i = 0, j = 0; i < a.size() && j < b.size();) {
        if (a[i].lo < b[j].hi && b[j].lo < a[i].hi)
            return true;
        if (a[i].hi <= b[j].hi)
            ++i;
        else
            ++j;
    }
    return false;
}

// Checks of one tensor with elements against the list's first.
int check_tensor(const zs_tensors* L, int32_t k, const zs_tensor& t)
{
    const bool states = L->state != ZS_STATE_NONE;
    if (!t.grad == L->grads || !t.param == L->params ||
        !t.master == L->master)
        return fail(ZS_EINVAL, "tensor %d: grad, param and master are given "
                    "for every tensor or for none", k);
    if (!t.m == states || !t.v == states)
        return fail(ZS_EINVAL, "tensor %d: m and v %s", k,
                    states ? "missing" : "given without a state type");
    if (!t.m_scale == (L->state == ZS_STATE_8) ||
        !t.v_scale == (L->state == ZS_STATE_8))
        return fail(ZS_EINVAL, "tensor %d: scales belong to 8-bit states",
                    k);
    if (t.master && (!t.param || L->param_type != ZS_BF16))
        return fail(ZS_EINVAL, "tensor %d: a master belongs to bf16 "
                    "parameters", k);
    const int gs = L->grad_type == ZS_F32 ? 4 : 2;
    const int ps = L->param_type == ZS_F32 ? 4 : 2;
    if (!aligned(t.grad, gs) || !aligned(t.param, ps) ||
        !aligned(t.master, 4) || !aligned(t.m, 4) || !aligned(t.v, 4) ||
        !aligned(t.m_scale, 4) || !aligned(t.v_scale, 4))
        return fail(ZS_EALIGN, "tensor %d: a pointer is not aligned to its "
                    "element (codes: to 4 bytes)", k);
    if (t.numel > kMaxReach)
        return fail(ZS_ERANGE, "tensor %d: %lld elements", k,
                    (long long)t.numel);
    if (t.grad && L->world > 1) {
        if (t.grad_stride < t.numel)
            return fail(ZS_ERANGE, "tensor %d: grad_stride %lld < %lld "
                        "elements", k, (long long)t.grad_stride,
                        (long long)t.numel);
        if (t.grad_stride > (kMaxReach - t.numel) / (L->world - 1))
            return fail(ZS_ERANGE, "tensor %d: slices reach past 2^46 "
                        "elements", k);
    }
    return ZS_OK;
}

// Where a tensor's units start.  Blocks of 8-bit states start at its first
// element; with fp32 states the units may start later, where what the step
// writes is aligned to lines of 128 bytes, or at least everything to four
// elements (a flat buffer's views share their distance from a line).
void place(const zs_tensors* L, Rec& r)
{
    const int gs = L->grad_type == ZS_F32 ? 4 : 2;
    const int ps = L->param_type == ZS_F32 ? 4 : 2;
    const int ss = L->state == ZS_STATE_8 ? 1 : 4;
    auto at = [](const void* p, int lead, int size, int to) {
        return !p || (reinterpret_cast<uintptr_t>(p) +
                      (uintptr_t)(lead * size)) % to == 0;
    };
    auto fours = [&](int lead) {
        return at(r.grad, lead, gs, 4 * gs) && r.gstride % 4 == 0 &&
               at(r.param, lead, ps, 4 * ps) && at(r.master, lead, 4, 16) &&
               at(r.m, lead, ss, 4 * ss) && at(r.v, lead, ss, 4 * ss);
    };
    auto lines = [&](int lead) {
        return fours(lead) && at(r.param, lead, ps, 128) &&
               at(r.master, lead, 4, 128) && at(r.m, lead, 4, 128) &&
               at(r.v, lead, 4, 128);
    };
    int lead = 0;
    if (L->state == ZS_STATE_32 && r.param) {
        while (lead < 64 && !lines(lead))
            ++lead;
        if (lead == 64)
            for (lead = 3; lead > 0 && !fours(lead);)
                --lead;
    }
    r.pre = (kBlock - lead) % kBlock;
    r.flags = (fours(lead) ? kRecFours : 0) |
              (at(r.grad, lead, gs, 128) && r.gstride * gs % 128 == 0 ? kRecLines
                                                              : 0);
}

int build_list(zs_tensors* L, int32_t count, const zs_tensor* ts)
{
    std::vector<Span> spans;
    std::vector<int32_t> late;          // records with one piece more
    int64_t pieces = 0;
    const int gs = L->grad_type == ZS_F32 ? 4 : 2;
    const int ps = L->param_type == ZS_F32 ? 4 : 2;
    for (int32_t k = 0; k < count; ++k) {
        const zs_tensor& t = ts[k];
        if (t.numel < 0)
            return fail(ZS_EINVAL, "tensor %d: numel %lld < 0", k,
                        (long long)t.numel);
        if (t.group < 0 || t.group >= ZS_TENSORS_MAX_GROUPS)
            return fail(ZS_EINVAL, "tensor %d: group %d outside [0, %d)", k,
                        t.group, ZS_TENSORS_MAX_GROUPS);
        L->numel.push_back(t.numel);
        if (t.numel == 0)
            continue;
        if (L->recs.empty()) {
            L->grads = t.grad;
            L->params = t.param;
            L->master = t.master;
        }
        if (int rc = check_tensor(L, k, t))
            return rc;
        L->max_group = std::max(L->max_group, t.group);
        Rec r = {};
        r.grad = t.grad;
        r.gstride = L->world > 1 ? t.grad_stride : 0;
        r.param = t.param;
        r.master = t.master;
        r.m = t.m;
        r.v = t.v;
        r.ms = t.m_scale;
        r.vs = t.v_scale;
        r.numel = t.numel;
        r.piece0 = (int32_t)pieces;
        r.group = t.group;
        place(L, r);
        const int64_t own = (t.numel + kPiece - 1) / kPiece;
        if ((r.pre + t.numel + kPiece - 1) / kPiece > own)
            late.push_back((int32_t)L->recs.size());
        pieces += own;
        if (pieces + (int64_t)late.size() > kMaxPieces)
            return fail(ZS_ERANGE, "tensors 0 to %d have too many elements",
                        k);
        L->tensor.resize((size_t)pieces, (int32_t)L->recs.size());
        L->recs.push_back(r);
        add_span(spans, r.param, r.numel * ps, true);
        add_span(spans, r.master, r.numel * 4, true);
        state_spans(L, r, L->states);
        if (L->grads) {
            if ((int64_t)L->recs.size() * L->world > kMaxSlices)
                return fail(ZS_ERANGE, "more than 2^22 gradient slices");
            for (int32_t s = 0; s < L->world; ++s)
                add_span(spans, static_cast<const char*>(r.grad) +
                         (int64_t)s * r.gstride * gs, r.numel * gs, false);
        }
    }
    L->own = (int32_t)pieces;
    L->tensor.insert(L->tensor.end(), late.begin(), late.end());
    spans.insert(spans.end(), L->states.begin(), L->states.end());
    if (overlap(spans))
        return fail(ZS_EINVAL, "arrays that a step writes overlap one "
                    "another or the gradients");
    std::sort(L->states.begin(), L->states.end(), before);
    return ZS_OK;
}

// A list's use by a call: its table, on the current device.
int check_list(const zs_tensors* L, const char* name)
{
    if (!L) return fail(ZS_EINVAL, "%s is NULL", name);
    if (L->recs.empty())
        return ZS_OK;
    if (!L->table.recs)
        return fail(ZS_EINVAL, "%s has no table (zs_tensors_upload)", name);
    int dev = -1;
    const hipError_t e = hipGetDevice(&dev);
    if (e != hipSuccess)
        return fail(ZS_EDEVICE, "hipGetDevice: %s", hipGetErrorString(e));
    if (dev != L->device)
        return fail(ZS_EINVAL, "%s has its table on device %d, the current "
                    "device is %d", name, L->device, dev);
    return ZS_OK;
}

int check_launch(const char* what)
{
    const hipError_t err = hipGetLastError();
    if (err != hipSuccess)
        return fail(ZS_EDEVICE, "%s: %s", what, hipGetErrorString(err));
    return ZS_OK;
}

Ranks ranks_of(int32_t W)
{
    return {W, (float)W, (float)(1.0 / (double)W), (W & (W - 1)) == 0};
}

// bits: of the states.
int make_hp(const zs_adamw& hp, int64_t t, int32_t k, int bits, Hp& h)
{
    if (!std::isfinite(hp.lr) || !std::isfinite(hp.weight_decay))
        return fail(ZS_EINVAL, "group %d: lr and weight_decay must be "
                    "finite", k);
    if (!(hp.beta1 >= 0 && hp.beta1 < 1) || !(hp.beta2 >= 0 && hp.beta2 < 1))
        return fail(ZS_EINVAL, "group %d: betas must be in [0, 1)", k);
    if (!(hp.eps >= FLT_MIN) || !std::isfinite(hp.eps))
        return fail(ZS_EINVAL, "group %d: eps must be finite and at least "
                    "2^-126", k);
    // double precision, each constant rounded to fp32 once
    const double b1 = hp.beta1, b2 = hp.beta2, lr = hp.lr;
    const double bc2 = std::sqrt(1.0 - std::pow(b2, (double)t));
    h.b1 = hp.beta1;
    h.b2 = hp.beta2;
    h.omb1 = (float)(1.0 - b1);
    h.omb2 = (float)(1.0 - b2);
    h.ss = (float)(lr / (1.0 - std::pow(b1, (double)t)));
    h.bc2s = (float)bc2;
    h.ibc2s = (float)(1.0 / bc2);
    h.dec = (float)(1.0 - lr * (double)hp.weight_decay);
    h.eps = hp.eps;
    if (!std::isfinite(h.ss) || !std::isfinite(h.dec))
        return fail(ZS_EINVAL, "group %d: lr/(1-beta1^t) or "
                    "1-lr*weight_decay is not finite in fp32", k);
    // the 8-bit step's reciprocals have no subnormal results: an eps that
    // would need them is taken with its step size by a sixteenth, as are the
    // roots beside it
    if (bits == 8 && h.eps > 0x1p124f) {
        h.eps *= 0x1p-4f;
        h.ibc2s *= 0x1p-4f;
        h.ss *= 0x1p-4f;
    }
    return ZS_OK;
}

// One launch for each kLaunchPieces pieces of a list: run(first, workgroups),
// U units to a workgroup.
template <int U, class Run>
void for_pieces(int64_t pieces, Run run)
{
    for (int64_t first = 0; first < pieces; first += kLaunchPieces)
        run((int32_t)first,
            (uint32_t)(std::min(pieces - first, kLaunchPieces) * (4 / U)));
}

// Bytes that a CU's workgroups may have on their way from memory in a step.  A
// few workgroups per CU keep the rows that are open in HBM few (zs_step.hip
// has the same cap): with fp32 states 50 KB run the 124 M step in 537 us
// against 573 at as many workgroups as fit, W = 8 in 1392 against 1508 and
// fp32 weights in 914 against 1018; 44 to 60 KB are within 2 %.  The 8-bit
// step's waves live longer for their arithmetic and want 80 to 100 KB (318
// against 328 us with a master, W = 4 763 against 824).
constexpr int kInFlight32 = 50 << 10, kInFlight8 = 88 << 10;

// Workgroups of U units per CU, 0 for as many as fit.
template <int BITS, int U, int WM, class G>
int step_residency(int32_t W)
{
    constexpr int kRest = (WM == kBf16 ? 2 : 4) + (BITS == 32 ? 8 : 2);
    const int64_t bytes =
        (int64_t)U * kBlock * (kRest + (int64_t)W * (int)sizeof(G));
    const int64_t k = (BITS == 32 ? kInFlight32 : kInFlight8) / bytes;
    return k > 24 ? 0 : (int)std::max<int64_t>(k, 6);
}

template <int BITS, int WM, int WT, class G>
void launch_step_u(const zs_tensors* L, StepArgs& a, hipStream_t s)
{
    constexpr int U = BITS == 32 ? kStep32Units : kStep8Units;
    const unsigned lds =
        zs::residency_lds(step_residency<BITS, U, WM, G>(a.ranks.W));
    for_pieces<U>((int64_t)L->tensor.size(), [&](int32_t first,
                                                 uint32_t groups) {
        a.t.first = first;
        step_kernel<BITS, U, WM, WT, G><<<groups, kWave, lds, s>>>(a);
    });
}

// Four and eight ranks at compile time have all loads on their way without a
// branch between them (W = 8 1390 us against 1463, W = 4 1123 against 1140;
// W = 2 984 both ways).
template <int BITS, int WM, class G>
void launch_step_w(const zs_tensors* L, StepArgs& a, hipStream_t s)
{
    switch (a.ranks.W) {
    case 1: launch_step_u<BITS, WM, 1, G>(L, a, s); break;
    case 4: launch_step_u<BITS, WM, 4, G>(L, a, s); break;
    case 8: launch_step_u<BITS, WM, 8, G>(L, a, s); break;
    default: launch_step_u<BITS, WM, 0, G>(L, a, s); break;
    }
}

template <int BITS, class G>
void launch_step_wm(const zs_tensors* L, StepArgs& a, hipStream_t s)
{
    if (L->master)
        launch_step_w<BITS, kMaster, G>(L, a, s);
    else if (L->param_type == ZS_BF16)
        launch_step_w<BITS, kBf16, G>(L, a, s);
    else
        launch_step_w<BITS, kF32, G>(L, a, s);
}

template <int BITS>
void launch_step(const zs_tensors* L, StepArgs& a, hipStream_t s)
{
    if (L->grad_type == ZS_BF16)
        launch_step_wm<BITS, uint16_t>(L, a, s);
    else
        launch_step_wm<BITS, float>(L, a, s);
}

template <bool PACK, int U>
void launch_convert(int64_t pieces, ConvertArgs& a, hipStream_t s)
{
    const unsigned lds = zs::residency_lds(PACK ? 0 : kUnpackResidency);
    for_pieces<U>(pieces, [&](int32_t first, uint32_t groups) {
        a.from.first = a.to.first = first;
        convert_kernel<PACK, U><<<groups, kWave, lds, s>>>(a);
    });
}

// How zs_tensors_sumsq cuts a list: pieces of each wave, and workgroups.
void sum_plan(const zs_tensors* L, int32_t& per_wave, int32_t& groups)
{
    const int64_t pieces = L->own;
    const int64_t most = pieces <= kSumOne ? 1 : kSumMaxGroups;
    const int64_t waves = most * kSumWaves;
    per_wave = (int32_t)std::max<int64_t>(1, (pieces + waves - 1) / waves);
    const int64_t per_group = (int64_t)per_wave * kSumWaves;
    groups = (int32_t)std::max<int64_t>(
        1, (pieces + per_group - 1) / per_group);
}

template <class G>
void launch_sum(const SumArgs& a, uint32_t groups, hipStream_t s)
{
    const dim3 block(kWave, kSumWaves);
    if (a.ranks.W == 1)
        sumsq_kernel<1, G><<<groups, block, 0, s>>>(a);
    else
        sumsq_kernel<0, G><<<groups, block, 0, s>>>(a);
}

}  // namespace

extern "C" int zs_tensors_create(int32_t count, const zs_tensor* tensors,
                                 int32_t world, int32_t grad_type,
                                 int32_t param_type, int32_t state,
                                 zs_tensors** out)
{
    zs::clear_error();
    if (!out) return fail(ZS_EINVAL, "out is NULL");
    *out = nullptr;
    if (count < 0) return fail(ZS_EINVAL, "count %d < 0", count);
    if (count > 0 && !tensors) return fail(ZS_EINVAL, "tensors is NULL");
    if (world < 1) return fail(ZS_EINVAL, "world %d < 1", world);
    if (grad_type != ZS_BF16 && grad_type != ZS_F32)
        return fail(ZS_EINVAL, "unknown grad_type %d", grad_type);
    if (param_type != ZS_BF16 && param_type != ZS_F32)
        return fail(ZS_EINVAL, "unknown param_type %d", param_type);
    if (state != ZS_STATE_NONE && state != ZS_STATE_32 &&
        state != ZS_STATE_8)
        return fail(ZS_EINVAL, "unknown state %d", state);
    zs_tensors* L = new (std::nothrow) zs_tensors;
    if (!L) return fail(ZS_ENOMEM, "host allocation");
    L->world = world;
    L->grad_type = grad_type;
    L->param_type = param_type;
    L->state = state;
    int rc;
    try {
        rc = build_list(L, count, tensors);
    } catch (const std::exception&) {
        rc = fail(ZS_ENOMEM, "host allocation");
    }
    if (rc != ZS_OK) {
        delete L;
        return rc;
    }
    *out = L;
    return ZS_OK;
}

extern "C" void zs_tensors_free(zs_tensors* L)
{
    delete L;
}

extern "C" int zs_tensors_table_bytes(const zs_tensors* L, int64_t* bytes)
{
    zs::clear_error();
    if (!L || !bytes) return fail(ZS_EINVAL, "list and bytes must be "
                                  "non-NULL");
    *bytes = recs_bytes(L) + (int64_t)L->tensor.size() * 4;
    return ZS_OK;
}

extern "C" int zs_tensors_upload(zs_tensors* L, void* table, int64_t bytes,
                                 void* hip_stream)
{
    int64_t need = 0;
    if (int rc = zs_tensors_table_bytes(L, &need))
        return rc;
    if (need == 0)
        return ZS_OK;
    if (L->table.recs)
        return fail(ZS_EINVAL, "the list has its table");
    if (!table) return fail(ZS_EINVAL, "table is NULL");
    if (!aligned(table, 16))
        return fail(ZS_EALIGN, "table not 16-byte aligned");
    if (bytes < need)
        return fail(ZS_ERANGE, "table of %lld bytes, %lld are needed",
                    (long long)bytes, (long long)need);
    hipStream_t s = static_cast<hipStream_t>(hip_stream);
    hipStreamCaptureStatus cap = hipStreamCaptureStatusNone;
    hipError_t e = hipStreamIsCapturing(s, &cap);
    if (e != hipSuccess) {
        (void)hipGetLastError();
        return fail(ZS_EDEVICE, "hipStreamIsCapturing: %s",
                    hipGetErrorString(e));
    }
    if (cap != hipStreamCaptureStatusNone)
        return fail(ZS_EINVAL, "the upload waits for its copy: not under "
                    "capture");
    int dev = -1;
    e = hipGetDevice(&dev);
    char* const at = static_cast<char*>(table);
    if (e == hipSuccess)
        e = hipMemcpyAsync(at, L->recs.data(), L->recs.size() * sizeof(Rec),
                           hipMemcpyHostToDevice, s);
    if (e == hipSuccess)
        e = hipMemcpyAsync(at + recs_bytes(L), L->tensor.data(),
                           L->tensor.size() * 4, hipMemcpyHostToDevice, s);
    // also after an error: the copies read the list's own memory
    const hipError_t waited = hipStreamSynchronize(s);
    if (e == hipSuccess)
        e = waited;
    if (e != hipSuccess) {
        (void)hipGetLastError();
        return fail(ZS_EDEVICE, "table copy: %s", hipGetErrorString(e));
    }
    L->table.recs = reinterpret_cast<const Rec*>(at);
    L->table.tensor = reinterpret_cast<const int32_t*>(at + recs_bytes(L));
    L->table.own = L->own;
    L->device = dev;
    return ZS_OK;
}

extern "C" int zs_tensors_step(const zs_tensors* L, const zs_adamw* hp,
                               int32_t n_hp, int64_t step,
                               const double* sumsq, float max_norm,
                               void* hip_stream)
{
    zs::clear_error();
    if (!L) return fail(ZS_EINVAL, "list is NULL");
    if (!hp) return fail(ZS_EINVAL, "hp is NULL");
    if (n_hp < 1 || n_hp > ZS_TENSORS_MAX_GROUPS)
        return fail(ZS_EINVAL, "n_hp %d outside [1, %d]", n_hp,
                    ZS_TENSORS_MAX_GROUPS);
    if (step < 1) return fail(ZS_EINVAL, "step %lld < 1", (long long)step);
    if (sumsq && !(max_norm > 0))
        return fail(ZS_EINVAL, "max_norm must be positive");
    if (!aligned(sumsq, 8)) return fail(ZS_EALIGN, "sumsq not 8-byte aligned");
    StepArgs a = {};
    for (int32_t k = 0; k < n_hp; ++k)
        if (int rc = make_hp(hp[k], step, k, L->state, a.hp[k]))
            return rc;
    if (L->recs.empty())
        return ZS_OK;
    if (!L->grads || !L->params || L->state == ZS_STATE_NONE)
        return fail(ZS_EINVAL, "a step needs gradients, parameters and "
                    "states");
    if (L->max_group >= n_hp)
        return fail(ZS_EINVAL, "a tensor of group %d, n_hp is %d",
                    L->max_group, n_hp);
    if (int rc = check_list(L, "list"))
        return rc;
    a.t = L->table;
    a.sumsq = sumsq;
    a.max_norm = max_norm;
    a.ranks = ranks_of(L->world);
    hipStream_t s = static_cast<hipStream_t>(hip_stream);
    if (L->state == ZS_STATE_32)
        launch_step<32>(L, a, s);
    else
        launch_step<8>(L, a, s);
    return check_launch("tensor step kernel");
}

extern "C" int zs_tensors_sumsq_workspace(const zs_tensors* L,
                                          int64_t* bytes)
{
    zs::clear_error();
    if (!L || !bytes) return fail(ZS_EINVAL, "list and bytes must be "
                                  "non-NULL");
    int32_t per_wave, groups;
    sum_plan(L, per_wave, groups);
    *bytes = groups > 1 ? (int64_t)groups * 8 : 0;
    return ZS_OK;
}

extern "C" int zs_tensors_sumsq(const zs_tensors* L, double* out,
                                void* workspace, int64_t workspace_bytes,
                                void* hip_stream)
{
    int64_t need = 0;
    if (int rc = zs_tensors_sumsq_workspace(L, &need))
        return rc;
    if (!out) return fail(ZS_EINVAL, "out is NULL");
    if (!aligned(out, 8)) return fail(ZS_EALIGN, "out not 8-byte aligned");
    if (!L->recs.empty() && !L->grads)
        return fail(ZS_EINVAL, "the list has no gradients");
    if (need > 0) {
        if (!workspace) return fail(ZS_EINVAL, "workspace is NULL");
        if (!aligned(workspace, 16))
            return fail(ZS_EALIGN, "workspace not 16-byte aligned");
    }
    if (workspace_bytes < need)
        return fail(ZS_ERANGE, "workspace of %lld bytes, %lld are needed",
                    (long long)workspace_bytes, (long long)need);
    if (int rc = check_list(L, "list"))
        return rc;
    SumArgs a = {};
    int32_t groups;
    sum_plan(L, a.per_wave, groups);
    a.t = L->table;
    a.ranks = ranks_of(L->world);
    a.out = groups > 1 ? static_cast<double*>(workspace) : out;
    hipStream_t s = static_cast<hipStream_t>(hip_stream);
    if (L->grad_type == ZS_BF16)
        launch_sum<uint16_t>(a, (uint32_t)groups, s);
    else
        launch_sum<float>(a, (uint32_t)groups, s);
    if (groups > 1)
        sumsq_last_kernel<<<1, kLastThreads, 0, s>>>(a.out, groups, out);
    return check_launch("sum of squares kernel");
}

extern "C" int zs_tensors_convert(const zs_tensors* from,
                                  const zs_tensors* to, void* hip_stream)
{
    zs::clear_error();
    if (!from || !to) return fail(ZS_EINVAL, "lists must be non-NULL");
    if (from->numel != to->numel)
        return fail(ZS_EINVAL, "the lists have other sizes");
    const bool pack = from->state == ZS_STATE_32 && to->state == ZS_STATE_8;
    if (!pack && !(from->state == ZS_STATE_8 && to->state == ZS_STATE_32))
        return fail(ZS_EINVAL, "need one list of 32-bit and one of 8-bit "
                    "states");
    if (from->recs.empty())
        return ZS_OK;
    if (shared(from->states, to->states))
        return fail(ZS_EINVAL, "the lists' states overlap");
    if (int rc = check_list(from, "from"))
        return rc;
    if (int rc = check_list(to, "to"))
        return rc;
    ConvertArgs a = {from->table, to->table};
    // those of the list in 8 bits, as in convert_kernel
    const int64_t pieces = (int64_t)(pack ? to : from)->tensor.size();
    hipStream_t s = static_cast<hipStream_t>(hip_stream);
    if (pack)
        launch_convert<true, kPackUnits>(pieces, a, s);
    else
        launch_convert<false, kUnpackUnits>(pieces, a, s);
    return check_launch("state conversion kernel");
}
