// Lists of tensors: the AdamW step with states in 32 bits or in 8, the
// gradients' sum of squares, and the conversion of states, with their host
// side.  Written for gfx950 (CDNA4, wave64).
//
// All four are streams bounded by HBM: per element a step reads W gradients,
// the weights and the states and writes weights and states back (28 bytes
// with bf16 gradients, a master and fp32 states; 16 with 8-bit ones; 10 with
// 8-bit states and no master).
//
// A list's tensors are cut into pieces of kPiece elements, one one-wave
// workgroup each, so one launch takes any number of tensors of any sizes.  A
// workgroup finds its tensor in the list's table in device memory (the
// tensor's number for each piece, then the tensor's record; both are
// wave-uniform and come by scalar loads).

#include <hip/hip_runtime.h>

#include <algorithm>
#include <cfloat>
#include <cmath>
#include <cstdint>
#include <new>
#include <vector>

#include "zs_device.h"
#include "zs_internal.h"
#include "zs_tensors.h"

namespace {

typedef unsigned int u32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
// the same at any element's address; the hardware takes vector accesses at
// such addresses whole
typedef u32x2 u32x2_2 __attribute__((aligned(2)));
typedef f32x4 f32x4_4 __attribute__((aligned(4)));

constexpr int kWave = 64;
constexpr int kBlock = ZS_STATE8_BLOCK;
static_assert(kBlock == 4 * kWave, "a wave's unit is one block");
constexpr int kUnits = 4;
constexpr int kPiece = kBlock * kUnits;
// HIP launches fewer than 2^32 work-items along x
constexpr int64_t kMaxPieces = (int64_t(1) << 26) - 1;
constexpr int64_t kMaxReach = int64_t(1) << 46;
constexpr int64_t kMaxSlices = int64_t(1) << 30;

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
    int32_t vec;        // every pointer and stride aligned to four elements
    int32_t pad;
};
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
};

struct StepArgs {
    Table t;
    const double* sumsq;        // nullable
    float max_norm;
    int32_t W;
    float fw, invw;             // W and 1/W
    int32_t pow2;               // W is a power of two (1/W exact)
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

// fp32 -> bf16 bits, nearest even; NaN -> quiet NaN keeping sign and the
// top payload bits.
__device__ __forceinline__ uint32_t to_bf16(float f)
{
    const uint32_t u = __float_as_uint(f);
    if ((u & 0x7fffffffu) > 0x7f800000u)
        return (u >> 16) | 0x40u;
    return (u + 0x7fffu + ((u >> 16) & 1u)) >> 16;
}

struct V4 {
    float x[4];
};

// Elements i .. i+3 of p.  FAST: all four exist and lie at an aligned
// address.  Else those below n; the others are 0.
template <bool FAST>
__device__ __forceinline__ V4 load4(const float* p, int i, int n)
{
    if constexpr (FAST) {
        const f32x4 a = __builtin_nontemporal_load(
            reinterpret_cast<const f32x4*>(p + i));
        return {a.x, a.y, a.z, a.w};
    }
    if (i + 4 <= n) {
        const f32x4 a = *reinterpret_cast<const f32x4_4*>(p + i);
        return {a.x, a.y, a.z, a.w};
    }
    V4 r = {0, 0, 0, 0};
#pragma unroll
    for (int j = 0; j < 3; ++j)
        if (i + j < n)
            r.x[j] = p[i + j];
    return r;
}

template <bool FAST>
__device__ __forceinline__ V4 load4(const uint16_t* p, int i, int n)
{
    u32x2 a;
    if constexpr (FAST) {
        a = __builtin_nontemporal_load(reinterpret_cast<const u32x2*>(p + i));
    } else if (i + 4 <= n) {
        a = *reinterpret_cast<const u32x2_2*>(p + i);
    } else {
        V4 r = {0, 0, 0, 0};
#pragma unroll
        for (int j = 0; j < 3; ++j)
            if (i + j < n)
                r.x[j] = __uint_as_float((uint32_t)p[i + j] << 16);
        return r;
    }
    return {bf16_lo(a.x), bf16_hi(a.x), bf16_lo(a.y), bf16_hi(a.y)};
}

// Stores of a piece whose first element is at p (wave-uniform): streamed on
// to HBM where it is whole, else element by element below n.
template <bool FAST>
__device__ __forceinline__ void store4(float* p, int i, int n, const V4& r)
{
    if constexpr (FAST) {
        zsdev::stream_store(p, kPiece * 4u, (uint32_t)i * 4u,
                            f32x4{r.x[0], r.x[1], r.x[2], r.x[3]});
        return;
    }
    if (i + 4 <= n) {
        *reinterpret_cast<f32x4_4*>(p + i) =
            f32x4{r.x[0], r.x[1], r.x[2], r.x[3]};
        return;
    }
#pragma unroll
    for (int j = 0; j < 3; ++j)
        if (i + j < n)
            p[i + j] = r.x[j];
}

template <bool FAST>
__device__ __forceinline__ void store4(uint16_t* p, int i, int n, const V4& r)
{
    const uint32_t b[4] = {to_bf16(r.x[0]), to_bf16(r.x[1]), to_bf16(r.x[2]),
                           to_bf16(r.x[3])};
    const u32x2 q = {b[0] | (b[1] << 16), b[2] | (b[3] << 16)};
    if constexpr (FAST) {
        zsdev::stream_store(p, kPiece * 2u, (uint32_t)i * 2u, q);
        return;
    }
    if (i + 4 <= n) {
        *reinterpret_cast<u32x2_2*>(p + i) = q;
        return;
    }
#pragma unroll
    for (int j = 0; j < 3; ++j)
        if (i + j < n)
            p[i + j] = (uint16_t)b[j];
}

// Four codes in a word.
template <bool FAST>
__device__ __forceinline__ uint32_t load_codes(const uint8_t* p, int i, int n)
{
    if constexpr (FAST)
        return __builtin_nontemporal_load(
            reinterpret_cast<const uint32_t*>(p + i));
    if (i + 4 <= n)
        return *reinterpret_cast<const uint32_t*>(p + i);
    uint32_t r = 0;
#pragma unroll
    for (int j = 0; j < 3; ++j)
        if (i + j < n)
            r |= (uint32_t)p[i + j] << (8 * j);
    return r;
}

template <bool FAST>
__device__ __forceinline__ void store_codes(uint8_t* p, int i, int n,
                                            uint32_t q)
{
    if constexpr (FAST) {
        zsdev::stream_store(p, kPiece, (uint32_t)i, q);
        return;
    }
    if (i + 4 <= n) {
        *reinterpret_cast<uint32_t*>(p + i) = q;
        return;
    }
#pragma unroll
    for (int j = 0; j < 3; ++j)
        if (i + j < n)
            p[i + j] = (uint8_t)(q >> (8 * j));
}

// The sum over W slices in rank order, from the first (so that the sign of a
// zero sum is its own), then the mean.  All loads of a batch of slices come
// before its adds.
template <bool FAST, int WT, class G>
__device__ __forceinline__ void mean4(const G* g0, int64_t gs, int n, int W,
                                      float fw, float invw, int pow2,
                                      V4 (&g)[kUnits])
{
    const int lane = (int)threadIdx.x;
    if constexpr (WT == 1) {
#pragma unroll
        for (int k = 0; k < kUnits; ++k)
            g[k] = load4<FAST>(g0, 4 * (k * kWave + lane), n);
        return;
    }
    constexpr int NB = 4;
#pragma unroll
    for (int k = 0; k < kUnits; ++k)
        g[k] = load4<FAST>(g0, 4 * (k * kWave + lane), n);
#pragma unroll 1
    for (int s0 = 1; s0 < W; s0 += NB) {
        V4 x[NB][kUnits];
#pragma unroll
        for (int s = 0; s < NB; ++s)
            if (s0 + s < W)
#pragma unroll
                for (int k = 0; k < kUnits; ++k)
                    x[s][k] = load4<FAST>(g0 + (int64_t)(s0 + s) * gs,
                                          4 * (k * kWave + lane), n);
#pragma unroll
        for (int s = 0; s < NB; ++s)
            if (s0 + s < W)
#pragma unroll
                for (int k = 0; k < kUnits; ++k)
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        g[k].x[j] = g[k].x[j] + x[s][k].x[j];
    }
#pragma unroll
    for (int k = 0; k < kUnits; ++k)
#pragma unroll
        for (int j = 0; j < 4; ++j)
            g[k].x[j] = pow2 ? g[k].x[j] * invw : g[k].x[j] / fw;
}

// ---- codes

// The largest of a wave's unsigned numbers, in every lane: bits of |x| order
// as |x| does, with infinity above all numbers and NaN above infinity.
__device__ __forceinline__ uint32_t wave_max(uint32_t x)
{
#define ZS_DPP_MAX(ctrl, rows)                                               \
    {                                                                        \
        const uint32_t y = (uint32_t)__builtin_amdgcn_update_dpp(            \
            0, (int)x, ctrl, rows, 0xf, false);                              \
        x = x > y ? x : y;                                                   \
    }
    ZS_DPP_MAX(0x111, 0xf)      // row_shr 1, 2, 4, 8: lane 15 of each row
    ZS_DPP_MAX(0x112, 0xf)
    ZS_DPP_MAX(0x114, 0xf)
    ZS_DPP_MAX(0x118, 0xf)
    ZS_DPP_MAX(0x142, 0xa)      // row_bcast 15 into rows 1 and 3
    ZS_DPP_MAX(0x143, 0xc)      // row_bcast 31 into rows 2 and 3
#undef ZS_DPP_MAX
    return (uint32_t)__builtin_amdgcn_readlane((int)x, 63);
}

__device__ __forceinline__ uint32_t abs_bits(float x)
{
    return __float_as_uint(x) & 0x7fffffffu;
}

// S and f32(top^2 / A) of a block whose largest |x| has the bits a.
template <int TOP>
__device__ __forceinline__ void scale_of(uint32_t a, float& S, float& inv)
{
    constexpr float kTop2 = (float)(TOP * TOP);
    const float A = __uint_as_float(a);
    S = A * (float)(1.0 / (double)(TOP * TOP));
    inv = kTop2 / A;
    if (a < 0x0d800000u) {              // below 2^-100
        S = 0.0f;
        inv = 0.0f;
    }
    if (a >= 0x7f800000u) {             // an infinity or a NaN
        S = __uint_as_float(0x7fc00000u);
        inv = 0.0f;
    }
}

// The whole number q with (q - 1/2)^2 <= y < (q + 1/2)^2, y >= 0, as a float.
// The hardware's root is within an ulp; less 2^-10 the guess is q or one
// below it, and (q + 1/2)^2 = (q^2 + 1/4) + q is exact in fp32 up to 255.
__device__ __forceinline__ float root_code(float y)
{
    float q = floorf(__builtin_amdgcn_sqrtf(y) + (0.5f - 0x1p-10f));
    const float up = __builtin_fmaf(q, q, 0.25f) + q;
    return up <= y ? q + 1.0f : q;
}

// ---- the step

// g c, or no step at all: *sumsq not finite.
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
    return s - s == 0.0;
}

// Kinds of weights.
constexpr int kMaster = 0, kBf16 = 1, kF32 = 2;

template <bool FAST, int WM>
struct Weights {
    V4 w[kUnits];
    __device__ void load(const Rec& r, int64_t off, int n)
    {
#pragma unroll
        for (int k = 0; k < kUnits; ++k) {
            const int i = 4 * (k * kWave + (int)threadIdx.x);
            if constexpr (WM == kMaster)
                w[k] = load4<FAST>(r.master + off, i, n);
            else if constexpr (WM == kBf16)
                w[k] = load4<FAST>(static_cast<const uint16_t*>(r.param) +
                                   off, i, n);
            else
                w[k] = load4<FAST>(static_cast<const float*>(r.param) + off,
                                   i, n);
        }
    }
    __device__ void store(const Rec& r, int64_t off, int n, int k) const
    {
        const int i = 4 * (k * kWave + (int)threadIdx.x);
        if constexpr (WM == kMaster)
            store4<FAST>(r.master + off, i, n, w[k]);
        if constexpr (WM == kF32)
            store4<FAST>(static_cast<float*>(r.param) + off, i, n, w[k]);
        else
            store4<FAST>(static_cast<uint16_t*>(r.param) + off, i, n, w[k]);
    }
};

template <bool FAST, int WM, int WT, class G>
__device__ __forceinline__ void step32_piece(const StepArgs& a, const Rec& r,
                                             int64_t off, int n)
{
    float* const mp = static_cast<float*>(r.m) + off;
    float* const vp = static_cast<float*>(r.v) + off;
    const int lane = (int)threadIdx.x;
    Weights<FAST, WM> w;
    V4 m[kUnits], v[kUnits], g[kUnits];
    w.load(r, off, n);
#pragma unroll
    for (int k = 0; k < kUnits; ++k) {
        m[k] = load4<FAST>(mp, 4 * (k * kWave + lane), n);
        v[k] = load4<FAST>(vp, 4 * (k * kWave + lane), n);
    }
    mean4<FAST, WT>(static_cast<const G*>(r.grad) + off, r.gstride, n, a.W,
                    a.fw, a.invw, a.pow2, g);
    const Hp h = a.hp[r.group];
    float c;
    if (!clip_of(a.sumsq, a.max_norm, c))
        return;
#pragma unroll
    for (int k = 0; k < kUnits; ++k) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float gi = g[k].x[j] * c;
            const float mi = h.b1 * m[k].x[j] + h.omb1 * gi;
            const float vi = h.b2 * v[k].x[j] + h.omb2 * (gi * gi);
            const float den = sqrtf(vi) / h.bc2s + h.eps;
            w.w[k].x[j] = w.w[k].x[j] * h.dec - h.ss * (mi / den);
            m[k].x[j] = mi;
            v[k].x[j] = vi;
        }
        w.store(r, off, n, k);
        store4<FAST>(mp, 4 * (k * kWave + lane), n, m[k]);
        store4<FAST>(vp, 4 * (k * kWave + lane), n, v[k]);
    }
}

template <bool FAST, int WM, int WT, class G>
__device__ __forceinline__ void step8_piece(const StepArgs& a, const Rec& r,
                                            int64_t off, int n)
{
    uint8_t* const mp = static_cast<uint8_t*>(r.m) + off;
    uint8_t* const vp = static_cast<uint8_t*>(r.v) + off;
    float* const msp = r.ms + off / kBlock;
    float* const vsp = r.vs + off / kBlock;
    const int lane = (int)threadIdx.x;
    Weights<FAST, WM> w;
    uint32_t mq[kUnits], vq[kUnits];
    float ms[kUnits], vs[kUnits];
    V4 g[kUnits];
    w.load(r, off, n);
#pragma unroll
    for (int k = 0; k < kUnits; ++k) {
        mq[k] = load_codes<FAST>(mp, 4 * (k * kWave + lane), n);
        vq[k] = load_codes<FAST>(vp, 4 * (k * kWave + lane), n);
        const bool there = FAST || k * kBlock < n;
        ms[k] = there ? msp[k] : 0.0f;
        vs[k] = there ? vsp[k] : 0.0f;
    }
    mean4<FAST, WT>(static_cast<const G*>(r.grad) + off, r.gstride, n, a.W,
                    a.fw, a.invw, a.pow2, g);
    const Hp h = a.hp[r.group];
    float c;
    if (!clip_of(a.sumsq, a.max_norm, c))
        return;
#pragma unroll
    for (int k = 0; k < kUnits; ++k) {
        if (!FAST && k * kBlock >= n)
            break;
        float m[4], root[4];
        uint32_t am = 0, ar = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float qm = (float)(int8_t)(mq[k] >> (8 * j));
            const float qv = (float)(uint8_t)(vq[k] >> (8 * j));
            const float r0 = (qv * qv) * vs[k];
            const float gi = g[k].x[j] * c;
            const float mi = h.b1 * ((qm * fabsf(qm)) * ms[k]) + h.omb1 * gi;
            const float vi = h.b2 * (r0 * r0) + h.omb2 * (gi * gi);
            root[j] = sqrtf(vi);
            m[j] = mi;
            const float den = root[j] * h.ibc2s + h.eps;
            w.w[k].x[j] = w.w[k].x[j] * h.dec -
                          h.ss * (mi * __builtin_amdgcn_rcpf(den));
            // elements behind the tensor's last are 0 here: gradient and
            // codes were loaded as 0
            am = max(am, abs_bits(mi));
            ar = max(ar, abs_bits(root[j]));
        }
        w.store(r, off, n, k);
        float Sm, im, Sr, ir;
        scale_of<127>(wave_max(am), Sm, im);
        scale_of<255>(wave_max(ar), Sr, ir);
        uint32_t cm = 0, cr = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            float q = root_code(fabsf(m[j]) * im);
            cm |= ((uint32_t)(int)copysignf(q, m[j]) & 0xffu) << (8 * j);
            q = root_code(root[j] * ir);
            if (root[j] > 0.0f && ir > 0.0f)
                q = fmaxf(q, 1.0f);
            cr |= (uint32_t)q << (8 * j);
        }
        store_codes<FAST>(mp, 4 * (k * kWave + lane), n, cm);
        store_codes<FAST>(vp, 4 * (k * kWave + lane), n, cr);
        if (lane == 0) {
            msp[k] = Sm;
            vsp[k] = Sr;
        }
    }
}

template <int BITS, int WM, int WT, class G>
__global__ __launch_bounds__(kWave) void step_kernel(StepArgs a)
{
    const int32_t p = (int32_t)blockIdx.x;
    const Rec& r = a.t.recs[a.t.tensor[p]];
    const int64_t off = (int64_t)(p - r.piece0) * kPiece;
    const int64_t left = r.numel - off;
    if (left >= kPiece && r.vec) {
        if constexpr (BITS == 32)
            step32_piece<true, WM, WT, G>(a, r, off, kPiece);
        else
            step8_piece<true, WM, WT, G>(a, r, off, kPiece);
    } else {
        const int n = left < kPiece ? (int)left : kPiece;
        if constexpr (BITS == 32)
            step32_piece<false, WM, WT, G>(a, r, off, n);
        else
            step8_piece<false, WM, WT, G>(a, r, off, n);
    }
}

// ---- the sum of squares

constexpr int kSumThreads = 256;
constexpr int kSumWaves = kSumThreads / kWave;
constexpr int kSumMaxGroups = 2048;     // workgroups, and so partial sums
constexpr int64_t kSumOne = 32;         // pieces that one workgroup takes alone

struct SumArgs {
    Table t;
    int32_t pieces;
    int32_t per_wave;           // consecutive pieces of a wave
    int32_t W;
    float fw, invw;
    int32_t pow2;
    double* out;                // one per workgroup
};

template <bool FAST, int WT, class G>
__device__ __forceinline__ double sum_piece(const SumArgs& a, const Rec& r,
                                            int64_t off, int n)
{
    V4 g[kUnits];
    const int lane = (int)threadIdx.x & (kWave - 1);
    (void)lane;
    mean4<FAST, WT>(static_cast<const G*>(r.grad) + off, r.gstride, n, a.W,
                    a.fw, a.invw, a.pow2, g);
    double s = 0.0;
#pragma unroll
    for (int k = 0; k < kUnits; ++k)
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

// threadIdx.x: lane, threadIdx.y: wave of the workgroup.
template <int WT, class G>
__global__ __launch_bounds__(kSumThreads) void sumsq_kernel(SumArgs a)
{
    __shared__ double lds[kSumWaves];
    const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.y);
    const int64_t first =
        ((int64_t)blockIdx.x * kSumWaves + wave) * a.per_wave;
    const int64_t end = min(first + a.per_wave, (int64_t)a.pieces);
    double s = 0.0;
    for (int64_t p = first; p < end; ++p) {
        const Rec& r = a.t.recs[a.t.tensor[p]];
        const int64_t off = (int64_t)((int32_t)p - r.piece0) * kPiece;
        const int64_t left = r.numel - off;
        if (left >= kPiece && r.vec)
            s += sum_piece<true, WT, G>(a, r, off, kPiece);
        else
            s += sum_piece<false, WT, G>(a, r, off,
                                         left < kPiece ? (int)left : kPiece);
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

template <bool FAST>
__device__ __forceinline__ void pack_piece(const Rec& f, const Rec& t,
                                           int64_t off, int n)
{
    const float* const mp = static_cast<const float*>(f.m) + off;
    const float* const vp = static_cast<const float*>(f.v) + off;
    const int lane = (int)threadIdx.x;
    V4 m[kUnits], v[kUnits];
#pragma unroll
    for (int k = 0; k < kUnits; ++k) {
        m[k] = load4<FAST>(mp, 4 * (k * kWave + lane), n);
        v[k] = load4<FAST>(vp, 4 * (k * kWave + lane), n);
    }
#pragma unroll
    for (int k = 0; k < kUnits; ++k) {
        if (!FAST && k * kBlock >= n)
            break;
        uint32_t am = 0, ar = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            v[k].x[j] = sqrtf(v[k].x[j]);
            am = max(am, abs_bits(m[k].x[j]));
            ar = max(ar, abs_bits(v[k].x[j]));
        }
        float Sm, im, Sr, ir;
        scale_of<127>(wave_max(am), Sm, im);
        scale_of<255>(wave_max(ar), Sr, ir);
        uint32_t cm = 0, cr = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            float q = root_code(fabsf(m[k].x[j]) * im);
            cm |= ((uint32_t)(int)copysignf(q, m[k].x[j]) & 0xffu)
                  << (8 * j);
            q = root_code(v[k].x[j] * ir);
            if (v[k].x[j] > 0.0f && ir > 0.0f)
                q = fmaxf(q, 1.0f);
            cr |= (uint32_t)q << (8 * j);
        }
        store_codes<FAST>(static_cast<uint8_t*>(t.m) + off,
                          4 * (k * kWave + lane), n, cm);
        store_codes<FAST>(static_cast<uint8_t*>(t.v) + off,
                          4 * (k * kWave + lane), n, cr);
        if (lane == 0) {
            t.ms[off / kBlock + k] = Sm;
            t.vs[off / kBlock + k] = Sr;
        }
    }
}

template <bool FAST>
__device__ __forceinline__ void unpack_piece(const Rec& f, const Rec& t,
                                             int64_t off, int n)
{
    const uint8_t* const mp = static_cast<const uint8_t*>(f.m) + off;
    const uint8_t* const vp = static_cast<const uint8_t*>(f.v) + off;
    const int lane = (int)threadIdx.x;
    uint32_t mq[kUnits], vq[kUnits];
    float ms[kUnits], vs[kUnits];
#pragma unroll
    for (int k = 0; k < kUnits; ++k) {
        mq[k] = load_codes<FAST>(mp, 4 * (k * kWave + lane), n);
        vq[k] = load_codes<FAST>(vp, 4 * (k * kWave + lane), n);
        const bool there = FAST || k * kBlock < n;
        ms[k] = there ? f.ms[off / kBlock + k] : 0.0f;
        vs[k] = there ? f.vs[off / kBlock + k] : 0.0f;
    }
#pragma unroll
    for (int k = 0; k < kUnits; ++k) {
        V4 m, v;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float qm = (float)(int8_t)(mq[k] >> (8 * j));
            const float qv = (float)(uint8_t)(vq[k] >> (8 * j));
            const float r0 = (qv * qv) * vs[k];
            m.x[j] = (qm * fabsf(qm)) * ms[k];
            v.x[j] = r0 * r0;
        }
        store4<FAST>(static_cast<float*>(t.m) + off, 4 * (k * kWave + lane),
                     n, m);
        store4<FAST>(static_cast<float*>(t.v) + off, 4 * (k * kWave + lane),
                     n, v);
    }
}

template <bool PACK>
__global__ __launch_bounds__(kWave) void convert_kernel(ConvertArgs a)
{
    const int32_t p = (int32_t)blockIdx.x;
    const int32_t i = a.from.tensor[p];
    const Rec& f = a.from.recs[i];
    const Rec& t = a.to.recs[i];
    const int64_t off = (int64_t)(p - f.piece0) * kPiece;
    const int64_t left = f.numel - off;
    if (left >= kPiece && f.vec && t.vec) {
        if constexpr (PACK)
            pack_piece<true>(f, t, off, kPiece);
        else
            unpack_piece<true>(f, t, off, kPiece);
    } else {
        const int n = left < kPiece ? (int)left : kPiece;
        if constexpr (PACK)
            pack_piece<false>(f, t, off, n);
        else
            unpack_piece<false>(f, t, off, n);
    }
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
    std::vector<Span> states;           // m, v and scales, in order
    Table table = {nullptr, nullptr};
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

int build_list(zs_tensors* L, int32_t count, const zs_tensor* ts)
{
    std::vector<Span> spans;
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
        const int ss = L->state == ZS_STATE_8 ? 1 : 4;
        r.vec = aligned(t.grad, 4 * gs) && r.gstride % 4 == 0 &&
                aligned(t.param, 4 * ps) && aligned(t.master, 16) &&
                aligned(t.m, 4 * ss) && aligned(t.v, 4 * ss);
        pieces += (t.numel + kPiece - 1) / kPiece;
        if (pieces > kMaxPieces)
            return fail(ZS_ERANGE, "tensors 0 to %d have too many elements",
                        k);
        L->tensor.resize((size_t)pieces, (int32_t)L->recs.size());
        L->recs.push_back(r);
        add_span(spans, r.param, r.numel * ps, true);
        add_span(spans, r.master, r.numel * 4, true);
        state_spans(L, r, L->states);
        if (L->grads) {
            if ((int64_t)L->recs.size() * L->world > kMaxSlices)
                return fail(ZS_ERANGE, "more than 2^30 gradient slices");
            for (int32_t s = 0; s < L->world; ++s)
                add_span(spans, static_cast<const char*>(r.grad) +
                         (int64_t)s * r.gstride * gs, r.numel * gs, false);
        }
    }
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

template <class A>
void set_world(A& a, int32_t W)
{
    a.W = W;
    a.fw = (float)W;
    a.invw = (float)(1.0 / (double)W);
    a.pow2 = (W & (W - 1)) == 0;
}

int make_hp(const zs_adamw& hp, int64_t t, int32_t k, Hp& h)
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
    return ZS_OK;
}

template <int BITS, int WM, class G>
void launch_step_w(const StepArgs& a, uint32_t pieces, hipStream_t s)
{
    if (a.W == 1)
        step_kernel<BITS, WM, 1, G><<<pieces, kWave, 0, s>>>(a);
    else
        step_kernel<BITS, WM, 0, G><<<pieces, kWave, 0, s>>>(a);
}

template <int BITS, class G>
void launch_step_wm(const zs_tensors* L, const StepArgs& a, hipStream_t s)
{
    const uint32_t pieces = (uint32_t)L->tensor.size();
    if (L->master)
        launch_step_w<BITS, kMaster, G>(a, pieces, s);
    else if (L->param_type == ZS_BF16)
        launch_step_w<BITS, kBf16, G>(a, pieces, s);
    else
        launch_step_w<BITS, kF32, G>(a, pieces, s);
}

template <int BITS>
void launch_step(const zs_tensors* L, const StepArgs& a, hipStream_t s)
{
    if (L->grad_type == ZS_BF16)
        launch_step_wm<BITS, uint16_t>(L, a, s);
    else
        launch_step_wm<BITS, float>(L, a, s);
}

// How zs_tensors_sumsq cuts a list: pieces of each wave, and workgroups.
void sum_plan(const zs_tensors* L, int32_t& per_wave, int32_t& groups)
{
    const int64_t pieces = (int64_t)L->tensor.size();
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
    if (a.W == 1)
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
        if (int rc = make_hp(hp[k], step, k, a.hp[k]))
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
    set_world(a, L->world);
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
    a.pieces = (int32_t)L->tensor.size();
    set_world(a, L->world);
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
    const ConvertArgs a = {from->table, to->table};
    const uint32_t pieces = (uint32_t)from->tensor.size();
    hipStream_t s = static_cast<hipStream_t>(hip_stream);
    if (pack)
        convert_kernel<true><<<pieces, kWave, 0, s>>>(a);
    else
        convert_kernel<false><<<pieces, kWave, 0, s>>>(a);
    return check_launch("state conversion kernel");
}
