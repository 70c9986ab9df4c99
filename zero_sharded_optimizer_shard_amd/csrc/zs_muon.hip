// Orthogonalisation by Newton-Schulz products and the Muon step over
// whole-tensor layouts (include/zs_muon.h).  gfx950 (CDNA4, wave64).
//
// With X = U / (|U|_F + eps) and m <= n its sides, one step is
//   gram     A = X X^T            symmetric: one triangle of tiles, m^2 n flops
//   poly     C = a + b A + c A A  symmetric: one triangle of tiles, m^3
//   update   X <- C X             2 m^2 n
// (X^T X and X C for a matrix with more rows than columns), on the matrix
// cores: D[i][j] = sum_k P[i][k] Q[j][k] with both operands contiguous along
// k.  gram multiplies the rows of X's shorter side, update needs the rows of
// its longer side, so X is kept in both orientations: Xd [rows][cols] as the
// caller has it and Xt [cols][rows].
//
// Numbers.  Operands are fp16 times 2^10: |X| <= 1, so entries reach from
// 2^10 down to the mean 2^10 / sqrt(rows cols) = 0.022 of the largest shapes
// (2^31 elements), in fp16's normal range.  Sums are fp32.  What is rounded to fp16, and what
// is not:
//  - X is a pair (hi, lo), 22 bits; products use hi, the term a X uses both.
//    Rounded to fp16 alone, the rounding of each step would enter the null
//    directions of a matrix of low rank and grow by a = 3.4 a step (rank 8 of
//    1024: 4e-2 of the result's norm against 3e-4).  What the products round
//    there grows all the same (zs_muon.h has what is left).
//    What is left is mostly hi's rounding in the gram (512 x 1024: 4.6e-4 of
//    5.7e-4; C's 2.2e-4, A's 2.1e-4, the update's 1.3e-4), which two more
//    products would take away: a quarter of the work three times over.
//  - The diagonals of A and C are fp32 vectors, and zero in the fp16
//    matrices: near the end A is close to the identity, and the rounding of
//    its diagonal would be most of the error.  (R + D)(R + D) = R R + D R +
//    R D + D D, the last three element by element.
//  - In full precision (FULL) the squares and X^T are pairs too and every
//    product is three: hi hi + hi lo + lo hi.
//  - fp16 ends at 2^-24, which is 2^-34 of X.  A matrix whose norm is below eps
//    starts at |X| = |U| / (|U| + eps) << 1 and would lose its bits there, so
//    it is held as 2^e X, with 2^e |X| in [1/2, 1).  A step that can multiply
//    it by g takes t = ceil(log2 g) from e, by way of C alone: with
//    e' = max(e - t, 0) and A' = 2^2e A as the gram gives it
//      2^(e' - e) C = 2^(e' - e) (a + b 2^-2e A' + c 2^-4e A' A')
//    (zs_muon_plan.h: shift_of).  Matrices of norm eps and above have e = 0,
//    and powers of two round nothing.
//
// Launches: the norm (or the momentum, which leaves U and its norm), X_0, and
// three products a step, for all matrices of a call at once; small matrices
// take all steps in one launch.  What bounds them on MI355X: from 4096 a side
// on the matrix cores, which are busy 52-66 % of the cycles of a square's
// launch and 43-57 % of an update's, whose epilogue moves ten bytes an element
// (more with the master) with nothing beside it; up to about 1024 a side the
// launches themselves, each 5-7 us plus 0.18 us for 64 k (0.5 us in full
// precision).
//
// Padding.  Every matrix is stored with its sides rounded up to 64 and zeros
// behind, which the products preserve, so the k loop has no edge; rows past
// the end of an operand are read from its last row and their results are not
// stored.

#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>

#include "zs_internal.h"
#include "zs_muon.h"
#include "zs_muon_plan.h"

namespace {

using namespace zs::muon;

typedef unsigned int u32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef _Float16 f16;
typedef f16 f16x4 __attribute__((ext_vector_type(4)));
typedef f16 f16x8 __attribute__((ext_vector_type(8)));

constexpr int kScaleBits = 10;
constexpr float kScale = 1 << kScaleBits, kUnscale = 1 / kScale;
constexpr int64_t kTile = ZS_TILE;

// Where its parts lie: E elements of X, S of a square, D of a diagonal, over
// the whole stack, and in one matrix e, s and mp.
//   Xd[2] hi, lo | Xt[2] hi (lo) | kSquares m x m matrices, each hi (lo)
//   | their diagonals | e (int32) of each matrix | partial sums (double)
// The momentum kernel's U (fp32) lies where Xd[1] will be: it is read by the
// normalising kernel, before the first update writes there.
constexpr int kSquares = 4;
enum Square { kA, kC, kT, kC2 };         // what they hold: run_steps

template <bool FULL>
struct Region {
    char* ws;
    int32_t rp, cp, mp;                 // padded sides, the smaller one
    int64_t e, s, E, S, D, exps;
    __host__ __device__ Region(char* w, int32_t R, int32_t C, int32_t batch)
        : ws(w), exps(((int64_t)batch + 1) / 2 * 8)
    {
        rp = padded(R);
        cp = padded(C);
        mp = rp < cp ? rp : cp;
        e = (int64_t)rp * cp;
        s = (int64_t)mp * mp;
        E = batch * e;
        S = batch * s;
        D = (int64_t)batch * mp;
    }
    __device__ f16* xd(int p) const { return (f16*)(ws + 4 * p * E); }
    __device__ f16* xt(int p) const
    {
        return (f16*)(ws + 8 * E + (FULL ? 4 : 2) * p * E);
    }
    __host__ __device__ int64_t x_bytes() const
    {
        return (FULL ? 16 : 12) * E;
    }
    __host__ __device__ int64_t d_off() const
    {
        return x_bytes() + (FULL ? 4 : 2) * kSquares * S;
    }
    __host__ __device__ int64_t exp_off() const
    {
        return d_off() + 4 * kSquares * D;
    }
    __host__ __device__ int64_t parts_off() const
    {
        return exp_off() + exps;
    }
    __device__ f16* square(int k) const
    {
        return (f16*)(ws + x_bytes() + (FULL ? 4 : 2) * k * S);
    }
    __device__ float* diag(int k) const
    {
        return (float*)(ws + d_off() + 4 * k * D);
    }
    __device__ int32_t* exponent() const
    {
        return (int32_t*)(ws + exp_off());
    }
    __host__ __device__ double* parts() const
    {
        return (double*)(ws + parts_off());
    }
    __host__ float* u() const { return (float*)(ws + 4 * E); }  // xd(1)
};

// The stack of workgroup `bid`, and the workgroup's index within it.  All
// starts are read at once: kernel arguments are far away, and a search would
// wait for each in turn.
__device__ __forceinline__ int find(const Group& g, uint32_t& bid)
{
    int p = 0;
    uint32_t s = 0;
#pragma unroll
    for (int k = 1; k < kMaxMats; ++k) {
        const uint32_t t = g.start[k];
        p = bid >= t ? k : p;
        s = bid >= t ? t : s;
    }
    bid -= s;
    return p;
}

__device__ __forceinline__ float bf16_to_f32(uint32_t u)
{
    return __uint_as_float(u << 16);
}

__device__ __forceinline__ uint32_t to_bf16(float f)
{
    const uint32_t u = __float_as_uint(f);
    if ((u & 0x7fffffffu) > 0x7f800000u)
        return (u >> 16) | 0x40u;
    return (u + 0x7fffu + ((u >> 16) & 1u)) >> 16;
}

// ---- sums of squares -------------------------------------------------------

constexpr int kNT = 256;                // threads of the elementwise kernels
// Elements behind one partial sum: a workgroup takes them at once, all loads
// before the arithmetic.
constexpr int kNormChunk = 8192, kMomChunk = 2048;
constexpr int32_t kMaxParts = 2048;     // more are summed by a launch of their
                                        // own

// Sum over the workgroup in a fixed order, for every thread.
template <int NT = kNT>
__device__ __forceinline__ double block_sum(double v)
{
    __shared__ double s[NT / 64];
    for (int d = 32; d; d >>= 1)
        v += __shfl_down(v, d, 64);
    if ((threadIdx.x & 63) == 0)
        s[threadIdx.x >> 6] = v;
    __syncthreads();
    double t = 0;
    for (int w = 0; w < NT / 64; ++w)
        t += s[w];
    return t;
}

struct Source {                         // a caller's stack of matrices
    const void* x;
    int64_t batch, row;                 // strides in elements
    int32_t vec;                        // four elements at a time
};

struct NormArgs {
    Group g;
    Source src[kMaxMats];
};

template <bool BF16>
__device__ __forceinline__ f32x4 load4(const void* x, int64_t i)
{
    if constexpr (BF16) {
        const u32x2 u = *reinterpret_cast<const u32x2*>(
            static_cast<const uint16_t*>(x) + i);
        return f32x4{bf16_to_f32(u.x), __uint_as_float(u.x & 0xffff0000u),
                     bf16_to_f32(u.y), __uint_as_float(u.y & 0xffff0000u)};
    } else {
        return *reinterpret_cast<const f32x4*>(
            static_cast<const float*>(x) + i);
    }
}

template <bool BF16>
__device__ __forceinline__ float load1(const void* x, int64_t i)
{
    if constexpr (BF16)
        return bf16_to_f32(static_cast<const uint16_t*>(x)[i]);
    else
        return static_cast<const float*>(x)[i];
}

__device__ __forceinline__ double sq4(f32x4 v)
{
    return (double)v.x * v.x + (double)v.y * v.y + (double)v.z * v.z +
           (double)v.w * v.w;
}

// Partial sums of squares of the callers' matrices: workgroup = one chunk of
// one matrix.  Squares and sums in 64 bits: a gradient's squares leave
// fp32's range long before the gradient does.
template <bool BF16, bool FULL>
__global__ __launch_bounds__(kNT) void ns_norm_kernel(NormArgs a)
{
    uint32_t bid = blockIdx.x;
    const int p = find(a.g, bid);
    const Mat& m = a.g.m[p];
    const Source& s = a.src[p];
    const uint32_t b = bid / m.nparts, part = bid % m.nparts;
    const uint32_t n = (uint32_t)m.R * m.C;
    const uint32_t e0 = part * kNormChunk;
    const uint32_t e1 = n - e0 < (uint32_t)kNormChunk ? n : e0 + kNormChunk;
    double sum = 0;
    if (s.vec) {
        constexpr int U = kNormChunk / (4 * kNT);
        f32x4 x[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const uint32_t e = e0 + 4 * (u * kNT + threadIdx.x);
            x[u] = f32x4{0, 0, 0, 0};
            if (e < e1) {
                const uint32_t r = e / m.C, c = e % m.C;
                x[u] = load4<BF16>(s.x, b * s.batch + r * s.row + c);
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
            sum += sq4(x[u]);
    } else {
        for (uint32_t e = e0 + threadIdx.x; e < e1; e += kNT) {
            const uint32_t r = e / m.C, c = e % m.C;
            const double v =
                load1<BF16>(s.x, b * s.batch + r * s.row + c);
            sum += v * v;
        }
    }
    sum = block_sum(sum);
    if (threadIdx.x == 0)
        Region<FULL>(m.ws, m.R, m.C, m.batch)
            .parts()[(int64_t)b * m.nparts + part] = sum;
}

// ---- the step's momentum ---------------------------------------------------

struct MomSrc {
    const uint16_t* grads;
    float* state;                       // the tensor's first tile
    float* u;                           // where U goes
    double* parts;                      // and its partial sums of squares,
                                        // NULL where nobody reads them
};

struct MomArgs {
    Group g;
    MomSrc src[kMaxMats];
    int64_t gstride;                    // slices: elements between slices
    int32_t W, nesterov;
    float mu, fw, invw;
    int32_t pow2;                       // W is a power of two (1/W exact)
};

// g = mean of the W slices, M <- mu M + g, U to the workspace, partial sums
// of U's squares.  2W + 8 bytes read and written in the state and gradients
// and 4 for U, per element; bound by HBM.  VEC: four elements a thread
// (every row of four stays inside a tile, tiles being multiples of four).
template <int WT, bool TILED, bool VEC>
__device__ __forceinline__ void momentum_part(const MomArgs& a, const Mat& m,
                                              const MomSrc& s, uint32_t bid)
{
    constexpr int V = VEC ? 4 : 1, U = kMomChunk / (V * kNT);
    constexpr int NB = WT ? WT : 8;     // slices loaded at a time
    constexpr int UB = VEC ? U : 2;     // and elements (V each)
    const uint32_t b = bid / m.nparts, part = bid % m.nparts;
    const uint32_t n = (uint32_t)m.R * m.C;
    const uint32_t e0 = part * kMomChunk;
    const uint32_t e1 = n - e0 < (uint32_t)kMomChunk ? n : e0 + kMomChunk;
    const int W = WT ? WT : a.W;
    double sum = 0;
#pragma unroll
    for (int u0 = 0; u0 < U; u0 += UB) {
        f32x4 mom[UB], acc[UB];         // V of each four in use
        float* mp[UB];
        const uint16_t* gp[UB];
        int64_t ge[UB];
        bool in[UB];
        const int64_t gs = TILED ? kTile : a.gstride;
#pragma unroll
        for (int u = 0; u < UB; ++u) {
            const uint32_t e = e0 + V * ((u0 + u) * kNT + threadIdx.x);
            in[u] = e < e1;
            ge[u] = (int64_t)b * n + e;
            const int64_t tile = ge[u] / kTile, pos = ge[u] % kTile;
            gp[u] = TILED ? s.grads + tile * W * kTile + pos : s.grads + ge[u];
            mp[u] = s.state + (tile * 3 + 1) * kTile + pos;
            if (in[u]) {
                if constexpr (VEC)
                    mom[u] = __builtin_nontemporal_load(
                        reinterpret_cast<const f32x4*>(mp[u]));
                else
                    mom[u].x = *mp[u];
            }
        }
        for (int s0 = 0; s0 < W; s0 += NB) {
            u32x2 x[UB][NB];
#pragma unroll
            for (int u = 0; u < UB; ++u)
#pragma unroll
                for (int i = 0; i < NB; ++i)
                    if (in[u] && (WT || s0 + i < W)) {
                        const uint16_t* const g = gp[u] + (s0 + i) * gs;
                        if constexpr (VEC)
                            x[u][i] = __builtin_nontemporal_load(
                                reinterpret_cast<const u32x2*>(g));
                        else
                            x[u][i].x = *g;
                    }
#pragma unroll
            for (int u = 0; u < UB; ++u)
#pragma unroll
                for (int i = 0; i < NB; ++i)
                    if (WT || s0 + i < W) {
                        const f32x4 v = {
                            bf16_to_f32(x[u][i].x),
                            __uint_as_float(x[u][i].x & 0xffff0000u),
                            bf16_to_f32(x[u][i].y),
                            __uint_as_float(x[u][i].y & 0xffff0000u)};
#pragma unroll
                        for (int k = 0; k < V; ++k)
                            acc[u][k] =
                                s0 + i == 0 ? v[k] : acc[u][k] + v[k];
                    }
        }
#pragma unroll
        for (int u = 0; u < UB; ++u) {
            if (!in[u])
                continue;
            f32x4 up;
#pragma unroll
            for (int k = 0; k < V; ++k) {
                const float g =
                    a.pow2 ? acc[u][k] * a.invw : acc[u][k] / a.fw;
                const float t = a.mu * mom[u][k];
                mom[u][k] = t + g;
                const float t2 = a.mu * mom[u][k];
                up[k] = a.nesterov ? g + t2 : mom[u][k];
                sum += (double)up[k] * up[k];
            }
            if constexpr (VEC) {
                __builtin_nontemporal_store(mom[u],
                                            reinterpret_cast<f32x4*>(mp[u]));
                *reinterpret_cast<f32x4*>(s.u + ge[u]) = up;
            } else {
                *mp[u] = mom[u].x;
                s.u[ge[u]] = up.x;
            }
        }
    }
    if (!s.parts)
        return;
    sum = block_sum(sum);
    if (threadIdx.x == 0)
        s.parts[(int64_t)b * m.nparts + part] = sum;
}

template <int WT, bool TILED>
__global__ __launch_bounds__(kNT) void muon_momentum_kernel(MomArgs a)
{
    uint32_t bid = blockIdx.x;
    const int p = find(a.g, bid);
    const Mat& m = a.g.m[p];
    if (((uint32_t)m.R * m.C) % 4 == 0)
        momentum_part<WT, TILED, true>(a, m, a.src[p], bid);
    else
        momentum_part<WT, TILED, false>(a, m, a.src[p], bid);
}

// A matrix's many partial sums into the first of them: workgroup = one matrix.
constexpr int kSumNT = 1024;

template <bool FULL>
__global__ __launch_bounds__(kSumNT) void ns_sum_kernel(Group g)
{
    uint32_t b = blockIdx.x;
    const Mat& m = g.m[find(g, b)];
    double* const parts = Region<FULL>(m.ws, m.R, m.C, m.batch).parts() +
                          (int64_t)b * m.nparts;
    double sum = 0;
    for (int i = threadIdx.x; i < m.nparts; i += 8 * kSumNT) {
        double x[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const int n = i + k * kSumNT;
            x[k] = n < m.nparts ? parts[n] : 0;
        }
#pragma unroll
        for (int k = 0; k < 8; ++k)
            sum += x[k];
    }
    sum = block_sum<kSumNT>(sum);       // every thread has read its own
    if (threadIdx.x == 0)
        parts[0] = sum;
}

// ---- X = U / (|U| + eps) into the workspace --------------------------------

struct InitArgs {
    Group g;
    Source src[kMaxMats];
    float eps;
    int32_t summed;                     // the first partial sum is the sum
};

__device__ __forceinline__ void split(float x, f16& hi, f16& lo)
{
    hi = (f16)x;
    lo = (f16)(x - (float)hi);
}

// What a matrix of this norm is multiplied by, and its e (at the top).  One
// with a NaN or an infinity is NaN everywhere.
__device__ __forceinline__ double start_scale(double norm, float eps, int& e)
{
    e = 0;
    if (!(norm < HUGE_VAL))
        return NAN;
    if (norm > 0) {
        int x;
        frexp(norm / (norm + (double)eps), &x);
        e = x < 0 ? -x : 0;
    }
    return ldexp((double)kScale / (norm + (double)eps), e);
}

// Workgroup = one 64 x 64 tile of one padded matrix: read U, scale, write Xd
// (hi, lo) and, through LDS, Xt.
template <bool BF16, bool FULL>
__global__ __launch_bounds__(kNT) void ns_init_kernel(InitArgs a)
{
    __shared__ f16 t[FULL ? 2 : 1][64][64 + 4];
    uint32_t bid = blockIdx.x;
    const int p = find(a.g, bid);
    const Mat& m = a.g.m[p];
    const Region<FULL> w(m.ws, m.R, m.C, m.batch);
    const uint32_t tc = w.cp / 64, tiles = tc * (w.rp / 64);
    const uint32_t b = bid / tiles;
    bid %= tiles;
    const int r0 = bid / tc * 64, c0 = bid % tc * 64;
    // the matrix's sum of squares, every workgroup in the same order
    double sum = 0;
    const double* const parts = w.parts() + (int64_t)b * m.nparts;
    const int nparts = a.summed ? 1 : m.nparts;
    for (int i = threadIdx.x; i < nparts; i += kNT)
        sum += parts[i];
    sum = block_sum(sum);
    int ex;
    const double inv = start_scale(sqrt(sum), a.eps, ex);
    if (bid == 0 && threadIdx.x == 0)
        w.exponent()[b] = ex;
    const Source& s = a.src[p];
    const int tx = threadIdx.x % 16 * 4, ty = threadIdx.x / 16;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const int r = r0 + ty + 16 * k, c = c0 + tx;
        f32x4 v = {0, 0, 0, 0};
        if (r < m.R && c < m.C) {
            const int64_t i = b * s.batch + r * s.row + c;
            if (s.vec) {
                v = load4<BF16>(s.x, i);
            } else {
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    if (c + q < m.C)
                        v[q] = load1<BF16>(s.x, i + q);
            }
        }
        f16x4 hi, lo;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            f16 h, l;
            split((float)((double)v[q] * inv), h, l);
            hi[q] = h;
            lo[q] = l;
            t[0][tx + q][ty + 16 * k] = h;
            if constexpr (FULL)
                t[1][tx + q][ty + 16 * k] = l;
        }
        const int64_t o = b * w.e + (int64_t)r * w.cp + c;
        *reinterpret_cast<f16x4*>(w.xd(0) + o) = hi;
        *reinterpret_cast<f16x4*>(w.xd(0) + w.E + o) = lo;
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const int c = ty + 16 * k;
        const int64_t o = b * w.e + (int64_t)(c0 + c) * w.rp + r0 + tx;
        *reinterpret_cast<f16x4*>(w.xt(0) + o) =
            *reinterpret_cast<const f16x4*>(&t[0][c][tx]);
        if constexpr (FULL)
            *reinterpret_cast<f16x4*>(w.xt(0) + w.E + o) =
                *reinterpret_cast<const f16x4*>(&t[1][c][tx]);
    }
}

// ---- the products ----------------------------------------------------------

struct OutMat {
    void* o;
    int64_t batch, row;
    int32_t vec;
};

struct StepMat {
    float* state;                       // the tensor's first tile
    uint16_t* pshard;                   // nullable, at the tensor
    uint16_t* flat;                     // nullable, at the tensor
    float s;                            // lr * shape's scale
};

struct GemmArgs {
    Group g;
    union {
        OutMat out[kMaxMats];
        StepMat st[kMaxMats];
    };
    int32_t parity;                     // which of the two X is read
    int8_t sp, sq, so;                  // squares: operands and result
    // kPoly: shifts before and after its step; the last update: all of them
    int16_t shift, shift1;
    float a, b, c;
    float dec;                          // 1 - lr*wd
};
static_assert(sizeof(GemmArgs) <= 4096 && sizeof(MomArgs) <= 4096 &&
              sizeof(NormArgs) <= 4096, "kernel arguments");

typedef __attribute__((address_space(1))) const void gptr;
typedef __attribute__((address_space(3))) void lptr;

// Workgroup shape of the products: a BT x BT tile of D, WI x WJ waves, each
// with FI x FJ accumulators of 16 x 16, ST stages of 64 k in LDS.
template <int BT_, int WI_, int WJ_, int ST_>
struct Shape {
    static constexpr int BT = BT_, WI = WI_, WJ = WJ_, ST = ST_;
    static constexpr int kWaves = WI * WJ, kThreads = 64 * kWaves;
    static constexpr bool kTurns = kWaves == 8;     // see the kernel
    static constexpr int FI = BT / WI / 16, FJ = BT / WJ / 16;
    static constexpr int kRow = 128;                // bytes of a stage's row
    static constexpr int kHalf = BT * kRow;         // bytes per operand
    // 1 KiB load instructions of a wave per stage; the first half of the
    // waves loads P, the second Q
    static constexpr int kLoads = 2 * kHalf / 1024 / kWaves;
    static_assert(kLoads * 512 * kWaves == kHalf && FI % 2 == 0, "shape");
};

// Two waves a SIMD taking turns (the loop is described in the kernel): the
// large tile feeds the matrix cores best (updates of 4096 x 4096 and 8192 x
// 8192, epilogues with them: 147 and 1025 us, 0.93 and 1.07 PFLOP/s; the 192
// tile 190 and 1312 us, the 128 tile 173 and 1165, the 64 tile 241 and 1830),
// the smaller ones fill the chip where there are few of the larger (squares of
// 4096: 136 tiles of 256 103 us, 256 of 192 85 us).
typedef Shape<256, 2, 4, 2> Shape256;
typedef Shape<192, 2, 4, 2> Shape192;
typedef Shape<128, 2, 4, 2> Shape128;
// Small matrices are bound by the latency of a launch and of a stage: four
// stages in LDS (eight in a longer loop cost 3 to 7 % more a call).
typedef Shape<64, 2, 2, 4> Shape64;

// s_waitcnt immediate: at most vm vector loads and lg LDS operations out.
constexpr int wait_count(int vm, int lg)
{
    return (vm & 15) | ((vm >> 4) << 14) | (7 << 4) | (lg << 8);
}

__device__ __forceinline__ void slot_barrier()
{
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
}

// Workgroups go to the 8 XCDs in turn; give each XCD a run of neighbouring
// tiles of each stack, whose operands its L2 then holds.  A stack's first
// workgroup is a multiple of 8.
__device__ __forceinline__ uint32_t xcd_order(uint32_t bid, uint32_t n)
{
    const uint32_t x = bid & 7, per = n >> 3, rem = n & 7;
    return x * per + (x < rem ? x : rem) + (bid >> 3);
}

// A lane's FJ columns of one row, v[0..FJ-1][q]; `left` columns are there.
template <int FJ>
__device__ __forceinline__ void store_cols(f16* o, const f16x8 (&v)[FJ],
                                           int q, int left)
{
    if constexpr (FJ == 3) {            // not a vector's size
#pragma unroll
        for (int j = 0; j < FJ; ++j)
            if (j < left)
                o[j] = v[j][q];
    } else {
        typedef f16 cols __attribute__((ext_vector_type(FJ)));
        cols t;
#pragma unroll
        for (int j = 0; j < FJ; ++j)
            t[j] = v[j][q];
        *reinterpret_cast<cols*>(o) = t;
    }
}

// The last update's results v[0..3], times 2^-un, at row j and columns
// i .. i+3 of matrix b (i a multiple of 4; columns past the last are not
// there), to the caller's matrix.
template <int EPI>
__device__ __forceinline__ void finish_out(const OutMat& om, const Mat& m,
                                           uint32_t b, int j, int i,
                                           const float* v, int un)
{
    const int64_t o = b * om.batch + j * om.row + i;
    float x[4];
#pragma unroll
    for (int q = 0; q < 4; ++q)
        x[q] = ldexpf(v[q], un);
    if constexpr (EPI == kOutF32) {
        float* const op = static_cast<float*>(om.o) + o;
        if (om.vec) {
            *reinterpret_cast<f32x4*>(op) = f32x4{x[0], x[1], x[2], x[3]};
        } else {
#pragma unroll
            for (int q = 0; q < 4; ++q)
                if (i + q < m.C)
                    op[q] = x[q];
        }
    } else {
        uint16_t* const op = static_cast<uint16_t*>(om.o) + o;
        if (om.vec) {
            *reinterpret_cast<u32x2*>(op) =
                u32x2{to_bf16(x[0]) | (to_bf16(x[1]) << 16),
                      to_bf16(x[2]) | (to_bf16(x[3]) << 16)};
        } else {
#pragma unroll
            for (int q = 0; q < 4; ++q)
                if (i + q < m.C)
                    op[q] = (uint16_t)to_bf16(x[q]);
        }
    }
}

// The same into the weights: by fours where rows are (`st`, already
// stepped), else one by one.
__device__ __forceinline__ void finish_step(const GemmArgs& a, int p,
                                            const Mat& m, uint32_t b, int j,
                                            int i, bool vec4, const float* v,
                                            int un, f32x4 st)
{
    const StepMat& sm = a.st[p];
    const int64_t e = ((int64_t)b * m.R + j) * m.C + i;
    if (vec4) {
        *reinterpret_cast<f32x4*>(sm.state + e / kTile * 3 * kTile +
                                  e % kTile) = st;
        const u32x2 h = {to_bf16(st[0]) | (to_bf16(st[1]) << 16),
                         to_bf16(st[2]) | (to_bf16(st[3]) << 16)};
        if (sm.pshard)
            *reinterpret_cast<u32x2*>(sm.pshard + e) = h;
        if (sm.flat)
            *reinterpret_cast<u32x2*>(sm.flat + e) = h;
    } else {
        const f32x4 vv = {v[0], v[1], v[2], v[3]};
        const int n = m.C - i < 4 ? m.C - i : 4;
#pragma unroll 1
        for (int q = 0; q < n; ++q) {
            const int64_t eq = e + q;
            float* const s1 = sm.state + eq / kTile * 3 * kTile + eq % kTile;
            const float t = *s1 * a.dec;
            const float u = sm.s * ldexpf(vv[q], un);
            const float x = t - u;
            *s1 = x;
            const uint16_t h = (uint16_t)to_bf16(x);
            if (sm.pshard)
                sm.pshard[eq] = h;
            if (sm.flat)
                sm.flat[eq] = h;
        }
    }
}

// Tiles go in bands of kBand along one side, the band's tiles of a column
// first: the 32 CUs of an XCD then work on about 8 x 4 tiles, 12 panels of the
// operands, where a row of 32 tiles would read 33.
constexpr uint32_t kBand = 8;

// Tile `n` of a lower triangle of t tiles a side.
__device__ __forceinline__ void lower_tile(uint32_t n, uint32_t t,
                                           uint32_t& ti, uint32_t& tj)
{
    // the band: rows r0 .. r0 + h - 1, after r0 (r0 + 1) / 2 tiles
    uint32_t r0 = 0;
    while (r0 + kBand < t && (r0 + kBand) * (r0 + kBand + 1) / 2 <= n)
        r0 += kBand;
    const uint32_t h = t - r0 < kBand ? t - r0 : kBand;
    n -= r0 * (r0 + 1) / 2;
    if (n < (r0 + 1) * h) {             // columns that the whole band has
        tj = n / h;
        ti = r0 + n % h;
        return;
    }
    n -= (r0 + 1) * h;                  // column r0 + k: h - k tiles
    uint32_t k = 1;
    while (n >= h - k)
        n -= h - k++;
    tj = r0 + k;
    ti = r0 + k + n;
}

template <class SH, int EPI, bool FULL>
__global__ __launch_bounds__(SH::kThreads) void ns_gemm_kernel(GemmArgs a)
{
    constexpr int BT = SH::BT, FI = SH::FI, FJ = SH::FJ, ST = SH::ST;
    constexpr int kRow = SH::kRow, NL = SH::kLoads;
    constexpr bool kTri = symmetric(EPI);
    // the stages; separate objects, so that the compiler sees that reading
    // one does not wait for the loads into another
    __shared__ __align__(1024) char lds0[2 * SH::kHalf];
    __shared__ __align__(1024) char lds1[2 * SH::kHalf];
    __shared__ __align__(1024) char lds2[ST > 2 ? 2 * SH::kHalf : 16];
    __shared__ __align__(1024) char lds3[ST > 2 ? 2 * SH::kHalf : 16];
    // the diagonals of the epilogue's squares along i and j
    __shared__ __align__(16) float diag[2][BT];

    uint32_t bid = blockIdx.x;
    const int p = find(a.g, bid);
    const Mat& m = a.g.m[p];
    if (bid >= m.tiles)
        return;                         // the whole workgroup
    bid = xcd_order(bid, m.tiles);
    const Region<FULL> w(m.ws, m.R, m.C, m.batch);
    const int32_t rp = w.rp, cp = w.cp, mp = w.mp;
    const bool tall = m.R > m.C;

    // D[i][j]: ti, tj its tile
    uint32_t b, ti, tj;
    int32_t ni, nj, nk;
    const f16 *P, *Q;
    int64_t plo, qlo;
    if constexpr (kTri) {
        const uint32_t tiles = tri_tiles<BT>(mp);
        b = bid / tiles;
        bid %= tiles;
        lower_tile(bid, (mp + BT - 1) / BT, ti, tj);
        ni = nj = mp;
        if constexpr (EPI == kGram) {
            P = (tall ? w.xt(a.parity) : w.xd(a.parity)) + b * w.e;
            nk = tall ? rp : cp;
            plo = w.E;
            Q = P;
        } else {
            P = w.square(a.sp) + b * w.s;
            Q = w.square(a.sq) + b * w.s;
            nk = mp;
            plo = w.S;
        }
        qlo = plo;
    } else {
        ni = cp;
        nj = rp;
        nk = mp;
        const uint32_t tni = (ni + BT - 1) / BT, tnj = (nj + BT - 1) / BT;
        b = bid / (tni * tnj);
        bid %= tni * tnj;
        const uint32_t band = bid / (kBand * tni) * kBand;
        const uint32_t h = tnj - band < kBand ? tnj - band : kBand;
        bid -= band * tni;
        tj = band + bid % h;
        ti = bid / h;
        const f16* const C = w.square(a.sp) + b * w.s;
        if (tall) {
            P = C;
            plo = w.S;
            Q = w.xd(a.parity) + b * w.e;
            qlo = w.E;
        } else {
            P = w.xt(a.parity) + b * w.e;
            plo = w.E;
            Q = C;
            qlo = w.S;
        }
    }
    const int i0 = ti * BT, j0 = tj * BT;
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wi = wave / SH::WJ, wj = wave % SH::WJ;

    // Which rows a fragment holds.  D's lane of a 16 x 16 has 4 rows 4 g ..
    // 4 g + 3 (g = lane / 16) of column lane % 16.  Rows and columns of D are
    // dealt to the fragments so that a lane's values lie side by side:
    //   fragments f, f + 1 (f even): its 4 + 4 rows are 8 in a row of P,
    //     32 (f / 2) + 8 g + 4 (f % 2) + 0..3
    //   fragments 0 .. FJ-1 along j: its columns are FJ in a row of Q,
    //     FJ (lane % 16) + 0..FJ-1
    // so out[j][i] is written 16 bytes a lane, 64 in a row, and its transpose
    // out[i][j] 2 FJ bytes a lane, 32 FJ in a row, straight from registers.
    //
    // A stage's row is 128 bytes, in 16-byte pieces: 64 k, or in full
    // precision 32 k, their high parts and then their low ones.  Piece c of a
    // row is stored at c ^ sw(row), with sw(row) spreading the 16 rows that a
    // fragment reads at one k over all eight places.  (Q's rows of one read
    // are then all even or all odd where FJ is 2 or 4, and use half of the
    // banks: a quarter of the LDS cycles, measured to cost no time, since the
    // products take three times as many.)  A load instruction fills 1 KiB of
    // LDS in lane order, 8 rows, so the lane fetches the piece that belongs at
    // its place.
    const bool isP = wave < SH::kWaves / 2;
    const char* const base = reinterpret_cast<const char*>(
        isP ? P + (int64_t)i0 * nk : Q + (int64_t)j0 * nk);
    constexpr int kStageK = FULL ? 32 : 64;
    const int64_t lo = 2 * (isP ? plo : qlo);       // bytes to the low parts
    uint32_t voff[NL];
    int64_t llo[NL];
#pragma unroll
    for (int q = 0; q < NL; ++q) {
        const int u = wave * NL + q;
        const int row = (isP ? u : u - BT / 8) * 8 + lane / 8;
        const int lim = isP ? ni - i0 : nj - j0;
        const int r = row < lim ? row : lim - 1;
        const int sw = isP ? (row & 3) | ((row >> 1) & 4) : (row / FJ) & 7;
        const int piece = (lane & 7) ^ sw;
        voff[q] = (uint32_t)r * nk * 2 + (FULL ? piece & 3 : piece) * 16;
        llo[q] = piece < 4 ? 0 : lo;
    }
    const int total = nk / kStageK;
    int next = 0;                                   // stage to be loaded
    auto load = [&](char* lds) {
        const char* const s = base + (int64_t)next * (kStageK * 2);
        ++next;
#pragma unroll
        for (int q = 0; q < NL; ++q) {
            const char* const from = FULL ? s + llo[q] + voff[q] : s + voff[q];
            __builtin_amdgcn_global_load_lds(
                (gptr*)from, (lptr*)(lds + (wave * NL + q) * 1024), 16, 0, 0);
        }
    };

    f32x4 acc[FI][FJ];
#pragma unroll
    for (int i = 0; i < FI; ++i)
#pragma unroll
        for (int j = 0; j < FJ; ++j)
            acc[i][j] = f32x4{0, 0, 0, 0};
    const int l16 = lane & 15, g = lane >> 4;
    const int fi = (wi * FI * 16 + (l16 >> 2) * 8 + (l16 & 3)) * kRow;
    const int fj = SH::kHalf + (wj * FJ * 16 + l16 * FJ) * kRow;
    const int fc = (g ^ (l16 & 7)) * 16;    // sw(row) = l16 & 7 for both
    // What the epilogue reads (the map of rows and columns is above), in units
    // of one column run: unit u is column u % FJ of fragments 2 (u / FJ) and
    // the next.  The first kEarly are fetched ahead of the products, the rest
    // kRing - 1 units ahead of their use: vector memory completes in order,
    // and a load behind stores waits for them.  Past the edges the nearest
    // values inside are read, and dropped.
    constexpr bool kX = EPI >= kUpdate;
    constexpr int kUnits = FI / 2 * FJ;
    // as many as the registers beside the largest tile's sums hold
    constexpr int kRing =
        EPI == kStep || FULL ? 3 : EPI == kProd ? 4 : 6;
    constexpr int kMost = EPI == kGram ? 0 : FULL ? 1 : kRing == 3 ? 2 : 3;
    constexpr int kEarly = kMost < kUnits ? kMost : kUnits;
    static_assert(kEarly < kRing, "units");
    const f16* const xin = w.xd(a.parity) + b * w.e;
    const f16* const pm = w.square(a.sp) + b * w.s;
    const f16* const qm = w.square(a.sq) + b * w.s;
    const float* const dp = w.diag(a.sp) + (int64_t)b * mp;
    const float* const dq = w.diag(a.sq) + (int64_t)b * mp;
    const int64_t olo = kTri ? w.S : w.E;
    const int ld = kTri ? w.mp : w.cp, ldT = kTri ? w.mp : w.rp;
    const int ib = i0 + wi * FI * 16 + g * 8;
    const int jb = j0 + (wj * 16 + l16) * FJ;
    const bool vec4 = m.C % 4 == 0;             // kStep's state by fours
    const int ex =
        EPI == kPoly || EPI > kUpdate ? w.exponent()[b] : 0;
    f16x8 inh[kRing], inl[kRing], inh2[kRing], inl2[kRing];
    f32x4 inS[kRing][2];
    auto fetch = [&](int u) {
        if constexpr (EPI == kGram)
            return;
        const int n = u % kRing, f = u / FJ * 2, jf = u % FJ;
        const int i = ib + f * 16 < ni ? ib + f * 16 : ni - 8;
        const int j = jb + jf < nj ? jb + jf : nj - 1;
        const int64_t o = (int64_t)j * ld + i;
        const f16* const in = kX ? xin : pm;
        inh[n] = *reinterpret_cast<const f16x8*>(in + o);
        if constexpr (FULL || kX)
            inl[n] = *reinterpret_cast<const f16x8*>(in + olo + o);
        if constexpr (EPI == kProd) {
            inh2[n] = *reinterpret_cast<const f16x8*>(qm + o);
            if constexpr (FULL)
                inl2[n] = *reinterpret_cast<const f16x8*>(qm + olo + o);
        }
        if constexpr (EPI == kStep) {
            if (vec4) {
                const int js = j < m.R ? j : m.R - 1;
                const int64_t r = ((int64_t)b * m.R + js) * m.C;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int is = i + 4 * h;
                    const int64_t e = r + (is < m.C ? is : m.C - 4);
                    inS[n][h] = *reinterpret_cast<const f32x4*>(
                        a.st[p].state + e / kTile * 3 * kTile + e % kTile);
                }
            }
        }
    };
    if constexpr (EPI != kGram) {
        // the diagonals along the tile's rows and columns: in an update the
        // one along X's shorter side counts (tall: i), the other is not read
        for (int t = threadIdx.x; t < BT; t += SH::kThreads) {
            const int i = i0 + t < ni ? i0 + t : ni - 1;
            const int j = j0 + t < nj ? j0 + t : nj - 1;
            if (!kX || tall)
                diag[0][t] = dp[i];
            if (!kX || !tall)
                diag[1][t] = (kX ? dp : dq)[j];
        }
#pragma unroll
        for (int u = 0; u < kEarly; ++u)
            fetch(u);
    }

    // Fragments: half h of a stage's rows (k 0..31 and 32..63, or the high and
    // the low parts).
    auto readx = [&](const char* lds, int h, f16x8 (&x)[FI]) {
#pragma unroll
        for (int i = 0; i < FI; ++i)
            x[i] = *reinterpret_cast<const f16x8*>(
                lds + fi + (i / 2 * 32 + i % 2 * 4) * kRow + (fc ^ (h * 64)));
    };
    auto ready = [&](const char* lds, int h, f16x8 (&y)[FJ]) {
#pragma unroll
        for (int j = 0; j < FJ; ++j)
            y[j] = *reinterpret_cast<const f16x8*>(lds + fj + j * kRow +
                                                   (fc ^ (h * 64)));
    };
    auto multiply = [&](const f16x8 (&x)[FI], const f16x8 (&y)[FJ]) {
#pragma unroll
        for (int i = 0; i < FI; ++i)
#pragma unroll
            for (int j = 0; j < FJ; ++j)
                acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_f16(
                    x[i], y[j], acc[i][j], 0, 0, 0);
    };
    if constexpr (SH::kTurns) {
        // A stage's products, each after its reads: k 0..31 and 32..63, or in
        // full precision high x high, high x low and low x high.
        constexpr int kParts = FULL ? 3 : 2;
        f16x8 x[FI], y[FULL ? 2 : 1][FJ];
        auto read = [&](const char* lds, int part) {
            if (!FULL || part < 2)
                ready(lds, part, y[FULL ? part : 0]);
            if (!FULL || part != 1)
                readx(lds, part != 0, x);
        };
        auto product = [&](int part) { multiply(x, y[FULL && part == 1]); };
        // The waves of a SIMD (w and w + 4) run one slot apart: while one
        // multiplies, the other reads its fragments and issues loads.  A
        // part of a stage takes a wave two slots, read and multiply, each
        // ended by a barrier.  The loads for the next stage go out in the
        // stage's first slot; they have landed for every wave when it waits
        // for its own before the barrier that ends the last part's reads,
        // the later half's one slot before the earlier half reads them.  What
        // they overwrite the later half may have read in the slot just before;
        // those reads have returned, as every wave waits for its own before
        // the barrier that ends their slot.
        auto stage = [&](const char* cur, char* other, int kt) {
            if (kt + 1 < total)
                load(other);
#pragma unroll
            for (int part = 0; part < kParts; ++part) {
                read(cur, part);
                if (part + 1 < kParts)
                    __builtin_amdgcn_s_waitcnt(wait_count(63, 0));
                else
                    __builtin_amdgcn_s_waitcnt(wait_count(0, 0));
                slot_barrier();
                __builtin_amdgcn_s_setprio(1);
                product(part);
                __builtin_amdgcn_s_setprio(0);
                slot_barrier();
            }
        };
        load(lds0);
        __builtin_amdgcn_s_waitcnt(wait_count(0, 0));
        slot_barrier();
        if (wave >= 4)
            slot_barrier();
        for (int kt = 0; kt < total; kt += 2) {
            stage(lds0, lds1, kt);
            if (kt + 1 < total)
                stage(lds1, lds0, kt + 1);
        }
        if (wave < 4)
            slot_barrier();
    } else {
        // ST stages in LDS, fragments in two register sets: while the products
        // of stage k run, stage k + 1 is read.  At the top of turn k stage
        // k + 1 is whole when at most the loads of the ST - 2 younger ones
        // are out, and this wave's reads of stage k have returned; after the
        // barrier that holds for every wave, and stage k's place is free.
        static_assert(SH::kTurns || ST == 4, "stages");
        char* const bufs[4] = {lds0, lds1, lds2, lds3};
        f16x8 fx[2][2][FI], fy[2][2][FJ];       // [set][half]
        auto readAll = [&](const char* lds, int set) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                readx(lds, h, fx[set][h]);
                ready(lds, h, fy[set][h]);
            }
        };
        auto mulAll = [&](int set) {
            multiply(fx[set][0], fy[set][0]);
            if constexpr (FULL) {
                multiply(fx[set][0], fy[set][1]);
                multiply(fx[set][1], fy[set][0]);
            } else {
                multiply(fx[set][1], fy[set][1]);
            }
        };
#pragma unroll
        for (int k = 0; k < ST; ++k)
            if (k < total)
                load(bufs[k]);
        if (total >= ST)
            __builtin_amdgcn_s_waitcnt(wait_count((ST - 1) * NL, 0));
        else
            __builtin_amdgcn_s_waitcnt(wait_count(0, 0));
        slot_barrier();
        readAll(bufs[0], 0);
        int kt = 0;
        for (; kt + 2 * ST <= total; kt += ST) {    // no stage is missing
#pragma unroll
            for (int k = 0; k < ST; ++k) {
                __builtin_amdgcn_s_waitcnt(wait_count((ST - 2) * NL, 0));
                slot_barrier();
                load(bufs[k]);
                readAll(bufs[(k + 1) % ST], (k + 1) % 2);
                __builtin_amdgcn_sched_barrier(0);
                mulAll(k % 2);
                __builtin_amdgcn_sched_barrier(0);
            }
        }
        for (; kt < total; kt += ST) {
#pragma unroll
            for (int k = 0; k < ST; ++k) {
                if (kt + k >= total)
                    break;
                // (apart from the loads', so that every path has it)
                __builtin_amdgcn_s_waitcnt(wait_count(63, 0));
                if (kt + k + ST - 1 < total)
                    __builtin_amdgcn_s_waitcnt(wait_count((ST - 2) * NL, 15));
                else
                    __builtin_amdgcn_s_waitcnt(wait_count(0, 15));
                slot_barrier();
                if (kt + k + ST < total)
                    load(bufs[k]);
                // past the last stage: what lies there, for nobody
                readAll(bufs[(k + 1) % ST], (k + 1) % 2);
                __builtin_amdgcn_sched_barrier(0);
                mulAll(k % 2);
                __builtin_amdgcn_sched_barrier(0);
            }
        }
    }

    // Epilogue, from registers.
    const int e0 = max(ex - a.shift, 0), e1 = max(ex - a.shift1, 0);
    const float pa = ldexpf(a.a, e1 - e0), pb = ldexpf(a.b, e1 - 3 * e0),
                pc = ldexpf(a.c, e1 - 5 * e0);
    const int un = -kScaleBits - e0;
    float* const dout = w.diag(a.so) + (int64_t)b * mp;
    f16* const out =
        kTri ? w.square(a.so) + b * w.s : w.xd(1 - a.parity) + b * w.e;
    f16* const outT = kTri ? out : w.xt(1 - a.parity) + b * w.e;
#pragma unroll
    for (int u = kEarly; u < kRing - 1 && u < kUnits; ++u)
        fetch(u);
#pragma unroll
    for (int f = 0; f < FI; f += 2) {
        const int i = ib + f * 16;
        f16x8 vh[FJ], vl[FJ];
        f32x4 di[2] = {};
        if constexpr (EPI != kGram) {
            const f32x4* const d4 = reinterpret_cast<const f32x4*>(
                &diag[0][(wi * FI + f) * 16 + g * 8]);
            di[0] = d4[0];
            di[1] = d4[1];
        }
#pragma unroll
        for (int jf = 0; jf < FJ; ++jf) {
            const float dj =
                EPI == kGram ? 0 : diag[1][(wj * 16 + l16) * FJ + jf];
            const int u = f / 2 * FJ + jf, n = u % kRing, j = jb + jf;
            if (u + kRing - 1 < kUnits)
                fetch(u + kRing - 1);
            float v[8];                     // the results, times kScale
#pragma unroll
            for (int q = 0; q < 8; ++q) {
                const float d = acc[f + q / 4][jf][q % 4] * kUnscale;
                const float dii = di[q / 4][q % 4];
                if constexpr (EPI == kGram) {
                    v[q] = d;
                } else if constexpr (EPI == kPoly || EPI == kProd) {
                    // (R + D)(S + F) = R S + D S + R F + D F, with D and F
                    // the diagonals
                    float r = (float)inh[n][q];
                    if constexpr (FULL)
                        r = r + (float)inl[n][q];
                    if constexpr (EPI == kPoly) {
                        v[q] = pb * r + pc * (d + (dii + dj) * r);
                    } else {
                        float t = (float)inh2[n][q];
                        if constexpr (FULL)
                            t = t + (float)inl2[n][q];
                        v[q] = d + (dii * t + r * dj);
                    }
                } else {
                    v[q] = (tall ? dii : dj) *
                               ((float)inh[n][q] + (float)inl[n][q]) + d;
                }
            }
            if constexpr (kTri) {
                // the diagonal, apart
                if (ti == tj) {
#pragma unroll
                    for (int q = 0; q < 8; ++q)
                        if (i + q == j && i < ni) {
                            const float d =
                                acc[f + q / 4][jf][q % 4] * kUnscale *
                                kUnscale;
                            const float dii = di[q / 4][q % 4];
                            const float dd =
                                EPI == kGram ? d : d + dii * dj;
                            dout[j] = EPI == kPoly
                                          ? pa + (pb * dj + pc * dd)
                                          : dd;
                            v[q] = 0;
                        }
                }
            }
            if constexpr (EPI <= kUpdate) {
#pragma unroll
                for (int q = 0; q < 8; ++q) {
                    f16 h, l;
                    split(v[q], h, l);
                    vh[jf][q] = h;
                    vl[jf][q] = l;
                }
                if (i < ni && j < nj) {
                    const int64_t o = (int64_t)j * ld + i;
                    *reinterpret_cast<f16x8*>(out + o) = vh[jf];
                    if constexpr (FULL || EPI == kUpdate)
                        *reinterpret_cast<f16x8*>(out + olo + o) = vl[jf];
                }
            } else {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    f32x4 st;
                    if constexpr (EPI == kStep) {
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            const float t = inS[n][h][q] * a.dec;
                            const float x =
                                a.st[p].s * ldexpf(v[4 * h + q], un);
                            st[q] = t - x;
                        }
                    }
                    if (j < m.R && i + 4 * h < m.C) {
                        if constexpr (EPI == kStep)
                            finish_step(a, p, m, b, j, i + 4 * h, vec4,
                                        v + 4 * h, un, st);
                        else
                            finish_out<EPI>(a.out[p], m, b, j, i + 4 * h,
                                            v + 4 * h, un);
                    }
                }
            }
        }
        // the other triangle (a tile on the diagonal holds both), or X^T
        if constexpr (EPI <= kUpdate) {
            if (i < ni && jb < nj && (!kTri || ti != tj)) {
#pragma unroll
                for (int q = 0; q < 8; ++q) {
                    f16* const o = outT + (int64_t)(i + q) * ldT + jb;
                    store_cols<FJ>(o, vh, q, nj - jb);
                    if constexpr (FULL)
                        store_cols<FJ>(o + olo, vl, q, nj - jb);
                }
            }
        }
    }
}

// ---- small matrices, whole in one workgroup --------------------------------

// A matrix whose shorter side is at most TM and whose longer one at most TN
// stays in one CU for all steps: one launch instead of three a step, each of
// which would cost its latency and little else (64 x 64, five steps: 16 us a
// call against 72 us).  Below, X is m x n with m the shorter side, transposed
// on the way in and out where the matrix is tall.  X itself is held by the
// threads in fp32, laid out as the update's sums; LDS holds the operands of
// the products: X by rows and by columns and the square A, then C.  The
// arithmetic is the large kernels', with X kept in fp32.  A step is three
// products of 64 or 128 k and five barriers, bound by their latency.
template <int TM_, int TN_, int NW_, int GI_, int UI_>
struct Small {
    static constexpr int TM = TM_, TN = TN_, NW = NW_;
    // waves along i and j: of the squares (m x m), of the update (i along n)
    static constexpr int GI = GI_, GJ = NW / GI, UI = UI_, UJ = NW / UI;
    static constexpr int kThreads = 64 * NW;
};

struct SmallArgs {
    Group g;
    Source src[kMaxMats];
    union {
        OutMat out[kMaxMats];
        StepMat st[kMaxMats];
    };
    int32_t bf16;                       // the source's type
    int32_t epi;                        // kOutBf16, kOutF32 or kStep
    int32_t steps;
    float eps, dec;
    float coef[ZS_NS_MAX_STEPS][3];
    int16_t shift[ZS_NS_MAX_STEPS];     // each step's by itself
};
static_assert(sizeof(SmallArgs) <= 4096, "kernel arguments");

// Byte offset of element (row, col) of an fp16 matrix of L columns in LDS:
// 16-byte pieces permuted within each 128 bytes by the row.
template <int L>
__device__ __forceinline__ int lds_at(int row, int col)
{
    return row * (2 * L) + (col >> 6) * 128 +
           ((((col >> 3) & 7) ^ (row & 7)) << 4) + (col & 7) * 2;
}

// acc[i][j] += sum over K columns of P's rows p0 + 16 i .. and Q's rows
// q0 + 16 j ..; FULL: high and low parts, the low ones LP and LQ bytes on.
template <int FI, int FJ, int K, bool FULL>
__device__ __forceinline__ void lds_product(f32x4 (&acc)[FI][FJ],
                                            const char* P, int LP, int p0,
                                            const char* Q, int LQ, int q0)
{
    const int l16 = threadIdx.x & 15, g = (threadIdx.x >> 4) & 3;
#pragma unroll
    for (int i = 0; i < FI; ++i)
#pragma unroll
        for (int j = 0; j < FJ; ++j)
            acc[i][j] = f32x4{0, 0, 0, 0};
#pragma unroll 2
    for (int k = 0; k < K; k += 32) {
#pragma unroll
        for (int part = 0; part < (FULL ? 3 : 1); ++part) {
            f16x8 x[FI], y[FJ];
#pragma unroll
            for (int i = 0; i < FI; ++i)
                x[i] = *reinterpret_cast<const f16x8*>(
                    P + (part == 2 ? LP : 0) +
                    lds_at<K>(p0 + 16 * i + l16, k + 8 * g));
#pragma unroll
            for (int j = 0; j < FJ; ++j)
                y[j] = *reinterpret_cast<const f16x8*>(
                    Q + (part == 1 ? LQ : 0) +
                    lds_at<K>(q0 + 16 * j + l16, k + 8 * g));
#pragma unroll
            for (int i = 0; i < FI; ++i)
#pragma unroll
                for (int j = 0; j < FJ; ++j)
                    acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_f16(
                        x[i], y[j], acc[i][j], 0, 0, 0);
        }
    }
}

template <class SM, bool FULL>
__global__ __launch_bounds__(SM::kThreads) void ns_small_kernel(SmallArgs a)
{
    constexpr int TM = SM::TM, TN = SM::TN, F = FULL ? 2 : 1;
    constexpr int GFI = TM / SM::GI / 16, GFJ = TM / SM::GJ / 16;
    constexpr int UFI = TN / SM::UI / 16, UFJ = TM / SM::UJ / 16;
    constexpr int LX = TM * TN * 2, LS = TM * TM * 2;
    __shared__ __align__(1024) char xm[LX * F];     // X  [m][n]
    __shared__ __align__(1024) char xt[LX * F];     // X^T [n][m]
    __shared__ __align__(1024) char sq[LS * F];     // A, then C
    __shared__ float dg[TM];                        // its diagonal
    __shared__ double red[SM::NW];

    uint32_t b = blockIdx.x;
    const int p = find(a.g, b);
    const Mat& m = a.g.m[p];
    const Source& s = a.src[p];
    const bool tall = m.R > m.C;
    const int M = tall ? m.C : m.R, N = tall ? m.R : m.C;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int l16 = lane & 15, g = lane >> 4;
    const int gi = wave / SM::GJ * GFI * 16, gj = wave % SM::GJ * GFJ * 16;
    const int ui = wave / SM::UJ * UFI * 16, uj = wave % SM::UJ * UFJ * 16;

    // X, this thread's elements: n index ui + 16 i + 4 g + q, m index
    // uj + 16 j + l16
    f32x4 x[UFI][UFJ];
    double sum = 0;
    const int64_t sn = tall ? s.row : 1, sm = tall ? 1 : s.row;
#pragma unroll
    for (int i = 0; i < UFI; ++i)
#pragma unroll
        for (int j = 0; j < UFJ; ++j)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int n = ui + 16 * i + 4 * g + q, r = uj + 16 * j + l16;
                float v = 0;
                if (n < N && r < M) {
                    const int64_t at = b * s.batch + r * sm + n * sn;
                    v = a.bf16 ? load1<true>(s.x, at) : load1<false>(s.x, at);
                }
                x[i][j][q] = v;
                sum += (double)v * v;
            }
    for (int d = 32; d; d >>= 1)
        sum += __shfl_down(sum, d, 64);
    if (lane == 0)
        red[wave] = sum;
    __syncthreads();
    sum = 0;
    for (int w = 0; w < SM::NW; ++w)
        sum += red[w];
    int ex;
    const double inv = start_scale(sqrt(sum), a.eps, ex);
#pragma unroll
    for (int i = 0; i < UFI; ++i)
#pragma unroll
        for (int j = 0; j < UFJ; ++j)
#pragma unroll
            for (int q = 0; q < 4; ++q)
                x[i][j][q] = (float)((double)x[i][j][q] * inv);

    for (int step = 0; step < a.steps; ++step) {
        const int e1 = max(ex - a.shift[step], 0);
        const float ca = ldexpf(a.coef[step][0], e1 - ex),
                    cb = ldexpf(a.coef[step][1], e1 - 3 * ex),
                    cc = ldexpf(a.coef[step][2], e1 - 5 * ex);
        ex = e1;
        // X's operands
#pragma unroll
        for (int i = 0; i < UFI; ++i)
#pragma unroll
            for (int j = 0; j < UFJ; ++j) {
                const int n = ui + 16 * i + 4 * g, r = uj + 16 * j + l16;
                f16x4 hi, lo;
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    f16 h, l;
                    split(x[i][j][q], h, l);
                    hi[q] = h;
                    lo[q] = l;
                    *reinterpret_cast<f16*>(xt + lds_at<TM>(n + q, r)) = h;
                    if constexpr (FULL)
                        *reinterpret_cast<f16*>(xt + LX +
                                                lds_at<TM>(n + q, r)) = l;
                }
                *reinterpret_cast<f16x4*>(xm + lds_at<TN>(r, n)) = hi;
                if constexpr (FULL)
                    *reinterpret_cast<f16x4*>(xm + LX + lds_at<TN>(r, n)) =
                        lo;
            }
        __syncthreads();
        // A = X X^T, its diagonal apart
        f32x4 A[GFI][GFJ], S[GFI][GFJ];
        auto store = [&](const f32x4 (&v)[GFI][GFJ]) {
#pragma unroll
            for (int i = 0; i < GFI; ++i)
#pragma unroll
                for (int j = 0; j < GFJ; ++j) {
                    const int at = lds_at<TM>(gj + 16 * j + l16,
                                              gi + 16 * i + 4 * g);
                    f16x4 hi, lo;
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        f16 h, l;
                        split(v[i][j][q], h, l);
                        hi[q] = h;
                        lo[q] = l;
                    }
                    *reinterpret_cast<f16x4*>(sq + at) = hi;
                    if constexpr (FULL)
                        *reinterpret_cast<f16x4*>(sq + LS + at) = lo;
                }
        };
        lds_product<GFI, GFJ, TN, FULL>(A, xm, LX, gi, xm, LX, gj);
#pragma unroll
        for (int i = 0; i < GFI; ++i)
#pragma unroll
            for (int j = 0; j < GFJ; ++j)
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    A[i][j][q] = A[i][j][q] * kUnscale;
                    if (gi + 16 * i + 4 * g + q == gj + 16 * j + l16) {
                        dg[gj + 16 * j + l16] = A[i][j][q] * kUnscale;
                        A[i][j][q] = 0;
                    }
                }
        store(A);
        __syncthreads();
        // C = a + b A + c A A
        lds_product<GFI, GFJ, TM, FULL>(S, sq, LS, gi, sq, LS, gj);
        float dc[GFI][GFJ];
#pragma unroll
        for (int i = 0; i < GFI; ++i)
#pragma unroll
            for (int j = 0; j < GFJ; ++j) {
                const float dj = dg[gj + 16 * j + l16];
                dc[i][j] = 0;
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const int t = gi + 16 * i + 4 * g + q;
                    const float d = S[i][j][q] * kUnscale;
                    const float r = A[i][j][q];
                    S[i][j][q] = cb * r + cc * (d + (dg[t] + dj) * r);
                    if (t == gj + 16 * j + l16) {
                        dc[i][j] = ca + (cb * dj +
                                         cc * (d * kUnscale + dj * dj));
                        S[i][j][q] = 0;
                    }
                }
            }
        __syncthreads();                // A and its diagonal have been read
#pragma unroll
        for (int i = 0; i < GFI; ++i)
#pragma unroll
            for (int j = 0; j < GFJ; ++j)
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    if (gi + 16 * i + 4 * g + q == gj + 16 * j + l16)
                        dg[gj + 16 * j + l16] = dc[i][j];
        store(S);
        __syncthreads();
        // X <- C X
        f32x4 U[UFI][UFJ];
        lds_product<UFI, UFJ, TM, FULL>(U, xt, LX, ui, sq, LS, uj);
#pragma unroll
        for (int i = 0; i < UFI; ++i)
#pragma unroll
            for (int j = 0; j < UFJ; ++j) {
                const float dj = dg[uj + 16 * j + l16];
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    x[i][j][q] = dj * x[i][j][q] + U[i][j][q] * kUnscale;
            }
        __syncthreads();                // the operands have been read
    }

#pragma unroll
    for (int i = 0; i < UFI; ++i)
#pragma unroll
        for (int j = 0; j < UFJ; ++j)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int n = ui + 16 * i + 4 * g + q, r = uj + 16 * j + l16;
                if (n >= N || r >= M)
                    continue;
                const float v = ldexpf(x[i][j][q], -kScaleBits - ex);
                const int64_t row = tall ? n : r, col = tall ? r : n;
                if (a.epi == kStep) {
                    const StepMat& o = a.st[p];
                    const int64_t e = (b * (int64_t)m.R + row) * m.C + col;
                    float* const s1 =
                        o.state + e / kTile * 3 * kTile + e % kTile;
                    const float t = *s1 * a.dec;
                    const float u = o.s * v;
                    const float w = t - u;
                    *s1 = w;
                    const uint16_t h = (uint16_t)to_bf16(w);
                    if (o.pshard)
                        o.pshard[e] = h;
                    if (o.flat)
                        o.flat[e] = h;
                } else {
                    const OutMat& o = a.out[p];
                    const int64_t at = b * o.batch + row * o.row + col;
                    if (a.epi == kOutBf16)
                        static_cast<uint16_t*>(o.o)[at] =
                            (uint16_t)to_bf16(v);
                    else
                        static_cast<float*>(o.o)[at] = v;
                }
            }
}

// ---- host ------------------------------------------------------------------

int check_launch(const char* what)
{
    const hipError_t err = hipGetLastError();
    if (err != hipSuccess)
        return zs::fail(ZS_EDEVICE, "%s: %s", what, hipGetErrorString(err));
    return ZS_OK;
}

constexpr int64_t kMaxSide = 32768;             // of the smaller side
constexpr int64_t kMaxLong = (int64_t)1 << 22;  // of the larger: a tile's rows
                                                // span less than 4 GiB
// Workgroups of a call's widest launch, at least: HIP allows fewer than 2^32
// threads, and the small kernel has 512 for a matrix of one tile.
constexpr int64_t kMaxTiles = ((int64_t)1 << 23) - 1;

// One member's sizes, checked; tiles: a matrix's 64 x 64 tiles or its pieces
// of the momentum, whichever are more.
int check_sizes(int32_t i, int64_t batch, int64_t rows, int64_t cols,
                int64_t& tiles)
{
    using zs::fail;
    if (batch < 0 || rows < 0 || cols < 0)
        return fail(ZS_EINVAL, "matrices %d: negative size", i);
    if (batch == 0 || rows == 0 || cols == 0)
        return ZS_OK;
    if (rows > INT32_MAX / cols)
        return fail(ZS_ERANGE, "matrices %d: %lld x %lld elements in one "
                    "matrix", i, (long long)rows, (long long)cols);
    const int64_t lo = rows < cols ? rows : cols;
    const int64_t hi = rows < cols ? cols : rows;
    if (lo > kMaxSide || hi > kMaxLong)
        return fail(ZS_ERANGE, "matrices %d: %lld x %lld is above %lld on "
                    "the smaller or %lld on the larger side", i,
                    (long long)rows, (long long)cols, (long long)kMaxSide,
                    (long long)kMaxLong);
    const int64_t per = ((rows + 63) / 64) * ((cols + 63) / 64);
    const int64_t parts = rows * cols / kMomChunk + 1;
    const int64_t most = per > parts ? per : parts;
    if (batch > kMaxTiles / most || (tiles += batch * most) > kMaxTiles)
        return fail(ZS_ERANGE, "more than %lld matrix tiles in one call",
                    (long long)kMaxTiles);
    return ZS_OK;
}

int check_precision(int32_t precision)
{
    if (precision != ZS_NS_FAST && precision != ZS_NS_FULL)
        return zs::fail(ZS_EINVAL, "unknown precision %d", precision);
    return ZS_OK;
}

int check_ns(const zs_newton_schulz* ns)
{
    using zs::fail;
    if (!ns) return fail(ZS_EINVAL, "ns is NULL");
    if (ns->steps < 1 || ns->steps > ZS_NS_MAX_STEPS)
        return fail(ZS_EINVAL, "steps %d outside [1, %d]", ns->steps,
                    ZS_NS_MAX_STEPS);
    if (const int rc = check_precision(ns->precision)) return rc;
    if (!(ns->eps > 0) || !std::isfinite(ns->eps))
        return fail(ZS_EINVAL, "eps must be positive and finite");
    for (int k = 0; k < ns->steps; ++k)
        for (int q = 0; q < 3; ++q)
            if (!std::isfinite(ns->coef[k][q]))
                return fail(ZS_EINVAL, "coef[%d][%d] is not finite", k, q);
    return ZS_OK;
}

bool aligned(const void* p, uintptr_t n)
{
    return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0;
}

// (Waves, 64 x 64: in full precision 8 take 17.4 us a call, 4 20.2; in fast
// precision a thousand matrices take 30.4 us with 4, 31.1 with 8.)
template <bool FULL>
using Small64 = Small<64, 64, FULL ? 8 : 4, 2, 2>;
typedef Small<64, 256, 8, 2, 8> Small256;
typedef Small<64, 512, 8, 2, 8> Small512;
typedef Small<128, 128, 8, 2, 2> Small128;
// A matrix counts for one tile in the first of these, for two and more in the
// others, and for four and more where sums have a launch of their own.
static_assert(kMaxTiles * Small64<true>::kThreads < (int64_t)1 << 32 &&
              kMaxTiles / 2 * 512 < (int64_t)1 << 32 &&
              kMaxTiles / 4 * kSumNT < (int64_t)1 << 32, "threads of a launch");

// A stack's bytes of workspace.
int64_t mat_bytes(const Mat& m, bool full)
{
    if (small_kind(m.R, m.C, full))     // U alone
        return (4 * (int64_t)m.batch * m.R * m.C + 255) / 256 * 256;
    const int64_t parts = 8 * (int64_t)m.batch * m.nparts;
    const int64_t off =
        full ? Region<true>(nullptr, m.R, m.C, m.batch).parts_off()
             : Region<false>(nullptr, m.R, m.C, m.batch).parts_off();
    return (off + parts + 255) / 256 * 256;
}

// Appends a stack to the group, with its part of the workspace.
void add_mat(Group& g, int64_t batch, int64_t rows, int64_t cols, int chunk,
             bool full, char* ws, int64_t& used)
{
    Mat& m = g.m[g.count++];
    m.R = (int32_t)rows;
    m.C = (int32_t)cols;
    m.batch = (int32_t)batch;
    m.nparts = (int32_t)((rows * cols + chunk - 1) / chunk);
    m.ws = ws + used;
    used += mat_bytes(m, full);
}

int64_t group_bytes(const Group& g, bool full)
{
    int64_t n = 0;
    for (int i = 0; i < g.count; ++i)
        n += mat_bytes(g.m[i], full);
    return n;
}

template <class SH, int EPI, bool FULL>
int launch_gemm(GemmArgs& a, hipStream_t s)
{
    const uint32_t n = set_starts(a.g, d_tiles<SH::BT, EPI>, 8);
    hipLaunchKernelGGL((ns_gemm_kernel<SH, EPI, FULL>), dim3(n),
                       dim3(SH::kThreads), 0, s, a);
    return check_launch("Newton-Schulz product");
}

template <int EPI, bool FULL>
int launch_product(GemmArgs& a, int tile, hipStream_t s)
{
    switch (tile) {
    case 64: return launch_gemm<Shape64, EPI, FULL>(a, s);
    case 128: return launch_gemm<Shape128, EPI, FULL>(a, s);
    case 192: return launch_gemm<Shape192, EPI, FULL>(a, s);
    default: return launch_gemm<Shape256, EPI, FULL>(a, s);
    }
}

template <int LAST, bool FULL>
int run_products(GemmArgs& a, const zs_newton_schulz& ns, const Part& part,
                 hipStream_t s)
{
    const Tiles& t = part.tiles;
    a.parity = 0;
    a.shift1 = 0;
    int rc = ZS_OK;
    auto poly = [&](int k, Square out) {
        a.a = ns.coef[k][0];
        a.b = ns.coef[k][1];
        a.c = ns.coef[k][2];
        a.shift = a.shift1;
        a.shift1 = (int16_t)(a.shift1 + shift_of(ns.coef[k]));
        a.sp = a.sq = kA;
        a.so = out;
        if (!rc) rc = launch_product<kPoly, FULL>(a, t.square.tile, s);
    };
    auto prod = [&](Square p, Square q, Square out) {
        a.sp = p;
        a.sq = q;
        a.so = out;
        if (!rc) rc = launch_product<kProd, FULL>(a, t.square.tile, s);
    };
    for (int k = 0; k < ns.steps && !rc;) {
        const bool two = part.pairs && together(ns, k);
        a.so = kA;
        rc = launch_product<kGram, FULL>(a, t.gram.tile, s);
        poly(k, kC);
        if (two) {
            prod(kC, kA, kT);
            prod(kT, kC, kA);
            poly(k + 1, kC2);
            prod(kC2, kC, kT);
        }
        k += two ? 2 : 1;
        a.sp = two ? kT : kC;
        if (k == ns.steps)
            a.shift = a.shift1;
        if (!rc)
            rc = k < ns.steps
                     ? launch_product<kUpdate, FULL>(a, t.update.tile, s)
                     : launch_product<LAST, FULL>(a, t.last.tile, s);
        a.parity ^= 1;
    }
    return rc;
}

// The steps on a group whose X[0] is in the workspace.
template <int LAST, bool FULL>
int run_steps(GemmArgs& a, const zs_newton_schulz& ns, hipStream_t s)
{
    Part parts[2];
    const int n = plan_steps<LAST, FULL>(a.g, ns, parts);
    if (n == 1)
        return run_products<LAST, FULL>(a, ns, parts[0], s);
    for (const Part& part : parts) {
        GemmArgs b = a;
        b.g.count = part.count;
        for (int k = 0; k < part.count; ++k) {
            const int i = part.at[k];
            b.g.m[k] = a.g.m[i];
            if (LAST == kStep)
                b.st[k] = a.st[i];
            else
                b.out[k] = a.out[i];
        }
        if (const int rc = run_products<LAST, FULL>(b, ns, part, s)) return rc;
    }
    return ZS_OK;
}

uint32_t init_tiles(const Mat& m)
{
    return (uint32_t)(padded(m.R) / 64) * (uint32_t)(padded(m.C) / 64);
}

template <bool BF16, bool FULL>
int launch_init(const Group& g, const Source* src, float eps, hipStream_t s)
{
    InitArgs a;
    a.g = g;
    for (int i = 0; i < g.count; ++i)
        a.src[i] = src[i];
    a.eps = eps;
    a.summed = 0;
    for (int i = 0; i < g.count; ++i)
        a.summed |= g.m[i].nparts > kMaxParts;
    if (a.summed) {
        const uint32_t n = set_starts(a.g, [](const Mat&) { return 1; });
        hipLaunchKernelGGL(ns_sum_kernel<FULL>, dim3(n), dim3(kSumNT), 0, s,
                           a.g);
        if (const int rc = check_launch("norm sums")) return rc;
    }
    const uint32_t n = set_starts(a.g, init_tiles);
    hipLaunchKernelGGL((ns_init_kernel<BF16, FULL>), dim3(n), dim3(kNT), 0, s,
                       a);
    return check_launch("Newton-Schulz start");
}

template <class SM, bool FULL>
int launch_small(SmallArgs& a, hipStream_t s)
{
    const uint32_t n = set_starts(a.g, [](const Mat&) { return 1; });
    hipLaunchKernelGGL((ns_small_kernel<SM, FULL>), dim3(n),
                       dim3(SM::kThreads), 0, s, a);
    return check_launch("Newton-Schulz steps");
}

// What a call does with the stacks of a group: src where they come from, out
// or st where they go.
struct Work {
    const Group* g;
    const Source* src;
    int32_t x_type;
    int epi;                            // kOutBf16, kOutF32 or kStep
    const OutMat* out;
    const StepMat* st;
    float dec;
    const zs_newton_schulz* ns;
};

// The small stacks of each kind, and the rest into `g` (with its members'
// places in the whole group in `at`).
template <bool FULL>
int run_small(const Work& w, Group& g, int* at, hipStream_t s)
{
    g.count = 0;
    for (int kind = 0; kind <= kSmalls; ++kind) {
        SmallArgs a;
        a.g.count = 0;
        for (int i = 0; i < w.g->count; ++i) {
            const Mat& m = w.g->m[i];
            if (small_kind(m.R, m.C, FULL) != kind)
                continue;
            if (kind == 0) {
                at[g.count] = i;
                g.m[g.count++] = m;
                continue;
            }
            const int n = a.g.count++;
            a.g.m[n] = m;
            a.src[n] = w.src[i];
            if (w.epi == kStep)
                a.st[n] = w.st[i];
            else
                a.out[n] = w.out[i];
        }
        if (kind == 0 || a.g.count == 0)
            continue;
        a.bf16 = w.x_type == ZS_BF16;
        a.epi = w.epi;
        a.steps = w.ns->steps;
        a.eps = w.ns->eps;
        a.dec = w.dec;
        for (int k = 0; k < ZS_NS_MAX_STEPS; ++k) {
            for (int q = 0; q < 3; ++q)
                a.coef[k][q] = k < a.steps ? w.ns->coef[k][q] : 0;
            a.shift[k] = (int16_t)shift_of(a.coef[k]);
        }
        int rc;
        if (kind == 1) {
            rc = launch_small<Small64<FULL>, FULL>(a, s);
        } else if (kind == 2) {
            rc = launch_small<Small256, FULL>(a, s);
        } else if constexpr (FULL) {
            rc = ZS_OK;
        } else {
            rc = kind == 3 ? launch_small<Small512, FULL>(a, s)
                           : launch_small<Small128, FULL>(a, s);
        }
        if (rc) return rc;
    }
    return ZS_OK;
}

// The large stacks, whose partial sums of squares are in the workspace.
template <bool FULL>
int run_large(const Work& w, const Group& g, const int* at, hipStream_t s)
{
    Source src[kMaxMats];
    for (int i = 0; i < g.count; ++i)
        src[i] = w.src[at[i]];
    const int rc = w.x_type == ZS_BF16
                       ? launch_init<true, FULL>(g, src, w.ns->eps, s)
                       : launch_init<false, FULL>(g, src, w.ns->eps, s);
    if (rc) return rc;
    GemmArgs a;
    a.g = g;
    a.dec = w.dec;
    for (int i = 0; i < g.count; ++i)
        if (w.epi == kStep)
            a.st[i] = w.st[at[i]];
        else
            a.out[i] = w.out[at[i]];
    return w.epi == kOutBf16  ? run_steps<kOutBf16, FULL>(a, *w.ns, s)
           : w.epi == kOutF32 ? run_steps<kOutF32, FULL>(a, *w.ns, s)
                              : run_steps<kStep, FULL>(a, *w.ns, s);
}

template <bool FULL>
int orthogonalize(const Work& w, hipStream_t s)
{
    NormArgs na;
    int at[kMaxMats];
    if (const int rc = run_small<FULL>(w, na.g, at, s)) return rc;
    if (na.g.count == 0) return ZS_OK;
    const Group g = na.g;
    for (int i = 0; i < g.count; ++i)
        na.src[i] = w.src[at[i]];
    const uint32_t n =
        set_starts(na.g, [](const Mat& m) { return m.nparts; });
    if (w.x_type == ZS_BF16)
        hipLaunchKernelGGL((ns_norm_kernel<true, FULL>), dim3(n), dim3(kNT),
                           0, s, na);
    else
        hipLaunchKernelGGL((ns_norm_kernel<false, FULL>), dim3(n), dim3(kNT),
                           0, s, na);
    if (const int rc = check_launch("norm kernel")) return rc;
    return run_large<FULL>(w, g, at, s);
}

}  // namespace

extern "C" int zs_orthogonalize_workspace(int32_t count,
                                          const zs_ns_matrices* mats,
                                          int32_t precision, int64_t* bytes)
{
    using zs::fail;
    zs::clear_error();
    if (!mats || !bytes) return fail(ZS_EINVAL, "NULL pointer");
    if (count < 1 || count > kMaxMats)
        return fail(ZS_EINVAL, "count %d outside [1, %d]", count, kMaxMats);
    if (const int rc = check_precision(precision)) return rc;
    Group g;
    g.count = 0;
    int64_t tiles = 0, used = 0;
    for (int32_t i = 0; i < count; ++i) {
        const zs_ns_matrices& m = mats[i];
        const int rc = check_sizes(i, m.batch, m.rows, m.cols, tiles);
        if (rc) return rc;
        if (m.batch && m.rows && m.cols)
            add_mat(g, m.batch, m.rows, m.cols, kNormChunk,
                    precision == ZS_NS_FULL,
                    nullptr, used);
    }
    *bytes = group_bytes(g, precision == ZS_NS_FULL);
    return ZS_OK;
}

extern "C" int zs_orthogonalize(int32_t count, const zs_ns_matrices* mats,
                                int32_t x_type, int32_t o_type,
                                const zs_newton_schulz* ns, void* workspace,
                                int64_t workspace_bytes, void* hip_stream)
{
    using zs::fail;
    zs::clear_error();
    if (!mats) return fail(ZS_EINVAL, "mats is NULL");
    if (count < 1 || count > kMaxMats)
        return fail(ZS_EINVAL, "count %d outside [1, %d]", count, kMaxMats);
    if ((x_type != ZS_BF16 && x_type != ZS_F32) ||
        (o_type != ZS_BF16 && o_type != ZS_F32))
        return fail(ZS_EINVAL, "unknown element type %d or %d", x_type,
                    o_type);
    if (const int rc = check_ns(ns)) return rc;
    const bool full = ns->precision == ZS_NS_FULL;
    const uintptr_t xe = x_type == ZS_BF16 ? 2 : 4;
    const uintptr_t oe = o_type == ZS_BF16 ? 2 : 4;
    Group g;
    g.count = 0;
    Source src[kMaxMats];
    OutMat out[kMaxMats];
    int64_t tiles = 0, used = 0;
    int32_t order[kMaxMats];
    sort_members(order, count, [&](int32_t i, int64_t& r, int64_t& c) {
        r = mats[i].rows;
        c = mats[i].cols;
    });
    for (int32_t n = 0; n < count; ++n) {
        const int32_t i = order[n];
        const zs_ns_matrices& m = mats[i];
        if (const int rc = check_sizes(i, m.batch, m.rows, m.cols, tiles))
            return rc;
        if (!(m.batch && m.rows && m.cols))
            continue;
        if (!m.x || !m.o)
            return fail(ZS_EINVAL, "matrices %d: NULL pointer", i);
        if (!aligned(m.x, xe) || !aligned(m.o, oe))
            return fail(ZS_EALIGN, "matrices %d: pointer not aligned to its "
                        "elements", i);
        if (m.x_row_stride < m.cols || m.o_row_stride < m.cols ||
            m.x_batch_stride < 0)
            return fail(ZS_EINVAL, "matrices %d: row stride below cols, or "
                        "a negative batch stride", i);
        // the furthest element has to have an address
        constexpr int64_t kFar = (int64_t)1 << 46;
        if (m.x_row_stride > kFar / m.rows || m.o_row_stride > kFar / m.rows ||
            m.x_batch_stride > kFar / m.batch ||
            m.o_batch_stride > kFar / m.batch)
            return fail(ZS_ERANGE, "matrices %d: strides too large", i);
        // a stack's outputs: one behind the other, or side by side in rows
        // of their own
        const bool behind =
            m.o_batch_stride >= (m.rows - 1) * m.o_row_stride + m.cols;
        const bool beside =
            m.o_batch_stride >= m.cols &&
            m.o_row_stride >= (m.batch - 1) * m.o_batch_stride + m.cols;
        if (m.batch > 1 && !behind && !beside)
            return fail(ZS_EINVAL, "matrices %d: outputs overlap", i);
        Source& s = src[g.count];
        s.x = m.x;
        s.batch = m.x_batch_stride;
        s.row = m.x_row_stride;
        s.vec = m.cols % 4 == 0 && s.row % 4 == 0 &&
                (m.batch == 1 || s.batch % 4 == 0) && aligned(m.x, 4 * xe);
        OutMat& o = out[g.count];
        o.o = m.o;
        o.batch = m.o_batch_stride;
        o.row = m.o_row_stride;
        o.vec = m.cols % 4 == 0 && o.row % 4 == 0 &&
                (m.batch == 1 || o.batch % 4 == 0) && aligned(m.o, 4 * oe);
        add_mat(g, m.batch, m.rows, m.cols, kNormChunk, full,
                static_cast<char*>(workspace), used);
    }
    if (g.count == 0) return ZS_OK;
    if (!workspace) return fail(ZS_EINVAL, "workspace is NULL");
    if (!aligned(workspace, 256))
        return fail(ZS_EALIGN, "workspace must be 256-byte aligned");
    if (workspace_bytes < used)
        return fail(ZS_ERANGE, "workspace of %lld bytes, %lld needed",
                    (long long)workspace_bytes, (long long)used);
    const hipStream_t s = static_cast<hipStream_t>(hip_stream);
    const Work w = {&g, src, x_type, o_type == ZS_BF16 ? kOutBf16 : kOutF32,
                    out, nullptr, 1.f, ns};
    return full ? orthogonalize<true>(w, s) : orthogonalize<false>(w, s);
}

namespace {

// The members of a muon call, checked against the layout; order[n]: which
// tensor the group's n-th stack is.
int muon_group(const zs_layout* L, int32_t count, const zs_muon_tensor* t,
               bool full, char* ws, Group& g, int32_t* order, int64_t& used)
{
    using zs::fail;
    if (!L) return fail(ZS_EINVAL, "layout is NULL");
    if (!t) return fail(ZS_EINVAL, "tensors is NULL");
    if (!L->whole_tensors)
        return fail(ZS_EINVAL, "the layout is not whole-tensor");
    if (count < 1 || count > kMaxMats)
        return fail(ZS_EINVAL, "count %d outside [1, %d]", count, kMaxMats);
    const int32_t nb = (int32_t)L->buckets.size();
    g.count = 0;
    used = 0;
    int64_t tiles = 0;
    for (int32_t i = 0; i < count; ++i) {
        const int32_t b = t[i].bucket_id;
        if (b < 0 || b >= nb)
            return fail(ZS_ERANGE, "tensors[%d]: bucket %d outside [0, %d)",
                        i, b, nb);
        for (int32_t k = 0; k < i; ++k)
            if (t[k].bucket_id == b)
                return fail(ZS_EINVAL, "bucket %d appears twice", b);
        if (const int rc = check_sizes(i, t[i].batch, t[i].rows, t[i].cols,
                                       tiles))
            return rc;
        // sizes are in range, and so is their product (kMaxTiles)
        const int64_t n = t[i].batch * t[i].rows * t[i].cols;
        if (n != L->chunks[b].numel)
            return fail(ZS_EINVAL, "tensors[%d]: %lld x %lld x %lld is not "
                        "the tensor's %lld elements", i,
                        (long long)t[i].batch, (long long)t[i].rows,
                        (long long)t[i].cols, (long long)L->chunks[b].numel);
    }
    sort_members(order, count, [&](int32_t i, int64_t& r, int64_t& c) {
        r = t[i].rows;
        c = t[i].cols;
    });
    for (int32_t n = 0; n < count; ++n) {
        const zs_muon_tensor& m = t[order[n]];
        add_mat(g, m.batch, m.rows, m.cols, kMomChunk, full, ws, used);
    }
    return ZS_OK;
}

template <int WT>
void launch_momentum(const MomArgs& a, bool tiled, uint32_t n, hipStream_t s)
{
    if (tiled)
        hipLaunchKernelGGL((muon_momentum_kernel<WT, true>), dim3(n),
                           dim3(kNT), 0, s, a);
    else
        hipLaunchKernelGGL((muon_momentum_kernel<WT, false>), dim3(n),
                           dim3(kNT), 0, s, a);
}

template <bool FULL>
int muon_step(const Group& g, MomArgs& ma, const StepMat* st, bool tiled,
              float dec, const zs_newton_schulz& ns, hipStream_t s)
{
    ma.g = g;
    Source src[kMaxMats] = {};
    for (int i = 0; i < g.count; ++i) {
        const Mat& m = g.m[i];
        const bool small = small_kind(m.R, m.C, FULL) != 0;
        const Region<FULL> r(m.ws, m.R, m.C, m.batch);
        ma.src[i].u = small ? (float*)m.ws : r.u();
        ma.src[i].parts = small ? nullptr : r.parts();
        src[i].x = ma.src[i].u;
        src[i].row = m.C;
        src[i].batch = (int64_t)m.R * m.C;
        src[i].vec = m.C % 4 == 0;
    }
    const uint32_t n =
        set_starts(ma.g, [](const Mat& m) { return m.nparts; });
    switch (ma.W) {
    case 1: launch_momentum<1>(ma, tiled, n, s); break;
    case 2: launch_momentum<2>(ma, tiled, n, s); break;
    case 4: launch_momentum<4>(ma, tiled, n, s); break;
    case 8: launch_momentum<8>(ma, tiled, n, s); break;
    default: launch_momentum<0>(ma, tiled, n, s); break;
    }
    if (const int rc = check_launch("momentum kernel")) return rc;
    const Work w = {&g, src, ZS_F32, kStep, nullptr, st, dec, &ns};
    Group large;
    int at[kMaxMats];
    if (const int rc = run_small<FULL>(w, large, at, s)) return rc;
    return large.count ? run_large<FULL>(w, large, at, s) : ZS_OK;
}

}  // namespace

extern "C" int zs_muon_workspace(const zs_layout* L, int32_t count,
                                 const zs_muon_tensor* tensors,
                                 int32_t precision, int64_t* bytes)
{
    zs::clear_error();
    if (!bytes) return zs::fail(ZS_EINVAL, "bytes is NULL");
    if (const int rc = check_precision(precision)) return rc;
    Group g;
    int64_t used;
    int32_t order[kMaxMats];
    const int rc = muon_group(L, count, tensors, precision == ZS_NS_FULL,
                              nullptr, g, order, used);
    if (!rc) *bytes = used;
    return rc;
}

extern "C" int zs_muon_step(const zs_layout* L, int32_t count,
                            const zs_muon_tensor* tensors,
                            const uint16_t* const* grads, int32_t grad_layout,
                            int64_t grad_stride, float* state,
                            uint16_t* param_shard, uint16_t* full_flat,
                            const zs_muon* hp, void* workspace,
                            int64_t workspace_bytes, void* hip_stream)
{
    using zs::fail;
    zs::clear_error();
    if (!hp) return fail(ZS_EINVAL, "hp is NULL");
    if (const int rc = check_ns(&hp->ns)) return rc;
    if (!std::isfinite(hp->lr) || !std::isfinite(hp->momentum) ||
        !std::isfinite(hp->weight_decay))
        return fail(ZS_EINVAL, "lr, momentum or weight_decay is not finite");
    if (hp->scale != ZS_MUON_SCALE_NONE && hp->scale != ZS_MUON_SCALE_SHAPE &&
        hp->scale != ZS_MUON_SCALE_RMS)
        return fail(ZS_EINVAL, "unknown scale %d", hp->scale);
    const float dec =
        (float)(1.0 - (double)hp->lr * (double)hp->weight_decay);
    if (!std::isfinite(dec))
        return fail(ZS_EINVAL, "1 - lr*weight_decay is not finite");
    const bool full = hp->ns.precision == ZS_NS_FULL;
    Group g;
    int64_t used;
    int32_t order[kMaxMats];
    if (const int rc = muon_group(L, count, tensors, full,
                                  static_cast<char*>(workspace), g, order,
                                  used))
        return rc;
    if (grad_layout != ZS_GRADS_SLICES && grad_layout != ZS_GRADS_TILED)
        return fail(ZS_EINVAL, "unknown grad_layout %d", grad_layout);
    if (!grads || !state || !workspace)
        return fail(ZS_EINVAL, "grads, state and workspace must be non-NULL");
    if (!param_shard && !full_flat)
        return fail(ZS_EINVAL, "need param_shard or full_flat");
    if (!aligned(state, 16) || !aligned(param_shard, 16) ||
        !aligned(full_flat, 16))
        return fail(ZS_EALIGN, "device pointers must be 16-byte aligned");
    if (!aligned(workspace, 256))
        return fail(ZS_EALIGN, "workspace must be 256-byte aligned");
    const bool tiled = grad_layout == ZS_GRADS_TILED;
    MomArgs ma;
    StepMat st[kMaxMats];
    for (int32_t n = 0; n < count; ++n) {
        const int32_t i = order[n];
        const zs_bucket& b = L->buckets[tensors[i].bucket_id];
        if (!grads[i]) return fail(ZS_EINVAL, "grads[%d] is NULL", i);
        if (!aligned(grads[i], 16))
            return fail(ZS_EALIGN, "grads[%d] is not 16-byte aligned", i);
        if (!tiled) {
            if (grad_stride % 8)
                return fail(ZS_EALIGN, "grad_stride %lld is not a multiple "
                            "of 8", (long long)grad_stride);
            if (grad_stride < b.slice_numel)
                return fail(ZS_ERANGE, "grad_stride %lld < %lld elements per "
                            "slice", (long long)grad_stride,
                            (long long)b.slice_numel);
            if (grad_stride > INT64_MAX / 2 / L->world)
                return fail(ZS_ERANGE, "W * grad_stride overflows");
        }
        ma.src[n].grads = grads[i];
        ma.src[n].state = state + b.tile_off * 3 * kTile;
        st[n].state = ma.src[n].state;
        st[n].pshard = param_shard ? param_shard + b.shard_off : nullptr;
        st[n].flat = full_flat ? full_flat + slice_flat_pos(L, b) : nullptr;
        const double r = (double)tensors[i].rows, c = (double)tensors[i].cols;
        const double scale =
            hp->scale == ZS_MUON_SCALE_SHAPE ? std::sqrt(r > c ? r / c : 1.0)
            : hp->scale == ZS_MUON_SCALE_RMS
                ? 0.2 * std::sqrt(r > c ? r : c)
                : 1.0;
        st[n].s = (float)((double)hp->lr * scale);
        if (!std::isfinite(st[n].s))
            return fail(ZS_EINVAL, "tensors[%d]: lr times its scale is not "
                        "finite", i);
    }
    if (workspace_bytes < used)
        return fail(ZS_ERANGE, "workspace of %lld bytes, %lld needed",
                    (long long)workspace_bytes, (long long)used);
    ma.gstride = grad_stride;
    ma.W = L->world;
    ma.nesterov = hp->nesterov != 0;
    ma.mu = hp->momentum;
    ma.fw = (float)L->world;
    ma.invw = 1.f / (float)L->world;
    ma.pow2 = (L->world & (L->world - 1)) == 0;
    const hipStream_t s = static_cast<hipStream_t>(hip_stream);
    return full ? muon_step<true>(g, ma, st, tiled, dec, hp->ns, s)
                : muon_step<false>(g, ma, st, tiled, dec, hp->ns, s);
}
