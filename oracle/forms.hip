// TEST INFRASTRUCTURE: the arithmetic of csrc/zs_codes.h against the
// compiler's forms and the definitions, for every input of its ranges.
// Written for gfx950 (CDNA4, wave64).

#include <hip/hip_runtime.h>

#include <cstdint>

#include "zs_codes.h"

namespace {

// What is compared.
constexpr int kBf16 = 0, kRoot = 1, kQuotient = 2, kCodes = 3, kHardware = 4;

struct Result {
    unsigned long long compared, wrong, first;
};

constexpr uint32_t kThreads = 256, kGroups = 4096;
constexpr uint32_t kAll = kThreads * kGroups;       // 2^20
constexpr uint32_t kTurns = 1u << 10;               // of four inputs a thread
static_assert((uint64_t)kAll * kTurns * 4 == 1ull << 32, "every input once");

// Nearest even in integers, NaN quiet with its sign and top payload bits.
__device__ uint32_t bf16_of(uint32_t u)
{
    if ((u & 0x7fffffffu) > 0x7f800000u)
        return u >> 16 | 0x40;
    return (u + 0x7fff + (u >> 16 & 1)) >> 16;
}

// The whole number q with (q - 1/2)^2 <= y < (q + 1/2)^2.
__device__ int code_of(float y)
{
    const double q = floor(sqrt((double)y));
    return (int)q + ((q + 0.5) * (q + 0.5) <= (double)y);
}

template <int WHAT>
__global__ __launch_bounds__(kThreads) void compare_kernel(Result* out)
{
    unsigned long long compared = 0, wrong = 0, first = ~0ull;
    auto look = [&](uint32_t u, bool in, bool ok) {
        compared += in;
        if (in && !ok) {
            ++wrong;
            if (u < first)
                first = u;
        }
    };
    // all lanes of a wave take the same number of turns
    for (uint32_t turn = 0; turn < kTurns; ++turn) {
        const uint32_t u0 =
            4 * (turn * kAll + blockIdx.x * kThreads + threadIdx.x);
        if constexpr (WHAT == kCodes) {
            // sizes of m up to A's own, signs in turn, and roots up to A's:
            // 0 and those that a root of fp32 can have over its A
            float m[4], r[4];
            bool in_m[4], in_r[4];
            for (int j = 0; j < 4; ++j) {
                const float y = __uint_as_float(u0 + j);
                in_m[j] = y >= 0.0f && y <= kTopM * (1.0f + 0x1p-20f);
                in_r[j] = y == 0.0f || (y >= 0x1p-123f &&
                                        y <= kTopR * (1.0f + 0x1p-20f));
                m[j] = in_m[j] ? (j % 2 ? -y : y) : 0.0f;
                r[j] = in_r[j] ? y : 0.0f;
            }
            uint32_t cm, cr;
            codes(m, r, 1.0f, 1.0f, cm, cr);
            for (int j = 0; j < 4; ++j) {
                const int qm = code_of(fabsf(m[j]));
                int qr = code_of(r[j]);
                if (r[j] > 0.0f && qr == 0)
                    qr = 1;
                look(u0 + j, in_m[j],
                     (int8_t)(cm >> (8 * j)) == (j % 2 ? -qm : qm));
                look(u0 + j, in_r[j], (int)(cr >> (8 * j) & 255) == qr);
            }
            continue;
        }
        for (int j = 0; j < 4; ++j) {
            const uint32_t u = u0 + j;
            const float x = __uint_as_float(u);
            if constexpr (WHAT == kBf16) {
                const uint32_t w = to_bf16(x, -x);
                look(u, true, w == (bf16_of(u) |
                                    bf16_of(u ^ 0x80000000u) << 16));
            } else if constexpr (WHAT == kRoot) {
                const bool in = x >= 0x1p-96f && u < 0x7f800000u;
                look(u, in, root_of(x) == sqrtf(x));
            } else if constexpr (WHAT == kQuotient) {
                const bool in = x >= 0x1p-100f && x < 0x1p126f;
                look(u, in, quotient_of(kTopM, x) == kTopM / x &&
                            quotient_of(kTopR, x) == kTopR / x);
            } else {
                const bool in = x >= 0.0f && x < 65536.0f;
                const double s = __builtin_amdgcn_sqrtf(x);
                look(u, in, fabs(s - sqrt((double)x)) <= 0x1p-16 &&
                            (x > kTopR || root_code(x) == code_of(x)));
            }
        }
    }
    atomicAdd(&out->compared, compared);
    if (wrong) {
        atomicAdd(&out->wrong, wrong);
        atomicMin(&out->first, first);
    }
}

}  // namespace

// Compares all of `what`; out: device memory, {0, 0, ~0} before the call.
// Returns a HIP error.
extern "C" int zs_forms_compare(int what, void* out, void* hip_stream)
{
    Result* const r = static_cast<Result*>(out);
    hipStream_t s = static_cast<hipStream_t>(hip_stream);
    switch (what) {
    case kBf16: compare_kernel<kBf16><<<kGroups, kThreads, 0, s>>>(r); break;
    case kRoot: compare_kernel<kRoot><<<kGroups, kThreads, 0, s>>>(r); break;
    case kQuotient:
        compare_kernel<kQuotient><<<kGroups, kThreads, 0, s>>>(r);
        break;
    case kCodes:
        compare_kernel<kCodes><<<kGroups, kThreads, 0, s>>>(r);
        break;
    case kHardware:
        compare_kernel<kHardware><<<kGroups, kThreads, 0, s>>>(r);
        break;
    default: return (int)hipErrorInvalidValue;
    }
    return (int)hipGetLastError();
}
