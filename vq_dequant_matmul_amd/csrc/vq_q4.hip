// vq_q4.hip -- dispatch of the 4-bit products (vq_q4_impl.hpp) and the
// router's bf16 product (gfx950).
#include <hip/hip_runtime.h>

#include "vq_common.hpp"
#include "vq_internal.hpp"

namespace vq {

template <int G>
hipError_t q4_group(const Q4Launch &L, hipStream_t stream);
extern template hipError_t q4_group<32>(const Q4Launch &, hipStream_t);
extern template hipError_t q4_group<64>(const Q4Launch &, hipStream_t);
extern template hipError_t q4_group<128>(const Q4Launch &, hipStream_t);

namespace {

// ---- the router's product -------------------------------------------------------
//
// logits[t][e] = sum_c w[e][c] x[t][c].  A few MB of bf16 weights: the time is
// one trip to memory for one token (512x4096: 2.6 us, an empty launch 2.5), and
// the reads of x from the caches for many (64 tokens of 512x4096: 10 us).  One
// wave takes TE experts and TN tokens, its lanes eight columns at a time, so
// that few experts still give many waves.  The sums are fp32 FMAs; matrix
// cores, fed with 16 experts and 16 tokens straight from memory, were slower (64
// tokens of 128x2816: 8.4 us against 5), for the 64 separate pieces of a load.

constexpr int kLogitWaves = 4;

// Keeps the loads before it there: they are not moved to their uses, into
// branches, where each would wait for the one before.
__device__ __forceinline__ void loads_first()
{
    asm volatile("" ::: "memory");
}

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ void widen(const u32x4 v, float (&f)[8])
{
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        f[2 * j] = __uint_as_float(v[j] << 16);
        f[2 * j + 1] = __uint_as_float(v[j] & 0xffff0000u);
    }
}

template <int TE, int TN, bool F32>
__global__ __launch_bounds__(64 * kLogitWaves) void k_logits(LogitsLaunch L)
{
    // Loads of w in flight.  With fp32 or two experts one step is 10 to 18 loads
    // already (64 tokens of 128x2816: fp32 6.0 us with one, 6.4 with two, bf16 6.1
    // and 5.3; two experts of 512x4096, bf16: 10.2 and 11.0, but fp32 14.0 and
    // 12.8).
    constexpr int kAhead = TN == 1 ? 8 : F32 || TE > 1 ? 1 : 2;
    const int lane = threadIdx.x & 63, t0 = blockIdx.y * TN;
    const int e0 =
        (blockIdx.x * kLogitWaves + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6)) * TE;
    if (e0 >= L.n_experts)
        return;
    const uint16_t *w[TE];
#pragma unroll
    for (int m = 0; m < TE; ++m)
        w[m] = L.w + (int64_t)min(e0 + m, L.n_experts - 1) * L.hidden;
    const char *x = static_cast<const char *>(L.x);
    constexpr int kBytes = F32 ? 4 : 2;
    float sum[TE][TN] = {};
    for (int c0 = lane * 8; c0 < L.hidden; c0 += 512 * kAhead) {
        u32x4 wr[kAhead][TE], xr[kAhead][TN][F32 ? 2 : 1];
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            const int c = min(c0 + i * 512, L.hidden - 8);
#pragma unroll
            for (int m = 0; m < TE; ++m)
                wr[i][m] = load_global(reinterpret_cast<const u32x4 *>(w[m] + c));
#pragma unroll
            for (int k = 0; k < TN; ++k) {
                const int t = min(t0 + k, L.n - 1);
                const u32x4 *p = reinterpret_cast<const u32x4 *>(
                    x + ((int64_t)t * L.hidden + c) * kBytes);
                xr[i][k][0] = load_global(p);
                if constexpr (F32)
                    xr[i][k][1] = load_global(p + 1);
            }
        }
        loads_first();
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            if (c0 + i * 512 >= L.hidden)
                break;
            float wf[TE][8], xf[8];
#pragma unroll
            for (int m = 0; m < TE; ++m)
                widen(wr[i][m], wf[m]);
#pragma unroll
            for (int k = 0; k < TN; ++k) {
                if constexpr (F32) {
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        xf[j] = __uint_as_float(xr[i][k][j / 4][j % 4]);
                } else {
                    widen(xr[i][k][0], xf);
                }
#pragma unroll
                for (int m = 0; m < TE; ++m)
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        sum[m][k] = fmaf(wf[m][j], xf[j], sum[m][k]);
            }
        }
    }
#pragma unroll
    for (int m = 0; m < TE; ++m)
#pragma unroll
        for (int k = 0; k < TN; ++k) {
            const float v = segment_sum_dpp(sum[m][k], 64);
            if (lane == 0 && e0 + m < L.n_experts && t0 + k < L.n)
                L.logits[(int64_t)(t0 + k) * L.n_experts + e0 + m] = v;
        }
}

template <int TE, int TN>
hipError_t logits_launch(const LogitsLaunch &L, hipStream_t stream)
{
    constexpr int kExperts = kLogitWaves * TE;
    const dim3 grid((L.n_experts + kExperts - 1) / kExperts, (L.n + TN - 1) / TN);
    if (L.x_f32)
        k_logits<TE, TN, true><<<grid, 64 * kLogitWaves, 0, stream>>>(L);
    else
        k_logits<TE, TN, false><<<grid, 64 * kLogitWaves, 0, stream>>>(L);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_q4(const Q4Launch &L, hipStream_t stream)
{
    switch (L.t[0].group) {
    case 32: return q4_group<32>(L, stream);
    case 64: return q4_group<64>(L, stream);
    default: return q4_group<128>(L, stream);
    }
}

hipError_t launch_router_logits(const LogitsLaunch &L, hipStream_t stream)
{
    // Two experts a wave, which halves the reads of x, where that leaves waves
    // enough for the chip (64 tokens of 512x4096: 10.2 us with two, 13.0 with one;
    // of 128x2816: 6.6 and 5.3); for fp32, whose x is twice as long, earlier
    // (of 256x4096: 10.1 and 11.3, in bf16 level: 7.8 and 7.5).
    const int64_t waves = (int64_t)L.n_experts * ((L.n + 7) / 8);
    return L.n == 1 ? logits_launch<1, 1>(L, stream)
         : L.n <= 4 ? logits_launch<1, 4>(L, stream)
         : waves > (L.x_f32 ? 1024 : 2048) ? logits_launch<2, 8>(L, stream)
                                           : logits_launch<1, 8>(L, stream);
}

}  // namespace vq
