// vq_route.hip -- selection of a token's experts from the router's logits,
// per-expert counts, the load-balance loss, and their gradient (gfx950).
//
// With p the token's softmax (or its sigmoid scores s over their sum), f_e =
// counts[e] / (N top_k) and N the tokens that count:
//   loss = E sum_e f_e (1/N) sum_t p[t][e]
//   d loss / d l[t][j] = (E/N) p_j (f_j - sum_e f_e p_e)  (* (1 - s_j), sigmoid)
// and for weights w = scale * s / sum(selected s) (renormalised):
//   d / d l_j = w_j (g_j - sum_i g_i w_i / scale)          (* (1 - s_j), sigmoid)
// for w = scale * s:
//   softmax: p_j (scale [j selected] g_j - sum_i g_i w_i), sigmoid: g_j w_j (1 - s_j).
//
// A segment of lanes works on a token, lane l of it owning experts
// [l VPL, (l + 1) VPL), so that the lowest lane of equal keys is the lowest
// index.  Each pass reads the logits once.  The chains of reductions and
// exchanges within a token bound the time, not HBM: 4096 tokens of 512 experts
// (sigmoid, bias, counts and loss, 8.7 MB) take 19.5 us, 14 for the selection
// and 5 for joining the partial sums in a fixed order; one token of 512 experts
// 4.5 us; the gradient for 16384 tokens of 128 (bf16, 9.5 MB) 9.6 us, 1.0 TB/s.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <type_traits>

#include "vq_bf16.hpp"
#include "vq_common.hpp"
#include "vq_internal.hpp"

namespace vq {
namespace {

constexpr int kRouteWaves = 8;      // waves per workgroup, forward (4096x512 with counts
                                    // and loss: 20.2 us, with 4 and two tokens each 22.3)
constexpr int kGradWaves = 4;       // and backward
constexpr int kRouteBlocks = 512;   // workgroups at most: rows of the partial sums
constexpr int kFinishExperts = 32;  // experts of a finishing workgroup: a line of each
                                    // row (4096x512: 20.2 us in all, 20.6 with 16, 21.5
                                    // with 64)
constexpr int kWsHeader = 2048;
constexpr float kNegInf = -__builtin_huge_valf();

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

// Workspace: a ticket (in its own 256 bytes), the finishing workgroups' partial
// losses, then per workgroup and expert the sum of p and the count.
struct RouteWs {
    uint32_t *ticket;
    double *part_loss;    // [32][2]: sum of count * p, sum of counts
    float *p;             // [blocks][n_experts]
    int32_t *c;           // [blocks][n_experts]
};

// Workgroups of `each` tokens, at most `most`, one at least.
int blocks_for(int n_tokens, int each, int most)
{
    const int64_t b = ((int64_t)n_tokens + each - 1) / each;
    return (int)std::max<int64_t>(1, std::min<int64_t>(b, most));
}

int route_blocks(int n_tokens) { return blocks_for(n_tokens, kRouteWaves, kRouteBlocks); }

RouteWs route_ws(void *ws, int n_experts, int blocks)
{
    char *p = static_cast<char *>(ws);
    RouteWs r;
    r.ticket = reinterpret_cast<uint32_t *>(p);
    r.part_loss = reinterpret_cast<double *>(p + 256);
    r.p = reinterpret_cast<float *>(p + kWsHeader);
    r.c = reinterpret_cast<int32_t *>(r.p + (size_t)blocks * n_experts);
    return r;
}

// ---- reductions over segments of S lanes (16, 32 or 64); every lane gets them ------

template <int S, class F>
__device__ __forceinline__ uint32_t segment_join(uint32_t v, F &&f)
{
    v = f(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0xb1, 0xf, 0xf, true));
    v = f(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x4e, 0xf, 0xf, true));
    v = f(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x141, 0xf, 0xf, true));
    v = f(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x140, 0xf, 0xf, true));
    if constexpr (S >= 32) {
        const auto r = __builtin_amdgcn_permlane16_swap(v, v, false, false);
        v = f(r[0], r[1]);
    }
    if constexpr (S >= 64) {
        const auto r = __builtin_amdgcn_permlane32_swap(v, v, false, false);
        v = f(r[0], r[1]);
    }
    return v;
}

template <int S>
__device__ __forceinline__ float segment_max(float v)
{
    return __uint_as_float(segment_join<S>(__float_as_uint(v), [](uint32_t a, uint32_t b) {
        return __float_as_uint(fmaxf(__uint_as_float(a), __uint_as_float(b)));
    }));
}

template <int S>
__device__ __forceinline__ float segment_sum(float v)
{
    return __uint_as_float(segment_join<S>(__float_as_uint(v), [](uint32_t a, uint32_t b) {
        return __float_as_uint(__uint_as_float(a) + __uint_as_float(b));
    }));
}

__device__ __forceinline__ double wave_sum(double v)
{
    for (int m = 32; m; m >>= 1)
        v += __shfl_xor(v, m);
    return v;
}

// ---- logits and scores ---------------------------------------------------------------

template <bool BF16>
__device__ __forceinline__ float logit_at(const void *p, int64_t i)
{
    if constexpr (BF16)
        return bf16_bits_to_float(static_cast<const uint16_t *>(p)[i]);
    else
        return static_cast<const float *>(p)[i];
}

// Logits [e0, e0 + VPL) of a row; -inf past the last expert.  by_four: rows of
// a multiple of four experts, aligned for vector loads.
template <int VPL, bool BF16>
__device__ __forceinline__ void load_logits(const void *p, int64_t row, int E, int e0,
                                            bool by_four, float (&l)[VPL])
{
    if (VPL >= 4 && by_four) {
#pragma unroll
        for (int j = 0; j < VPL; j += 4) {
            const int64_t i = row * E + (e0 + j < E ? e0 + j : 0);
            if constexpr (BF16) {
                const u32x2 v = load_global(reinterpret_cast<const u32x2 *>(
                    static_cast<const uint16_t *>(p) + i));
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    l[(j + k) % VPL] = __uint_as_float(k & 1 ? v[k / 2] & 0xffff0000u
                                                             : v[k / 2] << 16);
            } else {
                const u32x4 v = load_global(reinterpret_cast<const u32x4 *>(
                    static_cast<const float *>(p) + i));
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    l[(j + k) % VPL] = __uint_as_float(v[k]);
            }
        }
#pragma unroll
        for (int j = 0; j < VPL; ++j)
            l[j] = e0 + j < E ? l[j] : kNegInf;
    } else {
#pragma unroll
        for (int j = 0; j < VPL; ++j)
            l[j] = e0 + j < E ? logit_at<BF16>(p, row * E + e0 + j) : kNegInf;
    }
}

template <int VPL, bool BF16>
__device__ __forceinline__ void store_logits(void *p, int64_t row, int E, int e0, bool by_four,
                                             const float (&d)[VPL])
{
    if (VPL >= 4 && by_four) {
#pragma unroll
        for (int j = 0; j < VPL; j += 4) {
            if (e0 + j >= E)
                continue;
            const int64_t i = row * E + e0 + j;
            if constexpr (BF16) {
                u32x2 v;
#pragma unroll
                for (int k = 0; k < 2; ++k)
                    v[k] = float_to_bf16_bits(d[(j + 2 * k) % VPL]) |
                           (uint32_t)float_to_bf16_bits(d[(j + 2 * k + 1) % VPL]) << 16;
                *reinterpret_cast<u32x2 *>(static_cast<uint16_t *>(p) + i) = v;
            } else {
                f32x4 v;
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    v[k] = d[(j + k) % VPL];
                *reinterpret_cast<f32x4 *>(static_cast<float *>(p) + i) = v;
            }
        }
    } else {
#pragma unroll
        for (int j = 0; j < VPL; ++j)
            if (e0 + j < E) {
                if constexpr (BF16)
                    static_cast<uint16_t *>(p)[row * E + e0 + j] = float_to_bf16_bits(d[j]);
                else
                    static_cast<float *>(p)[row * E + e0 + j] = d[j];
            }
    }
}

// exp(x) by the hardware's exp2 at x log2(e), with what the product's rounding and
// the constant's leave out, d: 2^hi (1 + d ln 2), 2^-22 relative.  (Without that
// term the error grows with |x|, to 5e-6 at 80.)  Infinities of x make d NaN,
// which the median turns into a bound that changes no 0 and no infinity.
__device__ __forceinline__ float exp_fast(float x)
{
    constexpr float kLog2e = 0x1.715476p+0f, kLog2eLow = 0x1.4ae0cp-26f, kLn2 = 0x1.62e43p-1f;
    const float hi = kLog2e * x;
    const float d = fmaf(kLog2eLow, x, fmaf(kLog2e, x, -hi));
    return __builtin_amdgcn_exp2f(hi) *
           fmaf(kLn2, __builtin_amdgcn_fmed3f(d, -0x1p-10f, 0x1p-10f), 1.0f);
}

// FAST: exp_fast and the hardware's reciprocal.
template <bool FAST = false>
__device__ __forceinline__ float sigmoid(float v)
{
    if constexpr (FAST)
        return __builtin_amdgcn_rcpf(1.0f + exp_fast(-v));
    else
        return 1.0f / (1.0f + expf(-v));
}

// The lane's scores, p = score * inv (0 where no score is above 0), and the
// row's largest logit and sum of exponentials for the softmax.  Relative error
// a few 2^-24, with FAST (the order, which near ties decide in 64 bits, the loss
// and gradients that are rounded to bf16) a few 2^-23.
template <int VPL, int S, bool FAST>
__device__ __forceinline__ void scores(bool sig, const float (&l)[VPL], float (&s)[VPL],
                                       float &inv, float &top, float &total)
{
    top = kNegInf;
    total = 0.0f;
    if (!sig) {
#pragma unroll
        for (int j = 0; j < VPL; ++j)
            top = fmaxf(top, l[j]);
        top = segment_max<S>(top);
    }
#pragma unroll
    for (int j = 0; j < VPL; ++j) {
        s[j] = sig ? sigmoid<FAST>(l[j]) : FAST ? exp_fast(l[j] - top) : expf(l[j] - top);
        total += s[j];
    }
    total = segment_sum<S>(total);
    inv = total == 0.0f ? 0.0f : 1.0f / total;
    if (!sig) {
#pragma unroll
        for (int j = 0; j < VPL; ++j)
            s[j] *= inv;
        inv = 1.0f;
    }
}

// ---- selection -------------------------------------------------------------------------

// Order-preserving integers; 0 is below every key.  NaN is ordered as -inf,
// -0 as 0.
__device__ __forceinline__ uint32_t order_key(float v)
{
    v = v > kNegInf ? v + 0.0f : kNegInf;
    const uint32_t u = __float_as_uint(v);
    return (u >> 31) ? ~u : u | 0x80000000u;
}

__device__ __forceinline__ float key_value(uint32_t k)
{
    return __uint_as_float((k >> 31) ? k & 0x7fffffffu : ~k);
}

__device__ __forceinline__ uint64_t order_key(double v)
{
    if (!(v > -__builtin_huge_val()))
        return 1;
    const uint64_t u = (uint64_t)__double_as_longlong(v + 0.0);
    return (u >> 63) ? ~u : u | 0x8000000000000000ull;
}

// What a wave shares through LDS while it orders a token's experts.
template <int VPL>
struct RouteRow {
    float logit[64 * VPL];
    uint32_t key[64], expert[64];   // candidates
};

__device__ __forceinline__ void wave_lds_sync()
{
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// The number of the n candidates (one per lane) that come before the lane's.
template <class K>
__device__ __forceinline__ int rank_of(K key, int expert, int n)
{
    int before = 0;
    for (int i = 0; i < n; ++i) {
        K other;
        if constexpr (sizeof(K) == 4)
            other = (K)__builtin_amdgcn_readlane((int)key, i);
        else
            other = (K)(uint32_t)__builtin_amdgcn_readlane((int)key, i) |
                    (K)(uint32_t)__builtin_amdgcn_readlane((int)(key >> 32), i) << 32;
        const int at = __builtin_amdgcn_readlane(expert, i);
        before += other > key || (other == key && at < expert);
    }
    return before;
}

// One expert's key in 64 bits; top and total are the row's largest logit and
// sum of exponentials (softmax).
__device__ __forceinline__ uint64_t exact_key(float logit, float bias, bool sig, double top,
                                              double total)
{
    const double v = logit;
    if (!(logit > kNegInf))
        return 1;
    return order_key((sig ? 1.0 / (1.0 + exp(-v)) : exp(v - top) / total) + (double)bias);
}

__device__ __noinline__ void exact_softmax(const float *logit, int E, double &top, double &total)
{
    const int lane = threadIdx.x & 63;
    top = -__builtin_huge_val();
    for (int e = lane; e < E; e += 64)
        top = fmax(top, (double)logit[e]);
    for (int d = 32; d; d >>= 1)
        top = fmax(top, __shfl_xor(top, d));
    total = 0.0;
    for (int e = lane; e < E; e += 64)
        total += exp((double)logit[e] - top);
    total = wave_sum(total);
}

// The slots of n <= 64 candidates by 64-bit keys.
__device__ __noinline__ int exact_slot(const float *logit, const float *bias, bool sig, int E,
                                       int n, int expert)
{
    double top = 0.0, total = 1.0;
    if (!sig)
        exact_softmax(logit, E, top, total);
    const bool live = (int)(threadIdx.x & 63) < n;
    return rank_of(live ? exact_key(logit[expert], bias[expert], sig, top, total) : (uint64_t)0,
                   expert, n);
}

// The k largest of all E in order, one maximum of the wave after another, in
// 64 bits: for tokens with more than 64 candidates (many equal keys).
template <int VPL>
__device__ __noinline__ int select_all(const float *logit, const float *bias, bool sig, int k,
                                       int E)
{
    const int lane = threadIdx.x & 63;
    double top = 0.0, total = 1.0;
    if (bias && !sig)
        exact_softmax(logit, E, top, total);
    uint64_t key[VPL];
#pragma unroll
    for (int j = 0; j < VPL; ++j) {
        const int e = lane * VPL + j;
        key[j] = e >= E ? 0
                 : bias ? exact_key(logit[e], bias[e], sig, top, total)
                        : order_key((double)logit[e]);
    }
    int mine = 0;
    for (int s = 0; s < k; ++s) {
        uint64_t best = 0;
        int at = 0x7fffffff;
#pragma unroll
        for (int j = 0; j < VPL; ++j)
            if (key[j] > best) {
                best = key[j];
                at = lane * VPL + j;
            }
        for (int d = 32; d; d >>= 1) {
            const uint64_t ob = __shfl_xor(best, d);
            const int oa = __shfl_xor(at, d);
            if (ob > best || (ob == best && oa < at)) {
                best = ob;
                at = oa;
            }
        }
#pragma unroll
        for (int j = 0; j < VPL; ++j)
            if (at == lane * VPL + j)
                key[j] = 0;
        if (lane == s)
            mine = at;
    }
    return mine;
}

// The k largest keys in order: lane s returns the s-th expert.  The k-th
// largest of the lanes' own maxima is a bound that at least k keys reach and
// few others do: it is found bit by bit, each bit one compare and a count of
// the wave.  The keys that reach it move to one lane each and count those
// before them.  (One maximum of the wave per slot instead took two and a half
// times the instructions, most of them on the one scalar unit of a CU.)
//
// With a bias a key is off by less than kNear * (|key| + bias_max) / 2 (the
// scores by a few 2^-23 of them, and the rounding of the sum): what is within kNear of the bound is a candidate too, and if two
// neighbours among the first k + 1 are, the candidates are ordered by 64-bit
// keys.
template <int VPL>
__device__ __forceinline__ int select(const uint32_t (&key)[VPL], RouteRow<VPL> &row,
                                      const float *bias, bool sig, int k, int E, float bias_max)
{
    constexpr float kNear = 0x1p-15f;
    const int lane = threadIdx.x & 63;
    uint32_t most = key[0];
#pragma unroll
    for (int j = 1; j < VPL; ++j)
        most = max(most, key[j]);
    uint32_t bound = 0, reach = 1;
    uint64_t held[VPL];
    int n = E;
    // 16 bits (seven of the mantissa) mostly do, all 32 where keys lie close
    for (int bit = 31; bit >= 0 && n > 64; --bit) {
        const uint32_t next = bound | 1u << bit;
        if (__popcll(__ballot(most >= next)) >= k)
            bound = next;
        if (bit == 16 || bit == 0) {
            reach = max(bound, 1u);
            if (bias) {
                const float v = key_value(reach);
                reach = v > kNegInf ? order_key(v - kNear * (fabsf(v) + bias_max)) : 1u;
            }
            n = 0;
#pragma unroll
            for (int j = 0; j < VPL; ++j)
                n += __popcll(__ballot(key[j] >= reach));
        }
    }
    if (n > 64)
        return select_all<VPL>(row.logit, bias, sig, k, E);
    int base = 0;
#pragma unroll
    for (int j = 0; j < VPL; ++j) {
        held[j] = __ballot(key[j] >= reach);
        if (key[j] >= reach) {
            const int at = base + __builtin_amdgcn_mbcnt_hi(
                (uint32_t)(held[j] >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)held[j], 0));
            row.key[at] = key[j];
            row.expert[at] = lane * VPL + j;
        }
        base += __popcll(held[j]);
    }
    wave_lds_sync();
    const bool live = lane < n;
    const uint32_t mine = live ? row.key[lane] : 0;
    const int expert = live ? row.expert[lane] : 0;
    int slot = rank_of(mine, expert, n);
    if (bias) {
        // the ordered keys, and each one's distance from the next
        wave_lds_sync();
        if (live)
            row.key[slot] = mine;
        wave_lds_sync();
        bool close = false;
        if (lane < k && lane + 1 < n) {
            const float a = key_value(row.key[lane]), b = key_value(row.key[lane + 1]);
            close = a - b <= kNear * (fabsf(a) + bias_max);
        }
        if (__any(close))
            slot = exact_slot(row.logit, bias, sig, E, n, expert);
    }
    wave_lds_sync();
    if (live)
        row.expert[slot] = expert;
    wave_lds_sync();
    const int out = row.expert[lane];   // (lanes past the slots: not used)
    wave_lds_sync();
    return out;
}

// The sums of p over tokens: fp32 over kHeld tokens of a wave; where a wave has
// more, whole numbers of 2^-40 in LDS for the workgroup (whose order does not
// matter; at most 2^22 tokens, 2^62); 64 bits over the waves' last ones and the
// workgroups, with one rounding to fp32 between.  (Whole numbers for the last
// ones too: 4096x512 19.8 us, else 19.3.)
constexpr int kHeld = 16;

template <int VPL>
__device__ __forceinline__ void flush_sums(float (&psum)[VPL], unsigned long long *sums, bool *bad)
{
    const int lane = threadIdx.x & 63;
    bool nan = false;
#pragma unroll
    for (int j = 0; j < VPL; ++j) {
        nan |= psum[j] != psum[j];
        // below 2^52: the number is in the mantissa
        const double v = fma((double)psum[j], 0x1p40, 0x1p52);
        atomicAdd(&sums[j * 64 + lane],
                  (unsigned long long)__double_as_longlong(v) & 0xfffffffffffffull);
        psum[j] = 0.0f;
    }
    if (nan)
        *bad = true;
}

template <int VPL, bool BF16>
__global__ __launch_bounds__(64 * kRouteWaves, VPL <= 8 ? 4 : 2) void k_route(RouteLaunch L, RouteWs ws)
{
    __shared__ RouteRow<VPL> rows[kRouteWaves];   // at last, the sums of p in place of logits
    __shared__ unsigned long long lp[64 * VPL];   // [VPL][64]: a lane's experts apart
    __shared__ int lc[64 * VPL];
    __shared__ bool bad;                          // a NaN among the p
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, E = L.n_experts, k = L.top_k;
    const int e0 = lane * VPL;
    const bool stats = L.counts != nullptr, sig = L.sigmoid;
    const bool by_four = E % 4 == 0 &&
                         reinterpret_cast<uintptr_t>(L.logits) % (BF16 ? 8 : 16) == 0;
    if (stats) {
        if (blockIdx.x == 0 && threadIdx.x == 0)
            *ws.ticket = 0;
        if (threadIdx.x == 0)
            bad = false;
        for (int i = threadIdx.x; i < 64 * VPL; i += 64 * kRouteWaves) {
            lc[i] = 0;
            lp[i] = 0;
        }
        __syncthreads();
    }
    float bias[VPL], bias_max = 0.0f;
    if (L.bias) {
#pragma unroll
        for (int j = 0; j < VPL; ++j) {
            bias[j] = e0 + j < E ? L.bias[e0 + j] : 0.0f;
            bias_max = fmaxf(bias_max, fabsf(bias[j]));
        }
        bias_max = segment_max<64>(bias_max);
    }
    float psum[VPL] = {};
    const int64_t first = (int64_t)blockIdx.x * kRouteWaves + wave;
    const int64_t step = (int64_t)gridDim.x * kRouteWaves;
    int64_t flush_at = first + kHeld * step;
    for (int64_t t = first; t < L.n_tokens; t += step) {
        if (stats && t == flush_at) {
            flush_sums(psum, lp, &bad);
            flush_at += kHeld * step;
        }
        float l[VPL];
        load_logits<VPL, BF16>(L.logits, t, E, e0, by_four, l);
        bool some = false;
#pragma unroll
        for (int j = 0; j < VPL; ++j)
            some |= l[j] != kNegInf;
        if ((L.mask && !L.mask[t]) || !__any(some)) {
            if (lane < k) {
                L.ids[t * k + lane] = lane;
                L.weights[t * k + lane] = 0.0f;
            }
            continue;
        }
        // scores of all experts, where the order, the weights or the loss use them
        float sc[VPL], inv = 0.0f, top = 0.0f, total = 0.0f;
        if (L.bias || stats || (!sig && !L.renormalize))
            scores<VPL, 64, true>(sig, l, sc, inv, top, total);
        uint32_t key[VPL];
#pragma unroll
        for (int j = 0; j < VPL; ++j) {
            const float v = L.bias && l[j] > kNegInf ? sc[j] + bias[j] : l[j];
            key[j] = e0 + j < E ? order_key(v) : 0;
        }
#pragma unroll
        for (int j = 0; j < VPL; ++j)
            rows[wave].logit[e0 + j] = l[j];
        wave_lds_sync();
        const int mine = select<VPL>(key, rows[wave], L.bias, sig, k, E, bias_max);
        // weights, from the chosen logits
        const float v = lane < k ? rows[wave].logit[mine] : kNegInf;
        float w;
        if (sig)
            w = lane < k ? sigmoid(v) : 0.0f;
        else if (L.renormalize)
            w = expf(v - segment_max<64>(v));
        else
            w = expf(v - top) / total;
        if (L.renormalize) {
            const float tot = segment_sum<64>(w);
            w = tot == 0.0f ? 0.0f : w / tot;
        }
        if (lane < k) {
            L.ids[t * k + lane] = mine;
            L.weights[t * k + lane] = w * L.scale;
        }
        if (stats) {
            if (lane < k)
                atomicAdd(&lc[mine], 1);
#pragma unroll
            for (int j = 0; j < VPL; ++j)
                psum[j] += sc[j] * inv;
        }
    }
    if (!stats)
        return;
#pragma unroll
    for (int j = 0; j < VPL; ++j)
        rows[wave].logit[e0 + j] = psum[j];
    __syncthreads();
    for (int e = threadIdx.x; e < E; e += 64 * kRouteWaves) {
        double v = (double)lp[e % VPL * 64 + e / VPL] * 0x1p-40;
        for (int w = 0; w < kRouteWaves; ++w)
            v += rows[w].logit[e];
        ws.p[(size_t)blockIdx.x * E + e] = bad ? __builtin_nanf("") : (float)v;
        ws.c[(size_t)blockIdx.x * E + e] = lc[e];
    }
}

// Workgroup b joins the partial sums of experts [32 b, 32 b + 32): 32 rows of
// threads with eight workgroups' sums each in flight.  The last one to finish
// joins their contributions to the loss, in workgroup order.
__global__ __launch_bounds__(1024) void k_route_finish(RouteWs ws, int blocks, int E, int k,
                                                       int32_t *counts, float *loss)
{
    constexpr int kRows = 1024 / kFinishExperts, kAtOnce = 8;
    __shared__ double lp[kRows][kFinishExperts];
    __shared__ int lc[kRows][kFinishExperts];
    __shared__ bool last;
    const int col = threadIdx.x % kFinishExperts, row = threadIdx.x / kFinishExperts;
    const int e = blockIdx.x * kFinishExperts + col;
    double p = 0.0;
    int c = 0;
    if (e < E)
        for (int b0 = row; b0 < blocks; b0 += kRows * kAtOnce) {
            float pv[kAtOnce];
            int cv[kAtOnce];
#pragma unroll
            for (int i = 0; i < kAtOnce; ++i) {
                const int b = min(b0 + i * kRows, blocks - 1);
                pv[i] = ws.p[(size_t)b * E + e];
                cv[i] = ws.c[(size_t)b * E + e];
            }
#pragma unroll
            for (int i = 0; i < kAtOnce; ++i)
                if (b0 + i * kRows < blocks) {
                    p += pv[i];
                    c += cv[i];
                }
        }
    lp[row][col] = p;
    lc[row][col] = c;
    for (int n = kRows / 2; n > 0; n /= 2) {
        __syncthreads();
        if (row < n) {
            lp[row][col] += lp[row + n][col];
            lc[row][col] += lc[row + n][col];
        }
    }
    __syncthreads();
    if (threadIdx.x < 64) {
        const bool mine = threadIdx.x < kFinishExperts && e < E;
        p = mine ? lp[0][col] : 0.0;
        c = mine ? lc[0][col] : 0;
        if (mine)
            counts[e] = c;
        const double cp = wave_sum((double)c * p), cs = wave_sum((double)c);
        if (threadIdx.x == 0) {
            __hip_atomic_store(ws.part_loss + 2 * blockIdx.x, cp, __ATOMIC_RELAXED,
                               __HIP_MEMORY_SCOPE_AGENT);
            __hip_atomic_store(ws.part_loss + 2 * blockIdx.x + 1, cs, __ATOMIC_RELAXED,
                               __HIP_MEMORY_SCOPE_AGENT);
            last = __hip_atomic_fetch_add(ws.ticket, 1u, __ATOMIC_ACQ_REL,
                                          __HIP_MEMORY_SCOPE_AGENT) == gridDim.x - 1;
        }
    }
    __syncthreads();
    if (!last || threadIdx.x >= 64)
        return;
    // (at most 32 workgroups: one lane each)
    double cp = 0.0, cs = 0.0;
    if (threadIdx.x < gridDim.x) {
        cp = __hip_atomic_load(ws.part_loss + 2 * threadIdx.x, __ATOMIC_RELAXED,
                               __HIP_MEMORY_SCOPE_AGENT);
        cs = __hip_atomic_load(ws.part_loss + 2 * threadIdx.x + 1, __ATOMIC_RELAXED,
                               __HIP_MEMORY_SCOPE_AGENT);
    }
    cp = wave_sum(cp);
    cs = wave_sum(cs);
    // cs = N k, so cp / (N k) / N = cp k / cs^2
    if (threadIdx.x == 0)
        *loss = cs > 0.0 ? (float)(E * cp * k / (cs * cs)) : 0.0f;
}

// ---- gradient ----------------------------------------------------------------------------

// S lanes per token, 64 / S tokens per wave.
template <int VPL, int S, bool BF16>
__global__ __launch_bounds__(64 * kGradWaves) void k_route_grad(RouteGradLaunch L)
{
    __shared__ float rows[kGradWaves * 64 / S][S * VPL];
    __shared__ double sums[kGradWaves];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, E = L.n_experts, k = L.top_k;
    const int sl = lane % S, e0 = sl * VPL, seg = threadIdx.x / S;
    const bool sig = L.sigmoid;
    const bool by_four = E % 4 == 0 &&
                         reinterpret_cast<uintptr_t>(L.logits) % (BF16 ? 8 : 16) == 0 &&
                         reinterpret_cast<uintptr_t>(L.d_logits) % (BF16 ? 8 : 16) == 0;
    constexpr int kTokens = kGradWaves * 64 / S;     // of a workgroup at a time
    constexpr int KPL = kMaxRouteTopK / S;           // slots of a lane at most
    // A token's loads, issued together before the counts are summed.  Segments
    // past the last token work on it again and do not store.
    float l[VPL], g[KPL];
    int id[KPL];
    bool counted;
    const auto fetch = [&](int64_t t) {
        load_logits<VPL, BF16>(L.logits, t, E, e0, by_four, l);
        counted = !L.mask || L.mask[t];
#pragma unroll
        for (int i = 0; i < KPL; ++i) {
            const int slot = i * S + sl;
            const bool have = L.d_weights && slot < k;
            id[i] = have ? L.ids[t * k + slot] : -1;
            g[i] = have ? L.d_weights[t * k + slot] : 0.0f;
        }
    };
    const int64_t last = L.n_tokens - 1;
    fetch(min((int64_t)blockIdx.x * kTokens + seg, last));
    float f[VPL] = {};   // d_loss * E * counts / (N k) / N
    if (L.counts) {
        double cs = 0.0;   // the workgroup's sum of all counts
        for (int e = threadIdx.x; e < E; e += 64 * kGradWaves)
            cs += L.counts[e];
        cs = wave_sum(cs);
        if (lane == 0)
            sums[wave] = cs;
        __syncthreads();
        cs = 0.0;
        for (int w = 0; w < kGradWaves; ++w)
            cs += sums[w];
        const float a = cs > 0.0 ? (float)((double)L.d_loss[0] * E * k / (cs * cs)) : 0.0f;
#pragma unroll
        for (int j = 0; j < VPL; ++j)
            f[j] = e0 + j < E ? a * (float)L.counts[e0 + j] : 0.0f;
    }
    for (int64_t t0 = (int64_t)blockIdx.x * kTokens; t0 < L.n_tokens;
         t0 += (int64_t)gridDim.x * kTokens) {
        const int64_t t = min(t0 + seg, last);
        if (t0 != (int64_t)blockIdx.x * kTokens)
            fetch(t);
        float d[VPL] = {};
        bool some = false;
#pragma unroll
        for (int j = 0; j < VPL; ++j)
            some |= l[j] != kNegInf;
        const uint64_t bits = __ballot(some) >> (lane / S * S);
        const bool live = (S == 64 ? bits : bits & ((1ull << (S % 64)) - 1)) != 0 && counted;
        if (!live) {   // (no NaN into the sums below)
#pragma unroll
            for (int j = 0; j < VPL; ++j)
                l[j] = 0.0f;
        }
        float s[VPL], inv, top, total;
        scores<VPL, S, BF16>(sig, l, s, inv, top, total);
        if (L.counts) {
            float dot = 0.0f;
#pragma unroll
            for (int j = 0; j < VPL; ++j)
                dot += s[j] * inv * f[j];
            dot = segment_sum<S>(dot);
#pragma unroll
            for (int j = 0; j < VPL; ++j)
                d[j] = s[j] * inv * (f[j] - dot);
        }
        if (L.d_weights) {
            // the slots' scores over what divides them, and the mean they subtract
            float *row = rows[seg];
#pragma unroll
            for (int j = 0; j < VPL; ++j)
                row[e0 + j] = l[j];
            __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
            __builtin_amdgcn_wave_barrier();
            __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
            float w[KPL], sel_top = kNegInf, tot = 0.0f, mean = 0.0f;
#pragma unroll
            for (int i = 0; i < KPL; ++i) {
                if (id[i] < 0 || id[i] >= E)
                    id[i] = -1;
                g[i] = id[i] < 0 ? 0.0f : g[i] * L.scale;
                w[i] = id[i] < 0 || !live ? kNegInf : row[id[i]];
                sel_top = fmaxf(sel_top, w[i]);
            }
            if (!sig)
                sel_top = L.renormalize ? segment_max<S>(sel_top) : top;
#pragma unroll
            for (int i = 0; i < KPL; ++i) {
                w[i] = id[i] < 0 || !live ? 0.0f : sig ? sigmoid(w[i]) : expf(w[i] - sel_top);
                tot += w[i];
            }
            tot = L.renormalize ? segment_sum<S>(tot) : sig ? 1.0f : total;
            const float over = tot == 0.0f ? 0.0f : 1.0f / tot;
#pragma unroll
            for (int i = 0; i < KPL; ++i) {
                // the quotient with its remainder: the one weight of a single slot is
                // 1, and its gradient 0
                const float v = w[i] * over;
                w[i] = fmaf(fmaf(-v, tot, w[i]), over, v);
                mean += g[i] * w[i];
            }
            mean = segment_sum<S>(mean);
            const float sub = L.renormalize ? mean : 0.0f;       // from the slots
            const float all = !L.renormalize && !sig ? mean : 0.0f;   // from every expert
            // to their experts' lanes, through the segment's row
            __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
            __builtin_amdgcn_wave_barrier();
#pragma unroll
            for (int j = 0; j < VPL; ++j)
                row[e0 + j] = 0.0f;
            __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
            __builtin_amdgcn_wave_barrier();
#pragma unroll
            for (int i = 0; i < KPL; ++i)
                if (id[i] >= 0)
                    atomicAdd(&row[id[i]], w[i] * (g[i] - sub));
            __builtin_amdgcn_wave_barrier();
            __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
#pragma unroll
            for (int j = 0; j < VPL; ++j)
                d[j] += row[e0 + j] - s[j] * inv * all;
            __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
            __builtin_amdgcn_wave_barrier();
        }
#pragma unroll
        for (int j = 0; j < VPL; ++j) {
            if (sig)
                d[j] *= sigmoid<BF16>(-l[j]);   // 1 - s, without its cancellation near s = 1
            if (l[j] == kNegInf || !live)
                d[j] = 0.0f;
        }
        if (t0 + seg < L.n_tokens)
            store_logits<VPL, BF16>(L.d_logits, t, E, e0, by_four, d);
    }
}

template <class F>
hipError_t by_width(int n_experts, bool bf16, F &&f)
{
#define VQ_WIDTH(V)                                                                               \
    if (n_experts <= 64 * V)                                                                      \
        return bf16 ? f(std::integral_constant<int, V>(), std::true_type())                       \
                    : f(std::integral_constant<int, V>(), std::false_type());
    VQ_WIDTH(1)
    VQ_WIDTH(2)
    VQ_WIDTH(4)
    VQ_WIDTH(8)
    VQ_WIDTH(16)
#undef VQ_WIDTH
    return hipErrorInvalidValue;
}

template <int VPL, int S>
hipError_t grad_launch(const RouteGradLaunch &L, hipStream_t stream)
{
    constexpr int kTokens = kGradWaves * 64 / S;
    // at most eight workgroups per CU (256): each sums the counts first
    const int blocks = blocks_for(L.n_tokens, kTokens, 2048);
    if (L.logits_bf16)
        k_route_grad<VPL, S, true><<<blocks, 64 * kGradWaves, 0, stream>>>(L);
    else
        k_route_grad<VPL, S, false><<<blocks, 64 * kGradWaves, 0, stream>>>(L);
    return hipGetLastError();
}

}  // namespace

size_t route_workspace_bytes(int n_experts, int n_tokens)
{
    static_assert(256 + kMaxSelectExperts / kFinishExperts * 16 <= kWsHeader, "header too small");
    return kWsHeader + (size_t)route_blocks(n_tokens) * n_experts * 8;
}

hipError_t launch_route(const RouteLaunch &L, hipStream_t stream)
{
    const int blocks = L.counts ? route_blocks(L.n_tokens)
                                : blocks_for(L.n_tokens, kRouteWaves, 8192);
    const RouteWs ws = route_ws(L.ws, L.n_experts, blocks);
    hipError_t e = by_width(L.n_experts, L.logits_bf16, [&](auto v, auto bf) {
        k_route<decltype(v)::value, decltype(bf)::value>
            <<<blocks, 64 * kRouteWaves, 0, stream>>>(L, ws);
        return hipGetLastError();
    });
    if (e != hipSuccess || !L.counts)
        return e;
    k_route_finish<<<(L.n_experts + kFinishExperts - 1) / kFinishExperts, 1024, 0, stream>>>(
        ws, blocks, L.n_experts, L.top_k, L.counts, L.loss);
    return hipGetLastError();
}

hipError_t launch_route_grad(const RouteGradLaunch &L, hipStream_t stream)
{
    // eight experts per lane where that fills it: fewer lanes a token, shorter
    // chains of reductions (16384 tokens of 128: 16 lanes)
    if (L.n_experts <= 64)
        return grad_launch<4, 16>(L, stream);
    if (L.n_experts <= 128)
        return grad_launch<8, 16>(L, stream);
    if (L.n_experts <= 256)
        return grad_launch<8, 32>(L, stream);
    if (L.n_experts <= 512)
        return grad_launch<8, 64>(L, stream);
    return grad_launch<16, 64>(L, stream);
}

}  // namespace vq
