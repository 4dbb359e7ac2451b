// vq_norm.hip -- the norms at both ends of a block, fused with the residual
// add between them, and their gradient (gfx950).
//
// Per token, with n = hidden, q = 1/sqrt(mean(y^2) + eps), a = o + post_weight,
// r = 1/sqrt(mean(h'^2) + eps), b = o + pre_weight, g the gate:
//   z = q a y,   h' = skip h + block g z,   x = r b h'
// and backward, D the whole gradient by h' (u = b dx, B = block D):
//   D = dh' + r (u - h' r mean(u h' r))             dh = skip D
//   dy = q (a g B - y q mean(a g B y q))            (no post norm: dy = g B)
//   db = sum_t dx r h',  da = sum_t g B q y,  dg = sum B z
// A gate per channel (or none) is the same for every token, so da = g S and
// dg = a S with one sum over tokens, S = sum_t B q y.
//
// One workgroup holds a token's row in registers, V groups of four values per
// thread, so every array is read once: HBM bounds both directions (4096x4096,
// fp32 h and y, bf16 x: 235 MB in 51 us, 4.6 TB/s, on outputs that are new each
// time, 44 where the same ones stay in the 256 MB cache in part; the gradient
// of 8191x2816 in bf16: 277 MB in 67 us, 4.2 TB/s, 5 of them to join its partial
// sums).  Rows past 8192 do not fit the gradient's registers: 42 to 84 of a
// thread's are in scratch (2048x16384 in bf16: 181 us, 2.2 TB/s; 2048x8192: 64,
// 3.2 TB/s).
#include <hip/hip_runtime.h>

#include <algorithm>
#include <type_traits>

#include "vq_bf16.hpp"
#include "vq_common.hpp"
#include "vq_internal.hpp"

namespace vq {
namespace {

constexpr int kNormMaxThreads = 1024;

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

// Four values of an fp32 or bf16 array as they are in memory.
template <bool F32>
struct Raw4 {
    typedef std::conditional_t<F32, u32x4, u32x2> type;
};

// Group i of a row that starts at element `row` (the same in every lane): a
// uniform base and a 32-bit offset.
template <bool F32>
__device__ __forceinline__ typename Raw4<F32>::type load_raw(const void *p, int64_t row,
                                                             uint32_t i)
{
    typedef const __attribute__((address_space(1))) char *Bytes;
    typedef const __attribute__((address_space(1))) typename Raw4<F32>::type *Ptr;
    const Bytes base = (Bytes)(reinterpret_cast<uintptr_t>(p) + row * (F32 ? 4 : 2));
    return *(Ptr)(base + i * (F32 ? 16u : 8u));
}

__device__ __forceinline__ void expand(u32x4 a, float (&v)[4])
{
#pragma unroll
    for (int j = 0; j < 4; ++j)
        v[j] = __uint_as_float(a[j]);
}

__device__ __forceinline__ void expand(u32x2 a, float (&v)[4])
{
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        v[2 * j] = __uint_as_float(a[j] << 16);
        v[2 * j + 1] = __uint_as_float(a[j] & 0xffff0000u);
    }
}

template <bool F32>
__device__ __forceinline__ void store4(void *p, int64_t row, uint32_t i, const float (&v)[4])
{
    typedef __attribute__((address_space(1))) char *Bytes;
    typedef __attribute__((address_space(1))) typename Raw4<F32>::type *Ptr;
    const Bytes base = (Bytes)(reinterpret_cast<uintptr_t>(p) + row * (F32 ? 4 : 2));
    typename Raw4<F32>::type a;
    if constexpr (F32) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
            a[j] = __float_as_uint(v[j]);
    } else {
#pragma unroll
        for (int j = 0; j < 2; ++j)
            a[j] = float_to_bf16_bits(v[2 * j]) | (uint32_t)float_to_bf16_bits(v[2 * j + 1]) << 16;
    }
    *(Ptr)(base + i * (F32 ? 16u : 8u)) = a;
}

// The forward's weights and gates have their type at run time: a uniform branch.
__device__ __forceinline__ void load_weight(const void *p, uint32_t i, bool f32, float (&v)[4])
{
    if (f32)
        expand(load_raw<true>(p, 0, i), v);
    else
        expand(load_raw<false>(p, 0, i), v);
}

__device__ __forceinline__ float scalar_at(const void *p, int64_t i, bool f32)
{
    return f32 ? static_cast<const float *>(p)[i]
               : bf16_bits_to_float(static_cast<const uint16_t *>(p)[i]);
}

// Sums of N values over the workgroup; every thread gets them.  lds is one of
// two buffers used in turn, so that one barrier per sum is enough.
template <int N>
__device__ __forceinline__ void block_sum(float (&v)[N], float *lds)
{
    const int waves = blockDim.x >> 6;
#pragma unroll
    for (int i = 0; i < N; ++i)
        v[i] = segment_sum_dpp(v[i], 64);
    if (waves == 1)
        return;
    if ((threadIdx.x & 63) == 0)
#pragma unroll
        for (int i = 0; i < N; ++i)
            lds[(threadIdx.x >> 6) * N + i] = v[i];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i)
        v[i] = 0.0f;
    for (int w = 0; w < waves; ++w)
#pragma unroll
        for (int i = 0; i < N; ++i)
            v[i] += lds[w * N + i];
}

template <int V, bool HF, bool YF, bool XF>
__global__ __launch_bounds__(kNormMaxThreads) void k_norm(vq_block_norm_args a)
{
    __shared__ float lds[2][kNormMaxThreads / 64];
    const int n4 = a.hidden / 4, nt = blockDim.x;
    const bool wf = a.weight_dtype == VQ_F32;
    const float inv = 1.0f / (float)a.hidden;
    const int64_t t = blockIdx.x;
    float h[V][4], y[V][4];
    float sum[1] = {0.0f};
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int i = v * nt + threadIdx.x;
        if (i < n4) {
            expand(load_raw<HF>(a.h, t * a.h_stride, i), h[v]);
            if (a.y)
                expand(load_raw<YF>(a.y, t * a.y_stride, i), y[v]);
        }
    }
    if (a.post_weight) {
#pragma unroll
        for (int v = 0; v < V; ++v)
            if (v * nt + (int)threadIdx.x < n4)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    sum[0] += y[v][j] * y[v][j];
        block_sum<1>(sum, lds[0]);
    }
    const float q = 1.0f / sqrtf(sum[0] * inv + a.eps);
    float scale = a.block_scale;
    if (a.gate_kind == VQ_GATE_TOKEN)
        scale *= scalar_at(a.gate, t, wf);
    sum[0] = 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int i = v * nt + threadIdx.x;
        if (i >= n4)
            continue;
        float w[4];
        if (a.post_weight) {
            load_weight(a.post_weight, i, wf, w);
#pragma unroll
            for (int j = 0; j < 4; ++j)
                y[v][j] *= q * (w[j] + a.weight_offset);
        }
        if (a.gate_kind == VQ_GATE_CHANNEL) {
            load_weight(a.gate, i, wf, w);
#pragma unroll
            for (int j = 0; j < 4; ++j)
                y[v][j] *= w[j];
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            h[v][j] = a.skip_scale * h[v][j] + (a.y ? scale * y[v][j] : 0.0f);
            sum[0] += h[v][j] * h[v][j];
        }
        if (a.h_out)
            store4<HF>(a.h_out, t * a.h_out_stride, i, h[v]);
    }
    if (!a.x)
        return;
    block_sum<1>(sum, lds[1]);
    const float r = 1.0f / sqrtf(sum[0] * inv + a.eps);
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int i = v * nt + threadIdx.x;
        if (i >= n4)
            continue;
        float w[4];
        if (a.pre_weight)
            load_weight(a.pre_weight, i, wf, w);
#pragma unroll
        for (int j = 0; j < 4; ++j)
            h[v][j] *= a.pre_weight ? r * (w[j] + a.weight_offset) : r;
        store4<XF>(a.x, t * a.x_stride, i, h[v]);
    }
}

// Each workgroup takes every gridDim'th token and leaves its sums over them in
// the workspace, [2][hidden] per workgroup: S (or da with a gate per token),
// db.  The next token's values are on their way while one is worked on.
// WIDE: rows for more than 512 threads, whose registers leave no room for that.
template <int V, bool HF, bool YF, bool XF, bool WF, bool WIDE>
__global__ __launch_bounds__(WIDE ? kNormMaxThreads : 512, WIDE ? 4 : 3) void k_norm_grad(NormGradLaunch L)
{
    __shared__ float lds[2][3 * kNormMaxThreads / 64];
    const vq_block_norm_args &a = L.a;
    const int n4 = a.hidden / 4, nt = blockDim.x;
    const bool has_x = L.d_x != nullptr, has_y = a.y != nullptr;
    const bool channel = a.gate_kind == VQ_GATE_CHANNEL;
    const bool has_b = a.pre_weight && has_x;
    const float inv = 1.0f / (float)a.hidden;
    float s_post[V][4] = {}, s_pre[V][4] = {};
    typename Raw4<HF>::type hr[V], dr[V];
    typename Raw4<YF>::type yr[V];
    typename Raw4<XF>::type ur[V];
    typename Raw4<WF>::type pre_raw[V], post_raw[V], gate_raw[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int i = v * nt + threadIdx.x;
        pre_raw[v] = post_raw[v] = gate_raw[v] = typename Raw4<WF>::type{};
        if (i >= n4)
            continue;
        if (has_b)
            pre_raw[v] = load_raw<WF>(a.pre_weight, 0, i);
        if (a.post_weight)
            post_raw[v] = load_raw<WF>(a.post_weight, 0, i);
        if (channel)
            gate_raw[v] = load_raw<WF>(a.gate, 0, i);
    }
    // weight + offset, or 1 without the weight
    const float off_b = has_b ? a.weight_offset : 1.0f;
    const float off_p = a.post_weight ? a.weight_offset : 1.0f;
    const auto fetch = [&](int64_t t) {
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int i = v * nt + threadIdx.x;
            hr[v] = dr[v] = typename Raw4<HF>::type{};
            yr[v] = typename Raw4<YF>::type{};
            ur[v] = typename Raw4<XF>::type{};
            if (i >= n4)
                continue;
            if (has_x) {
                hr[v] = load_raw<HF>(a.h_out, t * a.h_out_stride, i);
                ur[v] = load_raw<XF>(L.d_x, t * a.x_stride, i);
            }
            if (L.d_h_out)
                dr[v] = load_raw<HF>(L.d_h_out, t * a.h_out_stride, i);
            if (has_y)
                yr[v] = load_raw<YF>(a.y, t * a.y_stride, i);
        }
    };
    if (!WIDE)
        fetch(blockIdx.x);
    for (int64_t t = blockIdx.x; t < a.n_tokens; t += gridDim.x) {
        float h[V][4], y[V][4], d[V][4], u[V][4];
        float s3[3] = {0.0f, 0.0f, 0.0f};   // h'^2, u h', y^2
        if (WIDE)
            fetch(t);
#pragma unroll
        for (int v = 0; v < V; ++v) {
            expand(hr[v], h[v]);
            expand(yr[v], y[v]);
            expand(dr[v], d[v]);
            expand(ur[v], u[v]);
        }
        if (!WIDE && t + gridDim.x < a.n_tokens)
            fetch(t + gridDim.x);
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int i = v * nt + threadIdx.x;
            if (i >= n4)
                continue;
            float b[4];
            expand(pre_raw[v], b);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                s3[0] += h[v][j] * h[v][j];
                s3[1] += (b[j] + off_b) * u[v][j] * h[v][j];
                s3[2] += y[v][j] * y[v][j];
            }
        }
        block_sum<3>(s3, lds[0]);
        const float r = has_x ? 1.0f / sqrtf(s3[0] * inv + a.eps) : 0.0f;
        const float mu = r * inv * s3[1];   // mean of u h' r
        const float q = a.post_weight ? 1.0f / sqrtf(s3[2] * inv + a.eps) : 1.0f;
        const float gt = a.gate_kind == VQ_GATE_TOKEN ? scalar_at(a.gate, t, WF) : 1.0f;
        float s2[2] = {0.0f, 0.0f};   // a g B y, B z
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int i = v * nt + threadIdx.x;
            if (i >= n4)
                continue;
            float b[4], p[4], g[4], dh[4];
            expand(pre_raw[v], b);
            expand(post_raw[v], p);
            expand(gate_raw[v], g);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float w = b[j] + off_b, po = p[j] + off_p;
                const float hn = h[v][j] * r;
                const float D = d[v][j] + r * (w * u[v][j] - hn * mu);
                s_pre[v][j] += u[v][j] * hn;
                dh[j] = a.skip_scale * D;
                const float B = a.block_scale * D, qy = q * y[v][j];
                s2[1] += po * qy * B;
                s_post[v][j] += gt * B * qy;
                d[v][j] = po * B * (channel ? g[j] : gt);
                s2[0] += d[v][j] * y[v][j];
            }
            if (L.d_h)
                store4<HF>(L.d_h, t * a.h_stride, i, dh);
        }
        // lds[1] is read before the next token's first sum lets anyone past
        block_sum<2>(s2, lds[1]);
        if (L.d_gate && a.gate_kind == VQ_GATE_TOKEN && threadIdx.x == 0)
            L.d_gate[t] = s2[1];
        if (!L.d_y)
            continue;
        const float nu = a.post_weight ? q * inv * s2[0] : 0.0f;   // mean of a g B y q
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int i = v * nt + threadIdx.x;
            if (i >= n4)
                continue;
            float dy[4];
#pragma unroll
            for (int j = 0; j < 4; ++j)
                dy[j] = q * (d[v][j] - y[v][j] * q * nu);
            store4<YF>(L.d_y, t * a.y_stride, i, dy);
        }
    }
    float *part = L.ws + (size_t)blockIdx.x * 2 * a.hidden;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int i = v * nt + threadIdx.x;
        if (i >= n4)
            continue;
        store4<true>(part, 0, i, s_post[v]);
        store4<true>(part, a.hidden, i, s_pre[v]);
    }
}

// Sums the workgroups' parts in a fixed order, 64 channels a workgroup: y = 0
// the post weight and the channel gate, y = 1 the pre weight.
constexpr int kFinishWaves = 16;

__global__ __launch_bounds__(64 * kFinishWaves) void k_norm_grad_finish(NormGradLaunch L,
                                                                        int blocks)
{
    __shared__ float lds[kFinishWaves][64];
    const vq_block_norm_args &a = L.a;
    const bool pre = blockIdx.y == 1, channel = a.gate_kind == VQ_GATE_CHANNEL;
    float *dgate = channel ? L.d_gate : nullptr;
    if (pre ? !L.d_pre_weight : !L.d_post_weight && !dgate)
        return;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, c = blockIdx.x * 64 + lane;
    constexpr int kAtOnce = 16;
    float sum = 0.0f;
    if (c < a.hidden) {
        const float *p = L.ws + (pre ? a.hidden : 0) + c;
        for (int b0 = wave; b0 < blocks; b0 += kFinishWaves * kAtOnce) {
            float v[kAtOnce];
#pragma unroll
            for (int k = 0; k < kAtOnce; ++k) {
                const int b = b0 + k * kFinishWaves;
                v[k] = b < blocks ? p[(size_t)b * 2 * a.hidden] : 0.0f;
            }
#pragma unroll
            for (int k = 0; k < kAtOnce; ++k)
                sum += v[k];
        }
    }
    lds[wave][lane] = sum;
    __syncthreads();
    if (wave != 0 || c >= a.hidden)
        return;
    sum = 0.0f;
    for (int w = 0; w < kFinishWaves; ++w)
        sum += lds[w][lane];
    const bool wf = a.weight_dtype == VQ_F32;
    if (pre) {
        L.d_pre_weight[c] = sum;
        return;
    }
    if (L.d_post_weight)
        L.d_post_weight[c] = channel ? sum * scalar_at(a.gate, c, wf) : sum;
    if (dgate)
        dgate[c] = a.post_weight ? sum * (scalar_at(a.post_weight, c, wf) + a.weight_offset) : sum;
}

// Workgroups of the backward pass: two per CU (256), which is what their
// registers leave room for (8191x2816 bf16: 71 us with 512, 93 with 256, 91 with
// 1023; rows past 4096 have room for one: 4096x16384 310 with 512, 285 with 256).
int grad_blocks(const vq_block_norm_args &a) { return std::min(a.n_tokens, 512); }

// f(groups of four values per thread, the types of h, y and x, threads) for
// workgroups of about `want` threads, more where a thread would get more than
// four groups.
template <class F>
hipError_t by_types(const vq_block_norm_args &a, int want, F &&f)
{
    using T = std::true_type;
    using N = std::false_type;
    int v = (a.hidden / 4 + want - 1) / want;
    v = v > 2 ? 4 : v;
    const int threads = ((a.hidden / 4 + v - 1) / v + 63) / 64 * 64;
    const auto with_v = [&](auto v) {
        const auto with_h = [&](auto h) {
            const auto with_y = [&](auto y) {
                return a.x_dtype == VQ_F32 ? f(v, h, y, T(), threads) : f(v, h, y, N(), threads);
            };
            return a.y_dtype == VQ_F32 ? with_y(T()) : with_y(N());
        };
        return a.h_dtype == VQ_F32 ? with_h(T()) : with_h(N());
    };
    switch (v) {
    case 1: return with_v(std::integral_constant<int, 1>());
    case 2: return with_v(std::integral_constant<int, 2>());
    default: return with_v(std::integral_constant<int, 4>());
    }
}

}  // namespace

hipError_t launch_block_norm(const vq_block_norm_args &a, hipStream_t stream)
{
    // few tokens: a row over as many threads as there are, for its latency (one
    // token of 4096: 3.5 us with 1024 threads, 4.9 with 256; 255 tokens 5.6 and
    // 7.7; 4096 tokens 52 and 46)
    return by_types(a, a.n_tokens < 256 ? kNormMaxThreads : 256,
                    [&](auto v, auto h, auto y, auto x, int threads) {
        k_norm<decltype(v)::value, decltype(h)::value, decltype(y)::value, decltype(x)::value>
            <<<a.n_tokens, threads, 0, stream>>>(a);
        return hipGetLastError();
    });
}

size_t block_norm_grad_workspace_bytes(const vq_block_norm_args &a)
{
    return (size_t)grad_blocks(a) * 2 * a.hidden * sizeof(float);
}

hipError_t launch_block_norm_grad(const NormGradLaunch &L, hipStream_t stream)
{
    const vq_block_norm_args &a = L.a;
    const int blocks = grad_blocks(a);
    if (blocks > 0) {
        const bool wide = a.hidden > 4096, wf = a.weight_dtype == VQ_F32;
        const hipError_t e = by_types(a, wide ? kNormMaxThreads : 512,
                                      [&](auto v, auto h, auto y, auto x, int threads) {
            constexpr int V = decltype(v)::value;
            constexpr bool H = decltype(h)::value, Y = decltype(y)::value, X = decltype(x)::value;
            if constexpr (V <= 2) {
                if (!wide) {
                    auto kern = wf ? k_norm_grad<V, H, Y, X, true, false>
                                   : k_norm_grad<V, H, Y, X, false, false>;
                    kern<<<blocks, threads, 0, stream>>>(L);
                    return hipGetLastError();
                }
            }
            if constexpr (V >= 2) {
                auto kern = wf ? k_norm_grad<V, H, Y, X, true, true>
                               : k_norm_grad<V, H, Y, X, false, true>;
                kern<<<blocks, threads, 0, stream>>>(L);
            }
            return hipGetLastError();
        });
        if (e != hipSuccess)
            return e;
    }
    if (!L.d_post_weight && !L.d_pre_weight &&
        !(L.d_gate && a.gate_kind == VQ_GATE_CHANNEL))
        return hipSuccess;
    k_norm_grad_finish<<<dim3((a.hidden + 63) / 64, 2), 64 * kFinishWaves, 0, stream>>>(L, blocks);
    return hipGetLastError();
}

}  // namespace vq
