// vq_q4_impl.hpp -- dense products with 4-bit weights and group scales, for up to
// 64 tokens (gfx950).
//
//   y[t][r] = sum_g ( s[r][g] sum_{c in g} q[r][c] x[t][c] + b[r][g] sum_{c in g} x[t][c] )
//
// The floor is one read of the codes and scales (HBM): one token of 65541x4096
// takes 32 us, 4.8 TB/s, 16 tokens 42, and two thousand rows the time of a
// launch and two trips to memory (2048x2048, one token: 3.2 us).  With more
// tokens, and three times over for fp32, reading x from LDS, unpacking and the
// products themselves take longer than the codes (4096x4096, 64 tokens: 14 us;
// gate and up of 8449x2816, 37 fp32 tokens: 36).  (The two sides of each rule
// below were timed in turn on one card, on weights past its 256 MB cache; from
// card to card and with the data such times differ by up to a tenth.)  The
// products run on
// the matrix cores (v_mfma_f32_16x16x32_bf16: A = 16 tokens of x, B = 16 rows
// of W), so that the vector units only turn codes into bf16, one instruction
// per weight: a code placed in the top mantissa bits of bf16 16.0 is 16 + q
// exactly, two codes per and-or.  The group sums of x that the added 16 and
// the bias need come from the same MFMA with B = 1; per group
//   y += s * sum (16 + q) x + (b - 16 s) * sum x
// in fp32.  (16 is the smallest offset that leaves four mantissa bits for the
// code; 128, with the code in the low bits, would amplify the rounding of the
// sums eight times.)  fp32 activations enter as three bf16 terms that hold
// all 24 bits.
//
// Weights reach the operand layout through LDS.  The layout gives neighbouring
// lanes neighbouring rows; loading that way asks the cache for 64 separate
// 16-byte pieces per instruction, and the address units then bound the kernel
// (65541x4096, 16 tokens: 102 us, loads prefetched four deep or not).  So a
// wave loads whole line pieces of its 16 rows into registers, writes them to
// a padded buffer of its own in LDS while the next ones are on their way, and
// reads operands from there.
#pragma once

#include <hip/hip_runtime.h>

#include <algorithm>

#include "vq_common.hpp"
#include "vq_internal.hpp"

namespace vq {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

constexpr int kQ4MaxWaves = 8;
constexpr int kQ4MaxLds = 160 << 10;

struct Q4Args {
    const uint32_t *codes[2];
    const uint16_t *scales[2];
    const uint16_t *biases[2];
    int rows, wpr, groups;   // wpr: words per row
    int nproj;
    int blocks;              // of SU units along a row
    int ks_log2;             // waves that share a row tile, splitting the blocks,
    int tail_log2;           // and in the workgroups from blockIdx.x == lead on
    int lead;
    int chunk;               // blocks of x held in LDS, a multiple of those waves
    int chunks;              // of a row
    const void *x;
    int n;                   // tokens, of which blockIdx.y takes every 16 * TT
    float *y;
    int accumulate;
};

// A unit is 128 columns, 16 words of a row: four MFMA operands ("slots") of
// four quarters (lane / 16).  Word of a slot and quarter: with groups of 128
// a lane reads 4 words at once, with 64 two and two, with 32 one by one, so
// that an operand never mixes groups.
template <int G>
__device__ __forceinline__ void place_of(int word, int &slot, int &q)
{
    if constexpr (G == 128) {
        q = word >> 2;
        slot = word & 3;
    } else if constexpr (G == 64) {
        q = (word >> 1) & 3;
        slot = (word >> 3) * 2 + (word & 1);
    } else {
        q = word & 3;
        slot = word >> 2;
    }
}

template <int G>
__device__ __forceinline__ void read_unit(const char *row, int q, uint32_t (&w)[4])
{
    if constexpr (G == 128) {
        const u32x4 v = *reinterpret_cast<const u32x4 *>(row + q * 16);
#pragma unroll
        for (int i = 0; i < 4; ++i)
            w[i] = v[i];
    } else if constexpr (G == 64) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const u32x2 v = *reinterpret_cast<const u32x2 *>(row + i * 32 + q * 8);
            w[2 * i] = v[0];
            w[2 * i + 1] = v[1];
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            w[i] = *reinterpret_cast<const uint32_t *>(row + i * 16 + q * 4);
    }
}

// Eight codes as bf16 16 + q, in the order 0 4 1 5 2 6 3 7.  mask 0x00780078
// and base 0x41804180 come in registers: as literals they would not fit one
// and-or instruction.
__device__ __forceinline__ bf16x8 unpack(uint32_t w, uint32_t mask, uint32_t base)
{
    u32x4 v;
    v[0] = ((w << 3) & mask) | base;
    v[1] = ((w >> 1) & mask) | base;
    v[2] = ((w >> 5) & mask) | base;
    v[3] = ((w >> 9) & mask) | base;
    return __builtin_bit_cast(bf16x8, v);
}

// Eight values of x: bf16 pairs (PL = 1), or fp32 to be split in three.
template <int PL>
struct XPiece {
    u32x4 v[PL == 1 ? 1 : 2];
};

// Piece i of x (at most 64 x 2^20 values: 32-bit offsets).
template <int PL>
__device__ __forceinline__ XPiece<PL> load_piece(const void *x, uint32_t i)
{
    typedef const __attribute__((address_space(1))) char *Bytes;
    typedef const __attribute__((address_space(1))) u32x4 *Ptr;
    XPiece<PL> p;
    const Ptr s = (Ptr)((Bytes)reinterpret_cast<uintptr_t>(x) + i * (PL == 1 ? 16u : 32u));
    p.v[0] = s[0];
    if constexpr (PL == 3)
        p.v[1] = s[1];
    return p;
}

// The piece in unpack()'s order as PL bf16 terms.  fp32 is cut, not rounded:
// 8 + 8 + 8 mantissa bits hold all 24, and nothing overflows.
template <int PL>
__device__ __forceinline__ void split_piece(const XPiece<PL> &p, u32x4 (&out)[PL])
{
    if constexpr (PL == 1) {
        const u32x4 d = p.v[0];
        out[0][0] = __builtin_amdgcn_perm(d[2], d[0], 0x05040100);
        out[0][1] = __builtin_amdgcn_perm(d[2], d[0], 0x07060302);
        out[0][2] = __builtin_amdgcn_perm(d[3], d[1], 0x05040100);
        out[0][3] = __builtin_amdgcn_perm(d[3], d[1], 0x07060302);
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            float a = __uint_as_float(p.v[0][j]), b = __uint_as_float(p.v[1][j]);
#pragma unroll
            for (int t = 0; t < PL; ++t) {
                const uint32_t ua = __float_as_uint(a), ub = __float_as_uint(b);
                out[t][j] = __builtin_amdgcn_perm(ub, ua, 0x07060302);
                a -= __uint_as_float(ua & 0xffff0000u);
                b -= __uint_as_float(ub & 0xffff0000u);
            }
        }
    }
}

// Scale i of the halves in v.
template <bool BF16>
__device__ __forceinline__ float scale_value(uint32_t v, int i)
{
    if constexpr (BF16)
        return __uint_as_float(i & 1 ? v & 0xffff0000u : v << 16);
    else
        return half_bits_to_float(i & 1 ? v >> 16 : v & 0xffffu);
}

// x in LDS is [PL][unit][slot][quarter][token] in 16-byte places: an odd number
// of places per token row, so that the staging writes of 16 words do not meet
// in a bank, and a constant one, so that reads have immediate offsets, where
// that wastes little (four tokens or fewer: the real count).
__host__ __device__ constexpr int q4_token_places(int TT, int NI, int n)
{
    return NI == 1 ? n | 1 : 16 * TT + 1;
}

// Per-wave LDS: the codes of TL tiles of 16 rows (rows padded by 16 bytes
// against bank conflicts), then their scales and biases.
template <int G, int SU, int TL>
struct Q4Lds {
    static constexpr int kGroups = SU * 128 / G;                 // of a block
    static constexpr int kRow = SU * 64 + 16;
    static constexpr int kScaleRow = kGroups * 2 == 32 ? 48 : kGroups * 2;
    static constexpr int kScales = TL * 16 * kRow;               // offset
    static constexpr int kBytes = (kScales + TL * 2 * 16 * kScaleRow + 15) / 16 * 16;
};

// PL: bf16 terms of an activation.  TT tiles of 16 tokens, of whose four
// accumulator registers NI are used (token t of a tile sits in register t/4,
// quarter t%4, so up to four tokens need one).  TL row tiles per wave: rows r
// and r + 16, or the same rows of gate and up.  SU units per block, the piece
// of 16 rows that a wave has in flight.  SB: bf16 scales, AF: biases.
// (Groups of 128 with two token tiles: 128 registers, so that a CU holds two
// workgroups; 64 fp32 tokens of 32768x4096: 103 us, else 113.)
template <int G, int PL, int TT, int NI, int TL, int SU, bool SB, bool AF>
__global__ __launch_bounds__(64 * kQ4MaxWaves, G == 128 && TT == 2 && TL == 1 ? 4 : 2) void k_q4(Q4Args a)
{
    using S = Q4Lds<G, SU, TL>;
    constexpr int NG = 128 / G;        // groups of a unit
    constexpr bool kEarly = NI == 4;   // the first x before the first codes (below)
    extern __shared__ __attribute__((aligned(16))) u32x4 lds[];
    // the workgroup's tokens
    const int t0 = blockIdx.y * 16 * TT, n = min(a.n - t0, 16 * TT);
    const void *x = static_cast<const char *>(a.x) + (int64_t)t0 * a.wpr * (PL == 1 ? 16 : 32);
    float *out = a.y + (int64_t)t0 * a.rows;
    const int lane = threadIdx.x & 63, waves = blockDim.x >> 6;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int q = lane >> 4, col = lane & 15;
    const int np = q4_token_places(TT, NI, n), cu = a.chunk * SU;
    char *mine = reinterpret_cast<char *>(lds) + wave * S::kBytes;
    u32x4 *xa = lds + waves * S::kBytes / 16;
    const bool tail = (int)blockIdx.x >= a.lead;
    const int ks_log2 = tail ? a.tail_log2 : a.ks_log2;
    const int ks = wave & ((1 << ks_log2) - 1), rg = wave >> ks_log2;
    const bool pair = a.nproj == 2;
    const int tile_rows = pair ? 16 : 16 * TL;
    const int first_tile = tail ? a.lead * (waves >> a.ks_log2) +
                                      (blockIdx.x - a.lead) * (waves >> ks_log2)
                                : blockIdx.x * (waves >> ks_log2);
    const int r0 = (first_tile + rg) * tile_rows;
    if (first_tile * tile_rows >= a.rows)
        return;   // a column that fills up the grid: the whole workgroup

    // what the lane loads: 16 bytes of row load_row + i * (16 / SU), i < SU;
    // PB bytes of the scales (lower lanes) or biases of one row
    constexpr int kPerRow = 4 * SU, kRowStep = 16 / SU;
    const int load_row = lane / kPerRow, piece = lane % kPerRow;
    constexpr int PB = S::kGroups * 2 < 16 ? S::kGroups * 2 : 16, PPR = S::kGroups * 2 / PB;
    const int s_kind = lane / (16 * PPR), s_row = lane / PPR % 16, s_part = lane % PPR;
    const bool s_live = lane < (AF ? 32 : 16) * PPR;
    const uint32_t *cp[TL][SU];
    const uint16_t *sp[TL];
#pragma unroll
    for (int l = 0; l < TL; ++l) {
        const int m = pair ? l : 0, first = r0 + (pair ? 0 : 16 * l);
#pragma unroll
        for (int i = 0; i < SU; ++i)
            cp[l][i] = a.codes[m] +
                       (int64_t)min(first + load_row + i * kRowStep, a.rows - 1) * a.wpr;
        sp[l] = (AF && s_kind ? a.biases[m] : a.scales[m]) +
                (int64_t)min(first + s_row, a.rows - 1) * a.groups;
    }

    u32x4 w[TL][SU];
    uint32_t sc[TL][(PB + 3) / 4];
    const auto load_block = [&](int blk) {
        // past the row's end its last piece again, against zeros in x
        const int word = min(blk * SU * 16 + piece * 4, a.wpr - 4);
        const int g0 = blk * S::kGroups + s_part * (PB / 2);
#pragma unroll
        for (int l = 0; l < TL; ++l)
#pragma unroll
            for (int i = 0; i < SU; ++i)
                w[l][i] = __builtin_nontemporal_load(
                    (const __attribute__((address_space(1))) u32x4 *)(cp[l][i] + word));
        if (!s_live)
            return;
#pragma unroll
        for (int l = 0; l < TL; ++l) {
            if ((blk + 1) * S::kGroups <= a.groups) {
                // rows of an odd number of groups start between dwords
                if constexpr (PB == 2) {
                    sc[l][0] = load_global(sp[l] + g0);
                } else {
                    typedef uint32_t Raw __attribute__((ext_vector_type(PB / 4), aligned(2)));
                    const Raw r = *(const __attribute__((address_space(1))) Raw *)(sp[l] + g0);
#pragma unroll
                    for (int i = 0; i < PB / 4; ++i)
                        sc[l][i] = r[i];
                }
            } else {
#pragma unroll
                for (int i = 0; i < PB / 2; i += 2) {
                    const uint32_t lo = g0 + i < a.groups ? load_global(sp[l] + g0 + i) : 0u;
                    const uint32_t hi = PB > 2 && g0 + i + 1 < a.groups
                                            ? load_global(sp[l] + g0 + i + 1) : 0u;
                    sc[l][i / 2] = lo | hi << 16;
                }
            }
        }
    };
    const auto store_block = [&]() {
#pragma unroll
        for (int l = 0; l < TL; ++l) {
#pragma unroll
            for (int i = 0; i < SU; ++i)
                *reinterpret_cast<u32x4 *>(mine + (l * 16 + load_row + i * kRowStep) * S::kRow +
                                           piece * 16) = w[l][i];
            if (s_live) {
                char *d = mine + S::kScales + ((l * 2 + s_kind) * 16 + s_row) * S::kScaleRow +
                          s_part * PB;
                if constexpr (PB == 2)
                    *reinterpret_cast<uint16_t *>(d) = (uint16_t)sc[l][0];
                else
#pragma unroll
                    for (int i = 0; i < PB / 4; ++i)
                        reinterpret_cast<uint32_t *>(d)[i] = sc[l][i];
            }
        }
    };

    // lane's A rows: MFMA row col holds token (col % 4) * 4 + col / 4 of a tile
    int tok[TT];
#pragma unroll
    for (int tt = 0; tt < TT; ++tt)
        tok[tt] = min(16 * tt + (col & 3) * 4 + (col >> 2), n - 1);
    const char *my_codes = mine + col * S::kRow, *my_scales = mine + S::kScales +
                                                              col * S::kScaleRow;
    float tot[TL][TT][NI] = {};
    uint32_t mask = 0x00780078u, base = 0x41804180u;
    asm("" : "+s"(mask));
    asm("" : "+v"(base));

    // x is staged in pieces of 8 columns of a token, XB per thread in flight.
    // Piece i is word i % cw of token i / cw (cw words a chunk, a multiple of
    // 16 as is the number of threads: a thread's place in a unit is fixed).
    constexpr int XB = 4;
    const int cw = cu * 16, nt = blockDim.x;
    const int step_t = nt / cw, step_w = nt - step_t * cw;
    const int first_t = threadIdx.x / cw, first_w = threadIdx.x - first_t * cw;
    int slot0, q0;
    place_of<G>(threadIdx.x & 15, slot0, q0);
    const int place0 = slot0 * 4 + q0;

    // blocks of this wave: ks, ks + step, ... of each chunk
    const bf16x8 ones = __builtin_bit_cast(
        bf16x8, u32x4{0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u});
    const int step = 1 << ks_log2;
    // pieces on their way, from token t and word w of a chunk
    XPiece<PL> px[XB];
    const auto advance = [&](int &t, int &w) {
        t += step_t;
        w += step_w;
        if (w >= cw) {
            w -= cw;
            ++t;
        }
    };
    const auto fetch_x = [&](int c, int t, int w) {
#pragma unroll
        for (int k = 0; k < XB; ++k) {
            px[k] = load_piece<PL>(x, (uint32_t)min(t, n - 1) * a.wpr +
                                          min(c * cw + w, a.wpr - 1));
            advance(t, w);
        }
    };
    const auto put_x = [&](int c, int &t, int &w) {
#pragma unroll
        for (int k = 0; k < XB; ++k) {
            if (t >= n)
                break;
            u32x4 v[PL];
            split_piece<PL>(px[k], v);
#pragma unroll
            for (int pl = 0; pl < PL; ++pl)
                xa[((pl * cu + (w >> 4)) * 16 + place0) * np + t] =
                    c * cw + w < a.wpr ? v[pl] : u32x4{0, 0, 0, 0};
            advance(t, w);
        }
    };
    const auto stage_x = [&](int c) {   // after fetch_x
        int t = first_t, w = first_w;
        put_x(c, t, w);
        while (t < n) {
            fetch_x(c, t, w);
            put_x(c, t, w);
        }
    };
    // the wave's own LDS writes, before other lanes' reads of them and after
    const auto wave_sync = [] {
        __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
        __builtin_amdgcn_wave_barrier();
        __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
    };
    const auto multiply = [&](int kb) {   // the block in LDS, block kb of the chunk
        wave_sync();
#pragma unroll
        for (int su = 0; su < SU; ++su) {
            const int uc = kb * SU + su;   // the unit's place in the chunk
            uint32_t ww[TL][4], sw[TL][(NG + 1) / 2], bw[TL][(NG + 1) / 2];
#pragma unroll
            for (int l = 0; l < TL; ++l) {
                read_unit<G>(my_codes + l * 16 * S::kRow + su * 64, q, ww[l]);
                const char *s = my_scales + l * 2 * 16 * S::kScaleRow + su * NG * 2;
                if constexpr (NG == 1) {
                    sw[l][0] = *reinterpret_cast<const uint16_t *>(s);
                    if (AF)
                        bw[l][0] =
                            *reinterpret_cast<const uint16_t *>(s + 16 * S::kScaleRow);
                } else {
#pragma unroll
                    for (int i = 0; i < NG / 2; ++i) {
                        sw[l][i] = reinterpret_cast<const uint32_t *>(s)[i];
                        if (AF)
                            bw[l][i] =
                                reinterpret_cast<const uint32_t *>(s + 16 * S::kScaleRow)[i];
                    }
                }
            }
#pragma unroll
            for (int g = 0; g < NG; ++g) {
                // The lower terms of x are summed first: next to the sums of the highest
                // one each of their steps would round as much as it adds (error of 640
                // columns in groups of 128: 2.4e-7, else 1.4e-6).  That keeps a group's
                // unpacked codes in registers; with few tokens, whose x is read ahead
                // into them, lower sums apart cost less (one token of 65536x4096: groups
                // of 64 49 us, else 63, of 128 50 and 60; of 32, one operand a group, 50
                // and 51).
                f32x4 acc[TL][TT] = {}, xs[TT] = {};
                const auto step_of = [&](int pl, int m, const bf16x8 (&wv)[TL],
                                         f32x4 (&to)[TL][TT], f32x4 (&xt)[TT]) {
                    const int slot = g * (4 / NG) + m;
#pragma unroll
                    for (int tt = 0; tt < TT; ++tt) {
                        const bf16x8 av = __builtin_bit_cast(
                            bf16x8, xa[((pl * cu + uc) * 16 + slot * 4 + q) * np + tok[tt]]);
                        xt[tt] =
                            __builtin_amdgcn_mfma_f32_16x16x32_bf16(av, ones, xt[tt], 0, 0, 0);
#pragma unroll
                        for (int l = 0; l < TL; ++l)
                            to[l][tt] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                                av, wv[l], to[l][tt], 0, 0, 0);
                    }
                };
                bf16x8 wv[4 / NG][TL];
                const auto unpack_slot = [&](int m) {
#pragma unroll
                    for (int l = 0; l < TL; ++l)
                        wv[m][l] = unpack(ww[l][g * (4 / NG) + m], mask, base);
                };
                if constexpr (PL > 1 && NI == 1 && G > 32) {
                    f32x4 low[TL][TT] = {}, xl[TT] = {};
#pragma unroll
                    for (int m = 0; m < 4 / NG; ++m) {
                        unpack_slot(m);
                        step_of(0, m, wv[m], acc, xs);
#pragma unroll
                        for (int pl = 1; pl < PL; ++pl)
                            step_of(pl, m, wv[m], low, xl);
                    }
#pragma unroll
                    for (int tt = 0; tt < TT; ++tt)
#pragma unroll
                        for (int i = 0; i < NI; ++i) {
                            xs[tt][i] += xl[tt][i];
#pragma unroll
                            for (int l = 0; l < TL; ++l)
                                acc[l][tt][i] += low[l][tt][i];
                        }
                } else {
#pragma unroll
                    for (int pl = PL - 1; pl >= 0; --pl)
#pragma unroll
                        for (int m = 0; m < 4 / NG; ++m) {
                            if (pl == PL - 1)
                                unpack_slot(m);
                            step_of(pl, m, wv[m], acc, xs);
                        }
                }
                float sv[TL], cv[TL];
#pragma unroll
                for (int l = 0; l < TL; ++l) {
                    sv[l] = scale_value<SB>(sw[l][g / 2], g);
                    cv[l] = AF ? fmaf(-16.0f, sv[l], scale_value<SB>(bw[l][g / 2], g))
                               : -24.0f * sv[l];
                }
#pragma unroll
                for (int tt = 0; tt < TT; ++tt)
#pragma unroll
                    for (int i = 0; i < NI; ++i)
#pragma unroll
                        for (int l = 0; l < TL; ++l)
                            tot[l][tt][i] = fmaf(sv[l], acc[l][tt][i],
                                                 fmaf(cv[l], xs[tt][i], tot[l][tt][i]));
            }
        }
        wave_sync();
    };

    // Loads return in order.  For more than four tokens x goes before the codes,
    // so that its staging does not wait for them (16 fp32 tokens, gate and up of
    // 2048x4096: 13.5 us, else 14.2; in bf16 this order costs 3 %: 10.0 and 9.7,
    // 4096x4096 8.0 and 7.7); for fewer, whose x is soon there, after them (one
    // token of 2048x2048: 3.6 us, else 3.9).
    if constexpr (kEarly) {
        fetch_x(0, first_t, first_w);
        load_block(ks);
        stage_x(0);
        __syncthreads();
    } else {
        load_block(ks);
    }
    for (int c = 0; c < a.chunks; ++c) {
        if (!kEarly || c) {
            if (c)
                __syncthreads();
            if constexpr (kEarly) {
                fetch_x(c, first_t, first_w);
                stage_x(c);
            } else {
                for (int t = first_t, w = first_w; t < n;) {
                    int t1 = t, w1 = w;
                    fetch_x(c, t, w);
                    put_x(c, t1, w1);
                    t = t1;
                    w = w1;
                }
            }
            __syncthreads();
        }
        for (int kb = ks; kb < a.chunk; kb += step) {
            const int blk = c * a.chunk + kb;
            if (blk >= a.blocks)
                break;
            store_block();
            if (blk + step < a.blocks)
                load_block(blk + step);
            multiply(kb);
        }
    }

    // y[t][r] of tile l from its sums v (both tiles' in a pair)
    const auto store = [&](int first, int t, const float (&v)[TL]) {
        if (t >= n)
            return;
        float *y = out + (int64_t)t * a.rows;
        if (pair) {
            if (first + col < a.rows)
                y[first + col] = silu_mul(v[0], v[TL - 1]);
            return;
        }
#pragma unroll
        for (int l = 0; l < TL; ++l) {
            const int r = first + 16 * l + col;
            if (r < a.rows)
                y[r] = a.accumulate ? y[r] + v[l] : v[l];
        }
    };
    constexpr int R = TT * NI;
    if (!ks_log2) {
#pragma unroll
        for (int k = 0; k < R; ++k) {
            float v[TL];
#pragma unroll
            for (int l = 0; l < TL; ++l)
                v[l] = tot[l][k / NI][k % NI];
            store(r0, 16 * (k / NI) + (k % NI) * 4 + q, v);
        }
        return;
    }
    // join the waves that split the blocks, in their order
    float *red = reinterpret_cast<float *>(lds);   // [wave][l][k][lane]
    __syncthreads();
#pragma unroll
    for (int l = 0; l < TL; ++l)
#pragma unroll
        for (int k = 0; k < R; ++k)
            red[((wave * TL + l) * R + k) * 64 + lane] = tot[l][k / NI][k % NI];
    __syncthreads();
    for (int k = ks; k < R; k += step) {
        float v[TL] = {};
        for (int i = 0; i < step; ++i)
#pragma unroll
            for (int l = 0; l < TL; ++l)
                v[l] += red[((((rg << ks_log2) + i) * TL + l) * R + k) * 64 + lane];
        store(r0, 16 * (k / NI) + (k % NI) * 4 + q, v);
    }
}

inline Q4Args q4_args(const Q4Launch &L)
{
    Q4Args a = {};
    for (int m = 0; m < L.nproj; ++m) {
        a.codes[m] = L.t[m].codes;
        a.scales[m] = static_cast<const uint16_t *>(L.t[m].scales);
        a.biases[m] = static_cast<const uint16_t *>(L.t[m].biases);
    }
    a.rows = L.t[0].rows;
    a.wpr = L.t[0].cols / 8;
    a.groups = L.t[0].cols / L.t[0].group;
    a.nproj = L.nproj;
    a.x = L.x;
    a.n = L.n;
    a.y = L.y;
    a.accumulate = L.accumulate;
    return a;
}

// LDS to join the sums of a workgroup's waves, `regs` a lane.
constexpr int q4_join_bytes(int waves, int regs)
{
    return waves * regs * 64 * 4;
}

// Sets the chunks of a launch with 1 << ks waves per tile: as much of x at a
// time as fits in `lds` bytes.  Returns the bytes, or 0.
template <int G, int PL, int TT, int NI, int TL, int SU>
int q4_fit(Q4Args &a, int ks, int waves, int lds)
{
    using S = Q4Lds<G, SU, TL>;
    const int step = 1 << ks, codes = waves * S::kBytes;
    const int block = SU * PL * 16 * q4_token_places(TT, NI, a.n) * 16;   // NI == 1: n <= 4
    a.ks_log2 = ks;
    a.chunk = std::min(std::max(lds - codes, 0) / block / step * step,
                       (a.blocks + step - 1) / step * step);
    if (a.chunk == 0)
        return 0;
    a.chunks = (a.blocks + a.chunk - 1) / a.chunk;
    return std::max(codes + a.chunk * block, ks ? q4_join_bytes(waves, TL * TT * NI) : 0);
}

template <int G, int PL, int TT, int NI, int TL, int SU, bool SB, bool AF>
hipError_t q4_launch(const Q4Launch &L, hipStream_t stream)
{
    Q4Args a = q4_args(L);
    const int units = (a.wpr + 15) / 16;
    a.blocks = (units + SU - 1) / SU;
    const int tile_rows = L.nproj == 2 ? 16 : 16 * TL;
    const int tiles = (a.rows + tile_rows - 1) / tile_rows;
    const int groups = (L.n + 16 * TT - 1) / (16 * TT);   // of tokens
    // Waves per tile, which split a row: as many as keep the chip at eight waves
    // per CU, a workgroup of eight sharing one staging of x (16 tokens of 4096
    // columns, 512 tiles: 10.4 us with four, 14.5 with eight; 4097 tiles: 45.8
    // with one, 49.9 with two; four tokens, 4096 tiles: 32.8 with one, 38.9 with
    // four).  One token, whose x is small: eight, or four where the tiles alone
    // fill the chip (512 tiles: 6.8 us with eight, 7.4 with four; 1024: 11.4 and
    // 10.2; 4097: 42.9 and 33.7).
    int ks = 3;
    if (L.n == 1)
        ks = tiles > 1024 ? 2 : 3;
    else
        while (ks > 0 && ((int64_t)tiles * groups) << ks > 256 * kQ4MaxWaves)
            --ks;
    while (1 << ks > a.blocks)
        --ks;
    const int waves = L.n == 1 ? std::max(4, 1 << ks) : kQ4MaxWaves;
    // half a CU's LDS if that holds a block of x per wave of a tile, else all
    int bytes = 0;
    for (; !bytes; --ks) {
        bytes = q4_fit<G, PL, TT, NI, TL, SU>(a, ks, waves, kQ4MaxLds / 2);
        if (!bytes)
            bytes = q4_fit<G, PL, TT, NI, TL, SU>(a, ks, waves, kQ4MaxLds);
    }
    const int per_wg = waves >> a.ks_log2;
    int columns = (tiles + per_wg - 1) / per_wg;
    a.lead = columns;
    // Work in whole waves per tile ends with a round that leaves CUs idle: of
    // its workgroups, where they fill half the CUs or less (or half of what
    // runs on them at once, two of half a CU's LDS), each is spread over more
    // waves per tile (16 tokens of 4096 columns, 32784 rows: 24.4 us, else 28.9;
    // 65541 rows: 42.2 and 46.4; gate and up of 40000 rows: 49 and 63).
    const int total = columns * groups;
    for (int slots = 256; slots <= (bytes > kQ4MaxLds / 2 ? 256 : 512); slots *= 2) {
        const int last = total % slots;
        if (a.ks_log2 || per_wg < 2 || total <= slots || !last || 2 * last > slots ||
            a.chunk < 2)
            continue;
        int t = 1;
        while (2 << t <= per_wg && last << (t + 1) <= slots && a.chunk >= 2 << t)
            ++t;
        a.tail_log2 = t;
        a.chunk = a.chunk >> t << t;
        a.chunks = (a.blocks + a.chunk - 1) / a.chunk;
        a.lead -= (last + groups - 1) / groups;
        const int rest = tiles - a.lead * per_wg;
        columns = a.lead + (rest + (per_wg >> t) - 1) / (per_wg >> t);
        bytes = std::max(bytes, q4_join_bytes(waves, TL * TT * NI));
        break;
    }
    const auto kern = k_q4<G, PL, TT, NI, TL, SU, SB, AF>;
    if (bytes > 65536) {
        const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void *>(kern),
                                                 hipFuncAttributeMaxDynamicSharedMemorySize,
                                                 bytes);
        if (e != hipSuccess)
            return e;
    }
    // Several groups of tokens: the columns of the grid are made a multiple of
    // the eight XCDs, so that one XCD's L2 serves all groups of a tile's codes
    // (8449x2816 gate and up, 37 fp32 tokens: 37.9 us, else 41.2).
    const dim3 grid(groups > 1 ? (columns + 7) / 8 * 8 : columns, groups);
    kern<<<grid, 64 * waves, bytes, stream>>>(a);
    return hipGetLastError();
}

template <int G, int PL, bool SB, bool AF>
hipError_t q4_by_tokens(const Q4Launch &L, hipStream_t stream)
{
    // Token tiles run as workgroups of their own, which read the codes again,
    // from L2 for the most part, until they fill the chip; then a wave takes two
    // (64 tokens of 4096 columns, 4096 rows: 13.6 us as single tiles, 14.3 in
    // twos; 8192 rows 18.9 and 19.7, 16384 rows 33.8 and 32.3, 32768 rows 70 and
    // 58).  fp32, with three times the products per code, later (8192 rows: 32
    // us as single tiles, 36 in twos; 16384 rows 59 and 65; 32768 rows 116 and
    // 103).
    //
    // Blocks of four units (512 columns) where there are many tiles, of two
    // where few waves must share the latency (16 tokens, 65541 rows: 43.3 us
    // with four, 45.5 with two; 4096 rows: 9.6 and 7.9; gate and up of 32768
    // rows: 39 and 43, of 1024: 12.5 and 9.9).  For fp32, whose x takes the
    // LDS, half of that (65541 rows: 79 us with two, 83 with one; 4096 rows:
    // 13.9 and 12.2).  Up to four tokens in the paired form, which has twice the
    // codes in flight: two (8192 rows, one token: 10.4 us, 14.2 with four; four
    // tokens: 10.7 and 11.9).
    //
    // Two row tiles per wave in the paired form only: they halve the reads of x
    // and cost as much in occupancy.
    const bool pair = L.nproj == 2;
    const int64_t jobs = (int64_t)((L.t[0].rows + 15) / 16) * ((L.n + 15) / 16);
    const bool many = jobs > (PL == 1 ? 1024 : 512);
    constexpr int kBig = PL == 1 ? 4 : 2, kSmall = PL == 1 ? 2 : 1;
    if (L.n <= 4)
        return pair   ? q4_launch<G, PL, 1, 1, 2, 2, SB, AF>(L, stream)
               : many ? q4_launch<G, PL, 1, 1, 1, 4, SB, AF>(L, stream)
                      : q4_launch<G, PL, 1, 1, 1, 2, SB, AF>(L, stream);
    if (L.n > 16 && jobs > (PL == 1 ? 1024 : 2048))
        return pair ? q4_launch<G, PL, 2, 4, 2, 2, SB, AF>(L, stream)
                    : q4_launch<G, PL, 2, 4, 1, 2, SB, AF>(L, stream);
    if (many)
        return pair ? q4_launch<G, PL, 1, 4, 2, kBig, SB, AF>(L, stream)
                    : q4_launch<G, PL, 1, 4, 1, kBig, SB, AF>(L, stream);
    return pair ? q4_launch<G, PL, 1, 4, 2, kSmall, SB, AF>(L, stream)
                : q4_launch<G, PL, 1, 4, 1, kSmall, SB, AF>(L, stream);
}

template <int G, int PL>
hipError_t q4_by_scales(const Q4Launch &L, hipStream_t stream)
{
    const bool affine = L.t[0].biases != nullptr;
    if (L.t[0].scale_bf16)
        return affine ? q4_by_tokens<G, PL, true, true>(L, stream)
                      : q4_by_tokens<G, PL, true, false>(L, stream);
    return affine ? q4_by_tokens<G, PL, false, true>(L, stream)
                  : q4_by_tokens<G, PL, false, false>(L, stream);
}

// One group size (the translation units instantiate it).
template <int G>
hipError_t q4_group(const Q4Launch &L, hipStream_t stream)
{
    return L.x_f32 ? q4_by_scales<G, 3>(L, stream) : q4_by_scales<G, 1>(L, stream);
}

}  // namespace vq
