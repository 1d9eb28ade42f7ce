// MX4 operators: the row quantiser and the grouped product of routed rows with MX4 expert weights.
//
// Product: rows r of group g (offsets[g] <= r < offsets[g + 1]) give
//     out[r] = act(W[g] x[src(r)]),   src(r) = perm[r] / k,   or r without a permutation,
// with W[g] of N rows by K columns.  Two kernels:
//  - product_mx4_kernel: x in MX4 too.  E2M1 x E2M1 with both block scales applied inside
//    v_mfma_scale_f32_16x16x128_f8f6f4; for batches of rows.
//  - product_wide_kernel: x in bf16 or fp32, entering exactly; weights widened to bf16; for few
//    rows per group, where streaming the weights is all that counts.
#include <hip/hip_runtime.h>

#include "moe_launch.hpp"
#include "mx4_dev.hpp"

namespace moe {
namespace {

// ---------------------------------------------------------------------------------------------
// Quantiser.  Blocks of 32 lie one after another in memory whatever the row, so the matrix is cut
// into pieces of 8 values: a lane loads one, the block's largest magnitude is exchanged within
// four lanes, and each lane writes its 4 bytes of codes.  Bound by memory.

template <typename XT, bool VALUES>
__global__ __launch_bounds__(256) void quantize_mx4_kernel(const XT *__restrict__ v, long long pieces,
                                                           uint32_t *__restrict__ q, uint8_t *__restrict__ scale,
                                                           XT *__restrict__ values)
{
    const long long i = (long long)blockIdx.x * 256 + threadIdx.x;
    if (i >= pieces) return;             // pieces is a multiple of 4: whole blocks leave together
    float f[8];
    if constexpr (sizeof(XT) == 2) {
        const uint4 u = *reinterpret_cast<const uint4 *>(v + i * 8);
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            f[2 * j] = __uint_as_float(w[j] << 16);
            f[2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
        }
    } else {
        const float4 a = *reinterpret_cast<const float4 *>(v + i * 8);
        const float4 b = *reinterpret_cast<const float4 *>(v + i * 8 + 4);
        f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
        f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
    }
    // magnitudes compare as their bits (a NaN's are the largest)
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) m = max(m, __float_as_uint(f[j]) & 0x7FFFFFFFu);
    m = max(m, dpp_u32<0xB1>(m));
    m = max(m, dpp_u32<0x4E>(m));
    const uint32_t s = mx4_scale(m);
    const float sf = e8m0_f32(s);
    const uint32_t codes = s == MX_NAN ? 0u : mx4_codes8(f, sf);
    q[i] = codes;
    if ((i & 3) == 0) scale[i >> 2] = (uint8_t)s;
    if constexpr (VALUES) {
        if constexpr (sizeof(XT) == 2) {
            U4 o;
            o.v = mx4_bf16x8(codes, sf);
            if (s == MX_NAN) o.w[0] = o.w[1] = o.w[2] = o.w[3] = 0x7FC07FC0u;
            *reinterpret_cast<uint4 *>(values + i * 8) = o.u;
        } else {
            float o[8];
            const f32x2v p0 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, sf, 0);
            const f32x2v p1 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, sf, 1);
            const f32x2v p2 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, sf, 2);
            const f32x2v p3 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, sf, 3);
            o[0] = p0[0]; o[1] = p0[1]; o[2] = p1[0]; o[3] = p1[1];
            o[4] = p2[0]; o[5] = p2[1]; o[6] = p3[0]; o[7] = p3[1];
            if (s == MX_NAN) {
#pragma unroll
                for (int j = 0; j < 8; ++j) o[j] = __uint_as_float(0x7FC00000u);
            }
            *reinterpret_cast<float4 *>(values + i * 8) = make_float4(o[0], o[1], o[2], o[3]);
            *reinterpret_cast<float4 *>(values + i * 8 + 4) = make_float4(o[4], o[5], o[6], o[7]);
        }
    }
}

// ---------------------------------------------------------------------------------------------
// Groups.  The offsets live on the device, so a block finds its rows itself: one wave holds the
// groups' row counts, 64 per register, and scans them.

struct Tile {
    int g, row0, rows;      // group, first row, rows (0: no such tile)
};

__device__ __forceinline__ int wave_scan_incl(int v, int lane)
{
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const int t = __shfl_up(v, o, WAVE);
        v += lane >= o ? t : 0;
    }
    return v;
}

// Tile number `tile` when every group's rows are cut into tiles of `bm`.  Offsets are clamped into
// [0, Pr] and taken as ascending, so no value of theirs leads outside the rows.
__device__ __forceinline__ Tile find_tile(const Mx4Product &p, int tile, int bm, int lane)
{
    if (p.offsets == nullptr) {
        const int r0 = tile * bm;
        return Tile{0, r0, min(bm, p.Pr - r0)};
    }
    const int G = p.E + p.S;
    int before = 0;
    for (int c = 0; c < G; c += 64) {
        const int g = c + lane;
        int lo = 0, hi = 0;
        if (g < p.E) {
            lo = min(max(p.offsets[g], 0), p.Pr);
            hi = min(max(p.offsets[g + 1], lo), p.Pr);
        } else if (g < G) {
            lo = p.Pr + (g - p.E) * p.T;
            hi = lo + p.T;
        }
        const int nt = (hi - lo + bm - 1) / bm;
        const int incl = wave_scan_incl(nt, lane);
        const unsigned long long m = __ballot(before + incl > tile);
        if (m) {
            const int at = __ffsll((long long)m) - 1;
            const int t = tile - before - __shfl(incl - nt, at, WAVE);
            const int glo = __shfl(lo, at, WAVE), ghi = __shfl(hi, at, WAVE);
            return Tile{c + at, glo + t * bm, min(bm, ghi - glo - t * bm)};
        }
        before += __shfl(incl, 63, WAVE);
    }
    return Tile{0, 0, 0};
}

__device__ __forceinline__ int source_row(const Mx4Product &p, int r)
{
    if (p.perm == nullptr) return min(r, p.rows_x - 1);
    const int pair = p.perm[r];
    return min(max(p.k == 1 ? pair : pair / p.k, 0), p.rows_x - 1);
}

__device__ __forceinline__ float activate(float v, int act)
{
    const float r = fmaxf(v, 0.f);
    // a NaN stays one (fmaxf drops it)
    return act == ACT_RELU2 ? (v != v ? v : r * r) : v;
}

__device__ __forceinline__ void store1(const Mx4Product &p, size_t at, float v)
{
    if (p.otype == X_F32) static_cast<float *>(p.out)[at] = v;
    else static_cast<uint16_t *>(p.out)[at] = __builtin_bit_cast(uint16_t, (__bf16)v);
}

// four consecutive outputs from n0 on, of which those below N exist
__device__ __forceinline__ void store4(const Mx4Product &p, int row, int n0, int NO, const float (&v)[4])
{
    const size_t at = (size_t)row * NO + n0;
    if ((NO & 3) == 0) {
        if (n0 >= NO) return;
        if (p.otype == X_F32) {
            *reinterpret_cast<float4 *>(static_cast<float *>(p.out) + at) = make_float4(v[0], v[1], v[2], v[3]);
        } else {
            const bf16x2v a = {(__bf16)v[0], (__bf16)v[1]}, b = {(__bf16)v[2], (__bf16)v[3]};
            *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(p.out) + at) =
                make_uint2(__builtin_bit_cast(uint32_t, a), __builtin_bit_cast(uint32_t, b));
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (n0 + i < NO) store1(p, at + i, v[i]);
}

// ---------------------------------------------------------------------------------------------
// Product of MX4 rows.  A block of 4 waves computes BM = 128 rows by BN = 256 weight rows (128 gate
// rows and their 128 up rows with SwiGLU); wave w owns 64 of the weight rows and all 128 rows.
// Weights are the A operand (their rows become 4 consecutive outputs of a lane), x the B operand.
// Weights go from global memory into registers (no other wave wants them); x goes through LDS.

constexpr int PB_M = 128, PB_N = 256, PB_KS = 256;     // rows, weight rows, K of an LDS stage

__device__ __forceinline__ void lds_dma16(const void *g, uint32_t lds)
{
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off"
                 :: "s"(__builtin_amdgcn_readfirstlane(lds)), "v"(g) : "memory", "m0");
}
template <typename T>
__device__ __forceinline__ uint32_t lds_addr(T *p)
{
    return (uint32_t)(uintptr_t)(__attribute__((address_space(3))) void *)p;
}

__device__ __forceinline__ i32x8v code_reg(const uint4 &v)
{
    return i32x8v{(int)v.x, (int)v.y, (int)v.z, (int)v.w, 0, 0, 0, 0};
}

// One K step's weights of a wave: 4 fragments of 16 rows by 128 columns.
struct WStep {
    uint4 c[4];
    uint32_t s[4];       // this lane's scale code in the low byte
};

// MG: 32-row groups of the tile that hold rows.
template <int MG>
__device__ __forceinline__ void product_tile(const Mx4Product &p, const Tile &t, int nt, uint8_t *lds)
{
    constexpr int MF = 2 * MG;           // 16-row fragments
    const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63, li = lane & 15, lg = lane >> 4;
    const bool glu = p.act == ACT_SWIGLU;
    const int F = p.N >> 1, NO = glu ? F : p.N;
    const int KB = p.K >> 1, KSC = p.K >> 5;              // bytes of codes, of scales per row
    const int steps = (p.K + 127) >> 7, stages = (p.K + PB_KS - 1) / PB_KS;
    const bool half = (p.K & 127) != 0;                   // the last step holds 64 columns
    uint8_t *xsc = lds + 2 * PB_M * (PB_KS / 2);          // x scales: [step][lane][fragment]

    // ---- x scales of the tile, transposed so that a lane reads all fragments' in one go
    for (int i = tid; i < 16 * (KSC >> 1); i += 256) {
        const int r = i & 15, pr = i >> 4;                // row within a fragment, pair of blocks
        uint32_t b[8];
#pragma unroll
        for (int f = 0; f < 8; ++f) {
            b[f] = 0;
            if (f < MF) {
                const int row = min(16 * f + r, t.rows - 1);
                b[f] = *reinterpret_cast<const uint16_t *>(p.xs + (size_t)source_row(p, t.row0 + row) * KSC + 2 * pr);
            }
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            uint32_t w[2];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                w[j] = 0;
#pragma unroll
                for (int f = 0; f < 4; ++f) w[j] |= ((b[4 * j + f] >> (8 * h)) & 0xFFu) << (8 * f);
            }
            const int kb = 2 * pr + h;                    // = 4 step + lane group
            *reinterpret_cast<uint2 *>(xsc + (size_t)(kb >> 2) * 512 + (kb & 3) * 128 + r * 8) = make_uint2(w[0], w[1]);
        }
    }
    if (half && tid < 32)                                 // the missing blocks' scales: 1
        *reinterpret_cast<uint2 *>(xsc + (size_t)(steps - 1) * 512 + 256 + tid * 8) = make_uint2(0x7F7F7F7Fu, 0x7F7F7F7Fu);

    // ---- x codes: an LDS stage holds 128 bytes of every row, chunk c of row r at c ^ ((r >> 1) & 7)
    const uint8_t *xp[MG];
    int xc[MG];
#pragma unroll
    for (int i = 0; i < MG; ++i) {
        const int slot = (i * 4 + wave) * 64 + lane, r = slot >> 3;
        xp[i] = static_cast<const uint8_t *>(p.x) + (size_t)source_row(p, t.row0 + min(r, t.rows - 1)) * KB;
        xc[i] = 16 * ((slot & 7) ^ ((r >> 1) & 7));
    }
    auto issue = [&](int st) {
        const uint32_t L = lds_addr(lds + (st & 1) * PB_M * (PB_KS / 2));
#pragma unroll
        for (int i = 0; i < MG; ++i)
            lds_dma16(xp[i] + min(st * (PB_KS / 2) + xc[i], KB - 16), L + (i * 4 + wave) * 1024);
    };

    // ---- weights
    const uint8_t *wp[4], *sp[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        int n;
        if (glu) {
            const int f = min(nt * 128 + wave * 32 + 16 * (j & 1) + li, F - 1);
            n = j < 2 ? f : F + f;
        } else {
            n = min(nt * 256 + wave * 64 + 16 * j + li, p.N - 1);
        }
        const size_t row = (size_t)t.g * p.N + n;
        wp[j] = p.w + row * KB + 16 * lg;
        sp[j] = p.ws + row * KSC + lg;
    }
    const bool live = (glu ? nt * 128 + wave * 32 : nt * 256 + wave * 64) < NO;
    auto wload = [&](WStep &w, int s) {
        const bool in = live && s < steps && !(half && s == steps - 1 && lg >= 2);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            w.c[j] = make_uint4(0, 0, 0, 0);
            w.s[j] = 127;
            if (in) {
                w.c[j] = *reinterpret_cast<const uint4 *>(wp[j] + (size_t)s * 64);
                w.s[j] = sp[j][s * 4];
            }
        }
    };

    f32x4 acc[4][MF];
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int f = 0; f < MF; ++f) acc[j][f] = zero4();

    auto step = [&](const WStep &w, int s) {
        const uint8_t *L = lds + ((s >> 1) & 1) * PB_M * (PB_KS / 2);
        const uint2 xs = *reinterpret_cast<const uint2 *>(xsc + (size_t)s * 512 + lane * 8);
        i32x8v a[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) a[j] = code_reg(w.c[j]);
#pragma unroll
        for (int f = 0; f < MF; ++f) {
            const int r = 16 * f + li, c = 4 * (s & 1) + lg;
            const i32x8v b = code_reg(*reinterpret_cast<const uint4 *>(L + r * 128 + 16 * (c ^ ((r >> 1) & 7))));
            const uint32_t xsf = f < 4 ? xs.x : xs.y;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                switch (f & 3) {                          // the scale's byte is part of the instruction
                case 0: acc[j][f] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a[j], b, acc[j][f], 4, 4, 0, (int)w.s[j], 0, (int)xsf); break;
                case 1: acc[j][f] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a[j], b, acc[j][f], 4, 4, 0, (int)w.s[j], 1, (int)xsf); break;
                case 2: acc[j][f] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a[j], b, acc[j][f], 4, 4, 0, (int)w.s[j], 2, (int)xsf); break;
                default: acc[j][f] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a[j], b, acc[j][f], 4, 4, 0, (int)w.s[j], 3, (int)xsf); break;
                }
            }
        }
    };

    issue(0);
    WStep w0, w1;
    wload(w0, 0);
    for (int st = 0; st < stages; ++st) {
        // this stage's loads have landed in every wave, and every wave has left the other buffer
        asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
        if (st + 1 < stages) issue(st + 1);
        wload(w1, 2 * st + 1);
        step(w0, 2 * st);
        wload(w0, 2 * st + 2);
        if (2 * st + 1 < steps) step(w1, 2 * st + 1);
    }

    // ---- epilogue: lane l, element i of acc[j][f] is output 16 j + 4 (l / 16) + i of row 16 f + l % 16
    if (!live) return;
#pragma unroll
    for (int f = 0; f < MF; ++f) {
        const int r = 16 * f + li;
        float v[4][4];
#pragma unroll
        for (int j = 0; j < (glu ? 2 : 4); ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i) v[j][i] = glu ? silu_f32(acc[j][f][i]) * acc[j + 2 > 3 ? 3 : j + 2][f][i] : activate(acc[j][f][i], p.act);
        const int nfr = glu ? 2 : 4, n0 = glu ? nt * 128 + wave * 32 : nt * 256 + wave * 64;
        if (p.otype == X_MX4) {
            // two fragments are one block of 32 outputs, spread over the four lanes of a row
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                if (2 * b >= nfr) break;
                float u[8];
                uint32_t m = 0;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    u[i] = v[2 * b + (i >> 2)][i & 3];
                    m = max(m, __float_as_uint(u[i]) & 0x7FFFFFFFu);
                }
                m = max(m, xor_lane_u32(m, 16, lane));
                m = max(m, xor_lane_u32(m, 32, lane));
                const uint32_t s = mx4_scale(m);
                const uint32_t q = s == MX_NAN ? 0u : mx4_codes8(u, e8m0_f32(s));
                const int nb = n0 + 32 * b;
                if (r < t.rows && nb < NO) {
                    uint8_t *o = static_cast<uint8_t *>(p.out) + (size_t)(t.row0 + r) * (NO >> 1) + (nb >> 1) + 2 * lg;
                    *reinterpret_cast<uint16_t *>(o) = (uint16_t)q;
                    *reinterpret_cast<uint16_t *>(o + 8) = (uint16_t)(q >> 16);
                    if (lg == 0) p.out_scales[(size_t)(t.row0 + r) * (NO >> 5) + (nb >> 5)] = (uint8_t)s;
                }
            }
        } else if (r < t.rows) {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (j < nfr) store4(p, t.row0 + r, n0 + 16 * j + 4 * lg, NO, v[j]);
        }
    }
}

__global__ __launch_bounds__(256, 2) void product_mx4_kernel(Mx4Product p, int ntiles)
{
    extern __shared__ __attribute__((aligned(16))) uint8_t mx4_lds[];
    const int b = blockIdx.x, mt = b / ntiles, nt = b - mt * ntiles;
    const Tile t = find_tile(p, mt, PB_M, threadIdx.x & 63);
    if (t.rows < 1) return;
    switch ((t.rows + 31) >> 5) {
    case 1: product_tile<1>(p, t, nt, mx4_lds); break;
    case 2: product_tile<2>(p, t, nt, mx4_lds); break;
    case 3: product_tile<3>(p, t, nt, mx4_lds); break;
    default: product_tile<4>(p, t, nt, mx4_lds); break;
    }
}

// ---------------------------------------------------------------------------------------------
// Product of bf16 / fp32 rows with MX4 weights.  A block owns TN 16-row weight tiles (with SwiGLU
// TN / 2 gate tiles and their up tiles) of one group; its waves split K and the partial sums meet
// in LDS in wave order.  Weights widen to bf16 exactly; an fp32 x is cut into three bf16 terms
// whose sum is x, so every product is exact and the sums are fp32.

template <int XK>
struct XTerms {
    static constexpr int N = XK == X_F32 ? 3 : 1;
};

// eight fp32 values as three bf16 terms by truncation: 8 + 8 + 8 significand bits
__device__ __forceinline__ void cut_f32x8(const float *v, bf16x8 (&terms)[3])
{
    U4 a, b, c;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float r[2], s[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const float x = v[2 * i + h];
            r[h] = x - __uint_as_float(__float_as_uint(x) & 0xFFFF0000u);
            s[h] = r[h] - __uint_as_float(__float_as_uint(r[h]) & 0xFFFF0000u);
        }
        a.w[i] = pack_bf16_exact(v[2 * i], v[2 * i + 1]);        // the upper halves
        b.w[i] = pack_bf16_exact(r[0], r[1]);
        c.w[i] = pack_bf16_exact(s[0], s[1]);
    }
    terms[0] = a.v;
    terms[1] = b.v;
    terms[2] = c.v;
}

template <int XK, int TN, int MT, int NW>
__global__ __launch_bounds__(64 * NW) void product_wide_kernel(Mx4Product p)
{
    constexpr int NTERM = XTerms<XK>::N;
    __shared__ float red[NW][TN * 256];
    const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63, li = lane & 15, lg = lane >> 4;
    const Tile t = find_tile(p, blockIdx.y, 1 << 30, lane);
    if (t.rows < 1) return;
    const bool glu = p.act == ACT_SWIGLU;
    const int F = p.N >> 1, NO = glu ? F : p.N;
    const int TO = glu ? TN / 2 : TN;                      // output tiles
    const int KB = p.K >> 1, KSC = p.K >> 5, steps = (p.K + 127) >> 7;
    const int n0 = blockIdx.x * TO * 16;

    const uint8_t *wp[TN], *sp[TN];
#pragma unroll
    for (int j = 0; j < TN; ++j) {
        int n;
        if (glu) {
            const int f = min(n0 + 16 * (j % (TN / 2)) + li, F - 1);
            n = j < TN / 2 ? f : F + f;
        } else {
            n = min(n0 + 16 * j + li, p.N - 1);
        }
        const size_t row = (size_t)t.g * p.N + n;
        wp[j] = p.w + row * KB + 16 * lg;
        sp[j] = p.ws + row * KSC + lg;
    }

    for (int r0 = 0; r0 < t.rows; r0 += 16 * MT) {
        f32x4 acc[TN][MT];
        const uint8_t *xp[MT];
        bool in[MT];
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            const int r = r0 + 16 * m + li;
            in[m] = r < t.rows;
            const size_t src = source_row(p, t.row0 + min(r, t.rows - 1));
            xp[m] = static_cast<const uint8_t *>(p.x) + (src * p.K + 32 * lg) * (XK == X_F32 ? 4 : 2);
#pragma unroll
            for (int j = 0; j < TN; ++j) acc[j][m] = zero4();
        }
        for (int s = wave; s < steps; s += NW) {
            const bool kin = 128 * s + 32 * lg < p.K;
            uint4 w[TN];
            float sc[TN];
#pragma unroll
            for (int j = 0; j < TN; ++j) {
                w[j] = make_uint4(0, 0, 0, 0);
                uint32_t sb = 127;
                if (kin) {
                    w[j] = *reinterpret_cast<const uint4 *>(wp[j] + (size_t)s * 64);
                    sb = sp[j][s * 4];
                }
                sc[j] = e8m0_f32(sb);
            }
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                if (MT > 1 && r0 + 16 * m >= t.rows) break;
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    bf16x8 xt[NTERM];
                    if constexpr (XK == X_F32) {
                        float v[8] = {};
                        if (in[m] && kin) {
                            const float4 *g = reinterpret_cast<const float4 *>(xp[m] + ((size_t)s * 128 + 8 * q) * 4);
                            const float4 a = g[0], b = g[1];
                            v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
                            v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
                        }
                        cut_f32x8(v, xt);
                    } else {
                        U4 u;
                        u.u = make_uint4(0, 0, 0, 0);
                        if (in[m] && kin) u.u = *reinterpret_cast<const uint4 *>(xp[m] + ((size_t)s * 128 + 8 * q) * 2);
                        xt[0] = u.v;
                    }
#pragma unroll
                    for (int j = 0; j < TN; ++j) {
                        const uint32_t c = q == 0 ? w[j].x : q == 1 ? w[j].y : q == 2 ? w[j].z : w[j].w;
                        const bf16x8 wb = mx4_bf16x8(c, sc[j]);
#pragma unroll
                        for (int k = NTERM - 1; k >= 0; --k) acc[j][m] = mfma16x16x32_bf16(wb, xt[k], acc[j][m]);
                    }
                }
            }
        }
        // ---- the waves' sums, then the activation; element i of a lane is weight row 4 lg + i of x row li
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            if (r0 + 16 * m >= t.rows) break;
            __syncthreads();
#pragma unroll
            for (int j = 0; j < TN; ++j)
                *reinterpret_cast<f32x4 *>(&red[wave][j * 256 + li * 16 + 4 * lg]) = acc[j][m];
            __syncthreads();
            for (int i = tid; i < TO * 256; i += 64 * NW) {
                const int n = i % (16 * TO), r = i / (16 * TO);
                const int at = (n >> 4) * 256 + r * 16 + (n & 15);
                float v = 0.f, u = 0.f;
#pragma unroll
                for (int k = 0; k < NW; ++k) {
                    v += red[k][at];
                    if (glu) u += red[k][at + (TN / 2) * 256];
                }
                if (r0 + 16 * m + r < t.rows && n0 + n < NO)
                    store1(p, (size_t)(t.row0 + r0 + 16 * m + r) * NO + n0 + n, glu ? silu_f32(v) * u : activate(v, p.act));
            }
        }
    }
}

template <int XK, int TN>
hipError_t launch_wide(const Mx4Product &p, hipStream_t s)
{
    constexpr int NW = 4;
    const int TO = p.act == ACT_SWIGLU ? TN / 2 : TN;
    const int NO = p.act == ACT_SWIGLU ? p.N / 2 : p.N;
    const int rows = p.Pr + p.S * p.T;
    const int G = p.offsets ? p.E + p.S : 1;
    const dim3 grid((NO + 16 * TO - 1) / (16 * TO), rows < G ? rows : G);
    if (rows <= 16) product_wide_kernel<XK, TN, 1, NW><<<grid, 64 * NW, 0, s>>>(p);
    else product_wide_kernel<XK, TN, 4, NW><<<grid, 64 * NW, 0, s>>>(p);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_quantize_mx4(const void *v, int xtype, int rows, int cols, uint8_t *q, uint8_t *scale, void *values,
                               hipStream_t s)
{
    ProfScope prof(K_QUANT, s);
    const long long pieces = (long long)rows * cols / 8;
    const unsigned blocks = (unsigned)((pieces + 255) / 256);
    uint32_t *q4 = reinterpret_cast<uint32_t *>(q);
    if (xtype == X_BF16) {
        const uint16_t *x = static_cast<const uint16_t *>(v);
        uint16_t *o = static_cast<uint16_t *>(values);
        if (values) quantize_mx4_kernel<uint16_t, true><<<blocks, 256, 0, s>>>(x, pieces, q4, scale, o);
        else quantize_mx4_kernel<uint16_t, false><<<blocks, 256, 0, s>>>(x, pieces, q4, scale, o);
    } else {
        const float *x = static_cast<const float *>(v);
        float *o = static_cast<float *>(values);
        if (values) quantize_mx4_kernel<float, true><<<blocks, 256, 0, s>>>(x, pieces, q4, scale, o);
        else quantize_mx4_kernel<float, false><<<blocks, 256, 0, s>>>(x, pieces, q4, scale, o);
    }
    return hipGetLastError();
}

hipError_t launch_product_mx4(const Mx4Product &p, hipStream_t s)
{
    ProfScope prof(K_PRODUCT_MX4, s);
    if (p.xtype == X_F32) return launch_wide<X_F32, 4>(p, s);
    if (p.xtype == X_BF16) return launch_wide<X_BF16, 2>(p, s);
    const int NO = p.act == ACT_SWIGLU ? p.N / 2 : p.N;
    const int per = p.act == ACT_SWIGLU ? PB_N / 2 : PB_N;
    const int ntiles = (NO + per - 1) / per;
    const int rows = p.Pr + p.S * p.T, G = p.offsets ? p.E + p.S : 1;
    const int mtiles = rows / PB_M + (rows < G ? rows : G);        // at least the sum of the groups' tiles
    const int lds = 2 * PB_M * (PB_KS / 2) + 512 * ((p.K + 127) / 128);
    if (lds > 64 * 1024) {
        const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void *>(product_mx4_kernel),
                                                 hipFuncAttributeMaxDynamicSharedMemorySize, lds);
        if (e != hipSuccess) return e;
    }
    product_mx4_kernel<<<(unsigned)mtiles * ntiles, 256, lds, s>>>(p, ntiles);
    return hipGetLastError();
}

}  // namespace moe
