// MX4 operators: the row quantiser and the grouped product of routed rows with MX4 expert weights.
//
// Product: rows r of group g (offsets[g] <= r < offsets[g + 1]) give
//     out[r] = act(W[g] x[src(r)]),   src(r) = perm[r] / k,   or r without a permutation,
// with W[g] of N rows by K columns.  Two kernels:
//  - product_mx4_kernel: x in MX4 too.  E2M1 x E2M1 with both block scales applied inside
//    v_mfma_scale_f32_32x32x64_f8f6f4; for batches of rows.
//  - product_wide_kernel: x in bf16 or fp32, entering exactly; weights widened to bf16; for few
//    rows per group, where streaming the weights is all that counts.
#include <hip/hip_runtime.h>

#include <type_traits>

#include "moe_launch.hpp"
#include "mx4_dev.hpp"

namespace moe {
namespace {

// ---------------------------------------------------------------------------------------------
// Quantiser.  Blocks of 32 lie one after another in memory whatever the row, so the matrix is cut
// into pieces of 8 values: a lane loads one, the block's largest magnitude is exchanged within
// four lanes, and each lane writes its 4 bytes of codes.  Bound by memory: 16384 x 704 fp32 with the
// values 16.5 us, 98 MB at 5.9 TB/s (a copy of the same device reaches 4.65); a single row 1.3 us, a
// launch.  Two or four pieces a thread changed nothing.

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
// Groups.  The offsets live on the device, so every wave finds its block's rows itself: lane l holds
// groups 8 l .. 8 l + 7, which three loads fetch, and one scan over the lanes numbers the tiles.  The
// S shared groups follow the E routed ones and need no loads.

struct Tile {
    int g, row0, rows;      // group, first row, rows (0: no such tile)
};

constexpr int GPL = 8;      // groups per lane
static_assert(GPL * WAVE >= MAX_E, "a wave holds every group");

// Offsets are clamped into [0, Pr] and taken as ascending, so no value of theirs leads outside the rows.
__device__ __forceinline__ void load_groups(const Mx4Product &p, int lane, int (&lo)[GPL], int (&hi)[GPL])
{
    const int g0 = GPL * lane;
    int o[GPL + 1] = {};
    if (g0 + GPL <= p.E) {
        const int4 a = *reinterpret_cast<const int4 *>(p.offsets + g0), b = *reinterpret_cast<const int4 *>(p.offsets + g0 + 4);
        o[0] = a.x; o[1] = a.y; o[2] = a.z; o[3] = a.w;
        o[4] = b.x; o[5] = b.y; o[6] = b.z; o[7] = b.w;
        o[8] = p.offsets[g0 + 8];
    } else if (g0 < p.E) {
#pragma unroll
        for (int i = 0; i <= GPL; ++i) o[i] = p.offsets[min(g0 + i, p.E)];
    }
#pragma unroll
    for (int i = 0; i < GPL; ++i) {
        lo[i] = min(max(o[i], 0), p.Pr);
        hi[i] = min(max(o[i + 1], lo[i]), p.Pr);
    }
}

// inclusive sum over the lanes up to this one
__device__ __forceinline__ int wave_scan_incl(int v)
{
    // within rows of 16 lanes by DPP row shifts, then the rows' ends onto the rows behind them
    v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xF, 0xF, false);
    v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xF, 0xF, false);
    v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xF, 0xF, false);
    v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xF, 0xF, false);
    v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xA, 0xF, false);
    v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xC, 0xF, false);
    return v;
}

// The tiles of all groups when each group's rows are cut into tiles of `bm`: their number, and tile
// `tile` (a negative one: none).
struct Tiling {
    int lo[GPL], hi[GPL], nt, incl, routed, total;
    __device__ __forceinline__ Tiling(const Mx4Product &p, int bm, int lane)
    {
        load_groups(p, lane, lo, hi);
        nt = 0;
#pragma unroll
        for (int i = 0; i < GPL; ++i) nt += (hi[i] - lo[i] + bm - 1) / bm;
        incl = wave_scan_incl(nt);
        routed = __builtin_amdgcn_readlane(incl, 63);
        total = routed + p.S * ((p.T + bm - 1) / bm);
    }
    __device__ __forceinline__ Tile find(const Mx4Product &p, int bm, int tile) const
    {
        if (tile < 0 || tile >= total) return Tile{0, 0, 0};
        if (tile >= routed) {
            const int per = (p.T + bm - 1) / bm, s = (tile - routed) / per, r = (tile - routed - s * per) * bm;
            return Tile{p.E + s, p.Pr + s * p.T + r, min(bm, p.T - r)};
        }
        const int at = __ffsll((long long)__ballot(incl > tile)) - 1;      // the lane that holds it
        int left = tile - __builtin_amdgcn_readlane(incl - nt, at), g = 0, l = 0, h = 0;
        bool open = true;
#pragma unroll
        for (int i = 0; i < GPL; ++i) {
            const int a = __builtin_amdgcn_readlane(lo[i], at), b = __builtin_amdgcn_readlane(hi[i], at), n = (b - a + bm - 1) / bm;
            if (open && left < n) {
                g = i;
                l = a;
                h = b;
                open = false;
            }
            if (open) left -= n;
        }
        return Tile{GPL * at + g, l + left * bm, min(bm, h - l - left * bm)};
    }
};

// Block b's tile when every group's rows are cut into tiles of `bm` and the weight rows into
// `ntiles`.  Blocks go to the 8 XCDs in turn, so each XCD takes a contiguous eighth of the tiles,
// weight tiles running fastest: the row tiles of one group, which read the same weights, and the
// weight tiles of one row tile, which read the same rows, meet in one L2.
__device__ __forceinline__ Tile find_tile(const Mx4Product &p, int b, int bm, int ntiles, int lane, int &nt)
{
    const auto mine = [&](int total) {
        const long long live = (long long)total * ntiles;
        const int x = b & 7, j0 = (int)(live * x / 8), j = j0 + (b >> 3);
        const bool in = j < (int)(live * (x + 1) / 8);
        // columns of 8 weight tiles, one after another
        const int c = total > 0 ? j / (8 * total) : 0, w = max(1, min(8, ntiles - 8 * c)), r = j - 8 * c * total;
        const int tile = r / w;
        nt = 8 * c + r - tile * w;
        return in ? tile : -1;
    };
    if (p.offsets == nullptr) {
        const int tile = mine((p.Pr + bm - 1) / bm);
        return tile < 0 ? Tile{0, 0, 0} : Tile{0, tile * bm, min(bm, p.Pr - tile * bm)};
    }
    const Tiling q(p, bm, lane);
    return q.find(p, bm, mine(q.total));
}

// Tile `tile` of all groups' rows cut into tiles of `bm`.
__device__ __forceinline__ Tile find_rows(const Mx4Product &p, int tile, int bm, int lane)
{
    if (p.offsets == nullptr) return Tile{0, tile * bm, min(bm, p.Pr - tile * bm)};
    return Tiling(p, bm, lane).find(p, bm, tile);
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

// silu(g) = g / (1 + 2^(-g log2 e)).  The exponent is split in two floats, so its rounding does not
// grow with |g|; exp and reciprocal instructions are good to 1 ulp.
__device__ __forceinline__ float silu_fast(float g)
{
    const float x = __builtin_amdgcn_fmed3f(-g, -88.5f, 88.5f);      // 2^127.7: sums and products stay finite
    const float hi = x * 1.44269504f, lo = fmaf(x, 1.44269504f, -hi) + x * 1.9259630e-8f;
    const float e = __builtin_amdgcn_exp2f(hi);
    return g * __builtin_amdgcn_rcpf(1.f + fmaf(e, lo * 0.69314718f, e));
}

template <int OT>
__device__ __forceinline__ void store1(const Mx4Product &p, size_t at, float v)
{
    if (OT == X_F32) static_cast<float *>(p.out)[at] = v;
    else static_cast<uint16_t *>(p.out)[at] = __builtin_bit_cast(uint16_t, (__bf16)v);
}

// four consecutive outputs from column n on, at element `at`; those below NO exist
__device__ __forceinline__ void store4(const Mx4Product &p, size_t at, int n, int NO, const float (&v)[4])
{
    if (NO & 3) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (n + i < NO) {
                if (p.otype == X_F32) store1<X_F32>(p, at + i, v[i]);
                else store1<X_BF16>(p, at + i, v[i]);
            }
    } else if (n < NO) {
        if (p.otype == X_F32) {
            *reinterpret_cast<float4 *>(static_cast<float *>(p.out) + at) = make_float4(v[0], v[1], v[2], v[3]);
        } else {
            typedef __bf16 b4 __attribute__((ext_vector_type(4)));
            const b4 o = {(__bf16)v[0], (__bf16)v[1], (__bf16)v[2], (__bf16)v[3]};
            *reinterpret_cast<b4 *>(static_cast<uint16_t *>(p.out) + at) = o;
        }
    }
}

// ---------------------------------------------------------------------------------------------
// Product of MX4 rows.  A block of 4 waves computes up to 160 rows by 256 weight rows (128 gate rows
// and their 128 up rows with SwiGLU); wave w owns 64 of the weight rows and all the rows.  Weights are
// the A operand (their rows become 4 consecutive outputs of a lane), x the B operand.
//
// An MFMA lane holds one row's 16 bytes, so neighbouring lanes hold different rows: loaded straight
// into registers, every lane would be a cache access of its own (64 per KB; gate/up of 2048 tokens 206
// us that way).  Both operands therefore go through LDS by direct-to-LDS loads whose neighbouring
// lanes read neighbouring bytes, in stages of 128 columns.  E2M1 products run at twice the rate in the
// 32x32x64 form (measured 9.1 PFLOP/s on registers alone) than in the 16x16x128 one (4.8).
//
// Measured: gate/up of 2048 tokens top-8 of 128 experts (1408 x 2816) 96 us, 2.8 TB/s of weights and
// 1.35 PFLOP/s; their down projection (2816 x 704, fp32 out) 99 us, half of it the 185 MB of results
// and a third a block's way to its first product; 4096 x 6144 x 6144 112 us, 2.8 PFLOP/s.  A copy
// without loads ran the first in 69 and the last in 84 us: what is left is latency at a block's start
// and the operands' way from L2 (about 17 bytes a cycle and CU), which the two blocks of a CU hide in
// part.  Tried and slower: 128 weight rows (162 / 233 / 164 us), four such blocks a CU (200 / 272 /
// 205), stages through registers (123 / 112 / 133 against 112 / 106 / 130 then).

constexpr int PB_M = 160, PB_N = 256;                  // rows, weight rows of a block
constexpr int PB_XST = PB_M * 64, PB_WST = PB_N * 64;  // bytes of a stage's codes (128 columns)
constexpr int PB_XBUF = 2, PB_WBUF = 3;                // weights come from HBM, rows mostly from L2
constexpr int PB_WLOADS = 4;                           // load instructions of a wave per weight stage
constexpr int PB_SST = 8 * (PB_M + PB_N);              // 8 scales (256 columns) of every row
constexpr int PB_LDS = PB_WBUF * PB_WST + PB_XBUF * PB_XST + 2 * PB_SST;

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

// Orders LDS between the waves of a block; unlike __syncthreads() it leaves global loads in flight.
__device__ __forceinline__ void lds_barrier() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

__device__ __forceinline__ i32x8v code_reg(const uint4 &v)
{
    return i32x8v{(int)v.x, (int)v.y, (int)v.z, (int)v.w, 0, 0, 0, 0};
}

// Where a stage keeps 16-byte chunk c of row r (64-byte rows): the 16 rows that the 16 lanes of a
// fragment read at once fall on different banks.
__device__ __forceinline__ int chunk64_at(int r, int c) { return r * 64 + 16 * (c ^ ((r >> 2) & 3)); }

// Scales 16 q .. 16 q + 15 of a row (`row`: its scales, n in all), 1 for those past the end.  Rows of
// scales start at even addresses only.
__device__ __forceinline__ uint4 scales16(const uint8_t *row, int q, int n)
{
    uint4 v;
    if (16 * q + 16 <= n) {
        __builtin_memcpy(&v, __builtin_assume_aligned(row + 16 * q, 2), 16);
        return v;
    }
    uint32_t h[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) h[i] = *reinterpret_cast<const uint16_t *>(row + min(16 * q + 2 * i, n - 2));
#pragma unroll
    for (int i = 0; i < 8; ++i) h[i] = 16 * q + 2 * i < n ? h[i] : 0x7F7Fu;
    return make_uint4(h[0] | (h[1] << 16), h[2] | (h[3] << 16), h[4] | (h[5] << 16), h[6] | (h[7] << 16));
}

// Codes of columns past K: E2M1 zeros.
__device__ const uint4 mx4_zeros = {0, 0, 0, 0};

// MG: 32-row groups of the tile that hold rows.
template <bool GLU, int OT, int MG>
__device__ __forceinline__ void product_tile(const Mx4Product &p, const Tile &t, int nt, uint8_t *lds)
{
    const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63, li = lane & 31, lh = lane >> 5;
    const int F = p.N >> 1, NO = GLU ? F : p.N;
    const int KB = p.K >> 1, KSC = p.K >> 5;              // bytes of codes, of scales per row
    const int steps = (p.K + 127) >> 7;                   // the last one may hold 64 columns

    // weight row that row r of the block's 256 stands for: wave w's 64 rows are 32 gate and their 32
    // up rows with SwiGLU
    auto weight_row = [&](int r) {
        int n = nt * 256 + r;
        if (GLU) n = min(nt * 128 + (r >> 6) * 32 + (r & 31), F - 1) + ((r & 32) ? F : 0);
        return (size_t)t.g * p.N + min(n, p.N - 1);
    };
    constexpr int WO = GLU ? 32 : 64;                     // a wave's outputs of a row
    const int n0 = (nt * 4 + wave) * WO;
    const bool live = n0 < NO;

    // ---- sources: 4 lanes read a row's 64 bytes; instruction i of a wave fills 16 rows.  Rows past the
    // tile's or the matrix's end read the last one, so that every wave issues the same loads.
    constexpr int XI = (MG + 1) / 2;                      // x code instructions of a wave
    const uint8_t *wsrc[4], *xsrc[XI];
    const int drow = lane >> 2, dchunk = 16 * ((lane & 3) ^ ((lane >> 4) & 3));   // (row >> 2) & 3 of row = lane / 4
    auto x_row = [&](int r) { return (size_t)source_row(p, t.row0 + min(r, t.rows - 1)); };
#pragma unroll
    for (int i = 0; i < 4; ++i) wsrc[i] = p.w + weight_row(64 * wave + 16 * i + drow) * KB;
    uint8_t *xlds = lds + PB_WBUF * PB_WST, *slds = xlds + PB_XBUF * PB_XST;
    auto issue_w = [&](int s, int buf) {
        const uint32_t L = lds_addr(lds + buf * PB_WST);
        const int off = min(s, steps - 1) * 64 + dchunk;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            lds_dma16(off < KB ? wsrc[i] + off : reinterpret_cast<const uint8_t *>(&mx4_zeros), L + (4 * wave + i) * 1024);
    };
    auto issue_x = [&](int s) {
        const uint32_t L = lds_addr(xlds + (s & 1) * PB_XST);
        const int off = min(s * 64 + dchunk, KB - 16);
#pragma unroll
        for (int i = 0; i < XI; ++i)
            if (wave + 4 * i < 2 * MG) lds_dma16(xsrc[i] + off, L + (wave + 4 * i) * 1024);
    };
    // the weights need only the group: they are on their way while the rows' places are looked up
    issue_w(0, 0);
    issue_w(1, 1);
    // thread r: the scales of weight row r and (the first 160) of row r
    const uint8_t *wsc = p.ws + weight_row(tid) * KSC;
    uint4 sw = scales16(wsc, 0, KSC);
#pragma unroll
    for (int i = 0; i < XI; ++i) xsrc[i] = static_cast<const uint8_t *>(p.x) + x_row(16 * (wave + 4 * i) + drow) * KB;
    issue_x(0);
    const uint8_t *xsc = p.xs + x_row(min(tid, PB_M - 1)) * KSC;
    uint4 sx = scales16(xsc, 0, KSC);
    // columns 256 q ..: two steps' scales of every row
    auto put_scales = [&](int q, uint32_t w0, uint32_t w1, uint32_t x0, uint32_t x1) {
        uint2 *S = reinterpret_cast<uint2 *>(slds + (q & 1) * PB_SST);
        S[tid] = make_uint2(w0, w1);
        if (tid < PB_M) S[PB_N + tid] = make_uint2(x0, x1);
    };

    f32x16v acc[2][MG];
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int f = 0; f < MG; ++f)
#pragma unroll
            for (int i = 0; i < 16; ++i) acc[j][f][i] = 0.f;

    // A lane holds half a row's 64 columns, blocks 2 u + lh of the step: with the row's scales shifted by
    // its half, byte 2 u is the one.
    auto step = [&](int s, int buf) {
        const uint8_t *X = xlds + (s & 1) * PB_XST, *W = lds + buf * PB_WST + wave * 4096;
        const uint32_t *S = reinterpret_cast<const uint32_t *>(slds + ((s >> 1) & 1) * PB_SST) + (s & 1) + 2 * li;
        const uint32_t *WS = S + 128 * wave, *XS = S + 2 * PB_N;
        int sa[2], sb[MG];
#pragma unroll
        for (int j = 0; j < 2; ++j) sa[j] = (int)(WS[64 * j] >> (8 * lh));
#pragma unroll
        for (int f = 0; f < MG; ++f) sb[f] = (int)(XS[64 * f] >> (8 * lh));
        i32x8v a[2][2], b[2][MG];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
#pragma unroll
            for (int j = 0; j < 2; ++j) a[u][j] = code_reg(*reinterpret_cast<const uint4 *>(W + chunk64_at(32 * j + li, 2 * u + lh)));
#pragma unroll
            for (int f = 0; f < MG; ++f) b[u][f] = code_reg(*reinterpret_cast<const uint4 *>(X + chunk64_at(32 * f + li, 2 * u + lh)));
        }
#pragma unroll
        for (int f = 0; f < MG; ++f)
#pragma unroll
            for (int j = 0; j < 2; ++j)
                acc[j][f] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(a[0][j], b[0][f], acc[j][f], 4, 4, 0, sa[j], 0, sb[f]);
#pragma unroll
        for (int f = 0; f < MG; ++f)
#pragma unroll
            for (int j = 0; j < 2; ++j)
                acc[j][f] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(a[1][j], b[1][f], acc[j][f], 4, 4, 2, sa[j], 2, sb[f]);
    };

    // Weights are asked for two steps ahead, x one step ahead.  At the top of step s the newest
    // loads in flight are the weights of step s + 1; everything older has to be there.  Every step
    // issues the same number of weight loads (past the end the last step's again), so the count
    // holds.  Scales go through registers, four steps' of a row at a time, and from there into LDS two
    // steps' at a time, into the buffer that is not being read.
    put_scales(0, sw.x, sw.y, sx.x, sx.y);
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    int buf = 0;
    for (int s = 0; s < steps; ++s) {
        // stage s has landed in every wave, and every wave has left the buffers filled next
        asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(PB_WLOADS) : "memory");
        const int q = (s >> 1) + 1;                       // the next two steps
        if ((s & 3) == 1 && s + 1 < steps) {
            put_scales(q, sw.z, sw.w, sx.z, sx.w);
            if (s + 3 < steps) {
                sw = scales16(wsc, (s >> 2) + 1, KSC);
                sx = scales16(xsc, (s >> 2) + 1, KSC);
            }
        }
        if (s + 1 < steps) issue_x(s + 1);
        issue_w(s + 2, buf == 0 ? 2 : buf - 1);
        if (live) step(s, buf);
        if ((s & 3) == 3 && s + 1 < steps) put_scales(q, sw.x, sw.y, sx.x, sx.y);
        buf = buf == 2 ? 0 : buf + 1;
    }
    // no load may still be writing LDS, and every wave is done reading it
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
    if (!live) return;

    // ---- epilogue: lane l, element i of acc[j][f] is output 32 j + 8 (i / 4) + 4 (l / 32) + i % 4 of row
    // 32 f + l % 32.  Each fragment's 32 rows turn round in the wave's own part of LDS, so that
    // neighbouring lanes store neighbouring outputs of a row; fp32 and bf16 results with the
    // non-temporal hint, so that they do not push operands out of L2 that other blocks read again (185
    // MB of fp32 results 105 -> 99 us, 50 MB of bf16 115 -> 112 us).
    constexpr int RS = WO + 4;
    float *T = reinterpret_cast<float *>(lds) + wave * 32 * (64 + 4);
    const bool whole = NO % (OT == X_F32 ? 4 : 8) == 0;
#pragma unroll
    for (int f = 0; f < MG; ++f) {
#pragma unroll
        for (int j = 0; j < (GLU ? 1 : 2); ++j)
#pragma unroll
            for (int i = 0; i < 16; i += 4) {
                f32x4 v;
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    v[k] = GLU ? silu_fast(acc[0][f][i + k]) * acc[1][f][i + k] : activate(acc[j][f][i + k], p.act);
                *reinterpret_cast<f32x4 *>(T + li * RS + 32 * j + 2 * i + 4 * lh) = v;
            }
        __builtin_amdgcn_wave_barrier();
        const int r0 = t.row0 + 32 * f, rn = t.rows - 32 * f;
        if (OT != X_MX4 && !whole) {
#pragma unroll 1
            for (int i = lane; i < 32 * WO; i += 64) {
                const int r = i / WO, n = i & (WO - 1);
                if (r < rn && n0 + n < NO) store1<OT>(p, (size_t)(r0 + r) * NO + n0 + n, T[r * RS + n]);
            }
        } else if (OT == X_F32) {
#pragma unroll
            for (int i = 0; i < 32 * WO / 4; i += 64) {
                const int r = (i + lane) / (WO / 4), n = 4 * ((i + lane) & (WO / 4 - 1));
                const f32x4 v = *reinterpret_cast<const f32x4 *>(T + r * RS + n);
                if (r < rn && n0 + n < NO)
                    __builtin_nontemporal_store(v, reinterpret_cast<f32x4 *>(static_cast<float *>(p.out) + (size_t)(r0 + r) * NO + n0 + n));
            }
        } else {
#pragma unroll
            for (int i = 0; i < 32 * WO / 8; i += 64) {
                const int r = (i + lane) / (WO / 8), n = 8 * ((i + lane) & (WO / 8 - 1));
                float u[8];
                *reinterpret_cast<f32x4 *>(u) = *reinterpret_cast<const f32x4 *>(T + r * RS + n);
                *reinterpret_cast<f32x4 *>(u + 4) = *reinterpret_cast<const f32x4 *>(T + r * RS + n + 4);
                const bool in = r < rn && n0 + n < NO;
                const size_t at = (size_t)(r0 + r) * NO + n0 + n;
                if (OT == X_BF16) {
                    typedef __bf16 b8 __attribute__((ext_vector_type(8)));
                    b8 o;
#pragma unroll
                    for (int k = 0; k < 8; ++k) o[k] = (__bf16)u[k];
                    if (in) __builtin_nontemporal_store(o, reinterpret_cast<b8 *>(static_cast<uint16_t *>(p.out) + at));
                } else {
                    // four lanes hold a block of 32 outputs
                    uint32_t m = 0;
#pragma unroll
                    for (int k = 0; k < 8; ++k) m = max(m, __float_as_uint(u[k]) & 0x7FFFFFFFu);
                    m = max(m, dpp_u32<0xB1>(m));
                    m = max(m, dpp_u32<0x4E>(m));
                    const uint32_t sc = mx4_scale(m);
                    const uint32_t q = sc == MX_NAN ? 0u : mx4_codes8(u, e8m0_f32(sc));
                    if (in) {
                        reinterpret_cast<uint32_t *>(p.out)[at >> 3] = q;
                        if ((lane & 3) == 0) p.out_scales[at >> 5] = (uint8_t)sc;
                    }
                }
            }
        }
        __builtin_amdgcn_wave_barrier();
    }
}

template <bool GLU, int OT>
__global__ __launch_bounds__(256, 2) void product_mx4_kernel(Mx4Product p, int bm, int ntiles)
{
    __shared__ __attribute__((aligned(16))) uint8_t mx4_lds[PB_LDS];
    int nt;
    const Tile t = find_tile(p, blockIdx.x, bm, ntiles, threadIdx.x & 63, nt);
    if (t.rows < 1) return;
    switch ((t.rows + 31) >> 5) {
    case 1: product_tile<GLU, OT, 1>(p, t, nt, mx4_lds); break;
    case 2: product_tile<GLU, OT, 2>(p, t, nt, mx4_lds); break;
    case 3: product_tile<GLU, OT, 3>(p, t, nt, mx4_lds); break;
    case 4: product_tile<GLU, OT, 4>(p, t, nt, mx4_lds); break;
    default: product_tile<GLU, OT, 5>(p, t, nt, mx4_lds); break;
    }
}

// ---------------------------------------------------------------------------------------------
// Product of bf16 / fp32 rows with MX4 weights: few rows per group, so streaming the weights is what
// counts.  Measured: 16 tokens top-22 of 512 experts (2688 x 1024) 78 us, 377 MB at 4.8 TB/s; 8 tokens'
// fp32 rows through 51 experts' down projection (2816 x 704) 17 us; one token's gate/up through 8
// experts (1408 x 2816) 9 us, which is a block's chain of loads: the groups' offsets, the row's place,
// the row, while the weights come (weights straight into the matrix cores' lanes: 302 / 66 / 11.5 us).
//
// A wave owns a set of 32 weight rows (with SwiGLU 16 gate rows and their up rows), or with
// KS > 1 every KS-th stage of 256 columns of one, and streams their codes and scales through a ring
// of its own in LDS by direct-to-LDS loads: neighbouring lanes read neighbouring bytes, whole 128-byte
// lines of a row, since a second load of a line that is still on its way stalls the cache.  Only its own loads fill
// the ring, so it runs without barriers.  The group's rows of x lie in LDS for all sets and waves of
// the block, as bf16: an fp32 x is cut into three terms whose sum is x, weights widen exactly, so
// every product is exact and the sums are fp32.

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

// The same with 128-byte rows.
__device__ __forceinline__ int chunk_at(int r, int c) { return r * 128 + 16 * (c ^ ((r >> 1) & 7)); }

constexpr int PW_WAVES = 4, PW_RING = 2;               // waves of a block, stages of a wave's ring
constexpr int PW_STAGE = 32 * 128 + 4 * 32 * 4;        // codes, then scales (four dwords per row) of 256 columns

// 2 bytes per lane, each zero-extended into the dword lds + 4 l of lane l.
__device__ __forceinline__ void lds_dma2(const void *g, uint32_t lds)
{
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_ushort %1, off"
                 :: "s"(__builtin_amdgcn_readfirstlane(lds)), "v"(g) : "memory", "m0");
}

// MT: 16-row fragments of x at a time.
template <int XK, int MT, int KS>
struct Wide {
    // x: three blocks to a CU where they are many and their groups small, else two
    static constexpr int SLAB = (KS == 1 && MT == 1 ? 16 : 40) * 1024;
    // rows of a block: as many as KS stages of x fit the slab for
    static constexpr int FIT = SLAB / (2 * XTerms<XK>::N * (KS * 256 + 8));
    static constexpr int RM = FIT < 16 * MT ? FIT : 16 * MT;
};

template <int XK, bool GLU, int MT, int KS>
__global__ __launch_bounds__(64 * PW_WAVES, KS == 1 && MT == 1 ? 3 : 2) void product_wide_kernel(Mx4Product p, int nblocks)
{
    constexpr int NTERM = XTerms<XK>::N, SETS = PW_WAVES / KS, RM = Wide<XK, MT, KS>::RM, PW_SLAB = Wide<XK, MT, KS>::SLAB;
    __shared__ __attribute__((aligned(16))) uint8_t s_ring[PW_WAVES * PW_RING * PW_STAGE];
    __shared__ __attribute__((aligned(16))) uint8_t s_slab[PW_SLAB];
    __shared__ int s_src[16 * MT];
    const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63, li = lane & 15, lg = lane >> 4;
    const int slot = blockIdx.x / nblocks;
    const Tile t = find_rows(p, slot, RM, lane);
    if (t.rows < 1) return;
    constexpr int WO = GLU ? 16 : 32, TN = 2;              // outputs of a set, 16-row weight tiles
    const int F = p.N >> 1, NO = GLU ? F : p.N;
    const int KB = p.K >> 1, KSC = p.K >> 5, steps = (p.K + 255) >> 8;   // stages of 256 columns
    const int ks = wave % KS, n0 = ((blockIdx.x - slot * nblocks) * SETS + wave / KS) * WO;
    const bool live = n0 < NO;
    uint8_t *ring = s_ring + wave * PW_RING * PW_STAGE;
    // sources: 8 lanes read a weight row's 128 bytes of a stage; lanes r and r + 32 the scales of row r
    auto weight_row = [&](int r) {
        int n = n0 + r;
        if (GLU) n = min(n0 + (r & 15), F - 1) + ((r & 16) ? F : 0);
        return (size_t)t.g * p.N + min(n, p.N - 1);
    };
    const uint8_t *wsrc[4];
    int dchunk[2];                                         // of even and odd instructions (8 rows each)
#pragma unroll
    for (int i = 0; i < 4; ++i) wsrc[i] = p.w + weight_row(8 * i + (lane >> 3)) * KB;
#pragma unroll
    for (int i = 0; i < 2; ++i) dchunk[i] = 16 * ((lane & 7) ^ (((8 * i + (lane >> 3)) >> 1) & 7));
    const uint8_t *wsc = p.ws + weight_row(lane & 31) * KSC;
    auto issue = [&](int s, int buf) {
        if (s >= steps) return;
        const uint32_t L = lds_addr(ring + buf * PW_STAGE);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int off = s * 128 + dchunk[i & 1];
            lds_dma16(off < KB ? wsrc[i] + off : reinterpret_cast<const uint8_t *>(&mx4_zeros), L + i * 1024);
        }
        // blocks past the end take the row's last scales (their codes are zeros)
#pragma unroll
        for (int h = 0; h < 2; ++h) lds_dma2(wsc + min(8 * s + 4 * h + ((lane >> 4) & 2), KSC - 2), L + 4096 + 256 * h);
    };

    const int R = t.rows;
    if (live) issue(ks, 0);

    // ---- x: [term][row][columns of a slab + 8]; the slab holds all of K where it fits
    if (tid < R) s_src[tid] = source_row(p, t.row0 + tid);
    const int SC = (PW_SLAB / (2 * NTERM * R) - 8) / 256 / KS * KS;   // stages of a slab, at least KS
    const int XS = min(SC, steps) * 256 + 8;                   // bf16 values of a slab row
    const int nslab = (steps + SC - 1) / SC;
    uint16_t *slab = reinterpret_cast<uint16_t *>(s_slab);
    auto load_slab = [&](int b) {
        const int c0 = b * SC * 256, pieces = (min(steps, (b + 1) * SC) * 256 - c0) / 8;
        for (int i = tid; i < R * pieces; i += 64 * PW_WAVES) {
            const int r = i / pieces, c = 8 * (i - r * pieces);
            const size_t at = (size_t)s_src[r] * p.K + c0 + c;
            const bool in = c0 + c < p.K;
            uint16_t *dst = slab + r * XS + c;
            if constexpr (XK == X_F32) {
                float v[8] = {};
                if (in) {
                    const float4 *g = reinterpret_cast<const float4 *>(static_cast<const float *>(p.x) + at);
                    const float4 a = g[0], b4 = g[1];
                    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
                    v[4] = b4.x; v[5] = b4.y; v[6] = b4.z; v[7] = b4.w;
                }
                bf16x8 xt[3];
                cut_f32x8(v, xt);
#pragma unroll
                for (int k = 0; k < 3; ++k) *reinterpret_cast<bf16x8 *>(dst + k * R * XS) = xt[k];
            } else {
                uint4 v = make_uint4(0, 0, 0, 0);
                if (in) v = *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(p.x) + at);
                *reinterpret_cast<uint4 *>(dst) = v;
            }
        }
    };

    int buf = 0;
    // With few rows the three terms of an fp32 x fit side by side: column li of the matrix product
    // is term li / R of row li % R, one instruction does the work of three, and the columns of a
    // row are added at the end (8 tokens' down projection 18.5 -> 17.3 us).
    const bool packed = XK == X_F32 && MT == 1 && 3 * R <= 16;
    const int xrow = packed ? min(li, 3 * R - 1) : li;

    f32x4 acc[TN][MT];
#pragma unroll
    for (int j = 0; j < TN; ++j)
#pragma unroll
        for (int m = 0; m < MT; ++m) acc[j][m] = zero4();
    for (int b = 0; b < nslab; ++b) {
        lds_barrier();
        load_slab(b);
        lds_barrier();
        const int send = live ? min(steps, (b + 1) * SC) : 0;
        for (int s = b * SC + ks; s < send; s += KS) {
            // this stage has landed, and what was read from the buffer to fill next has arrived
            asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
            issue(s + KS, buf ^ 1);
            const uint8_t *W = ring + buf * PW_STAGE;
            buf ^= 1;
#pragma unroll
            for (int u = 0; u < 2; ++u) {              // 128 columns
                const uint32_t *S = reinterpret_cast<const uint32_t *>(W + 4096) + 64 * u + (lg >> 1) * 32 + li;
                uint4 w[TN];
                float sc[TN];
#pragma unroll
                for (int j = 0; j < TN; ++j) {
                    w[j] = *reinterpret_cast<const uint4 *>(W + chunk_at(16 * j + li, 4 * u + lg));
                    sc[j] = e8m0_f32((S[16 * j] >> (8 * (lg & 1))) & 0xFFu);
                }
#pragma unroll
                for (int m = 0; m < MT; ++m) {
                    if (MT > 1 && 16 * m >= R) break;
                    const uint16_t *X = slab + (packed ? xrow : min(16 * m + li, R - 1)) * XS + (s - b * SC) * 256 + 128 * u + 32 * lg;
                    if (packed) {
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            const bf16x8 xt = *reinterpret_cast<const bf16x8 *>(X + 8 * q);
#pragma unroll
                            for (int j = 0; j < TN; ++j) {
                                const uint32_t c = q == 0 ? w[j].x : q == 1 ? w[j].y : q == 2 ? w[j].z : w[j].w;
                                acc[j][m] = mfma16x16x32_bf16(mx4_bf16x8(c, sc[j]), xt, acc[j][m]);
                            }
                        }
                        continue;
                    }
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        bf16x8 xt[NTERM];
#pragma unroll
                        for (int k = 0; k < NTERM; ++k) xt[k] = *reinterpret_cast<const bf16x8 *>(X + k * R * XS + 8 * q);
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
        }
    }
    // no load may still be writing LDS
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
    if (!live) return;
    if (packed) {
        // row r: the small terms first
#pragma unroll
        for (int j = 0; j < TN; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float mid = __shfl(acc[j][0][i], (lane & 48) | min(li + R, 15), WAVE);
                const float low = __shfl(acc[j][0][i], (lane & 48) | min(li + 2 * R, 15), WAVE);
                acc[j][0][i] += low + mid;
            }
    }
    // ---- element i of a lane's acc[j][m] is weight row 16 j + 4 lg + i of x row 16 m + li
    if constexpr (KS > 1) {
        // the KS waves' sums meet in LDS, in wave order (the rings are idle)
        float *red = reinterpret_cast<float *>(ring);
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            if (16 * m >= R) break;
            if (m > 0) lds_barrier();
#pragma unroll
            for (int j = 0; j < TN; ++j) *reinterpret_cast<f32x4 *>(red + li * 36 + 16 * j + 4 * lg) = acc[j][m];
            lds_barrier();
            const int rows = min(16, R - 16 * m);
            for (int i = ks * 64 + lane; i < rows * WO; i += KS * 64) {
                const int r = i / WO, n = i & (WO - 1);
                const float *q = reinterpret_cast<const float *>(s_ring + (wave - ks) * PW_RING * PW_STAGE) + r * 36 + n;
                float v = 0.f, u = 0.f;
#pragma unroll
                for (int k = 0; k < KS; ++k) {
                    v += q[k * (PW_RING * PW_STAGE / 4)];
                    if (GLU) u += q[k * (PW_RING * PW_STAGE / 4) + 16];
                }
                if (n0 + n < NO) {
                    v = GLU ? silu_fast(v) * u : activate(v, p.act);
                    const size_t at = (size_t)(t.row0 + 16 * m + r) * NO + n0 + n;
                    if (p.otype == X_F32) store1<X_F32>(p, at, v);
                    else store1<X_BF16>(p, at, v);
                }
            }
        }
    } else {
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            if (16 * m + li >= R) continue;
            const size_t row = (size_t)(t.row0 + 16 * m + li) * NO;
#pragma unroll
            for (int j = 0; j < (GLU ? 1 : 2); ++j) {
                const int n = n0 + 16 * j + 4 * lg;
                float v[4];
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    v[i] = GLU ? silu_fast(acc[j][m][i]) * acc[1][m][i] : activate(acc[j][m][i], p.act);
                store4(p, row + n, n, NO, v);
            }
        }
    }
}

template <int XK, bool GLU>
hipError_t launch_wide(const Mx4Product &p, hipStream_t s)
{
    const int WO = GLU ? 16 : 32, NO = GLU ? p.N / 2 : p.N;
    const int rows = p.Pr + p.S * p.T, G = p.offsets ? p.E + p.S : 1;
    const int slots = rows < G ? rows : G, sets = (NO + WO - 1) / WO;
    const auto go = [&](auto kernel, int rm, int per) {
        const int nblocks = (sets + per - 1) / per;
        kernel<<<(unsigned)(rows / rm + slots) * nblocks, 64 * PW_WAVES, 0, s>>>(p, nblocks);
    };
    // Where groups hold many rows: 64 (fp32: 25, which the slab holds) at a time, not 16.
    constexpr int MANY = XK == X_F32 ? 2 : 4;
    if (rows > 16 && rows >= 8 * G)
        go(product_wide_kernel<XK, GLU, MANY, 1>, Wide<XK, MANY, 1>::RM, PW_WAVES);
    // Four waves share a set's columns while the sets alone leave the GPU short of waves (256 CUs of
    // 12): one token's 44 sets x 8 experts 9.0 us split and 18 whole, 88 x 51 at 8 tokens 37 and 19.
    else if ((long long)sets * slots < 2048)
        go(product_wide_kernel<XK, GLU, 1, PW_WAVES>, Wide<XK, 1, PW_WAVES>::RM, 1);
    else
        go(product_wide_kernel<XK, GLU, 1, 1>, Wide<XK, 1, 1>::RM, PW_WAVES);
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
    if (p.xtype != X_MX4) {
        const bool g = p.act == ACT_SWIGLU;
        if (p.xtype == X_F32) return g ? launch_wide<X_F32, true>(p, s) : launch_wide<X_F32, false>(p, s);
        return g ? launch_wide<X_BF16, true>(p, s) : launch_wide<X_BF16, false>(p, s);
    }
    const int NO = p.act == ACT_SWIGLU ? p.N / 2 : p.N;
    const int per = p.act == ACT_SWIGLU ? PB_N / 2 : PB_N;
    const int ntiles = (NO + per - 1) / per;
    const int rows = p.Pr + p.S * p.T, G = p.offsets ? p.E + p.S : 1;
    // Groups of about a tile's size lie whole in one of 160 rows where 128 would leave many a second
    // tile of a few rows that reads all the weights again (groups of 128 +- 11 rows, gate/up of 2048
    // tokens: 96 us against 110).  Larger groups are cut into 128s (4096 rows by 6144 by
    // 6144: 114 us against 130).
    const int slots = rows < G ? rows : G, bm = rows <= 144 * slots ? PB_M : 128;
    const int mtiles = rows / bm + slots;                          // at least the sum of the groups' tiles
    const unsigned grid = ((unsigned)mtiles * ntiles + 7) / 8 * 8;
    const bool glu = p.act == ACT_SWIGLU;
    auto go = [&](auto g, auto o) { product_mx4_kernel<g.value, o.value><<<grid, 256, 0, s>>>(p, bm, ntiles); };
    auto by_out = [&](auto g) {
        if (p.otype == X_F32) go(g, std::integral_constant<int, X_F32>{});
        else if (p.otype == X_BF16) go(g, std::integral_constant<int, X_BF16>{});
        else go(g, std::integral_constant<int, X_MX4>{});
    };
    if (glu) by_out(std::true_type{});
    else by_out(std::false_type{});
    return hipGetLastError();
}

}  // namespace moe
