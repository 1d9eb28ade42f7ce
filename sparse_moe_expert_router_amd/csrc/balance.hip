// Router training statistics: the load-balancing loss and the z loss over a batch's logits, the
// experts' load counts, and the gradient with respect to the logits.
//
// For the n tokens that count (mask, and not every logit -inf), p_t = softmax(l_t),
// f_e = (pairs of counted tokens routed to e) / (n k), P_e = mean_t p_te:
//     balance = E sum_e f_e P_e,     z = mean_t lse(l_t)^2,
//     d l_te  = p_te (g_b E / n (f_e - sum_j f_j p_tj) + g_z 2 / n lse_t)
//             + [e in S_t] w_te (dw_te - sum_j w_tj dw_tj)          (renormalised top-k weights),
// f taken as a constant (it is a count).  The floor is reading the logits once (and writing the
// gradient): 17 MB and 37 MB for 32768 tokens of 128 experts, 4 and 8 us.  Measured there: the loss 10.3
// + 4.3 us (128 blocks of 16 waves, bound by their arithmetic and the rows' exchanges; then one block
// that adds up), the gradient 13.8 us, 2.7 TB/s.  A batch of 8 tokens takes one launch of 3.2 us.  The
// first form (256-thread blocks, no row ahead, library exp and log) took 40 + 6.8 and 16 us.
//
// A row's E logits lie in LPR lanes (a power of two) with NJ pieces of VEC values each: softmax
// needs only exchanges inside those lanes, and the per-expert sums stay in registers until a
// block's end.  Sums of any one output run in a fixed order; only integer counts use atomics.
#include <hip/hip_runtime.h>

#include <type_traits>

#include "moe_common.hpp"
#include "moe_launch.hpp"

namespace moe {
namespace {

constexpr int BL_THREADS = 1024;    // of the loss kernels
constexpr int BG_THREADS = 256;     // of the gradient kernel
constexpr int BL_BLOCKS = 128;      // most partial sums the second kernel adds up
constexpr int MAX_EPAD = 512;

template <int LPR>
__device__ __forceinline__ float group_sum(float v, int lane)
{
#pragma unroll
    for (int o = 1; o < LPR; o <<= 1) v += __uint_as_float(xor_lane_u32(__float_as_uint(v), o, lane));
    return v;
}
template <int LPR>
__device__ __forceinline__ float group_max(float v, int lane)
{
#pragma unroll
    for (int o = 1; o < LPR; o <<= 1) v = fmaxf(v, __uint_as_float(xor_lane_u32(__float_as_uint(v), o, lane)));
    return v;
}

__device__ __forceinline__ float load_logit(const void *l, int ltype, size_t at)
{
    if (ltype == X_F32) return static_cast<const float *>(l)[at];
    if (ltype == X_BF16) return bf16_bits_to_f32(static_cast<const uint16_t *>(l)[at]);
    return (float)static_cast<const double *>(l)[at];
}

template <int LPR, int NJ, int VEC>
__device__ __forceinline__ int expert_of(int sub, int j, int v)
{
    return (j * LPR + sub) * VEC + v;
}

// the row's logits, -inf past E
template <int LT, int LPR, int NJ, int VEC>
__device__ __forceinline__ void load_row(const void *logits, size_t base, int E, int sub, float (&l)[NJ * VEC])
{
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
        const int e0 = expert_of<LPR, NJ, VEC>(sub, j, 0);
        if constexpr (VEC == 4) {
            float4 a = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
            if (e0 < E) {                                     // E is a multiple of 4 here
                if constexpr (LT == X_F32) {
                    a = *reinterpret_cast<const float4 *>(static_cast<const float *>(logits) + base + e0);
                } else if constexpr (LT == X_BF16) {
                    const uint2 u = *reinterpret_cast<const uint2 *>(static_cast<const uint16_t *>(logits) + base + e0);
                    a = make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xFFFF0000u),
                                    __uint_as_float(u.y << 16), __uint_as_float(u.y & 0xFFFF0000u));
                } else {
                    const double *d = static_cast<const double *>(logits) + base + e0;
                    a = make_float4((float)d[0], (float)d[1], (float)d[2], (float)d[3]);
                }
            }
            l[4 * j] = a.x; l[4 * j + 1] = a.y; l[4 * j + 2] = a.z; l[4 * j + 3] = a.w;
        } else {
            l[j] = e0 < E ? load_logit(logits, LT, base + e0) : -INFINITY;
        }
    }
}

// In place: l becomes p = softmax(l).  Returns lse; `none`: every logit is -inf (p = 0, lse = 0).
// A NaN or +inf logit makes the row NaN.  The exponent, logarithm and reciprocal instructions are good
// to 1 ulp; the exponent's rounded argument adds |l - max| roundings of 2^-24 to p, as the fp32 logits
// themselves carry.
template <int LPR, int NV>
__device__ __forceinline__ float softmax_row(float (&l)[NV], int lane, bool &none)
{
    float m = -INFINITY;
#pragma unroll
    for (int i = 0; i < NV; ++i) m = fmaxf(m, l[i] != l[i] ? INFINITY : l[i]);
    m = group_max<LPR>(m, lane);
    none = m == -INFINITY;
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        l[i] = none ? 0.f : __builtin_amdgcn_exp2f((l[i] - m) * 1.44269504f);
        s += l[i];
    }
    s = group_sum<LPR>(s, lane);
    const float r = none ? 0.f : __builtin_amdgcn_rcpf(s);
#pragma unroll
    for (int i = 0; i < NV; ++i) l[i] *= r;
    return none ? 0.f : fmaf(__builtin_amdgcn_logf(s), 0.693147181f, m);
}

// The block's share of the rows: partial sums of p, of lse^2, and counts.  With one block
// (`last`), the results themselves.
struct BalanceOut {
    float *loss;
    int32_t *counts;
    float *mean_prob;
    float *part_p;          // [blocks][Epad]
    int32_t *part_c;        // [blocks][Epad]
    float *part_z;          // [blocks]
    int32_t *part_n;        // [blocks]
    int Epad;
};

// A row's share of a lane, as it is in memory: loaded a row ahead of its use.  Padding rows are loaded
// like the others (they lie inside the arrays) and dropped after.
template <int LT, int LPR, int NJ, int VEC>
struct Row {
    float l[NJ * VEC];
    int id;                 // slot `sub` of the row
    bool on;
    __device__ __forceinline__ void load(const void *logits, int t, int T, int E, const int32_t *idx, int k,
                                         const uint8_t *mask, int sub)
    {
        const int r = min(t, T - 1);
        load_row<LT, LPR, NJ, VEC>(logits, (size_t)r * E, E, sub, l);
        id = idx[(size_t)r * k + min(sub, k - 1)];
        on = t < T && (mask == nullptr || mask[r] != 0);
    }
    __device__ __forceinline__ void drop_padding()
    {
#pragma unroll
        for (int i = 0; i < NJ * VEC; ++i) l[i] = on ? l[i] : -INFINITY;
    }
};

// the block's sum of v: waves by exchange, then in wave order
__device__ __forceinline__ float block_sum(float v, float *s_red, int tid)
{
    v = wave_sum(v);
    if ((tid & 63) == 0) s_red[tid >> 6] = v;
    __syncthreads();
    float t = 0.f;
    for (int i = 0; i < BL_THREADS / 64; ++i) t += s_red[i];
    return t;
}

template <int LT, int LPR, int NJ, int VEC>
__global__ __launch_bounds__(BL_THREADS) void balance_rows_kernel(const void *__restrict__ logits, int T, int E,
                                                                  const int32_t *__restrict__ idx, int k,
                                                                  const uint8_t *__restrict__ mask, BalanceOut o)
{
    constexpr int NV = NJ * VEC, SUBS = BL_THREADS / LPR, NW = BL_THREADS / 64;   // SUBS rows at a time
    __shared__ int s_cnt[MAX_EPAD];
    __shared__ float s_p[NW * LPR * NV];
    __shared__ float s_z[NW];
    __shared__ int s_n[NW];
    __shared__ float s_red[NW];
    const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63, sub = tid % LPR, row_in = tid / LPR;
    const int per = (T + gridDim.x - 1) / gridDim.x;
    const int t0 = blockIdx.x * per, t1 = min(T, t0 + per);
    Row<LT, LPR, NJ, VEC> next;
    next.load(logits, t0 + row_in, T, E, idx, k, mask, sub);
    for (int e = tid; e < E; e += BL_THREADS) s_cnt[e] = 0;
    __syncthreads();

    float acc[NV] = {}, z = 0.f;
    int n = 0;
    for (int tb = t0; tb < t1; tb += SUBS) {
        const int t = tb + row_in;
        Row<LT, LPR, NJ, VEC> r = next;
        if (tb + SUBS < t1) next.load(logits, t + SUBS, T, E, idx, k, mask, sub);
        r.on = r.on && t < t1;
        r.drop_padding();
        bool none;
        const float lse = softmax_row<LPR, NV>(r.l, lane, none);
#pragma unroll
        for (int i = 0; i < NV; ++i) acc[i] += r.l[i];
        z += lse * lse;
        if (!none) {
            n += 1;
            if (sub < k) atomicAdd(&s_cnt[clamp_id(r.id, E)], 1);
            for (int j = sub + LPR; j < k; j += LPR) atomicAdd(&s_cnt[clamp_id(idx[(size_t)t * k + j], E)], 1);
        }
    }
    // the wave's rows, then the waves
#pragma unroll
    for (int s = LPR; s < 64; s <<= 1) {
#pragma unroll
        for (int i = 0; i < NV; ++i) acc[i] += __uint_as_float(xor_lane_u32(__float_as_uint(acc[i]), s, lane));
        z += __uint_as_float(xor_lane_u32(__float_as_uint(z), s, lane));
        n += (int)xor_lane_u32((uint32_t)n, s, lane);
    }
    if (lane < LPR) {
#pragma unroll
        for (int i = 0; i < NV; ++i) s_p[wave * LPR * NV + expert_of<LPR, NJ, VEC>(sub, i / VEC, i % VEC)] = acc[i];
    }
    if (lane == 0) {
        s_z[wave] = z;
        s_n[wave] = n;
    }
    __syncthreads();
    float zt = 0.f;
    int nt = 0;
#pragma unroll
    for (int i = 0; i < NW; ++i) {
        zt += s_z[i];
        nt += s_n[i];
    }
    const bool whole = gridDim.x == 1;
    const float inv = 1.f / (float)max(nt, 1);
    float dot = 0.f;
    if (tid < E) {
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < NW; ++i) s += s_p[i * LPR * NV + tid];
        const int c = s_cnt[tid];
        if (whole) {
            s *= inv;
            o.counts[tid] = c;
            o.mean_prob[tid] = s;
            dot = (float)c * (inv / (float)k) * s;
        } else {
            o.part_p[(size_t)blockIdx.x * o.Epad + tid] = s;
            o.part_c[(size_t)blockIdx.x * o.Epad + tid] = c;
        }
    }
    if (whole) {
        dot = block_sum(dot, s_red, tid);
        if (tid == 0) {
            o.loss[0] = (float)E * dot;
            o.loss[1] = zt * inv;
        }
    } else if (tid == 0) {
        o.part_z[blockIdx.x] = zt;
        o.part_n[blockIdx.x] = nt;
    }
}

// Adds the blocks' partial sums: thread groups take every G-th block, four experts a thread, then the
// groups are added in order.
__global__ __launch_bounds__(BL_THREADS) void balance_join_kernel(int blocks, int E, int k, BalanceOut o)
{
    __shared__ float4 s_p[BL_THREADS];
    __shared__ int4 s_c[BL_THREADS];
    __shared__ float s_red[BL_THREADS / 64];
    const int tid = threadIdx.x, C = o.Epad / 4, G = BL_THREADS / C, c = tid % C, g = tid / C;
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
    int4 n4 = make_int4(0, 0, 0, 0);
    if (g < G) {
#pragma unroll 4
        for (int b = g; b < blocks; b += G) {
            const float4 u = *reinterpret_cast<const float4 *>(o.part_p + (size_t)b * o.Epad + 4 * c);
            const int4 v = *reinterpret_cast<const int4 *>(o.part_c + (size_t)b * o.Epad + 4 * c);
            s.x += u.x; s.y += u.y; s.z += u.z; s.w += u.w;
            n4.x += v.x; n4.y += v.y; n4.z += v.z; n4.w += v.w;
        }
    }
    s_p[tid] = s;
    s_c[tid] = n4;
    // every wave adds the row counts and the z sums itself
    float zt = 0.f;
    int nt = 0;
    for (int b = tid & 63; b < blocks; b += 64) {
        zt += o.part_z[b];
        nt += o.part_n[b];
    }
    zt = wave_sum(zt);
    nt = wave_sum(nt);
    __syncthreads();
    const float inv = 1.f / (float)max(nt, 1);
    float dot = 0.f;
    if (tid < E) {
        float P = 0.f;
        int cnt = 0;
        for (int i = 0; i < G; ++i) {
            P += reinterpret_cast<const float *>(s_p + i * C)[tid];
            cnt += reinterpret_cast<const int *>(s_c + i * C)[tid];
        }
        P *= inv;
        o.counts[tid] = cnt;
        o.mean_prob[tid] = P;
        dot = (float)cnt * (inv / (float)k) * P;
    }
    dot = block_sum(dot, s_red, tid);
    if (tid == 0) {
        o.loss[0] = (float)E * dot;
        o.loss[1] = zt * inv;
    }
}

template <int LT, int LPR, int NJ, int VEC>
__global__ __launch_bounds__(BG_THREADS) void balance_grad_kernel(
    const void *__restrict__ logits, int T, int E, const int32_t *__restrict__ idx, int k,
    const uint8_t *__restrict__ mask, const int32_t *__restrict__ counts, const float *__restrict__ d_loss,
    const float *__restrict__ topk_w, const float *__restrict__ d_topk_w, void *__restrict__ d_logits, int gtype)
{
    constexpr int NV = NJ * VEC, SUBS = BG_THREADS / LPR;
    __shared__ int s_id[SUBS][MAX_K];
    __shared__ float s_dw[SUBS][MAX_K];
    const int tid = threadIdx.x, lane = tid & 63, sub = tid % LPR, row_in = tid / LPR;
    const bool wpart = topk_w != nullptr;
    Row<LT, LPR, NJ, VEC> next;
    float w_next = 0.f, dw_next = 0.f;
    auto fetch = [&](int t) {
        next.load(logits, t, T, E, idx, k, mask, sub);
        if (wpart) {
            const size_t at = (size_t)min(t, T - 1) * k + min(sub, k - 1);
            w_next = topk_w[at];
            dw_next = d_topk_w[at];
        }
    };
    fetch(blockIdx.x * SUBS + row_in);
    // f of this lane's experts; the counts sum to n k
    float f[NV];
    int c[NV], total = 0;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int e = expert_of<LPR, NJ, VEC>(sub, i / VEC, i % VEC);
        c[i] = e < E ? counts[e] : 0;
        total += c[i];
    }
#pragma unroll
    for (int o = 1; o < LPR; o <<= 1) total += (int)xor_lane_u32((uint32_t)total, o, lane);
    const float inv_nk = total > 0 ? 1.f / (float)total : 0.f, inv_n = inv_nk * (float)k;
#pragma unroll
    for (int i = 0; i < NV; ++i) f[i] = (float)c[i] * inv_nk;
    const float gb = d_loss[0] * (float)E * inv_n, gz = 2.f * d_loss[1] * inv_n;

    for (int tb = blockIdx.x * SUBS; tb < T; tb += gridDim.x * SUBS) {
        const int t = tb + row_in;
        Row<LT, LPR, NJ, VEC> r = next;
        const float w0 = w_next, dw0 = dw_next;
        if (tb + (int)gridDim.x * SUBS < T) fetch(t + gridDim.x * SUBS);
        r.drop_padding();
        float(&l)[NV] = r.l;
        bool none;
        const float lse = softmax_row<LPR, NV>(l, lane, none);
        float fp = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i) fp = fmaf(f[i], l[i], fp);
        fp = group_sum<LPR>(fp, lane);
#pragma unroll
        for (int i = 0; i < NV; ++i) l[i] = none ? 0.f : l[i] * fmaf(gb, f[i] - fp, gz * lse);
        if (wpart) {
            // the k selected experts' share, added in slot order by the lane that holds the expert
            const size_t base = (size_t)min(t, T - 1) * k;
            float wd = none || sub >= k ? 0.f : w0 * dw0;
            for (int j = sub + LPR; j < k; j += LPR) wd = none ? 0.f : fmaf(topk_w[base + j], d_topk_w[base + j], wd);
            wd = group_sum<LPR>(wd, lane);
            if (sub < k) {
                s_id[row_in][sub] = clamp_id(r.id, E);
                s_dw[row_in][sub] = none ? 0.f : w0 * (dw0 - wd);
            }
            for (int j = sub + LPR; j < k; j += LPR) {
                s_id[row_in][j] = clamp_id(idx[base + j], E);
                s_dw[row_in][j] = none ? 0.f : topk_w[base + j] * (d_topk_w[base + j] - wd);
            }
            // a row's lanes sit in one wave, whose LDS accesses stay in order
            __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
            __builtin_amdgcn_wave_barrier();
            __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
            for (int j = 0; j < k; ++j) {
                const int id = s_id[row_in][j];
                const float v = s_dw[row_in][j];
#pragma unroll
                for (int i = 0; i < NV; ++i)
                    if (id == expert_of<LPR, NJ, VEC>(sub, i / VEC, i % VEC)) l[i] += v;
            }
            __builtin_amdgcn_wave_barrier();
        }
        if (t >= T) continue;
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
            const int e0 = expert_of<LPR, NJ, VEC>(sub, j, 0);
            if (e0 >= E) continue;
            const size_t at = (size_t)t * E + e0;
            if constexpr (VEC == 4) {
                if (gtype == X_F32) {
                    *reinterpret_cast<float4 *>(static_cast<float *>(d_logits) + at) =
                        make_float4(l[4 * j], l[4 * j + 1], l[4 * j + 2], l[4 * j + 3]);
                } else {
                    typedef __bf16 b4 __attribute__((ext_vector_type(4)));
                    const b4 v = {(__bf16)l[4 * j], (__bf16)l[4 * j + 1], (__bf16)l[4 * j + 2], (__bf16)l[4 * j + 3]};
                    *reinterpret_cast<b4 *>(static_cast<uint16_t *>(d_logits) + at) = v;
                }
            } else if (gtype == X_F32) {
                static_cast<float *>(d_logits)[at] = l[j];
            } else {
                static_cast<uint16_t *>(d_logits)[at] = __builtin_bit_cast(uint16_t, (__bf16)l[j]);
            }
        }
    }
}

// Calls fn with the (LPR, NJ, VEC) that E takes: four values a lane where E allows whole pieces.
template <typename Fn>
hipError_t by_width(int E, Fn fn)
{
    using std::integral_constant;
#define MOE_SHAPE(L, J, V) fn(integral_constant<int, L>{}, integral_constant<int, J>{}, integral_constant<int, V>{})
    if (E % 4 == 0) {
        if (E <= 16) return MOE_SHAPE(4, 1, 4);
        if (E <= 64) return MOE_SHAPE(16, 1, 4);
        if (E <= 128) return MOE_SHAPE(32, 1, 4);
        if (E <= 256) return MOE_SHAPE(64, 1, 4);
        return MOE_SHAPE(64, 2, 4);
    }
    if (E <= 16) return MOE_SHAPE(16, 1, 1);
    if (E <= 64) return MOE_SHAPE(32, 2, 1);
    if (E <= 256) return MOE_SHAPE(64, 4, 1);
    return MOE_SHAPE(64, 8, 1);
#undef MOE_SHAPE
}

template <typename Fn>
hipError_t by_type(int ltype, Fn fn)
{
    using std::integral_constant;
    if (ltype == X_F32) return fn(integral_constant<int, X_F32>{});
    if (ltype == X_BF16) return fn(integral_constant<int, X_BF16>{});
    return fn(integral_constant<int, X_F64>{});
}

int epad(int E) { return (E + 3) / 4 * 4; }

int balance_blocks(int T, int E)
{
    // a block holds about 4096 logits at a time; four rounds of them cost less than a second launch,
    // and fewer blocks leave less to add up
    const long long values = (long long)T * E;
    const long long b = (values + 16383) / 16384;
    return (int)(b < 1 ? 1 : (b > BL_BLOCKS ? BL_BLOCKS : b));
}

size_t up256(size_t v) { return (v + 255) / 256 * 256; }

}  // namespace

size_t balance_workspace_bytes(int T, int E)
{
    const int nb = balance_blocks(T, E);
    return 2 * up256((size_t)nb * epad(E) * 4) + 2 * up256((size_t)nb * 4);
}

hipError_t launch_balance_loss(const void *logits, int ltype, int T, int E, const int32_t *idx, int k,
                               const uint8_t *mask, float *loss, int32_t *counts, float *mean_prob, void *ws,
                               hipStream_t s)
{
    ProfScope prof(K_BALANCE, s);
    const int nb = balance_blocks(T, E);
    char *w = static_cast<char *>(ws);
    const size_t pe = up256((size_t)nb * epad(E) * 4), pz = up256((size_t)nb * 4);
    BalanceOut o{loss, counts, mean_prob, reinterpret_cast<float *>(w), reinterpret_cast<int32_t *>(w + pe),
                 reinterpret_cast<float *>(w + 2 * pe), reinterpret_cast<int32_t *>(w + 2 * pe + pz), epad(E)};
    hipError_t e = by_type(ltype, [&](auto lt) {
        return by_width(E, [&](auto l, auto j, auto v) {
            balance_rows_kernel<lt.value, l.value, j.value, v.value><<<nb, BL_THREADS, 0, s>>>(logits, T, E, idx, k, mask, o);
            return hipGetLastError();
        });
    });
    if (e != hipSuccess || nb == 1) return e;
    balance_join_kernel<<<1, 1024, 0, s>>>(nb, E, k, o);
    return hipGetLastError();
}

hipError_t launch_balance_grad(const void *logits, int ltype, int T, int E, const int32_t *idx, int k,
                               const uint8_t *mask, const int32_t *counts, const float *d_loss, const float *topk_w,
                               const float *d_topk_w, void *d_logits, int gtype, hipStream_t s)
{
    ProfScope prof(K_BALANCE, s);
    return by_type(ltype, [&](auto lt) {
        return by_width(E, [&](auto l, auto j, auto v) {
            constexpr int subs = BG_THREADS / l.value;
            const int want = (T + subs - 1) / subs;
            const int blocks = want < 1024 ? want : 1024;
            balance_grad_kernel<lt.value, l.value, j.value, v.value><<<blocks, BG_THREADS, 0, s>>>(
                logits, T, E, idx, k, mask, counts, d_loss, topk_w, d_topk_w, d_logits, gtype);
            return hipGetLastError();
        });
    });
}

}  // namespace moe
