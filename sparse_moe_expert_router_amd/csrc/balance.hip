// Router training statistics: the load-balancing loss and the z loss over a batch's logits, the
// experts' load counts, and the gradient with respect to the logits.
//
// For the n tokens that count (mask, and not every logit -inf), p_t = softmax(l_t),
// f_e = (pairs of counted tokens routed to e) / (n k), P_e = mean_t p_te:
//     balance = E sum_e f_e P_e,     z = mean_t lse(l_t)^2,
//     d l_te  = p_te (g_b E / n (f_e - sum_j f_j p_tj) + g_z 2 / n lse_t)
//             + [e in S_t] w_te (dw_te - sum_j w_tj dw_tj)          (renormalised top-k weights),
// f taken as a constant (it is a count).  Bound by reading the logits once.
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

constexpr int BL_THREADS = 256;
constexpr int BL_BLOCKS = 128;      // partial sums the second kernel adds up
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
// A NaN or +inf logit makes the row NaN.
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
        l[i] = none ? 0.f : expf(l[i] - m);
        s += l[i];
    }
    s = group_sum<LPR>(s, lane);
    const float r = none ? 0.f : 1.f / s;
#pragma unroll
    for (int i = 0; i < NV; ++i) l[i] *= r;
    return none ? 0.f : m + logf(s);
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

// sum over the block of f_e P_e, in thread order within waves and wave order across them
__device__ __forceinline__ float block_sum(float v, float *s_red, int tid, int nwaves)
{
    v = wave_sum(v);
    __syncthreads();
    if ((tid & 63) == 0) s_red[tid >> 6] = v;
    __syncthreads();
    float t = 0.f;
    for (int i = 0; i < nwaves; ++i) t += s_red[i];
    return t;
}

template <int LT, int LPR, int NJ, int VEC>
__global__ __launch_bounds__(BL_THREADS) void balance_rows_kernel(const void *__restrict__ logits, int T, int E,
                                                                  const int32_t *__restrict__ idx, int k,
                                                                  const uint8_t *__restrict__ mask, BalanceOut o)
{
    constexpr int NV = NJ * VEC, SUBS = BL_THREADS / LPR;     // rows a block holds at a time
    __shared__ int s_cnt[MAX_EPAD];
    __shared__ float s_p[SUBS * LPR * NV];
    __shared__ float s_z[SUBS];
    __shared__ int s_n[SUBS];
    __shared__ float s_red[BL_THREADS / 64];
    const int tid = threadIdx.x, lane = tid & 63, sub = tid % LPR, row_in = tid / LPR;
    for (int e = tid; e < E; e += BL_THREADS) s_cnt[e] = 0;
    __syncthreads();

    float acc[NV] = {}, z = 0.f;
    int n = 0;
    const int per = (T + gridDim.x - 1) / gridDim.x;
    const int t0 = blockIdx.x * per, t1 = min(T, t0 + per);
    for (int tb = t0; tb < t1; tb += SUBS) {
        const int t = tb + row_in;
        float l[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i) l[i] = -INFINITY;
        const bool on = t < t1 && (mask == nullptr || mask[t] != 0);
        if (on) load_row<LT, LPR, NJ, VEC>(logits, (size_t)t * E, E, sub, l);
        bool none;
        const float lse = softmax_row<LPR, NV>(l, lane, none);
#pragma unroll
        for (int i = 0; i < NV; ++i) acc[i] += l[i];
        z += lse * lse;
        if (!none) {
            n += 1;
            for (int j = sub; j < k; j += LPR) atomicAdd(&s_cnt[clamp_id(idx[(size_t)t * k + j], E)], 1);
        }
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) s_p[row_in * LPR * NV + expert_of<LPR, NJ, VEC>(sub, i / VEC, i % VEC)] = acc[i];
    if (sub == 0) {
        s_z[row_in] = z;
        s_n[row_in] = n;
    }
    __syncthreads();
    float zt = 0.f;
    int nt = 0;
    for (int i = 0; i < SUBS; ++i) {
        zt += s_z[i];
        nt += s_n[i];
    }
    const bool whole = gridDim.x == 1;
    const float inv = 1.f / (float)max(nt, 1);
    float dot = 0.f;
    for (int e = tid; e < E; e += BL_THREADS) {
        float s = 0.f;
        for (int i = 0; i < SUBS; ++i) s += s_p[i * LPR * NV + e];
        if (whole) {
            s *= inv;
            o.counts[e] = s_cnt[e];
            o.mean_prob[e] = s;
            dot += (float)s_cnt[e] * (inv / (float)k) * s;
        } else {
            o.part_p[(size_t)blockIdx.x * o.Epad + e] = s;
            o.part_c[(size_t)blockIdx.x * o.Epad + e] = s_cnt[e];
        }
    }
    if (whole) {
        dot = block_sum(dot, s_red, tid, BL_THREADS / 64);
        if (tid == 0) {
            o.loss[0] = (float)E * dot;
            o.loss[1] = zt * inv;
        }
    } else if (tid == 0) {
        o.part_z[blockIdx.x] = zt;
        o.part_n[blockIdx.x] = nt;
    }
}

// Adds the blocks' partial sums in block order within 1024 / Epad strided groups, then the groups.
__global__ __launch_bounds__(1024) void balance_join_kernel(int blocks, int E, int k, BalanceOut o)
{
    __shared__ float s_p[1024];
    __shared__ int s_c[1024];
    __shared__ float s_red[16];
    const int tid = threadIdx.x, Ep = o.Epad, G = 1024 / Ep, e = tid % Ep, g = tid / Ep;
    float s = 0.f;
    int c = 0;
    if (e < E && g < G)
        for (int b = g; b < blocks; b += G) {
            s += o.part_p[(size_t)b * Ep + e];
            c += o.part_c[(size_t)b * Ep + e];
        }
    s_p[tid] = s;
    s_c[tid] = c;
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
            P += s_p[i * Ep + tid];
            cnt += s_c[i * Ep + tid];
        }
        P *= inv;
        o.counts[tid] = cnt;
        o.mean_prob[tid] = P;
        dot = (float)cnt * (inv / (float)k) * P;
    }
    dot = block_sum(dot, s_red, tid, 16);
    if (tid == 0) {
        o.loss[0] = (float)E * dot;
        o.loss[1] = zt * inv;
    }
}

template <int LT, int LPR, int NJ, int VEC>
__global__ __launch_bounds__(BL_THREADS) void balance_grad_kernel(
    const void *__restrict__ logits, int T, int E, const int32_t *__restrict__ idx, int k,
    const uint8_t *__restrict__ mask, const int32_t *__restrict__ counts, const float *__restrict__ d_loss,
    const float *__restrict__ topk_w, const float *__restrict__ d_topk_w, void *__restrict__ d_logits, int gtype)
{
    constexpr int NV = NJ * VEC, SUBS = BL_THREADS / LPR;
    __shared__ int s_id[SUBS][MAX_K];
    __shared__ float s_dw[SUBS][MAX_K];
    const int tid = threadIdx.x, lane = tid & 63, sub = tid % LPR, row_in = tid / LPR;
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
    const bool wpart = topk_w != nullptr;

    for (int tb = blockIdx.x * SUBS; tb < T; tb += gridDim.x * SUBS) {
        const int t = tb + row_in;
        float l[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i) l[i] = -INFINITY;
        const bool on = t < T && (mask == nullptr || mask[t] != 0);
        if (on) load_row<LT, LPR, NJ, VEC>(logits, (size_t)t * E, E, sub, l);
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
            float wd = 0.f;
            for (int j = sub; j < k; j += LPR) {
                const size_t at = (size_t)min(t, T - 1) * k + j;
                wd = none ? 0.f : fmaf(topk_w[at], d_topk_w[at], wd);
            }
            wd = group_sum<LPR>(wd, lane);
            for (int j = sub; j < k; j += LPR) {
                const size_t at = (size_t)min(t, T - 1) * k + j;
                s_id[row_in][j] = clamp_id(idx[at], E);
                s_dw[row_in][j] = none ? 0.f : topk_w[at] * (d_topk_w[at] - wd);
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
    // a block takes 16 KB of logits at a time; fewer blocks leave less to add up afterwards
    const long long values = (long long)T * E;
    const long long b = (values + 4095) / 4096;
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
            constexpr int subs = BL_THREADS / l.value;
            const int want = (T + subs - 1) / subs;
            const int blocks = want < 2048 ? want : 2048;
            balance_grad_kernel<lt.value, l.value, j.value, v.value><<<blocks, BL_THREADS, 0, s>>>(
                logits, T, E, idx, k, mask, counts, d_loss, topk_w, d_topk_w, d_logits, gtype);
            return hipGetLastError();
        });
    });
}

}  // namespace moe
