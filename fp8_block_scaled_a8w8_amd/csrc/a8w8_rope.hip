// a8w8_rope.hip -- what a served decoder block does between its qkv projection and its
// attention, for gfx950: norms of queries and keys for each head, the position rotation,
// and the new keys and values into the paged cache, in one pass.
//
//   x^    = w * x / sqrt(mean(x^2) + eps)               per token and head (optional)
//   theta = positions[axis_of[i], t] * inv_freq[i]      i < R/2
//   (a, b) -> (a cos theta - b sin theta, b cos theta + a sin theta)
//           (a, b) = (x_i, x_{i+R/2}) ("halves") or (x_2i, x_2i+1) ("pairs"); dimensions >= R pass
//
// q is rounded once to bf16; k and v once to the cache's type (e4m3: of value / scale[head],
// saturating at 448).  Bound by memory: 2 bytes in and 1 or 2 out per element.  A lane holds
// eight dimensions of one head (16-byte loads and stores), so a head's norm is a reduction over
// D/8 lanes and a pair of "halves" meets by a lane shuffle.  A workgroup serves heads of one
// token and forms the token's R/2 sines and cosines once, into LDS.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "a8w8_device.h"
#include "a8w8_internal.h"
#include "a8w8_quant_math.h"
#include "gemm_a8w8_blockscale.h"

namespace a8w8 {
namespace kern {

constexpr int kMaxHeadDim = 256;
constexpr int64_t kMaxGroups = 1 << 23;      // workgroups of a launch: a dimension has less than 2^32 threads

struct RopeArgs {
    const uint16_t *q, *k, *v;
    int64_t q_row, q_head, k_row, k_head, v_row, v_head;
    const float *q_weight, *k_weight;
    const int32_t *positions;
    const float *inv_freq;
    const int32_t *axis_of, *slots;
    uint16_t *q_out, *k_out;
    void *k_cache, *v_cache;
    const float *k_scale, *v_scale;
    int64_t T, first, cache_slots;           // first: this launch's first token
    int32_t Hq, Hkv, R, axes, pairs, fp8;
    float eps;
};


// Eight values to e4m3 codes of x / s; NaN keeps its code (the clamp alone would lose it).
__device__ __forceinline__ u32x2 codes8(const float (&x)[8], float s)
{
    float c[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float v = x[i] / s;
        c[i] = v != v ? v : __builtin_amdgcn_fmed3f(v, -448.0f, 448.0f);
    }
    u32x2 r;
    int w = __builtin_amdgcn_cvt_pk_fp8_f32(c[0], c[1], 0, false);
    r[0] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c[2], c[3], w, true);
    w = __builtin_amdgcn_cvt_pk_fp8_f32(c[4], c[5], 0, false);
    r[1] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c[6], c[7], w, true);
    return r;
}

__device__ __forceinline__ u32x4 bf16x8(const float (&x)[8])
{
    u32x4 r;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        r[i] = bf16_rne(x[2 * i]) | (bf16_rne(x[2 * i + 1]) << 16);
    return r;
}

template <int D>
__global__ __launch_bounds__(256) void rope_kernel(RopeArgs p)
{
    constexpr int LPH = D / 8;               // lanes of a head
    __shared__ float cs[kMaxHeadDim];        // cosine, sine of each frequency
    const int64_t t = p.first + blockIdx.x;
    const int half = p.R / 2;
    if ((int)threadIdx.x < half) {
        const int i = threadIdx.x;
        const int a = p.axis_of ? min(max(p.axis_of[i], 0), p.axes - 1) : 0;
        // The angle in turns, in 64 bits: far positions times frequencies near 1 have no
        // exact fp32 product.
        const double turns = (double)p.positions[(int64_t)a * p.T + t] * ((double)p.inv_freq[i] * 0.15915494309189533577);
        float s, c;
        sincospif(2.0f * (float)(turns - rint(turns)), &s, &c);
        cs[2 * i] = c;
        cs[2 * i + 1] = s;
    }
    __syncthreads();
    const int slot = p.slots ? p.slots[t] : -1;
    const bool keep = slot >= 0 && slot < p.cache_slots;
    const int heads = p.Hq + p.Hkv + (p.v_cache ? p.Hkv : 0);
    const int sub = threadIdx.x % LPH;
    const int per = 256 / LPH;               // heads of one trip
    for (int h0 = blockIdx.y * per; h0 < heads; h0 += gridDim.y * per) {
        const int h = h0 + threadIdx.x / LPH;
        if (h >= heads)
            continue;                        // whole heads leave: the shuffles below stay within one
        const int kind = h < p.Hq ? 0 : h < p.Hq + p.Hkv ? 1 : 2;
        const int hh = kind == 0 ? h : kind == 1 ? h - p.Hq : h - p.Hq - p.Hkv;
        const uint16_t *src = kind == 0 ? p.q + t * p.q_row + hh * p.q_head
                            : kind == 1 ? p.k + t * p.k_row + hh * p.k_head : p.v + t * p.v_row + hh * p.v_head;
        const u32x4 raw = *(reinterpret_cast<const u32x4 *>(src) + sub);
        float x[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = bf16_lo(raw[i]);
            x[2 * i + 1] = bf16_hi(raw[i]);
        }
        if (kind != 2) {
            const float *w = kind == 0 ? p.q_weight : p.k_weight;
            if (w) {
                float ss = 0.0f;
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    ss = __builtin_fmaf(x[i], x[i], ss);
#pragma unroll
                for (int m = 1; m < LPH; m *= 2)
                    ss += __shfl_xor(ss, m);
                const float r = 1.0f / sqrtf(ss * (1.0f / D) + p.eps);
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    x[i] = x[i] * r * w[sub * 8 + i];
            }
            if (p.pairs) {
                if (sub * 8 < p.R)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float c = cs[(sub * 4 + i) * 2], s = cs[(sub * 4 + i) * 2 + 1];
                        const float a = x[2 * i], b = x[2 * i + 1];
                        x[2 * i] = __builtin_fmaf(a, c, -b * s);
                        x[2 * i + 1] = __builtin_fmaf(b, c, a * s);
                    }
            } else if (half) {
                const int step = half / 8;   // lanes between a and b
                const bool first = sub < step, turn = sub < 2 * step;
                const int lane = threadIdx.x & 63;
                const int other = turn ? (first ? lane + step : lane - step) : lane;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float o = __shfl(x[i], other);
                    if (turn) {
                        const int f = (first ? sub : sub - step) * 8 + i;
                        const float c = cs[2 * f], s = cs[2 * f + 1];
                        x[i] = __builtin_fmaf(x[i], c, first ? -o * s : o * s);
                    }
                }
            }
        }
        if (kind == 0 || (kind == 1 && p.k_out)) {
            uint16_t *dst = kind == 0 ? p.q_out + (t * p.Hq + hh) * D : p.k_out + (t * p.Hkv + hh) * D;
            *(reinterpret_cast<u32x4 *>(dst) + sub) = bf16x8(x);
        } else if (keep) {
            const int64_t at = ((int64_t)slot * p.Hkv + hh) * LPH + sub;
            void *cache = kind == 1 ? p.k_cache : p.v_cache;
            if (p.fp8) {
                const float *sc = kind == 1 ? p.k_scale : p.v_scale;
                static_cast<u32x2 *>(cache)[at] = codes8(x, sc ? sc[hh] : 1.0f);
            } else {
                static_cast<u32x4 *>(cache)[at] = bf16x8(x);
            }
        }
    }
}

}  // namespace kern

namespace {
bool misaligned(const void *p, uintptr_t mask) { return (reinterpret_cast<uintptr_t>(p) & mask) != 0; }
}  // namespace
}  // namespace a8w8

using namespace a8w8;

extern "C" int a8w8_qk_norm_rope(const a8w8_rope_desc *d, void *stream)
{
    if (!d)
        return A8W8_ERR_NULL;
    const bool cached = d->k_cache || d->v_cache;
    if (d->T < 0 || d->T > (1 << 30) || d->q_heads < 1 || d->kv_heads < 1 || d->q_heads > 1024 || d->kv_heads > 1024 ||
        (d->head_dim != 64 && d->head_dim != 128 && d->head_dim != 256) || d->rotary_dim < 0 || d->rotary_dim > d->head_dim ||
        d->rotary_dim % 16 != 0 || (d->rotary_dim > 0 && (d->axes < 1 || d->axes > 16)) || d->layout < 0 || d->layout > 1 ||
        d->cache_dtype < 0 || d->cache_dtype > 1 || !(d->eps >= 0.0f) ||
        (cached && (d->cache_slots < 1 || d->cache_slots > (1ll << 31) - 1)))
        return A8W8_ERR_SHAPE;
    for (const int64_t s : {d->q_row, d->q_head, d->k_row, d->k_head, cached ? d->v_row : 0, cached ? d->v_head : 0})
        if (s < 0 || s % 8 != 0)
            return A8W8_ERR_SHAPE;
    if (d->T == 0)
        return A8W8_OK;
    if (!d->q || !d->k || !d->q_out || (cached ? (!d->k_cache || !d->v_cache || !d->v || !d->slots || d->k_out != nullptr) : !d->k_out) ||
        (d->rotary_dim > 0 && (!d->positions || !d->inv_freq)))
        return A8W8_ERR_NULL;
    const uintptr_t cache_mask = d->cache_dtype == A8W8_CACHE_E4M3 ? 7 : 15;
    if (misaligned(d->q, 15) || misaligned(d->k, 15) || misaligned(d->v, 15) || misaligned(d->q_out, 15) || misaligned(d->k_out, 15) ||
        misaligned(d->k_cache, cache_mask) || misaligned(d->v_cache, cache_mask) || misaligned(d->q_weight, 3) ||
        misaligned(d->k_weight, 3) || misaligned(d->positions, 3) || misaligned(d->inv_freq, 3) || misaligned(d->axis_of, 3) ||
        misaligned(d->slots, 3) || misaligned(d->k_scale, 3) || misaligned(d->v_scale, 3))
        return A8W8_ERR_ALIGN;
    int cus = 0;
    const int rc = device_ready(&cus);
    if (rc != A8W8_OK)
        return rc;
    kern::RopeArgs a;
    a.q = static_cast<const uint16_t *>(d->q);
    a.k = static_cast<const uint16_t *>(d->k);
    a.v = static_cast<const uint16_t *>(d->v);
    a.q_row = d->q_row, a.q_head = d->q_head, a.k_row = d->k_row, a.k_head = d->k_head, a.v_row = d->v_row, a.v_head = d->v_head;
    a.q_weight = d->q_weight, a.k_weight = d->k_weight;
    a.positions = d->positions, a.inv_freq = d->inv_freq, a.axis_of = d->axis_of, a.slots = d->slots;
    a.q_out = static_cast<uint16_t *>(d->q_out), a.k_out = static_cast<uint16_t *>(d->k_out);
    a.k_cache = d->k_cache, a.v_cache = d->v_cache, a.k_scale = d->k_scale, a.v_scale = d->v_scale;
    a.T = d->T, a.cache_slots = d->cache_slots;
    a.Hq = d->q_heads, a.Hkv = d->kv_heads, a.R = d->rotary_dim, a.axes = d->axes, a.pairs = d->layout == A8W8_ROPE_PAIRS;
    a.fp8 = d->cache_dtype == A8W8_CACHE_E4M3;
    a.eps = d->eps;
    const auto f = d->head_dim == 64 ? kern::rope_kernel<64> : d->head_dim == 128 ? kern::rope_kernel<128> : kern::rope_kernel<256>;
    // Few tokens: a workgroup takes one trip of a token's heads (one token of 24 gated heads of 256: 3.5 us replayed, against
    // 6.7 in one workgroup).  Many: one workgroup per token, which forms the angles once (8191 tokens: 64 us; a
    // workgroup per trip 78, several tokens a workgroup 89 and more, with fewer bytes in flight).
    const int per = 256 * 8 / d->head_dim, trips = (d->q_heads + (cached ? 2 : 1) * d->kv_heads + per - 1) / per;
    for (a.first = 0; a.first < d->T; a.first += kern::kMaxGroups) {
        const int64_t groups = d->T - a.first < kern::kMaxGroups ? d->T - a.first : kern::kMaxGroups;
        hipLaunchKernelGGL(f, dim3((unsigned)groups, (unsigned)(d->T <= 256 ? trips : 1)), dim3(256), 0, static_cast<hipStream_t>(stream), a);
        if (hipGetLastError() != hipSuccess)
            return A8W8_ERR_HIP;
    }
    return A8W8_OK;
}
