// a8w8_moe.hip -- expert routing and a whole mixture-of-experts layer for a few
// tokens on fp8 block-scaled expert weights, for gfx950.
//
//   routing   ids[t, 0..k) = the k experts of the largest logits of token t, best
//             first, ties to the lowest index; a logit of -inf or NaN masks its
//             expert (+inf counts as the largest finite value); slots left without
//             an expert get id -1 and weight 0.  Weights: softmax over the row or
//             sigmoid of the chosen logits, optionally divided by their sum, times
//             a constant.
//   layer     h[t,j] = silu(W13[e] gate . x_t) * (W13[e] up . x_t)      e = ids[t,j]
//             Y[t]   = bf16( sum_j w[t,j] * W2[e] . h[t,j] )
//
// with x bf16 and W13 [E, 2I, H] (gate rows, then up rows), W2 [E, H, I] e4m3fn with
// one fp32 scale per 128 x 128 block.  For a few tokens the layer is bound by the
// bytes of the experts' weights, so the activations stay bf16 (quantising them
// would save nothing and cost accuracy): a weight fragment is widened in registers
// to bf16, which is exact, and multiplied with v_mfma_f32_16x16x32_bf16; a K block's
// fp32 dot is then scaled into the fp32 accumulator, as in the GEMM kernels.  h is carried
// as two bf16 terms where experts have few slots, else as one.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <atomic>
#include <cmath>

#include "a8w8_device.h"
#include "a8w8_internal.h"
#include "gemm_a8w8_blockscale.h"

namespace a8w8 {
namespace kern {

// Wave-uniform read-only data through the constant address space: scalar loads.
typedef const __attribute__((address_space(4))) int32_t const_i32;
typedef int i4 __attribute__((ext_vector_type(4)));
typedef const __attribute__((address_space(4))) i4 const_i4;

typedef __bf16 v2b __attribute__((ext_vector_type(2)));

constexpr int kMaxTopk = 16;       // experts per token
constexpr int kMaxExperts = 1024;  // one workgroup's thread per expert
constexpr int kChunk = 256;        // tokens of one pass (the plan below and the down kernel's LDS)
// Beyond any buffer here: loads return zeros, no traffic.  (As a vector offset: the bounds check
// may leave the scalar offset out, so a load that is to read nothing must not depend on that one.)
constexpr uint32_t kOob = 0x7ffff000u;
constexpr int kHiddenPad = 1024;   // bytes of the workspace behind the hidden rows

struct RouteArgs {
    const void *logits;   // [T, E] fp32 or bf16
    float *weights;       // [T, k]
    int32_t *ids;         // [T, k]
    int64_t T;
    int32_t E, k, bf16, sigmoid, renorm;
    float scale;
};

// One chunk's plan: the reached experts {expert, first slot, slots, 0} in ascending order,
// and the slots' tokens and weights, grouped by expert in token order.
struct MoePlan {
    int32_t experts, slots, pad[14];
    int4 expert[kMaxExperts];
    int32_t token[kChunk * kMaxTopk];
    float weight[kChunk * kMaxTopk];
    // Routing as the workgroups that route leave it for the one that plans: [token][slot].
    int32_t routed_id[kChunk * kMaxTopk];
    float routed_weight[kChunk * kMaxTopk];
    int32_t place[kChunk * kMaxTopk];      // [token][slot]: its place among the slots, -1: none
};

struct MoeArgs {
    const uint16_t *X;    // bf16 [T, H]
    const uint8_t *W13;   // e4m3fn [E, 2I, H]
    const float *s13;     // [E, 2I/128, H/128]
    const uint8_t *W2;    // e4m3fn [E, H, I]
    const float *s2;      // [E, H/128, I/128]
    uint16_t *Y;          // bf16 [T, H]
    MoePlan *plan;        // (the up product writes it when it routes itself)
    uint16_t *h;          // bf16 [slots, I]; where lo is not 0, the second terms lo elements behind
    uint32_t lo;
    float *part;          // down product with splits: [H/16][splits][T][16]
    int32_t *cnt;         // one zeroed counter per 16 output columns
    int32_t T, H, I, E, splits, vec_store;
    RouteArgs route;
};

// ---------------------------------------------------------------------------
// Routing.  One wave per token; lane l holds the logits of experts l, l + 64, ...
// (VPL of them).
//
// Bound by instructions, so: the logits are compared as unsigned integers of the same order (a
// float's bits, inverted if negative, else with the sign bit set), whose maximum takes its DPP
// operand directly; each lane sorts its logits once, so that its best one is always the first;
// and taking an expert shifts one lane's list.  One token, 256 experts, top 8: 3.2 us.

constexpr uint32_t kMasked = 0u;

__device__ __forceinline__ uint32_t order_of(float x)
{
    const uint32_t b = __float_as_uint(x + 0.0f);  // (-0 becomes +0)
    return b ^ ((uint32_t)((int)b >> 31) | 0x80000000u);
}
// NaN masks its expert; +inf is the largest finite value.
__device__ __forceinline__ uint32_t key_of(float x)
{
    return x > -INFINITY ? order_of(fminf(x, 3.402823466e38f)) : kMasked;
}
__device__ __forceinline__ float value_of(uint32_t k)
{
    return __uint_as_float(k ^ ((uint32_t)((int)~k >> 31) | 0x80000000u));
}

__device__ __forceinline__ uint32_t max_u32(uint32_t a, uint32_t b) { return a > b ? a : b; }
template <int CTRL>
__device__ __forceinline__ uint32_t dpp_max(uint32_t x)   // lanes without a source: 0, the smallest
{
    return max_u32(x, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, CTRL, 0xF, 0xF, false));
}
// Maximum over the wave, in every lane: within the four rows of 16 lanes, then of their last lanes.
__device__ __forceinline__ uint32_t wave_max(uint32_t x)
{
    x = dpp_max<0x111>(x);
    x = dpp_max<0x112>(x);
    x = dpp_max<0x114>(x);
    x = dpp_max<0x118>(x);
    const uint32_t a = (uint32_t)__builtin_amdgcn_readlane((int)x, 15), b = (uint32_t)__builtin_amdgcn_readlane((int)x, 31);
    const uint32_t c = (uint32_t)__builtin_amdgcn_readlane((int)x, 47), d = (uint32_t)__builtin_amdgcn_readlane((int)x, 63);
    return max_u32(max_u32(a, b), max_u32(c, d));
}
// One DPP step of a sum: lanes without a source add nothing.
template <int CTRL, int ROWS>
__device__ __forceinline__ float dpp_add(float x)
{
    return x + __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), CTRL, ROWS, 0xF, false));
}
// Sum over the wave in a fixed order, in every lane.
__device__ __forceinline__ float wave_sum(float x)
{
    x = dpp_add<0x111, 0xF>(x);
    x = dpp_add<0x112, 0xF>(x);
    x = dpp_add<0x114, 0xF>(x);
    x = dpp_add<0x118, 0xF>(x);
    x = dpp_add<0x142, 0xA>(x);
    x = dpp_add<0x143, 0xC>(x);
    return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(x), 63));
}

template <int VPL>
__device__ __forceinline__ void load_logits(const RouteArgs &p, int64_t t, int lane, uint32_t (&v)[VPL])
{
    float x[VPL];
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
        const int e = i * 64 + lane;
        x[i] = -INFINITY;
        if (e < p.E) {
            if (p.bf16)
                x[i] = __uint_as_float((uint32_t)static_cast<const uint16_t *>(p.logits)[t * p.E + e] << 16);
            else
                x[i] = static_cast<const float *>(p.logits)[t * p.E + e];
        }
    }
#pragma unroll
    for (int i = 0; i < VPL; ++i)
        v[i] = key_of(x[i]);
}

// One logit's part of the softmax's sum.  (The hardware's exponential: the argument's rounding,
// 2^-24 of it, falls on terms that are e^argument.)
__device__ __forceinline__ float softmax_term(uint32_t key, float top_value)
{
    return __builtin_amdgcn_exp2f((value_of(key) - top_value) * 1.44269504088896340736f);
}

// A chosen logit's weight before it is divided.  Sigmoids that are to be divided by their sum:
// below 0, sigmoid(v) = exp(v) / (1 + exp(v)), and exp(top) cancels, so the quotients hold where
// every sigmoid itself would underflow.
__device__ __forceinline__ float slot_weight(const RouteArgs &p, uint32_t key, float top_value, bool chosen)
{
    const float x = value_of(key);
    return !chosen       ? 0.f
           : !p.sigmoid  ? expf(x - top_value)
           : p.renorm && top_value < 0.f ? expf(x - top_value) / (1.0f + expf(x))
                                         : 1.0f / (1.0f + expf(-x));
}

// The token's routing: lane j < k returns slot j's weight and expert.
template <int VPL>
__device__ __forceinline__ void route_row(const RouteArgs &p, uint32_t (&v)[VPL], int lane, float &w, int &id)
{
    // The lane's logits in descending order, equal ones in their own (neighbours swap only if
    // strictly out of order), with their places i (expert i * 64 + lane).
    int at[VPL];
#pragma unroll
    for (int i = 0; i < VPL; ++i)
        at[i] = i;
#pragma unroll
    for (int n = VPL - 1; n > 0; --n)
#pragma unroll
        for (int i = 0; i < n; ++i) {
            const bool swap = v[i + 1] > v[i];
            const uint32_t a = v[i], b = v[i + 1];
            const int c = at[i], d = at[i + 1];
            v[i] = swap ? b : a;
            v[i + 1] = swap ? a : b;
            at[i] = swap ? d : c;
            at[i + 1] = swap ? c : d;
        }
    uint32_t m = wave_max(v[0]);
    const float top_value = value_of(m);
    float all = 0.f;
    if (!p.sigmoid && !p.renorm && m != kMasked) {
#pragma unroll
        for (int i = 0; i < VPL; ++i)
            all += v[i] != kMasked ? softmax_term(v[i], top_value) : 0.f;
        all = wave_sum(all);
    }
    uint32_t val = kMasked;
    id = -1;
    for (int j = 0; j < p.k; ++j) {
        if (m == kMasked)
            break;
        // The lowest expert with the largest logit left: one lane's, or the lowest of several lanes'.
        uint64_t lanes = __ballot(v[0] == m);
        int l = __builtin_ctzll(lanes), e = __builtin_amdgcn_readlane(at[0], l) * 64 + l;
        for (lanes &= lanes - 1; lanes != 0; lanes &= lanes - 1) {
            const int l2 = __builtin_ctzll(lanes), e2 = __builtin_amdgcn_readlane(at[0], l2) * 64 + l2;
            l = e2 < e ? l2 : l;
            e = e2 < e ? e2 : e;
        }
        val = lane == j ? m : val;
        id = lane == j ? e : id;
        const bool mine = lane == l;
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
            v[i] = mine ? (i + 1 < VPL ? v[i + 1 < VPL ? i + 1 : i] : kMasked) : v[i];
            if (i + 1 < VPL)
                at[i] = mine ? at[i + 1 < VPL ? i + 1 : i] : at[i];
        }
        m = wave_max(v[0]);
    }
    w = slot_weight(p, val, top_value, id >= 0);
    const float total = p.renorm ? wave_sum(w) : p.sigmoid ? 1.0f : all;
    w = total > 0.f ? w / total * p.scale : 0.f;
}

template <int VPL>
__device__ __forceinline__ void route_token(const RouteArgs &p, int64_t t, int lane)
{
    uint32_t v[VPL];
    float w;
    int id;
    load_logits<VPL>(p, t, lane, v);
    route_row<VPL>(p, v, lane, w, id);
    if (lane < p.k) {
        p.weights[t * p.k + lane] = w;
        p.ids[t * p.k + lane] = id;
    }
}

template <int VPL>
__global__ __launch_bounds__(256) void route_kernel(RouteArgs p)
{
    const int lane = threadIdx.x & 63;
    const int64_t step = (int64_t)gridDim.x * 4;
    for (int64_t t = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); t < p.T; t += step)
        route_token<VPL>(p, t, lane);
}

// Routing many tokens to up to 8 of 256 experts each: sixteen lanes per token, four tokens a wave,
// lane l holding the logits of experts l, l + 16, ... (V of them).  The k-th largest of the 16
// lanes' largest logits cannot be above the k-th largest logit, so the logits from there on
// hold the chosen ones: 10.6 of them on average for random logits and k = 8.  They are gathered
// in LDS, one or two to a lane, and each counts the better ones, which is its slot.  A token with
// more than 32 of them (equal logits, mostly) is routed by the whole wave as above.  About 120
// instructions a token against 480.  Bound by them and by its narrow loads, one logit to a lane, which
// nothing overlaps with the ranking; not by bytes: 16381 tokens, 256 experts, top 8 take 8.7 us (2.0 TB/s),
// with bf16 logits 8.6, with 128 experts 5.8.  A wave per token: 15.6; with fewer tokens a wave's own
// time counts, which is the longer one here (4096 tokens: 5.0 against 5.5 us, 2048: 4.9 against 4.2).
// (Replayed graphs of 30 calls, a launch's 1-2 us each included.)
template <int D>
__device__ __forceinline__ uint32_t ror(uint32_t x)   // of the lane's row of 16
{
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x120 + D, 0xF, 0xF, false);
}
template <int LANE>
__device__ __forceinline__ uint32_t row_lane(uint32_t x)
{
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x150 + LANE, 0xF, 0xF, false);
}
// How many of the row's other lanes hold more.
template <int D = 1>
__device__ __forceinline__ int row_rank(uint32_t x)
{
    if constexpr (D == 16)
        return 0;
    else
        return (ror<D>(x) > x ? 1 : 0) + row_rank<D + 1>(x);
}
// How many of the row's lanes hold a better (key, expert) than `c` in `o`.
template <int D = 0>
__device__ __forceinline__ int row_better(uint2 o, uint2 c)
{
    if constexpr (D == 16) {
        return 0;
    } else {
        const uint32_t k = D > 0 ? ror<D>(o.x) : o.x, e = D > 0 ? ror<D>(o.y) : o.y;
        return (((uint64_t)k << 32 | (uint32_t)~e) > ((uint64_t)c.x << 32 | (uint32_t)~c.y) ? 1 : 0) + row_better<D + 1>(o, c);
    }
}
// Sum over the lane's row, in the order of wave_sum.
__device__ __forceinline__ float row_sum(float x)
{
    x = dpp_add<0x111, 0xF>(x);
    x = dpp_add<0x112, 0xF>(x);
    x = dpp_add<0x114, 0xF>(x);
    x = dpp_add<0x118, 0xF>(x);
    return __uint_as_float(row_lane<15>(__float_as_uint(x)));
}

constexpr int kRowTopk = 8, kRowExperts = 256, kRowTokens = 4096, kRowList = 32;

template <int V>
__global__ __launch_bounds__(256) void route_rows_kernel(RouteArgs p)
{
    __shared__ uint2 list[16][kRowList + 1];       // per token: key and expert (the last one: of no use)
    const int lane = threadIdx.x & 63, l16 = lane & 15;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    uint2 *mine = list[wave * 4 + (lane >> 4)];
    for (int64_t t0 = ((int64_t)blockIdx.x * 4 + wave) * 4; t0 < p.T; t0 += (int64_t)gridDim.x * 16) {
        const int64_t t = t0 + (lane >> 4);
        const bool live = t < p.T;
        uint32_t key[V];
        {
            float x[V];
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const int e = i * 16 + l16;
                x[i] = -INFINITY;
                if (live && e < p.E) {
                    if (p.bf16)
                        x[i] = __uint_as_float((uint32_t)static_cast<const uint16_t *>(p.logits)[t * p.E + e] << 16);
                    else
                        x[i] = static_cast<const float *>(p.logits)[t * p.E + e];
                }
            }
#pragma unroll
            for (int i = 0; i < V; ++i)
                key[i] = key_of(x[i]);
        }
        uint32_t m = key[0];
#pragma unroll
        for (int i = 1; i < V; ++i)
            m = max_u32(m, key[i]);
        uint32_t from = row_rank(m) < p.k ? m : 0xffffffffu;
        from = min(from, ror<8>(from));
        from = min(from, ror<4>(from));
        from = min(from, ror<2>(from));
        from = max_u32(min(from, ror<1>(from)), kMasked + 1u);
        int count = 0;
#pragma unroll
        for (int i = 0; i < V; ++i)
            count += key[i] >= from ? 1 : 0;
        int upto = count;
        upto += __builtin_amdgcn_update_dpp(0, upto, 0x111, 0xF, 0xF, false);
        upto += __builtin_amdgcn_update_dpp(0, upto, 0x112, 0xF, 0xF, false);
        upto += __builtin_amdgcn_update_dpp(0, upto, 0x114, 0xF, 0xF, false);
        upto += __builtin_amdgcn_update_dpp(0, upto, 0x118, 0xF, 0xF, false);
        const int total = (int)row_lane<15>((uint32_t)upto);
        int at = upto - count;
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (key[i] >= from) {
                mine[min(at, kRowList)] = make_uint2(key[i], (uint32_t)(i * 16 + l16));
                ++at;
            }
        __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
        __builtin_amdgcn_wave_barrier();
        const uint2 none = make_uint2(kMasked, 0xffffffffu);
        const uint2 c = l16 < total ? mine[l16] : none;
        int place = row_better(c, c);
        const bool more = __ballot(total > 16) != 0;
        if (more) {                                // a second one to each lane
            const uint2 d = l16 + 16 < total ? mine[min(l16 + 16, kRowList)] : none;
            place += row_better(d, c);
            const int place2 = row_better(d, d) + row_better(c, d);
            __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
            __builtin_amdgcn_wave_barrier();
            if (l16 + 16 < total)
                mine[place2] = d;
        }
        __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
        __builtin_amdgcn_wave_barrier();
        if (l16 < total)
            mine[place] = c;
        __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
        __builtin_amdgcn_wave_barrier();
        const bool chosen = l16 < min(total, p.k);
        const uint2 slot = chosen ? mine[l16] : none;
        const float top_value = value_of(row_lane<0>(slot.x));
        float all = 0.f;
        if (!p.sigmoid && !p.renorm) {
#pragma unroll
            for (int i = 0; i < V; ++i)
                all += key[i] != kMasked ? softmax_term(key[i], top_value) : 0.f;
            all = row_sum(all);
        }
        const float w = slot_weight(p, slot.x, top_value, chosen);
        const float total_w = p.renorm ? row_sum(w) : p.sigmoid ? 1.0f : all;
        if (live && total <= kRowList && l16 < p.k) {
            p.weights[t * p.k + l16] = total_w > 0.f ? w / total_w * p.scale : 0.f;
            p.ids[t * p.k + l16] = (int)slot.y;
        }
        for (uint64_t over = __ballot(live && total > kRowList && l16 == 0); over != 0; over &= over - 1)
            route_token<V / 4>(p, t0 + (__builtin_ctzll(over) >> 4), lane);
    }
}

// ---------------------------------------------------------------------------
// The layer's plan for one chunk of at most kChunk tokens: the experts that any
// token reached, and their slots (token, weight), grouped by expert in token order.

// Sixteen tokens per workgroup, one wave each; the last workgroup to finish (the only one,
// for up to 16 tokens) makes the plan from everyone's routing.  There a bitmap of tokens
// per expert gives every slot its place by counting, so the order is fixed whatever the
// order the waves run in.  256 tokens: 9.9 us against 52 us with one workgroup routing them
// all, sixteen tokens to a wave.
template <int VPL>
__global__ __launch_bounds__(1024) void moe_plan_kernel(RouteArgs p, MoePlan *plan, int32_t *cnt_done)
{
    __shared__ uint32_t mask[kMaxExperts][kChunk / 32];
    __shared__ int16_t s_id[kChunk * kMaxTopk];
    __shared__ int16_t s_off[kMaxExperts];
    __shared__ uint32_t s_wave[16];
    __shared__ int last;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int T = (int)p.T, E = p.E, k = p.k;
    const int t = (int)blockIdx.x * 16 + wave;
    if (t < T) {
        uint32_t v[VPL];
        float w;
        int id;
        load_logits<VPL>(p, t, lane, v);
        route_row<VPL>(p, v, lane, w, id);
        if (lane < k) {      // device-coherent: another XCD's workgroup may make the plan
            __hip_atomic_store(&plan->routed_id[t * k + lane], id, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            __hip_atomic_store(&plan->routed_weight[t * k + lane], w, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        }
    }
    for (int i = tid; i < E * (kChunk / 32); i += 1024)
        (&mask[0][0])[i] = 0u;
    wait_vmcnt<0>();                               // this wave's routing is out
    __syncthreads();                               // ... and every wave's
    if (gridDim.x > 1) {
        if (tid == 0)
            last = __hip_atomic_fetch_add(cnt_done, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == (int)gridDim.x - 1;
        __syncthreads();
        if (!last)
            return;
        if (tid == 0)
            __hip_atomic_store(cnt_done, 0, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
    float w[kChunk * kMaxTopk / 1024];
#pragma unroll
    for (int q = 0; q < kChunk * kMaxTopk / 1024; ++q) {
        const int i = tid + q * 1024;
        if (i < T * k) {
            const int id = __hip_atomic_load(&plan->routed_id[i], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            w[q] = __hip_atomic_load(&plan->routed_weight[i], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            s_id[i] = (int16_t)id;
            const int tok = i / k;
            if (id >= 0)
                atomicOr(&mask[id][tok >> 5], 1u << (tok & 31));
        }
    }
    __syncthreads();
    // Exclusive scan over the experts of (slots, reached) packed as 16 + 16 bits.
    int cnt = 0;
    if (tid < E) {
#pragma unroll
        for (int i = 0; i < kChunk / 32; ++i)
            cnt += __popc(mask[tid][i]);
    }
    const uint32_t mine = (uint32_t)cnt | (cnt > 0 ? 0x10000u : 0u);
    uint32_t sum = mine;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const uint32_t o = __shfl_up(sum, d);
        if (lane >= d)
            sum += o;
    }
    if (lane == 63)
        s_wave[wave] = sum;
    __syncthreads();
    uint32_t before = 0;
    for (int i = 0; i < wave; ++i)
        before += s_wave[i];
    const uint32_t at = before + sum - mine;
    if (cnt > 0) {
        const int4 a = {tid, (int)(at & 0xffffu), cnt, 0};
        plan->expert[at >> 16] = a;
        s_off[tid] = (int16_t)(at & 0xffffu);
    }
    if (tid == 1023) {
        plan->experts = (int)((before + sum) >> 16);
        plan->slots = (int)((before + sum) & 0xffffu);
    }
    __syncthreads();
#pragma unroll
    for (int q = 0; q < kChunk * kMaxTopk / 1024; ++q) {
        const int i = tid + q * 1024;
        const int id = i < T * k ? s_id[i] : -1;
        int pos = -1;
        if (id >= 0) {
            const int tok = i / k;
            pos = s_off[id] + __popc(mask[id][tok >> 5] & ((1u << (tok & 31)) - 1u));
            for (int b = 0; b < (tok >> 5); ++b)
                pos += __popc(mask[id][b]);
            plan->token[pos] = tok;
            plan->weight[pos] = w[q];
        }
        if (i < T * k)
            plan->place[i] = pos;
    }
}

// ---------------------------------------------------------------------------
// Products.

// Eight e4m3 codes (two words) as eight bf16, exactly.
__device__ __forceinline__ v8b widen8(int lo, int hi)
{
    const v2b a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((uint32_t)lo, 1.0f, false);
    const v2b b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((uint32_t)lo, 1.0f, true);
    const v2b c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((uint32_t)hi, 1.0f, false);
    const v2b d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((uint32_t)hi, 1.0f, true);
    return (v8b){a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

// A 16 x 128 weight fragment widened: lane l holds row l % 16; part q < 2 its columns
// 16 g + 8 q .. + 8, part q >= 2 its columns 64 + 16 g + 8 (q - 2) .. + 8, g = l / 16.
struct Wide {
    v8b part[4];
};
__device__ __forceinline__ Wide widen(v8i w)
{
    return {{widen8(w[0], w[1]), widen8(w[2], w[3]), widen8(w[4], w[5]), widen8(w[6], w[7])}};
}

// The 16 x 16 dot of a widened weight block with an activation block in the same K order
// (x[q]: eight bf16): lane l returns D[4 (l / 16) + i][l % 16].
__device__ __forceinline__ v4f block_dot(const Wide &w, const v4i (&x)[4])
{
    v4f d = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int q = 0; q < 4; ++q)
        d = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w.part[q], __builtin_bit_cast(v8b, x[q]), d, 0, 0, 0);
    return d;
}

// Byte offset of lane's load h (0, 1) of 16-row tile `tile` within an expert's weights, block 0:
// row-major loads take whole 128-byte lines (rows 0-7, then 8-15); packed ones two kilobytes.
template <bool PK>
__device__ __forceinline__ uint32_t tile_offset(uint32_t tile, int h, int lane, uint32_t K)
{
    if (PK)
        return packed_block(tile, 0u, K >> 7) + (uint32_t)(lane * 16 + h * 1024);
    const int r16 = lane & 15, g = lane >> 4;
    return (tile * 16 + 8 * h + (r16 & 7)) * K + (uint32_t)(g + 4 * (r16 >> 3)) * 16;
}

// Byte offsets of an activation row's four 16-byte parts of a block, from 32 g.
__device__ constexpr int part_offset(int q) { return (q & 1) * 16 + (q >> 1) * 128; }

// The product of one expert's weight rows with its slots.  Workgroup (a, c): expert a of the
// plan and 2 NT 16-row tiles.  Its NW waves take runs of D K blocks in turn; a pass serves NG
// groups of 16 slots (a further pass reads the expert's weights again, from the caches).  The
// wave partials are summed through LDS in wave order.
//
// Up product: NT tiles of gate rows from 16 NT c on and the same of up rows; h = silu(gate) *
// up goes to the down product as two bf16 terms or one, the type of its matrix instructions (see there).
// Bound by the weights' bytes (61 tokens, 256 experts of 512 x 2048: 75 us, 6.1 TB/s); with
// 16 slots per expert by the activations' as well, which a workgroup of NT = 4 reads half as
// often as one of NT = 2 (256 tokens, 128 experts of 768 x 2048: 78 us; a call with both products on
// NT = 4 takes 140, on NT = 2 148).
//
// DOWN, for many slots per expert: 2 NT neighbouring tiles of W2's rows on the slots' h; the
// products stay fp32, each slot's times its routing weight, and moe_combine_kernel adds a
// token's.  Bound like the up product (the same 256 tokens: 48 us, 4.2 TB/s, and 5 us for the
// sums; a call with the products for few slots instead, whose every down workgroup reads all hidden rows
// and keeps sums per token that leave room for four waves on a CU, takes 222 us).
//
// FUSED (up to 64 slots, 8 tokens and 256 experts): every workgroup routes the tokens
// itself, a wave a token, and finds its expert in a bitmap; workgroup 0 leaves the plan for
// the down product.  That saves the plan kernel's launch, 5 us of a one-token layer's 21.
constexpr int kFusedSlots = 64, kFusedTokens = 8, kFusedExperts = 256;

// What a workgroup needs to know of its expert; lane l's token of slot s comes from token().
struct UpExpert {
    int e, off, cnt;
    int tokens;               // FUSED: lane s holds slot s's token
};

// Routes the tokens and finds the workgroup's expert; e = -1: fewer than a + 1 are reached.
template <int NW>
__device__ __forceinline__ UpExpert fused_plan(const RouteArgs &r, MoePlan *plan, int a)
{
    __shared__ int s_id[kFusedSlots];
    __shared__ float s_w[kFusedSlots];
    __shared__ uint32_t s_map[kFusedExperts / 32];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int T = (int)r.T, k = r.k, n = T * k;
    constexpr int VPL = kFusedExperts / 64;
    uint32_t v[VPL];
    float w;
    int id;
    if (wave < T)
        load_logits<VPL>(r, wave, lane, v);
    if (threadIdx.x < kFusedExperts / 32)
        s_map[threadIdx.x] = 0u;
    __syncthreads();
    for (int t = wave; t < T; t += NW) {
        if (t >= NW)
            load_logits<VPL>(r, t, lane, v);
        route_row<VPL>(r, v, lane, w, id);
        if (lane < k) {
            s_id[t * k + lane] = id;
            s_w[t * k + lane] = w;
            if (id >= 0)
                atomicOr(&s_map[id >> 5], 1u << (id & 31));
        }
    }
    __syncthreads();
    // The a-th reached expert, in ascending order.
    const uint32_t word = lane < kFusedExperts / 32 ? s_map[lane] : 0u;
    int upto = __popc(word);
#pragma unroll
    for (int d = 1; d < kFusedExperts / 32; d <<= 1) {
        const int o = __shfl_up(upto, d);
        if (lane >= d)
            upto += o;
    }
    const int before = upto - __popc(word), reached = __builtin_amdgcn_readlane(upto, kFusedExperts / 32 - 1);
    id = lane < n ? s_id[lane] : -1;
    if (blockIdx.x == 0 && wave == 0) {
        // The plan: each slot's place is the slots of lower experts and the earlier ones of its own.
        int less = 0, same = 0, rank = 0;
        for (int i = 0; i < n; ++i) {
            const int o = __builtin_amdgcn_readlane(id, i);
            less += o >= 0 && o < id ? 1 : 0;
            same += o == id && i < lane ? 1 : 0;
        }
        const uint64_t live = __ballot(id >= 0), firsts = __ballot(id >= 0 && same == 0);
        for (int i = 0; i < n; ++i)
            rank += (firsts >> i & 1) != 0 && __builtin_amdgcn_readlane(id, i) < id ? 1 : 0;
        int cnt = 0;
        for (int i = 0; i < n; ++i)
            cnt += __builtin_amdgcn_readlane(id, i) == id ? 1 : 0;
        if (id >= 0) {
            plan->token[less + same] = lane / k;
            plan->weight[less + same] = s_w[lane];
            if (same == 0)
                plan->expert[rank] = make_int4(id, less, cnt, 0);
        }
        if (lane == 0) {
            plan->experts = reached;
            plan->slots = __builtin_popcountll(live);
        }
    }
    UpExpert x = {-1, 0, 0, 0};
    if (a >= reached)
        return x;
    const int l = __builtin_ctzll(__ballot(lane < kFusedExperts / 32 && before <= a && a < upto));
    uint32_t bits = (uint32_t)__builtin_amdgcn_readlane((int)word, l);
    for (int i = a - __builtin_amdgcn_readlane(before, l); i > 0; --i)
        bits &= bits - 1;
    x.e = 32 * l + __builtin_ctz(bits);
    const uint64_t mine = __ballot(id == x.e);
    x.off = __builtin_popcountll(__ballot(id >= 0 && id < x.e));
    x.cnt = __builtin_popcountll(mine);
    // Slot s's token to lane s (an expert holds a token once: at most kFusedTokens slots).
    const int pos = __builtin_amdgcn_mbcnt_hi((uint32_t)(mine >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)mine, 0));
    x.tokens = __builtin_amdgcn_ds_permute(4 * (id == x.e ? pos : 63), lane / k);
    return x;
}

template <int D, int NW, int NG, int NT, bool FUSED, bool DOWN, bool PK>
__device__ __forceinline__ void expert_rows(const MoeArgs &p)
{
    __shared__ v4f red[NW][2 * NG * NT][64];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int CB = DOWN ? p.H / (32 * NT) : p.I / (16 * NT), a = (int)blockIdx.x / CB, c = (int)blockIdx.x - a * CB;
    UpExpert ex;
    if constexpr (FUSED) {
        ex = fused_plan<NW>(p.route, p.plan, a);
        if (ex.e < 0)
            return;
    } else {
        if (a >= ((const_i32 *)p.plan)[0])
            return;
        const i4 x = ((const_i4 *)p.plan->expert)[a];
        ex = {x[0], x[1], x[2], 0};
    }
    const int e = ex.e, off = ex.off, cnt = ex.cnt;
    const int K = DOWN ? p.I : p.H, N = DOWN ? p.H : 2 * p.I, KB = K >> 7;
    const int r16 = lane & 15, g = lane >> 4;
    const uint32_t wbytes = (uint32_t)N * (uint32_t)K;
    const uint8_t *W = (DOWN ? p.W2 : p.W13) + (size_t)e * wbytes;
    const __amdgpu_buffer_rsrc_t wres = buffer_rsrc(W, wbytes), none = buffer_rsrc(W, 0u);
    const __amdgpu_buffer_rsrc_t xres = DOWN ? buffer_rsrc(p.h + (size_t)off * K, (uint32_t)cnt * (uint32_t)K * 2u)
                                             : buffer_rsrc(p.X, (uint32_t)p.T * (uint32_t)K * 2u);
    // The first tile of either half: DOWN neighbours, else of the gate's and of the up rows.
    const int first = DOWN ? c * 2 * NT : c * NT, second = DOWN ? first + NT : (N >> 5) + first;
    const_f32 *scales = (const_f32 *)((DOWN ? p.s2 : p.s13) + (size_t)e * (N >> 7) * KB);
    const_f32 *sg = scales + (size_t)(first >> 3) * KB, *su = scales + (size_t)(second >> 3) * KB;
    uint32_t woff[2 * NT][2];
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            woff[t][h] = tile_offset<PK>((uint32_t)(first + t), h, lane, (uint32_t)K);
            woff[NT + t][h] = tile_offset<PK>((uint32_t)(second + t), h, lane, (uint32_t)K);
        }
    for (int s0 = 16 * NG * (int)blockIdx.y; s0 < cnt; s0 += 16 * NG * (int)gridDim.y) {
        uint32_t xoff[NG];
#pragma unroll
        for (int n = 0; n < NG; ++n) {
            const int s = s0 + 16 * n + r16;
            int t = 0;
            if constexpr (FUSED)
                t = __builtin_amdgcn_ds_bpermute(4 * s, ex.tokens);
            else if constexpr (DOWN)
                t = s;
            else if (s < cnt)
                t = p.plan->token[off + s];
            xoff[n] = s < cnt ? (uint32_t)t * (uint32_t)K * 2u + 32u * (uint32_t)g : kOob;
        }
        v4f acc[2 * NT][NG];
#pragma unroll
        for (int t = 0; t < 2 * NT; ++t)
#pragma unroll
            for (int n = 0; n < NG; ++n)
                acc[t][n] = (v4f){0.f, 0.f, 0.f, 0.f};
        for (int kb0 = wave * D; kb0 < KB; kb0 += NW * D) {
            v4i wr[D][2 * NT][2];
            v4i xr[D][NG][4];
#pragma unroll
            for (int j = 0; j < D; ++j) {
                const int kb = kb0 + j;
                const bool live = kb < KB;
                const int so = live ? kb * (PK ? 2048 : 128) : 0;
#pragma unroll
                for (int t = 0; t < 2 * NT; ++t)
#pragma unroll
                    for (int h = 0; h < 2; ++h)
                        wr[j][t][h] = __builtin_amdgcn_raw_buffer_load_b128(live ? wres : none, (int)woff[t][h], so,
                                                                           NG > 1 ? 0 : 2 /* nt */);
#pragma unroll
                for (int n = 0; n < NG; ++n)
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        xr[j][n][q] = __builtin_amdgcn_raw_buffer_load_b128(live ? xres : none,
                                                                            (int)(xoff[n] + part_offset(q)),
                                                                            live ? kb * 256 : 0, 0);
            }
#pragma unroll
            for (int j = 0; j < D; ++j) {
                const int kb = kb0 + j;
                if (kb < KB) {
#pragma unroll
                    for (int t = 0; t < 2 * NT; ++t) {
                        const Wide w = widen(w_fragment(wr[j][t][0], wr[j][t][1], PK));
#pragma unroll
                        for (int n = 0; n < NG; ++n)
                            acc[t][n] = fma4(block_dot(w, xr[j][n]), t < NT ? sg[kb] : su[kb], acc[t][n]);
                    }
                }
            }
        }
        if (s0 >= 16 * NG * (int)gridDim.y)
            __syncthreads();                       // the previous pass's partials are read out
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int n = 0; n < NG; ++n) {
                red[wave][2 * (n * NT + t)][lane] = acc[t][n];
                red[wave][2 * (n * NT + t) + 1][lane] = acc[NT + t][n];
            }
        __syncthreads();
#pragma unroll
        for (int f0 = 0; f0 < NG * NT; f0 += NW) { // wave w finishes tile f % NT of group f / NT, f = w, w + NW, ..
            const int f = f0 + wave;
            if (f < NG * NT) {
                v4f v0 = red[0][2 * f][lane], v1 = red[0][2 * f + 1][lane];
#pragma unroll
                for (int w = 1; w < NW; ++w) {
                    v0 += red[w][2 * f][lane];
                    v1 += red[w][2 * f + 1][lane];
                }
                const int s = s0 + 16 * (f / NT) + r16;
                if (s < cnt) {
                    if constexpr (DOWN) {
                        const float weight = p.plan->weight[off + s];
                        float *to = p.part + (size_t)(off + s) * N + 16 * (first + f % NT) + 4 * g;
                        *reinterpret_cast<v4f *>(to) = v0 * weight;
                        *reinterpret_cast<v4f *>(to + 16 * NT) = v1 * weight;
                    } else {
                        v4f hv;
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            hv[i] = v0[i] / (1.0f + expf(-v0[i])) * v1[i];
                        const int64_t row = (int64_t)(off + s) * p.I;
                        store4(p.h, row, 16 * (first + f % NT) + 4 * g, p.I, true, hv);
                        if (NG == 1 && p.lo != 0) {            // (no second term beside an inf or NaN)
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                const float rest = hv[i] - __uint_as_float(bf16_rne(hv[i]) << 16);
                                hv[i] = rest - rest == 0.f ? rest : 0.f;
                            }
                            store4(p.h + p.lo, row, 16 * (first + f % NT) + 4 * g, p.I, true, hv);
                        }
                    }
                }
            }
        }
    }
}

template <int D, int NW, int NG, int NT, bool FUSED, bool PK>
__global__ __launch_bounds__(NW * 64) void moe_up_kernel(MoeArgs p)
{
    expert_rows<D, NW, NG, NT, FUSED, false, PK>(p);
}

template <int D, int NW, int NG, int NT, bool PK>
__global__ __launch_bounds__(NW * 64) void moe_slot_down_kernel(MoeArgs p)
{
    expert_rows<D, NW, NG, NT, false, true, PK>(p);
}

// The sum of a token's slots, in the order of its routing; a thread forms four columns.
__global__ __launch_bounds__(256) void moe_combine_kernel(MoeArgs p)
{
    const int n = ((int)blockIdx.x * 256 + (int)threadIdx.x) * 4, t = blockIdx.y, k = p.route.k;
    if (n >= p.H)
        return;
    const_i32 *place = (const_i32 *)p.plan->place + (size_t)t * k;
    v4f sum = {0.f, 0.f, 0.f, 0.f};
    for (int j0 = 0; j0 < k; j0 += 8) {
        v4f v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int at = j0 + j < k ? place[j0 + j] : -1;
            v[j] = at >= 0 ? *reinterpret_cast<const v4f *>(p.part + (size_t)at * p.H + n) : (v4f){0.f, 0.f, 0.f, 0.f};
        }
#pragma unroll
        for (int j = 0; j < 8; ++j)
            sum += v[j];
    }
    store4(p.Y, (int64_t)t * p.H, n, p.H, p.vec_store != 0, sum);
}

// Few slots per expert leave most of the 16 columns of a product empty, yet a block's hidden rows
// cost the same loads however many columns they fill (with one or two slots per expert those
// loads can take as long as the weights).  So the columns are two sets of 8 slots:
//
// TWO: the second set holds the hidden rows' second terms, so that h is carried as two bf16 terms
// (16 bits of mantissa, as the adapters' inner values are) and only Y's own rounding is left.  With
// one term h's rounding weighs as much as Y's: 1.4 times its error, up to 1.8 for one token.  For that a
// call takes up to 5% longer than with the columns dealt out to 4 K blocks of one term (17.7 and 18.4 us
// for one token and 128 experts of 768 x 2048, 80.3 and 81.0 for 5 and 32 of 1792 x 5120, 118.8 and 121.9
// for 61 and 256 of 512 x 2048), as long as experts have up to 3.5 slots on average.
//
// Else: the second set takes the next K block, and one block's loads fetch the hidden rows of two.
// Above 3.5 slots a second term costs up to 10% (128 tokens, 256 experts of 512 x 2048: 151 us and 158-165),
// and so many slots average the rounding out to the 1.4.
//
// Either way the sets are added at the end.
__device__ __forceinline__ float sum_sets(float v)   // (every lane of a 16-lane row gets it)
{
    return v + __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x128, 0xF, 0xF, false));   // row_ror 8
}

// Down product and combination.  Workgroup (cb, s): output columns 16 NT cb .. + 16 NT; its
// NW waves (of S workgroups per column block) split the (expert, D K blocks) units of every
// reached expert into equal runs.  A wave adds each unit's weighted products to its own
// fp32 sums per token in LDS (an expert holds a token once, so no two lanes add to one
// place); at the end the waves' sums are added in wave order.  With S > 1 the workgroups'
// sums meet in the workspace and the last to arrive adds them in order.  No output depends
// on which wave ran first.  The next unit's weights and first slots are in flight while a
// unit is multiplied.
struct DownUnit {
    int off, cnt, kb0;        // the expert's slots, the unit's first K block
};

template <int D, int NW, int RING, bool TWO, int NT, bool PK>
__global__ __launch_bounds__(NW * 64) void moe_down_kernel(MoeArgs p)
{
    constexpr int P = TWO ? 1 : 2;                                  // K blocks that share the columns
    static_assert(D % P == 0, "whole groups of P blocks");
    static_assert((D - 1) * 256 <= kHiddenPad, "a unit's blocks past K");
    constexpr int G = 8, DX = D / P;                                // slots per group, hidden-row loads per unit
    extern __shared__ __attribute__((aligned(16))) float sums[];    // [NW][T][16 NT]
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int T = p.T, H = p.H, I = p.I, KB = I >> 7, S = p.splits;
    const int cb = (int)blockIdx.x / S, split = (int)blockIdx.x - cb * S;
    const int r16 = lane & 15, g = lane >> 4, slot = r16 % G, set = r16 / G;
    const_i32 *head = (const_i32 *)p.plan;
    const_i4 *list = (const_i4 *)p.plan->expert;
    const int experts = head[0], slots = head[1];
    const int C = (KB + D - 1) / D;
    const int units = experts * C, part = split * NW + wave, parts = S * NW;
    const int u0 = (int)((int64_t)part * units / parts), u1 = (int)((int64_t)(part + 1) * units / parts);
    const uint32_t wbytes = (uint32_t)I * (uint32_t)H;
    const uint32_t srow = (uint32_t)(cb * NT >> 3) * (uint32_t)KB, sexp = (uint32_t)(H >> 7) * (uint32_t)KB;
    const __amdgpu_buffer_rsrc_t hres = buffer_rsrc(p.h, ((TWO ? p.lo : 0u) + (uint32_t)slots * (uint32_t)I) * 2u);
    const __amdgpu_buffer_rsrc_t tres = buffer_rsrc(p.plan->token, (uint32_t)slots * 4u);
    const __amdgpu_buffer_rsrc_t gres = buffer_rsrc(p.plan->weight, (uint32_t)slots * 4u);
    uint32_t woff[NT][2];
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int h = 0; h < 2; ++h)
            woff[t][h] = tile_offset<PK>((uint32_t)(cb * NT + t), h, lane, (uint32_t)I);
    const uint32_t lane_h = (uint32_t)slot * (uint32_t)I * 2u + 32u * (uint32_t)g + (uint32_t)set * (TWO ? p.lo * 2u : 256u);

    v4i wr[RING][D][NT][2], xr[RING][DX][4];
    float sr[RING][D];                             // the blocks' weight scales
    int tok[RING];
    float wt[RING];
    DownUnit un[RING];
    // Slots s0 .. s0 + G - 1 of unit n: their hidden rows' blocks, tokens and weights.  (A block
    // past K reads the row's neighbour, or behind the last row the kHiddenPad bytes that the
    // workspace keeps there; its products are not kept.)
    auto load_slots = [&](const DownUnit &n, int s0, v4i (&x)[DX][4], int &tk, float &w) __attribute__((always_inline)) {
        const uint32_t hoff = s0 + slot < n.cnt ? lane_h : kOob;
        const int row = (int)((uint32_t)(n.off + s0) * (uint32_t)I * 2u);
#pragma unroll
        for (int j = 0; j < DX; ++j)
#pragma unroll
            for (int q = 0; q < 4; ++q)
                x[j][q] = __builtin_amdgcn_raw_buffer_load_b128(hres, (int)(hoff + part_offset(q) + 256 * P * j),
                                                                row + n.kb0 * 256, 0);
        tk = __builtin_amdgcn_raw_buffer_load_b32(tres, 4 * slot, 4 * (n.off + s0), 0);
        w = __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(gres, 4 * slot, 4 * (n.off + s0), 0));
    };
    // The walk over the run's units: expert number a of the plan, chunk ch of its K blocks; the
    // plan entry of the next unit is read ahead of its use.
    int a = u0 / C, ch = u0 - a * C;
    i4 next = list[min(a, kMaxExperts - 1)];
    // Issues the loads of unit u, always the same number of them, so that the wait for one
    // unit's loads never has to cover the next one's: past the run's end, and for a block
    // past K, they read nothing (zero records, and no scalar offset).
    auto load = [&](int u, v4i (&w)[D][NT][2], v4i (&x)[DX][4], float (&sc)[D], int &tk, float &wgt, DownUnit &n)
        __attribute__((always_inline)) {
        const bool live = u < u1;
        const i4 ex = next;
        n.off = ex[1];
        n.cnt = live ? ex[2] : 0;
        n.kb0 = ch * D;
        if (++ch == C) {
            ch = 0;
            ++a;
        }
        next = list[u + 1 < u1 ? a : 0];
#pragma unroll
        for (int j = 0; j < D; ++j) {
            const bool block = live && n.kb0 + j < KB;
            const __amdgpu_buffer_rsrc_t wres = buffer_rsrc(p.W2 + (size_t)ex[0] * wbytes, block ? wbytes : 0u);
            const __amdgpu_buffer_rsrc_t sres = buffer_rsrc(p.s2, block ? (uint32_t)p.E * sexp * 4u : 0u);
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    w[j][t][h] = __builtin_amdgcn_raw_buffer_load_b128(wres, (int)woff[t][h] + j * (PK ? 2048 : 128),
                                                                       block ? n.kb0 * (PK ? 2048 : 128) : 0, 2 /* nt */);
            // (a vector load: a scalar one would make the wave wait for all its scalar loads)
            sc[j] = __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(
                                                  sres, 4 * j,
                                                  block ? (int)(((uint32_t)ex[0] * sexp + srow + (uint32_t)n.kb0) * 4u) : 0, 0));
        }
        load_slots(n, 0, x, tk, wgt);
    };
    float *own = sums + (size_t)wave * T * 16 * NT;
    auto compute = [&](const v4i (&w)[D][NT][2], const v4i (&x)[DX][4], const float (&sc)[D], int tk, float wgt, const DownUnit &n)
        __attribute__((always_inline)) {
        auto add = [&](const v4i (&xs)[DX][4], int s0, int t16, float w16) __attribute__((always_inline)) {
            v4f acc[NT];
#pragma unroll
            for (int t = 0; t < NT; ++t)
                acc[t] = (v4f){0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int j = 0; j < D; ++j) {
                if (n.kb0 + j < KB) {
#pragma unroll
                    for (int t = 0; t < NT; ++t) {
                        const Wide wf = widen(w_fragment(w[j][t][0], w[j][t][1], PK));
                        const v4f sum = fma4(block_dot(wf, xs[j / P]), sc[j], acc[t]);
                        if (TWO || set == j % P)
                            acc[t] = sum;
                    }
                }
            }
#pragma unroll
            for (int t = 0; t < NT; ++t) {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    acc[t][i] = sum_sets(acc[t][i]);
                if (s0 + slot < n.cnt && set == 0) {
                    v4f *to = reinterpret_cast<v4f *>(own + ((size_t)t16 * NT + t) * 16 + 4 * g);
                    *to = fma4(acc[t], w16, *to);
                }
            }
        };
        add(x, 0, tk, wgt);
        for (int s0 = G; s0 < n.cnt; s0 += G) {    // (registers of its own: the first slots' wait stays exact)
            v4i more[DX][4];
            int t16;
            float w16;
            load_slots(n, s0, more, t16, w16);
            add(more, s0, t16, w16);
        }
    };
    // (A wave without a unit -- every wave, where no token reaches an expert and the plan's list holds
    // whatever the workspace held before -- loads nothing.)
    if (u0 < u1) {
#pragma unroll
        for (int r = 0; r < RING - 1; ++r)
            load(u0 + r, wr[r], xr[r], sr[r], tok[r], wt[r], un[r]);
    }
    for (int i = lane; i < T * 4 * NT; i += 64)
        reinterpret_cast<v4f *>(own)[i] = (v4f){0.f, 0.f, 0.f, 0.f};
    for (int u = u0; u < u1; u += RING) {
#pragma unroll
        for (int r = 0; r < RING; ++r) {
            constexpr int LAST = RING - 1;
            const int to = (r + LAST) % RING;
            load(u + r + LAST, wr[to], xr[to], sr[to], tok[to], wt[to], un[to]);
            compute(wr[r], xr[r], sr[r], tok[r], wt[r], un[r]);
        }
    }
    __syncthreads();
    const bool whole = S == 1;
    constexpr int Q = 4 * NT;                                       // 4-column pieces of a token's columns
    const __amdgpu_buffer_rsrc_t pres = buffer_rsrc(p.part + (size_t)cb * S * T * 16 * NT, (uint32_t)(S * T) * 64u * NT);
    for (int i = threadIdx.x; i < T * Q; i += NW * 64) {
        v4f v = reinterpret_cast<const v4f *>(sums)[i];
#pragma unroll
        for (int w = 1; w < NW; ++w)
            v += reinterpret_cast<const v4f *>(sums)[(size_t)w * T * Q + i];
        if (whole)
            store4(p.Y, (int64_t)(i / Q) * H, 16 * NT * cb + 4 * (i % Q), H, p.vec_store != 0, v);
        else                                       // [cb][split][T][16 NT] fp32, device-coherent
            __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(v4i, v), pres, i * 16, split * T * 64 * NT, 16 /* sc1 */);
    }
    if (whole)
        return;
    __shared__ int last;
    wait_vmcnt<0>();                               // this wave's partial stores are complete
    __syncthreads();                               // ... and every wave's
    if (threadIdx.x == 0)
        last = __hip_atomic_fetch_add(p.cnt + cb, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == S - 1;
    __syncthreads();
    if (!last)
        return;
    for (int i = threadIdx.x; i < T * Q; i += NW * 64) {
        v4f v = {0.f, 0.f, 0.f, 0.f};
        for (int s = 0; s < S; ++s)
            v += __builtin_bit_cast(v4f, __builtin_amdgcn_raw_buffer_load_b128(pres, i * 16, s * T * 64 * NT, 16 /* sc1 */));
        store4(p.Y, (int64_t)(i / Q) * H, 16 * NT * cb + 4 * (i % Q), H, p.vec_store != 0, v);
    }
    if (threadIdx.x == 0)
        __hip_atomic_store(p.cnt + cb, 0, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

}  // namespace kern

namespace {

using namespace kern;

constexpr int kMaxDevices = 64;
std::atomic<int> g_lds_set[kMaxDevices];

typedef void (*RouteFn)(RouteArgs);
typedef void (*PlanFn)(RouteArgs, MoePlan *, int32_t *);
typedef void (*MoeFn)(MoeArgs);

// Logits per lane: the smallest power of two that covers E.
int vpl_index(int E) { return E <= 64 ? 0 : E <= 128 ? 1 : E <= 256 ? 2 : E <= 512 ? 3 : 4; }
const RouteFn kRoute[5] = {route_kernel<1>, route_kernel<2>, route_kernel<4>, route_kernel<8>, route_kernel<16>};
const RouteFn kRouteRows[3] = {route_rows_kernel<4>, route_rows_kernel<8>, route_rows_kernel<16>};
const PlanFn kPlan[5] = {moe_plan_kernel<1>, moe_plan_kernel<2>, moe_plan_kernel<4>, moe_plan_kernel<8>,
                         moe_plan_kernel<16>};
#define MOE_UP(D, NW, NG, NT, FUSED) \
    {{moe_up_kernel<D, NW, NG, NT, FUSED, false>, moe_up_kernel<D, NW, NG, NT, FUSED, true>}, NW, NT}
struct UpInstance {
    MoeFn fn[2];      // [packed]
    int waves, tiles; // tiles: 16-row tiles of gate rows per workgroup
};
// Few slots per expert, routing itself; few; many (more than six on average), wide and narrow.
const UpInstance kUp[4] = {MOE_UP(2, 4, 1, 1, true), MOE_UP(2, 4, 1, 1, false), MOE_UP(1, 4, 2, 4, false),
                           MOE_UP(1, 4, 2, 2, false)};

#define MOE_DOWN(D, NW, RING, TWO, NT) \
    {{moe_down_kernel<D, NW, RING, TWO, NT, false>, moe_down_kernel<D, NW, RING, TWO, NT, true>}, D, NW, NT, TWO}
struct DownInstance {
    MoeFn fn[2];      // [packed]
    int blocks, waves, tiles;
    bool two;         // two terms of the hidden rows
};
// Two widths with two terms of the hidden rows, two with one.
const DownInstance kDown[] = {MOE_DOWN(2, 4, 2, true, 1), MOE_DOWN(2, 4, 2, true, 2), MOE_DOWN(4, 4, 2, false, 1),
                              MOE_DOWN(4, 4, 2, false, 2)};
// Many slots per expert: wide (128 rows of W2 a workgroup) and narrow (64).
#define MOE_SLOT_DOWN(NT) \
    {{moe_slot_down_kernel<1, 4, 2, NT, false>, moe_slot_down_kernel<1, 4, 2, NT, true>}, 4, NT}
const UpInstance kSlotDown[2] = {MOE_SLOT_DOWN(4), MOE_SLOT_DOWN(2)};

int check_route(const void *logits, int32_t dtype, int64_t T, int64_t E, int32_t topk, int32_t score)
{
    if (T < 0 || T > ((int64_t)1 << 30) || E < 1 || E > kMaxExperts || topk < 1 || topk > kMaxTopk || topk > E ||
        dtype < 0 || dtype > 1 || score < 0 || score > 1)
        return A8W8_ERR_SHAPE;
    if (T == 0)
        return A8W8_OK;
    if (!logits)
        return A8W8_ERR_NULL;
    if (reinterpret_cast<uintptr_t>(logits) & (dtype == A8W8_LOGITS_BF16 ? 1 : 3))
        return A8W8_ERR_ALIGN;
    return A8W8_OK;
}

// The down product's plan: which instance (-1: the one that leaves the slots to the combination), and
// how many workgroups per column block.
struct DownPlan {
    int id, splits;
};

// The form by the average slots of a reached expert (the comment on the column sets).  Then the
// width and the split with the least estimated time, in us: the weights at 5.5 TB/s, more
// for the hidden rows' loads, times the unevenness of the last round of workgroups, plus 1
// per split (its partial sums) and 3 per further round.  Measured at 5, 16 and 61 tokens (5120 x 1792, 2048 x 768, 2048 x 512) for
// both widths and 1, 2, 3, 4 and 6 splits: the pick is the fastest or within 4%.
DownPlan down_plan(int64_t slots, int64_t experts, int64_t H, int64_t I, int cus)
{
    const double reached = experts * (1.0 - std::exp(-(double)slots / experts)), each = slots / reached;
    if (each > 6.0)
        return {-1, 1};
    const int first = each <= 3.5 ? 0 : 2;
    DownPlan best = {first, 1};
    double best_us = 1e30;
    for (int id = first; id < first + 2; ++id) {
        const DownInstance &d = kDown[id];
        const int64_t blocks = H / (16 * d.tiles);
        const double work = reached * H * I / 5.5e6 * (1.0 + 0.3 / ((d.two ? 1 : 2) * d.tiles)), units = reached * ((I / 128 + d.blocks - 1) / d.blocks);
        for (int S = 1; S <= 8 && (S == 1 || S * d.waves <= units); ++S) {
            const int64_t rounds = (blocks * S + cus - 1) / cus;
            const double us = work * rounds * cus / (blocks * S) + S + 3.0 * (rounds - 1);
            if (us < best_us) {
                best = {id, S};
                best_us = us;
            }
        }
    }
    return best;
}

struct MoeLayout {
    int64_t h, part, bytes;   // offsets from the workspace's start
    int64_t lo;               // elements from a hidden row's first term to its second (0: one term)
    DownPlan down;
};

MoeLayout moe_layout(int64_t T, int32_t topk, int32_t E, int64_t H, int64_t I, int cus)
{
    const int64_t t = T < kChunk ? T : kChunk, slots = t * topk;
    MoeLayout l;
    l.down = down_plan(slots, E, H, I, cus);
    l.h = A8W8_WORKSPACE_COUNTER_BYTES + (((int64_t)sizeof(MoePlan) + 255) & ~(int64_t)255);
    l.lo = l.down.id >= 0 && kDown[l.down.id].two ? slots * I : 0;
    l.part = l.h + (((slots * I + l.lo) * 2 + kHiddenPad + 255) & ~(int64_t)255);
    l.bytes = l.part + (l.down.id < 0 ? slots * H * 4 : l.down.splits > 1 ? l.down.splits * t * H * 4 : 0);
    return l;
}

int check_layer_shape(int64_t T, int32_t topk, int32_t E, int64_t H, int64_t I)
{
    if (T < 0 || T > ((int64_t)1 << 30) || E < 1 || E > kMaxExperts || topk < 1 || topk > kMaxTopk || topk > E)
        return A8W8_ERR_SHAPE;
    // 32-bit offsets inside one expert's weights, a chunk's activations and hidden rows;
    // one counter per 16 output columns.
    if (H < 128 || H % 128 != 0 || H > 65536 || I < 128 || I % 128 != 0 || I > 65536 ||
        2 * I * H >= (int64_t)kOob)
        return A8W8_ERR_SHAPE;
    return A8W8_OK;
}

}  // namespace
}  // namespace a8w8

using namespace a8w8;

extern "C" {

int a8w8_moe_route(const void *logits, int32_t logits_dtype, int64_t T, int64_t E, int32_t topk, int32_t score,
                   int32_t renormalize, float scale, float *weights, int32_t *ids, void *stream)
{
    int rc = check_route(logits, logits_dtype, T, E, topk, score);
    if (rc != A8W8_OK || T == 0)
        return rc;
    if (!weights || !ids)
        return A8W8_ERR_NULL;
    if ((reinterpret_cast<uintptr_t>(weights) & 3) || (reinterpret_cast<uintptr_t>(ids) & 3))
        return A8W8_ERR_ALIGN;
    int cus = 0;
    rc = device_ready(&cus);
    if (rc != A8W8_OK)
        return rc;
    const RouteArgs a = {logits, weights, ids, T, (int32_t)E, topk, logits_dtype, score, renormalize != 0, scale};
    const bool rows = T >= kRowTokens && topk <= kRowTopk && E <= kRowExperts;
    const int64_t wgs = rows ? (T + 15) / 16 : (T + 3) / 4, cap = (int64_t)cus * 8;
    hipLaunchKernelGGL((rows ? kRouteRows : kRoute)[vpl_index((int)E)], dim3((unsigned)(wgs < cap ? wgs : cap)), dim3(256), 0,
                       static_cast<hipStream_t>(stream), a);
    return hipGetLastError() == hipSuccess ? A8W8_OK : A8W8_ERR_HIP;
}

int a8w8_moe_workspace_bytes(int64_t T, int32_t topk, int32_t experts, int64_t H, int64_t I, int32_t cu_count,
                             int64_t *bytes)
{
    if (!bytes)
        return A8W8_ERR_NULL;
    const int rc = check_layer_shape(T, topk, experts, H, I);
    if (rc != A8W8_OK)
        return rc;
    // Fewer tokens may need more (another form or split of the down product): what any number up to T needs.
    *bytes = 0;
    for (int64_t t = 1; t <= std::min<int64_t>(T, kChunk); ++t)
        *bytes = std::max(*bytes, moe_layout(t, topk, experts, H, I, cu_count > 0 ? cu_count : 256).bytes);
    return A8W8_OK;
}

int a8w8_moe_layer(const a8w8_moe_desc *d, void *stream)
{
    if (!d)
        return A8W8_ERR_NULL;
    int rc = check_layer_shape(d->T, d->topk, d->experts, d->H, d->I);
    if (rc != A8W8_OK)
        return rc;
    if (d->w_packed < 0 || d->w_packed > 1)
        return A8W8_ERR_SHAPE;
    rc = check_route(d->logits, d->logits_dtype, d->T, d->experts, d->topk, d->score);
    if (rc != A8W8_OK || d->T == 0)
        return rc;
    if (!d->X || !d->W13 || !d->w13_scale || !d->W2 || !d->w2_scale || !d->Y)
        return A8W8_ERR_NULL;
    if ((reinterpret_cast<uintptr_t>(d->X) & 15) || (reinterpret_cast<uintptr_t>(d->W13) & 15) ||
        (reinterpret_cast<uintptr_t>(d->W2) & 15) || (reinterpret_cast<uintptr_t>(d->w13_scale) & 3) ||
        (reinterpret_cast<uintptr_t>(d->w2_scale) & 3) || (reinterpret_cast<uintptr_t>(d->Y) & 1) ||
        (reinterpret_cast<uintptr_t>(d->workspace) & 255))
        return A8W8_ERR_ALIGN;
    int cus = 0;
    rc = device_ready(&cus);
    if (rc != A8W8_OK)
        return rc;
    const MoeLayout l = moe_layout(d->T, d->topk, d->experts, d->H, d->I, cus);
    if (!d->workspace || d->workspace_bytes < l.bytes)
        return A8W8_ERR_WORKSPACE;
    int dev = 0;
    if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= kMaxDevices)
        return A8W8_ERR_HIP;
    if (g_lds_set[dev].load(std::memory_order_acquire) == 0) {
        for (const DownInstance &i : kDown)
            for (const MoeFn f : i.fn)
                if (hipFuncSetAttribute(reinterpret_cast<const void *>(f), hipFuncAttributeMaxDynamicSharedMemorySize,
                                        i.waves * i.tiles * kChunk * 64) != hipSuccess)
                    return A8W8_ERR_HIP;
        g_lds_set[dev].store(1, std::memory_order_release);
    }
    uint8_t *ws = static_cast<uint8_t *>(d->workspace);
    hipStream_t st = static_cast<hipStream_t>(stream);
    const int64_t lsize = d->logits_dtype == A8W8_LOGITS_BF16 ? 2 : 4;
    for (int64_t t0 = 0; t0 < d->T; t0 += kChunk) {
        const int64_t T = d->T - t0 < kChunk ? d->T - t0 : kChunk;
        const RouteArgs r = {static_cast<const uint8_t *>(d->logits) + t0 * d->experts * lsize, nullptr, nullptr, T,
                             d->experts, d->topk, d->logits_dtype, d->score, d->renormalize != 0, d->scale};
        MoeArgs m;
        m.X = static_cast<const uint16_t *>(d->X) + t0 * d->H;
        m.W13 = static_cast<const uint8_t *>(d->W13);
        m.s13 = d->w13_scale;
        m.W2 = static_cast<const uint8_t *>(d->W2);
        m.s2 = d->w2_scale;
        m.Y = static_cast<uint16_t *>(d->Y) + t0 * d->H;
        m.cnt = reinterpret_cast<int32_t *>(ws);
        MoePlan *plan = reinterpret_cast<MoePlan *>(ws + A8W8_WORKSPACE_COUNTER_BYTES);
        m.plan = plan;
        m.h = reinterpret_cast<uint16_t *>(ws + l.h);
        m.lo = (uint32_t)l.lo;
        m.part = reinterpret_cast<float *>(ws + l.part);
        m.T = (int32_t)T;
        m.H = (int32_t)d->H;
        m.I = (int32_t)d->I;
        m.E = d->experts;
        m.splits = l.down.splits;
        m.vec_store = (reinterpret_cast<uintptr_t>(d->Y) & 7) == 0;
        const int64_t slots = T * d->topk, reached = slots < d->experts ? slots : d->experts;
        m.route = r;
        const bool fused = T <= kFusedTokens && slots <= kFusedSlots && d->experts <= kFusedExperts && l.down.id >= 0;
        if (!fused)
            hipLaunchKernelGGL(kPlan[vpl_index(d->experts)], dim3((unsigned)((T + 15) / 16)), dim3(1024), 0, st, r, plan, m.cnt);
        if (l.down.id >= 0) {
            const UpInstance &up = kUp[fused ? 0 : 1];
            hipLaunchKernelGGL(up.fn[d->w_packed], dim3((unsigned)(reached * (d->I / (16 * up.tiles)))), dim3(up.waves * 64), 0,
                               st, m);
            const DownInstance &down = kDown[l.down.id];
            hipLaunchKernelGGL(down.fn[d->w_packed], dim3((unsigned)(d->H / (16 * down.tiles) * l.down.splits)),
                               dim3(down.waves * 64), (size_t)(down.waves * down.tiles * T * 64), st, m);
        } else {
            // The wide workgroups where they give three quarters of the CUs one, and, where even the
            // narrow ones are too few, workgroups of their own for an expert's passes of 32 slots.
            // 64 tokens, 8 experts of 512 x 1024, top 2: 20.6 us against 25.4 with wide ones; 32 tokens, 8
            // of 1792 x 4096: 46.6 against 44.7.  256 tokens on all of 8 experts of 128 x 1280: 37.0 us
            // against 114.8 with every pass in one workgroup.
            const auto launch = [&](const UpInstance *pair, int64_t wide) {
                const UpInstance &f = pair[4 * wide >= 3 * cus ? 0 : 1];
                const int64_t wgs = wide * pair[0].tiles / f.tiles, fill = (2 * cus + wgs - 1) / wgs, most = (T + 31) / 32;
                hipLaunchKernelGGL(f.fn[d->w_packed], dim3((unsigned)wgs, (unsigned)(fill < most ? fill : most)),
                                   dim3(f.waves * 64), 0, st, m);
            };
            launch(kUp + 2, reached * (d->I / 64));
            launch(kSlotDown, reached * (d->H / 128));
            hipLaunchKernelGGL(moe_combine_kernel, dim3((unsigned)((d->H + 1023) / 1024), (unsigned)T), dim3(256), 0, st, m);
        }
        if (hipGetLastError() != hipSuccess)
            return A8W8_ERR_HIP;
    }
    return A8W8_OK;
}

}  // extern "C"
