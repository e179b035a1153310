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
// fp32 dot is then scaled into the fp32 accumulator, as in the GEMM kernels.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <atomic>
#include <mutex>

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
constexpr uint32_t kOob = 0x7ffff000u;   // beyond any buffer here: loads return zeros, no traffic

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
};

struct MoeArgs {
    const uint16_t *X;    // bf16 [T, H]
    const uint8_t *W13;   // e4m3fn [E, 2I, H]
    const float *s13;     // [E, 2I/128, H/128]
    const uint8_t *W2;    // e4m3fn [E, H, I]
    const float *s2;      // [E, H/128, I/128]
    uint16_t *Y;          // bf16 [T, H]
    const MoePlan *plan;
    uint16_t *h;          // bf16 [slots, I]
    float *part;          // down product with splits: [H/16][splits][T][16]
    int32_t *cnt;         // one zeroed counter per 16 output columns
    int32_t T, H, I, E, splits, vec_store;
};

// ---------------------------------------------------------------------------
// Routing.  One wave per token; lane l holds the logits of experts l, l + 64, ...
// (VPL of them).

// One DPP step of a reduction over the wave: lanes without a source keep `x`'s neutral `old`.
template <int CTRL, int ROWS>
__device__ __forceinline__ float dpp_from(float old, float x)
{
    return __int_as_float(__builtin_amdgcn_update_dpp(__float_as_int(old), __float_as_int(x), CTRL, ROWS, 0xF, false));
}
// Maximum over the wave (row shifts, then row broadcasts: lane 63 has it), in every lane.
__device__ __forceinline__ float wave_max(float x)
{
    x = fmaxf(x, dpp_from<0x111, 0xF>(x, x));
    x = fmaxf(x, dpp_from<0x112, 0xF>(x, x));
    x = fmaxf(x, dpp_from<0x114, 0xF>(x, x));
    x = fmaxf(x, dpp_from<0x118, 0xF>(x, x));
    x = fmaxf(x, dpp_from<0x142, 0xA>(x, x));
    x = fmaxf(x, dpp_from<0x143, 0xC>(x, x));
    return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(x), 63));
}
// Sum over the wave in a fixed order, in every lane.
__device__ __forceinline__ float wave_sum(float x)
{
    x += dpp_from<0x111, 0xF>(0.f, x);
    x += dpp_from<0x112, 0xF>(0.f, x);
    x += dpp_from<0x114, 0xF>(0.f, x);
    x += dpp_from<0x118, 0xF>(0.f, x);
    x += dpp_from<0x142, 0xA>(0.f, x);
    x += dpp_from<0x143, 0xC>(0.f, x);
    return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(x), 63));
}

template <int VPL>
__device__ __forceinline__ void load_logits(const RouteArgs &p, int64_t t, int lane, float (&v)[VPL])
{
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
        const int e = i * 64 + lane;
        float x = -INFINITY;
        if (e < p.E) {
            if (p.bf16)
                x = __uint_as_float((uint32_t)static_cast<const uint16_t *>(p.logits)[t * p.E + e] << 16);
            else
                x = static_cast<const float *>(p.logits)[t * p.E + e];
        }
        // NaN masks its expert; +inf is the largest finite value.
        v[i] = x == x ? fminf(x, 3.402823466e38f) : -INFINITY;
    }
}

// The token's routing: lane j < k returns slot j's weight and expert.
template <int VPL>
__device__ __forceinline__ void route_row(const RouteArgs &p, float (&v)[VPL], int lane, float &w, int &id)
{
    float lm = v[0];
#pragma unroll
    for (int i = 1; i < VPL; ++i)
        lm = fmaxf(lm, v[i]);
    const float top = wave_max(lm);
    float all = 0.f;
    if (!p.sigmoid && !p.renorm && top > -INFINITY) {
#pragma unroll
        for (int i = 0; i < VPL; ++i)
            all += expf(v[i] - top);
        all = wave_sum(all);
    }
    float val = -INFINITY, m = top;
    id = -1;
    for (int j = 0; j < p.k; ++j) {
        if (m == -INFINITY)
            break;
        int e = -1;
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
            if (e < 0) {
                const uint64_t b = __ballot(v[i] == m);
                if (b)
                    e = i * 64 + __builtin_ctzll(b);
            }
        }
        if (lane == j) {
            val = m;
            id = e;
        }
        lm = -INFINITY;
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
            if (i * 64 + lane == e)
                v[i] = -INFINITY;
            lm = fmaxf(lm, v[i]);
        }
        m = wave_max(lm);
    }
    // Sigmoids that are to be divided by their sum: below 0, sigmoid(v) = exp(v) / (1 + exp(v)),
    // and exp(top) cancels, so the quotients hold where every sigmoid itself would underflow.
    w = 0.f;
    if (id >= 0)
        w = !p.sigmoid ? expf(val - top)
            : p.renorm && top < 0.f ? expf(val - top) / (1.0f + expf(val))
                                    : 1.0f / (1.0f + expf(-val));
    const float total = p.renorm ? wave_sum(w) : p.sigmoid ? 1.0f : all;
    w = total > 0.f ? w / total * p.scale : 0.f;
}

template <int VPL>
__global__ __launch_bounds__(256) void route_kernel(RouteArgs p)
{
    const int lane = threadIdx.x & 63;
    const int64_t step = (int64_t)gridDim.x * 4;
    for (int64_t t = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); t < p.T; t += step) {
        float v[VPL], w;
        int id;
        load_logits<VPL>(p, t, lane, v);
        route_row<VPL>(p, v, lane, w, id);
        if (lane < p.k) {
            p.weights[t * p.k + lane] = w;
            p.ids[t * p.k + lane] = id;
        }
    }
}

// ---------------------------------------------------------------------------
// The layer's plan for one chunk of at most kChunk tokens: the experts that any
// token reached, and their slots (token, weight), grouped by expert in token order.

// Sixteen tokens per workgroup, one wave each; the last workgroup to finish (the only one,
// for up to 16 tokens) makes the plan from everyone's routing.  There a bitmap of tokens
// per expert gives every slot its place by counting, so the order is fixed whatever the
// order the waves run in.  256 tokens: 6.9 us against 52 us with one workgroup routing them
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
        float v[VPL], w;
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
        if (id >= 0) {
            const int tok = i / k;
            int pos = s_off[id] + __popc(mask[id][tok >> 5] & ((1u << (tok & 31)) - 1u));
            for (int b = 0; b < (tok >> 5); ++b)
                pos += __popc(mask[id][b]);
            plan->token[pos] = tok;
            plan->weight[pos] = w[q];
        }
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

// Up product.  Workgroup (a, c): expert a of the plan, NT 16-row tiles of gate rows from
// 16 NT c on and the same of up rows.  Its NW waves take runs of D K blocks in turn; a pass
// serves NG groups of 16 slots (a further pass reads the expert's weights again, from the
// caches).  The wave partials are summed through LDS in wave order; h = silu(gate) * up is
// rounded once to bf16, the activation type of the down product's matrix instructions.
template <int D, int NW, int NG, int NT, bool PK>
__global__ __launch_bounds__(NW * 64) void moe_up_kernel(MoeArgs p)
{
    static_assert(NG * NT <= NW, "wave q finishes tile q % NT of group q / NT");
    __shared__ v4f red[NW][2 * NG * NT][64];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int CB = p.I / (16 * NT), a = (int)blockIdx.x / CB, c = (int)blockIdx.x - a * CB;
    if (a >= ((const_i32 *)p.plan)[0])
        return;
    const i4 ex = ((const_i4 *)p.plan->expert)[a];
    const int e = ex[0], off = ex[1], cnt = ex[2];
    const int H = p.H, I = p.I, KB = H >> 7;
    const int r16 = lane & 15, g = lane >> 4;
    const uint32_t wbytes = 2u * (uint32_t)I * (uint32_t)H;
    const uint8_t *W = p.W13 + (size_t)e * wbytes;
    const __amdgpu_buffer_rsrc_t wres = buffer_rsrc(W, wbytes), none = buffer_rsrc(W, 0u);
    const __amdgpu_buffer_rsrc_t xres = buffer_rsrc(p.X, (uint32_t)p.T * (uint32_t)H * 2u);
    const int NB = (2 * I) >> 7, sb = (c * NT) >> 3;
    const_f32 *sg = (const_f32 *)(p.s13 + ((size_t)e * NB + sb) * KB);
    const_f32 *su = (const_f32 *)(p.s13 + ((size_t)e * NB + ((I >> 7) + sb)) * KB);
    uint32_t woff[2 * NT][2];                      // gate tiles, then up tiles
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            woff[t][h] = tile_offset<PK>((uint32_t)(c * NT + t), h, lane, (uint32_t)H);
            woff[NT + t][h] = tile_offset<PK>((uint32_t)((I >> 4) + c * NT + t), h, lane, (uint32_t)H);
        }
    for (int s0 = 0; s0 < cnt; s0 += 16 * NG) {
        uint32_t xoff[NG];
#pragma unroll
        for (int n = 0; n < NG; ++n) {
            const int s = s0 + 16 * n + r16;
            xoff[n] = s < cnt ? (uint32_t)p.plan->token[off + s] * (uint32_t)H * 2u + 32u * (uint32_t)g : kOob;
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
        if (s0 > 0)
            __syncthreads();                       // the previous pass's partials are read out
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int n = 0; n < NG; ++n) {
                red[wave][2 * (n * NT + t)][lane] = acc[t][n];
                red[wave][2 * (n * NT + t) + 1][lane] = acc[NT + t][n];
            }
        __syncthreads();
        if (wave < NG * NT) {
            v4f vg = red[0][2 * wave][lane], vu = red[0][2 * wave + 1][lane];
#pragma unroll
            for (int w = 1; w < NW; ++w) {
                vg += red[w][2 * wave][lane];
                vu += red[w][2 * wave + 1][lane];
            }
            const int s = s0 + 16 * (wave / NT) + r16;
            if (s < cnt) {
                v4f hv;
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    hv[i] = vg[i] / (1.0f + expf(-vg[i])) * vu[i];
                store4(p.h, (int64_t)(off + s) * I, 16 * (c * NT + wave % NT) + 4 * g, I, true, hv);
            }
        }
    }
}

// Down product and combination.  Workgroup (cb, s): output columns 16 cb .. + 16; its NW
// waves (of S workgroups per column block) split the (expert, D K blocks) units of every
// reached expert into equal runs.  A wave adds each unit's weighted products to its own
// fp32 sums per token in LDS (lane l holds columns 4 (l / 16) .. + 4 of slot l % 16, and an
// expert holds a token once, so no two lanes add to one place); at the end the waves' sums
// are added in wave order.  With S > 1 the workgroups' sums meet in the workspace and the
// last to arrive adds them in order.  No output depends on which wave ran first.
// The next unit's weights and first 16 slots are in flight while a unit is multiplied.
struct DownUnit {
    int off, cnt, kb0;        // the expert's slots, the unit's first K block
};

template <int D, int NW, int RING, bool PK>
__global__ __launch_bounds__(NW * 64) void moe_down_kernel(MoeArgs p)
{
    extern __shared__ __attribute__((aligned(16))) float sums[];    // [NW][T][16]
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int T = p.T, H = p.H, I = p.I, KB = I >> 7, S = p.splits;
    const int cb = (int)blockIdx.x / S, split = (int)blockIdx.x - cb * S;
    const int r16 = lane & 15, g = lane >> 4;
    const_i32 *head = (const_i32 *)p.plan;
    const_i4 *list = (const_i4 *)p.plan->expert;
    const int experts = head[0], slots = head[1];
    const int C = (KB + D - 1) / D;
    const int units = experts * C, part = split * NW + wave, parts = S * NW;
    const int u0 = (int)((int64_t)part * units / parts), u1 = (int)((int64_t)(part + 1) * units / parts);
    const uint32_t wbytes = (uint32_t)I * (uint32_t)H;
    const uint32_t srow = (uint32_t)(cb >> 3) * (uint32_t)KB, sexp = (uint32_t)(H >> 7) * (uint32_t)KB;
    const __amdgpu_buffer_rsrc_t hres = buffer_rsrc(p.h, (uint32_t)slots * (uint32_t)I * 2u);
    const __amdgpu_buffer_rsrc_t sres = buffer_rsrc(p.s2, (uint32_t)p.E * sexp * 4u);
    const __amdgpu_buffer_rsrc_t tres = buffer_rsrc(p.plan->token, (uint32_t)slots * 4u);
    const __amdgpu_buffer_rsrc_t gres = buffer_rsrc(p.plan->weight, (uint32_t)slots * 4u);
    uint32_t woff[2];
#pragma unroll
    for (int h = 0; h < 2; ++h)
        woff[h] = tile_offset<PK>((uint32_t)cb, h, lane, (uint32_t)I);
    const uint32_t lane_h = (uint32_t)r16 * (uint32_t)I * 2u + 32u * (uint32_t)g;

    v4i wr[RING][D][2], xr[RING][D][4];
    float sr[RING][D];                             // the blocks' weight scales
    int tok[RING];
    float wt[RING];
    DownUnit un[RING];
    // Slots s0 .. s0 + 15 of unit n: their hidden rows' blocks, tokens and weights.
    auto load_slots = [&](const DownUnit &n, int s0, v4i (&x)[D][4], int &tk, float &w) __attribute__((always_inline)) {
        const uint32_t hoff = s0 + r16 < n.cnt ? lane_h : kOob;
        const int row = (int)((uint32_t)(n.off + s0) * (uint32_t)I * 2u);
#pragma unroll
        for (int j = 0; j < D; ++j)
#pragma unroll
            for (int q = 0; q < 4; ++q)
                x[j][q] = __builtin_amdgcn_raw_buffer_load_b128(hres, (int)(hoff + part_offset(q) + 256 * j),
                                                                row + n.kb0 * 256, 0);
        tk = __builtin_amdgcn_raw_buffer_load_b32(tres, 4 * r16, 4 * (n.off + s0), 0);
        w = __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(gres, 4 * r16, 4 * (n.off + s0), 0));
    };
    // The walk over the run's units: expert number a of the plan, chunk ch of its K blocks; the
    // plan entry of the next unit is read ahead of its use.
    int a = u0 / C, ch = u0 - a * C;
    i4 next = list[min(a, kMaxExperts - 1)];
    // Issues the loads of unit u, always the same number of them, so that the wait for one
    // unit's loads never has to cover the next one's: past the run's end they read nothing
    // (zero records) and no slot is live.  A block past K reads bytes nobody multiplies.
    auto load = [&](int u, v4i (&w)[D][2], v4i (&x)[D][4], float (&sc)[D], int &tk, float &wgt, DownUnit &n)
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
        const __amdgpu_buffer_rsrc_t wres = buffer_rsrc(p.W2 + (size_t)ex[0] * wbytes, live ? wbytes : 0u);
#pragma unroll
        for (int j = 0; j < D; ++j) {
#pragma unroll
            for (int h = 0; h < 2; ++h)
                w[j][h] = __builtin_amdgcn_raw_buffer_load_b128(wres, (int)woff[h] + j * (PK ? 2048 : 128),
                                                                n.kb0 * (PK ? 2048 : 128), 2 /* nt */);
            // (a vector load: a scalar one would make the wave wait for all its scalar loads)
            sc[j] = __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(
                                                  sres, 4 * j, (int)(((uint32_t)ex[0] * sexp + srow + (uint32_t)n.kb0) * 4u), 0));
        }
        load_slots(n, 0, x, tk, wgt);
    };
    float *own = sums + (size_t)wave * T * 16;
    auto compute = [&](const v4i (&w)[D][2], const v4i (&x)[D][4], const float (&sc)[D], int tk, float wgt, const DownUnit &n) __attribute__((always_inline)) {
        Wide wf[D];
#pragma unroll
        for (int j = 0; j < D; ++j)
            wf[j] = widen(w_fragment(w[j][0], w[j][1], PK));
        auto add = [&](const v4i (&x16)[D][4], int s0, int t16, float w16) __attribute__((always_inline)) {
            v4f acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int j = 0; j < D; ++j)
                if (n.kb0 + j < KB)
                    acc = fma4(block_dot(wf[j], x16[j]), sc[j], acc);
            if (s0 + r16 < n.cnt) {
                v4f *to = reinterpret_cast<v4f *>(own + (size_t)t16 * 16 + 4 * g);
                *to = fma4(acc, w16, *to);
            }
        };
        add(x, 0, tk, wgt);
        for (int s0 = 16; s0 < n.cnt; s0 += 16) {  // (registers of its own: the first 16 slots' wait stays exact)
            v4i more[D][4];
            int t16;
            float w16;
            load_slots(n, s0, more, t16, w16);
            add(more, s0, t16, w16);
        }
    };
#pragma unroll
    for (int r = 0; r < RING - 1; ++r)
        load(u0 + r, wr[r], xr[r], sr[r], tok[r], wt[r], un[r]);
    for (int i = lane; i < T * 4; i += 64)
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
    for (int i = threadIdx.x; i < T * 4; i += NW * 64) {
        v4f v = reinterpret_cast<const v4f *>(sums)[i];
#pragma unroll
        for (int w = 1; w < NW; ++w)
            v += reinterpret_cast<const v4f *>(sums)[(size_t)w * T * 4 + i];
        const int t = i >> 2, n = 16 * cb + 4 * (i & 3);
        if (whole) {
            store4(p.Y, (int64_t)t * H, n, H, p.vec_store != 0, v);
        } else {
            // [cb][split][T][16] fp32, device-coherent
            const __amdgpu_buffer_rsrc_t pres = buffer_rsrc(p.part + (size_t)cb * S * T * 16, (uint32_t)(S * T) * 64u);
            __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(v4i, v), pres, i * 16, split * T * 64,
                                                   16 /* sc1 */);
        }
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
    const __amdgpu_buffer_rsrc_t pres = buffer_rsrc(p.part + (size_t)cb * S * T * 16, (uint32_t)(S * T) * 64u);
    for (int i = threadIdx.x; i < T * 4; i += NW * 64) {
        v4f v = {0.f, 0.f, 0.f, 0.f};
        for (int s = 0; s < S; ++s)
            v += __builtin_bit_cast(v4f, __builtin_amdgcn_raw_buffer_load_b128(pres, i * 16, s * T * 64, 16 /* sc1 */));
        store4(p.Y, (int64_t)(i >> 2) * H, 16 * cb + 4 * (i & 3), H, p.vec_store != 0, v);
    }
    if (threadIdx.x == 0)
        __hip_atomic_store(p.cnt + cb, 0, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

}  // namespace kern

namespace {

using namespace kern;

constexpr int kDownWaves = 8, kDownBlocks = 2, kDownRing = 2;
constexpr int kUpWaves = 8, kUpBlocks = 2;
constexpr int kMaxDevices = 64;
std::atomic<int> g_lds_set[kMaxDevices];

typedef void (*RouteFn)(RouteArgs);
typedef void (*PlanFn)(RouteArgs, MoePlan *, int32_t *);
typedef void (*MoeFn)(MoeArgs);

// Logits per lane: the smallest power of two that covers E.
int vpl_index(int E) { return E <= 64 ? 0 : E <= 128 ? 1 : E <= 256 ? 2 : E <= 512 ? 3 : 4; }
const RouteFn kRoute[5] = {route_kernel<1>, route_kernel<2>, route_kernel<4>, route_kernel<8>, route_kernel<16>};
const PlanFn kPlan[5] = {moe_plan_kernel<1>, moe_plan_kernel<2>, moe_plan_kernel<4>, moe_plan_kernel<8>,
                         moe_plan_kernel<16>};
#define MOE_UP(D, NG, NT) {moe_up_kernel<D, kUpWaves, NG, NT, false>, moe_up_kernel<D, kUpWaves, NG, NT, true>}
struct UpInstance {
    MoeFn fn[2];      // [packed]
    int tiles;        // 16-row tiles of gate rows per workgroup
};
const UpInstance kUp[3] = {{MOE_UP(kUpBlocks, 1, 1), 1}, {MOE_UP(1, 2, 2), 2}, {MOE_UP(1, 4, 2), 2}};
const MoeFn kDown[2] = {moe_down_kernel<kDownBlocks, kDownWaves, kDownRing, false>,
                        moe_down_kernel<kDownBlocks, kDownWaves, kDownRing, true>};

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

// Workgroups per 16-column block of the down product: as many as fill the CUs
// in whole rounds.
int down_splits(int64_t T, int64_t H, int64_t units, int cus)
{
    (void)T;
    const int64_t blocks = H / 16;
    int best = 1;
    double best_cost = 1e30;
    for (int S = 1; S <= 8; ++S) {
        if (S > 1 && units < (int64_t)S * kDownWaves)
            break;
        const double rounds = (double)((blocks * S + cus - 1) / cus) / S + 0.02 * S;
        if (rounds < best_cost - 1e-9) {
            best = S;
            best_cost = rounds;
        }
    }
    return best;
}

struct MoeLayout {
    int64_t h, part, bytes;   // offsets from the workspace's start
    int splits;
};

MoeLayout moe_layout(int64_t T, int32_t topk, int32_t E, int64_t H, int64_t I, int cus)
{
    const int64_t t = T < kChunk ? T : kChunk, slots = t * topk;
    const int64_t reached = slots < E ? slots : E;
    MoeLayout l;
    l.splits = down_splits(t, H, reached * ((I / 128 + kDownBlocks - 1) / kDownBlocks), cus);
    l.h = A8W8_WORKSPACE_COUNTER_BYTES + (((int64_t)sizeof(MoePlan) + 255) & ~(int64_t)255);
    l.part = l.h + ((slots * I * 2 + 255) & ~(int64_t)255);
    l.bytes = l.part + (l.splits > 1 ? l.splits * t * H * 4 : 0);
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
    const int64_t wgs = (T + 3) / 4, cap = (int64_t)cus * 8;
    hipLaunchKernelGGL(kRoute[vpl_index((int)E)], dim3((unsigned)(wgs < cap ? wgs : cap)), dim3(256), 0,
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
    *bytes = T == 0 ? 0 : moe_layout(T, topk, experts, H, I, cu_count > 0 ? cu_count : 256).bytes;
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
        for (const MoeFn f : kDown)
            if (hipFuncSetAttribute(reinterpret_cast<const void *>(f), hipFuncAttributeMaxDynamicSharedMemorySize,
                                    kDownWaves * kChunk * 64) != hipSuccess)
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
        m.part = reinterpret_cast<float *>(ws + l.part);
        m.T = (int32_t)T;
        m.H = (int32_t)d->H;
        m.I = (int32_t)d->I;
        m.E = d->experts;
        m.splits = l.splits;
        m.vec_store = (reinterpret_cast<uintptr_t>(d->Y) & 7) == 0;
        const int64_t slots = T * d->topk, reached = slots < d->experts ? slots : d->experts;
        hipLaunchKernelGGL(kPlan[vpl_index(d->experts)], dim3((unsigned)((T + 15) / 16)), dim3(1024), 0, st, r, plan, m.cnt);
        // Groups of 16 slots per pass over an expert's weights, by the average slots per expert.
        const int64_t each = slots / d->experts;
        const int ng = each <= 6 ? 0 : each <= 20 ? 1 : 2;
        hipLaunchKernelGGL(kUp[ng].fn[d->w_packed], dim3((unsigned)(reached * (d->I / (16 * kUp[ng].tiles)))), dim3(kUpWaves * 64), 0, st, m);
        hipLaunchKernelGGL(kDown[d->w_packed], dim3((unsigned)(d->H / 16 * l.splits)), dim3(kDownWaves * 64),
                           (size_t)(kDownWaves * T * 64), st, m);
        if (hipGetLastError() != hipSuccess)
            return A8W8_ERR_HIP;
    }
    return A8W8_OK;
}

}  // extern "C"
