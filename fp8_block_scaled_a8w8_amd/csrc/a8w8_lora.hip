// a8w8_lora.hip -- low-rank adapters of many requests at once beside one shared a8w8
// projection, for gfx950:
//
//   Y[m] = bf16( a8w8 product of quantize_1x128(x_m) with W
//                + scaling[a] * B[a] (A[a] x_m) )            a = ids[m], none if negative
//
// in two launches.  The first (lora_inner_kernel, here) quantises X to the codes and
// scales the GEMM takes -- the step that precedes every a8w8 GEMM -- and in other
// workgroups of the same launch forms the inner products V[m] = scaling[a] A[a] x_m.  The
// second is the a8w8 GEMM itself, which adds B[a] V[m] to its fp32 accumulators before it
// rounds them (lora_fold in a8w8_kernels.hip).
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <cstring>

#include "a8w8_device.h"
#include "a8w8_internal.h"
#include "a8w8_quant_math.h"
#include "gemm_a8w8_blockscale.h"

namespace a8w8 {
namespace kern {

struct InnerArgs {
    const uint16_t *X;      // bf16 [M, K]
    const uint16_t *A;      // bf16 [L, R, K]
    const float *scaling;   // [L]
    const int32_t *ids;     // [M]
    uint8_t *codes;         // e4m3fn [M, K]
    float *scales;          // [M, K/128]
    uint16_t *V;            // bf16 [M][2 R]
    int32_t M, K, L, R;
    int32_t quant_wgs;      // workgroups that quantise; the rest form inner products
    int32_t share;          // workgroups per 16-row tile and 16 ranks that share its adapters out
};

constexpr int kInnerWaves = 8;
constexpr int kInnerUnroll = 5;   // 64-wide K chunks a wave has in flight

// Inner products.  A workgroup takes 16 rows of X, 16 ranks and every share-th distinct
// adapter of those rows; its waves take 64-wide chunks of K in turn.  Matrix operands:
// rows of A[a] (ranks), then rows of X, both straight from memory in one K order (lane l:
// row l % 16, 32 contiguous bytes 32 (l / 16) .. of a 128-byte chunk); rows of X that use
// another adapter are zero.  The waves' partials are summed through LDS in wave order.
__global__ __launch_bounds__(kInnerWaves * 64) void lora_inner_kernel(InnerArgs p)
{
    const int tid = threadIdx.x, lane = tid & 63;
    if ((int)blockIdx.x < p.quant_wgs) {
        const int64_t groups = (int64_t)p.M * (p.K >> 7);
        const int sub = tid & 15;
        for (int64_t gi = (int64_t)blockIdx.x * (kInnerWaves * 4) + (tid >> 4); gi < groups;
             gi += (int64_t)p.quant_wgs * (kInnerWaves * 4))
            quant_group(*(reinterpret_cast<const u32x4 *>(p.X + gi * 128) + sub), p.codes, p.scales, gi, sub);
        return;
    }
    __shared__ v4f red[kInnerWaves][64];
    constexpr uint32_t OOB = 0x7ffff000u;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int RT = (p.R + 15) >> 4;
    int b = (int)blockIdx.x - p.quant_wgs;
    const int rt = b % RT;
    b /= RT;
    const int first = b % p.share, m0 = b / p.share * 16;
    const int r16 = lane & 15, g = lane >> 4;
    const int K = p.K, chunks = K >> 6;
    int id = m0 + r16 < p.M ? p.ids[m0 + r16] : -1;
    if ((uint32_t)id >= (uint32_t)p.L)
        id = -1;
    uint32_t left = (uint32_t)__ballot(id >= 0) & 0xffffu;
    const __amdgpu_buffer_rsrc_t xres = buffer_rsrc(p.X + (size_t)m0 * K, 16u * (uint32_t)K * 2u);
    for (int number = 0; left != 0u; ++number) {
        const int a = __builtin_amdgcn_readlane(id, __builtin_ctz(left));
        left &= ~((uint32_t)__ballot(id == a) & 0xffffu);
        if (number % p.share != first)
            continue;
        const bool mine = id == a;
        const __amdgpu_buffer_rsrc_t ares = buffer_rsrc(p.A + (size_t)a * p.R * K, (uint32_t)p.R * (uint32_t)K * 2u);
        const int rank = 16 * rt + r16;
        const uint32_t aoff = rank < p.R ? (uint32_t)rank * (uint32_t)K * 2u + 32u * (uint32_t)g : OOB;
        const uint32_t xoff = mine ? (uint32_t)r16 * (uint32_t)K * 2u + 32u * (uint32_t)g : OOB;
        v4f acc = {0.f, 0.f, 0.f, 0.f};
        for (int c0 = wave; c0 < chunks; c0 += kInnerWaves * kInnerUnroll) {
            v4i ar[kInnerUnroll][2], xr[kInnerUnroll][2];
#pragma unroll
            for (int j = 0; j < kInnerUnroll; ++j) {
                const int c = c0 + j * kInnerWaves;
                const bool live = c < chunks;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    ar[j][h] = __builtin_amdgcn_raw_buffer_load_b128(ares, (int)(live ? aoff + 16 * h : OOB),
                                                                     live ? c * 128 : 0, 0);
                    xr[j][h] = __builtin_amdgcn_raw_buffer_load_b128(xres, (int)(live ? xoff + 16 * h : OOB),
                                                                     live ? c * 128 : 0, 0);
                }
            }
#pragma unroll
            for (int j = 0; j < kInnerUnroll; ++j)
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8b, ar[j][h]),
                                                                  __builtin_bit_cast(v8b, xr[j][h]), acc, 0, 0, 0);
        }
        red[wave][lane] = acc;
        __syncthreads();
        if (wave == 0) {
            v4f v = red[0][lane];
#pragma unroll
            for (int w = 1; w < kInnerWaves; ++w)
                v += red[w][lane];
            // lane: ranks 16 rt + 4 g .. + 4 of row r16, as two bf16 terms each (R is a multiple of 8)
            const int r = 16 * rt + 4 * g;
            if (mine && r < p.R) {
                const float sc = p.scaling[a];
                uint32_t hi[4], lo[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float f = v[i] * sc;
                    hi[i] = bf16_rne(f);
                    const float rest = f - __uint_as_float(hi[i] << 16);
                    lo[i] = rest - rest == 0.f ? bf16_rne(rest) : 0u;      // (no second term beside an inf or NaN)
                }
                uint16_t *to = p.V + (size_t)(m0 + r16) * 2 * p.R + r;
                *reinterpret_cast<uint2 *>(to) = make_uint2(hi[0] | (hi[1] << 16), hi[2] | (hi[3] << 16));
                *reinterpret_cast<uint2 *>(to + p.R) = make_uint2(lo[0] | (lo[1] << 16), lo[2] | (lo[3] << 16));
            }
        }
        __syncthreads();                                           // red is rewritten by the next adapter
    }
}

}  // namespace kern

namespace {

using namespace kern;

constexpr int kMaxRank = 256;
constexpr int64_t kMax32 = 0x7ffff000;   // 32-bit byte offsets inside one adapter, one 16-row tile

int64_t up256(int64_t n) { return (n + 255) & ~(int64_t)255; }

struct LoraLayout {
    int64_t codes, scales, v, bytes;   // offsets from the workspace's start
};

LoraLayout lora_layout(int64_t M, int64_t K, int64_t R)
{
    LoraLayout l;
    l.codes = A8W8_WORKSPACE_COUNTER_BYTES;
    l.scales = l.codes + up256(M * K);
    l.v = l.scales + up256(M * (K / 128) * 4);
    l.bytes = l.v + up256(M * 2 * R * 2);
    return l;
}

int check_lora_shape(int64_t M, int64_t N, int64_t K, int64_t L, int64_t R)
{
    const int rc = check_gemm_shape(M, N, K);
    if (rc != A8W8_OK)
        return rc;
    if (L < 1 || L > (1 << 20) || R < 8 || R > kMaxRank || R % 8 != 0 || N * R * 2 >= kMax32 || R * K * 2 >= kMax32 ||
        16 * K * 2 >= kMax32)
        return A8W8_ERR_SHAPE;
    return A8W8_OK;
}

}  // namespace
}  // namespace a8w8

using namespace a8w8;

extern "C" {

int gemm_a8w8_blockscale_lora_workspace_bytes(int64_t M, int64_t N, int64_t K, int32_t adapters, int32_t rank,
                                              int64_t *bytes)
{
    if (!bytes)
        return A8W8_ERR_NULL;
    const int rc = check_lora_shape(M, N, K, adapters, rank);
    if (rc != A8W8_OK)
        return rc;
    *bytes = M == 0 ? 0 : lora_layout(M, K, rank).bytes;
    return A8W8_OK;
}

int gemm_a8w8_blockscale_lora(const a8w8_lora_desc *d, void *stream)
{
    if (!d)
        return A8W8_ERR_NULL;
    int rc = check_lora_shape(d->M, d->N, d->K, d->adapters, d->rank);
    if (rc != A8W8_OK)
        return rc;
    if (d->w_packed < 0 || d->w_packed > 1)
        return A8W8_ERR_SHAPE;
    if (d->variant >= num_variants())
        return A8W8_ERR_PLAN;
    if (d->M == 0)
        return A8W8_OK;
    if (!d->X || !d->W || !d->w_scale || !d->A || !d->B || !d->scaling || !d->ids || !d->Y)
        return A8W8_ERR_NULL;
    if ((reinterpret_cast<uintptr_t>(d->X) & 15) || (reinterpret_cast<uintptr_t>(d->W) & 15) ||
        (reinterpret_cast<uintptr_t>(d->A) & 15) || (reinterpret_cast<uintptr_t>(d->B) & 15) ||
        (reinterpret_cast<uintptr_t>(d->w_scale) & 3) || (reinterpret_cast<uintptr_t>(d->scaling) & 3) ||
        (reinterpret_cast<uintptr_t>(d->ids) & 3) || (reinterpret_cast<uintptr_t>(d->Y) & 1) ||
        (reinterpret_cast<uintptr_t>(d->workspace) & 255))
        return A8W8_ERR_ALIGN;
    const LoraLayout l = lora_layout(d->M, d->K, d->rank);
    if (!d->workspace || d->workspace_bytes < l.bytes)
        return A8W8_ERR_WORKSPACE;
    int cus = 0;
    rc = device_ready(&cus);
    if (rc != A8W8_OK)
        return rc;
    if (d->variant >= 0 && !lora_accepts(d->variant, d->M, d->N, d->K, cus))
        return A8W8_ERR_PLAN;
    const int id = d->variant >= 0 ? d->variant : lora_variant(d->M, d->N, d->K, cus, d->w_packed != 0);
    uint8_t *ws = static_cast<uint8_t *>(d->workspace);
    hipStream_t st = static_cast<hipStream_t>(stream);

    InnerArgs in;
    in.X = static_cast<const uint16_t *>(d->X);
    in.A = static_cast<const uint16_t *>(d->A);
    in.scaling = d->scaling;
    in.ids = d->ids;
    in.codes = ws + l.codes;
    in.scales = reinterpret_cast<float *>(ws + l.scales);
    in.V = reinterpret_cast<uint16_t *>(ws + l.v);
    in.M = (int32_t)d->M;
    in.K = (int32_t)d->K;
    in.L = d->adapters;
    in.R = d->rank;
    const int64_t groups = d->M * (d->K / 128), qwgs = (groups + kInnerWaves * 4 - 1) / (kInnerWaves * 4);
    in.quant_wgs = (int32_t)(qwgs < 16 * cus ? qwgs : 16 * cus);
    const int64_t tiles = (d->M + 15) / 16, rts = (d->rank + 15) / 16;
    // Few rows: one workgroup per distinct adapter a tile can have; many: one takes them all
    // (most tiles of a prompt have one).
    int64_t share = d->M < 16 ? d->M : 16;
    if (share > d->adapters)
        share = d->adapters;
    if (tiles > 16)
        share = 1;
    in.share = (int32_t)share;
    hipLaunchKernelGGL(lora_inner_kernel, dim3((unsigned)(in.quant_wgs + tiles * rts * share)), dim3(kInnerWaves * 64), 0,
                       st, in);

    Args a;
    std::memset(&a, 0, sizeof(a));
    a.A = in.codes;
    a.a_scale = in.scales;
    a.W = static_cast<const uint8_t *>(d->W);
    a.w_scale = d->w_scale;
    a.Y = static_cast<uint16_t *>(d->Y);
    a.M = in.M;
    a.N = (int32_t)d->N;
    a.K = in.K;
    a.wpk = d->w_packed;
    a.splits = 1;
    a.lora = {in.V, static_cast<const uint16_t *>(d->B), d->ids, d->adapters, d->rank};
    if (launch_lora(id, a, cus, st) != hipSuccess || hipGetLastError() != hipSuccess)
        return A8W8_ERR_HIP;
    return A8W8_OK;
}

}  // extern "C"
