// a8w8_lora.hip -- low-rank adapters of many requests at once beside one shared a8w8
// projection, for gfx950:
//
//   Y[m] = bf16( a8w8 product of x_m quantised per 1 x 128 group with W
//                + scaling[a] * B[a] (A[a] x_m) )            a = ids[m], none if negative
//
// First X is quantised to the codes and scales the GEMM takes -- the step that precedes every
// a8w8 GEMM -- and the inner products V[m] = scaling[a] A[a] x_m are formed in
// other workgroups of the same launch.  Then the a8w8 GEMM adds
// B[a] V[m] to its fp32 accumulators before it rounds them (lora_add in a8w8_kernels.hip);
// for few rows on tile instances lora_expand_kernel forms those products beforehand.
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
    int32_t inner_wgs;      // workgroups that form inner products; the rest quantise
    int32_t quant_wgs;
    int32_t RS;             // workgroups per run of rows that share their ranks out
    int32_t width, expand_width;   // rows of a workgroup's run (a power of two up to 128): inner products, expansion
    const uint16_t *B;      // bf16 [L, N, R]      (expansion)
    float *D;               // fp32 [M][ldd]
    int32_t N, ldd;
};

constexpr int kInnerRows = 128;   // rows of a chunk

// Workgroups past the inner products' quantise X: one 1 x 128 group per 16 lanes of NW waves.
template <int NW>
__device__ __forceinline__ void quantise_part(const InnerArgs &p)
{
    const int64_t groups = (int64_t)p.M * (p.K >> 7);
    const int sub = threadIdx.x & 15;
    for (int64_t gi = (int64_t)((int)blockIdx.x - p.inner_wgs) * (NW * 4) + (threadIdx.x >> 4); gi < groups;
         gi += (int64_t)p.quant_wgs * (NW * 4))
        quant_group<true>(*(reinterpret_cast<const u32x4 *>(p.X + gi * 128) + sub), p.codes, p.scales, gi, sub);
}

// The work on low-rank products.  The rows are taken 128 at a time; the rows of a chunk that
// use one adapter, wherever in the chunk they are, are gathered into groups of ROWS, so that
// the adapter is read once per group and not once per row.  A group belongs to the
// workgroup whose rows hold its first one: the workgroup of rows [r0, r0 + width) calls
// task(a, row) for each, with lane l's row of the chunk the (l % ROWS)-th of the group
// (-1: none).  No list is made, and a workgroup without a group costs one look at the ids.
template <int ROWS, typename Task>
__device__ __forceinline__ void for_groups(const int32_t *ids, int M, int L, int m0, int r0, int width, Task task)
{
    const int lane = threadIdx.x & 63;
    int id[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int m = m0 + 64 * h + lane;
        id[h] = m < M ? ids[m] : -1;
    }
    for (int r = r0; r < r0 + width; ++r) {
        const int a = __builtin_amdgcn_readlane(r < 64 ? id[0] : id[1], r & 63);
        if ((uint32_t)a >= (uint32_t)L)
            continue;
        const uint64_t rows0 = __ballot(id[0] == a), rows1 = __ballot(id[1] == a);
        // Each lane's rows' places among the adapter's, in row order.
        const int in0 = __builtin_popcountll(rows0);
        const int pos0 = __builtin_amdgcn_mbcnt_hi((uint32_t)(rows0 >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)rows0, 0));
        const int pos1 = in0 + __builtin_amdgcn_mbcnt_hi((uint32_t)(rows1 >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)rows1, 0));
        const int first = __builtin_amdgcn_readlane(r < 64 ? pos0 : pos1, r & 63);
        if (first % ROWS != 0)
            continue;
        // Each row is pushed to the lane of its place (the others to lane 63, which is no
        // place), then read by every lane that stands for the place.
        const int to0 = id[0] == a && pos0 - first >= 0 && pos0 - first < ROWS ? pos0 - first : 63;
        const int to1 = id[1] == a && pos1 - first >= 0 && pos1 - first < ROWS ? pos1 - first : 63;
        const int got = max(__builtin_amdgcn_ds_permute(4 * to0, lane + 1), __builtin_amdgcn_ds_permute(4 * to1, lane + 65));
        task(a, __builtin_amdgcn_ds_bpermute(4 * (lane % ROWS), got) - 1);
    }
}

// Four consecutive inner values of a row, times the adapter's scaling, as two bf16 terms each.
__device__ __forceinline__ void store_inner(const InnerArgs &p, int m, int r, float sc, v4f v)
{
    uint32_t hi[4], lo[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float f = v[i] * sc;
        hi[i] = bf16_rne(f);
        const float rest = f - __uint_as_float(hi[i] << 16);
        lo[i] = rest - rest == 0.f ? bf16_rne(rest) : 0u;      // (no second term beside an inf or NaN)
    }
    uint16_t *to = p.V + (size_t)m * 2 * p.R + r;
    *reinterpret_cast<uint2 *>(to) = make_uint2(hi[0] | (hi[1] << 16), hi[2] | (hi[3] << 16));
    *reinterpret_cast<uint2 *>(to + p.R) = make_uint2(lo[0] | (lo[1] << 16), lo[2] | (lo[3] << 16));
}

// Inner products of few rows: a workgroup forms 4 ranks of up to 4 rows with
// v_mfma_f32_4x4x4_16b_bf16, whose 16 blocks take 16 pieces of K: lane l holds row l % 4 of
// either operand and 16 bytes of K at 16 (l / 4) of a 256-byte chunk, so that every lane of a
// load carries data (a 16 x 16 product of one row would issue the same loads for 15 empty
// ones).  The waves take U chunks each at a time; a wave's 16 block sums are added across
// its lanes, the waves' through LDS, both in a fixed order.  Bound by the latency of one
// chain ids -> A -> V, hence 4 ranks per workgroup.
constexpr int kFewWaves = 4;

template <int U>
__global__ __launch_bounds__(kFewWaves * 64) void lora_inner_few_kernel(InnerArgs p)
{
    if ((int)blockIdx.x >= p.inner_wgs) {
        quantise_part<kFewWaves>(p);
        return;
    }
    __shared__ v4f red[kFewWaves][4];
    constexpr uint32_t OOB = 0x7ffff000u;
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    // The runs of rows that take the same ranks on one XCD: its L2 reads their part of A once.
    const int runs = p.inner_wgs / p.RS, item = xcd_item((int)blockIdx.x, p.inner_wgs);
    const int at = item % runs * p.width, m0 = at / kInnerRows * kInnerRows;
    const int K = p.K, chunks = K >> 7;
    const __amdgpu_buffer_rsrc_t xres = buffer_rsrc(p.X + (size_t)m0 * K, (uint32_t)min(p.M - m0, kInnerRows) * (uint32_t)K * 2u);
    for_groups<4>(p.ids, p.M, p.L, m0, at - m0, p.width, [&](int a, int row) __attribute__((always_inline)) {
        const float scaling = p.scaling[a];
        const __amdgpu_buffer_rsrc_t ares = buffer_rsrc(p.A + (size_t)a * p.R * K, (uint32_t)p.R * (uint32_t)K * 2u);
        const uint32_t xoff = row >= 0 ? (uint32_t)row * (uint32_t)K * 2u + 16u * (uint32_t)(lane >> 2) : OOB;
        v4i xr[U];                                     // read once for all ranks where the waves take K at one go
        for (int rank0 = item / runs * 4, fresh = 1; rank0 < p.R; rank0 += 4 * p.RS, fresh = chunks > kFewWaves * U) {
            const uint32_t aoff = (uint32_t)(rank0 + (lane & 3)) * (uint32_t)K * 2u + 16u * (uint32_t)(lane >> 2);
            v4f acc = {0.f, 0.f, 0.f, 0.f};
            for (int c0 = wave; c0 < chunks; c0 += kFewWaves * U) {
                v4i ar[U];
#pragma unroll
                for (int j = 0; j < U; ++j) {
                    const int c = c0 + j * kFewWaves;
                    ar[j] = __builtin_amdgcn_raw_buffer_load_b128(ares, (int)(c < chunks ? aoff : OOB), c < chunks ? c * 256 : 0, 0);
                }
                if (fresh) {
#pragma unroll
                    for (int j = 0; j < U; ++j) {
                        const int c = c0 + j * kFewWaves;
                        xr[j] = __builtin_amdgcn_raw_buffer_load_b128(xres, (int)(c < chunks ? xoff : OOB),
                                                                      c < chunks ? c * 256 : 0, 0);
                    }
                }
                __builtin_amdgcn_sched_barrier(0);     // every load out before the first product
#pragma unroll
                for (int j = 0; j < U; ++j)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const v2u w = {(uint32_t)ar[j][2 * h], (uint32_t)ar[j][2 * h + 1]};
                        const v2u x = {(uint32_t)xr[j][2 * h], (uint32_t)xr[j][2 * h + 1]};
                        acc = __builtin_amdgcn_mfma_f32_4x4x4bf16_1k(__builtin_bit_cast(v4s, w), __builtin_bit_cast(v4s, x), acc,
                                                                     0, 0, 0);
                    }
            }
#pragma unroll
            for (int d = 4; d < 64; d <<= 1)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    acc[i] += __shfl_xor(acc[i], d);
            if (lane < 4)
                red[wave][lane] = acc;
            __syncthreads();
            if (wave == 0 && lane < 4 && row >= 0) {
                v4f v = red[0][lane];
#pragma unroll
                for (int w = 1; w < kFewWaves; ++w)
                    v += red[w][lane];
                store_inner(p, m0 + row, rank0, scaling, v);
            }
            __syncthreads();                                           // red is rewritten by the next ranks
        }
    });
}

// Inner products of more rows: a workgroup forms 16 ranks of up to 16 rows.  Matrix operands
// are rows of A[a], then the gathered rows of X, both straight from memory in one K order
// (lane l: row l % 16, 16 bytes 16 (l / 16) .. of each 64-byte half of a 128-byte chunk of K).
// The waves take U such chunks each at a time; their partials are summed through LDS in wave
// order.
constexpr int kInnerWaves = 8;

template <int U>
__global__ __launch_bounds__(kInnerWaves * 64) void lora_inner_kernel(InnerArgs p)
{
    __shared__ v4f red[kInnerWaves][64];
    constexpr uint32_t OOB = 0x7ffff000u;
    const int lane = threadIdx.x & 63, r16 = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    if ((int)blockIdx.x >= p.inner_wgs) {
        quantise_part<kInnerWaves>(p);
        return;
    }
    // Neighbouring runs of rows (a prompt's: one adapter) and the ranks of a run on one XCD: each
    // XCD's L2 then reads a few adapters and its rows of X once (2048 rows, 16 adapters of
    // rank 32).
    const int item = xcd_item((int)blockIdx.x, p.inner_wgs);
    const int at = item / p.RS * p.width, m0 = at / kInnerRows * kInnerRows;
    const int rank0 = item % p.RS * 16;
    const int K = p.K, chunks = K >> 6;
    const uint32_t aoff = rank0 + r16 < p.R ? (uint32_t)(rank0 + r16) * (uint32_t)K * 2u + 16u * (uint32_t)g : OOB;
    const __amdgpu_buffer_rsrc_t xres = buffer_rsrc(p.X + (size_t)m0 * K, (uint32_t)min(p.M - m0, kInnerRows) * (uint32_t)K * 2u);
    for_groups<16>(p.ids, p.M, p.L, m0, at - m0, p.width, [&](int a, int row) __attribute__((always_inline)) {
        const __amdgpu_buffer_rsrc_t ares = buffer_rsrc(p.A + (size_t)a * p.R * K, (uint32_t)p.R * (uint32_t)K * 2u);
        const uint32_t xoff = row >= 0 ? (uint32_t)row * (uint32_t)K * 2u + 16u * (uint32_t)g : OOB;
        v4f acc = {0.f, 0.f, 0.f, 0.f};
        for (int c0 = wave; c0 < chunks; c0 += kInnerWaves * U) {
            v4i ar[U][2], xr[U][2];
#pragma unroll
            for (int j = 0; j < U; ++j) {
                const int c = c0 + j * kInnerWaves;
                const bool live = c < chunks;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    ar[j][h] = __builtin_amdgcn_raw_buffer_load_b128(ares, (int)(live ? aoff + 64 * h : OOB),
                                                                     live ? c * 128 : 0, 0);
                    xr[j][h] = __builtin_amdgcn_raw_buffer_load_b128(xres, (int)(live ? xoff + 64 * h : OOB),
                                                                     live ? c * 128 : 0, 0);
                }
            }
            __builtin_amdgcn_sched_barrier(0);     // every load out before the first product
#pragma unroll
            for (int j = 0; j < U; ++j)
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
            const int r = rank0 + 4 * g;                           // four ranks of the lane's row (R is a multiple of 4)
            if (row >= 0 && r < p.R)
                store_inner(p, m0 + row, r, p.scaling[a], v);
        }
        __syncthreads();                                           // red is rewritten by the next group
    });
}

// Expansion D[m] = B[a] V[m] for calls of few rows on tiles: a workgroup takes a group of up
// to 16 rows of one adapter and 128 columns, a wave 32 of them (two 16-row fragments of B),
// so that B is read once per group (133 rows, 24 adapters of 5120 x 64: 8.6 us, 9.9 with
// 256 columns).  D is fp32: the GEMM adds it to its accumulators.
constexpr int kExpandCols = 128;

__global__ __launch_bounds__(256) void lora_expand_kernel(InnerArgs p)
{
    constexpr uint32_t OOB = 0x7ffff000u;
    constexpr int TN = 2, KS = 2;
    const int lane = threadIdx.x & 63, r16 = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int CBS = (p.N + kExpandCols - 1) / kExpandCols;
    const int at = (int)blockIdx.x / CBS * p.expand_width, m0 = at / kInnerRows * kInnerRows;
    const int n0 = (int)blockIdx.x % CBS * kExpandCols + wave * 16 * TN;
    for_groups<16>(p.ids, p.M, p.L, m0, at - m0, p.expand_width, [&](int a, int row) __attribute__((always_inline)) {
        const int R = p.R;
        const __amdgpu_buffer_rsrc_t vres = buffer_rsrc(p.V + (size_t)m0 * 2 * R, (uint32_t)kInnerRows * (uint32_t)R * 4u);
        const __amdgpu_buffer_rsrc_t bres = buffer_rsrc(p.B + (size_t)a * p.N * R, (uint32_t)p.N * (uint32_t)R * 2u);
        v4f acc[TN];
#pragma unroll
        for (int u = 0; u < TN; ++u)
            acc[u] = (v4f){0.f, 0.f, 0.f, 0.f};
        for (int k0 = 0; k0 < R; k0 += 32 * KS) {
            v4i br[KS][TN], v[KS][2];
#pragma unroll
            for (int s = 0; s < KS; ++s) {
                const int k = k0 + 32 * s + 8 * g;
#pragma unroll
                for (int u = 0; u < TN; ++u) {
                    const int n = n0 + 16 * u + r16;
                    br[s][u] = __builtin_amdgcn_raw_buffer_load_b128(
                        bres, k < R && n < p.N ? (int)(((uint32_t)n * (uint32_t)R + (uint32_t)k) * 2u) : (int)OOB, 0, 0);
                }
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    v[s][h] = __builtin_amdgcn_raw_buffer_load_b128(
                        vres, k < R && row >= 0 ? (row * 2 * R + h * R + k) * 2 : (int)OOB, 0, 0);
            }
#pragma unroll
            for (int s = 0; s < KS; ++s)
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int u = 0; u < TN; ++u)
                        acc[u] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8b, br[s][u]),
                                                                         __builtin_bit_cast(v8b, v[s][h]), acc[u], 0, 0, 0);
        }
        if (row >= 0) {
#pragma unroll
            for (int u = 0; u < TN; ++u) {
                const int n = n0 + 16 * u + 4 * g;
                if (n < p.ldd)
                    *reinterpret_cast<v4f *>(p.D + (size_t)(m0 + row) * p.ldd + n) = acc[u];
            }
        }
    });
}

}  // namespace kern

namespace {

using namespace kern;

constexpr int kMaxRank = 256;
constexpr int64_t kFewRows = 512;
constexpr int64_t kMax32 = 0x7ffff000;   // 32-bit byte offsets inside one adapter, one 16-row tile

int64_t up256(int64_t n) { return (n + 255) & ~(int64_t)255; }

struct LoraLayout {
    int64_t codes, scales, v, d, bytes;   // offsets from the workspace's start
};

int64_t d_stride(int64_t N) { return (N + 3) & ~(int64_t)3; }

LoraLayout lora_layout(int64_t M, int64_t N, int64_t K, int64_t R)
{
    LoraLayout l;
    l.codes = A8W8_WORKSPACE_COUNTER_BYTES;
    l.scales = l.codes + up256(M * K);
    l.v = l.scales + up256(M * (K / 128) * 4);
    l.d = l.v + up256(M * 2 * R * 2);
    l.bytes = l.d + (M <= kFewRows ? up256(M * d_stride(N) * 4) : 0);
    return l;
}

int check_lora_shape(int64_t M, int64_t N, int64_t K, int64_t L, int64_t R)
{
    const int rc = check_gemm_shape(M, N, K);
    if (rc != A8W8_OK)
        return rc;
    if (N > (1 << 22) || L < 1 || L > (1 << 20) || R < 8 || R > kMaxRank || R % 8 != 0 || N * R * 2 >= kMax32 || R * K * 2 >= kMax32 ||
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
    *bytes = M == 0 ? 0 : lora_layout(M, N, K, rank).bytes;
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
    const LoraLayout l = lora_layout(d->M, d->N, d->K, d->rank);
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
    // Up to kFewRows rows: groups of 4 rows, 4 ranks a workgroup, runs of one row (a decode batch's
    // adapters differ).  Above: groups of 16 rows, 16 ranks a workgroup, runs of 16 rows
    // (of a prompt each starts a group).  The quantisation's workgroups come after those.
    const bool few = d->M <= kFewRows;
    const int waves = few ? kFewWaves : kInnerWaves;
    const int64_t groups = d->M * (d->K / 128), qwgs = (groups + waves * 4 - 1) / (waves * 4);
    in.quant_wgs = (int32_t)(qwgs < 8 * cus ? qwgs : 8 * cus);
    in.RS = few ? d->rank / 4 : (d->rank + 15) / 16;
    in.width = few ? 1 : 16;
    in.expand_width = d->M <= 128 ? 1 : 2;
    in.inner_wgs = (int32_t)((d->M + in.width - 1) / in.width * in.RS);
    in.B = static_cast<const uint16_t *>(d->B);
    in.N = (int32_t)d->N;
    in.ldd = (int32_t)d_stride(d->N);
    // Tiles of few rows: the low-rank products are formed beforehand, adapter by adapter.
    in.D = few && variant(id).kernel != A8W8_KERNEL_RSKINNY ? reinterpret_cast<float *>(ws + l.d) : nullptr;
    const dim3 grid((unsigned)(in.inner_wgs + in.quant_wgs)), block(waves * 64);
    if (few)
        hipLaunchKernelGGL(lora_inner_few_kernel<12>, grid, block, 0, st, in);
    else
        hipLaunchKernelGGL(lora_inner_kernel<5>, grid, block, 0, st, in);
    if (in.D != nullptr)
        hipLaunchKernelGGL(lora_expand_kernel, dim3((unsigned)((d->M + in.expand_width - 1) / in.expand_width * ((d->N + kExpandCols - 1) / kExpandCols))), dim3(256),
                           0, st, in);

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
    a.lora = {in.V, in.B, d->ids, in.D, d->adapters, d->rank, in.ldd};
    if (launch_lora(id, a, cus, st) != hipSuccess || hipGetLastError() != hipSuccess)
        return A8W8_ERR_HIP;
    return A8W8_OK;
}

}  // extern "C"
