// a8w8_attention.hip -- attention of the new tokens of several sequences over a paged cache,
// for gfx950.
//
// Row i of the n new tokens of a sequence of `len` tokens (the new ones included, their keys
// already in the cache) stands at p = len - n + i and sees the keys j <= p; with a window only
// j > p - window, and the first `sinks` tokens:
//
//   out = (sum_j softmax_j(scale q . k_j) v_j) * sigmoid(gate)         (gate optional)
//
// A row that sees nothing gets zeros.  Softmax statistics and sums in fp32.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "a8w8_device.h"
#include "a8w8_internal.h"
#include "a8w8_quant_math.h"
#include "gemm_a8w8_blockscale.h"

namespace a8w8 {
namespace kern {

struct AttnArgs {
    const uint16_t *q, *gate;
    int64_t q_row, q_head, gate_row, gate_head;
    const uint8_t *k, *v;
    const float *k_scale, *v_scale;
    const int32_t *table, *q_start, *lens;
    uint16_t *out;
    int64_t T;
    int32_t B, P, pages, page_shift, Hq, Hkv, G, window, sinks;
    float scale;
};

template <bool FP8>
__device__ __forceinline__ float cached(const uint8_t *base, int64_t i)
{
    if constexpr (FP8)
        return __builtin_amdgcn_cvt_f32_fp8(base[i], 0);
    else
        return __uint_as_float((uint32_t) reinterpret_cast<const uint16_t *>(base)[i] << 16);
}

// One workgroup per row and query head; each wave takes every fourth key, a lane D/64 dimensions.
template <int D, bool FP8>
__global__ __launch_bounds__(256) void attention_kernel(AttnArgs p)
{
    constexpr int E = D / 64;
    __shared__ float part[4][D + 2];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int t = blockIdx.x, h = blockIdx.y;
    int b = -1, first = 0, n = 0;
    for (int i = 0; i < p.B; ++i) {
        const int s = p.q_start[i], e = p.q_start[i + 1];
        if (s >= 0 && e <= p.T && t >= s && t < e)
            b = i, first = s, n = e - s;
    }
    if (b < 0)
        return;
    const int pos = p.lens[b] - n + (t - first), hk = h / p.G;
    const int64_t keys = (int64_t)p.P << p.page_shift;
    const int end = (int)(pos + 1 < keys ? pos + 1 : keys);
    float q[E], o[E], m = -INFINITY, l = 0.0f;
#pragma unroll
    for (int e = 0; e < E; ++e) {
        q[e] = __uint_as_float((uint32_t)p.q[t * p.q_row + h * p.q_head + lane * E + e] << 16);
        o[e] = 0.0f;
    }
    const float sc = p.scale * (p.k_scale ? p.k_scale[hk] : 1.0f);
    for (int j = wave; j < end; j += 4) {
        if (p.window && j <= pos - p.window && j >= p.sinks)
            continue;
        const int page = p.table[(int64_t)b * p.P + (j >> p.page_shift)];
        if (page < 0 || page >= p.pages)
            continue;
        const int64_t at = ((((int64_t)page << p.page_shift) + (j & ((1 << p.page_shift) - 1))) * p.Hkv + hk) * D + lane * E;
        float s = 0.0f;
#pragma unroll
        for (int e = 0; e < E; ++e)
            s = __builtin_fmaf(q[e], cached<FP8>(p.k, at + e), s);
        for (int x = 32; x; x >>= 1)
            s += __shfl_xor(s, x);
        s *= sc;
        const float mn = fmaxf(m, s), a = m == -INFINITY ? 0.0f : __expf(m - mn), w = __expf(s - mn);
        m = mn;
        l = l * a + w;
#pragma unroll
        for (int e = 0; e < E; ++e)
            o[e] = o[e] * a + w * cached<FP8>(p.v, at + e);
    }
#pragma unroll
    for (int e = 0; e < E; ++e)
        part[wave][lane * E + e] = o[e];
    if (lane == 0)
        part[wave][D] = m, part[wave][D + 1] = l;
    __syncthreads();
    if (wave)
        return;
    float M = -INFINITY, L = 0.0f;
    for (int w = 0; w < 4; ++w)
        M = fmaxf(M, part[w][D]);
    for (int w = 0; w < 4; ++w)
        L += part[w][D] == -INFINITY ? 0.0f : part[w][D + 1] * __expf(part[w][D] - M);
#pragma unroll
    for (int e = 0; e < E; ++e) {
        float x = 0.0f;
        for (int w = 0; w < 4; ++w)
            x += part[w][D] == -INFINITY ? 0.0f : part[w][lane * E + e] * __expf(part[w][D] - M);
        x = M == -INFINITY ? 0.0f : x / L * (p.v_scale ? p.v_scale[hk] : 1.0f);
        if (p.gate)
            x /= 1.0f + __expf(-__uint_as_float((uint32_t)p.gate[t * p.gate_row + h * p.gate_head + lane * E + e] << 16));
        p.out[((int64_t)t * p.Hq + h) * D + lane * E + e] = (uint16_t)bf16_rne(x);
    }
}

}  // namespace kern

namespace {

bool misaligned(const void *p, uintptr_t mask) { return (reinterpret_cast<uintptr_t>(p) & mask) != 0; }

int check_attention_shape(int64_t T, int64_t B, int32_t q_heads, int32_t kv_heads, int32_t head_dim, int32_t cache_dtype)
{
    if (T < 0 || T > (1 << 22) || B < 0 || B > 4096 || kv_heads < 1 || q_heads < kv_heads || q_heads > 1024 ||
        q_heads % kv_heads != 0 || q_heads / kv_heads > 64 || (head_dim != 64 && head_dim != 128 && head_dim != 256) ||
        cache_dtype < 0 || cache_dtype > 1)
        return A8W8_ERR_SHAPE;
    return A8W8_OK;
}

}  // namespace
}  // namespace a8w8

using namespace a8w8;

extern "C" {

int a8w8_paged_attention_workspace_bytes(int64_t T, int64_t B, int32_t q_heads, int32_t kv_heads, int32_t head_dim,
                                         int32_t cache_dtype, int32_t cu_count, int64_t *bytes)
{
    if (!bytes)
        return A8W8_ERR_NULL;
    const int rc = check_attention_shape(T, B, q_heads, kv_heads, head_dim, cache_dtype);
    if (rc != A8W8_OK)
        return rc;
    *bytes = T == 0 || B == 0 ? 0 : A8W8_WORKSPACE_COUNTER_BYTES;
    return A8W8_OK;
}

int a8w8_paged_attention(const a8w8_attention_desc *d, void *stream)
{
    if (!d)
        return A8W8_ERR_NULL;
    int rc = check_attention_shape(d->T, d->B, d->q_heads, d->kv_heads, d->head_dim, d->cache_dtype);
    if (rc != A8W8_OK)
        return rc;
    if (d->pages < 1 || d->table_pages < 1 || d->page_size < 1 || d->page_size > 65536 || (d->page_size & (d->page_size - 1)) ||
        d->pages > (1ll << 31) / d->page_size || d->table_pages > (1ll << 30) / d->page_size || d->window < 0 || d->sinks < 0 ||
        d->max_new < 0 || d->scale != d->scale)
        return A8W8_ERR_SHAPE;
    for (const int64_t s : {d->q_row, d->q_head, d->gate ? d->gate_row : 0, d->gate ? d->gate_head : 0})
        if (s < 0 || s % 8 != 0)
            return A8W8_ERR_SHAPE;
    if (d->T == 0 || d->B == 0)
        return A8W8_OK;
    if (!d->q || !d->k_cache || !d->v_cache || !d->page_table || !d->q_start || !d->kv_lens || !d->out)
        return A8W8_ERR_NULL;
    if (misaligned(d->q, 15) || misaligned(d->gate, 15) || misaligned(d->k_cache, 15) || misaligned(d->v_cache, 15) ||
        misaligned(d->out, 15) || misaligned(d->k_scale, 3) || misaligned(d->v_scale, 3) || misaligned(d->page_table, 3) ||
        misaligned(d->q_start, 3) || misaligned(d->kv_lens, 3) || misaligned(d->workspace, 255))
        return A8W8_ERR_ALIGN;
    int cus = 0;
    rc = device_ready(&cus);
    if (rc != A8W8_OK)
        return rc;
    int64_t need = 0;
    rc = a8w8_paged_attention_workspace_bytes(d->T, d->B, d->q_heads, d->kv_heads, d->head_dim, d->cache_dtype, cus, &need);
    if (rc != A8W8_OK)
        return rc;
    if (!d->workspace || d->workspace_bytes < need)
        return A8W8_ERR_WORKSPACE;
    kern::AttnArgs a;
    a.q = static_cast<const uint16_t *>(d->q), a.gate = static_cast<const uint16_t *>(d->gate);
    a.q_row = d->q_row, a.q_head = d->q_head, a.gate_row = d->gate_row, a.gate_head = d->gate_head;
    a.k = static_cast<const uint8_t *>(d->k_cache), a.v = static_cast<const uint8_t *>(d->v_cache);
    a.k_scale = d->k_scale, a.v_scale = d->v_scale;
    a.table = d->page_table, a.q_start = d->q_start, a.lens = d->kv_lens;
    a.out = static_cast<uint16_t *>(d->out);
    a.T = d->T, a.B = (int32_t)d->B, a.P = (int32_t)d->table_pages, a.pages = (int32_t)d->pages;
    a.page_shift = __builtin_ctz((unsigned)d->page_size);
    a.Hq = d->q_heads, a.Hkv = d->kv_heads, a.G = d->q_heads / d->kv_heads, a.window = d->window, a.sinks = d->sinks;
    a.scale = d->scale;
    const bool f8 = d->cache_dtype == A8W8_CACHE_E4M3;
    const auto f = d->head_dim == 64 ? (f8 ? kern::attention_kernel<64, true> : kern::attention_kernel<64, false>)
                 : d->head_dim == 128 ? (f8 ? kern::attention_kernel<128, true> : kern::attention_kernel<128, false>)
                                      : (f8 ? kern::attention_kernel<256, true> : kern::attention_kernel<256, false>);
    hipLaunchKernelGGL(f, dim3((unsigned)d->T, (unsigned)d->q_heads), dim3(256), 0, static_cast<hipStream_t>(stream), a);
    return hipGetLastError() == hipSuccess ? A8W8_OK : A8W8_ERR_HIP;
}

}  // extern "C"
