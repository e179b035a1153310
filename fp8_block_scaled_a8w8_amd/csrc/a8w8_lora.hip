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

#include <algorithm>
#include <cstring>

#include "a8w8_device.h"
#include "a8w8_internal.h"
#include "a8w8_quant_math.h"
#include "gemm_a8w8_blockscale.h"

namespace a8w8 {
namespace kern {

// Up to 16 rows of one adapter (-1: no such group; no such row).
struct ExpandGroup {
    int32_t adapter, row[16];
};

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
    int32_t RS;             // workgroups that share the ranks of a run of rows, or of a group, out
    int32_t subs;                  // workgroups that share a run's groups out, many rows
    int32_t groups, expand_groups; // workgroups per chunk: inner products of few rows, expansion
    int32_t id_bits;               // of an adapter's number
    int32_t quotient;              // group scales are amax / 448, else amax times the fp32 reciprocal
    ExpandGroup *list;             // [chunk of 256 rows][expand_groups]
    const uint16_t *B;      // bf16 [L, N, R]      (expansion)
    float *D;               // fp32 [M][ldd]
    int32_t N, ldd;
};

constexpr int kInnerRows = 128;   // rows of a chunk
constexpr int kRunRows = 16;      // rows of a workgroup's run, many rows

// Workgroups past the inner products' quantise X: one 1 x 128 group per 16 lanes of NW waves, with
// either rounding of the group's scale.
template <int NW>
__device__ __forceinline__ void quantise_part(const InnerArgs &p)
{
    const int64_t groups = (int64_t)p.M * (p.K >> 7);
    const int sub = threadIdx.x & 15;
    for (int64_t gi = (int64_t)((int)blockIdx.x - p.inner_wgs) * (NW * 4) + (threadIdx.x >> 4); gi < groups;
         gi += (int64_t)p.quant_wgs * (NW * 4)) {
        const u32x4 x = *(reinterpret_cast<const u32x4 *>(p.X + gi * 128) + sub);
        if (p.quotient)
            quant_group<false>(x, p.codes, p.scales, gi, sub);
        else
            quant_group<true>(x, p.codes, p.scales, gi, sub);
    }
}

// The row of the chunk at place lane % ROWS of a group (-1: none), from the places of the lane's
// W rows (lane, lane + 64, ...; outside 0 .. ROWS - 1: not of the group).  Each row is pushed to
// the lane of its place (the others to lane 63, which is no place), then read by every lane that
// stands for the place.
template <int ROWS, int W>
__device__ __forceinline__ int group_row(const int (&place)[W])
{
    const int lane = threadIdx.x & 63;
    int got = 0;
#pragma unroll
    for (int h = 0; h < W; ++h)
        got = max(got, __builtin_amdgcn_ds_permute(4 * (place[h] >= 0 && place[h] < ROWS ? place[h] : 63), 64 * h + lane + 1));
    return __builtin_amdgcn_ds_bpermute(4 * (lane % ROWS), got) - 1;
}

// The work on low-rank products.  The rows are taken 128 at a time; the rows of a chunk that
// use one adapter, wherever in the chunk they are, are gathered into groups of ROWS, so that
// the adapter is read once per group and not once per row.  A group belongs to the
// workgroup whose rows hold its first one: the workgroup of rows [r0, r0 + width) calls
// task(a, row) for each, with lane l's row of the chunk the (l % ROWS)-th of the group
// (-1: none); of `subs` such workgroups number `sub` takes every subs-th of them.  No list is
// made, and a workgroup without a group costs one look at the ids.
template <int ROWS, typename Task>
__device__ __forceinline__ void for_groups(const int32_t *ids, int M, int L, int m0, int r0, int width, int sub, int subs, Task task)
{
    const int lane = threadIdx.x & 63;
    int id[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int m = m0 + 64 * h + lane;
        id[h] = m < M ? ids[m] : -1;
    }
    int nth = 0;
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
        if (nth++ % subs != sub)
            continue;
        const int place[2] = {id[0] == a ? pos0 - first : -1, id[1] == a ? pos1 - first : -1};
        task(a, group_row<ROWS>(place));
    }
}

// Which rows of a chunk of 256 have the adapter of row 64 h + lane, by comparing the ids bit by
// bit: the row's place among them, the first of them, and whether it has an adapter at all.
constexpr int kWideRows = 256, kWords = kWideRows / 64;

struct Ids {
    int id[kWords];                                // lane's rows lane, lane + 64, ..
    uint64_t valid[kWords];
};
__device__ __forceinline__ Ids load_ids(const int32_t *ids, int M, int L, int m0)
{
    Ids x;
#pragma unroll
    for (int w = 0; w < kWords; ++w) {
        const int m = m0 + 64 * w + (int)(threadIdx.x & 63);
        x.id[w] = m < M ? ids[m] : -1;
    }
#pragma unroll
    for (int w = 0; w < kWords; ++w)
        x.valid[w] = __ballot((uint32_t)x.id[w] < (uint32_t)L);
    return x;
}
__device__ __forceinline__ void count_before(const Ids &x, int bits, int (&pos)[kWords], int (&first)[kWords])
{
    uint64_t eq[kWords][kWords];
#pragma unroll
    for (int h = 0; h < kWords; ++h)
#pragma unroll
        for (int w = 0; w <= h; ++w)
            eq[h][w] = x.valid[w];
    for (int b = 0; b < bits; ++b) {
        uint64_t set[kWords];
#pragma unroll
        for (int w = 0; w < kWords; ++w)
            set[w] = __ballot((x.id[w] >> b & 1) != 0);
#pragma unroll
        for (int h = 0; h < kWords; ++h) {
            const uint64_t flip = (uint64_t)(int64_t)((x.id[h] >> b & 1) - 1);
#pragma unroll
            for (int w = 0; w <= h; ++w)           // (later rows do not count)
                eq[h][w] &= set[w] ^ flip;
        }
    }
    const uint64_t below = ((uint64_t)1 << (threadIdx.x & 63)) - 1;
#pragma unroll
    for (int h = 0; h < kWords; ++h) {
        pos[h] = __builtin_popcountll(eq[h][h] & below);
        first[h] = 64 * h + (int)(threadIdx.x & 63);
        if (pos[h] > 0)
            first[h] = 64 * h + __builtin_ctzll(eq[h][h]);
#pragma unroll
        for (int w = h - 1; w >= 0; --w) {
            pos[h] += __builtin_popcountll(eq[h][w]);
            first[h] = eq[h][w] != 0 ? 64 * w + __builtin_ctzll(eq[h][w]) : first[h];
        }
    }
}

// The j-th of such groups of a chunk of 256 rows alone: task(a, row) once, or never if the chunk
// has fewer.  For rows of few adapters, where the groups' first rows lie unevenly and a
// workgroup per row leaves some CUs two or three groups and others none (128 rows, 24
// adapters of 6144 x 64: 9.7 us against 13.1).
template <int ROWS, typename Task>
__device__ __forceinline__ void one_group(const int32_t *ids, int M, int L, int bits, int m0, int j, Task task)
{
    const Ids x = load_ids(ids, M, L, m0);
    int pos[kWords], unused[kWords], a = -1, first = 0, before = 0;
    count_before(x, bits, pos, unused);
#pragma unroll
    for (int h = 0; h < kWords; ++h) {
        const bool begins = (uint32_t)x.id[h] < (uint32_t)L && pos[h] % ROWS == 0;
        const uint64_t in = __ballot(begins);
        const int nth = before + __builtin_amdgcn_mbcnt_hi((uint32_t)(in >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)in, 0));
        const uint64_t hit = __ballot(begins && nth == j);
        if (hit != 0) {
            const int l = __builtin_ctzll(hit);
            a = __builtin_amdgcn_readlane(x.id[h], l);
            first = __builtin_amdgcn_readlane(pos[h], l);
        }
        before += __builtin_popcountll(in);
    }
    if (a < 0)
        return;
    int place[kWords];
#pragma unroll
    for (int h = 0; h < kWords; ++h)
        place[h] = x.id[h] == a ? pos[h] - first : -1;
    task(a, group_row<ROWS>(place));
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

// Lists the groups of a chunk for the expansion that follows, a thread per row: each finds its
// place among its adapter's rows; the rows that begin a group number the groups, and leave the
// numbers where the others look for them.
__device__ __forceinline__ void list_groups(const InnerArgs &p, int chunk)
{
    __shared__ int16_t number[kWideRows * 16];     // [first row of the adapter][group of the adapter]
    __shared__ int count[kWords];
    const int m0 = chunk * kWideRows, row = (int)threadIdx.x, wave = row >> 6;
    ExpandGroup *list = p.list + (size_t)chunk * p.expand_groups;
    for (int i = row; i < p.expand_groups * 17; i += kWideRows)
        reinterpret_cast<int32_t *>(list)[i] = -1;
    const Ids x = load_ids(p.ids, p.M, p.L, m0);
    int pos4[kWords], first4[kWords], pos = 0, first = 0, id = -1;
    count_before(x, p.id_bits, pos4, first4);
#pragma unroll
    for (int h = 0; h < kWords; ++h) {
        pos = wave == h ? pos4[h] : pos;
        first = wave == h ? first4[h] : first;
        id = wave == h ? x.id[h] : id;
    }
    const bool ok = (uint32_t)id < (uint32_t)p.L, begins = ok && pos % 16 == 0;
    const uint64_t in = __ballot(begins);
    if ((row & 63) == 0)
        count[wave] = __builtin_popcountll(in);
    __syncthreads();
    int nth = __builtin_amdgcn_mbcnt_hi((uint32_t)(in >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)in, 0));
    for (int w = 0; w < wave; ++w)
        nth += count[w];
    if (begins)
        number[first * 16 + pos / 16] = (int16_t)nth;
    wait_vmcnt<0>();                               // the -1s are out
    __syncthreads();
    if (ok) {
        ExpandGroup &g = list[number[first * 16 + pos / 16]];
        if (begins)
            g.adapter = id;
        g.row[pos % 16] = m0 + row;
    }
}

// Inner products of few rows: a workgroup forms 4 G ranks of up to 4 G rows with
// v_mfma_f32_4x4x4_16b_bf16, whose 16 blocks take 16 pieces of K: lane l holds row l % 4 of
// either operand and 16 bytes of K at 16 (l / 4) of a 256-byte chunk, so that every lane of a
// load carries data (a 16 x 16 product of one row would issue the same loads for 15 empty
// ones).  The waves take U chunks each at a time; a wave's 16 block sums are added across
// its lanes, the waves' through LDS, both in a fixed order.  A token's adapter is bound by the
// latency of one chain ids -> A -> V, hence 4 ranks per workgroup (one token, 6144 x 16: 4.4 us
// with the quantisation; 16 tokens of 5120 x 16: 5.3 us); rows that share adapters by the bytes a
// CU has in flight, hence 8 x 8 (133 rows, 24 adapters of 6144 x 64: 10.4 us; U of 3, 6 and 12, and 8
// waves, within 8%).
constexpr int kFewWaves = 4;

template <int U, int G>
__global__ __launch_bounds__(kFewWaves * 64) void lora_inner_few_kernel(InnerArgs p)
{
    static_assert(kFewWaves * 64 == kWideRows, "a thread per row");
    if ((int)blockIdx.x >= p.inner_wgs) {
        if ((int)blockIdx.x < p.inner_wgs + p.quant_wgs)
            quantise_part<kFewWaves>(p);
        else
            list_groups(p, (int)blockIdx.x - p.inner_wgs - p.quant_wgs);
        return;
    }
    __shared__ v4f red[kFewWaves * 4][G][4 * G];   // per wave and 16 lanes: ranks 4 g .. of a group's rows
    constexpr uint32_t OOB = 0x7ffff000u;
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    // The groups' workgroups that take the same ranks on one XCD: its L2 reads their part of A once.
    const int runs = p.inner_wgs / p.RS, item = xcd_item((int)blockIdx.x, p.inner_wgs);
    const int j = item % runs, chunk = G == 1 ? kInnerRows : kWideRows, m0 = G == 1 ? j / chunk * chunk : j / p.groups * chunk;
    const int K = p.K, chunks = K >> 7;
    const __amdgpu_buffer_rsrc_t xres = buffer_rsrc(p.X + (size_t)m0 * K, (uint32_t)min(p.M - m0, chunk) * (uint32_t)K * 2u);
    const auto task = [&](int a, int row) __attribute__((always_inline)) {
        const float scaling = p.scaling[a];
        const __amdgpu_buffer_rsrc_t ares = buffer_rsrc(p.A + (size_t)a * p.R * K, (uint32_t)p.R * (uint32_t)K * 2u);
        uint32_t xoff[G];
#pragma unroll
        for (int h = 0; h < G; ++h) {
            const int r = G == 1 ? row : __builtin_amdgcn_ds_bpermute(4 * ((lane & 3) + 4 * h), row);
            xoff[h] = r >= 0 ? (uint32_t)r * (uint32_t)K * 2u + 16u * (uint32_t)(lane >> 2) : OOB;
        }
        const int rank0 = item / runs * 4 * G;
        const uint32_t aoff = (uint32_t)(rank0 + (lane & 3)) * (uint32_t)K * 2u + 16u * (uint32_t)(lane >> 2);
        v4f acc[G][G];
#pragma unroll
        for (int i = 0; i < G * G; ++i)
            acc[i / G][i % G] = (v4f){0.f, 0.f, 0.f, 0.f};
        for (int c0 = wave; c0 < chunks; c0 += kFewWaves * U) {
            v4i ar[U][G], xr[U][G];
#pragma unroll
            for (int j = 0; j < U; ++j) {
                const int c = c0 + j * kFewWaves;
#pragma unroll
                for (int h = 0; h < G; ++h)
                    ar[j][h] = __builtin_amdgcn_raw_buffer_load_b128(
                        ares, (int)(c < chunks ? aoff + (uint32_t)(4 * h) * (uint32_t)K * 2u : OOB), c < chunks ? c * 256 : 0, 0);
            }
#pragma unroll
            for (int j = 0; j < U; ++j) {
                const int c = c0 + j * kFewWaves;
#pragma unroll
                for (int h = 0; h < G; ++h)
                    xr[j][h] = __builtin_amdgcn_raw_buffer_load_b128(xres, (int)(c < chunks ? xoff[h] : OOB),
                                                                     c < chunks ? c * 256 : 0, 0);
            }
            __builtin_amdgcn_sched_barrier(0);         // every load out before the first product
#pragma unroll
            for (int j = 0; j < U; ++j)
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int i = 0; i < G * G; ++i) {
                        const v4i &aw = ar[j][i / G], &xw = xr[j][i % G];
                        const v2u w = {(uint32_t)aw[2 * h], (uint32_t)aw[2 * h + 1]};
                        const v2u x = {(uint32_t)xw[2 * h], (uint32_t)xw[2 * h + 1]};
                        acc[i / G][i % G] = __builtin_amdgcn_mfma_f32_4x4x4bf16_1k(
                            __builtin_bit_cast(v4s, w), __builtin_bit_cast(v4s, x), acc[i / G][i % G], 0, 0, 0);
                    }
        }
        // The four blocks of each 16 lanes, then the sixteen sums of those in LDS.
#pragma unroll
        for (int i = 0; i < G * G; ++i) {
            v4f v = acc[i / G][i % G];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                v[q] += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v[q]), 0x128, 0xF, 0xF, false));  // row_ror 8
                v[q] += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v[q]), 0x124, 0xF, 0xF, false));  // row_ror 4
            }
            if ((lane & 12) == 0)
                red[4 * wave + (lane >> 4)][i / G][4 * (i % G) + (lane & 3)] = v;
        }
        __syncthreads();                               // (the only task of this workgroup: red is not written again)
        if (wave == 0 && lane < 4 * G * G) {           // lane: rank group lane / (4 G), row lane % (4 G) of the group
            const int h = lane / (4 * G), r = lane % (4 * G);
            v4f v = red[0][h][r];
#pragma unroll
            for (int w = 1; w < kFewWaves * 4; ++w)
                v += red[w][h][r];
            if (row >= 0)                              // (row: of the group's lane % (4 G)-th place)
                store_inner(p, m0 + row, rank0 + 4 * h, scaling, v);
        }
    };
    if constexpr (G == 1)
        for_groups<4 * G>(p.ids, p.M, p.L, m0, j - m0, 1, 0, 1, task);
    else
        one_group<4 * G>(p.ids, p.M, p.L, p.id_bits, m0, j % p.groups, task);
}

// Inner products of more rows: a workgroup forms 16 ranks of up to 16 rows.  Matrix operands
// are rows of A[a], then the gathered rows of X, both straight from memory in one K order
// (lane l: row l % 16, 16 bytes 16 (l / 16) .. of each 64-byte half of a 128-byte chunk of K).
// The waves take U such chunks each at a time; their partials are summed through LDS in wave
// order.  Bound by the lines a CU has in flight: X is read once per 16 ranks, A once per group
// (2048 rows of 5120, rank 32, 16 adapters, with the quantisation: 25.8 us, about 6 of them
// without either's loads; 16 waves, or U of 10, within 5%).
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
    const int base = p.inner_wgs / p.subs, sub = (int)blockIdx.x / base, item = xcd_item((int)blockIdx.x % base, base);
    const int at = item / p.RS * kRunRows, m0 = at / kInnerRows * kInnerRows;
    const int rank0 = item % p.RS * 16;
    const int K = p.K, chunks = K >> 6;
    const uint32_t aoff = rank0 + r16 < p.R ? (uint32_t)(rank0 + r16) * (uint32_t)K * 2u + 16u * (uint32_t)g : OOB;
    const __amdgpu_buffer_rsrc_t xres = buffer_rsrc(p.X + (size_t)m0 * K, (uint32_t)min(p.M - m0, kInnerRows) * (uint32_t)K * 2u);
    for_groups<16>(p.ids, p.M, p.L, m0, at - m0, kRunRows, sub, p.subs, [&](int a, int row) __attribute__((always_inline)) {
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

// Expansion D[m] = B[a] V[m] for calls of few rows on tiles: a workgroup takes a listed group
// of up to 16 rows of one adapter and 128 columns, a wave 32 of them (two 16-row fragments of B),
// so that B is read once per group.  Bound by B's bytes and the latency list -> B, V -> D (133
// rows, 24 adapters of 5120 x 64: 6.7 us, 8.8 with the groups found anew in every workgroup, a
// tenth more with 256 columns).  D is fp32: the GEMM adds it to its accumulators.
constexpr int kExpandCols = 128;

__global__ __launch_bounds__(256) void lora_expand_kernel(InnerArgs p)
{
    constexpr uint32_t OOB = 0x7ffff000u;
    constexpr int TN = 2, KS = 2;
    const int lane = threadIdx.x & 63, r16 = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int CBS = (p.N + kExpandCols - 1) / kExpandCols;
    const int n0 = (int)blockIdx.x % CBS * kExpandCols + wave * 16 * TN;
    const ExpandGroup &group = p.list[(int)blockIdx.x / CBS];
    const int a = __builtin_amdgcn_readfirstlane(group.adapter), row = group.row[r16], R = p.R;
    if (a < 0)
        return;
    const __amdgpu_buffer_rsrc_t vres = buffer_rsrc(p.V, (uint32_t)p.M * (uint32_t)R * 4u);
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
                *reinterpret_cast<v4f *>(p.D + (size_t)row * p.ldd + n) = acc[u];
        }
    }
}

}  // namespace kern

namespace {

using namespace kern;

constexpr int kMaxRank = 256;
constexpr int64_t kFewRows = 512;
constexpr int64_t kMax32 = 0x7ffff000;   // 32-bit byte offsets inside one adapter, one chunk of X's rows (the
                                         // offset that stands for nothing to read is beyond them)

int64_t up256(int64_t n) { return (n + 255) & ~(int64_t)255; }

struct LoraLayout {
    int64_t codes, scales, v, d, list, bytes;   // offsets from the workspace's start
};

int64_t d_stride(int64_t N) { return (N + 3) & ~(int64_t)3; }

LoraLayout lora_layout(int64_t M, int64_t N, int64_t K, int64_t R)
{
    LoraLayout l;
    l.codes = A8W8_WORKSPACE_COUNTER_BYTES;
    l.scales = l.codes + up256(M * K);
    l.v = l.scales + up256(M * (K / 128) * 4);
    l.d = l.v + up256(M * 2 * R * 2);
    l.list = l.d + (M <= kFewRows ? up256(M * d_stride(N) * 4) : 0);
    l.bytes = l.list + (M <= kFewRows ? (M + kWideRows - 1) / kWideRows * kWideRows * (int64_t)sizeof(ExpandGroup) : 0);
    return l;
}

// The most groups of `size` rows that a chunk of `rows` can fall into, and all chunks of M.
int64_t chunk_groups(int64_t rows, int64_t L, int size) { return std::min(rows, L + rows / size); }
int64_t all_groups(int64_t M, int64_t L, int size)
{
    return M / kWideRows * chunk_groups(kWideRows, L, size) + chunk_groups(M % kWideRows, L, size);
}

int check_lora_shape(int64_t M, int64_t N, int64_t K, int64_t L, int64_t R)
{
    const int rc = check_gemm_shape(M, N, K);
    if (rc != A8W8_OK)
        return rc;
    if (N > (1 << 22) || L < 1 || L > (1 << 20) || R < 8 || R > kMaxRank || R % 8 != 0 || N * R * 2 >= kMax32 || R * K * 2 >= kMax32 ||
        std::min<int64_t>(M, kWideRows) * K * 2 >= kMax32)
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
    // Fewer rows may need more (up to kFewRows the products are formed beforehand): what any number up to M needs.
    *bytes = M == 0 ? 0 : std::max(lora_layout(M, N, K, rank).bytes, lora_layout(std::min(M, kFewRows), N, K, rank).bytes);
    return A8W8_OK;
}

static int lora_impl(const a8w8_lora_desc *d, bool quotient, void *stream)
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
    in.quotient = quotient;
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
    // Up to kFewRows rows: 4 ranks a workgroup and groups of 4 rows, a workgroup per row (a decode
    // batch's adapters differ), or, where the adapters have more rows and half the CUs still get
    // one, 8 ranks and groups of 8 rows, a workgroup per group (133 rows, 24 adapters of 6144 x 64: 10.2
    // against 15.3 us; 16 rows, 2 adapters: 20.8 against 17.3 us a call).  Above: groups of 16 rows, 16
    // ranks a workgroup, runs of 16 rows (of a prompt each starts a group, seldom two), whose groups up
    // to four workgroups share out, the second ones of all runs after the first ones, as long as
    // there are at most four workgroups a CU.  One workgroup a run against that: 1024 rows of 5120 x 6144,
    // rank 16, 8 adapters 82 and 72 us a call for prompts, 152 and 87 with adapters that change row by row;
    // 2048 of 14336 x 5120, rank 32, 16 adapters 220 and 218, 340 and 294.  4096 of 2048 x 2048, rank 64, 24
    // adapters, where the rule takes one: 65 and 183 us; with four (16 a CU, most idle) 81 and 165.  The
    // quantisation's workgroups come after those, then those that list the groups for the expansion.
    //
    // kFewRows also decides whether the products are formed beforehand or in the tiles' epilogue.  Prompts, and
    // adapters that change row by row, in us a call: 14336 x 5120, rank 32, 16 adapters, 256 rows 62 and 63
    // beforehand against 57 and 84, 512 rows 90 and 88 against 74 and 99, 1024 rows 147 and 150 against 121
    // and 176; 5120 x 6144, rank 16, 8 adapters, 512 rows 57 and 58 against 58 and 74, 1024 rows 78 and 78 against 69
    // and 87; 2048 x 2048, rank 64, 24 adapters, 512 rows 28 and 29 against 27 and 54.  The host does not know the
    // ids: up to 512 rows are taken to be a decode batch, more to be prompts.
    const bool few = d->M <= kFewRows;
    const int waves = few ? kFewWaves : kInnerWaves;
    const int64_t groups = d->M * (d->K / 128), qwgs = (groups + waves * 4 - 1) / (waves * 4);
    const bool eights = few && d->M > 4 * (int64_t)in.L && (in.L + d->M / 8) * (in.R / 8) >= cus / 2;
    in.quant_wgs = (int32_t)(qwgs < 8 * cus ? qwgs : 8 * cus);
    in.RS = eights ? in.R / 8 : few ? in.R / 4 : (in.R + 15) / 16;
    const int64_t firsts = (d->M + kRunRows - 1) / kRunRows * in.RS;
    in.subs = few ? 1 : (int32_t)std::max<int64_t>(1, std::min<int64_t>(4, 4 * cus / firsts));
    in.groups = (int32_t)chunk_groups(kWideRows, in.L, 8);
    in.expand_groups = (int32_t)chunk_groups(kWideRows, in.L, 16);
    in.id_bits = 0;
    while (in.id_bits < 31 && ((in.L - 1) >> in.id_bits) != 0)
        ++in.id_bits;
    in.inner_wgs = (int32_t)(eights ? all_groups(d->M, in.L, 8) * in.RS : few ? d->M * in.RS : firsts * in.subs);
    in.B = static_cast<const uint16_t *>(d->B);
    in.N = (int32_t)d->N;
    in.ldd = (int32_t)d_stride(d->N);
    // Tiles of few rows: the low-rank products are formed beforehand, adapter by adapter.
    in.D = few && variant(id).kernel != A8W8_KERNEL_RSKINNY ? reinterpret_cast<float *>(ws + l.d) : nullptr;
    in.list = reinterpret_cast<ExpandGroup *>(ws + l.list);
    const int lists = in.D != nullptr ? (int)((d->M + kWideRows - 1) / kWideRows) : 0;
    const dim3 grid((unsigned)(in.inner_wgs + in.quant_wgs + lists)), block(waves * 64);
    if (eights)
        hipLaunchKernelGGL((lora_inner_few_kernel<6, 2>), grid, block, 0, st, in);
    else if (few)
        hipLaunchKernelGGL((lora_inner_few_kernel<12, 1>), grid, block, 0, st, in);
    else
        hipLaunchKernelGGL(lora_inner_kernel<5>, grid, block, 0, st, in);
    if (in.D != nullptr)
        hipLaunchKernelGGL(lora_expand_kernel, dim3((unsigned)(all_groups(d->M, in.L, 16) * ((d->N + kExpandCols - 1) / kExpandCols))),
                           dim3(256), 0, st, in);

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

int gemm_a8w8_blockscale_lora(const a8w8_lora_desc *desc, void *stream) { return lora_impl(desc, false, stream); }

int gemm_a8w8_blockscale_lora_quantize_1x128(const a8w8_lora_desc *desc, void *stream)
{
    return lora_impl(desc, true, stream);
}

}  // extern "C"
