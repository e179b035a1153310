// a8w8_attention.hip -- attention of the new tokens of several sequences over a paged cache,
// for gfx950.
//
// Row i of the n new tokens of a sequence of `len` tokens (the new ones included, their keys
// already in the cache) stands at p = len - n + i and sees the keys j <= p; with a window only
// j > p - window, and the first `sinks` tokens:
//
//   out = (sum_j softmax_j(scale q . k_j) v_j) * sigmoid(gate)         (gate optional)
//
// A row that sees nothing gets zeros (so does one whose keys all score -infinity, which the running maximum cannot tell
// from it).
//
// The query heads of one key head are rows of one matrix: row r of a sequence is token r / G,
// head r % G of the group, so that keys and values are read once for all of them.  One pass over
// the keys with the running maximum m and sum l of each row's softmax (base 2):
//
//   S^T = K Q^T,  P = 2^(S - m),  O^T = O^T 2^(m_old - m) + V^T P^T
//
// Both products have the row as their column index: a lane of a matrix instruction's result
// holds one row and several keys, so m, l and the rescaling are a lane's own scalars, and the
// result registers of the first product are the operand registers of the second one, for keys in
// the order that the instruction's lanes have them -- P never moves between lanes.  V is
// transposed on its way out of LDS (ds_read_b64_tr).
//
// Two kernels, by the sequence's rows (tokens times heads of the group):
//   few    up to 16: one tile of 16 rows on 16x16x32 instructions; bound by the cache's bytes.
//          Every wave streams tiles of 32 keys of its own through its own part of LDS.
//   many   more: tiles of 256 rows (head_dim 64, 256: 128) on 32x32x16 instructions, 32 rows a wave;
//          bound by the products.  The waves share tiles of 64 (head_dim 256: 32) keys.
// Both are launched where the host cannot know that one has nothing to do (see max_new), one behind
// the other; an empty launch of the few kernel takes 4.7 us.
// Work is cut in units (blocks of keys of one sequence, key head and row tile) and every
// workgroup takes an equal run of them, found from the lengths on the device; pieces of an item
// that was cut meet in the workspace, where the last one to arrive joins them in their order.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <atomic>

#include "a8w8_device.h"
#include "a8w8_internal.h"
#include "a8w8_quant_math.h"
#include "gemm_a8w8_blockscale.h"

namespace a8w8 {
namespace kern {

typedef float v2f __attribute__((ext_vector_type(2)));
typedef float v16f __attribute__((ext_vector_type(16)));
typedef __bf16 v2b __attribute__((ext_vector_type(2)));
typedef __bf16 v4b __attribute__((ext_vector_type(4)));
typedef int v2i __attribute__((ext_vector_type(2)));
typedef __attribute__((address_space(3))) void *lds_ptr_t;
typedef __attribute__((address_space(3))) v4s lds_v4s;
typedef __attribute__((address_space(3))) v2i lds_v2i;
typedef __attribute__((address_space(3))) v8b lds_v8b;

constexpr int kMaxSeqs = 2048;
constexpr int kFewRows = 16;
constexpr float kLowest = -3.0e38f;    // the running maximum before any key: 2^(-inf - kLowest) is 0

struct AttnArgs {
    const uint16_t *q, *gate;
    int64_t q_row, q_head, gate_row, gate_head;
    const uint8_t *k, *v;
    const float *k_scale, *v_scale;
    const int32_t *table, *q_start, *lens;
    uint16_t *out;
    float *part;       // pieces: [workgroup][2] of rows x head_dim sums, then rows x {m, l}
    int32_t *cnt;      // one zeroed counter per workgroup
    int32_t T, B, P, pages, page_shift, Hq, Hkv, G, window, sinks;
    int32_t few_only;  // no other kernel runs: every sequence is the few kernel's
    float scale;
};

// What copies of keys that no row sees read.
__device__ const uint4 kNothing = {0, 0, 0, 0};

// ---------------------------------------------------------------------------
// Memory

// Direct-to-LDS copies of 16 (4) bytes a lane to lds + 16 (4) * lane, as asm: the compiler would
// make every LDS read wait for all copies in flight.  The padding between the m0 write and the
// load is the hazard that it does not see inside the string.  Counted by vmcnt like any load: the
// loops below hold no other vector memory operation of the compiler's.
__device__ __forceinline__ void copy16(const void *src, uint32_t lds)
{
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\tglobal_load_lds_dwordx4 %1, off" : : "s"(lds), "v"(src) : "memory", "m0");
}
__device__ __forceinline__ void copy4(const void *src, uint32_t lds)
{
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\tglobal_load_lds_dword %1, off" : : "s"(lds), "v"(src) : "memory", "m0");
}
// The same from a wave-uniform address plus a lane's 32-bit offset.
__device__ __forceinline__ void copy16_at(const void *base, uint32_t off, uint32_t lds)
{
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\tglobal_load_lds_dwordx4 %1, %2" : : "s"(lds), "v"(off), "s"(base) : "memory", "m0");
}
// Two of them from wave-uniform addresses plus lanes' 32-bit offsets (the addresses are ready before the first
// wait, so the second needs the m0 write's alone).
__device__ __forceinline__ void copy16_pair(const void *base0, uint32_t off0, uint32_t lds0, const void *base1, uint32_t off1,
                                            uint32_t lds1)
{
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\tglobal_load_lds_dwordx4 %1, %2\n\t"
                 "s_mov_b32 m0, %3\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %4, %5"
                 :
                 : "s"(lds0), "v"(off0), "s"(base0), "s"(lds1), "v"(off1), "s"(base1)
                 : "memory", "m0");
}
template <int N>
__device__ __forceinline__ void wait_copies()
{
    asm volatile("s_waitcnt vmcnt(%0)" : : "n"(N) : "memory");
}
// This wave's LDS reads have returned (before a copy overwrites what they read).
__device__ __forceinline__ void wait_reads() { asm volatile("s_waitcnt lgkmcnt(0)" : : : "memory"); }

__device__ __forceinline__ uint32_t lds_addr(const void *p) { return (uint32_t)(uintptr_t)(lds_ptr_t)p; }

__device__ __forceinline__ v8b join(v4s a, v4s b)
{
    typedef short v8s __attribute__((ext_vector_type(8)));
    return __builtin_bit_cast(v8b, (v8s)__builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7));
}
// Eight e4m3 codes to bf16, exactly.
__device__ __forceinline__ v8b widen(v2i c)
{
    const v2b a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c[0], 1.0f, false);
    const v2b b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c[0], 1.0f, true);
    const v2b d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c[1], 1.0f, false);
    const v2b e = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c[1], 1.0f, true);
    return (v8b){a[0], a[1], b[0], b[1], d[0], d[1], e[0], e[1]};
}
__device__ __forceinline__ v2b round2(float a, float b) { return __builtin_convertvector((v2f){a, b}, v2b); }

// Reductions over the lanes that hold the same row (l ^ 16, l ^ 32).
__device__ __forceinline__ float max_swap32(float x)
{
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float max_swap16(float x)
{
    const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float sum_swap32(float x)
{
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}
__device__ __forceinline__ float sum_swap16(float x)
{
    const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

// The order of the instructions before stays before, of those behind behind.  (Left to itself the compiler
// reads each operand of a matrix instruction from LDS right before its use and waits for it.)
__device__ __forceinline__ void in_order() { __builtin_amdgcn_sched_barrier(0); }

__device__ __forceinline__ v16f zero16()
{
    v16f z;
#pragma unroll
    for (int i = 0; i < 16; ++i)
        z[i] = 0.0f;
    return z;
}

// Pieces of cut items go past the XCDs' own L2s (sc1): other workgroups read them in this launch.
__device__ __forceinline__ void put4(__amdgpu_buffer_rsrc_t r, uint32_t off, v4f x)
{
    __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(v4i, x), r, off, 0, 16);
}
__device__ __forceinline__ v4f get4(__amdgpu_buffer_rsrc_t r, uint32_t off)
{
    return __builtin_bit_cast(v4f, __builtin_amdgcn_raw_buffer_load_b128(r, off, 0, 16));
}
__device__ __forceinline__ void put2(__amdgpu_buffer_rsrc_t r, uint32_t off, v2f x)
{
    __builtin_amdgcn_raw_buffer_store_b64(__builtin_bit_cast(v2u, x), r, off, 0, 16);
}
__device__ __forceinline__ v2f get2(__amdgpu_buffer_rsrc_t r, uint32_t off)
{
    return __builtin_bit_cast(v2f, __builtin_amdgcn_raw_buffer_load_b64(r, off, 0, 16));
}

// ---------------------------------------------------------------------------
// What a sequence and a tile of its rows need

struct Seq {
    int q0, n, len;
};
__device__ __forceinline__ Seq load_seq(const AttnArgs &p, int b)
{
    const int s = p.q_start[b], e = p.q_start[b + 1];
    const bool inside = s >= 0 && e <= p.T && e > s;
    return {s, inside ? e - s : 0, max(p.lens[b], 0)};
}

// The keys that rows at positions first .. last see, as blocks of BK: [0, hi) without a window; with one
// blocks of the sinks first, then those from the first row's window on.  A tile that sees no key
// still is one block, whose result is zeros.
struct Keys {
    int hi, lo, sink, sink_blocks, skip, blocks;
    __device__ __forceinline__ int base(int x, int BK) const { return (x < sink_blocks ? x : x + skip) * BK; }
};
template <int BK>
__device__ __forceinline__ Keys keys_of(const AttnArgs &p, int first, int last)
{
    Keys k;
    k.hi = max(0, min(last + 1, p.P << p.page_shift));
    k.lo = k.sink = k.sink_blocks = k.skip = 0;
    if (p.window && first + 1 > p.window) {
        k.lo = first + 1 - p.window;
        k.sink = min(p.sinks, min(k.lo, k.hi));
        k.sink_blocks = (k.sink + BK - 1) / BK;
        // (a window that lies behind the table's end begins, as blocks go, at the last key that can be read: no block's
        // first key passes 2^30 by more than a few blocks, whatever the length)
        k.skip = max(0, min(k.lo, k.hi) / BK - k.sink_blocks);
    }
    const int all = (k.hi + BK - 1) / BK;
    k.blocks = max(1, all <= k.sink_blocks ? all : max(k.sink_blocks, all - k.skip));
    return k;
}
// First key of a row's window.
__device__ __forceinline__ int window_start(const AttnArgs &p, int pos)
{
    return p.window && pos + 1 > p.window ? pos + 1 - p.window : 0;
}

// What the scores of a key head are multiplied by: scale, its keys' scale and the softmax's change to base 2.  The sign
// goes into the queries (exactly), so that the size is positive and a masked score of -inf stays one.  A factor that is
// not finite makes the queries NaN: every row that sees a key is NaN then, as by the definition, and one that sees
// none still gets zeros.
struct ScoreFactor {
    float size;
    uint32_t sign, nan;      // of two bf16 queries
};
__device__ __forceinline__ ScoreFactor score_factor(const AttnArgs &p, int hk)
{
    const float x = p.scale * (p.k_scale ? p.k_scale[hk] : 1.0f) * 1.4426950408889634f, size = __builtin_fabsf(x);
    const bool finite = size < INFINITY;
    return {finite ? fmaxf(size, 1.17549435e-38f) : 1.0f, x < 0.0f ? 0x80008000u : 0u, finite ? 0u : 0x7fc07fc0u};
}

// Inclusive sums of x over a workgroup's WAVES waves; *total the whole sum.  `scratch`: WAVES values in LDS.
template <int WAVES>
__device__ __forceinline__ int64_t scan(int64_t x, int64_t *scratch, int64_t *total)
{
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
        const int64_t y = __shfl_up(x, d);
        x += lane >= d ? y : 0;
    }
    __syncthreads();
    if (lane == 63)
        scratch[wave] = x;
    __syncthreads();
    int64_t t = 0;
#pragma unroll
    for (int w = 0; w < WAVES; ++w) {
        x += w < wave ? scratch[w] : 0;
        t += scratch[w];
    }
    *total = t;
    return x;
}

// a / b for a >= 0, b > 0; almost always of 32 bits, which take a twentieth of the instructions.
__device__ __forceinline__ int64_t divide(int64_t a, int64_t b)
{
    return ((a | b) >> 32) == 0 ? (int64_t)((uint32_t)a / (uint32_t)b) : a / b;
}
__device__ __forceinline__ int64_t uniform(int64_t x)
{
    const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)x), hi = __builtin_amdgcn_readfirstlane((uint32_t)(x >> 32));
    return (int64_t)(((uint64_t)hi << 32) | lo);
}

// The next sequence from b on that belongs to this kernel (B: none).
template <bool MANY>
__device__ __forceinline__ bool mine(const AttnArgs &p, const Seq &s)
{
    return s.n > 0 && (MANY ? (int64_t)s.n * p.G > kFewRows : p.few_only || (int64_t)s.n * p.G <= kFewRows);
}
template <bool MANY>
__device__ __forceinline__ int next_seq(const AttnArgs &p, int b)
{
    for (; b < p.B; b += 64) {
        const int i = b + (int)(threadIdx.x & 63);
        const uint64_t any = __ballot(i < p.B && mine<MANY>(p, load_seq(p, min(i, p.B - 1))));
        if (any)
            return b + __builtin_ctzll(any);
    }
    return p.B;
}

// x * sigmoid(gate), reciprocal and exponential of the hardware (one ulp each).
__device__ __forceinline__ float gated(float x, float gate)
{
    return x * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(gate * -1.4426950408889634f));
}
// A value that the compiler must take as new here: what is computed from it is computed here and not kept in
// registers across the loops around.
__device__ __forceinline__ int fresh(int x)
{
    asm volatile("" : "+v"(x));
    return x;
}

// Where rows of a tile see different keys and some elements of V are not finite, a row that does not
// see such a key must not get 0 * inf.  In blocks that not all rows see whole, such elements are zeroed
// in LDS (clear_infinite), and where there were any, what they do to the sums of the rows that see them
// is added when the item is done (add_infinite), out of the main loop's way.
__device__ __forceinline__ v8b finite_part(v8b v)
{
    u32x4 w = __builtin_bit_cast(u32x4, v);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t lo = (w[i] & 0x7f80u) == 0x7f80u ? 0xffffu : 0u, hi = (w[i] & 0x7f800000u) == 0x7f800000u ? 0xffff0000u : 0u;
        w[i] &= ~(lo | hi);
    }
    return __builtin_bit_cast(v8b, w);
}
// Zeroes what is not finite in n KB that this wave copied (bf16, or e4m3 whose NaN is 0x7f), `step` KB apart;
// returns whether there was any.
template <bool FP8>
__device__ __forceinline__ bool clear_infinite(uint8_t *lds, int n, int step = 1)
{
    bool any = false;
#pragma unroll 1
    for (int i = 0; i < n; ++i) {
        u32x4 *at = reinterpret_cast<u32x4 *>(lds + i * step * 1024) + (threadIdx.x & 63);
        const u32x4 w = *at;
        u32x4 y = __builtin_bit_cast(u32x4, finite_part(__builtin_bit_cast(v8b, w)));
        if constexpr (FP8) {
            y = w;
#pragma unroll
            for (int c = 0; c < 16; ++c)
                if (((w[c / 4] >> (8 * (c % 4))) & 0x7f) == 0x7f)
                    y[c / 4] &= ~(0xffu << (8 * (c % 4)));
        }
        const bool other = y[0] != w[0] || y[1] != w[1] || y[2] != w[2] || y[3] != w[3];
        if (other)
            *at = y;
        any |= __ballot(other) != 0;
    }
    return any;
}
// Adds the infinities and NaN among the four values from `src` on.
template <bool FP8>
__device__ __forceinline__ void add_infinite(float *o, const uint8_t *src)
{
    if constexpr (FP8) {
        const uint32_t w = *reinterpret_cast<const uint32_t *>(src);
#pragma unroll
        for (int c = 0; c < 4; ++c)
            if (((w >> (8 * c)) & 0x7f) == 0x7f)
                o[c] = NAN;
    } else {
        const uint2 w = *reinterpret_cast<const uint2 *>(src);
        const float x[4] = {bf16_lo(w.x), bf16_hi(w.x), bf16_lo(w.y), bf16_hi(w.y)};
#pragma unroll
        for (int c = 0; c < 4; ++c)
            o[c] += __builtin_fabsf(x[c]) < INFINITY ? 0.0f : x[c];
    }
}
// The first n keys of 32 (none if n <= 0).
__device__ __forceinline__ uint32_t first_keys(int n) { return n >= 32 ? ~0u : n <= 0 ? 0u : (1u << n) - 1; }
// Which of the 32 keys from kb on a row sees of those in `seen`.
__device__ __forceinline__ uint32_t row_keys(uint32_t seen, int kb, int pos, int low, int sinks)
{
    return seen & first_keys(pos - kb + 1) & (~first_keys(low - kb) | first_keys(sinks - kb));
}

// ---------------------------------------------------------------------------
// Up to 16 rows

// A unit is read once from the cache and shared by nobody, so what counts is bytes in flight: every wave keeps
// its next tile's keys on the way while it multiplies, with waits counted per wave and no barrier in an item.
// Measured (one MI355X; a 4 GiB copy reaches 4.77 TB/s): bf16, 16 requests of 20000 tokens, head_dim 256, 4 key
// heads 162 us, 5.3 TB/s; one request of 131071 tokens, head_dim 128, 8 key heads 108 us, 5.0 TB/s; e4m3, 61
// requests of 4000 tokens 72 us, 4.4 TB/s (waves of a workgroup end apart, and each item costs its start and
// end).  A request of 501 tokens takes 15 us: 5.5 thousand cycles (2.4 us) to find the run, 6.4 to the first product,
// 2.7 for the tiles, up to 18 for joining waves and pieces.
//   WAVES   one workgroup of eight waves, against two of four with the same LDS: 131071 tokens 108 us (140), 16
//           x 20000 163 (173), since half as many pieces are joined.  head_dim 256 in bf16 has room for four.
//   PER_CU  two where LDS holds them; e4m3, whose codes are also converted, at one: 72 us against 80 - 92.
//   P       bf16 rounding of P would cost as much as the output's own; the second term's products are free
//           here (bound by bytes), so P is a sum of two.
template <int D, bool FP8>
struct Few {
    static constexpr int ROW = D * (FP8 ? 1 : 2);           // bytes of a cached head
    static constexpr int CH = ROW / 16;                     // its 16-byte chunks
    static constexpr int TILE = 32 * ROW;                   // a wave's keys or values
    static constexpr int LOADS = TILE / 1024;               // copies of a tile
    static constexpr int PAD = D + 4;                       // floats of a row of sums in LDS
    static constexpr int OUT = 16 * PAD * 4;
    static constexpr int WAVE = (2 * TILE > OUT ? 2 * TILE : OUT) + 512;   // tiles, then two sets of page numbers
    static constexpr int WAVES = 8 * WAVE > 144 * 1024 ? 4 : 8, THREADS = 64 * WAVES;
    static constexpr int LDS = WAVES * WAVE;
    static constexpr int PER_CU = !FP8 && 2 * LDS <= 150 * 1024 ? 2 : 1;
    static constexpr int KEYS = 32 * WAVES;                 // a unit
    static constexpr int ITEM = 2;                          // what an item costs beside its units, in units
    static constexpr int E = 16 * D / THREADS < 4 ? 4 : 16 * D / THREADS;  // neighbouring sums that a thread joins
    static constexpr int PIECE = 16 * D + 32;               // floats of a cut item's piece
    // chunk position of chunk c in row r: lanes of a fragment read hit all banks
    static __device__ __forceinline__ constexpr int turn_k(int r) { return ((r & 3) | ((r >> 1) & 4)) & (CH - 1); }
    static __device__ __forceinline__ constexpr int turn_v(int r) { return FP8 ? r & 7 & (CH - 1) : (r & 3) << 1; }
};

// A wave's copies of 32 keys (or values) from key kb on into LDS at dst; `seen`: bit r = some row sees key kb + r, whose
// page is in lane r of `pages`.
template <int D, bool FP8, bool IS_V>
__device__ __forceinline__ void few_copy(const AttnArgs &p, const int pages, int kb, uint32_t seen, int hk, uint32_t dst)
{
    using F = Few<D, FP8>;
    constexpr int R = 64 / F::CH;                // rows of a copy
    const int lane = fresh(threadIdx.x & 63), mask = (1 << p.page_shift) - 1;
    const uint8_t *cache = (IS_V ? p.v : p.k) + (int64_t)hk * F::ROW;
    const uint64_t stride = (uint64_t)p.Hkv * F::ROW;
    const auto turn = [](int r) { return IS_V ? F::turn_v(r) : F::turn_k(r); };
    if (seen == ~0u && (1 << p.page_shift) >= R) {       // every copy lies in one page: scalar addresses
        const uint32_t at = (lane / F::CH) * (uint32_t)stride + ((lane % F::CH) ^ turn(lane / F::CH)) * 16;
#pragma unroll
        for (int i = 0; i < F::LOADS; ++i) {
            const uint32_t page = __builtin_amdgcn_readlane(pages, i * R);
            copy16_at(cache + ((page << p.page_shift) | ((kb + i * R) & mask)) * stride, at ^ (turn(i * R) * 16), dst + i * 1024);
        }
    } else {
#pragma unroll
        for (int i = 0; i < F::LOADS; ++i) {
            const int r = i * R + lane / F::CH, c = (lane % F::CH) ^ turn(r);
            const uint32_t slot = ((uint32_t)__builtin_amdgcn_ds_bpermute(r * 4, pages) << p.page_shift) | ((kb + r) & mask);
            const uint8_t *src = cache + slot * stride + c * 16;
            copy16((seen >> r) & 1 ? (const void *)src : (const void *)&kNothing, dst + i * 1024);
        }
    }
}

template <int D, bool FP8>
__global__ __launch_bounds__((Few<D, FP8>::THREADS), (Few<D, FP8>::PER_CU * Few<D, FP8>::WAVES / 4)) void few_kernel(AttnArgs p)
{
    using F = Few<D, FP8>;
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ int64_t scratch[F::WAVES];
    __shared__ int64_t at;
    __shared__ int at_b, last;
    __shared__ float wave_m[F::WAVES][16], wave_l[F::WAVES][16];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int i16 = lane & 15, g = lane >> 4;

    // Units of all sequences, and this workgroup's run of them.
    const auto units_of = [&](int b) -> int64_t {
        const Seq s = load_seq(p, b);
        if (!mine<false>(p, s))
            return 0;
        // (a sequence of several tiles: each is given the blocks of all its rows)
        return (int64_t)(keys_of<F::KEYS>(p, s.len - s.n, s.len - 1).blocks + F::ITEM) *
               (((int64_t)s.n * p.G + kFewRows - 1) / kFewRows) * p.Hkv;
    };
    const int wg = blockIdx.x;
    int64_t total, run, u, rem;
    int b;
    if (p.B <= 64) {                         // one sequence a lane, every wave by itself
        const int64_t own = lane < p.B ? units_of(lane) : 0;
        int64_t sum = own;
#pragma unroll
        for (int d = 1; d < 64; d *= 2) {
            const int64_t y = __shfl_up(sum, d);
            sum += lane >= d ? y : 0;
        }
        total = uniform(__shfl(sum, 63));
        run = divide(total + gridDim.x - 1, gridDim.x);
        u = wg * run;
        if (u >= total)
            return;
        b = __builtin_ctzll(__ballot(u < sum));
        rem = u - uniform(__shfl(sum - own, b));
    } else {
        const int per = (p.B + F::THREADS - 1) / F::THREADS;
        int64_t own = 0;
        for (int i = 0; i < per; ++i) {
            const int c = threadIdx.x * per + i;
            own += c < p.B ? units_of(c) : 0;
        }
        int64_t before = scan<F::WAVES>(own, scratch, &total) - own;
        run = divide(total + gridDim.x - 1, gridDim.x);
        u = wg * run;
        if (u >= total)
            return;
        if (u >= before && u < before + own) {
            for (int c = threadIdx.x * per;; ++c) {
                const int64_t all = units_of(c);
                if (u < before + all) {
                    at = u - before;
                    at_b = c;
                    break;
                }
                before += all;
            }
        }
        __syncthreads();
        b = __builtin_amdgcn_readfirstlane(at_b);
        rem = uniform(at);
    }
    const int64_t u_end = min(u + run, total);

    uint8_t *mem = smem + wave * F::WAVE;
    uint8_t *kt_mem = mem, *vt_mem = mem + F::TILE;
    int *page_mem = reinterpret_cast<int *>(mem + F::WAVE - 512);      // [2][64]
    const uint32_t kt_lds = lds_addr(kt_mem), vt_lds = lds_addr(vt_mem), page_lds = lds_addr(page_mem);

    while (u < u_end) {
        const Seq s = load_seq(p, b);
        const int rows = s.n * p.G, tiles = (rows + kFewRows - 1) / kFewRows;
        // the blocks of the whole sequence, the visible range of the tile's rows (below)
        Keys k = keys_of<F::KEYS>(p, s.len - s.n, s.len - 1);
        const int blocks = k.blocks, units = blocks + F::ITEM;       // an item's first block is unit ITEM
        const int item = (int)divide(rem, units), v0 = (int)(rem - (int64_t)item * units);
        const int hk = __builtin_amdgcn_readfirstlane(item / tiles), tile = __builtin_amdgcn_readfirstlane(item % tiles);
        const int v1 = (int)min((int64_t)units, v0 + (u_end - u));
        const int x0 = max(v0 - F::ITEM, 0), x1 = max(v1 - F::ITEM, 0);
        if (x1 == 0)
            break;                           // (the run ends before the item's first block)
        const int r0 = tile * kFewRows, r_last = min(r0 + kFewRows, rows) - 1;
        const int first = s.len - s.n + r0 / p.G, final = s.len - s.n + r_last / p.G;
        {
            const Keys own_keys = keys_of<F::KEYS>(p, first, final);
            k.hi = own_keys.hi, k.lo = own_keys.lo, k.sink = own_keys.sink;
        }
        // Rows past the last one repeat it; their results are not stored.
        const int r = min(r0 + i16, rows - 1), token = r / p.G, head = hk * p.G + r % p.G;
        const int pos = s.len - s.n + token, low = window_start(p, pos), low_final = window_start(p, final);

        // Rows to operand registers (score_factor says what goes into them).
        u32x4 q_raw[D / 32];
        {
            const uint16_t *src = p.q + (int64_t)(s.q0 + token) * p.q_row + (int64_t)head * p.q_head + g * 8;
#pragma unroll
            for (int d = 0; d < D / 32; ++d)
                q_raw[d] = *reinterpret_cast<const u32x4 *>(src + d * 32);
        }
        const ScoreFactor factor = score_factor(p, hk);
        float sc = factor.size;
        float vs = p.v_scale ? p.v_scale[hk] : 1.0f;

        float m = kLowest, l = 0.0f;
        v4f o[D / 16];
#pragma unroll
        for (int d = 0; d < D / 16; ++d)
            o[d] = (v4f){0.0f, 0.0f, 0.0f, 0.0f};

        bool left_out = false;                       // (the same in all lanes)
        int mixed_from = x1, mixed_to = x0;          // the mixed blocks lie between
        const int32_t *row_table = p.table + (int64_t)b * p.P;
        // Do not all rows see all of the 32 keys?
        const auto is_mixed = [&](uint32_t seen, int kb) {
            return !(seen == 0xffffffffu && kb + 31 <= first && (kb >= low_final || kb + 31 < p.sinks));
        };
        const auto base = [&](int x) { return k.base(x, F::KEYS) + wave * 32; };
        const auto fetch_pages = [&](int x) {
            const int i = min((base(x) + (lane & 31)) >> p.page_shift, p.P - 1);
            copy4(row_table + i, page_lds + (x & 1) * 256);
        };
        const auto seen_keys = [&](int x, int &pg) {
            const int j = base(x) + (lane & 31);
            pg = page_mem[(x & 1) * 64 + (lane & 31)];
            return (uint32_t)__ballot(pg >= 0 && pg < p.pages && j < k.hi && (j >= k.lo || j < k.sink));
        };
        fetch_pages(x0);
        wait_copies<0>();
        int pages;                                   // of the tile that is copied, a key a lane
        uint32_t seen = seen_keys(x0, pages);
        fetch_pages(x0 + 1);
        few_copy<D, FP8, false>(p, pages, base(x0), seen, hk, kt_lds);
        few_copy<D, FP8, true>(p, pages, base(x0), seen, hk, vt_lds);

        // (here, so that the loop below waits for nothing but the copies)
        v8b q[D / 32];
#pragma unroll
        for (int d = 0; d < D / 32; ++d) {
            q_raw[d] = (q_raw[d] ^ factor.sign) | factor.nan;
            asm volatile("" : "+v"(q_raw[d]));
            q[d] = __builtin_bit_cast(v8b, q_raw[d]);
        }
        asm volatile("" : "+v"(sc), "+v"(vs));

        for (int x = x0; x < x1; ++x) {
            const int kb = base(x);
            const bool more = x + 1 < x1;
            wait_copies<F::LOADS>();                 // the keys are here, the values may be under way
            v4f sv[2];
            if (seen) {
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    // tile t's row i is key 8 (i / 4) + i % 4 + 4 t: a lane's results are keys 8 g .. 8 g + 7
                    const int key = 8 * (i16 >> 2) + (i16 & 3) + 4 * t;
                    const uint8_t *row = kt_mem + key * F::ROW;
                    const int turn = F::turn_k(key);
                    sv[t] = (v4f){0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                    for (int d = 0; d < D / 32; ++d) {
                        v8b a;
                        if constexpr (FP8)
                            a = widen(*reinterpret_cast<const v2i *>(row + ((2 * d + (g >> 1)) ^ turn) * 16 + (g & 1) * 8));
                        else
                            a = *reinterpret_cast<const v8b *>(row + ((4 * d + g) ^ turn) * 16);
                        sv[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, q[d], sv[t], 0, 0, 0);
                    }
                }
            }
            wait_reads();
            uint32_t seen_next = 0;
            if (more) {
                seen_next = seen_keys(x + 1, pages);
                wait_reads();
                fetch_pages(x + 2);
                few_copy<D, FP8, false>(p, pages, base(x + 1), seen_next, hk, kt_lds);
            }
            u32x4 up;
            v8b lo;
            bool mixed = false;
            if (seen) {
                mixed = is_mixed(seen, kb);
                float pr[8], top = kLowest;
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    pr[j] = sv[j >> 2][j & 3] * sc;
                if (mixed) {
                    mixed_from = min(mixed_from, x);
                    mixed_to = x;
                    const uint32_t mine8 = row_keys(seen, kb, pos, low, p.sinks) >> (8 * g);
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        pr[j] = (mine8 >> j) & 1 ? pr[j] : -INFINITY;
                }
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    top = fmaxf(top, pr[j]);
                top = max_swap32(max_swap16(top));
                if (__ballot(top > m)) {
                    const float mn = fmaxf(m, top), a = __builtin_amdgcn_exp2f(m - mn);
                    m = mn;
                    l *= a;
#pragma unroll
                    for (int d = 0; d < D / 16; ++d)
                        o[d] *= a;
                }
#pragma unroll
                for (int j = 0; j < 8; j += 2) {
                    const float e0 = __builtin_amdgcn_exp2f(pr[j] - m), e1 = __builtin_amdgcn_exp2f(pr[j + 1] - m);
                    l += e0 + e1;
                    // Two bf16 terms, 16 bits of mantissa, at no cost where memory is the bound: the upper half of the
                    // bits, and what is left plus 2^-16 of the value (the sums' end takes that out of l as well), so that
                    // both terms of a positive numerator are positive and an infinite value stays infinite.
                    const uint32_t b0 = __float_as_uint(e0), b1 = __float_as_uint(e1);
                    up[j / 2] = __builtin_amdgcn_perm(b1, b0, 0x07060302u);
                    const v2b r2 = round2(__builtin_fmaf(e0, 0x1p-16f, e0 - __uint_as_float(b0 & 0xffff0000u)),
                                          __builtin_fmaf(e1, 0x1p-16f, e1 - __uint_as_float(b1 & 0xffff0000u)));
                    lo[j] = r2[0], lo[j + 1] = r2[1];
                }
            }
            if (more)
                wait_copies<F::LOADS + 1>();
            else
                wait_copies<0>();
            if (seen) {
                const auto fragment = [&](int d) {
                    if constexpr (FP8) {
                        const int key = 8 * g + (i16 >> 1);
                        return widen(__builtin_amdgcn_ds_read_tr8_b64_v2i32(
                            (lds_v2i *)(vt_mem + key * F::ROW + (d ^ F::turn_v(key)) * 16 + (i16 & 1) * 8)));
                    } else {
                        const int key = 8 * g + (i16 >> 2);
                        const uint8_t *src = vt_mem + key * F::ROW + ((2 * d + ((i16 & 3) >> 1)) ^ F::turn_v(key)) * 16 + (i16 & 1) * 8;
                        return join(__builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s *)src),
                                    __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s *)(src + 4 * F::ROW)));
                    }
                };
                if (mixed && clear_infinite<FP8>(vt_mem, F::LOADS))
                    left_out = true;
#pragma unroll
                for (int d = 0; d < D / 16; ++d) {
                    const v8b a = fragment(d);
                    o[d] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, __builtin_bit_cast(v8b, up), o[d], 0, 0, 0);
                    o[d] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, lo, o[d], 0, 0, 0);
                }
            }
            wait_reads();
            if (more)
                few_copy<D, FP8, true>(p, pages, base(x + 1), seen_next, hk, vt_lds);
            seen = seen_next;
        }

        if (left_out) {
#pragma unroll 1
            for (int x = mixed_from; x <= mixed_to; ++x)
#pragma unroll 1
                for (int c = 0; c < 32; ++c) {
                    const int key = base(x) + c;
                    if (key >= k.hi)
                        break;
                    const int pg = row_table[key >> p.page_shift];
                    if (pg < 0 || pg >= p.pages || key > pos || (key < low && key >= p.sinks))
                        continue;
                    const uint64_t slot = ((uint32_t)pg << p.page_shift) | (key & ((1 << p.page_shift) - 1));
                    const uint8_t *src = p.v + (slot * p.Hkv + hk) * F::ROW;
#pragma unroll
                    for (int d = 0; d < D / 16; ++d)
                        add_infinite<FP8>(reinterpret_cast<float *>(&o[d]), src + (d * 16 + g * 4) * (F::ROW / D));
                }
        }

        // The four waves' sums to LDS, over their own tiles.
        l = sum_swap32(sum_swap16(l)) * (1.0f + 0x1p-16f);
        float *sums = reinterpret_cast<float *>(mem);
#pragma unroll
        for (int d = 0; d < D / 16; ++d)
            *reinterpret_cast<v4f *>(sums + i16 * F::PAD + d * 16 + g * 4) = o[d];
        if (g == 0) {
            wave_m[wave][i16] = m;
            wave_l[wave][i16] = l;
        }
        __syncthreads();
        // A thread joins E neighbouring sums of one row.
        constexpr int E = F::E, SEGS = D / E;
        const int row = threadIdx.x / SEGS, d0 = threadIdx.x % SEGS * E;
        const bool joins = row < 16 && r0 + row < rows;
        float M = kLowest, L = 0.0f, acc[E];
#pragma unroll
        for (int e = 0; e < E; ++e)
            acc[e] = 0.0f;
        if (joins) {
#pragma unroll
            for (int w = 0; w < F::WAVES; ++w)
                M = fmaxf(M, wave_m[w][row]);
#pragma unroll
            for (int w = 0; w < F::WAVES; ++w) {
                const float f = __builtin_amdgcn_exp2f(wave_m[w][row] - M);
                L += f * wave_l[w][row];
                const float *src = reinterpret_cast<const float *>(smem + w * F::WAVE) + row * F::PAD + d0;
#pragma unroll
                for (int e = 0; e < E; e += 4) {
                    const v4f x = *reinterpret_cast<const v4f *>(src + e);
#pragma unroll
                    for (int c = 0; c < 4; ++c)
                        acc[e + c] = __builtin_fmaf(f, x[c], acc[e + c]);
                }
            }
        }
        __syncthreads();
        bool write = x0 == 0 && x1 == blocks;
        if (!write) {
            // This piece to the workspace; the last one of the item joins them all.
            const int64_t a0 = u - v0 + F::ITEM;             // the item's blocks are units a0 .. a0 + blocks
            const int w_lo = (int)divide(a0, run), w_hi = (int)divide(a0 + blocks - 1, run);
            const auto piece = [&](int w) {
                return buffer_rsrc(p.part + ((int64_t)w * 2 + (w == w_lo ? 1 : 0)) * F::PIECE, F::PIECE * 4);
            };
            if (joins) {
                const __amdgpu_buffer_rsrc_t dst = piece(wg);
#pragma unroll
                for (int e = 0; e < E; e += 4)
                    put4(dst, (row * D + d0 + e) * 4, (v4f){acc[e], acc[e + 1], acc[e + 2], acc[e + 3]});
                if (d0 == 0)
                    put2(dst, (16 * D + row * 2) * 4, (v2f){M, L});
            }
            wait_copies<0>();
            __syncthreads();
            if (threadIdx.x == 0)
                last = __hip_atomic_fetch_add(p.cnt + w_lo, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == w_hi - w_lo;
            __syncthreads();
            write = last;
            if (write) {
                // The threads of the rows there are not take part of the pieces: slice s of S a run of them, the
                // slices' results then meet in LDS in their order.
                const int live = min(16, rows - r0), lines = live <= 1 ? 1 : live <= 2 ? 2 : live <= 4 ? 4 : live <= 8 ? 8 : 16;
                const int S = F::THREADS / SEGS / lines, slice = row / lines, my_row = row % lines;
                const int n = w_hi - w_lo + 1, each = (n + S - 1) / S;
                const int from = w_lo + slice * each, to = min(from + each, w_hi + 1);
                M = kLowest, L = 0.0f;
#pragma unroll
                for (int e = 0; e < E; ++e)
                    acc[e] = 0.0f;
                if (my_row < live) {
#pragma unroll 8
                    for (int w = from; w < to; ++w) {
                        const __amdgpu_buffer_rsrc_t src = piece(w);
                        const v2f ml = get2(src, (16 * D + my_row * 2) * 4);
                        v4f x[E / 4];
#pragma unroll
                        for (int e = 0; e < E / 4; ++e)
                            x[e] = get4(src, (my_row * D + d0 + e * 4) * 4);
                        const float mn = fmaxf(M, ml[0]), fa = __builtin_amdgcn_exp2f(M - mn), fb = __builtin_amdgcn_exp2f(ml[0] - mn);
                        M = mn;
                        L = L * fa + ml[1] * fb;
#pragma unroll
                        for (int e = 0; e < E; ++e)
                            acc[e] = acc[e] * fa + x[e >> 2][e & 3] * fb;
                    }
                }
                float *meet = reinterpret_cast<float *>(smem);       // [S][lines][D + 4]
#pragma unroll
                for (int e = 0; e < E; e += 4)
                    *reinterpret_cast<v4f *>(meet + row * F::PAD + d0 + e) = (v4f){acc[e], acc[e + 1], acc[e + 2], acc[e + 3]};
                if (d0 == 0)
                    *reinterpret_cast<v2f *>(meet + row * F::PAD + D) = (v2f){M, L};
                __syncthreads();
                if (row < live) {
                    for (int t = 1; t < S; ++t) {
                        const float *src = meet + (t * lines + row) * F::PAD;
                        const float m2 = src[D], l2 = src[D + 1];
                        const float mn = fmaxf(M, m2), fa = __builtin_amdgcn_exp2f(M - mn), fb = __builtin_amdgcn_exp2f(m2 - mn);
                        M = mn;
                        L = L * fa + l2 * fb;
#pragma unroll
                        for (int e = 0; e < E; ++e)
                            acc[e] = acc[e] * fa + src[d0 + e] * fb;
                    }
                }
                __syncthreads();
                if (threadIdx.x == 0)
                    __hip_atomic_store(p.cnt + w_lo, 0, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            }
        }
        if (write && joins) {
            const int t = s.q0 + (r0 + row) / p.G, h = hk * p.G + (r0 + row) % p.G;
            const float f = L != 0.0f ? vs / L : 0.0f;           // (nothing seen: zeros)
            uint32_t *dst = reinterpret_cast<uint32_t *>(p.out + ((int64_t)t * p.Hq + h) * D + d0);
#pragma unroll
            for (int e = 0; e < E; ++e)
                acc[e] *= f;
            if (p.gate && L != 0.0f) {                           // (zeros whatever the gate)
                const uint32_t *gt = reinterpret_cast<const uint32_t *>(p.gate + t * p.gate_row + h * p.gate_head + d0);
#pragma unroll
                for (int e = 0; e < E; e += 2) {
                    acc[e] = gated(acc[e], bf16_lo(gt[e / 2]));
                    acc[e + 1] = gated(acc[e + 1], bf16_hi(gt[e / 2]));
                }
            }
#pragma unroll
            for (int e = 0; e < E; e += 2)
                dst[e / 2] = bf16_rne(acc[e]) | (bf16_rne(acc[e + 1]) << 16);
        }
        u += v1 - v0;
        rem += v1 - v0;
        if (rem >= (int64_t)units * tiles * p.Hkv) {
            rem = 0;
            b = __builtin_amdgcn_readfirstlane(next_seq<false>(p, b + 1));
        }
        wait_copies<0>();
    }
}

// ---------------------------------------------------------------------------
// More rows

// 4 D operations per row and key on the matrix units, and 2^x, maximum, sum and conversion of every element on the
// vector unit, which take about as long: the loop therefore issues the next block's K Q^T between the numerators
// of this one and this one's V^T P^T between the maxima of the next.  Measured (one MI355X; a bf16 product of
// 8192^3 reaches 1419 TFLOP/s): a prompt of 8191 tokens, 32 heads over 8, head_dim 128, 572 us, 962 TFLOP/s; the matrix
// units are busy in 42 % of the cycles and vector instructions issue in 38 %.  Chunks of 2 x 2048 tokens behind 8000,
// head_dim 256, 932 us, 720 TFLOP/s, 29 % and 22 %.
//   WAVES   head_dim 128: eight waves on one set of tiles, against four and two workgroups a CU with tiles of 32
//           keys: 570 us against 694.  head_dim 256: one wave a SIMD, whose registers (324 of 512) hold 32 rows of
//           queries (64) and of sums (128), two blocks of scores (32) and the operands read ahead; 64 keys do not
//           fit LDS in four stages.
//   ITEM    what the start and the end of an item cost, as blocks, so that workgroups with many short items (a
//           window) end with those of few long ones: prompt 757 us without, 698 619 603 577 585 595 at 1 3 4 6
//           9 13.
//   AHEAD   LDS operands read before their use; 2, 4 and 8 are alike, 0 (the compiler's own order) 8 % slower.
//   Not kept: copies spread between the matrix instructions (577 -> 625; head_dim 256 912 -> 1200), numerators
//           in three skewed steps (593), all before or all behind the products (706, 575).
//   P       is one bf16 here: a term is off by at most 2^-8 of itself, of either sign, so that sums of many are off by
//           less: results are 2.1e-3 (2-norm) from 64 bits, where their own rounding to bf16 alone makes 1.65e-3.  A
//           second term would take that away and costs a quarter of the rate: prompt 766 us against 577, chunks with
//           head_dim 256 1115 against 926, e4m3 chunk and decodes 266 against 208, window prompt of 8000 tokens 249
//           against 201.
template <int D, bool FP8>
struct Many {
    static constexpr int BK = D == 256 ? 32 : 64;           // keys of a block
    static constexpr int ROW = D * 2;                       // bytes of a head in LDS (bf16)
    static constexpr int CH = ROW / 16;
    static constexpr int TILE = BK * ROW;
    static constexpr int WAVES = D == 128 ? 8 : 4, THREADS = 64 * WAVES, ROWS = 32 * WAVES;
    static constexpr int LOADS = TILE / (16 * THREADS);     // 16-byte copies of a thread per tile
    static constexpr int STAGES = FP8 ? 3 : 4;              // blocks in LDS (e4m3: one more in registers)
    static constexpr int SCRATCH = kMaxSeqs * 12 + 16;      // what finding the run needs
    static constexpr int LDS = 2 * STAGES * TILE > SCRATCH ? 2 * STAGES * TILE : SCRATCH;
    static constexpr int ITEM = 6;                          // what an item costs beside its blocks, in blocks
    static constexpr int JOIN = 4;                          // what joining a piece costs, in blocks
    static constexpr int PIECE = ROWS * D + ROWS * 2;   // floats
    static constexpr int AHEAD = 4;                         // operands read before their use
    // Chunk position of chunk c in row r: c ^ turn, so that 16 lanes of a read of keys (16 rows, one chunk) and
    // 32 of one of values (4 rows, 4 chunks) meet all 64 banks.
    static __device__ __forceinline__ constexpr int turn_k(int r) { return D == 64 ? (r >> 1) & 7 : r & 15; }
    static __device__ __forceinline__ constexpr int turn_v(int r) { return D == 64 ? (r & 2) << 1 : (r & 3) << 2; }
    static constexpr int KV = D == 64 ? 4 : 8, VV = D == 64 ? 2 : 4;   // addresses that differ by more than a constant
};

template <int D, bool FP8>
__global__ __launch_bounds__((Many<D, FP8>::THREADS)) __attribute__((amdgpu_waves_per_eu(D == 256 ? 1 : 2, D == 256 ? 1 : 2))) void many_kernel(AttnArgs p)
{
    using F = Many<D, FP8>;
    constexpr int BK = F::BK, NK = BK / 32, ND = D / 32;
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ int64_t scratch[F::WAVES];
    __shared__ int64_t at;
    __shared__ int at_t, last, longest;
    __shared__ int left_out;             // the last of this workgroup's items (counted from 1) of which values were zeroed
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int i32 = lane & 31, h2 = lane >> 5;

    const auto tiles_of = [&](const Seq &s) { return mine<true>(p, s) ? (int)(((int64_t)s.n * p.G + F::ROWS - 1) / F::ROWS) : 0; };
    const auto tile_keys = [&](const Seq &s, int tile) {
        const int r0 = tile * F::ROWS, r1 = min(r0 + F::ROWS, s.n * p.G) - 1;
        return keys_of<BK>(p, s.len - s.n + r0 / p.G, s.len - s.n + r1 / p.G);
    };
    int b, tile, hk;
    int64_t u, u_end, rem, total, run;
    int wg;
    {
        // Units of each sequence (per key head), from all its tiles.
        int64_t *units = reinterpret_cast<int64_t *>(smem);                    // [B]: units, then their sums before b
        int *tiles = reinterpret_cast<int *>(smem + kMaxSeqs * 8);             // [B + 1]: tiles before b
        const int per = (p.B + F::THREADS - 1) / F::THREADS;
        int64_t own = 0, all;
        if (threadIdx.x == 0)
            longest = 0;
        for (int i = 0; i < per; ++i) {
            const int c = threadIdx.x * per + i;
            if (c < p.B)
                own += tiles_of(load_seq(p, c));
        }
        int64_t before = scan<F::WAVES>(own, scratch, &all) - own;
        for (int i = 0; i < per; ++i) {
            const int c = threadIdx.x * per + i;
            if (c < p.B) {
                units[c] = 0;
                tiles[c] = (int)before;
                before += tiles_of(load_seq(p, c));
            }
        }
        __syncthreads();
        const int n_tiles = (int)all;
        for (int i = threadIdx.x; i < n_tiles; i += F::THREADS) {
            int lo = 0, hi = p.B;            // the last sequence with tiles[c] <= i (it has tiles of its own)
            while (hi - lo > 1) {
                const int mid = (lo + hi) / 2;
                if (tiles[mid] <= i)
                    lo = mid;
                else
                    hi = mid;
            }
            const int blocks = tile_keys(load_seq(p, lo), i - tiles[lo]).blocks;
            atomicAdd(reinterpret_cast<unsigned long long *>(units + lo), (unsigned long long)(blocks + F::ITEM));
            atomicMax(&longest, blocks);
        }
        __syncthreads();
        own = 0;
        for (int i = 0; i < per; ++i) {
            const int c = threadIdx.x * per + i;
            own += c < p.B ? units[c] * p.Hkv : 0;
        }
        before = scan<F::WAVES>(own, scratch, &total) - own;
        if (total == 0)
            return;
        // Equal runs, but none so short that joining the pieces of the longest item, one after the other, takes
        // longer than the blocks of a run: n / run pieces of JOIN blocks' time against run blocks.  (70 tokens of 8
        // heads behind 8383, beside 5 decodes: 395 us with equal runs over all CUs, 114 122 138 at JOIN 3 7 14; 3263
        // tokens of one head: 184, 79 81 90; long prompts, whose runs are longer by themselves, are the same.)
        run = max(divide(total + gridDim.x - 1, gridDim.x), (int64_t)sqrtf((float)F::JOIN * (float)longest));
        const int wgs = (int)divide(total + run - 1, run);
        if ((int)blockIdx.x >= wgs)
            return;
        wg = xcd_item(blockIdx.x, wgs);      // neighbouring runs, which share keys, on one XCD
        u = wg * run;
        u_end = min(u + run, total);
        if (u >= before && u < before + own) {
            int64_t left = u - before;
            for (int i = 0; i < per; ++i) {
                const int c = threadIdx.x * per + i;
                if (c >= p.B)
                    break;
                if (left < units[c] * p.Hkv) {
                    at = left;
                    at_t = c;
                    break;
                }
                left -= units[c] * p.Hkv;
            }
        }
        __syncthreads();
        b = __builtin_amdgcn_readfirstlane(at_t);
        const int64_t per_head = uniform(units[b]);
        rem = uniform(at);
        hk = __builtin_amdgcn_readfirstlane((int)divide(rem, per_head));
        rem -= hk * per_head;
        // the tile of that head
        const Seq s = load_seq(p, b);
        const int n = tiles_of(s);
        tile = 0;
        for (int t0 = 0; t0 < n; t0 += F::THREADS) {
            const int t = t0 + threadIdx.x;
            const int64_t x = t < n ? tile_keys(s, t).blocks + F::ITEM : 0;
            int64_t sum;
            const int64_t upto = scan<F::WAVES>(x, scratch, &sum);
            if (rem >= upto - x && rem < upto) {
                at = rem - (upto - x);
                at_t = t;
            }
            __syncthreads();
            if (rem < sum) {
                tile = __builtin_amdgcn_readfirstlane(at_t);
                rem = at;
                break;
            }
            rem -= sum;
        }
        __syncthreads();
    }

    uint8_t *k_mem = smem, *v_mem = smem + F::STAGES * F::TILE;
    const uint32_t k_lds = lds_addr(k_mem), v_lds = lds_addr(v_mem);
    // LDS addresses of this lane's parts of the fragments in the first block: keys by chunk 2 d + h2 of row i32,
    // values by chunks 4 d ..; further d are constants behind.
    uint32_t k_frag[F::KV], v_frag[F::VV];
#pragma unroll
    for (int d = 0; d < F::KV; ++d)
        k_frag[d] = k_lds + i32 * F::ROW + ((2 * d + h2) ^ F::turn_k(i32)) * 16;
#pragma unroll
    for (int d = 0; d < F::VV; ++d) {
        const int key = 4 * h2 + ((lane & 15) >> 2);
        v_frag[d] = v_lds + key * F::ROW + ((4 * d + 2 * ((lane >> 4) & 1) + ((lane & 3) >> 1)) ^ F::turn_v(key)) * 16 + (lane & 1) * 8;
    }

    // A lane's part of a piece of keys (values) in the cache, see `fetch`.
    uint32_t k_lane, v_lane;
    {
        constexpr int SIZE = FP8 ? D : F::ROW, C = SIZE / 16, R = 64 / C;
        const int row = wave * R + lane / C, c = lane % C;
        k_lane = (lane / C) * p.Hkv * SIZE + (FP8 ? c : c ^ F::turn_k(row)) * 16;
        v_lane = (lane / C) * p.Hkv * SIZE + (FP8 ? c : c ^ F::turn_v(row)) * 16;
    }

    if (threadIdx.x == 0)
        left_out = 0;
    __syncthreads();

    for (int items = 1; u < u_end; ++items) {
        const Seq s = load_seq(p, b);
        const int rows = s.n * p.G;
        const Keys k = tile_keys(s, tile);
        const int units = k.blocks + F::ITEM;         // this item's; its first block is unit ITEM
        const int v0 = __builtin_amdgcn_readfirstlane((int)rem), v1 = (int)min((int64_t)units, v0 + (u_end - u));
        const int x0 = max(v0 - F::ITEM, 0), x1 = max(v1 - F::ITEM, 0);
        if (x1 == 0)
            break;                                   // (the run ends before the item's first block)
        const int r0 = tile * F::ROWS + wave * 32;         // this wave's rows
        const bool busy = r0 < rows;
        const int first = s.len - s.n + r0 / p.G, final = s.len - s.n + (min(r0 + 32, rows) - 1) / p.G;
        const int low_final = window_start(p, final);
        const int tile_first = s.len - s.n + tile * F::ROWS / p.G;     // of the whole tile
        const int tile_low = window_start(p, s.len - s.n + (min((tile + 1) * F::ROWS, rows) - 1) / p.G);
        // Rows past the last one repeat it; their results are not stored.
        const int r = min(r0 + i32, rows - 1), token = r / p.G, head = hk * p.G + r % p.G;
        const int pos = s.len - s.n + token, low = window_start(p, pos);

        u32x4 q_raw[D / 16];
        {
            const uint16_t *src = p.q + (int64_t)(s.q0 + token) * p.q_row + (int64_t)head * p.q_head + h2 * 8;
#pragma unroll
            for (int d = 0; d < D / 16; ++d)
                q_raw[d] = *reinterpret_cast<const u32x4 *>(src + d * 16);
        }
        const ScoreFactor factor = score_factor(p, hk);
        float sc = factor.size;
        float vs = p.v_scale ? p.v_scale[hk] : 1.0f;

        float m = kLowest, l = 0.0f;
        v16f o[ND];
#pragma unroll
        for (int d = 0; d < ND; ++d)
#pragma unroll
            for (int i = 0; i < 16; ++i)
                o[d][i] = 0.0f;

        const int32_t *row_table = p.table + (int64_t)b * p.P;
        const int in_page = (1 << p.page_shift) - 1;
        int mixed_from = x1, mixed_to = x0;          // the blocks that not all rows see whole lie between
        constexpr uint64_t kAll = ~0ull >> (64 - BK);
        // Does no row from `from` on to the one whose window begins at `low` miss a key of the block?
        const auto is_whole = [&](uint64_t seen, int kb, int from, int low) {
            return seen == kAll && kb + BK - 1 <= from && (kb >= low || kb + BK - 1 < p.sinks);
        };
        // Numbers of the 64 pages from page `page0` on, one a lane, and which of them are pages of the cache.
        int page0 = -(1 << 30), pages = 0;
        uint64_t good = 0;
        // Which keys of block x any row sees, with its pages at hand.
        const auto seen_keys = [&](int x) -> uint64_t {
            const int kb = k.base(x, BK), from = kb >> p.page_shift, to = (kb + BK - 1) >> p.page_shift;
            if (from < page0 || to >= page0 + 64) {
                page0 = from;
                pages = row_table[min(page0 + lane, p.P - 1)];
                good = __ballot(pages >= 0 && pages < p.pages);
            }
            const uint64_t used = (~0ull >> (63 - (to - from))) << (from - page0);
            if ((good & used) == used && kb + BK <= k.hi && kb >= k.lo)
                return kAll;
            const int j = kb + lane;
            const bool ok = (good >> (((kb + (lane & (BK - 1))) >> p.page_shift) - page0)) & 1;
            return __ballot(lane < BK && ok && j < k.hi && (j >= k.lo || j < k.sink));
        };
        // Copies of a block's keys and values (bf16: straight to LDS; e4m3: to registers, widened to LDS by `widen_block`).
        u32x4 held[2][FP8 ? F::LOADS / 2 : 1];
        const uint64_t stride = (uint64_t)p.Hkv * (FP8 ? D : F::ROW);
        const uint8_t *k_head = p.k + (int64_t)hk * (FP8 ? D : F::ROW), *v_head = p.v + (int64_t)hk * (FP8 ? D : F::ROW);
        const auto fetch = [&](int x, int stage, uint64_t seen) {
            static_assert(F::turn_v(F::WAVES * 1024 / F::ROW) == 0, "v_lane is for every piece");
            const int kb = k.base(x, BK);
            constexpr int SIZE = FP8 ? D : F::ROW, C = SIZE / 16, R = 64 / C, N = FP8 ? F::LOADS / 2 : F::LOADS;
            // Piece i of this wave: R rows from (WAVES i + wave) R on, a lane 16 bytes of one.  Where the pieces lie in
            // one page each and every key is seen, their addresses are scalar.
            const auto piece = [&](int i, const uint8_t *kp, const uint8_t *vp) {
                if constexpr (FP8) {
                    held[0][i] = *reinterpret_cast<const u32x4 *>(kp + k_lane);
                    held[1][i] = *reinterpret_cast<const u32x4 *>(vp + k_lane);
                } else {
                    const uint32_t dst = stage * F::TILE + (i * F::WAVES + wave) * 1024;
                    copy16_pair(kp, k_lane ^ (F::turn_k(i * F::WAVES * R) * 16), k_lds + dst, vp, v_lane, v_lds + dst);
                }
            };
            if (seen == kAll && (1 << p.page_shift) >= BK) {
                const uint32_t page = __builtin_amdgcn_readlane(pages, (kb >> p.page_shift) - page0);
                uint64_t off = ((page << p.page_shift) | ((kb + wave * R) & in_page)) * stride;
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    piece(i, k_head + off, v_head + off);
                    off += F::WAVES * R * stride;
                }
            } else if (seen == kAll && (1 << p.page_shift) >= R) {
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    const int key = kb + (i * F::WAVES + wave) * R;
                    const uint32_t page = __builtin_amdgcn_readlane(pages, (key >> p.page_shift) - page0);
                    const uint64_t off = ((page << p.page_shift) | (key & in_page)) * stride;
                    piece(i, k_head + off, v_head + off);
                }
            } else {
                const int ln = fresh(lane);
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    const int row = (i * F::WAVES + wave) * R + ln / C, c = ln % C;
                    const uint32_t page = __builtin_amdgcn_ds_bpermute((((kb + row) >> p.page_shift) - page0) * 4, pages);
                    const uint64_t off = ((page << p.page_shift) | ((kb + row) & in_page)) * stride;
                    const bool ok = (seen >> row) & 1;
                    const uint8_t *none = reinterpret_cast<const uint8_t *>(&kNothing);
                    if constexpr (FP8) {
                        held[0][i] = *reinterpret_cast<const u32x4 *>(ok ? k_head + off + c * 16 : none);
                        held[1][i] = *reinterpret_cast<const u32x4 *>(ok ? v_head + off + c * 16 : none);
                    } else {
                        const uint32_t dst = stage * F::TILE + (i * F::WAVES + wave) * 1024;
                        copy16(ok ? k_head + off + (c ^ F::turn_k(row)) * 16 : none, k_lds + dst);
                        copy16(ok ? v_head + off + (c ^ F::turn_v(row)) * 16 : none, v_lds + dst);
                    }
                }
            }
        };
        const auto widen_block = [&](int stage) {
            if constexpr (FP8) {
                constexpr int CH8 = D / 16;
                const int ln = fresh(lane);
#pragma unroll
                for (int i = 0; i < F::LOADS / 2; ++i) {
                    const int row = (i * F::WAVES + wave) * (64 / CH8) + ln / CH8, c = ln % CH8;
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        uint8_t *line = smem + stage * F::TILE + row * F::ROW;
                        const v2i ck = {(int)held[0][i][2 * half], (int)held[0][i][2 * half + 1]};
                        const v2i cv = {(int)held[1][i][2 * half], (int)held[1][i][2 * half + 1]};
                        *reinterpret_cast<v8b *>(line + ((2 * c + half) ^ F::turn_k(row)) * 16) = widen(ck);
                        *reinterpret_cast<v8b *>(line + F::STAGES * F::TILE + ((2 * c + half) ^ F::turn_v(row)) * 16) = widen(cv);
                    }
                }
            }
        };
        // Copies run ahead of the products: those of block x + STAGES - 1 (e4m3: loads into registers, widened into LDS
        // at the step's end) are issued in step x, into the place that block x - 1 leaves.
        constexpr int LEAD = F::STAGES - 1;
        uint64_t seen[F::STAGES];                    // of blocks x, x + 1, ..
#pragma unroll
        for (int i = 0; i < LEAD; ++i) {
            seen[i] = 0;
            if (x0 + i < x1) {
                seen[i] = seen_keys(x0 + i);
                fetch(x0 + i, i, seen[i]);
                widen_block(i);
            }
        }
        seen[LEAD] = 0;
        // (here, so that the loop below waits for nothing but the copies)
        v8b q[D / 16];
#pragma unroll
        for (int d = 0; d < D / 16; ++d) {
            q_raw[d] = (q_raw[d] ^ factor.sign) | factor.nan;
            asm volatile("" : "+v"(q_raw[d]));
            q[d] = __builtin_bit_cast(v8b, q_raw[d]);
        }
        asm volatile("" : "+v"(sc), "+v"(vs));

        // Step x forms the scores of block x + 1 while the numerators of block x are computed, and the sums of block
        // x while the maximum of block x + 1 is taken: a wave's matrix and vector instructions run side by side.
        constexpr int NQ = NK * D / 16, NV = BK / 16 * ND, PAIRS = BK / 4, EARLY = PAIRS / 2, A = F::AHEAD;
        static_assert(NQ % A == 0 && NV % 2 == 0 && EARLY % (BK / 32) == 0, "");
        const auto key_part = [&](const uint32_t (&at)[F::KV], int i) {
            const int t = i % NK, d = i / NK;
            return *(const lds_v8b *)(at[d % F::KV] + d / F::KV * (F::KV * 32) + 32 * t * F::ROW);
        };
        // a lane's keys of 16: 4 h2 .. + 3, then 8 + 4 h2 .. + 3, as the first product left them
        const auto value_part = [&](const uint32_t (&at)[F::VV], int i) {
            const int t = i / ND, d = i % ND;
            const uint32_t src = at[d % F::VV] + d / F::VV * (F::VV * 64) + 16 * t * F::ROW;
            return join(__builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s *)src),
                        __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s *)(src + 8 * F::ROW)));
        };
        const auto mask_block = [&](v16f (&sv)[NK], uint64_t seen, int kb) {
#pragma unroll
            for (int t = 0; t < NK; ++t) {
                const uint32_t keys = row_keys((uint32_t)(seen >> (32 * t)), kb + 32 * t, pos, low, p.sinks) >> (4 * h2);
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    sv[t][i] = (keys >> (8 * (i >> 2) + (i & 3))) & 1 ? sv[t][i] : -INFINITY;
            }
        };
        // The maximum that is subtracted may lag by 2^8: numerators stay far from the types' ends, and the sums are
        // seldom rescaled.
        const auto raise = [&](float top) {
            top = max_swap32(top) * sc;
            if (__ballot(top > m + 8.0f)) {
                const float mn = fmaxf(m, top), f = __builtin_amdgcn_exp2f(m - mn);
                m = mn;
                l *= f;
#pragma unroll
                for (int d = 0; d < ND; ++d)
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        o[d][i] *= f;
            }
        };
        int stage = 0;                               // of block x
        const auto turn = [&](int x, v16f (&sv)[NK], v16f (&sn)[NK]) __attribute__((always_inline)) {
            const int kb = k.base(x, BK);
            const bool next = x + 1 < x1;
            // This wave's copies up to block x + 1 (behind them may be those of block x + 2).
            if (!FP8 && x + 2 < x1)
                wait_copies<2 * F::LOADS>();
            else
                wait_copies<0>();
            if (!is_whole(seen[0], kb, tile_first, tile_low)) {
                mixed_from = min(mixed_from, x);
                mixed_to = x;
                // (what this wave has copied, or widened: 1 or 2 KB of every so many)
                uint8_t *own = v_mem + stage * F::TILE + wave * (FP8 ? 2048 : 1024);
                bool any = clear_infinite<false>(own, FP8 ? F::LOADS / 2 : F::LOADS, (FP8 ? 2 : 1) * F::WAVES);
                if (FP8)
                    any |= clear_infinite<false>(own + 1024, F::LOADS / 2, 2 * F::WAVES);
                if (any)
                    left_out = items;
            }
            __syncthreads();                         // everyone's copies; and block x - 1 is read
            const int ahead = x + LEAD, free_stage = stage == 0 ? F::STAGES - 1 : stage - 1;
            if (ahead < x1) {
                seen[LEAD] = seen_keys(ahead);
                fetch(ahead, free_stage, seen[LEAD]);
            }
            const int next_stage = stage + 1 == F::STAGES ? 0 : stage + 1;
            if (busy) {
                v8b a[A];
                uint32_t k_at[F::KV], v_at[F::VV];   // (so that the reads differ by constants)
                if (x == x0) {
#pragma unroll
                    for (int d = 0; d < F::KV; ++d)
                        k_at[d] = fresh(k_frag[d] + stage * F::TILE);
#pragma unroll
                    for (int i = 0; i < A; ++i)
                        a[i] = key_part(k_at, i);
#pragma unroll
                    for (int i = 0; i < NQ; ++i) {
                        const int t = i % NK, d = i / NK;
                        if (d == 0)
                            sv[t] = zero16();
                        in_order();
                        sv[t] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a[i % A], q[d], sv[t], 0, 0, 0);
                        if (i + A < NQ)
                            a[i % A] = key_part(k_at, i + A);
                    }
                    in_order();
                    if (!is_whole(seen[0], kb, first, low_final))
                        mask_block(sv, seen[0], kb);
                    float top = kLowest;
#pragma unroll
                    for (int i = 0; i < 16 * NK; i += 2)
                        top = fmaxf(fmaxf(top, sv[i / 16][i % 16]), sv[i / 16][i % 16 + 1]);
                    raise(top);
                }
                v8b pr[BK / 16];
                const auto numerators = [&](int j) {
                    const int t = j >> 3, i = (2 * j) & 15;
                    const float e0 = __builtin_amdgcn_exp2f(__builtin_fmaf(sv[t][i], sc, -m));
                    const float e1 = __builtin_amdgcn_exp2f(__builtin_fmaf(sv[t][i + 1], sc, -m));
                    const v2b e = round2(e0, e1);
                    l = __builtin_amdgcn_fdot2_f32_bf16(e, (v2b){(__bf16)1.0f, (__bf16)1.0f}, l, false);
                    pr[j >> 2][(2 * j) & 7] = e[0];
                    pr[j >> 2][((2 * j) & 7) + 1] = e[1];
                };
#pragma unroll
                for (int d = 0; d < F::VV; ++d)
                    v_at[d] = fresh(v_frag[d] + stage * F::TILE);
                if (next) {
#pragma unroll
                    for (int d = 0; d < F::KV; ++d)
                        k_at[d] = fresh(k_frag[d] + next_stage * F::TILE);
#pragma unroll
                    for (int i = 0; i < A; ++i)
                        a[i] = key_part(k_at, i);
#pragma unroll
                    for (int i = 0; i < NQ; ++i) {
                        const int t = i % NK, d = i / NK;
                        if (d == 0)
                            sn[t] = zero16();
                        in_order();
                        sn[t] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a[i % A], q[d], sn[t], 0, 0, 0);
                        a[i % A] = i + A < NQ ? key_part(k_at, i + A) : value_part(v_at, i + A - NQ);
#pragma unroll
                        for (int j = i * EARLY / NQ; j < (i + 1) * EARLY / NQ; ++j)
                            numerators(j);
                    }
                    in_order();
                    if (!is_whole(seen[1], k.base(x + 1, BK), first, low_final))
                        mask_block(sn, seen[1], k.base(x + 1, BK));
                } else {
#pragma unroll
                    for (int i = 0; i < A; ++i)
                        a[i] = value_part(v_at, i);
#pragma unroll
                    for (int j = 0; j < EARLY; ++j)
                        numerators(j);
                }
                float top = kLowest;
#pragma unroll
                for (int i = 0; i < NV; ++i) {
                    const int t = i / ND, d = i % ND;
                    in_order();
                    o[d] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a[i % A], pr[t], o[d], 0, 0, 0);
                    if (i + A < NV)
                        a[i % A] = value_part(v_at, i + A);
                    if (i < NV / 2) {
#pragma unroll
                        for (int j = EARLY + i * 2 * EARLY / NV; j < EARLY + (i + 1) * 2 * EARLY / NV; ++j)
                            numerators(j);
                    } else {
#pragma unroll
                        for (int c = (2 * i - NV) * 8 * NK / NV; c < (2 * i + 2 - NV) * 8 * NK / NV; ++c)
                            top = fmaxf(fmaxf(top, sn[c / 8][2 * c % 16]), sn[c / 8][2 * c % 16 + 1]);
                    }
                }
                in_order();
                raise(next ? top : kLowest);
            }
            if (ahead < x1)
                widen_block(free_stage);
#pragma unroll
            for (int i = 0; i < LEAD; ++i)
                seen[i] = seen[i + 1];
            stage = next_stage;
        };
        v16f score[2][NK];
#pragma unroll
        for (int t = 0; t < NK; ++t)
            score[0][t] = score[1][t] = zero16();
        for (int x = x0; x < x1; x += 2) {
            turn(x, score[0], score[1]);
            if (x + 1 < x1)
                turn(x + 1, score[1], score[0]);
        }
        l = sum_swap32(l);
        if (left_out == items) {
#pragma unroll 1
            for (int x = mixed_from; x <= mixed_to; ++x)
#pragma unroll 1
                for (int c = 0; c < BK; ++c) {
                    const int key = k.base(x, BK) + c;
                    if (key >= k.hi)
                        break;
                    const int pg = row_table[key >> p.page_shift];
                    if (pg < 0 || pg >= p.pages || key > pos || (key < low && key >= p.sinks))
                        continue;
                    const uint64_t slot = ((uint32_t)pg << p.page_shift) | (key & in_page);
                    const uint8_t *src = p.v + (slot * p.Hkv + hk) * (D * (FP8 ? 1 : 2));
#pragma unroll
                    for (int d = 0; d < ND; ++d)
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            add_infinite<FP8>(reinterpret_cast<float *>(&o[d]) + 4 * i, src + (d * 32 + i * 8 + h2 * 4) * (FP8 ? 1 : 2));
                }
        }

        bool write = x0 == 0 && x1 == k.blocks;
        if (!write) {
            const int64_t a0 = u - v0 + F::ITEM;     // its blocks are units a0 .. a0 + blocks
            const int w_lo = (int)divide(a0, run), w_hi = (int)divide(a0 + k.blocks - 1, run);
            const auto piece = [&](int w) {
                return buffer_rsrc(p.part + ((int64_t)w * 2 + (w == w_lo ? 1 : 0)) * F::PIECE, F::PIECE * 4);
            };
            const uint32_t off = wave * (32 * D * 4) + fresh(lane) * 16, ml_off = (F::ROWS * D + (wave * 32 + i32) * 2) * 4;
            {
                const __amdgpu_buffer_rsrc_t dst = piece(wg);
                if (busy) {
#pragma unroll
                    for (int d = 0; d < ND; ++d)
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            put4(dst, off + (d * 4 + i) * 1024, (v4f){o[d][4 * i], o[d][4 * i + 1], o[d][4 * i + 2], o[d][4 * i + 3]});
                    if (h2 == 0)
                        put2(dst, ml_off, (v2f){m, l});
                }
            }
            wait_copies<0>();
            __syncthreads();
            if (threadIdx.x == 0)
                last = __hip_atomic_fetch_add(p.cnt + w_lo, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == w_hi - w_lo;
            __syncthreads();
            write = last;
            if (write && busy) {
                m = kLowest, l = 0.0f;
                for (int w = w_lo; w <= w_hi; ++w) {
                    const __amdgpu_buffer_rsrc_t src = piece(w);
                    const v2f ml = get2(src, ml_off);
                    const float mn = fmaxf(m, ml[0]), fa = __builtin_amdgcn_exp2f(m - mn), fb = __builtin_amdgcn_exp2f(ml[0] - mn);
                    m = mn;
                    l = l * fa + ml[1] * fb;
#pragma unroll
                    for (int d = 0; d < ND; ++d)
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const v4f y = get4(src, off + (d * 4 + i) * 1024);
#pragma unroll
                            for (int c = 0; c < 4; ++c)
                                o[d][4 * i + c] = (w == w_lo ? 0.0f : o[d][4 * i + c] * fa) + y[c] * fb;
                        }
                }
            }
            if (write && threadIdx.x == 0)
                __hip_atomic_store(p.cnt + w_lo, 0, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        }
        const int r_out = r0 + (fresh(lane) & 31);
        if (write && r_out < rows) {
            const int t = s.q0 + r_out / p.G, h = hk * p.G + r_out % p.G;
            const float f = l != 0.0f ? vs / l : 0.0f;
#pragma unroll
            for (int d = 0; d < ND; ++d)
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    o[d][i] *= f;
            if (p.gate && l != 0.0f) {               // (a row that sees nothing: zeros whatever the gate)
                const uint16_t *gt = p.gate + t * p.gate_row + h * p.gate_head + 4 * h2;
#pragma unroll
                for (int d = 0; d < ND; ++d)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const uint2 w = *reinterpret_cast<const uint2 *>(gt + d * 32 + i * 8);
                        o[d][4 * i] = gated(o[d][4 * i], bf16_lo(w.x));
                        o[d][4 * i + 1] = gated(o[d][4 * i + 1], bf16_hi(w.x));
                        o[d][4 * i + 2] = gated(o[d][4 * i + 2], bf16_lo(w.y));
                        o[d][4 * i + 3] = gated(o[d][4 * i + 3], bf16_hi(w.y));
                    }
            }
            uint16_t *dst = p.out + ((int64_t)t * p.Hq + h) * D + 4 * h2;
#pragma unroll
            for (int d = 0; d < ND; ++d)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    uint2 w;
                    w.x = bf16_rne(o[d][4 * i]) | (bf16_rne(o[d][4 * i + 1]) << 16);
                    w.y = bf16_rne(o[d][4 * i + 2]) | (bf16_rne(o[d][4 * i + 3]) << 16);
                    *reinterpret_cast<uint2 *>(dst + d * 32 + i * 8) = w;
                }
        }
        u += v1 - v0;
        rem = 0;
        if (u < u_end) {
            if ((int64_t)(tile + 1) * F::ROWS < rows) {
                ++tile;
            } else {
                tile = 0;
                if (++hk == p.Hkv) {
                    hk = 0;
                    b = __builtin_amdgcn_readfirstlane(next_seq<true>(p, b + 1));
                }
            }
        }
        __syncthreads();                             // the tiles are free
    }
}

}  // namespace kern

namespace {

bool misaligned(const void *p, uintptr_t mask) { return (reinterpret_cast<uintptr_t>(p) & mask) != 0; }

int check_attention_shape(int64_t T, int64_t B, int32_t q_heads, int32_t kv_heads, int32_t head_dim, int32_t cache_dtype)
{
    if (T < 0 || T > (1 << 22) || B < 0 || B > kern::kMaxSeqs || kv_heads < 1 || q_heads < kv_heads || q_heads > 1024 ||
        q_heads % kv_heads != 0 || q_heads / kv_heads > 64 || (head_dim != 64 && head_dim != 128 && head_dim != 256) ||
        cache_dtype < 0 || cache_dtype > 1)
        return A8W8_ERR_SHAPE;
    return A8W8_OK;
}

typedef void (*AttnFn)(kern::AttnArgs);
struct Instance {
    AttnFn fn;
    int threads, lds, per_cu, piece;      // piece: floats of a cut item's piece
};
template <int D, bool FP8>
constexpr Instance few_instance()
{
    using F = kern::Few<D, FP8>;
    return {kern::few_kernel<D, FP8>, F::THREADS, F::LDS, F::PER_CU, F::PIECE};
}
template <int D, bool FP8>
constexpr Instance many_instance()
{
    using F = kern::Many<D, FP8>;
    return {kern::many_kernel<D, FP8>, F::THREADS, F::LDS, D == 64 ? 2 : 1, F::PIECE};
}
const Instance kFew[3][2] = {{few_instance<64, false>(), few_instance<64, true>()},
                             {few_instance<128, false>(), few_instance<128, true>()},
                             {few_instance<256, false>(), few_instance<256, true>()}};
const Instance kMany[3][2] = {{many_instance<64, false>(), many_instance<64, true>()},
                              {many_instance<128, false>(), many_instance<128, true>()},
                              {many_instance<256, false>(), many_instance<256, true>()}};
int dim_index(int head_dim) { return head_dim == 64 ? 0 : head_dim == 128 ? 1 : 2; }

constexpr int kMaxDevices = 64;
std::atomic<int> g_lds_set[kMaxDevices];

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
    *bytes = 0;
    if (T == 0 || B == 0)
        return A8W8_OK;
    const Instance &few = kFew[dim_index(head_dim)][cache_dtype], &many = kMany[dim_index(head_dim)][cache_dtype];
    const int64_t cus = cu_count > 0 ? cu_count : 256;
    int64_t floats = cus * few.per_cu * 2 * few.piece;
    if (T * (q_heads / kv_heads) > kern::kFewRows)
        floats = std::max(floats, cus * many.per_cu * 2 * many.piece);
    *bytes = A8W8_WORKSPACE_COUNTER_BYTES + floats * 4;
    return A8W8_OK;
}

int a8w8_paged_attention(const a8w8_attention_desc *d, void *stream)
{
    if (!d)
        return A8W8_ERR_NULL;
    int rc = check_attention_shape(d->T, d->B, d->q_heads, d->kv_heads, d->head_dim, d->cache_dtype);
    if (rc != A8W8_OK)
        return rc;
    if (d->page_size < 1 || d->page_size > 65536 || (d->page_size & (d->page_size - 1)) || d->window < 0 || d->sinks < 0 ||
        d->max_new < 0 || d->scale != d->scale)
        return A8W8_ERR_SHAPE;
    for (const int64_t s : {d->q_row, d->q_head, d->gate ? d->gate_row : 0, d->gate ? d->gate_head : 0})
        if (s < 0 || s % 8 != 0)
            return A8W8_ERR_SHAPE;
    if (d->T == 0 || d->B == 0)
        return A8W8_OK;                      // (also with a table of no pages, which a batch of no sequences has)
    if (d->pages < 1 || d->table_pages < 1 || d->pages > ((1ll << 31) - 1) / d->page_size ||
        d->table_pages > (1ll << 30) / d->page_size)
        return A8W8_ERR_SHAPE;
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
    int dev = 0;
    if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= kMaxDevices)
        return A8W8_ERR_HIP;
    if (g_lds_set[dev].load(std::memory_order_acquire) == 0) {
        for (const auto *set : {kFew, kMany})
            for (int i = 0; i < 6; ++i)
                if (hipFuncSetAttribute(reinterpret_cast<const void *>(set[i / 2][i % 2].fn),
                                        hipFuncAttributeMaxDynamicSharedMemorySize, set[i / 2][i % 2].lds) != hipSuccess)
                    return A8W8_ERR_HIP;
        g_lds_set[dev].store(1, std::memory_order_release);
    }
    kern::AttnArgs a;
    a.q = static_cast<const uint16_t *>(d->q), a.gate = static_cast<const uint16_t *>(d->gate);
    a.q_row = d->q_row, a.q_head = d->q_head, a.gate_row = d->gate_row, a.gate_head = d->gate_head;
    a.k = static_cast<const uint8_t *>(d->k_cache), a.v = static_cast<const uint8_t *>(d->v_cache);
    a.k_scale = d->k_scale, a.v_scale = d->v_scale;
    a.table = d->page_table, a.q_start = d->q_start, a.lens = d->kv_lens;
    a.out = static_cast<uint16_t *>(d->out);
    a.T = (int32_t)d->T, a.B = (int32_t)d->B, a.P = (int32_t)d->table_pages, a.pages = (int32_t)d->pages;
    a.page_shift = __builtin_ctz((unsigned)d->page_size);
    a.Hq = d->q_heads, a.Hkv = d->kv_heads, a.G = d->q_heads / d->kv_heads, a.window = d->window, a.sinks = d->sinks;
    a.scale = d->scale;
    a.cnt = static_cast<int32_t *>(d->workspace);
    a.part = reinterpret_cast<float *>(static_cast<uint8_t *>(d->workspace) + A8W8_WORKSPACE_COUNTER_BYTES);
    hipStream_t st = static_cast<hipStream_t>(stream);
    const Instance &few = kFew[dim_index(d->head_dim)][d->cache_dtype], &many = kMany[dim_index(d->head_dim)][d->cache_dtype];
    const int64_t most = d->max_new > 0 ? std::min<int64_t>(d->max_new, d->T) : d->T;      // rows of one sequence
    a.few_only = most * a.G <= kern::kFewRows;
    if (!a.few_only)
        hipLaunchKernelGGL(many.fn, dim3((unsigned)(cus * many.per_cu)), dim3(many.threads), (size_t)many.lds, st, a);
    hipLaunchKernelGGL(few.fn, dim3((unsigned)(cus * few.per_cu)), dim3(few.threads), (size_t)few.lds, st, a);
    return hipGetLastError() == hipSuccess ? A8W8_OK : A8W8_ERR_HIP;
}

}  // extern "C"
