// a8w8_device.h -- device helpers shared by the kernel files: vector types, buffer
// descriptors, the weight fragment's lane layout, and the bf16 store.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace a8w8 {
namespace kern {

typedef float v4f __attribute__((ext_vector_type(4)));
typedef int v4i __attribute__((ext_vector_type(4)));
typedef uint32_t v2u __attribute__((ext_vector_type(2)));
typedef int v8i __attribute__((ext_vector_type(8)));
typedef __bf16 v8b __attribute__((ext_vector_type(8)));
typedef short v4s __attribute__((ext_vector_type(4)));
// Read-only global data read through the constant address space: wave-uniform
// loads from it become scalar loads.
typedef const __attribute__((address_space(4))) float const_f32;

// Raw buffer descriptor over `bytes` bytes at `base` (stride 0, 32-bit data
// format word of the CDNA buffer resource).
__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer_rsrc(const void *base, uint32_t bytes)
{
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(base), (short)0, (int)bytes, 0x00020000);
}

__device__ __forceinline__ v8i cat(v4i lo, v4i hi)
{
    return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
}

__device__ __forceinline__ v4f fma4(v4f d, float s, v4f acc)
{
    acc[0] = __builtin_fmaf(d[0], s, acc[0]);
    acc[1] = __builtin_fmaf(d[1], s, acc[1]);
    acc[2] = __builtin_fmaf(d[2], s, acc[2]);
    acc[3] = __builtin_fmaf(d[3], s, acc[3]);
    return acc;
}

// fp32 -> bf16 bits, round to nearest even (NaN stays a quiet NaN).
__device__ __forceinline__ uint32_t bf16_rne(float f)
{
    uint32_t u = __float_as_uint(f);
    if ((u & 0x7fffffffu) > 0x7f800000u)
        return 0x7fc0u;
    u += 0x7fffu + ((u >> 16) & 1u);
    return u >> 16;
}

// Store the 4 consecutive columns n..n+3 of row m (n < N checked per element
// unless the vector path is allowed and all four exist).
__device__ __forceinline__ void store4(uint16_t *Y, int64_t row_off, int n, int N, bool vec, v4f v)
{
    const uint32_t b0 = bf16_rne(v[0]), b1 = bf16_rne(v[1]);
    const uint32_t b2 = bf16_rne(v[2]), b3 = bf16_rne(v[3]);
    if (vec && n + 3 < N) {
        uint2 pk;
        pk.x = b0 | (b1 << 16);
        pk.y = b2 | (b3 << 16);
        *reinterpret_cast<uint2 *>(Y + row_off + n) = pk;
    } else {
        if (n < N) Y[row_off + n] = (uint16_t)b0;
        if (n + 1 < N) Y[row_off + n + 1] = (uint16_t)b1;
        if (n + 2 < N) Y[row_off + n + 2] = (uint16_t)b2;
        if (n + 3 < N) Y[row_off + n + 3] = (uint16_t)b3;
    }
}

// The whole-line weight loads' lane exchange (see the skinny kernel's comment on weight loads):
// two loads of rows 0-7 and 8-15 of a 16-row tile become the MFMA operand layout, lane l holding
// row l % 16, chunks l / 16 and l / 16 + 4 of the 128-wide block.
__device__ __forceinline__ v8i fix_row_layout(v4i v0, v4i v1)
{
    // lanes 8-15 of each row take v1 from lane p-8; lanes 0-7 take v0 from lane p+8
    v4i a, b;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        a[i] = __builtin_amdgcn_update_dpp(v0[i], v1[i], 0x128, 0xF, 0xC, false);
        b[i] = __builtin_amdgcn_update_dpp(v1[i], v0[i], 0x128, 0xF, 0x3, false);
    }
    return cat(a, b);
}

// Wait until at most N vector-memory operations of this wave are outstanding.
template <int N>
__device__ __forceinline__ void wait_vmcnt()
{
    static_assert(N >= 0 && N < 64, "vmcnt is a 6-bit counter");
    // s_waitcnt immediate (gfx9): vmcnt[3:0] | expcnt[6:4] | lgkmcnt[11:8] | vmcnt[5:4] << 14
    __builtin_amdgcn_s_waitcnt((N & 15) | (7 << 4) | (15 << 8) | ((N >> 4) << 14));
}

// Packed weights (the optional offline layout a8w8_prepack_weights writes):
// rows padded with zeros to a multiple of 16; for every 16-row tile t and K
// block kb, 2 KB in MFMA operand order, [h][lane][16 bytes], lane l holding
// row 16t + l%16, 16-byte chunk l/16 + 4h of the block.  A wave then reads
// each half of a fragment (1 KB) with one contiguous load and needs no lane
// exchange.  Byte offset of tile t, block kb:
__device__ __forceinline__ uint32_t packed_block(uint32_t tile, uint32_t kb, uint32_t KB)
{
    return (tile * KB + kb) << 11;
}
// Weight fragment from its two 16-byte loads (row layout needs the lane exchange).
__device__ __forceinline__ v8i w_fragment(v4i w0, v4i w1, bool pk)
{
    return pk ? cat(w0, w1) : fix_row_layout(w0, w1);
}
// Work item of workgroup b of T: workgroups go to the 8 XCDs in turn, so each XCD gets a
// contiguous run of items (and its L2 what they share).
__device__ __forceinline__ int xcd_item(int b, int T)
{
    const int xcd = b & 7, local = b >> 3;
    const int q = T >> 3, r = T & 7;
    return xcd * q + min(xcd, r) + local;
}
}  // namespace kern
}  // namespace a8w8
