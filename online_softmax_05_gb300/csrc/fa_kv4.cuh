// fa_kv4.cuh -- the layout of the 4-bit paged key/value cache.
//
// The pool is (pages, Hkv, page_size / 16) blocks.  A block holds 16 tokens of
// one head: key codes (16 rows of D/2 bytes), key scales (16 rows of D/G pairs
// of bf16: s, m), then value codes and value scales alike.  A group of G
// channels stands for s * code + m with
//   m = min,  s = bf16((max - min) / 15),  code = round((x - m) / s) in 0..15.
// s below 2^-100 is stored as 0 (the group is its minimum); a group with a NaN
// or an infinite range has s = m = NaN and reads back as NaN.
//
// Channel order.  The decoding kernel feeds the codes to matrix instructions
// straight from the bytes, so a row's codes lie as their fragments want them:
//   keys    channel 32 g + 8 j + i: nibble i of 32-bit word j D/32 + g
//   values  channel 32 g + 4 r + i: nibble i of 16-bit half-word r D/32 + g
// A lane that reads 16 (D = 128) or 8 (D = 64) consecutive bytes of a key row
// gets 8 channels of every 32, and a lane that reads 8 or 4 bytes of a value
// row 4 channels of every 32: no matrix instruction mixes two groups.
#pragma once

#include <cuda_bf16.h>

#include <cstdint>

namespace fa {

template <int D_, int G_>
struct Kv4 {
    static constexpr int D = D_, G = G_;
    static constexpr int kGroups = D / G;
    static constexpr int kRow = D / 2;            // bytes of a token's codes
    static constexpr int kScaleRow = kGroups * 4;  // bytes of a token's scales
    static constexpr int kKeyCodes = 0;
    static constexpr int kKeyScales = 16 * kRow;
    static constexpr int kValueCodes = kKeyScales + 16 * kScaleRow;
    static constexpr int kValueScales = kValueCodes + 16 * kRow;
    static constexpr int kBlock = kValueScales + 16 * kScaleRow;
};

// Where a token of a sequence lies: the paged table, read with its bounds.
struct Kv4Pages {
    unsigned char* pool;
    const int* table;    // [B][width]
    int width;           // table entries per sequence
    int num_pages;
    int heads;           // Hkv
    int blocks_page;     // page_size / 16
    int shift;           // its logarithm, or -1 if it is no power of two
    long long block_bytes;

    // Byte offset of head 0's block holding slots 16 n .. 16 n + 15 of sequence
    // b, or -1 if the table names no page of the pool there.
    __host__ __device__ __forceinline__ long long block_of(int b, int n) const {
        const int at = shift >= 0 ? n >> shift : n / blocks_page;
        if (at >= width) return -1;
        const int page = table[static_cast<long long>(b) * width + at];
        if (page < 0 || page >= num_pages) return -1;
        return (static_cast<long long>(page) * heads * blocks_page + (n - at * blocks_page)) * block_bytes;
    }
    __host__ __device__ __forceinline__ long long head_bytes() const { return blocks_page * block_bytes; }
    __host__ __device__ __forceinline__ long long capacity() const {
        return static_cast<long long>(width) * blocks_page * 16;
    }
};

inline Kv4Pages kv4_pages(unsigned char* pool, const int* table, int width, int num_pages, int heads, int page_size,
                          int D, int group) {
    Kv4Pages x;
    x.pool = pool;
    x.table = table;
    x.width = width;
    x.num_pages = num_pages;
    x.heads = heads;
    x.blocks_page = page_size / 16;
    x.shift = -1;
    for (int s = 0; s < 16; ++s)
        if (x.blocks_page == 1 << s) x.shift = s;
    x.block_bytes = 16LL * (D + 8 * D / group);
    return x;
}

__device__ __forceinline__ float2 kv4_scale(uint32_t pair) {  // (s, m)
    return make_float2(__uint_as_float(pair << 16), __uint_as_float(pair & 0xffff0000u));
}

}  // namespace fa
