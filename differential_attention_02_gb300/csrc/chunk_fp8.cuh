// What the chunk attention's kernels do for an fp8 (e4m3) cache. The operands of one
// tensor-core product have one type; every e4m3 value is an fp16 value, and a bf16 query
// row becomes one of fp16 times a power of two, which goes into the row's score scale.
// So K and V are brought into shared memory raw and rewritten as fp16 by a warpgroup,
// and P is fp16, eight times finer than bf16 down to 2^-21 of a row's largest
// weight (kWeightShift).
//
// The conversion is the instruction cvt.rn.f16x2.e4m3x2 on the halves of a word. Through the
// intrinsic, whose result comes in two halves that have to be joined again, it was slower than four
// integer instructions a pair; written out it is faster: 2 x 1024 tokens at the end of 8192, 16 query and
// 8 KV heads 262 -> 211 us, d = 128 (2 x 1024 of 4096, 8 heads) 184 -> 152 us, 16 x 5 drafted tokens over
// 8192 keys 104 -> 84 us (69 with the later steps of chunk_few_tcgen05.cu). Over a bf16 cache the two
// prompts take 183 and 107 us: the rest is this conversion, done again by every query tile.
//
// What else the path cost on the way, on those drafted tokens in 128-row tiles: K to bf16 beside a
// bf16 query 217 us, K to fp16 197, eight chunks of a thread loaded before the first is stored 164,
// the same in loops small enough for the instruction cache 153, warps without rows kept out 144.
// (Tiles of few rows now have a kernel of their own, chunk_few_tcgen05.cu.)
#pragma once

#include "common.cuh"

namespace da {

// The weights beside an fp16 V are fp16 too, whose values end at 2^-24 (weights below 2^-25 become 0 in
// the product), while the fp32 sum of the weights keeps them. So the running maximum is held lower by this many
// powers of two: a row's largest weight is 2^7, up to 2^15 where the maximum lags by its threshold of 2^8, both
// within fp16's 65504, and a weight is off by at most 2^-32 of the row's largest. Sums, accumulators and partial
// states all carry the factor, and it leaves with the division by the sum. It costs nothing (a constant in the
// maximum's multiplication). A tail of 8191 keys 15, 17 and 18 nats below one key whose V row is zero, relative RMS
// of the output: up to 9e-3, 5e-2 and 1.4e-1 without it, 3e-4, 5e-4 and 1.2e-3 with it.
constexpr float kWeightShift = 7.f;  // log2 units

// fp8 cache: a query row of D bf16 values as fp16 values of the same row times 2^shift, in
// place in its swizzled boxes, by the thread that owns the row; returns 2^-shift. The row's
// largest exponent goes to 2^15, so nothing overflows, and what falls below fp16's normal
// range is smaller than the row's maximum by 2^-29 and more: less than the fp32 sums of the
// scores keep, unless K is zero in the row's largest channels. (Rows below 2^-111 keep a
// factor of 2^126, the last whose inverse is a normal number; their values still come to
// 2^-7 and more, well inside fp16's normal range.)
template <int D>
__device__ __forceinline__ float q_row_to_f16(uint8_t* boxes, int r) {
    uint32_t m = 0;  // largest magnitude of a packed pair's halves
#pragma unroll
    for (int c = 0; c < D / 8; ++c) {
        const uint4 v = *reinterpret_cast<const uint4*>(boxes + (c >> 3) * (128 * 128) + sw128_offset(r, c & 7));
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) m = max(m, max(w[i] & 0x7fffu, (w[i] >> 16) & 0x7fffu));
    }
    const int shift = min(142 - (int)(m >> 7), 126);
    const float up = __uint_as_float((uint32_t)(127 + shift) << 23);
#pragma unroll
    for (int c = 0; c < D / 8; ++c) {
        uint4* at = reinterpret_cast<uint4*>(boxes + (c >> 3) * (128 * 128) + sw128_offset(r, c & 7));
        const uint4 v = *at;
        *at = make_uint4(pack_f16x2(bf16lo_to_f32(v.x) * up, bf16hi_to_f32(v.x) * up),
                         pack_f16x2(bf16lo_to_f32(v.y) * up, bf16hi_to_f32(v.y) * up),
                         pack_f16x2(bf16lo_to_f32(v.z) * up, bf16hi_to_f32(v.z) * up),
                         pack_f16x2(bf16lo_to_f32(v.w) * up, bf16hi_to_f32(v.w) * up));
    }
    fence_proxy_async_shared();  // before the score products read the row
    return __uint_as_float((uint32_t)(127 - shift) << 23);
}

// The score scale of a query row (log2 units): its map's times the row's 2^-shift, kept above zero. Masked
// scores are -inf, and -inf times a scale that underflowed to 0 would be NaN. A row whose scale is raised
// here has raw scores below 2^32 (2^16 x 448 x 128 channels), so scores below 2^-94: 0 either way.
__device__ __forceinline__ float row_score_scale(float map_scale, float down) {
    return fmaxf(map_scale * down, 0x1p-126f);
}

// Sixteen e4m3 values as fp16 values in pairs, exactly.
__device__ __forceinline__ void e4m3x16_to_f16(uint4 x, uint32_t* y) {
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int i = 0; i < 4; ++i)
        asm("{\n\t.reg .b16 lo, hi;\n\t"
            "mov.b32 {lo, hi}, %2;\n\t"
            "cvt.rn.f16x2.e4m3x2 %0, lo;\n\t"
            "cvt.rn.f16x2.e4m3x2 %1, hi;\n\t}"
            : "=r"(y[2 * i]), "=r"(y[2 * i + 1])
            : "r"(w[i]));
}

// Raw chunk c of row r into its two chunks of a swizzled fp16 box.
__device__ __forceinline__ void put_e4m3x16(uint8_t* box, int r, int c, uint4 x) {
    uint32_t y[8];
    e4m3x16_to_f16(x, y);
    *reinterpret_cast<uint4*>(box + sw128_offset(r, 2 * c)) = make_uint4(y[0], y[1], y[2], y[3]);
    *reinterpret_cast<uint4*>(box + sw128_offset(r, 2 * c + 1)) = make_uint4(y[4], y[5], y[6], y[7]);
}

// Four raw chunks, `step` bytes and `rows` rows apart, all loaded before the first is stored; rows
// from `hidden` on become zeros.
__device__ __forceinline__ void convert4(const uint8_t* raw, int step, uint8_t* box, int r, int rows, int c, int hidden) {
    uint4 x[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) x[u] = *reinterpret_cast<const uint4*>(raw + u * step);
#pragma unroll
    for (int u = 0; u < 4; ++u) {
        if (r + u * rows >= hidden) x[u] = make_uint4(0, 0, 0, 0);
        put_e4m3x16(box, r + u * rows, c, x[u]);
    }
}

}  // namespace da
