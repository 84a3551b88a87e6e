// Rotary positions for the query and key halves, and the append of many new
// tokens to a paged KV cache with that rotation applied on the way.
//
// The rotation turns each pair of channels j of a row at position p by the angle
// p f_j and multiplies it by m:
//   (a, b) -> m (a cos - b sin, a sin + b cos).
// Differential attention scores two halves, Q1 K1^T and Q2 K2^T; each half is
// rotated like a head of width d, so a rotation is always asked of several
// operands with the same positions. (The source pages take Q and K as given; the
// rotation is what a model applies to them first.)
//
// Angles. f_j arrives as a 0.64 fixed-point number of turns per position, so the
// low 64 bits of p * F_j are the fraction of a turn exactly, whatever the
// position: no range reduction and no 64-bit floating point. Its upper 32 bits,
// as a signed number, are the angle in [-1/2, 1/2) turns (error 2^-32 turns);
// rounding them to fp32 adds at most 2^-25 of a turn, 1.9e-7 rad.
//
// Both kernels move each channel once and are bound by HBM (by latency for a few
// tokens). A thread owns eight channels of one token, four pairs of them rotated,
// and walks over heads with the same four sines and cosines; the rows it loads are
// batched, so that several loads are in flight before the first store.
#include <cuda_fp8.h>
#include <math.h>

#include <type_traits>

#include "common.cuh"
#include "kernels.h"

namespace da {
namespace {

constexpr int kRowsBatch = 4;  // rows loaded before the first is stored

// ---------------------------------------------------------------- eight channels of a row
template <typename T>
struct Vec4 {  // four consecutive 16-bit values
    uint2 v;
};
template <>
struct Vec4<float> {
    float4 v;
};

template <typename T>
__device__ __forceinline__ void unpack4(const Vec4<T>& x, float* f) {
    if constexpr (std::is_same<T, float>::value) {
        f[0] = x.v.x; f[1] = x.v.y; f[2] = x.v.z; f[3] = x.v.w;
    } else if constexpr (std::is_same<T, __half>::value) {
        const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&x.v.x));
        const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&x.v.y));
        f[0] = a.x; f[1] = a.y; f[2] = b.x; f[3] = b.y;
    } else {
        f[0] = bf16lo_to_f32(x.v.x); f[1] = bf16hi_to_f32(x.v.x);
        f[2] = bf16lo_to_f32(x.v.y); f[3] = bf16hi_to_f32(x.v.y);
    }
}

template <typename T>
__device__ __forceinline__ Vec4<T> pack4(const float* f) {
    Vec4<T> x;
    if constexpr (std::is_same<T, float>::value) x.v = make_float4(f[0], f[1], f[2], f[3]);
    else if constexpr (std::is_same<T, __half>::value) x.v = make_uint2(pack_f16x2(f[0], f[1]), pack_f16x2(f[2], f[3]));
    else x.v = make_uint2(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]));
    return x;
}

// The two channel quartets of chunk j of a row: for a rotated chunk of the half
// layout channels 4j.. and r/2 + 4j.. (the pairs' first and second members), else
// 8 consecutive channels. Rows are 16-byte aligned and r a multiple of 8, so a
// quartet is aligned to its own size.
struct Quartets {
    int a, b;
};
__device__ __forceinline__ Quartets quartets(int j, int rotary, int interleaved) {
    if (!interleaved && j < rotary / 8) return {4 * j, rotary / 2 + 4 * j};
    return {8 * j, 8 * j + 4};
}

// Sines and cosines (times the magnitude) of the four pairs of chunk j at a position.
__device__ __forceinline__ void chunk_angles(const RopeTable& t, int j, int64_t pos, float* c, float* s) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const uint64_t turns = (uint64_t)pos * t.freqs[4 * j + k];  // mod 1 turn, for either sign of pos
        const float x = (float)(int32_t)(turns >> 32) * 0x1p-31f;   // angle / pi in [-1, 1)
        sincospif(x, &s[k], &c[k]);
        s[k] *= t.magnitude;
        c[k] *= t.magnitude;
    }
}

// Rotates the eight channels (two quartets) of a rotated chunk in place.
__device__ __forceinline__ void turn(float* a, float* b, const float* c, const float* s, int interleaved) {
    if (interleaved) {  // pairs (a0, a1), (a2, a3), (b0, b1), (b2, b3)
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            float* q = k < 2 ? a + 2 * k : b + 2 * (k - 2);
            const float x = q[0], y = q[1];
            q[0] = x * c[k] - y * s[k];
            q[1] = x * s[k] + y * c[k];
        }
    } else {  // pairs (a_k, b_k)
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const float x = a[k], y = b[k];
            a[k] = x * c[k] - y * s[k];
            b[k] = x * s[k] + y * c[k];
        }
    }
}

// ---------------------------------------------------------------- rotation of up to four operands
// grid.x: blocks of 256 / (d / 8) tokens; grid.y: ranges of the (operand, head) rows
// of a token, so that a few tokens still fill the GPU while many share their sines.
template <typename TI, typename TO>
__global__ void __launch_bounds__(256, sizeof(TI) == 2 ? 4 : 2) rope_kernel(const __grid_constant__ RopeParams p) {
    const int chunks = p.d / 8, per_block = 256 / chunks;
    const int j = threadIdx.x % chunks;
    const int64_t t = (int64_t)blockIdx.x * per_block + threadIdx.x / chunks;
    if (threadIdx.x >= per_block * chunks || t >= (int64_t)p.B * p.N) return;
    const int b = (int)(t / p.N), n = (int)(t % p.N);
    const bool rotated = j < p.table.rotary / 8;
    const Quartets q = quartets(j, p.table.rotary, p.table.interleaved);
    float c[4], s[4];
    if (rotated) {
        chunk_angles(p.table, j, p.positions ? p.positions[t] : n, c, s);
        if (p.backward) {
#pragma unroll
            for (int k = 0; k < 4; ++k) s[k] = -s[k];
        }
    }
    int lo = (int)((int64_t)p.rows * blockIdx.y / gridDim.y);
    const int hi = (int)((int64_t)p.rows * (blockIdx.y + 1) / gridDim.y);
    int o = 0, first = 0;  // operand of row lo, and its first row
    while (lo < hi) {
        while (lo >= first + p.heads[o]) first += p.heads[o++];
        const int end = min(hi, first + p.heads[o]);
        const TI* in = static_cast<const TI*>(p.in[o]) + b * p.in_stride[o][0] + n * p.in_stride[o][2];
        TO* out = static_cast<TO*>(p.out[o]) + b * p.out_stride[o][0] + n * p.out_stride[o][2];
        for (; lo < end; lo += kRowsBatch) {
            Vec4<TI> va[kRowsBatch], vb[kRowsBatch];
#pragma unroll
            for (int u = 0; u < kRowsBatch; ++u) {
                if (lo + u < end) {
                    const TI* row = in + (lo + u - first) * p.in_stride[o][1];
                    va[u] = *reinterpret_cast<const Vec4<TI>*>(row + q.a);
                    vb[u] = *reinterpret_cast<const Vec4<TI>*>(row + q.b);
                }
            }
#pragma unroll
            for (int u = 0; u < kRowsBatch; ++u) {
                if (lo + u < end) {
                    TO* row = out + (lo + u - first) * p.out_stride[o][1];
                    float fa[4], fb[4];
                    unpack4(va[u], fa);
                    unpack4(vb[u], fb);
                    if (rotated) turn(fa, fb, c, s, p.table.interleaved);
                    *reinterpret_cast<Vec4<TO>*>(row + q.a) = pack4<TO>(fa);
                    *reinterpret_cast<Vec4<TO>*>(row + q.b) = pack4<TO>(fb);
                }
            }
        }
        lo = end;
    }
}

template <typename TI>
cudaError_t launch_rope_t(const RopeParams& p, dim3 grid, cudaStream_t stream) {
    if (p.out_dtype == 0) rope_kernel<TI, float><<<grid, 256, 0, stream>>>(p);
    else if (p.out_dtype == 1) rope_kernel<TI, __nv_bfloat16><<<grid, 256, 0, stream>>>(p);
    else rope_kernel<TI, __half><<<grid, 256, 0, stream>>>(p);
    return cudaGetLastError();
}

// ---------------------------------------------------------------- ragged append to a paged cache
// The number of entries of a sorted array that are <= t, by one warp: each step
// narrows the range to one of 32 parts, so up to 32 sequences take one load and up
// to 1024 two. For an unsorted array the result is some number in [0, n].
__device__ __forceinline__ int warp_count_le(const int32_t* a, int n, int t, int lane) {
    int lo = 0, len = n;
    while (len > 0) {
        const int step = (len + 31) / 32;
        const int i = lo + (lane + 1) * step - 1;  // last entry of this lane's part
        const bool le = i < lo + len && a[i] <= t;
        const int full = __popc(__ballot_sync(0xffffffffu, le));  // whole parts that are <= t
        const int end = lo + len;
        lo += full * step;
        len = step == 1 ? 0 : min(step - 1, end - lo);
    }
    return lo;
}

// x / scale, correctly rounded. With the correctly rounded inverse one residual corrects the product
// (Markstein, IBM J. Res. Dev. 34, 1990); infinities, NaN and signed zeros stay what the product says. The residual must
// not underflow where the quotient is an e4m3 value, hence the range of scales that the host allows (inv 0: the
// division itself; 5 sequences of up to 777 tokens, 8 heads, d = 128: 16.3 us with it, 14.6 without).
__device__ __forceinline__ float quotient(float x, float scale, float inv) {
    if (inv == 0.f) return __fdiv_rn(x, scale);
    const float q = x * inv;
    return fabsf(q) < 1e30f && q != 0.f ? fmaf(fmaf(-q, scale, x), inv, q) : q;
}

// Four values as e4m3(x / scale), saturating.
__device__ __forceinline__ uint32_t e4m3x4(const float* f, float scale, float inv) {
    const float2 a = make_float2(quotient(f[0], scale, inv), quotient(f[1], scale, inv));
    const float2 b = make_float2(quotient(f[2], scale, inv), quotient(f[3], scale, inv));
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(a, __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(b, __NV_SATFINITE, __NV_E4M3);
    return lo | (hi << 16);
}

// One warp per (token, range of KV heads); its lanes take the row's chunks of eight
// channels: first K1's d / 8, then K2's, then V's Dv / 8. The token's rows are loaded
// before its sequence is searched for, so that the chain of dependent loads (chunk
// starts, length, page) overlaps them.
template <typename TI, bool FP8>
__global__ void __launch_bounds__(256) append_chunk_kernel(const __grid_constant__ AppendChunkParams p) {
    const int lane = threadIdx.x & 31;
    const int64_t w = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
    const int t = (int)(w / p.head_splits), part = (int)(w % p.head_splits);
    if (t >= p.T) return;
    const int h0 = p.H_kv * part / p.head_splits, h1 = p.H_kv * (part + 1) / p.head_splits;
    const int ck = p.d / 8, total = 2 * ck + p.Dv / 8;
    int64_t page = -1;
    int row = 0, pos = 0;
    bool found = false;
    for (int c0 = 0; c0 < total; c0 += 32) {
        const int cc = c0 + lane;
        const bool active = cc < total;
        const int o = cc < ck ? 0 : cc < 2 * ck ? 1 : 2;
        const int j = cc - o * ck;  // chunk within the row (of V for o == 2)
        const bool rotated = active && o < 2 && j < p.table.rotary / 8;
        const Quartets q = o < 2 ? quartets(j, p.table.rotary, p.table.interleaved) : Quartets{8 * j, 8 * j + 4};
        const TI* in = static_cast<const TI*>(p.in[o]) + (int64_t)t * p.in_stride_t[o];
        float c[4], s[4];
        for (int h = h0; h < h1; h += kRowsBatch) {
            Vec4<TI> va[kRowsBatch], vb[kRowsBatch];
#pragma unroll
            for (int u = 0; u < kRowsBatch; ++u) {
                if (active && h + u < h1) {
                    const TI* r = in + (h + u) * p.in_stride_h[o];
                    va[u] = *reinterpret_cast<const Vec4<TI>*>(r + q.a);
                    vb[u] = *reinterpret_cast<const Vec4<TI>*>(r + q.b);
                }
            }
            if (!found) {
                found = true;
                int b, first, next, len;
                if (p.B <= 32) {  // starts and lengths of all sequences in one step
                    const int end = lane < p.B ? p.q_start[lane + 1] : INT32_MAX;
                    const int lens = lane < p.B ? p.seq_lens[lane] : 0;
                    const int start0 = p.q_start[0];
                    b = __popc(__ballot_sync(0xffffffffu, end <= t));
                    next = __shfl_sync(0xffffffffu, end, b & 31);
                    first = b == 0 ? start0 : __shfl_sync(0xffffffffu, end, (b - 1) & 31);
                    len = __shfl_sync(0xffffffffu, lens, b & 31);
                    if (t < first || b >= p.B) return;  // a row before the first sequence or behind the last
                } else {
                    b = warp_count_le(p.q_start, p.B + 1, t, lane) - 1;
                    if (b < 0 || b >= p.B) return;
                    first = p.q_start[b];
                    next = p.q_start[b + 1];
                    len = p.seq_lens[b];
                }
                const int64_t at = (int64_t)len - ((int64_t)next - first) + (t - first);
                if (at < 0 || at / 64 >= p.max_pages) return;
                page = p.block_table[(int64_t)b * p.max_pages + at / 64];
                if (page < 0 || page >= p.num_pages) return;
                pos = (int)at;
                row = (int)(at % 64);
            }
            if (h == h0 && rotated) chunk_angles(p.table, j, pos, c, s);
#pragma unroll
            for (int u = 0; u < kRowsBatch; ++u) {
                if (active && h + u < h1) {
                    float fa[4], fb[4];
                    unpack4(va[u], fa);
                    unpack4(vb[u], fb);
                    if (rotated) turn(fa, fb, c, s, p.table.interleaved);
                    const int64_t off = page * p.page_stride[o] + (h + u) * p.head_stride[o] + row * p.row_stride[o];
                    if constexpr (FP8) {
                        uint8_t* dst = static_cast<uint8_t*>(p.pages[o]) + off;
                        *reinterpret_cast<uint32_t*>(dst + q.a) = e4m3x4(fa, p.scale[o], p.inv[o]);
                        *reinterpret_cast<uint32_t*>(dst + q.b) = e4m3x4(fb, p.scale[o], p.inv[o]);
                    } else {
                        __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(p.pages[o]) + off;
                        *reinterpret_cast<Vec4<__nv_bfloat16>*>(dst + q.a) = pack4<__nv_bfloat16>(fa);
                        *reinterpret_cast<Vec4<__nv_bfloat16>*>(dst + q.b) = pack4<__nv_bfloat16>(fb);
                    }
                }
            }
        }
    }
}

}  // namespace

cudaError_t launch_rope(const RopeParams& p, cudaStream_t stream) {
    int sms = 0;
    cudaError_t e = device_sm_count(&sms);
    if (e != cudaSuccess) return e;
    const int per_block = 256 / (p.d / 8);
    const int64_t blocks = ((int64_t)p.B * p.N + per_block - 1) / per_block;
    // One resident round of blocks (four per SM) where a token's rows allow it: a thread then keeps
    // its sines for more rows and nothing runs on in a second round.
    int64_t split = (int64_t)sms * 4 / blocks;
    const int64_t most = (p.rows + 1) / 2;
    split = split < most ? split : most;
    const dim3 grid((unsigned)blocks, (unsigned)(split > 1 ? split : 1));
    if (p.in_dtype == 0) return launch_rope_t<float>(p, grid, stream);
    if (p.in_dtype == 1) return launch_rope_t<__nv_bfloat16>(p, grid, stream);
    return launch_rope_t<__half>(p, grid, stream);
}

cudaError_t launch_append_chunk(AppendChunkParams p, cudaStream_t stream) {
    int sms = 0;
    cudaError_t e = device_sm_count(&sms);
    if (e != cudaSuccess) return e;
    // The warps that are resident at once (24 per SM) share the heads of few tokens, a head each at the
    // least: more would start in a second round and look their token up again.
    const int64_t split = (int64_t)sms * 24 / p.T;
    p.head_splits = (int)(split < 1 ? 1 : split < p.H_kv ? split : p.H_kv);
    for (int o = 0; o < 3; ++o) p.inv[o] = p.scale[o] >= 0x1p-60f && p.scale[o] <= 0x1p60f ? 1.f / p.scale[o] : 0.f;
    const int64_t blocks = ((int64_t)p.T * p.head_splits + 7) / 8;
    if (p.in_f16) {
        if (p.fp8) append_chunk_kernel<__half, true><<<(unsigned)blocks, 256, 0, stream>>>(p);
        else append_chunk_kernel<__half, false><<<(unsigned)blocks, 256, 0, stream>>>(p);
    } else {
        if (p.fp8) append_chunk_kernel<__nv_bfloat16, true><<<(unsigned)blocks, 256, 0, stream>>>(p);
        else append_chunk_kernel<__nv_bfloat16, false><<<(unsigned)blocks, 256, 0, stream>>>(p);
    }
    return cudaGetLastError();
}

}  // namespace da
