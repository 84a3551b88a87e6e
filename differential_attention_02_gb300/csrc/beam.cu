// Beam search: the best continuations over a sequence's beams and the vocabulary, and
// the reordering of per-beam states that follows.
//
// A live beam k with logits x has a candidate for every token v, with the score
//   s = score_k + (x_v - m) - log(sum_u exp(x_u - m)),  m = max x,
// a finished one a single candidate, itself. Candidates are ranked by s / max(n, 1)^a with
// their length n. Within a beam the ranking is that of the logits, so a row only has to
// give its W best logits, its maximum and its sum; the beams' lists are then merged.
//
// The sum's terms are fp32, each within 2^-22 of itself; partial sums are joined in 64
// bits, and scores are formed and compared in 64 bits, so that the order of two
// candidates of different beams does not hang on fp32's rounding of sums near -50.
#include <limits.h>
#include <math.h>

#include <type_traits>

#include "common.cuh"
#include "kernels.h"

namespace da {
namespace {

constexpr int kThreads = 256;

template <typename T>
__device__ __forceinline__ float load_logit(const T* p) {
    if constexpr (std::is_same<T, float>::value) return *p;
    else if constexpr (std::is_same<T, __half>::value) return __half2float(*p);
    else return __bfloat162float(*p);
}

// A logit and its token as one key: larger is better, equal logits go to the lowest token.
// 0: no candidate (-inf or NaN).
__device__ __forceinline__ uint64_t make_key(float x, int v) {
    if (!(x > -INFINITY)) return 0;
    const uint32_t u = __float_as_uint(x == 0.f ? 0.f : x);  // -0 is +0
    const uint32_t o = u & 0x80000000u ? ~u : u | 0x80000000u;
    return (uint64_t)o << 32 | (uint32_t)~v;
}
__device__ __forceinline__ float key_logit(uint64_t k) {
    const uint32_t o = (uint32_t)(k >> 32);
    return __uint_as_float(o & 0x80000000u ? o & 0x7fffffffu : ~o);
}
__device__ __forceinline__ int key_token(uint64_t k) { return (int)~(uint32_t)k; }

template <typename T, typename F>
__device__ __forceinline__ T block_reduce(T v, F f, T* shared) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = f(v, __shfl_xor_sync(0xffffffffu, v, o));
    __syncthreads();
    if ((threadIdx.x & 31) == 0) shared[threadIdx.x >> 5] = v;
    __syncthreads();
    v = shared[0];
    for (int i = 1; i < kThreads / 32; ++i) v = f(v, shared[i]);
    return v;
}

// One block per row: maximum, sum and, one after the other, the W best logits.
template <typename T>
__global__ void __launch_bounds__(kThreads) beam_rows_kernel(const __grid_constant__ BeamParams p) {
    __shared__ uint64_t keys[kThreads / 32];
    __shared__ double sums[kThreads / 32];
    __shared__ float maxima[kThreads / 32];
    const int row = blockIdx.x, b = row / p.K, k = row % p.K;
    if (p.finished && p.finished[row]) return;
    const T* x = static_cast<const T*>(p.logits) + b * p.stride_b + k * p.stride_k;
    float m = -INFINITY;
    for (int v = threadIdx.x; v < p.V; v += kThreads) m = fmaxf(m, load_logit(x + v));
    m = block_reduce(m, [](float a, float c) { return fmaxf(a, c); }, maxima);
    double sum = 0;
    for (int v = threadIdx.x; v < p.V; v += kThreads) {
        const float y = load_logit(x + v);
        sum += y == m ? 1. : y < m ? (double)expf(y - m) : 0.;
    }
    sum = block_reduce(sum, [](double a, double c) { return a + c; }, sums);
    if (threadIdx.x == 0) {
        p.maxima[row] = m;
        p.sums[row] = sum;
    }
    uint64_t last = ~0ull;
    for (int w = 0; w < p.W; ++w) {
        uint64_t best = 0;
        for (int v = threadIdx.x; v < p.V; v += kThreads) {
            const uint64_t key = make_key(load_logit(x + v), v);
            if (key < last && key > best) best = key;
        }
        last = block_reduce(best, [](uint64_t a, uint64_t c) { return a > c ? a : c; }, keys);
        if (threadIdx.x == 0) p.keys[(int64_t)row * p.W + w] = last;
        if (last == 0) {
            for (int i = w + 1 + threadIdx.x; i < p.W; i += kThreads) p.keys[(int64_t)row * p.W + i] = 0;
            break;
        }
    }
}

// One warp per sequence merges its beams' lists, a beam to a lane.
__global__ void __launch_bounds__(32) beam_merge_kernel(const __grid_constant__ BeamParams p) {
    const int b = blockIdx.x, lane = threadIdx.x, row = b * p.K + lane;
    const bool beam = lane < p.K;
    const double score = beam ? (double)p.scores[row] : -INFINITY;
    const bool ended = beam && p.finished && p.finished[row];
    const int length = beam && p.lengths ? p.lengths[row] : 0;
    const int n = length < INT_MAX && !ended ? length + 1 : length;
    const double weight = p.length_penalty == 0. ? 1. : pow((double)(n > 1 ? n : 1), p.length_penalty);
    const double m = beam && !ended ? (double)p.maxima[row] : 0.;
    const double lse = beam && !ended ? log(p.sums[row]) : 0.;
    const uint64_t* list = p.keys + (int64_t)row * p.W;
    int at = 0;
    double s = -INFINITY, rank = -INFINITY;
    uint64_t key = 0;
    auto head = [&]() {  // the lane's best candidate that is left
        s = -INFINITY;
        key = beam && !ended && at < p.W ? list[at] : 0;
        if (ended && at == 0) s = score;
        else if (key) {
            const double x = key_logit(key);
            s = score + ((x == m ? 0. : x - m) - lse);
        }
        if (!(s > -INFINITY)) s = -INFINITY;
        rank = s > -INFINITY ? s / weight : -INFINITY;
        if (!(rank > -INFINITY)) rank = s = -INFINITY;
    };
    head();
    __syncwarp();  // every lane has read what the outputs may overwrite
    for (int w = 0; w < p.W; ++w) {
        double best = rank;
        int from = lane;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            const double r = __shfl_xor_sync(0xffffffffu, best, o);
            const int f = __shfl_xor_sync(0xffffffffu, from, o);
            if (r > best || (r == best && f < from)) best = r, from = f;
        }
        const int64_t out = (int64_t)b * p.W + w;
        if (!(best > -INFINITY)) {
            if (lane == 0) {
                p.scores_out[out] = -INFINITY;
                p.tokens[out] = p.eos >= 0 ? p.eos : 0;
                p.parents[out] = -1;
                if (p.finished_out) p.finished_out[out] = 1;
                if (p.lengths_out) p.lengths_out[out] = 0;
            }
        } else if (lane == from) {
            const int token = ended ? p.eos : key_token(key);
            p.scores_out[out] = (float)s;
            p.tokens[out] = token;
            p.parents[out] = lane;
            if (p.finished_out) p.finished_out[out] = ended || token == p.eos;
            if (p.lengths_out) p.lengths_out[out] = n;
            ++at;
            head();
        }
        __syncwarp();
    }
}

// ---------------------------------------------------------------- reordering
// A thread owns one unit of every beam of a group: it loads the units of all beams whose
// parent is another, then stores them, so that the group's rows change places in place
// without a second buffer or a barrier. Beams that are their own parent cost nothing.
template <typename U, int KMAX>
__global__ void __launch_bounds__(256) beam_reorder_kernel(const __grid_constant__ ReorderParams p) {
    const ReorderState& s = p.state[blockIdx.z];
    const int64_t t = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (t >= (int64_t)s.parts * s.rows * s.units) return;
    const int64_t line = t / s.units;
    const int unit = (int)(t % s.units), row = (int)(line % s.rows), part = (int)(line / s.rows);
    const int first = blockIdx.y * p.K;
    uint8_t* base = s.ptr + first * s.stride_state + part * s.stride_part + row * s.stride_row + (int64_t)unit * sizeof(U);
    U v[KMAX];
    uint32_t moved = 0;
#pragma unroll
    for (int k = 0; k < KMAX; ++k) {
        if (k >= p.K) break;
        const int parent = p.parents[first + k];
        if (parent == k || parent < 0 || parent >= p.K) continue;
        if (s.by_len && row >= p.lens[first + parent]) continue;
        moved |= 1u << k;
        v[k] = *reinterpret_cast<const U*>(base + parent * s.stride_state);
    }
#pragma unroll
    for (int k = 0; k < KMAX; ++k)
        if (moved >> k & 1) *reinterpret_cast<U*>(base + k * s.stride_state) = v[k];
}

template <typename U>
cudaError_t launch_reorder_u(const ReorderParams& p, dim3 grid, cudaStream_t stream) {
    if (p.K <= 4) beam_reorder_kernel<U, 4><<<grid, 256, 0, stream>>>(p);
    else if (p.K <= 8) beam_reorder_kernel<U, 8><<<grid, 256, 0, stream>>>(p);
    else if (p.K <= 16) beam_reorder_kernel<U, 16><<<grid, 256, 0, stream>>>(p);
    else beam_reorder_kernel<U, kMaxBeams><<<grid, 256, 0, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_beam_select(const BeamParams& p, int in_dtype, cudaStream_t stream) {
    const unsigned rows = (unsigned)(p.B * p.K);
    if (in_dtype == 0) beam_rows_kernel<float><<<rows, kThreads, 0, stream>>>(p);
    else if (in_dtype == 1) beam_rows_kernel<__nv_bfloat16><<<rows, kThreads, 0, stream>>>(p);
    else beam_rows_kernel<__half><<<rows, kThreads, 0, stream>>>(p);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    beam_merge_kernel<<<(unsigned)p.B, 32, 0, stream>>>(p);
    return cudaGetLastError();
}

cudaError_t launch_beam_reorder(const ReorderParams& p, int unit, int count, cudaStream_t stream) {
    int64_t most = 0;
    for (int i = 0; i < count; ++i) {
        const int64_t n = (int64_t)p.state[i].parts * p.state[i].rows * p.state[i].units;
        most = n > most ? n : most;
    }
    if (most == 0) return cudaSuccess;
    const dim3 grid((unsigned)((most + 255) / 256), (unsigned)p.B, (unsigned)count);
    if (unit == 16) return launch_reorder_u<uint4>(p, grid, stream);
    if (unit == 4) return launch_reorder_u<uint32_t>(p, grid, stream);
    if (unit == 2) return launch_reorder_u<uint16_t>(p, grid, stream);
    return launch_reorder_u<uint8_t>(p, grid, stream);
}

}  // namespace da
