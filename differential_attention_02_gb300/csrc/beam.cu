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
//
// A row is read once. Blocks share a row in chunks; a warp reads segments of 256 logits,
// adds their exponentials and keeps each segment's maximum. The W best logits of a chunk
// lie in the W segments of the largest maxima (equal ones in order): any other segment has
// W segments before it that each hold a logit to be preferred. So the selection looks at
// the maxima, reads W segments once more (from L2), and its time does not hang on the
// order of the logits.
#include <limits.h>
#include <math.h>

#include <type_traits>

#include "common.cuh"
#include "kernels.h"

namespace da {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kSegment = kBeamSegment;  // a warp's step, eight logits a lane

// ---------------------------------------------------------------- logits as keys
// Bits whose order as unsigned numbers is that of the values; above -inf's for every candidate.
__device__ __forceinline__ uint32_t ordered(float x) {
    const uint32_t u = __float_as_uint(x + 0.f);  // -0 is +0
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}
// The same, 0 for -inf and NaN: no candidate.
__device__ __forceinline__ uint32_t candidate(float x) { return x > -INFINITY ? ordered(x) : 0; }
// A logit and its token as one key: larger is better, equal logits go to the lowest token. 0: none.
__device__ __forceinline__ uint64_t make_key(uint32_t x, int v) { return x == 0 ? 0 : (uint64_t)x << 32 | (uint32_t)~v; }
__device__ __forceinline__ float key_logit(uint64_t k) {
    const uint32_t o = (uint32_t)(k >> 32);
    return __uint_as_float(o & 0x80000000u ? o & 0x7fffffffu : ~o);
}
__device__ __forceinline__ int key_token(uint64_t k) { return (int)~(uint32_t)k; }

__device__ __forceinline__ uint64_t warp_max_key(uint64_t k) {
    const uint32_t hi = __reduce_max_sync(0xffffffffu, (uint32_t)(k >> 32));
    const uint32_t lo = __reduce_max_sync(0xffffffffu, (uint32_t)(k >> 32) == hi ? (uint32_t)k : 0u);
    return (uint64_t)hi << 32 | lo;
}

// ---------------------------------------------------------------- a row in 16-byte vectors
// Rows begin at any element. Positions count from the 16-byte boundary at or before the row's first logit;
// those outside [off, end) read as -inf, and only vectors that lie inside are loaded whole.
template <typename T>
struct RowView {
    static constexpr int kVec = 16 / sizeof(T);  // logits of a vector
    static constexpr int kLoads = 8 / kVec;      // vectors of a lane in a segment
    const T* base;
    int off, end;

    __device__ __forceinline__ RowView(const T* row, int V) {
        off = (int)((reinterpret_cast<uintptr_t>(row) & 15) / sizeof(T));
        base = row - off;
        end = off + V;
    }
    __device__ __forceinline__ static int position(int segment, int lane, int load) {
        return segment * kSegment + (load * 32 + lane) * kVec;
    }
    __device__ __forceinline__ uint4 load(int at) const {
        uint4 v;
        if (at >= off && at + kVec <= end) {
            asm("ld.global.nc.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(base + at));
        } else {
            uint32_t w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if constexpr (sizeof(T) == 4) {
                    w[i] = at + i >= off && at + i < end ? *reinterpret_cast<const uint32_t*>(base + at + i) : 0xff800000u;
                } else {
                    constexpr uint32_t none = std::is_same<T, __half>::value ? 0xfc00u : 0xff80u;
                    const int lo = at + 2 * i, hi = lo + 1;
                    w[i] = (lo >= off && lo < end ? *reinterpret_cast<const uint16_t*>(base + lo) : none) |
                           (hi >= off && hi < end ? *reinterpret_cast<const uint16_t*>(base + hi) : none) << 16;
                }
            }
            v = make_uint4(w[0], w[1], w[2], w[3]);
        }
        return v;
    }
    // The logits of one vector, and the largest of them (NaN left out unless all are).
    __device__ __forceinline__ static void unpack(uint4 v, float* x) {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (sizeof(T) == 4) {
                x[i] = __uint_as_float(w[i]);
            } else if constexpr (std::is_same<T, __half>::value) {
                const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
                x[2 * i] = f.x;
                x[2 * i + 1] = f.y;
            } else {
                x[2 * i] = bf16lo_to_f32(w[i]);
                x[2 * i + 1] = bf16hi_to_f32(w[i]);
            }
        }
    }
    __device__ __forceinline__ static float largest(uint4 v) {
        if constexpr (sizeof(T) == 4) {
            return fmaxf(fmaxf(__uint_as_float(v.x), __uint_as_float(v.y)), fmaxf(__uint_as_float(v.z), __uint_as_float(v.w)));
        } else if constexpr (std::is_same<T, __half>::value) {
            const __half2* h = reinterpret_cast<const __half2*>(&v);
            const float2 f = __half22float2(__hmax2(__hmax2(h[0], h[1]), __hmax2(h[2], h[3])));
            return fmaxf(f.x, f.y);
        } else {
            const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&v);
            const __nv_bfloat162 m = __hmax2(__hmax2(h[0], h[1]), __hmax2(h[2], h[3]));
            const uint32_t w = *reinterpret_cast<const uint32_t*>(&m);
            return fmaxf(bf16lo_to_f32(w), bf16hi_to_f32(w));
        }
    }
};

// ---------------------------------------------------------------- sums of exponentials
// A lane's sum of e^x, scaled by a base that the warp shares. For maxima below 2^20 the sum is that of
// 2^(x L - c) with the whole number c = ceil(m L), L = log2 e rounded to fp32: one fused product and one
// exponential a term, and a new base changes the sum by a power of two exactly. What L's rounding takes,
// 2^(x (log2 e - L)), is put back for x = m when the sum is done; the rest, of |x - m| 1.4e-8, is below the
// terms' own errors. Other maxima (infinite ones among them) take the terms from x - m.
constexpr float kLog2e = 1.44269504f;
constexpr double kLog2eRest = 1.4426950408889634 - (double)kLog2e, kLn2 = 0.69314718055994531;

__device__ __forceinline__ bool plain_max(float m) { return fabsf(m) < 0x1p20f; }
// Any maximum, and logits with NaN among them (which count as nothing).
__device__ __forceinline__ float any_term(float x, float m, float c) {
    if (plain_max(m)) return x == x ? fast_exp2(fmaf(x, kLog2e, -c)) : 0.f;
    return x == m ? 1.f : x < m ? fast_exp2((x - m) * kLog2e) : 0.f;
}
// The factor between two bases: maxima m (0 behind it: none yet) with their c.
__device__ __forceinline__ float rebase(float from, float to) {
    if (from == -INFINITY) return 0.f;
    if (plain_max(from) && plain_max(to)) {
        const float power = ceilf(from * kLog2e) - ceilf(to * kLog2e);  // not above 0
        return power < -126.f ? 0.f : __int_as_float(((int)power + 127) << 23);
    }
    const double a = plain_max(from) ? kLn2 * ceilf(from * kLog2e) : (double)from;
    const double b = plain_max(to) ? kLn2 * ceilf(to * kLog2e) : (double)to;
    return (float)exp(a - b);
}
// The base's logarithm: the sum is total * exp(base).
__device__ __forceinline__ double base_log(float m) {
    return plain_max(m) ? kLn2 * (ceilf(m * kLog2e) + kLog2eRest * (double)m) : (double)m;
}

// The sum of a lane's four vectors where that takes care; rare, and out of the way of the instruction cache.
template <typename T>
__device__ __noinline__ float any_sum(const uint4* v, float m, float c) {
    float t = 0.f;
#pragma unroll 1
    for (int i = 0; i < 4; ++i) {
        float x[RowView<T>::kVec];
        RowView<T>::unpack(v[i], x);
        for (int j = 0; j < RowView<T>::kVec; ++j) t += any_term(x[j], m, c);
    }
    return t;
}

// One warp: the segments of the W largest maxima, equal ones in order, up to 32 N of them. Returns how many
// there are, and the last one's maximum.
template <int N>
__device__ __forceinline__ int choose_segments(const uint32_t* best, int segments, int W, int lane, int* chosen, uint32_t* last) {
    uint32_t mine[N], u = 0;
    int at = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) mine[i] = i * 32 + lane < segments ? best[i * 32 + lane] : 0;
    int n = 0;
    for (; n < W; ++n) {
        u = 0;
#pragma unroll
        for (int i = N - 1; i >= 0; --i)
            if (mine[i] >= u) u = mine[i], at = i * 32 + lane;
        const uint32_t top = __reduce_max_sync(0xffffffffu, u);
        if (top == 0) break;
        const int segment = __reduce_min_sync(0xffffffffu, u == top ? at : INT_MAX);
        *last = top;
        if (lane == 0) chosen[n] = segment;
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (segment == i * 32 + lane) mine[i] = 0;
    }
    return n;
}

// One block per chunk of a row: its sum of exponentials and its W best logits.
template <typename T>
__global__ void __launch_bounds__(kThreads) beam_rows_kernel(const __grid_constant__ BeamParams p) {
    using View = RowView<T>;
    constexpr int kStep = 4 / View::kLoads;  // segments of a warp's round: four vectors a lane in flight
    __shared__ uint32_t best[kBeamSegments];  // a segment's largest logit
    __shared__ double sums[kWarps];
    __shared__ float maxima[kWarps];
    __shared__ int chosen[kMaxBeamWidth];
    __shared__ int n_chosen;
    __shared__ uint32_t least;
    extern __shared__ uint64_t lists[];  // [W][W]: the best of each chosen segment
    const int row = blockIdx.x / p.chunks, chunk = blockIdx.x % p.chunks;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    pdl_trigger();
    if (p.finished && p.finished[row]) return;
    const View view(static_cast<const T*>(p.logits) + row / p.K * p.stride_b + row % p.K * p.stride_k, p.V);
    const int first = chunk * p.chunk_segments;
    const int segments = min(p.chunk_segments, (view.end + kSegment - 1) / kSegment - first);  // may be none

    float m = -INFINITY, c = 0.f, sum = 0.f;
    for (int s = warp * kStep; s < segments; s += kWarps * kStep) {
        uint4 v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int segment = s + i / View::kLoads;  // one behind the chunk's last reads as nothing
            v[i] = view.load(segment < segments ? View::position(first + segment, lane, i % View::kLoads) : view.end);
        }
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < kStep; ++i) {
            float x = View::largest(v[i * View::kLoads]);
            if (View::kLoads == 2) x = fmaxf(x, View::largest(v[i * View::kLoads + 1]));
            const uint32_t u = __reduce_max_sync(0xffffffffu, candidate(x));
            if (lane == 0 && s + i < segments) best[s + i] = u;
            top = max(top, u);
        }
        if (top == 0) continue;
        const float now = key_logit((uint64_t)top << 32);
        if (now > m) {
            sum *= rebase(m, now);
            m = now;
            c = ceilf(m * kLog2e);
        }
        float t = NAN;
        if (plain_max(m)) {
            float2 t2 = make_float2(0.f, 0.f);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float x[View::kVec];
                View::unpack(v[i], x);
#pragma unroll
                for (int j = 0; j < View::kVec; j += 2) {
                    const float2 y = __ffma2_rn(make_float2(x[j], x[j + 1]), make_float2(kLog2e, kLog2e), make_float2(-c, -c));
                    t2 = __fadd2_rn(t2, make_float2(fast_exp2(y.x), fast_exp2(y.y)));
                }
            }
            t = t2.x + t2.y;
        }
        if (t != t) t = any_sum<T>(v, m, c);
        sum += t;
    }
    double total = sum;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
    if (lane == 0) {
        sums[warp] = total;
        maxima[warp] = m;
    }
    __syncthreads();

    const int64_t out = (int64_t)row * p.chunks + chunk;
    if (warp == 0) {
        uint32_t last = 0;
        const int n = segments <= 128   ? choose_segments<4>(best, segments, p.W, lane, chosen, &last)
                      : segments <= 256 ? choose_segments<8>(best, segments, p.W, lane, chosen, &last)
                                        : choose_segments<kBeamSegments / 32>(best, segments, p.W, lane, chosen, &last);
        if (lane == 0) {
            n_chosen = n;
            least = n == p.W ? last : 1;  // a logit below the last chosen maximum is not among the W best
        }
    } else if (warp == 1) {
        float top = lane < kWarps ? maxima[lane] : -INFINITY;
        const float mine = top;
        top = warp_max(top);
        double s = lane < kWarps && mine > -INFINITY ? sums[lane] * (mine == top ? 1. : exp(base_log(mine) - base_log(top))) : 0.;
#pragma unroll
        for (int o = 4; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        if (lane == 0) {
            p.sums[out] = s;
            p.maxima[out] = top;
        }
    }
    __syncthreads();

    // A warp per chosen segment: its logits that may be among the W best, best first.
    for (int w = warp; w < n_chosen; w += kWarps) {
        uint32_t x[8];
        const int segment = first + chosen[w];
#pragma unroll
        for (int i = 0; i < View::kLoads; ++i) {
            float f[View::kVec];
            View::unpack(view.load(View::position(segment, lane, i)), f);
#pragma unroll
            for (int j = 0; j < View::kVec; ++j) x[i * View::kVec + j] = candidate(f[j]);
        }
        // a token's place in the segment, for the lane's j-th logit
        const auto place = [lane](int j) { return (j / View::kVec * 32 + lane) * View::kVec + j % View::kVec; };
        int n = 0;
        for (; n < p.W; ++n) {
            uint32_t u = 0;
#pragma unroll
            for (int j = 0; j < 8; ++j) u = max(u, x[j]);
            const uint32_t top = __reduce_max_sync(0xffffffffu, u);
            if (top < least) break;
            int at = kSegment;
#pragma unroll
            for (int j = 7; j >= 0; --j) at = x[j] == top ? place(j) : at;
            at = __reduce_min_sync(0xffffffffu, at);
            if (lane == 0) lists[w * p.W + n] = make_key(top, segment * kSegment + at - view.off);
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (place(j) == at) x[j] = 0;
        }
        if (lane == 0 && n < p.W) lists[w * p.W + n] = 0;
    }
    __syncthreads();
    if (warp == 0) {  // the segments' lists, two to a lane, into one
        int at[2] = {0, 0};
        uint64_t head[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) head[i] = i * 32 + lane < n_chosen ? lists[(i * 32 + lane) * p.W] : 0;
        for (int w = 0; w < p.W; ++w) {
            const uint64_t top = warp_max_key(max(head[0], head[1]));
            if (lane == 0) p.keys[out * p.W + w] = top;
            if (top == 0) {
                for (int i = w + 1 + lane; i < p.W; i += 32) p.keys[out * p.W + i] = 0;
                break;
            }
#pragma unroll
            for (int i = 0; i < 2; ++i)
                if (head[i] == top) head[i] = ++at[i] < p.W ? lists[(i * 32 + lane) * p.W + at[i]] : 0;
        }
    }
}

// One block per sequence, a warp per beam: the beam's chunks are merged by their logits, then the
// beams by their ranks.
__global__ void __launch_bounds__(32 * kMaxBeams) beam_merge_kernel(const __grid_constant__ BeamParams p) {
    extern __shared__ uint64_t shared[];  // [K][chunks W] keys, then [K][W] keys, [K][W] scores, [K][W] ranks
    const int b = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31, row = b * p.K + warp;
    const int n = p.chunks * p.W;
    uint64_t* in = shared + (int64_t)warp * n;
    uint64_t* keys = shared + (int64_t)p.K * n;
    double* scores = reinterpret_cast<double*>(keys + p.K * p.W);
    uint64_t* ranks = reinterpret_cast<uint64_t*>(scores + p.K * p.W);
    __shared__ int s_length[kMaxBeams];
    __shared__ bool s_ended[kMaxBeams];
    pdl_wait();
    const double score = p.scores[row];
    const bool ended = p.finished && p.finished[row];
    const int length = p.lengths ? p.lengths[row] : 0;
    const int after = length < INT_MAX && !ended ? length + 1 : length;
    if (lane == 0) {
        s_length[warp] = after;
        s_ended[warp] = ended;
    }
    const double weight = p.length_penalty == 0. ? 1. : pow((double)(after > 1 ? after : 1), p.length_penalty);
    double base = 0., lse = 0.;
    if (!ended) {
        const int64_t at = (int64_t)row * p.chunks;
        for (int i = lane; i < n; i += 32) in[i] = p.keys[at * p.W + i];
        float m[2];
        double s[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            m[i] = i * 32 + lane < p.chunks ? p.maxima[at + i * 32 + lane] : -INFINITY;
            s[i] = m[i] > -INFINITY ? p.sums[at + i * 32 + lane] : 0.;
        }
        const float top = warp_max(fmaxf(m[0], m[1]));
        double sum = 0.;
#pragma unroll
        for (int i = 0; i < 2; ++i) sum += m[i] == top || s[i] == 0. ? s[i] : s[i] * exp(base_log(m[i]) - base_log(top));
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        base = base_log(top);
        lse = log(sum);
        __syncwarp();
        int from[2] = {0, 0};
        uint64_t head[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) head[i] = i * 32 + lane < p.chunks ? in[(i * 32 + lane) * p.W] : 0;
        for (int w = 0; w < p.W; ++w) {
            const uint64_t best = warp_max_key(max(head[0], head[1]));
            if (lane == 0) keys[warp * p.W + w] = best;
#pragma unroll
            for (int i = 0; i < 2; ++i)
                if (best != 0 && head[i] == best) head[i] = ++from[i] < p.W ? in[(i * 32 + lane) * p.W + from[i]] : 0;
        }
        __syncwarp();
    }
    for (int w = lane; w < p.W; w += 32) {
        double s = -INFINITY;
        if (ended) {
            if (w == 0) s = score;
        } else if (const uint64_t key = keys[warp * p.W + w]) {
            const double x = key_logit(key);
            s = score + ((x == base ? 0. : x - base) - lse);
        }
        const double rank = s / weight;
        const bool some = rank > -INFINITY && s > -INFINITY;
        scores[warp * p.W + w] = s;
        const uint64_t u = (uint64_t)__double_as_longlong(rank + 0.);
        ranks[warp * p.W + w] = !some ? 0 : u >> 63 ? ~u : u | 1ull << 63;
    }
    __syncthreads();
    if (warp > 0) return;
    int at = 0;
    uint64_t head = lane < p.K ? ranks[lane * p.W] : 0;
    for (int w = 0; w < p.W; ++w) {
        const int64_t out = (int64_t)b * p.W + w;
        const uint64_t top = warp_max_key(head);
        if (top == 0) {
            if (lane == 0) {
                p.scores_out[out] = -INFINITY;
                p.tokens[out] = p.eos >= 0 ? p.eos : 0;
                p.parents[out] = -1;
                if (p.finished_out) p.finished_out[out] = 1;
                if (p.lengths_out) p.lengths_out[out] = 0;
            }
        } else if (lane == __ffs(__ballot_sync(0xffffffffu, head == top)) - 1) {  // the lowest of equal beams
            const int token = s_ended[lane] ? p.eos : key_token(keys[lane * p.W + at]);
            p.scores_out[out] = (float)scores[lane * p.W + at];
            p.tokens[out] = token;
            p.parents[out] = lane;
            if (p.finished_out) p.finished_out[out] = s_ended[lane] || token == p.eos;
            if (p.lengths_out) p.lengths_out[out] = s_length[lane];
            head = ++at < p.W ? ranks[lane * p.W + at] : 0;
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
    const unsigned blocks = (unsigned)(p.B * p.K * p.chunks);
    const size_t lists = (size_t)p.W * p.W * sizeof(uint64_t);
    if (in_dtype == 0) beam_rows_kernel<float><<<blocks, kThreads, lists, stream>>>(p);
    else if (in_dtype == 1) beam_rows_kernel<__nv_bfloat16><<<blocks, kThreads, lists, stream>>>(p);
    else beam_rows_kernel<__half><<<blocks, kThreads, lists, stream>>>(p);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    e = prepare_once<beam_merge_kernel>(kBeamMergeBytes);
    if (e != cudaSuccess) return e;
    return launch_pdl(beam_merge_kernel, dim3((unsigned)p.B), dim3((unsigned)(32 * p.K)),
                      (size_t)p.K * p.W * (p.chunks + 3) * sizeof(uint64_t), stream, p);
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
