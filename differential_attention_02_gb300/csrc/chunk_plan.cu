// Work plan and merge of the attention of ragged new tokens over a paged cache.
//
// The chunk starts and lengths live on the device (a captured graph replays with new
// ones), so the device cuts the work: one block lists the query tiles, chooses how
// many key tiles one entry takes, and writes the list of entries that the attention
// kernel's CTAs index. A few microseconds, most of them overlapped with the launch of
// the attention kernel (a programmatic dependent).
//
// Why a split length chosen from the batch: one sequence's last 16 tokens have one
// tile per KV head and fill the GPU only if their keys are split; four prompts'
// chunks have thousands of tiles, and splitting them only costs partial states; a
// batch of both has a few long tiles that would run on alone. With entries of at most
// k key tiles, W key tiles in all and C work items at a time, k >= W / (2 C) bounds
// the number of extra entries by 2 C and the slots of split tiles by 4 C (a tile of
// n > k key tiles has ceil(n / k) <= 2 n / k entries), which sizes the workspace on
// the host. Among the k that cut the longest tile into 1 .. 64 parts, the one with the
// shortest estimated makespan is taken.
#include <math.h>

#include "common.cuh"
#include "kernels.h"

namespace da {
namespace {

constexpr int kPlanThreads = 1024;
constexpr int kMaxParts = 64;
// Fixed cost of an entry (start, epilogue) and of one that leaves a partial state, in
// key tiles: about 4 us and 1.3 us a key tile.
constexpr float kEntryCost = 3.f, kSplitCost = 5.f;

__device__ __forceinline__ int tile_keys(const ChunkTile& t) {  // key tiles that the tile's last token sees
    const int keys = t.pos0 + t.ntok;
    return keys > 0 ? (keys + kChunkKeys - 1) / kChunkKeys : 0;
}

// Exclusive sum over the block of one int per thread; *total gets the whole sum.
__device__ __forceinline__ int block_scan(int v, int* warp_sums, int* total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    __syncthreads();  // earlier readers of warp_sums are done
    if (lane == 31) warp_sums[warp] = x;
    __syncthreads();
    if (warp == 0) {
        const int w = warp_sums[lane];
        int y = w;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int z = __shfl_up_sync(0xffffffffu, y, o);
            if (lane >= o) y += z;
        }
        warp_sums[lane] = y - w;
        if (lane == 31) warp_sums[32] = y;
    }
    __syncthreads();
    *total = warp_sums[32];
    return warp_sums[warp] + x - v;
}

__global__ void __launch_bounds__(kPlanThreads) chunk_plan_kernel(const __grid_constant__ ChunkParams p) {
    __shared__ int warp_sums[33];
    __shared__ long long work_sum;
    __shared__ int work_max;
    __shared__ float est[kMaxParts];
    pdl_trigger();
    pdl_wait();  // the lengths may be the previous kernel's output, and it may still read this workspace
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (tid == 0) {
        work_sum = 0;
        work_max = 0;
    }
    // 1. Query tiles, each sequence's last (longest) one first.
    int n_tiles = 0;
    for (int b0 = 0; b0 < p.B; b0 += kPlanThreads) {
        const int b = b0 + tid;
        int first = 0, n = 0, len = 0;
        if (b < p.B) {
            first = min(max(p.q_start[b], 0), p.T);
            n = min(max(p.q_start[b + 1], first), p.T) - first;
            len = min(max(p.seq_lens[b], 0), p.L);
        }
        const int nt = (n + p.tm - 1) / p.tm;
        int sum;
        const int at = n_tiles + block_scan(nt, warp_sums, &sum);
        for (int i = 0; i < nt && at + i < p.max_tiles; ++i) {
            const int k = nt - 1 - i;
            p.tiles[at + i] = ChunkTile{b, first + k * p.tm, min(p.tm, n - k * p.tm), len - n + k * p.tm};
        }
        n_tiles += sum;
    }
    n_tiles = min(n_tiles, p.max_tiles);  // only starts that are not sorted exceed it
    __syncthreads();
    // 2. Key tiles in all, and of the longest tile.
    long long w = 0;
    int wm = 0;
    for (int i = tid; i < n_tiles; i += kPlanThreads) {
        const int k = tile_keys(p.tiles[i]);
        w += k;
        wm = max(wm, k);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        w += __shfl_xor_sync(0xffffffffu, w, o);
        wm = max(wm, __shfl_xor_sync(0xffffffffu, wm, o));
    }
    if (lane == 0) {
        atomicAdd(reinterpret_cast<unsigned long long*>(&work_sum), (unsigned long long)w);
        atomicMax(&work_max, wm);
    }
    __syncthreads();
    const long long W = work_sum * p.H_kv;
    const int longest = max(work_max, 1);
    // 3. Key tiles per entry: a warp estimates one candidate at a time.
    const int least = max(1, (int)((W + 2 * p.ctas - 1) / (2 * p.ctas)));
    for (int s = 1 + warp; s <= kMaxParts; s += kPlanThreads / 32) {
        const int k = (longest + s - 1) / s;
        float e = INFINITY;
        if (s == 1 || (k >= least && p.max_slots > 0)) {
            float items = 0.f, split = 0.f;
            for (int i = lane; i < n_tiles; i += 32) {
                const int n = tile_keys(p.tiles[i]), parts = max(1, (n + k - 1) / k);
                items += (float)parts;
                if (parts > 1) split += (float)parts;
            }
            items = warp_sum(items) * (float)p.H_kv;
            split = warp_sum(split) * (float)p.H_kv;
            const float ctas = (float)p.ctas, cost = (float)k + (s > 1 ? kSplitCost : kEntryCost);
            const float all = (float)W + kEntryCost * items + (kSplitCost - kEntryCost) * split;
            e = fminf(ceilf(items / ctas) * cost, all / ctas + 0.5f * cost);
        }
        if (lane == 0) est[s - 1] = e;
    }
    __syncthreads();
    int best = 1;
    for (int s = 2; s <= kMaxParts; ++s)
        if (est[s - 1] < est[best - 1]) best = s;
    const int k = (longest + best - 1) / best;
    // 4. Entries, slots and merges.
    int n_entries = 0, n_slots = 0, n_merges = 0;
    for (int i0 = 0; i0 < n_tiles; i0 += kPlanThreads) {
        const int i = i0 + tid;
        ChunkTile t{};
        int n = 0, parts = 0;
        if (i < n_tiles) {
            t = p.tiles[i];
            n = tile_keys(t);
            parts = max(1, (n + k - 1) / k);
        }
        int se, ss, sm;
        const int ae = n_entries + block_scan(parts, warp_sums, &se);
        const int as = n_slots + block_scan(parts > 1 ? parts : 0, warp_sums, &ss);
        const int am = n_merges + block_scan(parts > 1 ? 1 : 0, warp_sums, &sm);
        // The bounds hold for every batch (see the top); the checks keep the writes inside all the same.
        for (int j = 0; j < parts && ae + j < p.max_entries; ++j) {
            const int lo = (int)((long long)n * j / parts), hi = (int)((long long)n * (j + 1) / parts);
            const int slot = parts > 1 && as + j < p.max_slots ? as + j : -1;
            p.entries[ae + j] = ChunkEntry{t, lo, hi - lo, slot, 0};
        }
        if (parts > 1 && am < p.max_merges && as + parts <= p.max_slots) p.merges[am] = ChunkMerge{t, as, parts, {0, 0}};
        n_entries += se;
        n_slots += ss;
        n_merges += sm;
    }
    if (tid == 0) *p.plan = ChunkPlan{n_tiles, min(n_entries, p.max_entries), min(n_merges, p.max_merges), k};
}

// Joins the partial states of a split tile: block (merge, KV head) x eight rows; a thread
// owns four output columns of one row. Then the combination, the row's RMSNorm and the
// (1 - lambda_init) scale, as the attention kernels' own epilogues. The slots are
// added in the order of their keys.
constexpr int kMergeRows = 8;

template <int DV>
__global__ void __launch_bounds__(kMergeRows * DV / 4) chunk_merge_kernel(const __grid_constant__ ChunkParams p) {
    constexpr int CG = DV / 4;
    __shared__ float red[CG][kMergeRows + 1];
    pdl_trigger();
    pdl_wait();
    const int m = blockIdx.x / p.H_kv, hk = blockIdx.x % p.H_kv;
    if (m >= p.plan->merges) return;
    const ChunkMerge g = p.merges[m];
    const int row = blockIdx.y * kMergeRows + threadIdx.x % kMergeRows, cg = threadIdx.x / kMergeRows;
    const int rows = g.tile.ntok * p.group;
    if (blockIdx.y * kMergeRows >= rows) return;
    const bool live = row < rows;
    const int r = live ? row : 0;
    float M[2] = {kChunkNoMax, kChunkNoMax}, l[2] = {0.f, 0.f};
    float o[2][4] = {};
    for (int s = 0; s < g.count; ++s) {
        const int64_t item = (int64_t)(g.slot + s) * p.H_kv + hk;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const float2 st = *reinterpret_cast<const float2*>(p.part_stats + ((item * 2 + k) * p.rows + r) * 2);
            const float4 v = *reinterpret_cast<const float4*>(p.part_o + (((item * 2 + k) * CG + cg) * p.rows + r) * 4);
            const float n = fmaxf(M[k], st.x), a = fast_exp2(M[k] - n), c = fast_exp2(st.x - n);
            M[k] = n;
            l[k] = l[k] * a + st.y * c;
            o[k][0] = o[k][0] * a + v.x * c;
            o[k][1] = o[k][1] * a + v.y * c;
            o[k][2] = o[k][2] * a + v.z * c;
            o[k][3] = o[k][3] * a + v.w * c;
        }
    }
    // A row that sees no key has l = 0 and gives zeros.
    const float i1 = l[0] > 0.f ? p.v_scale / l[0] : 0.f, i2 = l[1] > 0.f ? p.lambda * p.v_scale / l[1] : 0.f;
    float x[4], ss = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[i] = o[0][i] * i1 - o[1][i] * i2;
        ss = fmaf(x[i], x[i], ss);
    }
    red[cg][threadIdx.x % kMergeRows] = ss;
    __syncthreads();
    float tot = 0.f;
#pragma unroll 8
    for (int c = 0; c < CG; ++c) tot += red[c][threadIdx.x % kMergeRows];
    if (!live) return;
    const float sc = (1.0f - p.lambda_init) / sqrtf(tot / (float)DV + p.eps);
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] *= tot > 0.f ? sc : 0.f;
    if (p.norm_w) {
        const float4 wv = *reinterpret_cast<const float4*>(p.norm_w + cg * 4);
        x[0] *= wv.x; x[1] *= wv.y; x[2] *= wv.z; x[3] *= wv.w;
    }
    const int64_t at = ((int64_t)(g.tile.t0 + row / p.group) * p.H + hk * p.group + row % p.group) * DV + cg * 4;
    if (p.out_bf16 || p.out_f16)
        *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.out) + at) =
            make_uint2(pack_16x2(x[0], x[1], p.out_f16 != 0), pack_16x2(x[2], x[3], p.out_f16 != 0));
    else
        *reinterpret_cast<float4*>(static_cast<float*>(p.out) + at) = make_float4(x[0], x[1], x[2], x[3]);
}

}  // namespace

cudaError_t launch_chunk_plan(const ChunkParams& p, cudaStream_t stream) {
    return launch_pdl(chunk_plan_kernel, dim3(1), dim3(kPlanThreads), 0, stream, p);
}

cudaError_t launch_chunk_merge(const ChunkParams& p, cudaStream_t stream) {
    const dim3 grid(p.max_merges * p.H_kv, (p.rows + kMergeRows - 1) / kMergeRows);
    if (p.Dv == 128) return launch_pdl(chunk_merge_kernel<128>, grid, dim3(kMergeRows * 32), 0, stream, p);
    return launch_pdl(chunk_merge_kernel<256>, grid, dim3(kMergeRows * 64), 0, stream, p);
}

}  // namespace da
