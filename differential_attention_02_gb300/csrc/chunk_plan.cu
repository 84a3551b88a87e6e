// Work plan and merge of the attention of ragged new tokens over a paged cache.
//
// The chunk starts and lengths live on the device (a captured graph replays with new
// ones), so the device cuts the work: one block lists the query tiles, chooses how many
// key tiles one entry takes and writes the list of entries that the attention kernel's
// CTAs index, longest first.
//
// Why a split length chosen from the batch: one sequence's last 16 tokens have one item
// (a tile and a KV head) per head and fill the GPU only if their keys are split; four
// prompts' chunks have a thousand items, and splitting them only costs partial states.
// Of the lengths that cut the longest item into 1 .. 64 parts, the one with the shortest
// estimated makespan is taken, at a fixed cost per entry (start and epilogue: about 4 us
// against 1.3 us a key tile; 5 against 0.8 in tiles of few rows), a further one per partial
// state, and the merge's own time. With W key tiles in all and room for E more entries (three rounds of CTAs, api.cu),
// a length k >= W / E adds at most E entries and leaves at most 2 E of them partial (an
// item of n > k key tiles has ceil(n / k) <= 2 n / k parts), which sizes the lists and
// the workspace on the host. Batches of two rounds of items and more stay whole: a mixed
// batch of 428 items took 106 us cut and 102 whole, and cutting the whole row of items
// at every multiple of W / C, which balances any batch within an entry, was no faster either
// (four prompts' chunks 592 against 586 us, the mixed batch 110 against 104), since
// every cut costs a partial state of 128 KB and its merge. The rule looks at the number of
// items alone and those batches were of like lengths: one sequence much longer than the others in a
// batch of that size stays whole, one CTA per head, and sets the time.
//
// The costs per entry, state and merge step were fitted to the single-CTA kernels and are used for
// the CTA pairs as well.
#include <math.h>

#include "common.cuh"
#include "kernels.h"

namespace da {
namespace {

constexpr int kPlanThreads = 512, kPlanWarps = kPlanThreads / 32;
constexpr int kMaxParts = 64;  // two estimates a lane; one sequence with one KV head leaves 88 of 152 SMs without work
constexpr int kTilesInSmem = 2048;  // longer lists are read back from the workspace
constexpr float kEntryCost = 3.f, kFewEntryCost = 6.f, kMergeCost = 3.f, kMergeStep = 0.45f;  // key tiles' times

__device__ __forceinline__ int tile_keys(const ChunkTile& t) {  // key tiles that the tile's last token sees
    const int keys = t.pos0 + t.ntok;
    return keys > 0 ? (keys + kChunkKeys - 1) / kChunkKeys : 0;
}

// Exclusive sum over the block of one value per thread; *total gets the whole sum.
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
    // Every warp adds up the warps' sums itself: one barrier less than handing them out.
    const int w = lane < kPlanWarps ? warp_sums[lane] : 0;
    int y = w;
#pragma unroll
    for (int o = 1; o < kPlanWarps; o <<= 1) {
        const int z = __shfl_up_sync(0xffffffffu, y, o);
        if (lane >= o) y += z;
    }
    *total = __shfl_sync(0xffffffffu, y, kPlanWarps - 1);
    return __shfl_sync(0xffffffffu, y - w, warp) + x - v;
}

__global__ void __launch_bounds__(kPlanThreads) chunk_plan_kernel(const __grid_constant__ ChunkLists lists) {
    const ChunkParams& p = lists.p[blockIdx.x];
    __shared__ int warp_sums[kPlanWarps];
    __shared__ float est[kMaxParts];
    __shared__ int est_items[kMaxParts];
    __shared__ int keys_s[kTilesInSmem];
    __shared__ int count[5];  // entries of each class of length, merges
    __shared__ int longest_s;
    __shared__ unsigned long long row_s;  // key tiles of all tiles
    pdl_trigger();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (tid < 5) count[tid] = 0;
    if (tid == 5) longest_s = 0;
    if (tid == 6) row_s = 0;
    pdl_wait();  // the lengths may be the previous kernel's output, and it may still read this workspace
    // 1. Query tiles, each sequence's last (longest) one first.
    int n_tiles = 0;
    for (int b0 = 0; b0 < p.B; b0 += kPlanThreads) {
        const int b = b0 + tid;
        int first = 0, n = 0, len = 0;
        if (b < p.B) {
            first = p.q_start[b];
            const int next = p.q_start[b + 1], m = p.seq_lens[b];
            first = min(max(first, 0), p.T);
            n = min(max(next, first), p.T) - first;
            len = min(max(m, 0), p.L);
        }
        // Only a sequence's last tile may have few rows.
        int nt = (n + p.tm - 1) / p.tm, end = nt;
        if (p.which != kTilesAll && nt > 0) {
            const bool few = (n - (nt - 1) * p.tm) * p.group <= kFewRows;
            if (p.which == kTilesMany) nt = end -= few;
            else nt = few;
        }
        int sum;
        const int at = n_tiles + block_scan(nt, warp_sums, &sum);
        unsigned long long keys = 0;
        int most = 0;
        for (int i = 0; i < nt && at + i < p.max_tiles; ++i) {
            const int k = end - 1 - i;
            const ChunkTile t{b, first + k * p.tm, min(p.tm, n - k * p.tm), len - n + k * p.tm};
            p.tiles[at + i] = t;
            const int q = tile_keys(t);
            if (at + i < kTilesInSmem) keys_s[at + i] = q;
            keys += q;
            most = max(most, q);
        }
        if (most > 0) {
            atomicAdd(&row_s, keys);
            atomicMax(&longest_s, most);
        }
        n_tiles += sum;
    }
    n_tiles = min(n_tiles, p.max_tiles);  // only starts that are not sorted exceed it
    __syncthreads();
    auto keys_of = [&](int i) { return i < kTilesInSmem ? keys_s[i] : tile_keys(p.tiles[i]); };
    const int longest = max(longest_s, 1), n_items = n_tiles * p.H_kv;
    const long long W = (long long)row_s * p.H_kv;
    // 2. Key tiles per entry: a warp estimates one number of parts at a time. Batches of two rounds of
    // items and more stay whole.
    int k = longest, entries = n_items;
    const bool may_split = p.max_slots > 0 && W > 0 && n_items < 2 * p.ctas;
    if (may_split) {
        const int least = (int)((W + p.max_merges - 1) / p.max_merges);  // where it is above `longest`, nothing is split
        const float entry_cost = p.which == kTilesFew ? kFewEntryCost : kEntryCost;
        const float split_cost = entry_cost + 5.f * (float)p.rows / kChunkRows, ctas = (float)p.ctas;
        int width = 32;  // lanes that the merge gives to a row's parts: 32 / width (below)
        while (width / 2 >= p.rows) width /= 2;
        for (int s = 1 + warp; s <= kMaxParts; s += kPlanWarps) {
            const int ks = (longest + s - 1) / s;
            float e = INFINITY;
            int all = 0;
            if (s == 1 || ks >= least) {
                int items = 0, split = 0;
                for (int i = lane; i < n_tiles; i += 32) {
                    const int n = keys_of(i), parts = n > ks ? (n + ks - 1) / ks : 1;
                    items += parts;
                    split += parts > 1 ? parts : 0;
                }
                all = __reduce_add_sync(0xffffffffu, items) * p.H_kv;
                const float all_items = (float)all;
                const float all_split = (float)__reduce_add_sync(0xffffffffu, split) * (float)p.H_kv;
                const float cost = (float)ks + (s > 1 ? split_cost : entry_cost);
                const float sum = (float)W + entry_cost * all_items + (split_cost - entry_cost) * all_split;
                // Whole items differ in length and the short ones fill in behind the long ones; parts are alike
                // (with one factor 160 ragged decoding items were cut, 84 us against 77 whole, and 64 of d = 128, 109
                // against 92; without the merge's steps one item of 98 key tiles got 49 parts, 53 us against 33).
                e = fminf(ceilf(all_items / ctas) * cost, sum / ctas + (s > 1 ? 0.75f : 0.5f) * cost) +
                    (s > 1 ? kMergeCost + kMergeStep * (float)((s * width + 31) / 32) : 0.f);
            }
            if (lane == 0) {
                est[s - 1] = e;
                est_items[s - 1] = all;
            }
        }
        __syncthreads();
        // Every warp finds the same minimum; the fewest parts among equals.
        const float a = est[lane], b = est[lane + 32];
        float e = fminf(a, b);
        int s = a <= b ? lane + 1 : lane + 33;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            const float e2 = __shfl_xor_sync(0xffffffffu, e, o);
            const int s2 = __shfl_xor_sync(0xffffffffu, s, o);
            if (e2 < e || (e2 == e && s2 < s)) {
                e = e2;
                s = s2;
            }
        }
        k = (longest + s - 1) / s;
        entries = est_items[s - 1];
    }
    // 3. Entries by class of length (over 1/2, 1/4, 1/8 of the longest, shorter) and their slots.
    // Two lists of two classes each, one from the front and one from the back, so that one pass places
    // them. The place within a class depends on the order of the atomics; the slots, and with them
    // every sum, do not.
    int n_slots = 0;
    for (int i0 = 0; i0 < n_items; i0 += kPlanThreads) {
        const int i = i0 + tid;
        ChunkTile t{};
        int n = 0, parts = 0, hk = 0;
        if (i < n_items) {
            const int ti = (unsigned)i / (unsigned)p.H_kv;
            hk = i - ti * p.H_kv;
            t = p.tiles[ti];
            n = tile_keys(t);
            parts = n > k ? (n + k - 1) / k : 1;
        }
        // Where all entries run at once their order does not matter: they take the places of a running sum
        // (no atomics: one token of 16 heads 8.8 -> 6.8 us). One round, since entries <= ctas <= threads.
        if (entries <= p.ctas && entries <= kPlanThreads) {
            int sum;
            const int split = parts > 1 ? parts : 0;
            const int at = block_scan(parts | split << 16, warp_sums, &sum);  // 512 entries at most
            const int ae = at & 0xffff, as = at >> 16;
            if (split > 0 && as + parts <= p.max_slots) {
                const int m = atomicAdd(&count[4], 1);
                if (m < p.max_merges) p.merges[m] = ChunkMerge{t, as, parts, hk, 0};
            }
            int lo = 0;
            for (int j = 0; j < parts && ae + j < p.max_entries; ++j) {
                const int hi = (int)((unsigned)(n * (j + 1)) / (unsigned)parts);
                p.entries[ae + j] = ChunkEntry{t, lo, hi - lo, split > 0 && as + j < p.max_slots ? as + j : -1, hk};
                lo = hi;
            }
            if (tid == 0) count[0] = min(sum & 0xffff, p.max_entries);
            break;
        }
        int as = 0;
        if (k < longest) {
            int sum;
            as = n_slots + block_scan(parts > 1 ? parts : 0, warp_sums, &sum);
            n_slots += sum;
            if (parts > 1 && as + parts <= p.max_slots) {
                const int m = atomicAdd(&count[4], 1);
                if (m < p.max_merges) p.merges[m] = ChunkMerge{t, as, parts, hk, 0};
            }
        }
        const int most = __reduce_max_sync(0xffffffffu, parts);
        for (int j = 0; j < most; ++j) {
            int lo = 0, hi = 0, c = 4;
            if (j < parts) {
                lo = (int)((unsigned)(n * j) / (unsigned)parts);  // n < 2^25 (L < 2^31), parts <= 64
                hi = (int)((unsigned)(n * (j + 1)) / (unsigned)parts);
                const int len = hi - lo;
                c = 2 * len > k ? 0 : 4 * len > k ? 1 : 8 * len > k ? 2 : 3;
            }
            // One atomic per warp and class.
            int place = 0;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const unsigned m = __ballot_sync(0xffffffffu, c == q);
                if (m == 0) continue;
                int base = 0;
                if (lane == 0) base = atomicAdd(&count[q], __popc(m));
                base = __shfl_sync(0xffffffffu, base, 0);
                if (c == q) place = base + __popc(m & ((1u << lane) - 1));
            }
            // The bounds hold for every batch (see the top); the checks keep the writes inside all the same.
            if (j < parts && place < p.max_entries) {
                const int slot = parts > 1 && as + j < p.max_slots ? as + j : -1;
                const int at = (c & 1) ? p.max_entries - 1 - place : place;
                p.entries[(int64_t)(c >> 1) * p.max_entries + at] = ChunkEntry{t, lo, hi - lo, slot, hk};
            }
        }
    }
    __syncthreads();
    if (tid == 0) {
        const int c0 = count[0], c1 = c0 + count[1], c2 = c1 + count[2], c3 = c2 + count[3];
        *p.plan = ChunkPlan{{c0, c1, c2, c3}, n_tiles, min(count[4], p.max_merges), k, 0};
    }
}

// Joins the partial states of the split items. What each entry left per row and map is
// the unnormalised accumulator, the running maximum and the sum; the parts are added
// in the order of their keys, then the combination, the row's RMSNorm and the
// (1 - lambda_init) scale, as in the attention kernels' own epilogues. A kernel of its
// own because one SM takes about 10 us to read the two states of a 128-row item, which
// the last of the item's CTAs would add to its run (measured: 35 us on a batch of 100
// such items); spread over the GPU they are read at the L2's rate.
//
// A block takes 32 rows of an item: lane = row, warp w column quartets 4 w .. 4 w + 3, so that
// every load of a warp is 512 contiguous bytes, as the states were stored. An item of at most 16 rows
// leaves lanes over: they take parts of the keys each, joined by shuffles (16 items of one row in 10 parts:
// 13.5 -> 5.7 us). The order of the additions depends on the numbers of rows and parts alone.
constexpr int kMergeRows = 32;

// Adds the state (M2, l2, o2) of one map to (M, l, o).
__device__ __forceinline__ void add_state(float& M, float& l, float4* o, float M2, float l2, const float4* o2) {
    const float n = fmaxf(M, M2), a = fast_exp2(M - n), b = fast_exp2(M2 - n);
    M = n;
    l = l * a + l2 * b;
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        o[c].x = o[c].x * a + o2[c].x * b;
        o[c].y = o[c].y * a + o2[c].y * b;
        o[c].z = o[c].z * a + o2[c].z * b;
        o[c].w = o[c].w * a + o2[c].w * b;
    }
}

template <int DV>
__global__ void __launch_bounds__(DV * 2) chunk_merge_kernel(const __grid_constant__ ChunkLists lists) {
    const ChunkParams& p = lists.p[blockIdx.y];
    constexpr int CG = DV / 4, WARPS = CG / 4;
    __shared__ float red[WARPS][kMergeRows];
    pdl_trigger();
    pdl_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int blocks = (p.rows + kMergeRows - 1) / kMergeRows, work = p.plan->merges * blocks;
    for (int w = blockIdx.x; w < work; w += gridDim.x) {
        const ChunkMerge g = p.merges[w / blocks];
        const int rows = g.tile.ntok * p.group, r0 = w % blocks * kMergeRows;
        if (r0 >= rows) continue;
        int width = kMergeRows;  // lanes of a group of keys: a power of two
        while (width / 2 >= rows) width /= 2;
        const int row = r0 + lane % width, r = min(row, rows - 1);
        float M[2] = {kChunkNoMax, kChunkNoMax}, l[2] = {0.f, 0.f};
        float4 o[2][4];
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
            for (int c = 0; c < 4; ++c) o[k][c] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 2
        for (int s = lane / width; s < g.count; s += kMergeRows / width) {
            const int64_t item = g.slot + s;
            float2 ml[2];
            float4 v[2][4];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                ml[k] = *reinterpret_cast<const float2*>(p.part_stats + ((item * 2 + k) * p.rows + r) * 2);
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    v[k][c] = *reinterpret_cast<const float4*>(
                        p.part_o + (((item * 2 + k) * CG + warp * 4 + c) * p.rows + r) * 4);
            }
#pragma unroll
            for (int k = 0; k < 2; ++k) add_state(M[k], l[k], o[k], ml[k].x, ml[k].y, v[k]);
        }
        for (int d = width; d < kMergeRows; d *= 2) {  // the same in every lane of the block
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const float M2 = __shfl_xor_sync(0xffffffffu, M[k], d), l2 = __shfl_xor_sync(0xffffffffu, l[k], d);
                float4 v[4];
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    v[c] = make_float4(__shfl_xor_sync(0xffffffffu, o[k][c].x, d), __shfl_xor_sync(0xffffffffu, o[k][c].y, d),
                                       __shfl_xor_sync(0xffffffffu, o[k][c].z, d), __shfl_xor_sync(0xffffffffu, o[k][c].w, d));
                add_state(M[k], l[k], o[k], M2, l2, v);
            }
        }
        // A row that sees no key has l = 0 and gives zeros; a NaN sum stays one.
        const float i1 = l[0] != 0.f ? p.v_scale / l[0] : 0.f, i2 = l[1] != 0.f ? p.lambda * p.v_scale / l[1] : 0.f;
        float x[16], ss = 0.f;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            x[4 * c] = o[0][c].x * i1 - o[1][c].x * i2;
            x[4 * c + 1] = o[0][c].y * i1 - o[1][c].y * i2;
            x[4 * c + 2] = o[0][c].z * i1 - o[1][c].z * i2;
            x[4 * c + 3] = o[0][c].w * i1 - o[1][c].w * i2;
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) ss = fmaf(x[i], x[i], ss);
        __syncthreads();  // the previous round's readers are done
        red[warp][lane] = ss;
        __syncthreads();
        ss = 0.f;
#pragma unroll
        for (int i = 0; i < WARPS; ++i) ss += red[i][lane];
        if (row >= rows || lane >= width) continue;
        const float sc = ss == 0.f ? 0.f : (1.0f - p.lambda_init) / sqrtf(ss / (float)DV + p.eps);
#pragma unroll
        for (int i = 0; i < 16; ++i) x[i] *= p.norm_w ? sc * p.norm_w[warp * 16 + i] : sc;
        const int64_t at = ((int64_t)(g.tile.t0 + r / p.group) * p.H + g.hk * p.group + r % p.group) * DV + warp * 16;
        if (p.out_bf16 || p.out_f16) {
            const bool f16 = p.out_f16 != 0;
            uint4* dst = reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.out) + at);
#pragma unroll
            for (int i = 0; i < 2; ++i)
                dst[i] = make_uint4(pack_16x2(x[8 * i], x[8 * i + 1], f16), pack_16x2(x[8 * i + 2], x[8 * i + 3], f16),
                                    pack_16x2(x[8 * i + 4], x[8 * i + 5], f16), pack_16x2(x[8 * i + 6], x[8 * i + 7], f16));
        } else {
            float4* dst = reinterpret_cast<float4*>(static_cast<float*>(p.out) + at);
#pragma unroll
            for (int i = 0; i < 4; ++i) dst[i] = make_float4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
        }
    }
}

}  // namespace

cudaError_t launch_chunk_plan(const ChunkLists& lists, int n, cudaStream_t stream) {
    return launch_pdl(chunk_plan_kernel, dim3(n), dim3(kPlanThreads), 0, stream, lists);
}

cudaError_t launch_chunk_merge(const ChunkLists& lists, int n, cudaStream_t stream) {
    int sms = 0;
    const cudaError_t e = device_sm_count(&sms);
    if (e != cudaSuccess) return e;
    int64_t most = 0;
    for (int i = 0; i < n; ++i) {
        const ChunkParams& p = lists.p[i];
        const int64_t blocks = (int64_t)p.max_merges * ((p.rows + kMergeRows - 1) / kMergeRows);
        if (blocks > most) most = blocks;
    }
    const dim3 grid((unsigned)(most < 4 * sms ? most : 4 * sms), n);  // one resident round at most
    return lists.p[0].Dv == 128 ? launch_pdl(chunk_merge_kernel<128>, grid, dim3(256), 0, stream, lists)
                                : launch_pdl(chunk_merge_kernel<256>, grid, dim3(512), 0, stream, lists);
}

}  // namespace da
