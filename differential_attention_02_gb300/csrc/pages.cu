// Which pages of a paged cache each sequence holds: a fork of the block table (rows that
// continue others, grow, roll back, start or end), the compaction of the pool, and the
// copies that both ask for.
//
// State: a table [S, M] of page numbers, the tokens of each row, and of each page the
// number of its holders; a page without holders is free. Both planning kernels are one
// block that passes over the table and the counts. Counts change by integer atomics,
// whose order does not matter; free pages are handed out lowest first, to the rows in
// order, so that equal states give equal results.
#include <limits.h>

#include "common.cuh"
#include "kernels.h"

namespace da {
namespace {

constexpr int kPage = 64;
constexpr int kPlanThreads = 1024;

__device__ __forceinline__ int pages_of(int tokens) { return (int)(((int64_t)tokens + kPage - 1) / kPage); }

// Exclusive scan over the block; *total is the sum in every thread.
__device__ __forceinline__ int block_scan(int v, int* shared, int* total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    __syncthreads();  // of an earlier scan's reads
    if (lane == 31) shared[warp] = x;
    __syncthreads();
    int w = shared[lane];  // 32 warps
    int s = w;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, s, o);
        if (lane >= o) s += y;
    }
    *total = __shfl_sync(0xffffffffu, s, 31);
    return __shfl_sync(0xffffffffu, s - w, warp) + x - v;
}

struct Row {  // what becomes of a row
    int parent;  // the row that it continues, or -1
    int kept;    // tokens kept of it
    int tokens;  // tokens after
    int over;    // pages wanted beyond the table's columns
};
__device__ __forceinline__ int row_tokens(const ForkParams& p, int i) {
    return min(max(p.lens[i], 0), (int)min((int64_t)p.M * kPage, (int64_t)INT_MAX));
}
__device__ __forceinline__ Row row_after(const ForkParams& p, int i) {
    const bool done = p.done && p.done[i];
    int parent = i;
    if (p.parents) {
        const int k = p.parents[i];
        parent = k < 0 || k >= p.K ? -1 : i / p.K * p.K + k;
    }
    if (done) parent = -1;
    const int before = parent < 0 ? 0 : row_tokens(p, parent);
    int64_t want = p.new_lens ? p.new_lens[i] : parent < 0 ? 0 : (int64_t)before + p.grow;
    if (done || want < 0) want = 0;
    const int64_t most = min((int64_t)p.M * kPage, (int64_t)INT_MAX);
    Row r;
    r.parent = parent;
    r.over = want > most ? (int)min((want - most + kPage - 1) / kPage, (int64_t)(1 << 18)) : 0;
    r.tokens = (int)min(want, most);
    r.kept = min(before, r.tokens);
    return r;
}

__global__ void __launch_bounds__(kPlanThreads) pages_fork_kernel(const __grid_constant__ ForkParams p, int cols) {
    extern __shared__ int shared[];
    __shared__ int scan[32];
    __shared__ int s_over;
    int* parent = shared;         // [S] each
    int* kept = parent + p.S;
    int* tokens = kept + p.S;
    int* held = tokens + p.S;     // pages of the old row
    int* stage = held + p.S;      // [S][cols]
    const int tid = threadIdx.x;
    if (tid == 0) s_over = 0;
    __syncthreads();
    for (int i = tid; i < p.S; i += kPlanThreads) {
        const Row r = row_after(p, i);
        parent[i] = r.parent;
        kept[i] = r.kept;
        tokens[i] = r.tokens;
        held[i] = pages_of(row_tokens(p, i));
        p.tail[i] = -1;
        if (r.over) atomicAdd(&s_over, r.over);
    }
    for (int i = tid; i < p.P; i += kPlanThreads) p.refs_out[i] = p.refs[i];
    __syncthreads();
    for (int i = tid; i < p.S; i += kPlanThreads) p.lens_out[i] = tokens[i];  // lens may be the same array

    // Columns of all rows through shared memory: the table may be rewritten in place, and the counts
    // follow the pages that rows lose and gain. What a row keeps of itself changes nothing.
    for (int c0 = 0; c0 < p.M; c0 += cols) {
        const int n = min(cols, p.M - c0);
        for (int t = tid; t < p.S * n; t += kPlanThreads) {
            const int i = t / n, c = c0 + t % n;
            const int page = c < held[i] ? p.table[(int64_t)i * p.M + c] : -1;
            stage[t] = page >= 0 && page < p.P ? page : -1;
        }
        __syncthreads();
        for (int t = tid; t < p.S * n; t += kPlanThreads) {
            const int i = t / n, j = t % n, c = c0 + j, from = parent[i], full = kept[i] / kPage;
            const int got = from >= 0 && c < full ? stage[from * n + j] : -1;
            const bool same = from == i && c < full;
            p.table_out[(int64_t)i * p.M + c] = got;
            if (stage[t] >= 0 && !same) atomicAdd(&p.refs_out[stage[t]], -1);
            if (got >= 0 && !same) atomicAdd(&p.refs_out[got], 1);
            if (from >= 0 && c == full && kept[i] % kPage) p.tail[i] = stage[from * n + j];
        }
        __syncthreads();
    }

    // The begun page stays with the first row that has it, if it has no other holder.
    for (int i = tid; i < p.S; i += kPlanThreads)
        if (__ldcg(&p.tail[i]) >= 0) p.claim[__ldcg(&p.tail[i])] = INT_MAX;
    __syncthreads();
    for (int i = tid; i < p.S; i += kPlanThreads)
        if (__ldcg(&p.tail[i]) >= 0) atomicMin(&p.claim[__ldcg(&p.tail[i])], i);
    __syncthreads();
    int base = 0, copies = 0;
    for (int i0 = 0; i0 < p.S; i0 += kPlanThreads) {
        const int i = i0 + tid;
        int need = 0, copy = 0;
        if (i < p.S) {
            const int t = __ldcg(&p.tail[i]), full = kept[i] / kPage;
            const bool stays = t >= 0 && __ldcg(&p.claim[t]) == i && __ldcg(&p.refs_out[t]) <= 0;
            copy = t >= 0 && !stays;
            need = pages_of(tokens[i]) - full - stays;
            p.first[i] = full + stays;
        }
        int total, total_copies;
        const int at = block_scan(need, scan, &total), copy_at = block_scan(copy, scan, &total_copies);
        if (i < p.S) {
            p.prefix[i] = base + at;
            p.copy_at[i] = copy ? copies + copy_at : -1;
        }
        base += total;
        copies += total_copies;
    }
    __syncthreads();  // all claims have seen the counts
    for (int i = tid; i < p.S; i += kPlanThreads) {
        const int full = kept[i] / kPage;
        if (__ldcg(&p.first[i]) > full) {
            const int t = __ldcg(&p.tail[i]);
            p.refs_out[t] = 1;
            p.table_out[(int64_t)i * p.M + full] = t;
        }
    }
    __syncthreads();

    // Free pages, lowest first, to the entries that need one, in the rows' order.
    const int wanted = base;
    int free_pages = 0;
    for (int p0 = 0; p0 < p.P; p0 += kPlanThreads) {
        const int page = p0 + tid;
        const int count = page < p.P ? __ldcg(&p.refs_out[page]) : 1;
        int total;
        const int number = free_pages + block_scan(count <= 0, scan, &total);
        if (count <= 0) {
            if (number < wanted) {
                int lo = 0, hi = p.S - 1;  // the last row whose entries begin at or before `number`
                while (lo < hi) {
                    const int mid = (lo + hi + 1) / 2;
                    if (__ldcg(&p.prefix[mid]) <= number) lo = mid;
                    else hi = mid - 1;
                }
                const int begin = __ldcg(&p.prefix[lo]), first = __ldcg(&p.first[lo]);
                p.table_out[(int64_t)lo * p.M + first + (number - begin)] = page;
                p.refs_out[page] = 1;
                const int at = __ldcg(&p.copy_at[lo]);
                if (number == begin && at >= 0) {
                    p.copies[3 * at] = __ldcg(&p.tail[lo]);
                    p.copies[3 * at + 1] = page;
                    p.copies[3 * at + 2] = kept[lo] % kPage;
                }
            } else if (count < 0) {
                p.refs_out[page] = 0;
            }
        }
        free_pages += total;
    }
    // The copies whose page was found come first, in the rows' order.
    int done = 0;
    for (int i0 = 0; i0 < p.S; i0 += kPlanThreads) {
        const int i = i0 + tid;
        int total;
        block_scan(i < p.S && __ldcg(&p.copy_at[i]) >= 0 && __ldcg(&p.prefix[i]) < free_pages, scan, &total);
        done += total;
    }
    for (int i = done + tid; i < p.S; i += kPlanThreads) p.copies[3 * i] = p.copies[3 * i + 1] = p.copies[3 * i + 2] = -1;
    if (tid == 0) {
        const int given = min(wanted, free_pages);
        p.info[0] = done;
        p.info[1] = wanted - given + s_over;
        p.info[2] = free_pages - given;
        p.info[3] = p.P - (free_pages - given);
    }
}

__global__ void __launch_bounds__(kPlanThreads) pages_compact_kernel(const __grid_constant__ CompactParams p) {
    __shared__ int scan[32];
    const int tid = threadIdx.x;
    int used = 0;
    for (int p0 = 0; p0 < p.P; p0 += kPlanThreads) {
        int total;
        block_scan(p0 + tid < p.P && p.refs[p0 + tid] > 0, scan, &total);
        used += total;
    }
    // The i-th highest held page behind place `used` moves to the i-th lowest free one before it.
    int below = 0, behind = 0;  // held pages before this place; of them behind place `used`
    for (int p0 = 0; p0 < p.P; p0 += kPlanThreads) {
        const int page = p0 + tid;
        const int count = page < p.P ? p.refs[page] : 0;
        const bool held = count > 0;
        int total;
        const int at = below + block_scan(held, scan, &total);
        if (page < p.P) {
            p.refs_out[page] = held ? count : 0;
            p.moved[page] = held ? page : -1;
            if (held && page >= used && used - 1 - at < p.max_copies) p.src[used - 1 - at] = page;
            if (!held && page < used && page - at < p.max_copies) p.dst[page - at] = page;
        }
        below += total;
        block_scan(held && page >= used, scan, &total);
        behind += total;
    }
    __syncthreads();
    const int moves = min(behind, p.max_copies);
    for (int i = tid; i < p.max_copies; i += kPlanThreads) {
        const bool some = i < moves;
        const int src = some ? p.src[i] : -1, dst = some ? p.dst[i] : -1;
        p.copies[3 * i] = src;
        p.copies[3 * i + 1] = dst;
        p.copies[3 * i + 2] = some ? kPage : -1;
        if (some) {
            p.moved[src] = dst;
            p.refs_out[dst] = p.refs_out[src];
            p.refs_out[src] = 0;
        }
    }
    __syncthreads();
    for (int64_t t = tid; t < (int64_t)p.S * p.M; t += kPlanThreads) {
        const int i = (int)(t / p.M), c = (int)(t % p.M);
        const int page = c < pages_of(max(p.lens[i], 0)) ? p.table[t] : -1;
        p.table_out[t] = page >= 0 && page < p.P ? p.moved[page] : -1;
    }
    if (tid == 0) {
        p.info[0] = moves;
        p.info[1] = 0;
        p.info[2] = p.P - used;
        p.info[3] = used;
    }
}

// grid.x: blocks over (copy, head); grid.y: pools.
__global__ void __launch_bounds__(256) pages_copy_kernel(const __grid_constant__ CopyParams p) {
    const CopyPool& pool = p.pool[blockIdx.y];
    const int n = p.count ? min(max(*p.count, 0), p.max_copies) : p.max_copies;
    for (int64_t u = blockIdx.x; u < (int64_t)n * pool.heads; u += gridDim.x) {
        const int64_t i = u / pool.heads;
        const int head = (int)(u % pool.heads);
        const int src = p.copies[3 * i], dst = p.copies[3 * i + 1], rows = min(p.copies[3 * i + 2], kPage);
        if (src < 0 || src >= p.P || dst < 0 || dst >= p.P || src == dst) continue;
        const uint8_t* from = pool.ptr + src * pool.stride_page + head * pool.stride_head;
        uint8_t* to = pool.ptr + dst * pool.stride_page + head * pool.stride_head;
        for (int t = threadIdx.x; t < rows * pool.row_vecs; t += 256) {
            const int64_t at = (t / pool.row_vecs) * pool.stride_row + (t % pool.row_vecs) * 16;
            *reinterpret_cast<uint4*>(to + at) = *reinterpret_cast<const uint4*>(from + at);
        }
    }
}

}  // namespace

cudaError_t launch_pages_fork(const ForkParams& p, cudaStream_t stream) {
    // Rows of 16 bytes in shared memory, and columns for up to 96 KB beside them.
    const int cols = p.S == 0 ? 1 : p.S * 8 > 24576 ? 8 : min(p.M, 24576 / p.S);
    const size_t smem = (size_t)p.S * (16 + 4 * cols);
    cudaError_t e = prepare_once<pages_fork_kernel>(200 * 1024);
    if (e != cudaSuccess) return e;
    pages_fork_kernel<<<1, kPlanThreads, smem, stream>>>(p, cols);
    return cudaGetLastError();
}

cudaError_t launch_pages_compact(const CompactParams& p, cudaStream_t stream) {
    pages_compact_kernel<<<1, kPlanThreads, 0, stream>>>(p);
    return cudaGetLastError();
}

cudaError_t launch_pages_copy(const CopyParams& p, int pools, cudaStream_t stream) {
    int sms = 0;
    cudaError_t e = device_sm_count(&sms);
    if (e != cudaSuccess) return e;
    int heads = 1;
    for (int i = 0; i < pools; ++i) heads = p.pool[i].heads > heads ? p.pool[i].heads : heads;
    const int64_t units = (int64_t)p.max_copies * heads, most = (int64_t)sms * 8;
    const dim3 grid((unsigned)(units < most ? units : most), (unsigned)pools);
    pages_copy_kernel<<<grid, 256, 0, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace da
