// Differential attention of few new tokens over an fp8 paged cache, d = 64 and Dv = 128:
// the entries of the plan (chunk_plan.cu) whose tile has at most 16 rows (tokens x query
// heads of a KV head), as a batch of decoding or verifying sequences has.
//
// In chunk_tcgen05.cu a 128-row tile spends its time on rows that do not exist: the products
// read each K/V tile once per map as their second operand, and 128 threads per map take the
// exponentials of rows that nobody needs. Here the keys are the rows instead,
//   S_m^T = K_m Q_m^T  [128 keys x 16],   O^T += V^T [P_1^T | P_2^T]  [Dv x 32],
// so each tile is read once, V for both maps together, and the softmax has one thread per
// key and map with 16 exponentials. A row's maximum then lies across the threads; it is
// moved as lazily as there (a stale maximum of up to 2^8 costs fp16 nothing), so in most
// steps the warps only vote that none has to move, and take the exponentials meanwhile. A
// step is two key tiles: the hand-overs cost as much as the arithmetic of one.
//
// K goes from the raw tile into tensor memory (the products' first operand), V into shared
// memory as fp16 (chunk_fp8.cuh), by four warps each; K and V have rings and producers of
// their own, and the scores and P V issuers of their own, so that K runs ahead and neither
// waits behind the other. Queries, sums, scales, masks, hidden V rows and the partial
// states are those of chunk_tcgen05.cu.
//
// Measured on 16 sequences x 5 drafted tokens over 8192 keys, 16 query and 8 KV heads (10 rows a
// tile; the bytes take 40 us): 113 us in 128-row tiles; here 104 with the conversion's
// result joined by hand, 84 with the instruction written out, 78 with steps of two tiles and
// rings of their own, 74 with two issuers (69 to 72 with the lists' bounds of api.cu). A
// key tile takes 1,500 cycles, 1.2 times what the
// bytes need on the 128 SMs that have an item; a start takes 8 us, most of it
// instructions fetched for the first time. Slower were the exponentials of 32 rows (94 against 84 us),
// two streams of tiles with accumulators of their own (98), loops over the rows with more code
// than the instruction cache takes (129), the maxima four rows at a time in a loop (76
// against 74).
//
// 20 warps: 0..3 softmax of map 1 and output, 4..7 softmax of map 2, 8 producer of Q and K, 9
// issuer of the scores, 10 producer of V, 11 issuer of P V, 12..15 convert K, 16..19 convert V.
#include <math.h>

#include "chunk_fp8.cuh"
#include "common.cuh"
#include "kernels.h"

namespace da {
namespace {

constexpr int BN = kChunkKeys, D = 64, DV = 128, R = kFewRows;  // a multiple of 16, a lane per row
constexpr int kWarpProducer = 8, kWarpMma = 9, kWarpProducerV = 10, kWarpPv = 11, kWarpK = 12, kWarpV = 16, kThreads = 640;
constexpr float kRescaleThreshold = 8.0f + kWeightShift;  // log2 units over the maximum as it is held (chunk_fp8.cuh)

// Register split (see fwd_tcgen05.cu): 2 x 144 + 3 x 64 = 5 x 96, what the block is launched with.
constexpr int kRegsLaunch = 96, kRegsSoftmax = 144, kRegsOther = 64;
static_assert(2 * kRegsSoftmax + 3 * kRegsOther <= 5 * kRegsLaunch, "register split");

constexpr int kQBytes = R * D * 2, kVBytes = BN * DV * 2, kPBytes = BN * 128;
constexpr int kBoxBytes = 128 * 128;  // [128 rows][64 16-bit values], 128-byte swizzle
constexpr int kRawBytes = 2 * BN * D;  // K1 and K2, or V: e4m3
static_assert(kRawBytes == BN * DV, "one size");
constexpr int kKRaw = 4, kVRaw = 3, kKStages = 4, kStages = 2;  // raw tiles; operand tiles of K (TMEM) and V
constexpr int kOffP = 0, kOffV = 2 * kPBytes, kOffRaw = kOffV + kStages * kVBytes;
constexpr int kOffRawV = kOffRaw + kKRaw * kRawBytes, kOffQ = kOffRawV + kVRaw * kRawBytes, kOffBar = kOffQ + 2 * kQBytes;
// S: two buffers of two tiles of two maps; O; K: four buffers of two maps, a key's 64 fp16 values in 32 columns.
constexpr uint32_t kTmemCols = 512, kColS = 0, kColO = 8 * R, kColK = 10 * R;
static_assert(R == 16 && 10 * R + kKStages * D <= (int)kTmemCols, "TMEM budget");

struct Bars {
    uint64_t q_full, q_ready;
    uint64_t rawk_full[kKRaw], rawk_empty[kKRaw], rawv_full[kVRaw], rawv_empty[kVRaw];
    uint64_t k_full[kKStages], k_empty[kKStages], v_full[2], v_empty[2];
    uint64_t s_full[2], s_empty[2], vote[2], p_full, o_done, drain;
    uint32_t tmem_base;
    int abort, word[2][3];
    ChunkEntry e;
    // Per map and row: the running maximum, the factor of its last move, the score scale, the sum of the weights,
    // the warps' maxima.
    alignas(16) float m[2][R], alpha[2][R], scale[2][R], sum[2][R], most[2][4][R];
};
constexpr size_t kSmem = 1024 + (size_t)kOffBar + sizeof(Bars);
static_assert(kSmem <= 232448, "shared memory budget");

// Order-preserving map of a float to an integer (NaN aside).
__device__ __forceinline__ int float_order(float x) {
    const int b = __float_as_int(x);
    return b ^ ((b >> 31) & 0x7fffffff);
}
__device__ __forceinline__ float order_float(int b) { return __int_as_float(b ^ ((b >> 31) & 0x7fffffff)); }

__global__ void __launch_bounds__(kThreads, 1) chunk_few_kernel(const __grid_constant__ ChunkParams p) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    Bars* bars = reinterpret_cast<Bars*>(smem + kOffBar);
    volatile int* abort_flag = &bars->abort;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        mbar_init(&bars->q_full, 1);
        mbar_init(&bars->q_ready, 2);
        for (int s = 0; s < kKRaw; ++s) {
            mbar_init(&bars->rawk_full[s], 1);
            mbar_init(&bars->rawk_empty[s], 4);
        }
        for (int s = 0; s < kVRaw; ++s) {
            mbar_init(&bars->rawv_full[s], 1);
            mbar_init(&bars->rawv_empty[s], 4);
        }
        for (int s = 0; s < kKStages; ++s) {
            mbar_init(&bars->k_full[s], 4);
            mbar_init(&bars->k_empty[s], 1);
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(&bars->vote[s], 4);
            mbar_init(&bars->v_full[s], 4);
            mbar_init(&bars->v_empty[s], 1);
            mbar_init(&bars->s_full[s], 1);
            mbar_init(&bars->s_empty[s], 8);
        }
        mbar_init(&bars->p_full, 8);
        mbar_init(&bars->o_done, 1);
        mbar_init(&bars->drain, 2);  // the issuers of S and of P V
        bars->abort = 0;
        for (int i = 0; i < 6; ++i) bars->word[i / 3][i % 3] = 0;
        fence_mbarrier_init();
    }
    pdl_trigger();
    pdl_wait();  // the plan, Q and the newest cache rows come from earlier kernels
    const int ei = (int)blockIdx.x;
    ChunkEntry guess{};
    if (threadIdx.x == 0) guess = p.entries[ei];  // the right one in the longest class: one latency instead of two
    const ChunkPlan plan = *p.plan;
    if (ei >= plan.upto[3]) return;  // every thread of the CTA
    if (threadIdx.x == 0) bars->e = ei < plan.upto[0] ? guess : p.entries[chunk_entry(plan.upto, p.max_entries, ei)];
    if (warp == kWarpMma) {
        tmem_alloc(&bars->tmem_base, kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = bars->tmem_base;
    const ChunkEntry& e = bars->e;
    const int nkv = e.nkt, rows = e.tile.ntok * p.group, hk = e.hk;
    const int last = nkv - 1, steps = (nkv + 1) / 2;  // two key tiles a step

    uint8_t* ps = smem + kOffP;
    uint8_t* vs = smem + kOffV;
    uint8_t* qs = smem + kOffQ;

    if (warp >= 8) {
        setmaxnreg_dec<kRegsOther>();
        const int key_end = e.tile.pos0 + e.tile.ntok;          // keys that the tile's last token sees
        const int tail_row = key_end - (e.kt0 + last) * BN;     // first hidden row of the last key tile
        if (warp == kWarpProducer || warp == kWarpProducerV) {
            // ------------------------------------------------------------ producers, of Q and K and of V
            const bool of_k = warp == kWarpProducer;
            if (lane == 0 && nkv > 0) {
                if (of_k) {
                    tma_prefetch_desc(&p.tm_k1);
                    tma_prefetch_desc(&p.tm_k2);
                    mbar_arrive_expect_tx(&bars->q_full, 2 * (uint32_t)p.q_rows * 128u);
                    index_ok(e.tile.t0 >= 0 && e.tile.t0 < p.T && hk < p.H_kv, p.err, 0xC0);
                    tma_load_4d(qs, &p.tm_q1, &bars->q_full, 0, 0, e.tile.t0, hk);
                    tma_load_4d(qs + kQBytes, &p.tm_q2, &bars->q_full, 0, 0, e.tile.t0, hk);
                } else {
                    tma_prefetch_desc(&p.tm_v);
                }
                // Physical pages, read one key tile ahead; num_pages (zeros) where none is needed.
                const int32_t* table = p.block_table + (int64_t)e.tile.b * p.max_pages;
                const int pages = (key_end + 63) / 64;
                auto page_at = [&](int i) -> int {
                    if (i >= pages) return p.num_pages;
                    const int pg = table[i];
                    return index_ok(pg >= 0 && pg < p.num_pages, p.err, 0xC1) ? pg : p.num_pages;
                };
                int next0 = page_at(2 * e.kt0), next1 = page_at(2 * e.kt0 + 1);
                const int ring = of_k ? kKRaw : kVRaw;
                uint64_t* full = of_k ? bars->rawk_full : bars->rawv_full;
                uint64_t* empty = of_k ? bars->rawk_empty : bars->rawv_empty;
                uint8_t* raw = smem + (of_k ? kOffRaw : kOffRawV);
                int j = 0, s = 0;
                uint32_t ph = 1;
                for (; j < nkv; ++j) {
                    const int pg[2] = {next0, next1};
                    if (j + 1 < nkv) {
                        next0 = page_at(2 * (e.kt0 + j + 1));
                        next1 = page_at(2 * (e.kt0 + j + 1) + 1);
                    }
                    if (!mbar_wait(&empty[s], ph, abort_flag, p.err, 0x31)) break;
                    mbar_arrive_expect_tx(&full[s], kRawBytes);
                    uint8_t* st = raw + s * kRawBytes;
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        if (of_k) {
                            tma_load_4d(st + h * 64 * D, &p.tm_k1, &full[s], 0, 0, hk, pg[h]);
                            tma_load_4d(st + BN * D + h * 64 * D, &p.tm_k2, &full[s], 0, 0, hk, pg[h]);
                        } else {
                            tma_load_4d(st + h * 64 * DV, &p.tm_v, &full[s], 0, 0, hk, pg[h]);
                        }
                    }
                    if (++s == ring) {
                        s = 0;
                        ph ^= 1;
                    }
                }
                // Drain: no copy may still be landing in shared memory when the CTA exits.
                if (of_k) mbar_wait(&bars->q_full, 0, nullptr, p.err, 0x32);
                for (int u = max(0, j - ring); u < j; ++u) mbar_wait(&full[u % ring], (u / ring) & 1, nullptr, p.err, 0x33);
            }
        } else if (warp == kWarpMma) {
            // ------------------------------------------------------------ scores, as early as their buffers allow
            const uint32_t id_s = idesc_kind_f16(BN, R, 0, 0, 1);
            const uint64_t dq = sdesc_sw128(smem_u32(qs), 16, 1024);
            bool ok = nkv > 0 && mbar_wait_warp(&bars->q_ready, 0, abort_flag, p.err, 0x34);
            for (int j = 0; ok && j < nkv; ++j) {
                const int i = j >> 1, s = j % kKStages;
                ok = mbar_wait_warp(&bars->k_full[s], (j / kKStages) & 1, abort_flag, p.err, 0x38);
                if ((j & 1) == 0) ok = ok && mbar_wait_warp(&bars->s_empty[i & 1], ((i >> 1) & 1) ^ 1, abort_flag, p.err, 0x36);
                if (!ok) break;
                tc_fence_after();
                if (elect_one()) {
                    const uint32_t tS = tmem + kColS + (i & 1) * 4 * R + (j & 1) * 2 * R;
#pragma unroll
                    for (int m = 0; m < 2; ++m)
#pragma unroll
                        for (int kk = 0; kk < D / 16; ++kk)
                            umma_ts(tS + m * R, tmem + kColK + s * D + m * (D / 2) + kk * 8,
                                    dq + (uint64_t)(m * (kQBytes >> 4) + kk * 2), id_s, kk > 0 ? 1u : 0u);
                    umma_commit(&bars->k_empty[s]);
                    if ((j & 1) || j == last) umma_commit(&bars->s_full[i & 1]);
                }
                __syncwarp();
            }
            // Every MMA issued (also before an abort) must finish before TMEM is freed.
            if (elect_one()) umma_commit(&bars->drain);
            __syncwarp();
            mbar_wait(&bars->drain, 0, nullptr, p.err, 0x39);
        } else if (warp == kWarpPv) {
            // ------------------------------------------------------------ P V
            const uint32_t id_o = idesc_kind_f16(DV, 2 * R, 1, 1, 1);
            const uint64_t dv0 = sdesc_sw128(smem_u32(vs), kBoxBytes, 1024);
            const uint64_t dp = sdesc_sw128(smem_u32(ps), kBoxBytes, 1024);
            bool ok = nkv > 0;
            for (int j = 0; ok && j < nkv; ++j) {
                const int s = j % kStages;
                ok = mbar_wait_warp(&bars->v_full[s], (j / kStages) & 1, abort_flag, p.err, 0x3a);
                if ((j & 1) == 0) ok = ok && mbar_wait_warp(&bars->p_full, (j >> 1) & 1, abort_flag, p.err, 0x3b);
                if (!ok) break;
                tc_fence_after();
                if (elect_one()) {
                    const uint64_t dv = dv0 + (uint64_t)s * (kVBytes >> 4), du = dp + (uint64_t)(j & 1) * (kPBytes >> 4);
#pragma unroll
                    for (int kk = 0; kk < BN / 16; ++kk)
                        umma_ss(tmem + kColO, dv + (uint64_t)(kk * 128), du + (uint64_t)(kk * 128), id_o,
                                j > 0 || kk > 0 ? 1u : 0u);
                    umma_commit(&bars->v_empty[s]);
                    if ((j & 1) || j == last) umma_commit(&bars->o_done);
                }
                __syncwarp();
            }
            if (elect_one()) umma_commit(&bars->drain);
            __syncwarp();
            mbar_wait(&bars->drain, 0, nullptr, p.err, 0x39);
        } else if (warp >= kWarpV) {
            // ------------------------------------------------------------ V: e4m3 -> fp16
            const int ct = (warp - kWarpV) * 32 + lane;
            // Lanes 4..7 of eight take the next row's other box, so that neither the loads nor the
            // swizzled stores of a quarter warp meet in a bank.
            const int in = ct % 16, box = (in / 4 + in / 8) & 1, r0 = 2 * (ct / 16) + ((in / 4) & 1), c = in % 4;
            for (int j = 0; j < nkv; ++j) {
                const int s = j % kStages, rs = j % kVRaw;
                if (!mbar_wait_warp(&bars->rawv_full[rs], (j / kVRaw) & 1, abort_flag, p.err, 0x4a)) break;
                if (!mbar_wait_warp(&bars->v_empty[s], ((j / kStages) & 1) ^ 1, abort_flag, p.err, 0x4b)) break;
                const uint8_t* raw = smem + kOffRawV + rs * kRawBytes;
                uint8_t* v = vs + s * kVBytes;
                const int hidden = j == last ? tail_row : BN;
#pragma unroll 1
                for (int r = r0; r < BN; r += 64)
                    convert4(raw + r * DV + box * 64 + c * 16, 16 * DV, v + box * kBoxBytes, r, 16, c, hidden);
                fence_proxy_async_shared();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(&bars->v_full[s]);
                    mbar_arrive(&bars->rawv_empty[rs]);
                }
            }
        } else if (warp >= kWarpK) {
            // ------------------------------------------------------------ K: e4m3 -> fp16
            // Into TMEM, the operand of a product whose rows they are: thread = key. The 64-byte swizzle
            // of the raw rows keeps a quarter warp's loads on different banks.
            const int r = (warp - kWarpK) * 32 + lane;
            const uint32_t tK = tmem + ((uint32_t)((warp - kWarpK) * 32) << 16) + kColK;
            for (int j = 0; j < nkv; ++j) {
                const int s = j % kKStages;  // of the raw ring too
                static_assert(kKRaw == kKStages, "one stage index");
                const uint32_t ph = (uint32_t)(j / kKStages) & 1;
                if (!mbar_wait_warp(&bars->rawk_full[s], ph, abort_flag, p.err, 0x48)) break;
                if (!mbar_wait_warp(&bars->k_empty[s], ph ^ 1, abort_flag, p.err, 0x49)) break;
                tc_fence_after();
                const uint8_t* raw = smem + kOffRaw + s * kRawBytes + r * D;
#pragma unroll 1
                for (int m = 0; m < 2; ++m) {
                    uint32_t y[32];
#pragma unroll
                    for (int c = 0; c < 4; ++c)
                        e4m3x16_to_f16(*reinterpret_cast<const uint4*>(raw + m * BN * D + ((c ^ ((r >> 1) & 3)) << 4)), y + 8 * c);
                    tmem_st32(tK + s * D + m * (D / 2), y);
                }
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(&bars->k_full[s]);
                    mbar_arrive(&bars->rawk_empty[s]);
                }
            }
        }
    } else {
        setmaxnreg_inc<kRegsSoftmax>();
        // ------------------------------------------------------------ softmax of map m: thread = key of the tile
        // Columns of P and O: 16 map + row.
        const int m = warp >> 2, t = threadIdx.x & 127;
        const uint32_t lane_base = tmem + ((uint32_t)((warp & 3) * 32) << 16);
        const int pos0 = e.tile.pos0;
        const float* scale = bars->scale[m];
        float* mx = bars->m[m];
        bool ok = true;
        if ((warp & 3) == 0) {  // row = lane
            if (lane < R) mx[lane] = kChunkNoMax;
            if (nkv > 0) {
                ok = mbar_wait_warp(&bars->q_full, 0, abort_flag, p.err, 0x46);
                float f = 0.f;  // rows that are not there: scores of 0
                if (ok && lane < rows) f = q_row_to_f16<D>(qs + m * kQBytes, lane) * (m == 0 ? p.scale1_log2 : p.scale2_log2);
                if (lane < R) bars->scale[m][lane] = f;
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars->q_ready);
            }
        }
        named_bar_sync(4, 256);
        float l[R];
#pragma unroll
        for (int i = 0; i < R; ++i) l[i] = 0.f;

        for (int i = 0; i < steps; ++i) {
            ok = ok && mbar_wait_warp(&bars->s_full[i & 1], (i >> 1) & 1, abort_flag, p.err, 0x40);
            tc_fence_after();
            const uint32_t tS = lane_base + kColS + (i & 1) * 4 * R + m * R;
            const int key0 = (e.kt0 + 2 * i) * BN + t;  // the second tile's: 128 further
            const bool single = 2 * i + 1 == nkv;       // the entry has no second tile: every row is before its keys
            int hide[2];                                // rows before the key
#pragma unroll
            for (int u = 0; u < 2; ++u)
                hide[u] = key0 + u * BN > pos0 ? (int)min((int64_t)(key0 + u * BN - pos0) * p.group, (int64_t)R) : 0;
            if (single) hide[1] = R;
            float x[2][R], top = -INFINITY;
#pragma unroll
            for (int u = 0; u < 2; ++u) tmem_ld16(tS + u * 2 * R, reinterpret_cast<uint32_t*>(x[u]));
            tmem_ld_wait();
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const float sc = scale[r], neg = -mx[r];
                x[0][r] = fmaf(x[0][r], sc, neg);
                x[1][r] = fmaf(x[1][r], sc, neg);
            }
            if (__builtin_expect(single || (e.kt0 + 2 * i + 2) * BN - 1 > pos0, 0)) {
#pragma unroll
                for (int u = 0; u < 2; ++u)
#pragma unroll
                    for (int r = 0; r < R; ++r)
                        if (r < hide[u]) x[u][r] = -INFINITY;
            }
#pragma unroll
            for (int r = 0; r < R; ++r) top = fmax3(top, x[0][r], x[1][r]);
            // Does a maximum have to move (1), has a wait run out (2)? One word per step, of three: the
            // word of the step before is cleared behind this step's vote for the step after next.
            const bool bad = !ok || *abort_flag;
            const int say = (__any_sync(0xffffffffu, top > kRescaleThreshold) ? 1 : 0) | (__any_sync(0xffffffffu, bad) ? 2 : 0);
            if (lane == 0) {
                if (say) atomicOr(&bars->word[m][i % 3], say);
                mbar_arrive(&bars->vote[m]);
            }
            // The weights against the maxima as they stand, while the votes come in.
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int r = 0; r < R; ++r) x[u][r] = fast_exp2(x[u][r]);
            // Every warp of the map votes on every step up to the one that ends it, so this wait needs no abort
            // flag; with one, a warp could leave the others alone at the barriers below.
            mbar_wait_warp(&bars->vote[m], i & 1, nullptr, p.err, 0x41);
            const int word = *(volatile int*)&bars->word[m][i % 3];
            if (t == 0) bars->word[m][(i + 2) % 3] = 0;
            if (__builtin_expect(word & 2, 0)) {  // the same decision in every warp of the map
                ok = false;
                break;
            }
            if (__builtin_expect(word, 0)) {
                // Scores again; the maxima over the keys; the sums to the new ones.
#pragma unroll
                for (int u = 0; u < 2; ++u) tmem_ld16(tS + u * 2 * R, reinterpret_cast<uint32_t*>(x[u]));
                tmem_ld_wait();
#pragma unroll
                for (int r = 0; r < R; ++r) {
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        x[u][r] *= scale[r];
                        if (r < hide[u]) x[u][r] = -INFINITY;
                    }
                    const int most = __reduce_max_sync(0xffffffffu, float_order(fmaxf(x[0][r], x[1][r])));
                    if (lane == 0) bars->most[m][warp & 3][r] = order_float(most);
                }
                named_bar_sync(1 + m, 128);
                if (t < R) {
                    const float m0 = mx[t];
                    const float m1 = fmaxf(fmaxf(fmaxf(bars->most[m][0][t], bars->most[m][1][t]),
                                                 fmaxf(bars->most[m][2][t], bars->most[m][3][t])) - kWeightShift, m0);
                    mx[t] = m1;
                    bars->alpha[m][t] = fast_exp2(m0 - m1);
                }
                named_bar_sync(1 + m, 128);
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    x[0][r] = fast_exp2(x[0][r] - mx[r]);
                    x[1][r] = fast_exp2(x[1][r] - mx[r]);
                    l[r] *= bars->alpha[m][r];
                }
            }
            if (i > 0) ok = mbar_wait_warp(&bars->o_done, (i - 1) & 1, abort_flag, p.err, 0x42);  // P is free, O at rest
            if (__builtin_expect(word && i > 0, 0)) {
                tc_fence_after();
                uint32_t o[R];
                tmem_ld16(lane_base + kColO + m * R, o);
                tmem_ld_wait();
#pragma unroll
                for (int r = 0; r < R; ++r) o[r] = __float_as_uint(__uint_as_float(o[r]) * bars->alpha[m][r]);
                tmem_st16(lane_base + kColO + m * R, o);
                tmem_st_wait();
            }
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    uint32_t w[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const int r = h * 8 + 2 * k;
                        l[r] += x[u][r];
                        l[r + 1] += x[u][r + 1];
                        w[k] = pack_f16x2(x[u][r], x[u][r + 1]);
                    }
                    *reinterpret_cast<uint4*>(ps + u * kPBytes + sw128_offset(t, m * 2 + h)) = make_uint4(w[0], w[1], w[2], w[3]);
                }
            tc_fence_before();
            fence_proxy_async_shared();  // before the products read P
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&bars->s_empty[i & 1]);
                mbar_arrive(&bars->p_full);
            }
        }

        // ------------------------------------------------------------ epilogue
        if (ok && nkv > 0) ok = mbar_wait_warp(&bars->o_done, (steps - 1) & 1, abort_flag, p.err, 0x44);
        ok = __all_sync(0xffffffffu, ok && !*abort_flag);
        tc_fence_after();
        // Sums over the keys, through the idle operand tiles: [map][row][129].
        float* scratch = reinterpret_cast<float*>(vs);
        const bool partial = e.slot >= 0;
        const int64_t item = e.slot;
        named_bar_sync(4, 256);  // every warp is past its last P
#pragma unroll
        for (int i = 0; i < R; ++i)
            scratch[(m * R + i) * 129 + t] = l[i];
        named_bar_sync(1 + m, 128);
        {
            const int row = t >> 2, part = t & 3;  // four threads a row
            float sum = 0.f;
            if (row < rows)
#pragma unroll 8
                for (int i = 0; i < 32; ++i) sum += scratch[(m * R + row) * 129 + part * 32 + i];
            sum += __shfl_xor_sync(0xffffffffu, sum, 1);
            sum += __shfl_xor_sync(0xffffffffu, sum, 2);
            if (part == 0 && row < R) {
                bars->sum[m][row] = sum;
                if (partial && ok && row < rows)
                    *reinterpret_cast<float2*>(p.part_stats + ((item * 2 + m) * p.rows + row) * 2) = make_float2(mx[row], sum);
            }
        }
        named_bar_sync(4, 256);
        if (ok) {
            // Thread = column of V. Partial states: each group its own map's; else the first group combines them.
            if (partial || m == 0) {
                uint32_t o[R], o2[R];
                tmem_ld16(lane_base + kColO + m * R, o);
                if (!partial) tmem_ld16(lane_base + kColO + R, o2);
                tmem_ld_wait();
#pragma unroll
                for (int row = 0; row < R; ++row) {
                    if (row >= rows) break;
                    if (partial) {
                        p.part_o[(((item * 2 + m) * (DV / 4) + t / 4) * p.rows + row) * 4 + t % 4] = __uint_as_float(o[row]);
                    } else {
                        const float l1 = bars->sum[0][row], l2 = bars->sum[1][row];
                        // 0 for a row that sees no key, which gives zeros; a NaN sum stays one
                        const float i1 = l1 > 0.f || !(l1 == l1) ? p.v_scale / l1 : 0.f;
                        const float i2 = l2 > 0.f || !(l2 == l2) ? p.lambda * p.v_scale / l2 : 0.f;
                        // without a key tile the accumulators hold another kernel's values
                        scratch[row * 132 + t] = nkv > 0 ? __uint_as_float(o[row]) * i1 - __uint_as_float(o2[row]) * i2 : 0.f;
                    }
                }
            }
        }
        named_bar_sync(4, 256);
        if (!partial && ok) {
            for (int row = warp; row < rows; row += 8) {  // a warp per row, four columns a lane
                const float4 v = *reinterpret_cast<const float4*>(scratch + row * 132 + lane * 4);
                float ss = v.x * v.x + v.y * v.y + v.z * v.z + v.w * v.w;
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
                const float sc = ss == 0.f ? 0.f : (1.0f - p.lambda_init) / sqrtf(ss / (float)DV + p.eps);
                float4 w = make_float4(sc, sc, sc, sc);
                if (p.norm_w) {
                    const float4 gain = *reinterpret_cast<const float4*>(p.norm_w + lane * 4);
                    w = make_float4(sc * gain.x, sc * gain.y, sc * gain.z, sc * gain.w);
                }
                const float4 y = make_float4(v.x * w.x, v.y * w.y, v.z * w.z, v.w * w.w);
                const int64_t at =
                    ((int64_t)(e.tile.t0 + row / p.group) * p.H + hk * p.group + row % p.group) * DV + lane * 4;
                if (p.out_bf16 || p.out_f16) {
                    const bool f16 = p.out_f16 != 0;
                    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.out) + at) =
                        make_uint2(pack_16x2(y.x, y.y, f16), pack_16x2(y.z, y.w, f16));
                } else {
                    *reinterpret_cast<float4*>(static_cast<float*>(p.out) + at) = y;
                }
            }
        }
    }
    tc_fence_before();
    named_bar_sync(3, kThreads);  // every role is done with TMEM and shared memory
    if (warp == kWarpMma) {
        tc_fence_after();
        tmem_dealloc(tmem, kTmemCols);
    }
}

}  // namespace

cudaError_t launch_chunk_few(const ChunkParams& p, cudaStream_t stream) {
    const cudaError_t e = prepare_once<chunk_few_kernel>((int)kSmem, kRegsLaunch);  // the split assumes it
    if (e != cudaSuccess) return e;
    return launch_pdl(chunk_few_kernel, dim3((unsigned)p.max_entries), dim3(kThreads), kSmem, stream, p);
}

}  // namespace da
