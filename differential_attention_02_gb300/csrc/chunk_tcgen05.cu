// Differential attention of ragged new tokens over a paged KV cache, d = 64 and
// Dv = 128, on the 5th-generation tensor cores.
//
// Per query head, token i of a sequence's n new ones stands at position
// p = len - n + i and sees the cache entries 0 .. p (its own among them):
//   O = softmax(Q1 K1^T / sqrt d) V - lambda softmax(Q2 K2^T / sqrt d) V,
// then the head's RMSNorm and the (1 - lambda_init) scale; the mathematics, the two
// running softmax states and their lazily moved maxima are those of fwd_tcgen05.cu.
//
// A CTA works on one entry of the plan (chunk_plan.cu): 128 query rows = tm
// consecutive tokens x the query heads that share one KV head (row r is token
// r / group, head r % group), and a range of 128-key tiles. Packing the heads
// of a group into the rows reads each K/V tile once for all of them and fills the
// 128 MMA rows with few tokens. Rows past the entry's tokens compute on whatever
// follows in Q (rows are independent) and are not stored.
//
// 12 warps: 0..3 softmax of map 1, 4..7 of map 2, 8 TMA producer, 9 MMA issuer,
// 10 clears V rows behind the last visible key, 11 idle. With an fp8 cache 16 warps:
// 12..15 convert (below).
//
// Pages: a key tile is two 64-token pages, each fetched by its own TMA boxes at
// (0, head, page); a page that the tile does not need is asked for behind the pool's
// end, which the copy engine fills with zeros. The cache's bytes behind the last
// visible key are not trusted: scores there are replaced by -inf, and since 0 x NaN
// would still reach the output through P V, the V rows of the last page behind the
// last visible key are cleared in shared memory before that product.
//
// fp8 cache: e4m3 tiles are brought into shared memory raw and a fourth warpgroup
// converts them into the fp16 tiles that the MMAs read; the softmax warps convert the
// query rows once (chunk_fp8.cuh). The K scales go into the maps' score scales, V's into
// the epilogue.
//
// Weights. The operands of a product have one type, so beside a bf16 V the weights are bf16:
// each is off by up to 2^-8 of itself, 1.66e-3 RMS per map, while their sum is fp32 of the
// unrounded ones. On the operators' cases the two maps' difference is off by 2.0e-3 RMS and a
// bf16 output by 2.6e-3, where fp32 weights (the decode kernels) give 1.7e-3; the
// prefill kernels make the same choice. Weights in two bf16 parts would take 320 multiply-adds
// a row, key and map instead of 192, on a tensor pipe that long prompts already keep 52% busy.
//
// Entries that finish their tile store the output; the others leave per row and map
// the unnormalised accumulator, running maximum and sum (columns in quartets, rows
// innermost, so that a warp's 32 rows store 512 contiguous bytes).
#include <math.h>

#include "chunk_fp8.cuh"
#include "common.cuh"
#include "kernels.h"

namespace da {
namespace {

constexpr int BM = kChunkRows, BN = kChunkKeys, D = 64, DV = 128;
constexpr int kWarpProducer = 8, kWarpMma = 9, kWarpTail = 10, kWarpConvert = 12;
constexpr float kRescaleThreshold = 8.0f;  // log2 units

template <bool FP8>
struct Cfg {
    static constexpr int kThreads = (FP8 ? 16 : 12) * 32;
    // Register split (see fwd_tcgen05.cu): the softmax warpgroups' share plus the others' must
    // not exceed what the block was launched with, or setmaxnreg.inc would wait forever.
    static constexpr int kRegsLaunch = FP8 ? 128 : 168;
    static constexpr int kRegsSoftmax = FP8 ? 192 : 208, kRegsOther = FP8 ? 64 : 88;
    static_assert(2 * 128 * kRegsSoftmax + (kThreads - 256) * kRegsOther <= kThreads * kRegsLaunch, "register split");
    static constexpr int kQBytes = BM * D * 2, kKBytes = BN * D * 2, kVBytes = BN * DV * 2;
    static constexpr int kBoxBytes = 128 * 128;   // [128 rows][64 16-bit values], 128-byte swizzle
    static constexpr int kStageBytes = 2 * kKBytes + kVBytes;
    static constexpr int kStages = FP8 ? 2 : 3;    // operand tiles
    static constexpr int kRawStages = FP8 ? 2 : 0; // e4m3 tiles: K1, K2 [128][64 B], V [128][128 B]
    static constexpr int kRawBytes = kStageBytes / 2;
    static constexpr int kOffQ1 = 0, kOffQ2 = kQBytes, kOffStages = 2 * kQBytes;
    static constexpr int kOffRaw = kOffStages + kStages * kStageBytes;
    static constexpr int kOffBar = kOffRaw + kRawStages * kRawBytes;
    static constexpr int kBarBytes = 320;
    static constexpr size_t kSmem = 1024 + (size_t)kOffBar + kBarBytes;
    static_assert(kSmem <= 232448, "shared memory budget");
    static constexpr uint32_t kTmemCols = 512, kColS = 0, kColO = 2 * BN;
    static_assert(2 * BN + 2 * DV <= 512, "TMEM budget");
};

struct Bars {
    uint64_t q_full, q_ready;  // landed; fp8: converted by the softmax warps
    uint64_t kv_full[3], kv_empty[3];            // operand tiles (fp8: K1 and K2 only)
    uint64_t v_full[2], v_empty[2];              // fp8: V tiles
    uint64_t raw_full[2][2], raw_empty[2][2];    // fp8: e4m3 tiles, [stage][K, V]
    uint64_t s_full[2], p_half[2], p_full[2], o_done[2];
    uint64_t tail_full, tail_done;  // V of a last key tile that gets rows cleared: landed, cleared
    uint64_t drain;
    uint32_t tmem_base;
    int abort;
    ChunkEntry e;
};
static_assert(sizeof(Bars) <= Cfg<true>::kBarBytes, "barrier block fits its reserve");

template <bool FP8>
__device__ __forceinline__ void issue_qk(uint32_t s_tmem, uint64_t q_desc, uint64_t k_desc) {
    constexpr uint32_t idesc = idesc_kind_f16(BM, BN, 0, 0, FP8);
#pragma unroll
    for (int kk = 0; kk < D / 16; ++kk)
        umma_ss(s_tmem, q_desc + (uint64_t)(kk * 2), k_desc + (uint64_t)(kk * 2), idesc, kk > 0 ? 1u : 0u);
}

// Half of O (+)= P V: P from TMEM (16 keys per 8 columns), V boxes of [128 keys][64 columns].
template <bool FP8>
__device__ __forceinline__ void issue_pv_half(uint32_t o_tmem, uint32_t p_tmem, uint64_t v_desc, int half, uint32_t acc) {
    constexpr uint32_t idesc = idesc_kind_f16(BM, DV, 0, 1, FP8);
#pragma unroll
    for (int k = 0; k < BN / 32; ++k) {
        const int kk = half * (BN / 32) + k;
        umma_ts(o_tmem, p_tmem + kk * 8, v_desc + (uint64_t)(kk * 128), idesc, (acc || kk > 0) ? 1u : 0u);
    }
}

template <bool FP8>
__global__ void __launch_bounds__(Cfg<FP8>::kThreads, 1) chunk_kernel(const __grid_constant__ ChunkParams p) {
    using C = Cfg<FP8>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    Bars* bars = reinterpret_cast<Bars*>(smem + C::kOffBar);
    float* epi = reinterpret_cast<float*>(smem + C::kOffQ1);  // row exchange, once the Q1 tile is idle
    volatile int* abort_flag = &bars->abort;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        mbar_init(&bars->q_full, 1);
        for (int s = 0; s < C::kStages; ++s) {
            mbar_init(&bars->kv_full[s], FP8 ? 4 : 1);  // fp8: one arrival per converting warp
            mbar_init(&bars->kv_empty[s], 1);
        }
        for (int s = 0; s < C::kRawStages; ++s) {
            mbar_init(&bars->v_full[s], 4);
            mbar_init(&bars->v_empty[s], 1);
            for (int u = 0; u < 2; ++u) {
                mbar_init(&bars->raw_full[s][u], 1);
                mbar_init(&bars->raw_empty[s][u], 4);
            }
        }
        for (int g = 0; g < 2; ++g) {
            mbar_init(&bars->s_full[g], 1);
            if (!FP8) {
                mbar_init(&bars->p_half[g], 4);  // one arrival per softmax warp
                mbar_init(&bars->p_full[g], 4);
            }
            mbar_init(&bars->o_done[g], 1);
        }
        mbar_init(&bars->tail_full, 1);
        mbar_init(&bars->tail_done, 1);
        mbar_init(&bars->drain, 1);
        bars->abort = 0;
        fence_mbarrier_init();
    }
    pdl_trigger();
    pdl_wait();  // the plan, Q and the newest cache rows come from earlier kernels
    const int ei = (int)(blockIdx.x);
    ChunkEntry guess{};
    if (threadIdx.x == 0) guess = p.entries[ei];  // the right one in the longest class: one latency instead of two
    const ChunkPlan plan = *p.plan;
    if (ei >= plan.upto[3]) return;  // every thread of the CTA
    // The entry lives in shared memory, so that the softmax loop keeps its registers for scores.
    if (threadIdx.x == 0) {
        bars->e = ei < plan.upto[0] ? guess : p.entries[chunk_entry(plan.upto, p.max_entries, ei)];
        if constexpr (FP8) {
            // One arrival per softmax warp that has rows of the entry: with few tokens the others stay out
            // and leave the sub-partitions to the conversion (153 -> 144 us for 10 rows a tile; with a bf16
            // cache, where nothing competes with them, it gained nothing).
            const uint32_t warps = (uint32_t)min(4, (bars->e.tile.ntok * p.group + 31) / 32);
            for (int g = 0; g < 2; ++g) {
                mbar_init(&bars->p_half[g], warps);
                mbar_init(&bars->p_full[g], warps);
            }
            mbar_init(&bars->q_ready, 2 * warps);
            fence_mbarrier_init();
        }
    }
    if (warp == kWarpMma) {
        tmem_alloc(&bars->tmem_base, C::kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = bars->tmem_base;
    const ChunkEntry& e = bars->e;

    uint8_t* q1s = smem + C::kOffQ1;
    uint8_t* q2s = smem + C::kOffQ2;
    uint8_t* stages = smem + C::kOffStages;
    const int nkv = e.nkt;

    if (warp >= 8) {
        const int hk = e.hk;
        const int key_end = e.tile.pos0 + e.tile.ntok;      // keys that the tile's last token sees
        const int last = nkv - 1;
        const int tail_row = key_end - (e.kt0 + last) * BN;  // first hidden row of the last key tile
        const bool tail = nkv > 0 && tail_row < BN;
        setmaxnreg_dec<C::kRegsOther>();
        if (warp == kWarpProducer) {
            // ------------------------------------------------------------ producer
            if (lane == 0 && nkv > 0) {
                tma_prefetch_desc(&p.tm_k1);
                tma_prefetch_desc(&p.tm_k2);
                tma_prefetch_desc(&p.tm_v);
                const uint32_t q_bytes = (uint32_t)(p.group * p.tm) * 128u;
                mbar_arrive_expect_tx(&bars->q_full, 2 * q_bytes);
                index_ok(e.tile.t0 >= 0 && e.tile.t0 < p.T && hk < p.H_kv, p.err, 0xC0);
                tma_load_4d(q1s, &p.tm_q1, &bars->q_full, 0, 0, e.tile.t0, hk);
                tma_load_4d(q2s, &p.tm_q2, &bars->q_full, 0, 0, e.tile.t0, hk);
                // Physical pages, read one key tile ahead; num_pages (zeros) where none is needed.
                const int32_t* table = p.block_table + (int64_t)e.tile.b * p.max_pages;
                const int pages = (key_end + 63) / 64;
                auto page_at = [&](int i) -> int {
                    if (i >= pages) return p.num_pages;
                    const int pg = table[i];
                    return index_ok(pg >= 0 && pg < p.num_pages, p.err, 0xC1) ? pg : p.num_pages;
                };
                int next0 = page_at(2 * e.kt0), next1 = page_at(2 * e.kt0 + 1);
                constexpr int kRing = FP8 ? C::kRawStages : C::kStages;
                int j = 0, v = 0;  // tiles of K (bf16: K and V) and of V loaded
                for (; j < nkv; ++j) {
                    const int s = j % kRing;
                    const uint32_t free_ph = ((j / kRing) & 1) ^ 1;
                    const int pg[2] = {next0, next1};
                    if (j + 1 < nkv) {
                        next0 = page_at(2 * (e.kt0 + j + 1));
                        next1 = page_at(2 * (e.kt0 + j + 1) + 1);
                    }
                    if constexpr (FP8) {
                        uint8_t* st = smem + C::kOffRaw + s * C::kRawBytes;
                        if (!mbar_wait(&bars->raw_empty[s][0], free_ph, abort_flag, p.err, 0x31)) break;
                        mbar_arrive_expect_tx(&bars->raw_full[s][0], 2 * BN * D);
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            tma_load_4d(st + h * 64 * D, &p.tm_k1, &bars->raw_full[s][0], 0, 0, hk, pg[h]);
                            tma_load_4d(st + BN * D + h * 64 * D, &p.tm_k2, &bars->raw_full[s][0], 0, 0, hk, pg[h]);
                        }
                        if (!mbar_wait(&bars->raw_empty[s][1], free_ph, abort_flag, p.err, 0x31)) {
                            ++j;  // this tile's K is on its way
                            break;
                        }
                        mbar_arrive_expect_tx(&bars->raw_full[s][1], BN * DV);
#pragma unroll
                        for (int h = 0; h < 2; ++h)
                            tma_load_4d(st + 2 * BN * D + h * 64 * DV, &p.tm_v, &bars->raw_full[s][1], 0, 0, hk, pg[h]);
                        v = j + 1;
                    } else {
                        if (!mbar_wait(&bars->kv_empty[s], free_ph, abort_flag, p.err, 0x31)) break;
                        uint8_t* st = stages + s * C::kStageBytes;
                        // A last tile that gets V rows cleared has a barrier of its own for V: the
                        // clearing warp follows no other phase of the ring.
                        const bool own = tail && j == last;
                        uint64_t* full = &bars->kv_full[s];
                        uint64_t* vfull = own ? &bars->tail_full : full;
                        mbar_arrive_expect_tx(full, own ? 2 * C::kKBytes : C::kStageBytes);
                        if (own) mbar_arrive_expect_tx(vfull, C::kVBytes);
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            tma_load_4d(st + h * 64 * 128, &p.tm_k1, full, 0, 0, hk, pg[h]);
                            tma_load_4d(st + C::kKBytes + h * 64 * 128, &p.tm_k2, full, 0, 0, hk, pg[h]);
                        }
#pragma unroll
                        for (int h = 0; h < 2; ++h)
#pragma unroll
                            for (int x = 0; x < DV / 64; ++x)
                                tma_load_4d(st + 2 * C::kKBytes + x * C::kBoxBytes + h * 64 * 128, &p.tm_v, vfull, x * 64,
                                            0, hk, pg[h]);
                    }
                }
                // Drain: no copy may still be landing in shared memory when the CTA exits.
                mbar_wait(&bars->q_full, 0, nullptr, p.err, 0x32);
                if constexpr (FP8) {
                    for (int u = max(0, j - kRing); u < j; ++u)
                        mbar_wait(&bars->raw_full[u % kRing][0], (u / kRing) & 1, nullptr, p.err, 0x33);
                    for (int u = max(0, v - kRing); u < v; ++u)
                        mbar_wait(&bars->raw_full[u % kRing][1], (u / kRing) & 1, nullptr, p.err, 0x33);
                } else {
                    for (int u = max(0, j - kRing); u < j; ++u)
                        mbar_wait(&bars->kv_full[u % kRing], (u / kRing) & 1, nullptr, p.err, 0x33);
                    if (tail && j == nkv) mbar_wait(&bars->tail_full, 0, nullptr, p.err, 0x33);
                }
            }
        } else if (warp == kWarpMma) {
            // ------------------------------------------------------------ MMA issuer
            const uint32_t tS[2] = {tmem + C::kColS, tmem + C::kColS + BN};
            const uint32_t tO[2] = {tmem + C::kColO, tmem + C::kColO + DV};
            const uint64_t dq[2] = {sdesc_sw128(smem_u32(q1s), 16, 1024), sdesc_sw128(smem_u32(q2s), 16, 1024)};
            const uint64_t dk0 = sdesc_sw128(smem_u32(stages), 16, 1024);
            const uint64_t dv0 = sdesc_sw128(smem_u32(stages) + 2 * C::kKBytes, BN * 128, 1024);
            constexpr uint64_t kStageStep = C::kStageBytes >> 4, kK2Step = C::kKBytes >> 4;
            bool ok = nkv > 0 && mbar_wait_warp(FP8 ? &bars->q_ready : &bars->q_full, 0, abort_flag, p.err, 0x34) &&
                      mbar_wait_warp(&bars->kv_full[0], 0, abort_flag, p.err, 0x35);
            if (ok) {
                tc_fence_after();
                if (elect_one()) {
                    issue_qk<FP8>(tS[0], dq[0], dk0);
                    umma_commit(&bars->s_full[0]);
                    issue_qk<FP8>(tS[1], dq[1], dk0 + kK2Step);
                    umma_commit(&bars->s_full[1]);
                    if (FP8) umma_commit(&bars->kv_empty[0]);
                }
                __syncwarp();
            }
            for (int j = 0; ok && j < nkv; ++j) {
                const int s = j % C::kStages, s1 = (j + 1) % C::kStages;
                const uint64_t dv = dv0 + s * kStageStep, dk1 = dk0 + s1 * kStageStep;
                const bool more = j + 1 < nkv;
                if (!FP8 && j == last && tail && !mbar_wait_warp(&bars->tail_done, 0, abort_flag, p.err, 0x3a)) break;
                if (FP8 && !mbar_wait_warp(&bars->v_full[s], (uint32_t)(j / C::kStages) & 1, abort_flag, p.err, 0x3a)) break;
                // S_m(j+1) follows PV_m(j). With an fp8 cache the next K tiles may still be in conversion: then
                // S_0(j+1) waits behind PV_1(j) rather than PV_1(j) behind it.
                bool s0_late = false;
                for (int m = 0; m < 2; ++m) {
                    if (!mbar_wait_warp(&bars->p_half[m], j & 1, abort_flag, p.err, 0x36 + m)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    if (elect_one()) issue_pv_half<FP8>(tO[m], tS[m], dv, 0, j > 0 ? 1u : 0u);
                    __syncwarp();
                    const uint32_t ph1 = (uint32_t)((j + 1) / C::kStages) & 1;
                    bool next = more;
                    if (!FP8 && m == 0 && more && !mbar_wait_warp(&bars->kv_full[s1], ph1, abort_flag, p.err, 0x38)) {
                        ok = false;
                        break;
                    }
                    if (!mbar_wait_warp(&bars->p_full[m], j & 1, abort_flag, p.err, 0x3b + m)) {
                        ok = false;
                        break;
                    }
                    if (FP8 && m == 0 && more) {
                        next = __all_sync(0xffffffffu, mbar_try_wait(&bars->kv_full[s1], ph1));
                        s0_late = !next;
                    }
                    tc_fence_after();
                    if (elect_one()) {
                        issue_pv_half<FP8>(tO[m], tS[m], dv, 1, 1u);
                        umma_commit(&bars->o_done[m]);
                        if (m == 1) umma_commit(FP8 ? &bars->v_empty[s] : &bars->kv_empty[s]);
                        if (next && !(FP8 && m == 1)) {
                            issue_qk<FP8>(tS[m], dq[m], dk1 + m * kK2Step);
                            umma_commit(&bars->s_full[m]);
                        }
                    }
                    __syncwarp();
                    if (FP8 && m == 1 && more) {
                        if (!mbar_wait_warp(&bars->kv_full[s1], ph1, abort_flag, p.err, 0x38)) {
                            ok = false;
                            break;
                        }
                        tc_fence_after();
                        if (elect_one()) {
                            if (s0_late) {
                                issue_qk<FP8>(tS[0], dq[0], dk1);
                                umma_commit(&bars->s_full[0]);
                            }
                            issue_qk<FP8>(tS[1], dq[1], dk1 + kK2Step);
                            umma_commit(&bars->s_full[1]);
                            umma_commit(&bars->kv_empty[s1]);
                        }
                        __syncwarp();
                    }
                }
            }
            // Every MMA issued (also before an abort) must finish before TMEM is freed.
            if (elect_one()) umma_commit(&bars->drain);
            __syncwarp();
            mbar_wait(&bars->drain, 0, nullptr, p.err, 0x39);
        } else if (!FP8 && warp == kWarpTail && tail) {
            // ------------------------------------------------------------ hidden V rows
            const int s = last % C::kStages;
            if (mbar_wait_warp(&bars->tail_full, 0, abort_flag, p.err, 0x3e)) {
                // Up to the end of the page: a page that was not needed holds zeros.
                const int rows = ((tail_row + 63) & ~63) - tail_row;
                uint8_t* v = stages + s * C::kStageBytes + 2 * C::kKBytes;
                for (int i = lane; i < rows * 8 * (DV / 64); i += 32) {
                    const int x = i / (rows * 8), rest = i % (rows * 8);
                    *reinterpret_cast<uint4*>(v + x * C::kBoxBytes + (tail_row * 8 + rest) * 16) = make_uint4(0, 0, 0, 0);
                }
                fence_proxy_async_shared();  // before the products read them
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars->tail_done);
            }
        } else if (FP8 && warp >= kWarpConvert) {
            // ------------------------------------------------------------ e4m3 -> fp16
            const int cw = warp - kWarpConvert, ct = cw * 32 + lane;
            for (int j = 0; j < nkv; ++j) {
                static_assert(!FP8 || (C::kRawStages == 2 && C::kStages == 2), "one stage index");
                const int s = j % 2;
                const uint32_t ph = (uint32_t)(j / 2) & 1;
                if (!mbar_wait_warp(&bars->raw_full[s][0], ph, abort_flag, p.err, 0x48)) break;
                if (!mbar_wait_warp(&bars->kv_empty[s], ph ^ 1, abort_flag, p.err, 0x49)) break;
                const uint8_t* raw = smem + C::kOffRaw + s * C::kRawBytes;
                uint8_t* st = stages + s * C::kStageBytes;
                // K1, K2 and V in batches of four 16-byte chunks a thread, each batch loaded before the first
                // chunk is stored (the compiler must assume that they overlap), in loops that stay small:
                // three roles share an SM sub-partition's instruction cache. K and V have barriers of their
                // own, so that the next scores do not wait for V nor its conversion for the last products.
                // K: a warp takes 8 rows x 4 chunks.
#pragma unroll 1
                for (int m = 0; m < 2; ++m)
                    convert4(raw + m * BN * D + ct * 16, 128 * 16, st + m * C::kKBytes, ct / 4, 32, ct % 4, BN);
                fence_proxy_async_shared();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(&bars->kv_full[s]);
                    mbar_arrive(&bars->raw_empty[s][0]);
                }
                if (!mbar_wait_warp(&bars->raw_full[s][1], ph, abort_flag, p.err, 0x4a)) break;
                if (!mbar_wait_warp(&bars->v_empty[s], ph ^ 1, abort_flag, p.err, 0x4b)) break;
                // V: lanes 4..7 of eight take the next row's other box, so that neither the loads nor
                // the swizzled stores of a quarter warp meet in a bank.
                const int hidden = j == last ? tail_row : BN;
                const int in = ct % 16, box = (in / 4 + in / 8) & 1, r0 = 2 * (ct / 16) + ((in / 4) & 1), c = in % 4;
#pragma unroll 1
                for (int r = r0; r < BN; r += 64)
                    convert4(raw + 2 * BN * D + r * DV + box * 64 + c * 16, 16 * DV, st + 2 * C::kKBytes + box * C::kBoxBytes,
                             r, 16, c, hidden);
                fence_proxy_async_shared();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(&bars->v_full[s]);
                    mbar_arrive(&bars->raw_empty[s][1]);
                }
            }
        }
        tc_fence_before();
        named_bar_sync(2, C::kThreads);  // every role is done with TMEM and shared memory
        if (warp == kWarpMma) {
            tc_fence_after();
            tmem_dealloc(tmem, C::kTmemCols);
        }
    } else {
        setmaxnreg_inc<C::kRegsSoftmax>();
        // ------------------------------------------------------------ softmax (map g)
        const int g = warp >> 2, lg = warp & 3;
        const int r = lg * 32 + lane;  // query row within the tile == TMEM lane
        const uint32_t lane_base = tmem + ((uint32_t)(lg * 32) << 16);
        const uint32_t tS = lane_base + C::kColS + g * BN;
        const uint32_t tO = lane_base + C::kColO + g * DV;
        // (A bf16 cache has one score scale for both maps: a kernel constant in the loop's FMAs.)
        float sl2 = !FP8 || g == 0 ? p.scale1_log2 : p.scale2_log2;
        const int pos0 = e.tile.pos0, kb0 = e.kt0 * BN;
        const int lim = r < e.tile.ntok * p.group ? pos0 + r / p.group + 1 : 0;  // keys that this row sees
        // fp8: a warp none of whose rows belongs to the entry skips the key tiles. Its rows' weights are
        // whatever the scores' columns hold, and nothing reads their sums.
        const int n_mine = FP8 && lg * 32 >= e.tile.ntok * p.group ? 0 : nkv;
        float m_used = kChunkNoMax, l = 0.f;
        bool ok = true;
        if (FP8 && n_mine > 0) {
            ok = mbar_wait_warp(&bars->q_full, 0, abort_flag, p.err, 0x46);
            if (ok) sl2 = row_score_scale(sl2, q_row_to_f16<D>(g == 0 ? q1s : q2s, r));
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars->q_ready);
        }

        for (int j = 0; ok && j < n_mine; ++j) {
            if (!mbar_wait_warp(&bars->s_full[g], j & 1, abort_flag, p.err, 0x40 + g)) {
                ok = false;
                break;
            }
            tc_fence_after();
            uint32_t sr[BN];
#pragma unroll
            for (int c = 0; c < BN / 32; ++c) tmem_ld32(tS + c * 32, sr + c * 32);
            tmem_ld_wait();
            const int kbase = kb0 + j * BN;
            if (kbase + BN - 1 > pos0) {
#pragma unroll
                for (int i = 0; i < BN; ++i)
                    if (kbase + i >= lim) sr[i] = __float_as_uint(-INFINITY);
            }
            float mx0 = -INFINITY, mx1 = -INFINITY, mx2 = -INFINITY, mx3 = -INFINITY;
#pragma unroll
            for (int i = 0; i < BN; i += 8) {
                mx0 = fmax3(mx0, __uint_as_float(sr[i]), __uint_as_float(sr[i + 1]));
                mx1 = fmax3(mx1, __uint_as_float(sr[i + 2]), __uint_as_float(sr[i + 3]));
                mx2 = fmax3(mx2, __uint_as_float(sr[i + 4]), __uint_as_float(sr[i + 5]));
                mx3 = fmax3(mx3, __uint_as_float(sr[i + 6]), __uint_as_float(sr[i + 7]));
            }
            // The maximum starts at the finite floor kChunkNoMax: a row that has seen no key keeps it,
            // so that its weights are exp2(-inf) = 0, and its first real maximum rescales the empty
            // sums by exp2(floor - max) = 0.
            const float top = fmax3(fmaxf(mx0, mx1), mx2, mx3);
            const float m_new = FP8 ? fmaf(top, sl2, -kWeightShift) : top * sl2;
            float alpha = 1.f;
            bool rescale = false;
            if (m_new > m_used + kRescaleThreshold) {
                alpha = fast_exp2(m_used - m_new);
                m_used = m_new;
                rescale = true;
            }
            if (j > 0 && __any_sync(0xffffffffu, rescale)) {
                if (!mbar_wait_warp(&bars->o_done[g], (j - 1) & 1, abort_flag, p.err, 0x42 + g)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
#pragma unroll 1
                for (int c = 0; c < DV / 32; ++c) {
                    uint32_t o[32];
                    tmem_ld32(tO + c * 32, o);
                    tmem_ld_wait();
#pragma unroll
                    for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
                    tmem_st32(tO + c * 32, o);
                }
            }
            float rs[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
                uint32_t pk[BN / 4];
#pragma unroll
                for (int i = 0; i < BN / 2; i += 2) {
                    const int k = hf * (BN / 2) + i;
                    const float e0 = fast_exp2(fmaf(__uint_as_float(sr[k]), sl2, -m_used));
                    const float e1 = fast_exp2(fmaf(__uint_as_float(sr[k + 1]), sl2, -m_used));
                    rs[(i >> 1) & 3] += e0 + e1;
                    pk[i / 2] = pack_p<FP8>(e0, e1);
                }
                tmem_st32(tS + hf * (BN / 4), pk);
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(hf == 0 ? &bars->p_half[g] : &bars->p_full[g]);
            }
            l = l * alpha + ((rs[0] + rs[1]) + (rs[2] + rs[3]));
        }

        // ------------------------------------------------------------ epilogue
        if (ok && n_mine > 0) {
            ok = mbar_wait_warp(&bars->o_done[0], (nkv - 1) & 1, abort_flag, p.err, 0x44) &&
                 mbar_wait_warp(&bars->o_done[1], (nkv - 1) & 1, abort_flag, p.err, 0x45);
        }
        tc_fence_after();
        const int rows = e.tile.ntok * p.group, hk = e.hk;
        if (e.slot >= 0) {
            // Partial state of map g: this thread's row.
            if (ok) {
                const int64_t item = e.slot;
                float* o = p.part_o + (item * 2 + g) * (DV / 4) * p.rows * 4 + r * 4;
#pragma unroll 1
                for (int c = 0; c < DV / 32; ++c) {
                    uint32_t x[32];
                    tmem_ld32(tO + c * 32, x);
                    tmem_ld_wait();
                    if (r < rows) {
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            *reinterpret_cast<uint4*>(o + (int64_t)(c * 8 + i) * p.rows * 4) =
                                make_uint4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
                    }
                }
                if (r < rows)
                    *reinterpret_cast<float2*>(p.part_stats + ((item * 2 + g) * p.rows + r) * 2) = make_float2(m_used, l);
            }
        } else {
            named_bar_sync(1, 256);  // both groups past their last PV: the Q1 tile is free
            // Weight of map g in the output row; 0 for a row that sees no key, which gives zeros.
            epi[g * BM + r] = l > 0.f || !(l == l) ? (g == 0 ? p.v_scale : p.lambda * p.v_scale) / l : 0.f;
            named_bar_sync(1, 256);
            const float inv1 = epi[r], inv2 = epi[BM + r];
            constexpr int kHalf = DV / 2;  // columns handled by this group
            float oh[kHalf];
            float ss = 0.f;
            const bool mine = lg * 32 < rows;  // a warp without rows has nothing to add up or store
            if (ok && mine) {
#pragma unroll
                for (int c = 0; c < kHalf / 32; ++c) {
                    uint32_t o1[32], o2[32];
                    tmem_ld32(lane_base + C::kColO + g * kHalf + c * 32, o1);
                    tmem_ld32(lane_base + C::kColO + DV + g * kHalf + c * 32, o2);
                    tmem_ld_wait();
#pragma unroll
                    for (int i = 0; i < 32; ++i) {
                        // without a key tile the accumulators hold another kernel's values
                        const float x = nkv > 0 ? __uint_as_float(o1[i]) * inv1 - __uint_as_float(o2[i]) * inv2 : 0.f;
                        oh[c * 32 + i] = x;
                        ss = fmaf(x, x, ss);
                    }
                }
            }
            epi[(2 + g) * BM + r] = ss;
            named_bar_sync(1, 256);
            // Staged as 128-byte-swizzled boxes of 128 rows in the idle operand ring; then whole
            // rows (256 or 512 contiguous bytes) by a warp each, since the tile may end inside
            // the row range of the next sequence.
            uint8_t* stage = stages;
            const bool out16 = p.out_bf16 || p.out_f16;
            if (ok && mine) {
                const float tot = epi[2 * BM + r] + epi[3 * BM + r];
                const float rsc = tot == 0.f ? 0.f : (1.0f - p.lambda_init) / sqrtf(tot / (float)DV + p.eps);
                const float* w = p.norm_w ? p.norm_w + g * kHalf : nullptr;
                if (out16) {
                    const bool f16 = p.out_f16 != 0;
#pragma unroll
                    for (int c = 0; c < 8; ++c) {
                        float y[8];
#pragma unroll
                        for (int i = 0; i < 8; ++i) y[i] = oh[c * 8 + i] * rsc * (w ? w[c * 8 + i] : 1.f);
                        *reinterpret_cast<uint4*>(stage + g * C::kBoxBytes + sw128_offset(r, c)) =
                            make_uint4(pack_16x2(y[0], y[1], f16), pack_16x2(y[2], y[3], f16),
                                       pack_16x2(y[4], y[5], f16), pack_16x2(y[6], y[7], f16));
                    }
                } else {
#pragma unroll
                    for (int bx = 0; bx < 2; ++bx)
#pragma unroll
                        for (int c = 0; c < 8; ++c) {
                            float y[4];
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                const int k = bx * 32 + c * 4 + i;
                                y[i] = oh[k] * rsc * (w ? w[k] : 1.f);
                            }
                            *reinterpret_cast<float4*>(stage + (g * 2 + bx) * C::kBoxBytes + sw128_offset(r, c)) =
                                make_float4(y[0], y[1], y[2], y[3]);
                        }
                }
            }
            named_bar_sync(1, 256);
            if (!*abort_flag) {
                for (int row = warp; row < rows; row += 8) {
                    const int64_t at =
                        ((int64_t)(e.tile.t0 + row / p.group) * p.H + hk * p.group + row % p.group) * DV + lane * 4;
                    if (out16)
                        *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.out) + at) = *reinterpret_cast<const uint2*>(
                            stage + (lane >> 4) * C::kBoxBytes + sw128_offset(row, (lane >> 1) & 7) + (lane & 1) * 8);
                    else
                        *reinterpret_cast<uint4*>(static_cast<float*>(p.out) + at) = *reinterpret_cast<const uint4*>(
                            stage + (lane >> 3) * C::kBoxBytes + sw128_offset(row, lane & 7));
                }
            }
        }
        tc_fence_before();
        named_bar_sync(2, C::kThreads);  // releases the MMA warp to free TMEM
    }
}

template <bool FP8>
cudaError_t launch_t(const ChunkParams& p, cudaStream_t stream) {
    using C = Cfg<FP8>;
    // The register split assumes the compiled per-thread count.
    const cudaError_t e = prepare_once<chunk_kernel<FP8>>((int)C::kSmem, C::kRegsLaunch);
    if (e != cudaSuccess) return e;
    return launch_pdl(chunk_kernel<FP8>, dim3((unsigned)p.max_entries), dim3(C::kThreads), C::kSmem, stream, p);
}

}  // namespace

cudaError_t launch_chunk_64(const ChunkParams& p, cudaStream_t stream) {
    return p.kv_fp8 ? launch_t<true>(p, stream) : launch_t<false>(p, stream);
}

}  // namespace da
