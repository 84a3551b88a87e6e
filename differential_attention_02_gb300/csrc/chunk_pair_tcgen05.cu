// Differential attention of ragged new tokens over a paged KV cache for wide heads
// (d = 128, Dv = 256), on a pair of CTAs (a 2-CTA cluster), tcgen05 MMAs.
//
// The computation, the entries of the plan, the packing of rows, the pages and the
// treatment of bytes behind the last visible key are those of chunk_tcgen05.cu; the
// division of labour is that of fwd_pair_tcgen05.cu, because the two accumulators of
// 256 columns and the scores do not fit one CTA's tensor memory: CTA rank m of the
// pair computes map m alone with a double-buffered score tile, and the epilogue
// forms O1/l1 - lambda O2/l2 across the pair through distributed shared memory.
// An entry that leaves a partial state needs no exchange: each CTA stores its map's.
//
// Warps: 0 TMA producer, 1 MMA issuer, 2..5 softmax and epilogue, then with a bf16
// cache 6 (clears V rows behind the last visible key), with an fp8 cache 6..9, which
// convert e4m3 tiles to fp16 (chunk_fp8.cuh).
//
// fp8 cache: K tiles (two pages) and V half tiles (one page) are 16 KB raw units in
// one ring, loaded and converted in the order in which the MMAs consume them:
// K(0) K(1) V(0a) V(0b) K(2) V(1a) V(1b) K(3) ..; any other order could leave the
// MMA warp waiting for a K tile behind a V tile whose buffer it has not freed yet.
#include <math.h>

#include "chunk_fp8.cuh"
#include "common.cuh"
#include "kernels.h"

namespace da {
namespace {

constexpr int BM = kChunkRows, BN = kChunkKeys, D = 128, DV = 256;
constexpr int kWarpExtra = 6;  // tail (bf16 cache) or the first converting warp (fp8)
constexpr float kRescaleThreshold = 8.0f;  // log2 units

template <bool FP8>
struct Cfg {
    static constexpr int kThreads = (FP8 ? 10 : 7) * 32;
    static constexpr int kQBytes = BM * D * 2, kKBytes = BN * D * 2;
    static constexpr int kVHBytes = BN / 2 * DV * 2;  // half a V tile: one page of 64 keys
    static constexpr int kBoxBytes = 128 * 128;
    static constexpr int kKStages = 2, kVHStages = FP8 ? 2 : 4;
    static constexpr int kRawStages = FP8 ? 4 : 0, kRawBytes = 128 * 128;  // K tile or V page in e4m3
    static constexpr int kOffQ = 0, kOffK = kQBytes, kOffV = kOffK + kKStages * kKBytes;
    static constexpr int kOffRaw = kOffV + kVHStages * kVHBytes;
    static constexpr int kOffBar = kOffRaw + kRawStages * kRawBytes;
    static constexpr int kBarBytes = 320;
    static constexpr size_t kSmem = 1024 + (size_t)kOffBar + kBarBytes;
    static constexpr int kHalf = DV / 2, kXStride = kHalf + 4;
    static constexpr int kOffX = kOffK;  // exchange buffer (peer's part of this CTA's half) in the rings
    static constexpr int kOffSS = kOffX + BM * kXStride * 4;
    static constexpr int kOffOut = kOffK + 96 * 1024;  // output staging behind it: up to 64 KB
    static_assert(kOffOut >= kOffSS + BM * 4 && kOffOut % 1024 == 0, "staging after the exchange buffers");
    static_assert(kOffOut + BM * 128 * (kHalf / 32) <= kOffBar, "fp32 staging fits");
    static_assert(kSmem <= 232448, "shared memory budget");
    static constexpr uint32_t kTmemCols = 512, kColO = 2 * BN;
};

struct Bars {
    uint64_t q_full, q_ready;  // landed; fp8: converted by the softmax warps
    uint64_t k_full[2], k_empty[2];
    uint64_t v_full[4], v_empty[4];
    uint64_t raw_full[4], raw_empty[4];
    uint64_t s_full[2], p_half[2], p_full[2];
    uint64_t o_done, drain;
    uint64_t tail_full, tail_done;  // the half tile that gets V rows cleared: landed, cleared
    uint64_t xsync;  // epilogue rendezvous of the pair: one local and one remote arrival per phase
    uint32_t tmem_base;
    int abort;
};
static_assert(sizeof(Bars) <= 320, "barrier block");

template <bool FP8>
__device__ __forceinline__ void issue_qk(uint32_t s_tmem, uint64_t q_desc, uint64_t k_desc) {
    constexpr uint32_t idesc = idesc_kind_f16(BM, BN, 0, 0, FP8);
#pragma unroll
    for (int kk = 0; kk < D / 16; ++kk) {
        const uint64_t off = (uint64_t)(((kk >> 2) * (128 * 128) + (kk & 3) * 32) >> 4);
        umma_ss(s_tmem, q_desc + off, k_desc + off, idesc, kk > 0 ? 1u : 0u);
    }
}

// O (+)= P V for one half of the keys: V from a half tile, boxes of [64 keys][64 columns].
template <bool FP8>
__device__ __forceinline__ void issue_pv_half(uint32_t o_tmem, uint32_t p_tmem, uint64_t vh_desc, int half, uint32_t acc) {
    constexpr uint32_t idesc = idesc_kind_f16(BM, DV, 0, 1, FP8);
#pragma unroll
    for (int k = 0; k < BN / 32; ++k) {
        const int kk = half * (BN / 32) + k;
        umma_ts(o_tmem, p_tmem + kk * 8, vh_desc + (uint64_t)(k * 128), idesc, (acc || kk > 0) ? 1u : 0u);
    }
}

// Raw units in consumption order. Unit i of an entry with n key tiles: K(0), K(1) (if any),
// then per tile j: V(j a), V(j b), K(j + 2) (if any). Calls k(tile) or v(half tile) until one
// returns false.
template <typename FK, typename FV>
__device__ __forceinline__ void for_units(int n, FK k, FV v) {
    if (n < 1 || !k(0)) return;
    if (n > 1 && !k(1)) return;
    for (int j = 0; j < n; ++j) {
        if (!v(2 * j) || !v(2 * j + 1)) return;
        if (j + 2 < n && !k(j + 2)) return;
    }
}

template <bool FP8>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(Cfg<FP8>::kThreads, 1)
    chunk_pair_kernel(const __grid_constant__ ChunkParams p) {
    using C = Cfg<FP8>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    Bars* bars = reinterpret_cast<Bars*>(smem + C::kOffBar);
    volatile int* abort_flag = &bars->abort;
    const uint32_t rank = cluster_ctarank();  // which map this CTA computes
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const CUtensorMap* tm_q = rank ? &p.tm_q2 : &p.tm_q1;
    const CUtensorMap* tm_k = rank ? &p.tm_k2 : &p.tm_k1;

    if (threadIdx.x == 0) {
        mbar_init(&bars->q_full, 1);
        mbar_init(&bars->q_ready, 4);
        for (int s = 0; s < 2; ++s) {
            mbar_init(&bars->k_full[s], FP8 ? 4 : 1);  // fp8: one arrival per converting warp
            mbar_init(&bars->k_empty[s], 1);
            mbar_init(&bars->s_full[s], 1);
            mbar_init(&bars->p_half[s], 4);  // one arrival per softmax warp
            mbar_init(&bars->p_full[s], 4);
        }
        for (int s = 0; s < 4; ++s) {
            mbar_init(&bars->v_full[s], FP8 ? 4 : 1);
            mbar_init(&bars->v_empty[s], 1);
            mbar_init(&bars->raw_full[s], 1);
            mbar_init(&bars->raw_empty[s], 4);
        }
        mbar_init(&bars->o_done, 1);
        mbar_init(&bars->drain, 1);
        mbar_init(&bars->tail_full, 1);
        mbar_init(&bars->tail_done, 1);
        mbar_init(&bars->xsync, 2);
        bars->abort = 0;
        fence_mbarrier_init();
    }
    // The peer arrives on xsync later, so its initialisation must be visible cluster-wide first.
    cluster_sync_start();
    pdl_trigger();
    pdl_wait();  // the plan, Q and the newest cache rows come from earlier kernels
    const int ei = (int)(blockIdx.x >> 1);
    ChunkEntry e = p.entries[ei];  // the right one in the longest class: one latency instead of two
    const ChunkPlan plan = *p.plan;
    if (ei >= plan.upto[3]) return;  // every thread of both CTAs
    if (ei >= plan.upto[0]) e = p.entries[chunk_entry(plan.upto, p.max_entries, ei)];
    const int hk = e.hk;
    if (warp == 1) {
        tmem_alloc(&bars->tmem_base, C::kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = bars->tmem_base;
    uint8_t* qs = smem + C::kOffQ;
    uint8_t* ks = smem + C::kOffK;
    uint8_t* vs = smem + C::kOffV;
    uint8_t* raws = smem + C::kOffRaw;
    const int nkv = e.nkt, last = nkv - 1;
    const int key_end = e.tile.pos0 + e.tile.ntok;       // keys that the tile's last token sees
    const int tail_row = key_end - (e.kt0 + last) * BN;  // first hidden row of the last key tile
    const int rows = e.tile.ntok * p.group;
    // The half tile (page) in which the visible keys end, if they end inside one.
    const bool tail = nkv > 0 && tail_row < BN && (tail_row & 63) != 0;
    const int tail_half = 2 * last + (tail_row >> 6);

    bool ok = true;
    float l = 0.f, m_used = kChunkNoMax;
    if (warp == 0) {
        // ------------------------------------------------------------ producer
        if (lane == 0 && nkv > 0) {
            tma_prefetch_desc(tm_k);
            tma_prefetch_desc(&p.tm_v);
            const uint32_t q_rows = (uint32_t)(p.group * p.tm);
            mbar_arrive_expect_tx(&bars->q_full, q_rows * D * 2);
            index_ok(e.tile.t0 >= 0 && e.tile.t0 < p.T && hk < p.H_kv, p.err, 0xC2);
#pragma unroll
            for (int x = 0; x < D / 64; ++x)
                tma_load_4d(qs + x * C::kBoxBytes, tm_q, &bars->q_full, x * 64, 0, e.tile.t0, hk);
            const int32_t* table = p.block_table + (int64_t)e.tile.b * p.max_pages;
            const int pages = (key_end + 63) / 64;
            // Physical page i of the sequence; num_pages (zeros) where the tile needs none.
            auto page_at = [&](int i) -> int {
                if (i >= pages) return p.num_pages;
                const int pg = table[i];
                return index_ok(pg >= 0 && pg < p.num_pages, p.err, 0xC3) ? pg : p.num_pages;
            };
            if constexpr (FP8) {
                int n = 0;
                auto unit = [&]() -> uint8_t* {  // the next raw stage, once it is free
                    const int s = n % C::kRawStages;
                    if (!mbar_wait(&bars->raw_empty[s], ((n / C::kRawStages) & 1) ^ 1, abort_flag, p.err, 0x51)) return nullptr;
                    mbar_arrive_expect_tx(&bars->raw_full[s], C::kRawBytes);
                    return raws + s * C::kRawBytes;
                };
                for_units(
                    nkv,
                    [&](int j) {
                        const int p0 = page_at(2 * (e.kt0 + j)), p1 = page_at(2 * (e.kt0 + j) + 1);
                        uint8_t* dst = unit();
                        if (!dst) return false;
                        tma_load_4d(dst, tm_k, &bars->raw_full[n % C::kRawStages], 0, 0, hk, p0);
                        tma_load_4d(dst + 64 * D, tm_k, &bars->raw_full[n % C::kRawStages], 0, 0, hk, p1);
                        ++n;
                        return true;
                    },
                    [&](int u) {
                        const int pg = page_at(2 * e.kt0 + u);
                        uint8_t* dst = unit();
                        if (!dst) return false;
                        tma_load_4d(dst, &p.tm_v, &bars->raw_full[n % C::kRawStages], 0, 0, hk, pg);
                        ++n;
                        return true;
                    });
                mbar_wait(&bars->q_full, 0, nullptr, p.err, 0x53);
                for (int u = max(0, n - C::kRawStages); u < n; ++u)
                    mbar_wait(&bars->raw_full[u % C::kRawStages], (u / C::kRawStages) & 1, nullptr, p.err, 0x53);
            } else {
                int jk = 0, jv = 0;
                bool go = true;
                int next0 = page_at(2 * e.kt0), next1 = page_at(2 * e.kt0 + 1);
                for (int j = 0; go && j < nkv; ++j) {
                    const int pg[2] = {next0, next1};
                    if (j + 1 < nkv) {
                        next0 = page_at(2 * (e.kt0 + j + 1));
                        next1 = page_at(2 * (e.kt0 + j + 1) + 1);
                    }
                    const int sk = j % C::kKStages;
                    go = mbar_wait(&bars->k_empty[sk], ((j / C::kKStages) & 1) ^ 1, abort_flag, p.err, 0x51);
                    if (!go) break;
                    mbar_arrive_expect_tx(&bars->k_full[sk], C::kKBytes);
#pragma unroll
                    for (int x = 0; x < D / 64; ++x)
#pragma unroll
                        for (int h = 0; h < 2; ++h)
                            tma_load_4d(ks + sk * C::kKBytes + x * C::kBoxBytes + h * 64 * 128, tm_k, &bars->k_full[sk],
                                        x * 64, 0, hk, pg[h]);
                    jk = j + 1;
                    for (int h = 0; go && h < 2; ++h) {
                        const int u = 2 * j + h, su = u % C::kVHStages;
                        go = mbar_wait(&bars->v_empty[su], ((u / C::kVHStages) & 1) ^ 1, abort_flag, p.err, 0x52);
                        if (!go) break;
                        // The half tile that gets rows cleared has a barrier of its own: the clearing
                        // warp follows no other phase of the ring.
                        uint64_t* full = tail && u == tail_half ? &bars->tail_full : &bars->v_full[su];
                        mbar_arrive_expect_tx(full, C::kVHBytes);
#pragma unroll
                        for (int x = 0; x < DV / 64; ++x)
                            tma_load_4d(vs + su * C::kVHBytes + x * 64 * 128, &p.tm_v, full, x * 64, 0, hk, pg[h]);
                        jv = u + 1;
                    }
                }
                // Drain: no copy may still be landing in shared memory when the CTA exits.
                mbar_wait(&bars->q_full, 0, nullptr, p.err, 0x53);
                for (int u = max(0, jk - C::kKStages); u < jk; ++u)
                    mbar_wait(&bars->k_full[u % C::kKStages], (u / C::kKStages) & 1, nullptr, p.err, 0x53);
                for (int u = max(0, jv - C::kVHStages); u < jv; ++u) {
                    if (tail && u == tail_half) mbar_wait(&bars->tail_full, 0, nullptr, p.err, 0x53);
                    else mbar_wait(&bars->v_full[u % C::kVHStages], (u / C::kVHStages) & 1, nullptr, p.err, 0x53);
                }
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        // ------------------------------------------------------------ MMA issuer
        const uint32_t tS[2] = {tmem, tmem + BN};
        const uint32_t tO = tmem + C::kColO;
        const uint64_t dq = sdesc_sw128(smem_u32(qs), 16, 1024);
        const uint64_t dk0 = sdesc_sw128(smem_u32(ks), 16, 1024);
        const uint64_t dv0 = sdesc_sw128(smem_u32(vs), (BN / 2) * 128, 1024);
        constexpr uint64_t kKStep = C::kKBytes >> 4, kVHStep = C::kVHBytes >> 4;
        auto issue_s = [&](int j) -> bool {  // S(j) into score buffer j % 2, then K(j) is released
            const int sk = j % C::kKStages;
            if (!mbar_wait_warp(&bars->k_full[sk], (j / C::kKStages) & 1, abort_flag, p.err, 0x55)) return false;
            tc_fence_after();
            if (elect_one()) {
                issue_qk<FP8>(tS[j & 1], dq, dk0 + sk * kKStep);
                umma_commit(&bars->s_full[j & 1]);
                umma_commit(&bars->k_empty[sk]);
            }
            __syncwarp();
            return true;
        };
        bool go = nkv > 0 && mbar_wait_warp(FP8 ? &bars->q_ready : &bars->q_full, 0, abort_flag, p.err, 0x54) && issue_s(0) &&
                  (nkv < 2 || issue_s(1));
        for (int j = 0; go && j < nkv; ++j) {
            const int bf = j & 1;
            for (int h = 0; go && h < 2; ++h) {
                const int u = 2 * j + h, su = u % C::kVHStages;
                go = (!FP8 && tail && u == tail_half
                          ? mbar_wait_warp(&bars->tail_done, 0, abort_flag, p.err, 0x5b)
                          : mbar_wait_warp(&bars->v_full[su], (u / C::kVHStages) & 1, abort_flag, p.err, 0x58)) &&
                     mbar_wait_warp(h == 0 ? &bars->p_half[bf] : &bars->p_full[bf], (j >> 1) & 1, abort_flag, p.err,
                                    0x56 + h);
                if (!go) break;
                tc_fence_after();
                if (elect_one()) {
                    issue_pv_half<FP8>(tO, tS[bf], dv0 + su * kVHStep, h, j > 0 || h > 0 ? 1u : 0u);
                    if (h == 1) umma_commit(&bars->o_done);
                    umma_commit(&bars->v_empty[su]);
                }
                __syncwarp();
            }
            // S(j+2) reuses buffer bf: issued after PV(j), which reads P(j) there.
            if (go && j + 2 < nkv && !issue_s(j + 2)) break;
        }
        // Every MMA issued (also before an abort) must finish before TMEM is freed.
        if (elect_one()) umma_commit(&bars->drain);
        __syncwarp();
        mbar_wait(&bars->drain, 0, nullptr, p.err, 0x59);
        __syncwarp();
    } else if (warp < kWarpExtra) {
        // ------------------------------------------------------------ softmax
        const int lg = warp & 3;
        const int r = lg * 32 + lane;  // query row within the tile == TMEM lane
        const uint32_t lane_base = tmem + ((uint32_t)(lg * 32) << 16);
        const uint32_t tO = lane_base + C::kColO;
        float sl2 = rank ? p.scale2_log2 : p.scale1_log2;
        if (FP8 && nkv > 0) {
            ok = mbar_wait_warp(&bars->q_full, 0, abort_flag, p.err, 0x69);
            if (ok) sl2 = row_score_scale(sl2, q_row_to_f16<D>(qs, r));
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars->q_ready);
        }
        const int lim = r < rows ? e.tile.pos0 + r / p.group + 1 : 0;  // keys that this row sees
        const bool idle = lg * 32 >= rows;  // no row of the warp belongs to the entry: see chunk_tcgen05.cu
        for (int j = 0; ok && j < nkv; ++j) {
            const int bf = j & 1;
            const uint32_t tS = lane_base + bf * BN;
            if (!mbar_wait_warp(&bars->s_full[bf], (j >> 1) & 1, abort_flag, p.err, 0x60)) {
                ok = false;
                break;
            }
            if (idle) {
                if (lane == 0) {
                    mbar_arrive(&bars->p_half[bf]);
                    mbar_arrive(&bars->p_full[bf]);
                }
                continue;
            }
            tc_fence_after();
            uint32_t sr[BN];
#pragma unroll
            for (int c = 0; c < BN / 32; ++c) tmem_ld32(tS + c * 32, sr + c * 32);
            tmem_ld_wait();
            const int kbase = (e.kt0 + j) * BN;
            if (kbase + BN - 1 > e.tile.pos0) {
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
            // kChunkNoMax: see chunk_tcgen05.cu (rows that have seen no key).
            const float top = fmax3(fmaxf(mx0, mx1), mx2, mx3);
            const float m_new = FP8 ? fmaf(top, sl2, -kWeightShift) : top * sl2;
            float alpha = 1.f;
            bool rescale = false;
            if (m_new > m_used + kRescaleThreshold) {
                alpha = fast_exp2(m_used - m_new);
                m_used = m_new;
                rescale = true;
            }
            // S(j) was issued after PV(j-2), so o_done is at most one phase behind.
            if (j > 0 && __any_sync(0xffffffffu, rescale)) {
                if (!mbar_wait_warp(&bars->o_done, (j - 1) & 1, abort_flag, p.err, 0x61)) {
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
                    const int kx = hf * (BN / 2) + i;
                    const float e0 = fast_exp2(fmaf(__uint_as_float(sr[kx]), sl2, -m_used));
                    const float e1 = fast_exp2(fmaf(__uint_as_float(sr[kx + 1]), sl2, -m_used));
                    rs[(i >> 1) & 3] += e0 + e1;
                    pk[i / 2] = pack_p<FP8>(e0, e1);
                }
                tmem_st32(tS + hf * (BN / 4), pk);
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(hf == 0 ? &bars->p_half[bf] : &bars->p_full[bf]);
            }
            l = l * alpha + ((rs[0] + rs[1]) + (rs[2] + rs[3]));
        }
        // S(nkv-1) may land before PV(nkv-2) is done, two phases before the last one: a parity wait
        // tells neighbouring phases apart only, so both are waited for.
        if (ok && nkv > 1) ok = mbar_wait_warp(&bars->o_done, nkv & 1, abort_flag, p.err, 0x62);
        if (ok && nkv > 0) ok = mbar_wait_warp(&bars->o_done, (nkv - 1) & 1, abort_flag, p.err, 0x62);
        tc_fence_after();
    } else if constexpr (!FP8) {
        // ------------------------------------------------------------ hidden V rows
        if (tail) {
            const int su = tail_half % C::kVHStages, row0 = tail_row & 63;
            if (mbar_wait_warp(&bars->tail_full, 0, abort_flag, p.err, 0x5c)) {
                uint8_t* v = vs + su * C::kVHBytes;
                const int n = (64 - row0) * 8;  // 16-byte chunks per box
                for (int i = lane; i < n * (DV / 64); i += 32)
                    *reinterpret_cast<uint4*>(v + (i / n) * 64 * 128 + (row0 * 8 + i % n) * 16) = make_uint4(0, 0, 0, 0);
                fence_proxy_async_shared();  // before the products read them
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars->tail_done);
            }
        }
    } else {
        // ------------------------------------------------------------ e4m3 -> fp16
        const int ct = (warp - kWarpExtra) * 32 + lane;
        int n = 0;
        auto raw_unit = [&]() -> const uint8_t* {
            const int s = n % C::kRawStages;
            if (!mbar_wait_warp(&bars->raw_full[s], (n / C::kRawStages) & 1, abort_flag, p.err, 0x5d)) return nullptr;
            return raws + s * C::kRawBytes;
        };
        auto done = [&](uint64_t* full) {
            fence_proxy_async_shared();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(full);
                mbar_arrive(&bars->raw_empty[n % C::kRawStages]);
            }
            ++n;
        };
        for_units(
            nkv,
            [&](int j) {
                const uint8_t* raw = raw_unit();
                const int s = j % C::kKStages;
                if (!raw || !mbar_wait_warp(&bars->k_empty[s], ((j / C::kKStages) & 1) ^ 1, abort_flag, p.err, 0x5e))
                    return false;
                // [128 rows][128 bytes] -> two boxes of 64 channels. Lanes 4..7 of eight take the next row's
                // other box: neither loads nor swizzled stores of a quarter warp meet in a bank.
                const int in = ct % 16, box = (in / 4 + in / 8) & 1, r0 = 2 * (ct / 16) + ((in / 4) & 1), c = in % 4;
#pragma unroll 1
                for (int r = r0; r < BN; r += 64)
                    convert4(raw + r * D + box * 64 + c * 16, 16 * D, ks + s * C::kKBytes + box * C::kBoxBytes, r, 16, c, BN);
                done(&bars->k_full[s]);
                return true;
            },
            [&](int u) {
                const uint8_t* raw = raw_unit();
                const int su = u % C::kVHStages;
                if (!raw || !mbar_wait_warp(&bars->v_empty[su], ((u / C::kVHStages) & 1) ^ 1, abort_flag, p.err, 0x5f))
                    return false;
                // [64 rows][256 bytes] -> four boxes of 64 columns, with the same lane order per box pair.
                const int hidden = tail && u == tail_half ? (tail_row & 63) : 64;
                const int in = ct % 16, box = 2 * ((ct / 16) & 1) + ((in / 4 + in / 8) & 1);
                const int r0 = 2 * (ct / 32) + ((in / 4) & 1), c = in % 4;
#pragma unroll 1
                for (int r = r0; r < 64; r += 32)
                    convert4(raw + r * DV + box * 64 + c * 16, 8 * DV, vs + su * C::kVHBytes + box * 64 * 128, r, 8, c, hidden);
                done(&bars->v_full[su]);
                return true;
            });
    }

    // ---------------------------------------------------------------- epilogue
    const bool epi = warp >= 2 && warp < kWarpExtra;
    const int lg = warp & 3;
    const int r = lg * 32 + lane;
    const uint32_t tO = tmem + ((uint32_t)(lg * 32) << 16) + C::kColO;
    if (e.slot >= 0) {
        // Partial state of this CTA's map: the thread's row.
        if (epi && ok) {
            const int64_t it = e.slot;
            float* o = p.part_o + (it * 2 + rank) * (DV / 4) * p.rows * 4 + r * 4;
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
                *reinterpret_cast<float2*>(p.part_stats + ((it * 2 + rank) * p.rows + r) * 2) = make_float2(m_used, l);
        }
    } else {
        // Every thread of both CTAs takes part in the three pair_sync calls below. The pair
        // exchanges data by pushing it into the peer's shared memory.
        constexpr int H2 = C::kHalf;
        float* xbuf = reinterpret_cast<float*>(smem + C::kOffX);
        float* ssbuf = reinterpret_cast<float*>(smem + C::kOffSS);
        const uint32_t peer = rank ^ 1u;
        // Weight of this map in the row; 0 for a row that sees no key, which gives zeros.
        const bool seen = nkv > 0 && (l > 0.f || !(l == l));
        const float coef = !seen ? 0.f : (rank == 0) ? p.v_scale / l : -p.lambda * p.v_scale / l;
        const uint32_t own0 = rank * H2, other0 = peer * H2;
        // Without a key tile the accumulator holds another kernel's values.
        auto val = [&](uint32_t bits) { return nkv > 0 ? __uint_as_float(bits) * coef : 0.f; };
        // The exchange buffers live in the K/V rings: both CTAs must be past their last MMA.
        ok = pair_sync(&bars->xsync, peer, 0, abort_flag, p.err, 0x63) && ok;
        ok = __all_sync(0xffffffffu, ok);
        // A warp without rows has nothing to exchange or store (272 items of 1 or 2 rows: 61 -> 51 us).
        const bool mine = epi && lg * 32 < rows;
        if (mine && ok) {
            // The half of this map's row the peer finishes -> the peer's buffer.
            const uint32_t peer_x = mapa_shared(smem_u32(xbuf + r * C::kXStride), peer);
#pragma unroll 1
            for (int c = 0; c < H2 / 32; ++c) {
                uint32_t o[32];
                tmem_ld32(tO + other0 + c * 32, o);
                tmem_ld_wait();
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    st_dsmem_f4(peer_x + (uint32_t)(c * 32 + 4 * i) * 4u,
                                make_float4(val(o[4 * i]), val(o[4 * i + 1]), val(o[4 * i + 2]), val(o[4 * i + 3])));
            }
        }
        ok = pair_sync(&bars->xsync, peer, 1, abort_flag, p.err, 0x64) && ok;
        ok = __all_sync(0xffffffffu, ok);
        const float* xrow = xbuf + r * C::kXStride;
        float ss = 0.f;
        if (mine && ok) {
#pragma unroll 1
            for (int c = 0; c < H2 / 32; ++c) {
                uint32_t o[32];
                tmem_ld32(tO + own0 + c * 32, o);
                tmem_ld_wait();
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float4 q = *reinterpret_cast<const float4*>(xrow + c * 32 + 4 * i);
                    const float x0 = val(o[4 * i]) + q.x, x1 = val(o[4 * i + 1]) + q.y, x2 = val(o[4 * i + 2]) + q.z,
                                x3 = val(o[4 * i + 3]) + q.w;
                    ss = fmaf(x0, x0, fmaf(x1, x1, fmaf(x2, x2, fmaf(x3, x3, ss))));
                }
            }
            st_dsmem_f32(mapa_shared(smem_u32(ssbuf + r), peer), ss);
        }
        ok = pair_sync(&bars->xsync, peer, 2, abort_flag, p.err, 0x65) && ok;
        ok = __all_sync(0xffffffffu, ok && !*abort_flag);
        uint8_t* stage = smem + C::kOffOut;
        const bool out16 = p.out_bf16 || p.out_f16;
        if (mine && ok) {
            const float tot = ss + ssbuf[r];
            const float rsc = tot == 0.f ? 0.f : (1.0f - p.lambda_init) / sqrtf(tot / (float)DV + p.eps);
            const bool f16 = p.out_f16 != 0;
#pragma unroll 1
            for (int c = 0; c < H2 / 32; ++c) {
                uint32_t o[32];
                tmem_ld32(tO + own0 + c * 32, o);
                tmem_ld_wait();
                float y[32];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float4 q = *reinterpret_cast<const float4*>(xrow + c * 32 + 4 * i);
                    y[4 * i] = (val(o[4 * i]) + q.x) * rsc;
                    y[4 * i + 1] = (val(o[4 * i + 1]) + q.y) * rsc;
                    y[4 * i + 2] = (val(o[4 * i + 2]) + q.z) * rsc;
                    y[4 * i + 3] = (val(o[4 * i + 3]) + q.w) * rsc;
                }
                if (p.norm_w) {
#pragma unroll
                    for (int i = 0; i < 32; ++i) y[i] *= p.norm_w[own0 + c * 32 + i];
                }
                if (out16) {
                    uint8_t* box = stage + (c >> 1) * (BM * 128);
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        *reinterpret_cast<uint4*>(box + sw128_offset(r, (c & 1) * 4 + i)) =
                            make_uint4(pack_16x2(y[8 * i], y[8 * i + 1], f16), pack_16x2(y[8 * i + 2], y[8 * i + 3], f16),
                                       pack_16x2(y[8 * i + 4], y[8 * i + 5], f16),
                                       pack_16x2(y[8 * i + 6], y[8 * i + 7], f16));
                } else {
                    uint8_t* box = stage + c * (BM * 128);
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        *reinterpret_cast<float4*>(box + sw128_offset(r, i)) =
                            make_float4(y[4 * i], y[4 * i + 1], y[4 * i + 2], y[4 * i + 3]);
                }
            }
            // The warp's own 32 rows, each half row (256 or 512 contiguous bytes) by the whole warp: the
            // tile may end inside the row range of the next sequence.
            __syncwarp();
            for (int q = lg * 32; q < min(rows, lg * 32 + 32); ++q) {
                const int64_t at =
                    ((int64_t)(e.tile.t0 + q / p.group) * p.H + hk * p.group + q % p.group) * DV + own0 + lane * 4;
                if (out16)
                    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.out) + at) = *reinterpret_cast<const uint2*>(
                        stage + (lane >> 4) * (BM * 128) + sw128_offset(q, (lane >> 1) & 7) + (lane & 1) * 8);
                else
                    *reinterpret_cast<uint4*>(static_cast<float*>(p.out) + at) = *reinterpret_cast<const uint4*>(
                        stage + (lane >> 3) * (BM * 128) + sw128_offset(q, lane & 7));
            }
        }
        // No remote access follows the third rendezvous, so either CTA may exit.
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, C::kTmemCols);
    }
}

template <bool FP8>
cudaError_t launch_t(const ChunkParams& p, cudaStream_t stream) {
    using C = Cfg<FP8>;
    const cudaError_t e = prepare_once<chunk_pair_kernel<FP8>>((int)C::kSmem);
    if (e != cudaSuccess) return e;
    return launch_pdl(chunk_pair_kernel<FP8>, dim3((unsigned)(2 * p.max_entries)), dim3(C::kThreads), C::kSmem,
                      stream, p);
}

}  // namespace

cudaError_t launch_chunk_pair(const ChunkParams& p, cudaStream_t stream) {
    return p.kv_fp8 ? launch_t<true>(p, stream) : launch_t<false>(p, stream);
}

}  // namespace da
