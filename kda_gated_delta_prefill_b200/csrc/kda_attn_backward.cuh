// kda_attn_backward.cuh -- gradients of causal softmax attention, on the
// 5th-generation tensor cores.
//
// With P_ij = exp(s_ij - lse_i) and delta_i = o_i . do_i (= sum_j P_ij dP_ij):
//   dV_j = sum_i P_ij do_i          dP_ij = do_i . v_j          dS_ij = P_ij (dP_ij - delta_i)
//   dQ_i = scale sum_j dS_ij k_j    dK_j = scale sum_i dS_ij q_i
// dK and dV of a shared key/value head are sums over its query heads.
//
// Three launches: the statistics (delta, and lse in units of log 2, in tiles of 128 rows), dQ, and dK/dV.  dK/dV walks
// the queries for a tile of keys and dQ the keys for a tile of queries, so every sum has one owner and a fixed
// order: no atomics, the same bits every time.  The price is that S and dP are formed twice (7 matrix products
// instead of 5).
//
// Precision.  P and dS are rounded to bf16 for the products (2^-9 relative).  o . do inherits the rounding of o and of the
// P that formed it, and where one key has most of a row's probability, dP_ij - delta_i is a small difference of it: dQ and
// dK would be 2e-2 to 1.1 (of the 2-norm) off for probabilities of 0.96 to 0.9998.  But sum_j dS_ij is zero, so what dQ finds
// it to be is delta's error.  dQ leaves the corrected delta for dK/dV, and corrects itself by taking the sum out at the key
// whose P_ij is above 1/2 (at most one; without one, delta's error counts for little).  Rows that see at most 16 keys get
// delta in fp32 from its definition (statistics, below).  dQ and dK are 2.4e-3 off for scores of unit variance and 2e-3 to
// 5e-3 for those rows (1.7e-3 is bf16 results alone).  It costs 5 % (D = 128) and 8 % (D = 64) of the dQ kernel, and dQ has
// to come first, where behind dK/dV it filled the SMs that the last key tiles leave idle: 2,675 -> 2,802 us for 16,384
// tokens of 16/4 heads, 709 -> 760 for 8,192, 125 -> 150 for 2,048 of 32/8.
//
// dK/dV works on the transposes: a thread owns a key row of S^T = K Q^T and dP^T = V dO^T, so P^T and dS^T go back to
// TMEM in bf16 and are the A operands of dV += P^T dO and dK += dS^T Q; only Q and dO tiles move through shared memory.
// TMEM (D = 128): S^T/P^T, dP^T/dS^T, dV, dK with 128 columns each.  The order of the MMAs,
//   dV(i), S^T(i+1), dK(i), dP^T(i+1), dV(i+1), ...
// leaves two products' time for each of P (between S^T and dV) and dS (between dP^T and dK).  At D = 64, where P and dS
// have columns of their own, S^T of the next tile does not wait for dV, and one issuing warp was what everything waited
// for (a wait costs it 120 cycles and an MMA 40): two warps issue, S^T and dV the one, dP^T and dK the other, so every
// sum still has one order (8,192 tokens, 16/16 heads: 327 -> 291 us).  At D = 128 that is slower (1,600 -> 1,750 us for
// 16,384 tokens of 16/4 heads): dP and dK come between dV and S, which are the longest chain.
//
// The launches depend on one another on the device only as far as they have to: each is set up while the one before it
// ends.  Where key tiles are few, a cluster of CTAs shares the heads of a group and adds up over distributed shared memory,
// in the CTAs' order.
#pragma once
#include "kda_attn_common.cuh"

namespace kda {

struct AttnBwdParams {
    SeqView seq;
    int H, HKV, qslots;  // slots of 128 rows of q
    int split;           // CTAs (a cluster) that share a key tile's query heads
    float scale, scale_log2;
    const __nv_bfloat16 *q, *k, *v, *o, *dout;
    int64_t q_stride, k_stride, v_stride, do_stride;
    const float *lse;
    float *stats;  // [H][qslots][2][128]: -lse * log2(e) (-inf: no probability), -delta
    __nv_bfloat16 *dq, *dk, *dv;
    unsigned *err;
};

// ---------------------------------------------------------------------------------------------------- statistics
// A warp for two or four rows: bound by reading o and dout once.
//
// Rows that see few keys get delta from its definition, sum_j P_ij dP_ij in fp32: there P is large and dP_ij - delta_i
// a small difference of two numbers, for which o . do with its rounded o is too coarse (sequences of two tokens: dQ
// 2.7e-2 off, 2.5e-3 so).  They are the first 16 of a sequence's rows that see any; CTAs of their own take them, a
// thread for each row and key (in the tiles' CTAs, behind the other rows, they cost 4 us of a 52 us backward).
constexpr int kAttnStatThreads = 256, kAttnExactKeys = 16;
// Eight products of bf16 values, summed.
__device__ __forceinline__ float dot8(uint4 a, uint4 b)
{
    const uint32_t x[4] = {a.x, a.y, a.z, a.w}, y[4] = {b.x, b.y, b.z, b.w};
    float s = 0.f;
#pragma unroll
    for (int e = 0; e < 4; ++e) s += bf16lo(x[e]) * bf16lo(y[e]) + bf16hi(x[e]) * bf16hi(y[e]);
    return s;
}
// -lse * log2(e) of a row; -inf where it has no probability.
__device__ __forceinline__ float neg_lse(const AttnBwdParams &p, int n, int h, const Seq &sq, int row)
{
    const int64_t at = p.seq.cu_q ? static_cast<int64_t>(h) * p.seq.T + sq.q0 + row
                                  : (static_cast<int64_t>(n) * p.H + h) * p.seq.T + row;
    return p.lse[at] == -INFINITY ? -INFINITY : -p.lse[at] * kLog2e;
}
template <int D>
__device__ __forceinline__ void attn_exact_delta(const AttnBwdParams &p, int n, int h)
{
    static_assert(kAttnStatThreads == kAttnExactKeys * kAttnExactKeys, "a thread for each row and key");
    const Seq sq = seq_of(p.seq, n);
    const int diff = sq.lk - sq.lq;  // row i sees i + 1 + diff keys
    const int row = max(0, -diff) + threadIdx.x / kAttnExactKeys, key = threadIdx.x % kAttnExactKeys;
    const bool mine = row < min(sq.lq, kAttnExactKeys - diff);
    const int hk = h / (p.H / p.HKV);
    float x = 0.f;
    if (mine && key <= row + diff) {
        const int64_t i = static_cast<int64_t>(sq.q0) + row, j = static_cast<int64_t>(sq.k0) + key;
        const uint4 *q = reinterpret_cast<const uint4 *>(p.q + i * p.q_stride + h * D),
                    *g = reinterpret_cast<const uint4 *>(p.dout + i * p.do_stride + h * D),
                    *k = reinterpret_cast<const uint4 *>(p.k + j * p.k_stride + hk * D),
                    *v = reinterpret_cast<const uint4 *>(p.v + j * p.v_stride + hk * D);
        float s = 0.f, dp = 0.f;
#pragma unroll 2
        for (int d = 0; d < D / 8; ++d) {
            s += dot8(q[d], k[d]);
            dp += dot8(g[d], v[d]);
        }
        x = ex2(fmaf(s, p.scale_log2, neg_lse(p, n, h, sq, row))) * dp;
    }
#pragma unroll
    for (int off = kAttnExactKeys / 2; off > 0; off >>= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
    const int slot = (p.seq.cu_q ? sq.q0 / AT + n : n * ((sq.lq + AT - 1) / AT)) + row / AT;
    if (mine && key == 0) p.stats[(static_cast<int64_t>(h) * p.qslots + slot) * (2 * AT) + AT + row % AT] = -x;
}
// CTAs: of each head, the sequences (rows that see few keys), then the tiles.  32 registers, so that eight of them fit an
// SM and keep enough loads in flight (40 registers: 33 us instead of 29 for 16,384 tokens and 16 heads).
template <int D>
__global__ void __launch_bounds__(kAttnStatThreads, 8) kda_attn_stats_kernel(const AttnBwdParams p)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int h = blockIdx.x % p.H, slot = blockIdx.x / p.H - p.seq.N;
    asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
    if (slot < 0) {
        attn_exact_delta<D>(p, slot + p.seq.N, h);
        return;
    }
    int n, blk;
    if (!find_block<AT>(p.seq.cu_q, p.seq.N, p.seq.T, slot, lane, n, blk)) return;
    const Seq sq = seq_of(p.seq, n);
    const int few = kAttnExactKeys - (sq.lk - sq.lq);  // rows before it that see a key are left to the others
    float *out = p.stats + (static_cast<int64_t>(h) * p.qslots + slot) * (2 * AT);
    constexpr int R = AT / (kAttnStatThreads / 32);
    constexpr int LPR = D / 8, RPW = 32 / LPR;  // lanes of a row, rows of a warp at a time
    for (int i = 0; i < R; i += RPW) {
        const int r = warp * R + i + lane / LPR, row = blk * AT + r;
        float s = 0.f;
        if (row < sq.lq)
            s = dot8(*reinterpret_cast<const uint4 *>(p.o + ((static_cast<int64_t>(sq.q0) + row) * p.H + h) * D +
                                                      8 * (lane % LPR)),
                     *reinterpret_cast<const uint4 *>(p.dout + (static_cast<int64_t>(sq.q0) + row) * p.do_stride +
                                                      h * D + 8 * (lane % LPR)));
#pragma unroll
        for (int off = LPR / 2; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
        if (lane % LPR == 0) {
            out[r] = row < sq.lq ? neg_lse(p, n, h, sq, row) : -INFINITY;
            if (row >= min(few, sq.lq) || row < sq.lq - sq.lk) out[AT + r] = -s;
        }
    }
}

// ---------------------------------------------------------------------------------------------------- dK and dV
template <int D>
struct AttnDkvSmem {
    static constexpr int TILE = AT * D * 2;
    static constexpr int NST = D == 128 ? 2 : 4;
    static constexpr int Q = 2 * TILE;              // K, V, then the rings of Q, dO and statistics
    static constexpr int DO = Q + NST * TILE;
    static constexpr int STAT = DO + NST * TILE;
    // qfull qempty dofull doempty [NST], kfull vfull sfull pready dpfull dsready done sfree dpfree
    static constexpr int BAR = STAT + NST * 1024;
    static constexpr int TMEM_SLOT = BAR + (4 * NST + 9) * 8;
    static constexpr int ABORT = TMEM_SLOT + 4;
    static constexpr int TOTAL = ABORT + 4;
};
// 16 warps of arithmetic (a quarter of the rows, 32 columns each), then two of MMAs and one of loads: five warpgroups
// for the register split (512 * 104 + 128 * 64 = 640 * 96).  With 8 warps of 64 columns, two on a scheduler and both in
// the same step, most cycles issued nothing: 133 -> 124 us for 2,048 tokens of 32/8 heads, 246 -> 229 for 4,096 of
// 16/4.  The statistics of the 32 columns are read from shared memory ahead of the scores and of dP, not behind them
// (the MMAs take most of its bandwidth): with them stored negated and masks set in a branch of their own, 134 -> 127 us
// and 173 -> 166 us (4,096 tokens, 16/16 heads, D = 64).
constexpr int kAttnBwdWarps = 16, kAttnBwdThreads = 32 * (kAttnBwdWarps + 4);
constexpr int kAttnBwdMma = kAttnBwdWarps, kAttnBwdLoad = kAttnBwdWarps + 2;  // two warps issue MMAs
#define ATTN_BWD_MORE_REGISTERS() asm volatile("setmaxnreg.inc.sync.aligned.u32 104;\n")
#define ATTN_BWD_FEWER_REGISTERS() asm volatile("setmaxnreg.dec.sync.aligned.u32 64;\n")

template <int D>
__global__ void __launch_bounds__(kAttnBwdThreads, 1)
    kda_attn_dkv_kernel(const AttnBwdParams p, const __grid_constant__ CUtensorMap mq,
                        const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv,
                        const __grid_constant__ CUtensorMap mdo)
{
    using S = AttnDkvSmem<D>;
    constexpr int NST = S::NST, TILE = S::TILE, HALVES = D / 64;
    constexpr bool kOwn = D == 64;           // P and dS have columns of their own
    constexpr int kIssuers = kOwn ? 2 : 1;  // warps that issue MMAs
    constexpr uint32_t TM_S = 0, TM_DP = 128, TM_DV = 256, TM_DK = 256 + D, TM_COLS = 512;
    constexpr uint32_t TM_P = kOwn ? 384 : TM_S, TM_DS = kOwn ? 448 : TM_DP, TM_GROUP = kOwn ? 16 : 32;  // 32 queries
    extern __shared__ __align__(1024) uint8_t sm[];
    const uint32_t sb = smem_u32(sm);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int rank = blockIdx.x % p.split, unit = blockIdx.x / p.split;
    const int hk = unit % p.HKV, G = p.H / p.HKV / p.split, head0 = (hk * p.split + rank) * G;
    int n, blk;
    if (!pick_block<AT, false>(p.seq.cu_k, p.seq.N, p.seq.Tk, unit / p.HKV, lane, n, blk)) {
        // (where no sequence has a key, all CTAs leave here: what follows in the stream waits for this launch only)
        asm volatile("griddepcontrol.wait;\n" ::: "memory");
        return;
    }
    const Seq sq = seq_of(p.seq, n);
    const int diff = sq.lk - sq.lq, j0 = blk * AT;
    // query tiles that see a key of this tile: first .. nq - 1 of each of this CTA's heads
    const int nq = (sq.lq + AT - 1) / AT, first = j0 > diff ? (j0 - diff) / AT : 0;
    const int cnt = max(nq - first, 0), total = cnt * G;
    const int qslot0 = p.seq.cu_q ? sq.q0 / AT + n : n * nq;  // the sequence's first slot of statistics

    const uint32_t qfull = sb + S::BAR, qempty = qfull + 8 * NST, dofull = qempty + 8 * NST, doempty = dofull + 8 * NST,
                   kfull = doempty + 8 * NST, vfull = kfull + 8, sfull = kfull + 16, pready = kfull + 24,
                   dpfull = kfull + 32, dsready = kfull + 40, done = kfull + 48, sfree = kfull + 56, dpfree = kfull + 64;
    volatile int *abort_flag = reinterpret_cast<volatile int *>(sm + S::ABORT);
    if (tid == 0) {
        for (int s = 0; s < 3 * NST; ++s) mbar_init(qfull + 8 * s, 1);
        for (int s = 0; s < NST; ++s) mbar_init(doempty + 8 * s, kIssuers);  // dP and dV are done with the tile
        for (uint32_t b : {kfull, vfull, sfull, dpfull}) mbar_init(b, 1);
        mbar_init(done, kIssuers);
        for (uint32_t b : {pready, dsready, sfree, dpfree}) mbar_init(b, kAttnBwdWarps);
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == kAttnBwdMma) tc_alloc(sb + S::TMEM_SLOT, TM_COLS);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t *>(sm + S::TMEM_SLOT);
    auto fail = [&](unsigned code) {
        atomicOr(p.err, code);
        *abort_flag = 1;
    };

    if (warp < kAttnBwdWarps) {
        // ---------------- P^T and dS^T: key row, 32 of the query columns ----------------
        ATTN_BWD_MORE_REGISTERS();
        const int group = warp >> 2, quarter = warp & 3;
        const uint32_t lb = static_cast<uint32_t>(32 * quarter) << 16;
        const uint32_t ts = tmem + lb + TM_S + 32 * group, td = tmem + lb + TM_DP + 32 * group;
        const uint32_t tp = tmem + lb + TM_P + TM_GROUP * group, tds = tmem + lb + TM_DS + TM_GROUP * group;
        auto arrive = [&](uint32_t bar) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar);
        };
        // the MMAs of iteration it - 1 that read P (or dS) are done with it
        auto reusable = [&](uint32_t bars, int it) {
            if (!kOwn || it == 0) return true;
            return __all_sync(0xffffffffu, mbar_wait_quiet(bars + 8 * ((it - 1) % NST), ((it - 1) / NST) & 1)) != 0;
        };
        const int key = j0 + 32 * quarter + lane;
        const float c = p.scale_log2;
        bool ok = true;
        // queries q >= key - diff see the key; counted from this warp's first column of tile i
        const int seen = key - diff - 32 * group;
        for (int it = 0, i = first; it < total; ++it, i = i + 1 == nq ? first : i + 1) {
            const int st = it % NST;
            ok = __all_sync(0xffffffffu, mbar_wait_quiet(qfull + 8 * st, (it / NST) & 1));
            if (!ok) break;
            const float4 *stat = reinterpret_cast<const float4 *>(sm + S::STAT + st * 1024) + 8 * group;
            float4 l[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) l[e] = stat[e];
            ok = __all_sync(0xffffffffu, mbar_wait_quiet(sfull, it & 1));
            if (!ok) break;
            tc_fence_after();
            uint32_t r[32];
            tc_ld32(ts, r);
            tc_wait_ld();
            if (kOwn) arrive(sfree);
            const int from = seen - i * AT;
            if (__any_sync(0xffffffffu, from > 0)) {
#pragma unroll
                for (int e = 0; e < 32; ++e)
                    if (e < from) r[e] = 0xff800000u;  // -inf
            }
            float2 pr[16];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const uint32_t *x = &r[4 * e];
                const float2 a = fma2(make_float2(__uint_as_float(x[0]), __uint_as_float(x[1])), make_float2(c, c),
                                      make_float2(l[e].x, l[e].y));
                const float2 b = fma2(make_float2(__uint_as_float(x[2]), __uint_as_float(x[3])), make_float2(c, c),
                                      make_float2(l[e].z, l[e].w));
                pr[2 * e] = make_float2(ex2_ftz(a.x), ex2_ftz(a.y));
                pr[2 * e + 1] = make_float2(ex2_ftz(b.x), ex2_ftz(b.y));
            }
            ok = reusable(doempty, it);
            if (!ok) break;
            uint32_t w[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) w[e] = pack_bf16(pr[e].x, pr[e].y);
            tc_st16(tp, w);
            tc_wait_st();
            arrive(pready);

#pragma unroll
            for (int e = 0; e < 8; ++e) l[e] = stat[32 + e];
            ok = __all_sync(0xffffffffu, mbar_wait_quiet(dpfull, it & 1));
            if (!ok) break;
            tc_fence_after();
            // (in halves: fewer registers)
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                uint32_t x[16];
                tc_ld16(td + 16 * half, x);
                tc_wait_ld();
                if (half == 1) {
                    if (kOwn) arrive(dpfree);
                    ok = reusable(qempty, it);
                }
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float4 d4 = l[4 * half + e / 2];
                    const float2 a = mul2(pr[8 * half + e],
                                          add2(make_float2(__uint_as_float(x[2 * e]), __uint_as_float(x[2 * e + 1])),
                                               e & 1 ? make_float2(d4.z, d4.w) : make_float2(d4.x, d4.y)));
                    w[8 * half + e] = pack_bf16(a.x, a.y);
                }
            }
            if (!ok) break;
            tc_st16(tds, w);
            tc_wait_st();
            arrive(dsready);
        }
        if (ok && total > 0) ok = __all_sync(0xffffffffu, mbar_wait_quiet(done, 0));
        if (!ok) {
            if (lane == 0) fail(ERR_PIPE_FULL_WAIT);
        } else if (p.split > 1 && total > 0) {
            // this CTA's sums over its heads, fp32, to shared memory: dV (groups 0, 1: half the columns each), dK (2,
            // 3); nothing else uses the tiles any more
            tc_fence_after();
            const int half = group >> 1, c0 = (group & 1) * (D / 2);
            const int row = 32 * quarter + lane;
            float4 *dst = reinterpret_cast<float4 *>(sm) + (half * AT + row) * (D / 4);
#pragma unroll
            for (int i = 0; i < D / 64; ++i) {
                uint32_t v[32];
                tc_ld32(tmem + lb + (half ? TM_DK : TM_DV) + c0 + 32 * i, v);
                tc_wait_ld();
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    dst[(c0 / 4 + 8 * i + e) ^ (row & (D / 4 - 1))] =
                        make_float4(__uint_as_float(v[4 * e]), __uint_as_float(v[4 * e + 1]),
                                    __uint_as_float(v[4 * e + 2]), __uint_as_float(v[4 * e + 3]));
            }
        } else if (rank == 0 && group < 2) {
            // warps 0-3 store dV, 4-7 dK, through the K and V tiles (no MMA reads them any more)
            tc_fence_after();
            const int half = group;
            const int row = j0 + 32 * quarter;
            const int64_t at = ((static_cast<int64_t>(sq.k0) + row) * p.HKV + hk) * D;
            store_rows<D>(tmem + lb + (half ? TM_DK : TM_DV), total > 0, half ? p.scale : 1.f,
                          sb + half * TILE + quarter * (32 * D * 2), lane, sq.lk - row, (half ? p.dk : p.dv) + at,
                          static_cast<int64_t>(p.HKV) * D);
        }
    } else {
        ATTN_BWD_FEWER_REGISTERS();
        if (warp == kAttnBwdLoad + 1 && lane == 0) {
            // (also in CTAs without work: what follows in the stream waits for this launch only)
            asm volatile("griddepcontrol.wait;\n" ::: "memory");
        }
        if (warp == kAttnBwdLoad && lane == 0 && total > 0) {
            // ---------------- loads ----------------
            int nqi = 0, ndo = 0;  // tiles of Q and of dO requested
            bool ok = true;
            auto tile = [&](const CUtensorMap *m, uint32_t dst, int head, int row, uint32_t bar) {
                for (int c = 0; c < HALVES; ++c) tma_load_3d(dst + c * kHalfBytes, m, 64 * c, head, row, bar);
            };
            mbar_expect_tx(kfull, TILE);
            tile(&mk, sb, hk, sq.k0 + j0, kfull);
            mbar_expect_tx(vfull, TILE);
            tile(&mv, sb + TILE, hk, sq.k0 + j0, vfull);
            // the statistics, with dQ's corrections (nothing else depends on that launch)
            asm volatile("griddepcontrol.wait;\n" ::: "memory");
            for (int it = 0, hq = head0, i = first; it < total && ok && !*abort_flag; ++it) {
                const int st = it % NST;
                const uint32_t par = ((it / NST) - 1) & 1;
                if (it >= NST && !mbar_wait(qempty + 8 * st, par)) {
                    ok = false;
                    break;
                }
                mbar_expect_tx(qfull + 8 * st, TILE + 1024);
                tile(&mq, sb + S::Q + st * TILE, hq, sq.q0 + i * AT, qfull + 8 * st);
                bulk_load(sb + S::STAT + st * 1024,
                          p.stats + (static_cast<int64_t>(hq) * p.qslots + qslot0 + i) * (2 * AT), 1024, qfull + 8 * st);
                ++nqi;
                if (it >= NST && !mbar_wait(doempty + 8 * st, par)) {
                    ok = false;
                    break;
                }
                mbar_expect_tx(dofull + 8 * st, TILE);
                tile(&mdo, sb + S::DO + st * TILE, hq, sq.q0 + i * AT, dofull + 8 * st);
                ++ndo;
                if (++i == nq) {
                    i = first;
                    ++hq;
                }
            }
            if (!ok) fail(ERR_PIPE_EMPTY_WAIT);
            if (!ok || *abort_flag) {  // let the copies in flight land before the CTA leaves
                mbar_wait(kfull, 0);
                mbar_wait(vfull, 0);
                for (int i = max(0, nqi - NST); i < nqi; ++i) mbar_wait(qfull + 8 * (i % NST), (i / NST) & 1);
                for (int i = max(0, ndo - NST); i < ndo; ++i) mbar_wait(dofull + 8 * (i % NST), (i / NST) & 1);
            }
        } else if (warp < kAttnBwdMma + kIssuers && total > 0) {
            // ---------------- MMAs ----------------
            constexpr uint32_t id_s = idesc_bf16(128, AT, false, false), id_d = idesc_bf16(128, D, false, true);
            const TileDesc desc(sb);
            const int tail = sq.lq - (nq - 1) * AT;  // rows of the last query tile
            bool ok = true;
            auto wait = [&](uint32_t bar, uint32_t parity) {
                ok = ok && __all_sync(0xffffffffu, mbar_wait_quiet(bar, parity));
                tc_fence_after();
                return ok;
            };
            // the tile of iteration it of a ring, once it is there; left: tiles to the end of its head
            auto arrived = [&](uint32_t full, int ring, int it, int &left) {
                const int st = it % NST;
                if (!wait(full + 8 * st, (it / NST) & 1)) return false;
                if (--left == 0) {
                    left = cnt;
                    if (tail < AT) zero_tail_rows<D>(sb + ring + st * TILE, tail, lane);
                }
                return true;
            };
            // D[128 keys][128 queries] = (K or V) (Q or dO)^T
            auto product = [&](uint32_t d, int keys, int at, uint32_t commit) {
#pragma unroll
                for (int ks = 0; ks < D / 16; ++ks)
                    tc_mma_ss_warp(d, desc.k(keys, ks), desc.k(at, ks), id_s, ks > 0);
                tc_commit_warp(commit);
            };
            // D += A B, A in groups of 32 queries
            auto accumulate = [&](uint32_t d, uint32_t a, int at, bool more) {
#pragma unroll
                for (int ks = 0; ks < AT / 16; ++ks)
                    tc_mma_ts_warp(d, a + (ks >> 1) * TM_GROUP + (ks & 1) * 8, desc.mn(at, ks), id_d, more || ks > 0);
            };
            int left = cnt, left_do = cnt;
            auto score = [&](int it) {
                if (arrived(qfull, S::Q, it, left)) product(tmem + TM_S, 0, S::Q + (it % NST) * TILE, sfull);
            };
            auto dprob = [&](int it) {
                if (!arrived(dofull, S::DO, it, left_do)) return;
                product(tmem + TM_DP, TILE, S::DO + (it % NST) * TILE, dpfull);
                if (kIssuers == 2) tc_commit_warp(doempty + 8 * (it % NST));  // (else dV's commit covers it)
            };
            auto dv = [&](int it) {
                accumulate(tmem + TM_DV, tmem + TM_P, S::DO + (it % NST) * TILE, it > 0);
                tc_commit_warp(doempty + 8 * (it % NST));
            };
            auto dk = [&](int it) {
                accumulate(tmem + TM_DK, tmem + TM_DS, S::Q + (it % NST) * TILE, it > 0);
                tc_commit_warp(qempty + 8 * (it % NST));
            };
            auto go = [&](int it) { return it < total && ok && !__any_sync(0xffffffffu, *abort_flag); };
            if (!kOwn) {
                if (wait(kfull, 0)) score(0);
                if (wait(vfull, 0)) dprob(0);
                for (int it = 0; go(it); ++it) {
                    const bool more = it + 1 < total;
                    if (!wait(pready, it & 1)) break;
                    dv(it);
                    if (more) score(it + 1);
                    if (!ok || !wait(dsready, it & 1)) break;
                    dk(it);
                    if (more) dprob(it + 1);
                }
            } else if (warp == kAttnBwdMma) {  // S and dV
                if (wait(kfull, 0)) score(0);
                for (int it = 0; go(it); ++it) {
                    if (it + 1 < total && wait(sfree, it & 1)) score(it + 1);
                    // (dO's tile for this warp too: the other may not be there yet)
                    if (!ok || !arrived(dofull, S::DO, it, left_do) || !wait(pready, it & 1)) break;
                    dv(it);
                }
            } else {  // dP and dK
                if (wait(vfull, 0)) dprob(0);
                for (int it = 0; go(it); ++it) {
                    if (it + 1 < total && wait(dpfree, it & 1)) dprob(it + 1);
                    // (S of this tile is complete: what follows the sequence in Q is zero)
                    if (!ok || !wait(qfull + 8 * (it % NST), (it / NST) & 1) || !wait(dsready, it & 1)) break;
                    dk(it);
                }
            }
            tc_commit_warp(done);
            if (!ok && lane == 0) fail(ERR_PIPE_FULL_WAIT);
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == kAttnBwdMma) tc_dealloc(tmem, TM_COLS);
    if (p.split > 1 && total > 0) {
        // the cluster's sums: each CTA adds up its share of the rows over all CTAs, in their order
        cluster_sync();
        constexpr int Q4 = D / 4;
        const int rows = AT / p.split, r0 = rank * rows;
        // (the arithmetic warps: the others gave their registers away)
        for (int i = tid; warp < kAttnBwdWarps && i < 2 * rows * Q4; i += 32 * kAttnBwdWarps) {
            const int half = i / (rows * Q4), row = r0 + i / Q4 % rows, ch = i % Q4;
            const uint32_t at = sb + ((half * AT + row) * Q4 + (ch ^ (row & (Q4 - 1)))) * 16;
            float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
            for (int c = 0; c < p.split; ++c) {
                const float4 v = cluster_load4(at, c);
                a = make_float4(a.x + v.x, a.y + v.y, a.z + v.z, a.w + v.w);
            }
            const float m = half ? p.scale : 1.f;
            if (j0 + row < sq.lk)
                *reinterpret_cast<uint2 *>((half ? p.dk : p.dv) +
                                           ((static_cast<int64_t>(sq.k0) + j0 + row) * p.HKV + hk) * D + 4 * ch) =
                    make_uint2(pack_bf16(a.x * m, a.y * m), pack_bf16(a.z * m, a.w * m));
        }
        __syncwarp();    // (an aligned barrier, and rows past the end took no part in the stores)
        cluster_sync();  // no CTA leaves while another reads its sums
    }
}

// ---------------------------------------------------------------------------------------------------- dQ
// One CTA per tile of 128 queries of a head; a thread owns a query row of S and dP.  TMEM: S in two buffers (dS in
// bf16 over the one it came from), dP, dQ.  S of the next key tile is formed while this one's exponentials run, and
// dP of the next while P of the next is formed.  Two warps issue MMAs, S and dP the one and dQ the other, and K and V
// have rings of their own, as V's tiles are done with earlier: 1,340 -> 1,190 us (16,384 tokens, 16/4 heads), 266 ->
// 242 (8,192 tokens, 16/16 heads, D = 64) against one warp and one ring.
template <int D>
struct AttnDqSmem {
    static constexpr int TILE = AT * D * 2;
    static constexpr int NK = D == 128 ? 3 : 4, NV = D == 128 ? 2 : 4;
    static constexpr int K = 2 * TILE, V = K + NK * TILE;  // Q, dO, then the rings of K and V
    // kfull[NK] kempty[NK] vfull[NV] vempty[NV] qfull dofull sfull[2] dpfull dsready[2] done dpfree
    static constexpr int BAR = V + NV * TILE;
    static constexpr int TMEM_SLOT = BAR + (2 * (NK + NV) + 9) * 8;
    static constexpr int ABORT = TMEM_SLOT + 4;
    static constexpr int TOTAL = ABORT + 4;
};

template <int D>
__global__ void __launch_bounds__(kAttnBwdThreads, 1)
    kda_attn_dq_kernel(const AttnBwdParams p, const __grid_constant__ CUtensorMap mq,
                       const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv,
                       const __grid_constant__ CUtensorMap mdo)
{
    using S = AttnDqSmem<D>;
    constexpr int NK = S::NK, NV = S::NV, TILE = S::TILE, HALVES = D / 64;
    constexpr uint32_t TM_S = 0, TM_DP = 256, TM_DQ = 384, TM_COLS = 512;
    extern __shared__ __align__(1024) uint8_t sm[];
    const uint32_t sb = smem_u32(sm);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int h = blockIdx.x % p.H;
    int n, blk;
    asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
    if (!pick_block<AT, true>(p.seq.cu_q, p.seq.N, p.seq.T, blockIdx.x / p.H, lane, n, blk)) {
        asm volatile("griddepcontrol.wait;\n" ::: "memory");  // (what follows waits for this launch only)
        return;
    }
    const Seq sq = seq_of(p.seq, n);
    const int diff = sq.lk - sq.lq, r0 = blk * AT;
    const int seen_tile = min(r0 + AT, sq.lq) + diff;  // keys that the tile's last row sees
    const int nt = seen_tile <= 0 ? 0 : (seen_tile + AT - 1) / AT;

    const uint32_t kfull = sb + S::BAR, kempty = kfull + 8 * NK, vfull = kempty + 8 * NK, vempty = vfull + 8 * NV,
                   qfull = vempty + 8 * NV, dofull = qfull + 8, sfull0 = qfull + 16, dpfull = qfull + 32, dsready0 = qfull + 40, done = qfull + 56, dpfree = qfull + 64;
    volatile int *abort_flag = reinterpret_cast<volatile int *>(sm + S::ABORT);
    if (tid == 0) {
        for (int s = 0; s < 2 * (NK + NV); ++s) mbar_init(kfull + 8 * s, 1);
        for (uint32_t b : {qfull, dofull, sfull0, sfull0 + 8, dpfull}) mbar_init(b, 1);
        mbar_init(done, 2);
        for (int b = 0; b < 2; ++b) mbar_init(dsready0 + 8 * b, kAttnBwdWarps);
        mbar_init(dpfree, kAttnBwdWarps);
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == kAttnBwdMma) tc_alloc(sb + S::TMEM_SLOT, TM_COLS);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t *>(sm + S::TMEM_SLOT);
    auto fail = [&](unsigned code) {
        atomicOr(p.err, code);
        *abort_flag = 1;
    };

    if (warp < kAttnBwdWarps) {
        // ---------------- P and dS: query row, 32 of the key columns ----------------
        ATTN_BWD_MORE_REGISTERS();
        const int group = warp >> 2, quarter = warp & 3;
        const uint32_t lb = static_cast<uint32_t>(32 * quarter) << 16;
        const uint32_t td = tmem + lb + TM_DP + 32 * group;
        const int r = 32 * quarter + lane;
        const int slot = (p.seq.cu_q ? sq.q0 / AT + n : n * ((sq.lq + AT - 1) / AT)) + blk;
        float *stat = p.stats + (static_cast<int64_t>(h) * p.qslots + slot) * (2 * AT);
        asm volatile("griddepcontrol.wait;\n" ::: "memory");
        const float2 l2 = make_float2(stat[r], stat[r]), delta = make_float2(stat[AT + r], stat[AT + r]);
        // keys of this group that the row sees (rows past the end: p = 0)
        const int seen = r0 + r + 1 + diff - 32 * group;
        const float c = p.scale_log2;
        float2 sum = make_float2(0.f, 0.f);  // of dS over this thread's keys
        int best = -1;                       // the key whose probability is above 1/2, if it is one of them
        bool ok = true;
        for (int j = 0; j < nt; ++j) {
            const uint32_t ts = tmem + lb + TM_S + 128 * (j & 1) + 32 * group;
            ok = __all_sync(0xffffffffu, mbar_wait_quiet(sfull0 + 8 * (j & 1), (j >> 1) & 1));
            if (!ok) break;
            tc_fence_after();
            uint32_t x[32];
            tc_ld32(ts, x);
            tc_wait_ld();
            const int keys = seen - j * AT;
            if (__any_sync(0xffffffffu, keys < 32)) {
#pragma unroll
                for (int e = 0; e < 32; ++e)
                    if (e >= keys) x[e] = 0xff800000u;  // -inf
            }
            float2 pr[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                const float2 a = fma2(make_float2(__uint_as_float(x[2 * e]), __uint_as_float(x[2 * e + 1])),
                                      make_float2(c, c), l2);
                pr[e] = make_float2(ex2_ftz(a.x), ex2_ftz(a.y));
            }
            float top = fmaxf(pr[0].x, pr[0].y);
#pragma unroll
            for (int e = 1; e < 16; ++e) top = max3(top, pr[e].x, pr[e].y);
            if (__any_sync(0xffffffffu, top > 0.5f)) {
#pragma unroll
                for (int e = 0; e < 32; ++e)
                    if ((e & 1 ? pr[e >> 1].y : pr[e >> 1].x) > 0.5f) best = j * AT + 32 * group + e;
            }
            ok = __all_sync(0xffffffffu, mbar_wait_quiet(dpfull, j & 1));
            if (!ok) break;
            tc_fence_after();
            tc_ld32(td, x);
            tc_wait_ld();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(dpfree);
            uint32_t w[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                const float2 a = mul2(pr[e], add2(make_float2(__uint_as_float(x[2 * e]), __uint_as_float(x[2 * e + 1])),
                                                  delta));
                sum = add2(sum, a);
                w[e] = pack_bf16(a.x, a.y);
            }
            tc_st16(ts, w);
            tc_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(dsready0 + 8 * (j & 1));
        }
        if (ok && nt > 0) ok = __all_sync(0xffffffffu, mbar_wait_quiet(done, 0));
        // the rows' sums of dS over all keys (through the K tiles: no MMA reads them any more)
        float *sums = reinterpret_cast<float *>(sm + S::K);
        int *bests = reinterpret_cast<int *>(sums + 4 * AT);
        if (ok) {
            sums[group * AT + r] = sum.x + sum.y;
            bests[group * AT + r] = best;
        }
        asm volatile("bar.sync 1, %0;\n" ::"n"(32 * kAttnBwdWarps) : "memory");
        if (!ok) {
            if (lane == 0) fail(ERR_PIPE_FULL_WAIT);
        } else if (group == 0) {
            const float off = (sums[r] + sums[AT + r]) + (sums[2 * AT + r] + sums[3 * AT + r]);
            const int key = max(max(bests[r], bests[AT + r]), max(bests[2 * AT + r], bests[3 * AT + r]));
            if (r0 + r < sq.lq) stat[AT + r] = delta.x - off;  // (a row behind them may hold anything)
            // through the Q tile
            tc_fence_after();
            const int row = r0 + 32 * quarter, hk = h / (p.H / p.HKV);
            store_rows<D, true>(tmem + lb + TM_DQ, nt > 0, p.scale, sb + quarter * (32 * D * 2), lane, sq.lq - row,
                                p.dq + ((static_cast<int64_t>(sq.q0) + row) * p.H + h) * D,
                                static_cast<int64_t>(p.H) * D, -off,
                                key < 0 ? nullptr : p.k + (static_cast<int64_t>(sq.k0) + key) * p.k_stride + hk * D);
        }
    } else {
        ATTN_BWD_FEWER_REGISTERS();
        if (warp == kAttnBwdLoad && lane == 0 && nt > 0) {
            // ---------------- loads ----------------
            const int hk = h / (p.H / p.HKV);
            bool ok = true;
            auto tile = [&](const CUtensorMap *m, uint32_t dst, int head, int row, uint32_t bar) {
                mbar_expect_tx(bar, TILE);
                for (int c = 0; c < HALVES; ++c) tma_load_3d(dst + c * kHalfBytes, m, 64 * c, head, row, bar);
            };
            tile(&mq, sb, h, sq.q0 + r0, qfull);
            int nk = 0, nv = 0;  // tiles of K and of V requested
            for (int j = 0; j < nt && ok && !*abort_flag; ++j) {
                if (j >= NK && !mbar_wait(kempty + 8 * (j % NK), (j / NK - 1) & 1)) {
                    ok = false;
                    break;
                }
                tile(&mk, sb + S::K + (j % NK) * TILE, hk, sq.k0 + j * AT, kfull + 8 * (j % NK));
                ++nk;
                if (j == 0) tile(&mdo, sb + TILE, h, sq.q0 + r0, dofull);
                if (j >= NV && !mbar_wait(vempty + 8 * (j % NV), (j / NV - 1) & 1)) {
                    ok = false;
                    break;
                }
                tile(&mv, sb + S::V + (j % NV) * TILE, hk, sq.k0 + j * AT, vfull + 8 * (j % NV));
                ++nv;
            }
            if (!ok) fail(ERR_PIPE_EMPTY_WAIT);
            if (!ok || *abort_flag) {  // let the copies in flight land before the CTA leaves
                mbar_wait(qfull, 0);
                if (nk) mbar_wait(dofull, 0);
                for (int j = max(0, nk - NK); j < nk; ++j) mbar_wait(kfull + 8 * (j % NK), (j / NK) & 1);
                for (int j = max(0, nv - NV); j < nv; ++j) mbar_wait(vfull + 8 * (j % NV), (j / NV) & 1);
            }
        } else if (warp < kAttnBwdLoad && nt > 0) {
            // ---------------- MMAs: S and dP by one warp, dQ by the other ----------------
            constexpr uint32_t id_s = idesc_bf16(128, AT, false, false), id_d = idesc_bf16(128, D, false, true);
            const TileDesc desc(sb);
            const int tail = sq.lk - (nt - 1) * AT;  // rows of the last key tile, if fewer than 128
            bool ok = true;
            auto wait = [&](uint32_t bar, uint32_t parity) {
                ok = ok && __all_sync(0xffffffffu, mbar_wait_quiet(bar, parity));
                tc_fence_after();
                return ok;
            };
            if (warp == kAttnBwdMma) {
                // D[128 queries][128 keys] = (Q or dO) (K or V)^T, once the tile is there and what follows the sequence
                // taken out
                auto product = [&](uint32_t d, int rows, uint32_t full, uint32_t parity, int at, int j, uint32_t commit) {
                    if (!wait(full, parity)) return;
                    if (tail < AT && j == nt - 1) zero_tail_rows<D>(sb + at, tail, lane);
#pragma unroll
                    for (int ks = 0; ks < D / 16; ++ks)
                        tc_mma_ss_warp(d, desc.k(rows, ks), desc.k(at, ks), id_s, ks > 0);
                    tc_commit_warp(commit);
                };
                auto score = [&](int j) {
                    const int st = j % NK;
                    product(tmem + TM_S + 128 * (j & 1), 0, kfull + 8 * st, (j / NK) & 1, S::K + st * TILE, j,
                            sfull0 + 8 * (j & 1));
                };
                auto dprob = [&](int j) {
                    const int st = j % NV;
                    product(tmem + TM_DP, TILE, vfull + 8 * st, (j / NV) & 1, S::V + st * TILE, j, dpfull);
                    if (ok) tc_commit_warp(vempty + 8 * st);
                };
                if (wait(qfull, 0)) score(0);
                if (wait(dofull, 0)) dprob(0);
                if (ok && nt > 1) score(1);
                for (int j = 0; j + 1 < nt && ok && !__any_sync(0xffffffffu, *abort_flag); ++j) {
                    if (wait(dpfree, j & 1)) dprob(j + 1);
                    // dQ is done with dS of this tile, where S of the next but one goes
                    if (j + 2 < nt && wait(kempty + 8 * (j % NK), (j / NK) & 1)) score(j + 2);
                }
            } else {
                for (int j = 0; j < nt && ok && !__any_sync(0xffffffffu, *abort_flag); ++j) {
                    const int st = j % NK;
                    const uint32_t a = tmem + TM_S + 128 * (j & 1);
                    // (two barriers for dS: dP of the next tile is on its way, so the warps may be done with that one's
                    // dS before this one's arrival is seen; the one after next waits for S, which waits for dQ)
                    if (!wait(kfull + 8 * st, (j / NK) & 1) || !wait(dsready0 + 8 * (j & 1), (j >> 1) & 1)) break;
#pragma unroll
                    for (int ks = 0; ks < AT / 16; ++ks)
                        tc_mma_ts_warp(tmem + TM_DQ, a + (ks >> 1) * 32 + (ks & 1) * 8, desc.mn(S::K + st * TILE, ks),
                                       id_d, j > 0 || ks > 0);
                    tc_commit_warp(kempty + 8 * st);
                }
            }
            tc_commit_warp(done);
            if (!ok && lane == 0) fail(ERR_PIPE_FULL_WAIT);
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == kAttnBwdMma) tc_dealloc(tmem, TM_COLS);
}

}  // namespace kda
