// kda_attn_forward.cuh -- causal softmax attention of packed or plain batches
// with shared key/value heads, on the 5th-generation tensor cores.
//
// For a sequence of Lq queries and Lk keys, query i sees keys j <= i + Lk - Lq:
//   s_ij = scale q_i . k_j,   lse_i = log sum_j exp(s_ij),   o_i = sum_j exp(s_ij - lse_i) v_j
// in one pass over the keys: with a reference m_i near the running maximum,
//   l_i += sum_j exp(s_ij - m_i),   O_i += sum_j exp(s_ij - m_i) v_j,
// both multiplied by exp(m_old - m_new) when the reference moves.  The reference moves only when the maximum has
// grown past it by more than 2^8: exponentials then stay below 2^8, far inside the range of the fp32 sums and of the
// bf16 operand P, and most key tiles skip the read-modify-write of O.
//
// One CTA takes 256 queries of one head as two tiles of 128 (A and B) and walks the key tiles of 128.
//   warps 0-3, 4-7  softmax of tile A, B: a thread per row
//   warp 8 (and 9)  issues the MMAs: S = Q K^T (both operands in shared memory) and O += P V (P in TMEM)
//   warp 10         TMA loads of Q, and of K and V tiles through a ring
// TMEM: S_A, S_B (128 columns each), O_A, O_B and, where there is room (D = 64), P_A and P_B.  P is handed over in
// halves of 64 keys, so that O += P V starts while the second half is formed (at D = 128: 4.07 -> 3.46 ms for 32,768
// tokens and 16 heads).
//  D = 128: P lies over S, so S of the next key tile is issued behind O += P V of this one, and one warp issues for
//    both tiles in turn, which keeps them half a period apart: while one is in its softmax, the tensor cores work on
//    the other. A softmax warp that sees S may also rescale O: no MMA writes it then.
//  D = 64: S of the next key tile is issued as soon as the softmax has read this one into registers, and each tile has
//    its own issuer (0.69-0.75 ms for 16,384 tokens and 16 heads; 0.83 with P over S).
// Bound at D = 64 by the exponentials (16 a cycle and SM: 2,048 cycles for both tiles, of about 2,700), and at D = 128 by
// the chain from S to P to O and by power: for 32,768 tokens of 16/4 heads the tensor pipe is busy in 58 % of the cycles,
// and back to back the clock falls to 1.59 GHz under the 1 kW limit (3.9 ms, 1,130 TFLOP/s; a single call on a rested card
// 3.5 ms).  The pairs of times here were taken in turn on rested cards.  Measured without gain: a polynomial on the FMA
// pipe for a quarter of the exponentials; scores in halves with N = 64, so that neither waits for the other (fewer cycles,
// but Q read twice: less clock, 3.86 ms).  Waiting warps are suspended (mbarrier.try_wait): polling took
// issue slots from the softmax (3.46 -> 3.36 ms).
#pragma once
#include <type_traits>

#include "kda_attn_common.cuh"

namespace kda {

struct AttnFwdParams {
    SeqView seq;
    int H, HKV;
    float scale, scale_log2;  // scale, scale * log2(e)
    __nv_bfloat16 *o;         // [rows, H, D]
    float *lse;               // [B, H, T] (packed: B = 1)
    unsigned *err;
};

template <int D>
struct AttnFwdSmem {
    static constexpr int TILE = AT * D * 2;
    static constexpr int NST = D == 128 ? 5 : 8;
    static constexpr int RING = 2 * TILE;
    static constexpr int BAR = RING + NST * TILE;  // full[NST] empty[NST] qfull[2] sfull[2] pready[2][2] sfree[2] odone[2]
    static constexpr int TMEM_SLOT = BAR + (2 * NST + 12) * 8;
    static constexpr int ABORT = TMEM_SLOT + 4;
    static constexpr int TOTAL = ABORT + 4;
};
// Three warpgroups: 168 registers a thread at launch (64,512 in all), of which the softmax warps take 208 and the
// third warpgroup (two of its warps idle) keeps 88: 256 * 208 + 128 * 88 = 64,512.
constexpr int kAttnFwdThreads = 384;
constexpr int kAttnFwdRows = 2 * AT;

template <int D>
__global__ void __launch_bounds__(kAttnFwdThreads, 1)
    kda_attn_fwd_kernel(const AttnFwdParams p, const __grid_constant__ CUtensorMap mq,
                        const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv)
{
    using S = AttnFwdSmem<D>;
    constexpr int NST = S::NST, TILE = S::TILE, HALVES = D / 64;
    constexpr bool kOwnP = D == 64;          // P has columns of its own
    constexpr int kIssuers = kOwnP ? 2 : 1;  // warps that issue MMAs
    constexpr uint32_t TM_O = 256, TM_P = kOwnP ? 384 : 0, TM_PSTEP = kOwnP ? 64 : 128, TM_COLS = 512;
    extern __shared__ __align__(1024) uint8_t sm[];
    const uint32_t sb = smem_u32(sm);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    // heads of one block of queries beside one another (they share keys), the blocks with most keys first
    const int h = blockIdx.x % p.H;
    int n, blk;
    if (!pick_block<kAttnFwdRows, true>(p.seq.cu_q, p.seq.N, p.seq.T, blockIdx.x / p.H, lane, n, blk)) return;
    const Seq sq = seq_of(p.seq, n);
    const int diff = sq.lk - sq.lq, r0 = blk * kAttnFwdRows;
    // key tiles that tile w (0, 1) of the block sees
    auto tiles = [&](int w) {
        const int a = r0 + w * AT;
        if (a >= sq.lq) return 0;
        const int seen = min(a + AT, sq.lq) + diff;
        return seen <= 0 ? 0 : (seen + AT - 1) / AT;
    };
    const int nt[2] = {tiles(0), tiles(1)};
    const int nmax = max(nt[0], nt[1]);

    const uint32_t full0 = sb + S::BAR, empty0 = full0 + 8 * NST, qfull0 = empty0 + 8 * NST, sfull0 = qfull0 + 16,
                   pready0 = qfull0 + 32, sfree0 = qfull0 + 64, odone0 = qfull0 + 80;
    volatile int *abort_flag = reinterpret_cast<volatile int *>(sm + S::ABORT);
    if (tid == 0) {
        for (int s = 0; s < NST; ++s) {
            mbar_init(full0 + 8 * s, 1);
            mbar_init(empty0 + 8 * s, kIssuers);
        }
        for (int w = 0; w < 2; ++w) {
            mbar_init(qfull0 + 8 * w, 1);
            mbar_init(sfull0 + 8 * w, 1);
            mbar_init(pready0 + 16 * w, 4);
            mbar_init(pready0 + 16 * w + 8, 4);
            mbar_init(sfree0 + 8 * w, 4);
            mbar_init(odone0 + 8 * w, 1);
        }
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 8) tc_alloc(sb + S::TMEM_SLOT, TM_COLS);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t *>(sm + S::TMEM_SLOT);
    auto fail = [&](unsigned code) {
        atomicOr(p.err, code);
        *abort_flag = 1;
    };

    if (warp < 8) {
        // ---------------- softmax: row `row` of tile w ----------------
        asm volatile("setmaxnreg.inc.sync.aligned.u32 208;\n");
        const int w = warp >> 2, quarter = warp & 3;
        const uint32_t lb = static_cast<uint32_t>(32 * quarter) << 16;
        const uint32_t ts = tmem + lb + 128 * w, tp = tmem + lb + TM_P + TM_PSTEP * w, to = tmem + lb + TM_O + D * w;
        const int row = r0 + w * AT + 32 * quarter + lane;
        const int seen = min(row, sq.lq - 1) + 1 + diff;  // keys that the row sees (rows past the end: any)
        const float c = p.scale_log2;
        float m = 0.f, l = 0.f;  // reference (in units of the scores), sum
        bool ok = true;
        auto rescale = [&](float alpha) {
#pragma unroll
            for (int i = 0; i < D / 16; ++i) {
                uint32_t ov[16];
                tc_ld16(to + 16 * i, ov);
                tc_wait_ld();
#pragma unroll
                for (int e = 0; e < 16; ++e) ov[e] = __float_as_uint(__uint_as_float(ov[e]) * alpha);
                tc_st16(to + 16 * i, ov);
            }
        };
        for (int j = 0; j < nt[w]; ++j) {
            ok = __all_sync(0xffffffffu, mbar_wait_quiet(sfull0 + 8 * w, j & 1));
            if (!ok) break;
            tc_fence_after();
            uint32_t r[4][32];
#pragma unroll
            for (int i = 0; i < 4; ++i) tc_ld32(ts + 32 * i, r[i]);
            tc_wait_ld();
            if (kOwnP) {  // the next scores may be formed
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(sfree0 + 8 * w);
            }
            const int keys = seen - j * AT;
            const bool cut = __any_sync(0xffffffffu, keys < AT);
            if (cut) {
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int e = 0; e < 32; ++e)
                        if (32 * i + e >= keys) r[i][e] = 0xff800000u;
            }
            float mx[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                mx[i] = __uint_as_float(r[i][0]);
#pragma unroll
                for (int e = 1; e < 31; e += 2)
                    mx[i] = max3(mx[i], __uint_as_float(r[i][e]), __uint_as_float(r[i][e + 1]));
                mx[i] = fmaxf(mx[i], __uint_as_float(r[i][31]));
            }
            const float top = fmaxf(max3(mx[0], mx[1], mx[2]), mx[3]);
            float alpha = 1.f;
            if (j == 0) {
                m = top == -INFINITY ? 0.f : top;
            } else if ((top - m) * c > 8.f || (l == 0.f && top != -INFINITY)) {
                // (a row that has seen no key yet takes its first finite maximum as the reference)
                alpha = l == 0.f ? 0.f : ex2((m - top) * c);
                m = top;
                l *= alpha;
            }
            const bool move = __any_sync(0xffffffffu, alpha != 1.f);
            if (kOwnP && j > 0) {  // O += P V of the tile before has read P and written O
                ok = __all_sync(0xffffffffu, mbar_wait_quiet(odone0 + 8 * w, (j - 1) & 1));
                if (!ok) break;
                tc_fence_after();
                if (move) rescale(alpha);
            }
            const float2 c2 = make_float2(c, c), b2 = make_float2(-m * c, -m * c);
            float2 sum = make_float2(0.f, 0.f), sum1 = sum;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                uint32_t pk[16];
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    float2 x =
                        fma2(make_float2(__uint_as_float(r[i][2 * e]), __uint_as_float(r[i][2 * e + 1])), c2, b2);
                    x = make_float2(ex2_ftz(x.x), ex2_ftz(x.y));
                    if (e & 1) sum1 = add2(sum1, x);
                    else sum = add2(sum, x);
                    pk[e] = pack_bf16(x.x, x.y);
                }
                if (!kOwnP && i == 0 && move) rescale(alpha);  // (off the way to the first exponentials)
                tc_st16(tp + 16 * i, pk);
                if (i & 1) {
                    tc_wait_st();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(pready0 + 8 * (2 * w + (i >> 1)));
                }
            }
            l += (sum.x + sum.y) + (sum1.x + sum1.y);
        }
        // ---------------- o = O / l, through this warp's rows of the Q tile ----------------
        if (ok && nt[w] > 0) ok = __all_sync(0xffffffffu, mbar_wait_quiet(odone0 + 8 * w, kOwnP ? (nt[w] - 1) & 1 : 0));
        if (!ok) {
            if (lane == 0) fail(ERR_PIPE_FULL_WAIT);
        } else {
            tc_fence_after();
            const float inv = l > 0.f || l != l ? 1.f / l : 0.f;
            const int first = r0 + w * AT + 32 * quarter;
            store_rows<D>(to, nt[w] > 0, inv, sb + w * TILE + quarter * (32 * D * 2), lane, sq.lq - first,
                          p.o + ((static_cast<int64_t>(sq.q0) + first) * p.H + h) * D, static_cast<int64_t>(p.H) * D);
            if (row < sq.lq) {
                const int64_t at = p.seq.cu_q ? static_cast<int64_t>(h) * p.seq.T + sq.q0 + row
                                              : (static_cast<int64_t>(n) * p.H + h) * p.seq.T + row;
                p.lse[at] = inv == 0.f ? -INFINITY : m * p.scale + logf(l);
            }
        }
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 88;\n");
        if (warp == 10) {
            // ---------------- loads: Q_A, K_0, Q_B, V_0, K_1, V_1, ... ----------------
            if (lane == 0) {
                const int hk = h / (p.H / p.HKV);
                auto load_q = [&](int w) {
                    if (nt[w] == 0) return;
                    mbar_expect_tx(qfull0 + 8 * w, TILE);
                    for (int c = 0; c < HALVES; ++c)
                        tma_load_3d(sb + w * TILE + c * kHalfBytes, &mq, 64 * c, h, sq.q0 + r0 + w * AT, qfull0 + 8 * w);
                };
                int issued = 0;
                auto load_kv = [&](const CUtensorMap *m, int j) {
                    const int s = issued % NST;
                    if (issued >= NST && !mbar_wait(empty0 + 8 * s, ((issued / NST) - 1) & 1)) {
                        fail(ERR_PIPE_EMPTY_WAIT);
                        return false;
                    }
                    mbar_expect_tx(full0 + 8 * s, TILE);
                    for (int c = 0; c < HALVES; ++c)
                        tma_load_3d(sb + S::RING + s * TILE + c * kHalfBytes, m, 64 * c, hk, sq.k0 + j * AT,
                                    full0 + 8 * s);
                    ++issued;
                    return true;
                };
                if (nmax > 0) {
                    load_q(0);
                    bool ok = load_kv(&mk, 0);
                    load_q(1);
                    ok = ok && load_kv(&mv, 0);
                    for (int j = 1; j < nmax && ok && !*abort_flag; ++j) ok = load_kv(&mk, j) && load_kv(&mv, j);
                    if (!ok || *abort_flag) {  // let the copies in flight land before the CTA leaves
                        for (int i = max(0, issued - NST); i < issued; ++i)
                            mbar_wait(full0 + 8 * (i % NST), (i / NST) & 1);
                        for (int w = 0; w < 2; ++w)
                            if (nt[w]) mbar_wait(qfull0 + 8 * w, 0);
                    }
                }
            }
        } else if (warp < 8 + kIssuers) {
            // ---------------- MMAs of both tiles in turn, or of one each ----------------
            auto issue = [&](auto first, auto last) {
                constexpr int w0 = decltype(first)::value, w1 = decltype(last)::value;
                constexpr uint32_t id_s = idesc_bf16(128, AT, false, false), id_o = idesc_bf16(128, D, false, true);
                const TileDesc desc(sb);
                bool ok = true;
                auto wait = [&](uint32_t bar, uint32_t parity) {
                    ok = ok && __all_sync(0xffffffffu, mbar_wait_quiet(bar, parity));
                    tc_fence_after();
                    return ok;
                };
                // ring positions: K_j at 2 j, V_j at 2 j + 1
                // (one issuer asks for each once, not for A, for B and to let it go: 229 -> 222 us, 8,192 tokens 16/4
                // heads)
                int seen[2] = {-1, -1};
                auto arrived = [&](int pos) {
                    if (!kOwnP && pos <= seen[pos & 1]) return ok;
                    seen[pos & 1] = pos;
                    return wait(full0 + 8 * (pos % NST), (pos / NST) & 1);
                };
                // An issuer lets go of every position, also of those that its tile does not use, but of none before it
                // is there: an arrival ahead of the loads would count for the position's predecessor in the ring.
                auto release = [&](int pos) {
                    if (arrived(pos)) tc_commit_warp(empty0 + 8 * (pos % NST));
                };
                auto score = [&](int w, int j) {  // S_w = Q_w K_j^T
                    if (!arrived(2 * j)) return;
                    const int at = S::RING + ((2 * j) % NST) * TILE;
#pragma unroll
                    for (int ks = 0; ks < D / 16; ++ks)
                        tc_mma_ss_warp(tmem + 128 * w, desc.k(w * TILE, ks), desc.k(at, ks), id_s, ks > 0);
                    tc_commit_warp(sfull0 + 8 * w);
                };
#pragma unroll
                for (int w = w0; w < w1; ++w)
                    if (nt[w] > 0 && wait(qfull0 + 8 * w, 0)) score(w, 0);
                if (nmax > 0) release(0);
                for (int j = 0; j < nmax && ok && !__any_sync(0xffffffffu, *abort_flag); ++j) {
                    const int st = (2 * j + 1) % NST;
#pragma unroll
                    for (int w = w0; w < w1; ++w) {
                        if (!ok || j >= nt[w]) continue;
                        if (kOwnP && j + 1 < nt[w] && wait(sfree0 + 8 * w, j & 1)) score(w, j + 1);
                        if (!ok || !arrived(2 * j + 1)) continue;
                        if (sq.lk - j * AT < AT) zero_tail_rows<D>(sb + S::RING + st * TILE, sq.lk - j * AT, lane);
                        const int at = S::RING + st * TILE;
#pragma unroll
                        for (int hf = 0; hf < 2; ++hf) {
                            if (!wait(pready0 + 8 * (2 * w + hf), j & 1)) break;
#pragma unroll
                            for (int ks = 4 * hf; ks < 4 * hf + 4; ++ks)
                                tc_mma_ts_warp(tmem + TM_O + D * w, tmem + TM_P + TM_PSTEP * w + 8 * ks,
                                               desc.mn(at, ks), id_o, j > 0 || ks > 0);
                        }
                        if (!ok) continue;
                        if (kOwnP || j + 1 == nt[w]) tc_commit_warp(odone0 + 8 * w);
                        if (!kOwnP && j + 1 < nt[w]) score(w, j + 1);
                    }
                    if (!ok) break;
                    // (a tile with fewer key tiles than the other lets theirs go as well)
                    release(2 * j + 1);
                    if (j + 1 < nmax) release(2 * j + 2);
                }
                if (!ok && lane == 0) fail(ERR_PIPE_FULL_WAIT);
            };
            using I0 = std::integral_constant<int, 0>;
            using I1 = std::integral_constant<int, 1>;
            using I2 = std::integral_constant<int, 2>;
            if constexpr (kIssuers == 1) issue(I0{}, I2{});
            else if (warp == 8) issue(I0{}, I1{});
            else issue(I1{}, I2{});
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 8) tc_dealloc(tmem, TM_COLS);
}

}  // namespace kda
