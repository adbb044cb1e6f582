// kda_attn_decode.cuh -- one-token attention over the paged 8-bit cache.
//
//   s_j = scale q . (ks_b code_k[j]),  o = sum_j softmax(s)_j vs_b code_v[j],  lse = log sum_j exp(s_j)
// with ks_b and vs_b the scales of token j's block and head.  Bound by reading the codes once: 2 D bytes per token and
// key/value head.
//
// The work is cut evenly over the CTAs, whatever the lengths: the tiles of all (row, key/value head)
// units stand in one line of W, and CTA c of G <= W takes tiles [c W / G, (c + 1) W / G) of it.  A unit inside one CTA
// is finished there; of a unit that several CTAs share, each leaves its maximum, sum and accumulator, and a second,
// dependent launch joins them in the order of the CTAs.
//
// Few short requests take another form: a cluster of eight CTAs per unit, which join over distributed shared memory,
// with no scan of the lengths and no second launch (one request of 777 tokens, 32/8 heads: 5.8 us on the device, 8.9 in
// the other).  What the host knows of the lengths is the table's width: in a table wider than 128 tiles a short request
// takes the first form.
//
// In a CTA, one warp requests the tiles' pages by TMA through a ring; four warps take 16 tokens of a tile each, with a
// running softmax of their own, and join at the end of the unit.  All query heads of a group share one pass over the
// codes, as columns of mma.sync: S^T = K Q^T and O^T += V^T P^T, whose M dimension is the tokens, or the head
// dimension.  The codes become fp16 exactly in registers (both code types fit), a query row becomes fp16 after a power
// of two makes its largest element 1..2 (exact, but for elements 2^-14 smaller than it, which round at 2^-24 of it).
// tcgen05 would want the codes in shared memory as fp16, and at 24 bytes per cycle and SM mma.sync is not what bounds.
//
// The value scale goes into the exponent: with x_j = s_j log2(e) and t_j = x_j + log2(vs_b), the weights 2^(t_j - M) are
// what multiplies the codes.  M is a running reference of t, so a weight is small only where its product with the codes
// is.  Weights are fp16 (11 bits), 2^12 where M is set and at most 2^15, which keeps what is flushed below 2^-37 of the
// largest.  The softmax's sum has a running reference of its own, L of x, and adds 2^(x_j - L).  (With one reference for
// both, 1 / vs_b is a factor of the sum, which then overflows for small scales, such as 65,536 tokens of a cache of zeros
// at scale 2^-100, and loses blocks whose scales are far below another's.)  The term is the weight times
// 2^(M - L) / vs_b, one factor for 16 tokens of a block.  Where that factor passes 2^48 the weights, which fp16 flushes
// anyway, are formed with the scale 2^(M - L - 48), so that they do not underflow before the sum has them.
// What leaves a warp, a CTA or a piece is M, the accumulator, and log2 of the whole sum.
#pragma once
#include "kda_attn_common.cuh"
#include "kda_cache.cuh"

namespace kda {

// A tile is 16 KB of codes: 64 tokens at D = 128, 128 at D = 64, where a warp takes two slices of 16 tokens at once.
// The warps' work on a tile is a chain of latencies (shared memory, MMAs, shuffles, exponentials, MMAs), so three CTAs
// share an SM where registers allow it (up to 8 query heads): 161 -> 147 us for 64 int8 requests of 500 to
// 12,000 tokens, 32/8 heads.
__host__ __device__ constexpr int ad_tile(int D) { return 64 * (128 / D); }
__host__ __device__ constexpr int ad_ctas(int NT) { return NT == 1 ? 3 : 2; }
constexpr int kAdWarps = 4, kAdThreads = 32 * kAdWarps + 32, kAdMaxCtas = 512;
// The form for few short requests: CTAs of a unit, and the most tiles that its table may hold (one request, 32/8 heads,
// D = 128; us on the device with a cluster and without: 500 tokens 5.4, 8.5; 2,000: 7.1, 10.2; 8,000: 13, 15; 32,000:
// 37, 21).
constexpr int kAdCluster = 8, kAdClusterTiles = 128;
// The longest request: token indices, rounded up to tiles and looked up ahead, stay below 2^31.
constexpr int kAdMaxTokens = INT_MAX - 4095;
// The join's threads, and the pieces times float4s of a unit that it joins in one CTA: eight for each thread.
constexpr int kAdJoinThreads = 512, kAdJoinItems = 8 * kAdJoinThreads;

struct AttnDecodeParams {
    const __nv_bfloat16 *q;  // row b at q + b * q_stride: [H, D]
    int64_t q_stride;
    const float *kscale, *vscale;  // [num_blocks, HKV]
    const int32_t *table;          // [B, width], rows table_stride apart
    int64_t table_stride;
    const int32_t *lens;           // [B]
    __nv_bfloat16 *o;              // [B, H, D]
    float *lse;                    // [B, H]
    float *part;                   // [G][2] pieces: accumulators [HB][D], then reference and log2 of the sum [HB][2]
    int4 *shared_unit;             // [G][2]: the unit that begins in CTA c and goes on behind it, and the one that comes in
                                   // from before (or -1); each with the CTAs behind its first, and that CTA
    unsigned *err;
    int B, H, HKV, chunks, width, num_blocks;  // chunks of HB query heads of a group
    float scale_log2;
};

template <int D, int NT>
struct AttnDecodeSmem {
    static constexpr int HB = 8 * NT;                  // query heads of a unit
    static constexpr int SL = 128 / D;                 // slices of a warp
    static constexpr int HALF = ad_tile(D) * D;        // K or V codes of a tile: 8 KB
    static constexpr int NST = NT == 1 ? 3 : 4;
    static constexpr int JOIN = NST * 2 * HALF;        // fp32 [4 warps][HB][D]
    static constexpr int QROWS = JOIN + kAdWarps * HB * D * 4;       // bf16 [2][HB][D]: queries of this unit and the next
    static constexpr int STATS = QROWS + 2 * HB * D * 2;             // fp32 [4 warps][HB][2]
    static constexpr int META = STATS + kAdWarps * HB * 2 * 4;       // float4 [NST][4 SL slices]
    static constexpr int SCAN = META + NST * kAdWarps * SL * 16;     // int64 [5 warps], start {b, tile}
    static constexpr int BAR = SCAN + 64 + 16;                       // full[NST] empty[NST] qfull[2] qempty[2]
    static constexpr int ABORT = BAR + (2 * NST + 4) * 8;
    static constexpr int TOTAL = ABORT + 8;
};

// Where CTA c's share of W tiles begins.
__device__ __forceinline__ int64_t share(int64_t W, int c, int G) { return W * c / G; }

__device__ __forceinline__ uint32_t movmatrix(uint32_t x)
{
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;\n" : "=r"(y) : "r"(x));
    return y;
}
// Codes to fp16 pairs: bytes 0 and 1 of w into lo, 2 and 3 into hi.
template <bool FP8>
__device__ __forceinline__ void codes_to_f16(uint32_t w, uint32_t &lo, uint32_t &hi)
{
    if constexpr (FP8) {
        asm("{\n .reg .b16 a, b;\n mov.b32 {a, b}, %2;\n cvt.rn.f16x2.e4m3x2 %0, a;\n cvt.rn.f16x2.e4m3x2 %1, b;\n}\n"
            : "=r"(lo), "=r"(hi)
            : "r"(w));
    } else {
        // byte u = code + 128 as the low bits of fp16 1024 + u; minus 1152
        const uint32_t u = w ^ 0x80808080u;
        const uint32_t a = __byte_perm(u, 0x64646464u, 0x4140), b = __byte_perm(u, 0x64646464u, 0x4342);
        const uint32_t off = 0x64806480u;  // 1152
        asm("sub.rn.f16x2 %0, %1, %2;\n" : "=r"(lo) : "r"(a), "r"(off));
        asm("sub.rn.f16x2 %0, %1, %2;\n" : "=r"(hi) : "r"(b), "r"(off));
    }
}

// log2 of a sum with its reference; -inf: no token counted.
// (lg2.approx is off by 2^-22, of itself or, between 1/2 and 2, absolutely)
__device__ __forceinline__ float log_sum(float L, float l)
{
    float y;
    asm("lg2.approx.ftz.f32 %0, %1;\n" : "=f"(y) : "f"(l));
    return l == 0.f ? -INFINITY : L + y;
}
// What a piece's accumulator (its reference Mk at most M) and sum are multiplied by and add, when pieces are joined.
__device__ __forceinline__ float join_weight(float Mk, float Lk, float M)
{
    return Mk == -INFINITY ? (Lk == -INFINITY ? 0.f : 1.f) : ex2_ftz(Mk - M);
}
__device__ __forceinline__ float join_sum(float Lk, float L) { return Lk == -INFINITY ? 0.f : ex2_ftz(Lk - L); }

// Four dims of a head's result from its accumulator, reference and log2 of the sum.
template <int D>
__device__ __forceinline__ void store_attention(const AttnDecodeParams &p, int b, int h, int d, float4 a, float M, float L)
{
    const int64_t at = static_cast<int64_t>(b) * p.H + h;
    const bool none = L == -INFINITY;
    const float f = ex2(0.5f * (M - L));  // in two steps: the whole may be below 2^-149
    *reinterpret_cast<uint2 *>(p.o + at * D + d) =
        none ? make_uint2(0u, 0u)
             : make_uint2(pack_bf16(a.x * f * f, a.y * f * f), pack_bf16(a.z * f * f, a.w * f * f));
    if (d == 0) p.lse[at] = none ? -INFINITY : L * kLn2;
}

template <bool FP8, int D, int NT, bool CL>
__global__ void __launch_bounds__(kAdThreads, ad_ctas(NT))
    kda_attn_decode_kernel(const AttnDecodeParams p, const __grid_constant__ CUtensorMap mk,
                           const __grid_constant__ CUtensorMap mv, const int shift)
{
    using S = AttnDecodeSmem<D, NT>;
    constexpr int NST = S::NST, HB = S::HB, HALF = S::HALF, SL = S::SL, KS = D / 16, MT = D / 16;
    constexpr int TILE = ad_tile(D), SLICES = TILE / 16, BATCH = 32 / SLICES;  // (tiles looked up at once)
    extern __shared__ __align__(1024) uint8_t sm[];
    const uint32_t sb = smem_u32(sm);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int c = blockIdx.x;
    const int units_row = p.HKV * p.chunks, group = p.H / p.HKV;
    const int bs = 1 << shift;
    // (lengths are rounded up to tiles, and a batch of tiles, 512 tokens, is looked up ahead)
    const int cap = static_cast<int>(min(static_cast<int64_t>(p.width) << shift, static_cast<int64_t>(kAdMaxTokens)));
    const uint32_t full0 = sb + S::BAR, empty0 = full0 + 8 * NST, qfull0 = empty0 + 8 * NST, qempty0 = qfull0 + 16;
    float4 *meta = reinterpret_cast<float4 *>(sm + S::META);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(sm + S::ABORT);
    auto len_of = [&](int b) { return min(max(p.lens[b], 0), cap); };
    auto tiles_of = [&](int b) { return (len_of(b) + TILE - 1) / TILE; };
    asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
    if (tid == 0) {
        for (int s = 0; s < NST; ++s) {
            mbar_init(full0 + 8 * s, 1);
            mbar_init(empty0 + 8 * s, kAdWarps);
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(qfull0 + 8 * s, 1);
            mbar_init(qempty0 + 8 * s, kAdWarps);
        }
        *abort_flag = 0;
        fence_mbar_init();
    }
    // this CTA's share as pieces: row, unit in the row, tiles [t0, t1) of the unit's n
    int b, u, n, t0, G = 0;
    int64_t left, W = 0, g1 = 0;
    if constexpr (CL) {
        const int unit = c / kAdCluster, rank = c % kAdCluster;
        b = unit / units_row;
        u = unit % units_row;
        n = tiles_of(b);
        if (p.lens[b] > cap && u == 0 && rank == 0 && tid == 0) atomicOr(p.err, ERR_BLOCK_ID);
        if (n == 0) {  // (the whole cluster leaves)
            const int heads = min(HB, group - u % p.chunks * HB);
            const int64_t at = static_cast<int64_t>(b) * p.H + u / p.chunks * group + u % p.chunks * HB;
            for (int i = tid; rank == 0 && i < heads * D / 2; i += kAdThreads)
                reinterpret_cast<uint32_t *>(p.o + at * D)[i] = 0u;
            if (rank == 0 && tid < heads) p.lse[at + tid] = -INFINITY;
            return;
        }
        t0 = n * rank / kAdCluster;
        left = n * (rank + 1) / kAdCluster - t0;
        __syncthreads();
    } else {
        // ---------------- W, and the row in which this CTA's share begins ----------------
        int64_t *scan = reinterpret_cast<int64_t *>(sm + S::SCAN);
        const int per = (p.B + kAdThreads - 1) / kAdThreads;
        const int b0 = min(tid * per, p.B), b1 = min(b0 + per, p.B);
        int64_t mine = 0;
        for (int i = b0; i < b1; ++i) mine += tiles_of(i);
        int64_t inc = mine;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int64_t x = __shfl_up_sync(0xffffffffu, inc, off);
            if (lane >= off) inc += x;
        }
        if (lane == 31) scan[warp] = inc;
        __syncthreads();
        int64_t before = inc - mine;
        for (int w = 0; w < kAdThreads / 32; ++w) {
            if (w < warp) before += scan[w];
            W += scan[w];
        }
        W *= units_row;
        G = static_cast<int>(min(W, static_cast<int64_t>(gridDim.x)));  // CTAs with work: a tile each at least
        const int64_t g0 = c < G ? share(W, c, G) : 0;
        g1 = c < G ? share(W, c + 1, G) : 0;
        // rows without tokens: zeros (every CTA some of them); too long for the table: an error
        for (int row = c; row < p.B; row += gridDim.x) {
            if (p.lens[row] > cap && tid == 0) atomicOr(p.err, ERR_BLOCK_ID);
            if (len_of(row) > 0) continue;
            for (int i = tid; i < p.H * D / 2; i += kAdThreads)
                reinterpret_cast<uint32_t *>(p.o + static_cast<int64_t>(row) * p.H * D)[i] = 0u;
            for (int i = tid; i < p.H; i += kAdThreads) p.lse[static_cast<int64_t>(row) * p.H + i] = -INFINITY;
        }
        int *start = reinterpret_cast<int *>(sm + S::SCAN + 64);
        if (g0 < g1 && g0 >= before * units_row && g0 < (before + mine) * units_row) {
            int64_t at = before;
            int row = b0;
            for (; g0 >= (at + tiles_of(row)) * units_row; ++row) at += tiles_of(row);
            start[0] = row;
            *reinterpret_cast<int64_t *>(start + 2) = g0 - at * units_row;
        }
        if (tid < 2) p.shared_unit[2 * c + tid] = make_int4(-1, 0, 0, 0);
        __syncthreads();
        if (g0 >= g1) return;
        b = start[0];
        n = tiles_of(b);
        const int64_t inrow = *reinterpret_cast<int64_t *>(start + 2);
        u = static_cast<int>(inrow / n);
        t0 = static_cast<int>(inrow - static_cast<int64_t>(u) * n);
        left = g1 - g0;
    }
    const bool idle = left == 0;
    auto next = [&](int t1) {  // behind tile t1 - 1 of this unit
        left -= t1 - t0;
        t0 = 0;
        if (left > 0 && ++u == units_row) {
            u = 0;
            do ++b;
            while ((n = tiles_of(b)) == 0);
        }
    };

    if (warp == kAdWarps) {
        // ---------------- loads: lane = tile of a batch * SLICES + slice of 16 tokens ----------------
        const int slices_page = min(bs / 16, SLICES), rows = 16 * slices_page;  // slices and rows of one copy
        const int my_tile = lane / SLICES, my_slice = lane % SLICES;
        int it = 0, pieces = 0;
        bool ok = true;
        while (left > 0 && ok) {
            const int t1 = static_cast<int>(min(static_cast<int64_t>(n), t0 + left));
            const int len = len_of(b), hk = u / p.chunks, hc = u % p.chunks;
            auto ids = [&](int t) {  // the block of this lane's slice
                const int tok = (t + my_tile) * TILE + 16 * my_slice;
                if (t + my_tile >= t1 || tok >= len) return -2;
                const int id = p.table[b * p.table_stride + (tok >> shift)];
                return id >= 0 && id < p.num_blocks ? id : -1;
            };
            int id = ids(t0);
            // the unit's queries: its heads stand beside one another in the row
            const int qs = pieces & 1;
            if (pieces >= 2) ok = __all_sync(0xffffffffu, mbar_wait(qempty0 + 8 * qs, ((pieces >> 1) - 1) & 1));
            if (!ok) break;
            if (lane == 0) {
                const int bytes = min(HB, group - hc * HB) * D * 2;
                mbar_expect_tx(qfull0 + 8 * qs, bytes);
                bulk_load(sb + S::QROWS + qs * HB * D * 2, p.q + b * p.q_stride + (hk * group + hc * HB) * D, bytes,
                          qfull0 + 8 * qs);
            }
            ++pieces;
            for (int t = t0; t < t1 && ok; t += BATCH) {
                const int far = ids(t + BATCH);
                float ks = 0.f, vs = 0.f;
                if (id >= 0) {
                    ks = p.kscale[static_cast<int64_t>(id) * p.HKV + hk];
                    vs = p.vscale[static_cast<int64_t>(id) * p.HKV + hk];
                }
                if (__any_sync(0xffffffffu, id == -1) && lane == 0) atomicOr(p.err, ERR_BLOCK_ID);
                // scale of the scores, log2 of the value scale and that + 48, whether the slice counts (1 or 2).  All
                // of a block's values are zero where its scale is (2): any scale will do then
                const float lv = log2f(vs > 0.f ? vs : 1.f);
                const float4 m = make_float4(ks, lv, lv + 48.f, id >= 0 ? (vs > 0.f ? 1.f : 2.f) : 0.f);
                const bool copies = id >= 0 && my_slice % slices_page == 0;  // the lane of a copy's first slice
                const uint32_t who = __ballot_sync(0xffffffffu, copies);
                for (int k = 0; k < BATCH && t + k < t1; ++k, ++it) {
                    const int st = it % NST;
                    if (it >= NST) {
                        ok = __all_sync(0xffffffffu, mbar_wait(empty0 + 8 * st, ((it / NST) - 1) & 1));
                        if (!ok || *abort_flag) {
                            ok = false;
                            break;
                        }
                    }
                    if (my_tile == k) meta[st * SLICES + my_slice] = m;
                    __syncwarp();
                    const int copies_k = __popc((who >> (SLICES * k)) & ((1u << SLICES) - 1));
                    if (lane == 0) mbar_expect_tx(full0 + 8 * st, copies_k * 2 * rows * D);
                    __syncwarp();
                    if (my_tile == k && copies) {
                        const int tok = (t + k) * TILE + 16 * my_slice;
                        const uint32_t dst = sb + st * 2 * HALF + 16 * my_slice * D;
                        const int row = hk * bs + (tok & (bs - 1));
                        tma_load_3d(dst, &mk, 0, row, id, full0 + 8 * st);
                        tma_load_3d(dst + HALF, &mv, 0, row, id, full0 + 8 * st);
                    }
                }
                id = far;
            }
            // A unit of several CTAs: from the one with its first tile to the one with its last.  (The CTAs behind the
            // first only where the join may want their help; at most n G / W + 2 CTAs have a piece.)
            if (!CL && lane == 0 && t1 - t0 < n &&
                (t0 == 0 || (static_cast<int64_t>(n) * G + 2 * W) * (HB * D / 4) >= 2 * kAdJoinItems * W)) {
                auto owner = [&](int64_t tile) {  // k with share(k) <= tile < share(k + 1)
                    int k = static_cast<int>(tile * G / W);
                    while (share(W, k + 1, G) <= tile) ++k;
                    while (share(W, k, G) > tile) --k;
                    return k;
                };
                const int64_t begin = g1 - left - t0;
                const int k0 = t0 == 0 ? c : owner(begin), k1 = t1 == n ? c : owner(begin + n - 1);
                p.shared_unit[2 * c + (t0 > 0)] = make_int4(b * units_row + u, k1 - k0, k0, 0);
            }
            next(t1);
        }
        if (!ok) {  // let the copies in flight land before the CTA leaves
            if (lane == 0) {
                atomicOr(p.err, ERR_PIPE_EMPTY_WAIT);
                *abort_flag = 1;
            }
            for (int i = max(0, it - NST); i < it; ++i) mbar_wait(full0 + 8 * (i % NST), (i / NST) & 1);
            for (int i = max(0, pieces - 2); i < pieces; ++i) mbar_wait(qfull0 + 8 * (i & 1), (i >> 1) & 1);
        }
    } else {
        // ---------------- arithmetic: warp w takes slices SL w .. SL w + SL - 1 of every tile ----------------
        const int r = lane >> 2, cc = lane & 3;
        float *join = reinterpret_cast<float *>(sm + S::JOIN), *stats = reinterpret_cast<float *>(sm + S::STATS);
        int it = 0, pieces = 0;
        bool ok = true;
        while (left > 0) {
            const int t1 = static_cast<int>(min(static_cast<int64_t>(n), t0 + left));
            const int len = len_of(b), hk = u / p.chunks, hc = u % p.chunks;
            const int heads = min(HB, group - hc * HB), head0 = hk * group + hc * HB;
            const int qs = pieces & 1;
            if (ok) ok = __all_sync(0xffffffffu, mbar_wait(qfull0 + 8 * qs, (pieces >> 1) & 1));
            ++pieces;
            // query rows as B operands: column r (head), the dims that this lane's K words hold
            uint32_t qf[NT][KS][2];
            float f0[NT], f1[NT];  // score factors of heads 2 cc and 2 cc + 1
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                const int hd = 8 * nt + r;
                const uint8_t *src = sm + S::QROWS + ((qs * HB + hd) * D + cc * (D / 4)) * 2;
                uint4 raw[D / 32];
#pragma unroll
                for (int i = 0; i < D / 32; ++i)
                    raw[i] = hd < heads ? reinterpret_cast<const uint4 *>(src)[i] : make_uint4(0u, 0u, 0u, 0u);
                uint32_t top = 0;
                auto word = [&](int k) {
                    const uint4 &v = raw[k >> 2];
                    return (k & 3) == 0 ? v.x : (k & 3) == 1 ? v.y : (k & 3) == 2 ? v.z : v.w;
                };
#pragma unroll
                for (int k = 0; k < D / 8; ++k) {
                    const uint32_t a = word(k) & 0x7fff7fffu;
                    top = max(top, max(a & 0xffffu, a >> 16));
                }
                top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
                top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
                const int e = min(max(static_cast<int>(top >> 7), 1), 253);  // exponent of the largest element
                const float down = __int_as_float((254 - e) << 23), up = __int_as_float(e << 23);
#pragma unroll
                for (int k = 0; k < D / 8; ++k)
                    qf[nt][k >> 1][k & 1] = pack_f16(bf16lo(word(k)) * down, bf16hi(word(k)) * down);
                const float f = up * p.scale_log2;
                f0[nt] = __shfl_sync(0xffffffffu, f, 8 * cc);
                f1[nt] = __shfl_sync(0xffffffffu, f, 8 * cc + 4);
            }
            if (ok && lane == 0) mbar_arrive(qempty0 + 8 * qs);
            float acc[NT][MT][4], l0[NT], l1[NT];
            float M0[NT], M1[NT], Q0[NT], Q1[NT];  // M, M - L
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                M0[nt] = M1[nt] = -INFINITY;
                Q0[nt] = Q1[nt] = l0[nt] = l1[nt] = 0.f;
#pragma unroll
                for (int i = 0; i < MT; ++i) acc[nt][i][0] = acc[nt][i][1] = acc[nt][i][2] = acc[nt][i][3] = 0.f;
            }
            // after a wait that ran out the warp only keeps the others company at the barriers
            for (int t = t0; t < t1 && ok; ++t, ++it) {
                const int st = it % NST;
                ok = __all_sync(0xffffffffu, mbar_wait(full0 + 8 * st, (it / NST) & 1));
                if (!ok) break;
                const uint8_t *kt = sm + st * 2 * HALF, *vt = kt + HALF;
                float4 m[SL];
                int have[SL];  // tokens of the slice
                bool counts = false;
#pragma unroll
                for (int y = 0; y < SL; ++y) {
                    m[y] = meta[st * SLICES + SL * warp + y];
                    have[y] = m[y].w != 0.f ? len - t * TILE - 16 * (SL * warp + y) : 0;
                    counts = counts || have[y] > 0;
                }
                if (counts) {
                    float s[SL][NT][4];
#pragma unroll
                    for (int y = 0; y < SL; ++y) {
                        uint32_t kw[2][KS];  // token r and r + 8: the words of this lane's D / 4 dims
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const int rw = 16 * (SL * warp + y) + r + 8 * i;
#pragma unroll
                            for (int j = 0; j < D / 64; ++j) {
                                const int ch = D == 128 ? ((2 * cc + j) ^ (rw & 7)) : (cc ^ ((rw >> 1) & 3));
                                const uint4 v = *reinterpret_cast<const uint4 *>(kt + rw * D + 16 * ch);
                                kw[i][4 * j] = v.x;
                                kw[i][4 * j + 1] = v.y;
                                kw[i][4 * j + 2] = v.z;
                                kw[i][4 * j + 3] = v.w;
                            }
                        }
                        // two chains of MMAs, half as long
                        float s1[NT][4];
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                            for (int e = 0; e < 4; ++e) s[y][nt][e] = s1[nt][e] = 0.f;
#pragma unroll
                        for (int k = 0; k < KS; ++k) {
                            uint32_t a[4];
                            codes_to_f16<FP8>(kw[0][k], a[0], a[2]);
                            codes_to_f16<FP8>(kw[1][k], a[1], a[3]);
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt) mma_f16(k & 1 ? s1[nt] : s[y][nt], a, qf[nt][k][0], qf[nt][k][1]);
                        }
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                            for (int e = 0; e < 4; ++e) s[y][nt][e] += s1[nt][e];
                    }
                    uint32_t pb[SL][NT][2];
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        float h0 = -INFINITY, h1 = -INFINITY;  // largest t
                        bool low = false;
#pragma unroll
                        for (int y = 0; y < SL; ++y) {
                            const float a = f0[nt] * m[y].x, bq = f1[nt] * m[y].x;
                            float(&x)[4] = s[y][nt];
                            x[0] = fmaf(x[0], a, m[y].y);
                            x[1] = fmaf(x[1], bq, m[y].y);
                            x[2] = fmaf(x[2], a, m[y].y);
                            x[3] = fmaf(x[3], bq, m[y].y);
                            if (r >= have[y]) x[0] = x[1] = -INFINITY;
                            if (r + 8 >= have[y]) x[2] = x[3] = -INFINITY;
                            h0 = fmaxf(h0, fmaxf(x[0], x[2]));
                            h1 = fmaxf(h1, fmaxf(x[1], x[3]));
                            low = low || m[y].z < Q0[nt] || m[y].z < Q1[nt];
                        }
#pragma unroll
                        for (int off = 4; off < 32; off <<= 1) {
                            h0 = fmaxf(h0, __shfl_xor_sync(0xffffffffu, h0, off));
                            h1 = fmaxf(h1, __shfl_xor_sync(0xffffffffu, h1, off));
                        }
                        // L moves where M does: a term is at most its weight, 2^15, times 2^48 without
                        const bool g0_ = h0 > M0[nt] + 15.f, g1_ = h1 > M1[nt] + 15.f;
                        const bool moves = __any_sync(0xffffffffu, g0_ || g1_ || low) != 0;
                        if (moves) {
                            float x0 = -INFINITY, x1 = -INFINITY;  // largest x
#pragma unroll
                            for (int y = 0; y < SL; ++y) {
                                x0 = fmaxf(x0, (SL == 1 ? h0 : fmaxf(s[y][nt][0], s[y][nt][2])) - m[y].y);
                                x1 = fmaxf(x1, (SL == 1 ? h1 : fmaxf(s[y][nt][1], s[y][nt][3])) - m[y].y);
                            }
#pragma unroll
                            for (int off = 4; SL > 1 && off < 32; off <<= 1) {
                                x0 = fmaxf(x0, __shfl_xor_sync(0xffffffffu, x0, off));
                                x1 = fmaxf(x1, __shfl_xor_sync(0xffffffffu, x1, off));
                            }
                            // the accumulators' factor; the sum's reference M - Q goes from M - Q to Mn - Qn
                            auto move = [](float &M, float &Q, float &l, bool g, float h, float x) {
                                const float Mn = g ? h - 12.f : M, L = M - Q;
                                const float Qn = g || x > L ? Mn - fmaxf(L, x) : Q, dm = g ? M - Mn : 0.f;
                                l *= ex2_ftz(dm + (Qn - Q));
                                M = Mn;
                                Q = Qn;
                                return ex2_ftz(dm);
                            };
                            const float al0 = move(M0[nt], Q0[nt], l0[nt], g0_, h0, x0);
                            const float al1 = move(M1[nt], Q1[nt], l1[nt], g1_, h1, x1);
#pragma unroll
                            for (int i = 0; i < MT; ++i) {
                                acc[nt][i][0] *= al0;
                                acc[nt][i][1] *= al1;
                                acc[nt][i][2] *= al0;
                                acc[nt][i][3] *= al1;
                            }
                        }
#pragma unroll
                        for (int y = 0; y < SL; ++y) {
                            float(&x)[4] = s[y][nt];
                            float e0 = -M0[nt], e1 = -M1[nt], c0 = Q0[nt] - m[y].y, c1 = Q1[nt] - m[y].y;
                            if (moves) {  // factors of 2^48 at most
                                const float u0 = fmaxf(c0 - 48.f, 0.f), u1 = fmaxf(c1 - 48.f, 0.f);
                                e0 += u0;
                                e1 += u1;
                                c0 -= u0;
                                c1 -= u1;
                            }
                            x[0] = ex2_ftz(x[0] + e0);
                            x[1] = ex2_ftz(x[1] + e1);
                            x[2] = ex2_ftz(x[2] + e0);
                            x[3] = ex2_ftz(x[3] + e1);
                            if (SL > 1 && have[y] <= 0) x[0] = x[1] = x[2] = x[3] = 0.f;  // (before any token: M is -inf)
                            l0[nt] = fmaf(x[0] + x[2], ex2_ftz(c0), l0[nt]);
                            l1[nt] = fmaf(x[1] + x[3], ex2_ftz(c1), l1[nt]);
                            pb[y][nt][0] = movmatrix(pack_f16(x[0], x[1]));
                            pb[y][nt][1] = movmatrix(pack_f16(x[2], x[3]));
                        }
                    }
#pragma unroll
                    for (int y = 0; y < SL; ++y) {
                        // V words: tokens 2 cc, 2 cc + 1, 2 cc + 8, 2 cc + 9; dims of chunk r
                        uint32_t vw[4][D / 32];
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int tok = 2 * cc + (i & 1) + 8 * (i >> 1), rw = 16 * (SL * warp + y) + tok;
                            if constexpr (D == 128) {
                                const uint4 v = *reinterpret_cast<const uint4 *>(vt + rw * D + 16 * (r ^ (rw & 7)));
                                vw[i][0] = v.x;
                                vw[i][1] = v.y;
                                vw[i][2] = v.z;
                                vw[i][3] = v.w;
                            } else {
                                const uint2 v = *reinterpret_cast<const uint2 *>(
                                    vt + rw * D + 16 * ((r >> 1) ^ ((rw >> 1) & 3)) + 8 * (r & 1));
                                vw[i][0] = v.x;
                                vw[i][1] = v.y;
                            }
                            // codes behind the last token, and of a block without a scale, may be anything
                            if (tok >= have[y] || m[y].w == 2.f)
#pragma unroll
                                for (int k = 0; k < D / 32; ++k) vw[i][k] = 0u;
                        }
#pragma unroll
                        for (int w = 0; w < D / 32; ++w) {
                            // bytes of two tokens side by side: A operand pairs along the tokens
                            uint32_t a[2][4];  // dims 4 w + {0, 1} and {2, 3} of the chunk: a0 a1 a2 a3
#pragma unroll
                            for (int pr = 0; pr < 2; ++pr) {
                                const uint32_t lo = __byte_perm(vw[2 * pr][w], vw[2 * pr + 1][w], 0x5140);
                                const uint32_t hi = __byte_perm(vw[2 * pr][w], vw[2 * pr + 1][w], 0x7362);
                                codes_to_f16<FP8>(lo, a[0][2 * pr], a[0][2 * pr + 1]);
                                codes_to_f16<FP8>(hi, a[1][2 * pr], a[1][2 * pr + 1]);
                            }
#pragma unroll
                            for (int i = 0; i < 2; ++i)
#pragma unroll
                                for (int nt = 0; nt < NT; ++nt)
                                    mma_f16(acc[nt][2 * w + i], a[i], pb[y][nt][0], pb[y][nt][1]);
                        }
                    }
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(empty0 + 8 * st);
            }
            if (!ok && lane == 0) {
                atomicOr(p.err, ERR_PIPE_FULL_WAIT);
                *abort_flag = 1;
            }
            // ---------------- join the four warps (the unit before has been read) ----------------
            asm volatile("bar.sync 1, %0;\n" ::"n"(32 * kAdWarps) : "memory");
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
                for (int off = 4; off < 32; off <<= 1) {
                    l0[nt] += __shfl_xor_sync(0xffffffffu, l0[nt], off);
                    l1[nt] += __shfl_xor_sync(0xffffffffu, l1[nt], off);
                }
#pragma unroll
                for (int hh = 0; hh < 2; ++hh) {
                    float *dst = join + (warp * HB + 8 * nt + 2 * cc + hh) * D + r * (D / 8);
#pragma unroll
                    for (int i = 0; i < MT; i += 2)
                        *reinterpret_cast<float4 *>(dst + 2 * i) = make_float4(
                            acc[nt][i][hh], acc[nt][i][2 + hh], acc[nt][i + 1][hh], acc[nt][i + 1][2 + hh]);
                }
                if (r == 0) {
                    float *st = stats + (warp * HB + 8 * nt + 2 * cc) * 2;
                    st[0] = M0[nt];
                    st[1] = log_sum(M0[nt] - Q0[nt], l0[nt]);
                    st[2] = M1[nt];
                    st[3] = log_sum(M1[nt] - Q1[nt], l1[nt]);
                }
            }
            asm volatile("bar.sync 1, %0;\n" ::"n"(32 * kAdWarps) : "memory");
            const bool whole = t0 == 0 && t1 == n;
            float *part = p.part + static_cast<int64_t>(2 * c + (t0 > 0 ? 0 : 1)) * (HB * (D + 2));
            for (int i = tid; i < heads * (D / 4); i += 32 * kAdWarps) {
                const int hd = i / (D / 4), d = 4 * (i % (D / 4));
                float M = -INFINITY, L = -INFINITY;
#pragma unroll
                for (int w = 0; w < kAdWarps; ++w) {
                    M = fmaxf(M, stats[(w * HB + hd) * 2]);
                    L = fmaxf(L, stats[(w * HB + hd) * 2 + 1]);
                }
                float l = 0.f;
                float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                for (int w = 0; w < kAdWarps; ++w) {
                    const float Mw = stats[(w * HB + hd) * 2], Lw = stats[(w * HB + hd) * 2 + 1];
                    const float f = join_weight(Mw, Lw, M);
                    const float4 v = *reinterpret_cast<const float4 *>(join + (w * HB + hd) * D + d);
                    l += join_sum(Lw, L);
                    a = make_float4(fmaf(v.x, f, a.x), fmaf(v.y, f, a.y), fmaf(v.z, f, a.z), fmaf(v.w, f, a.w));
                }
                L = log_sum(L, l);
                if constexpr (CL) {  // this CTA's piece, in shared memory
                    reinterpret_cast<float4 *>(sm + S::QROWS)[i] = a;
                    if (d == 0) reinterpret_cast<float2 *>(sm + S::META)[hd] = make_float2(M, L);
                } else if (whole) {
                    store_attention<D>(p, b, head0 + hd, d, a, M, L);
                } else {
                    *reinterpret_cast<float4 *>(part + hd * D + d) = a;
                    if (d == 0) *reinterpret_cast<float2 *>(part + HB * D + 2 * hd) = make_float2(M, L);
                }
            }
            next(t1);
        }
        if (CL && idle) {  // fewer tiles than CTAs: an empty piece
            for (int i = tid; i < HB * D / 4; i += 32 * kAdWarps)
                reinterpret_cast<float4 *>(sm + S::QROWS)[i] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (tid < HB) reinterpret_cast<float2 *>(sm + S::META)[tid] = make_float2(-INFINITY, -INFINITY);
        }
    }
    if constexpr (CL) {
        // the unit's result from its CTAs' pieces, in their order: HB / 8 heads a CTA
        __syncwarp();
        cluster_sync();
        const int hc = u % p.chunks, heads = min(HB, group - hc * HB);
        for (int i = tid; i < HB / kAdCluster * (D / 4); i += kAdThreads) {
            const int hd = c % kAdCluster * (HB / kAdCluster) + i / (D / 4), d = 4 * (i % (D / 4));
            if (hd >= heads) continue;
            float2 ml[kAdCluster];
            float4 v[kAdCluster];
            float M = -INFINITY, L = -INFINITY, l = 0.f;
#pragma unroll
            for (int k = 0; k < kAdCluster; ++k) {
                ml[k] = cluster_load2(sb + S::META + 8 * hd, k);
                v[k] = cluster_load4(sb + S::QROWS + (hd * D + d) * 4, k);
            }
#pragma unroll
            for (int k = 0; k < kAdCluster; ++k) {
                M = fmaxf(M, ml[k].x);
                L = fmaxf(L, ml[k].y);
            }
            float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int k = 0; k < kAdCluster; ++k) {
                const float f = join_weight(ml[k].x, ml[k].y, M);
                l += join_sum(ml[k].y, L);
                a = make_float4(fmaf(v[k].x, f, a.x), fmaf(v[k].y, f, a.y), fmaf(v[k].z, f, a.z), fmaf(v[k].w, f, a.w));
            }
            store_attention<D>(p, b, u / p.chunks * group + hc * HB + hd, d, a, M, log_sum(L, l));
        }
        __syncwarp();
        cluster_sync();  // no CTA leaves while another reads its piece
    }
}

// Joins the pieces of a unit that began in CTA c, in their order.  A thread takes a head, four dims and a run of the
// pieces; the runs are joined through shared memory.  Bound by the latency of its dependent loads (which unit;
// references and accumulators, eight pieces at a time).
struct AttnPiece {
    float M, L, l;  // references of the weights and of the sum
    float4 a;
    __device__ __forceinline__ void add(float Mk, float Lk, float4 v)  // the other's references at most M and L
    {
        const float f = join_weight(Mk, Lk, M);
        l += join_sum(Lk, L);
        a = make_float4(fmaf(v.x, f, a.x), fmaf(v.y, f, a.y), fmaf(v.z, f, a.z), fmaf(v.w, f, a.w));
    }
    __device__ __forceinline__ void refer(float Mn, float Ln)
    {
        const float f = join_weight(M, l == 0.f ? -INFINITY : 0.f, Mn);
        l = l == 0.f ? 0.f : l * ex2_ftz(L - Ln);
        M = Mn;
        L = Ln;
        a = make_float4(a.x * f, a.y * f, a.z * f, a.w * f);
    }
};
template <int D, int NT>
__global__ void __launch_bounds__(kAdJoinThreads) kda_attn_decode_join_kernel(const AttnDecodeParams p)
{
    constexpr int HB = 8 * NT, PIECE = HB * (D + 2);
    __shared__ AttnPiece runs[kAdJoinThreads];
    asm volatile("griddepcontrol.wait;\n" ::: "memory");
    const int tid = threadIdx.x, units_row = p.HKV * p.chunks, group = p.H / p.HKV;
    // A share of a unit's heads: all of them, unless there are so many pieces that a run would be longer than eight;
    // then the CTAs behind the first take shares too (one request of 131,072 tokens, 8/1 heads: 44 -> 20 us for the
    // step).
    auto join = [&](int4 su, int part) {
        const int c = su.z, b = su.x / units_row, u = su.x % units_row, hk = u / p.chunks, hc = u % p.chunks;
        const int heads = min(HB, group - hc * HB), n = su.y + 1;
        const int parts = max(1, min(heads, n * heads * (D / 4) / kAdJoinItems));
        if (part >= parts) return;
        const int h0 = heads * part / parts, items = (heads * (part + 1) / parts - h0) * (D / 4);
        const int nr = kAdJoinThreads / items;  // runs
        const int item = tid % items, run = tid / items, hd = h0 + item / (D / 4), d = 4 * (item % (D / 4));
        const int k_begin = n * run / nr, k_end = run < nr ? n * (run + 1) / nr : 0;
        // the piece of CTA c is its last one, those of the CTAs behind their first
        const float *first = p.part + (2ll * c + 1) * PIECE, *rest = p.part + 2ll * c * PIECE;
        AttnPiece all{-INFINITY, -INFINITY, 0.f, make_float4(0.f, 0.f, 0.f, 0.f)};
        for (int k0 = k_begin; k0 < k_end; k0 += 8) {
            float2 ml[8];
            float4 v[8];
            float M = all.M, L = all.L;
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                ml[k] = make_float2(-INFINITY, -INFINITY);
                v[k] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (k0 + k < k_end) {
                    const float *src = k0 + k == 0 ? first : rest + 2ll * (k0 + k) * PIECE;
                    ml[k] = *reinterpret_cast<const float2 *>(src + HB * D + 2 * hd);
                    v[k] = *reinterpret_cast<const float4 *>(src + hd * D + d);
                }
            }
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                M = fmaxf(M, ml[k].x);
                L = fmaxf(L, ml[k].y);
            }
            all.refer(M, L);
#pragma unroll
            for (int k = 0; k < 8; ++k) all.add(ml[k].x, ml[k].y, v[k]);
        }
        __syncthreads();  // (the runs of the share before are read)
        runs[tid] = all;
        __syncthreads();
        if (run > 0) return;
        for (int r = 1; r < nr; ++r) {
            const AttnPiece &o = runs[r * items + item];
            const float Lo = log_sum(o.L, o.l);
            all.refer(fmaxf(all.M, o.M), fmaxf(all.L, Lo));
            all.add(o.M, Lo, o.a);
        }
        store_attention<D>(p, b, hk * group + hc * HB + hd, d, all.a, all.M, log_sum(all.L, all.l));
    };
    const int4 out = p.shared_unit[2 * blockIdx.x], in = p.shared_unit[2 * blockIdx.x + 1];
    if (out.x >= 0) join(out, 0);
    if (in.x >= 0) join(in, blockIdx.x - in.z);
}

}  // namespace kda
