// kda_attn_common.cuh -- what the softmax-attention kernels share: sequence
// lookup, tensor-core wrappers for bf16 operands, and pair arithmetic.
#pragma once
#include "kda_common.cuh"
#include "ptx.cuh"
#include "tc.cuh"

namespace kda {

// further bits of the device error word
enum : unsigned { ERR_BLOCK_ID = 16u, ERR_CACHE_FULL = 32u };

// Wait for a phase without taking issue slots from the scheduler's other warps: mbarrier.try_wait suspends the warp for
// a time that the hardware chooses (with a long limit of one's own it also resumes late).  Bounded like mbar_wait.
__device__ __forceinline__ bool mbar_try(uint32_t bar, uint32_t parity)
{
    uint32_t ok;
    asm volatile(
        "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}\n"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}
__device__ __forceinline__ bool mbar_wait_quiet(uint32_t bar, uint32_t parity)
{
    if (mbar_try(bar, parity)) return true;
    const long long t0 = clock64();
    while (!mbar_try(bar, parity))
        if (clock64() - t0 > kWaitBudget) return false;
    return true;
}

constexpr int AT = 128;  // rows of an attention tile, of queries and of keys
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// kind::f16 instruction descriptor: bf16 A and B, fp32 accumulator, either operand MN-major
__host__ __device__ constexpr uint32_t idesc_bf16(int M, int N, bool a_mn, bool b_mn)
{
    return (1u << 4) | (1u << 7) | (1u << 10) | (a_mn ? (1u << 15) : 0u) | (b_mn ? (1u << 16) : 0u) |
           (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24);
}
// D[tmem] (+)= A[smem] B[smem], called by a whole converged warp (one elected lane issues)
__device__ __forceinline__ void tc_mma_ss_warp(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                               uint32_t accumulate)
{
    asm volatile(
        "{\n .reg .pred p, e;\n elect.sync _|e, 0xffffffff;\n setp.ne.b32 p, %4, 0;\n"
        " @e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate));
}

// A [128 rows][D] bf16 tile is D / 64 column halves of [128][64], each 16 KB in the 128-byte-swizzle layout of a
// TMA load.  K-major (the rows are M or N): 32 bytes further per 16-column step, 16 KB per half.  MN-major (the
// rows are K): 64-column blocks 16 KB apart, 16-row steps 2 KB apart.
constexpr int kHalfBytes = AT * 128;
__device__ __forceinline__ uint64_t tile_desc_k(uint32_t saddr) { return sw128_desc(saddr, 16, 1024); }
__device__ __forceinline__ uint64_t tile_desc_mn(uint32_t saddr) { return sw128_desc(saddr, kHalfBytes, 1024); }
__device__ __forceinline__ uint32_t kstep_k(int ks)
{
    return static_cast<uint32_t>((ks >> 2) * (kHalfBytes >> 4) + (ks & 3) * 2);
}
__device__ __forceinline__ uint32_t kstep_mn(int ks) { return static_cast<uint32_t>(ks * (2048 >> 4)); }

// Descriptors of the tiles at byte offsets of the CTA's shared memory: a constant high word, and a low word (addresses
// below 2^18 bytes) that only offsets are added to, so that an MMA costs its issuer little more than itself.
struct TileDesc {
    uint32_t khi, klo, mhi, mlo;
    __device__ __forceinline__ explicit TileDesc(uint32_t sb)
    {
        const uint64_t k = tile_desc_k(sb), m = tile_desc_mn(sb);
        khi = static_cast<uint32_t>(k >> 32);
        klo = static_cast<uint32_t>(k);
        mhi = static_cast<uint32_t>(m >> 32);
        mlo = static_cast<uint32_t>(m);
    }
    __device__ __forceinline__ uint64_t k(int at, int ks) const  // step ks of 16 columns, rows are M or N
    {
        return (static_cast<uint64_t>(khi) << 32) | (klo + (at >> 4) + kstep_k(ks));
    }
    __device__ __forceinline__ uint64_t mn(int at, int ks) const  // step ks of 16 rows, columns are N
    {
        return (static_cast<uint64_t>(mhi) << 32) | (mlo + (at >> 4) + kstep_mn(ks));
    }
};

// Rows [first, 128) of a tile become zero (whole warp; the async proxy sees it).  Tail tiles of a sequence hold
// whatever follows it, and 0 * NaN in a matrix product would carry that into the sequence's results.
template <int D>
__device__ __forceinline__ void zero_tail_rows(uint32_t tile, int first, int lane)
{
    for (int i = lane; i < (AT - first) * 8; i += 32)
#pragma unroll
        for (int h = 0; h < D / 64; ++h)
            asm volatile("st.shared.v4.b32 [%0], {%1,%1,%1,%1};\n" ::"r"(
                             tile + h * kHalfBytes + (first + (i >> 3)) * 128 + (i & 7) * 16),
                         "r"(0)
                         : "memory");
    fence_proxy_async();
    __syncwarp();
}

// Thread-block clusters: a barrier of all their threads, and four or two floats of CTA `rank`'s shared memory.
__device__ __forceinline__ void cluster_sync()
{
    asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;\n" ::: "memory");
}
__device__ __forceinline__ float4 cluster_load4(uint32_t saddr, int rank)
{
    float4 v;
    asm volatile(
        "{\n .reg .b32 a;\n mapa.shared::cluster.u32 a, %4, %5;\n"
        " ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [a];\n}\n"
        : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
        : "r"(saddr), "r"(rank)
        : "memory");
    return v;
}

__device__ __forceinline__ float2 cluster_load2(uint32_t saddr, int rank)
{
    float2 v;
    asm volatile(
        "{\n .reg .b32 a;\n mapa.shared::cluster.u32 a, %2, %3;\n ld.shared::cluster.v2.f32 {%0, %1}, [a];\n}\n"
        : "=f"(v.x), "=f"(v.y)
        : "r"(saddr), "r"(rank)
        : "memory");
    return v;
}

// The sequences of a batch: packed (cu given, clamped to the tensors' rows) or plain.
struct SeqView {
    const int32_t *cu_q, *cu_k;  // [N+1], null for a plain batch
    int N, T, Tk;                // sequences; rows of q and of k (plain: of each sequence)
};
struct Seq {
    int q0, lq, k0, lk;  // first row and length, of queries and of keys
};
__device__ __forceinline__ void seq_range(const int32_t *cu, int n, int T, int &first, int &len)
{
    const int a = min(max(cu[n], 0), T), b = min(max(cu[n + 1], 0), T);
    first = a;
    len = max(b - a, 0);
}
__device__ __forceinline__ Seq seq_of(const SeqView &s, int n)
{
    Seq r;
    if (s.cu_q) {
        seq_range(s.cu_q, n, s.T, r.q0, r.lq);
        seq_range(s.cu_k, n, s.Tk, r.k0, r.lk);
    } else {
        r = Seq{n * s.T, s.T, n * s.Tk, s.Tk};
    }
    return r;
}
// Blocks of BLK rows are numbered so that no scan of the lengths is needed: sequence n's first block is
// cu[n] / BLK + n, which leaves room for all of its blocks (and sometimes one that stays empty).
template <int BLK>
__host__ __device__ constexpr int block_slots(int N, int T, bool packed)
{
    return packed ? T / BLK + N : N * ((T + BLK - 1) / BLK);
}
// The sequence and the block in it of slot t; false for an empty slot.  Whole warp; a 32-way search, so two
// dependent loads find one sequence of a thousand.
template <int BLK>
__device__ __forceinline__ bool find_block(const int32_t *cu, int N, int T, int t, int lane, int &n, int &blk)
{
    if (!cu) {
        const int per = (T + BLK - 1) / BLK;
        n = t / per;
        blk = t - n * per;
        return true;
    }
    int lo = 0, hi = N;
    while (hi - lo > 1) {
        const int step = (hi - lo + 31) / 32, i = lo + lane * step;
        const bool at = i < hi && min(max(cu[i], 0), T) / BLK + i <= t;
        const int c = max(__popc(__ballot_sync(0xffffffffu, at)), 1);
        lo += (c - 1) * step;
        hi = min(hi, lo + step);
    }
    int first, len;
    seq_range(cu, lo, T, first, len);
    n = lo;
    blk = t - (first / BLK + lo);
    return blk >= 0 && static_cast<int64_t>(blk) * BLK < len;
}

// The warp's 32 rows of a [128 rows][D] fp32 accumulator (TMEM, row = lane), times mul, rounded to bf16 and stored
// to dst + row * stride for the first `rows` of them, through 32 * D * 2 bytes of shared memory so that the global
// accesses are whole rows.  Without `any` the rows are zeros and TMEM is not read; a row whose mul is 0 is zeros.
// ADD: a row with an `other` row of D bf16 gets `weight` times that before the multiplication.
template <int D, bool ADD = false>
__device__ __forceinline__ void store_rows(uint32_t taddr, bool any, float mul, uint32_t stage, int lane, int rows,
                                           __nv_bfloat16 *dst, int64_t stride, float weight = 0.f,
                                           const __nv_bfloat16 *other = nullptr)
{
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
        uint32_t v[32];
        if (any) {
            tc_ld32(taddr + 32 * i, v);
            tc_wait_ld();
        }
        if (ADD && other) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const uint4 x = reinterpret_cast<const uint4 *>(other)[4 * i + e];
                const uint32_t u[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    v[8 * e + 2 * k] = __float_as_uint(fmaf(bf16lo(u[k]), weight, __uint_as_float(v[8 * e + 2 * k])));
                    v[8 * e + 2 * k + 1] =
                        __float_as_uint(fmaf(bf16hi(u[k]), weight, __uint_as_float(v[8 * e + 2 * k + 1])));
                }
            }
        }
        const bool zero = !any || mul == 0.f;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            uint32_t u[4];
#pragma unroll
            for (int k = 0; k < 4; ++k)
                u[k] = zero ? 0u
                            : pack_bf16(__uint_as_float(v[8 * e + 2 * k]) * mul,
                                        __uint_as_float(v[8 * e + 2 * k + 1]) * mul);
            const int ch = 4 * i + e;  // 16-byte piece of the row, swizzled by the row
            asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};\n" ::"r"(stage + lane * (D * 2) +
                                                                           ((ch ^ (lane & 7)) << 4)),
                         "r"(u[0]), "r"(u[1]), "r"(u[2]), "r"(u[3])
                         : "memory");
        }
    }
    __syncwarp();
    constexpr int PER = D * 2 / 16, ROWS = 32 / PER;  // pieces of a row, rows of one warp access
#pragma unroll
    for (int i = 0; i < 32 / ROWS; ++i) {
        const int rr = i * ROWS + lane / PER, ch = lane % PER;
        if (rr >= rows) continue;
        uint4 u;
        asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];\n"
                     : "=r"(u.x), "=r"(u.y), "=r"(u.z), "=r"(u.w)
                     : "r"(stage + rr * (D * 2) + ((ch ^ (rr & 7)) << 4)));
        *reinterpret_cast<uint4 *>(dst + rr * stride + 8 * ch) = u;
    }
}

// The sequence and block of the t-th CTA (of block_slots<BLK>()), those with most work first: blocks in levels by their
// place in their sequence, the last ones first (LAST) or the first ones.  With up to 128 packed sequences a warp holds
// their block counts and searches for the level; with more, blocks go in the order of their slots.
template <int BLK, bool LAST>
__device__ __forceinline__ bool pick_block(const int32_t *cu, int N, int T, int t, int lane, int &n, int &blk)
{
    const uint32_t all = 0xffffffffu;
    if (!cu) {
        const int level = t / N;
        n = t - level * N;
        blk = LAST ? (T + BLK - 1) / BLK - 1 - level : level;
        return true;
    }
    if (N > 128) return find_block<BLK>(cu, N, T, LAST ? block_slots<BLK>(N, T, true) - 1 - t : t, lane, n, blk);
    int nb[4], most = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const int i = lane + 32 * k;
        int first, len = 0;
        if (i < N) seq_range(cu, i, T, first, len);
        nb[k] = (len + BLK - 1) / BLK;
        most = max(most, nb[k]);
    }
    most = __reduce_max_sync(all, most);
    // CTAs before level b: blocks at places above b, or below it
    auto before = [&](int b) {
        int c = 0;
#pragma unroll
        for (int k = 0; k < 4; ++k) c += LAST ? max(nb[k] - b - 1, 0) : min(nb[k], b);
        return static_cast<int>(__reduce_add_sync(all, static_cast<unsigned>(c)));
    };
    if (t >= before(LAST ? -1 : most)) return false;
    int lo = 0, hi = most;  // the level is in [lo, hi)
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        // LAST: levels mid .. hi - 1 hold the CTAs before before(mid - 1)
        if (LAST ? t < before(mid - 1) : t >= before(mid)) lo = mid;
        else hi = mid;
    }
    blk = lo;
    int r = t - before(lo);  // the r-th sequence that has this block
    n = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const uint32_t m = __ballot_sync(all, nb[k] > lo);
        const int c = __popc(m);
        const uint32_t it = __ballot_sync(all, (m >> lane & 1) && __popc(m & ((1u << lane) - 1)) == r);
        if (r >= 0 && r < c) n = 32 * k + __ffs(it) - 1;
        r -= c;
    }
    return true;
}

__device__ __forceinline__ float max3(float a, float b, float c) { return fmaxf(fmaxf(a, b), c); }

}  // namespace kda
