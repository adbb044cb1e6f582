// kda_cache.cuh -- the paged 8-bit key/value cache: block tables and slot
// maps from request lengths, and storing new keys and values.
//
// A cache holds blocks of BS tokens, [HKV][BS][D] codes each, with one fp32 scale per (block, head); value = code *
// scale.  Codes are e4m3 or int8.  Scales are powers of two:
//   scale = the smallest 2^e with max |x| <= 2^e * (448 | 127) over the block's tokens of that head
// When tokens join a block that already holds some, its scale may have to grow, and the earlier codes are rounded
// again.  With powers of two that is exact for e4m3 (but for its subnormals) and adds at most half a step per doubling
// for int8, half + quarter + ... < one step in all, however many times tokens join; with scales of max / 448 every
// single token could move the scale and cost another rounding.  The price is up to one bit of int8's range.
#pragma once
#include "kda_attn_common.cuh"

namespace kda {

// ------------------------------------------------------------------------------------------ block tables, slot maps
struct CachePlanParams {
    const int32_t *context_lens, *new_lens;  // [B]
    int32_t *block_table;                    // [B, width], rows table_stride apart
    const int32_t *free_blocks;              // [num_free]
    int32_t *cu_seqlens, *seq_lens, *slot_map, *used;
    int64_t table_stride;
    int B, width, num_free, tokens, shift;   // block size = 1 << shift
    unsigned *err;
};
constexpr int kPlanThreads = 512, kPlanMaxRows = 16384;

// Every CTA scans all B rows by itself (a few KB from L2) and then writes its share of the slot map and of the new
// table entries, so one launch does it: the operator is bound by its launch and by that scan's latency.
__global__ void __launch_bounds__(kPlanThreads) kda_cache_plan_kernel(const CachePlanParams p)
{
    extern __shared__ int32_t plan_sm[];
    int32_t *cu = plan_sm, *take = plan_sm + p.B + 1;  // [B + 1] tokens before row b, [B] blocks taken before it
    __shared__ int2 part[kPlanThreads / 32];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int bs = 1 << p.shift, per = (p.B + kPlanThreads - 1) / kPlanThreads;
    auto blocks = [&](int tokens) { return (tokens >> p.shift) + ((tokens & (bs - 1)) != 0); };
    auto ctx = [&](int b) { return max(p.context_lens[b], 0); };
    auto add = [&](int b) { return max(p.new_lens[b], 0); };
    // this thread's rows b0 .. b1 - 1, then an exclusive scan over the threads
    const int b0 = min(tid * per, p.B), b1 = min(b0 + per, p.B);
    int2 s = make_int2(0, 0);
    for (int b = b0; b < b1; ++b) {
        const int c = ctx(b), a = add(b);
        s.x += a;
        s.y += blocks(c + a) - blocks(c);
    }
    int2 inc = s;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, inc.x, off), y = __shfl_up_sync(0xffffffffu, inc.y, off);
        if (lane >= off) {
            inc.x += x;
            inc.y += y;
        }
    }
    if (lane == 31) part[warp] = inc;
    __syncthreads();
    int2 at = make_int2(inc.x - s.x, inc.y - s.y), all = make_int2(0, 0);
    for (int w = 0; w < kPlanThreads / 32; ++w) {
        if (w < warp) {
            at.x += part[w].x;
            at.y += part[w].y;
        }
        all.x += part[w].x;
        all.y += part[w].y;
    }
    for (int b = b0; b < b1; ++b) {
        const int c = ctx(b), a = add(b);
        cu[b] = at.x;
        take[b] = at.y;
        if (blockIdx.x == 0) {
            p.cu_seqlens[b] = at.x;
            p.seq_lens[b] = c + a;
        }
        at.x += a;
        at.y += blocks(c + a) - blocks(c);
    }
    if (tid == 0) {
        cu[p.B] = all.x;
        if (blockIdx.x == 0) {
            p.cu_seqlens[p.B] = all.x;
            *p.used = min(all.y, p.num_free);
            if (all.y > p.num_free || all.x > p.tokens) atomicOr(p.err, ERR_CACHE_FULL);
        }
    }
    __syncthreads();
    // new table entries: a warp per row
    const int warps = gridDim.x * (kPlanThreads / 32);
    for (int b = blockIdx.x * (kPlanThreads / 32) + warp; b < p.B; b += warps) {
        const int have = blocks(ctx(b)), need = blocks(ctx(b) + add(b));
        if (need > p.width && lane == 0) atomicOr(p.err, ERR_CACHE_FULL);
        for (int k = have + lane; k < min(need, p.width); k += 32) {
            const int f = take[b] + k - have;
            p.block_table[b * p.table_stride + k] = f < p.num_free ? p.free_blocks[f] : -1;
        }
    }
    // the slot of each token; -1 behind the last one, and where there is no block
    for (int t = blockIdx.x * kPlanThreads + tid; t < p.tokens; t += gridDim.x * kPlanThreads) {
        int slot = -1;
        if (t < all.x) {
            int lo = 0, hi = p.B;  // the last row that starts at or before t (rows without tokens start where the next does)
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (cu[mid] <= t) lo = mid;
                else hi = mid;
            }
            const int c = ctx(lo), pos = c + t - cu[lo], k = pos >> p.shift, have = blocks(c);
            if (k < p.width) {
                const int f = take[lo] + k - have;
                const int id = k < have          ? p.block_table[lo * p.table_stride + k]
                               : f < p.num_free  ? p.free_blocks[f]
                                                 : -1;
                if (id >= 0 && id <= (INT_MAX >> p.shift)) slot = (id << p.shift) + (pos & (bs - 1));
            }
        }
        p.slot_map[t] = slot;
    }
}

// ------------------------------------------------------------------------------------------ storing keys and values
struct CacheAppendParams {
    const __nv_bfloat16 *x[2];  // k, v: row t at x + t * stride, [HKV][D]
    int64_t stride[2];
    uint8_t *cache[2];          // codes: block b at cache + b * block_stride, [HKV][BS][D]
    int64_t block_stride;
    float *scale[2];            // [num_blocks, HKV]
    const int32_t *slots;       // [T]
    int T, HKV, num_blocks, window;
    unsigned *err;
};
constexpr int kAppendThreads = 256;

// four floats -> four codes
template <bool FP8>
__device__ __forceinline__ uint32_t encode4(float a, float b, float c, float d)
{
    if constexpr (FP8) {
        uint16_t lo, hi;
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;\n" : "=h"(lo) : "f"(b), "f"(a));
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;\n" : "=h"(hi) : "f"(d), "f"(c));
        return static_cast<uint32_t>(lo) | (static_cast<uint32_t>(hi) << 16);
    } else {
        // nearest even; NaN becomes 0, infinities the largest code
        auto one = [](float x) { return static_cast<uint32_t>(min(max(__float2int_rn(x), -127), 127)) & 0xffu; };
        return one(a) | (one(b) << 8) | (one(c) << 16) | (one(d) << 24);
    }
}
// four codes -> four floats
template <bool FP8>
__device__ __forceinline__ float4 decode4(uint32_t w)
{
    if constexpr (FP8) {
        uint32_t lo, hi;
        asm("{\n .reg .b16 a, b;\n mov.b32 {a, b}, %2;\n cvt.rn.f16x2.e4m3x2 %0, a;\n cvt.rn.f16x2.e4m3x2 %1, b;\n}\n"
            : "=r"(lo), "=r"(hi)
            : "r"(w));
        const float2 x = unpack_f16(lo), y = unpack_f16(hi);
        return make_float4(x.x, x.y, y.x, y.y);
    } else {
        auto one = [w](int i) { return static_cast<float>(static_cast<int8_t>(w >> (8 * i))); };
        return make_float4(one(0), one(1), one(2), one(3));
    }
}

// A run is the tokens of one block that stand beside one another in the call; its first token leads it.  A CTA looks
// at `window` tokens and, for each leader among them, stores the run's tokens of 8 / (BS / 16) (head, k or v) units:
// BS / 16 warps a unit, 16 tokens a warp, held in registers between the maximum and the rounding, so every input byte
// is read once.  Windows are one token where there are few tokens (each may lead its own block) and up to a block where
// there are many (most of them follow a leader).  Bound by HBM for prompts (2 bytes in, 1 out per element), by latency
// for one token per request.
template <bool FP8, int D, int BS>
__global__ void __launch_bounds__(kAppendThreads) kda_cache_append_kernel(const CacheAppendParams p)
{
    constexpr int WPU = BS / 16, UNITS = 8 / WPU;         // warps of a unit, units of a CTA
    constexpr int LPT = D / 4, TPS = 32 / LPT, STEPS = 16 / TPS;  // lanes of a token, tokens of a step
    __shared__ uint32_t tops[8];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int groups = (2 * p.HKV + UNITS - 1) / UNITS;
    const int64_t t0 = static_cast<int64_t>(blockIdx.x / groups) * p.window;
    const int unit = (blockIdx.x % groups) * UNITS + warp / WPU, ws = warp % WPU;
    const bool live = unit < 2 * p.HKV;
    const int kv = unit & 1, h = min(unit >> 1, p.HKV - 1);
    const __nv_bfloat16 *in = kv ? p.x[1] : p.x[0];
    const int64_t stride = kv ? p.stride[1] : p.stride[0];
    uint8_t *cache = kv ? p.cache[1] : p.cache[0];
    float *scale = kv ? p.scale[1] : p.scale[0];
    const int slots = p.num_blocks * BS;
    for (int64_t t = t0; t < min(t0 + p.window, static_cast<int64_t>(p.T)); ++t) {
        const int lead = p.slots[t];
        if (lead < 0) continue;
        if (lead >= slots) {
            if (tid == 0) atomicOr(p.err, ERR_BLOCK_ID);
            continue;
        }
        const int blk = lead / BS;
        if (t > 0) {
            const int before = p.slots[t - 1];
            if (before >= 0 && before / BS == blk) continue;
        }
        // this warp's 16 tokens of the run: offset in the block (or -1), and whether all before it belong to the run
        int off = -1;
        bool whole = true;
#pragma unroll
        for (int w = 0; w < WPU; ++w) {
            const int64_t at = t + 16 * w + lane;
            const int s = whole && w <= ws && lane < 16 && at < p.T ? p.slots[at] : -1;
            const bool in = s >= 0 && s / BS == blk;
            const uint32_t m = __ballot_sync(0xffffffffu, in) & 0xffffu;
            const int n = whole && w <= ws ? __ffs(~m) - 1 : 0;  // leading tokens that belong to it
            if (w == ws) off = lane < n ? s % BS : -1;
            whole = whole && n == 16;
        }
        const __nv_bfloat16 *src = in + (t + 16 * ws) * stride + h * D + 4 * (lane % LPT);
        uint2 x[STEPS];
        int o[STEPS];
        uint32_t top2 = 0;  // largest |x| of either half, as bf16 pairs
#pragma unroll
        for (int i = 0; i < STEPS; ++i) {
            const int k = i * TPS + lane / LPT;
            o[i] = __shfl_sync(0xffffffffu, off, k);
            x[i] = make_uint2(0u, 0u);
            if (live && o[i] >= 0) x[i] = *reinterpret_cast<const uint2 *>(src + k * stride);
        }
#pragma unroll
        for (int i = 0; i < STEPS; ++i) {
            // max drops NaN
            asm("max.bf16x2 %0, %0, %1;\n" : "+r"(top2) : "r"(x[i].x & 0x7fff7fffu));
            asm("max.bf16x2 %0, %0, %1;\n" : "+r"(top2) : "r"(x[i].y & 0x7fff7fffu));
        }
        uint32_t top = max(top2 & 0xffffu, top2 >> 16);  // bits of non-negative bf16 order as integers
        top = __reduce_max_sync(0xffffffffu, top);
        if (top >= 0x7f80u) {  // infinities saturate: the maximum is over the finite values
            top = 0;
#pragma unroll
            for (int i = 0; i < STEPS; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const uint32_t a = ((e & 2 ? x[i].y : x[i].x) >> (16 * (e & 1))) & 0x7fffu;
                    if (a < 0x7f80u) top = max(top, a);
                }
            top = __reduce_max_sync(0xffffffffu, top);
        }
        const int first = lead % BS;  // tokens of the block before the run: kept
        float *sp = scale + static_cast<int64_t>(blk) * p.HKV + h;
        const float was = first > 0 ? *sp : 0.f;
        if (WPU > 1) {
            __syncthreads();  // (also: the run before has read tops)
            if (lane == 0) tops[warp] = top;
            __syncthreads();
#pragma unroll
            for (int w = 0; w < WPU; ++w) top = max(top, tops[warp / WPU * WPU + w]);
        }
        // the smallest power of two that holds it: 448 = 1.75 * 2^8, 127 = 1.984375 * 2^6
        const int e = static_cast<int>(top >> 7) - 127 - (FP8 ? 8 : 6) + ((top & 0x7fu) > (FP8 ? 0x60u : 0x7eu));
        float s = __int_as_float((max(e, -100) + 127) << 23);
        if (first > 0) s = fmaxf(was, s);
        if (!live) continue;
        uint8_t *dst = cache + blk * p.block_stride + static_cast<int64_t>(h) * BS * D + 4 * (lane % LPT);
        if (first > 0 && s != was) {  // the earlier tokens' codes at the new scale
            const float r = was / s;
            for (int k = ws * TPS + lane / LPT; k < first; k += WPU * TPS) {
                uint32_t *c = reinterpret_cast<uint32_t *>(dst + k * D);
                const float4 v = decode4<FP8>(*c);
                *c = encode4<FP8>(v.x * r, v.y * r, v.z * r, v.w * r);
            }
        }
        const float inv = 1.f / s;
#pragma unroll
        for (int i = 0; i < STEPS; ++i)
            if (o[i] >= 0)
                *reinterpret_cast<uint32_t *>(dst + o[i] * D) =
                    encode4<FP8>(bf16lo(x[i].x) * inv, bf16hi(x[i].x) * inv, bf16lo(x[i].y) * inv,
                                 bf16hi(x[i].y) * inv);
        if (ws == 0 && lane == 0) *sp = s;
    }
}

}  // namespace kda
