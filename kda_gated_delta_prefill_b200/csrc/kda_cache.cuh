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
    // [B + 1] tokens before row b; [B] blocks taken before it; [B] tokens held
    int32_t *cu = plan_sm, *take = cu + p.B + 1, *held = take + p.B;
    __shared__ int2 part[kPlanThreads / 32];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int bs = 1 << p.shift, per = (p.B + kPlanThreads - 1) / kPlanThreads;
    auto blocks = [&](int tokens) { return (tokens >> p.shift) + ((tokens & (bs - 1)) != 0); };
    // lengths, and sums of them and of blocks, stop at 2^31 - 1: no index below may come from a sum that wrapped
    auto ctx = [&](int b) { return max(p.context_lens[b], 0); };
    auto add = [&](int b, int c) { return min(max(p.new_lens[b], 0), INT_MAX - c); };
    auto sum = [](int x, int y) { return x > INT_MAX - y ? INT_MAX : x + y; };
    // this thread's rows b0 .. b1 - 1, then an exclusive scan over the threads
    const int b0 = min(tid * per, p.B), b1 = min(b0 + per, p.B);
    int2 s = make_int2(0, 0);
    for (int b = b0; b < b1; ++b) {
        const int c = ctx(b), a = add(b, c);
        s.x = sum(s.x, a);
        s.y = sum(s.y, blocks(c + a) - blocks(c));
    }
    int2 inc = s;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, inc.x, off), y = __shfl_up_sync(0xffffffffu, inc.y, off);
        if (lane >= off) {
            inc.x = sum(inc.x, x);
            inc.y = sum(inc.y, y);
        }
    }
    if (lane == 31) part[warp] = inc;
    __syncthreads();
    int2 at = make_int2(__shfl_up_sync(0xffffffffu, inc.x, 1), __shfl_up_sync(0xffffffffu, inc.y, 1));
    if (lane == 0) at = make_int2(0, 0);
    int2 all = make_int2(0, 0);
    for (int w = 0; w < kPlanThreads / 32; ++w) {
        if (w == warp) at = make_int2(sum(all.x, at.x), sum(all.y, at.y));
        all = make_int2(sum(all.x, part[w].x), sum(all.y, part[w].y));
    }
    for (int b = b0; b < b1; ++b) {
        const int c = ctx(b), a = add(b, c);
        cu[b] = at.x;
        take[b] = at.y;
        held[b] = c;
        if (blockIdx.x == 0) {
            p.cu_seqlens[b] = at.x;
            p.seq_lens[b] = c + a;
        }
        at.x = sum(at.x, a);
        at.y = sum(at.y, blocks(c + a) - blocks(c));
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
        const int have = blocks(ctx(b)), need = blocks(ctx(b) + add(b, ctx(b))), left = p.num_free - take[b];
        if (need > p.width && lane == 0) atomicOr(p.err, ERR_CACHE_FULL);
        for (int k = have + lane; k < min(need, p.width); k += 32) {
            p.block_table[b * p.table_stride + k] = k - have < left ? p.free_blocks[take[b] + k - have] : -1;
        }
    }
    // The slot of each token; -1 behind the last one, and where there is no block.  A thread takes four tokens: one
    // search and one table entry, unless a row or a block ends among them.
    int steps = 0;
    while ((1 << steps) < p.B) ++steps;
    const bool wide = (reinterpret_cast<uintptr_t>(p.slot_map) & 15) == 0;
    bool lost = false;  // a token without a slot, also for want of a block in an earlier call
    for (int t = 4 * (blockIdx.x * kPlanThreads + tid); t < p.tokens; t += 4 * gridDim.x * kPlanThreads) {
        int slot[4] = {-1, -1, -1, -1};
        if (t < all.x) {
            int row = 0;  // the last row that starts at or before t (rows without tokens start where the next does)
            for (int w = 1 << steps >> 1; w > 0; w >>= 1)
                if (row + w < p.B && cu[row + w] <= t) row += w;
            auto place = [&](int r, int pos) {
                const int k = pos >> p.shift;
                if (k >= p.width) return -1;
                const int have = blocks(held[r]), more = k - have;
                const int id = more < 0                        ? p.block_table[r * p.table_stride + k]
                               : more < p.num_free - take[r] ? p.free_blocks[take[r] + more]
                                                             : -1;
                return id >= 0 && id <= (INT_MAX >> p.shift) ? (id << p.shift) + (pos & (bs - 1)) : -1;
            };
            const int pos = held[row] + t - cu[row];
            if (t + 4 <= cu[row + 1] && (pos & (bs - 1)) + 4 <= bs) {
                const int s0 = place(row, pos);
#pragma unroll
                for (int j = 0; j < 4; ++j) slot[j] = s0 < 0 ? -1 : s0 + j;
                lost = lost || s0 < 0;
            } else {
                for (int j = 0; j < 4 && t + j < all.x; ++j) {
                    while (cu[row + 1] <= t + j) ++row;
                    slot[j] = place(row, held[row] + t + j - cu[row]);
                    lost = lost || slot[j] < 0;
                }
            }
        }
        if (wide && t + 4 <= p.tokens) {
            *reinterpret_cast<int4 *>(p.slot_map + t) = make_int4(slot[0], slot[1], slot[2], slot[3]);
        } else {
            for (int j = 0; j < 4 && t + j < p.tokens; ++j) p.slot_map[t + j] = slot[j];
        }
    }
    if (__any_sync(0xffffffffu, lost) && lane == 0) atomicOr(p.err, ERR_CACHE_FULL);
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
// four finite bf16 values times a power of two -> four codes.  int8 rounds by adding 1.5 * 2^23: the sum's low byte is
// the integer nearest the product (exact, at most 127), ties to even.
template <bool FP8>
__device__ __forceinline__ uint32_t encode4(uint2 x, float inv)
{
    const float2 a = unpack_bf16(x.x), b = unpack_bf16(x.y), i2 = make_float2(inv, inv);
    if constexpr (!FP8) {
        const float2 magic = make_float2(12582912.f, 12582912.f);
        const float2 u = fma2(a, i2, magic), v = fma2(b, i2, magic);
        const uint32_t lo = __byte_perm(__float_as_uint(u.x), __float_as_uint(u.y), 0x0040);
        const uint32_t hi = __byte_perm(__float_as_uint(v.x), __float_as_uint(v.y), 0x0040);
        return __byte_perm(lo, hi, 0x5410);
    } else {
        const float2 u = mul2(a, i2), v = mul2(b, i2);
        return encode4<FP8>(u.x, u.y, v.x, v.y);
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
// at `window` tokens and, for each leader among them, stores the run's tokens of 8 / WPU (head, k or v) units, WPU
// warps a unit, 16 tokens a warp at a time.  With many tokens windows are as long as a block (most tokens follow a
// leader) and WPU = BS / 16: a warp's 16 tokens stay in registers between the maximum and the rounding, and every
// input byte is read once.  With few tokens (each may lead its own block) a window is one token and WPU = 1, so
// that no warp is without a token; a longer run is then read twice.  Bound by HBM for prompts (2 bytes in, 1 out per
// element), by the latency of slot, scale, row and store for one token per request.
template <bool FP8, int D, int BS, int WPU>
__global__ void __launch_bounds__(kAppendThreads, 3) kda_cache_append_kernel(const CacheAppendParams p)
{
    constexpr int UNITS = 8 / WPU, CHUNKS = BS / 16 / WPU;        // units of a CTA; 16-token pieces of a warp
    constexpr int LPT = D / 4, TPS = 32 / LPT, STEPS = 16 / TPS;  // lanes of a token, tokens of a step
    __shared__ uint32_t tops[8];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, sub = lane / LPT;
    const int groups = (2 * p.HKV + UNITS - 1) / UNITS;
    const int64_t t0 = static_cast<int64_t>(blockIdx.x / groups) * p.window;
    const int unit = (blockIdx.x % groups) * UNITS + warp / WPU, ws = warp % WPU;
    const bool live = unit < 2 * p.HKV;
    const int kv = unit & 1, h = min(unit >> 1, p.HKV - 1);
    const int64_t stride = kv ? p.stride[1] : p.stride[0];
    const __nv_bfloat16 *in = (kv ? p.x[1] : p.x[0]) + h * D + 4 * (lane % LPT);
    uint8_t *cache = kv ? p.cache[1] : p.cache[0];
    float *scale = kv ? p.scale[1] : p.scale[0];
    const int slots = p.num_blocks * BS;
    const int64_t t_end = min(t0 + p.window, static_cast<int64_t>(p.T));
    // the leaders among 32 tokens at a time
    uint32_t leads = 0;
    int s_lane = -1;
    int64_t base = t0 - 32;
    for (;;) {
        while (leads == 0) {
            base += 32;
            if (base >= t_end) return;
            const int64_t at = base + lane;
            s_lane = at < t_end ? p.slots[at] : -1;
            int before = __shfl_up_sync(0xffffffffu, s_lane, 1);
            if (lane == 0) before = base > 0 ? p.slots[base - 1] : -1;
            if (s_lane >= slots) {
                if (blockIdx.x % groups == 0 && warp == 0) atomicOr(p.err, ERR_BLOCK_ID);
                s_lane = -1;
            }
            leads = __ballot_sync(0xffffffffu, s_lane >= 0 && (before < 0 || before / BS != s_lane / BS));
        }
        const int bit = __ffs(leads) - 1;
        leads &= leads - 1;
        const int64_t t = base + bit;
        const int lead = __shfl_sync(0xffffffffu, s_lane, bit);
        const int blk = lead / BS, first = lead % BS;  // tokens of the block before the run are kept
        float *sp = scale + static_cast<int64_t>(blk) * p.HKV + h;
        const float was = first > 0 ? *sp : 0.f;
        // 16 tokens of the run from its token 16 * piece on: this lane's offset in the block, or -1 behind the run
        bool whole = true;
        auto offsets = [&](int piece) {
            const int64_t at = t + 16 * piece + lane;
            const int s = whole && lane < 16 && at < p.T ? p.slots[at] : -1;
            const uint32_t m = __ballot_sync(0xffffffffu, s >= 0 && s / BS == blk) & 0xffffu;
            const int n = whole ? __ffs(~m) - 1 : 0;
            whole = n == 16;
            return lane < n ? s % BS : -1;
        };
        // a whole piece of consecutive slots needs no lookups
        auto straight = [&](int off) {
            const int o0 = __shfl_sync(0xffffffffu, off, 0);
            return __all_sync(0xffffffffu, lane >= 16 || (off >= 0 && off == o0 + lane)) != 0;
        };
        uint2 x[STEPS];
        auto load = [&](int piece, int off) {
            const __nv_bfloat16 *src = in + (t + 16 * piece + sub) * stride;
            if (straight(off)) {
#pragma unroll
                for (int i = 0; i < STEPS; ++i, src += TPS * stride)
                    x[i] = live ? *reinterpret_cast<const uint2 *>(src) : make_uint2(0u, 0u);
                return;
            }
#pragma unroll
            for (int i = 0; i < STEPS; ++i, src += TPS * stride) {
                const int o = __shfl_sync(0xffffffffu, off, i * TPS + sub);
                x[i] = make_uint2(0u, 0u);
                if (live && o >= 0) x[i] = *reinterpret_cast<const uint2 *>(src);
            }
        };
        // largest |x| as bits (those of non-negative bf16 order as integers)
        int off = -1, pieces = 0;
        uint32_t top2 = 0;
        for (int w = 0; w < ws; ++w) offsets(w);
#pragma unroll 1
        for (int c = 0; c < CHUNKS; ++c) {
            const int o = offsets(c * WPU + ws);
            if (c > 0 && !__any_sync(0xffffffffu, o >= 0)) break;
            load(c * WPU + ws, o);
            off = o;
            pieces = c + 1;
#pragma unroll
            for (int i = 0; i < STEPS; ++i)
                top2 = __vmaxu2(top2, __vmaxu2(x[i].x & 0x7fff7fffu, x[i].y & 0x7fff7fffu));
            if (!whole) break;
        }
        uint32_t top = __reduce_max_sync(0xffffffffu, max(top2 & 0xffffu, top2 >> 16));
        const bool fine = top < 0x7f80u;
        const bool again = CHUNKS > 1 && pieces > 1;  // only the last piece's rows are still in registers
        if (!fine) {  // infinities and NaN do not count
            top = 0;
            whole = true;
            for (int w = 0; w < ws; ++w) offsets(w);
#pragma unroll 1
            for (int c = 0; c < CHUNKS; ++c) {
                const int o16 = offsets(c * WPU + ws);
#pragma unroll 1
                for (int k = sub; k < 16; k += TPS) {
                    if (__shfl_sync(0xffffffffu, o16, k) < 0) continue;
                    const uint2 v = *reinterpret_cast<const uint2 *>(in + (t + 16 * (c * WPU + ws) + k) * stride);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const uint32_t a = ((e & 2 ? v.y : v.x) >> (16 * (e & 1))) & 0x7fffu;
                        if (a < 0x7f80u) top = max(top, a);
                    }
                }
                if (!whole) break;
            }
            top = __reduce_max_sync(0xffffffffu, top);
        }
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
#pragma unroll 4
            for (int k = ws * TPS + sub; k < first; k += WPU * TPS) {
                uint32_t *c = reinterpret_cast<uint32_t *>(dst + k * D);
                const float4 v = decode4<FP8>(*c);
                *c = encode4<FP8>(v.x * r, v.y * r, v.z * r, v.w * r);
            }
        }
        const float inv = 1.f / s;
        auto store = [&](int o16) {
            if (straight(o16)) {
                uint8_t *row = dst + (__shfl_sync(0xffffffffu, o16, 0) + sub) * D;
#pragma unroll
                for (int i = 0; i < STEPS; ++i)
                    *reinterpret_cast<uint32_t *>(row + i * TPS * D) = encode4<FP8>(x[i], inv);
                return;
            }
#pragma unroll
            for (int i = 0; i < STEPS; ++i) {
                const int o = __shfl_sync(0xffffffffu, o16, i * TPS + sub);
                if (o >= 0) *reinterpret_cast<uint32_t *>(dst + o * D) = encode4<FP8>(x[i], inv);
            }
        };
        if (!fine) {  // token by token
            whole = true;
            for (int w = 0; w < ws; ++w) offsets(w);
#pragma unroll 1
            for (int c = 0; c < CHUNKS; ++c) {
                const int o16 = offsets(c * WPU + ws);
#pragma unroll 1
                for (int k = sub; k < 16; k += TPS) {
                    const int o = __shfl_sync(0xffffffffu, o16, k);
                    if (o < 0) continue;
                    const uint2 v = *reinterpret_cast<const uint2 *>(in + (t + 16 * (c * WPU + ws) + k) * stride);
                    *reinterpret_cast<uint32_t *>(dst + o * D) =
                        encode4<FP8>(bf16lo(v.x) * inv, bf16hi(v.x) * inv, bf16lo(v.y) * inv, bf16hi(v.y) * inv);
                }
                if (!whole) break;
            }
        } else if (!again) {
            store(off);
        } else {
            whole = true;
#pragma unroll 1
            for (int c = 0; c < CHUNKS; ++c) {
                const int o = offsets(c);
                load(c, o);
                store(o);
                if (!whole) break;
            }
        }
        if (ws == 0 && lane == 0) *sp = s;
    }
}

}  // namespace kda
