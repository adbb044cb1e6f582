// kda_attn_api.cuh -- C ABI of the softmax-attention operators (declared in
// include/kda_prefill.h): host-side argument checks, tensor maps, launches.
#pragma once
#include "kda_attn_backward.cuh"
#include "kda_attn_decode.cuh"
#include "kda_attn_forward.cuh"
#include "kda_cache.cuh"

namespace {

// Bytes that `rows` rows of `inner` elements, `stride` elements apart, span.
size_t span(int64_t rows, int64_t stride, int64_t inner, int elem)
{
    return rows <= 0 ? 0 : (static_cast<size_t>(rows - 1) * stride + inner) * elem;
}

struct Range {
    const void *p;
    size_t n;
};
// Whether any of the outputs overlaps an input or another output.
template <int NO, int NI>
bool outputs_overlap(const Range (&out)[NO], const Range (&in)[NI])
{
    for (int i = 0; i < NO; ++i) {
        for (int j = 0; j < NI; ++j)
            if (overlaps(out[i].p, out[i].n, in[j].p, in[j].n)) return true;
        for (int j = i + 1; j < NO; ++j)
            if (overlaps(out[i].p, out[i].n, out[j].p, out[j].n)) return true;
    }
    return false;
}

// [rows][heads][D] bf16 with a row stride as a 3D tiled map; a box is 64 columns of 128 rows of one head.
bool attn_map(CUtensorMap *m, const void *base, int heads, int64_t rows, int64_t row_stride, int D)
{
    auto enc = tensor_map_encoder();
    if (!enc) return false;
    cuuint64_t dims[3] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(heads), static_cast<cuuint64_t>(rows)};
    cuuint64_t strides[2] = {static_cast<cuuint64_t>(D) * 2, static_cast<cuuint64_t>(row_stride) * 2};
    cuuint32_t box[3] = {64, 1, static_cast<cuuint32_t>(kda::AT)};
    cuuint32_t estr[3] = {1, 1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(base), dims, strides, box, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

struct AttnDims {
    int B, T, Tk, H, HKV, D, N;
    bool packed;
    int64_t rows, krows;
};

// Sizes of an attention over whole prompts; `rows` rows of queries and `krows` of keys in all.
kda_status_t attn_dims(int B, int T, int Tk, int H, int HKV, int D, float scale, const int32_t *cu, const int32_t *cu_k,
                       int num_seqs, AttnDims &d)
{
    if (B <= 0 || T < 0 || Tk < 0 || H <= 0 || HKV <= 0 || H % HKV != 0) return KDA_ERR_INVALID_ARG;
    if (!(scale > 0.f) || scale > 3e38f) return KDA_ERR_INVALID_ARG;
    if (D != 64 && D != 128) return KDA_ERR_UNSUPPORTED;
    const bool packed = cu != nullptr;
    if (packed != (cu_k != nullptr) || packed != (num_seqs > 0)) return KDA_ERR_INVALID_ARG;
    if (packed && B != 1) return KDA_ERR_INVALID_ARG;
    if (!aligned(cu, 4) || !aligned(cu_k, 4)) return KDA_ERR_MISALIGNED;
    d = AttnDims{B, T, Tk, H, HKV, D, packed ? num_seqs : B, packed, static_cast<int64_t>(B) * T,
                 static_cast<int64_t>(B) * Tk};
    // token rows are TMA coordinates (int32); grids and row indices stay below 2^31
    if (d.rows > INT_MAX - 1024 || d.krows > INT_MAX - 1024) return KDA_ERR_UNSUPPORTED;
    const int64_t slots = std::max(d.rows, d.krows) / kda::AT + d.N;
    if (slots * H > INT_MAX) return KDA_ERR_UNSUPPORTED;
    return KDA_OK;
}

// A strided [rows][heads][D] bf16 operand.
kda_status_t check_rows(const void *p, int64_t rows, int64_t stride, int64_t inner)
{
    if (rows == 0) return KDA_OK;
    if (!p || stride < inner) return KDA_ERR_INVALID_ARG;
    if (!aligned(p, 16) || stride % 8 || stride >= (1ll << 38)) return KDA_ERR_MISALIGNED;
    return KDA_OK;
}

}  // namespace

extern "C" kda_status_t kda_attention_forward(const void *q, int64_t q_row_stride, const void *k, int64_t k_row_stride,
                                              const void *v, int64_t v_row_stride, const int32_t *cu_seqlens,
                                              const int32_t *cu_seqlens_k, int num_seqs, int B, int T, int Tk, int H,
                                              int HKV, int D, float scale, void *o, float *lse, void *stream)
{
    AttnDims d;
    kda_status_t st = attn_dims(B, T, Tk, H, HKV, D, scale, cu_seqlens, cu_seqlens_k, num_seqs, d);
    if (st != KDA_OK) return st;
    if (d.rows == 0) return KDA_OK;
    const int64_t wq = static_cast<int64_t>(H) * D, wk = static_cast<int64_t>(HKV) * D;
    if ((st = check_rows(q, d.rows, q_row_stride, wq)) != KDA_OK ||
        (st = check_rows(k, d.krows, k_row_stride, wk)) != KDA_OK ||
        (st = check_rows(v, d.krows, v_row_stride, wk)) != KDA_OK)
        return st;
    if (!o || !lse) return KDA_ERR_INVALID_ARG;
    if (!aligned(o, 16) || !aligned(lse, 4)) return KDA_ERR_MISALIGNED;
    const size_t ncu = static_cast<size_t>(d.N + 1) * 4;
    const Range out[] = {{o, span(d.rows, wq, wq, 2)}, {lse, static_cast<size_t>(d.rows) * H * 4}};
    const Range in[] = {{q, span(d.rows, q_row_stride, wq, 2)}, {k, span(d.krows, k_row_stride, wk, 2)},
                        {v, span(d.krows, v_row_stride, wk, 2)}, {cu_seqlens, ncu}, {cu_seqlens_k, ncu}};
    if (outputs_overlap(out, in)) return KDA_ERR_INVALID_ARG;

    DeviceInfo info;
    if (device_info(info) != cudaSuccess) return KDA_ERR_CUDA;
    using namespace kda;
    AttnFwdParams p{};
    p.seq = SeqView{cu_seqlens, cu_seqlens_k, d.N, T, Tk};
    p.H = H;
    p.HKV = HKV;
    p.scale = scale;
    p.scale_log2 = scale * kLog2e;
    p.o = static_cast<__nv_bfloat16 *>(o);
    p.lse = lse;
    p.err = info.err;
    CUtensorMap mq, mk, mv;
    if (!attn_map(&mq, q, H, d.rows, q_row_stride, D)) return KDA_ERR_CUDA;
    if (d.krows == 0) {
        mk = mv = mq;  // no key tile is loaded
    } else if (!attn_map(&mk, k, HKV, d.krows, k_row_stride, D) || !attn_map(&mv, v, HKV, d.krows, v_row_stride, D)) {
        return KDA_ERR_CUDA;
    }
    const int grid = block_slots<kAttnFwdRows>(d.N, T, d.packed) * H;
    auto launch = [&](auto kern, int smem) {
        if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
            return KDA_ERR_CUDA;
        kern<<<grid, kAttnFwdThreads, smem, static_cast<cudaStream_t>(stream)>>>(p, mq, mk, mv);
        return cudaGetLastError() == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
    };
    return D == 128 ? launch(kda_attn_fwd_kernel<128>, AttnFwdSmem<128>::TOTAL)
                    : launch(kda_attn_fwd_kernel<64>, AttnFwdSmem<64>::TOTAL);
}

namespace {

// CTAs (a cluster) that share the query heads of a key tile: until there are twice as many as SMs.  With fewer a key
// tile's loop over all heads of its group is the longest chain there is; with more the clusters cost more than they
// balance (D = 128, 32/8 heads; us per backward with 1, 2 and 4 CTAs):
//   512 tokens (32 key tiles): 53, 47, 41    1,024 (64): 110, 80, 80    2,048 (128): 182, 150, 172
// 16/4 heads, 4,096 tokens (128): 307, 219, 250, and 8,192 (256): 762, 782, 860; 8/1 heads, 2,048 tokens (16 key tiles): 240,
// 176, 108 and, with 8, 76.
int backward_split(int group, int64_t units, int sms)
{
    int split = 1;
    while (split < 8 && group % (2 * split) == 0 && split * units <= sms) split *= 2;
    return split;
}

}  // namespace

extern "C" size_t kda_attention_backward_workspace_size(int B, int T, int H, int num_seqs)
{
    if (B <= 0 || T < 0 || H <= 0 || num_seqs < 0 || (num_seqs > 0 && B != 1)) return 0;
    const int64_t slots = num_seqs > 0 ? static_cast<int64_t>(T) / kda::AT + num_seqs
                                       : static_cast<int64_t>(B) * ((static_cast<int64_t>(T) + kda::AT - 1) / kda::AT);
    return static_cast<size_t>(slots) * H * 2 * kda::AT * sizeof(float);
}

extern "C" kda_status_t kda_attention_backward(const void *q, int64_t q_row_stride, const void *k, int64_t k_row_stride,
                                               const void *v, int64_t v_row_stride, const void *o, const float *lse,
                                               const void *dout, int64_t dout_row_stride, const int32_t *cu_seqlens,
                                               const int32_t *cu_seqlens_k, int num_seqs, int B, int T, int Tk, int H,
                                               int HKV, int D, float scale, void *dq, void *dk, void *dv,
                                               void *workspace, size_t workspace_bytes, void *stream)
{
    AttnDims d;
    kda_status_t st = attn_dims(B, T, Tk, H, HKV, D, scale, cu_seqlens, cu_seqlens_k, num_seqs, d);
    if (st != KDA_OK) return st;
    const int64_t wq = static_cast<int64_t>(H) * D, wk = static_cast<int64_t>(HKV) * D;
    if ((st = check_rows(q, d.rows, q_row_stride, wq)) != KDA_OK ||
        (st = check_rows(k, d.krows, k_row_stride, wk)) != KDA_OK ||
        (st = check_rows(v, d.krows, v_row_stride, wk)) != KDA_OK || (st = check_rows(o, d.rows, wq, wq)) != KDA_OK ||
        (st = check_rows(dout, d.rows, dout_row_stride, wq)) != KDA_OK)
        return st;
    if ((d.rows && (!lse || !dq || !workspace)) || (d.krows && (!dk || !dv))) return KDA_ERR_INVALID_ARG;
    if (!aligned(lse, 4) || !aligned(dq, 16) || !aligned(dk, 16) || !aligned(dv, 16) || !aligned(workspace, 16))
        return KDA_ERR_MISALIGNED;
    const size_t need = kda_attention_backward_workspace_size(B, T, H, num_seqs);
    if (d.rows && workspace_bytes < need) return KDA_ERR_WORKSPACE;
    const size_t ncu = static_cast<size_t>(d.N + 1) * 4, nq = span(d.rows, wq, wq, 2), nk = span(d.krows, wk, wk, 2);
    const Range out[] = {{dq, nq}, {dk, nk}, {dv, nk}, {workspace, need}};
    const Range in[] = {{q, span(d.rows, q_row_stride, wq, 2)}, {k, span(d.krows, k_row_stride, wk, 2)},
                        {v, span(d.krows, v_row_stride, wk, 2)}, {o, nq},
                        {lse, static_cast<size_t>(d.rows) * H * 4}, {dout, span(d.rows, dout_row_stride, wq, 2)},
                        {cu_seqlens, ncu}, {cu_seqlens_k, ncu}};
    if (outputs_overlap(out, in)) return KDA_ERR_INVALID_ARG;
    if (d.rows == 0 && d.krows == 0) return KDA_OK;

    DeviceInfo info;
    if (device_info(info) != cudaSuccess) return KDA_ERR_CUDA;
    using namespace kda;
    AttnBwdParams p{};
    p.seq = SeqView{cu_seqlens, cu_seqlens_k, d.N, T, Tk};
    p.H = H;
    p.HKV = HKV;
    p.qslots = block_slots<AT>(d.N, T, d.packed);
    const int64_t kunits = static_cast<int64_t>(block_slots<AT>(d.N, Tk, d.packed)) * HKV;  // key tiles of all heads
    p.scale = scale;
    p.scale_log2 = scale * kLog2e;
    p.q = static_cast<const __nv_bfloat16 *>(q);
    p.k = static_cast<const __nv_bfloat16 *>(k);
    p.v = static_cast<const __nv_bfloat16 *>(v);
    p.q_stride = q_row_stride;
    p.k_stride = k_row_stride;
    p.v_stride = v_row_stride;
    p.o = static_cast<const __nv_bfloat16 *>(o);
    p.dout = static_cast<const __nv_bfloat16 *>(dout);
    p.do_stride = dout_row_stride;
    p.lse = lse;
    p.stats = static_cast<float *>(workspace);
    p.dq = static_cast<__nv_bfloat16 *>(dq);
    p.dk = static_cast<__nv_bfloat16 *>(dk);
    p.dv = static_cast<__nv_bfloat16 *>(dv);
    p.err = info.err;
    CUtensorMap mq, mk, mv, mdo;
    if (d.rows && (!attn_map(&mq, q, H, d.rows, q_row_stride, D) ||
                   !attn_map(&mdo, dout, H, d.rows, dout_row_stride, D)))
        return KDA_ERR_CUDA;
    if (d.krows && (!attn_map(&mk, k, HKV, d.krows, k_row_stride, D) ||
                    !attn_map(&mv, v, HKV, d.krows, v_row_stride, D)))
        return KDA_ERR_CUDA;
    // a side without rows: the kernels write zeros to the other side's gradients and load nothing
    if (!d.rows) mq = mdo = mk;
    if (!d.krows) mk = mv = mq;
    p.split = backward_split(H / HKV, kunits, info.sms);
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    // a launch is set up while the one before it ends, where SMs are idle
    auto launch = [&](auto kern, int64_t grid, int smem, int cluster, bool early) {
        if (grid > INT_MAX) return KDA_ERR_UNSUPPORTED;
        if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
            return KDA_ERR_CUDA;
        cudaLaunchConfig_t cfg{};
        cfg.gridDim = dim3(static_cast<unsigned>(grid));
        cfg.blockDim = dim3(kAttnBwdThreads);
        cfg.dynamicSmemBytes = smem;
        cfg.stream = s;
        cudaLaunchAttribute attr[2]{};
        cfg.attrs = attr;
        if (early) {
            attr[cfg.numAttrs].id = cudaLaunchAttributeProgrammaticStreamSerialization;
            attr[cfg.numAttrs++].val.programmaticStreamSerializationAllowed = 1;
        }
        if (cluster > 1) {
            attr[cfg.numAttrs].id = cudaLaunchAttributeClusterDimension;
            attr[cfg.numAttrs].val.clusterDim.x = cluster;
            attr[cfg.numAttrs].val.clusterDim.y = attr[cfg.numAttrs].val.clusterDim.z = 1;
            ++cfg.numAttrs;
        }
        return cudaLaunchKernelEx(&cfg, kern, p, mq, mk, mv, mdo) == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
    };
    auto run = [&](auto stats, auto dkv, int dkv_smem, auto dqk, int dq_smem) {
        kda_status_t r = KDA_OK;
        if (d.rows) {
            const int64_t grid = (static_cast<int64_t>(p.qslots) + d.N) * H;
            if (grid > INT_MAX) return KDA_ERR_UNSUPPORTED;
            stats<<<static_cast<int>(grid), kAttnStatThreads, 0, s>>>(p);
            if (cudaGetLastError() != cudaSuccess) return KDA_ERR_CUDA;
        }
        if (d.rows) r = launch(dqk, static_cast<int64_t>(p.qslots) * H, dq_smem, 1, true);
        if (r == KDA_OK && d.krows)
            r = launch(dkv, kunits * p.split, dkv_smem, p.split, d.rows > 0);
        return r;
    };
    return D == 128 ? run(kda_attn_stats_kernel<128>, kda_attn_dkv_kernel<128>, AttnDkvSmem<128>::TOTAL,
                          kda_attn_dq_kernel<128>, AttnDqSmem<128>::TOTAL)
                    : run(kda_attn_stats_kernel<64>, kda_attn_dkv_kernel<64>, AttnDkvSmem<64>::TOTAL,
                          kda_attn_dq_kernel<64>, AttnDqSmem<64>::TOTAL);
}

// ---------------------------------------------------------------------------------------------- the 8-bit cache
namespace {

// log2 of a cache's block size, or -1.
int block_shift(int block_size)
{
    return block_size == 16 ? 4 : block_size == 32 ? 5 : block_size == 64 ? 6 : block_size == 128 ? 7 : -1;
}

kda_status_t cache_dims(int code_type, int num_blocks, int block_size, int HKV, int D, int64_t block_stride)
{
    if (num_blocks <= 0 || HKV <= 0 || block_size <= 0) return KDA_ERR_INVALID_ARG;
    if ((code_type != KDA_CACHE_E4M3 && code_type != KDA_CACHE_INT8) || block_shift(block_size) < 0 ||
        (D != 64 && D != 128))
        return KDA_ERR_UNSUPPORTED;
    const int64_t block = static_cast<int64_t>(HKV) * block_size * D;
    if (block_stride < block) return KDA_ERR_INVALID_ARG;
    // slots and the rows of a block are int32
    if (static_cast<int64_t>(num_blocks) * block_size > INT_MAX || block > INT_MAX) return KDA_ERR_UNSUPPORTED;
    if (block_stride % 16 || block_stride >= (1ll << 39)) return KDA_ERR_MISALIGNED;
    return KDA_OK;
}

// The codes as a 3D map: D bytes, the rows of a block, the blocks; a box is `rows` rows of one block.
bool cache_map(CUtensorMap *m, const void *base, int D, int block_rows, int num_blocks, int64_t block_stride, int rows)
{
    auto enc = tensor_map_encoder();
    if (!enc) return false;
    cuuint64_t dims[3] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(block_rows),
                          static_cast<cuuint64_t>(num_blocks)};
    cuuint64_t strides[2] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(block_stride)};
    cuuint32_t box[3] = {static_cast<cuuint32_t>(D), static_cast<cuuint32_t>(rows), 1};
    cuuint32_t estr[3] = {1, 1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void *>(base), dims, strides, box, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE, D == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

extern "C" kda_status_t kda_cache_plan(const int32_t *context_lens, const int32_t *new_lens, int B,
                                       int32_t *block_table, int64_t table_stride, int table_width,
                                       const int32_t *free_blocks, int num_free, int block_size, int32_t *cu_seqlens,
                                       int32_t *seq_lens, int32_t *slot_map, int num_tokens, int32_t *used,
                                       void *stream)
{
    if (B <= 0 || table_width <= 0 || num_free < 0 || num_tokens < 0) return KDA_ERR_INVALID_ARG;
    const int shift = block_shift(block_size);
    // (the kernel's token index goes a step, 2,048 tokens a CTA, past the last token)
    if (shift < 0 || B > kda::kPlanMaxRows || num_tokens > INT_MAX - (1 << 20)) return KDA_ERR_UNSUPPORTED;
    if (table_stride < table_width) return KDA_ERR_INVALID_ARG;
    if (!context_lens || !new_lens || !block_table || (num_free && !free_blocks) || !cu_seqlens || !seq_lens ||
        (num_tokens && !slot_map) || !used)
        return KDA_ERR_INVALID_ARG;
    for (const void *p : {static_cast<const void *>(context_lens), static_cast<const void *>(new_lens),
                          static_cast<const void *>(block_table), static_cast<const void *>(free_blocks),
                          static_cast<const void *>(cu_seqlens), static_cast<const void *>(seq_lens),
                          static_cast<const void *>(slot_map), static_cast<const void *>(used)})
        if (!aligned(p, 4)) return KDA_ERR_MISALIGNED;
    const size_t nb = static_cast<size_t>(B) * 4;
    const Range out[] = {{block_table, span(B, table_stride, table_width, 4)}, {cu_seqlens, nb + 4}, {seq_lens, nb},
                         {slot_map, static_cast<size_t>(num_tokens) * 4}, {used, 4}};
    const Range in[] = {{context_lens, nb}, {new_lens, nb}, {free_blocks, static_cast<size_t>(num_free) * 4}};
    if (outputs_overlap(out, in)) return KDA_ERR_INVALID_ARG;
    DeviceInfo info;
    if (device_info(info) != cudaSuccess) return KDA_ERR_CUDA;
    using namespace kda;
    const CachePlanParams p{context_lens, new_lens, block_table, free_blocks, cu_seqlens, seq_lens,  slot_map, used,
                            table_stride, B,        table_width, num_free,    num_tokens, shift,     info.err};
    // enough CTAs for four tokens a thread, or a warp per 4 rows, up to one CTA per SM
    const int64_t want = std::max<int64_t>((num_tokens + 4ll * kPlanThreads - 1) / (4 * kPlanThreads), (B + 63) / 64);
    const int grid = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(want, info.sms)));
    const int smem = (3 * B + 1) * 4;
    if (cudaFuncSetAttribute(kda_cache_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
        return KDA_ERR_CUDA;
    kda_cache_plan_kernel<<<grid, kPlanThreads, smem, static_cast<cudaStream_t>(stream)>>>(p);
    return cudaGetLastError() == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

extern "C" kda_status_t kda_cache_append(const void *k, int64_t k_row_stride, const void *v, int64_t v_row_stride,
                                         void *k_cache, void *v_cache, int64_t block_stride, float *k_scale,
                                         float *v_scale, int code_type, int num_blocks, int block_size,
                                         const int32_t *slot_map, int T, int HKV, int D, void *stream)
{
    if (T < 0) return KDA_ERR_INVALID_ARG;
    kda_status_t st = cache_dims(code_type, num_blocks, block_size, HKV, D, block_stride);
    if (st != KDA_OK) return st;
    if (T == 0) return KDA_OK;
    const int64_t w = static_cast<int64_t>(HKV) * D;
    if ((st = check_rows(k, T, k_row_stride, w)) != KDA_OK || (st = check_rows(v, T, v_row_stride, w)) != KDA_OK)
        return st;
    if (!k_cache || !v_cache || !k_scale || !v_scale || !slot_map) return KDA_ERR_INVALID_ARG;
    if (!aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(k_scale, 4) || !aligned(v_scale, 4) ||
        !aligned(slot_map, 4))
        return KDA_ERR_MISALIGNED;
    const size_t pool = span(num_blocks, block_stride, w * block_size, 1), ns = static_cast<size_t>(num_blocks) * HKV * 4;
    // k_cache and v_cache may interleave (one pool of [block][k, v]), but not at the same place
    const int64_t apart = static_cast<const char *>(v_cache) - static_cast<const char *>(k_cache);
    const int64_t block = w * block_size, gap = ((apart % block_stride) + block_stride) % block_stride;
    if (overlaps(k_cache, pool, v_cache, pool) && (gap < block || gap > block_stride - block)) return KDA_ERR_INVALID_ARG;
    const Range caches[] = {{k_cache, pool}, {v_cache, pool}};
    const Range out[] = {{k_scale, ns}, {v_scale, ns}};
    const Range in[] = {{k, span(T, k_row_stride, w, 2)}, {v, span(T, v_row_stride, w, 2)},
                        {slot_map, static_cast<size_t>(T) * 4}};
    if (outputs_overlap(out, in)) return KDA_ERR_INVALID_ARG;
    for (const Range &c : caches) {
        for (const Range &r : in)
            if (overlaps(c.p, c.n, r.p, r.n)) return KDA_ERR_INVALID_ARG;
        for (const Range &r : out)
            if (overlaps(c.p, c.n, r.p, r.n)) return KDA_ERR_INVALID_ARG;
    }
    DeviceInfo info;
    if (device_info(info) != cudaSuccess) return KDA_ERR_CUDA;
    using namespace kda;
    CacheAppendParams p{};
    p.x[0] = static_cast<const __nv_bfloat16 *>(k);
    p.x[1] = static_cast<const __nv_bfloat16 *>(v);
    p.stride[0] = k_row_stride;
    p.stride[1] = v_row_stride;
    p.cache[0] = static_cast<uint8_t *>(k_cache);
    p.cache[1] = static_cast<uint8_t *>(v_cache);
    p.block_stride = block_stride;
    p.scale[0] = k_scale;
    p.scale[1] = v_scale;
    p.slots = slot_map;
    p.T = T;
    p.HKV = HKV;
    p.num_blocks = num_blocks;
    p.err = info.err;
    // Windows as small as leaves 32 CTAs for each SM at most (3 fit at a time): one token for a step of requests, a
    // block for prompts.  256 single tokens (8 heads, blocks of 64): 6 us with one warp a unit, 14 with four; prompts
    // of 95,000 tokens (blocks of 16, where both are the same) do not differ.
    const int wpu = block_size / 16;
    const int64_t wide = (2ll * HKV * wpu + 7) / 8;  // CTAs of a run with BS / 16 warps a unit
    const int64_t fits = T * wide / (32ll * info.sms);
    p.window = static_cast<int>(std::min<int64_t>(block_size, std::max<int64_t>(1, fits)));
    const bool few = p.window == 1;
    const int64_t grid = (T + p.window - 1ll) / p.window * (few ? (2ll * HKV + 7) / 8 : wide);
    if (grid > INT_MAX) return KDA_ERR_UNSUPPORTED;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    auto go = [&](auto fp8, auto d) {
        constexpr bool F = decltype(fp8)::value;
        constexpr int DD = decltype(d)::value;
        auto run = [&](auto kern) { kern<<<static_cast<int>(grid), kAppendThreads, 0, s>>>(p); };
        auto pick = [&](auto one, auto wide) { few ? run(one) : run(wide); };
        if (block_size == 16) run(kda_cache_append_kernel<F, DD, 16, 1>);
        else if (block_size == 32) pick(kda_cache_append_kernel<F, DD, 32, 1>, kda_cache_append_kernel<F, DD, 32, 2>);
        else if (block_size == 64) pick(kda_cache_append_kernel<F, DD, 64, 1>, kda_cache_append_kernel<F, DD, 64, 4>);
        else pick(kda_cache_append_kernel<F, DD, 128, 1>, kda_cache_append_kernel<F, DD, 128, 8>);
    };
    using D64 = std::integral_constant<int, 64>;
    using D128 = std::integral_constant<int, 128>;
    if (code_type == KDA_CACHE_E4M3) D == 128 ? go(std::true_type{}, D128{}) : go(std::true_type{}, D64{});
    else D == 128 ? go(std::false_type{}, D128{}) : go(std::false_type{}, D64{});
    return cudaGetLastError() == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

namespace {

// Query heads of a unit, and the most CTAs that a decode step uses, whatever the device.
int decode_heads(int H, int HKV) { return H / HKV <= 8 ? 8 : 16; }
int64_t decode_ctas(int B, int H, int HKV, int D, int table_width, int block_size)
{
    const int64_t hb = decode_heads(H, HKV), chunks = (H / HKV + hb - 1) / hb;
    const int64_t tiles = (static_cast<int64_t>(table_width) * block_size + kda::ad_tile(D) - 1) / kda::ad_tile(D);
    const int64_t row = HKV * chunks;  // each factor may be near 2^31
    return tiles >= kda::kAdMaxCtas || row >= kda::kAdMaxCtas ? kda::kAdMaxCtas
                                                              : std::min<int64_t>(kda::kAdMaxCtas, B * (tiles * row));
}
size_t decode_part_bytes(int64_t ctas, int H, int HKV, int D)
{
    return round_up(static_cast<size_t>(ctas) * 2 * decode_heads(H, HKV) * (D + 2) * 4, kAlign);
}

}  // namespace

extern "C" size_t kda_attention_decode_workspace_size(int B, int H, int HKV, int D, int table_width, int block_size)
{
    if (B <= 0 || H <= 0 || HKV <= 0 || H % HKV || (D != 64 && D != 128) || table_width <= 0 ||
        block_shift(block_size) < 0)
        return 0;
    const int64_t ctas = decode_ctas(B, H, HKV, D, table_width, block_size);
    return decode_part_bytes(ctas, H, HKV, D) + round_up(static_cast<size_t>(ctas) * 2 * sizeof(int4), kAlign);
}

extern "C" kda_status_t kda_attention_decode(const void *q, int64_t q_row_stride, const void *k_cache,
                                             const void *v_cache, int64_t block_stride, const float *k_scale,
                                             const float *v_scale, int code_type, int num_blocks, int block_size,
                                             const int32_t *block_table, int64_t table_stride, int table_width,
                                             const int32_t *seq_lens, int B, int H, int HKV, int D, float scale,
                                             void *o, float *lse, void *workspace, size_t workspace_bytes, void *stream)
{
    if (B < 0 || H <= 0 || HKV <= 0 || H % HKV != 0 || table_width <= 0 || !(scale > 0.f) || scale > 3e38f)
        return KDA_ERR_INVALID_ARG;
    kda_status_t st = cache_dims(code_type, num_blocks, block_size, HKV, D, block_stride);
    if (st != KDA_OK) return st;
    if (B == 0) return KDA_OK;
    if (static_cast<int64_t>(B) * H > INT_MAX) return KDA_ERR_UNSUPPORTED;
    const int64_t wq = static_cast<int64_t>(H) * D;
    if ((st = check_rows(q, B, q_row_stride, wq)) != KDA_OK) return st;
    if (!k_cache || !v_cache || !k_scale || !v_scale || !block_table || !seq_lens || !o || !lse ||
        table_stride < table_width)
        return KDA_ERR_INVALID_ARG;
    const size_t need = kda_attention_decode_workspace_size(B, H, HKV, D, table_width, block_size);
    if (!workspace || workspace_bytes < need) return KDA_ERR_WORKSPACE;
    if (!aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(k_scale, 4) || !aligned(v_scale, 4) ||
        !aligned(block_table, 4) || !aligned(seq_lens, 4) || !aligned(o, 16) || !aligned(lse, 4) ||
        !aligned(workspace, 16))
        return KDA_ERR_MISALIGNED;
    const size_t pool = span(num_blocks, block_stride, static_cast<int64_t>(HKV) * block_size * D, 1);
    const size_t ns = static_cast<size_t>(num_blocks) * HKV * 4;
    const Range out[] = {{o, span(B, wq, wq, 2)}, {lse, static_cast<size_t>(B) * H * 4}, {workspace, need}};
    const Range in[] = {{q, span(B, q_row_stride, wq, 2)}, {k_cache, pool}, {v_cache, pool}, {k_scale, ns},
                        {v_scale, ns}, {block_table, span(B, table_stride, table_width, 4)},
                        {seq_lens, static_cast<size_t>(B) * 4}};
    if (outputs_overlap(out, in)) return KDA_ERR_INVALID_ARG;
    DeviceInfo info;
    if (device_info(info) != cudaSuccess) return KDA_ERR_CUDA;
    using namespace kda;
    const int hb = decode_heads(H, HKV);
    const int64_t ctas = decode_ctas(B, H, HKV, D, table_width, block_size);
    AttnDecodeParams p{};
    p.q = static_cast<const __nv_bfloat16 *>(q);
    p.q_stride = q_row_stride;
    p.kscale = k_scale;
    p.vscale = v_scale;
    p.table = block_table;
    p.table_stride = table_stride;
    p.lens = seq_lens;
    p.o = static_cast<__nv_bfloat16 *>(o);
    p.lse = lse;
    p.part = static_cast<float *>(workspace);
    p.shared_unit = reinterpret_cast<int4 *>(static_cast<char *>(workspace) + decode_part_bytes(ctas, H, HKV, D));
    p.err = info.err;
    p.B = B;
    p.H = H;
    p.HKV = HKV;
    p.chunks = (H / HKV + hb - 1) / hb;
    p.width = table_width;
    p.num_blocks = num_blocks;
    p.scale_log2 = scale * kLog2e;
    const int rows = std::min(block_size, ad_tile(D)), shift = block_shift(block_size);
    CUtensorMap mk, mv;
    if (!cache_map(&mk, k_cache, D, HKV * block_size, num_blocks, block_stride, rows) ||
        !cache_map(&mv, v_cache, D, HKV * block_size, num_blocks, block_stride, rows))
        return KDA_ERR_CUDA;
    const int grid = static_cast<int>(std::min<int64_t>(ctas, static_cast<int64_t>(info.sms) * ad_ctas(hb / 8)));
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    // few short requests: a cluster per unit
    const int64_t units = static_cast<int64_t>(B) * HKV * p.chunks;
    const bool clusters = units * kAdCluster <= static_cast<int64_t>(info.sms) * ad_ctas(hb / 8) &&
                          static_cast<int64_t>(table_width) * block_size <= kAdClusterTiles * ad_tile(D);
    auto launch = [&](auto kern, int blocks, int threads, int smem, cudaLaunchAttribute attr, auto... args) {
        if (smem && cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
            return KDA_ERR_CUDA;
        cudaLaunchConfig_t cfg{};
        cfg.gridDim = dim3(blocks);
        cfg.blockDim = dim3(threads);
        cfg.dynamicSmemBytes = smem;
        cfg.stream = s;
        cfg.attrs = &attr;
        cfg.numAttrs = attr.id == cudaLaunchAttributeIgnore ? 0 : 1;
        return cudaLaunchKernelEx(&cfg, kern, p, args...) == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
    };
    auto go = [&](auto fp8, auto d, auto nt) {
        constexpr bool F = decltype(fp8)::value;
        constexpr int DD = decltype(d)::value, N = decltype(nt)::value;
        constexpr int smem = AttnDecodeSmem<DD, N>::TOTAL;
        cudaLaunchAttribute attr{};
        attr.id = cudaLaunchAttributeIgnore;
        if (clusters) {
            attr.id = cudaLaunchAttributeClusterDimension;
            attr.val.clusterDim.x = kAdCluster;
            attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
            return launch(kda_attn_decode_kernel<F, DD, N, true>, static_cast<int>(units * kAdCluster), kAdThreads, smem,
                          attr, mk, mv, shift);
        }
        kda_status_t r = launch(kda_attn_decode_kernel<F, DD, N, false>, grid, kAdThreads, smem, attr, mk, mv, shift);
        if (r != KDA_OK) return r;
        // the join waits for the pieces on the device (griddepcontrol.wait), so its launch overlaps the step
        attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr.val.programmaticStreamSerializationAllowed = 1;
        return launch(kda_attn_decode_join_kernel<DD, N>, grid, kAdJoinThreads, 0, attr);
    };
    using D64 = std::integral_constant<int, 64>;
    using D128 = std::integral_constant<int, 128>;
    using N1 = std::integral_constant<int, 1>;
    using N2 = std::integral_constant<int, 2>;
    auto by_heads = [&](auto fp8, auto d) { return hb == 8 ? go(fp8, d, N1{}) : go(fp8, d, N2{}); };
    auto by_dim = [&](auto fp8) { return D == 128 ? by_heads(fp8, D128{}) : by_heads(fp8, D64{}); };
    return code_type == KDA_CACHE_E4M3 ? by_dim(std::true_type{}) : by_dim(std::false_type{});
}
