// kda_attn_api.cuh -- C ABI of the softmax-attention operators (declared in
// include/kda_prefill.h): host-side argument checks, tensor maps, launches.
#pragma once
#include "kda_attn_backward.cuh"
#include "kda_attn_forward.cuh"

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
    p.slots = block_slots<kAttnFwdRows>(d.N, T, d.packed);
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
    const int grid = p.slots * H;
    auto launch = [&](auto kern, int smem) {
        if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
            return KDA_ERR_CUDA;
        kern<<<grid, kAttnFwdThreads, smem, static_cast<cudaStream_t>(stream)>>>(p, mq, mk, mv);
        return cudaGetLastError() == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
    };
    return D == 128 ? launch(kda_attn_fwd_kernel<128>, AttnFwdSmem<128>::TOTAL)
                    : launch(kda_attn_fwd_kernel<64>, AttnFwdSmem<64>::TOTAL);
}

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
    p.kslots = block_slots<AT>(d.N, Tk, d.packed);
    p.scale = scale;
    p.scale_log2 = scale * kLog2e;
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
    if (d.rows && (!attn_map(&mq, q, H, d.rows, q_row_stride, D) || !attn_map(&mdo, dout, H, d.rows, dout_row_stride, D)))
        return KDA_ERR_CUDA;
    if (d.krows && (!attn_map(&mk, k, HKV, d.krows, k_row_stride, D) || !attn_map(&mv, v, HKV, d.krows, v_row_stride, D)))
        return KDA_ERR_CUDA;
    // a side without rows: the kernels write zeros to the other side's gradients and load nothing
    if (!d.rows) mq = mdo = mk;
    if (!d.krows) mk = mv = mq;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    auto run = [&](auto stats, auto dkv, int dkv_smem, auto dqk, int dq_smem) {
        if (cudaFuncSetAttribute(dkv, cudaFuncAttributeMaxDynamicSharedMemorySize, dkv_smem) != cudaSuccess ||
            cudaFuncSetAttribute(dqk, cudaFuncAttributeMaxDynamicSharedMemorySize, dq_smem) != cudaSuccess)
            return KDA_ERR_CUDA;
        if (d.rows) stats<<<p.qslots * H, kAttnStatThreads, 0, s>>>(p);
        if (d.krows) dkv<<<p.kslots * HKV, kAttnBwdThreads, dkv_smem, s>>>(p, mq, mk, mv, mdo);
        if (d.rows) dqk<<<p.qslots * H, kAttnBwdThreads, dq_smem, s>>>(p, mq, mk, mv, mdo);
        return cudaGetLastError() == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
    };
    return D == 128 ? run(kda_attn_stats_kernel<128>, kda_attn_dkv_kernel<128>, AttnDkvSmem<128>::TOTAL,
                          kda_attn_dq_kernel<128>, AttnDqSmem<128>::TOTAL)
                    : run(kda_attn_stats_kernel<64>, kda_attn_dkv_kernel<64>, AttnDkvSmem<64>::TOTAL,
                          kda_attn_dq_kernel<64>, AttnDqSmem<64>::TOTAL);
}
