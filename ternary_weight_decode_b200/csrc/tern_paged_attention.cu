// tern_paged_attention.cu -- attention over the paged 8-bit KV cache.
//
// out = sum_j softmax_j(scale q . k_j) v_j, one pass over the tokens with the
// running maximum m and sum z of the softmax: a new maximum m' scales what was
// summed before by exp(m - m').
#include "tern_paged.cuh"

namespace tern {

namespace {

constexpr int kAttnThreads = 128;

__device__ __forceinline__ float code_value(uint8_t c, int kind) {
    if (kind == TERN_KV_INT8) return static_cast<float>(static_cast<int8_t>(c));
    return __half2float(__half(__nv_cvt_fp8_to_halfraw(c, __NV_E4M3)));
}

// A warp per (row, query head), four dimensions a lane.
__global__ void __launch_bounds__(kAttnThreads)
    attn_paged_kernel(PagedView v, const float *q, int ldq, int Hq, int window, int sinks, float scale, float *out,
                      int ldo) {
    extern __shared__ int32_t starts[];
    const int tid = threadIdx.x, lane = tid & 31;
    pdl_wait();
    for (int i = tid; i <= v.B; i += kAttnThreads) starts[i] = v.row_start[i];
    __syncthreads();
    const int64_t u = static_cast<int64_t>(blockIdx.x) * (kAttnThreads / 32) + (tid >> 5);
    const int64_t row = u / Hq;
    const int b = row < v.T ? row_sequence(starts, v.B, static_cast<int>(row)) : -1;
    if (b >= 0) {
        const int t = static_cast<int>(row), h = static_cast<int>(u - row * Hq);
        const int g = h / (Hq / v.Hkv);
        const int tok = v.ctx[b] - starts[b + 1] + t;
        const float4 qv = *reinterpret_cast<const float4 *>(q + static_cast<int64_t>(t) * ldq + h * kPD + 4 * lane);
        const float qs[4] = {qv.x * scale, qv.y * scale, qv.z * scale, qv.w * scale};
        float m = -INFINITY, z = 0.0f, acc[4] = {};
        const int low = window > 0 ? max(0, tok - window + 1) : 0;
        for (int j = 0; j <= tok; ++j) {
            if (window > 0 && j >= sinks && j < low) j = low;
            const int64_t bi0 = block_index(v, b, j / kPB);
            if (bi0 < 0) {
                j = (j / kPB) * kPB + kPB - 1;
                if (j >= v.pages_ld * static_cast<int64_t>(v.page_size)) break;
                continue;
            }
            const int64_t bi = bi0 + static_cast<int64_t>(g) * v.bpp;
            const int64_t at = (bi * kPB + j % kPB) * kPD + 4 * lane;
            const uint32_t kw = *reinterpret_cast<const uint32_t *>(v.kc + at);
            const uint32_t vw = *reinterpret_cast<const uint32_t *>(v.vc + at);
            const float ks = v.ks[bi], vs = v.vs[bi];
            float d = 0.0f;
#pragma unroll
            for (int e = 0; e < 4; ++e) d = fmaf(qs[e], code_value(static_cast<uint8_t>(kw >> (8 * e)), v.kind), d);
            const float x = warp_sum(d) * ks;
            const float mn = fmaxf(m, x);
            const float r = m == -INFINITY ? 0.0f : expf(m - mn), w = expf(x - mn);
            z = z * r + w;
            m = mn;
#pragma unroll
            for (int e = 0; e < 4; ++e)
                acc[e] = fmaf(w * vs, code_value(static_cast<uint8_t>(vw >> (8 * e)), v.kind), acc[e] * r);
        }
        const float iz = z > 0.0f ? 1.0f / z : 0.0f;
        *reinterpret_cast<float4 *>(out + static_cast<int64_t>(t) * ldo + h * kPD + 4 * lane) =
            make_float4(acc[0] * iz, acc[1] * iz, acc[2] * iz, acc[3] * iz);
    }
    pdl_launch_dependents();
}

}  // namespace

size_t attention_paged_workspace_bytes(int Hq, int Hkv, int num_sms) {
    (void)Hq;
    (void)Hkv;
    (void)num_sms;
    return 16;
}

cudaError_t launch_attention_paged(const PagedAttentionLaunch &A, cudaStream_t s) {
    const int64_t warps = static_cast<int64_t>(A.batch.T) * A.Hq;
    return launch_pdl(attn_paged_kernel, dim3(static_cast<unsigned>(ceil_div(warps, kAttnThreads / 32))), kAttnThreads,
                      static_cast<size_t>(A.batch.B + 1) * sizeof(int32_t), s, paged_view(A.batch, A.cache), A.q, A.ldq,
                      A.Hq, A.window, A.sinks, A.scale, A.out, A.ldo);
}

}  // namespace tern
