// Softmax cross entropy of the head, row by row: from a block of logits to
// the loss, the normaliser and the logits' gradient.
//
//   lse = ln sum_v exp z_v;  loss = lse - z_target
//   g_v = r (exp(z_v - lse) - [v == target])
#include <math.h>

#include "train.h"

namespace muon {
namespace {

constexpr int kRowThreads = 512;

__device__ __forceinline__ float finite_max(float m) { return isinf(m) ? 0.f : m; }

// One CTA per token.
template <int DT>
__global__ void __launch_bounds__(kRowThreads) ce_rows_kernel(const CeRows r) {
    typedef typename Elem<DT>::T TG;
    __shared__ float red_m[kRowThreads / 32], red_s[kRowThreads / 32];
    const int64_t t = blockIdx.x;
    float* z = r.Z + t * r.z_ld;
    const int64_t target = load_index(r.targets, r.targets64, t);
    const bool inside = target >= 0 && target < r.vocab;
    const bool live = inside && target != r.ignore_index;
    if (!inside && target != r.ignore_index && threadIdx.x == 0) *r.status = MUON_ERR_INVALID_ARG;
    float m = -INFINITY, s = 0.f;
    for (int64_t v = threadIdx.x; v < r.vocab; v += kRowThreads) {
        const float x = z[v] * r.logit_scale;
        if (x > m || isnan(x)) {
            s = (m == -INFINITY ? 0.f : s * expf(finite_max(m) - finite_max(x))) + expf(x - finite_max(x));
            m = x;
        } else {
            s += expf(x - finite_max(m));
        }
    }
    for (int o = 16; o > 0; o >>= 1) {
        const float m2 = __shfl_xor_sync(0xffffffffu, m, o), s2 = __shfl_xor_sync(0xffffffffu, s, o);
        const float n = fmaxf(m, m2);
        s = (m == -INFINITY ? 0.f : s * expf(finite_max(m) - finite_max(n))) +
            (m2 == -INFINITY ? 0.f : s2 * expf(finite_max(m2) - finite_max(n)));
        m = n;
    }
    if ((threadIdx.x & 31) == 0) {
        red_m[threadIdx.x >> 5] = m;
        red_s[threadIdx.x >> 5] = s;
    }
    __syncthreads();
    m = -INFINITY;
    for (int i = 0; i < kRowThreads / 32; ++i) m = fmaxf(m, red_m[i]);
    s = 0.f;
    for (int i = 0; i < kRowThreads / 32; ++i)
        if (red_m[i] != -INFINITY) s += red_s[i] * expf(finite_max(red_m[i]) - finite_max(m));
    const float lse = finite_max(m) + logf(s);
    if (threadIdx.x == 0) {
        r.lse[t] = lse;
        r.loss[t] = live ? lse - z[target] * r.logit_scale : 0.f;
    }
    if (!r.with_grad) return;
    const float top = r.scale_max ? *r.scale_max : 1.f;
    const float scale = ce_grad_lift(DT) * (r.row_scale ? (top > 0.f ? r.row_scale[t] / top : 0.f) : 1.f);
    TG* g = reinterpret_cast<TG*>(z);
    for (int64_t v0 = 0; v0 < r.vocab; v0 += kRowThreads) {
        const int64_t v = v0 + threadIdx.x;
        __syncthreads();
        float x = v < r.vocab ? z[v] * r.logit_scale : 0.f;
        __syncthreads();  // the row's reads stay ahead of its writes, which take half the space
        x = live ? scale * (expf(x - lse) - (v == target ? 1.f : 0.f)) : 0.f;
        if (v < r.vocab) g[v] = Elem<DT>::store(x);
    }
    if (!live)
        for (int64_t c = threadIdx.x; c < r.dim; c += kRowThreads)
            static_cast<TG*>(r.hidden)[t * r.hidden_ld + c] = Elem<DT>::store(0.f);
}

__global__ void ce_scale_kernel(const float* row_scale, int64_t tokens, float mult, float* out, int* status) {
    __shared__ float red[32];
    float m = row_scale ? 0.f : 1.f;
    if (row_scale)
        for (int64_t t = threadIdx.x; t < tokens; t += blockDim.x) {
            const float a = fabsf(row_scale[t]);
            m = isnan(a) || a > m ? a : m;
        }
    for (int o = 16; o > 0; o >>= 1) {
        const float x = __shfl_xor_sync(0xffffffffu, m, o);
        m = isnan(x) || x > m ? x : m;
    }
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = m;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int i = 1; i < static_cast<int>(blockDim.x >> 5); ++i) m = isnan(red[i]) || red[i] > m ? red[i] : m;
        out[0] = m;
        out[1] = m * mult;
        *status = 0;
    }
}

template <int DT>
__global__ void round_kernel(const float* src, typename Elem<DT>::T* dst, int64_t n) {
    for (int64_t i = blockIdx.x * int64_t(blockDim.x) + threadIdx.x; i < n; i += int64_t(gridDim.x) * blockDim.x)
        dst[i] = Elem<DT>::store(src[i]);
}

}  // namespace

cudaError_t launch_ce_rows(const CeRows& r, cudaStream_t st) {
    launch_begin(MUON_KERNEL_CE_ROWS, st);
    const int grid = static_cast<int>(r.tokens);
    if (r.dtype == MUON_BF16) ce_rows_kernel<MUON_BF16><<<grid, kRowThreads, 0, st>>>(r);
    else ce_rows_kernel<MUON_F16><<<grid, kRowThreads, 0, st>>>(r);
    launch_end(MUON_KERNEL_CE_ROWS, st);
    return cudaGetLastError();
}

cudaError_t launch_ce_scale(const float* row_scale, int64_t tokens, float mult, float* out, int* status,
                            cudaStream_t st) {
    launch_begin(MUON_KERNEL_CE_ROWS, st);
    ce_scale_kernel<<<1, 1024, 0, st>>>(row_scale, tokens, mult, out, status);
    launch_end(MUON_KERNEL_CE_ROWS, st);
    return cudaGetLastError();
}

cudaError_t launch_round(const float* src, void* dst, int dtype, int64_t n, int num_sms, cudaStream_t st) {
    launch_begin(MUON_KERNEL_CE_ROWS, st);
    if (dtype == MUON_BF16)
        round_kernel<MUON_BF16><<<num_sms * 8, 256, 0, st>>>(src, static_cast<__nv_bfloat16*>(dst), n);
    else
        round_kernel<MUON_F16><<<num_sms * 8, 256, 0, st>>>(src, static_cast<__half*>(dst), n);
    launch_end(MUON_KERNEL_CE_ROWS, st);
    return cudaGetLastError();
}

}  // namespace muon
