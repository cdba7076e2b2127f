// Softmax cross entropy of the head, row by row: the targets' logits, the
// loss and the normaliser from the logits tiles' sums, and the logits'
// gradient.
//
//   lse = ln sum_v exp z_v;  loss = lse - z_target
//   g_v = r (exp(z_v - lse) - [v == target])
//
// The target's logit is a plain fp32 dot product, apart from the tensor
// cores, and the tiles' sums leave its column out: a trained model's loss is
// the difference of a normaliser that the target's logit dominates and that
// same logit, and the tensor core's accumulator truncates (2e-6 of the result
// at 2048 terms against 4e-7 for fp32 sums).
#include <math.h>

#include "train.h"

namespace muon {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// (top, sum) pairs of disjoint column sets; an infinite top is not subtracted.
__device__ __forceinline__ float2 join(float2 a, float2 b) {
    const float m = fmaxf(a.x, b.x);
    const float ref = isinf(m) ? 0.f : m;
    const float sa = a.x == -INFINITY ? a.y : a.y * exp2_fast((isinf(a.x) ? 0.f : a.x) - ref);
    const float sb = b.x == -INFINITY ? b.y : b.y * exp2_fast((isinf(b.x) ? 0.f : b.x) - ref);
    return make_float2(m, sa + sb);
}

// One warp per token.
template <int DT>
__global__ void __launch_bounds__(256) ce_prepare_kernel(const CeBlock b) {
    typedef typename Elem<DT>::T T;
    pdl_wait_then_release();
    const int lane = threadIdx.x & 31;
    for (int64_t t = blockIdx.x * 8 + (threadIdx.x >> 5); t < b.tokens; t += gridDim.x * 8) {
        const int64_t target = load_index(b.targets, b.targets64, t);
        const bool inside = target >= 0 && target < b.vocab;
        const T* h = static_cast<const T*>(b.hidden) + t * b.hidden_ld;
        const T* w = static_cast<const T*>(b.weight) + (inside ? target : 0) * b.weight_ld;
        T* copy = static_cast<T*>(b.packed) + t * b.packed_ld;
        float s = 0.f;
        for (int64_t c = lane; c < b.dim; c += 32) {
            const T x = h[c];
            if (b.packed) copy[c] = x;
            s = fmaf(Elem<DT>::load(x), Elem<DT>::load(w[c]), s);
        }
        for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        if (lane == 0) {
            b.z_target[t] = inside ? b.logit_scale * s : -INFINITY;
            if (!inside && target != b.ignore_index) *b.status = MUON_ERR_INVALID_ARG;
        }
    }
}

// 32 tokens per CTA, one per lane; the warps share the column tiles.
__global__ void __launch_bounds__(1024) ce_finish_kernel(const CeBlock b) {
    __shared__ float2 part[32][32];
    pdl_wait_then_release();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t t = blockIdx.x * int64_t(32) + lane;
    float2 acc = make_float2(-INFINITY, 0.f);
    if (t < b.tokens)
        for (int64_t i = warp; i < b.col_tiles; i += 32) acc = join(acc, b.sums[i * b.tokens + t]);
    part[warp][lane] = acc;
    __syncthreads();
    if (warp != 0 || t >= b.tokens) return;
    for (int i = 1; i < 32; ++i) acc = join(acc, part[i][lane]);
    const int64_t target = load_index(b.targets, b.targets64, t);
    const bool inside = target >= 0 && target < b.vocab;
    const float zt = b.z_target[t];
    if (inside) acc = join(acc, make_float2(zt * kLog2e, isnan(zt) ? zt : 1.f));
    const float lse2 = (isinf(acc.x) ? 0.f : acc.x) + log2f(acc.y);
    const float lse = lse2 * kLn2;
    b.lse2[t] = lse2;
    b.lse[t] = lse;
    b.loss[t] = inside && target != b.ignore_index ? lse - zt : 0.f;
}

constexpr int kRowThreads = 512;

// One CTA per token.
template <int DT>
__global__ void __launch_bounds__(kRowThreads) ce_grad_rows_kernel(const CeBlock b) {
    typedef typename Elem<DT>::T TG;
    pdl_wait_then_release();
    const int64_t t = blockIdx.x;
    float* z = b.Z + t * b.z_ld;
    TG* g = reinterpret_cast<TG*>(z);
    const int64_t target = load_index(b.targets, b.targets64, t);
    const bool live = target >= 0 && target < b.vocab && target != b.ignore_index;
    const float top = *b.scale_max;
    const float scale = ce_grad_lift(DT) * (b.row_scale ? (top > 0.f ? b.row_scale[t] / top : 0.f) : 1.f);
    const float c2 = b.logit_scale * kLog2e, lse2 = b.lse2[t];
    const float pt = exp2_fast(b.z_target[t] * kLog2e - lse2);
    for (int64_t v0 = 0; v0 < b.vocab; v0 += kRowThreads) {
        const int64_t v = v0 + threadIdx.x;
        const float x = v < b.vocab ? z[v] : 0.f;
        __syncthreads();  // the row's reads stay ahead of its writes, which take half the space
        float d = v == target ? pt - 1.f : exp2_fast(fmaf(x, c2, -lse2));
        d = live ? scale * d : 0.f;
        if (v < b.vocab) g[v] = Elem<DT>::store(d);
    }
    if (!live)
        for (int64_t c = threadIdx.x; c < b.dim; c += kRowThreads)
            static_cast<TG*>(b.packed)[t * b.packed_ld + c] = Elem<DT>::store(0.f);
}

__global__ void ce_scale_kernel(const float* row_scale, int64_t tokens, float mult, float* out, int* status) {
    __shared__ float red[32];
    pdl_wait_then_release();
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
    pdl_wait_then_release();
    for (int64_t i = blockIdx.x * int64_t(blockDim.x) + threadIdx.x; i < n; i += int64_t(gridDim.x) * blockDim.x)
        dst[i] = Elem<DT>::store(src[i]);
}

}  // namespace

cudaError_t launch_ce_prepare(const CeBlock& b, int num_sms, cudaStream_t st) {
    const int64_t blocks = (b.tokens + 7) / 8;
    const dim3 grid(static_cast<unsigned>(blocks < num_sms * 8 ? blocks : num_sms * 8));
    launch_begin(MUON_KERNEL_CE_ROWS, st);
    const cudaError_t e = launch_pdl(b.dtype == MUON_BF16 ? ce_prepare_kernel<MUON_BF16> : ce_prepare_kernel<MUON_F16>,
                                     grid, dim3(256), 0, st, b);
    launch_end(MUON_KERNEL_CE_ROWS, st);
    return e;
}

cudaError_t launch_ce_finish(const CeBlock& b, cudaStream_t st) {
    launch_begin(MUON_KERNEL_CE_ROWS, st);
    const cudaError_t e =
        launch_pdl(ce_finish_kernel, dim3(static_cast<unsigned>((b.tokens + 31) / 32)), dim3(1024), 0, st, b);
    launch_end(MUON_KERNEL_CE_ROWS, st);
    return e;
}

cudaError_t launch_ce_grad_rows(const CeBlock& b, cudaStream_t st) {
    launch_begin(MUON_KERNEL_CE_ROWS, st);
    const cudaError_t e =
        launch_pdl(b.dtype == MUON_BF16 ? ce_grad_rows_kernel<MUON_BF16> : ce_grad_rows_kernel<MUON_F16>,
                   dim3(static_cast<unsigned>(b.tokens)), dim3(kRowThreads), 0, st, b);
    launch_end(MUON_KERNEL_CE_ROWS, st);
    return e;
}

cudaError_t launch_ce_scale(const float* row_scale, int64_t tokens, float mult, float* out, int* status,
                            cudaStream_t st) {
    launch_begin(MUON_KERNEL_CE_ROWS, st);
    const cudaError_t e = launch_pdl(ce_scale_kernel, dim3(1), dim3(1024), 0, st, row_scale, tokens, mult, out, status);
    launch_end(MUON_KERNEL_CE_ROWS, st);
    return e;
}

cudaError_t launch_round(const float* src, void* dst, int dtype, int64_t n, int num_sms, cudaStream_t st) {
    launch_begin(MUON_KERNEL_CE_ROWS, st);
    cudaError_t e;
    if (dtype == MUON_BF16)
        e = launch_pdl(round_kernel<MUON_BF16>, dim3(num_sms * 8), dim3(256), 0, st, src,
                       static_cast<__nv_bfloat16*>(dst), n);
    else
        e = launch_pdl(round_kernel<MUON_F16>, dim3(num_sms * 8), dim3(256), 0, st, src, static_cast<__half*>(dst), n);
    launch_end(MUON_KERNEL_CE_ROWS, st);
    return e;
}

}  // namespace muon
