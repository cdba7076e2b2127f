// Matrix products of the head and the experts: C = alpha * A B with 16-bit
// operands and fp32 sums, plain or grouped by expert.
#include "train.h"

namespace muon {
namespace {

constexpr int TS = 64;  // tile rows and columns
constexpr int TK = 16;

__device__ __forceinline__ int64_t clamped_offset(const TrainGemm& g, int64_t e) {
    const int64_t n = g.group == GROUP_M ? g.M : g.K;
    const int64_t o = load_index(g.offsets, g.offsets64, e);
    return o < 0 ? 0 : o > n ? n : o;
}

// Range [lo, hi) of group e.  GROUP_M has two more, e = -1 and e = groups:
// the rows before the first and after the last, whose products are zeros.
__device__ __forceinline__ void group_range(const TrainGemm& g, int64_t e, int64_t* lo, int64_t* hi) {
    *lo = e < 0 ? 0 : clamped_offset(g, e);
    *hi = e >= g.groups ? g.M : clamped_offset(g, e + 1);
    if (*hi < *lo) *hi = *lo;
}

template <int DT>
__device__ __forceinline__ float ld(const void* p, int64_t i) {
    return Elem<DT>::load(static_cast<const typename Elem<DT>::T*>(p)[i]);
}

template <int DT>
__global__ void __launch_bounds__(256) gemm_kernel(const TrainGemm g) {
    __shared__ float sa[TK][TS + 1], sb[TK][TS + 1];
    if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0 && g.status) *g.status = 0;
    int64_t row0 = static_cast<int64_t>(blockIdx.y) * TS, rows_end = g.M, k_lo = 0, k_hi = g.K;
    int64_t b_off = 0, c_off = 0;
    if (g.group == GROUP_M) {
        int64_t tile = blockIdx.y, e = -1, lo = 0, hi = 0;
        for (; e <= g.groups; ++e) {
            group_range(g, e, &lo, &hi);
            const int64_t n = (hi - lo + TS - 1) / TS;
            if (tile < n) break;
            tile -= n;
        }
        if (e > g.groups) return;
        row0 = lo + tile * TS;
        rows_end = hi;
        if (e < 0 || e == g.groups) k_hi = 0;
        else b_off = e * g.b_stride;
    } else if (g.group == GROUP_K) {
        const int64_t tm = (g.M + TS - 1) / TS;
        const int64_t e = blockIdx.y / tm;
        row0 = (blockIdx.y - e * tm) * TS;
        group_range(g, e, &k_lo, &k_hi);
        c_off = e * g.c_stride;
    }
    const int64_t col0 = static_cast<int64_t>(blockIdx.x) * TS;
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    float acc[4][4] = {};
    for (int64_t k0 = k_lo; k0 < k_hi; k0 += TK) {
        for (int i = threadIdx.x; i < TS * TK; i += 256) {
            const int ka = g.a_mn ? i / TS : i % TK, ma = g.a_mn ? i % TS : i / TK;
            const int kb = g.b_mn ? i / TS : i % TK, nb = g.b_mn ? i % TS : i / TK;
            const int64_t m = row0 + ma, n = col0 + nb;
            sa[ka][ma] = m < rows_end && k0 + ka < k_hi
                             ? ld<DT>(g.A, g.a_mn ? (k0 + ka) * g.lda + m : m * g.lda + k0 + ka) : 0.f;
            sb[kb][nb] = n < g.N && k0 + kb < k_hi
                             ? ld<DT>(g.B, b_off + (g.b_mn ? (k0 + kb) * g.ldb + n : n * g.ldb + k0 + kb)) : 0.f;
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < TK; ++k)
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[i][j] += sa[k][ty * 4 + i] * sb[k][tx * 4 + j];
        __syncthreads();
    }
    const float alpha = g.alpha_dev ? g.alpha * *g.alpha_dev : g.alpha;
    for (int i = 0; i < 4; ++i)
        for (int j = 0; j < 4; ++j) {
            const int64_t m = row0 + ty * 4 + i, n = col0 + tx * 4 + j;
            if (m >= rows_end || n >= g.N) continue;
            const int64_t at = c_off + m * g.ldc + n;
            const float v = alpha * acc[i][j];
            if (g.c_dtype == MUON_F32) {
                float* c = static_cast<float*>(g.C) + at;
                *c = g.accumulate ? *c + v : v;
            } else if (g.c_dtype == MUON_BF16) {
                static_cast<__nv_bfloat16*>(g.C)[at] = __float2bfloat16_rn(v);
            } else {
                static_cast<__half*>(g.C)[at] = __float2half_rn(v);
            }
        }
}

__global__ void pack_kernel(const uint16_t* src, int64_t src_ld, uint16_t* dst, int64_t dst_ld, int64_t rows,
                            int64_t cols) {
    for (int64_t r = blockIdx.x; r < rows; r += gridDim.x)
        for (int64_t c = threadIdx.x; c < cols; c += blockDim.x) dst[r * dst_ld + c] = src[r * src_ld + c];
}

}  // namespace

cudaError_t train_gemm(const TrainGemm& g, int num_sms, cudaStream_t st) {
    int64_t ty = (g.M + TS - 1) / TS;
    if (g.group == GROUP_M) ty += g.groups + 2;
    if (g.group == GROUP_K) ty *= g.groups;
    const dim3 grid(static_cast<unsigned>((g.N + TS - 1) / TS), static_cast<unsigned>(ty));
    launch_begin(g.kind, st);
    if (g.dtype == MUON_BF16) gemm_kernel<MUON_BF16><<<grid, 256, 0, st>>>(g);
    else gemm_kernel<MUON_F16><<<grid, 256, 0, st>>>(g);
    launch_end(g.kind, st);
    return cudaGetLastError();
}

cudaError_t launch_pack(const void* src, int64_t src_ld, void* dst, int64_t dst_ld, int64_t rows, int64_t cols,
                        int num_sms, cudaStream_t st) {
    const int grid = static_cast<int>(rows < num_sms * 8 ? rows : num_sms * 8);
    launch_begin(MUON_KERNEL_PACK, st);
    pack_kernel<<<grid, 256, 0, st>>>(static_cast<const uint16_t*>(src), src_ld, static_cast<uint16_t*>(dst), dst_ld,
                                      rows, cols);
    launch_end(MUON_KERNEL_PACK, st);
    return cudaGetLastError();
}

}  // namespace muon
