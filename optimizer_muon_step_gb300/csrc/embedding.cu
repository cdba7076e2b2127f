// The embedding: rows of a table by token id, and the table's gradient.
//
//   y[t]  = scale * E[id_t]
//   dE[v] = scale * sum over t with id_t = v of dy[t]
#include "train.h"

namespace muon {
namespace {

template <int TD, int OD>
__global__ void embed_lookup_kernel(const EmbedLookup a) {
    typedef typename Elem<TD>::T TI;
    typedef typename Elem<OD>::T TO;
    for (int64_t t = blockIdx.x; t < a.tokens; t += gridDim.x) {
        const int64_t id = load_index(a.ids, a.ids64, t);
        const bool live = id >= 0 && id < a.vocab && id != a.padding_idx;
        const TI* src = static_cast<const TI*>(a.table) + (live ? id : 0) * a.table_ld;
        TO* dst = static_cast<TO*>(a.out) + t * a.out_ld;
        for (int64_t c = threadIdx.x; c < a.dim; c += blockDim.x)
            dst[c] = Elem<OD>::store(live ? a.scale * Elem<TD>::load(src[c]) : 0.f);
    }
}

// One CTA per table row: the tokens' ids are scanned in order.
template <int GD>
__global__ void embed_grad_kernel(const EmbedGrad a, int* status) {
    typedef typename Elem<GD>::T TG;
    __shared__ int list[256];
    __shared__ int found;
    const int64_t v = blockIdx.x;
    if (v == 0 && threadIdx.x == 0) *status = 0;
    bool any = false;
    for (int64_t c0 = 0; c0 < a.dim; c0 += blockDim.x) {
        const int64_t c = c0 + threadIdx.x;
        float sum = 0.f;
        any = false;
        for (int64_t t0 = 0; t0 < a.tokens; t0 += 256) {
            __syncthreads();
            if (threadIdx.x < 32) {
                int n = 0;
                for (int k = 0; k < 8; ++k) {
                    const int64_t t = t0 + 32 * k + threadIdx.x;
                    const bool hit = t < a.tokens && v != a.padding_idx && load_index(a.ids, a.ids64, t) == v;
                    const unsigned m = __ballot_sync(0xffffffffu, hit);
                    if (hit) list[n + __popc(m & ((1u << threadIdx.x) - 1))] = 32 * k + threadIdx.x;
                    n += __popc(m);
                }
                if (threadIdx.x == 0) found = n;
            }
            __syncthreads();
            any |= found > 0;
            if (c < a.dim)
                for (int i = 0; i < found; ++i)
                    sum += Elem<GD>::load(static_cast<const TG*>(a.grad)[(t0 + list[i]) * a.grad_ld + c]);
        }
        if (c < a.dim) {
            float* d = a.d_table + v * a.dim + c;
            if (a.accumulate) {
                if (any) *d += a.scale * sum;
            } else {
                *d = a.scale * sum;
            }
        }
    }
}

__global__ void embed_check_kernel(const EmbedGrad a, int* status) {
    for (int64_t t = blockIdx.x * int64_t(blockDim.x) + threadIdx.x; t < a.tokens; t += int64_t(gridDim.x) * blockDim.x) {
        const int64_t id = load_index(a.ids, a.ids64, t);
        if (id != a.padding_idx && (id < 0 || id >= a.vocab)) *status = MUON_ERR_INVALID_ARG;
    }
}

template <int TD>
void lookup_out(const EmbedLookup& a, int grid, cudaStream_t st) {
    if (a.out_dtype == MUON_F32) embed_lookup_kernel<TD, MUON_F32><<<grid, 256, 0, st>>>(a);
    else if (a.out_dtype == MUON_BF16) embed_lookup_kernel<TD, MUON_BF16><<<grid, 256, 0, st>>>(a);
    else embed_lookup_kernel<TD, MUON_F16><<<grid, 256, 0, st>>>(a);
}

}  // namespace

cudaError_t launch_embed_lookup(const EmbedLookup& a, int num_sms, cudaStream_t st) {
    const int grid = static_cast<int>(a.tokens < num_sms * 8 ? a.tokens : num_sms * 8);
    launch_begin(MUON_KERNEL_EMBED_LOOKUP, st);
    if (a.table_dtype == MUON_F32) lookup_out<MUON_F32>(a, grid, st);
    else if (a.table_dtype == MUON_BF16) lookup_out<MUON_BF16>(a, grid, st);
    else lookup_out<MUON_F16>(a, grid, st);
    launch_end(MUON_KERNEL_EMBED_LOOKUP, st);
    return cudaGetLastError();
}

size_t embed_grad_workspace(int64_t tokens, int64_t vocab, int64_t dim) { return kHeaderBytes; }

cudaError_t launch_embed_grad(const EmbedGrad& a, void* workspace, int num_sms, cudaStream_t st) {
    int* status = static_cast<int*>(workspace);
    launch_begin(MUON_KERNEL_EMBED_GRAD, st);
    const int grid = static_cast<int>(a.vocab);
    if (a.grad_dtype == MUON_F32) embed_grad_kernel<MUON_F32><<<grid, 256, 0, st>>>(a, status);
    else if (a.grad_dtype == MUON_BF16) embed_grad_kernel<MUON_BF16><<<grid, 256, 0, st>>>(a, status);
    else embed_grad_kernel<MUON_F16><<<grid, 256, 0, st>>>(a, status);
    launch_end(MUON_KERNEL_EMBED_GRAD, st);
    if (a.tokens > 0) {
        launch_begin(MUON_KERNEL_EMBED_SORT, st);
        embed_check_kernel<<<num_sms, 256, 0, st>>>(a, status);
        launch_end(MUON_KERNEL_EMBED_SORT, st);
    }
    return cudaGetLastError();
}

}  // namespace muon
