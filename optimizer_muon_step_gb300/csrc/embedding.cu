// The embedding: rows of a table by token id, and the table's gradient.
//
//   y[t]  = scale * E[id_t]
//   dE[v] = scale * sum over t with id_t = v of dy[t]
//
// The lookup moves bytes and nothing else: one warp per token and 1024
// columns, four independent 16- or 32-byte loads per lane in flight.
//
// The gradient is dense (AdamW steps the whole table), so most of its bytes
// are the rows of ids that do not occur.  The token positions are sorted by
// id first, stably, so that every row is summed in token order by one warp
// and written once; no atomic adds, and the same bits on every call.  Three
// launches up to 16384 tokens:
//   sort   the first CTA sorts, least significant digit first, ids in
//          registers; the others meanwhile write the zero rows, each for its
//          share of the table, after a look through all ids
//   sums   per 8 to 32 sorted positions and 256 columns, the sums of the runs of
//          equal ids: a run inside them goes straight to its row, the
//          pieces of one that crosses go to the workspace
//   join   the crossing runs' pieces, in order
// More tokens are sorted by several CTAs, three launches a digit, and the
// zero rows are found in the sorted ids by the launch of the sums.
#include <mutex>
#include <type_traits>

#include "train.h"

namespace muon {
namespace {

// ---------------------------------------------------------------------------
// Lookup
// ---------------------------------------------------------------------------
constexpr int kVec = 8;                      // elements of a lane's load
constexpr int kUnroll = 4;
constexpr int kSeg = 32 * kVec * kUnroll;    // columns of a warp's task

// 8 elements as they lie in memory.
template <int DT>
struct Raw8 {
    uint4 w[DT == MUON_F32 ? 2 : 1];
};

template <int DT>
__device__ __forceinline__ Raw8<DT> load_raw8(const typename Elem<DT>::T* p) {
    Raw8<DT> r;
    r.w[0] = *reinterpret_cast<const uint4*>(p);
    if constexpr (DT == MUON_F32) r.w[1] = *reinterpret_cast<const uint4*>(p + 4);
    return r;
}

template <int DT>
__device__ __forceinline__ void widen8(const Raw8<DT>& r, float (&v)[8]) {
    if constexpr (DT == MUON_F32) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            v[4 * i] = __uint_as_float(r.w[i].x);
            v[4 * i + 1] = __uint_as_float(r.w[i].y);
            v[4 * i + 2] = __uint_as_float(r.w[i].z);
            v[4 * i + 3] = __uint_as_float(r.w[i].w);
        }
    } else {
        const uint32_t w[4] = {r.w[0].x, r.w[0].y, r.w[0].z, r.w[0].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (DT == MUON_BF16) {
                v[2 * i] = __uint_as_float(w[i] << 16);
                v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
            } else {
                const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
                v[2 * i] = f.x;
                v[2 * i + 1] = f.y;
            }
        }
    }
}

template <int DT>
__device__ __forceinline__ void store8(typename Elem<DT>::T* p, const float (&v)[8]) {
    if constexpr (DT == MUON_F32) {
        __stcs(reinterpret_cast<float4*>(p), make_float4(v[0], v[1], v[2], v[3]));
        __stcs(reinterpret_cast<float4*>(p + 4), make_float4(v[4], v[5], v[6], v[7]));
    } else {
        typename Elem<DT>::T h[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) h[i] = Elem<DT>::store(v[i]);
        __stcs(reinterpret_cast<uint4*>(p), *reinterpret_cast<const uint4*>(h));
    }
}

// kWide: every row of both matrices starts on 16 bytes and has a multiple of
// 8 elements; otherwise the warp moves single elements, side by side.
template <int TD, int OD, bool kWide>
__global__ void __launch_bounds__(256) embed_lookup_kernel(const __grid_constant__ EmbedLookup a, int segs) {
    typedef typename Elem<TD>::T TI;
    typedef typename Elem<OD>::T TO;
    const int lane = threadIdx.x & 31;
    const int64_t task = blockIdx.x * int64_t(8) + (threadIdx.x >> 5);
    const int64_t t = task / segs;
    if (t >= a.tokens) return;
    const int64_t c0 = (task - t * segs) * kSeg;
    const int64_t id = load_index(a.ids, a.ids64, t);
    const bool live = id >= 0 && id < a.vocab && id != a.padding_idx;
    const TI* src = static_cast<const TI*>(a.table) + (live ? id : 0) * a.table_ld;
    TO* dst = static_cast<TO*>(a.out) + t * a.out_ld;
    if constexpr (kWide) {
        float v[kUnroll][8];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int64_t c = c0 + (u * 32 + lane) * kVec;
#pragma unroll
            for (int i = 0; i < 8; ++i) v[u][i] = 0.f;
            if (live && c < a.dim) widen8<TD>(load_raw8<TD>(src + c), v[u]);
        }
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int64_t c = c0 + (u * 32 + lane) * kVec;
#pragma unroll
            for (int i = 0; i < 8; ++i) v[u][i] = live ? a.scale * v[u][i] : 0.f;
            if (c < a.dim) store8<OD>(dst + c, v[u]);
        }
    } else {
        const int64_t end = c0 + kSeg < a.dim ? c0 + kSeg : a.dim;
#pragma unroll 8
        for (int64_t c = c0 + lane; c < end; c += 32)
            dst[c] = Elem<OD>::store(live ? a.scale * Elem<TD>::load(src[c]) : 0.f);
    }
}

template <int TD, int OD>
void lookup_go(const EmbedLookup& a, cudaStream_t st) {
    const size_t te = dtype_bytes(TD), oe = dtype_bytes(OD);
    const bool wide = a.dim % 8 == 0 && (reinterpret_cast<uintptr_t>(a.table) & 15) == 0 && a.table_ld * te % 16 == 0 &&
                      (reinterpret_cast<uintptr_t>(a.out) & 15) == 0 && a.out_ld * oe % 16 == 0;
    const int segs = static_cast<int>((a.dim + kSeg - 1) / kSeg);
    const unsigned grid = static_cast<unsigned>((a.tokens * segs + 7) / 8);
    if (wide) embed_lookup_kernel<TD, OD, true><<<grid, 256, 0, st>>>(a, segs);
    else embed_lookup_kernel<TD, OD, false><<<grid, 256, 0, st>>>(a, segs);
}

template <int TD>
void lookup_out(const EmbedLookup& a, cudaStream_t st) {
    if (a.out_dtype == MUON_F32) lookup_go<TD, MUON_F32>(a, st);
    else if (a.out_dtype == MUON_BF16) lookup_go<TD, MUON_BF16>(a, st);
    else lookup_go<TD, MUON_F16>(a, st);
}

// ---------------------------------------------------------------------------
// Sort: (key, position) pairs by key, stable.  Ids that take no gradient get
// the key `vocab`, after all others.
// ---------------------------------------------------------------------------
constexpr int kSortThreads = 1024;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kDigitBits = 9;
constexpr int kBins = 1 << kDigitBits;
constexpr int kItems = 16;                            // per thread
constexpr int kSortTile = kSortThreads * kItems;      // pairs of one CTA

struct SortArgs {
    const void* ids;
    const int32_t* keys_in;  // null in the first pass: from ids
    const int32_t* pos_in;
    int32_t* keys;
    int32_t* pos;
    uint32_t* hist;          // [bin][tile], several tiles only
    int* status;
    int64_t tokens, vocab, padding_idx;
    int32_t ids64, shift, bits, tiles;
};

// The keys of a thread's items; -1 for an id outside the table, which the
// caller turns into `vocab` once it has reported it (a store to the status
// between the loads would put them in a row).
__device__ __forceinline__ int32_t raw_key(const SortArgs& a, int64_t t) {
    const int64_t id = load_index(a.ids, a.ids64, t);
    return id == a.padding_idx ? static_cast<int32_t>(a.vocab) : id < 0 || id >= a.vocab ? -1 : static_cast<int32_t>(id);
}

__device__ __forceinline__ void settle_keys(const SortArgs& a, int32_t (&key)[kItems]) {
    bool bad = false;
#pragma unroll
    for (int r = 0; r < kItems; ++r) {
        bad |= key[r] < 0;
        if (key[r] < 0) key[r] = static_cast<int32_t>(a.vocab);
    }
    if (bad) *a.status = MUON_ERR_INVALID_ARG;
}

// Rank of each of the warp's items among those of the same digit, in order:
// warp w has items [w, w + 1) * 32 * rounds, round r the r-th 32 of them.
// Lanes of equal digit are found by one ballot per bit: __match_any_sync took
// about 300 cycles a round, the sort of 16384 ids 47 us instead of SORTUS.
__device__ __forceinline__ void warp_ranks(const int32_t (&key)[kItems], uint16_t (&rank)[kItems], int rounds, int shift,
                                           int bits, uint16_t* hist, int lane) {
    const int bins = 1 << bits;
    for (int i = lane; i < bins; i += 32) hist[i] = 0;
    __syncwarp();
#pragma unroll
    for (int r = 0; r < kItems; ++r) {
        if (r < rounds) {
            const int d = (key[r] >> shift) & (bins - 1);
            unsigned same = 0xffffffffu;
#pragma unroll
            for (int k = 0; k < kDigitBits; ++k) {
                const bool one = (d >> k) & 1;
                const unsigned m = __ballot_sync(0xffffffffu, one);
                same &= one ? m : ~m;
            }
            const int before = __popc(same & ((1u << lane) - 1));
            const int base = hist[d];
            __syncwarp();
            if (before == 0) hist[d] = static_cast<uint16_t>(base + __popc(same));
            __syncwarp();
            rank[r] = static_cast<uint16_t>(base + before);
        }
    }
}

// Turns the warps' counts into first ranks within the CTA and returns, for
// threads below `bins`, the digit's count; the digits' starts go to `start`.
__device__ __forceinline__ int scan_counts(uint16_t* hist, int bins, uint32_t* start, uint32_t* scratch) {
    int total = 0;
    if (static_cast<int>(threadIdx.x) < bins) {
#pragma unroll
        for (int w0 = 0; w0 < kSortWarps; w0 += 8) {
            int n[8];
#pragma unroll
            for (int w = 0; w < 8; ++w) n[w] = hist[(w0 + w) * kBins + threadIdx.x];
#pragma unroll
            for (int w = 0; w < 8; ++w) {
                hist[(w0 + w) * kBins + threadIdx.x] = static_cast<uint16_t>(total);
                total += n[w];
            }
        }
    }
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int incl = total;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += x;
    }
    if (lane == 31) scratch[warp] = incl;
    __syncthreads();
    int before = 0;
    for (int w = 0; w < warp; ++w) before += scratch[w];
    if (static_cast<int>(threadIdx.x) < bins) start[threadIdx.x] = before + incl - total;
    __syncthreads();
    return total;
}

struct SortShared {
    uint16_t hist[kSortWarps * kBins];
    uint32_t start[kBins];
    uint32_t scratch[kSortWarps];
    int32_t keys[kSortTile];
    uint16_t pos[kSortTile];
};

// Zeros into `cols` floats, by a warp.
__device__ __forceinline__ void zero_floats(float* p, int64_t cols, int lane) {
    const int head = static_cast<int>((4 - ((reinterpret_cast<uintptr_t>(p) >> 2) & 3)) & 3);  // to 16 bytes
    const int64_t lead = head < cols ? head : cols;
    if (lane < lead) p[lane] = 0.f;
    const int64_t quads = (cols - lead) / 4;
    float4* q = reinterpret_cast<float4*>(p + lead);
#pragma unroll 8
    for (int64_t i = lane; i < quads; i += 32) __stcs(q + i, make_float4(0.f, 0.f, 0.f, 0.f));
    const int64_t done = lead + 4 * quads;
    if (done + lane < cols) p[done + lane] = 0.f;
}

// Zeros into the rows of this CTA's share of the table that no id names: a
// bit per row in shared memory, set in one pass over the ids.
__device__ __forceinline__ void zero_share(const SortArgs& a, float* d_table, int64_t dim, uint32_t* bits) {
    const int64_t per = (a.vocab + gridDim.x - 2) / (gridDim.x - 1);
    const int64_t v0 = (blockIdx.x - 1) * per, v1 = v0 + per < a.vocab ? v0 + per : a.vocab;
    for (int64_t i = threadIdx.x; i < (per + 31) / 32; i += kSortThreads) bits[i] = 0;
    __syncthreads();
#pragma unroll 8
    for (int64_t t = threadIdx.x; t < a.tokens; t += kSortThreads) {
        const int64_t id = load_index(a.ids, a.ids64, t);
        if (id >= v0 && id < v1 && id != a.padding_idx) atomicOr(&bits[(id - v0) >> 5], 1u << ((id - v0) & 31));
    }
    __syncthreads();
    for (int64_t v = v0 + (threadIdx.x >> 5); v < v1; v += kSortWarps)
        if (!((bits[(v - v0) >> 5] >> ((v - v0) & 31)) & 1)) zero_floats(d_table + v * dim, dim, threadIdx.x & 31);
}

// All passes in the first CTA; the zero rows by the others (none when the
// gradient is accumulated).
__global__ void __launch_bounds__(kSortThreads, 1)
    sort_one_kernel(const __grid_constant__ SortArgs a, int passes, float* d_table, int64_t dim) {
    extern __shared__ __align__(16) uint8_t sort_smem[];
    SortShared& s = *reinterpret_cast<SortShared*>(sort_smem);
    pdl_wait_then_release();
    if (blockIdx.x > 0) {
        zero_share(a, d_table, dim, reinterpret_cast<uint32_t*>(sort_smem));
        return;
    }
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int n = static_cast<int>(a.tokens);
    const int rounds = (n + kSortThreads - 1) / kSortThreads;
    const int first = warp * 32 * rounds + lane;
    if (threadIdx.x == 0) *a.status = 0;
    __syncthreads();
    int32_t key[kItems];
    uint16_t pos[kItems], rank[kItems];
#pragma unroll
    for (int r = 0; r < kItems; ++r) {
        key[r] = 0x7fffffff;  // past the end: after everything, in every pass
        pos[r] = 0;
        const int i = first + 32 * r;
        if (r < rounds && i < n) {
            key[r] = raw_key(a, i);
            pos[r] = static_cast<uint16_t>(i);
        }
    }
    settle_keys(a, key);
    const int bins = 1 << a.bits;
    for (int p = 0; p < passes; ++p) {
        const int shift = p * a.bits;
        warp_ranks(key, rank, rounds, shift, a.bits, s.hist + warp * kBins, lane);
        __syncthreads();
        scan_counts(s.hist, bins, s.start, s.scratch);
#pragma unroll
        for (int r = 0; r < kItems; ++r) {
            if (r < rounds) {
                const int d = (key[r] >> shift) & (bins - 1);
                const int to = static_cast<int>(s.start[d]) + s.hist[warp * kBins + d] + rank[r];
                s.keys[to] = key[r];
                s.pos[to] = pos[r];
            }
        }
        __syncthreads();
#pragma unroll
        for (int r = 0; r < kItems; ++r) {
            if (r < rounds) {
                key[r] = s.keys[first + 32 * r];
                pos[r] = s.pos[first + 32 * r];
            }
        }
        // the next pass writes keys and pos only after two more barriers
    }
#pragma unroll
    for (int r = 0; r < kItems; ++r) {
        const int i = first + 32 * r;
        if (r < rounds && i < n) {
            a.keys[i] = key[r];
            a.pos[i] = pos[r];
        }
    }
}

// Several tiles: counts per tile, one scan over [bin][tile], stable scatter.
template <bool kScatter>
__global__ void __launch_bounds__(kSortThreads, 1) sort_tile_kernel(const __grid_constant__ SortArgs a) {
    extern __shared__ __align__(16) uint8_t sort_smem[];
    SortShared& s = *reinterpret_cast<SortShared*>(sort_smem);
    pdl_wait_then_release();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t tile0 = blockIdx.x * int64_t(kSortTile);
    const int64_t first = tile0 + warp * 32 * kItems + lane;
    int32_t key[kItems];
    uint16_t rank[kItems];
#pragma unroll
    for (int r = 0; r < kItems; ++r) {
        const int64_t i = first + 32 * r;
        key[r] = 0x7fffffff;
        if (i < a.tokens) key[r] = a.keys_in ? a.keys_in[i] : raw_key(a, i);
    }
    if (!a.keys_in) settle_keys(a, key);
    const int bins = 1 << a.bits;
    warp_ranks(key, rank, kItems, a.shift, a.bits, s.hist + warp * kBins, lane);
    __syncthreads();
    const int total = scan_counts(s.hist, bins, s.start, s.scratch);
    if constexpr (!kScatter) {
        // the pairs past the end count too: they are the last ones of the last bin
        if (static_cast<int>(threadIdx.x) < bins) a.hist[threadIdx.x * int64_t(a.tiles) + blockIdx.x] = total;
    } else {
#pragma unroll
        for (int r = 0; r < kItems; ++r) {
            const int64_t i = first + 32 * r;
            const int d = (key[r] >> a.shift) & (bins - 1);
            const int64_t to = static_cast<int64_t>(a.hist[d * int64_t(a.tiles) + blockIdx.x]) +
                               s.hist[warp * kBins + d] + rank[r];
            if (i < a.tokens) {
                a.keys[to] = key[r];
                a.pos[to] = a.pos_in ? a.pos_in[i] : static_cast<int32_t>(i);
            }
        }
    }
}

// Exclusive scan of hist in place, one CTA.
__global__ void __launch_bounds__(1024) sort_scan_kernel(uint32_t* hist, int64_t n) {
    __shared__ uint32_t sums[32];
    pdl_wait_then_release();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t per = (n + 1023) / 1024;
    const int64_t lo = threadIdx.x * per < n ? threadIdx.x * per : n, hi = lo + per < n ? lo + per : n;
    uint32_t total = 0;
    for (int64_t i = lo; i < hi; ++i) total += hist[i];
    uint32_t incl = total;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t x = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += x;
    }
    if (lane == 31) sums[warp] = incl;
    __syncthreads();
    uint32_t at = incl - total;
    for (int w = 0; w < warp; ++w) at += sums[w];
    for (int64_t i = lo; i < hi; ++i) {
        const uint32_t x = hist[i];
        hist[i] = at;
        at += x;
    }
}

// ---------------------------------------------------------------------------
// Sums
// ---------------------------------------------------------------------------
constexpr int kMaxPiece = 32;  // sorted positions of one warp's task: 8, 16 or 32, see launch_embed_grad
constexpr int kMinPiece = 8;
constexpr int kCols = 256;     // and columns: 8 per lane
constexpr int kSumWarps = 4;
constexpr int kZeroRows = 32;  // table rows of one warp's zero task
constexpr int kZeroCols = 1024;

struct SumArgs {
    const void* grad;
    const int32_t* keys;
    const int32_t* pos;
    float* parts;          // [2 * piece + slot][part_ld]: slot 0 a run that began before, 1 one that goes on
    float* d_table;
    int64_t grad_ld, part_ld, vocab, dim;
    int32_t tokens, piece, pieces, col_tasks, zero_tasks_x, accumulate;
    int32_t sum_blocks;    // blocks before the zero tasks' ones
    float scale;
};

// Columns of lane `lane`, element i of its 8.
template <bool kWide>
__device__ __forceinline__ int64_t column(int64_t c0, int lane, int i) {
    return kWide ? c0 + lane * 8 + i : c0 + i * 32 + lane;
}

template <bool kWide>
__device__ __forceinline__ void put_row(float* row, int64_t c0, int64_t dim, int lane, const float (&v)[8], float scale,
                                        bool accumulate) {
    if constexpr (kWide) {
        const int64_t c = c0 + lane * 8;
        if (c >= dim) return;
        float4* p = reinterpret_cast<float4*>(row + c);
        float4 a = make_float4(scale * v[0], scale * v[1], scale * v[2], scale * v[3]);
        float4 b = make_float4(scale * v[4], scale * v[5], scale * v[6], scale * v[7]);
        if (accumulate) {
            const float4 x = p[0], y = p[1];
            a = make_float4(x.x + a.x, x.y + a.y, x.z + a.z, x.w + a.w);
            b = make_float4(y.x + b.x, y.y + b.y, y.z + b.z, y.w + b.w);
        }
        __stcs(p, a);
        __stcs(p + 1, b);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int64_t c = column<false>(c0, lane, i);
            if (c < dim) row[c] = accumulate ? row[c] + scale * v[i] : scale * v[i];
        }
    }
}

template <int GD, bool kWide>
__device__ __forceinline__ void sum_piece(const SumArgs& a, int piece, int64_t c0, int lane) {
    typedef typename Elem<GD>::T TG;
    const TG* grad = static_cast<const TG*>(a.grad);
    const int i0 = piece * a.piece;
    const int n = a.tokens - i0 < a.piece ? a.tokens - i0 : a.piece;
    const int dead = static_cast<int>(a.vocab);
    const int key = lane < n ? a.keys[i0 + lane] : dead;
    const int pos = lane < n ? a.pos[i0 + lane] : 0;
    const int prev = i0 > 0 ? a.keys[i0 - 1] : -1;
    const int next = i0 + n < a.tokens ? a.keys[i0 + n] : -1;
    const int live = __popc(__ballot_sync(0xffffffffu, key != dead));  // dead keys sort last
    float acc[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[i] = 0.f;
    bool began = __shfl_sync(0xffffffffu, key, 0) != prev;  // the current run's first token is in this piece
    constexpr int kBatch = kWide && GD == MUON_F32 ? 4 : 8;  // tokens loaded together
    for (int j0 = 0; j0 < live; j0 += kBatch) {
        typename std::conditional<kWide, Raw8<GD>, float[8]>::type v[kBatch];
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
            const int64_t t = __shfl_sync(0xffffffffu, pos, (j0 + j) & 31);
            const TG* src = grad + t * a.grad_ld;
            if constexpr (kWide) {
                if (j0 + j < live && c0 + lane * 8 < a.dim) v[j] = load_raw8<GD>(src + c0 + lane * 8);
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) v[j][i] = 0.f;
                if (j0 + j < live) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const int64_t c = column<false>(c0, lane, i);
                        if (c < a.dim) v[j][i] = Elem<GD>::load(src[c]);
                    }
                }
            }
        }
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
            const int l = j0 + j;
            if (l < live) {
                if constexpr (kWide) {
                    float f[8];
                    widen8<GD>(v[j], f);
#pragma unroll
                    for (int i = 0; i < 8; ++i) acc[i] += f[i];
                } else {
#pragma unroll
                    for (int i = 0; i < 8; ++i) acc[i] += v[j][i];
                }
                const int k = __shfl_sync(0xffffffffu, key, l);
                const int after = l + 1 < n ? __shfl_sync(0xffffffffu, key, (l + 1) & 31) : next;
                const bool last = l + 1 == n;
                if (k != after || last) {
                    const bool ends = k != after;
                    if (began && ends) {
                        put_row<kWide>(a.d_table + static_cast<int64_t>(k) * a.dim, c0, a.dim, lane, acc, a.scale, a.accumulate);
                    } else {
                        float* part = a.parts + (2 * static_cast<int64_t>(piece) + (began ? 1 : 0)) * a.part_ld;
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const int64_t c = column<kWide>(c0, lane, i);
                            if (c < a.dim) part[c] = acc[i];
                        }
                    }
#pragma unroll
                    for (int i = 0; i < 8; ++i) acc[i] = 0.f;
                    began = true;
                }
            }
        }
    }
}

__device__ __forceinline__ int lower_bound(const int32_t* keys, int n, int64_t v) {
    int lo = 0, hi = n;
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (keys[mid] < v) lo = mid + 1;
        else hi = mid;
    }
    return lo;
}

// Zeros into the rows [v0, v0 + 32) that have no token: lane l looks for row
// v0 + l.
__device__ __forceinline__ void zero_rows(const SumArgs& a, int64_t v0, int64_t c0, int lane) {
    const int64_t v = v0 + lane;
    bool empty = false;
    if (v < a.vocab) {
        const int at = lower_bound(a.keys, a.tokens, v);
        empty = at >= a.tokens || a.keys[at] != v;
    }
    unsigned todo = __ballot_sync(0xffffffffu, empty);
    const int64_t cols = a.dim - c0 < kZeroCols ? a.dim - c0 : kZeroCols;
    while (todo) {
        const int r = __ffs(todo) - 1;
        todo &= todo - 1;
        zero_floats(a.d_table + (v0 + r) * a.dim + c0, cols, lane);
    }
}

template <int GD, bool kWide>
__global__ void __launch_bounds__(32 * kSumWarps, kWide ? 6 : 4) embed_sum_kernel(const __grid_constant__ SumArgs a) {
    pdl_wait_then_release();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (static_cast<int>(blockIdx.x) < a.sum_blocks) {
        const int64_t task = blockIdx.x * int64_t(kSumWarps) + warp;
        const int64_t piece = task / a.col_tasks;
        if (piece < a.pieces) sum_piece<GD, kWide>(a, static_cast<int>(piece), (task - piece * a.col_tasks) * kCols, lane);
    } else {
        const int64_t task = (blockIdx.x - a.sum_blocks) * int64_t(kSumWarps) + warp;
        const int64_t row = task / a.zero_tasks_x;
        if (row * kZeroRows < a.vocab) zero_rows(a, row * kZeroRows, (task - row * a.zero_tasks_x) * kZeroCols, lane);
    }
}

// The runs that cross pieces: the piece where one begins owns it.  A warp
// adds the run's pieces over 256 columns, in order; a run of more than 64
// pieces is shared by the CTA's warps, whose sums the first one adds.
template <bool kWide>
__device__ __forceinline__ void add_pieces(const SumArgs& a, int piece, int lo, int hi, int64_t c0, int lane,
                                           float (&acc)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[i] = 0.f;
#pragma unroll 8
    for (int k = lo; k < hi; ++k) {
        const float* part = a.parts + (2 * static_cast<int64_t>(piece + k) + (k == 0 ? 1 : 0)) * a.part_ld;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int64_t c = column<kWide>(c0, lane, i);
            acc[i] += c < a.dim ? part[c] : 0.f;
        }
    }
}

template <bool kWide>
__global__ void __launch_bounds__(256) embed_join_kernel(const __grid_constant__ SumArgs a) {
    __shared__ float share[8][32][9];
    pdl_wait_then_release();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int piece = blockIdx.x;
    const int start = piece * a.piece, end = start + a.piece;
    if (end >= a.tokens) return;
    const int key = a.keys[end - 1], after = a.keys[end], head = a.keys[start], before = start > 0 ? a.keys[start - 1] : -1;
    // no run crosses, or the one that does began before this piece
    if (key == static_cast<int>(a.vocab) || after != key || (head == key && before == key)) return;
    int count = 1;  // pieces of the run: those whose first key is its key
    for (;;) {
        const int64_t first = (piece + count + lane) * static_cast<int64_t>(a.piece);
        const int n = __popc(__ballot_sync(0xffffffffu, first < a.tokens && a.keys[first < a.tokens ? first : 0] == key));
        count += n;
        if (n < 32) break;
    }
    float* row = a.d_table + static_cast<int64_t>(key) * a.dim;
    float acc[8];
    if (count <= 64) {
        const int64_t c0 = (blockIdx.y * int64_t(8) + warp) * kCols;
        if (c0 >= a.dim) return;
        add_pieces<kWide>(a, piece, 0, count, c0, lane, acc);
        put_row<kWide>(row, c0, a.dim, lane, acc, a.scale, a.accumulate);
        return;
    }
    const int per = (count + 7) / 8;
    for (int s = 0; s < 8; ++s) {
        const int64_t c0 = (blockIdx.y * int64_t(8) + s) * kCols;
        if (c0 >= a.dim) return;
        add_pieces<kWide>(a, piece, warp * per, warp * per + per < count ? warp * per + per : count, c0, lane, acc);
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 8; ++i) share[warp][lane][i] = acc[i];
        __syncthreads();
        if (warp == 0) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                acc[i] = 0.f;
                for (int w = 0; w < 8; ++w) acc[i] += share[w][lane][i];
            }
            put_row<kWide>(row, c0, a.dim, lane, acc, a.scale, a.accumulate);
        }
    }
}

// Workspace of the gradient: header, the sorted keys and positions (two sets
// when several sort tiles hand them on), the tiles' counts, the runs' pieces.
struct GradLayout {
    int64_t tiles, part_ld;
    size_t keys, pos, keys2, pos2, hist, parts, total;
};

// Long pieces leave fewer runs to join, short ones more warps: the longest
// that gives every warp slot of 152 SMs (24 each) a task, as 32 does for 16384
// tokens of 7168 (4099 tokens of 1003: 64 us with 32, PIECEUS with 8).
int sum_piece_size(int64_t tokens, int64_t dim) {
    const int64_t cols = (dim + kCols - 1) / kCols;
    int piece = kMaxPiece;
    while (piece > kMinPiece && (tokens + piece - 1) / piece * cols < 152 * 24) piece /= 2;
    return piece;
}

GradLayout grad_layout(int64_t tokens, int64_t dim) {
    GradLayout L = {};
    auto take = [&L](int64_t bytes) {
        const size_t o = L.total;
        L.total += static_cast<size_t>((bytes + 255) / 256 * 256);
        return o;
    };
    L.total = kHeaderBytes;
    L.tiles = (tokens + kSortTile - 1) / kSortTile;
    L.part_ld = (dim + 7) / 8 * 8;
    L.keys = take(4 * tokens);
    L.pos = take(4 * tokens);
    L.keys2 = take(L.tiles > 1 ? 4 * tokens : 0);
    L.pos2 = take(L.tiles > 1 ? 4 * tokens : 0);
    L.hist = take(L.tiles > 1 ? 4 * L.tiles * kBins : 0);
    const int64_t piece = sum_piece_size(tokens, dim);
    L.parts = take(8 * ((tokens + piece - 1) / piece) * L.part_ld);
    return L;
}

cudaError_t sort_setup() {
    static std::mutex mu;
    static bool done[64] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    std::lock_guard<std::mutex> lock(mu);
    if (done[dev]) return cudaSuccess;
    const auto attr = cudaFuncAttributeMaxDynamicSharedMemorySize;
    e = cudaFuncSetAttribute(sort_one_kernel, attr, sizeof(SortShared));
    if (e == cudaSuccess) e = cudaFuncSetAttribute(sort_tile_kernel<false>, attr, sizeof(SortShared));
    if (e == cudaSuccess) e = cudaFuncSetAttribute(sort_tile_kernel<true>, attr, sizeof(SortShared));
    done[dev] = e == cudaSuccess;
    return e;
}

template <typename F>
cudaError_t counted(int kind, cudaStream_t st, F launch) {
    launch_begin(kind, st);
    const cudaError_t e = launch();
    launch_end(kind, st);
    return e;
}

template <int GD>
cudaError_t sum_go(const SumArgs& s, bool wide, unsigned blocks, cudaStream_t st) {
    return launch_pdl(wide ? embed_sum_kernel<GD, true> : embed_sum_kernel<GD, false>, dim3(blocks), dim3(32 * kSumWarps), 0, st, s);
}

}  // namespace

cudaError_t launch_embed_lookup(const EmbedLookup& a, cudaStream_t st) {
    launch_begin(MUON_KERNEL_EMBED_LOOKUP, st);
    if (a.table_dtype == MUON_F32) lookup_out<MUON_F32>(a, st);
    else if (a.table_dtype == MUON_BF16) lookup_out<MUON_BF16>(a, st);
    else lookup_out<MUON_F16>(a, st);
    launch_end(MUON_KERNEL_EMBED_LOOKUP, st);
    return cudaGetLastError();
}

size_t embed_grad_workspace(int64_t tokens, int64_t dim) { return grad_layout(tokens, dim).total; }

cudaError_t launch_embed_grad(const EmbedGrad& a, void* workspace, int num_sms, cudaStream_t st) {
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    const GradLayout L = grad_layout(a.tokens, a.dim);
    cudaError_t e = sort_setup();
    if (e != cudaSuccess) return e;
    int key_bits = 1;
    while ((a.vocab >> key_bits) != 0) ++key_bits;  // keys 0 .. vocab
    const int passes = (key_bits + kDigitBits - 1) / kDigitBits;
    SortArgs s = {};
    s.ids = a.ids;
    s.keys = reinterpret_cast<int32_t*>(ws + L.keys);
    s.pos = reinterpret_cast<int32_t*>(ws + L.pos);
    s.hist = reinterpret_cast<uint32_t*>(ws + L.hist);
    s.status = reinterpret_cast<int*>(ws);
    s.tokens = a.tokens;
    s.vocab = a.vocab;
    s.padding_idx = a.padding_idx;
    s.ids64 = a.ids64;
    s.bits = (key_bits + passes - 1) / passes;
    s.tiles = static_cast<int32_t>(L.tiles);
    bool zeros = !a.accumulate;  // zero rows still to be written
    if (L.tiles <= 1) {
        // a share's bits must fit its CTA's shared memory (tables up to 1.6e8 rows)
        const int others = num_sms - 1;
        const bool fused = zeros && ((a.vocab + others - 1) / others + 31) / 32 * 4 <= static_cast<int64_t>(sizeof(SortShared));
        e = counted(MUON_KERNEL_EMBED_SORT, st, [&] {
            return launch_pdl(sort_one_kernel, dim3(fused ? num_sms : 1), dim3(kSortThreads), sizeof(SortShared), st, s,
                              passes, a.d_table, a.dim);
        });
        if (fused) zeros = false;
    } else {
        e = cudaMemsetAsync(ws, 0, kHeaderBytes, st);
        int32_t* bk[2] = {s.keys, reinterpret_cast<int32_t*>(ws + L.keys2)};
        int32_t* bp[2] = {s.pos, reinterpret_cast<int32_t*>(ws + L.pos2)};
        for (int p = 0; p < passes && e == cudaSuccess; ++p) {
            const int out = (passes - 1 - p) & 1;  // the last pass writes keys and pos
            s.shift = p * s.bits;
            s.keys_in = p ? bk[out ^ 1] : nullptr;
            s.pos_in = p ? bp[out ^ 1] : nullptr;
            s.keys = bk[out];
            s.pos = bp[out];
            const dim3 grid(static_cast<unsigned>(L.tiles));
            e = counted(MUON_KERNEL_EMBED_SORT, st, [&] {
                return launch_pdl(sort_tile_kernel<false>, grid, dim3(kSortThreads), sizeof(SortShared), st, s);
            });
            if (e == cudaSuccess)
                e = counted(MUON_KERNEL_EMBED_SORT, st, [&] {
                    return launch_pdl(sort_scan_kernel, dim3(1), dim3(1024), 0, st, s.hist, L.tiles << s.bits);
                });
            if (e == cudaSuccess)
                e = counted(MUON_KERNEL_EMBED_SORT, st, [&] {
                    return launch_pdl(sort_tile_kernel<true>, grid, dim3(kSortThreads), sizeof(SortShared), st, s);
                });
        }
    }
    if (e != cudaSuccess) return e;
    const size_t ge = dtype_bytes(a.grad_dtype);
    const bool wide = a.dim % 8 == 0 && (reinterpret_cast<uintptr_t>(a.grad) & 15) == 0 && a.grad_ld * ge % 16 == 0 &&
                      (reinterpret_cast<uintptr_t>(a.d_table) & 15) == 0;
    SumArgs m = {};
    m.grad = a.grad;
    m.keys = reinterpret_cast<int32_t*>(ws + L.keys);
    m.pos = reinterpret_cast<int32_t*>(ws + L.pos);
    m.parts = reinterpret_cast<float*>(ws + L.parts);
    m.d_table = a.d_table;
    m.grad_ld = a.grad_ld;
    m.part_ld = L.part_ld;
    m.vocab = a.vocab;
    m.dim = a.dim;
    m.tokens = static_cast<int32_t>(a.tokens);
    m.col_tasks = static_cast<int32_t>((a.dim + kCols - 1) / kCols);
    m.piece = sum_piece_size(a.tokens, a.dim);
    m.pieces = static_cast<int32_t>((a.tokens + m.piece - 1) / m.piece);
    m.zero_tasks_x = static_cast<int32_t>((a.dim + kZeroCols - 1) / kZeroCols);
    m.accumulate = a.accumulate;
    m.scale = a.scale;
    const int64_t sum_blocks = (static_cast<int64_t>(m.pieces) * m.col_tasks + kSumWarps - 1) / kSumWarps;
    const int64_t zero_blocks =
        zeros ? ((a.vocab + kZeroRows - 1) / kZeroRows * m.zero_tasks_x + kSumWarps - 1) / kSumWarps : 0;
    if (sum_blocks + zero_blocks > INT32_MAX) return cudaErrorInvalidValue;
    m.sum_blocks = static_cast<int32_t>(sum_blocks);
    const unsigned blocks = static_cast<unsigned>(sum_blocks + zero_blocks);
    if (blocks > 0)
        e = counted(MUON_KERNEL_EMBED_GRAD, st, [&] {
            return a.grad_dtype == MUON_F32    ? sum_go<MUON_F32>(m, wide, blocks, st)
                   : a.grad_dtype == MUON_BF16 ? sum_go<MUON_BF16>(m, wide, blocks, st)
                                               : sum_go<MUON_F16>(m, wide, blocks, st);
        });
    if (e == cudaSuccess && m.pieces > 1)
        e = counted(MUON_KERNEL_EMBED_GRAD, st, [&] {
            return launch_pdl(wide ? embed_join_kernel<true> : embed_join_kernel<false>,
                              dim3(static_cast<unsigned>(m.pieces - 1), static_cast<unsigned>((m.col_tasks + 7) / 8)),
                              dim3(256), 0, st, m);
        });
    return e;
}

}  // namespace muon
