// embedding.hip -- rows of a table looked up by token, and the table's gradient.
//
//   forward:   y[t] = scale * table[ids[t]]
//   backward:  dtable[v] = scale * sum over the tokens t with ids[t] = v of dy[t]
//
// The backward sorts the tokens by entry and sums each entry's rows in the
// order of their tokens, so that repeated calls give equal bits and no atomics
// meet.  Three launches:
//
//  sort:  workgroup b owns `span` entries of the table.  It reads all ids once
//         to count those below its entries (where its first token goes) and
//         those of each of its entries, a wavefront counting its own
//         contiguous part of the tokens; then again to place its tokens, each
//         wavefront in order behind the wavefronts before it.  No workgroup
//         waits for another: 512 workgroups reading 32768 ids are 64 MB from
//         the L2s, less time than the second launch of a counting sort by
//         blocks.
//  sum:   a wavefront per entry adds its rows and writes the entry, zeros
//         where it has no token.  Entries of more than kLong tokens (text has a
//         few that make up several percent of it) are left to further
//         wavefronts, each of which adds the rows of kLong consecutive sorted
//         tokens: at most two such entries have tokens there, and their two sums
//         are kept.
//  join:  the sums of a long entry are added in order by the wavefronts of the
//         workgroup at its start.
//
// Bound by memory: T rows read, V rows written (or, added, T at most read and written).
#include "mfma_common.h"

#include "../../include/moe_ffn.h"

#include <algorithm>
#include <cstdint>

namespace moe {
namespace {

using namespace mfma;

constexpr int kSortThreads = 512;
constexpr int kSortWaves = kSortThreads / 64;
constexpr int kMaxSpan = 512;          // entries of a sorting workgroup
constexpr int kLong = 64;              // tokens of an entry that one wavefront adds
constexpr int kMaxD = 16384;

bool aligned(const void* p, size_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

// ---- forward

struct FwdArgs {
    const int32_t* ids;
    const void* table;
    void* y;
    int64_t T;
    int D, V;
    float scale;
    int rows;        // rows of a workgroup
};

// Elements of 16 bytes.
template <typename E>
struct Vec {
    static constexpr int n = 16 / sizeof(E);
};

__device__ __forceinline__ u32x4_t scaled(u32x4_t v, float s, uint16_t*) {
    u32x4_t o;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        o[i] = pack_bf16(__uint_as_float(v[i] << 16) * s, __uint_as_float(v[i] & 0xffff0000u) * s);
    return o;
}
__device__ __forceinline__ u32x4_t scaled(u32x4_t v, float s, float*) {
    u32x4_t o;
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = __float_as_uint(__uint_as_float(v[i]) * s);
    return o;
}
__device__ __forceinline__ float to_float(uint16_t v) { return __uint_as_float((uint32_t)v << 16); }
__device__ __forceinline__ float to_float(float v) { return v; }
__device__ __forceinline__ void put(uint16_t* p, float v) { *p = (uint16_t)pack_bf16(v, 0.f); }
__device__ __forceinline__ void put(float* p, float v) { *p = v; }

// 16 bytes a lane where rows are a multiple of that, else an element a lane.
template <typename E, bool VEC>
__global__ __launch_bounds__(256) void embedding_forward_kernel(const FwdArgs a) {
    constexpr int W = VEC ? Vec<E>::n : 1;
    const int per_row = a.D / W;
    const int64_t t0 = (int64_t)blockIdx.x * a.rows;
    const int rows = (int)min((int64_t)a.rows, a.T - t0);
    for (int i = threadIdx.x; i < rows * per_row; i += 256) {
        const int r = i / per_row, c = (i - r * per_row) * W;
        const int64_t t = t0 + r;
        const int id = a.ids[t];
        const bool in = id >= 0 && id < a.V;
        const E* src = (const E*)a.table + (int64_t)(in ? id : 0) * a.D + c;
        E* dst = (E*)a.y + t * a.D + c;
        if constexpr (VEC)
            *(u32x4_t*)dst = in ? scaled(*(const u32x4_t*)src, a.scale, (E*)nullptr) : u32x4_t{0, 0, 0, 0};
        else
            put(dst, in ? to_float(*src) * a.scale : 0.f);
    }
}

// ---- backward

// order: the tokens with ids in [0, V), sorted by id and then by token;
// start[v]: where those of entry v begin, start[V] how many there are.
__global__ __launch_bounds__(kSortThreads) void embedding_sort_kernel(const int32_t* __restrict__ ids, int64_t T, int V,
                                                                      int span, int32_t* __restrict__ order,
                                                                      int32_t* __restrict__ start) {
    __shared__ int32_t at[kSortWaves][kMaxSpan];   // counts, then places
    __shared__ int32_t below[kSortWaves], sums[kSortWaves];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int lo = blockIdx.x * span, hi = min(lo + span, V);
    for (int i = tid; i < kSortWaves * kMaxSpan; i += kSortThreads) (&at[0][0])[i] = 0;
    __syncthreads();
    // this wavefront's tokens
    const int64_t per = (T + kSortThreads - 1) / kSortThreads * 64;
    const int64_t t0 = min(per * wave, T), t1 = min(t0 + per, T);
    int under = 0;
    for (int64_t base = t0; base < t1; base += 512) {
        int32_t id[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int64_t t = base + 64 * j + lane;
            id[j] = t < t1 ? ids[t] : -1;
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            under += id[j] >= 0 && id[j] < lo;
            if (id[j] >= lo && id[j] < hi) atomicAdd(&at[wave][id[j] - lo], 1);
        }
    }
    for (int d = 32; d; d >>= 1) under += __shfl_xor(under, d);
    if (lane == 0) below[wave] = under;
    __syncthreads();
    // exclusive prefix over (entry, wavefront)
    int mine = 0;
    int32_t c[kSortWaves];
#pragma unroll
    for (int w = 0; w < kSortWaves; ++w) {
        c[w] = at[w][tid];
        mine += c[w];
    }
    int incl = mine;
    for (int d = 1; d < 64; d <<= 1) {
        const int o = __shfl_up(incl, d);
        if (lane >= d) incl += o;
    }
    if (lane == 63) sums[wave] = incl;
    __syncthreads();
    int place = incl - mine;
#pragma unroll
    for (int w = 0; w < kSortWaves; ++w) {
        place += below[w];
        if (w < wave) place += sums[w];
    }
    if (lo + tid < hi) {
        start[lo + tid] = place;
        if (lo + tid == V - 1) start[V] = place + mine;
    }
#pragma unroll
    for (int w = 0; w < kSortWaves; ++w) {
        at[w][tid] = place;
        place += c[w];
    }
    __syncthreads();
    for (int64_t base = t0; base < t1; base += 512) {
        int32_t id[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int64_t t = base + 64 * j + lane;
            id[j] = t < t1 ? ids[t] : -1;
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const bool in = id[j] >= lo && id[j] < hi;
            uint64_t todo = __ballot(in);
            while (todo) {       // one entry at a time; every lane of the wavefront is here
                const int first = __ffsll((unsigned long long)todo) - 1;
                const int v = __shfl(id[j], first);
                const uint64_t same = __ballot(in && id[j] == v);
                const int p = at[wave][v - lo];
                if (in && id[j] == v)
                    order[p + __popcll(same & ((1ull << lane) - 1))] = (int32_t)(base + 64 * j + lane);
                if (lane == first) at[wave][v - lo] = p + __popcll(same);
                todo &= ~same;
            }
        }
    }
}

struct SumArgs {
    const int32_t *ids, *order, *start;
    const void* dy;
    void* out;
    float* part;         // [chunks][2][D]
    int64_t T;
    int D, V;
    float scale;
    int add;
    int64_t row_blocks;  // workgroups of 4 entries; those behind them take 4 chunks each
};

// Four columns, or one (VEC false), of a row.
template <typename E, bool VEC>
__device__ __forceinline__ float4 load_cols(const E* p) {
    if constexpr (!VEC) {
        return make_float4(to_float(*p), 0.f, 0.f, 0.f);
    } else if constexpr (sizeof(E) == 4) {
        return *(const float4*)p;
    } else {
        const uint2 v = *(const uint2*)p;
        return make_float4(__uint_as_float(v.x << 16), __uint_as_float(v.x & 0xffff0000u), __uint_as_float(v.y << 16),
                           __uint_as_float(v.y & 0xffff0000u));
    }
}
template <typename O, bool VEC>
__device__ __forceinline__ void store_cols(O* p, float4 v) {
    if constexpr (!VEC) put(p, v.x);
    else if constexpr (sizeof(O) == 4) *(float4*)p = v;
    else *(uint2*)p = make_uint2(pack_bf16(v.x, v.y), pack_bf16(v.z, v.w));
}
__device__ __forceinline__ float4 plus(float4 a, float4 b) {
    return make_float4(a.x + b.x, a.y + b.y, a.z + b.z, a.w + b.w);
}
__device__ __forceinline__ float4 times(float4 a, float s) { return make_float4(a.x * s, a.y * s, a.z * s, a.w * s); }

// The sum of columns c.. of the rows of sorted tokens p0 .. p1 - 1, in order.
template <typename E, bool VEC>
__device__ __forceinline__ float4 sum_rows(const SumArgs& a, int p0, int p1, int c) {
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
    const E* dy = (const E*)a.dy + c;
    int p = p0;
    for (; p + 8 <= p1; p += 8) {
        float4 v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = load_cols<E, VEC>(dy + (int64_t)a.order[p + j] * a.D);
#pragma unroll
        for (int j = 0; j < 8; ++j) s = plus(s, v[j]);
    }
    for (; p < p1; ++p) s = plus(s, load_cols<E, VEC>(dy + (int64_t)a.order[p] * a.D));
    return s;
}

template <typename O, bool VEC>
__device__ __forceinline__ void write_cols(const SumArgs& a, int v, int c, float4 s) {
    O* p = (O*)a.out + (int64_t)v * a.D + c;
    s = times(s, a.scale);
    if (a.add) s = plus(s, load_cols<O, VEC>(p));
    store_cols<O, VEC>(p, s);
}

template <typename E, typename O, bool VEC>
__global__ __launch_bounds__(256) void embedding_sum_kernel(const SumArgs a) {
    constexpr int W = VEC ? 4 : 1;
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    if (blockIdx.x < a.row_blocks) {
        const int64_t v = (int64_t)blockIdx.x * 4 + wave;
        if (v >= a.V) return;
        const int s = a.start[v], e = a.start[v + 1];
        if (e - s > kLong || (a.add && e == s)) return;
        for (int c = lane * W; c < a.D; c += 64 * W) write_cols<O, VEC>(a, (int)v, c, sum_rows<E, VEC>(a, s, e, c));
        return;
    }
    const int64_t chunk = ((int64_t)blockIdx.x - a.row_blocks) * 4 + wave;
    const int all = a.start[a.V];
    if (chunk * kLong >= all) return;
    const int p0 = (int)(chunk * kLong), p1 = min(p0 + kLong, all);
    // the entry of the chunk's first token, and that of its last, if long
    const int va = a.ids[a.order[p0]], vb = a.ids[a.order[p1 - 1]];
    const int ae = a.start[va + 1], bs = a.start[vb];
    float* part = a.part + chunk * 2 * a.D;
    if (ae - a.start[va] > kLong)
        for (int c = lane * W; c < a.D; c += 64 * W)
            store_cols<float, VEC>(part + c, sum_rows<E, VEC>(a, p0, min(ae, p1), c));
    if (vb != va && a.start[vb + 1] - bs > kLong)
        for (int c = lane * W; c < a.D; c += 64 * W)
            store_cols<float, VEC>(part + a.D + c, sum_rows<E, VEC>(a, bs, p1, c));
}

// Workgroup: the long entry that begins in this chunk, if one does (it then
// holds the chunk's last token).
template <typename O, bool VEC>
__global__ __launch_bounds__(256) void embedding_join_kernel(const SumArgs a) {
    constexpr int W = VEC ? 4 : 1;
    const int64_t chunk = blockIdx.x;
    const int all = a.start[a.V];
    if (chunk * kLong >= all) return;
    const int p0 = (int)(chunk * kLong), p1 = min(p0 + kLong, all);
    const int v = a.ids[a.order[p1 - 1]];
    const int s = a.start[v], e = a.start[v + 1];
    if (e - s <= kLong || s < p0) return;
    // the first sum is the chunk's second where the entry begins behind another
    const int64_t last = (e - 1) / kLong;
    for (int c = threadIdx.x * W; c < a.D; c += 256 * W) {
        float4 sum = load_cols<float, VEC>(a.part + (chunk * 2 + (a.ids[a.order[p0]] != v)) * a.D + c);
        int64_t k = chunk + 1;
        for (; k + 8 <= last + 1; k += 8) {
            float4 x[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) x[j] = load_cols<float, VEC>(a.part + (k + j) * 2 * a.D + c);
#pragma unroll
            for (int j = 0; j < 8; ++j) sum = plus(sum, x[j]);
        }
        for (; k <= last; ++k) sum = plus(sum, load_cols<float, VEC>(a.part + k * 2 * a.D + c));
        write_cols<O, VEC>(a, v, c, sum);
    }
}

constexpr size_t kAlign = 256;
size_t padded(size_t n) { return (n + kAlign - 1) / kAlign * kAlign; }

struct Layout {
    size_t order, start, part, total;
    int64_t chunks;
};
Layout layout_of(int64_t T, int D, int V) {
    Layout l;
    l.chunks = (T + kLong - 1) / kLong;
    l.order = 0;
    l.start = padded((size_t)T * 4);
    l.part = l.start + padded(((size_t)V + 1) * 4);
    l.total = l.part + padded((size_t)l.chunks * 2 * D * 4);
    return l;
}

moe_status check(int64_t T, int D, int V, float scale, moe_dtype dtype) {
    if (T < 0 || T >= (1ll << 31) || D <= 0 || V <= 0 || (dtype != MOE_F32 && dtype != MOE_BF16)) return MOE_ERR_INVALID_ARG;
    if (!(scale >= -3.4e38f && scale <= 3.4e38f)) return MOE_ERR_INVALID_ARG;
    if (D > kMaxD || V > (1 << 24) || T > (1 << 29)) return MOE_ERR_UNSUPPORTED;
    return MOE_OK;
}

template <typename E, typename O>
hipError_t launch_backward(SumArgs a, int64_t chunks, hipStream_t s) {
    const unsigned grid = (unsigned)(a.row_blocks + (chunks + 3) / 4);
    // rows of 4 columns a lane, where every row begins at a multiple of them
    if (a.D % 4 == 0) embedding_sum_kernel<E, O, true><<<grid, 256, 0, s>>>(a);
    else embedding_sum_kernel<E, O, false><<<grid, 256, 0, s>>>(a);
    if (hipError_t e = hipGetLastError()) return e;
    if (a.T > kLong) {
        if (a.D % 4 == 0) embedding_join_kernel<O, true><<<(unsigned)chunks, 256, 0, s>>>(a);
        else embedding_join_kernel<O, false><<<(unsigned)chunks, 256, 0, s>>>(a);
    }
    return hipGetLastError();
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

moe_status moe_embedding_forward(const int32_t* ids, const void* table, void* y, int64_t T, int D, int V, float scale,
                                 moe_dtype dtype, hipStream_t stream) {
    const moe_status st = check(T, D, V, scale, dtype);
    if (st != MOE_OK) return st;
    if (T > 0 && (!ids || !table || !y)) return MOE_ERR_INVALID_ARG;
    if (!aligned(ids, 4) || !aligned(table, 16) || !aligned(y, 16)) return MOE_ERR_INVALID_ARG;
    if (T == 0) return MOE_OK;
    FwdArgs a = {ids, table, y, T, D, V, scale, 1};
    const int e = dtype == MOE_BF16 ? 2 : 4;
    const bool vec = D * e % 16 == 0;
    // four 16-byte loads a thread
    a.rows = std::max(1, 1024 / (vec ? D * e / 16 : D));
    // and fewer than 2^32 threads a grid (at most 64 rows of 16384 then)
    a.rows = std::max(a.rows, (int)((T + (1 << 23) - 1) >> 23));
    const unsigned grid = (unsigned)((T + a.rows - 1) / a.rows);
    (void)hipGetLastError();
    if (dtype == MOE_BF16) {
        if (vec) embedding_forward_kernel<uint16_t, true><<<grid, 256, 0, stream>>>(a);
        else embedding_forward_kernel<uint16_t, false><<<grid, 256, 0, stream>>>(a);
    } else {
        if (vec) embedding_forward_kernel<float, true><<<grid, 256, 0, stream>>>(a);
        else embedding_forward_kernel<float, false><<<grid, 256, 0, stream>>>(a);
    }
    return hipGetLastError() == hipSuccess ? MOE_OK : MOE_ERR_HIP;
}

size_t moe_embedding_backward_workspace_size(int64_t T, int D, int V) {
    if (check(T, D, V, 1.f, MOE_F32) != MOE_OK) return 0;
    return layout_of(T, D, V).total;
}

moe_status moe_embedding_backward(const int32_t* ids, const void* dy, void* dtable, int64_t T, int D, int V, float scale,
                                  int accumulate, moe_dtype dtype, moe_dtype table_dtype, void* workspace, size_t ws_bytes,
                                  hipStream_t stream) {
    const moe_status st = check(T, D, V, scale, dtype);
    if (st != MOE_OK) return st;
    if (table_dtype != MOE_F32 && table_dtype != dtype) return MOE_ERR_INVALID_ARG;
    if (!dtable || (T > 0 && (!ids || !dy)) || !workspace) return MOE_ERR_INVALID_ARG;
    if (!aligned(ids, 4) || !aligned(dy, 16) || !aligned(dtable, 16) || !aligned(workspace, kAlign)) return MOE_ERR_INVALID_ARG;
    const Layout l = layout_of(T, D, V);
    if (ws_bytes < l.total) return MOE_ERR_WORKSPACE;
    if (T == 0 && accumulate) return MOE_OK;
    char* ws = (char*)workspace;
    SumArgs a = {ids, (const int32_t*)(ws + l.order), (const int32_t*)(ws + l.start), dy, dtable, (float*)(ws + l.part),
                 T, D, V, scale, accumulate ? 1 : 0, ((int64_t)V + 3) / 4};
    // about 512 workgroups, each with a power of two of entries
    int span = 16;
    while (span < kMaxSpan && (int64_t)span * 512 < V) span *= 2;
    (void)hipGetLastError();
    embedding_sort_kernel<<<(V + span - 1) / span, kSortThreads, 0, stream>>>(ids, T, V, span, (int32_t*)(ws + l.order),
                                                                             (int32_t*)(ws + l.start));
    if (hipGetLastError() != hipSuccess) return MOE_ERR_HIP;
    const bool in16 = dtype == MOE_BF16, out16 = table_dtype == MOE_BF16;
    const hipError_t e = in16 && out16 ? launch_backward<uint16_t, uint16_t>(a, l.chunks, stream)
                         : in16        ? launch_backward<uint16_t, float>(a, l.chunks, stream)
                                       : launch_backward<float, float>(a, l.chunks, stream);
    return e == hipSuccess ? MOE_OK : MOE_ERR_HIP;
}

}  // extern "C"
