// embedding.hip -- rows of a table looked up by token, and the table's gradient.
//
//   forward:   y[t] = scale * table[ids[t]]
//   backward:  dtable[v] = scale * sum over the tokens t with ids[t] = v of dy[t]
//
// The backward sorts the tokens by entry and sums each entry's rows in the
// order of their tokens, so that repeated calls give equal bits and no atomics
// meet.  Three launches:
//
//  sort:  workgroup b owns every 256th entry of the table.  It reads all ids once
//         to count those of the workgroups before it (where its first token goes) and
//         those of each of its entries, a wavefront counting its own
//         contiguous part of the tokens; then again to place its tokens, each
//         wavefront in order behind the wavefronts before it, the lanes of one
//         entry found by a ballot a bit.  No workgroup
//         waits for another: 256 workgroups reading 32768 ids twice are 64 MB
//         from the L2s, against two more launches of a sort by digits.
//  sum:   adds each entry's rows and writes the entry, zeros where it has no
//         token.  Entries of more than kLong tokens (text has a
//         few that make up several percent of it) are left to further
//         wavefronts, each of which adds the rows of kLong consecutive sorted
//         tokens: at most two such entries have tokens there, and their two sums
//         are kept.
//  join:  the sums of a long entry are added, in a fixed order, by the workgroup
//         at its start.
//
// Up to kFewTokens tokens one launch does all of it: each workgroup finds the
// tokens of its own entries (512 of 32768 entries x 768: 21 -> 13 us).
//
// Bound by memory: T rows read, V rows written (or, added, T at most read and written).
#include "mfma_common.h"

#include "../../include/moe_ffn.h"

#include <algorithm>
#include <cstdint>

namespace moe {
namespace {

using namespace mfma;

constexpr int kSortThreads = 1024;
constexpr int kSortWaves = kSortThreads / 64;
constexpr int kLong = 32;              // tokens of an entry that one wavefront adds
constexpr int kFewTokens = 1024;       // in one launch
constexpr int kFewEntries = 2048;      // of a workgroup, at most
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

// order: the tokens with ids in [0, V), those of an entry together and in order;
// first[v]: where those of entry v begin, count[v] how many they are; first[V] how
// many there are in all.  Workgroup b owns entries b, b + 2^shift, b + 2 2^shift..,
// at most 2^BITS of them, so that text's frequent entries, which are next to each
// other, fall to different workgroups (32768 tokens, one in 11 / (v + 1) of them
// entry v: 26 us with ranges of entries, 17 so).
template <int BITS>
__global__ __launch_bounds__(kSortThreads) void embedding_sort_kernel(const int32_t* __restrict__ ids, int64_t T, int V,
                                                                      int shift, int32_t* __restrict__ order,
                                                                      int32_t* __restrict__ first,
                                                                      int32_t* __restrict__ counts) {
    constexpr int SPAN = 1 << BITS;
    __shared__ int32_t at[kSortWaves][SPAN];   // counts, then places
    __shared__ int32_t below[kSortWaves], sums[kSortWaves];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int mask = (1 << shift) - 1, own = blockIdx.x;
    for (int i = tid; i < kSortWaves * SPAN; i += kSortThreads) (&at[0][0])[i] = 0;
    __syncthreads();
    // This wavefront's tokens, 64 consecutive ones a load.  Every workgroup looks at
    // every token, and that is most of its time: a few instructions for 64.
    const int per = (int)((T + kSortThreads - 1) / kSortThreads * 64);
    const int t0 = (int)min((int64_t)per * wave, T), t1 = (int)min((int64_t)t0 + per, T);
    auto each = [&](auto&& look) {
        int base = t0;
        if (base + 512 <= t1) {
            int32_t id[8], next[8];
            auto load = [&](const int32_t* p, int32_t (&to)[8]) {
#pragma unroll
                for (int j = 0; j < 8; ++j) to[j] = p[64 * j + lane];
            };
            load(ids + base, id);
            for (; base + 512 <= t1; base += 512) {
                load(ids + (base + 1024 <= t1 ? base + 512 : base), next);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    look(id[j], base + 64 * j);
                    id[j] = next[j];
                }
            }
        }
        for (; base < t1; base += 64) look(base + lane < t1 ? ids[base + lane] : -1, base);
    };
    int under = 0;
    bool any = false;
    each([&](int32_t id, int) {
        // -1 for what is outside the table: no workgroup's number is above mask
        id = (uint32_t)id < (uint32_t)V ? id : -1;
        const int of = id & mask;
        under += of < own;
        const bool in = of == own && id >= 0;
        if (__ballot(in)) {
            any = true;
            if (in) atomicAdd(&at[wave][id >> shift], 1);
        }
    });
    for (int d = 32; d; d >>= 1) under += __shfl_xor(under, d);
    if (lane == 0) below[wave] = under;
    __syncthreads();
    // exclusive prefix over (entry, wavefront), an entry a thread
    const bool entry = tid < SPAN;
    int mine = 0;
    if (entry)
        for (int w = 0; w < kSortWaves; ++w) mine += at[w][tid];
    int incl = mine;
    for (int d = 1; d < 64; d <<= 1) {
        const int o = __shfl_up(incl, d);
        if (lane >= d) incl += o;
    }
    if (lane == 63) sums[wave] = incl;
    __syncthreads();
    int place = incl - mine;
    for (int w = 0; w < kSortWaves; ++w) {
        place += below[w];
        if (w < wave) place += sums[w];
    }
    if (entry) {
        const int64_t v = ((int64_t)tid << shift) + own;
        if (v < V) {
            first[v] = place;
            counts[v] = mine;
        }
        if (own == mask && tid == SPAN - 1) first[V] = place + mine;
        for (int w = 0; w < kSortWaves; ++w) {
            const int c = at[w][tid];
            at[w][tid] = place;
            place += c;
        }
    }
    __syncthreads();
    if (!any) return;
    // in order
    each([&](int32_t id, int base) {
        const bool in = (id & mask) == own && (uint32_t)id < (uint32_t)V;
        uint64_t todo = __ballot(in);
        if (!todo) return;
        const int e = in ? id >> shift : -1;
        if (__popcll(todo) <= 8) {
            // few lanes: one entry after the other
            do {
                const int v = __builtin_amdgcn_readlane(e, __ffsll((unsigned long long)todo) - 1);
                const uint64_t same = __ballot(e == v);
                const int p = at[wave][v];
                if (e == v) order[p + __popcll(same & ((1ull << lane) - 1))] = base + lane;
                if (lane == 0) at[wave][v] = p + __popcll(same);
                todo &= ~same;
            } while (todo);
            return;
        }
        // the lanes with this lane's entry: those that agree in every bit
#pragma unroll
        for (int b = 0; b < BITS; ++b) {
            const uint64_t set = __ballot(e >> b & 1);
            todo &= e >> b & 1 ? set : ~set;
        }
        const int before = __popcll(todo & ((1ull << lane) - 1));
        if (in) {
            const int p = at[wave][e];
            order[p + before] = base + lane;
            // one of them moves the place on, behind all their reads
            if (before == 0) at[wave][e] = p + __popcll(todo);
        }
    });
}

struct SumArgs {
    const int32_t *ids, *order, *first, *count;
    const void* dy;
    void* out;
    float* part;         // [chunks][2][D]
    int64_t T;
    int D, V;
    float scale;
    int add;
    int rows;            // entries of a workgroup
    int64_t row_blocks;  // workgroups of entries; those behind them take 4 chunks each
};

// W consecutive columns (8 of bf16, 4 of fp32: 16 bytes; or 1) in fp32.
template <int W>
struct Cols {
    float x[W];
};
template <typename E, int W>
__device__ __forceinline__ Cols<W> load_cols(const E* p) {
    Cols<W> o;
    if constexpr (W == 1) {
        o.x[0] = to_float(*p);
    } else if constexpr (sizeof(E) == 4) {
#pragma unroll
        for (int i = 0; i < W; i += 4) *(float4*)(o.x + i) = *(const float4*)(p + i);
    } else if constexpr (W == 4) {
        const uint2 v = *(const uint2*)p;
        o.x[0] = __uint_as_float(v.x << 16), o.x[1] = __uint_as_float(v.x & 0xffff0000u);
        o.x[2] = __uint_as_float(v.y << 16), o.x[3] = __uint_as_float(v.y & 0xffff0000u);
    } else {
        const u32x4_t v = *(const u32x4_t*)p;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            o.x[2 * i] = __uint_as_float(v[i] << 16);
            o.x[2 * i + 1] = __uint_as_float(v[i] & 0xffff0000u);
        }
    }
    return o;
}
template <typename O, int W>
__device__ __forceinline__ void store_cols(O* p, const Cols<W>& v) {
    if constexpr (W == 1) {
        put(p, v.x[0]);
    } else if constexpr (sizeof(O) == 4) {
#pragma unroll
        for (int i = 0; i < W; i += 4) *(float4*)(p + i) = *(const float4*)(v.x + i);
    } else if constexpr (W == 4) {
        *(uint2*)p = make_uint2(pack_bf16(v.x[0], v.x[1]), pack_bf16(v.x[2], v.x[3]));
    } else {
        u32x4_t o;
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] = pack_bf16(v.x[2 * i], v.x[2 * i + 1]);
        *(u32x4_t*)p = o;
    }
}
template <int W>
__device__ __forceinline__ void add_to(Cols<W>& a, const Cols<W>& b) {
#pragma unroll
    for (int i = 0; i < W; ++i) a.x[i] += b.x[i];
}

// The sum of columns c.. of the rows of sorted tokens p0 .. p1 - 1, in order;
// token(p): which they are.
template <typename E, int W, typename F>
__device__ __forceinline__ Cols<W> sum_rows(const SumArgs& a, int p0, int p1, int c, F&& token) {
    Cols<W> s = {};
    const E* dy = (const E*)a.dy + c;
    int p = p0;
    for (; p + 8 <= p1; p += 8) {
        Cols<W> v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = load_cols<E, W>(dy + (int64_t)token(p + j) * a.D);
#pragma unroll
        for (int j = 0; j < 8; ++j) add_to(s, v[j]);
    }
    for (; p < p1; ++p) add_to(s, load_cols<E, W>(dy + (int64_t)token(p) * a.D));
    return s;
}
template <typename E, int W>
__device__ __forceinline__ Cols<W> sum_rows(const SumArgs& a, int p0, int p1, int c) {
    return sum_rows<E, W>(a, p0, p1, c, [&](int p) { return a.order[p]; });
}

template <typename O, int W>
__device__ __forceinline__ void write_cols(const SumArgs& a, int v, int c, Cols<W> s) {
    O* p = (O*)a.out + (int64_t)v * a.D + c;
#pragma unroll
    for (int i = 0; i < W; ++i) s.x[i] *= a.scale;
    if (a.add) add_to(s, load_cols<O, W>(p));
    // the table's gradient is not read again here: past the caches (32768 entries x
    // 768 in bf16, nearly all zeros: 14.4 -> 12.2 us)
    if constexpr (W % 4 == 0 && sizeof(O) * W % 16 == 0) {
        u32x4_t o[sizeof(O) * W / 16];
        store_cols<O, W>((O*)o, s);
#pragma unroll
        for (int i = 0; i < (int)(sizeof(O) * W / 16); ++i) __builtin_nontemporal_store(o[i], (u32x4_t*)p + i);
    } else {
        store_cols<O, W>(p, s);
    }
}

// Zeros, past the caches too.
template <typename O, int W>
__device__ __forceinline__ void clear_cols(O* p) {
    if constexpr (W % 4 == 0 && sizeof(O) * W % 16 == 0) {
#pragma unroll
        for (int i = 0; i < (int)(sizeof(O) * W / 16); ++i) __builtin_nontemporal_store(u32x4_t{}, (u32x4_t*)p + i);
    } else {
        store_cols<O, W>(p, Cols<W>{});
    }
}

template <typename E, typename O, int W>
__global__ __launch_bounds__(256) void embedding_sum_kernel(const SumArgs a) {
    if (blockIdx.x < a.row_blocks) {
        // W columns of an entry a thread.  The entries that a workgroup sums lie far
        // apart, since text has its frequent ones next to each other; those that it
        // clears follow one another, so that lines are written whole (rows of 632 fp32,
        // 63069 of them: 41 -> 31 us).
        const int per_row = a.D / W;
        const float inv = 1.f / per_row;
        // i / per_row: i is less than 2^16, so the product is off by less than 2^-7
        // of one column group's share
        auto row_of = [&](int i) { return (int)((i + 0.5f) * inv); };
        if (!a.add) {
            const int v0 = (int)blockIdx.x * a.rows;
            for (int i0 = threadIdx.x; i0 < a.rows * per_row; i0 += 1024) {
                bool none[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int v = v0 + row_of(i0 + 256 * j);
                    none[j] = i0 + 256 * j < a.rows * per_row && v < a.V && a.count[min(v, a.V - 1)] == 0;
                }
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (none[j]) clear_cols<O, W>((O*)a.out + (int64_t)v0 * a.D + (int64_t)(i0 + 256 * j) * W);
            }
        }
        for (int i0 = threadIdx.x; i0 < a.rows * per_row; i0 += 1024) {
            int s[4], n[4], v[4], c[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int i = i0 + 256 * j, r = row_of(i);
                c[j] = (i - r * per_row) * W;
                v[j] = r < a.rows ? (int)blockIdx.x + r * (int)a.row_blocks : a.V;
                const int at = min(v[j], a.V - 1);
                s[j] = a.first[at];
                n[j] = a.count[at];
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if (v[j] >= a.V || n[j] > kLong || n[j] == 0) continue;
                write_cols<O, W>(a, v[j], c[j], sum_rows<E, W>(a, s[j], s[j] + n[j], c[j]));
            }
        }
        return;
    }
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t chunk = ((int64_t)blockIdx.x - a.row_blocks) * 4 + wave;
    const int all = a.first[a.V];
    if (chunk * kLong >= all) return;
    const int p0 = (int)(chunk * kLong), p1 = min(p0 + kLong, all);
    // the entry of the chunk's first token, and that of its last, if long
    const int va = a.ids[a.order[p0]], vb = a.ids[a.order[p1 - 1]];
    const int ae = a.first[va] + a.count[va], bs = a.first[vb];
    float* part = a.part + chunk * 2 * a.D;
    if (a.count[va] > kLong)
        for (int c = lane * W; c < a.D; c += 64 * W)
            store_cols<float, W>(part + c, sum_rows<E, W>(a, p0, min(ae, p1), c));
    if (vb != va && a.count[vb] > kLong)
        for (int c = lane * W; c < a.D; c += 64 * W)
            store_cols<float, W>(part + a.D + c, sum_rows<E, W>(a, bs, p1, c));
}

// Few tokens, in one launch: each workgroup looks through all ids for those of the
// entries that it clears and of those that it sums (as above), sorts the latter by
// entry and token in LDS and adds; an entry of more than kLong tokens has its
// wavefronts side by side, a quarter of the tokens each.  Most workgroups find none.
template <typename E, typename O, int W>
__global__ __launch_bounds__(256) void embedding_few_kernel(const SumArgs a) {
    constexpr int J = kFewTokens / 256;
    __shared__ uint64_t hits[4 * J];
    __shared__ int list[kFewTokens], sorted[kFewTokens];       // entry << 10 | token
    __shared__ uint16_t begin[kFewEntries], count[kFewEntries];
    __shared__ uint32_t taken[kFewEntries / 32];               // of the entries that it clears
    __shared__ Cols<W> sums[4][64];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const unsigned blocks = (unsigned)a.row_blocks;
    const int per_row = a.D / W;
    const float inv = 1.f / per_row;
    // an item's entry and columns; entries past the table are V
    auto item = [&](int i, int& r, int& c) {
        r = (int)((i + 0.5f) * inv);       // i / per_row, as above
        c = (i - r * per_row) * W;
        return r < a.rows ? min((int)blockIdx.x + r * (int)blocks, a.V) : a.V;
    };
    const unsigned v0 = blockIdx.x * (unsigned)a.rows;
    if (tid < kFewEntries / 32) taken[tid] = 0;
    __syncthreads();
    int key[J];
#pragma unroll
    for (int j = 0; j < J; ++j) {
        const int t = 256 * j + tid;
        const int id = t < a.T ? a.ids[t] : -1;
        const unsigned r = (unsigned)id / blocks, own = (unsigned)id - v0;
        if (id >= 0 && own < (unsigned)a.rows) atomicOr(taken + (own >> 5), 1u << (own & 31));
        key[j] = id >= 0 && id < a.V && (unsigned)id - r * blocks == blockIdx.x ? (int)(r << 10) | t : -1;
        const uint64_t m = __ballot(key[j] >= 0);
        if (lane == 0) hits[4 * j + wave] = m;
    }
    __syncthreads();
    int n = 0;
#pragma unroll
    for (int j = 0; j < J; ++j)
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            const uint64_t m = hits[4 * j + w];
            if (w == wave && key[j] >= 0) list[n + __popcll(m & ((1ull << lane) - 1))] = key[j];
            n += __popcll(m);
        }
    if (!a.add) {
        O* out = (O*)a.out + (int64_t)v0 * a.D;
        for (int i = tid; i < a.rows * per_row; i += 256) {
            int r, c;
            item(i, r, c);
            if (v0 + r < (unsigned)a.V && !(taken[r >> 5] >> (r & 31) & 1)) clear_cols<O, W>(out + (int64_t)i * W);
        }
    }
    if (n == 0) return;
    for (int r = tid; r < a.rows; r += 256) count[r] = 0;
    __syncthreads();
    for (int i = tid; i < n; i += 256) {
        int rank = 0;
        for (int k = 0; k < n; ++k) rank += list[k] < list[i];
        sorted[rank] = list[i];
    }
    __syncthreads();
    for (int i = tid; i < n; i += 256) {
        const int r = sorted[i] >> 10;
        if (i && sorted[i - 1] >> 10 == r) continue;
        int e = i + 1;
        while (e < n && sorted[e] >> 10 == r) ++e;
        begin[r] = (uint16_t)i;
        count[r] = (uint16_t)(e - i);
    }
    __syncthreads();
    auto token = [&](int p) { return sorted[p] & 1023; };
    for (int i = tid; i < a.rows * per_row; i += 256) {
        int r, c;
        const int v = item(i, r, c);
        if (v >= a.V || count[r] > kLong || count[r] == 0) continue;
        const int p = begin[r];
        write_cols<O, W>(a, v, c, sum_rows<E, W>(a, p, p + count[r], c, token));
    }
    for (int p = 0; p < n;) {
        const int r = sorted[p] >> 10, m = count[r];
        if (m > kLong) {
            for (int c0 = 0; c0 < a.D; c0 += 64 * W) {
                const int c = c0 + lane * W;
                Cols<W> s = {};
                if (c < a.D) s = sum_rows<E, W>(a, p + m * wave / 4, p + m * (wave + 1) / 4, c, token);
                sums[wave][lane] = s;
                __syncthreads();
                if (wave == 0 && c < a.D) {
                    for (int w = 1; w < 4; ++w) add_to(s, sums[w][lane]);
                    write_cols<O, W>(a, (int)(blockIdx.x + r * blocks), c, s);
                }
                __syncthreads();
            }
        }
        p += m;
    }
}

// Workgroup: the long entry that begins in this chunk, if one does (it then
// holds the chunk's last token).  64 groups of columns at a time, 16 wavefronts
// each over every 16th part, then over the 16.
template <typename O, int W>
__global__ __launch_bounds__(1024) void embedding_join_kernel(const SumArgs a) {
    __shared__ Cols<W> sums[16][64];
    const int64_t chunk = blockIdx.x;
    const int all = a.first[a.V];
    if (chunk * kLong >= all) return;
    const int p0 = (int)(chunk * kLong), p1 = min(p0 + kLong, all);
    const int v = a.ids[a.order[p1 - 1]];
    const int s = a.first[v], e = s + a.count[v];
    if (e - s <= kLong || s < p0) return;
    // the first sum is the chunk's second where the entry begins behind another
    const int64_t last = (e - 1) / kLong;
    const int64_t skip = a.ids[a.order[p0]] != v ? a.D : 0;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    for (int c0 = 0; c0 < a.D; c0 += 64 * W) {
        const int c = c0 + lane * W;
        Cols<W> sum = {};
        if (c < a.D) {
#pragma unroll 4
            for (int64_t k = chunk + wave; k <= last; k += 16)
                add_to(sum, load_cols<float, W>(a.part + k * 2 * a.D + (k == chunk ? skip : 0) + c));
        }
        sums[wave][lane] = sum;
        __syncthreads();
        if (wave == 0 && c < a.D) {
            for (int w = 1; w < 16; ++w) add_to(sum, sums[w][lane]);
            write_cols<O, W>(a, v, c, sum);
        }
        __syncthreads();
    }
}

constexpr size_t kAlign = 256;
size_t padded(size_t n) { return (n + kAlign - 1) / kAlign * kAlign; }

struct Layout {
    size_t order, first, count, part, total;
    int64_t chunks;
};
Layout layout_of(int64_t T, int D, int V) {
    Layout l;
    l.chunks = (T + kLong - 1) / kLong;
    l.order = 0;
    l.first = padded((size_t)T * 4);
    l.count = l.first + padded(((size_t)V + 1) * 4);
    l.part = l.count + padded((size_t)V * 4);
    l.total = l.part + padded((size_t)l.chunks * 2 * D * 4);
    return l;
}

moe_status check(int64_t T, int D, int V, float scale, moe_dtype dtype) {
    if (T < 0 || T >= (1ll << 31) || D <= 0 || V <= 0 || (dtype != MOE_F32 && dtype != MOE_BF16)) return MOE_ERR_INVALID_ARG;
    if (!(scale >= -3.4e38f && scale <= 3.4e38f)) return MOE_ERR_INVALID_ARG;
    if (D > kMaxD || V > (1 << 24) || T > (1 << 26)) return MOE_ERR_UNSUPPORTED;
    return MOE_OK;
}

// Each workgroup reads all ids: with 1024 of 32768 entries x 768 17 us against 23 of the
// three launches, of 300 x 64, the smallest tables, 19 against 17.
bool few_tokens(int64_t T) { return T <= kFewTokens; }

template <typename E, typename O, int W>
hipError_t launch_sums(SumArgs a, int64_t chunks, hipStream_t s) {
    // about eight column groups a thread (32768 entries x 768 in bf16: 14.8 us, with
    // four 16.3, with two 19.1)
    // and fewer than 2^32 threads a grid
    const int least = (a.V + (1 << 23) - 1) >> 23;
    a.rows = std::max(least, kFewEntries / (a.D / W));
    a.row_blocks = ((int64_t)a.V + a.rows - 1) / a.rows;
    if (few_tokens(a.T)) {
        // and at least 1024 workgroups, where a few have most of the tokens
        a.rows = std::max(least, std::min(a.rows, a.V >> 10));
        a.row_blocks = ((int64_t)a.V + a.rows - 1) / a.rows;
        embedding_few_kernel<E, O, W><<<(unsigned)a.row_blocks, 256, 0, s>>>(a);
        return hipGetLastError();
    }
    embedding_sum_kernel<E, O, W><<<(unsigned)(a.row_blocks + (chunks + 3) / 4), 256, 0, s>>>(a);
    if (hipError_t e = hipGetLastError()) return e;
    // 4 columns a thread: more loads in flight for the few rows there are
    constexpr int J = W == 8 ? 4 : W;
    if (a.T > kLong) embedding_join_kernel<O, J><<<(unsigned)chunks, 1024, 0, s>>>(a);
    return hipGetLastError();
}

template <typename E, typename O>
hipError_t launch_backward(const SumArgs& a, int64_t chunks, hipStream_t s) {
    // 16 bytes of dy a load where every row begins at a multiple of them; 16 bytes of a
    // table that is written whole (two stores of 16 side by side write half lines: fp32
    // of 65536 x 768 86 us against 51, but added to 30 against 32)
    constexpr int W = Vec<E>::n;
    if constexpr (sizeof(E) < sizeof(O)) {
        if (!a.add && a.D % 4 == 0) return launch_sums<E, O, 4>(a, chunks, s);
    }
    if (a.D % W == 0) return launch_sums<E, O, W>(a, chunks, s);
    return launch_sums<E, O, 1>(a, chunks, s);
}

hipError_t launch_sort(const int32_t* ids, int64_t T, int V, int32_t* order, int32_t* first, int32_t* count, hipStream_t s) {
    // Every workgroup reads every id, so there is one a CU, and more only for more
    // than 1024 entries each.
    int shift = 8;
    while ((int64_t)V > 1024ll << shift) ++shift;
    const unsigned grid = 1u << shift;
    if (V <= 64 << shift) embedding_sort_kernel<6><<<grid, kSortThreads, 0, s>>>(ids, T, V, shift, order, first, count);
    else if (V <= 256 << shift) embedding_sort_kernel<8><<<grid, kSortThreads, 0, s>>>(ids, T, V, shift, order, first, count);
    else embedding_sort_kernel<10><<<grid, kSortThreads, 0, s>>>(ids, T, V, shift, order, first, count);
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
    // and fewer than 2^32 threads a grid (at most 8 rows then, T being 2^26 at most)
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
    SumArgs a = {ids, (const int32_t*)(ws + l.order), (const int32_t*)(ws + l.first), (const int32_t*)(ws + l.count), dy, dtable, (float*)(ws + l.part),
                 T, D, V, scale, accumulate ? 1 : 0, 1, 0};
    (void)hipGetLastError();
    if (!few_tokens(T) && launch_sort(ids, T, V, (int32_t*)(ws + l.order), (int32_t*)(ws + l.first),
                    (int32_t*)(ws + l.count), stream) != hipSuccess) return MOE_ERR_HIP;
    const bool in16 = dtype == MOE_BF16, out16 = table_dtype == MOE_BF16;
    const hipError_t e = in16 && out16 ? launch_backward<uint16_t, uint16_t>(a, l.chunks, stream)
                         : in16        ? launch_backward<uint16_t, float>(a, l.chunks, stream)
                                       : launch_backward<float, float>(a, l.chunks, stream);
    return e == hipSuccess ? MOE_OK : MOE_ERR_HIP;
}

}  // extern "C"
