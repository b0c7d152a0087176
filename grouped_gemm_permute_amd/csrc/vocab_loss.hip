// vocab_loss.hip -- cross entropy and distillation over a large vocabulary
// from the rows h [T, D] in front of it and its table W [V, D], with their
// gradients, without the logits z = h W^T in memory.
//
//   cross entropy   lse[t] = log sum_v exp z[t, v],  loss[t] = lse[t] - z[t, target[t]]
//                   dz[t, v] = g[t] (exp(z[t, v] - lse[t]) - [v = target[t]])
//   distillation    q[t] = softmax over the row's K entries of the teacher's logits / tau
//                   lse[t] = log sum_v exp(z[t, v] / tau)
//                   loss[t] = sum_k q[t, k] (log q[t, k] - z[t, ids[t, k]] / tau) + lse[t]
//                   dz[t, v] = g[t] / tau (exp(z[t, v] / tau - lse[t]) - sum of q[t, k] over ids[t, k] = v)
//   both            dh = dz W,  dW = dz^T h
//
// The forward is one pass of the tile kernel that keeps a largest value and a
// sum for each row and 256 entries, and a small kernel that joins those.  The
// backward makes the logits again, a piece of the vocabulary at a time, turns
// them into dz (at most kDzBytes of it) and multiplies that with W and with h.
// dz is rounded to the operands' precision: three planes of bf16 for fp32
// operands, one for bf16 ones, which takes half a step, up to 2^-8, of each entry, as
// much as rounding a bf16 result does (few rows have two, 16 bits).  Most of a row of
// dz is its target's entry (the teacher's largest), and what the rounding took from
// that one is given back in dh, which is off by 1.0 to 1.3 times what its own rounding
// is (1.4 without).  dW gets nothing back: bf16 is off by 1.0 to 1.4 times its own
// rounding, and fp32 by that of dz alone, 6e-4 to 1.6e-3 of it (512 to 16384 rows of 768
// columns): more planes would be as many more products.
//
// Rows that have no target (prompts, padding) take no part: from kListRows rows
// on the rest are listed first and the products run on those alone; fewer are
// not worth the launch, their dz is zero instead.
#include "mfma_common.h"
#include "vocab_internal.h"

#include "../../include/moe_ffn.h"

#include <algorithm>
#include <cmath>
#include <cstdint>

namespace moe {
namespace {

using namespace mfma;

constexpr size_t kAlign = 256;
constexpr int kMaxD = 16384, kMaxTop = 256;
constexpr int64_t kMaxV = 1 << 24, kMaxT = 1 << 28;
constexpr int64_t kListRows = 1024, kListRowsF32 = 512;
// Whether the products of few rows (vocab_few.hip) are the faster ones: they read the
// table once for 64 rows, the tiles of 128 or 256 rows less often, but those leave
// compute units idle where they are few, and in fp32 they begin with a copy of the
// table in planes.  Measured in us, few rows against tiles, rows x entries x D:
//   bf16 backward  65 x 20000 x 768 58/70, 192 x 20000 x 768 78/78, 256 x 16000 x 768 76/81, 65 x 40000 x 768 91/87,
//                  320 x 16384 x 768 96/83, 192 x 40000 x 768 130/108, 512 x 8000 x 512 68/79, 512 x 20000 x 256 84/81
//   bf16 forward   128 x 32768 x 768 23/26, 65 x 40000 x 768 31/26, 256 x 16000 x 512 18/18, 512 x 16000 x 256 22/15
//   fp32 backward  100 x 65536 x 768 400/479, 150 x 65536 x 768 515/493, 300 x 16000 x 768 253/264, 384 x 20000 x 768 341/308
//   fp32 forward   128 x 65536 x 768 126/220, 256 x 65536 x 768 236/233, 384 x 65536 x 768 345/380, 384 x 8000 x 512 45/76,
//                  40 x 10^7 x 64 1503/4108, 130 x 3 10^6 x 256 2980/3590, 256 x 2 10^6 x 256 2670/2480
bool few_rows(int64_t T, int D, int V, bool f32, bool backward) {
    if (D % (f32 ? 4 : 8)) return false;
    if (T <= 64) return true;
    const int64_t work = (T + 63) / 64 * V * std::max(D, 512);
    if (f32 && backward) return T <= 384 && work <= (T <= 256 ? 1 << 27 : 1 << 26);
    if (f32) return T <= 192 || (T <= 384 && T * V <= (1ll << 31) / 6);
    if (T > 512) return false;
    return work <= (backward ? 7 << 23 : T <= 192 ? 3 << 24 : 1 << 25);
}
// dW of few rows on its own kernel: bf16 always (22 against 48 at 64 rows of 65536 x
// 768); fp32 to 64 rows and for small tables (150 x 8000 x 512 31 against 37, 100 x
// 16000 x 768 36 against 32, 100 x 65536 x 768 126 against 88, 384 x 2000 x 256 63
// against 27).
bool few_dw(int64_t T, int D, int V, bool f32) {
    return !f32 || T <= 64 || (T <= 192 && (T + 63) / 64 * V * D <= 1 << 24);
}
// dz of one piece of the vocabulary: what ordinary steps take whole or in a few
// pieces (32768 rows: 32768 entries), little of 288 GB.
constexpr int64_t kDzBytes = 1ll << 31;
constexpr float kLog2E = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// Rows of one launch of a kernel with up to 256 threads a row: fewer than 2^32 threads
// in a grid.
constexpr int64_t kLaunchRows = 1 << 23;

bool aligned(const void* p, size_t a) { return ((uintptr_t)p & (a - 1)) == 0; }
size_t padded(size_t n) { return (n + kAlign - 1) / kAlign * kAlign; }

__device__ __forceinline__ float to_float(uint16_t v) { return __uint_as_float((uint32_t)v << 16); }
__device__ __forceinline__ float to_float(float v) { return v; }
__device__ __forceinline__ uint16_t to_bf16(float v) { return (uint16_t)pack_bf16(v, 0.f); }

// Whether row t has a target (ids null), or an entry with some probability.
__device__ __forceinline__ bool counts(int32_t id, float logit, int V) {
    return id >= 0 && id < V && !(logit == -INFINITY);
}

struct Targets {
    const int32_t* target;    // [T]; or
    const int32_t* ids;       // [T, K]
    const float* logits;      // [T, K]
    int K, V;
};

__device__ __forceinline__ bool live_row(const Targets& a, int64_t t) {
    if (a.target) return a.target[t] >= 0 && a.target[t] < a.V;
    for (int k = 0; k < a.K; ++k)
        if (counts(a.ids[t * a.K + k], a.logits[t * a.K + k], a.V)) return true;
    return false;
}

// live[t] of a distillation's rows t0.. : a wavefront a row.
__global__ __launch_bounds__(256) void vocab_live_kernel(const Targets a, int64_t t0, int64_t T, int32_t* __restrict__ live) {
    const int64_t t = t0 + (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
    const int lane = threadIdx.x & 63;
    if (t >= T) return;
    bool any = false;
    for (int k = lane; k < a.K; k += 64) any |= counts(a.ids[t * a.K + k], a.logits[t * a.K + k], a.V);
    const uint64_t m = __ballot(any);
    if (lane == 0) live[t] = m != 0;
}

// Which of rows t .. t + 3 count, those that are there (less than T).
__device__ __forceinline__ int four_rows(const int32_t* target, const int32_t* live, int V, int64_t t, int64_t T) {
    const int32_t* p = (target ? target : live) + t;
    int in = 0;
    auto look = [&](int32_t x, int j) { in |= (target ? x >= 0 && x < V : x != 0) << j; };
    if (t + 4 <= T) {
        int32_t x[4];
        __builtin_memcpy(x, p, 16);
#pragma unroll
        for (int j = 0; j < 4; ++j) look(x[j], j);
    } else {
        for (int j = 0; t + j < T; ++j) look(p[j], j);
    }
    return in;
}

// How many rows of each chunk count.
constexpr int kListChunk = 4096;
__global__ __launch_bounds__(1024) void vocab_count_kernel(const int32_t* __restrict__ target, const int32_t* __restrict__ live,
                                                           int V, int64_t T, int32_t* __restrict__ counts) {
    __shared__ int32_t sums[16];
    const int tid = threadIdx.x;
    int n = __popc(four_rows(target, live, V, (int64_t)blockIdx.x * kListChunk + 4 * tid, T));
    for (int d = 32; d; d >>= 1) n += __shfl_xor(n, d);
    if ((tid & 63) == 0) sums[tid >> 6] = n;
    __syncthreads();
    if (tid) return;
    for (int w = 1; w < 16; ++w) n += sums[w];
    counts[blockIdx.x] = n;
}

// The rows that count, in order: rows[0 .. *count), and pos[t], a row's place
// among them or -1.  A workgroup lists kListChunk rows; of up to kListCounted it
// counts those before them itself, in one launch (32768 rows: 0.5 MB read by 8
// workgroups, 7.8 us against 6.0 and 2.6 for the counts), and of more it takes `counts`,
// since that work grows with T^2 (65536 rows 11 us against 6.1 and 2.6, 131072 18 against
// 5.9 and 4.1, 2^22 745 against 26 and 6).  zero0, zero1 (or null): set to 0 for the
// other rows.
constexpr int64_t kListCounted = 1 << 15;
__global__ __launch_bounds__(1024) void vocab_list_kernel(const int32_t* __restrict__ target, const int32_t* __restrict__ live,
                                                          int V, int64_t T, const int32_t* __restrict__ counts,
                                                          int32_t* __restrict__ rows, int32_t* __restrict__ pos,
                                                          int32_t* __restrict__ count, float* zero0, float* zero1) {
    __shared__ int32_t sums[2][16];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int64_t base = (int64_t)blockIdx.x * kListChunk, t0 = base + 4 * tid;
    int before = 0;
    if (counts) {
#pragma unroll 4
        for (int c = tid; c < (int)blockIdx.x; c += 1024) before += counts[c];
    } else {
#pragma unroll 4
        for (int64_t t = 4 * tid; t < base; t += 4096) before += __popc(four_rows(target, live, V, t, base));
    }
    const int in = four_rows(target, live, V, t0, T);
    const int mine = __popc(in);
    int incl = mine;
    for (int d = 1; d < 64; d <<= 1) {
        const int o = __shfl_up(incl, d);
        if (lane >= d) incl += o;
    }
    for (int d = 32; d; d >>= 1) before += __shfl_xor(before, d);
    if (lane == 63) sums[0][wave] = incl, sums[1][wave] = before;
    __syncthreads();
    int place = incl - mine, n = 0;
    for (int w = 0; w < 16; ++w) {
        if (w < wave) place += sums[0][w];
        place += sums[1][w];
        n += sums[0][w] + sums[1][w];
    }
    for (int j = 0; j < 4 && t0 + j < T; ++j) {
        const int64_t t = t0 + j;
        if (in >> j & 1) {
            rows[place] = (int32_t)t;
            pos[t] = place++;
        } else {
            pos[t] = -1;
            if (zero0) zero0[t] = 0.f;
            if (zero1) zero1[t] = 0.f;
        }
    }
    if (tid == 0 && base + kListChunk >= T) *count = n;
}

// The backward's rows: row t of h to row pos[t] of the copy, as bf16 (one plane)
// or as three bf16 planes whose sum it is, zeros behind its D columns; g / tau
// and lse beside it.  Without pos every row is copied to its own place, those
// that do not count as zeros with a dz of zero.  With pos those rows' dh is
// written here, as zeros.
struct CopyArgs {
    const void* src;
    int64_t T;
    int D, Dp;
    uint16_t* dst;
    int64_t plane;
    const int32_t* pos;
    Targets targets;          // rows that count (pos null); target and ids null: all
    const int32_t* count;     // rows in the copy (with pos)
    const float *g, *lse;     // [T], or null
    float inv_tau;
    float *g_out, *lse_out;
    float4* info;             // g / tau, lse and the target's bits, or null
    int32_t* entry;           // the target, or null
    void* dh;                 // or null
};

template <typename E>
__global__ __launch_bounds__(256) void vocab_copy_kernel(const CopyArgs a) {
    const int lane = threadIdx.x & 63;
    // behind the last row zeros up to the next multiple of 32
    const int64_t n = a.count ? *a.count : a.T, end = (n + 31) / 32 * 32;
    for (int64_t t = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); t < a.T + 32; t += (int64_t)gridDim.x * 4) {
        int64_t to = t;
        bool live = true;
        if (t >= a.T) {
            to = n + (t - a.T);
            live = false;
            if (to >= end) break;
        } else if (a.pos) {
            to = a.pos[t];
            live = to >= 0;
            if (!live) {
                if (a.dh)
                    for (int c = lane; c < a.D; c += 64) ((E*)a.dh)[t * a.D + c] = E(0);
                continue;
            }
        } else if (a.targets.target || a.targets.ids) {
            if (a.targets.target) {
                live = live_row(a.targets, t);
            } else {
                bool any = false;
                for (int k = lane; k < a.targets.K; k += 64)
                    any |= counts(a.targets.ids[t * a.targets.K + k], a.targets.logits[t * a.targets.K + k], a.targets.V);
                live = __ballot(any) != 0;
            }
        }
        if (lane == 0 && t < a.T && (a.g || a.info)) {
            const float g = a.g && live ? a.g[t] * a.inv_tau : 0.f, lse = a.lse && live ? a.lse[t] : INFINITY;
            const int target = a.targets.target && live ? a.targets.target[t] : -1;
            if (a.entry) a.entry[to] = target;
            if (a.info) a.info[to] = make_float4(g, lse, __int_as_float(target), 0.f);
            if (a.g_out) {
                a.g_out[to] = g;
                a.lse_out[to] = lse;
            }
        }
        const E* src = (const E*)a.src + t * a.D;
        uint16_t* dst = a.dst + to * a.Dp;
        if (a.D % 8 == 0) {
            for (int c = 8 * lane; c < a.Dp; c += 512) {
                float x[8];
                if (c < a.D && live) {
                    if constexpr (sizeof(E) == 2) {
                        *(u32x4_t*)(dst + c) = *(const u32x4_t*)(src + c);
                        continue;
                    } else {
                        *(float4*)x = *(const float4*)(src + c);
                        *(float4*)(x + 4) = *(const float4*)(src + c + 4);
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < 8; ++i) x[i] = 0.f;
                }
#pragma unroll
                for (int pl = 0; pl < (sizeof(E) == 2 ? 1 : 3); ++pl) {
                    u32x4_t o;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        o[i] = pack_bf16(x[2 * i], x[2 * i + 1]);
                        x[2 * i] -= __uint_as_float(o[i] << 16);
                        x[2 * i + 1] -= __uint_as_float(o[i] & 0xffff0000u);
                    }
                    *(u32x4_t*)(dst + pl * a.plane + c) = o;
                }
            }
        } else {
            for (int c = lane; c < a.Dp; c += 64) {
                float x = c < a.D && live ? to_float(src[c]) : 0.f;
#pragma unroll
                for (int pl = 0; pl < (sizeof(E) == 2 ? 1 : 3); ++pl) {
                    const uint16_t o = to_bf16(x);
                    dst[pl * a.plane + c] = o;
                    x -= to_float(o);
                }
            }
        }
    }
}

// Joins the tiles' largest values and sums: LANES threads a row, each over every
// LANESth tile, then 16 of them over theirs.  Few rows of many tiles have a quarter of
// a workgroup or all of one each (of 131072 entries, one row 8.3 us with 16 lanes, 4.2
// with 256, 100 rows 5.9 and with 64 4.2; 1000 rows of 32768 4.4 and 4.7).
struct FinishArgs {
    const float2* part;
    int64_t pitch;
    int n_tiles;
    VocabRows rows;
    Targets targets;
    float c;
    const float* zt;          // cross entropy: the targets' logits
    float *loss, *lse;        // [T]; loss null: lse alone
    int64_t first;            // of the launch's (compact) rows
};

template <int LANES>
__global__ __launch_bounds__(256) void vocab_finish_kernel(const FinishArgs a) {
    constexpr int ROWS = 256 / LANES;
    __shared__ float2 sums[LANES][ROWS + 1];
    const int r = threadIdx.x % ROWS, sl = threadIdx.x / ROWS;
    const int64_t n = a.rows.count ? *a.rows.count : a.rows.T;
    const int64_t i = a.first + (int64_t)blockIdx.x * ROWS + r;
    if (i - r >= n) return;
    auto join = [](float2 x, float2 y) {
        const float m = fmaxf(x.x, y.x), off = m == -INFINITY ? 0.f : m;
        return make_float2(m, x.y * __builtin_amdgcn_exp2f(x.x - off) + y.y * __builtin_amdgcn_exp2f(y.x - off));
    };
    float2 sum = make_float2(-INFINITY, 0.f);
    if (i < n) {
#pragma unroll 4
        for (int k = sl; k < a.n_tiles; k += LANES) sum = join(sum, a.part[k * a.pitch + i]);
    }
    sums[sl][r] = sum;
    __syncthreads();
    // of more than 16, each of the first 16 has every 16th
    if constexpr (LANES > 16) {
        if (sl < 16) {
            for (int k = sl + 16; k < LANES; k += 16) sum = join(sum, sums[k][r]);
        }
        __syncthreads();
        if (sl < 16) sums[sl][r] = sum;
        __syncthreads();
    }
    if (sl || i >= n) return;
    float m = -INFINITY;
    for (int k = 0; k < 16; ++k) m = fmaxf(m, sums[k][r].x);
    const float off = m == -INFINITY ? 0.f : m;
    float s = 0.f;
    for (int k = 0; k < 16; ++k) s += sums[k][r].y * __builtin_amdgcn_exp2f(sums[k][r].x - off);
    const int64_t t = a.rows.rows ? a.rows.rows[i] : i;
    const bool live = a.rows.rows || live_row(a.targets, t);
    const float l = __builtin_amdgcn_logf(s);       // log2
    a.lse[t] = live ? (off + l) * kLn2 : 0.f;
    // the two large terms first: their difference is exact where the target leads
    if (a.loss) a.loss[t] = live ? (l + (off - a.zt[i] * a.c)) * kLn2 : 0.f;
}

// A teacher's row in LDS: q and log q of its K entries (0 for those that do not
// count); true if any counts.  Called by the whole first wavefront.
__device__ __forceinline__ bool teacher_row(const Targets& a, int64_t t, float inv_tau, float* q, float* logq, int32_t* id) {
    const int lane = threadIdx.x & 63;
    float top = -INFINITY;
    bool any = false, nan = false;
    for (int k = lane; k < a.K; k += 64) {
        const int32_t v = a.ids[t * a.K + k];
        const float x = a.logits[t * a.K + k];
        const bool in = counts(v, x, a.V);
        id[k] = in ? v : -1;
        logq[k] = x;
        if (in) {
            any = true;
            nan |= x != x;
            top = fmaxf(top, x);
        }
    }
    for (int d = 32; d; d >>= 1) top = fmaxf(top, __shfl_xor(top, d));
    if (__ballot(nan)) top = NAN;
    float sum = 0.f;
    for (int k = lane; k < a.K; k += 64) {
        // differences first: logits of the lowest value stay finite at any tau
        const float x = (logq[k] - top) * inv_tau, e = id[k] >= 0 ? expf(x) : 0.f;
        logq[k] = x;
        q[k] = e;
        sum += e;
    }
    for (int d = 32; d; d >>= 1) sum += __shfl_xor(sum, d);
    const float l = logf(sum);
    for (int k = lane; k < a.K; k += 64) {
        const bool in = id[k] >= 0;
        q[k] = in ? q[k] / sum : 0.f;
        logq[k] = in ? logq[k] - l : 0.f;
    }
    return __ballot(any) != 0;
}

// z[t, k] = h[t] . W[ids[t, k]] and the row's loss: a workgroup a row, 16 lanes
// an entry.  Gathers T K rows of the table, most of them from the last-level
// cache.
struct TopArgs {
    const void *h, *W;
    Targets targets;
    int D;
    float inv_tau;
    const float* lse;
    float *loss, *z;
    int64_t first;            // of the launch's rows
};

template <typename E, bool VEC>
__global__ __launch_bounds__(256) void vocab_top_kernel(const TopArgs a) {
    __shared__ float q[kMaxTop], logq[kMaxTop], zs[kMaxTop];
    __shared__ int32_t id[kMaxTop];
    const int64_t t = a.first + blockIdx.x;
    const int tid = threadIdx.x, K = a.targets.K;
    const E* h = (const E*)a.h + t * a.D;
    bool live = false;
    if (tid < 64) live = teacher_row(a.targets, t, a.inv_tau, q, logq, id);
    __syncthreads();
    const int sub = tid & 15;
    for (int k = tid >> 4; k < K; k += 16) {
        const int32_t v = a.targets.ids[t * K + k];
        float s = 0.f;
        if (v >= 0 && v < a.targets.V) {
            const E* w = (const E*)a.W + (int64_t)v * a.D;
            if constexpr (VEC) {
                constexpr int n = 16 / sizeof(E);
#pragma unroll 4
                for (int c = n * sub; c < a.D; c += 16 * n) {
                    const u32x4_t x = *(const u32x4_t*)(w + c), y = *(const u32x4_t*)(h + c);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        if constexpr (sizeof(E) == 2) {
                            s = fmaf(__uint_as_float(x[i] << 16), __uint_as_float(y[i] << 16), s);
                            s = fmaf(__uint_as_float(x[i] & 0xffff0000u), __uint_as_float(y[i] & 0xffff0000u), s);
                        } else {
                            s = fmaf(__uint_as_float(x[i]), __uint_as_float(y[i]), s);
                        }
                    }
                }
            } else {
                for (int c = sub; c < a.D; c += 16) s = fmaf(to_float(w[c]), to_float(h[c]), s);
            }
        }
        for (int d = 8; d; d >>= 1) s += __shfl_xor(s, d, 16);
        if (sub == 0) {
            zs[k] = s;
            a.z[t * K + k] = s;
        }
    }
    __syncthreads();
    if (tid >= 64) return;
    float sum = 0.f;
    for (int k = tid; k < K; k += 64)
        if (!(q[k] == 0.f)) sum += q[k] * (logq[k] - zs[k] * a.inv_tau);
    for (int d = 32; d; d >>= 1) sum += __shfl_xor(sum, d);
    if (tid == 0) a.loss[t] = live ? sum + a.lse[t] : 0.f;
}

// The teacher's share of dz: entries of the piece that a row's ids name are
// written anew, g / tau (exp(z / tau - lse) - q) from the z of the forward, q
// summed over ids that name the same one.  A wavefront a row.
struct TeacherArgs {
    Targets targets;
    VocabRows rows;
    const float *z;           // [T, K]
    const float *g, *lse;     // of compact rows; g already divided by tau
    float inv_tau;
    int64_t v0;
    int len;
    uint16_t* dz;
    int64_t pitch, plane;
    int planes;
    float* dz32;              // the same in fp32, or null
    float* err;               // or null: what rounding takes from the largest of the
    int32_t* entry;           // row's entries, and which it is (see VocabGrad)
    int64_t first;            // of the launch's (compact) rows
};

__global__ __launch_bounds__(64) void vocab_teacher_kernel(const TeacherArgs a) {
    __shared__ float q[kMaxTop], logq[kMaxTop];
    __shared__ int32_t id[kMaxTop];
    const int64_t i = a.first + blockIdx.x;
    if (i >= (a.rows.count ? *a.rows.count : a.rows.T)) return;
    const int64_t t = a.rows.rows ? a.rows.rows[i] : i;
    const int K = a.targets.K, lane = threadIdx.x;
    const bool some = teacher_row(a.targets, t, a.inv_tau, q, logq, id);
    __syncthreads();
    const float g = a.g[i], lse = a.lse[i];
    const bool first_piece = a.err && a.v0 == 0;
    float most = -1.f, rest = 0.f;
    int which = -1;
    for (int k = lane; some && k < K; k += 64) {
        const int32_t v = id[k];
        const bool here = v >= a.v0 && v < a.v0 + a.len;
        if (v < 0 || !(here || first_piece)) continue;
        float share = 0.f;
        bool first = true;
        for (int o = 0; o < K; ++o) {
            if (id[o] != v) continue;
            if (o < k) first = false;
            share += q[o];
        }
        if (!first) continue;
        float x = g * (exp_fp32(fmaf(a.z[t * K + k], a.inv_tau, -lse)) - share);
        if (fabsf(x) > most) {
            most = fabsf(x);
            rest = x - to_float(to_bf16(x));
            which = v;
        }
        if (!here) continue;
        uint16_t* p = a.dz + i * a.pitch + (v - a.v0);
        if (a.dz32) a.dz32[i * a.pitch + (v - a.v0)] = x;
        for (int pl = 0; pl < a.planes; ++pl) {
            const uint16_t o = to_bf16(x);
            p[pl * a.plane] = o;
            x -= to_float(o);
        }
    }
    if (!first_piece) return;
    for (int d = 32; d; d >>= 1) {
        const float m = __shfl_xor(most, d), r = __shfl_xor(rest, d);
        const int w = __shfl_xor(which, d);
        // the lower entry where two are alike, so that all lanes agree
        if (m > most || (m == most && w < which)) most = m, rest = r, which = w;
    }
    if (lane == 0) {
        a.err[i] = rest;
        a.entry[i] = which;
    }
}

template <typename O>
__global__ __launch_bounds__(256) void vocab_zero_kernel(O* p, int64_t n) {
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) p[i] = O(0);
}

// ---- plan and workspace

struct Plan {
    bool list;                // rows that count are listed first
    bool whole;               // logits by 256 x 256 tiles
    bool few, few_dw;         // the products of few rows, dW's among them
    bool copy_W, copy_h;      // operands as padded bf16 planes
    int planes, products, Dp;
    int dz_planes;
    bool give_back;           // what rounding takes from a row's largest entry of dz
    int64_t n_tiles;          // stats: column tiles
    int64_t piece, pieces;    // entries of a piece (a multiple of 256), and how many
    int64_t pitch;            // elements between rows of its dz
    size_t rows, pos, count, counts, live, hc, info, Wc, part, zt, g, lse, err, entry, dz, dz32, dh_part, acc, total;
};

// Whether rows that are not listed take the tiles of 256 x 256 (one workgroup a CU)
// rather than those of 128 x 256 (two): where there is one for every CU and the last
// row tile is more than half full.  Measured, bf16, forward with the copy of h that
// they need, and dz: 512 rows of 32768 x 768 36 us against 38 and 31 against 38, 768
// of 65536 82 against 93 and 105 against 126; 640 of 50001 74 against 65 and 72
// against 67 (half full), 1000 of 8000 x 1024 38 against 31 (half the CUs).
bool whole_tiles(int64_t T, int V) {
    return (T - 1) % 256 >= 128 && (T + 255) / 256 * ((V + kVocabTileCols - 1) / kVocabTileCols) >= 256;
}

Plan plan_of(int64_t T, int D, int V, int K, moe_dtype dtype, bool backward) {
    Plan p = {};
    p.list = T >= (dtype == MOE_BF16 ? kListRows : kListRowsF32);
    p.planes = dtype == MOE_BF16 ? 1 : 3;
    p.products = dtype == MOE_BF16 ? 1 : 6;
    const bool f32 = dtype != MOE_BF16;
    p.few = few_rows(T, D, V, f32, backward);
    p.few_dw = p.few && few_dw(T, D, V, f32);
    // bf16 rows of whole K steps are read where they are
    p.copy_W = !p.few && (f32 || D % 32 != 0);
    const bool many = p.list || (!p.few && whole_tiles(T, V));
    p.copy_h = p.copy_W || many || backward;
    p.dz_planes = p.few && !f32 ? 2 : p.planes;
    p.give_back = p.dz_planes == 1 && D % 4 == 0;
    // what is copied is padded to what the tiles of many rows take
    const int unit = p.copy_W && many ? 128 : 32;
    p.Dp = (D + unit - 1) / unit * unit;
    p.whole = many && p.Dp % 128 == 0;
    p.n_tiles = ((int64_t)V + kVocabTileCols - 1) / kVocabTileCols;
    if (p.few && !backward) p.n_tiles = ((int64_t)V + vocab_few_cols(T, V) - 1) / vocab_few_cols(T, V);
    size_t at = 0;
    auto take = [&](bool want, size_t bytes) {
        const size_t o = at;
        if (want) at += padded(bytes);
        return o;
    };
    p.rows = take(p.list, (size_t)T * 4);
    p.pos = take(p.list, (size_t)T * 4);
    p.count = take(p.list, 4);
    p.counts = take(p.list && T > kListCounted, (size_t)((T + kListChunk - 1) / kListChunk) * 4);
    p.live = take(p.list && K > 0, (size_t)T * 4);
    p.hc = take(p.copy_h, (size_t)p.planes * (T + 32) * p.Dp * 2);
    p.info = take(p.whole, (size_t)T * 16);
    p.Wc = take(p.copy_W, (size_t)p.planes * (V + 32ll) * p.Dp * 2);
    if (!backward) {
        p.part = take(true, (size_t)p.n_tiles * T * 8);
        p.zt = take(K == 0, (size_t)T * 4);
    } else {
        const int64_t tile = kVocabTileCols;
        // bytes of an entry of dz: its planes, or of few fp32 rows fp32 and what planes dW's tiles read
        const int64_t each = !p.few || !f32 ? 2 * p.dz_planes : p.few_dw ? 4 : 4 + 2 * p.dz_planes;
        // tiles of a piece
        const int64_t most = std::min(std::max<int64_t>(1, kDzBytes / (T * each) / tile), kVocabGradTiles / ((D + 255) / 256));
        p.pieces = (p.n_tiles + most - 1) / most;
        p.piece = (p.n_tiles + p.pieces - 1) / p.pieces * tile;
        p.pieces = (p.n_tiles * tile + p.piece - 1) / p.piece;
        p.g = take(true, (size_t)T * 4);
        p.lse = take(true, (size_t)T * 4);
        p.err = take(p.give_back, (size_t)T * 4);
        p.entry = take(p.give_back, (size_t)T * 4);
        // an odd number of 512 bytes: rows 2^n bytes apart meet in a few of the memory's
        // channels (131072 bytes: dz 1318 us, 131584: 1150)
        p.pitch = (p.piece / 256 | 1) * 256;
        p.dz = take(!f32 || !p.few_dw, (size_t)p.dz_planes * T * p.pitch * 2);
        p.dz32 = take(p.few && f32, (size_t)T * p.pitch * 4);
        p.dh_part = take(p.few, (size_t)(p.few ? p.pieces * vocab_few_splits(T, D, p.pieces > 1 ? (int)p.piece : V, f32) : 0) * T * D * 4);
        p.part = take(!p.few_dw, vocab_grad_partial_bytes(D));
        p.acc = take(p.pieces > 1 && !p.few, (size_t)T * p.Dp * 4);
    }
    p.total = at;
    return p;
}

struct Call {
    const void *h, *W;
    Targets targets;
    int64_t T;
    int D;
    float tau;
    moe_dtype dtype;
};

moe_status check(const Call& a) {
    if (a.T < 0 || a.D <= 0 || a.targets.V <= 0 || (a.dtype != MOE_F32 && a.dtype != MOE_BF16)) return MOE_ERR_INVALID_ARG;
    // log2(e) / tau, the forward's factor, is finite
    if (!(a.tau > 0.f) || a.tau > 3.4e38f || kLog2E / a.tau > 3.4e38f) return MOE_ERR_INVALID_ARG;
    if (a.D > kMaxD || a.targets.V > kMaxV || a.T > kMaxT || a.targets.K > kMaxTop) return MOE_ERR_UNSUPPORTED;
    // workgroups of a grid
    const int64_t t = (a.T + 127) / 128, v = (a.targets.V + 255) / 256, d = (a.D + 255) / 256;
    if (t * v > (1 << 22) || t * d > (1 << 22) || v * d > (1 << 22)) return MOE_ERR_UNSUPPORTED;
    return MOE_OK;
}

#define TRY(x)                                     \
    do {                                           \
        if ((x) != hipSuccess) return MOE_ERR_HIP; \
    } while (0)

// One launch after the other over T rows: launch(first row, rows).
template <typename L>
hipError_t by_rows(int64_t T, L&& launch) {
    for (int64_t t = 0; t < T; t += kLaunchRows) {
        launch(t, std::min(kLaunchRows, T - t));
        if (hipError_t e = hipGetLastError()) return e;
    }
    return hipSuccess;
}

hipError_t copy_rows(const CopyArgs& a, moe_dtype dtype, hipStream_t s) {
    const unsigned grid = (unsigned)std::min<int64_t>((a.T + 32 + 3) / 4, 8192);
    if (dtype == MOE_BF16) vocab_copy_kernel<uint16_t><<<grid, 256, 0, s>>>(a);
    else vocab_copy_kernel<float><<<grid, 256, 0, s>>>(a);
    return hipGetLastError();
}

// The list of rows and the table's planes, where the plan has them.
moe_status begin(const Call& a, const Plan& p, char* ws, VocabRows* rows, VocabOperand* W, float* zero0, float* zero1,
                 hipStream_t s) {
    *rows = {nullptr, nullptr, a.T};
    if (p.list) {
        int32_t* live = (int32_t*)(ws + p.live);
        if (!a.targets.target) {
            TRY(by_rows(a.T, [&](int64_t t, int64_t n) {
                vocab_live_kernel<<<(unsigned)((n + 3) / 4), 256, 0, s>>>(a.targets, t, a.T, live);
            }));
        }
        *rows = {(const int32_t*)(ws + p.rows), (const int32_t*)(ws + p.count), a.T};
        const unsigned chunks = (unsigned)((a.T + kListChunk - 1) / kListChunk);
        int32_t* counts = a.T > kListCounted ? (int32_t*)(ws + p.counts) : nullptr;
        if (counts) {
            vocab_count_kernel<<<chunks, 1024, 0, s>>>(a.targets.target, live, a.targets.V, a.T, counts);
            TRY(hipGetLastError());
        }
        vocab_list_kernel<<<chunks, 1024, 0, s>>>(a.targets.target, live, a.targets.V, a.T, counts, (int32_t*)(ws + p.rows),
                                            (int32_t*)(ws + p.pos), (int32_t*)(ws + p.count), zero0, zero1);
        TRY(hipGetLastError());
    }
    *W = {(const uint16_t*)a.W, a.D, 0};
    if (p.copy_W) {
        uint16_t* to = (uint16_t*)(ws + p.Wc);
        *W = {to, p.Dp, (a.targets.V + 32ll) * p.Dp};
        CopyArgs c = {a.W, a.targets.V, a.D, p.Dp, to, W->plane};
        TRY(copy_rows(c, a.dtype, s));
    }
    return MOE_OK;
}

moe_status forward(const Call& a, float* loss, float* lse, float* z, void* workspace, size_t ws_bytes, hipStream_t s) {
    if (a.T == 0) return MOE_OK;
    const Plan p = plan_of(a.T, a.D, a.targets.V, a.targets.K, a.dtype, false);
    if (!workspace || !aligned(workspace, kAlign)) return MOE_ERR_INVALID_ARG;
    if (ws_bytes < p.total) return MOE_ERR_WORKSPACE;
    char* ws = (char*)workspace;
    (void)hipGetLastError();
    VocabRows rows;
    VocabOperand W, h = {(const uint16_t*)a.h, a.D, 0};
    if (const moe_status st = begin(a, p, ws, &rows, &W, lse, a.targets.target ? loss : nullptr, s)) return st;
    if (p.copy_h) {
        uint16_t* to = (uint16_t*)(ws + p.hc);
        h = {to, p.Dp, (a.T + 32) * p.Dp};
        CopyArgs c = {a.h, a.T, a.D, p.Dp, to, h.plane};
        if (p.list) c.pos = (const int32_t*)(ws + p.pos), c.count = rows.count;
        if (p.whole) c.targets = a.targets, c.info = (float4*)(ws + p.info);
        TRY(copy_rows(c, a.dtype, s));
    }
    const float inv_tau = 1.f / a.tau;
    VocabStats st = {h, W, rows, a.targets.V, p.Dp, p.products, kLog2E * inv_tau,
                     (float2*)(ws + p.part), a.T, a.targets.target, (float*)(ws + p.zt)};
    if (p.few) {
        VocabFew w = {a.dtype != MOE_BF16, a.h, a.W, a.D, a.T, a.D, a.targets.V, st.c, a.targets.target, st.part, a.T, st.zt};
        TRY(launch_vocab_few_stats(w, s));
    } else
        TRY(p.whole ? launch_vocab_stats_whole(st, (const float4*)(ws + p.info), s) : launch_vocab_stats(st, s));
    FinishArgs f = {st.part, a.T, (int)p.n_tiles, rows, a.targets, st.c, st.zt, a.targets.target ? loss : nullptr, lse};
    TRY(by_rows(a.T, [&](int64_t t, int64_t n) {
        f.first = t;
        if (a.T <= 64 && f.n_tiles > 64) vocab_finish_kernel<256><<<(unsigned)n, 256, 0, s>>>(f);
        else if (a.T <= 512 && f.n_tiles > 64) vocab_finish_kernel<64><<<(unsigned)((n + 3) / 4), 256, 0, s>>>(f);
        else vocab_finish_kernel<16><<<(unsigned)((n + 15) / 16), 256, 0, s>>>(f);
    }));
    if (!a.targets.target) {
        TopArgs t = {a.h, a.W, a.targets, a.D, inv_tau, lse, loss, z};
        TRY(by_rows(a.T, [&](int64_t first, int64_t n) {
            t.first = first;
            const unsigned grid = (unsigned)n;
            if (a.dtype == MOE_BF16) {
                if (a.D % 8 == 0) vocab_top_kernel<uint16_t, true><<<grid, 256, 0, s>>>(t);
                else vocab_top_kernel<uint16_t, false><<<grid, 256, 0, s>>>(t);
            } else {
                if (a.D % 4 == 0) vocab_top_kernel<float, true><<<grid, 256, 0, s>>>(t);
                else vocab_top_kernel<float, false><<<grid, 256, 0, s>>>(t);
            }
        }));
    }
    return MOE_OK;
}

moe_status backward(const Call& a, const float* z, const float* lse, const float* dloss, void* dh, void* dW,
                    moe_dtype dW_dtype, void* workspace, size_t ws_bytes, hipStream_t s) {
    const int V = a.targets.V;
    if (a.T == 0) {
        if (!dW) return MOE_OK;
        const int64_t n = (int64_t)V * a.D;
        const unsigned grid = (unsigned)std::min<int64_t>((n + 255) / 256, 65536);
        (void)hipGetLastError();
        if (dW_dtype == MOE_BF16) vocab_zero_kernel<<<grid, 256, 0, s>>>((uint16_t*)dW, n);
        else vocab_zero_kernel<<<grid, 256, 0, s>>>((float*)dW, n);
        TRY(hipGetLastError());
        return MOE_OK;
    }
    const Plan p = plan_of(a.T, a.D, V, a.targets.K, a.dtype, true);
    if (dh && !p.few && vocab_grad_tiles(a.T, a.D) > kVocabGradTiles) return MOE_ERR_UNSUPPORTED;
    if (!workspace || !aligned(workspace, kAlign)) return MOE_ERR_INVALID_ARG;
    if (ws_bytes < p.total) return MOE_ERR_WORKSPACE;
    char* ws = (char*)workspace;
    (void)hipGetLastError();
    VocabRows rows;
    VocabOperand W;
    if (const moe_status st = begin(a, p, ws, &rows, &W, nullptr, nullptr, s)) return st;
    const float inv_tau = 1.f / a.tau;
    float *g = (float*)(ws + p.g), *l = (float*)(ws + p.lse);
    VocabOperand h = {(const uint16_t*)(ws + p.hc), p.Dp, (a.T + 32) * p.Dp};
    {
        CopyArgs c = {a.h, a.T, a.D, p.Dp, (uint16_t*)(ws + p.hc), h.plane};
        if (p.list) c.pos = (const int32_t*)(ws + p.pos), c.count = rows.count;
        if (p.whole) c.info = (float4*)(ws + p.info);
        if (p.give_back) c.entry = (int32_t*)(ws + p.entry);
        c.targets = a.targets;
        c.g = dloss, c.lse = lse, c.inv_tau = inv_tau, c.g_out = g, c.lse_out = l;
        c.dh = dh;
        TRY(copy_rows(c, a.dtype, s));
    }
    uint16_t* dz = (uint16_t*)(ws + p.dz);
    const int64_t dz_plane = a.T * p.pitch;
    const bool h16 = a.dtype == MOE_BF16;
    int parts = 0;            // of few rows' dh
    for (int64_t v0 = 0; v0 < V; v0 += p.piece) {
        const int len = (int)std::min<int64_t>(p.piece, V - v0);
        const VocabDz d = {h, W, rows, V, v0, len, p.Dp, p.products, inv_tau, g, l, a.targets.target, dz, p.pitch, dz_plane,
                           p.give_back ? (float*)(ws + p.err) : nullptr};
        VocabFew w = {!h16, h16 ? (const void*)h.p : a.h, (const char*)a.W + v0 * a.D * (h16 ? 2 : 4), h16 ? h.pitch : a.D,
                      a.T, a.D, len, inv_tau, a.targets.target};
        w.v0 = v0;
        w.g = g, w.lse = l;
        // of fp32 operands, planes only for a dW by tiles
        const bool planes = !p.few || h16 || (dW && !p.few_dw);
        w.dz = planes ? dz : nullptr, w.dz32 = p.few && !h16 ? (float*)(ws + p.dz32) : nullptr;
        w.dz_pitch = p.pitch, w.dz_plane = dz_plane;
        w.dh_part = (float*)(ws + p.dh_part) + (int64_t)parts * a.T * a.D;
        if (p.few) TRY(launch_vocab_few_dz(w, s));
        else TRY(p.whole ? launch_vocab_dz_whole(d, (const float4*)(ws + p.info), s) : launch_vocab_dz(d, s));
        if (!a.targets.target) {
            TeacherArgs t = {a.targets, rows, z, g, l, inv_tau, v0, len, dz, p.pitch, dz_plane, planes ? p.dz_planes : 0, w.dz32,
                             d.err, (int32_t*)(ws + p.entry)};
            TRY(by_rows(a.T, [&](int64_t first, int64_t n) {
                t.first = first;
                vocab_teacher_kernel<<<(unsigned)n, 64, 0, s>>>(t);
            }));
        }
        VocabGrad q = {};
        q.m = {dz, p.pitch, dz_plane};
        q.rows = rows;
        q.len = len;
        q.N = a.D;
        q.products = p.products;
        q.partial = (float*)(ws + p.part);
        if (dh && p.few) {
            TRY(launch_vocab_few_dh(w, s));
            parts += vocab_few_splits(a.T, a.D, len, !h16);
            if (v0 + p.piece >= V) TRY(launch_vocab_few_sum((const float*)(ws + p.dh_part), parts, a.T, a.D, h16, dh, s));
        } else if (dh) {
            q.dW = false;
            q.n = {W.p + v0 * W.pitch, W.pitch, W.plane};
            q.acc = p.pieces > 1 ? (float*)(ws + p.acc) : nullptr;
            q.acc_pitch = p.Dp;
            q.add = v0 > 0;
            q.last = v0 + p.piece >= V;
            q.out = dh;
            q.out_bf16 = h16;
            q.err = d.err;
            q.entry = (const int32_t*)(ws + p.entry);
            q.table = (const uint16_t*)a.W, q.table_pitch = a.D;
            TRY(launch_vocab_grad(q, s));
        }
        if (dW && p.few_dw) {
            const bool out16 = dW_dtype == MOE_BF16;
            TRY(launch_vocab_few_dw(w, (char*)dW + v0 * a.D * (out16 ? 2 : 4), out16, s));
        } else if (dW) {
            q.dW = true;
            q.err = nullptr;
            q.n = h;
            q.acc = nullptr;
            q.add = false;
            q.last = true;
            q.out_bf16 = dW_dtype == MOE_BF16;
            q.out = q.out_bf16 ? (void*)((uint16_t*)dW + v0 * a.D) : (void*)((float*)dW + v0 * a.D);
            TRY(launch_vocab_grad(q, s));
        }
    }
    return MOE_OK;
}

Call call_of(const void* h, const void* W, const int32_t* target, const int32_t* ids, const float* logits, int64_t T, int D,
             int V, int K, float tau, moe_dtype dtype) {
    return {h, W, {target, ids, logits, K, V}, T, D, tau, dtype};
}

// Pointers: 16 bytes for arrays of dtype, 4 for the others; null only where
// there is nothing to read or write.
bool bad(const void* p, size_t a, bool needed) { return (needed && !p) || !aligned(p, a); }

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

size_t moe_cross_entropy_workspace_size(int64_t T, int D, int V, moe_dtype dtype, int backward) {
    const Call a = call_of(nullptr, nullptr, nullptr, nullptr, nullptr, T, D, V, 0, 1.f, dtype);
    return check(a) != MOE_OK || T == 0 ? 0 : plan_of(T, D, V, 0, dtype, backward != 0).total;
}

moe_status moe_cross_entropy_forward(const void* h, const void* W, const int32_t* targets, float* loss, float* lse,
                                     int64_t T, int D, int V, moe_dtype dtype, void* workspace, size_t ws_bytes,
                                     hipStream_t stream) {
    const Call a = call_of(h, W, targets, nullptr, nullptr, T, D, V, 0, 1.f, dtype);
    if (const moe_status st = check(a)) return st;
    const bool any = T > 0;
    if (bad(h, 16, any) || bad(W, 16, any) || bad(targets, 4, any) || bad(loss, 4, any) || bad(lse, 4, any))
        return MOE_ERR_INVALID_ARG;
    return forward(a, loss, lse, nullptr, workspace, ws_bytes, stream);
}

moe_status moe_cross_entropy_backward(const void* h, const void* W, const int32_t* targets, const float* lse,
                                      const float* dloss, void* dh, void* dW, int64_t T, int D, int V, moe_dtype dtype,
                                      moe_dtype dW_dtype, void* workspace, size_t ws_bytes, hipStream_t stream) {
    const Call a = call_of(h, W, targets, nullptr, nullptr, T, D, V, 0, 1.f, dtype);
    if (const moe_status st = check(a)) return st;
    const bool any = T > 0;
    if (bad(h, 16, any) || bad(W, 16, any) || bad(targets, 4, any) || bad(lse, 4, any) || bad(dloss, 4, any) ||
        bad(dh, 16, any && !dW) || bad(dW, 16, false) || (dW_dtype != MOE_F32 && dW_dtype != dtype))
        return MOE_ERR_INVALID_ARG;
    return backward(a, nullptr, lse, dloss, dh, dW, dW_dtype, workspace, ws_bytes, stream);
}

size_t moe_distillation_workspace_size(int64_t T, int D, int V, int K, moe_dtype dtype, int backward) {
    const Call a = call_of(nullptr, nullptr, nullptr, nullptr, nullptr, T, D, V, K, 1.f, dtype);
    return K <= 0 || check(a) != MOE_OK || T == 0 ? 0 : plan_of(T, D, V, K, dtype, backward != 0).total;
}

moe_status moe_distillation_forward(const void* h, const void* W, const int32_t* ids, const float* logits, float* loss,
                                    float* lse, float* z, int64_t T, int D, int V, int K, float temperature, moe_dtype dtype,
                                    void* workspace, size_t ws_bytes, hipStream_t stream) {
    const Call a = call_of(h, W, nullptr, ids, logits, T, D, V, K, temperature, dtype);
    if (K <= 0) return MOE_ERR_INVALID_ARG;
    if (const moe_status st = check(a)) return st;
    const bool any = T > 0;
    if (bad(h, 16, any) || bad(W, 16, any) || bad(ids, 4, any) || bad(logits, 4, any) || bad(loss, 4, any) ||
        bad(lse, 4, any) || bad(z, 4, any))
        return MOE_ERR_INVALID_ARG;
    return forward(a, loss, lse, z, workspace, ws_bytes, stream);
}

moe_status moe_distillation_backward(const void* h, const void* W, const int32_t* ids, const float* logits, const float* z,
                                     const float* lse, const float* dloss, void* dh, void* dW, int64_t T, int D, int V, int K,
                                     float temperature, moe_dtype dtype, moe_dtype dW_dtype, void* workspace,
                                     size_t ws_bytes, hipStream_t stream) {
    const Call a = call_of(h, W, nullptr, ids, logits, T, D, V, K, temperature, dtype);
    if (K <= 0) return MOE_ERR_INVALID_ARG;
    if (const moe_status st = check(a)) return st;
    const bool any = T > 0;
    if (bad(h, 16, any) || bad(W, 16, any) || bad(ids, 4, any) || bad(logits, 4, any) || bad(z, 4, any) || bad(lse, 4, any) ||
        bad(dloss, 4, any) || bad(dh, 16, any && !dW) || bad(dW, 16, false) || (dW_dtype != MOE_F32 && dW_dtype != dtype))
        return MOE_ERR_INVALID_ARG;
    return backward(a, z, lse, dloss, dh, dW, dW_dtype, workspace, ws_bytes, stream);
}

}  // extern "C"
