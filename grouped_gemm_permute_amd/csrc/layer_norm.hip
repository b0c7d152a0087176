// layer_norm.hip -- layer norm in front of the layer: forward, backward, and
// the C entry points moe_layer_norm_forward / moe_layer_norm_backward.
//
//   forward   h = x (+ residual, rounded once to the storage type)
//             mean = sum(h) / D (0 with rms),  var = sum((h - mean)^2) / D
//             rstd = 1 / sqrt(var + eps),  y = (h - mean) rstd w + b
//   backward  z = (h - mean) rstd,  g = dy w
//             dx = rstd (g - sum(g) / D - z sum(g z) / D) (+ dh)
//             dweight = sum over rows of dy z,  dbias = sum over rows of dy
//             (rms: the sum(g) / D term is absent)
//
// Both are bound by memory: a row is read once, held in registers as fp32
// while its sums are formed (so the variance is the sum of squared
// deviations, not a difference of large sums), and written once.  A row
// belongs to LANES lanes, each holding up to NV vectors of 16 bytes, 3 of bf16 or 4 of
// fp32: 8, 32 or 64 lanes of a wavefront with shuffle sums for rows of up to 24, 96
// and 192 vectors of bf16 (32, 128 and 256 of fp32), a whole workgroup of 256 or 1024
// threads with sums through LDS for longer ones.  16-byte accesses are taken at any element alignment (the
// global memory path splits those that straddle a line), so an odd D costs
// only the element-wise tail of each row.
//
// The weight's gradient is a sum down the rows: every lane keeps the sums of
// its own columns in registers over the rows its workgroup walks, the
// workgroup adds its wavefronts' sums through LDS and writes one partial
// row, and a second kernel adds the partial rows in a fixed order (no
// atomics, so repeated calls give equal bits).  With few rows further
// workgroups of the same launch take it, each some columns of all rows.
#include "moe_ffn.h"

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

namespace {

typedef __attribute__((ext_vector_type(2))) float f32x2_t;
typedef __attribute__((ext_vector_type(2))) __bf16 bf16x2_t;
typedef __attribute__((ext_vector_type(4))) float f32x4_t;

struct bf16_t {
    uint16_t bits;
};

// 16 bytes at the alignment of one element.
template <typename T>
struct __attribute__((packed, aligned(sizeof(T)))) Raw {
    uint32_t w[4];
};

template <typename T>
constexpr int vec_of() {
    return 16 / (int)sizeof(T);
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2_t{lo, hi}, bf16x2_t));
}
__device__ __forceinline__ float to_float(float v) { return v; }
__device__ __forceinline__ float to_float(bf16_t v) { return __uint_as_float((uint32_t)v.bits << 16); }

__device__ __forceinline__ void unpack(const Raw<float>& r, float* v) {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = __uint_as_float(r.w[i]);
}
__device__ __forceinline__ void unpack(const Raw<bf16_t>& r, float* v) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(r.w[i] << 16);
        v[2 * i + 1] = __uint_as_float(r.w[i] & 0xffff0000u);
    }
}
__device__ __forceinline__ void pack(const float* v, Raw<float>& r) {
#pragma unroll
    for (int i = 0; i < 4; ++i) r.w[i] = __float_as_uint(v[i]);
}
__device__ __forceinline__ void pack(const float* v, Raw<bf16_t>& r) {
#pragma unroll
    for (int i = 0; i < 4; ++i) r.w[i] = pack_bf16(v[2 * i], v[2 * i + 1]);
}

template <typename T>
struct __attribute__((packed, aligned(sizeof(T)))) Raw2 {
    uint32_t w[2];
};
template <typename T>
struct __attribute__((packed, aligned(sizeof(T)))) Raw1 {
    uint32_t w;
};

// `left` elements of the row remain from p: a whole vector, its tail (TAIL:
// rows that have one), or nothing (left <= 0); what is not there reads as zero.
// A tail is taken from the row's last 16 bytes and shifted down, one load like
// any other; only a row shorter than a vector (SHORT: rows that may be) has no
// such 16 bytes and reads its elements, each at a place that exists.
template <bool TAIL, bool SHORT, typename T>
__device__ __forceinline__ Raw<T> load_raw(const T* p, int left, int D) {
    constexpr int VEC = vec_of<T>();
    Raw<T> r = {{0, 0, 0, 0}};
    if constexpr (!TAIL) {
        if (left > 0) r = *(const Raw<T>*)p;
        return r;
    }
    if (left <= 0) return r;
    if constexpr (SHORT) {
        if (D < VEC) {
            float v[VEC];
#pragma unroll
            for (int i = 0; i < VEC; ++i) v[i] = to_float(p[i < left ? i : 0]);
#pragma unroll
            for (int i = 0; i < VEC; ++i) v[i] = i < left ? v[i] : 0.f;
            pack(v, r);
            return r;
        }
    }
    const int over = left < VEC ? VEC - left : 0, bits = over * (int)sizeof(T) * 8;
    r = *(const Raw<T>*)(p - over);
    uint64_t lo = r.w[0] | (uint64_t)r.w[1] << 32, hi = r.w[2] | (uint64_t)r.w[3] << 32;
    if (bits >= 64) {
        lo = hi;
        hi = 0;
    }
    const int b = bits & 63;
    lo = lo >> b | (hi << 1) << (63 - b);
    hi >>= b;
    r.w[0] = (uint32_t)lo;
    r.w[1] = (uint32_t)(lo >> 32);
    r.w[2] = (uint32_t)hi;
    r.w[3] = (uint32_t)(hi >> 32);
    return r;
}
// Four elements, two and one for the tail.
template <bool TAIL, typename T>
__device__ __forceinline__ void store_vec(T* p, int left, const float* v) {
    constexpr int VEC = vec_of<T>();
    Raw<T> r;
    pack(v, r);
    if (TAIL ? left >= VEC : left > 0) {
        *(Raw<T>*)p = r;
        return;
    }
    if (!TAIL || left <= 0) return;
    if constexpr (sizeof(T) == 4) {
        if (left & 2) *(Raw2<T>*)p = {{r.w[0], r.w[1]}};
        if (left & 1) *(uint32_t*)(p + (left & 2)) = left & 2 ? r.w[2] : r.w[0];
    } else {
        if (left & 4) *(Raw2<T>*)p = {{r.w[0], r.w[1]}};
        const uint32_t w0 = left & 4 ? r.w[2] : r.w[0], w1 = left & 4 ? r.w[3] : r.w[1];
        if (left & 2) *(Raw1<T>*)(p + (left & 4)) = {w0};
        if (left & 1) p[left & 6].bits = (uint16_t)(left & 2 ? w1 : w0);
    }
}

// Sum over the LANES lanes of a row, the same bits in each.  Rows wider than
// a wavefront go through LDS: `red` holds one float per wavefront, and a row's
// successive sums alternate between two such buffers, so that the barrier of
// one separates the reads of the other from its next writes.
template <int LANES>
__device__ __forceinline__ float row_sum(float v, float* red) {
    constexpr int W = LANES < 64 ? LANES : 64;
#pragma unroll
    for (int o = W / 2; o > 0; o >>= 1) v += __shfl_xor(v, o, 64);
    if constexpr (LANES > 64) {
        if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
        __syncthreads();
        v = 0.f;
#pragma unroll
        for (int i = 0; i < LANES / 64; ++i) v += red[i];
    }
    return v;
}

template <int LANES>
constexpr int threads_of() {
    return LANES > 256 ? LANES : 256;
}

struct FwdArgs {
    const void *x, *r, *w, *b;
    void *y, *h;
    float *mean, *rstd;
    int64_t T;
    int D, rms;
    float eps;
};

template <typename T, int LANES, int NV, bool TAIL>
__global__ __launch_bounds__(threads_of<LANES>()) void norm_forward_kernel(const FwdArgs a) {
    constexpr int VEC = vec_of<T>(), NT = threads_of<LANES>(), ROWS = NT / LANES;
    __shared__ float red[2][LANES > 64 ? LANES / 64 : 1];
    const int lane = threadIdx.x % LANES;
    const float inv_d = 1.f / (float)a.D;
    int col[NV];
    // vectors before a lane's last are whole: the last, partial or absent
    // vector of a row falls to the last one of some lanes
    auto left = [&](int i) { return i < NV - 1 ? VEC : a.D - col[i]; };
    auto load = [&](const void* base, int64_t at, int i) {
        const T* p = (const T*)base + at + col[i];
        if (i < NV - 1) return *(const Raw<T>*)p;
        return load_raw<TAIL, LANES == 8 && NV == 1>(p, left(i), a.D);
    };
    Raw<T> w[NV], b[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        col[i] = (lane + i * LANES) * VEC;
        if (a.w) w[i] = load(a.w, 0, i);
        if (a.b) b[i] = load(a.b, 0, i);
    }
    // rows of a workgroup-wide LANES advance together (one row per workgroup),
    // so every thread reaches the barriers of row_sum
    for (int64_t t = (int64_t)blockIdx.x * ROWS + threadIdx.x / LANES; t < a.T;
         t += (int64_t)gridDim.x * ROWS) {
        const int64_t at = t * a.D;
        float v[NV][VEC];
        Raw<T> rx[NV], rr[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i) rx[i] = load(a.x, at, i);
        if (a.r) {
#pragma unroll
            for (int i = 0; i < NV; ++i) rr[i] = load(a.r, at, i);
        }
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            unpack(rx[i], v[i]);
            if (a.r) {
                float u[VEC];
                unpack(rr[i], u);
#pragma unroll
                for (int e = 0; e < VEC; ++e) v[i][e] += u[e];
                // the norm is that of the stored sum
                Raw<T> s;
                pack(v[i], s);
                unpack(s, v[i]);
                store_vec<TAIL>((T*)a.h + at + col[i], left(i), v[i]);
            }
        }
        float mean = 0.f;
        if (!a.rms) {
            float s = 0.f;
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
                for (int e = 0; e < VEC; ++e) s += v[i][e];
            mean = row_sum<LANES>(s, red[0]) * inv_d;
        } else if constexpr (LANES > 64) {
            __syncthreads();   // stands for the first sum's barrier
        }
        float q = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                v[i][e] = e < left(i) ? v[i][e] - mean : 0.f;
                q = fmaf(v[i][e], v[i][e], q);
            }
        const float rstd = 1.f / sqrtf(row_sum<LANES>(q, red[1]) * inv_d + a.eps);
        if (lane == 0) {
            if (a.mean) a.mean[t] = mean;
            if (a.rstd) a.rstd[t] = rstd;
        }
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            float u[VEC];
#pragma unroll
            for (int e = 0; e < VEC; ++e) v[i][e] *= rstd;
            if (a.w) {
                unpack(w[i], u);
#pragma unroll
                for (int e = 0; e < VEC; ++e) v[i][e] *= u[e];
            }
            if (a.b) {
                unpack(b[i], u);
#pragma unroll
                for (int e = 0; e < VEC; ++e) v[i][e] += u[e];
            }
            store_vec<TAIL>((T*)a.y + at + col[i], left(i), v[i]);
        }
    }
}

struct BwdArgs {
    const void *h, *dy, *w, *dh;
    const float *mean, *rstd;
    void* dx;
    float* part;      // [2][row_blocks][D] partial dweight, dbias; null: none
    float *dw, *db;   // the workgroups past row_blocks: the sums themselves
    int64_t T;
    int D, row_blocks;
};

// The weight's gradients of CV vectors of columns over all rows, for few rows: a
// thread takes one vector and a slice of the rows, and the slices are added by
// shuffles and through LDS.
constexpr int CV = 4;
template <typename T, int NT, bool TAIL>
__device__ __forceinline__ void column_sums(const BwdArgs& a) {
    constexpr int VEC = vec_of<T>(), SLICES = NT / CV, WAVES = NT / 64;
    __shared__ float sums[WAVES][2][CV * VEC];
    const int first = ((int)blockIdx.x - a.row_blocks) * CV * VEC;
    const int vec = threadIdx.x % CV, col = first + vec * VEC, left = a.D - col;
    auto load = [&](const void* base, int64_t at) {
        const T* p = (const T*)base + at;
        if (!TAIL || left >= VEC) return load_raw<false, false>(p, left, a.D);
        return load_raw<TAIL, TAIL>(p, left, a.D);
    };
    float dw[VEC], db[VEC];
#pragma unroll
    for (int e = 0; e < VEC; ++e) dw[e] = db[e] = 0.f;
#pragma unroll 4
    for (int t = threadIdx.x / CV; t < (int)a.T; t += SLICES) {
        const Raw<T> rh = load(a.h, (int64_t)t * a.D + col), ry = load(a.dy, (int64_t)t * a.D + col);
        const float mean = a.mean ? a.mean[t] : 0.f, rstd = a.rstd[t];
        float z[VEC], dy[VEC];
        unpack(rh, z);
        unpack(ry, dy);
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            dw[e] = fmaf(dy[e], (z[e] - mean) * rstd, dw[e]);
            db[e] += dy[e];
        }
    }
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
#pragma unroll
        for (int o = CV; o < 64; o <<= 1) {
            dw[e] += __shfl_xor(dw[e], o, 64);
            db[e] += __shfl_xor(db[e], o, 64);
        }
        if ((threadIdx.x & 63) < CV) {
            sums[threadIdx.x >> 6][0][vec * VEC + e] = dw[e];
            sums[threadIdx.x >> 6][1][vec * VEC + e] = db[e];
        }
    }
    __syncthreads();
    const int which = threadIdx.x / (CV * VEC), c = threadIdx.x % (CV * VEC);
    float* out = which ? a.db : a.dw;
    if (which > 1 || !out || first + c >= a.D) return;
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < WAVES; ++w) v += sums[w][which][c];
    out[first + c] = v;
}

template <typename T, int LANES, int NV, bool TAIL>
__global__ __launch_bounds__(threads_of<LANES>()) void norm_backward_kernel(const BwdArgs a) {
    constexpr int VEC = vec_of<T>(), NT = threads_of<LANES>(), ROWS = NT / LANES;
    constexpr int WAVES = NT / 64, COLS = LANES * NV * VEC;
    __shared__ float red[2][LANES > 64 ? LANES / 64 : 1];
    __shared__ __attribute__((aligned(16))) float wsum[LANES > 64 ? 1 : WAVES * COLS];
    if ((int)blockIdx.x >= a.row_blocks) return column_sums<T, NT, TAIL>(a);
    const int lane = threadIdx.x % LANES;
    const float inv_d = 1.f / (float)a.D;
    int col[NV];
    // vectors before a lane's last are whole: the last, partial or absent
    // vector of a row falls to the last one of some lanes
    auto left = [&](int i) { return i < NV - 1 ? VEC : a.D - col[i]; };
    auto load = [&](const void* base, int64_t at, int i) {
        const T* p = (const T*)base + at + col[i];
        if (i < NV - 1) return *(const Raw<T>*)p;
        return load_raw<TAIL, LANES == 8 && NV == 1>(p, left(i), a.D);
    };
    Raw<T> w[NV];
    float dw[NV][VEC], db[NV][VEC];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        col[i] = (lane + i * LANES) * VEC;
        w[i] = a.w ? load(a.w, 0, i) : Raw<T>{};
#pragma unroll
        for (int e = 0; e < VEC; ++e) dw[i][e] = db[i][e] = 0.f;
    }
    // z and g stay in fp32 between the sums and their use; rows wider than 256
    // lanes hold form them twice from the packed row, in half the registers
    constexpr bool KEEP = LANES <= 256;
    for (int64_t t = (int64_t)blockIdx.x * ROWS + threadIdx.x / LANES; t < a.T;
         t += (int64_t)a.row_blocks * ROWS) {
        const int64_t at = t * a.D;
        Raw<T> rh[NV], ry[NV], rd[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            rh[i] = load(a.h, at, i);
            ry[i] = load(a.dy, at, i);
        }
        if (a.dh) {
#pragma unroll
            for (int i = 0; i < NV; ++i) rd[i] = load(a.dh, at, i);
        }
        const float mean = a.mean ? a.mean[t] : 0.f, rstd = a.rstd[t];
        auto values = [&](int i, float* dy, float* z, float* g) {
            unpack(rh[i], z);
            unpack(ry[i], dy);
            unpack(w[i], g);
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                z[e] = (z[e] - mean) * rstd;
                if (TAIL) z[e] = e < left(i) ? z[e] : 0.f;
                g[e] = a.w ? g[e] * dy[e] : dy[e];
            }
        };
        float z[KEEP ? NV : 1][VEC], g[KEEP ? NV : 1][VEC];
        float sg = 0.f, sgz = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            constexpr int one = KEEP ? 1 : 0;
            float dy[VEC], *zi = z[i * one], *gi = g[i * one];
            values(i, dy, zi, gi);
            // past the row's end nothing is added: dy is 0 there, but z, -mean rstd, may be
            // infinite where no (h - mean) rstd is
            if (left(i) <= 0) continue;
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                dw[i][e] = fmaf(dy[e], zi[e], dw[i][e]);
                db[i][e] += dy[e];
                sg += gi[e];
                sgz = fmaf(gi[e], zi[e], sgz);
            }
        }
        sg = row_sum<LANES>(sg, red[0]);
        sgz = row_sum<LANES>(sgz, red[1]);
        if constexpr (!KEEP) {
            // the packed values stand for new ones: nothing unpacked is carried over
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
                for (int k = 0; k < 4; ++k) asm volatile("" : "+v"(rh[i].w[k]), "+v"(ry[i].w[k]), "+v"(w[i].w[k]));
        }
        const float mg = a.mean ? sg * inv_d : 0.f, mgz = sgz * inv_d;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            constexpr int one = KEEP ? 1 : 0;
            float dy[VEC], u[VEC], *zi = z[i * one], *gi = g[i * one];
            if constexpr (!KEEP) values(i, dy, zi, gi);
            if (a.dh) unpack(rd[i], u);
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                const float t0 = fmaf(-zi[e], mgz, gi[e] - mg);
                gi[e] = a.dh ? fmaf(rstd, t0, u[e]) : rstd * t0;
            }
            store_vec<TAIL>((T*)a.dx + at + col[i], left(i), gi);
        }
    }
    if (!a.part) return;
    float* out[2] = {a.part + (int64_t)blockIdx.x * a.D,
                     a.part + ((int64_t)a.row_blocks + blockIdx.x) * a.D};
    if constexpr (LANES > 64) {
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int e = 0; e < VEC; ++e)
                if (e < left(i)) {
                    out[0][col[i] + e] = dw[i][e];
                    out[1][col[i] + e] = db[i][e];
                }
    } else {
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            if (s) __syncthreads();
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                float v[VEC];
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    v[e] = s ? db[i][e] : dw[i][e];
#pragma unroll
                    for (int o = LANES; o < 64; o <<= 1) v[e] += __shfl_xor(v[e], o, 64);
                }
                // 16 bytes a store: element by element a lane's stride of VEC is
                // as many bank conflicts
                if ((threadIdx.x & 63) < LANES)
#pragma unroll
                    for (int e = 0; e < VEC; e += 4)
                        *(f32x4_t*)&wsum[(threadIdx.x >> 6) * COLS + col[i] + e] = f32x4_t{v[e], v[e + 1], v[e + 2], v[e + 3]};
            }
            __syncthreads();
            for (int c = threadIdx.x; c < a.D; c += NT) {
                float v = 0.f;
#pragma unroll
                for (int k = 0; k < WAVES; ++k) v += wsum[k * COLS + c];
                out[s][c] = v;
            }
        }
    }
}

// dweight / dbias: column sums of the [rows, D] partials, one workgroup per
// SUM_COLS columns of one of the two, SUM_SLICES threads per column.
constexpr int SUM_COLS = 32, SUM_SLICES = 32;
__global__ __launch_bounds__(SUM_COLS * SUM_SLICES) void norm_partial_sum_kernel(
    const float* __restrict__ part, int rows, int D, float* __restrict__ dw, float* __restrict__ db) {
    __shared__ float s[SUM_SLICES][SUM_COLS];
    float* out = blockIdx.y ? db : dw;
    if (!out) return;
    const float* p = part + (int64_t)blockIdx.y * rows * D;
    const int cl = threadIdx.x % SUM_COLS, sl = threadIdx.x / SUM_COLS;
    const int c = blockIdx.x * SUM_COLS + cl;
    float v = 0.f;
    if (c < D) {
#pragma unroll 16
        for (int r = sl; r < rows; r += SUM_SLICES) v += p[(int64_t)r * D + c];
    }
    s[sl][cl] = v;
    __syncthreads();
    if (sl == 0 && c < D) {
        float t = 0.f;
#pragma unroll
        for (int k = 0; k < SUM_SLICES; ++k) t += s[k][cl];
        out[c] = t;
    }
}

// ---- host side

constexpr int kMaxD = 16384;
constexpr size_t kAlign = 256;

struct Shape {
    int lanes, nv;
};
// Lanes per row and 16-byte vectors per lane: the fewest lanes that hold the
// row in 24 bf16 or 16 fp32 elements each.  Their fp32 copies and, in the
// backward, their gradient sums stay in registers, but for the backward of more than
// 8192 elements, whose 1024 threads have 128 registers each: it keeps the packed row and still
// spills (10 registers a lane in bf16, 28 with tails; 20 to 109 in fp32), which with one workgroup
// a unit leaves 2.8 TB/s (2048 x 16384 bf16 73 us without dh) where narrower rows have
// 4.2 to 5.7.  With a fourth bf16 vector
// the backward has one wavefront a SIMD (4096 x 777: 24 us instead of 16).
Shape shape_of(int D, moe_dtype dt) {
    const int vec = dt == MOE_BF16 ? 8 : 4, most = dt == MOE_BF16 ? 3 : 4, nvec = (D + vec - 1) / vec;
    int lanes = 1024;
    for (int l : {256, 64, 32, 8})
        if (nvec <= l * most) lanes = l;
    return {lanes, (nvec + lanes - 1) / lanes};
}
int threads_for(int lanes) { return lanes > 256 ? lanes : 256; }

constexpr int64_t kFwdMaxBlocks = 2048;
// Partial rows of the backward: two workgroups a unit, one where it is 1024 threads
// wide (with dh: 8192 x 8191 fp32 216 -> 207 us, 2048 x 16384 bf16 113 -> 92; with 256 of the narrower
// 8192 x 4096 bf16 would be 56 -> 70, 32768 x 768 36 -> 42).
int64_t bwd_blocks(int lanes) { return lanes == 1024 ? 256 : 512; }
unsigned grid_of(int64_t T, int lanes, int64_t most) {
    const int64_t rows = threads_for(lanes) / lanes, need = (T + rows - 1) / rows;
    return (unsigned)(need < most ? need : most);
}

bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }

// Few rows: the weight's gradients come from workgroups of their own beside the rows'
// (one launch, h and dy read twice) instead of partial rows and a second launch.
// (512 x 768 bf16 9.6 -> 5.2 us, 1024 x 768 10.4 -> 8.0, 2048 x 768 would be 12.3 ->
// 14.5; 512 x 4096 25 -> 8.6, 1024 x 4096 fp32 20.5 -> 18.9; with tails 512 x 1001 8.6 ->
// 8.1, 1024 x 1001 would be 10.7 -> 18.3.)
bool few_rows(int64_t T, int D, moe_dtype dt) {
    return T > 0 && T <= (D % (dt == MOE_BF16 ? 8 : 4) ? 512 : 1024);
}

moe_status check_sizes(int64_t T, int D, moe_dtype dt) {
    if (T < 0 || T >= ((int64_t)1 << 31) || D <= 0) return MOE_ERR_INVALID_ARG;
    if (dt != MOE_F32 && dt != MOE_BF16) return MOE_ERR_INVALID_ARG;
    if (D > kMaxD) return MOE_ERR_UNSUPPORTED;
    return MOE_OK;
}

// Calls f(LANES, NV, TAIL) for the shape, of the values that shape_of gives.
template <typename T, typename F>
void dispatch(Shape p, int D, F&& f) {
    using std::integral_constant;
    constexpr int most = sizeof(T) == 2 ? 3 : 4;
    // NV from the least that the next fewer lanes leave to `most` (of kMaxD
    // elements, where that is less)
    auto nv = [&](auto lanes, auto low) {
        constexpr int longest = kMaxD / vec_of<T>() / decltype(lanes)::value;
        constexpr int top = longest < most ? longest : most;
        auto at = [&](auto self, auto n) -> void {
            if (p.nv == n.value) {
                if (D % vec_of<T>()) return f(lanes, n, std::true_type{});
                return f(lanes, n, std::false_type{});
            }
            if constexpr (n.value < top) self(self, integral_constant<int, n.value + 1>{});
        };
        at(at, low);
    };
    switch (p.lanes) {
        case 8: return nv(integral_constant<int, 8>{}, integral_constant<int, 1>{});
        case 32: return nv(integral_constant<int, 32>{}, integral_constant<int, most * 8 / 32 + 1>{});
        case 64: return nv(integral_constant<int, 64>{}, integral_constant<int, most * 32 / 64 + 1>{});
        case 256: return nv(integral_constant<int, 256>{}, integral_constant<int, most * 64 / 256 + 1>{});
        default: return nv(integral_constant<int, 1024>{}, integral_constant<int, most * 256 / 1024 + 1>{});
    }
}

template <typename T>
hipError_t launch_forward(const FwdArgs& a, Shape p, unsigned grid, hipStream_t s) {
    dispatch<T>(p, a.D, [&](auto lanes, auto nv, auto tail) {
        constexpr int L = decltype(lanes)::value;
        norm_forward_kernel<T, L, decltype(nv)::value, decltype(tail)::value><<<grid, threads_of<L>(), 0, s>>>(a);
    });
    return hipGetLastError();
}
template <typename T>
hipError_t launch_backward(const BwdArgs& a, Shape p, unsigned grid, hipStream_t s) {
    dispatch<T>(p, a.D, [&](auto lanes, auto nv, auto tail) {
        constexpr int L = decltype(lanes)::value;
        norm_backward_kernel<T, L, decltype(nv)::value, decltype(tail)::value><<<grid, threads_of<L>(), 0, s>>>(a);
    });
    return hipGetLastError();
}

}  // namespace

extern "C" {

moe_status moe_layer_norm_forward(const void* x, const void* residual, const void* weight,
                                  const void* bias, void* y, void* h, float* mean, float* rstd,
                                  int64_t T, int D, int rms, float eps, moe_dtype dtype,
                                  hipStream_t stream) {
    const moe_status st = check_sizes(T, D, dtype);
    if (st != MOE_OK) return st;
    if (!(eps >= 0.f) || eps > 3.4e38f) return MOE_ERR_INVALID_ARG;
    if ((residual != nullptr) != (h != nullptr)) return MOE_ERR_INVALID_ARG;
    if (rms && mean) return MOE_ERR_INVALID_ARG;
    if (T > 0 && (!x || !y)) return MOE_ERR_INVALID_ARG;
    const void* ptrs[] = {x, residual, weight, bias, y, h};
    for (const void* p : ptrs)
        if (p && !aligned(p, 16)) return MOE_ERR_INVALID_ARG;
    if (!aligned(mean, 4) || !aligned(rstd, 4)) return MOE_ERR_INVALID_ARG;
    if (T == 0) return MOE_OK;
    const Shape p = shape_of(D, dtype);
    const FwdArgs a = {x, residual, weight, bias, y, h, mean, rstd, T, D, rms ? 1 : 0, eps};
    const unsigned grid = grid_of(T, p.lanes, kFwdMaxBlocks);
    (void)hipGetLastError();
    const hipError_t e = dtype == MOE_BF16 ? launch_forward<bf16_t>(a, p, grid, stream)
                                           : launch_forward<float>(a, p, grid, stream);
    return e == hipSuccess ? MOE_OK : MOE_ERR_HIP;
}

size_t moe_layer_norm_backward_workspace_size(int64_t T, int D, moe_dtype dtype) {
    if (check_sizes(T, D, dtype) != MOE_OK || few_rows(T, D, dtype)) return 0;
    const size_t rows = grid_of(T, shape_of(D, dtype).lanes, bwd_blocks(shape_of(D, dtype).lanes));
    const size_t bytes = 2 * rows * (size_t)D * sizeof(float);
    return (bytes + kAlign - 1) / kAlign * kAlign;
}

moe_status moe_layer_norm_backward(const void* h, const float* mean, const float* rstd,
                                   const void* weight, const void* dy, const void* dh, void* dx,
                                   float* dweight, float* dbias, int64_t T, int D, moe_dtype dtype,
                                   void* workspace, size_t ws_bytes, hipStream_t stream) {
    const moe_status st = check_sizes(T, D, dtype);
    if (st != MOE_OK) return st;
    if (T > 0 && (!h || !rstd || !dy || !dx)) return MOE_ERR_INVALID_ARG;
    const void* ptrs[] = {h, weight, dy, dh, dx};
    for (const void* p : ptrs)
        if (p && !aligned(p, 16)) return MOE_ERR_INVALID_ARG;
    const void* floats[] = {mean, rstd, dweight, dbias};
    for (const void* p : floats)
        if (!aligned(p, 4)) return MOE_ERR_INVALID_ARG;
    const bool sums = dweight || dbias, apart = sums && !few_rows(T, D, dtype);
    if (apart && T > 0) {
        if (!workspace || !aligned(workspace, kAlign)) return MOE_ERR_INVALID_ARG;
        if (ws_bytes < moe_layer_norm_backward_workspace_size(T, D, dtype)) return MOE_ERR_WORKSPACE;
    }
    const Shape p = shape_of(D, dtype);
    const unsigned grid = grid_of(T, p.lanes, bwd_blocks(p.lanes));
    (void)hipGetLastError();
    BwdArgs a = {h, dy, weight, dh, mean, rstd, dx, apart ? (float*)workspace : nullptr, dweight, dbias, T, D, (int)grid};
    auto launch = [&](unsigned blocks) {
        return dtype == MOE_BF16 ? launch_backward<bf16_t>(a, p, blocks, stream) : launch_backward<float>(a, p, blocks, stream);
    };
    if (T > 0) {
        const unsigned cols = sums && !apart ? (unsigned)((D * (dtype == MOE_BF16 ? 2 : 4) + 16 * CV - 1) / (16 * CV)) : 0;
        if (cols && (dx == h || dx == dy)) {
            // dx would be written over what the columns' workgroups read
            a.row_blocks = 0;
            if (launch(cols) != hipSuccess) return MOE_ERR_HIP;
            a.row_blocks = (int)grid;
            if (launch(grid) != hipSuccess) return MOE_ERR_HIP;
        } else if (launch(grid + cols) != hipSuccess) {
            return MOE_ERR_HIP;
        }
    }
    if (apart) {
        // with T == 0 there are no partial rows, and the sums are written as zeros
        norm_partial_sum_kernel<<<dim3((D + SUM_COLS - 1) / SUM_COLS, 2), SUM_COLS * SUM_SLICES, 0,
                                  stream>>>((const float*)workspace, (int)grid, D, dweight, dbias);
        if (hipGetLastError() != hipSuccess) return MOE_ERR_HIP;
    }
    return MOE_OK;
}

}  // extern "C"
