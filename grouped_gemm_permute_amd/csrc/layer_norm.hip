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
// belongs to LANES lanes, each holding NV vectors of 16 bytes: 8, 32 or 64
// lanes of a wavefront with shuffle sums for rows of up to 32, 128 and 256
// vectors, a whole workgroup of 256 or 1024 threads with sums through LDS for
// longer ones.  16-byte accesses are taken at any element alignment (the
// global memory path splits those that straddle a line), so an odd D costs
// only the element-wise tail of each row.
//
// The weight's gradient is a sum down the rows: every lane keeps the sums of
// its own columns in registers over the rows its workgroup walks, the
// workgroup adds its wavefronts' sums through LDS and writes one partial
// row, and a second kernel adds the partial rows in a fixed order (no
// atomics, so repeated calls give equal bits).
#include "moe_ffn.h"

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

namespace {

typedef __attribute__((ext_vector_type(2))) float f32x2_t;
typedef __attribute__((ext_vector_type(2))) __bf16 bf16x2_t;

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
__device__ __forceinline__ void store_one(float* p, float v) { *p = v; }
__device__ __forceinline__ void store_one(bf16_t* p, float v) { p->bits = (uint16_t)pack_bf16(v, 0.f); }

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

// `left` elements remain from p: a whole vector, the tail's elements, or
// nothing (left <= 0); what is not there reads as zero.
template <typename T>
__device__ __forceinline__ Raw<T> load_raw(const T* p, int left) {
    constexpr int VEC = vec_of<T>();
    Raw<T> r = {{0, 0, 0, 0}};
    if (left >= VEC) {
        r = *(const Raw<T>*)p;
    } else if (left > 0) {
        float v[VEC];
#pragma unroll
        for (int i = 0; i < VEC; ++i) v[i] = i < left ? to_float(p[i]) : 0.f;
        pack(v, r);
    }
    return r;
}
template <typename T>
__device__ __forceinline__ void store_vec(T* p, int left, const float* v) {
    constexpr int VEC = vec_of<T>();
    if (left >= VEC) {
        Raw<T> r;
        pack(v, r);
        *(Raw<T>*)p = r;
    } else {
#pragma unroll
        for (int i = 0; i < VEC; ++i)
            if (i < left) store_one(p + i, v[i]);
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

template <typename T, int LANES, int NV>
__global__ __launch_bounds__(threads_of<LANES>()) void norm_forward_kernel(const FwdArgs a) {
    constexpr int VEC = vec_of<T>(), NT = threads_of<LANES>(), ROWS = NT / LANES;
    __shared__ float red[2][LANES > 64 ? LANES / 64 : 1];
    const int lane = threadIdx.x % LANES;
    const float inv_d = 1.f / (float)a.D;
    int col[NV];
    // vectors before a lane's last are whole: the last, partial or absent
    // vector of a row falls to the last one of some lanes
    auto left = [&](int i) { return i < NV - 1 ? VEC : a.D - col[i]; };
    Raw<T> w[NV], b[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        col[i] = (lane + i * LANES) * VEC;
        if (a.w) w[i] = load_raw((const T*)a.w + col[i], left(i));
        if (a.b) b[i] = load_raw((const T*)a.b + col[i], left(i));
    }
    // rows of a workgroup-wide LANES advance together (one row per workgroup),
    // so every thread reaches the barriers of row_sum
    for (int64_t t = (int64_t)blockIdx.x * ROWS + threadIdx.x / LANES; t < a.T;
         t += (int64_t)gridDim.x * ROWS) {
        const int64_t at = t * a.D;
        float v[NV][VEC];
        Raw<T> rx[NV], rr[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i) rx[i] = load_raw((const T*)a.x + at + col[i], left(i));
        if (a.r) {
#pragma unroll
            for (int i = 0; i < NV; ++i) rr[i] = load_raw((const T*)a.r + at + col[i], left(i));
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
                store_vec((T*)a.h + at + col[i], left(i), v[i]);
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
            store_vec((T*)a.y + at + col[i], left(i), v[i]);
        }
    }
}

struct BwdArgs {
    const void *h, *dy, *w, *dh;
    const float *mean, *rstd;
    void* dx;
    float* part;      // [2][gridDim.x][D] partial dweight, dbias; null: neither is wanted
    int64_t T;
    int D;
};

template <typename T, int LANES, int NV>
__global__ __launch_bounds__(threads_of<LANES>()) void norm_backward_kernel(const BwdArgs a) {
    constexpr int VEC = vec_of<T>(), NT = threads_of<LANES>(), ROWS = NT / LANES;
    constexpr int WAVES = NT / 64, COLS = LANES * NV * VEC;
    __shared__ float red[2][LANES > 64 ? LANES / 64 : 1];
    __shared__ float wsum[LANES > 64 ? 1 : WAVES * COLS];
    const int lane = threadIdx.x % LANES;
    const float inv_d = 1.f / (float)a.D;
    int col[NV];
    // vectors before a lane's last are whole: the last, partial or absent
    // vector of a row falls to the last one of some lanes
    auto left = [&](int i) { return i < NV - 1 ? VEC : a.D - col[i]; };
    Raw<T> w[NV];
    float dw[NV][VEC], db[NV][VEC];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        col[i] = (lane + i * LANES) * VEC;
        if (a.w) w[i] = load_raw((const T*)a.w + col[i], left(i));
#pragma unroll
        for (int e = 0; e < VEC; ++e) dw[i][e] = db[i][e] = 0.f;
    }
    for (int64_t t = (int64_t)blockIdx.x * ROWS + threadIdx.x / LANES; t < a.T;
         t += (int64_t)gridDim.x * ROWS) {
        const int64_t at = t * a.D;
        Raw<T> rh[NV], ry[NV], rd[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            rh[i] = load_raw((const T*)a.h + at + col[i], left(i));
            ry[i] = load_raw((const T*)a.dy + at + col[i], left(i));
        }
        if (a.dh) {
#pragma unroll
            for (int i = 0; i < NV; ++i) rd[i] = load_raw((const T*)a.dh + at + col[i], left(i));
        }
        const float mean = a.mean ? a.mean[t] : 0.f, rstd = a.rstd[t];
        float z[NV][VEC], g[NV][VEC];
        float sg = 0.f, sgz = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            unpack(rh[i], z[i]);
            unpack(ry[i], g[i]);
            float u[VEC];
            if (a.w) unpack(w[i], u);
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                // past the row's end dy is zero, and so is every sum's share
                z[i][e] = (z[i][e] - mean) * rstd;
                dw[i][e] = fmaf(g[i][e], z[i][e], dw[i][e]);
                db[i][e] += g[i][e];
                if (a.w) g[i][e] *= u[e];
                sg += g[i][e];
                sgz = fmaf(g[i][e], z[i][e], sgz);
            }
        }
        sg = row_sum<LANES>(sg, red[0]);
        sgz = row_sum<LANES>(sgz, red[1]);
        const float mg = a.mean ? sg * inv_d : 0.f, mgz = sgz * inv_d;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            float u[VEC];
            if (a.dh) unpack(rd[i], u);
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                const float t0 = fmaf(-z[i][e], mgz, g[i][e] - mg);
                g[i][e] = a.dh ? fmaf(rstd, t0, u[e]) : rstd * t0;
            }
            store_vec((T*)a.dx + at + col[i], left(i), g[i]);
        }
    }
    if (!a.part) return;
    float* out[2] = {a.part + (int64_t)blockIdx.x * a.D,
                     a.part + ((int64_t)gridDim.x + blockIdx.x) * a.D};
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
            for (int i = 0; i < NV; ++i)
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    float v = s ? db[i][e] : dw[i][e];
#pragma unroll
                    for (int o = LANES; o < 64; o <<= 1) v += __shfl_xor(v, o, 64);
                    if ((threadIdx.x & 63) < LANES)
                        wsum[(threadIdx.x >> 6) * COLS + col[i] + e] = v;
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
constexpr int SUM_COLS = 32, SUM_SLICES = 16;
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
#pragma unroll 8
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
// Lanes per row and 16-byte vectors per lane: at most four vectors a lane
// (their fp32 copies and, in the backward, their gradient sums stay in
// registers), the fewest lanes that hold the row.
Shape shape_of(int D, moe_dtype dt) {
    const int vec = dt == MOE_BF16 ? 8 : 4, nvec = (D + vec - 1) / vec;
    const int lanes = nvec <= 32 ? 8 : nvec <= 128 ? 32 : nvec <= 256 ? 64 : nvec <= 1024 ? 256 : 1024;
    return {lanes, (nvec + lanes - 1) / lanes};
}
int threads_for(int lanes) { return lanes > 256 ? lanes : 256; }

constexpr int64_t kFwdMaxBlocks = 2048;
constexpr int64_t kBwdMaxBlocks = 512;
unsigned grid_of(int64_t T, int lanes, int64_t most) {
    const int64_t rows = threads_for(lanes) / lanes, need = (T + rows - 1) / rows;
    return (unsigned)(need < most ? need : most);
}

bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }

moe_status check_sizes(int64_t T, int D, moe_dtype dt) {
    if (T < 0 || T >= ((int64_t)1 << 31) || D <= 0) return MOE_ERR_INVALID_ARG;
    if (dt != MOE_F32 && dt != MOE_BF16) return MOE_ERR_INVALID_ARG;
    if (D > kMaxD) return MOE_ERR_UNSUPPORTED;
    return MOE_OK;
}

// Calls f<LANES, NV>() for the shape; only the pairs that shape_of gives.
template <typename F>
void dispatch(Shape p, F&& f) {
    auto nv = [&](auto lanes, auto least) {
        constexpr int N = decltype(least)::value;
        if constexpr (N <= 1)
            if (p.nv == 1) return f(lanes, std::integral_constant<int, 1>{});
        if constexpr (N <= 2)
            if (p.nv == 2) return f(lanes, std::integral_constant<int, 2>{});
        if (p.nv == 3) return f(lanes, std::integral_constant<int, 3>{});
        f(lanes, std::integral_constant<int, 4>{});
    };
    switch (p.lanes) {
        case 8: return nv(std::integral_constant<int, 8>{}, std::integral_constant<int, 1>{});
        case 32: return nv(std::integral_constant<int, 32>{}, std::integral_constant<int, 2>{});
        case 64: return nv(std::integral_constant<int, 64>{}, std::integral_constant<int, 3>{});
        case 256: return nv(std::integral_constant<int, 256>{}, std::integral_constant<int, 2>{});
        default: return nv(std::integral_constant<int, 1024>{}, std::integral_constant<int, 2>{});
    }
}

template <typename T>
hipError_t launch_forward(const FwdArgs& a, Shape p, unsigned grid, hipStream_t s) {
    dispatch(p, [&](auto lanes, auto nv) {
        constexpr int L = decltype(lanes)::value, N = decltype(nv)::value;
        // a row of kMaxD elements of two bytes has two vectors a thread at most
        if constexpr (sizeof(T) == 4 || L < 1024 || N <= 2)
            norm_forward_kernel<T, L, N><<<grid, threads_of<L>(), 0, s>>>(a);
    });
    return hipGetLastError();
}
template <typename T>
hipError_t launch_backward(const BwdArgs& a, Shape p, unsigned grid, hipStream_t s) {
    dispatch(p, [&](auto lanes, auto nv) {
        constexpr int L = decltype(lanes)::value, N = decltype(nv)::value;
        if constexpr (sizeof(T) == 4 || L < 1024 || N <= 2)
            norm_backward_kernel<T, L, N><<<grid, threads_of<L>(), 0, s>>>(a);
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
    if (check_sizes(T, D, dtype) != MOE_OK) return 0;
    const size_t rows = grid_of(T, shape_of(D, dtype).lanes, kBwdMaxBlocks);
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
    const bool sums = dweight || dbias;
    if (sums && T > 0) {
        if (!workspace || !aligned(workspace, kAlign)) return MOE_ERR_INVALID_ARG;
        if (ws_bytes < moe_layer_norm_backward_workspace_size(T, D, dtype)) return MOE_ERR_WORKSPACE;
    }
    const Shape p = shape_of(D, dtype);
    const unsigned grid = grid_of(T, p.lanes, kBwdMaxBlocks);
    (void)hipGetLastError();
    if (T > 0) {
        const BwdArgs a = {h, dy, weight, dh, mean, rstd, dx, sums ? (float*)workspace : nullptr, T, D};
        const hipError_t e = dtype == MOE_BF16 ? launch_backward<bf16_t>(a, p, grid, stream)
                                               : launch_backward<float>(a, p, grid, stream);
        if (e != hipSuccess) return MOE_ERR_HIP;
    }
    if (sums) {
        // with T == 0 there are no partial rows, and the sums are written as zeros
        norm_partial_sum_kernel<<<dim3((D + SUM_COLS - 1) / SUM_COLS, 2), SUM_COLS * SUM_SLICES, 0,
                                  stream>>>((const float*)workspace, (int)grid, D, dweight, dbias);
        if (hipGetLastError() != hipSuccess) return MOE_ERR_HIP;
    }
    return MOE_OK;
}

}  // extern "C"
