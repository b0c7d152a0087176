// newton_schulz.hip -- orthogonalisation of a batch of matrices by
// Newton-Schulz products, and the Muon step around it; the C entry points
// moe_newton_schulz and moe_muon_step.
//
//   X_0 = U / (|U| + eps),  |U| the Frobenius norm
//   A = X X^T on the shorter side m,  X <- a X + (b A + c A A) X,  `steps` times
//   newton_schulz: U = G, out = X
//   muon:          momentum <- beta momentum + dW,  U = dW + beta momentum
//                  (or momentum),  W <- (1 - lr decay) W - lr scale X
//
// Every product is a matrix product on the matrix cores with fp32 accuracy.
// An operand is held as two fp16 planes, hi = f16(v s) and lo = f16(v s - hi)
// with a power of two s, 22 bits of v together, and a product takes the
// three terms hi hi + hi lo + lo hi, summed in fp32: 3 of the fast fp16
// instructions (16x the fp32 ones' rate) keep the iteration at 0.3 to 1.3 of
// fp32's own error, where one fp16 or bf16 plane leaves 2e-3 to 2e-2, since
// small singular values grow by a factor a in each step and their rounding
// with them.  s comes from a bound on the singular values: the host follows
// the largest value of |x (a + b x^2 + c x^4)| from [0, 1] through the steps, an
// entry is never larger than the largest singular value, and s puts the bound
// at 2^15 at most (fp16 ends at 65504).  That bound assumes |X_0| = 1; where eps holds X_0
// down to rho = |U| / (|U| + eps) its planes would lose bits, and vanish below 2^-40.  So each matrix
// has a power of two of its own, lift = log2(1 / rho) rounded down, found with its norm: its planes
// hold 2^e X with e = max(0, lift + room_k) before step k, where 2^room_k is the bound of [0, 1] over
// the largest product of polynomials so far, so that 2^e X stays below the bound.  X's products are
// linear in X, so e enters as one factor of what a tile writes.
//
// Layout: a matrix of planes is cut into blocks of 32 rows by 32 columns of
// 4 KiB, each in the order in which the matrix instruction's lanes take it (plane,
// half of the columns, then 16 bytes for each of the 64 lanes), so a fragment
// is 1 KiB of consecutive memory for its wavefront, whether it goes to LDS or
// to registers, and needs no swizzle there.  Sizes are padded with zeros to multiples of
// 64 (they stay zero through the iteration), so only the first and the last
// kernel know the matrix's own sizes.
//
// Each product is C = P Q^T over row-major operands: A = X X^T takes X's rows
// twice, S = b A + c A A takes A's (A is symmetric), and X <- a X + S X takes S's
// rows and those of X^T; so X is kept in both orders, and an epilogue writes its
// tile in both.  For the symmetric results only tiles on and below the diagonal
// are computed, and their transposed tile is written beside them.
//
// What bounds the products: a compute unit draws 36 to 46 bytes a clock from its
// L2, whether through LDS or straight to registers.  A K step of 32 columns is
// 16, 32 and 64 KiB of a 64-, 128- and 256-tile, so at 36 bytes 450, 900 and 1800 clocks,
// against 192, 768 and about 3000 of matrix instructions: tiles of 64 are bound
// by it, those of 128 by both, those of 256 by the matrix cores (52% of their
// cycles at sixteen 1024 x 4096, the rest the epilogues of one workgroup a unit).
// Few or small matrices fill 256 units with small tiles only, and the smallest
// products are bound by the 4 us of a launch.
#include "mfma_common.h"
#include "moe_ffn.h"

#include <math.h>

#include <type_traits>

namespace moe {
namespace {

using namespace mfma;

typedef __attribute__((address_space(3))) float lds_float_t;
typedef __attribute__((ext_vector_type(8))) _Float16 f16x8_t;
typedef __attribute__((ext_vector_type(2))) _Float16 f16x2_t;

// ---------------------------------------------------------------- elements

struct __attribute__((packed, aligned(4))) Raw4f {
    float v[4];
};
struct __attribute__((packed, aligned(2))) Raw8h {
    uint32_t w[4];
};

// Eight consecutive fp32 or bf16 elements, `left` of which exist.
__device__ __forceinline__ void load8(const void* base, int64_t at, int left, bool bf16, float* v) {
    if (bf16) {
        const uint16_t* p = (const uint16_t*)base + at;
        if (left >= 8) {
            const Raw8h r = *(const Raw8h*)p;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                v[2 * i] = __uint_as_float(r.w[i] << 16);
                v[2 * i + 1] = __uint_as_float(r.w[i] & 0xffff0000u);
            }
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = i < left ? __uint_as_float((uint32_t)p[i] << 16) : 0.f;
        }
    } else {
        const float* p = (const float*)base + at;
        if (left >= 8) {
            const Raw4f r0 = *(const Raw4f*)p, r1 = *(const Raw4f*)(p + 4);
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = r0.v[i], v[4 + i] = r1.v[i];
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = i < left ? p[i] : 0.f;
        }
    }
}
__device__ __forceinline__ void store8(void* base, int64_t at, int left, bool bf16, const float* v) {
    if (bf16) {
        uint16_t* p = (uint16_t*)base + at;
        if (left >= 8) {
            Raw8h r;
#pragma unroll
            for (int i = 0; i < 4; ++i) r.w[i] = pack_bf16(v[2 * i], v[2 * i + 1]);
            *(Raw8h*)p = r;
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (i < left) p[i] = (uint16_t)pack_bf16(v[i], 0.f);
        }
    } else {
        float* p = (float*)base + at;
        if (left >= 8) {
            Raw4f r0, r1;
#pragma unroll
            for (int i = 0; i < 4; ++i) r0.v[i] = v[i], r1.v[i] = v[4 + i];
            *(Raw4f*)p = r0;
            *(Raw4f*)(p + 4) = r1;
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (i < left) p[i] = v[i];
        }
    }
}

// Where U comes from and the result goes.
struct Source {
    const void* g;      // G (newton_schulz, fp32 or bf16) or dW (muon, fp32)
    float* mom;         // muon: momentum; null: newton_schulz
    float beta;
    int nesterov;
    int g_bf16;
};
struct Target {
    void* out;          // newton_schulz: X; muon: W, read and written
    uint16_t* copy;     // muon: bf16 copy of W, or null
    float keep, rate;   // muon: W <- keep W - rate X
    int muon;
    int out_bf16;
};

// U of the muon step from dW and the momentum already moved on.
__device__ __forceinline__ void source8(const Source& s, int64_t at, int left, float* u) {
    load8(s.g, at, left, s.g_bf16, u);
    if (s.mom) {
        float m[8];
        load8(s.mom, at, left, false, m);
#pragma unroll
        for (int i = 0; i < 8; ++i) u[i] = s.nesterov ? fmaf(s.beta, m[i], u[i]) : m[i];
    }
}
// The same for the first pass, which moves the momentum on.
__device__ __forceinline__ void source8_first(const Source& s, int64_t at, int left, float* u) {
    load8(s.g, at, left, s.g_bf16, u);
    if (s.mom) {
        float m[8];
        load8(s.mom, at, left, false, m);
#pragma unroll
        for (int i = 0; i < 8; ++i) m[i] = fmaf(s.beta, m[i], u[i]);
        store8(s.mom, at, left, false, m);
#pragma unroll
        for (int i = 0; i < 8; ++i) u[i] = s.nesterov ? fmaf(s.beta, m[i], u[i]) : m[i];
    }
}
// The weights that eight results will change (muon), and the change: apart, so
// that a thread's loads are all on their way before its first store.
__device__ __forceinline__ void target8_load(const Target& t, int64_t at, int left, float* w) {
    if (t.muon) load8(t.out, at, left, t.out_bf16, w);
}
__device__ __forceinline__ void target8_store(const Target& t, int64_t at, int left, float* v, const float* w) {
    if (t.muon) {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = fmaf(-t.rate, v[i], t.keep * w[i]);
        if (t.copy) store8(t.copy, at, left, true, v);
    }
    store8(t.out, at, left, t.out_bf16, v);
}

// ------------------------------------------------------- norm and planes

// Sum of squares of one matrix's U, by norm_blocks(size) workgroups, in fp64
// (fp32 squares would overflow or vanish for gradients of 1e20 or 1e-20).
// Four turns of 8 elements a thread, or one while that makes at most 128 workgroups
// (1000 x 333: 4.1 -> 3.2 us).
constexpr int kNormMaxBlocks = 256;
int norm_blocks(int64_t size) {
    const int64_t one = (size + 2047) / 2048, four = (size + 8191) / 8192, n = one < 128 ? one : four < 128 ? 128 : four;
    return (int)(n < kNormMaxBlocks ? n : kNormMaxBlocks);
}

__device__ __forceinline__ double block_sum(double v, double* red, int waves) {
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o, 64);
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
    __syncthreads();
    v = 0.;
    for (int i = 0; i < waves; ++i) v += red[i];
    return v;
}

__global__ __launch_bounds__(256) void ns_norm_kernel(const Source s, int64_t size, double* part) {
    __shared__ double red[4];
    const int64_t base = (int64_t)blockIdx.y * size;
    double sum = 0.;
    for (int64_t at = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 8; at < size;
         at += (int64_t)gridDim.x * 256 * 8) {
        float u[8];
        source8_first(s, base + at, (int)min((int64_t)8, size - at), u);
#pragma unroll
        for (int i = 0; i < 8; ++i) sum = fma((double)u[i], (double)u[i], sum);
    }
    sum = block_sum(sum, red, 4);
    if (threadIdx.x == 0) part[(int64_t)blockIdx.y * gridDim.x + blockIdx.x] = sum;
}

// hi and lo of eight scaled values.
__device__ __forceinline__ void split8(const float* v, u32x4_t& hi, u32x4_t& lo) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const f16x2_t h = {(_Float16)v[2 * i], (_Float16)v[2 * i + 1]};
        const f16x2_t l = {(_Float16)(v[2 * i] - (float)h[0]), (_Float16)(v[2 * i + 1] - (float)h[1])};
        hi[i] = __builtin_bit_cast(uint32_t, h);
        lo[i] = __builtin_bit_cast(uint32_t, l);
    }
}
// Planes of a 32 x 32 block: [hi, lo][columns 0..15, 16..31][lane][8 values],
// lane = row % 32 + 32 for the second eight columns of a half.
constexpr int BLOCK = 4096, LO = 2048, HALF = 1024;
// Byte offset of the hi values of columns c .. c + 7 (c a multiple of 8) of a
// row; ld is the padded row length.  The lo values are LO bytes on.
__device__ __forceinline__ int64_t plane_at(int row, int ld, int c) {
    return ((int64_t)(row >> 5) * (ld >> 5) + (c >> 5)) * BLOCK + ((c >> 4) & 1) * HALF + ((c >> 3) & 1) * 512 +
           (row & 31) * 16;
}
__device__ __forceinline__ void store_planes(char* base, int64_t at, const float* v) {
    u32x4_t hi, lo;
    split8(v, hi, lo);
    *(u32x4_t*)(base + at) = hi;
    *(u32x4_t*)(base + at + LO) = lo;
}
__device__ __forceinline__ void add_planes(const u32x4_t hi, const u32x4_t lo, float f, float* v) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t hw = hi[i], lw = lo[i];
        const f16x2_t h = __builtin_bit_cast(f16x2_t, hw), l = __builtin_bit_cast(f16x2_t, lw);
        v[2 * i] = fmaf(f, (float)h[0] + (float)l[0], v[2 * i]);
        v[2 * i + 1] = fmaf(f, (float)h[1] + (float)l[1], v[2 * i + 1]);
    }
}

struct SplitArgs {
    Source s;
    const double* part;     // [B][nb]
    int nb;
    int M, N;               // U's own sizes
    int Mp, Np;             // padded
    double eps;
    float scale;
    int* lift;              // [B], out
    char *rows, *cols;      // planes [B][Mp][Np] (U's rows) and [B][Np][Mp] (its columns)
};
constexpr int ST = 64;
__global__ __launch_bounds__(256) void ns_split_kernel(const SplitArgs a) {
    __shared__ float tile[ST][ST + 1];
    __shared__ double red[4];
    const int b = blockIdx.z, i0 = blockIdx.y * ST, j0 = blockIdx.x * ST, tid = threadIdx.x;
    const int64_t base = (int64_t)b * a.M * a.N;
    char* rows = a.rows + (int64_t)b * a.Mp * a.Np * 4;
    char* cols = a.cols + (int64_t)b * a.Mp * a.Np * 4;
    const double mine = tid < a.nb ? a.part[(int64_t)b * a.nb + tid] : 0.;
    float in[2][8];              // on their way while the norm is added up
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const int r = (tid >> 3) + 32 * k, left = a.N - (j0 + (tid & 7) * 8);
        if (i0 + r < a.M && left > 0) source8(a.s, base + (int64_t)(i0 + r) * a.N + j0 + (tid & 7) * 8, left, in[k]);
    }
    const double norm = sqrt(block_sum(mine, red, 4)), more = (norm + a.eps) / norm;
    // finite: neither a zero matrix nor one that holds an infinity or NaN
    const int lift = more >= 2. && more < INFINITY ? ilogb(more) : 0;
    if (blockIdx.x == 0 && blockIdx.y == 0 && tid == 0) a.lift[b] = lift;
    const double inv = ldexp((double)a.scale / (norm + a.eps), lift);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const int r = (tid >> 3) + 32 * k, c = (tid & 7) * 8, left = i0 + r < a.M ? a.N - (j0 + c) : 0;
#pragma unroll
        for (int e = 0; e < 8; ++e) tile[r][c + e] = e < left ? (float)((double)in[k][e] * inv) : 0.f;
    }
    __syncthreads();
    // consecutive lanes take consecutive rows of the planes written
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const int r = tid & 63, c = ((tid >> 6) + 4 * k) * 8;
        float u[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) u[e] = tile[r][c + e];
        store_planes(rows, plane_at(i0 + r, a.Np, j0 + c), u);
#pragma unroll
        for (int e = 0; e < 8; ++e) u[e] = tile[c + e][r];
        store_planes(cols, plane_at(j0 + r, a.Mp, i0 + c), u);
    }
}

// ---------------------------------------------------------------- products

// GRAM:  C = f P P^T
// SYMM:  C = f P Q + fa P + fq Q for symmetric P and Q that commute (polynomials
//        of one matrix), so that C is symmetric
// APPLY: C = f P Q^T + fa X, P on the short side, Q = X^T
// FINAL: the same into the target
enum : int { GRAM = 0, SYMM = 1, APPLY = 2, FINAL = 3 };

constexpr int BT = 128;                       // tile rows and columns
constexpr int KB = 32;                        // K step
constexpr int TLD = BT + 1;                   // row of the fp32 tile in LDS

struct MulArgs {
    const char *p, *q;          // planes [B][pr][K], [B][qr][K]
    int64_t p_stride, q_stride; // bytes per matrix
    int pr, qr, K;              // padded rows of each side, reduction length
    int ti, tj;                 // tiles of each side
    int whole;                  // mixed tiles: how many of 128
    float f;                    // factor of the product
    const char* add;            // SYMM: P; APPLY, FINAL: X
    int64_t add_stride;
    float fa;                   // factor of the addend
    float fq;                   // SYMM: factor of Q, added too (0: not)
    float so;                   // scale of the stored planes
    char *c, *ct;               // planes out, as computed and transposed
    int64_t c_stride;
    const int* lift;            // [B]; room: before this product and after it
    int room, room_after;
    int swap;                   // FINAL: the target is the transposed tile
    int M, N;                   // FINAL: the target's sizes
    Target t;
};

// Row of accumulator register g within its 32 x 32 block (the column is lane % 32).
__device__ __forceinline__ int acc_row(int g, int kh) { return 8 * (g >> 2) + (g & 3) + 4 * kh; }

// acc[i][j] += (ph[i] + pl[i])(qh[j] + ql[j])^T without the product of the two
// low parts, term by term over the blocks, so that instructions in a row do not
// wait for each other's sums.
template <int NI, int NJ>
__device__ __forceinline__ void mul3(f32x16_t (&acc)[NI][NJ], const f16x8_t* ph, const f16x8_t* pl,
                                     const f16x8_t* qh, const f16x8_t* ql) {
#pragma unroll
    for (int t = 0; t < 3; ++t)
#pragma unroll
        for (int i = 0; i < NI; ++i)
#pragma unroll
            for (int j = 0; j < NJ; ++j)
                acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(t == 2 ? pl[i] : ph[i], t == 1 ? ql[j] : qh[j],
                                                                   acc[i][j], 0, 0, 0);
}

// The matrix and tile of number id; of a symmetric result the tiles on and
// below the diagonal.  Each XCD takes a contiguous range (xcd_remap), so its L2
// holds one matrix's operands (or a band of rows).
template <bool SYM>
__device__ __forceinline__ void tile_of(const MulArgs& a, int id, int& b, int& ti, int& tj) {
    const int per = SYM ? a.ti * (a.ti + 1) / 2 : a.ti * a.tj;
    b = id / per;
    const int t = id - b * per;
    if constexpr (SYM) {
        ti = (int)((sqrtf(8.f * t + 1.f) - 1.f) * 0.5f);
        while (ti * (ti + 1) / 2 > t) --ti;
        while ((ti + 1) * (ti + 2) / 2 <= t) ++ti;
        tj = t - ti * (ti + 1) / 2;
    } else {
        ti = t % a.ti;
        tj = t / a.ti;
    }
}

// What a matrix's own power of two comes to in what a product writes.
template <int MODE>
__device__ __forceinline__ float lift_factor(const MulArgs& a, int b) {
    if constexpr (MODE == SYMM) return 1.f;
    const int lift = a.lift[b], e = max(0, lift + a.room);
    return ldexpf(1.f, MODE == GRAM ? -2 * e : MODE == APPLY ? max(0, lift + a.room_after) - e : -e);
}

// From the sums of a TS x TS tile (sum8: eight of a row) to what the mode
// writes: eight values a thread along the rows, and, through the fp32 tile
// `at` in LDS, along the columns for the transposed order.
template <int MODE, int TS, int NT, typename Sum8, typename At>
__device__ __forceinline__ void epilogue(const MulArgs& a, float lift, int b, int i0, int j0, bool both,
                                         Sum8 sum8, At at) {
    constexpr int SEGS = TS / 8, PASSES = (TS * SEGS + NT - 1) / NT;
    // consecutive lanes take consecutive rows (the planes' order), or, for the
    // target, the segments of a row
    auto place = [](int id, int& row, int& seg) {
        row = MODE == FINAL ? id / SEGS : id % TS;
        seg = 8 * (MODE == FINAL ? id % SEGS : id / TS);
    };
    if (MODE == FINAL) both = a.swap;
    const float so = a.so * lift;
    auto here = [&](int r, int c) { return r < TS && c < TS && i0 + r < a.pr && j0 + c < a.qr; };
    // FINAL: where a piece of the target's row `row` begins
    auto target_at = [&](int row, int seg) {
        return a.swap ? ((int64_t)b * a.M + j0 + row) * a.N + i0 + seg : ((int64_t)b * a.M + i0 + row) * a.N + j0 + seg;
    };
    auto target_left = [&](int row, int seg) {
        if ((a.swap ? j0 : i0) + row >= a.M) return 0;
        return a.N - (a.swap ? i0 : j0) - seg;
    };
    // all addends, and the weights of the target, on their way before the first store
    float w[MODE == FINAL ? PASSES : 1][8];
    if constexpr (MODE == FINAL) {
#pragma unroll
        for (int k = 0; k < PASSES; ++k) {
            int row, seg;
            place(threadIdx.x + k * NT, row, seg);
            const int left = row < TS && seg < TS ? target_left(row, seg) : 0;
            if (left > 0) target8_load(a.t, target_at(row, seg), left, w[k]);
        }
    }
    u32x4_t hi[PASSES], lo[PASSES], qhi[PASSES], qlo[PASSES];
    if constexpr (MODE != GRAM) {
#pragma unroll
        for (int k = 0; k < PASSES; ++k) {
            int r, c;
            place(threadIdx.x + k * NT, r, c);
            if (!here(r, c)) continue;
            const int64_t from = plane_at(i0 + r, a.qr, j0 + c);
            const char* p = a.add + b * a.add_stride + from;
            hi[k] = *(const u32x4_t*)p;
            lo[k] = *(const u32x4_t*)(p + LO);
            if (MODE == SYMM && a.fq != 0.f) {
                p = a.q + b * a.q_stride + from;
                qhi[k] = *(const u32x4_t*)p;
                qlo[k] = *(const u32x4_t*)(p + LO);
            }
        }
    }
#pragma unroll
    for (int k = 0; k < PASSES; ++k) {
        int r, c;
        place(threadIdx.x + k * NT, r, c);
        if (!here(r, c)) continue;
        float v[8];
        sum8(r, c, v);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] *= a.f;
        if constexpr (MODE != GRAM) add_planes(hi[k], lo[k], a.fa, v);
        if (MODE == SYMM && a.fq != 0.f) add_planes(qhi[k], qlo[k], a.fq, v);
        if constexpr (MODE != FINAL) {
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] *= so;
            store_planes(a.c + b * a.c_stride, plane_at(i0 + r, a.qr, j0 + c), v);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] *= lift;
            const int left = a.swap ? 0 : target_left(r, c);
            if (left > 0) target8_store(a.t, target_at(r, c), left, v, w[k]);
        }
        if (both) {
#pragma unroll
            for (int e = 0; e < 8; ++e) at(r, c + e) = v[e];
        }
    }
    if (!both) return;
    __syncthreads();
#pragma unroll
    for (int k = 0; k < PASSES; ++k) {
        int c, r;
        place(threadIdx.x + k * NT, c, r);
        if (!here(r, c)) continue;
        float v[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = at(r + e, c);
        if constexpr (MODE != FINAL) {
            store_planes(a.ct + b * a.c_stride, plane_at(j0 + c, a.pr, i0 + r), v);
        } else {
            const int left = target_left(c, r);
            if (left > 0) target8_store(a.t, target_at(c, r), left, v, w[k]);
        }
    }
}

// The same from accumulators, for the modes that write planes, a wavefront's
// 32 x 32 blocks by themselves.  A lane holds four rows in a row of one column, half
// of a 16-byte piece of the transposed block, which goes out as it is (64 lanes,
// 512 consecutive bytes); for the other order the block's planes pass through 4 KiB of
// LDS of the wavefront's own, written in the transposed order and read back with
// the transposing read.  The addends are blocks at the transposed place, of the
// symmetric operands or of X^T, in the order of the accumulators.  Through an
// fp32 tile and two passes of 8 values a thread the same took about 7 us of a
// 128-tile; this takes 2.
template <int MODE, int NI, int NJ>
__device__ __forceinline__ void epilogue_blocks(const MulArgs& a, float lift, int b, int ib0, int jb0, bool both,
                                                const f32x16_t (&acc)[NI][NJ], char* lds) {
    const float so = a.so * lift;
    const int lane = threadIdx.x & 63, rl = lane & 31, kh = lane >> 5;
    const int pb = a.pr >> 5, qb = a.qr >> 5;
    // piece q (rows 8 q .. + 7) of the transposed block; + LO for the low plane
    auto piece = [&](int q) { return (q >> 1) * HALF + (q & 1) * 512 + rl * 16 + kh * 8; };
    struct Addend {
        uint2 hi[4], lo[4];
    };
    auto fetch = [&](const char* base, int64_t stride, int i, int j, Addend& d) {
        const int ib = min(ib0 + i, pb - 1), jb = min(jb0 + j, qb - 1);
        const char* p = base + b * stride + ((int64_t)jb * pb + ib) * BLOCK;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            d.hi[q] = *(const uint2*)(p + piece(q));
            d.lo[q] = *(const uint2*)(p + piece(q) + LO);
        }
    };
    auto add4 = [&](const Addend& d, int q, float f, float* v) {
        const uint32_t hw[2] = {d.hi[q].x, d.hi[q].y}, lw[2] = {d.lo[q].x, d.lo[q].y};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const f16x2_t h = __builtin_bit_cast(f16x2_t, hw[e >> 1]), l = __builtin_bit_cast(f16x2_t, lw[e >> 1]);
            v[e] = fmaf(f, (float)h[e & 1] + (float)l[e & 1], v[e]);
        }
    };
    const bool second = MODE == SYMM && a.fq != 0.f;
    auto one = [&](int i, int j, const Addend& d, const Addend& dq) {
        const int ib = ib0 + i, jb = jb0 + j;
        if (ib >= pb || jb >= qb) return;
        char* ct = a.ct + b * a.c_stride + ((int64_t)jb * pb + ib) * BLOCK;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            float v[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = acc[i][j][4 * q + e] * a.f;
            if constexpr (MODE != GRAM) add4(d, q, a.fa, v);
            if (second) add4(dq, q, a.fq, v);
            uint32_t oh[2], ol[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const float x = v[2 * e] * so, y = v[2 * e + 1] * so;
                const f16x2_t h = {(_Float16)x, (_Float16)y};
                const f16x2_t l = {(_Float16)(x - (float)h[0]), (_Float16)(y - (float)h[1])};
                oh[e] = __builtin_bit_cast(uint32_t, h);
                ol[e] = __builtin_bit_cast(uint32_t, l);
            }
            *(uint2*)(ct + piece(q)) = make_uint2(oh[0], oh[1]);
            *(uint2*)(ct + piece(q) + LO) = make_uint2(ol[0], ol[1]);
            if (both) {
                *(uint2*)(lds + piece(q)) = make_uint2(oh[0], oh[1]);
                *(uint2*)(lds + piece(q) + LO) = make_uint2(ol[0], ol[1]);
            }
        }
        if (!both) return;
        // the other lanes' writes: LDS serves a wavefront in order
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
        char* c = a.c + b * a.c_stride + ((int64_t)ib * qb + jb) * BLOCK;
        // a read gives lane s of 16 row 16 (G & 1) + s of the block, four columns;
        // group G = lane / 16 takes the eight columns 8 (G >> 1) of each half
        const int G = lane >> 4, sl = lane & 15;
        const int src = (G & 1) * HALF + ((sl >> 1) & 1) * 512 + (8 * (G >> 1) + (sl >> 2)) * 16 + (sl & 1) * 8;
#pragma unroll
        for (int p = 0; p < 2; ++p)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const char* at = lds + p * LO + src + 256 * h;
                const s16x4_t x = read_tr(at), y = read_tr(at + 64);
                const s16x8_t w = __builtin_shufflevector(x, y, 0, 1, 2, 3, 4, 5, 6, 7);
                *(s16x8_t*)(c + p * LO + h * HALF + lane * 16) = w;
            }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
    };
#pragma unroll
    for (int i = 0; i < NI; ++i) {
        Addend d[NJ], dq[NJ];
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
            if constexpr (MODE == SYMM) fetch(a.p, a.p_stride, i, j, d[j]);
            if constexpr (MODE == APPLY) fetch(a.q, a.q_stride, i, j, d[j]);
            if (second) fetch(a.q, a.q_stride, i, j, dq[j]);
        }
#pragma unroll
        for (int j = 0; j < NJ; ++j) one(i, j, d[j], dq[j]);
    }
}

// Tiles of T = 64 NI rows and columns, four wavefronts of 32 NI x 32 NI each.  A
// stage holds KS halves of a K step (16 columns each), in a ring of NS stages;
// operands are in registers for the stage that is multiplied and the one that is
// read.  As many workgroups as fit share a compute unit, one's epilogue under
// the others' matrix instructions.
//  * KS = 1, NS = 4: a stage has three half steps to arrive, in the LDS of two
//    whole ones (against a ring of two whole steps: 576 128-tiles, k = 128: 253 ->
//    213 us; 4096 tiles, k = 32: 451 -> 429; 78 64-tiles, k = 48: 21.8 -> 14.5)
//  * KS = 2, NS = 2: half the barriers, for 64-tiles with two or three workgroups a
//    unit (528 tiles, k = 256: 158 -> 134 us; 640, k = 32: 25.8 -> 23.8; at 408,
//    k = 64, it loses: 25.7 -> 32.4)
// 64-tiles whose wavefronts hold the whole tile and share out the K steps,
// straight from memory to registers, halve the LDS reads and gain nothing (624
// tiles, k = 48: 33 us, 31.5 here): LDS is not what they wait for.
template <int NI, int KS>
constexpr int stage_bytes() {
    return 4 * NI * KS * (BLOCK / 2);
}
// Bytes of a stage's buffer; in the end each holds rows of the fp32 tile, T / NS of them.
template <int NI, int KS, int NS>
constexpr int buffer_bytes() {
    constexpr int T = 64 * NI, rows = T / NS * (T + 1) * 4;
    return rows > stage_bytes<NI, KS>() ? rows : stage_bytes<NI, KS>();
}
// The tile at rows i0, columns j0 of matrix b.  The stages are separate objects, so
// that a read of one does not wait for the transfers into the others (st2 and
// st3 with NS = 4 only).
template <int MODE, int NI, int KS, int NS>
__device__ __forceinline__ void product_tile(const MulArgs& a, int b, int i0, int j0, bool both, char* st0,
                                             char* st1, char* st2, char* st3) {
    constexpr int T = 64 * NI, NB = T / 32, LD = T + 1;
    constexpr int PIECE = 1024, ENTRY = 2 * KS * PIECE;      // a block's share of a stage: [plane][half]
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const float lift = lift_factor<MODE>(a, b);

    // stage sources: wavefront w brings blocks w NB / 2 .. of the P then Q block
    // rows, 2 KS transfers of 1 KiB each.  Block rows past the padded end (tiles
    // that end outside) read the last one and are not stored.
    const int KT = a.K / KB;     // even
    constexpr int MINE = NB / 2, PER_STAGE = 2 * KS * MINE;
    const char* src[MINE];
#pragma unroll
    for (int i = 0; i < MINE; ++i) {
        const int blk = wave * MINE + i;
        const bool second = blk >= NB;
        const int row = second ? min((j0 >> 5) + blk - NB, (a.qr >> 5) - 1) : min((i0 >> 5) + blk, (a.pr >> 5) - 1);
        src[i] = (second ? a.q + b * a.q_stride : a.p + b * a.p_stride) + (int64_t)row * KT * BLOCK;
    }
    auto issue = [&](int n, char* st) {
        const int64_t o = KS == 2 ? (int64_t)n * BLOCK : (int64_t)(n >> 1) * BLOCK + (n & 1) * HALF;
#pragma unroll
        for (int j = 0; j < 2 * KS; ++j)
#pragma unroll
            for (int i = 0; i < MINE; ++i)
                load_lds16(src[i] + o + (j / KS) * LO + (j % KS) * HALF + lane * 16,
                           st + (wave * MINE + i) * ENTRY + j * PIECE);
    };

    const int wi = wave >> 1, wj = wave & 1, rl = lane & 31, kh = lane >> 5;
    f32x16_t acc[NI][NI];
#pragma unroll
    for (int i = 0; i < NI; ++i)
#pragma unroll
        for (int j = 0; j < NI; ++j) acc[i][j] = f32x16_t{};

    struct Frags {
        f16x8_t ph[KS][NI], pl[KS][NI], qh[KS][NI], ql[KS][NI];
    };
    auto read = [&](const char* st, Frags& f) {
        auto frag = [&](const char* p) { return __builtin_bit_cast(f16x8_t, *(const u32x4_t*)(p + lane * 16)); };
#pragma unroll
        for (int ks = 0; ks < KS; ++ks)
#pragma unroll
            for (int i = 0; i < NI; ++i) {
                const char* pb = st + (NI * wi + i) * ENTRY + ks * PIECE;
                const char* qb = st + (NB + NI * wj + i) * ENTRY + ks * PIECE;
                f.ph[ks][i] = frag(pb);
                f.pl[ks][i] = frag(pb + KS * PIECE);
                f.qh[ks][i] = frag(qb);
                f.ql[ks][i] = frag(qb + KS * PIECE);
            }
    };
    // Stage n, its operands already in registers: wait until stage n + 1 has
    // landed and this wavefront's reads of stage n are done; after the barrier
    // stage n's buffer is free, so stage n + NS is sent there, stage n + 1 is
    // read into the other registers and the matrix instructions of stage n run
    // over both.  Past the last stage the last one is sent and read again, so
    // that every step is alike.
    const int last = 2 * KT / KS - 1;
    auto step = [&](int n, const Frags& fc, Frags& fn, char* cur, const char* nxt) {
        __builtin_amdgcn_s_waitcnt(waitcnt_imm((NS - 2) * PER_STAGE, 0));
        __builtin_amdgcn_s_barrier();
        __builtin_amdgcn_sched_barrier(0);
        issue(min(n + NS, last), cur);
        read(nxt, fn);
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) mul3(acc, fc.ph[ks], fc.pl[ks], fc.qh[ks], fc.ql[ks]);
        if constexpr (NI == 2) {
#pragma unroll
            for (int i = 0; i < 4 * KS; ++i) {
                __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);   // matrix instruction
                __builtin_amdgcn_sched_group_barrier(0x010, 1, 0);   // transfer
                __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
                __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);   // LDS read
                __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
                __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
            }
        }
        __builtin_amdgcn_sched_barrier(0);
    };
    static_assert(NS == 2 || (NS == 4 && KS == 1), "stages in fours: 2 KT is a multiple of 4");
    Frags f0, f1;
    issue(0, st0);
    issue(1, st1);
    if constexpr (NS == 4) {
        issue(2, st2);
        issue(3, st3);
    }
    __builtin_amdgcn_s_waitcnt(waitcnt_imm((NS - 1) * PER_STAGE, 15));   // stage 0 has landed
    __builtin_amdgcn_s_barrier();
    read(st0, f0);
    for (int n = 0; n <= last; n += NS) {
        step(n, f0, f1, st0, st1);
        if constexpr (NS == 2) {
            step(n + 1, f1, f0, st1, st0);
        } else {
            step(n + 1, f1, f0, st1, st2);
            step(n + 2, f0, f1, st2, st3);
            step(n + 3, f1, f0, st3, st0);
        }
    }
    __builtin_amdgcn_s_waitcnt(waitcnt_imm(0, 0));           // before the buffers are used anew
    __syncthreads();

    if constexpr (MODE != FINAL) {
        char* mine = NS == 2 ? st0 + wave * BLOCK : wave == 0 ? st0 : wave == 1 ? st1 : wave == 2 ? st2 : st3;
        epilogue_blocks<MODE>(a, lift, b, (i0 >> 5) + NI * wi, (j0 >> 5) + NI * wj, both, acc, mine);
        return;
    }
    // ---- the target: the fp32 tile through LDS, T / NS rows a buffer
    // (a sum of distances: choosing among four pointers kept them in scratch memory)
    lds_float_t* const first = (lds_float_t*)st0;
    const int d1 = (lds_float_t*)st1 - first, d2 = (lds_float_t*)st2 - (lds_float_t*)st1,
              d3 = (lds_float_t*)st3 - (lds_float_t*)st2;
    auto at = [=](int r, int c) -> lds_float_t& {
        constexpr int rows = T / NS;
        const int to = (r >= rows ? d1 : 0) + (NS == 4 && r >= 2 * rows ? d2 : 0) + (NS == 4 && r >= 3 * rows ? d3 : 0);
        return first[to + (r & (rows - 1)) * LD + c];
    };
#pragma unroll
    for (int i = 0; i < NI; ++i)
#pragma unroll
        for (int j = 0; j < NI; ++j)
#pragma unroll
            for (int g = 0; g < 16; ++g)
                at(32 * (NI * wi + i) + acc_row(g, kh), 32 * (NI * wj + j) + rl) = acc[i][j][g];
    __syncthreads();
    auto sum8 = [&](int r, int c, float* v) {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = at(r, c + e);
    };
    epilogue<MODE, T, 256>(a, lift, b, i0, j0, true, sum8, at);
}

template <int MODE, int NI, int KS, int NS>
__global__ __launch_bounds__(256, 2) void ns_product_kernel(const MulArgs a) {
    constexpr bool SYM = MODE == GRAM || MODE == SYMM;
    constexpr int BYTES = buffer_bytes<NI, KS, NS>(), MORE = NS == 4 ? BYTES : 16;
    __shared__ __attribute__((aligned(1024))) char st0[BYTES];
    __shared__ __attribute__((aligned(1024))) char st1[BYTES];
    __shared__ __attribute__((aligned(1024))) char st2[MORE];
    __shared__ __attribute__((aligned(1024))) char st3[MORE];
    int b, ti, tj;
    tile_of<SYM>(a, xcd_remap(blockIdx.x, gridDim.x), b, ti, tj);
    product_tile<MODE, NI, KS, NS>(a, b, 64 * NI * ti, 64 * NI * tj, !SYM || ti != tj, st0, st1, st2, st3);
}

// 128-tiles in full rounds of 256 and the few that remain as four 64-tiles each,
// so that they end sooner than a round of their own: a.whole tiles of 128,
// then 4 (all - whole) workgroups of 64.  576 tiles, k = 32: 60 us, 68 with every
// tile of 128; k = 128: 213 and 238; 288 tiles, k = 24: 27.5 and 33.9.
template <int MODE>
__global__ __launch_bounds__(256, 2) void ns_product_mixed_kernel(const MulArgs a) {
    constexpr bool SYM = MODE == GRAM || MODE == SYMM;
    constexpr int BYTES = buffer_bytes<2, 1, 4>();
    __shared__ __attribute__((aligned(1024))) char st0[BYTES];
    __shared__ __attribute__((aligned(1024))) char st1[BYTES];
    __shared__ __attribute__((aligned(1024))) char st2[BYTES];
    __shared__ __attribute__((aligned(1024))) char st3[BYTES];
    int b, ti, tj;
    if ((int)blockIdx.x < a.whole) {
        tile_of<SYM>(a, xcd_remap(blockIdx.x, a.whole), b, ti, tj);
        product_tile<MODE, 2, 1, 4>(a, b, BT * ti, BT * tj, !SYM || ti != tj, st0, st1, st2, st3);
        return;
    }
    const int id = xcd_remap(blockIdx.x - a.whole, gridDim.x - a.whole);
    tile_of<SYM>(a, a.whole + (id >> 2), b, ti, tj);
    const int i0 = BT * ti + 64 * ((id >> 1) & 1), j0 = BT * tj + 64 * (id & 1);
    if (i0 >= a.pr || j0 >= a.qr || (SYM && i0 < j0)) return;
    product_tile<MODE, 1, 1, 4>(a, b, i0, j0, !SYM || i0 != j0, st0, st1, st2, st3);
}

// 256 x 256 tiles for long grids: eight wavefronts of 128 x 64, one workgroup a
// compute unit.  A byte from memory feeds twice the products of a 128-tile,
// and an LDS byte 1.5 times.  A stage is one half of the columns of a K step
// (32 KiB), in a ring of four, held in registers for the one that is multiplied
// and the one that is read: a stage has three half steps to arrive.
constexpr int LT = 256;
template <int MODE>
__global__ __launch_bounds__(512, 2) void ns_product_large_kernel(const MulArgs a) {
    constexpr bool SYM = MODE == GRAM || MODE == SYMM;
    constexpr int NB = LT / 32, PIECE = 1024, OPB = NB * 2 * PIECE;      // a block's hi and lo halves
    // in the end two of them hold a quadrant of the fp32 tile
    constexpr int BYTES = BT / 2 * TLD * 4;
    static_assert(BYTES >= 2 * OPB, "a stage fits");
    __shared__ __attribute__((aligned(1024))) char st0[BYTES];
    __shared__ __attribute__((aligned(1024))) char st1[BYTES];
    __shared__ __attribute__((aligned(1024))) char st2[BYTES];
    __shared__ __attribute__((aligned(1024))) char st3[BYTES];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    int b, ti, tj;
    tile_of<SYM>(a, xcd_remap(blockIdx.x, gridDim.x), b, ti, tj);
    const int i0 = ti * LT, j0 = tj * LT;
    const float lift = lift_factor<MODE>(a, b);
    const int KT = a.K / KB;     // even
    const char* ps = a.p + b * a.p_stride + (int64_t)min((i0 >> 5) + wave, (a.pr >> 5) - 1) * KT * BLOCK;
    const char* qs = a.q + b * a.q_stride + (int64_t)min((j0 >> 5) + wave, (a.qr >> 5) - 1) * KT * BLOCK;
    // half step h: columns 16 (h & 1) .. of block h / 2
    auto issue = [&](int h, char* st) {
        const int64_t o = (int64_t)(h >> 1) * BLOCK + (h & 1) * HALF + lane * 16;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            load_lds16(ps + o + j * LO, st + (2 * wave + j) * PIECE);
            load_lds16(qs + o + j * LO, st + OPB + (2 * wave + j) * PIECE);
        }
    };
    const int wi = wave >> 2, wj = wave & 3, rl = lane & 31, kh = lane >> 5;
    f32x16_t acc[4][2];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) acc[i][j] = f32x16_t{};
    struct Frags {
        f16x8_t ph[4], pl[4], qh[2], ql[2];
    };
    auto read = [&](const char* st, Frags& f) {
        auto frag = [&](const char* p) { return __builtin_bit_cast(f16x8_t, *(const u32x4_t*)(p + lane * 16)); };
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const char* qb = st + OPB + (2 * wj + j) * 2 * PIECE;
            f.qh[j] = frag(qb);
            f.ql[j] = frag(qb + PIECE);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const char* pb = st + (4 * wi + i) * 2 * PIECE;
            f.ph[i] = frag(pb);
            f.pl[i] = frag(pb + PIECE);
        }
    };
    // Half step h, its operands already in registers: wait until stage h + 1 has
    // landed (the two after it may be on their way) and this wavefront's reads
    // of stage h are done; after the barrier its buffer takes stage h + 4.
    const int last = 2 * KT - 1;
    auto step = [&](int h, const Frags& fc, Frags& fn, char* cur, const char* nxt) {
        __builtin_amdgcn_s_waitcnt(waitcnt_imm(8, 0));
        __builtin_amdgcn_s_barrier();
        __builtin_amdgcn_sched_barrier(0);
        issue(min(h + 4, last), cur);
        read(nxt, fn);
        mul3(acc, fc.ph, fc.pl, fc.qh, fc.ql);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);   // matrix instruction
            __builtin_amdgcn_sched_group_barrier(0x010, 1, 0);   // transfer
            __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
            __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);   // LDS read
            __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
            __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
            __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
            __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
        }
        __builtin_amdgcn_sched_barrier(0);
    };
    Frags f0, f1;
    issue(0, st0);
    issue(1, st1);
    issue(2, st2);               // 2 KT >= 4
    issue(3, st3);
    __builtin_amdgcn_s_waitcnt(waitcnt_imm(12, 15));
    __builtin_amdgcn_s_barrier();
    read(st0, f0);
    __builtin_amdgcn_sched_barrier(0);
    for (int h = 0; h <= last; h += 4) {
        step(h, f0, f1, st0, st1);
        step(h + 1, f1, f0, st1, st2);
        step(h + 2, f0, f1, st2, st3);
        step(h + 3, f1, f0, st3, st0);
    }
    __builtin_amdgcn_s_waitcnt(waitcnt_imm(0, 0));
    __syncthreads();

    if constexpr (MODE != FINAL) {
        epilogue_blocks<MODE>(a, lift, b, (i0 >> 5) + 4 * wi, (j0 >> 5) + 2 * wj, !SYM || ti != tj, acc, st0 + wave * BLOCK);
        return;
    }
    // ---- the target by quadrants, a row of two at a time
    for (int qi = 0; qi < 2; ++qi) {
        if (i0 + BT * qi >= a.pr) break;
        if (wi == qi) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 2; ++j)
#pragma unroll
                    for (int g = 0; g < 16; ++g)
                        ((float*)(wj < 2 ? (i < 2 ? st0 : st1) : (i < 2 ? st2 : st3)))[(32 * (i & 1) + acc_row(g, kh)) * TLD +
                                                                                    64 * (wj & 1) + 32 * j + rl] = acc[i][j][g];
        }
        __syncthreads();
        auto quadrant = [&](char* top, char* bottom, int qj) {
            if (j0 + BT * qj >= a.qr) return;
            lds_float_t* const first = (lds_float_t*)top;
            const int down = (lds_float_t*)bottom - first;
            auto at = [=](int r, int c) -> lds_float_t& {
                return first[(r < 64 ? 0 : down) + (r & 63) * TLD + c];
            };
            auto sum8 = [&](int r, int c, float* v) {
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] = at(r, c + e);
            };
            epilogue<MODE, BT, 512>(a, lift, b, i0 + BT * qi, j0 + BT * qj, true, sum8, at);
        };
        quadrant(st0, st1, 0);
        quadrant(st2, st3, 1);
        __syncthreads();
    }
}

// The same product for grids that would leave most of the GPU idle: 32 x 32
// tiles whose eight wavefronts share out the K steps among them and add their
// sums through LDS, so that a product of a few hundred rows runs on hundreds of
// compute units and a wavefront's chain of loads is an eighth as long.  Operands go
// from memory straight to registers: nothing in a tile is read twice, so LDS
// would only add its latency.
constexpr int DT = 32, DW = 8;
template <int MODE>
__global__ __launch_bounds__(64 * DW, 2) void ns_product_split_kernel(const MulArgs a) {
    constexpr bool SYM = MODE == GRAM || MODE == SYMM;
    constexpr int LD = DT + 1;
    __shared__ float part[DW][DT * LD];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    int b, ti, tj;
    tile_of<SYM>(a, xcd_remap(blockIdx.x, gridDim.x), b, ti, tj);
    const int rl = lane & 31, kh = lane >> 5;
    const float lift = lift_factor<MODE>(a, b);
    const int KT = a.K / KB;
    const char* pp = a.p + b * a.p_stride + (int64_t)ti * KT * BLOCK;
    const char* qp = a.q + b * a.q_stride + (int64_t)tj * KT * BLOCK;
    const uint32_t at16 = lane * 16;
    struct Frags {
        f16x8_t ph[2][1], pl[2][1], qh[2][1], ql[2][1];   // [k16 slice]
    };
    auto load = [&](int kt, Frags& f) {
        const char *pb = pp + (int64_t)kt * BLOCK, *qb = qp + (int64_t)kt * BLOCK;
#pragma unroll
        for (int ks = 0; ks < 2; ++ks) {
            f.ph[ks][0] = *(const f16x8_t*)(pb + at16 + ks * HALF);
            f.pl[ks][0] = *(const f16x8_t*)(pb + at16 + ks * HALF + LO);
            f.qh[ks][0] = *(const f16x8_t*)(qb + at16 + ks * HALF);
            f.ql[ks][0] = *(const f16x8_t*)(qb + at16 + ks * HALF + LO);
        }
    };
    f32x16_t acc[1][1] = {{f32x16_t{}}};
    auto compute = [&](const Frags& f) {
#pragma unroll
        for (int ks = 0; ks < 2; ++ks) mul3(acc, f.ph[ks], f.pl[ks], f.qh[ks], f.ql[ks]);
    };
    Frags f0, f1;
    if (wave < KT) {
        load(wave, f0);
#pragma unroll 1
        for (int kt = wave; kt < KT; kt += 2 * DW) {
            if (kt + DW < KT) load(kt + DW, f1);
            compute(f0);
            if (kt + DW >= KT) break;
            if (kt + 2 * DW < KT) load(kt + 2 * DW, f0);
            compute(f1);
        }
    }
#pragma unroll
    for (int g = 0; g < 16; ++g) part[wave][acc_row(g, kh) * LD + rl] = acc[0][0][g];
    __syncthreads();
    // a thread's results replace the first partial sums of its own entries
    auto at = [&](int r, int c) -> float& { return part[0][r * LD + c]; };
    auto sum8 = [&](int r, int c, float* v) {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = part[0][r * LD + c + e];
#pragma unroll
        for (int w = 1; w < DW; ++w)
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] += part[w][r * LD + c + e];
    };
    epilogue<MODE, DT, 64 * DW>(a, lift, b, ti * DT, tj * DT, !SYM || ti != tj, sum8, at);
}

// ------------------------------------------------- short sides of up to 64

// With a short side m of at most 32, or 64 in few matrices, nothing is worth planes or
// tiles: since every step multiplies X by a polynomial of A, and those commute, the steps run on
// the m x m side alone,
//   A <- P A P,  Q <- Q P  with P = a I + b A + c A A,
// in fp64 (whose rounding the growth of small singular values leaves far below
// fp32's; for long runs see ns_small_kernel), and X = Q U / (|U| + eps), |U|^2 = trace(U U^T),
// takes U once more.
// One workgroup sums A for a chunk of the long side; each workgroup of the second
// launch adds the chunks' sums, runs the steps by itself and multiplies its
// own chunk.  A matrix of one chunk takes a single launch.
//
// All products are fp64 matrix instructions of 16 x 16 x 4: a lane (g = lane / 16,
// c = lane % 16) holds A[c][k] and B[k][c] and receives rows 4 v + g, column c of the
// result in its value v.  The four instructions of a 16-block take k = 4 v + g, so
// a result block is an operand as it stands: mfma4(X, Y) = X^T Y.  Short sides of up
// to 16 need one block, and the steps stay in one wavefront's registers (0.83 us a
// step through LDS with a barrier for each product, 0.4 there, 0.2 up to 8 rows);
// larger ones are 4, 6 or 10 blocks, one a wavefront, and go through LDS (1.5, 4 and 8 us a
// step, bound by the fp64 instructions).
typedef __attribute__((ext_vector_type(4))) double f64x4_t;
constexpr int kMaxSteps = 64;

// Which short sides go this way.  Up to 32 all: of 91 batches of 1 to 2048 matrices of 8, 16, 24 and 32 by 64
// to 32768 the planes, padded to 64 rows, took 1.9 to 25 times as long (2048 of 8 x 64: 24 us, 258
// in planes; one 32 x 4096 23, 111; 128 of them 305, 714; 512 1383, 2645, the nearest; 128 of
// 32 x 32768 1461, 5756).  Beyond 32 by the workgroups that would run, each of which takes the
// steps by itself: up to 512 with short sides of up to 48 (512 of 48 x 48: 62 us, 107 in planes;
// 8 of 48 x 768 39, 67), 256 up to 64 (64 x 64: 51, 62; 64 x 4096 69, 108; 256 of 64 x 64 54, 71, 300
// would be 102, 85).
constexpr int64_t small_most(int m) { return m <= 32 ? INT64_MAX : m <= 48 ? 512 : m <= 64 ? 256 : -1; }
// Columns of the long side a workgroup takes: all of up to 384 (short sides of
// up to 16) or 256, in turns of 256 by 16 wavefronts in one launch (256 x 8: 6.9 us,
// 9.3 in two launches; 384 x 8: 8.3, 9.3; 768 x 8: 11.7, 9.7; 768 x 16: 15.3, 10.5; 32 x 192:
// 16.6, 17.2; 32 x 256: 18.7, 17.7); otherwise 128, one turn of 8 wavefronts, or more
// where that would be over 64 chunks, whose sums each workgroup adds (32 x 4096:
// 23 us, 331 by one workgroup).
int small_chunk(int M, int N) {
    const int m = M < N ? M : N, n = M < N ? N : M;
    if (m <= 32 && n <= (m <= 16 ? 384 : 256)) return n;
    return n <= 64 * 128 ? 128 : ((n + 63) / 64 + 127) / 128 * 128;
}
int small_chunks(int M, int N) {
    const int n = M < N ? N : M, chunk = small_chunk(M, N);
    return (n + chunk - 1) / chunk;
}

struct SmallArgs {
    Source s;
    Target t;
    int M, N, steps, chunk;      // chunk: columns of the long side a workgroup takes
    double a, b, c, eps;
    double* part;                // [B][chunks][blocks][256] sums of A's blocks on and below the diagonal
};
// What a long run adds to the diagonal of the A that step k starts with (see ns_small_kernel): a
// kernel argument of its own, since 512 bytes more cost every launch 0.15 us.
template <bool LONG>
struct Shifts {
    double of[kMaxSteps];
};
template <>
struct Shifts<false> {};

__device__ __forceinline__ f64x4_t mfma4(f64x4_t x, f64x4_t y, f64x4_t acc) {
#pragma unroll
    for (int v = 0; v < 4; ++v) acc = __builtin_amdgcn_mfma_f64_16x16x4f64(x[v], y[v], acc, 0, 0, 0);
    return acc;
}
__device__ __forceinline__ float load1(const void* base, int64_t at, int bf16) {
    return bf16 ? __uint_as_float((uint32_t)((const uint16_t*)base)[at] << 16) : ((const float*)base)[at];
}
__device__ __forceinline__ float source1(const Source& s, int64_t at, bool first) {
    const float g = load1(s.g, at, s.g_bf16);
    if (!s.mom) return g;
    float m = s.mom[at];
    if (first) s.mom[at] = m = fmaf(s.beta, m, g);
    return s.nesterov ? fmaf(s.beta, m, g) : m;
}
__device__ __forceinline__ void target1(const Target& t, int64_t at, float v) {
    if (t.muon) {
        v = fmaf(-t.rate, v, t.keep * load1(t.out, at, t.out_bf16));
        if (t.copy) t.copy[at] = (uint16_t)pack_bf16(v, 0.f);
    }
    if (t.out_bf16)
        ((uint16_t*)t.out)[at] = (uint16_t)pack_bf16(v, 0.f);
    else
        ((float*)t.out)[at] = v;
}

// Block index of (i, j), i >= j, and how many there are.
__host__ __device__ constexpr int low_block(int i, int j) { return i * (i + 1) / 2 + j; }
__host__ __device__ constexpr int low_blocks(int nb) { return low_block(nb, 0); }

// This workgroup's sum of U U^T over columns lo .. hi - 1 of the long side, NB x NB
// blocks of 16: blocks (0,0), (1,0), (1,1), .. of `sum` ([blocks][256], in LDS).
// A wavefront takes 16 columns at a time.
template <int NB, int NT>
__device__ __forceinline__ void small_gram(const SmallArgs& a, int lo, int hi, double* sum) {
    constexpr int BLOCKS = low_blocks(NB), WAVES = NT / 64;
    __shared__ double part[WAVES][BLOCKS][256];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, g = lane >> 4, c = lane & 15;
    const bool tall = a.M > a.N;
    const int m = tall ? a.N : a.M, n = tall ? a.M : a.N;
    const int64_t base = (int64_t)blockIdx.y * a.M * a.N;
    f64x4_t acc[BLOCKS];
#pragma unroll
    for (int k = 0; k < BLOCKS; ++k) acc[k] = f64x4_t{0., 0., 0., 0.};
#pragma unroll 2
    for (int l0 = lo + 16 * wave; l0 < hi; l0 += 16 * WAVES) {
        f64x4_t u[NB];
#pragma unroll
        for (int k = 0; k < NB; ++k)
#pragma unroll
            for (int v = 0; v < 4; ++v) {
                // four consecutive columns a lane, so that a wide row's are one line's
                const int p = 16 * k + c, l = l0 + 4 * g + v;
                u[k][v] = p < m && l < hi
                              ? (double)source1(a.s, base + (tall ? (int64_t)l * m + p : (int64_t)p * n + l), true)
                              : 0.;
            }
#pragma unroll
        for (int i = 0; i < NB; ++i)
#pragma unroll
            for (int j = 0; j <= i; ++j) acc[low_block(i, j)] = mfma4(u[i], u[j], acc[low_block(i, j)]);
    }
#pragma unroll
    for (int k = 0; k < BLOCKS; ++k)
#pragma unroll
        for (int v = 0; v < 4; ++v) part[wave][k][(4 * v + g) * 16 + c] = acc[k][v];
    __syncthreads();
    for (int e = tid; e < BLOCKS * 256; e += NT) {
        double t = 0.;
#pragma unroll
        for (int w = 0; w < WAVES; ++w) t += part[w][e >> 8][e & 255];
        sum[e] = t;
    }
    __syncthreads();
}

constexpr int kOneThreads = 1024;
// Four blocks a side: fewer wavefronts for the sums (their 10 blocks each go through
// LDS), one for each of the 10 blocks in the steps.
constexpr int gram_threads(int nb) { return nb == 4 ? 256 : 512; }
constexpr int step_threads(int nb, bool one) { return one ? kOneThreads : nb == 4 ? 640 : 512; }
template <int NB>
__global__ __launch_bounds__(gram_threads(NB)) void ns_small_gram_kernel(const SmallArgs a) {
    constexpr int BLOCKS = low_blocks(NB), NT = gram_threads(NB);
    __shared__ double sum[BLOCKS * 256];
    const int n = a.M > a.N ? a.M : a.N, lo = blockIdx.x * a.chunk;
    small_gram<NB, NT>(a, lo, min(lo + a.chunk, n), sum);
    double* out = a.part + ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * (BLOCKS * 256);
    for (int e = threadIdx.x; e < BLOCKS * 256; e += NT) out[e] = sum[e];
}

// ONE: the whole matrix is this workgroup's chunk, and its sums are taken here.
//
// LONG: steps that would multiply A's rounding by more than it can bear.  Where U has no
// component A = 0, and what rounding leaves there, n of either sign, grows by P^2 = a^2 a step as a
// small singular value's square does; a negative one is no square of anything, meets no bound
// and ends in infinity (rank 3 of 8, a = 3.44: 12 steps do, 20 are NaN).  Three measures keep
// such a run an iteration of real singular values, those above fp32's resolution untouched:
//  * shift_k = 2^-46 of the largest square is added to A's diagonal in every step, more than its
//    rounding, so A stays positive, and X X^T <= A stays below the host's bound.  A direction of
//    s |U| is off by 2^-47 / s^2, less than the 2^-24 / s of fp32 arithmetic from s = 2^-23 on.  It
//    holds Q below 2^23 of the bound, so that Q U is off by 2^-30 at most.
//  * A is made symmetric in every step: its skew part would grow alike.
//  * Q <- P Q, the order of X <- P X: by then P and Q share their directions to rounding only, and
//    Q P would multiply it by the large entries of Q.
// Short runs (7 of the usual coefficients, see is_long) need none of it and keep what precision fp64 has.
template <int NB, bool ONE, bool LONG>
__global__ __launch_bounds__(step_threads(NB, ONE)) void ns_small_kernel(const SmallArgs a, const Shifts<LONG> shift) {
    constexpr int BLOCKS = low_blocks(NB), NT = step_threads(NB, ONE), NQ = NB > 2 ? 1 : 2;
    __shared__ double sum[BLOCKS * 256];
    // whole matrices, blocks [i][j] of 16 x 16 in result order: value v of a lane at 64 v + lane
    __shared__ double A[NB][NB][256], P[NB][NB][256], U[NB][NB][256], Q[NQ][NB][NB][256];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, g = lane >> 4, c = lane & 15;
    const bool tall = a.M > a.N;
    const int m = tall ? a.N : a.M, n = tall ? a.M : a.N;
    const int lo = blockIdx.x * a.chunk, hi = min(lo + a.chunk, n);
    if constexpr (ONE) {
        small_gram<NB, NT>(a, lo, hi, sum);
    } else {
        for (int e = tid; e < BLOCKS * 256; e += NT) {
            double t = 0.;
#pragma unroll 8
            for (unsigned k = 0; k < gridDim.x; ++k)
                t += a.part[((int64_t)blockIdx.y * gridDim.x + k) * (BLOCKS * 256) + e];
            sum[e] = t;
        }
        __syncthreads();
    }
    double trace = lane < m ? sum[low_block(lane >> 4, lane >> 4) * 256 + (lane & 15) * 17] : 0.;
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) trace += __shfl_xor(trace, o, 64);
    trace = __shfl(trace, 0, 64);
    const double inv = 1. / (sqrt(trace) + a.eps);

    // this wavefront's next columns of U for the end: the first on their way during the
    // steps, where registers allow
    const int64_t base = (int64_t)blockIdx.y * a.M * a.N;
    float raw[NB][4];
    auto load = [&](int l0) {
#pragma unroll
        for (int k = 0; k < NB; ++k)
#pragma unroll
            for (int v = 0; v < 4; ++v) {
                const int p = 16 * k + 4 * v + g, l = l0 + c;
                raw[k][v] = p < m && l < hi
                                ? source1(a.s, base + (tall ? (int64_t)l * m + p : (int64_t)p * n + l), false)
                                : 0.f;
            }
    };
    int l0 = lo + 16 * wave;
    if (NB == 1 && l0 < hi) load(l0);

    // LONG: a diagonal block's symmetric part (its transpose is its product with 1), the shift added
    auto symmetric = [&](f64x4_t x, double more) {
        f64x4_t one;
#pragma unroll
        for (int v = 0; v < 4; ++v) one[v] = 4 * v + g == c ? 1. : 0.;
        const f64x4_t t = mfma4(x, one, f64x4_t{0., 0., 0., 0.});
#pragma unroll
        for (int v = 0; v < 4; ++v) x[v] = 0.5 * (x[v] + t[v]) + more * one[v];
        return x;
    };
    int q = 0;
    if constexpr (NB == 1) {
        // ---- the steps, all in the registers of one wavefront.  Past m everything is
        // zero, so that up to 8 half of the terms are left out
        if (wave == 0) {
            auto product = [&](f64x4_t x, f64x4_t y) {
                f64x4_t r = {0., 0., 0., 0.};
#pragma unroll
                for (int v = 0; v < 2; ++v) r = __builtin_amdgcn_mfma_f64_16x16x4f64(x[v], y[v], r, 0, 0, 0);
                if (m > 8) {
#pragma unroll
                    for (int v = 2; v < 4; ++v) r = __builtin_amdgcn_mfma_f64_16x16x4f64(x[v], y[v], r, 0, 0, 0);
                }
                return r;
            };
            f64x4_t A1, Q1;
#pragma unroll
            for (int v = 0; v < 4; ++v) A1[v] = sum[(4 * v + g) * 16 + c] * inv * inv;
            if constexpr (LONG) A1 = symmetric(A1, shift.of[0]);
            for (int k = 0; k < a.steps; ++k) {
                f64x4_t P1 = product(A1, A1);
#pragma unroll
                for (int v = 0; v < 4; ++v) {
                    const int i = 4 * v + g;
                    P1[v] = (i == c && i < m ? a.a : 0.) + a.b * A1[v] + a.c * P1[v];
                }
                Q1 = k == 0 ? P1 : LONG ? product(P1, Q1) : product(Q1, P1);
                if (k + 1 < a.steps) A1 = product(product(A1, P1), P1);
                if constexpr (LONG) {
                    if (k + 1 < a.steps) A1 = symmetric(A1, shift.of[k + 1]);
                }
            }
#pragma unroll
            for (int v = 0; v < 4; ++v) Q[0][0][0][LONG ? 16 * c + 4 * v + g : 64 * v + lane] = Q1[v];
        }
        __syncthreads();
    } else {
        // ---- the steps: a wavefront owns block (bi, bj) of every matrix; from three
        // blocks a side on, and in long runs, only those on and below the diagonal, and
        // writes their mirror images too
        constexpr bool LOWER = NB > 2 || LONG;
        const bool works = wave < (LOWER ? BLOCKS : NB * NB);
        const int bi = !LOWER ? wave >> 1 & 1 : !works || wave < 1 ? 0 : wave < 3 ? 1 : wave < 6 ? 2 : 3;
        const int bj = !LOWER ? wave & 1 : works ? wave - low_block(bi, 0) : 0;
        auto block = [&](double (*x)[NB][256], double (*y)[NB][256], int i, int j) {
            f64x4_t acc = {0., 0., 0., 0.};
#pragma unroll
            for (int k = 0; k < NB; ++k) {
                f64x4_t p, q;
#pragma unroll
                for (int v = 0; v < 4; ++v) p[v] = x[k][i][64 * v + lane], q[v] = y[k][j][64 * v + lane];
                acc = mfma4(p, q, acc);          // block (k, i)^T = block (i, k)
            }
            return acc;
        };
        auto product = [&](double (*x)[NB][256], double (*y)[NB][256]) { return block(x, y, bi, bj); };
        auto put = [&](double (*x)[NB][256], f64x4_t r) {
#pragma unroll
            for (int v = 0; v < 4; ++v) {
                x[bi][bj][64 * v + lane] = r[v];
                if (LOWER && bi != bj) x[bj][bi][64 * (c >> 2) + 16 * (c & 3) + 4 * v + g] = r[v];
            }
        };
        // LONG: all blocks of Q, which is not symmetric there, by turns of the wavefronts; the
        // last step leaves its transpose, from which X's product reads
        constexpr int QS = LONG ? (NB * NB + NT / 64 - 1) / (NT / 64) : 1;
        f64x4_t own;
#pragma unroll
        for (int v = 0; v < 4; ++v) {
            const int i = 4 * v + g;
            const double* blk = sum + low_block(max(bi, bj), min(bi, bj)) * 256;
            own[v] = (bi >= bj ? blk[i * 16 + c] : blk[c * 16 + i]) * inv * inv;
        }
        if constexpr (LONG) {
            if (bi == bj) own = symmetric(own, shift.of[0]);
        }
        if (works) put(A, own);
        __syncthreads();
        for (int k = 0; k < a.steps; ++k) {
            if (works) {
                const f64x4_t sq = product(A, A);
                f64x4_t r;
#pragma unroll
                for (int v = 0; v < 4; ++v) {
                    const int i = 16 * bi + 4 * v + g;
                    r[v] = (i == 16 * bj + c && i < m ? a.a : 0.) + a.b * own[v] + a.c * sq[v];
                }
                put(P, r);
                if (k == 0) put(Q[0], r);
            }
            __syncthreads();
            f64x4_t qn[QS], un;
            if constexpr (LONG) {
#pragma unroll
                for (int t = 0; t < QS; ++t) {
                    const int id = wave + t * (NT / 64);
                    if (k > 0 && id < NB * NB) qn[t] = block(P, Q[q], id / NB, id % NB);
                }
            } else {
                if (works && k > 0) qn[0] = product(Q[q], P);
            }
            if (works && k + 1 < a.steps) un = product(A, P);
            if (NQ == 1 && k > 0) __syncthreads();       // one Q: all have read it
            if (NQ == 2 && k > 0) q ^= 1;
            if constexpr (LONG) {
#pragma unroll
                for (int t = 0; t < QS; ++t) {
                    const int id = wave + t * (NT / 64);
                    if (k == 0 || id >= NB * NB) continue;
                    const bool last = k + 1 == a.steps;
                    double* to = last ? Q[q][id % NB][id / NB] : Q[q][id / NB][id % NB];
#pragma unroll
                    for (int v = 0; v < 4; ++v) to[last ? 16 * c + 4 * v + g : 64 * v + lane] = qn[t][v];
                }
            } else {
                if (works && k > 0) put(Q[q], qn[0]);
            }
            if (works && k + 1 < a.steps) put(U, un);
            __syncthreads();
            if (k + 1 < a.steps) {
                if (works) {
                    own = product(U, P);
                    if constexpr (LONG) {
                        if (bi == bj) own = symmetric(own, shift.of[k + 1]);
                    }
                    put(A, own);
                }
                __syncthreads();
            }
        }
    }

    // ---- X = Q U / (|U| + eps) for columns lo .. hi - 1, 16 a wavefront at a time
    if (NB > 1 && l0 < hi) load(l0);
    f64x4_t qb[NB > 2 ? 1 : NB][NB];         // held in registers up to two blocks a side
    auto fetch = [&](int i, int j) {
        f64x4_t r;
#pragma unroll
        for (int v = 0; v < 4; ++v) r[v] = Q[q][i][j][64 * v + lane];
        return r;
    };
    if constexpr (NB <= 2) {
#pragma unroll
        for (int i = 0; i < NB; ++i)
#pragma unroll
            for (int j = 0; j < NB; ++j) qb[i][j] = fetch(i, j);
    }
#pragma unroll 1
    for (; l0 < hi; l0 += NT / 4) {
        f64x4_t u[NB];
#pragma unroll
        for (int k = 0; k < NB; ++k)
#pragma unroll
            for (int v = 0; v < 4; ++v) u[k][v] = raw[k][v];
        if (l0 + NT / 4 < hi) load(l0 + NT / 4);
#pragma unroll (NB > 2 ? 1 : NB)
        for (int i = 0; i < NB; ++i) {
            f64x4_t r = {0., 0., 0., 0.};
#pragma unroll
            for (int k = 0; k < NB; ++k) {
                const f64x4_t x = NB > 2 ? fetch(k, i) : qb[NB > 2 ? 0 : k][i];
                r = tall ? mfma4(u[k], x, r) : mfma4(x, u[k], r);
            }
#pragma unroll
            for (int v = 0; v < 4; ++v) {
                // the result's rows are columns of the long side when tall, of the short otherwise
                const int p = 16 * i + (tall ? c : 4 * v + g), l = l0 + (tall ? 4 * v + g : c);
                if (p < m && l < hi)
                    target1(a.t, base + (tall ? (int64_t)l * m + p : (int64_t)p * n + l), (float)(r[v] * inv));
            }
        }
    }
}

// ---------------------------------------------------------------- host side

constexpr size_t kAlign = 256;
constexpr int kMaxSide = 32768;
constexpr int kSyms = 5;      // symmetric matrices of a call: A, A P and three of S and R
size_t align_up(size_t v) { return (v + kAlign - 1) / kAlign * kAlign; }
bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }
int pad64(int v) { return (v + 63) / 64 * 64; }

bool is_small(int B, int M, int N) {
    const int m = M < N ? M : N;
    return (int64_t)B * small_chunks(M, N) <= small_most(m);
}
int small_blocks(int M, int N) {
    const int m = M < N ? M : N;
    return (m + 15) / 16;
}

// 128 x 128 tiles of a matrix's planes.
int64_t tiles128(int M, int N) {
    return (int64_t)((pad64(M) + BT - 1) / BT) * ((pad64(N) + BT - 1) / BT);
}

struct Layout {
    size_t part, lift, x, xt[2], sym[kSyms], total;
};

moe_status check_sizes(int B, int M, int N) {
    if (B < 0 || M <= 0 || N <= 0) return MOE_ERR_INVALID_ARG;
    if (M > kMaxSide || N > kMaxSide || B > 65535) return MOE_ERR_UNSUPPORTED;
    // a grid's threads are fewer than 2^32
    if (!is_small(B, M, N) && B * tiles128(M, N) >= 1 << 24) return MOE_ERR_UNSUPPORTED;
    return MOE_OK;
}

Layout layout_of(int B, int M, int N) {
    Layout L = {};
    if (is_small(B, M, N)) {
        const size_t chunks = small_chunks(M, N), blocks = low_blocks(small_blocks(M, N));
        L.total = chunks > 1 || blocks > 3 ? (size_t)B * chunks * blocks * 256 * sizeof(double) : 0;
        return L;
    }
    const size_t m = pad64(M < N ? M : N), n = pad64(M < N ? N : M);
    size_t off = 0;
    auto take = [&](size_t bytes) {
        const size_t at = off;
        off = align_up(off + bytes);
        return at;
    };
    L.part = take((size_t)B * norm_blocks((int64_t)M * N) * sizeof(double));
    L.lift = take((size_t)B * sizeof(int));
    L.x = take((size_t)B * m * n * 4);
    L.xt[0] = take((size_t)B * m * n * 4);
    L.xt[1] = take((size_t)B * m * n * 4);
    for (size_t& at : L.sym) at = take((size_t)B * m * m * 4);
    L.total = off;
    return L;
}

// Largest |v(x)| over [0, s] for v's values at the ends and at the points given.
struct Bound {
    double best = 0.;
    bool fine = true;
    void at(double v) {
        if (!(fabs(v) <= 1e4)) fine = false;
        if (fabs(v) > best) best = fabs(v);
    }
};
// Bounds of a step that starts with singular values in [0, s]: of S = b A + c A A,
// of P = a I + S, and of the singular values after it.
bool step_bounds(double a, double b, double c, double s, double* mid, double* whole, double* next) {
    Bound p, w, q;
    const double y = s * s;
    auto inside = [&](double t) { return t >= 0. && t <= y; };
    auto both = [&](double t) {
        p.at(b * t + c * t * t);
        w.at(a + b * t + c * t * t);
    };
    both(0.);
    both(y);
    if (c != 0. && inside(-b / (2. * c))) both(-b / (2. * c));
    auto f = [&](double t) { return sqrt(t) * (a + b * t + c * t * t); };
    q.at(f(y));
    if (c != 0.) {
        const double d = 9. * b * b - 20. * a * c;
        if (d >= 0.)
            for (int k = -1; k <= 1; k += 2) {
                const double t = (-3. * b + k * sqrt(d)) / (10. * c);
                if (inside(t)) q.at(f(t));
            }
    } else if (b != 0. && inside(-a / (3. * b))) {
        q.at(f(-a / (3. * b)));
    }
    *mid = p.best * (1. + 1e-3);
    *whole = w.best * (1. + 1e-3);
    *next = q.best * (1. + 1e-3);
    return p.fine && w.fine && q.fine;
}
// The largest power of two that keeps `bound` at 2^15 at most.
double scale_for(double bound) {
    double s = 1.;
    while (s * bound > 32768.) s *= 0.5;
    while (s < 1099511627776. && 2. * s * bound <= 32768.) s *= 2.;
    return s;
}

// The tile a product runs on: the one whose estimate is the least.  The estimates
// are fits (us of one launch; n tiles, k steps of 32; 256 compute units) to 40
// products of 1 to 64 matrices with short sides of 256 to 4096 and k of 8 to 256, each
// timed on every tile.  They are within 15% mostly, and their choice
// is within 6% of the best of them, most often the best:
//  * 32, split over K:  each tile costs by itself, and more where an operand
//    outgrows an XCD's 4 MiB of L2
//  * 64 and 128:        a floor by the waits of a K step while units are idle, then by
//    the tiles; 128-tiles mixed with 64 where at most 64 are over a multiple of 256
//    (336 tiles: 57, mixed 56; 528 tiles: 227, mixed 195)
//  * 256:               by rounds of 256 workgroups, one a unit, and tiles
// Measured on both sides of the borders, 32 / 64 (half steps, whole) / 128 (or mixed) /
// 256: k = 48, one 768 x 1536 matrix's A 10.4 / 14.5, 21.8 / 25.7 / 78 us, two of them 14.2 /
// 14.9, 21.9 / 26.0 / 77, eight 39.9 / 31.6, 31.5 / 32.2 / 78; k = 24, S X of two 24.7 /
// 18.9, 18.5 / 18.9 / 50, of four 44.8 / 30.7, 34.2 / 27.5 / 51, of sixteen 208 / 139, 137 / 108 /
// 131; k = 32, of sixteen 1024 x 4096 matrices - / 622, 584 / 429 / 406.
struct Choice {
    int tile;
    bool halves;     // 64: four half steps; else two whole ones
    int whole;       // 128, mixed: how many of 128
};
Choice choose(int64_t n32, int64_t n64, int64_t n128, int64_t n256, int k, bool outgrown) {
    const int64_t r = (n256 + 255) / 256, over = n128 % 256;
    const bool mixed = n128 > 256 && over > 0 && over <= 64;
    const int64_t n = mixed ? n128 - over : n128;
    const struct {
        Choice c;
        double us;
    } all[] = {
        {{32, false, 0}, 4. + n32 * (0.0022 + (outgrown ? 0.0005 : 0.0003) * k)},
        {{64, true, 0}, 4. + k * fmax(0.22, 0.00096 * n64)},
        {{64, false, 0}, 4. + k * fmax(0.385, n64 <= 1000 ? 0.13 + 0.00072 * n64 : 0.0011 * n64)},
        {{128, true, mixed ? (int)n : 0},
         (mixed ? 12. : 8.) + k * fmax(0.48, (n <= 256 ? 0.0028 : n <= 512 ? 0.0032 : outgrown ? 0.0033 : 0.0031) * n)},
        {{256, false, 0}, 24. * r - 12. + k * (1.1 * r + 0.0048 * n256)},
    };
    int best = 0;
    for (int i = 1; i < 5; ++i)
        if (all[i].us < all[best].us) best = i;
    return all[best].c;
}

template <int MODE>
bool launch_product(MulArgs& g, int B, hipStream_t stream) {
    constexpr bool SYM = MODE == GRAM || MODE == SYMM;
    auto grid = [&](int tile) {
        g.ti = (g.pr + tile - 1) / tile;
        g.tj = (g.qr + tile - 1) / tile;
        return (int64_t)B * (SYM ? (int64_t)g.ti * (g.ti + 1) / 2 : (int64_t)g.ti * g.tj);
    };
    const bool outgrown = (int64_t)g.qr * g.K * 4 > 4 << 20;
    const Choice c = choose(grid(DT), grid(64), grid(128), grid(LT), g.K / KB, outgrown);
    const unsigned n = (unsigned)grid(c.tile);
    if (c.tile == 32)
        ns_product_split_kernel<MODE><<<n, 64 * DW, 0, stream>>>(g);
    else if (c.tile == 64 && c.halves)
        ns_product_kernel<MODE, 1, 1, 4><<<n, 256, 0, stream>>>(g);
    else if (c.tile == 64)
        ns_product_kernel<MODE, 1, 2, 2><<<n, 256, 0, stream>>>(g);
    else if (c.whole) {
        g.whole = c.whole;
        ns_product_mixed_kernel<MODE><<<c.whole + 4 * (n - c.whole), 256, 0, stream>>>(g);
    } else if (c.tile == 128)
        ns_product_kernel<MODE, 2, 1, 4><<<n, 256, 0, stream>>>(g);
    else
        ns_product_large_kernel<MODE><<<n, 512, 0, stream>>>(g);
    return hipGetLastError() == hipSuccess;
}

// Whether a run on the short side is a long one: what A's rounding, 2^-46 of the largest square and
// less, has grown to by the last step's polynomial is beyond 2^-24.
bool is_long(int steps, const double* whole) {
    double grown = 0x1p-46;
    for (int k = 0; k + 1 < steps; ++k) grown *= fmax(1., whole[k] * whole[k]);
    return grown > 0x1p-24;
}

moe_status run(const Source& src, const Target& tgt, int B, int M, int N, int steps, double a, double b,
               double c, double eps, void* workspace, size_t ws_bytes, hipStream_t stream) {
    if (steps < 1 || steps > kMaxSteps) return MOE_ERR_INVALID_ARG;
    if (!(eps >= 0.) || !isfinite(eps) || !isfinite(a) || !isfinite(b) || !isfinite(c))
        return MOE_ERR_INVALID_ARG;
    double mid[kMaxSteps], whole[kMaxSteps], top[kMaxSteps + 1], grown = 1.;
    int room[kMaxSteps + 1] = {};
    top[0] = 1.;
    for (int k = 0; k < steps; ++k) {
        if (!step_bounds(a, b, c, top[k], &mid[k], &whole[k], &top[k + 1])) return MOE_ERR_UNSUPPORTED;
        // what shrinks this far leaves fp16's range at the largest scale (all
        // zero coefficients are exact)
        if (top[k] != 0. && top[k] < 1e-9) return MOE_ERR_UNSUPPORTED;
        if (whole[k] != 0. && whole[k] < (1. + fabs(b) + fabs(c)) * 1e-12) return MOE_ERR_UNSUPPORTED;
        // top is at most what the polynomials' product lets 1 grow to; all is zero with whole
        grown *= whole[k];
        if (grown > 0.) room[k + 1] = ilogb(top[k + 1] / grown);
    }
    if (B == 0) return MOE_OK;
    (void)hipGetLastError();
    auto ok = [] { return hipGetLastError() == hipSuccess; };
    const Layout L = layout_of(B, M, N);
    if (L.total) {
        if (!workspace || !aligned(workspace, kAlign)) return MOE_ERR_INVALID_ARG;
        if (ws_bytes < L.total) return MOE_ERR_WORKSPACE;
    }
    if (is_small(B, M, N)) {
        const int chunks = small_chunks(M, N);
        const SmallArgs s = {src, tgt, M, N, steps, small_chunk(M, N), a, b, c, eps, (double*)workspace};
        const dim3 grid(chunks, B);
        auto launch = [&](auto blocks, auto long_run) {
            constexpr int NB = decltype(blocks)::value;
            constexpr bool LONG = decltype(long_run)::value;
            Shifts<LONG> shift;
            if constexpr (LONG) {
                for (int k = 0; k < kMaxSteps; ++k) shift.of[k] = k < steps ? 0x1p-46 * top[k] * top[k] : 0.;
            }
            if constexpr (NB <= 2) {
                if (chunks == 1) {
                    ns_small_kernel<NB, true, LONG><<<grid, kOneThreads, 0, stream>>>(s, shift);
                    return ok();
                }
            }
            ns_small_gram_kernel<NB><<<grid, gram_threads(NB), 0, stream>>>(s);
            if (!ok()) return false;
            ns_small_kernel<NB, false, LONG><<<grid, step_threads(NB, false), 0, stream>>>(s, shift);
            return ok();
        };
        auto of_blocks = [&](auto long_run) {
            const int blocks = small_blocks(M, N);
            return blocks == 1   ? launch(std::integral_constant<int, 1>{}, long_run)
                   : blocks == 2 ? launch(std::integral_constant<int, 2>{}, long_run)
                   : blocks == 3 ? launch(std::integral_constant<int, 3>{}, long_run)
                                 : launch(std::integral_constant<int, 4>{}, long_run);
        };
        const bool done = is_long(steps, whole) ? of_blocks(std::true_type{}) : of_blocks(std::false_type{});
        return done ? MOE_OK : MOE_ERR_HIP;
    }
    char* ws = (char*)workspace;
    const bool tall = M > N;
    const int m = pad64(tall ? N : M), n = pad64(tall ? M : N);
    // Steps in groups trade 3 m^2 n products of a step for up to 4 m^3, and lose
    // precision: A's rounding grows by P^2 in each step that A takes by itself, where that of a
    // new X X^T does not.  Five steps against 64 bits, in errors of the same iteration in fp32:
    // eight 768 x 1536 1.9 (one by one 0.8), four 1024 x 4096 1.6 (0.75), sixteen 256 x 512 2.1 (0.9),
    // 40 of 200 x 500 with strong directions 2.9 (0.8), 5e-6 to 7e-6 of |X|; the most 5.9, for three
    // steps of 128 of 70 x 200.  So they are not for fp32 results, but for those that
    // are rounded to bf16 (2^-8) or added to weights, W - rate X: at a rate of 0.02 that is 1e-7 of X, the
    // half step of an fp32 weight of X's size.  They pay from long sides of 1.5 times the short on and
    // enough tiles to share out: eight 768 x 1024 417 us one by one, 419 in groups, 768 x 1152 439,
    // 432, 768 x 1536 537, 478; sixteen 1024 x 4096 3559, 2321; one 768 x 1536 (72
    // tiles) 163, 167, two 231, 219.
    const bool grouped = (tgt.muon || tgt.out_bf16) && 2 * n >= 3 * m && B * tiles128(M, N) >= 128;
    const int nb = norm_blocks((int64_t)M * N);
    ns_norm_kernel<<<dim3(nb, B), 256, 0, stream>>>(src, (int64_t)M * N, (double*)(ws + L.part));
    if (!ok()) return MOE_ERR_HIP;

    char* x = ws + L.x;
    char* xt[2] = {ws + L.xt[0], ws + L.xt[1]};
    double sx = scale_for(top[0]);
    const int Mp = pad64(M), Np = pad64(N);
    int* lift = (int*)(ws + L.lift);
    const SplitArgs sp = {src, (const double*)(ws + L.part), nb, M, N, Mp, Np, eps, (float)sx, lift,
                          tall ? xt[0] : x, tall ? x : xt[0]};
    ns_split_kernel<<<dim3(Np / ST, Mp / ST, B), 256, 0, stream>>>(sp);
    if (!ok()) return MOE_ERR_HIP;

    // ---- the steps, in groups of one, two or three.  A group takes X's Gram
    // matrix A once and X once more in its end; between them
    //   S_j = b A_j + c A_j A_j,  P_j = a I + S_j,
    //   A_{j+1} = P_j A_j P_j = a U + U S_j with U = a A_j + A_j S_j,
    //   P_0 .. P_j = alpha I + R_j,  R_j = a R_{j-1} + alpha' S_j + R_{j-1} S_j,
    // all on the short side, where a I stays out of the stored planes.
    struct Plane {
        char* p;
        double scale;
    };
    const int64_t xs = (int64_t)m * n * 4, as = (int64_t)m * m * 4;
    MulArgs y = {};      // a product on the short side
    y.p_stride = y.q_stride = y.add_stride = y.c_stride = as;
    y.pr = y.qr = y.K = m;
    y.lift = lift;
    auto symm = [&](Plane P, Plane Q, double f, double fp, double fq, Plane out) {
        MulArgs g = y;
        g.p = g.add = P.p;
        g.q = Q.p;
        g.f = (float)(f / (P.scale * Q.scale));
        g.fa = (float)(fp / P.scale);
        g.fq = (float)(fq / Q.scale);
        g.so = (float)out.scale;
        g.c = g.ct = out.p;
        return launch_product<SYMM>(g, B, stream);
    };
    int turn = 0;
    for (int k = 0; k < steps;) {
        int group = grouped ? ((steps - k) % 2 && steps - k > 1 ? 3 : (steps - k > 1 ? 2 : 1)) : 1;
        // alpha and R cancel where the steps bring a singular value near 1: what
        // their 22 bits leave there is 2^-22 of the largest product of the P_j,
        // which stays at 2^-16 (three steps of the usual coefficients: 41)
        double product = 1.;
        for (int j = 0; j < group; ++j) {
            product *= whole[k + j];
            if (product > 64.) group = j > 0 ? j : 1;
        }
        Plane A = {ws + L.sym[0], scale_for(top[k] * top[k])}, U = {ws + L.sym[1], 0.};
        // where S and R are by turns: an S may be the R of the next step
        Plane S = {}, R = {};
        int free_at = 0;
        auto fresh = [&](double scale) {
            for (;; free_at = (free_at + 1) % 3) {
                char* p = ws + L.sym[2 + free_at];
                if (p != S.p && p != R.p) return Plane{p, scale};
            }
        };
        MulArgs g = y;
        g.p = g.q = x;
        g.p_stride = g.q_stride = xs;
        g.K = n;
        g.room = room[k];
        g.f = (float)(1. / (sx * sx));
        g.so = (float)A.scale;
        g.c = g.ct = A.p;
        if (!launch_product<GRAM>(g, B, stream)) return MOE_ERR_HIP;
        double alpha = 1., bound = 1.;
        for (int j = 0; j < group; ++j) {
            const int at = k + j;
            S = Plane{};
            S = fresh(scale_for(mid[at]));
            if (!symm(A, A, c, b, 0., S)) return MOE_ERR_HIP;
            bound *= whole[at];
            if (j == 0) {
                R = S;
            } else {
                const Plane next = fresh(scale_for(bound + fabs(alpha * a)));
                if (!symm(R, S, 1., a, alpha, next)) return MOE_ERR_HIP;
                R = next;
            }
            alpha *= a;
            if (j + 1 < group) {
                U.scale = scale_for(top[at] * top[at + 1]);
                const Plane next = {A.p, scale_for(top[at + 1] * top[at + 1])};
                if (!symm(A, S, 1., a, 0., U) || !symm(U, S, 1., a, 0., next)) return MOE_ERR_HIP;
                A = next;
            }
        }
        MulArgs z = y;
        z.room = room[k];
        k += group;
        z.room_after = room[k];
        z.p = R.p;
        z.q = xt[turn];
        z.q_stride = z.add_stride = z.c_stride = xs;
        z.qr = n;
        z.add = x;
        z.f = (float)(1. / (R.scale * sx));
        z.fa = (float)(alpha / sx);
        if (k < steps) {
            sx = scale_for(top[k]);
            turn ^= 1;
            z.so = (float)sx;
            z.c = x;
            z.ct = xt[turn];
            if (!launch_product<APPLY>(z, B, stream)) return MOE_ERR_HIP;
        } else {
            z.swap = tall;
            z.M = M;
            z.N = N;
            z.t = tgt;
            if (!launch_product<FINAL>(z, B, stream)) return MOE_ERR_HIP;
        }
    }
    return MOE_OK;
}

}  // namespace
}  // namespace moe

extern "C" {

size_t moe_newton_schulz_workspace_size(int B, int M, int N) {
    if (moe::check_sizes(B, M, N) != MOE_OK) return 0;
    return moe::layout_of(B, M, N).total;
}

moe_status moe_newton_schulz(const void* G, void* out, int B, int M, int N, int steps, double a, double b,
                             double c, double eps, moe_dtype dtype, void* workspace, size_t ws_bytes,
                             hipStream_t stream) {
    const moe_status st = moe::check_sizes(B, M, N);
    if (st != MOE_OK) return st;
    if (dtype != MOE_F32 && dtype != MOE_BF16) return MOE_ERR_INVALID_ARG;
    if (B > 0 && (!G || !out)) return MOE_ERR_INVALID_ARG;
    if (!moe::aligned(G, 16) || !moe::aligned(out, 16)) return MOE_ERR_INVALID_ARG;
    const int bf16 = dtype == MOE_BF16;
    const moe::Source src = {G, nullptr, 0.f, 0, bf16};
    const moe::Target tgt = {out, nullptr, 0.f, 0.f, 0, bf16};
    return moe::run(src, tgt, B, M, N, steps, a, b, c, eps, workspace, ws_bytes, stream);
}

moe_status moe_muon_step(void* W, void* W_bf16, const float* dW, float* momentum, int B, int M, int N,
                         float lr, float beta, float weight_decay, float scale, int nesterov, int steps,
                         double a, double b, double c, double eps, moe_dtype dtype, void* workspace,
                         size_t ws_bytes, hipStream_t stream) {
    const moe_status st = moe::check_sizes(B, M, N);
    if (st != MOE_OK) return st;
    if (dtype != MOE_F32 && dtype != MOE_BF16) return MOE_ERR_INVALID_ARG;
    if (W_bf16 && dtype != MOE_F32) return MOE_ERR_INVALID_ARG;
    if (!isfinite(lr) || !isfinite(beta) || !isfinite(weight_decay) || !isfinite(scale))
        return MOE_ERR_INVALID_ARG;
    if (B > 0 && (!W || !dW || !momentum)) return MOE_ERR_INVALID_ARG;
    const void* ptrs[] = {W, W_bf16, dW, momentum};
    for (const void* p : ptrs)
        if (!moe::aligned(p, 16)) return MOE_ERR_INVALID_ARG;
    const moe::Source src = {dW, momentum, beta, nesterov ? 1 : 0, 0};
    const moe::Target tgt = {W, (uint16_t*)W_bf16, (float)(1. - (double)lr * weight_decay),
                             (float)((double)lr * scale), 1, dtype == MOE_BF16};
    return moe::run(src, tgt, B, M, N, steps, a, b, c, eps, workspace, ws_bytes, stream);
}

}  // extern "C"
