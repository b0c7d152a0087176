// vocab_few.hip -- the products of the losses over a vocabulary for few rows
// (a decoding step's tokens, small chunks), where reading the table is all
// the work:
//
//  logits:  z = h W^T for 128 entries (of small tables 32, K divided over the
//           wavefronts) and 32 or 64 rows a workgroup, and from it the tile's
//           largest value and sum, or dz (as in vocab_gemm.hip)
//  dh:      dz W for 256 columns and a part of the entries a workgroup, and the
//           sum of the parts
//  dW:      dz^T h, 64 entries x 256 columns a workgroup: a few steps of K, then
//           the store, which is all of the time; several workgroups a CU
//
// dz of bf16 operands is two planes of bf16, 16 bits together: there are matrix
// instructions to spare, and so the gradients' own rounding is the only one
// that counts.
//
// The table is read once, in its own type: bf16 on the bf16 matrix
// instructions, fp32 on the fp32 ones (a sixteenth of the rate, which 64 rows
// still do not need), with no copy in planes.  Four wavefronts, each with its
// own 32 entries (64 columns), a ring of 16 KiB stages of the table and the few
// rows beside it, filled by 16-byte DMA; two workgroups a CU keep 64 to 96 KiB a CU
// on their way.
#include "mfma_common.h"
#include "vocab_internal.h"

#include <algorithm>

namespace moe {
namespace {

using namespace mfma;

constexpr int FN = kVocabFewCols;     // 128 entries of a logits tile
constexpr int N_BYTES = 16384;        // of a stage, either product

// What a row's bytes past its end are read as.
__device__ __attribute__((aligned(16))) u32x4_t few_zeros[1];

template <bool F32>
struct Elem {
    typedef uint16_t type;
};
template <>
struct Elem<true> {
    typedef float type;
};

// acc += the 32 x 32 product of 16 bytes a lane of each operand: lane l holds
// row l % 32 and, of 8 (fp32) or 16 (bf16) k, those of its half.
template <bool F32>
__device__ __forceinline__ f32x16_t multiply(u32x4_t n, u32x4_t m, f32x16_t acc) {
    if constexpr (F32) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            acc = __builtin_amdgcn_mfma_f32_32x32x2f32(__uint_as_float(n[i]), __uint_as_float(m[i]), acc, 0, 0, 0);
        return acc;
    } else {
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8_t, n), __builtin_bit_cast(bf16x8_t, m),
                                                       acc, 0, 0, 0);
    }
}

// Steps of a ring of NS stages: before step s its stage has landed, and the stage
// NS - 1 on is issued into the buffer that step s - 1 read.  PER: a wavefront's
// loads a stage.  `issue(s, buffer)` may be asked for stages past the last.
template <int NS, int PER, typename I, typename W>
__device__ __forceinline__ void ring(int steps, char* const (&st)[NS], I&& issue, W&& work) {
    if (steps <= 0) return;
#pragma unroll
    for (int u = 0; u + 1 < NS; ++u) issue(u, st[u]);
    for (int s = 0; s < steps; s += NS) {
#pragma unroll
        for (int u = 0; u < NS; ++u) {
            if (s + u >= steps) break;
            __builtin_amdgcn_s_waitcnt(waitcnt_imm((NS - 2) * PER, 0));
            __builtin_amdgcn_s_barrier();
            __builtin_amdgcn_sched_barrier(0);
            issue(s + u + NS - 1, st[(u + NS - 1) % NS]);
            work(st[u]);
            __builtin_amdgcn_sched_barrier(0);
        }
    }
    __builtin_amdgcn_s_waitcnt(waitcnt_imm(0, 0));
    __syncthreads();
}

// dz of a lane's 16 entries from their logits z(v) in 64 bits, `at` of them (or none)
// the target; those from `left` on are past the table.  fp32: at the target e^d - 1
// by itself, without the rounding of an e^d near 1.
template <bool F32, typename Z>
__device__ __forceinline__ void few_dz(float (&x)[16], Z&& z, float scale, float lse, float g, int at, int left) {
    float dt = 0.f;
#pragma unroll
    for (int v = 0; v < 16; ++v) {
        const int e = 8 * (v / 4) + v % 4;
        const float d = (float)fma(z(v), (double)scale, -(double)lse);
        float p = F32 ? exp_fp32(d) : __builtin_amdgcn_exp2f(d * 1.4426950408889634f);
        if (at == e) {
            dt = d;
            p -= 1.f;
        }
        // a row that does not count has an infinite lse: zeros, whatever h holds
        x[v] = e >= left || lse == INFINITY ? 0.f : p * g;
    }
    if constexpr (F32) {
        if (__ballot(at >= 0)) {
            const float p = expm1f(dt) * g;
#pragma unroll
            for (int v = 0; v < 16; ++v)
                if (at == 8 * (v / 4) + v % 4 && lse != INFINITY) x[v] = p;
        }
    }
}

// RB: blocks of 32 rows.
template <bool F32, int RB, bool DZ>
__global__ __launch_bounds__(256, 2) void vocab_few_logits_kernel(const VocabFew a, int m_tiles) {
    using E = typename Elem<F32>::type;
    constexpr int NS = RB == 1 ? 4 : 3, PER = 4 + RB, SB = N_BYTES + RB * 4096;
    __shared__ __attribute__((aligned(1024))) char st0[SB];
    __shared__ __attribute__((aligned(1024))) char st1[SB];
    __shared__ __attribute__((aligned(1024))) char st2[SB];
    __shared__ __attribute__((aligned(1024))) char st3[NS == 4 ? SB : 16];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    // row tiles of the same entries next to each other
    const int64_t row0 = (int64_t)(blockIdx.x % m_tiles) * (32 * RB), v0 = (int64_t)(blockIdx.x / m_tiles) * FN;
    const int64_t bytes = a.D * (int64_t)sizeof(E);          // of a row, a multiple of 16
    const int steps = (int)((bytes + 127) / 128);

    // DMA instruction: 8 rows of 128 bytes; lane -> row lane / 8, physical
    // chunk lane % 8 holding logical chunk (lane % 8) ^ swz8(row)
    const char* n_src[4];
    const char* m_src[RB];
    int n_c[4], m_c[RB];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int r = 32 * wave + 8 * j + (lane >> 3);
        n_c[j] = 16 * ((lane & 7) ^ swz8(r));
        n_src[j] = (const char*)a.W + min(v0 + r, (int64_t)a.V - 1) * bytes + n_c[j];
    }
#pragma unroll
    for (int j = 0; j < RB; ++j) {
        const int r = 8 * (RB * wave + j) + (lane >> 3);
        m_c[j] = 16 * ((lane & 7) ^ swz8(r));
        m_src[j] = (const char*)a.h + min(row0 + r, a.T - 1) * a.h_pitch * (int64_t)sizeof(E) + m_c[j];
    }
    // each tile begins elsewhere in K where rows are whole 2 KiB apart and the table's
    // bytes are all there is to wait for: else all tiles read from the same few of the
    // memory's channels (one row, fp32 32768 x 4096 145 -> 107 us, 131072 x 1024 128 ->
    // 108, bf16 131072 x 4096 216 -> 177; 64 rows lose 5%)
    const int turn = RB == 1 && bytes % 2048 == 0 ? blockIdx.x / m_tiles % steps : 0;
    auto issue = [&](int s, char* st) {
        int at = min(s, steps - 1);
        if (RB == 1) at = at + turn < steps ? at + turn : at + turn - steps;
        const int64_t k = (int64_t)at * 128;
#pragma unroll
        for (int j = 0; j < 4; ++j)
            load_lds16(k + n_c[j] < bytes ? n_src[j] + k : (const char*)few_zeros, st + (4 * wave + j) * 1024);
#pragma unroll
        for (int j = 0; j < RB; ++j)
            load_lds16(k + m_c[j] < bytes ? m_src[j] + k : (const char*)few_zeros, st + N_BYTES + (RB * wave + j) * 1024);
    };
    const int l = lane & 31, half = lane >> 5;
    // D / 2 (bf16: D / 16) terms follow one another in a sum, so there are several sums
    // (one of them was off by twice what a library's product is), joined in 64 bits:
    // a row's entry at its target is a small difference of large ones
    constexpr int CH = F32 && RB == 1 ? 8 : 4;
    f32x16_t sum[CH][RB];
#pragma unroll
    for (int q = 0; q < CH; ++q)
#pragma unroll
        for (int rb = 0; rb < RB; ++rb) sum[q][rb] = f32x16_t{};
    auto work = [&](const char* st) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const u32x4_t n = *(const u32x4_t*)(st + (32 * wave + l) * 128 + (((2 * i + half) ^ swz8(32 * wave + l)) << 4));
#pragma unroll
            for (int rb = 0; rb < RB; ++rb) {
                const u32x4_t m = *(const u32x4_t*)(st + N_BYTES + (32 * rb + l) * 128 + (((2 * i + half) ^ swz8(32 * rb + l)) << 4));
                if constexpr (F32) {
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        sum[(4 * i + q) % CH][rb] = __builtin_amdgcn_mfma_f32_32x32x2f32(
                            __uint_as_float(n[q]), __uint_as_float(m[q]), sum[(4 * i + q) % CH][rb], 0, 0, 0);
                } else {
                    sum[i][rb] = multiply<false>(n, m, sum[i][rb]);
                }
            }
        }
    };
    if constexpr (NS == 4) {
        char* const st[4] = {st0, st1, st2, st3};
        ring<4, PER>(steps, st, issue, work);
    } else {
        char* const st[3] = {st0, st1, st2};
        ring<3, PER>(steps, st, issue, work);
    }

    f32x16_t (&acc)[RB] = sum[0];
    auto joined = [&](int rb, int v) {
        double z = 0;
#pragma unroll
        for (int q = 0; q < CH; ++q) z += sum[q][rb][v];
        return z;
    };
    if constexpr (!DZ) {
#pragma unroll
        for (int rb = 0; rb < RB; ++rb)
#pragma unroll
            for (int v = 0; v < 16; ++v) acc[rb][v] = (float)joined(rb, v);
    }

    // element v of acc on lane l: row l % 32, entry v0 + 32 w + 8 (v / 4) + 4 (l / 32) + v % 4
    const int64_t c0 = v0 + 32 * wave + 4 * half;
    const int left = (int)min((int64_t)a.V - c0, (int64_t)32);
    float2* sums = (float2*)st0;                              // [4][32 RB]
#pragma unroll
    for (int rb = 0; rb < RB; ++rb) {
        const int64_t row = row0 + 32 * rb + l;
        const bool there = row < a.T;
        const int64_t target = there && a.target ? a.target[row] - a.v0 : -1;
        const int at = target >= c0 && target < c0 + 32 && target < a.V ? (int)(target - c0) : -1;
        if constexpr (!DZ) {
            if (__ballot(at >= 0)) {
#pragma unroll
                for (int v = 0; v < 16; ++v)
                    if (at == 8 * (v / 4) + v % 4) a.zt[row] = acc[rb][v];
            }
            float top = -INFINITY;
#pragma unroll
            for (int v = 0; v < 16; ++v) {
                if (8 * (v / 4) + v % 4 >= left) acc[rb][v] = -INFINITY;
                top = fmaxf(top, acc[rb][v]);
            }
            top = fmaxf(top, __shfl_xor(top, 32)) * a.scale;
            const float off = top == -INFINITY ? 0.f : top;
            float sum = 0.f;
#pragma unroll
            for (int v = 0; v < 16; ++v) sum += __builtin_amdgcn_exp2f(fmaf(acc[rb][v], a.scale, -off));
            sum += __shfl_xor(sum, 32);
            if (half == 0) sums[wave * 32 * RB + 32 * rb + l] = make_float2(top, sum);
        } else {
            // Through LDS, so that rows go out in whole lines: 32 of 128 entries in fp32,
            // 16-byte chunks XOR-swizzled by the row.
            const float lse = there ? a.lse[row] : INFINITY, g = there ? a.g[row] : 0.f;
            if (rb) __syncthreads();
            float x[16];
            few_dz<F32>(x, [&](int v) { return joined(rb, v); }, a.scale, lse, g, at, left);
#pragma unroll
            for (int vg = 0; vg < 4; ++vg)
                *(float4*)(st0 + l * 512 + (((8 * wave + 2 * vg + half) ^ l) << 4)) =
                    make_float4(x[4 * vg], x[4 * vg + 1], x[4 * vg + 2], x[4 * vg + 3]);
            __syncthreads();
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int r = 8 * i + (tid >> 5);
                const int64_t m = row0 + 32 * rb + r;
                if (m >= a.T) break;
                float4 x = *(const float4*)(st0 + r * 512 + (((tid & 31) ^ r) << 4));
                const int64_t to = m * a.dz_pitch + v0 + 4 * (tid & 31);
                if constexpr (F32) {
                    *(float4*)(a.dz32 + to) = x;
                    if (!a.dz) continue;
                }
#pragma unroll
                for (int pl = 0; pl < (F32 ? 3 : 2); ++pl) {
                    const uint32_t lo = pack_bf16(x.x, x.y), hi = pack_bf16(x.z, x.w);
                    *(uint2*)(a.dz + pl * a.dz_plane + to) = make_uint2(lo, hi);
                    x.x -= __uint_as_float(lo << 16);
                    x.y -= __uint_as_float(lo & 0xffff0000u);
                    x.z -= __uint_as_float(hi << 16);
                    x.w -= __uint_as_float(hi & 0xffff0000u);
                }
            }
        }
    }
    if constexpr (!DZ) {
        __syncthreads();
        if (tid < 32 * RB && row0 + tid < a.T) {
            float top = -INFINITY, sum = 0.f;
            float2 p[4];
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                p[w] = sums[w * 32 * RB + tid];
                top = fmaxf(top, p[w].x);
            }
            const float off = top == -INFINITY ? 0.f : top;
#pragma unroll
            for (int w = 0; w < 4; ++w) sum += p[w].y * __builtin_amdgcn_exp2f(p[w].x - off);
            a.part[v0 / FN * a.part_pitch + row0 + tid] = make_float2(top, sum);
        }
    }
}

// The same for 32 entries a workgroup, its wavefronts each with a quarter of K: where
// there are few tiles of 128 entries, a tile's steps are all of the time (four rows of
// 2000 x 768 fp32 20 -> 9 us, 40 rows of 8000 x 1536 68 -> 25, bf16 16 -> 9).
template <bool F32, int RB, bool DZ>
__global__ __launch_bounds__(256, 2) void vocab_few_split_kernel(const VocabFew a, int m_tiles) {
    using E = typename Elem<F32>::type;
    constexpr int NS = RB == 1 ? 4 : 3, PER = 2 + 2 * RB, NB = 8192, SB = NB + RB * 8192;
    __shared__ __attribute__((aligned(1024))) char st0[SB];
    __shared__ __attribute__((aligned(1024))) char st1[SB];
    __shared__ __attribute__((aligned(1024))) char st2[SB];
    __shared__ __attribute__((aligned(1024))) char st3[NS == 4 ? SB : 16];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int64_t row0 = (int64_t)(blockIdx.x % m_tiles) * (32 * RB), v0 = (int64_t)(blockIdx.x / m_tiles) * 32;
    const int64_t bytes = a.D * (int64_t)sizeof(E);          // of a row, a multiple of 16
    const int steps = (int)((bytes + 255) / 256);

    // DMA instruction: 4 rows of 256 bytes; lane -> row lane / 16, physical chunk
    // lane % 16 holding logical chunk (lane % 16) ^ (row % 16)
    const char* n_src[2];
    const char* m_src[2 * RB];
    int n_c[2], m_c[2 * RB];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const int r = 8 * wave + 4 * j + (lane >> 4);
        n_c[j] = 16 * ((lane & 15) ^ (r & 15));
        n_src[j] = (const char*)a.W + min(v0 + r, (int64_t)a.V - 1) * bytes + n_c[j];
    }
#pragma unroll
    for (int j = 0; j < 2 * RB; ++j) {
        const int r = 8 * RB * wave + 4 * j + (lane >> 4);
        m_c[j] = 16 * ((lane & 15) ^ (r & 15));
        m_src[j] = (const char*)a.h + min(row0 + r, a.T - 1) * a.h_pitch * (int64_t)sizeof(E) + m_c[j];
    }
    auto issue = [&](int s, char* st) {
        const int64_t k = (int64_t)min(s, steps - 1) * 256;
#pragma unroll
        for (int j = 0; j < 2; ++j)
            load_lds16(k + n_c[j] < bytes ? n_src[j] + k : (const char*)few_zeros, st + (2 * wave + j) * 1024);
#pragma unroll
        for (int j = 0; j < 2 * RB; ++j)
            load_lds16(k + m_c[j] < bytes ? m_src[j] + k : (const char*)few_zeros, st + NB + (2 * RB * wave + j) * 1024);
    };
    const int l = lane & 31, half = lane >> 5;
    constexpr int CH = 2;                // sums of a wavefront, as above
    f32x16_t sum[CH][RB];
#pragma unroll
    for (int q = 0; q < CH; ++q)
#pragma unroll
        for (int rb = 0; rb < RB; ++rb) sum[q][rb] = f32x16_t{};
    auto work = [&](const char* st) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int c = ((4 * wave + 2 * i + half) ^ (l & 15)) << 4;
            const u32x4_t n = *(const u32x4_t*)(st + l * 256 + c);
#pragma unroll
            for (int rb = 0; rb < RB; ++rb) {
                const u32x4_t m = *(const u32x4_t*)(st + NB + (32 * rb + l) * 256 + c);
                if constexpr (F32) {
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        sum[q % CH][rb] = __builtin_amdgcn_mfma_f32_32x32x2f32(
                            __uint_as_float(n[q]), __uint_as_float(m[q]), sum[q % CH][rb], 0, 0, 0);
                } else {
                    sum[i][rb] = multiply<false>(n, m, sum[i][rb]);
                }
            }
        }
    };
    if constexpr (NS == 4) {
        char* const st[4] = {st0, st1, st2, st3};
        ring<4, PER>(steps, st, issue, work);
    } else {
        char* const st[3] = {st0, st1, st2};
        ring<3, PER>(steps, st, issue, work);
    }

    // a block of rows a wavefront from here on
    auto part = [&](int w) { return (float*)(w < 2 ? st0 : st1) + (w & 1) * RB * 1024; };
#pragma unroll
    for (int rb = 0; rb < RB; ++rb)
#pragma unroll
        for (int v = 0; v < 16; ++v) {
            part(wave)[(16 * rb + v) * 64 + lane] = sum[0][rb][v] + sum[1][rb][v];
        }
    __syncthreads();
    if (wave >= RB) return;
    auto joined = [&](int v) {
        double z = 0;
#pragma unroll
        for (int w = 0; w < 4; ++w) z += part(w)[(16 * wave + v) * 64 + lane];
        return z;
    };
    // element v on lane l: row l % 32, entry v0 + 8 (v / 4) + 4 (l / 32) + v % 4
    const int64_t c0 = v0 + 4 * half, row = row0 + 32 * wave + l;
    const int left = (int)min((int64_t)a.V - c0, (int64_t)32);
    const bool there = row < a.T;
    const int64_t target = there && a.target ? a.target[row] - a.v0 : -1;
    const int at = target >= c0 && target < c0 + 32 && target < a.V ? (int)(target - c0) : -1;
    if constexpr (!DZ) {
        float z[16], top = -INFINITY;
#pragma unroll
        for (int v = 0; v < 16; ++v) {
            z[v] = (float)joined(v);
            if (at == 8 * (v / 4) + v % 4) a.zt[row] = z[v];
            if (8 * (v / 4) + v % 4 >= left) z[v] = -INFINITY;
            top = fmaxf(top, z[v]);
        }
        top = fmaxf(top, __shfl_xor(top, 32)) * a.scale;
        const float off = top == -INFINITY ? 0.f : top;
        float s = 0.f;
#pragma unroll
        for (int v = 0; v < 16; ++v) s += __builtin_amdgcn_exp2f(fmaf(z[v], a.scale, -off));
        s += __shfl_xor(s, 32);
        if (half == 0 && there) a.part[v0 / 32 * a.part_pitch + row] = make_float2(top, s);
    } else {
        const float lse = there ? a.lse[row] : INFINITY, g = there ? a.g[row] : 0.f;
        char* own = st2 + 4096 * wave;
        float x[16];
        few_dz<F32>(x, joined, a.scale, lse, g, at, left);
#pragma unroll
        for (int vg = 0; vg < 4; ++vg)
            *(float4*)(own + l * 128 + (((2 * vg + half) ^ (l & 7)) << 4)) =
                make_float4(x[4 * vg], x[4 * vg + 1], x[4 * vg + 2], x[4 * vg + 3]);
        wave_sync();
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = 8 * i + (lane >> 3);
            const int64_t m = row0 + 32 * wave + r;
            if (m >= a.T) break;
            float4 x = *(const float4*)(own + r * 128 + (((lane & 7) ^ (r & 7)) << 4));
            const int64_t to = m * a.dz_pitch + v0 + 4 * (lane & 7);
            if constexpr (F32) {
                *(float4*)(a.dz32 + to) = x;
                if (!a.dz) continue;
            }
#pragma unroll
            for (int pl = 0; pl < (F32 ? 3 : 2); ++pl) {
                const uint32_t lo = pack_bf16(x.x, x.y), hi = pack_bf16(x.z, x.w);
                *(uint2*)(a.dz + pl * a.dz_plane + to) = make_uint2(lo, hi);
                x.x -= __uint_as_float(lo << 16);
                x.y -= __uint_as_float(lo & 0xffff0000u);
                x.z -= __uint_as_float(hi << 16);
                x.w -= __uint_as_float(hi & 0xffff0000u);
            }
        }
    }
}

// dh's parts: columns 256 of a tile, K: entries, 32 (bf16) or 16 (fp32) a step.
template <bool F32, int RB>
__global__ __launch_bounds__(256, 2) void vocab_few_dh_kernel(const VocabFew a, int n_tiles, int m_tiles, int splits) {
    using E = typename Elem<F32>::type;
    constexpr int KS = F32 ? 16 : 32, RPI = F32 ? 1 : 2;       // k rows of a DMA instruction
    // dz: 16 rows of 64 bytes an instruction, of fp32 or of two planes of bf16
    constexpr int PLANES = F32 ? 1 : 2, MI = 2 * RB * PLANES, MJ = MI / 4 ? MI / 4 : 1;
    constexpr int NS = RB == 1 ? 4 : 3, PER = 4 + MJ;
    constexpr int ROW = 256 * sizeof(E), SB = N_BYTES + MI * 1024;
    __shared__ __attribute__((aligned(1024))) char st0[SB];
    __shared__ __attribute__((aligned(1024))) char st1[SB];
    __shared__ __attribute__((aligned(1024))) char st2[SB];
    __shared__ __attribute__((aligned(1024))) char st3[NS == 4 ? SB : 16];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int mt = blockIdx.x % m_tiles, rest = blockIdx.x / m_tiles;
    const int nt = rest % n_tiles, split = rest / n_tiles;
    const int64_t row0 = (int64_t)mt * (32 * RB);
    const int all = (a.V + KS - 1) / KS, per = (all + splits - 1) / splits;
    const int first = min(split * per, all), steps = min(per, all - first);

    // the table: instruction j of wavefront w fills k rows RPI (4 w + j)..; 16-byte
    // chunks swizzled so that neither the transposing reads (bf16) nor lanes l and
    // l + 32, four k rows apart (fp32), meet in a bank
    auto swz = [](int k) { return F32 ? 8 * ((k >> 2) & 1) : swz_tr(k); };
    constexpr int CPR = ROW / 16;                            // chunks of a k row: 64 or 32
    int n_k[4];
    int64_t n_c[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        n_k[j] = RPI * (4 * wave + j) + lane / CPR;
        const int c = nt * 256 + ((lane % CPR) ^ swz(n_k[j])) * (16 / (int)sizeof(E));
        n_c[j] = c < a.D ? c : 0;                            // a column that exists; its sums are not stored
    }
    // instruction m of a stage: plane m / (2 RB), rows 16 (m % (2 RB)).. (fp32 with one
    // block of rows has two for four wavefronts: twice over)
    const char* m_src[MJ];
#pragma unroll
    for (int j = 0; j < MJ; ++j) {
        const int m = (MJ * wave + j) % MI, r = 16 * (m % (2 * RB)) + (lane >> 2);
        const int c = (lane & 3) ^ ((r >> 2) & 3);
        m_src[j] = (F32 ? (const char*)a.dz32 : (const char*)(a.dz + m / (2 * RB) * a.dz_plane)) +
                   (min(row0 + r, a.T - 1) * a.dz_pitch * (int64_t)sizeof(E) + 16 * c);
    }
    auto issue = [&](int s, char* st) {
        const int64_t k = (int64_t)(first + min(s, steps - 1)) * KS;
#pragma unroll
        for (int j = 0; j < 4; ++j)
            load_lds16((const E*)a.W + min(k + n_k[j], (int64_t)a.V - 1) * a.D + n_c[j], st + (4 * wave + j) * 1024);
#pragma unroll
        for (int j = 0; j < MJ; ++j)
            load_lds16(m_src[j] + k * (int64_t)sizeof(E), st + N_BYTES + (MJ * wave + j) % MI * 1024);
    };
    const int l = lane & 31, half = lane >> 5, G = lane >> 4, sl = lane & 15;
    f32x16_t acc[2][RB];
#pragma unroll
    for (int b = 0; b < 2; ++b)
#pragma unroll
        for (int rb = 0; rb < RB; ++rb) acc[b][rb] = f32x16_t{};
    auto work = [&](const char* st) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            u32x4_t m[PLANES][RB];
#pragma unroll
            for (int pl = 0; pl < PLANES; ++pl)
#pragma unroll
                for (int rb = 0; rb < RB; ++rb)
                    m[pl][rb] = *(const u32x4_t*)(st + N_BYTES + (32 * (RB * pl + rb) + l) * 64 +
                                                  (((2 * i + half) ^ ((l >> 2) & 3)) << 4));
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                u32x4_t n;
                if constexpr (F32) {
                    const int d = 64 * wave + 32 * b + l;
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const int k = 8 * i + 4 * half + q;
                        n[q] = *(const uint32_t*)(st + k * ROW + (((d >> 2) ^ swz(k)) << 4) + 4 * (d & 3));
                    }
                } else {
                    const int R = 64 * wave + 32 * b + 16 * (G & 1) + 4 * (sl & 3);
                    s16x4_t h[2];
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        const int k = 8 * (G >> 1) + 4 * r + (sl >> 2);
                        h[r] = read_tr(st + (16 * i + k) * ROW + (((R >> 3) ^ swz_tr(k)) << 4) + 8 * ((R >> 2) & 1));
                    }
                    n = __builtin_bit_cast(u32x4_t, cat_bf16(h[0], h[1]));
                }
#pragma unroll
                for (int pl = PLANES - 1; pl >= 0; --pl)
#pragma unroll
                    for (int rb = 0; rb < RB; ++rb) acc[b][rb] = multiply<F32>(n, m[pl][rb], acc[b][rb]);
            }
        }
    };
    if constexpr (NS == 4) {
        char* const st[4] = {st0, st1, st2, st3};
        ring<4, PER>(steps, st, issue, work);
    } else {
        char* const st[3] = {st0, st1, st2};
        ring<3, PER>(steps, st, issue, work);
    }
#pragma unroll
    for (int rb = 0; rb < RB; ++rb) {
        const int64_t row = row0 + 32 * rb + l;
        if (row >= a.T) continue;
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
            for (int vg = 0; vg < 4; ++vg) {
                const int c = nt * 256 + 64 * wave + 32 * b + 8 * vg + 4 * half;
                const f32x16_t& x = acc[b][rb];
                if (c < a.D)       // D is a multiple of 4
                    *(float4*)(a.dh_part + ((int64_t)split * a.T + row) * a.D + c) =
                        make_float4(x[4 * vg], x[4 * vg + 1], x[4 * vg + 2], x[4 * vg + 3]);
            }
    }
}

// dh = the sum of its parts: 16 groups of 4 columns a workgroup, 16 threads each
// over every 16th part, then over the 16, in order.
__global__ __launch_bounds__(256) void vocab_few_sum_kernel(const float* __restrict__ part, int splits, int64_t n4,
                                                            bool bf16, void* __restrict__ dh) {
    __shared__ float4 sums[16][16];
    const int c = threadIdx.x & 15, sl = threadIdx.x >> 4;
    const int64_t i = (int64_t)blockIdx.x * 16 + c;
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
    if (i < n4) {
#pragma unroll 8
        for (int k = sl; k < splits; k += 16) {
            const float4 v = *(const float4*)(part + (k * n4 + i) * 4);
            s.x += v.x, s.y += v.y, s.z += v.z, s.w += v.w;
        }
    }
    sums[sl][c] = s;
    __syncthreads();
    if (sl || i >= n4) return;
#pragma unroll
    for (int k = 1; k < 16; ++k) {
        const float4 v = sums[k][c];
        s.x += v.x, s.y += v.y, s.z += v.z, s.w += v.w;
    }
    if (bf16) *(uint2*)((uint16_t*)dh + i * 4) = make_uint2(pack_bf16(s.x, s.y), pack_bf16(s.z, s.w));
    else *(float4*)((float*)dh + i * 4) = s;
}

// dW: K is the rows, 32 (bf16) or 16 (fp32) a step.
template <bool F32, bool OUT16>
__global__ __launch_bounds__(256, 4) void vocab_few_dw_kernel(const VocabFew a, int n_tiles, void* __restrict__ out) {
    using E = typename Elem<F32>::type;
    constexpr int KS = F32 ? 16 : 32, PLANES = F32 ? 1 : 2;
    constexpr int HROW = 256 * sizeof(E), ZROW = 64 * sizeof(E);   // bytes of a k row of h, of dz
    __shared__ __attribute__((aligned(1024))) char lds[32768];     // h's rows, dz's rows; then the output's
    constexpr int Z = 16384;
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int nt = blockIdx.x % n_tiles;
    const int64_t v0 = (int64_t)(blockIdx.x / n_tiles) * 64;
    const int l = lane & 31, half = lane >> 5, G = lane >> 4, sl = lane & 15;
    auto swz_z = [](int k) { return F32 ? 0 : 2 * (k & 3); };       // of dz's 128-byte rows

    f32x16_t acc[2][2];                                             // [columns][entries]
#pragma unroll
    for (int b = 0; b < 2; ++b)
#pragma unroll
        for (int e = 0; e < 2; ++e) acc[b][e] = f32x16_t{};
    for (int64_t k0 = 0; k0 < a.T; k0 += KS) {
        if (k0) __syncthreads();
        constexpr int HC = HROW / 16, HR = 64 / HC, ZC = ZROW / 16, ZR = 64 / ZC;   // chunks of a row, rows of a DMA instruction
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int k = HR * (4 * wave + j) + lane / HC;
            const int c = nt * 256 + ((lane % HC) ^ (F32 ? 0 : swz_tr(k))) * (16 / (int)sizeof(E));
            // a row that does not count is read as zeros, whatever it holds
            const bool there = k0 + k < a.T && (!F32 || a.lse[k0 + k] != INFINITY);
            const E* p = (const E*)a.h + (k0 + k) * a.h_pitch + (c < a.D ? c : 0);
            load_lds16(there ? (const void*)p : (const void*)few_zeros, lds + (4 * wave + j) * 1024);
        }
#pragma unroll
        for (int pl = 0; pl < PLANES; ++pl) {
            const int k = ZR * wave + lane / ZC;
            const E* p = (F32 ? (const E*)a.dz32 : (const E*)a.dz + pl * a.dz_plane) + (k0 + k) * a.dz_pitch + v0 +
                         ((lane % ZC) ^ swz_z(k)) * (16 / (int)sizeof(E));
            load_lds16(k0 + k < a.T ? (const void*)p : (const void*)few_zeros, lds + Z + (4 * pl + wave) * 1024);
        }
        wait_vmem();
        __syncthreads();
        if constexpr (F32) {
#pragma unroll
            for (int i = 0; i < KS / 2; ++i) {
                const int k = 2 * i + half;
                float n[2], m[2];
#pragma unroll
                for (int b = 0; b < 2; ++b) {
                    n[b] = *(const float*)(lds + k * HROW + 4 * (64 * wave + 32 * b + l));
                    m[b] = *(const float*)(lds + Z + k * ZROW + 4 * (32 * b + l));
                }
#pragma unroll
                for (int b = 0; b < 2; ++b)
#pragma unroll
                    for (int e = 0; e < 2; ++e) acc[b][e] = __builtin_amdgcn_mfma_f32_32x32x2f32(n[b], m[e], acc[b][e], 0, 0, 0);
            }
        } else {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                auto frag = [&](const char* at, int row, int R, int swz_of_k(int)) {
                    s16x4_t x[2];
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        const int k = 8 * (G >> 1) + 4 * r + (sl >> 2);
                        x[r] = read_tr(at + (16 * i + k) * row + (((R >> 3) ^ swz_of_k(k)) << 4) + 8 * ((R >> 2) & 1));
                    }
                    return cat_bf16(x[0], x[1]);
                };
                const int R = 16 * (G & 1) + 4 * (sl & 3);
                bf16x8_t n[2];
#pragma unroll
                for (int b = 0; b < 2; ++b) n[b] = frag(lds, HROW, 64 * wave + 32 * b + R, [](int k) { return swz_tr(k); });
#pragma unroll
                for (int pl = PLANES - 1; pl >= 0; --pl)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const bf16x8_t m = frag(lds + Z + 4096 * pl, ZROW, 32 * e + R, [](int k) { return 2 * (k & 3); });
#pragma unroll
                        for (int b = 0; b < 2; ++b)
                            acc[b][e] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(n[b], m, acc[b][e], 0, 0, 0);
                    }
            }
        }
    }
    __syncthreads();
    // 32 entries x 64 columns of the wavefront's own at a time through LDS, so that
    // a store writes whole rows of 128 or 256 bytes
    using O = typename Elem<!OUT16>::type;
    constexpr int OROW = 64 * sizeof(O), OC = OROW / 16, OR = 64 / OC;
    char* own = lds + wave * 8192;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
            for (int vg = 0; vg < 4; ++vg) {
                const f32x16_t& x = acc[b][e];
                if constexpr (OUT16)
                    *(uint2*)(own + l * OROW + (((4 * b + vg) ^ (l & 7)) << 4) + 8 * half) =
                        make_uint2(pack_bf16(x[4 * vg], x[4 * vg + 1]), pack_bf16(x[4 * vg + 2], x[4 * vg + 3]));
                else
                    *(float4*)(own + l * OROW + (((8 * b + 2 * vg + half) ^ (l & 15)) << 4)) =
                        make_float4(x[4 * vg], x[4 * vg + 1], x[4 * vg + 2], x[4 * vg + 3]);
            }
#pragma unroll
        for (int q = 0; q < 32 / OR; ++q) {
            const int r = OR * q + lane / OC, c = lane % OC;
            const u32x4_t v = *(const u32x4_t*)(own + r * OROW + ((c ^ (r & (OC - 1))) << 4));
            const int64_t row = v0 + 32 * e + r;
            const int col = nt * 256 + 64 * wave + c * (16 / (int)sizeof(O));
            if (row < a.V && col < a.D) *(u32x4_t*)((O*)out + row * a.D + col) = v;
        }
    }
}

bool fits(const VocabFew& a) {
    return a.T > 0 && a.V > 0 && a.D > 0 && a.D % (a.f32 ? 4 : 8) == 0 && a.h_pitch >= a.D;
}

template <bool DZ>
hipError_t launch_logits(const VocabFew& a, hipStream_t s) {
    if (!fits(a)) return hipErrorInvalidValue;
    const int rb = a.T <= 32 ? 1 : 2;
    // dz is written to the end of its rows: what reads it takes whole tiles, and
    // zeros times what the workspace held would be no zeros
    const int cols = vocab_few_cols(a.T, a.V);
    const int64_t m_tiles = (a.T + 32 * rb - 1) / (32 * rb), grid = m_tiles * (((DZ ? a.dz_pitch : (int64_t)a.V) + cols - 1) / cols);
    if (grid > 1 << 23) return hipErrorInvalidValue;
    auto go = [&](auto* kernel) { kernel<<<(unsigned)grid, 256, 0, s>>>(a, (int)m_tiles); };
    if (cols == FN) {
        if (a.f32) go(rb == 1 ? vocab_few_logits_kernel<true, 1, DZ> : vocab_few_logits_kernel<true, 2, DZ>);
        else go(rb == 1 ? vocab_few_logits_kernel<false, 1, DZ> : vocab_few_logits_kernel<false, 2, DZ>);
    } else {
        if (a.f32) go(rb == 1 ? vocab_few_split_kernel<true, 1, DZ> : vocab_few_split_kernel<true, 2, DZ>);
        else go(rb == 1 ? vocab_few_split_kernel<false, 1, DZ> : vocab_few_split_kernel<false, 2, DZ>);
    }
    return hipGetLastError();
}

}  // namespace

// With 125 tiles of 128 entries those of 32 take 15 us against 23 (4 rows of 16000 x 768
// fp32), 22 against 38 (256 of 3900), 7 against 9 (bf16); with 235 26 against 25, bf16
// 14 against 12.
int vocab_few_cols(int64_t T, int V) {
    const int rows = T <= 32 ? 32 : 64;
    return ((int64_t)V + FN - 1) / FN * ((T + rows - 1) / rows) < 160 ? 32 : FN;
}

int vocab_few_splits(int64_t T, int D, int V, bool f32) {
    const int64_t m_tiles = (T + (T <= 32 ? 31 : 63)) / (T <= 32 ? 32 : 64), n_tiles = (D + 255) / 256;
    const int64_t steps = (V + (f32 ? 15 : 31)) / (f32 ? 16 : 32);
    // a workgroup a CU, of 4 steps at least
    return (int)std::max<int64_t>(1, std::min<int64_t>(256 / (m_tiles * n_tiles), steps / 4));
}

hipError_t launch_vocab_few_stats(const VocabFew& a, hipStream_t s) { return launch_logits<false>(a, s); }
hipError_t launch_vocab_few_dz(const VocabFew& a, hipStream_t s) {
    if (a.dz_pitch % FN || a.dz_pitch < a.V) return hipErrorInvalidValue;
    return launch_logits<true>(a, s);
}

hipError_t launch_vocab_few_dw(const VocabFew& a, void* dW, bool out16, hipStream_t s) {
    if (!fits(a) || a.dz_pitch % FN || a.dz_pitch < a.V || (a.f32 && out16)) return hipErrorInvalidValue;
    const int n_tiles = (a.D + 255) / 256;
    const int64_t grid = ((int64_t)a.V + 63) / 64 * n_tiles;
    if (grid > 1 << 23) return hipErrorInvalidValue;
    if (a.f32) vocab_few_dw_kernel<true, false><<<(unsigned)grid, 256, 0, s>>>(a, n_tiles, dW);
    else if (out16) vocab_few_dw_kernel<false, true><<<(unsigned)grid, 256, 0, s>>>(a, n_tiles, dW);
    else vocab_few_dw_kernel<false, false><<<(unsigned)grid, 256, 0, s>>>(a, n_tiles, dW);
    return hipGetLastError();
}

hipError_t launch_vocab_few_dh(const VocabFew& a, hipStream_t s) {
    if (!fits(a) || a.dz_pitch % FN || a.dz_pitch < a.V) return hipErrorInvalidValue;
    const int rb = a.T <= 32 ? 1 : 2;
    const int m_tiles = (int)((a.T + 32 * rb - 1) / (32 * rb)), n_tiles = (a.D + 255) / 256;
    const int splits = vocab_few_splits(a.T, a.D, a.V, a.f32);
    const unsigned grid = (unsigned)(m_tiles * n_tiles * splits);
    if (a.f32) {
        if (rb == 1) vocab_few_dh_kernel<true, 1><<<grid, 256, 0, s>>>(a, n_tiles, m_tiles, splits);
        else vocab_few_dh_kernel<true, 2><<<grid, 256, 0, s>>>(a, n_tiles, m_tiles, splits);
    } else {
        if (rb == 1) vocab_few_dh_kernel<false, 1><<<grid, 256, 0, s>>>(a, n_tiles, m_tiles, splits);
        else vocab_few_dh_kernel<false, 2><<<grid, 256, 0, s>>>(a, n_tiles, m_tiles, splits);
    }
    return hipGetLastError();
}

hipError_t launch_vocab_few_sum(const float* part, int parts, int64_t T, int D, bool bf16, void* dh, hipStream_t s) {
    const int64_t n4 = T * D / 4;
    vocab_few_sum_kernel<<<(unsigned)((n4 + 15) / 16), 256, 0, s>>>(part, parts, n4, bf16, dh);
    return hipGetLastError();
}

}  // namespace moe
