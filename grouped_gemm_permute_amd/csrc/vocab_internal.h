// vocab_internal.h -- what the products of the vocabulary's losses
// (vocab_gemm.hip) take from their entry points (vocab_loss.hip).  Internal
// to libmoe_ffn.so.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace moe {

// e^d for fp32 results: d log2(e) is rounded by up to |d| 2^-24 of the result, and
// that rounding is made good.
__device__ __forceinline__ float exp_fp32(float d) {
    const float t = d * 1.4426950408889634f;
    const float r = fmaf(d, 1.4426950408889634f, -t) + d * 1.9259629911266175e-8f;   // log2(e) - its fp32 value
    const float e = __builtin_amdgcn_exp2f(t);
    return t > -126.f ? fmaf(e, r * 0.6931471805599453f, e) : e;
}

// Orders a wavefront's LDS accesses for the compiler (the hardware keeps their
// order), where lanes read what other lanes wrote.
__device__ __forceinline__ void wave_sync() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// One operand of a product: bf16 rows, `planes` arrays of them `plane`
// elements apart (an fp32 array is the sum of three such planes).
struct VocabOperand {
    const uint16_t* p;
    int64_t pitch;            // elements between rows
    int64_t plane;            // elements between planes
};

// Rows of tokens that count: `rows` lists them in order and `count` says how
// many they are (both on the device); null: all T of them.
struct VocabRows {
    const int32_t* rows;
    const int32_t* count;
    int64_t T;
};

constexpr int kVocabTileRows = 128;   // rows of tokens of a logits tile
constexpr int kVocabTileCols = 256;   // entries of the vocabulary of a logits tile

// z = h W^T by tiles; per tile and row the largest z c and the sum of
// 2^(z c - largest), to part[tile][row] (row pitch `part_pitch`); z of a
// row's target to zt.  Rows of h, part and zt are compact.  c = log2(e) / temperature.
struct VocabStats {
    VocabOperand h, W;
    VocabRows rows;
    int64_t V;
    int K;                    // a multiple of 32
    int products;             // 1, or 6 products of three planes
    float c;
    float2* part;
    int64_t part_pitch;
    const int32_t* target;    // [T] or null
    float* zt;
};
hipError_t launch_vocab_stats(const VocabStats& a, hipStream_t s);

// dz = g (exp(z inv_tau - lse) - [v = target]) for entries v0 .. v0 + len - 1,
// to dz (bf16 [compact rows, pitch], or three planes of it), zeros up to the
// next multiple of 256.  g and lse are of compact rows, g already divided by
// the temperature; target (or null) is of token rows.
struct VocabDz {
    VocabOperand h, W;
    VocabRows rows;
    int64_t V, v0;
    int len;
    int K;
    int products;
    float inv_tau;
    const float *g, *lse;
    const int32_t* target;
    uint16_t* dz;
    int64_t dz_pitch, dz_plane;
    float* err;               // or null; [compact rows], with target: see VocabGrad
};
hipError_t launch_vocab_dz(const VocabDz& a, hipStream_t s);

// The same for many rows; info: of compact rows g / tau, lse and the target's
// bits (negative: none), instead of g, lse and target.  K a multiple of 128.
hipError_t launch_vocab_stats_whole(const VocabStats& a, const float4* info, hipStream_t s);
hipError_t launch_vocab_dz_whole(const VocabDz& a, const float4* info, hipStream_t s);

// C[m][n] = sum over k of M and N operands:
//   dh (dW = false): m = compact row, k = entry of the piece, n = column of D
//   dW (dW = true):  m = entry of the piece, k = compact row, n = column of D
// added to acc's (fp32, row pitch acc_pitch) if `add`, and written to acc, or with
// `last` to out (fp32 or bf16, row pitch N; dh's rows mapped through rows.rows).
// Two launches: the tiles, and the sums of those that several workgroups made.
struct VocabGrad {
    bool dW;
    VocabOperand m, n;        // dh: dz, the table; dW: dz, h with zeros up to the next 32nd row
    VocabRows rows;
    int len;                  // entries of the piece
    int N;                    // columns of D
    int products;
    float* partial;           // vocab_grad_partial_bytes()
    float* acc;               // null where neither `add` nor !last
    int64_t acc_pitch;
    bool add, last;
    void* out;
    bool out_bf16;
    // dh, or null: what rounding dz to bf16 took from entry `entry[m]` of row m, which
    // makes up most of the row (its target); it is given back with the sum
    const float* err;
    const int32_t* entry;     // negative: none
    const uint16_t* table;    // bf16, all of it
    int64_t table_pitch;
    bool halves;              // of the launch: set by launch_vocab_grad
};
// Tiles of 256 rows (entries of the piece) x 256 columns, at most: their sums are 8
// workgroups of 256 threads each, fewer than 2^32 in a grid.
constexpr int64_t kVocabGradTiles = 1 << 20;
inline int64_t vocab_grad_tiles(int64_t M, int N) { return (M + 255) / 256 * ((N + 255) / 256); }
size_t vocab_grad_partial_bytes(int N);
hipError_t launch_vocab_grad(const VocabGrad& a, hipStream_t s);

// Few rows (vocab_few.hip): the products that read the table once, in its own
// type.  Rows of 16 bytes' multiples; every row is a row of its own, those that
// do not count have an infinite lse (dz) and are left to the caller (stats).
constexpr int kVocabFewCols = 128;    // entries of a logits tile, or, K divided over its wavefronts, 32
struct VocabFew {
    bool f32;
    const void *h, *W;        // bf16, or fp32; W: of the piece's first entry
    int64_t h_pitch;          // elements
    int64_t T;
    int D, V;                 // V: entries of the piece
    float scale;              // stats: log2(e) / tau; dz: 1 / tau
    const int32_t* target;    // [T] or null
    float2* part;             // stats
    int64_t part_pitch;
    float* zt;                // stats
    const float *g, *lse;     // dz: g / tau, lse
    uint16_t* dz;             // two planes of bf16 (bf16), three (f32; or null): [T, pitch]
    float* dz32;              // the same in fp32 (f32)
    int64_t dz_pitch, dz_plane;
    float* dh_part;           // [splits, T, D]
    int64_t v0;               // dz: the piece's first entry
};
int vocab_few_cols(int64_t T, int V);          // entries of a logits tile
int vocab_few_splits(int64_t T, int D, int V, bool f32);
hipError_t launch_vocab_few_stats(const VocabFew& a, hipStream_t s);
hipError_t launch_vocab_few_dz(const VocabFew& a, hipStream_t s);
hipError_t launch_vocab_few_dh(const VocabFew& a, hipStream_t s);     // vocab_few_splits() parts
// dh = the sum of `parts` parts [T, D], in order.
hipError_t launch_vocab_few_sum(const float* part, int parts, int64_t T, int D, bool bf16, void* dh, hipStream_t s);
hipError_t launch_vocab_few_dw(const VocabFew& a, void* dW, bool out16, hipStream_t s);

}  // namespace moe
