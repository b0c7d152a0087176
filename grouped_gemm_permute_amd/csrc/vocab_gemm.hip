// vocab_gemm.hip -- the matrix products behind the losses over a vocabulary,
// on bf16 MFMA, none of which leaves the logits in memory:
//
//  stats:  z = h W^T, tile by tile; of each row of a tile the largest z c and
//          the sum of 2^(z c - largest) are kept (c = log2(e) / temperature),
//          8 bytes for 256 logits
//  dz:     the same product again, for a piece of the vocabulary, and from it
//          the logits' gradient g (exp(z / tau - lse) - [v = target]) in bf16
//  grad:   dh = dz W (K: the piece's entries) and dW = dz^T h (K: tokens)
//
// fp32 operands come as three bf16 planes whose sum they are (8 + 8 + 8 bits),
// and their product is the six products of planes i, j with i + j <= 2 run
// through the same loop, the smallest first: what is left out is of the size of
// an fp32 product's own rounding.  Matrix cores take fp32 operands directly at
// a sixteenth of the bf16 rate, six bf16 products cost a sixth.
//
// Tile engines (after that of gemm_bf16.hip, with either layout of each operand):
// operands global -> LDS with 16-byte DMA into a ring of stages, the next
// fragments read from LDS under this step's MFMAs.  The MFMA's A operand is 32
// columns of N, its B operand 32 rows of M, so that a lane ends with 4 consecutive
// columns of one row.
//  * stats and dz, many rows: 256 x 256, 8 wavefronts, K steps of 64 in two stages of
//    64 KiB, one workgroup a CU that goes from tile to tile and loads the next one
//    under the epilogue's exponentials (stats of 32768 x 768 x 65536: 2.61 to 2.93 ms, 1130
//    to 1260 TFLOP/s, MFMA 58% busy at 2.0 GHz; a library's product of that shape, the
//    logits written: 1130.  dz of half of it: 1.68 ms, 980 with its 2 GiB written, 53%);
//  * stats and dz, fewer rows, or a D that is no multiple of 128: 128 x 256, 4
//    wavefronts, K steps of 32 in 3 stages of 24 KiB, two workgroups a CU: the
//    exponentials of one run under the other's MFMAs;
//  * grad: 256 x 256, 8 wavefronts, K steps of 32 in 4 stages of 32 KiB, a workgroup a
//    CU that goes from part to part (dh and dW of 32768 x 768 x 32768: 1.26 and 1.28 ms, 1300
//    TFLOP/s, MFMA 70 to 74% busy).  In steps of 64 as above the same products took 2%
//    longer.
#include "mfma_common.h"
#include "vocab_internal.h"

#include <type_traits>

namespace moe {
namespace {

using namespace mfma;

constexpr int BK = 32;
constexpr int TN = 256;                       // columns of N of a tile
constexpr int KC_ROW = BK * 2;                // bytes of a K-contiguous row in a stage
constexpr int KS_ROW = 512;                   // bytes of a k row of 256 columns
constexpr int N_BYTES = TN * KC_ROW;          // 16 KiB either way

constexpr int64_t kMaxTiles = 1 << 22;         // of 512 threads: fewer than 2^32 in a grid

static_assert(kVocabTileCols == TN && kVocabTileRows == 128, "tile sizes");

// 64-byte rows (4 chunks): 16 consecutive rows read at one logical chunk hit
// 16 distinct bank groups.
__device__ __forceinline__ int swz_kc(int row) { return (row >> 2) & 3; }

// The products of planes, smallest first: (1,1) (2,0) (0,2) (1,0) (0,1) (0,0),
// two bits each; one product alone is the last.
constexpr int kPlaneM = 1 | 2 << 2 | 0 << 4 | 1 << 6 | 0 << 8 | 0 << 10;
constexpr int kPlaneN = 1 | 0 << 2 | 2 << 4 | 0 << 6 | 1 << 8 | 0 << 10;

// The lane's number, made where it stands: kept in a register over a K loop it,
// and what follows from it, would be one too many.
__device__ __forceinline__ int fresh_lane() {
    int z = 0;
    asm volatile("" : "+v"(z));
    return __builtin_amdgcn_mbcnt_hi(~0u, __builtin_amdgcn_mbcnt_lo(~0u, z));
}

// The K loop of one tile.  MC / NC: the M / N operand's rows are contiguous in
// K; else its rows are k and the tile's 256 columns are contiguous.
template <bool MC, bool NC, int ROWS>
struct Engine {
    static constexpr int NW = ROWS == 256 ? 8 : 4;
    static constexpr int NT = 64 * NW;
    static constexpr int NJ = 4;                          // 32-row blocks of a wavefront
    static constexpr int MJ = ROWS / (16 * NW), WJ = 16 / NW;   // DMA instructions a stage
    static constexpr int M_BYTES = ROWS * KC_ROW;
    static constexpr int SBYTES = M_BYTES + N_BYTES;
    static constexpr int NS = ROWS == 256 ? 4 : 3;
    static constexpr int PER_STAGE = MJ + WJ;
    static_assert(MC || ROWS == 256, "k rows of 256 columns");

    // What the loads read: a base for the whole tile and a lane's offset from it,
    // in bytes (one address register a load).  K-contiguous: the lane's row, its
    // chunk of it; else its k row of a step, its chunk of columns.  A last step
    // that ends inside has the largest offset that it may read; lanes past it
    // read there.
    const char *m_base, *n_base;
    uint32_t m_at[MJ], n_at[WJ], m_most, n_most;
    int64_t m_plane, n_plane;         // bytes between planes
    int64_t m_step, n_step;           // bytes between K steps
    int steps;                        // K steps of a product
    int ik, ip;                       // the next stage: its step, its product
    int lane, wave, fw, rw;
    int m_off[NJ][2], n_off[2][2];    // fragment offsets in a stage

    f32x16_t acc[2][NJ];

    struct Frags {
        bf16x8_t n[2][2], m[2][NJ];
    };

    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int mi = 0; mi < 2; ++mi)
#pragma unroll
            for (int nj = 0; nj < NJ; ++nj) acc[mi][nj] = f32x16_t{};
    }

    __device__ __forceinline__ void begin() {
        const int tid = threadIdx.x;
        lane = tid & 63;
        wave = __builtin_amdgcn_readfirstlane(tid >> 6);
        fw = wave & 3;
        rw = wave >> 2;
        clear();
        const int G = lane >> 4, sl = lane & 15, xr = lane & 31;
        auto tr_off = [&](int R, int r) {
            const int k = 8 * (G >> 1) + 4 * r + (sl >> 2);
            return k * KS_ROW + (((R >> 3) ^ swz_tr(k)) << 4) + 8 * ((R >> 2) & 1);
        };
        auto kc_off = [&](int row0, int ks) {
            return (row0 + xr) * KC_ROW + (((2 * ks + (lane >> 5)) ^ swz_kc(xr)) << 4);
        };
        const int tr_col = 16 * (G & 1) + 4 * (sl & 3);
#pragma unroll
        for (int r = 0; r < 2; ++r) {
#pragma unroll
            for (int nj = 0; nj < NJ; ++nj)
                m_off[nj][r] = MC ? kc_off(128 * rw + 32 * nj, r) : tr_off(128 * rw + 32 * nj + tr_col, r);
#pragma unroll
            for (int mi = 0; mi < 2; ++mi)
                n_off[mi][r] = M_BYTES + (NC ? kc_off(64 * fw + 32 * mi, r) : tr_off(64 * fw + 32 * mi + tr_col, r));
        }
    }

    // Rows of a lane's loads: DMA instruction j fills 16 K-contiguous rows, or 2
    // k rows, of a tile.
    __device__ __forceinline__ int kc_row(int j, int per) const { return 16 * (per * wave + j) + (lane >> 2); }
    __device__ __forceinline__ int kc_chunk(int row) const { return (lane & 3) ^ swz_kc(row); }
    __device__ __forceinline__ int ks_row(int j, int per) const { return 2 * (per * wave + j) + (lane >> 5); }
    __device__ __forceinline__ int ks_chunk(int row) const { return (lane & 31) ^ swz_tr(row); }

    // A lane's offsets in tiles of `rows` rows (at least 1) `pitch` bytes apart.
    __device__ __forceinline__ void m_rows(int rows, int64_t pitch) {
#pragma unroll
        for (int j = 0; j < MJ; ++j) {
            const int row = kc_row(j, MJ);
            m_at[j] = (uint32_t)min(row, rows - 1) * (uint32_t)pitch + 16 * kc_chunk(row);
        }
        m_step = KC_ROW;
    }
    __device__ __forceinline__ void n_rows(int rows, int64_t pitch) {
#pragma unroll
        for (int j = 0; j < WJ; ++j) {
            const int row = kc_row(j, WJ);
            n_at[j] = (uint32_t)min(row, rows - 1) * (uint32_t)pitch + 16 * kc_chunk(row);
        }
        n_step = KC_ROW;
    }
    // ... and of k rows, `last` of them (at least 1) in the last step; columns from
    // `cols` on are read as the first ones, and their sums not stored.
    static __device__ __forceinline__ uint32_t most(int last, int64_t pitch, int cols) {
        return (uint32_t)(last - 1) * (uint32_t)pitch + 2 * min(cols, 256) - 16;
    }
    __device__ __forceinline__ void m_ks(int last, int64_t pitch) {
#pragma unroll
        for (int j = 0; j < MJ; ++j) {
            const int k = ks_row(j, MJ);
            m_at[j] = (uint32_t)k * (uint32_t)pitch + 16 * ks_chunk(k);
        }
        m_most = most(last, pitch, 256);
        m_step = BK * pitch;
    }
    __device__ __forceinline__ void n_ks(int last, int64_t pitch, int cols) {
#pragma unroll
        for (int j = 0; j < WJ; ++j) {
            const int k = ks_row(j, WJ);
            n_at[j] = (uint32_t)k * (uint32_t)pitch + (8 * ks_chunk(k) < cols ? 16 * ks_chunk(k) : 0);
        }
        n_most = most(last, pitch, cols);
        n_step = BK * pitch;
    }

    __device__ __forceinline__ void issue(char* st) {
        const int pm = (kPlaneM >> (2 * ip)) & 3, pn = (kPlaneN >> (2 * ip)) & 3;
        const char* m = m_base + pm * m_plane + ik * m_step;
        const char* n = n_base + pn * n_plane + ik * n_step;
        const bool end = ik + 1 == steps;
#pragma unroll
        for (int j = 0; j < MJ; ++j)
            load_lds16(m + (MC ? m_at[j] : min(m_at[j], end ? m_most : ~0u)), st + (MJ * wave + j) * 1024);
#pragma unroll
        for (int j = 0; j < WJ; ++j)
            load_lds16(n + (NC ? n_at[j] : min(n_at[j], end ? n_most : ~0u)), st + M_BYTES + (WJ * wave + j) * 1024);
        // the next stage; past the last one it is read again, into a buffer
        // that is never computed on, so that the loads in flight can be counted
        const bool turn = end && ip < 5;
        ik = turn ? 0 : ik + (end ? 0 : 1);
        ip += turn ? 1 : 0;
    }

    __device__ __forceinline__ void read_frags(const char* st, Frags& f) const {
#pragma unroll
        for (int ks = 0; ks < 2; ++ks) {
#pragma unroll
            for (int mi = 0; mi < 2; ++mi) {
                if constexpr (NC)
                    f.n[ks][mi] = __builtin_bit_cast(bf16x8_t, *(const u32x4_t*)(st + n_off[mi][ks]));
                else
                    f.n[ks][mi] = cat_bf16(read_tr(st + n_off[mi][0] + ks * 16 * KS_ROW),
                                           read_tr(st + n_off[mi][1] + ks * 16 * KS_ROW));
            }
#pragma unroll
            for (int nj = 0; nj < NJ; ++nj) {
                if constexpr (MC)
                    f.m[ks][nj] = __builtin_bit_cast(bf16x8_t, *(const u32x4_t*)(st + m_off[nj][ks]));
                else
                    f.m[ks][nj] = cat_bf16(read_tr(st + m_off[nj][0] + ks * 16 * KS_ROW),
                                           read_tr(st + m_off[nj][1] + ks * 16 * KS_ROW));
            }
        }
    }

    __device__ __forceinline__ void mfmas(const Frags& f) {
#pragma unroll
        for (int ks = 0; ks < 2; ++ks)
#pragma unroll
            for (int nj = 0; nj < NJ; ++nj)
#pragma unroll
                for (int mi = 0; mi < 2; ++mi)
                    acc[mi][nj] =
                        __builtin_amdgcn_mfma_f32_32x32x16_bf16(f.n[ks][mi], f.m[ks][nj], acc[mi][nj], 0, 0, 0);
    }

    static __device__ __forceinline__ void fence() { __builtin_amdgcn_sched_barrier(0); }

    // Step s, its operands in fc: wait for stage s + 1, issue the stage NS - 1
    // on into the buffer of stage s - 1, read stage s + 1's operands into fn, run
    // the MFMAs on fc.
    __device__ __forceinline__ void step(const Frags& fc, Frags& fn, const char* nxt, char* dma) {
        __builtin_amdgcn_s_waitcnt(waitcnt_imm(NS == 4 ? PER_STAGE : 0, 0));
        __builtin_amdgcn_s_barrier();
        fence();
        work(fc, fn, nxt, dma);
    }
    __device__ __forceinline__ void work(const Frags& fc, Frags& fn, const char* nxt, char* dma) {
        issue(dma);
        read_frags(nxt, fn);
        mfmas(fc);
        constexpr int reads = 2 * ((NC ? 2 : 4) + (MC ? 4 : 8));   // LDS reads a step: 12, 16 or 24
#pragma unroll
        for (int i = 0; i < (NW == 8 ? 4 : 6); ++i) {
            __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);   // MFMA
            __builtin_amdgcn_sched_group_barrier(0x010, 1, 0);   // vector memory
            __builtin_amdgcn_sched_group_barrier(0x100, reads > 16 ? 2 : 1, 0);   // LDS reads
            if constexpr (NW == 8) {
                __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
                __builtin_amdgcn_sched_group_barrier(0x100, reads > 16 ? 2 : 1, 0);
                __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
                __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
                __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
                __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
            }
        }
        if constexpr (NW == 4) {
#pragma unroll
            for (int i = 0; i < 6; ++i) {
                __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
                __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
            }
        }
        fence();
    }

    // The loads and barriers of run() for a wavefront without rows of its own.
    __device__ __forceinline__ void idle(const int KT, char* st0, char* st1, char* st2, char* st3) {
        static_assert(NS == 4, "stages");
        for (int kt = 0; kt < KT; ++kt) {
            __builtin_amdgcn_s_waitcnt(waitcnt_imm(PER_STAGE, 0));
            __builtin_amdgcn_s_barrier();
            fence();
            const int to = (kt + 3) & 3;
            issue(to == 0 ? st0 : to == 1 ? st1 : to == 2 ? st2 : st3);
        }
        __builtin_amdgcn_s_waitcnt(waitcnt_imm(0, 0));
        __syncthreads();
    }

    // `KT` K steps (at least 1); on return no load is in flight and every wavefront
    // has read the stages.  256 rows: the caller has issued the first three stages and
    // seen them land.
    __device__ __forceinline__ void run(const int KT, char* st0, char* st1, char* st2, char* st3) {
        Frags fa, fb;
        if constexpr (NS == 3) {
            issue(st0);
            issue(st1);
            __builtin_amdgcn_s_waitcnt(waitcnt_imm(PER_STAGE, 15));
            __builtin_amdgcn_s_barrier();
        }
        fence();
        read_frags(st0, fa);
        fence();
        int kt = 0;
        if constexpr (NS == 4) {
            for (; kt + 4 <= KT; kt += 4) {
                step(fa, fb, st1, st3);
                step(fb, fa, st2, st0);
                step(fa, fb, st3, st1);
                step(fb, fa, st0, st2);
            }
            if (kt < KT) {
                step(fa, fb, st1, st3);
                if (kt + 1 < KT) {
                    step(fb, fa, st2, st0);
                    if (kt + 2 < KT) step(fa, fb, st3, st1);
                }
            }
        } else {
            // buffers turn with period 3 and the operands' registers with period 2
            for (; kt + 3 <= KT; kt += 3) {
                step(fa, fb, st1, st2);
                step(fb, fa, st2, st0);
                step(fa, fb, st0, st1);
                const Frags t = fa;
                fa = fb;
                fb = t;
            }
            if (kt < KT) {
                step(fa, fb, st1, st2);
                if (kt + 1 < KT) step(fb, fa, st2, st0);
            }
        }
        __builtin_amdgcn_s_waitcnt(waitcnt_imm(0, 0));
        __syncthreads();
    }
};

// A logits tile's place: the XCDs take contiguous ranges of tiles, in groups of
// kGroup row tiles that walk over the columns, so that the tiles in flight on
// one XCD (64) are about 16 row tiles x 4 column tiles and share both operands
// through its L2.
constexpr int kGroup = 16;
__device__ __forceinline__ bool logits_tile(int m_tiles, int n_tiles, int& mt, int& nt) {
    const int id = xcd_remap_work(blockIdx.x, m_tiles * n_tiles);
    if (id < 0) return false;
    const int g = id / (kGroup * n_tiles);
    const int rows = min(kGroup, m_tiles - g * kGroup);
    const int r = id - g * kGroup * n_tiles;
    nt = r / rows;
    mt = g * kGroup + (r - nt * rows);
    return true;
}

using Logits = Engine<true, true, 128>;

// Rows row0.. of h (`rows` in all) and v0.. of W (V) of a logits tile.
template <typename E>
__device__ __forceinline__ void logits_sources(E& e, const VocabOperand& h, const VocabOperand& W, int products, int K,
                                               int64_t row0, int64_t rows, int64_t v0, int64_t V) {
    e.m_base = (const char*)(h.p + row0 * h.pitch);
    e.n_base = (const char*)(W.p + v0 * W.pitch);
    e.m_rows((int)min(rows - row0, (int64_t)256), 2 * h.pitch);
    e.n_rows((int)min(V - v0, (int64_t)256), 2 * W.pitch);
    e.m_plane = 2 * h.plane;
    e.n_plane = 2 * W.plane;
    e.steps = K / BK;
    e.ip = 6 - products;
    e.ik = 0;
}

// A lane's 32 values of a row stand for columns 32 (v / 16) + 8 (v / 4 % 4) + v % 4
// of 64 (less 4 for the upper lanes): whether column `at` is among them, and it.
__device__ __forceinline__ bool has_column(int at) { return at >= 0 && at < 64 && !(at & 4); }
__device__ __forceinline__ float column(const f32x16_t& x, const f32x16_t& y, int at) {
    float e = 0.f;
#pragma unroll
    for (int v = 0; v < 16; ++v) {
        e = at == 8 * (v / 4) + v % 4 ? x[v] : e;
        e = at == 32 + 8 * (v / 4) + v % 4 ? y[v] : e;
    }
    return e;
}
// What rounding to bf16 takes from a value.
__device__ __forceinline__ float rounding_of(float e) { return e - __uint_as_float(pack_bf16(e, 0.f) << 16); }

// Of the 64 logits of a row that lanes l and l + 32 hold: the largest times c,
// and the sum of 2^(z c - that).
__device__ __forceinline__ float2 row_stats(const f32x16_t& x, const f32x16_t& y, float c) {
    // the larger of two as the middle of them and infinity: fmaxf would first quieten
    // what may be a signalling NaN, 58 instructions for these 32 values against 24
    float top = -INFINITY, most = INFINITY;
    asm volatile("" : "+s"(most));
#pragma unroll
    for (int v = 0; v < 16; ++v) top = fmaxf(top, __builtin_amdgcn_fmed3f(x[v], y[v], most));
    top = fmaxf(top, __shfl_xor(top, 32)) * c;
    const float off = top == -INFINITY ? 0.f : top;
    float sum = 0.f;
#pragma unroll
    for (int v = 0; v < 16; ++v) sum += __builtin_amdgcn_exp2f(fmaf(x[v], c, -off));
#pragma unroll
    for (int v = 0; v < 16; ++v) sum += __builtin_amdgcn_exp2f(fmaf(y[v], c, -off));
    return make_float2(top, sum + __shfl_xor(sum, 32));
}
__device__ __forceinline__ float2 join_stats(const float2 (&p)[4]) {
    const float top = fmaxf(fmaxf(p[0].x, p[1].x), fmaxf(p[2].x, p[3].x));
    const float off = top == -INFINITY ? 0.f : top;
    float sum = 0.f;
#pragma unroll
    for (int w = 0; w < 4; ++w) sum += p[w].y * __builtin_amdgcn_exp2f(p[w].x - off);
    return make_float2(top, sum);
}

// Element v of acc[mi][nj] on lane l: row 32 nj + l % 32 of the tile, column
// 64 w + 32 mi + 8 (v / 4) + 4 (l / 32) + v % 4.
__global__ __launch_bounds__(256, 2) void vocab_stats_kernel(const VocabStats a, int n_tiles) {
    __shared__ __attribute__((aligned(1024))) char st0[Logits::SBYTES];
    __shared__ __attribute__((aligned(1024))) char st1[Logits::SBYTES];
    __shared__ __attribute__((aligned(1024))) char st2[Logits::SBYTES];
    const int64_t rows = a.rows.count ? *a.rows.count : a.rows.T;
    int mt, nt;
    if (!logits_tile((int)((rows + 127) / 128), n_tiles, mt, nt)) return;
    const int64_t row0 = (int64_t)mt * 128, v0 = (int64_t)nt * TN;
    Logits e;
    e.begin();
    logits_sources(e, a.h, a.W, a.products, a.K, row0, rows, v0, a.V);
    e.run(e.steps * a.products, st0, st1, st2, nullptr);

    const int l = e.lane & 31, half = e.lane >> 5;
    const int left = (int)min(a.V - v0, (int64_t)TN);
    float2* tile = (float2*)st0;                              // [4][128]
#pragma unroll
    for (int nj = 0; nj < 4; ++nj) {
        const int64_t row = row0 + 32 * nj + l;
        // the target's logit, where it is among this wavefront's 64 columns
        if (a.target) {
            const int64_t target = row < rows ? a.target[a.rows.rows ? a.rows.rows[row] : row] : -1;
            const bool mine = target >= v0 + 64 * e.fw && target < min(v0 + 64 * e.fw + 64, a.V);
            if (__ballot(mine)) {
                const int at = mine ? (int)(target - v0) - 64 * e.fw - 4 * half : -1;
                const float z = column(e.acc[0][nj], e.acc[1][nj], at);
                if (has_column(at)) a.zt[row] = z;
            }
        }
        if (left < TN) {
#pragma unroll
            for (int mi = 0; mi < 2; ++mi)
#pragma unroll
                for (int v = 0; v < 16; ++v)
                    if (64 * e.fw + 32 * mi + 8 * (v / 4) + 4 * half + v % 4 >= left) e.acc[mi][nj][v] = -INFINITY;
        }
        const float2 s = row_stats(e.acc[0][nj], e.acc[1][nj], a.c);
        if (half == 0) tile[e.fw * 128 + 32 * nj + l] = s;
    }
    __syncthreads();
    const int r = threadIdx.x;
    if (r < 128 && row0 + r < rows) {
        float2 p[4];
#pragma unroll
        for (int w = 0; w < 4; ++w) p[w] = tile[w * 128 + r];
        a.part[nt * a.part_pitch + row0 + r] = join_stats(p);
    }
}

// e^d, by way of 2^x for bf16 results.
template <int PLANES>
__device__ __forceinline__ float softmax_of(float d) {
    return PLANES == 1 ? __builtin_amdgcn_exp2f(d * 1.4426950408889634f) : exp_fp32(d);
}

// PLANES: 1 (bf16) or 3.
template <int PLANES>
__global__ __launch_bounds__(256, 2) void vocab_dz_kernel(const VocabDz a, int n_tiles) {
    __shared__ __attribute__((aligned(1024))) char st0[Logits::SBYTES];
    __shared__ __attribute__((aligned(1024))) char st1[Logits::SBYTES];
    __shared__ __attribute__((aligned(1024))) char st2[Logits::SBYTES];
    const int64_t rows = a.rows.count ? *a.rows.count : a.rows.T;
    int mt, nt;
    if (!logits_tile((int)((rows + 127) / 128), n_tiles, mt, nt)) return;
    const int64_t row0 = (int64_t)mt * 128, c0 = (int64_t)nt * TN, v0 = a.v0 + c0;
    Logits e;
    e.begin();
    logits_sources(e, a.h, a.W, a.products, a.K, row0, rows, v0, a.V);
    const int l = e.lane & 31, half = e.lane >> 5;
    const int left = (int)min((int64_t)a.len - c0, (int64_t)TN);
    // the rows' values are on their way during the K loop
    float lse[4], g[4];
    int target[4];
#pragma unroll
    for (int nj = 0; nj < 4; ++nj) {
        const int64_t row = min(row0 + 32 * nj + l, rows - 1);
        lse[nj] = a.lse[row], g[nj] = a.g[row];
        target[nj] = a.target ? a.target[a.rows.rows ? a.rows.rows[row] : row] : -1;
    }
    e.run(e.steps * a.products, st0, st1, st2, nullptr);

#pragma unroll
    for (int nj = 0; nj < 4; ++nj) {
#pragma unroll
        for (int mi = 0; mi < 2; ++mi)
#pragma unroll
            for (int v = 0; v < 16; ++v)
                e.acc[mi][nj][v] = softmax_of<PLANES>(fmaf(e.acc[mi][nj][v], a.inv_tau, -lse[nj]));
        if (a.target) {
            const bool mine = target[nj] >= v0 + 64 * e.fw && target[nj] < min(v0 + 64 * e.fw + 64, a.V);
            if (__ballot(mine)) {
                const int at = mine ? (int)(target[nj] - v0) - 64 * e.fw - 4 * half : -1;
#pragma unroll
                for (int mi = 0; mi < 2; ++mi)
#pragma unroll
                    for (int v = 0; v < 16; ++v)
                        if (at == 32 * mi + 8 * (v / 4) + v % 4) e.acc[mi][nj][v] -= 1.f;
            }
        }
#pragma unroll
        for (int mi = 0; mi < 2; ++mi)
#pragma unroll
            for (int v = 0; v < 16; ++v) e.acc[mi][nj][v] *= g[nj];
        if (PLANES == 1 && a.err) {
            const bool mine = target[nj] >= v0 + 64 * e.fw && target[nj] < min(v0 + 64 * e.fw + 64, a.V);
            if (__ballot(mine)) {
                const int at = mine ? (int)(target[nj] - v0) - 64 * e.fw - 4 * half : -1;
                const float x = column(e.acc[0][nj], e.acc[1][nj], at);
                if (has_column(at)) a.err[min(row0 + 32 * nj + l, rows - 1)] = rounding_of(x);
            }
        }
        if (left < TN) {
#pragma unroll
            for (int mi = 0; mi < 2; ++mi)
#pragma unroll
                for (int v = 0; v < 16; ++v)
                    if (64 * e.fw + 32 * mi + 8 * (v / 4) + 4 * half + v % 4 >= left) e.acc[mi][nj][v] = 0.f;
        }
    }
    // through LDS, so that the stores write whole rows of 512 bytes; 48 rows a
    // stage buffer, 16-byte chunks XOR-swizzled by the row
    constexpr int RPB = Logits::SBYTES / 512;
    static_assert(RPB % 16 == 0 && 3 * RPB >= 128, "the stage buffers hold the tile");
    auto orow = [&](int r) -> char* {
        const int q = r / RPB;
        return (q == 0 ? st0 : q == 1 ? st1 : st2) + (r - q * RPB) * 512;
    };
#pragma unroll
    for (int pl = 0; pl < PLANES; ++pl) {
        if (pl) __syncthreads();
#pragma unroll
        for (int nj = 0; nj < 4; ++nj) {
            const int r = 32 * nj + l;
            char* p = orow(r);
#pragma unroll
            for (int mi = 0; mi < 2; ++mi)
#pragma unroll
                for (int vg = 0; vg < 4; ++vg) {
                    f32x16_t& x = e.acc[mi][nj];
                    const uint32_t lo = pack_bf16(x[4 * vg], x[4 * vg + 1]), hi = pack_bf16(x[4 * vg + 2], x[4 * vg + 3]);
                    *(uint2*)(p + (((8 * e.fw + 4 * mi + vg) ^ (r & 15)) << 4) + 8 * half) = make_uint2(lo, hi);
                    if (pl + 1 < PLANES) {
                        x[4 * vg] -= __uint_as_float(lo << 16);
                        x[4 * vg + 1] -= __uint_as_float(lo & 0xffff0000u);
                        x[4 * vg + 2] -= __uint_as_float(hi << 16);
                        x[4 * vg + 3] -= __uint_as_float(hi & 0xffff0000u);
                    }
                }
        }
        __syncthreads();
        const int c = threadIdx.x & 31;
        uint16_t* out = a.dz + pl * a.dz_plane + c0 + 8 * c;
#pragma unroll 4
        for (int r = threadIdx.x >> 5; r < 128; r += 8) {
            if (row0 + r >= rows) break;
            __builtin_nontemporal_store(*(const u32x4_t*)(orow(r) + ((c ^ (r & 15)) << 4)),
                                        (u32x4_t*)(out + (row0 + r) * a.dz_pitch));
        }
    }
}

// ---- many rows: stats and dz on 256 x 256 tiles, one workgroup a CU that goes
// through its tiles without a pause: the last steps of a tile load the next
// one's first stages, which land under the epilogue.  What the epilogue wants of
// a row (its g, lse and target) comes into LDS with a stage's loads.  K is a
// multiple of 128: a tile begins and ends with the same stage buffer.
constexpr int kWholeUnits = 256;

// The K loop of a tile, in steps of 64: rows of 128 bytes, whole lines, in two
// stage buffers of 64 KiB, one barrier a step.  A step begins with the operands of
// its first half in registers:
//   read the second half's, run the first half's MFMAs;
//   wait for those and for the next stage, barrier: nobody reads this stage any
//   more;
//   load the stage after the next into its buffer, read the next stage's first
//   half, run the second half's MFMAs.
struct Wide {
    static constexpr int ROW = 128, BYTES = 256 * ROW, NJ = 4;
    const char *m_base, *n_base;
    uint32_t m_at[4], n_at[4];
    int64_t m_plane, n_plane;
    int steps, ik, ip;                // K steps of a product; the next stage
    int wave, fw, rw;
    int m_off[4], n_off[4];           // of a lane's chunks, by 16 k of a step; its rows are constants away
    f32x16_t acc[2][NJ];

    struct Frags {
        bf16x8_t n[2][2], m[2][NJ];
    };

    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int mi = 0; mi < 2; ++mi)
#pragma unroll
            for (int nj = 0; nj < NJ; ++nj) acc[mi][nj] = f32x16_t{};
    }
    // chunk c of row r, bytes from the row's first
    // (swizzled by the row's place among 32: the blocks of 32 rows are alike)
    static __device__ __forceinline__ int chunk(int c, int r) { return (c ^ ((r ^ ((r & 31) >> 3)) & 7)) << 4; }

    __device__ __forceinline__ void begin() {
        const int lane = threadIdx.x & 63;
        wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
        fw = wave & 3;
        rw = wave >> 2;
        clear();
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int at = (lane & 31) * ROW + chunk(2 * k + (lane >> 5), lane & 31);
            m_off[k] = 128 * rw * ROW + at;
            n_off[k] = 64 * fw * ROW + at;
        }
    }

    // Rows row0.. of h (`rows` in all) and v0.. of W (V).  DMA instruction j of a
    // wavefront: rows 8 (4 w + j)..; lane -> row lane / 8, physical chunk lane % 8.
    __device__ __forceinline__ void sources(const VocabOperand& h, const VocabOperand& W, int products, int64_t row0,
                                            int64_t rows, int64_t v0, int64_t V) {
        const int lane = fresh_lane();
        m_base = (const char*)(h.p + row0 * h.pitch);
        n_base = (const char*)(W.p + v0 * W.pitch);
        const int mr = (int)min(rows - row0, (int64_t)256), nr = (int)min(V - v0, (int64_t)256);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int r = 8 * (4 * wave + j) + (lane >> 3), c = chunk(lane & 7, r);
            m_at[j] = (uint32_t)min(r, mr - 1) * (uint32_t)(2 * h.pitch) + c;
            n_at[j] = (uint32_t)min(r, nr - 1) * (uint32_t)(2 * W.pitch) + c;
        }
        ip = 6 - products;
        ik = 0;
    }

    __device__ __forceinline__ void issue(char* ms, char* ns) {
        const int pm = (kPlaneM >> (2 * ip)) & 3, pn = (kPlaneN >> (2 * ip)) & 3;
        const char* m = m_base + pm * m_plane + (int64_t)ik * ROW;
        const char* n = n_base + pn * n_plane + (int64_t)ik * ROW;
#pragma unroll
        for (int j = 0; j < 4; ++j) load_lds16(m + m_at[j], ms + (4 * wave + j) * 1024);
#pragma unroll
        for (int j = 0; j < 4; ++j) load_lds16(n + n_at[j], ns + (4 * wave + j) * 1024);
        // past the last stage it is read again
        const bool end = ik + 1 == steps, turn = end && ip < 5;
        ik = turn ? 0 : ik + (end ? 0 : 1);
        ip += turn ? 1 : 0;
    }

    // Operands of half `h` of a stage: k 32 h + 16 ks + 8 (lane / 32)..
    __device__ __forceinline__ void read_frags(const char* ms, const char* ns, int h, Frags& f) const {
#pragma unroll
        for (int ks = 0; ks < 2; ++ks) {
#pragma unroll
            for (int mi = 0; mi < 2; ++mi)
                f.n[ks][mi] = __builtin_bit_cast(bf16x8_t, *(const u32x4_t*)(ns + n_off[2 * h + ks] + 32 * mi * ROW));
#pragma unroll
            for (int nj = 0; nj < NJ; ++nj)
                f.m[ks][nj] = __builtin_bit_cast(bf16x8_t, *(const u32x4_t*)(ms + m_off[2 * h + ks] + 32 * nj * ROW));
        }
    }

    __device__ __forceinline__ void mfmas(const Frags& f) {
#pragma unroll
        for (int ks = 0; ks < 2; ++ks)
#pragma unroll
            for (int nj = 0; nj < NJ; ++nj)
#pragma unroll
                for (int mi = 0; mi < 2; ++mi)
                    acc[mi][nj] =
                        __builtin_amdgcn_mfma_f32_32x32x16_bf16(f.n[ks][mi], f.m[ks][nj], acc[mi][nj], 0, 0, 0);
    }
    static __device__ __forceinline__ void fence() { __builtin_amdgcn_sched_barrier(0); }

    // The halves of a step around its wait and barrier.
    __device__ __forceinline__ void first(const Frags& fa, Frags& fb, const char* ms, const char* ns) {
        fence();
        read_frags(ms, ns, 1, fb);
        mfmas(fa);
#pragma unroll
        for (int i = 0; i < 12; ++i) {
            __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);   // MFMA
            __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);   // LDS read
        }
        fence();
    }
    __device__ __forceinline__ void second(Frags& fa, const Frags& fb, char* ms, char* ns, const char* mnext, const char* nnext) {
        fence();
        issue(ms, ns);
        read_frags(mnext, nnext, 0, fa);
        mfmas(fb);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);   // MFMA
            __builtin_amdgcn_sched_group_barrier(0x010, 1, 0);   // vector memory
            __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);   // LDS read
            __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
            __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
        }
        fence();
    }
};

struct WholeArgs {
    VocabOperand h, W;
    VocabRows rows;
    const float4* info;       // of compact rows: g / tau, lse, target (as bits)
    int64_t V, v0;
    int len, K, products;
    float scale;              // stats: log2(e) / tau; dz: 1 / tau
    float2* part;             // stats
    int64_t part_pitch;
    float* zt;                // stats, of compact rows
    uint16_t* dz;
    int64_t dz_pitch, dz_plane;
    float* err;
};

template <bool DZ, int PLANES>
__global__ __launch_bounds__(512, 1) void vocab_whole_kernel(const WholeArgs a, int n_tiles) {
    __shared__ __attribute__((aligned(1024))) char m0[Wide::BYTES];
    __shared__ __attribute__((aligned(1024))) char m1[Wide::BYTES];
    __shared__ __attribute__((aligned(1024))) char n0[Wide::BYTES];
    __shared__ __attribute__((aligned(1024))) char n1[Wide::BYTES];
    __shared__ __attribute__((aligned(1024))) float4 infos[256];
    __shared__ __attribute__((aligned(1024))) char extra[DZ ? 8 * 2048 : 4 * 256 * 8];   // dz on its way out, or the wavefronts' sums
    const int64_t rows = a.rows.count ? *a.rows.count : a.rows.T;
    const int m_tiles = (int)((rows + 255) / 256);
    // an XCD takes a contiguous range of tiles, its workgroups every 32nd of it;
    // 8 row tiles walk over the columns together
    constexpr int kRows = 8;
    const int total = m_tiles * n_tiles, xcd = blockIdx.x & 7;
    const int base = xcd * (total >> 3) + min(xcd, total & 7), count = (total >> 3) + (xcd < (total & 7) ? 1 : 0);
    int i = blockIdx.x >> 3;
    if (i >= count) return;

    Wide e;
    e.begin();
    int64_t row0, c0;
    auto place = [&](int i) {
        const int id = base + i, g = id / (kRows * n_tiles);
        const int in = min(kRows, m_tiles - g * kRows), r = id - g * kRows * n_tiles;
        const int nt = r / in;
        row0 = (int64_t)(g * kRows + (r - nt * in)) * 256;
        c0 = (int64_t)nt * TN;
    };
    auto sources = [&] { e.sources(a.h, a.W, a.products, row0, rows, a.v0 + c0, a.V); };
    e.m_plane = 2 * a.h.plane;
    e.n_plane = 2 * a.W.plane;
    e.steps = a.K / 64;
    place(i);
    sources();
    const int pairs = e.steps * a.products / 2;      // of steps
    // at a step's barrier the next stage has landed; right behind a tile's epilogue
    // its stores may still be on their way
    constexpr int after = DZ ? 16 * PLANES : 0;
    auto ready = [](bool early) {
        if (early) __builtin_amdgcn_s_waitcnt(waitcnt_imm(after, 0));
        else __builtin_amdgcn_s_waitcnt(waitcnt_imm(0, 0));
        __builtin_amdgcn_s_barrier();
    };

    Wide::Frags fa, fb;
    e.issue(m0, n0);
    e.issue(m1, n1);
    ready(false);
    Wide::fence();
    e.read_frags(m0, n0, 0, fa);
    for (;;) {
        const int64_t tile_row = row0, tile_col = c0;
        const bool more = i + 32 < count;
        i += 32;
        for (int g = 0; g < pairs; ++g) {
            e.first(fa, fb, m0, n0);
            ready(g == 0);
            if (g == 0) {
                // 64 rows a wavefront (twice over)
                const int r = 64 * (e.wave & 3);
                const int in = min(fresh_lane(), (int)min(rows - 1 - tile_row - r, (int64_t)63));
                load_lds16(a.info + tile_row + r + in, (char*)infos + 16 * r);
            }
            // the next tile's sources, once this one's last stage is on its way
            if (g + 1 == pairs && more) {
                place(i);
                sources();
            }
            e.second(fa, fb, m0, n0, m1, n1);
            e.first(fa, fb, m1, n1);
            ready(false);
            e.second(fa, fb, m1, n1, m0, n0);
        }

        // ---- epilogue.  Element v of acc[mi][nj] on lane l: row 128 rw + 32 nj +
        // l % 32, column 64 fw + 32 mi + 8 (v / 4) + 4 (l / 32) + v % 4.
        const int lane = fresh_lane();
        const int l = lane & 31, half = lane >> 5;
        const int64_t v0 = a.v0 + tile_col;
        const int left = (int)min(a.v0 + a.len - v0, (int64_t)TN) - 64 * e.fw - 4 * half;
#pragma unroll
        for (int nj = 0; nj < 4; ++nj) {
            const int r = 128 * e.rw + 32 * nj + l;
            const float4 in = infos[r];
            const int64_t row = tile_row + r;
            const int target = (int)__float_as_uint(in.z) - (int)v0 - 64 * e.fw - 4 * half;   // its column here
            const bool mine = __float_as_int(in.z) >= 0 && target >= -4 && target < 64;
            const bool any = __ballot(mine);
            if constexpr (DZ) {
#pragma unroll
                for (int mi = 0; mi < 2; ++mi)
#pragma unroll
                    for (int v = 0; v < 16; ++v)
                        e.acc[mi][nj][v] = softmax_of<PLANES>(fmaf(e.acc[mi][nj][v], a.scale, -in.y));
                if (any) {
#pragma unroll
                    for (int mi = 0; mi < 2; ++mi)
#pragma unroll
                        for (int v = 0; v < 16; ++v)
                            if (mine && target == 32 * mi + 8 * (v / 4) + v % 4) e.acc[mi][nj][v] -= 1.f;
                }
#pragma unroll
                for (int mi = 0; mi < 2; ++mi)
#pragma unroll
                    for (int v = 0; v < 16; ++v) e.acc[mi][nj][v] *= in.x;
                if (PLANES == 1 && any && a.err) {
                    const float x = column(e.acc[0][nj], e.acc[1][nj], target);
                    if (mine && has_column(target) && row < rows) a.err[row] = rounding_of(x);
                }
                if (left < 64) {
#pragma unroll
                    for (int mi = 0; mi < 2; ++mi)
#pragma unroll
                        for (int v = 0; v < 16; ++v)
                            if (32 * mi + 8 * (v / 4) + v % 4 >= left) e.acc[mi][nj][v] = 0.f;
                }
                // Through LDS, 16 rows of 128 bytes of the wavefront's own at a time
                // (16-byte chunks XOR-swizzled by the row), so that a store writes
                // whole lines (half lines, 131072 bytes apart: 1415 us against 1150).
                char* own = extra + 2048 * e.wave;
                const int sr = lane >> 3, sc = lane & 7;
                uint16_t* out = a.dz + (tile_row + 128 * e.rw + 32 * nj + sr) * a.dz_pitch + tile_col + 64 * e.fw + 8 * sc;
                // rows behind the last are computed as the last, and stored as it
                const int behind = (int)min(rows - 1 - (tile_row + 128 * e.rw + 32 * nj + sr), (int64_t)32);
#pragma unroll
                for (int pl = 0; pl < PLANES; ++pl) {
                    uint2 p[2][4];
#pragma unroll
                    for (int mi = 0; mi < 2; ++mi)
#pragma unroll
                        for (int vg = 0; vg < 4; ++vg) {
                            f32x16_t& x = e.acc[mi][nj];
                            const uint32_t lo = pack_bf16(x[4 * vg], x[4 * vg + 1]), hi = pack_bf16(x[4 * vg + 2], x[4 * vg + 3]);
                            p[mi][vg] = make_uint2(lo, hi);
                            if (pl + 1 < PLANES) {
                                x[4 * vg] -= __uint_as_float(lo << 16);
                                x[4 * vg + 1] -= __uint_as_float(lo & 0xffff0000u);
                                x[4 * vg + 2] -= __uint_as_float(hi << 16);
                                x[4 * vg + 3] -= __uint_as_float(hi & 0xffff0000u);
                            }
                        }
#pragma unroll
                    for (int part = 0; part < 2; ++part) {
                        if (l >> 4 == part) {
#pragma unroll
                            for (int mi = 0; mi < 2; ++mi)
#pragma unroll
                                for (int vg = 0; vg < 4; ++vg)
                                    *(uint2*)(own + (l & 15) * 128 + (((4 * mi + vg) ^ (l & 7)) << 4) + 8 * half) = p[mi][vg];
                        }
                        wave_sync();       // half the lanes wrote what all of them read
#pragma unroll
                        for (int q = 0; q < 2; ++q) {
                            const int r = 16 * part + 8 * q;
                            const u32x4_t v = *(const u32x4_t*)(own + (8 * q + sr) * 128 + ((sc ^ sr) << 4));
                            // non-temporal: the tiles keep their L2 (1% of the whole backward)
                            __builtin_nontemporal_store(
                                v, (u32x4_t*)(out + pl * a.dz_plane + min(r, behind) * a.dz_pitch));
                        }
                        wave_sync();
                    }
                }
            } else {
                if (any) {
                    const float z = column(e.acc[0][nj], e.acc[1][nj], target);
                    if (mine && has_column(target) && row < rows) a.zt[row] = z;
                }
                if (left < 64) {
#pragma unroll
                    for (int mi = 0; mi < 2; ++mi)
#pragma unroll
                        for (int v = 0; v < 16; ++v)
                            if (32 * mi + 8 * (v / 4) + v % 4 >= left) e.acc[mi][nj][v] = -INFINITY;
                }
                const float2 s = row_stats(e.acc[0][nj], e.acc[1][nj], a.scale);
                if (half == 0) ((float2*)extra)[256 * e.fw + r] = s;
            }
        }
        if constexpr (!DZ) {
            // LDS alone is waited for: the next tile's stages stay in flight
            __builtin_amdgcn_s_waitcnt(waitcnt_imm(63, 0));
            __builtin_amdgcn_s_barrier();
            const int r = 64 * e.wave + lane;
            if (r < 256 && tile_row + r < rows) {
                float2 p[4];
#pragma unroll
                for (int w = 0; w < 4; ++w) p[w] = ((const float2*)extra)[256 * w + r];
                a.part[tile_col / TN * a.part_pitch + tile_row + r] = join_stats(p);
            }
        }
        if (!more) return;
        e.clear();
    }
}

// The gradients' products run on one workgroup per CU.  Where the tiles of all K
// steps fill the CUs well enough, each workgroup takes whole ones (of a last round
// that is no more than half full, 128 of the rows each: dW of 1000 x 8000 x 1024 37
// -> 29 us, of 512 x 32768 x 768 45 -> 41) and they go straight out.  Else the steps
// are shared out: a team of workgroups takes the column tiles of the same 256 rows
// side by side, so that they read the M operand once through their XCD's L2, and
// writes its parts of tiles, which a second kernel adds in order.  For dW each team
// first takes as many whole tiles as there are for all: the teams go through K
// together and read the same of h, which the L2s then hold.  Of what remains, where
// its row tiles divide the teams well, each team has a range of the steps of one, the
// teams of one range next to each other; else the teams share out its steps evenly,
// each a contiguous range of them: at most one part that it does not begin and one
// that it does not end, and whole tiles between.  Against the even shares alone, in
// teams for whole tiles too, of 768 columns: dh of 512 rows and 32768 entries 47 -> 37
// us, dW of 512 and 65536 100 -> 68.
constexpr int kGradUnits = 256;

struct GradWork {
    int m_tiles, n_tiles, teams;
    int steps;                // K steps of one product
    int virt;                 // of a tile: those of all products, at least 1
    int per;                  // of a team
    bool split;               // tiles are divided between teams, from tile `shared` on
    bool even;                // ... evenly, else range by range
    bool halves;              // not split: those of the last round are, by rows
    int gain;                 // steps that dividing saves
    int rounds, shared;       // whole tiles of a team before, of all teams
};

__host__ __device__ __forceinline__ GradWork grad_work(const VocabGrad& a, int64_t rows) {
    GradWork w;
    const int64_t M = a.dW ? a.len : rows;
    const int K = a.dW ? (int)rows : a.len;
    w.m_tiles = (int)((M + 255) / 256);
    w.n_tiles = (a.N + TN - 1) / TN;
    w.teams = kGradUnits / w.n_tiles;
    w.steps = (K + BK - 1) / BK;
    w.virt = w.steps ? w.steps * a.products : 1;
    // (dh gains nothing from whole tiles first: 32768 x 768 x 65536 2640 us against
    // 2553, dW 2520 against 2578)
    w.rounds = a.dW ? w.m_tiles / w.teams : 0;
    w.shared = w.rounds * w.teams;
    const int rest = w.m_tiles - w.shared;
    // parts cost what their write and their sum take, about 32 steps (measured from 4 to
    // 40: 512 to 9000 rows, even between 20 and 40)
    const int even = (int)(((int64_t)rest * w.virt + w.teams - 1) / w.teams);
    // half a tile takes about three quarters of a whole one's time (fp32 dW of 1000 x
    // 16001 x 512, 126 tiles: in halves 113 us, divided 107)
    const int tiles = w.m_tiles * w.n_tiles, left = tiles % kGradUnits;
    w.halves = a.halves && 0 < left && 2 * left <= kGradUnits;
    const int whole = tiles / kGradUnits * w.virt + (w.halves ? (3 * w.virt + 3) / 4 : left ? w.virt : 0);
    w.gain = whole - w.rounds * w.virt - even;
    w.split = w.gain > 32;
    // ranges, unless they leave more than an eighth of the teams without work
    const int ranges = rest && rest <= w.teams ? w.teams / rest : 1;
    const int range = (w.virt + ranges - 1) / ranges;
    w.even = rest > w.teams || range > even + even / 8;
    const int per = w.even ? even : range;
    w.per = per > 8 ? per : 8;
    return w;
}

// A workgroup's part of the work: steps k0 to k1 of a tile.
struct GradPart {
    int mt, nt, k0, k1;
    int half;                 // the 128 rows of the tile that are wanted; -1: all
    int round;                // those taken so far; below 0: none
    int at;                   // the first step of the next part (even)
};

// The workgroup's first (round < 0) or next part; false: none.
__device__ __forceinline__ bool grad_next(const GradWork& w, int place, GradPart& p) {
    ++p.round;
    p.k0 = 0;
    p.k1 = w.virt;
    p.half = -1;
    if (!w.split) {
        int tile = place + p.round * kGradUnits;
        const int last = w.m_tiles * w.n_tiles / kGradUnits;
        if (w.halves && p.round >= last) {
            p.half = place & 1;
            tile = p.round > last ? w.m_tiles * w.n_tiles : last * kGradUnits + (place >> 1);
        }
        p.mt = tile / w.n_tiles;
        p.nt = tile - p.mt * w.n_tiles;
        return p.mt < w.m_tiles;
    }
    const int team = place / w.n_tiles;
    if (team >= w.teams) return false;
    p.nt = place - team * w.n_tiles;
    if (p.round < w.rounds) {
        p.mt = p.round * w.teams + team;
        return true;
    }
    const int rest = w.m_tiles - w.shared;
    if (!w.even) {
        const int range = team / rest;
        p.mt = w.shared + team - range * rest;
        p.k0 = range * w.per;
        p.k1 = min(w.virt, p.k0 + w.per);
        return p.round == w.rounds && p.k0 < w.virt;
    }
    if (p.round == w.rounds) p.at = team * w.per;
    const int end = min((team + 1) * w.per, rest * w.virt);
    if (p.at >= end) return false;
    p.mt = p.at / w.virt;
    p.k0 = p.at - p.mt * w.virt;
    p.k1 = min(w.virt, p.k0 + (end - p.at));
    p.at += p.k1 - p.k0;
    p.mt += w.shared;
    return true;
}

// Where a team's part of a tile goes: [256][256] fp32; slot 1 if the team begins
// a tile that it shares with the next.
__device__ __forceinline__ float* grad_part(const VocabGrad& a, const GradWork& w, int team, int slot, int nt) {
    return a.partial + (((int64_t)team * 2 + slot) * w.n_tiles + nt) * 65536;
}

// Four columns n0.. of row m on their way out.
__device__ __forceinline__ void grad_out(const VocabGrad& a, int64_t m, int n0, float4 v) {
    if (a.acc && n0 < a.acc_pitch) {
        float4* p = (float4*)(a.acc + m * a.acc_pitch + n0);
        if (a.add) {
            const float4 o = *p;
            v.x += o.x, v.y += o.y, v.z += o.z, v.w += o.w;
        }
        if (!a.last) *p = v;
    }
    if (!a.last || n0 >= a.N) return;
    if (!a.dW && a.err) {
        const int entry = a.entry[m];
        if (entry >= 0) {
            const float e = a.err[m];
            const uint2 w = *(const uint2*)(a.table + (int64_t)entry * a.table_pitch + n0);
            v.x = fmaf(e, __uint_as_float(w.x << 16), v.x), v.y = fmaf(e, __uint_as_float(w.x & 0xffff0000u), v.y);
            v.z = fmaf(e, __uint_as_float(w.y << 16), v.z), v.w = fmaf(e, __uint_as_float(w.y & 0xffff0000u), v.w);
        }
    }
    const int64_t at = (!a.dW && a.rows.rows ? (int64_t)a.rows.rows[m] : m) * a.N + n0;
    if (a.N % 4 == 0) {
        if (a.out_bf16)
            *(uint2*)((uint16_t*)a.out + at) = make_uint2(pack_bf16(v.x, v.y), pack_bf16(v.z, v.w));
        else
            *(float4*)((float*)a.out + at) = v;
        return;
    }
    const float x[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int q = 0; q < 4; ++q)
        if (n0 + q < a.N) {
            if (a.out_bf16)
                ((uint16_t*)a.out)[at + q] = (uint16_t)pack_bf16(x[q], 0.f);
            else
                ((float*)a.out)[at + q] = x[q];
        }
}

// DW: both operands are k rows of columns; else M is K-contiguous.  A part's first
// three stages are loaded under the epilogue of the one before.
// HALVES: see GradWork; apart, since the large products lose 1% by it.
template <bool DW, bool HALVES>
__global__ __launch_bounds__(512, 1) void vocab_grad_kernel(const VocabGrad a) {
    using Eng = Engine<!DW, false, 256>;
    __shared__ __attribute__((aligned(1024))) char st0[Eng::SBYTES];
    __shared__ __attribute__((aligned(1024))) char st1[Eng::SBYTES];
    __shared__ __attribute__((aligned(1024))) char st2[Eng::SBYTES];
    __shared__ __attribute__((aligned(1024))) char st3[Eng::SBYTES];
    __shared__ __attribute__((aligned(1024))) char out_[8 * 4096];
    const int64_t rows = a.rows.count ? *a.rows.count : a.rows.T;
    const GradWork w = grad_work(a, rows);
    // 32 consecutive places on an XCD
    const int place = (blockIdx.x & 7) * (kGradUnits / 8) + (blockIdx.x >> 3);
    const int64_t M = DW ? a.len : rows;
    const int last = ((DW ? (int)rows : a.len) - 1) % BK + 1;
    GradPart now;
    now.round = -1;
    if (!grad_next(w, place, now)) return;

    Eng e;
    e.begin();
    e.steps = w.steps;
    e.m_plane = 2 * a.m.plane;
    e.n_plane = 2 * a.n.plane;
    auto start = [&] {
        if (!w.steps) return;
        const int64_t row0 = (int64_t)now.mt * 256;
        e.ip = 6 - a.products + now.k0 / w.steps;
        e.ik = now.k0 % w.steps;
        if constexpr (DW) {
            e.m_base = (const char*)(a.m.p + row0);      // dz's rows are whole tiles
            e.m_ks(last, 2 * a.m.pitch);
        } else {
            e.m_base = (const char*)(a.m.p + row0 * a.m.pitch);
            e.m_rows((int)min(M - row0, (int64_t)256), 2 * a.m.pitch);
        }
        // k rows past the last: zeros behind h (dW), any of the table's against
        // dz's zeros (dh)
        e.n_base = (const char*)(a.n.p + now.nt * TN);
        e.n_ks(DW ? BK : last, 2 * a.n.pitch, (int)a.n.pitch - now.nt * TN);
        e.issue(st0);
        e.issue(st1);
        e.issue(st2);
    };
    start();
    __builtin_amdgcn_s_waitcnt(waitcnt_imm(0, 15));
    for (;;) {
        __builtin_amdgcn_s_barrier();
        const bool mine = !HALVES || now.half < 0 || now.half == e.rw;
        if (w.steps) {
            if (mine) e.run(now.k1 - now.k0, st0, st1, st2, st3);
            else e.idle(now.k1 - now.k0, st0, st1, st2, st3);
        }
        const GradPart was = now;
        const bool more = grad_next(w, place, now);
        if (more) start();
        if (!mine) {
            if (!more) return;
            __builtin_amdgcn_s_waitcnt(waitcnt_imm(0, 15));
            continue;
        }

        // Through LDS, 16 rows of the wavefront's 64 columns at a time (16-byte chunks
        // XOR-swizzled by the row), so that stores write whole lines.
        const int64_t row0 = (int64_t)was.mt * 256;
        float* part = nullptr;
        if (was.k1 - was.k0 < w.virt) part = grad_part(a, w, place / w.n_tiles, w.even && was.k0 == 0, was.nt);
        const int lane = fresh_lane(), l = lane & 31, half = lane >> 5, sr = lane >> 4, sc = lane & 15;
        char* own = out_ + 4096 * e.wave;
        const int n0 = was.nt * TN + 64 * e.fw + 4 * sc;
        const bool plain = DW && a.N % 4 == 0;
#pragma unroll
        for (int nj = 0; nj < 4; ++nj)
#pragma unroll 1
            for (int p = 0; p < 2; ++p) {      // kept small: the instructions are fetched as they run
                if (l >> 4 == p) {
#pragma unroll
                    for (int mi = 0; mi < 2; ++mi)
#pragma unroll
                        for (int vg = 0; vg < 4; ++vg) {
                            const f32x16_t& v = e.acc[mi][nj];
                            *(float4*)(own + (l & 15) * 256 + (((8 * mi + 2 * vg + half) ^ (l & 15)) << 4)) =
                                make_float4(v[4 * vg], v[4 * vg + 1], v[4 * vg + 2], v[4 * vg + 3]);
                        }
                }
                wave_sync();       // half the lanes wrote what all of them read
                // the next part's stages have landed, before more stores than can be counted
                if (nj == 2) __builtin_amdgcn_s_waitcnt(waitcnt_imm(0, 15));
                const int tr = 128 * e.rw + 32 * nj + 16 * p + sr;
                auto sum = [&](int q) { return *(const float4*)(own + (4 * q + sr) * 256 + ((sc ^ (4 * q + sr)) << 4)); };
                if (part) {
#pragma unroll
                    for (int q = 0; q < 4; ++q) *(float4*)(part + (tr + 4 * q) * 256 + 64 * e.fw + 4 * sc) = sum(q);
                } else if (plain) {
                    const int64_t at = (row0 + tr) * a.N + n0;
                    const int behind = n0 < a.N ? (int)min(M - row0 - tr, (int64_t)16) : 0;
                    if (a.out_bf16) {
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            const float4 v = sum(q);
                            if (4 * q < behind)
                                *(uint2*)((uint16_t*)a.out + at + 4 * q * a.N) = make_uint2(pack_bf16(v.x, v.y), pack_bf16(v.z, v.w));
                        }
                    } else {
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            const float4 v = sum(q);
                            if (4 * q < behind) *(float4*)((float*)a.out + at + 4 * q * a.N) = v;
                        }
                    }
                } else {
#pragma unroll 1
                    for (int q = 0; q < 4; ++q)
                        if (row0 + tr + 4 * q < M) grad_out(a, row0 + tr + 4 * q, n0, sum(q));
                }
                wave_sync();
            }
        if (!more) return;
        e.clear();
    }
}

// The tiles that more than one team made.  MANY (few row tiles, each of many
// parts): a row a workgroup, its wavefronts over every fourth part and then over
// the four; else 32 rows a workgroup, 8 a wavefront.
template <bool MANY>
__global__ __launch_bounds__(256) void vocab_grad_sum_kernel(const VocabGrad a) {
    __shared__ float4 sums[MANY ? 4 : 1][64];
    constexpr int PER = MANY ? 256 : 8;        // workgroups of a tile
    const int64_t rows = a.rows.count ? *a.rows.count : a.rows.T;
    const GradWork w = grad_work(a, rows);
    const int slab = blockIdx.x % PER, tile = blockIdx.x / PER;
    const int mt = tile / w.n_tiles, nt = tile - mt * w.n_tiles;
    if (mt >= w.m_tiles) return;
    const int64_t M = a.dW ? a.len : rows;
    if (!w.split || mt < w.shared) return;
    // the tile's parts
    const int of = mt - w.shared, rest = w.m_tiles - w.shared;
    const int t0 = w.even ? of * w.virt / w.per : 0;
    const int parts = w.even ? ((of + 1) * w.virt - 1) / w.per - t0 + 1 : (w.virt + w.per - 1) / w.per;
    if (parts == 1) return;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, n0 = nt * TN + 4 * lane;
    auto part = [&](int t, int tr) {
        const float* p = w.even ? grad_part(a, w, t0 + t, t == 0, nt) : grad_part(a, w, t * rest + of, 0, nt);
        return *(const float4*)(p + tr * 256 + 4 * lane);
    };
    auto add = [](float4& v, float4 o) { v.x += o.x, v.y += o.y, v.z += o.z, v.w += o.w; };
    if constexpr (MANY) {
        const int64_t m = (int64_t)mt * 256 + slab;
        if (m >= M) return;
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
        for (int t = wave; t < parts; t += 4) add(v, part(t, slab));
        sums[wave][lane] = v;
        __syncthreads();
        if (wave || n0 >= a.N) return;
#pragma unroll
        for (int q = 1; q < 4; ++q) add(v, sums[q][lane]);
        grad_out(a, m, n0, v);
    } else {
        if (n0 >= a.N) return;
#pragma unroll 2
        for (int i = 0; i < 8; ++i) {
            const int tr = 32 * slab + 4 * i + wave;
            const int64_t m = (int64_t)mt * 256 + tr;
            if (m >= M) break;
            float4 v = part(0, tr);
#pragma unroll 4
            for (int t = 1; t < parts; ++t) add(v, part(t, tr));
            grad_out(a, m, n0, v);
        }
    }
}

}  // namespace

hipError_t launch_vocab_stats(const VocabStats& a, hipStream_t s) {
    if (a.K <= 0 || a.K % BK || (a.products != 1 && a.products != 6) || a.rows.T <= 0 || a.V <= 0) return hipErrorInvalidValue;
    const int n_tiles = (int)((a.V + TN - 1) / TN);
    const int64_t tiles = (a.rows.T + 127) / 128 * n_tiles;
    if (tiles > kMaxTiles) return hipErrorInvalidValue;
    vocab_stats_kernel<<<grid_for_work(tiles), 256, 0, s>>>(a, n_tiles);
    return hipGetLastError();
}

hipError_t launch_vocab_dz(const VocabDz& a, hipStream_t s) {
    if (a.K <= 0 || a.K % BK || (a.products != 1 && a.products != 6) || a.rows.T <= 0 || a.len <= 0) return hipErrorInvalidValue;
    const int n_tiles = (a.len + TN - 1) / TN;
    if ((int64_t)n_tiles * TN > a.dz_pitch) return hipErrorInvalidValue;
    const int64_t tiles = (a.rows.T + 127) / 128 * n_tiles;
    if (tiles > kMaxTiles) return hipErrorInvalidValue;
    if (a.products == 1) vocab_dz_kernel<1><<<grid_for_work(tiles), 256, 0, s>>>(a, n_tiles);
    else vocab_dz_kernel<3><<<grid_for_work(tiles), 256, 0, s>>>(a, n_tiles);
    return hipGetLastError();
}

hipError_t launch_vocab_stats_whole(const VocabStats& a, const float4* info, hipStream_t s) {
    if (a.K <= 0 || a.K % (4 * BK) || (a.products != 1 && a.products != 6) || a.rows.T <= 0 || a.V <= 0 || !info) return hipErrorInvalidValue;
    const int64_t n_tiles = (a.V + TN - 1) / TN;
    if ((a.rows.T + 255) / 256 * n_tiles > kMaxTiles) return hipErrorInvalidValue;
    const WholeArgs w = {a.h, a.W, a.rows, info, a.V, 0, (int)a.V, a.K, a.products, a.c, a.part, a.part_pitch, a.zt, nullptr, 0, 0, nullptr};
    vocab_whole_kernel<false, 1><<<kWholeUnits, 512, 0, s>>>(w, (int)n_tiles);
    return hipGetLastError();
}

hipError_t launch_vocab_dz_whole(const VocabDz& a, const float4* info, hipStream_t s) {
    if (a.K <= 0 || a.K % (4 * BK) || (a.products != 1 && a.products != 6) || a.rows.T <= 0 || a.len <= 0 || !info) return hipErrorInvalidValue;
    const int64_t n_tiles = ((int64_t)a.len + TN - 1) / TN;
    if (n_tiles * TN > a.dz_pitch || (a.rows.T + 255) / 256 * n_tiles > kMaxTiles) return hipErrorInvalidValue;
    const WholeArgs w = {a.h, a.W, a.rows, info, a.V, a.v0, a.len, a.K, a.products, a.inv_tau, nullptr, 0, nullptr, a.dz, a.dz_pitch, a.dz_plane, a.err};
    if (a.products == 1) vocab_whole_kernel<true, 1><<<kWholeUnits, 512, 0, s>>>(w, (int)n_tiles);
    else vocab_whole_kernel<true, 3><<<kWholeUnits, 512, 0, s>>>(w, (int)n_tiles);
    return hipGetLastError();
}

size_t vocab_grad_partial_bytes(int N) {
    const int n_tiles = (N + TN - 1) / TN;
    return (size_t)(kGradUnits / n_tiles) * 2 * n_tiles * 65536 * 4;
}

hipError_t launch_vocab_grad(const VocabGrad& a, hipStream_t s) {
    if ((a.products != 1 && a.products != 6) || a.rows.T <= 0 || a.len <= 0 || a.N <= 0 || a.N > kGradUnits * TN ||
        a.n.pitch % BK || a.m.pitch % TN || a.n.pitch < a.N || !a.partial || ((a.add || !a.last) && !a.acc))
        return hipErrorInvalidValue;
    const int64_t tiles = vocab_grad_tiles(a.dW ? a.len : a.rows.T, a.N);
    if (tiles > kVocabGradTiles) return hipErrorInvalidValue;
    VocabGrad b = a;
    b.halves = a.dW || !a.rows.count;
    GradWork w = grad_work(b, a.rows.T);
    b.halves = w.halves && !w.split;
    if (b.halves) {
        if (a.dW) vocab_grad_kernel<true, true><<<kGradUnits, 512, 0, s>>>(b);
        else vocab_grad_kernel<false, true><<<kGradUnits, 512, 0, s>>>(b);
    } else {
        if (a.dW) vocab_grad_kernel<true, false><<<kGradUnits, 512, 0, s>>>(b);
        else vocab_grad_kernel<false, false><<<kGradUnits, 512, 0, s>>>(b);
    }
    if (hipError_t e = hipGetLastError()) return e;
    // with the rows known here, or more of them than there can be (dW: fewer rows
    // are fewer steps, which gain less by being divided, but for the rounding of two
    // quotients), tiles that are whole need no sum
    w = grad_work(b, a.rows.T);
    if (!a.rows.count ? !w.split : a.dW && w.gain <= 30) return hipSuccess;
    if (w.m_tiles * 8 <= w.teams) vocab_grad_sum_kernel<true><<<(unsigned)(tiles * 256), 256, 0, s>>>(b);
    else vocab_grad_sum_kernel<false><<<(unsigned)(tiles * 8), 256, 0, s>>>(b);
    return hipGetLastError();
}

}  // namespace moe
