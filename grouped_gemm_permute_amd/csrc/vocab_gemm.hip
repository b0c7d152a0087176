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
// Tile engine (that of gemm_bf16.hip, with either layout of each operand): K
// steps of 32, operands global -> LDS with 16-byte DMA into a ring of stages,
// the next step's fragments read from LDS under this step's MFMAs.  The MFMA's
// A operand is 32 columns of N, its B operand 32 rows of M, so that a lane ends
// with 4 consecutive columns of one row.
//  * stats and dz: 128 rows x 256 entries, 4 wavefronts, 3 stages of 24 KiB, two
//    workgroups a CU: the exponentials of one (quarter rate, 128 a lane) run
//    under the other's MFMAs;
//  * grad: 256 x 256, 8 wavefronts, 4 stages of 32 KiB; K is long, the epilogue
//    small.
#include "mfma_common.h"
#include "vocab_internal.h"

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

// What an N operand's k rows past its last one are read as.
__device__ __attribute__((aligned(16))) u32x4_t zero_chunk[1];

// The products of planes, smallest first: (1,1) (2,0) (0,2) (1,0) (0,1) (0,0),
// two bits each; one product alone is the last.
constexpr int kPlaneM = 1 | 2 << 2 | 0 << 4 | 1 << 6 | 0 << 8 | 0 << 10;
constexpr int kPlaneN = 1 | 0 << 2 | 2 << 4 | 0 << 6 | 1 << 8 | 0 << 10;

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

    // What a lane's loads read: for a K-contiguous operand the addresses of its
    // rows' chunks, else of its column chunk in k row 0.
    const char* m_src[MJ];
    const char* n_src[WJ];
    int64_t m_plane, n_plane;         // bytes between planes
    int64_t m_pitch, n_pitch;         // bytes between k rows
    int k_m, k_n;                     // k rows that exist (not K-contiguous operands)
    int steps, kt_total;              // K steps of a product and of all
    int ik, ip;                       // the next stage: its step, its product
    int lane, wave, fw, rw;
    int m_off[NJ][2], n_off[2][2];    // fragment offsets in a stage

    f32x16_t acc[2][NJ];

    struct Frags {
        bf16x8_t n[2][2], m[2][NJ];
    };

    __device__ __forceinline__ void begin() {
        const int tid = threadIdx.x;
        lane = tid & 63;
        wave = __builtin_amdgcn_readfirstlane(tid >> 6);
        fw = wave & 3;
        rw = wave >> 2;
#pragma unroll
        for (int mi = 0; mi < 2; ++mi)
#pragma unroll
            for (int nj = 0; nj < NJ; ++nj) acc[mi][nj] = f32x16_t{};
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

    __device__ __forceinline__ void issue(char* st) {
        const int pm = (kPlaneM >> (2 * ip)) & 3, pn = (kPlaneN >> (2 * ip)) & 3;
        const int64_t om = pm * m_plane, on = pn * n_plane;
#pragma unroll
        for (int j = 0; j < MJ; ++j) {
            const char* p;
            if constexpr (MC) {
                p = m_src[j] + (om + (int64_t)ik * KC_ROW);
            } else {
                const uint32_t k = min(ik * BK + ks_row(j, MJ), k_m - 1);
                p = m_src[j] + om + (uint64_t)k * (uint32_t)m_pitch;
            }
            load_lds16(p, st + (MJ * wave + j) * 1024);
        }
#pragma unroll
        for (int j = 0; j < WJ; ++j) {
            const char* p;
            if constexpr (NC) {
                p = n_src[j] + (on + (int64_t)ik * KC_ROW);
            } else {
                const int k = ik * BK + ks_row(j, WJ);
                const char* row = n_src[j] + on + (uint64_t)(uint32_t)min(k, k_n - 1) * (uint32_t)n_pitch;
                // opaque, so that the product does not move into a branch
                asm volatile("" : "+v"(row));
                p = k < k_n ? row : (const char*)zero_chunk;
            }
            load_lds16(p, st + M_BYTES + (WJ * wave + j) * 1024);
        }
        // the next stage; past the last one it is read again, into a buffer
        // that is never computed on, so that the loads in flight can be counted
        if (ik + 1 < steps) {
            ++ik;
        } else if (ip < 5) {
            ++ip;
            ik = 0;
        }
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

    // All K steps; on return no load is in flight and every wavefront has read
    // the stages.
    __device__ __forceinline__ void run(char* st0, char* st1, char* st2, char* st3) {
        if (kt_total <= 0) return;
        Frags fa, fb;
        issue(st0);
        issue(st1);
        if constexpr (NS == 4) issue(st2);
        __builtin_amdgcn_s_waitcnt(waitcnt_imm((NS - 2) * PER_STAGE, 15));
        __builtin_amdgcn_s_barrier();
        fence();
        read_frags(st0, fa);
        fence();
        int kt = 0;
        const int KT = kt_total;
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

// h's rows and W's rows of a logits tile.
__device__ __forceinline__ void logits_sources(Logits& e, const VocabOperand& h, const VocabOperand& W, int products,
                                               int K, int64_t row0, int64_t rows, const int32_t* gather, int64_t v0,
                                               int64_t V) {
    int64_t r[Logits::MJ];
#pragma unroll
    for (int j = 0; j < Logits::MJ; ++j) r[j] = min(row0 + e.kc_row(j, Logits::MJ), rows - 1);
    if (gather) {
#pragma unroll
        for (int j = 0; j < Logits::MJ; ++j) r[j] = gather[r[j]];
    }
#pragma unroll
    for (int j = 0; j < Logits::MJ; ++j)
        e.m_src[j] = (const char*)(h.p + r[j] * h.pitch + 8 * e.kc_chunk(e.kc_row(j, Logits::MJ)));
#pragma unroll
    for (int j = 0; j < Logits::WJ; ++j) {
        const int row = e.kc_row(j, Logits::WJ);
        const int64_t v = min(v0 + row, V - 1);
        e.n_src[j] = (const char*)(W.p + v * W.pitch + 8 * e.kc_chunk(row));
    }
    e.m_plane = 2 * h.plane;
    e.n_plane = 2 * W.plane;
    e.steps = K / BK;
    e.ip = 6 - products;
    e.ik = 0;
    e.kt_total = e.steps * products;
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
    logits_sources(e, a.h, a.W, a.products, a.K, row0, rows, a.gather ? a.rows.rows : nullptr, v0, a.V);
    e.run(st0, st1, st2, nullptr);

    const int l = e.lane & 31, half = e.lane >> 5;
    const int left = (int)min(a.V - v0, (int64_t)TN);
    float2* tile = (float2*)st0;                              // [4][128]
#pragma unroll
    for (int nj = 0; nj < 4; ++nj) {
        const int64_t row = row0 + 32 * nj + l;
        // the target's logit, where it is among this wavefront's 64 columns
        if (a.target) {
            const int64_t t = row < rows ? (a.rows.rows ? a.rows.rows[row] : row) : 0;
            const int64_t target = row < rows ? a.target[t] : -1;
            const bool mine = target >= v0 + 64 * e.fw && target < min(v0 + 64 * e.fw + 64, a.V);
            if (__ballot(mine)) {
                const int at = mine ? (int)(target - v0) - 64 * e.fw - 4 * half : -1;
#pragma unroll
                for (int mi = 0; mi < 2; ++mi)
#pragma unroll
                    for (int v = 0; v < 16; ++v)
                        if (at == 32 * mi + 8 * (v / 4) + v % 4) a.zt[t] = e.acc[mi][nj][v];
            }
        }
        if (left < TN) {
#pragma unroll
            for (int mi = 0; mi < 2; ++mi)
#pragma unroll
                for (int v = 0; v < 16; ++v)
                    if (64 * e.fw + 32 * mi + 8 * (v / 4) + 4 * half + v % 4 >= left) e.acc[mi][nj][v] = -INFINITY;
        }
        float top = -INFINITY;
#pragma unroll
        for (int mi = 0; mi < 2; ++mi)
#pragma unroll
            for (int v = 0; v < 16; ++v) top = fmaxf(top, e.acc[mi][nj][v]);
        top = fmaxf(top, __shfl_xor(top, 32));
        top *= a.c;
        const float off = top == -INFINITY ? 0.f : top;
        float sum = 0.f;
#pragma unroll
        for (int mi = 0; mi < 2; ++mi)
#pragma unroll
            for (int v = 0; v < 16; ++v) sum += __builtin_amdgcn_exp2f(fmaf(e.acc[mi][nj][v], a.c, -off));
        sum += __shfl_xor(sum, 32);
        if (half == 0) tile[e.fw * 128 + 32 * nj + l] = make_float2(top, sum);
    }
    __syncthreads();
    const int r = threadIdx.x;
    if (r < 128 && row0 + r < rows) {
        float2 p[4];
        float top = -INFINITY;
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            p[w] = tile[w * 128 + r];
            top = fmaxf(top, p[w].x);
        }
        const float off = top == -INFINITY ? 0.f : top;
        float sum = 0.f;
#pragma unroll
        for (int w = 0; w < 4; ++w) sum += p[w].y * __builtin_amdgcn_exp2f(p[w].x - off);
        a.part[nt * a.part_pitch + row0 + r] = make_float2(top, sum);
    }
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
    logits_sources(e, a.h, a.W, a.products, a.K, row0, rows, nullptr, v0, a.V);
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
    e.run(st0, st1, st2, nullptr);

#pragma unroll
    for (int nj = 0; nj < 4; ++nj) {
#pragma unroll
        for (int mi = 0; mi < 2; ++mi)
#pragma unroll
            for (int v = 0; v < 16; ++v)
                e.acc[mi][nj][v] = __builtin_amdgcn_exp2f(fmaf(e.acc[mi][nj][v], a.inv_tau, -lse[nj]) * 1.4426950408889634f);
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

// The gradients' products run on one workgroup per CU.  A team of workgroups
// takes the column tiles of the same 256 rows side by side, so that they read the
// M operand once through their XCD's L2; the teams share out the K steps of all
// row tiles evenly, each a contiguous range of them.  A tile whose steps one team
// makes goes straight out; of any other each team writes its part (at most one
// that it does not begin and one that it does not end) and a second kernel adds
// them in order.
constexpr int kGradUnits = 256;

struct GradWork {
    int m_tiles, n_tiles, teams;
    int steps;                // K steps of one product
    int virt;                 // of a tile: those of all products, at least 1
    int per;                  // of a team
};

__device__ __forceinline__ GradWork grad_work(const VocabGrad& a, int64_t rows) {
    GradWork w;
    const int64_t M = a.dW ? a.len : rows;
    const int K = a.dW ? (int)rows : a.len;
    w.m_tiles = (int)((M + 255) / 256);
    w.n_tiles = (a.N + TN - 1) / TN;
    w.teams = kGradUnits / w.n_tiles;
    w.steps = (K + BK - 1) / BK;
    w.virt = max(w.steps * a.products, 1);
    // parts cost what their write and their sum take, about 24 steps
    const int even = (int)(((int64_t)w.m_tiles * w.virt + w.teams - 1) / w.teams);
    const int whole = (w.m_tiles + w.teams - 1) / w.teams * w.virt;
    w.per = max(even + 24 < whole ? max(even, 8) : whole, 1);
    return w;
}

// Where a team's part of a tile goes: [256][256] fp32.
__device__ __forceinline__ float* grad_part(const VocabGrad& a, const GradWork& w, int team, bool begun, int nt) {
    return a.partial + (((int64_t)team * 2 + (begun ? 0 : 1)) * w.n_tiles + nt) * 65536;
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

// DW: both operands are k rows of columns; else M is K-contiguous.
template <bool DW>
__global__ __launch_bounds__(512, 1) void vocab_grad_kernel(const VocabGrad a) {
    using Eng = Engine<!DW, false, 256>;
    __shared__ __attribute__((aligned(1024))) char st0[Eng::SBYTES];
    __shared__ __attribute__((aligned(1024))) char st1[Eng::SBYTES];
    __shared__ __attribute__((aligned(1024))) char st2[Eng::SBYTES];
    __shared__ __attribute__((aligned(1024))) char st3[Eng::SBYTES];
    const int64_t rows = a.rows.count ? *a.rows.count : a.rows.T;
    const GradWork w = grad_work(a, rows);
    // 32 consecutive places on an XCD
    const int place = (blockIdx.x & 7) * (kGradUnits / 8) + (blockIdx.x >> 3);
    const int team = place / w.n_tiles, nt = place - team * w.n_tiles;
    if (team >= w.teams) return;
    const int64_t M = DW ? a.len : rows;
    const int64_t total = (int64_t)w.m_tiles * w.virt;
    const int64_t end = min((int64_t)(team + 1) * w.per, total);
    Eng e;
    for (int64_t at = (int64_t)team * w.per; at < end;) {
        const int mt = (int)(at / w.virt);
        const int k0 = (int)(at - (int64_t)mt * w.virt), k1 = (int)min((int64_t)w.virt, k0 + (end - at));
        at += k1 - k0;
        const int64_t m0 = (int64_t)mt * 256;

        e.begin();
        e.k_m = e.k_n = DW ? (int)rows : a.len;
        e.steps = w.steps;
        e.ip = 6 - a.products + (w.steps ? k0 / w.steps : 0);
        e.ik = w.steps ? k0 % w.steps : 0;
        e.kt_total = w.steps ? k1 - k0 : 0;
        e.m_plane = 2 * a.m.plane;
        e.n_plane = 2 * a.n.plane;
        e.m_pitch = 2 * a.m.pitch;
        e.n_pitch = 2 * a.n.pitch;
#pragma unroll
        for (int j = 0; j < Eng::MJ; ++j) {
            if constexpr (DW) {
                e.m_src[j] = (const char*)(a.m.p + m0 + 8 * e.ks_chunk(e.ks_row(j, Eng::MJ)));   // dz's rows are whole tiles
            } else {
                const int row = e.kc_row(j, Eng::MJ);
                e.m_src[j] = (const char*)(a.m.p + min(m0 + row, M - 1) * a.m.pitch + 8 * e.kc_chunk(row));
            }
        }
#pragma unroll
        for (int j = 0; j < Eng::WJ; ++j) {
            int n = nt * TN + 8 * e.ks_chunk(e.ks_row(j, Eng::WJ));
            if (n >= a.n.pitch) n = 0;       // an address that exists; its sums are never stored
            e.n_src[j] = (const char*)(a.n.p + n);
        }
        e.run(st0, st1, st2, st3);

        // Through LDS in two passes of 128 rows (those of the wavefronts rw =
        // pass), block nj in stage buffer nj as 32 rows of 1 KiB, 16-byte chunks
        // XOR-swizzled by the row; then each wavefront stores 16 rows.
        float* part = k1 - k0 < w.virt ? grad_part(a, w, team, k0 > 0, nt) : nullptr;
        auto buf = [&](int q) -> char* { return q == 0 ? st0 : q == 1 ? st1 : q == 2 ? st2 : st3; };
        const int l = e.lane & 31;
#pragma unroll
        for (int pass = 0; pass < 2; ++pass) {
            if (pass) __syncthreads();
            if (e.rw == pass) {
#pragma unroll
                for (int nj = 0; nj < 4; ++nj)
#pragma unroll
                    for (int mi = 0; mi < 2; ++mi)
#pragma unroll
                        for (int vg = 0; vg < 4; ++vg) {
                            const int c = 16 * e.fw + 8 * mi + 2 * vg + (e.lane >> 5);
                            const f32x16_t& v = e.acc[mi][nj];
                            *(float4*)(buf(nj) + l * 1024 + ((c ^ l) << 4)) =
                                make_float4(v[4 * vg], v[4 * vg + 1], v[4 * vg + 2], v[4 * vg + 3]);
                        }
            }
            __syncthreads();
            const char* sq = buf(e.wave >> 1);
#pragma unroll 4
            for (int i = 0; i < 16; ++i) {
                const int r = 16 * (e.wave & 1) + i, tr = 128 * pass + 32 * (e.wave >> 1) + r;
                const int64_t m = m0 + tr;
                if (m >= M) break;
                const float4 v = *(const float4*)(sq + r * 1024 + ((e.lane ^ r) << 4));
                if (part) *(float4*)(part + tr * 256 + 4 * e.lane) = v;
                else grad_out(a, m, nt * TN + 4 * e.lane, v);
            }
        }
        __syncthreads();       // the stages are read out before they are filled again
    }
}

// The tiles that more than one team made: 32 rows of one a workgroup.
__global__ __launch_bounds__(256) void vocab_grad_sum_kernel(const VocabGrad a) {
    const int64_t rows = a.rows.count ? *a.rows.count : a.rows.T;
    const GradWork w = grad_work(a, rows);
    const int slab = blockIdx.x & 7, tile = blockIdx.x >> 3;
    const int mt = tile / w.n_tiles, nt = tile - mt * w.n_tiles;
    if (mt >= w.m_tiles) return;
    const int64_t M = a.dW ? a.len : rows;
    const int64_t s0 = (int64_t)mt * w.virt, s1 = s0 + w.virt;
    const int t0 = (int)(s0 / w.per), t1 = (int)((s1 - 1) / w.per);
    if (t0 == t1) return;
    const int lane = threadIdx.x & 63, n0 = nt * TN + 4 * lane;
    if (n0 >= a.N) return;
#pragma unroll 2
    for (int i = 0; i < 8; ++i) {
        const int tr = 32 * slab + 4 * i + (threadIdx.x >> 6);
        const int64_t m = (int64_t)mt * 256 + tr;
        if (m >= M) break;
        const int at = tr * 256 + 4 * lane;
        float4 v = *(const float4*)(grad_part(a, w, t0, false, nt) + at);
#pragma unroll 4
        for (int t = t0 + 1; t <= t1; ++t) {
            const float4 o = *(const float4*)(grad_part(a, w, t, true, nt) + at);
            v.x += o.x, v.y += o.y, v.z += o.z, v.w += o.w;
        }
        grad_out(a, m, n0, v);
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

size_t vocab_grad_partial_bytes(int N) {
    const int n_tiles = (N + TN - 1) / TN;
    return (size_t)(kGradUnits / n_tiles) * 2 * n_tiles * 65536 * 4;
}

hipError_t launch_vocab_grad(const VocabGrad& a, hipStream_t s) {
    if ((a.products != 1 && a.products != 6) || a.rows.T <= 0 || a.len <= 0 || a.N <= 0 || a.N > kGradUnits * TN ||
        a.n.pitch % BK || a.m.pitch % TN || a.n.pitch < a.N || !a.partial || ((a.add || !a.last) && !a.acc))
        return hipErrorInvalidValue;
    const int64_t tiles = ((a.dW ? a.len : a.rows.T) + 255) / 256 * ((a.N + TN - 1) / TN);
    if (tiles > kMaxTiles / 4) return hipErrorInvalidValue;
    if (a.dW) vocab_grad_kernel<true><<<kGradUnits, 512, 0, s>>>(a);
    else vocab_grad_kernel<false><<<kGradUnits, 512, 0, s>>>(a);
    if (hipError_t e = hipGetLastError()) return e;
    vocab_grad_sum_kernel<<<(unsigned)(tiles * 8), 256, 0, s>>>(a);
    return hipGetLastError();
}

}  // namespace moe
