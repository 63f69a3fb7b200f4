// ssm_device.h -- building blocks of the state space scan's kernels: products
// of operands held as sums of bf16 parts, LDS tiles read along and across
// their rows, and the segments a sequence is cut into.
//
// Parts.  v_mfma_f32_16x16x32_bf16 multiplies bf16 exactly and adds in fp32,
// so an fp32 operand enters as up to three bf16 parts whose sum it is (8 bits
// of the 24 each): two cut off by truncation, the rest rounded.  Products of
// parts i and j with i + j > 2 are under 2^-24 of the whole and left out.  On
// this part six such products are 2.7 times faster than fp32 MFMA on the same
// tile, and a bf16 input (one part) needs three at most.
//
// k order.  Both operands of a 32-wide product hold, in lane l and slot j, the
// k index 16 (j / 4) + 4 (l / 16) + j % 4.  That is the order in which two
// accumulator tiles (rows 4 (l / 16) + e of rows 0..15 and 16..31) hold their
// rows, so an accumulator becomes the next product's operand without moving.
#pragma once

#include "kda_lanes.h"
#include "layer_device.h"

namespace kda {

template <int NP> struct Parts { bf16x8 v[NP]; };

__device__ __forceinline__ float top_bits(float x) {
    return __uint_as_float(__float_as_uint(x) & 0xffff0000u);
}

// Eight floats as NP parts; NP = 1 rounds to nearest.
template <int NP> __device__ __forceinline__ Parts<NP> split(const float (&f)[8]) {
    Parts<NP> p;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        float r = f[i];
#pragma unroll
        for (int k = 0; k < NP - 1; ++k) {
            const float h = top_bits(r);
            p.v[k][i] = static_cast<bf16>(h);
            r -= h;
        }
        p.v[NP - 1][i] = static_cast<bf16>(r);
    }
    return p;
}

// acc += A B, smallest products first.
template <int NA, int NB>
__device__ __forceinline__ f32x4 mma(const Parts<NA> &a, const Parts<NB> &b, f32x4 acc) {
#pragma unroll
    for (int s = (NA + NB - 2 < 2 ? NA + NB - 2 : 2); s >= 0; --s)
#pragma unroll
        for (int i = 0; i < NA; ++i)
            if (s - i >= 0 && s - i < NB)
                acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a.v[i], b.v[s - i], acc, 0, 0, 0);
    return acc;
}

// A tile of ROWS x COLS values as NP bf16 planes in LDS, COLS 32, 64 or 128.
// The 8-element chunks of a row change places by an XOR with `turn(row)`, which
// takes every value once over 16 rows and runs through the even values first.
// Sixteen rows' chunks of one column then lie in 16 different places of the 64
// banks, and so do two neighbouring columns' chunks of eight rows: both reads
// below are free of bank conflicts (rows padded by 32 bytes were so only along
// columns: 157 million conflict cycles in the 32K-token scan, 0.83 ms).
template <int NP, int ROWS, int COLS> struct Tile {
    static_assert(COLS == 32 || COLS == 64 || COLS == 128, "swizzle");
    static constexpr int LD = COLS;
    static constexpr int PLANE = ROWS * COLS;
    static constexpr int ELEMS = NP * PLANE;
    __device__ static int turn(int row) {
        constexpr int C = COLS / 8;       // chunks of a row
        const int q = row / (16 / C);     // rows that share the 64 banks count as one
        return ((2 * q) & (C - 1)) | ((q / (C / 2)) & 1);
    }
    // Element (row, col); runs of col % 8 stay together.
    __device__ static int at(int row, int col) {
        return row * COLS + (((col >> 3) ^ turn(row)) << 3) + (col & 7);
    }
};

// Operand with outer index = row: rows row0 + l % 16, k = columns 32 ks ...
// row0 is a multiple of 16.
template <typename TL, int NP>
__device__ __forceinline__ Parts<NP> read_rows(const bf16 *tile, int row0, int ks, int lane) {
    Parts<NP> p;
    const bf16 *at = tile + TL::at(row0 + (lane & 15), 32 * ks + 4 * (lane >> 4));
    const bf16 *up = tile + TL::at(row0 + (lane & 15), 32 * ks + 16 + 4 * (lane >> 4));
#pragma unroll
    for (int q = 0; q < NP; ++q) {
        const bf16x4 a = *reinterpret_cast<const bf16x4 *>(at + q * TL::PLANE);
        const bf16x4 b = *reinterpret_cast<const bf16x4 *>(up + q * TL::PLANE);
        p.v[q] = __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
    }
    return p;
}

// Operand with outer index = column: columns col0 + l % 16, k = rows 32 ks ...
// (transposing LDS reads: lane l of 16 receives column l of the four rows whose
// 8-byte pieces lanes l / 4 + 4 e address, e = 0..3).
template <typename TL, int NP>
__device__ __forceinline__ Parts<NP> read_cols(const bf16 *tile, int ks, int col0, int lane) {
    typedef __attribute__((address_space(3))) bf16x4 lds4;
    Parts<NP> p;
    const int row = 4 * (lane >> 4) + ((lane & 15) >> 2);
    const bf16 *at = tile + 32 * ks * TL::LD + TL::at(row, col0 + 4 * (lane & 3));
    const bf16 *up = at + 16 * TL::LD;  // turn() repeats after 16 rows
#pragma unroll
    for (int q = 0; q < NP; ++q) {
        const bf16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4bf16((lds4 *)(at + q * TL::PLANE));
        const bf16x4 b = __builtin_amdgcn_ds_read_tr16_b64_v4bf16((lds4 *)(up + q * TL::PLANE));
        p.v[q] = __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
    }
    return p;
}

// ROWS x COLS values of T, row r at p + r * stride, staged by NT threads:
// global to registers in 16-byte pieces (rows at and past `valid` as zeros),
// later registers to LDS as parts.
template <typename T, int ROWS, int COLS, int NT> struct Stage {
    static constexpr int E = 16 / sizeof(T), PER_ROW = COLS / E, COUNT = ROWS * PER_ROW / NT;
    static_assert(COUNT * NT == ROWS * PER_ROW, "pieces over threads");
    u32x4 r[COUNT];
    __device__ __forceinline__ void load(const T *p, int64_t stride, int valid, int tid) {
#pragma unroll
        for (int i = 0; i < COUNT; ++i) {
            const int piece = tid + i * NT, row = piece / PER_ROW;
            r[i] = row < valid ? *reinterpret_cast<const u32x4 *>(p + row * stride +
                                                                   piece % PER_ROW * E)
                               : u32x4{0u, 0u, 0u, 0u};
        }
    }
    template <typename TL> __device__ __forceinline__ void store(bf16 *tile, int tid) const {
#pragma unroll
        for (int i = 0; i < COUNT; ++i) {
            const int piece = tid + i * NT, row = piece / PER_ROW;
            bf16 *at = tile + TL::at(row, piece % PER_ROW * E);
            if constexpr (sizeof(T) == 2) {
                *reinterpret_cast<u32x4 *>(at) = r[i];
            } else {
                float v[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) v[e] = __uint_as_float(r[i][e]);
#pragma unroll
                for (int q = 0; q < 3; ++q) {
                    bf16x4 h;
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float t = q < 2 ? top_bits(v[e]) : v[e];
                        h[e] = static_cast<bf16>(t);
                        v[e] -= t;
                    }
                    *reinterpret_cast<bf16x4 *>(at + q * TL::PLANE) = h;
                }
            }
        }
    }
};

// Workgroup barrier that waits for this wave's LDS operations only: global
// loads on their way into registers and stores stay in flight across it.
__device__ __forceinline__ void lds_barrier() {
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
}

// The lane number as a value the compiler cannot trace: LDS addresses formed
// from it inside a loop are formed again in every iteration (an XOR and an add
// each) and do not fill the registers as loop constants.
__device__ __forceinline__ int here(int lane) {
    asm volatile("" : "+v"(lane));
    return lane;
}

// Inclusive sum over the 64 lanes in fp64.
__device__ __forceinline__ double wave_prefix(double v, int lane) {
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const double o = __shfl_up(v, d, 64);
        v += lane >= d ? o : 0.0;
    }
    return v;
}

constexpr double kLog2eD = 1.4426950408889634073599;

// Tokens of a block of the scan (and of a checkpoint of its backward).
template <typename T> constexpr int kSsmBlock = sizeof(T) == 2 ? 64 : 32;

// Pieces of `len` tokens of the sequences: piece j of sequence n, whose first
// token is t0, has number t0 / len + n + j, so numbers of different sequences
// never meet, and an empty sequence has one (empty) piece.
__host__ __device__ __forceinline__ int64_t piece_count(int64_t total, int64_t num, int64_t len) {
    return total / len + num + 1;
}
struct Piece {
    int seq, index, beg, end;  // sequence, number in it, tokens [beg, end)
    int seq_beg, seq_end;
    bool first, last, any;     // any: the number belongs to a sequence
};
__device__ __forceinline__ Piece find_piece(const Seqs &q, int64_t number, int len) {
    int lo = 0, hi = q.num - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (seq_first_token(q.cu, q.seq_len, q.total, mid) / len + mid <= number)
            lo = mid;
        else
            hi = mid - 1;
    }
    Piece p;
    p.seq = lo;
    p.seq_beg = (int)seq_first_token(q.cu, q.seq_len, q.total, lo);
    p.seq_end = seq_end_token(q, lo);
    if (p.seq_end < p.seq_beg) p.seq_end = p.seq_beg;  // malformed offsets
    const int64_t index = number - (p.seq_beg / len + lo);
    const int64_t count = p.seq_end > p.seq_beg ? (p.seq_end - p.seq_beg + (int64_t)len - 1) / len : 1;
    p.any = index >= 0 && index < count;
    p.index = (int)index;
    p.first = index == 0;
    p.last = index == count - 1;
    const int64_t beg = p.seq_beg + index * len, end = beg + len;
    p.beg = (int)beg;
    p.end = end < p.seq_end ? (int)end : p.seq_end;
    return p;
}

// Workgroups of one XCD (blockIdx % 8) take consecutive units, so that the
// heads that read the same B and C rows share an L2.  Returns -1 past the end.
__device__ __forceinline__ int64_t xcd_unit(int64_t units) {
    const int64_t per = (units + 7) / 8;
    const int64_t u = (int64_t)(blockIdx.x % 8) * per + blockIdx.x / 8;
    return blockIdx.x / 8 < per && u < units ? u : -1;
}
inline unsigned xcd_blocks(int64_t units) { return (unsigned)((units + 7) / 8 * 8); }

}  // namespace kda
