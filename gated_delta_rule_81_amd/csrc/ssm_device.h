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

__device__ __forceinline__ bool finite(float x) {
    return __builtin_fabsf(x) < __builtin_inff();
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

// Four floats as three parts, a plane each.
template <int PLANE> __device__ __forceinline__ void store_parts(bf16 *at, float (&v)[4]) {
#pragma unroll
    for (int q = 0; q < 3; ++q) {
        bf16x4 h;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float t = q < 2 ? top_bits(v[e]) : v[e];
            h[e] = static_cast<bf16>(t);
            v[e] -= t;
        }
        *reinterpret_cast<bf16x4 *>(at + q * PLANE) = h;
    }
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
// The 8-element chunks of a row change places by an XOR with `turn(row)`, a
// linear map that takes every value once over the rows that share the 64 banks.
// Measured, 16 waves reading: 3.3 cycles a wave for 8 bytes a lane along rows
// and for the transposing reads along columns, 4.1 for 16 bytes along rows; the
// plain XOR with the row costs the transposing reads 4.1, other maps the 16-byte
// reads 8, unswizzled rows 16 to 32.  By the counters, each kind of access in a loop
// of its own: 16-byte row reads, transposing reads, reads of fp32 rows and the staged
// 16-byte stores have no conflict cycles; two 8-byte row reads that the compiler joins
// into one instruction, and stores of accumulators (M, Q, E: 16 rows x 4 pieces a
// wave) have 8 in 16.
template <int NP, int ROWS, int COLS> struct Tile {
    static_assert(COLS == 32 || COLS == 64 || COLS == 128, "swizzle");
    static constexpr int LD = COLS;
    static constexpr int PLANE = ROWS * COLS;
    static constexpr int ELEMS = NP * PLANE;
    __device__ static int turn(int row) {
        constexpr int C = COLS / 8;       // chunks of a row
        const int q = row / (16 / C);     // rows that share the 64 banks count as one
        return ((2 * q) & (C - 1)) ^ (q & (C / 2) ? C / 2 + 1 : 0);
    }
    // Element (row, col); runs of col % 8 stay together.
    __device__ static int at(int row, int col) {
        return row * COLS + (((col >> 3) ^ turn(row)) << 3) + (col & 7);
    }
};

// Where a lane's pieces of an operand lie: element offsets that depend on the
// lane alone, formed once and used for every row tile (rows) or row step
// (columns) by immediate offsets, since turn() repeats after 16 rows.
//   rows:    outer index = row row0 + l % 16 (row0 a multiple of 16), k =
//            columns 32 ks ..; two 8-byte pieces
//   columns: outer index = column col0 + l % 16, k = rows 32 ks ..; two
//            transposing reads (lane l of 16 receives column l of the four rows
//            whose 8-byte pieces lanes l / 4 + 4 e address, e = 0..3)
template <typename TL> struct RowsAt {
    int o[TL::LD / 32][2];
    __device__ __forceinline__ explicit RowsAt(int lane) {
#pragma unroll
        for (int ks = 0; ks < TL::LD / 32; ++ks)
#pragma unroll
            for (int q = 0; q < 2; ++q)
                o[ks][q] = TL::at(lane & 15, 32 * ks + 16 * q + 4 * (lane >> 4));
    }
};
template <typename TL> __device__ __forceinline__ int cols_at(int col0, int lane) {
    return TL::at(4 * (lane >> 4) + ((lane & 15) >> 2), col0 + 4 * (lane & 3));
}

typedef __attribute__((address_space(3))) const bf16 lds_bf16;
typedef __attribute__((address_space(3))) bf16x4 lds_bf16x4;

template <typename TL, int NP>
__device__ __forceinline__ Parts<NP> read_rows(const bf16 *tile, int row0, int ks,
                                               const RowsAt<TL> &at) {
    Parts<NP> p;
    lds_bf16 *a = (lds_bf16 *)tile + at.o[ks][0], *b = (lds_bf16 *)tile + at.o[ks][1];
#pragma unroll
    for (int q = 0; q < NP; ++q) {
        const bf16x4 u = *(lds_bf16x4 *)(a + (q * TL::PLANE + row0 * TL::LD));
        const bf16x4 v = *(lds_bf16x4 *)(b + (q * TL::PLANE + row0 * TL::LD));
        p.v[q] = __builtin_shufflevector(u, v, 0, 1, 2, 3, 4, 5, 6, 7);
    }
    return p;
}

// The rows of a tile of fp32 values (TL in elements: two a value), in that k order,
// split into their three parts here.
template <typename TL> struct FloatRowsAt {
    int o[TL::LD / 64][2];
    __device__ __forceinline__ explicit FloatRowsAt(int lane) {
#pragma unroll
        for (int ks = 0; ks < TL::LD / 64; ++ks)
#pragma unroll
            for (int q = 0; q < 2; ++q)
                o[ks][q] = TL::at(lane & 15, 2 * (32 * ks + 16 * q + 4 * (lane >> 4)));
    }
};
template <typename TL, int NP>
__device__ __forceinline__ Parts<NP> read_rows(const bf16 *tile, int row0, int ks,
                                               const FloatRowsAt<TL> &at) {
    const bf16 *a = tile + row0 * TL::LD;
    const f32x4 u = *reinterpret_cast<const f32x4 *>(a + at.o[ks][0]);
    const f32x4 v = *reinterpret_cast<const f32x4 *>(a + at.o[ks][1]);
    const float f[8] = {u[0], u[1], u[2], u[3], v[0], v[1], v[2], v[3]};
    return split<NP>(f);
}

// The same outer index with k = 32 ks + 8 (l / 16) + j, for products whose two
// operands are both read so: one 16-byte read where the order above takes two of
// 8 bytes at half their rate.
template <typename TL> struct WideAt {
    int o[TL::LD / 32];
    __device__ __forceinline__ explicit WideAt(int lane) {
#pragma unroll
        for (int ks = 0; ks < TL::LD / 32; ++ks)
            o[ks] = TL::at(lane & 15, 32 * ks + 8 * (lane >> 4));
    }
};
template <typename TL, int NP>
__device__ __forceinline__ Parts<NP> read_wide(const bf16 *tile, int row0, int ks,
                                               const WideAt<TL> &at) {
    typedef __attribute__((address_space(3))) bf16x8 lds_bf16x8;
    Parts<NP> p;
    lds_bf16 *a = (lds_bf16 *)tile + at.o[ks];
#pragma unroll
    for (int q = 0; q < NP; ++q)
        p.v[q] = *(lds_bf16x8 *)(a + (q * TL::PLANE + row0 * TL::LD));
    return p;
}

// at = cols_at<TL>(col0, lane)
template <typename TL, int NP>
__device__ __forceinline__ Parts<NP> read_cols(const bf16 *tile, int ks, int at) {
    Parts<NP> p;
    lds_bf16 *a = (lds_bf16 *)tile + at;
#pragma unroll
    for (int q = 0; q < NP; ++q) {
        const bf16x4 u = __builtin_amdgcn_ds_read_tr16_b64_v4bf16(
            (lds_bf16x4 *)(a + (q * TL::PLANE + 32 * ks * TL::LD)));
        const bf16x4 v = __builtin_amdgcn_ds_read_tr16_b64_v4bf16(
            (lds_bf16x4 *)(a + (q * TL::PLANE + (32 * ks + 16) * TL::LD)));
        p.v[q] = __builtin_shufflevector(u, v, 0, 1, 2, 3, 4, 5, 6, 7);
    }
    return p;
}

// Word 3 of a raw buffer descriptor (32-bit format, no swizzle).
constexpr int kRsrcRaw = 0x00020000;

// ROWS x COLS values of T, row r at p + r * stride, staged by NT threads:
// global to registers in 16-byte pieces (rows at and past `valid` as zeros),
// later registers to LDS as parts.  Buffer loads whose descriptor ends behind the
// last valid row: rows past it read as zeros without a branch (64 rows of a
// tensor span less than 2^31 bytes).
template <typename T, int ROWS, int COLS, int NT> struct Stage {
    static constexpr int E = 16 / sizeof(T), PER_ROW = COLS / E, COUNT = ROWS * PER_ROW / NT;
    static constexpr int RS = NT / PER_ROW;
    static_assert(COUNT * NT == ROWS * PER_ROW && RS * PER_ROW == NT, "pieces over threads");
    u32x4 r[COUNT];
    __device__ __forceinline__ void load(const T *p, int64_t stride, int valid, int tid) {
        const int row_bytes = (int)stride * (int)sizeof(T);
        const auto rsrc = __builtin_amdgcn_make_buffer_rsrc(
            (void *)p, 0, (valid - 1) * row_bytes + COLS * (int)sizeof(T), kRsrcRaw);
        const int off = tid / PER_ROW * row_bytes + tid % PER_ROW * 16;
#pragma unroll
        for (int i = 0; i < COUNT; ++i)
            r[i] = __builtin_amdgcn_raw_buffer_load_b128(rsrc, off + i * RS * row_bytes, 0, 0);
    }
    // A sum of this thread's values: finite if all of them are (and none is huge).
    __device__ __forceinline__ float sum() const {
        typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
        unsigned ones = 0x3f803f80u;  // in a register: as a constant it would be one value
        asm("" : "+s"(ones));
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < COUNT; ++i) {
            float p = 0.f;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const unsigned v = r[i][e];
                if constexpr (sizeof(T) == 2)
                    p = __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2, v),
                                                        __builtin_bit_cast(bf16x2, ones), p, false);
                else
                    p += __uint_as_float(v);
            }
            s += p;
        }
        return s;
    }
    template <typename TL> __device__ __forceinline__ void store(bf16 *tile, int tid) const {
        const int row = tid / PER_ROW, col = tid % PER_ROW * E, first = TL::at(row, col);
#pragma unroll
        for (int i = 0; i < COUNT; ++i) {
            bf16 *at = tile + (RS % 16 == 0 ? first + i * RS * TL::LD : TL::at(row + i * RS, col));
            if constexpr (sizeof(T) == 2) {
                *reinterpret_cast<u32x4 *>(at) = r[i];
            } else {
                float v[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) v[e] = __uint_as_float(r[i][e]);
                store_parts<TL::PLANE>(at, v);
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

// Sums over the 64 lanes by DPP inside each 16-lane row and the rows' totals
// read into scalars: no LDS round trips, which six shuffle steps would be (the
// lane that forms a block's decays keeps the workgroup waiting).
template <int CTRL> __device__ __forceinline__ float dpp_or_zero(float x) {
    return __int_as_float(
        __builtin_amdgcn_update_dpp(0, __float_as_int(x), CTRL, 0xf, 0xf, true));
}
template <int CTRL> __device__ __forceinline__ double dpp_or_zero(double x) {
    const int lo = __builtin_amdgcn_update_dpp(0, __double2loint(x), CTRL, 0xf, 0xf, true);
    const int hi = __builtin_amdgcn_update_dpp(0, __double2hiint(x), CTRL, 0xf, 0xf, true);
    return __hiloint2double(hi, lo);
}
__device__ __forceinline__ float from_lane(float x, int lane) {
    return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(x), lane));
}
__device__ __forceinline__ double from_lane(double x, int lane) {
    return __hiloint2double(__builtin_amdgcn_readlane(__double2hiint(x), lane),
                            __builtin_amdgcn_readlane(__double2loint(x), lane));
}
// Inclusive sum over lanes 0 .. l.
template <typename V> __device__ __forceinline__ V wave_prefix(V v, int lane) {
    v += dpp_or_zero<0x111>(v);  // row_shr 1, 2, 4, 8
    v += dpp_or_zero<0x112>(v);
    v += dpp_or_zero<0x114>(v);
    v += dpp_or_zero<0x118>(v);
    const V r0 = from_lane(v, 15), r1 = from_lane(v, 31), r2 = from_lane(v, 47);
    return v + (lane < 16 ? V(0) : lane < 32 ? r0 : lane < 48 ? r0 + r1 : r0 + r1 + r2);
}
// Inclusive sum over lanes l .. 63.
template <typename V> __device__ __forceinline__ V wave_suffix(V v, int lane) {
    v += dpp_or_zero<0x101>(v);  // row_shl 1, 2, 4, 8
    v += dpp_or_zero<0x102>(v);
    v += dpp_or_zero<0x104>(v);
    v += dpp_or_zero<0x108>(v);
    const V r1 = from_lane(v, 16), r2 = from_lane(v, 32), r3 = from_lane(v, 48);
    return v + (lane < 16 ? r1 + r2 + r3 : lane < 32 ? r2 + r3 : lane < 48 ? r3 : V(0));
}

constexpr double kLog2eD = 1.4426950408889634073599;

// Tokens of a block of the scan (and of a checkpoint of its backward).
template <typename T> constexpr int kSsmBlock = sizeof(T) == 2 ? 64 : 32;

// One of the pieces the sequences are cut into (piece_count).
struct Piece {
    int seq, index, beg, end;  // sequence, number in it, tokens [beg, end)
    int seq_beg, seq_end;
    bool first, last, any;     // any: the number belongs to a sequence
    int64_t slot;              // of a sequence in several pieces
};
// By the piece's number, or by its slot (which sequences in one piece have none of;
// a sequence's slots all lie before those where the next one would have its own).
template <bool BY_SLOT = false>
__device__ __forceinline__ Piece find_piece(const Seqs &q, int64_t number, int len) {
    auto first_of = [&](int64_t t0, int n) {
        return BY_SLOT ? first_slot(q, len, t0, n) : first_piece(q, len, t0, n);
    };
    int lo = 0, hi = q.num - 1;
    if (!q.cu) lo = (int)(number / pieces_per_row(q, len));
    while (q.cu && lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (first_of(seq_first(q, mid), mid) <= number)
            lo = mid;
        else
            hi = mid - 1;
    }
    Piece p;
    p.seq = lo;
    p.seq_beg = seq_first(q, lo);
    p.seq_end = seq_end_token(q, lo);
    if (p.seq_end < p.seq_beg) p.seq_end = p.seq_beg;  // malformed offsets
    const int64_t index = number - first_of(p.seq_beg, lo);
    const int64_t count = p.seq_end > p.seq_beg ? (p.seq_end - p.seq_beg + (int64_t)len - 1) / len : 1;
    p.any = index >= 0 && index < count && (count > 1 || !BY_SLOT);
    p.slot = first_slot(q, len, p.seq_beg, lo) + index;
    p.index = (int)index;
    p.first = index == 0;
    p.last = index == count - 1;
    const int64_t beg = p.seq_beg + index * len, end = beg + len;
    p.beg = (int)beg;
    p.end = end < p.seq_end ? (int)end : p.seq_end;
    return p;
}

// The heads of one (piece, group) read the same B and C rows: their workgroups
// go to one XCD (blockIdx % 8) and share its L2, and the (piece, group) bundles
// are dealt to the XCDs in turn, so that pieces without tokens spread evenly.
// Returns number * heads + head, or -1 past the end.
__device__ __forceinline__ int64_t xcd_unit(unsigned block, int64_t numbers, int heads,
                                            int groups) {
    const int per = heads / groups;
    const int64_t i = block / 8, bundle = i / per * 8 + block % 8;
    if (bundle >= numbers * groups) return -1;
    return bundle / groups * heads + bundle % groups * per + i % per;
}
inline int64_t xcd_blocks(int64_t numbers, int heads, int groups) {
    return (numbers * groups + 7) / 8 * 8 * (heads / groups);
}

}  // namespace kda
