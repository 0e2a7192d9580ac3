// kda_latent_common.h -- device code that the latent attention kernels share:
// 32 x 32 matrix instructions, tiles in LDS, a block's sequence.
//
// Lane l of a wave is (n = l % 32, g = l / 32).  v_mfma_f32_32x32x16_bf16 takes 16
// values of k: A row n and B column n each in 8 k's of lane group g, and leaves in
// accumulator i of lane l the row 8 (i / 4) + 4 g + i % 4 of column n.  A product's
// accumulators are fed back as the B operand of the next one without leaving the
// lane: for k-block s of 16 rows, accumulators 8 s .. 8 s + 7 of the lane stand for
// the rows perm(s, g, j) = 16 s + 8 (j / 4) + 4 g + j % 4, and the A operand takes
// its columns in the same order, which is what two transposing LDS reads of 4 rows
// each deliver (ds_read_tr16_b64: of 4 rows x 16 columns, lane i of 16 gets column i).
#pragma once
#include "kda_latent_args.h"

namespace kda {

typedef float f16v __attribute__((ext_vector_type(16)));
typedef float f2v __attribute__((ext_vector_type(2)));
typedef __bf16 b2v __attribute__((ext_vector_type(2)));
typedef short s4 __attribute__((ext_vector_type(4)));
typedef int i4v __attribute__((ext_vector_type(4)));
typedef uint32_t u2v __attribute__((ext_vector_type(2)));
typedef uint32_t u4v __attribute__((ext_vector_type(4)));

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

__device__ __forceinline__ f16v mfma32(const s8 &a, const s8 &b, const f16v &c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(as_b8(a), as_b8(b), c, 0, 0, 0);
}

__device__ __forceinline__ f16v zero16() {
    f16v z;
#pragma unroll
    for (int i = 0; i < 16; ++i) z[i] = 0.0f;
    return z;
}

// Two fp32 -> two bf16 in one word (one conversion instruction, round to nearest even).
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    const f2v v = {lo, hi};
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, b2v));
}
// Accumulators 8 s .. 8 s + 7 as a B operand.
__device__ __forceinline__ s8 pack8(const f16v &v, int s) {
    u4v w;
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = pack2(v[8 * s + 2 * i], v[8 * s + 2 * i + 1]);
    return __builtin_bit_cast(s8, w);
}

// The value of lanes n and n + 32, combined in both.
__device__ __forceinline__ float pair_max(float x) {
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float pair_sum(float x) {
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

// ---- tiles in LDS -----------------------------------------------------------------
// A tile holds rows of 16-byte chunks, 8 (or a multiple) to a row, with chunk c of row
// r at place c ^ swap(r): 16 bytes of 8 neighbouring rows then lie in 8 different places
// of 128 bytes (swap takes 8 values), and so do the transposing read's 32 bytes of 4 rows
// (swap / 2 takes 4).  (A swap over 256 bytes, which are what LDS delivers a cycle, leaves
// no conflicts at all, 57% of the LDS cycles, but needs twice the addresses: the forward
// 762 -> 865 us, the gradient 2473 -> 2620.)
__device__ __forceinline__ int swap(int r) { return ((r & 3) << 1) | ((r >> 2) & 1); }

typedef const __attribute__((address_space(3))) s8 *lds_s8;
typedef __attribute__((address_space(3))) s4 *lds_s4;
__device__ __forceinline__ s8 read8(uint32_t at) { return *reinterpret_cast<lds_s8>(at); }
__device__ __forceinline__ s8 read_tr(uint32_t first, uint32_t second) {
    const s4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16(reinterpret_cast<lds_s4>(first));
    const s4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16(reinterpret_cast<lds_s4>(second));
    return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
}

// Row operand of rows 0 .. 31 of a tile of ROW bytes a row, k-block ks: at row_at(...) ^
// 32 ks within 128 bytes, 128 bytes further for every 4 k-blocks, 32 rows further for the
// next rows.
template <int ROW>
__device__ __forceinline__ uint32_t row_at(uint32_t base, int lane) {
    const int n = lane & 31, g = lane >> 5;
    return base + n * ROW + ((g ^ swap(n)) << 4);
}
template <int ROW>
__device__ __forceinline__ s8 row_operand(uint32_t at, int rows32, int ks) {
    return read8((at ^ ((ks & 3) << 5)) + (ks >> 2) * 128 + rows32 * 32 * ROW);
}
// Column operand: 32 columns from 32 dt, the rows perm(s, g, j) of k-block s: 4 rows,
// and 4 that are 8 further.
template <int ROW>
__device__ __forceinline__ uint32_t col_at(uint32_t base, int lane) {
    const int i = lane & 15, c16 = (lane >> 4) & 1, g = lane >> 5;
    const int r = 4 * g + (i >> 2);
    return base + r * ROW + (((2 * c16 + ((i & 3) >> 1)) ^ swap(r)) << 4) + (i & 1) * 8;
}
template <int ROW>
__device__ __forceinline__ s8 col_operand(uint32_t at, int s, int dt) {
    const uint32_t x = (at ^ ((dt & 1) << 6)) + (dt >> 1) * 128 + s * 16 * ROW;
    return read_tr(x, x + 8 * ROW);
}

// Copies from global memory straight into LDS, 16 bytes a lane: the wave's 64 lanes
// fill 1 KiB from `lds`.  Lanes whose offset is out of the descriptor's range write
// zeros.  Issued through inline asm, so that the compiler does not wait for them
// before other LDS reads; they are waited for by copies_done.
__device__ __forceinline__ void copy16(const i4v &rsrc, uint32_t off, uint32_t lds) {
    asm volatile("s_nop 0\n\tbuffer_load_dwordx4 %0, %1, 0 offen lds" :: "v"(off), "s"(rsrc), "{m0}"(lds) : "memory");
}
__device__ __forceinline__ void copy4(const i4v &rsrc, uint32_t off, uint32_t lds) {  // 256 bytes
    asm volatile("s_nop 0\n\tbuffer_load_dword %0, %1, 0 offen lds" :: "v"(off), "s"(rsrc), "{m0}"(lds) : "memory");
}
__device__ __forceinline__ i4v buffer_of(const void *p, uint32_t bytes) {
    const uint64_t a = reinterpret_cast<uint64_t>(p);
    i4v r;
    r[0] = __builtin_amdgcn_readfirstlane((int)(uint32_t)a);
    r[1] = __builtin_amdgcn_readfirstlane((int)((uint32_t)(a >> 32) & 0xffffu));
    r[2] = __builtin_amdgcn_readfirstlane((int)bytes);
    r[3] = 0x00020000;
    return r;
}
// This wave's copies and LDS accesses are done, and every wave's behind the barrier.
// (The wait is a builtin, which the compiler counts: loads of its own from before are
// not waited for again later, when the next copies are under way.)
__device__ __forceinline__ void copies_done() {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(0x0070);  // vmcnt(0) lgkmcnt(0)
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

// `rows` (at most 64) rows of 2 W bytes, `stride` bytes apart, into a tile, by the
// workgroup's WAVES waves.  off: tile_offset's.
template <int W>
__device__ __forceinline__ uint32_t tile_offset(int tid, uint32_t stride) {
    constexpr int C = W / 8;
    const int r = tid / C, c = tid % C;
    return (uint32_t)r * stride + (uint32_t)((c ^ swap(r)) << 4);
}
template <int W, int WAVES = 4>
__device__ __forceinline__ void copy_tile(const uint16_t *p, int rows, uint32_t stride, uint32_t off, uint32_t lds, int wave) {
    constexpr int C = W / 8, kRows = WAVES * 64 / C;
    const i4v rsrc = buffer_of(p, rows > 0 ? (uint32_t)(rows - 1) * stride + 2 * W : 0u);
#pragma unroll
    for (int i = 0; i < kKeys / kRows; ++i)
        copy16(rsrc, off + (uint32_t)(i * kRows) * stride, lds + (i * WAVES + wave) * 1024);
}

// ---- rows that leave a wave ----------------------------------------------------------
// 32 rows of CHUNKS x 16 bytes are staged in LDS (their own 512 CHUNKS bytes of it) and stored
// whole: lanes hold 8 bytes of a row at a time, and stored as such rows took 1.3 us longer a
// workgroup.  Chunk c of row r is at place c ^ (r % 16 or 8).
template <int CHUNKS>
__device__ __forceinline__ char *staged(char *stage, int r, int c) {
    return stage + r * (16 * CHUNKS) + ((c ^ (r & (CHUNKS % 16 == 0 ? 15 : 7))) << 4);
}
// Accumulators of 32 values from chunk `first` on, times f, as bf16.
template <int CHUNKS>
__device__ __forceinline__ void stage_values(char *stage, int lane, int first, const f16v &v, float f) {
#pragma unroll
    for (int e = 0; e < 4; ++e)
        *reinterpret_cast<u2v *>(staged<CHUNKS>(stage, lane & 31, first + e) + 8 * (lane >> 5)) =
            u2v{pack2(v[4 * e] * f, v[4 * e + 1] * f), pack2(v[4 * e + 2] * f, v[4 * e + 3] * f)};
}
// The first `rows` rows to `out`, `stride` values apart.
template <int CHUNKS>
__device__ __forceinline__ void store_rows(char *stage, int lane, uint16_t *out, int64_t stride, int rows) {
#pragma unroll
    for (int k = 0; k < CHUNKS / 2; ++k) {
        const int r = (64 * k + lane) / CHUNKS, c = (64 * k + lane) % CHUNKS;
        const u4v x = *reinterpret_cast<const u4v *>(staged<CHUNKS>(stage, r, c));
        if (r < rows) *reinterpret_cast<u4v *>(out + r * stride + 8 * c) = x;
    }
}

// ---- a block's sequence ----------------------------------------------------------
struct Span {
    int64_t q0, k0;  // first query and key, in rows of the tensors' token dimension
    int lq, lk;
    int64_t b;       // batch row
    int block;
};

__device__ __forceinline__ int64_t clamp64(int64_t v, int64_t lo, int64_t hi) { return v < lo ? lo : v > hi ? hi : v; }

__device__ __forceinline__ void bounds_of(const int64_t *cu, int64_t n, int64_t T, int64_t &first, int &len) {
    const int64_t lo = clamp64(cu[n], 0, T), hi = clamp64(cu[n + 1], lo, T);
    first = lo;
    len = (int)(hi - lo);
}

// Tiles of a part of a block whose sequence has `tiles` of the other side.  The host plans by the
// tiles of all sequences together, which are a batch row's own; of a packed batch each sequence is
// cut into as many parts as one that had all tiles would be (by that one's part 8 sequences of 16 queries over
// 8208 keys x 4 heads were not split at all: 149 -> 37 us; 4 of 1000 tokens, one head, 22 -> 20, their
// gradient 50 -> 40).  (Sequences of up to kFewTiles, too: the joining is launched for all of them; 5 of
// 768 tokens, one head, take 20.0 us, whole 22.9.)  Even, as the forward has tile j in buffer j % 2.
__device__ __forceinline__ int part_tiles_of(const LatentArgs &a, int tiles) {
    if (!a.cu) return a.part_tiles;
    const int parts = (int)a.parts;
    return (max(kPartTiles, (tiles + parts - 1) / parts) + 1) / 2 * 2;
}

// The sequence and block of unit e (a workgroup's number over the heads); false where
// there is none.  size: tokens of a block, of the keys with BY_KEYS, else of the queries;
// reversed: the last blocks, which see the most, come first.  Without a table the blocks
// of a packed batch (of at most 64 sequences) are counted through by the wave.
template <int SIZE, bool BY_KEYS>
__device__ __forceinline__ bool span_of(const LatentArgs &a, int64_t e, bool reversed, Span &s) {
    if (!a.cu) {
        s.b = e % a.B;
        s.block = (int)(e / a.B);
        if (reversed) s.block = (int)a.blocks - 1 - s.block;
        s.q0 = s.k0 = 0;
        s.lq = (int)a.T;
        s.lk = (int)a.Tk;
        return true;
    }
    int64_t n;
    if (a.table) {
        if (e >= a.table[0]) return false;
        n = a.table[2 + 2 * e];
        s.block = a.table[3 + 2 * e];
    } else {
        const int lane = threadIdx.x & 63;
        int blocks = 0;
        if (lane < a.seqs) {
            int64_t first;
            int len;
            bounds_of(BY_KEYS ? a.cuk : a.cu, lane, BY_KEYS ? a.Tk : a.T, first, len);
            blocks = (len + SIZE - 1) / SIZE;
        }
        int upto = blocks;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const int o = __shfl_up(upto, d);
            if (lane >= d) upto += o;
        }
        const uint64_t behind = __builtin_amdgcn_ballot_w64(upto > e);
        if (behind == 0) return false;
        n = __builtin_ctzll(behind);
        s.block = __builtin_amdgcn_readlane(upto, (int)n) - 1 - (int)e;  // from the sequence's end
        if (!reversed) s.block = __builtin_amdgcn_readlane(blocks, (int)n) - 1 - s.block;
    }
    bounds_of(a.cu, n, a.T, s.q0, s.lq);
    bounds_of(a.cuk, n, a.Tk, s.k0, s.lk);
    s.b = 0;
    return true;
}

}  // namespace kda
