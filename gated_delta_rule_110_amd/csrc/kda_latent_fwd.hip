// kda_latent_fwd.hip -- latent attention in its expanded form (kda_latent_fwd in
// include/kda_latent.h), and the table of a packed batch's blocks.
//
// A workgroup of four or eight waves has 32 queries a wave of one head and runs once
// through the keys they see, 64 at a time.  Scores are taken transposed, S^T = K Q^T, so that a
// lane holds one query's: its maximum and sum are the lane's own but for one exchange
// between lanes n and n + 32, and the accumulators, rounded to bf16, are the B operand
// of O^T += V^T P^T as they stand.  Queries stay in registers, keys and values come by
// copies straight into LDS, two tiles of each, and the scores of tile j + 1 are
// computed beside the exponentials of tile j.  Where there are few queries, workgroups
// share a block's keys and a second kernel joins what they leave.
//
// The matrix instructions bound it: 8192 tokens x 32 heads take 598 us, 1.15 PFLOP/s, and a
// stream of nothing but those instructions 538.  Both are held by the card's power, which
// lowers the clock (1.7 GHz here, where they fill 64% of the cycles), so that every LDS read
// and vector instruction costs time although there are slots for it: without exponentials
// the kernel took 26 us less, without LDS reads 70 and without copies 84 (of 715).
//
// Precision: scores, maxima, sums and outputs are fp32.  Probabilities are rounded to
// bf16 for the second product (at most 2^-8 of each; the outputs' own rounding is as large);
// the sum, and with it lse, takes them unrounded.
#include "kda_latent_common.h"

namespace kda {

namespace {

// LDS of a workgroup: two tiles of keys (128 and 64 values) and of values.
struct FwdSmem {
    uint16_t kn[2][kKeys * kNope];
    uint16_t kp[2][kKeys * kPe];
    uint16_t v[2][kKeys * kVal];
};

struct FwdState {
    s8 q[kQk / 16];
    f16v o[kVal / 32];
    float mc, l;   // running maximum (times scale, log2 units) and this lane's part of the sum
};

struct FwdAddr {
    uint32_t kn, kp, v;  // this lane's in buffer 0
};

// Where the lane's operands lie in a tile: the A operand of slot n (two 32-key halves of
// the scores' product, 12 k-blocks each), and that of slot m of the outputs' product (4
// k-blocks, 4 groups of 32 values).
__device__ __forceinline__ s8 key_operand(const FwdAddr &at, int buf, int n) {
    const uint32_t kn = at.kn + buf * (uint32_t)sizeof(FwdSmem::kn[0]), kp = at.kp + buf * (uint32_t)sizeof(FwdSmem::kp[0]);
    const int t = n & 1, ks = n >> 1;
    return ks < kNope / 16 ? row_operand<2 * kNope>(kn, t, ks) : row_operand<2 * kPe>(kp, t, ks - kNope / 16);
}
__device__ __forceinline__ s8 value_operand(const FwdAddr &at, int buf, int m) {
    return col_operand<2 * kVal>(at.v + buf * (uint32_t)sizeof(FwdSmem::v[0]), m >> 2, m & 3);
}
constexpr int kKeySlots = 2 * kQk / 16, kValueSlots = 4 * kVal / 32;

// Scores of keys that the lane's query does not see become -infinity.  base: the tile's
// first key; seen: keys that the query sees.
__device__ __forceinline__ void mask(f16v (&s)[2], int seen, int base, int g) {
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int i = 0; i < 16; ++i) s[t][i] = base + 32 * t + 8 * (i / 4) + 4 * g + i % 4 < seen ? s[t][i] : -INFINITY;
}

// The maximum of n of the lane's scores of either half, from `first` on.
__device__ __forceinline__ void maxima(const f16v (&s)[2], float &top, int first, int n) {
#pragma unroll
    for (int i = first; i < first + n; ++i) top = fmaxf(fmaxf(top, s[0][i]), s[1][i]);
}

// A rise of the maximum scales the accumulators.  The maximum in use may stay up to 2^8
// below the true one: probabilities up to 256 lose nothing, and the accumulators are
// scaled a few times a row instead of once a tile.
__device__ __forceinline__ void rise(FwdState &f, float lane_top, float c) {
    constexpr float kSlack = 8.0f;
    const float top = pair_max(lane_top) * c;
    if (__builtin_amdgcn_ballot_w64(top > f.mc + kSlack) == 0) return;
    const float m = fmaxf(f.mc, top);
    const float w = m == -INFINITY ? 1.0f : __builtin_amdgcn_exp2f(f.mc - m);
    f.mc = m;
    f.l *= w;
#pragma unroll
    for (int d = 0; d < kVal / 32; ++d)
#pragma unroll
        for (int i = 0; i < 16; ++i) f.o[d][i] *= w;
}

// Probability x of a tile's 32 in the lane, those of the first 32 keys first.  Every
// second one completes a word of the B operand.
struct Probs {
    u4v w[4];
    float last;
};
__device__ __forceinline__ void probability(FwdState &f, const f16v (&s)[2], float c, float m, int x, Probs &p) {
    const int t = x / 16, i = x % 16;
    const float e = __builtin_amdgcn_exp2f(fmaf(s[t][i], c, -m));
    f.l += e;
    if (i & 1) p.w[2 * t + i / 8][i % 8 / 2] = pack2(p.last, e);
    else p.last = e;
}

// Tile j's probabilities and outputs; with NEXT the scores of tile j + 1 too (and their
// maxima), whose 24 products come first, with an exponential each; the last 8 are taken
// beside the first half of the outputs' products, which need them in the second.
// Operands are read kAhead products before their use.  The order is fixed by the
// fences: left to itself the compiler reads all operands at once and spills.
template <bool NEXT>
__device__ __forceinline__ void tile_step(FwdState &f, const FwdAddr &at, int buf, const f16v (&s)[2], f16v (&next)[2], float &top, float c) {
    constexpr int kAhead = 4, kFirst = NEXT ? 0 : kKeySlots;
    const float m = f.mc == -INFINITY ? 0.0f : f.mc;
    Probs p;
    s8 ring[kAhead];
    const auto operand = [&](int n) { return n < kKeySlots ? key_operand(at, buf ^ 1, n) : value_operand(at, buf, n - kKeySlots); };
#pragma unroll
    for (int n = 0; n < kAhead; ++n) ring[(kFirst + n) % kAhead] = operand(kFirst + n);
    if (NEXT) {
        next[0] = next[1] = zero16();
        top = -INFINITY;
    } else {
#pragma unroll
        for (int x = 0; x < kKeySlots; ++x) probability(f, s, c, m, x, p);
    }
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int n = kFirst; n < kKeySlots + kValueSlots; ++n) {
        const s8 a = ring[n % kAhead];
        const int v = n - kKeySlots;
        if (v < 0) next[n & 1] = mfma32(a, f.q[n >> 1], next[n & 1]);
        else f.o[v & 3] = mfma32(a, __builtin_bit_cast(s8, p.w[v >> 2]), f.o[v & 3]);
        if (n + kAhead < kKeySlots + kValueSlots) ring[n % kAhead] = operand(n + kAhead);
        if (v < kValueSlots / 2) probability(f, s, c, m, n, p);
        else if (NEXT) maxima(next, top, 2 * (v - kValueSlots / 2), 2);
        __builtin_amdgcn_sched_barrier(0);
    }
}

__device__ __forceinline__ void first_scores(const FwdState &f, const FwdAddr &at, int buf, f16v (&s)[2], float &top) {
    s[0] = s[1] = zero16();
#pragma unroll
    for (int n = 0; n < kKeySlots; ++n) {
        s[n & 1] = mfma32(key_operand(at, buf, n), f.q[n >> 1], s[n & 1]);
        if (n % 4 == 3) __builtin_amdgcn_sched_barrier(0);
    }
    top = -INFINITY;
    maxima(s, top, 0, 16);
}

// Values that are NaN or infinite meet the zero probabilities of queries that do not see
// them.  Where a tile has hidden keys, those values are added apart, to the queries that
// see their keys, and then taken as zeros.
__device__ __forceinline__ bool odd_bits(uint32_t bf16) { return (bf16 & 0x7f80u) == 0x7f80u; }
__device__ __forceinline__ void add_odd(FwdState &f, const uint16_t *v, int seen, int base, int g) {
#pragma unroll 1
    for (int r = 0; r < kKeys; ++r) {
#pragma unroll
        for (int e = 0; e < kVal / 8; ++e) {  // the lane's four values of each 8
            const u2v w = *reinterpret_cast<const u2v *>(v + r * kVal + ((e ^ swap(r)) << 3) + 4 * g);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const uint32_t b = (w[k / 2] >> (16 * (k & 1))) & 0xffffu;
                const float x = odd_bits(b) ? bf16_bits_to_f32(b) : 0.0f;
                f.o[e / 4][4 * (e % 4) + k] += base + r < seen ? x : 0.0f;
            }
        }
    }
}
__device__ __forceinline__ void clear_odd(uint16_t *v, int tid, int threads) {
    uint32_t *w = reinterpret_cast<uint32_t *>(v);
    for (int i = tid; i < kKeys * kVal / 2; i += threads) {
        uint32_t x = w[i];
        if (odd_bits(x)) x &= 0xffff0000u;
        if (odd_bits(x >> 16)) x &= 0x0000ffffu;
        w[i] = x;
    }
}

// WAVES of 32 queries each.  SPLIT: a workgroup takes a part of its block's keys.
template <int WAVES, bool SPLIT>
__global__ __launch_bounds__(64 * WAVES, 2) void latent_fwd_kernel(LatentArgs a) {
    __shared__ __attribute__((aligned(1024))) FwdSmem sm;
    constexpr int kBlock = 32 * WAVES;
    const int tid = threadIdx.x, lane = tid & 63, g = lane >> 5;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int64_t place = a.base + blockIdx.x, unit = SPLIT ? place / a.parts : place, h = unit % a.H;
    Span sp;
    if (!span_of<kBlock, false>(a, unit / a.H, a.causal, sp)) return;
    const int q_first = sp.block * kBlock + wave * 32;  // of this wave
    const int block_last = min(sp.lq, (sp.block + 1) * kBlock) - 1;
    if (block_last < sp.block * kBlock) return;

    const auto sees = [&](int i) { return a.causal ? max(0, min(sp.lk, i + 1 + sp.lk - sp.lq)) : sp.lk; };
    const int all = (sees(block_last) + kKeys - 1) / kKeys;                      // tiles of the block
    const int part_tiles = SPLIT ? part_tiles_of(a, (sp.lk + kKeys - 1) / kKeys) : 0;
    const int t0 = SPLIT ? (int)(place - unit * a.parts) * part_tiles : 0;       // even: tile j is in buffer j % 2
    if (SPLIT && t0 >= max(all, 1)) return;
    const int tiles = SPLIT ? min(all, t0 + part_tiles) : all;                   // (behind the last) of the workgroup
    const int last = min(sp.lq - 1, q_first + 31);
    const int mine = last < q_first ? 0 : min(tiles, (sees(last) + kKeys - 1) / kKeys);  // of this wave
    const int whole = sees(q_first) / kKeys;                                 // of them without hidden keys

    const uint16_t *kv = a.kv + sp.b * a.kvb + sp.k0 * a.kvt + h * kKvRow;
    const uint16_t *pe = a.pe + sp.b * a.peb + sp.k0 * a.pet;
    const uint32_t kv_bytes = (uint32_t)a.kvt * 2, pe_bytes = (uint32_t)a.pet * 2;
    const uint32_t off_n = tile_offset<kNope>(tid, kv_bytes), off_p = tile_offset<kPe>(tid, pe_bytes);
    const uint32_t lds_kn = lds_addr(sm.kn), lds_kp = lds_addr(sm.kp), lds_v = lds_addr(sm.v);
    const auto copy_keys = [&](int j) {
        const int rows = min(kKeys, sp.lk - j * kKeys), buf = j & 1;
        copy_tile<kNope, WAVES>(kv + (int64_t)j * kKeys * a.kvt, rows, kv_bytes, off_n, lds_kn + buf * (uint32_t)sizeof(sm.kn[0]), wave);
        copy_tile<kPe, WAVES>(pe + (int64_t)j * kKeys * a.pet, rows, pe_bytes, off_p, lds_kp + buf * (uint32_t)sizeof(sm.kp[0]), wave);
    };
    const auto copy_values = [&](int j) {
        const int rows = min(kKeys, sp.lk - j * kKeys), buf = j & 1;
        copy_tile<kVal, WAVES>(kv + kNope + (int64_t)j * kKeys * a.kvt, rows, kv_bytes, off_n, lds_v + buf * (uint32_t)sizeof(sm.v[0]), wave);
    };
    if (tiles > t0) {
        copy_keys(t0);
        if (tiles > t0 + 1) copy_keys(t0 + 1);
        copy_values(t0);
    }

    FwdState f;
    const int i = q_first + (lane & 31), seen = sees(i);
    {
        const uint16_t *p = a.q + sp.b * a.qb + (sp.q0 + min(i, sp.lq - 1)) * a.qt + h * kQk + 8 * g;
#pragma unroll
        for (int ks = 0; ks < kQk / 16; ++ks) f.q[ks] = *reinterpret_cast<const s8 *>(p + 16 * ks);
    }
    const auto reset = [&]() {
        f.mc = -INFINITY;
        f.l = 0.0f;
#pragma unroll
        for (int d = 0; d < kVal / 32; ++d) f.o[d] = zero16();
    };
    reset();
    const FwdAddr at = {row_at<2 * kNope>(lds_kn, lane), row_at<2 * kPe>(lds_kp, lane), col_at<2 * kVal>(lds_v, lane)};
    const float c = a.scale * kLog2e;

    // Tile j's scores are in `s`, their maximum in `top`; those of j + 1 go to `next`.
    float top = -INFINITY;
    const auto begin = [&](int j) {
        copies_done();
        if (j + 2 < tiles) copy_keys(j + 2);
        if (j + 1 < tiles) copy_values(j + 1);
    };
    const auto hide = [&](int j, f16v (&s)[2]) {
        mask(s, seen, j * kKeys, g);
        top = -INFINITY;
        maxima(s, top, 0, 16);
    };
    const auto step = [&](int j, f16v (&s)[2], f16v (&next)[2]) {
        begin(j);
        if (j >= whole) hide(j, s);
        rise(f, top, c);
        tile_step<true>(f, at, j & 1, s, next, top, c);
    };
    if (tiles > t0) {
        f16v s0[2], s1[2];
        copies_done();
        int j = t0;
        if (mine > t0) {
            first_scores(f, at, 0, s0, top);
            for (; j + 2 < mine; j += 2) {
                step(j, s0, s1);
                step(j + 1, s1, s0);
            }
            if (j + 1 < mine) {
                step(j++, s0, s1);
                s0[0] = s1[0];
                s0[1] = s1[1];
            }
            begin(j);
            if (j >= whole) hide(j, s0);
            rise(f, top, c);
            tile_step<false>(f, at, j & 1, s0, s0, top, c);
            ++j;
        }
        for (; j < tiles; ++j) begin(j);
    }

    // NaN or infinity among the outputs: perhaps by way of keys that the query does not
    // see.  The block runs again, tile by tile, with those apart.
    f4 odd = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int e = 0; e < 16; ++e)
#pragma unroll
        for (int d = 0; d < kVal / 32; ++d) odd[d] = fmaf(f.o[d][e], 0.0f, odd[d]);
    static_assert(kVal / 32 == 4, "");
    uint32_t *flag = reinterpret_cast<uint32_t *>(sm.v[1]);  // behind what the outputs are staged in
    copies_done();
    const bool found = __builtin_amdgcn_ballot_w64(!((odd[0] + odd[1]) + (odd[2] + odd[3]) == 0.0f)) != 0;
    if (lane == 0) flag[wave] = found;
    __syncthreads();
    uint32_t again = 0;
#pragma unroll
    for (int k = 0; k < WAVES; ++k) again |= flag[k];
    if (again) {
        __syncthreads();
        reset();
        const int block_whole = sees(sp.block * kBlock) / kKeys;
#pragma unroll 1
        for (int j = t0; j < tiles; ++j) {
            copy_keys(j);
            copy_values(j);
            copies_done();
            f16v s[2];
            if (j < mine) {
                first_scores(f, at, j & 1, s, top);
                hide(j, s);
                rise(f, top, c);
            }
            if (j >= block_whole) {
                if (j < mine) add_odd(f, sm.v[j & 1], seen, j * kKeys, g);
                __syncthreads();
                clear_odd(sm.v[j & 1], tid, 64 * WAVES);
                __syncthreads();
            }
            if (j < mine) tile_step<false>(f, at, j & 1, s, s, top, c);
            __syncthreads();
        }
    }

    const float l = pair_sum(f.l);
    if (SPLIT && all > part_tiles) {
        f4 *y = reinterpret_cast<f4 *>(a.part) + (place * WAVES + wave) * (kVal / 8 * 64) + lane;
#pragma unroll
        for (int d = 0; d < kVal / 32; ++d)
#pragma unroll
            for (int e = 0; e < 4; ++e) y[(4 * d + e) * 64] = f4{f.o[d][4 * e], f.o[d][4 * e + 1], f.o[d][4 * e + 2], f.o[d][4 * e + 3]};
        if (g == 0) {
            float *st = a.part_stat + (place * WAVES + wave) * 64 + lane;
            st[0] = f.mc;
            st[32] = l;
        }
        return;
    }
    const float w = l == 0.0f ? 0.0f : 1.0f / l;
    const int64_t row0 = (sp.b * a.T + sp.q0 + q_first) * a.H + h;
    char *stage = reinterpret_cast<char *>(&sm) + wave * 32 * 2 * kVal;
    static_assert(sizeof(sm.kn) + sizeof(sm.kp) + sizeof(sm.v[0]) >= 8 * 32 * 2 * kVal, "");
#pragma unroll
    for (int d = 0; d < kVal / 32; ++d) stage_values<kVal / 8>(stage, lane, 4 * d, f.o[d], w);
    store_rows<kVal / 8>(stage, lane, a.out + row0 * kVal, a.H * kVal, sp.lq - q_first);
    // l == 0: no key is seen
    if (a.lse && g == 0 && i < sp.lq) a.lse[row0 + (lane & 31) * a.H] = l == 0.0f ? -INFINITY : (f.mc + __builtin_amdgcn_logf(l)) * kLn2;
}

// A block's parts added up in their order: 32 queries and 32 of their values a wave.
__global__ __launch_bounds__(64) void latent_fwd_join_kernel(LatentArgs a) {
    constexpr int kWaves = 4, kPieces = kVal / 32;
    const int lane = threadIdx.x, g = lane >> 5;
    const int64_t place = a.base + blockIdx.x, unit = place / (kWaves * kPieces), h = unit % a.H;
    const int wave = (int)(place / kPieces % kWaves), d = (int)(place % kPieces);
    Span sp;
    if (!span_of<32 * kWaves, false>(a, unit / a.H, a.causal, sp)) return;
    const int q_first = sp.block * 32 * kWaves + wave * 32, block_last = min(sp.lq, (sp.block + 1) * 32 * kWaves) - 1;
    if (q_first > block_last) return;
    const int keys = a.causal ? max(0, min(sp.lk, block_last + 1 + sp.lk - sp.lq)) : sp.lk, all = (keys + kKeys - 1) / kKeys;
    const int part_tiles = part_tiles_of(a, (sp.lk + kKeys - 1) / kKeys), parts = (all + part_tiles - 1) / part_tiles;
    if (parts < 2) return;
    const auto factor = [](float from, float to) { return to == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(from - to); };
    f4 o[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) o[e] = f4{0.0f, 0.0f, 0.0f, 0.0f};
    float m = -INFINITY, l = 0.0f;
#pragma unroll 4
    for (int p = 0; p < parts; ++p) {
        const int64_t s = (unit * a.parts + p) * kWaves + wave;
        const f4 *y = reinterpret_cast<const f4 *>(a.part) + (s * kPieces + d) * 4 * 64 + lane;
        const float *st = a.part_stat + s * 64 + (lane & 31);
        const float top = fmaxf(m, st[0]), was = factor(m, top), is = factor(st[0], top);
#pragma unroll
        for (int e = 0; e < 4; ++e) o[e] = o[e] * was + y[e * 64] * is;
        l = l * was + st[32] * is;
        m = top;
    }
    const int i = q_first + (lane & 31);
    if (i > block_last) return;
    const float w = l == 0.0f ? 0.0f : 1.0f / l;
    const int64_t row = (sp.b * a.T + sp.q0 + i) * a.H + h;
    uint16_t *out = a.out + row * kVal + 32 * d + 4 * g;
#pragma unroll
    for (int e = 0; e < 4; ++e) *reinterpret_cast<u2v *>(out + 8 * e) = u2v{pack2(o[e][0] * w, o[e][1] * w), pack2(o[e][2] * w, o[e][3] * w)};
    if (a.lse && d == 0 && g == 0) a.lse[row] = l == 0.0f ? -INFINITY : (m + __builtin_amdgcn_logf(l)) * kLn2;
}

// The blocks of a packed batch in order of falling length, by buckets of their tiles'
// number.  Which of a bucket's blocks comes first is left to chance: it decides when
// a block runs, not what it computes.  Blocks are counted in 64 bits: offsets that
// overlap, which valid ones do not, describe up to sequences times tokens / size of them.
constexpr int kBuckets = 1024;
struct TableArgs {
    const int64_t *cu, *cuk;
    int64_t T, Tk, seqs;
    int64_t cap;               // entries of the table
    int size, by_keys, causal;
    int32_t *table;
};
__global__ __launch_bounds__(1024) void latent_table_kernel(TableArgs by_queries, TableArgs by_keys) {
    const TableArgs &a = blockIdx.x == 0 ? by_queries : by_keys;
    __shared__ unsigned long long count[kBuckets];
    __shared__ int64_t part[16];
    __shared__ int most;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    for (int i = tid; i < kBuckets; i += 1024) count[i] = 0;
    if (tid == 0) most = 1;
    __syncthreads();
    const auto lengths = [&](int64_t n, int &lq, int &lk) {
        int64_t first;
        bounds_of(a.cu, n, a.T, first, lq);
        bounds_of(a.cuk, n, a.Tk, first, lk);
    };
    int top = 1;
    for (int64_t n = tid; n < a.seqs; n += 1024) {
        int lq, lk;
        lengths(n, lq, lk);
        top = max(top, ((a.by_keys ? lq : lk) + kKeys - 1) / kKeys);
    }
    atomicMax(&most, top);
    __syncthreads();
    int shift = 0;
    while ((most >> shift) >= kBuckets) ++shift;
    // Tiles that block i of a sequence runs through.
    const auto work = [&](int lq, int lk, int i) {
        if (a.by_keys) {
            const int first = a.causal ? max(0, i * a.size - (lk - lq)) : 0;  // query that sees the first key
            return max(0, lq - first + kKeys - 1) / kKeys;
        }
        const int last = min(lq, (i + 1) * a.size) - 1;
        return (max(0, a.causal ? min(lk, last + 1 + lk - lq) : lk) + kKeys - 1) / kKeys;
    };
    // visit(sequence, lq, lk, block) for every block.  A wave takes 64 sequences at a time:
    // lanes run through the blocks of short ones, the wave through those of long ones.
    constexpr int kShort = 8;
    const auto each = [&](auto visit) {
        for (int64_t first = wave * 64; first < a.seqs; first += 1024) {
            const int64_t n = first + lane;
            int lq = 0, lk = 0;
            if (n < a.seqs) lengths(n, lq, lk);
            const int blocks = ((a.by_keys ? lk : lq) + a.size - 1) / a.size;
            if (blocks <= kShort)
                for (int i = 0; i < blocks; ++i) visit(n, lq, lk, i);
            uint64_t who = __builtin_amdgcn_ballot_w64(blocks > kShort);
            while (who) {
                const int m = __builtin_ctzll(who);
                who &= who - 1;
                const int q = __shfl(lq, m), k = __shfl(lk, m), all = __shfl(blocks, m);
                for (int i = lane; i < all; i += 64) visit(first + m, q, k, i);
            }
        }
    };
    each([&](int64_t, int lq, int lk, int i) { atomicAdd(&count[work(lq, lk, i) >> shift], 1ull); });
    __syncthreads();
    // each bucket's first entry: the blocks of all larger ones
    const int64_t mine = (int64_t)count[kBuckets - 1 - tid];
    int64_t upto = mine;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int64_t o = __shfl_up(upto, d);
        if (lane >= d) upto += o;
    }
    if (lane == 63) part[wave] = upto;
    __syncthreads();
    int64_t before = 0;
    for (int w = 0; w < wave; ++w) before += part[w];
    count[kBuckets - 1 - tid] = before + upto - mine;
    if (tid == 1023) a.table[0] = (int)min(before + upto, a.cap);
    __syncthreads();
    each([&](int64_t n, int lq, int lk, int i) {
        const int64_t at = (int64_t)atomicAdd(&count[work(lq, lk, i) >> shift], 1ull);
        if (at >= a.cap) return;  // sequences that overlap
        a.table[2 + 2 * at] = (int)n;
        a.table[3 + 2 * at] = i;
    });
}

}  // namespace

}  // namespace kda

using namespace kda;

bool kda_latent_counted(int64_t seqs, int64_t units) { return seqs <= 64 && units <= 1024; }

hipError_t kda_launch_latent_table(const LatentArgs &a, int size, int32_t *queries, int64_t q_blocks, int32_t *keys, int64_t k_blocks,
                                   hipStream_t s) {
    const TableArgs q{a.cu, a.cuk, a.T, a.Tk, a.seqs, q_blocks, size, 0, a.causal, queries};
    const TableArgs k{a.cu, a.cuk, a.T, a.Tk, a.seqs, k_blocks, size, 1, a.causal, keys};
    hipLaunchKernelGGL(latent_table_kernel, dim3(keys ? 2 : 1), dim3(1024), 0, s, q, k);
    return hipGetLastError();
}

// With eight waves half as much is copied into LDS, but blocks are twice as long: 4096
// and 8192 tokens x 32 heads 178 and 609 us (with four waves 187 and 621); 16384 x 4 heads, 256
// workgroups, 437 (387); 16 sequences of 512 x 32 heads 101 (96).
int kda_latent_block(int64_t B, int64_t T, int64_t H, int64_t seqs) {
    return T * B / seqs >= 2048 && (T + 255) / 256 * B * H >= 512 ? 256 : 128;
}

hipError_t kda_launch_latent_fwd(const LatentArgs &a, int block, hipStream_t s) {
    const int64_t units = a.blocks * a.B * a.H;
    const hipError_t e = launch_groups(units * a.parts, a.launch_cap, [&](int64_t base, dim3 grid) {
        LatentArgs p = a;
        p.base = base;
        if (a.parts > 1) hipLaunchKernelGGL((latent_fwd_kernel<4, true>), grid, dim3(256), 0, s, p);
        else if (block == 128) hipLaunchKernelGGL((latent_fwd_kernel<4, false>), grid, dim3(256), 0, s, p);
        else hipLaunchKernelGGL((latent_fwd_kernel<8, false>), grid, dim3(512), 0, s, p);
    });
    if (e != hipSuccess || a.parts < 2) return e;
    return launch_groups(units * 16, a.launch_cap, [&](int64_t base, dim3 grid) {
        LatentArgs p = a;
        p.base = base;
        hipLaunchKernelGGL(latent_fwd_join_kernel, grid, dim3(64), 0, s, p);
    });
}
