// kda_latent_decode.hip -- latent attention in its absorbed form, over a paged cache
// (kda_latent_decode in include/kda_latent.h).
//
// All heads of a token read the same cached rows, so a workgroup has 32 or 64 rows of
// (token, head) and 32 cached rows at a time in LDS, which serve as keys (576 values)
// and as values (their first 512): 1152 bytes for 2 x 64 x 1088 operations a row.
//
// With 32 rows the cache's bytes are the bound: 64 requests of 4096 rows, 32 heads, take
// 57 us for 286 MB, 7 of them until the first rows are there, and their joining 7.  With 64
// rows a step's chain of scores, exponentials and barrier takes 1.3 us, for which its rows
// come at 7 TB/s: enough where a sequence has one row tile; with two, one request of 131072
// rows and 128 heads takes 53 to 60 us and its joining 8 (its bytes 25).
//
// Steps (32 cached rows of one row tile) of all sequences are lined up and shared out
// evenly among 256 workgroups, one a CU, whatever the lengths (with an allowance for the
// changes from one row tile to the next): each computes the line from the lengths, so that
// no plan has to be made on the host or launched ahead.  A
// row tile that ends up in several workgroups is joined by a second kernel from their
// fp32 accumulators, maxima and sums.
//
// A workgroup's steps are one stream, across sequences: four waves take the scores of
// step i (S^T = K Q^T, queries in registers) and leave the probabilities in LDS, four
// take the outputs of step i - 1 (O^T += V^T P^T, 128 of the 512 values each), and the copies
// of the steps i + 1 and i + 2 run meanwhile, with one barrier a step.  (Each SIMD has a
// wave of either kind; waves that do both need more registers than they have, or twice
// the LDS reads.)  The table's entries are copied into LDS two steps ahead of the rows.
//
// Precision: as in the expanded form, probabilities are rounded to bf16, all else is fp32.
#include <type_traits>
#include "kda_latent_common.h"

namespace kda {

namespace {

constexpr int kStep = 32;                      // cached rows a step
constexpr int kSub = kStep * 128;              // bytes of 64 values of a step's rows
constexpr int kSubs = kRow / 64;
constexpr int kBuffers = 4, kEntries = 8;      // steps in LDS; steps whose table entries are
constexpr int kOutWaves = 4;
constexpr int kWaveDims = kLat / kOutWaves;    // values of an output wave

struct DecodeSmem {
    uint16_t row[kBuffers][kSubs][kStep * 64];
    uint16_t p[2][64 * kStep];                 // [row][key], 16-byte chunk c of row r at c ^ (r / 4 % 4)
    int32_t entry[kEntries][64];               // page of every row of a step (32 of them)
    float top[2][64], sum[2][2][64];           // [half of the keys][row]; of two segments
    int rise[2];
    int64_t wave_sum[8];
    int wave_tiles[8];
    int64_t begin_rest, real[2];               // steps of all workgroups ahead of this one's, and with it
    int begin_n, begin_len, uneven;
};

// Chunk c of row r lies at place c ^ place(r) of its 128 bytes: reads of 16 bytes of 16
// rows, and transposing ones of 64 bytes of 4 rows, are without bank conflicts.
__device__ __forceinline__ int place(int r) { return ((r >> 1 & 1) << 2) | ((r >> 2) & 3); }

// Copies 16 bytes a lane from p + OFF into LDS from lds on.
template <int OFF>
__device__ __forceinline__ void copy16_at(const uint16_t *p, uint32_t lds) {
    asm volatile("s_nop 0\n\tglobal_load_lds_dwordx4 %0, off offset:%c2" :: "v"(p), "{m0}"(lds - OFF), "i"(OFF) : "memory");
}

// Waits until at most `left` of the wave's memory operations (the youngest) and none of its LDS
// accesses are under way, then for the other waves.
template <int LEFT>
__device__ __forceinline__ void arrive() {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(0x0070 | LEFT);
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

// The values of lanes n, n + 16, n + 32 and n + 48, combined in all of them.
__device__ __forceinline__ float quad_max(float x) {
    const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return pair_max(fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1])));
}
__device__ __forceinline__ float quad_sum(float x) {
    const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return pair_sum(__uint_as_float(r[0]) + __uint_as_float(r[1]));
}

// Scales from one maximum in use to another.
__device__ __forceinline__ float rescale(float from, float to) { return to == -INFINITY ? 1.0f : __builtin_amdgcn_exp2f(from - to); }

// A position in the line of steps.  Lengths are read by scalar loads, which are not
// counted with the copies.
typedef const __attribute__((address_space(4))) int64_t *const_i64;
struct Cursor {
    int n, rt, t;              // sequence, row tile, step within it
    int len, steps;            // of the sequence
};
__device__ __forceinline__ int length_of(const LatentDecodeArgs &a, int64_t n) {
    return (int)clamp64(reinterpret_cast<const_i64>(reinterpret_cast<uintptr_t>(a.len))[n], 0, a.max_pages << a.page_shift);
}
__device__ __forceinline__ void advance(const LatentDecodeArgs &a, Cursor &x) {
    if (++x.t < x.steps) return;
    x.t = 0;
    if (++x.rt < a.row_tiles) return;
    x.rt = 0;
    do {
        if (++x.n >= a.N) return;  // behind the last step
        x.len = length_of(a, x.n);
        x.steps = (x.len + kStep - 1) / kStep;
    } while (x.steps == 0);
}

// The copies of a step: this thread's row among the step's, from its table entry.  The
// score waves take the even 64-value parts, the output waves the odd ones.
template <bool EVEN>
__device__ __forceinline__ void copy_step(const LatentDecodeArgs &a, const Cursor &x, int32_t page, int row, int chunk, uint32_t lds) {
    const int pos = min(x.t * kStep + row, x.len - 1);  // rows behind the length: the last one again
    const uint32_t slot = ((uint32_t)min(max(page, 0), (int)a.pages - 1) << a.page_shift) + (pos & ((1 << a.page_shift) - 1));
    const uint16_t *p = a.cache + (uint64_t)slot * kRow + ((chunk ^ place(row)) << 3);
    if (EVEN) {
        copy16_at<0>(p, lds);
        copy16_at<256>(p, lds + 2 * kSub);
        copy16_at<512>(p, lds + 4 * kSub);
        copy16_at<768>(p, lds + 6 * kSub);
        copy16_at<1024>(p, lds + 8 * kSub);
    } else {
        copy16_at<128>(p, lds + kSub);
        copy16_at<384>(p, lds + 3 * kSub);
        copy16_at<640>(p, lds + 5 * kSub);
        copy16_at<896>(p, lds + 7 * kSub);
    }
}
constexpr int kEvenCopies = 5, kOddCopies = 4;

// What both kinds of waves share: the copies ahead of their work.
template <bool EVEN>
struct Feed {
    Cursor copy, look;         // two and four steps ahead
    int row, chunk;            // this thread's
    uint32_t lds;              // its wave's place in a 64-value part of buffer 0

    // Step i's share: copies of step i + 2, entries of step i + 4.
    __device__ __forceinline__ void ahead(const LatentDecodeArgs &a, DecodeSmem &sm, int i, int count, int tid) {
        if (i + 4 < count) {
            if (tid < 64) {
                const int pos = min(look.t * kStep + (tid & (kStep - 1)), look.len - 1);
                const int32_t *p = a.table + look.n * a.max_pages + (pos >> a.page_shift);
                asm volatile("s_nop 0\n\tglobal_load_lds_dword %0, off" :: "v"(p), "{m0}"(lds_addr(sm.entry[(i + 4) % kEntries])) : "memory");
            }
            advance(a, look);
        }
        if (i + 2 < count) {
            copy_step<EVEN>(a, copy, sm.entry[(i + 2) % kEntries][row], row, chunk, lds + (i + 2) % kBuffers * (uint32_t)sizeof(sm.row[0]));
            advance(a, copy);
        }
    }
};

// R: 32-row tiles of the workgroup's rows, and 16-row tiles of a score wave's.
template <int R>
__global__ __launch_bounds__(512, 2) void latent_decode_kernel(LatentDecodeArgs a) {
    __shared__ __attribute__((aligned(1024))) DecodeSmem sm;
    const int tid = threadIdx.x, lane = tid & 63, g = lane >> 5, n16 = lane & 15, g16 = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int64_t w = blockIdx.x;

    // The line of steps: sequence after sequence, row tile after row tile.  Thread t sums up an even
    // share of the sequences.
    const int64_t share = (a.N + 511) / 512, n0 = min(a.N, tid * share), n1 = min(a.N, n0 + share);
    const auto length = [&](int64_t n) { return clamp64(a.len[n], 0, a.max_pages << a.page_shift); };
    const auto steps_of = [&](int64_t n) { return (length(n) + kStep - 1) / kStep; };  // a row tile's, below 2^26
    int64_t sum = 0;
    int tiles = 0;
    for (int64_t n = n0; n < n1; ++n) {
        const int64_t t = steps_of(n);
        sum += t * a.row_tiles;
        if (t > 0) tiles += (int)a.row_tiles;
        else if (w == 0)
            for (int64_t r = 0; r < a.row_tiles; ++r) a.seg[2 * (n * a.row_tiles + r)] = -2;
    }
    int64_t upto = sum;
    int tiles_upto = tiles;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int64_t o = __shfl_up(upto, d);
        const int p = __shfl_up(tiles_upto, d);
        if (lane >= d) {
            upto += o;
            tiles_upto += p;
        }
    }
    if (lane == 63) {
        sm.wave_sum[wave] = upto;
        sm.wave_tiles[wave] = tiles_upto;
    }
    if (tid < 2) sm.rise[tid] = 0;
    if (tid == 0) sm.uneven = 0;
    __syncthreads();
    int64_t total = 0;
    int all_tiles = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        if (i < wave) {
            upto += sm.wave_sum[i];
            tiles_upto += sm.wave_tiles[i];
        }
        total += sm.wave_sum[i];
        all_tiles += sm.wave_tiles[i];
    }
    // A change to other queries within a workgroup takes about as long as kChange steps: where any has
    // one, as many units without work lie ahead of every row tile (12 sequences of up to 15000 rows x 64: 55
    // -> 44 us; where none has, as with two row tiles of 4096 steps, the units would make it 33 steps a
    // workgroup instead of 32, 66 -> 70 us).
    constexpr int kChange = R == 1 ? 3 : 5;
    {
        const uint32_t even = max((uint32_t)((total + a.groups - 1) / a.groups), 1u);
        for (int64_t n = n0; n < n1; ++n)
            if ((uint32_t)steps_of(n) % even != 0) sm.uneven = 1;
    }
    __syncthreads();
    const int change = sm.uneven ? kChange : 0;
    const int64_t ahead = upto - sum + (int64_t)(tiles_upto - tiles) * change;
    upto += (int64_t)tiles_upto * change;
    total += (int64_t)all_tiles * change;
    const int64_t per = (total + a.groups - 1) / a.groups;
    const int64_t first = w * per, behind = min(total, first + per);
    if (first >= behind) return;
    // A point of the line: its sequence, how far it lies in it, and the steps ahead of it.
    const auto locate = [&](int64_t point, int64_t &n, int64_t &rest) {
        int64_t at = ahead, before = tiles_upto - tiles, t;
        for (n = n0;; ++n) {
            t = steps_of(n);
            const int64_t u = t > 0 ? (t + change) * a.row_tiles : 0;
            if (point < at + u) break;
            at += u;
            if (u > 0) before += a.row_tiles;
        }
        rest = point - at;
        const int64_t unit = t + change, rt = rest >> 32 ? rest / unit : (uint32_t)rest / (uint32_t)unit;
        return point - (before + rt) * change - min(rest - rt * unit, (int64_t)change);
    };
    if (ahead <= first && first < upto) {
        int64_t n, rest;
        sm.real[0] = locate(first, n, rest);
        sm.begin_n = (int)n;
        sm.begin_len = (int)length(n);
        sm.begin_rest = rest;
    }
    if (ahead <= behind && behind < upto) {
        int64_t n, rest;
        sm.real[1] = locate(behind, n, rest);
    }
    if (tid == 0 && behind == total) sm.real[1] = total - (int64_t)all_tiles * change;
    __syncthreads();
    const int count = __builtin_amdgcn_readfirstlane((int)(sm.real[1] - sm.real[0]));
    if (count == 0) return;
    Cursor at;
    at.n = __builtin_amdgcn_readfirstlane(sm.begin_n);
    at.len = __builtin_amdgcn_readfirstlane(sm.begin_len);
    at.steps = (at.len + kStep - 1) / kStep;
    int64_t begin_unit;  // where this workgroup's first step stands in the line
    {
        const int64_t rest = sm.begin_rest;
        const int unit = at.steps + change;
        const int rt = rest >> 32 ? (int)(rest / unit) : (int)((uint32_t)rest / (uint32_t)unit);
        const int within = (int)(rest - (int64_t)rt * unit);
        at.rt = __builtin_amdgcn_readfirstlane(rt);
        at.t = __builtin_amdgcn_readfirstlane(max(0, within - change));
        begin_unit = first + max(0, change - within);
    }

    const uint32_t rows = (uint32_t)(a.T * a.H), H = (uint32_t)a.H;
    const float c = a.scale * kLog2e;
    const uint32_t lds = lds_addr(sm.row), lds_p = lds_addr(sm.p);
    // Keys that a row of a row tile sees; rows behind the last stand for it and are not stored.
    const auto seen_by = [&](const Cursor &x, int row) {
        const uint32_t i = min((uint32_t)(x.rt * R * 32 + row), rows - 1);
        return min(max(x.len - (int)a.T + 1 + (int)(i / H), 0), x.len);
    };

    // The first two steps' copies, and the next two's entries: here every thread reads its row's.
    const int my_row = 8 * (wave & 3) + (lane >> 3);
    Cursor copy = at, look = at;
    int32_t page[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        page[i] = 0;
        if (i < count) {
            page[i] = a.table[look.n * a.max_pages + (min(look.t * kStep + my_row, look.len - 1) >> a.page_shift)];
            advance(a, look);
        }
    }
    // Ahead of them the first segment's queries, by way of the buffers that are still free: where the score
    // waves ask for them, 16 rows a load and twice each, they come later (131072 rows x 128 heads 64 -> 60
    // us, 12 sequences of drafted tokens 41 -> 39).
    constexpr int kQueries = 2;  // first of the buffers
    {
        asm volatile("" ::"v"(page[0]), "v"(page[1]), "v"(page[2]), "v"(page[3]));  // waited for ahead of the copies, not behind them
        const int group = R == 2 ? wave : wave & 3, row = 8 * group + (lane >> 3);
        const uint32_t x = min((uint32_t)(at.rt * R * 32 + row), rows - 1), tok = x / H, head = x - tok * H;
        const int chunk = ((lane & 7) ^ place(row & 31)) << 3;
        const uint16_t *ql = a.ql + at.n * a.qln + (int64_t)tok * a.qlt + (int64_t)head * a.qlh + chunk;
        const uint16_t *qp = a.qp + at.n * a.qpn + (int64_t)tok * a.qpt + (int64_t)head * a.qph + chunk;
        const uint32_t to = lds + (kQueries + (group >> 2)) * (uint32_t)sizeof(sm.row[0]) + (group & 3) * 1024;
        if (R == 2 || wave < 4) {
            copy16_at<0>(ql, to);
            copy16_at<128>(ql, to + kSub);
            copy16_at<256>(ql, to + 2 * kSub);
            copy16_at<384>(ql, to + 3 * kSub);
        }
        if (R == 2 || wave >= 4) {
            copy16_at<512>(ql, to + 4 * kSub);
            copy16_at<640>(ql, to + 5 * kSub);
            copy16_at<768>(ql, to + 6 * kSub);
            copy16_at<896>(ql, to + 7 * kSub);
            copy16_at<0>(qp, to + 8 * kSub);
        }
    }
    const auto first_copies = [&](auto even) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
            if (i < count) {
                copy_step<decltype(even)::value>(a, copy, page[i], my_row, lane & 7, lds + (wave & 3) * 1024 + i * (uint32_t)sizeof(sm.row[0]));
                advance(a, copy);
            }
    };

    // Probabilities use the maximum that is in use, which may stay 2^40 behind the true one
    // (bf16 has fp32's exponents, so that nothing is lost): only a larger step, as at a segment's
    // start, makes all waves agree on new maxima before they go on.
    constexpr float kSlack = 40.0f;

    if (wave < 4) {
        // ---- scores: 16 keys and 16 R rows a wave --------------------------------------
        const int kg = wave >> 1, r0 = (wave & 1) * 16 * R;
        const uint32_t at_k = lds + (kg * 16 + n16) * 128 + ((g16 ^ place(n16)) << 4);
        s8 q[R][kRow / 32];
        int seen[R], all_see = 0, segment = 0;
        float m[R], l[R];
        const auto begin_segment = [&]() {
            all_see = seen_by(at, 0);
#pragma unroll
            for (int r = 0; r < R; ++r) {
                seen[r] = seen_by(at, r0 + 16 * r + n16);
                m[r] = -INFINITY;
                l[r] = 0.0f;
            }
        };
        const auto load_queries = [&]() {
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const uint32_t x = min((uint32_t)(at.rt * R * 32 + r0 + 16 * r + n16), rows - 1), tok = x / H, head = x - tok * H;
                const uint16_t *ql = a.ql + at.n * a.qln + (int64_t)tok * a.qlt + (int64_t)head * a.qlh + 8 * g16;
                const uint16_t *qp = a.qp + at.n * a.qpn + (int64_t)tok * a.qpt + (int64_t)head * a.qph + 8 * g16;
#pragma unroll
                for (int ks = 0; ks < kRow / 32; ++ks)
                    q[r][ks] = ks < kLat / 32 ? *reinterpret_cast<const s8 *>(ql + 32 * ks)
                                              : *reinterpret_cast<const s8 *>(qp + 32 * ks - kLat);
            }
        };
        first_copies(std::true_type());
        begin_segment();
        if ((lane & 7) == 0)
#pragma unroll
            for (int i = 2; i < 4; ++i) sm.entry[i][my_row] = page[i];
        Feed<true> feed{copy, look, my_row, lane & 7, lds + (wave & 3) * 1024};
        bool fresh = false;
        if (count > 1) arrive<2 * kEvenCopies>();
        else arrive<kEvenCopies>();
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int row = r0 + 16 * r + n16;
            const uint32_t at_q = lds + (kQueries + (row >> 5)) * (uint32_t)sizeof(sm.row[0]) + (row & 31) * 128 + ((g16 ^ place(row & 31)) << 4);
#pragma unroll
            for (int ks = 0; ks < kRow / 32; ++ks) q[r][ks] = read8((at_q ^ ((ks & 1) << 6)) + (ks >> 1) * kSub);
        }
        if (count > 1) arrive<kEvenCopies>();
        else arrive<0>();
#pragma unroll 1
        for (int i = 0; i <= count; ++i) {
            feed.ahead(a, sm, i, count, tid);
            float part[R];
            f4 s[R];
            const bool last = i == count - 1 || at.t == at.steps - 1;
            const auto probabilities = [&]() {
                const uint32_t put = lds_p + (i & 1) * (uint32_t)sizeof(sm.p[0]);
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    const int row = r0 + 16 * r + n16;
                    const float x = m[r] == -INFINITY ? 0.0f : m[r];
                    float e[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) e[k] = __builtin_amdgcn_exp2f(fmaf(s[r][k], c, -x));
                    part[r] = (e[0] + e[1]) + (e[2] + e[3]);
                    *reinterpret_cast<__attribute__((address_space(3))) u2v *>(
                        put + row * 64 + (((2 * kg + (g16 >> 1)) ^ (row >> 2 & 3)) << 4) + (g16 & 1) * 8) = u2v{pack2(e[0], e[1]), pack2(e[2], e[3])};
                    if (last) {
                        const float z = quad_sum(l[r] + part[r]);
                        if (g16 == 0) sm.sum[segment & 1][kg][row] = z;
                    }
                }
            };
            if (i < count) {
                if (fresh) {
                    // Waited for here, once a segment: at their uses, every step would wait, and with
                    // them for the copies.
                    begin_segment();
                    load_queries();
                    asm volatile("" ::: "memory");
                    __builtin_amdgcn_s_waitcnt(0x0f70);  // vmcnt(0)
                    asm volatile("" ::: "memory");
                }
                // One 16-row tile has two sums, two have one each: every second product waits for none.
                constexpr int kAhead = 5;
                const uint32_t k = at_k + i % kBuffers * (uint32_t)sizeof(sm.row[0]);
                const auto operand = [&](int x) { return read8((k ^ ((x & 1) << 6)) + (x >> 1) * kSub); };
                s8 ring[kAhead];
                f4 sums[2];
#pragma unroll
                for (int x = 0; x < kAhead; ++x) ring[x] = operand(x);
                sums[0] = sums[1] = f4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                for (int x = 0; x < kRow / 32; ++x) {
#pragma unroll
                    for (int r = 0; r < R; ++r)
                        sums[R == 1 ? x & 1 : r] = mfma16x16x32_bf16(ring[x % kAhead], q[r][x], sums[R == 1 ? x & 1 : r]);
                    if (x + kAhead < kRow / 32) ring[x % kAhead] = operand(x + kAhead);
                    __builtin_amdgcn_sched_barrier(0);
                }
                s[0] = R == 1 ? sums[0] + sums[1] : sums[0];
                if (R == 2) s[R - 1] = sums[1];
                if ((at.t + 1) * kStep > all_see) {
#pragma unroll
                    for (int r = 0; r < R; ++r)
#pragma unroll
                        for (int x = 0; x < 4; ++x) s[r][x] = at.t * kStep + kg * 16 + 4 * g16 + x < seen[r] ? s[r][x] : -INFINITY;
                }
                bool need = false;
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    const float top = quad_max(fmaxf(fmaxf(s[r][0], s[r][1]), fmaxf(s[r][2], s[r][3]))) * c;
                    if (g16 == 0) sm.top[kg][r0 + 16 * r + n16] = top;
                    need |= top > m[r] + kSlack;
                }
                if (__builtin_amdgcn_ballot_w64(need) != 0 && lane == 0) sm.rise[i & 1] = 1;
                probabilities();
            }
            if (i + 2 < count) arrive<kEvenCopies>();
            else arrive<0>();
            if (i < count) {
                if (sm.rise[i & 1]) {
#pragma unroll
                    for (int r = 0; r < R; ++r) {
                        const int row = r0 + 16 * r + n16;
                        const float x = fmaxf(m[r], fmaxf(sm.top[0][row], sm.top[1][row]));
                        l[r] *= rescale(m[r], x);
                        m[r] = x;
                    }
                    probabilities();
                    lds_barrier();
                    if (tid == 0) sm.rise[i & 1] = 0;  // set again two steps on
                }
#pragma unroll
                for (int r = 0; r < R; ++r) l[r] += part[r];
                fresh = at.t == at.steps - 1;
                segment += fresh;
                advance(a, at);
            }
        }
    } else {
        // ---- outputs: 128 values of all rows a wave -------------------------------------
        first_copies(std::false_type());
        Feed<false> feed{copy, look, my_row, lane & 7, lds + (wave & 3) * 1024};
        const int ow = wave - 4;
        const int vr = 8 * g + (n16 >> 2);  // keys 8 g .. of every 16, by two reads of 4 keys each
        const uint32_t at_v = lds + ow * (kWaveDims / 64) * kSub + vr * 128 + (((2 * (g16 & 1) + ((n16 & 3) >> 1)) ^ place(vr)) << 4) + (n16 & 1) * 8;
        const int pr = lane & 31;
        const uint32_t at_p = lds_p + pr * 64 + ((g ^ (pr >> 2 & 3)) << 4);
        f16v o[R][kWaveDims / 32];
        float m[R];
        int segment = 0, begin = 0;  // begin: the segment's first step
        const auto reset = [&]() {
#pragma unroll
            for (int r = 0; r < R; ++r) {
                m[r] = -INFINITY;
#pragma unroll
                for (int d = 0; d < kWaveDims / 32; ++d) o[r][d] = zero16();
            }
        };
        reset();
        if (count > 1) arrive<2 * kOddCopies>();
        else arrive<kOddCopies>();
        if (count > 1) arrive<kOddCopies>();
        else arrive<0>();
#pragma unroll 1
        for (int i = 0; i <= count; ++i) {
            feed.ahead(a, sm, i, count, tid);
            if (i > 0) {  // step i - 1, at `at`
                const int x = i - 1, buf = x % kBuffers;
                if ((at.t + 1) * kStep > seen_by(at, 0)) {
                    // Hidden keys: their values meet zero probabilities.  Where any of the wave's is NaN or
                    // infinite, those are added apart, to the rows that see their keys, and then taken as zeros.
                    u4v *v = reinterpret_cast<u4v *>(sm.row[buf][ow * (kWaveDims / 64)]);
                    bool odd = false;
                    for (int y = lane; y < kWaveDims / 64 * kSub / 16; y += 64) {
                        const u4v z = v[y];
#pragma unroll
                        for (int k = 0; k < 4; ++k) odd |= (z[k] & 0x7f80u) == 0x7f80u || (z[k] & 0x7f800000u) == 0x7f800000u;
                    }
                    if (__builtin_amdgcn_ballot_w64(odd) != 0) {
                        int sees[R];
#pragma unroll
                        for (int r = 0; r < R; ++r) sees[r] = seen_by(at, 32 * r + pr);
#pragma unroll 1
                        for (int k = 0; k < kStep; ++k) {
#pragma unroll
                            for (int e = 0; e < kWaveDims / 8; ++e) {
                                const uint16_t *y = sm.row[buf][ow * (kWaveDims / 64) + (e >> 3)] + k * 64 + (((e & 7) ^ place(k)) << 3) + 4 * g;
                                const u2v z = *reinterpret_cast<const u2v *>(y);
#pragma unroll
                                for (int j = 0; j < 4; ++j) {
                                    const uint32_t b = (z[j / 2] >> (16 * (j & 1))) & 0xffffu;
                                    const float f = (b & 0x7f80u) == 0x7f80u ? bf16_bits_to_f32(b) : 0.0f;
#pragma unroll
                                    for (int r = 0; r < R; ++r) o[r][e / 4][4 * (e % 4) + j] += at.t * kStep + k < sees[r] ? f : 0.0f;
                                }
                            }
                        }
                        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
                        uint32_t *y = reinterpret_cast<uint32_t *>(v);
                        for (int k = lane; k < kWaveDims / 64 * kSub / 4; k += 64) {
                            uint32_t z = y[k];
                            if ((z & 0x7f80u) == 0x7f80u) z &= 0xffff0000u;
                            if ((z & 0x7f800000u) == 0x7f800000u) z &= 0x0000ffffu;
                            y[k] = z;
                        }
                        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
                    }
                }
                constexpr int kSlots = kStep / 16 * kWaveDims / 32, kAhead = 3;
                const uint32_t v = at_v + buf * (uint32_t)sizeof(sm.row[0]);
                const auto operand = [&](int y) {
                    const int d = y % (kWaveDims / 32);
                    const uint32_t z = (v ^ ((d & 1) << 6)) + (d >> 1) * kSub + y / (kWaveDims / 32) * 16 * 128;
                    return read_tr(z, (z ^ 16) + 4 * 128);
                };
                s8 p[R][2], ring[kAhead];
#pragma unroll
                for (int ks = 0; ks < 2; ++ks)
#pragma unroll
                    for (int r = 0; r < R; ++r) p[r][ks] = read8((at_p ^ (ks << 5)) + (x & 1) * (uint32_t)sizeof(sm.p[0]) + r * 32 * 64);
#pragma unroll
                for (int y = 0; y < kAhead; ++y) ring[y] = operand(y);
#pragma unroll
                for (int y = 0; y < kSlots; ++y) {
#pragma unroll
                    for (int r = 0; r < R; ++r)
                        o[r][y % (kWaveDims / 32)] = mfma32(ring[y % kAhead], p[r][y / (kWaveDims / 32)], o[r][y % (kWaveDims / 32)]);
                    if (y + kAhead < kSlots) ring[y % kAhead] = operand(y + kAhead);
                    __builtin_amdgcn_sched_barrier(0);
                }
                const bool ends = at.t == at.steps - 1;
                if (ends || i == count) {
                    const int64_t tile = (int64_t)at.n * a.row_tiles + at.rt;
                    const bool begins = at.t - (x - begin) == 0;  // its first step is this workgroup's, too
                    const int64_t slot = 2 * w + (begin == 0 ? 0 : 1);
#pragma unroll
                    for (int r = 0; r < R; ++r) {
                        const float z = sm.sum[segment & 1][0][32 * r + pr] + sm.sum[segment & 1][1][32 * r + pr];
                        const uint32_t j = (uint32_t)(at.rt * R + r) * 32 + pr;
                        if (begins && ends) {
                            const float f = z == 0.0f ? 0.0f : 1.0f / z;
                            if (j >= rows) continue;
                            uint16_t *out = a.out + (at.n * (int64_t)rows + j) * kLat + ow * kWaveDims + 4 * g;
#pragma unroll
                            for (int d = 0; d < kWaveDims / 32; ++d)
#pragma unroll
                                for (int e = 0; e < 4; ++e) {
                                    const u2v y = {pack2(o[r][d][4 * e] * f, o[r][d][4 * e + 1] * f),
                                                   pack2(o[r][d][4 * e + 2] * f, o[r][d][4 * e + 3] * f)};
                                    *reinterpret_cast<u2v *>(out + 32 * d + 8 * e) = y;
                                }
                            if (a.lse && g == 0 && ow == 0)
                                a.lse[at.n * (int64_t)rows + j] = z == 0.0f ? -INFINITY : (m[r] + __builtin_amdgcn_logf(z)) * kLn2;
                        } else {
                            f4 *y = reinterpret_cast<f4 *>(a.part) + ((slot * kOutWaves + ow) * R + r) * (kWaveDims / 8 * 64) + lane;
#pragma unroll
                            for (int d = 0; d < kWaveDims / 32; ++d)
#pragma unroll
                                for (int e = 0; e < 4; ++e)
                                    y[(4 * d + e) * 64] = f4{o[r][d][4 * e], o[r][d][4 * e + 1], o[r][d][4 * e + 2], o[r][d][4 * e + 3]};
                            if (g == 0 && ow == 0) {
                                float *st = a.part_stat + (slot * R + r) * 64 + lane;
                                st[0] = m[r];
                                st[32] = z;
                            }
                        }
                    }
                    if (lane == 0 && ow == 0 && begins) {
                        a.seg[2 * tile] = ends ? -1 : (int32_t)slot;
                        a.seg[2 * tile + 1] = (int32_t)((begin_unit + begin + (int64_t)segment * change + at.steps - 1) / per);
                    }
                    reset();
                    begin = i;
                    ++segment;
                }
                advance(a, at);
            }
            if (i + 2 < count) arrive<kOddCopies>();
            else arrive<0>();
            if (i < count && sm.rise[i & 1]) {
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    const float x = fmaxf(m[r], fmaxf(sm.top[0][32 * r + pr], sm.top[1][32 * r + pr])), f = rescale(m[r], x);
                    m[r] = x;
#pragma unroll
                    for (int d = 0; d < kWaveDims / 32; ++d)
#pragma unroll
                        for (int e = 0; e < 16; ++e) o[r][d][e] *= f;
                }
                lds_barrier();
            }
        }
    }
}

// The parts of a row tile added up: 8 of a wave's values of 32 rows, 4 a lane, with a running
// maximum.  With MANY parts a workgroup's eight waves take every eighth of them, and their sums
// are added in their order; with few each of its waves has values of its own.
constexpr int kJoinWaves = 8;
template <int R, bool MANY>
__global__ __launch_bounds__(64 * kJoinWaves) void latent_join_kernel(LatentDecodeArgs a, int64_t base) {
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, n32 = lane & 31;
    const int64_t unit = MANY ? base + blockIdx.x : (base + blockIdx.x) * kJoinWaves + wave, tile = unit / (64 * R);
    const int piece = (int)(unit & 63), r = (int)(unit / 64 % R);
    const int pw = piece >> 4, pv = piece & 15;  // wave and group of values
    const int32_t head = a.seg[2 * tile];
    if (head == -1) return;
    const int64_t rows = a.T * a.H, n = tile / a.row_tiles, rt = tile - n * a.row_tiles;
    const int64_t i = (rt * R + r) * 32 + n32;
    if (__builtin_amdgcn_ballot_w64(i < rows) == 0) return;
    f4 o = f4{0.0f, 0.0f, 0.0f, 0.0f};
    float m = -INFINITY, l = 0.0f;
    const auto factor = [](float from, float to) { return to == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(from - to); };
    if (head >= 0) {
        const int w0 = head >> 1, w1 = a.seg[2 * tile + 1];
#pragma unroll 8
        for (int w = w0 + (MANY ? wave : 0); w <= w1; w += MANY ? kJoinWaves : 1) {
            const int64_t s = (int64_t)(w == w0 ? head : 2 * w) * R + r;
            const float *st = a.part_stat + s * 64 + n32;
            const f4 x = reinterpret_cast<const f4 *>(a.part)[((s / R * kOutWaves + pw) * R + r) * (kWaveDims / 8 * 64) + pv * 64 + lane];
            const float top = fmaxf(m, st[0]), f = factor(m, top), e = factor(st[0], top);
            o = o * f + x * e;
            l = l * f + st[32] * e;
            m = top;
        }
    }
    if (MANY) {
        __shared__ f4 acc[kJoinWaves][64];
        __shared__ float tops[kJoinWaves][32], sums[kJoinWaves][32];
        acc[wave][lane] = o;
        if (lane < 32) {
            tops[wave][lane] = m;
            sums[wave][lane] = l;
        }
        __syncthreads();
        if (wave > 0) return;
#pragma unroll
        for (int w = 1; w < kJoinWaves; ++w) m = fmaxf(m, tops[w][n32]);
        o = f4{0.0f, 0.0f, 0.0f, 0.0f};
        l = 0.0f;
#pragma unroll
        for (int w = 0; w < kJoinWaves; ++w) {
            const float f = factor(tops[w][n32], m);
            o += acc[w][lane] * f;
            l += sums[w][n32] * f;
        }
    }
    if (i >= rows) return;
    const float f = l == 0.0f ? 0.0f : 1.0f / l;
    uint16_t *out = a.out + (n * rows + i) * kLat + pw * kWaveDims + 32 * (pv >> 2) + 8 * (pv & 3) + 4 * (lane >> 5);
    *reinterpret_cast<u2v *>(out) = u2v{pack2(o[0] * f, o[1] * f), pack2(o[2] * f, o[3] * f)};
    if (a.lse && piece == 0 && lane < 32) a.lse[n * rows + i] = l == 0.0f ? -INFINITY : (m + __builtin_amdgcn_logf(l)) * kLn2;
}

}  // namespace

}  // namespace kda

using namespace kda;

hipError_t kda_launch_latent_decode(const LatentDecodeArgs &a, hipStream_t s) {
    const dim3 grid((unsigned)a.groups);
    if (a.rows32 == 1) hipLaunchKernelGGL(latent_decode_kernel<1>, grid, dim3(512), 0, s, a);
    else hipLaunchKernelGGL(latent_decode_kernel<2>, grid, dim3(512), 0, s, a);
    return hipGetLastError();
}

hipError_t kda_launch_latent_join(const LatentDecodeArgs &a, hipStream_t s) {
    // A row tile has about groups / (N row_tiles) parts: 128 parts of 64 rows take 8 us by eight waves, 28 by
    // two; with few parts a second wave only costs (64 row tiles of 5 parts: this kernel's and the steps' times
    // 64 -> 63 us, of a call that takes 68; 16 sequences x 128 heads 42 -> 40).
    const bool many = a.N * a.row_tiles * 16 <= a.groups;
    const int64_t units = a.N * a.row_tiles * a.rows32 * 64;
    return launch_groups(many ? units : units / kJoinWaves, 0, [&](int64_t base, dim3 grid) {
        const dim3 block(64 * kJoinWaves);
        if (a.rows32 == 1 && many) hipLaunchKernelGGL((latent_join_kernel<1, true>), grid, block, 0, s, a, base);
        else if (a.rows32 == 1) hipLaunchKernelGGL((latent_join_kernel<1, false>), grid, block, 0, s, a, base);
        else if (many) hipLaunchKernelGGL((latent_join_kernel<2, true>), grid, block, 0, s, a, base);
        else hipLaunchKernelGGL((latent_join_kernel<2, false>), grid, block, 0, s, a, base);
    });
}
