// kda_latent_decode.hip -- latent attention in its absorbed form, over a paged cache
// (kda_latent_decode in include/kda_latent.h).
//
// All heads of a token read the same cached rows, so a workgroup has 32 or 64 rows of
// (token, head) and 64 cached rows at a time in LDS, which serve as keys (576 values)
// and as values (their first 512): 1152 bytes for 2 x 64 x 1088 operations a row.  Up to
// 64 rows the cache's bytes are the bound, beyond that they come from L2.
//
// Steps (64 cached rows of one row tile) of all sequences are lined up and shared out
// evenly among 256 workgroups, one a CU, whatever the lengths: each computes the line
// from the lengths, so that no plan has to be made on the host or launched ahead.  A
// row tile that ends up in several workgroups is joined by a second kernel from their
// fp32 accumulators, maxima and sums.
//
// Of a step, wave w takes the scores of 32 keys for 32 rows (S^T = K Q^T, queries in
// registers), leaves their probabilities in LDS where each lane finds its operand again,
// and then takes 128 of the 512 values of all rows (O^T += V^T P^T).  The copies of the
// next 64 rows run meanwhile.
//
// Precision: as in the expanded form, probabilities are rounded to bf16, all else is fp32.
#include "kda_latent_common.h"

namespace kda {

namespace {

constexpr int kSub = kKeys * 128;              // bytes of 64 values of a tile's rows
constexpr int kSubs = kRow / 64;
constexpr int kWaveDims = kLat / 4;

struct DecodeSmem {
    uint16_t row[2][kSubs][kKeys * 64];
    u4v p[2][2][2][64];                        // [32 rows][32 keys][16 keys][lane]
    float top[2][2][32], sum[2][2][32];        // [32 rows][32 keys][row]
    int rise[2];
    int64_t wave_sum[4];
    int64_t begin_n, begin_rest;
};

// Copies 16 bytes a lane from p + off into LDS from lds on.
template <int OFF>
__device__ __forceinline__ void copy16_at(const uint16_t *p, uint32_t lds) {
    asm volatile("s_nop 0\n\tglobal_load_lds_dwordx4 %0, off offset:%c2" :: "v"(p), "{m0}"(lds - OFF), "i"(OFF) : "memory");
}

// This thread's two rows (tid / 8 and 32 further) of a tile, chunk tid % 8 of every 128
// bytes, at p[0] and p[1].
__device__ __forceinline__ void copy_rows(const uint16_t *const (&p)[2], uint32_t lds, int wave) {
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        const uint32_t at = lds + r * 4096 + wave * 1024;
        copy16_at<0>(p[r], at);
        copy16_at<128>(p[r], at + kSub);
        copy16_at<256>(p[r], at + 2 * kSub);
        copy16_at<384>(p[r], at + 3 * kSub);
        copy16_at<512>(p[r], at + 4 * kSub);
        copy16_at<640>(p[r], at + 5 * kSub);
        copy16_at<768>(p[r], at + 6 * kSub);
        copy16_at<896>(p[r], at + 7 * kSub);
        copy16_at<1024>(p[r], at + 8 * kSub);
    }
}

template <int R>
__global__ __launch_bounds__(256, 1) void latent_decode_kernel(LatentDecodeArgs a) {
    __shared__ __attribute__((aligned(1024))) DecodeSmem sm;
    const int tid = threadIdx.x, lane = tid & 63, g = lane >> 5;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int64_t w = blockIdx.x;
    const int kh = wave & 1, rh = R == 2 ? wave >> 1 : 0;  // this wave's keys and rows among the scores
    const int64_t top_len = a.max_pages << a.page_shift;
    const auto length = [&](int64_t n) { return clamp64(a.len[n], 0, top_len); };
    const auto tiles_of = [&](int64_t n) { return (length(n) + kKeys - 1) / kKeys; };

    // The line of steps: sequence after sequence, row tile after row tile.  Thread t sums
    // up an even share of the sequences.
    const int64_t share = (a.N + 255) / 256, n0 = min(a.N, tid * share), n1 = min(a.N, n0 + share);
    int64_t sum = 0;
    for (int64_t n = n0; n < n1; ++n) {
        const int64_t t = tiles_of(n) * a.row_tiles;
        sum += t;
        if (t == 0 && w == 0)
            for (int64_t r = 0; r < a.row_tiles; ++r) a.seg[2 * (n * a.row_tiles + r)] = -2;
    }
    int64_t upto = sum;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int64_t o = __shfl_up(upto, d);
        if (lane >= d) upto += o;
    }
    if (lane == 63) sm.wave_sum[wave] = upto;
    if (tid < 2) sm.rise[tid] = 0;
    __syncthreads();
    int64_t total = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (i < wave) upto += sm.wave_sum[i];
        total += sm.wave_sum[i];
    }
    const int64_t per = (total + a.groups - 1) / a.groups;
    const int64_t first = w * per, end = min(total, first + per);
    if (first >= end) return;
    if (upto - sum <= first && first < upto) {
        int64_t at = upto - sum, n = n0;
        for (;; ++n) {
            const int64_t t = tiles_of(n) * a.row_tiles;
            if (first < at + t) break;
            at += t;
        }
        sm.begin_n = n;
        sm.begin_rest = first - at;
    }
    __syncthreads();

    const float c = a.scale * kLog2e;
    const uint32_t lds = lds_addr(sm.row);
    const uint32_t at_k = row_at<128>(lds, lane) + kh * 32 * 128, at_v = col_at<128>(lds, lane) + wave * (kWaveDims / 64) * kSub;
    const int64_t rows = a.T * a.H;
    int64_t n = sm.begin_n, rest = sm.begin_rest, step = first;
    bool opening = true;
    while (step < end) {
        // A segment: tiles t0 .. t1 - 1 of row tile rt of sequence n.
        const int64_t tiles = tiles_of(n), len = length(n);
        if (tiles * a.row_tiles <= rest) {
            ++n;
            rest = 0;
            continue;
        }
        const int64_t rt = rest / tiles, t0 = rest - rt * tiles, t1 = min(tiles, t0 + (end - step));
        const bool alone = t0 == 0 && t1 == tiles;

        const int64_t row = (rt * R + rh) * 32 + (lane & 31), tok = min(row, rows - 1) / a.H, head = min(row, rows - 1) - tok * a.H;
        const int64_t seen = clamp64(len - a.T + 1 + tok, 0, len);
        const int64_t all_see = clamp64(len - a.T + 1 + rt * R * 32 / a.H, 0, len);  // keys that the tile's first row sees
        s8 q[kRow / 16];
        {
            const uint16_t *ql = a.ql + n * a.qln + tok * a.qlt + head * a.qlh + 8 * g;
            const uint16_t *qp = a.qp + n * a.qpn + tok * a.qpt + head * a.qph + 8 * g;
#pragma unroll
            for (int ks = 0; ks < kRow / 16; ++ks)
                q[ks] = ks < kLat / 16 ? *reinterpret_cast<const s8 *>(ql + 16 * ks) : *reinterpret_cast<const s8 *>(qp + 16 * ks - kLat);
        }
        f16v o[R][kWaveDims / 32];
        float m[R], l = 0.0f;  // m: of rows lane % 32 of each 32-row tile; l: of this wave's keys and rows

        // Where this thread's rows of tile t lie; rows behind the length take the last one's place.
        int32_t page[2];
        const auto look_up = [&](int64_t t) {
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const int64_t pos = min(t * kKeys + (tid >> 3) + 32 * r, len - 1);
                page[r] = a.table[n * a.max_pages + (pos >> a.page_shift)];
            }
        };
        const auto copy = [&](int64_t t) {
            const uint16_t *p[2];
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const int i = (tid >> 3) + 32 * r;
                const int64_t pos = min(t * kKeys + i, len - 1);
                const int64_t slot = (clamp64(page[r], 0, a.pages - 1) << a.page_shift) + (pos & ((int64_t(1) << a.page_shift) - 1));
                p[r] = a.cache + slot * kRow + (((tid & 7) ^ swap(i)) << 3);
            }
            copy_rows(p, lds + (uint32_t)(t & 1) * (uint32_t)sizeof(sm.row[0]), wave);
        };

        // apart: hidden keys' NaNs and infinities are kept from the rows that do not see them
        // (as in the expanded form: the segment runs again with them added apart).
        for (int apart = 0; apart < 2; ++apart) {
#pragma unroll
            for (int r = 0; r < R; ++r) {
                m[r] = -INFINITY;
#pragma unroll
                for (int d = 0; d < kWaveDims / 32; ++d) o[r][d] = zero16();
            }
            l = 0.0f;
            look_up(t0);
            copies_done();  // the last segment's reads, too
            copy(t0);
            look_up(min(t0 + 1, tiles - 1));
#pragma unroll 1
            for (int64_t t = t0; t < t1; ++t) {
                copies_done();
                if (t + 1 < t1) {
                    copy(t + 1);
                    look_up(min(t + 2, tiles - 1));
                }
                const uint32_t buf = (uint32_t)(t & 1) * (uint32_t)sizeof(sm.row[0]);
                // scores
                f16v s, s2;
                {
                    constexpr int kAhead = 6;
                    const uint32_t k = at_k + buf;
                    s8 ring[kAhead];
#pragma unroll
                    for (int i = 0; i < kAhead; ++i) ring[i] = row_operand<128>(k + (i >> 2) * kSub, 0, i & 3);
                    s = s2 = zero16();
#pragma unroll
                    for (int i = 0; i < kRow / 16; ++i) {
                        if (i & 1) s2 = mfma32(ring[i % kAhead], q[i], s2);
                        else s = mfma32(ring[i % kAhead], q[i], s);
                        const int x = i + kAhead;
                        if (x < kRow / 16) ring[i % kAhead] = row_operand<128>(k + (x >> 2) * kSub, 0, x & 3);
                        __builtin_amdgcn_sched_barrier(0);
                    }
                }
                float top = -INFINITY;
#pragma unroll
                for (int i = 0; i < 16; ++i) s[i] += s2[i];
                if ((t + 1) * kKeys > all_see) {
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const int64_t key = t * kKeys + kh * 32 + 8 * (i / 4) + 4 * g + i % 4;
                        s[i] = key < seen ? s[i] : -INFINITY;
                    }
                }
#pragma unroll
                for (int i = 0; i < 16; ++i) top = fmaxf(top, s[i]);
                top = pair_max(top) * c;
                const bool mine = R == 2 || wave < 2;  // with 32 rows, waves 2 and 3 have the scores of 0 and 1 again
                // Probabilities by the maximum in use, which may stay 2^40 behind the true one (bf16
                // has fp32's exponents, so that nothing is lost): only a larger step, as in a segment's first
                // tile, makes the waves agree on new maxima first.
                constexpr float kSlack = 40.0f;
                const bool need = top > m[rh] + kSlack;
                if (g == 0) sm.top[rh][kh][lane & 31] = top;
                if (__builtin_amdgcn_ballot_w64(need) != 0 && lane == 0) sm.rise[t & 1] = 1;
                float part = 0.0f;
                const auto probabilities = [&]() {
                    const float x = m[rh] == -INFINITY ? 0.0f : m[rh];
                    f16v e;
                    part = 0.0f;
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        e[i] = __builtin_amdgcn_exp2f(fmaf(s[i], c, -x));
                        part += e[i];
                    }
                    if (mine) {
                        sm.p[rh][kh][0][lane] = __builtin_bit_cast(u4v, pack8(e, 0));
                        sm.p[rh][kh][1][lane] = __builtin_bit_cast(u4v, pack8(e, 1));
                    }
                };
                probabilities();
                lds_barrier();
                if (sm.rise[t & 1]) {
#pragma unroll
                    for (int r = 0; r < R; ++r) {
                        const float x = fmaxf(m[r], fmaxf(sm.top[r][0][lane & 31], sm.top[r][1][lane & 31]));
                        const float f = x == -INFINITY ? 1.0f : __builtin_amdgcn_exp2f(m[r] - x);
                        if (r == rh) l *= f;
                        m[r] = x;
#pragma unroll
                        for (int d = 0; d < kWaveDims / 32; ++d)
#pragma unroll
                            for (int i = 0; i < 16; ++i) o[r][d][i] *= f;
                    }
                    probabilities();
                    lds_barrier();
                    if (tid == 0) sm.rise[t & 1] = 0;  // set again two tiles on
                }
                l += part;
                if (apart && (t + 1) * kKeys > all_see) {
#pragma unroll 1
                    for (int i = 0; i < kKeys; ++i) {
                        const int64_t key = t * kKeys + i;
#pragma unroll
                        for (int e = 0; e < kWaveDims / 8; ++e) {
                            const uint16_t *x = sm.row[t & 1][wave * (kWaveDims / 64) + (e >> 3)] + i * 64 + (((e & 7) ^ swap(i)) << 3) + 4 * g;
                            const u2v v = *reinterpret_cast<const u2v *>(x);
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                const uint32_t b = (v[j / 2] >> (16 * (j & 1))) & 0xffffu;
                                const float f = (b & 0x7f80u) == 0x7f80u ? bf16_bits_to_f32(b) : 0.0f;
#pragma unroll
                                for (int r = 0; r < R; ++r) {
                                    const int64_t k = min((rt * R + r) * 32 + (lane & 31), rows - 1) / a.H;
                                    o[r][e / 4][4 * (e % 4) + j] += key < len - a.T + 1 + k ? f : 0.0f;
                                }
                            }
                        }
                    }
                    __syncthreads();
                    uint32_t *x = reinterpret_cast<uint32_t *>(sm.row[t & 1]);
                    for (int i = tid; i < kLat / 64 * kSub / 4; i += 256) {
                        uint32_t v = x[i];
                        if ((v & 0x7f80u) == 0x7f80u) v &= 0xffff0000u;
                        if ((v >> 16 & 0x7f80u) == 0x7f80u) v &= 0x0000ffffu;
                        x[i] = v;
                    }
                    __syncthreads();
                }
                // outputs
                {
                    constexpr int kSlots = 4 * kWaveDims / 32, kAhead = 4;
                    const uint32_t v = at_v + buf;
                    s8 p[R][4], ring[kAhead];
#pragma unroll
                    for (int r = 0; r < R; ++r)
#pragma unroll
                        for (int ks = 0; ks < 4; ++ks) p[r][ks] = __builtin_bit_cast(s8, sm.p[r][ks >> 1][ks & 1][lane]);
                    const auto operand = [&](int i) {
                        const int d = i % (kWaveDims / 32);
                        return col_operand<128>(v + (d >> 1) * kSub, i / (kWaveDims / 32), d & 1);
                    };
#pragma unroll
                    for (int i = 0; i < kAhead; ++i) ring[i] = operand(i);
#pragma unroll
                    for (int i = 0; i < kSlots; ++i) {
#pragma unroll
                        for (int r = 0; r < R; ++r)
                            o[r][i % (kWaveDims / 32)] = mfma32(ring[i % kAhead], p[r][i / (kWaveDims / 32)], o[r][i % (kWaveDims / 32)]);
                        if (i + kAhead < kSlots) ring[i % kAhead] = operand(i + kAhead);
                        __builtin_amdgcn_sched_barrier(0);
                    }
                }
            }
            if (apart || t1 * kKeys <= all_see || a.T == 1) break;
            float odd = 0.0f;
#pragma unroll
            for (int r = 0; r < R; ++r)
#pragma unroll
                for (int d = 0; d < kWaveDims / 32; ++d)
#pragma unroll
                    for (int i = 0; i < 16; ++i) odd = fmaf(o[r][d][i], 0.0f, odd);
            __syncthreads();
            if (tid == 0) sm.begin_n = 0;
            __syncthreads();
            if (!(odd == 0.0f)) sm.begin_n = 1;
            __syncthreads();
            if (!sm.begin_n) break;
        }

        // The sums of both halves of the keys.
        const float half = pair_sum(l);
        __syncthreads();
        if (g == 0) sm.sum[rh][kh][lane & 31] = half;
        __syncthreads();
        if (alone) {
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const int64_t i = (rt * R + r) * 32 + (lane & 31);
                const float z = sm.sum[r][0][lane & 31] + sm.sum[r][1][lane & 31];
                const float f = z == 0.0f ? 0.0f : 1.0f / z;
                if (i >= rows) continue;
                uint16_t *out = a.out + (n * rows + i) * kLat + wave * kWaveDims + 4 * g;
#pragma unroll
                for (int d = 0; d < kWaveDims / 32; ++d)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const u2v x = {pack2(o[r][d][4 * e] * f, o[r][d][4 * e + 1] * f), pack2(o[r][d][4 * e + 2] * f, o[r][d][4 * e + 3] * f)};
                        *reinterpret_cast<u2v *>(out + 32 * d + 8 * e) = x;
                    }
                if (a.lse && g == 0 && wave == 0)
                    a.lse[n * rows + i] = z == 0.0f ? -INFINITY : (m[r] + __builtin_amdgcn_logf(z)) * kLn2;
            }
            if (tid == 0) a.seg[2 * (n * a.row_tiles + rt)] = -1;
        } else {
            const int64_t slot = 2 * w + (opening ? 0 : 1);
#pragma unroll
            for (int r = 0; r < R; ++r) {
                f4 *p = reinterpret_cast<f4 *>(a.part) + ((slot * 4 + wave) * R + r) * (kWaveDims / 8 * 64) + lane;
#pragma unroll
                for (int d = 0; d < kWaveDims / 32; ++d)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        p[(4 * d + e) * 64] = f4{o[r][d][4 * e], o[r][d][4 * e + 1], o[r][d][4 * e + 2], o[r][d][4 * e + 3]};
                if (g == 0 && wave == 0) {
                    float *st = a.part_stat + (slot * R + r) * 64 + lane;
                    st[0] = m[r];
                    st[32] = sm.sum[r][0][lane] + sm.sum[r][1][lane];
                }
            }
            if (t0 == 0 && tid == 0) {
                a.seg[2 * (n * a.row_tiles + rt)] = (int32_t)slot;
                a.seg[2 * (n * a.row_tiles + rt) + 1] = (int32_t)((step + tiles - 1) / per);
            }
        }
        step += t1 - t0;
        rest += t1 - t0;
        opening = false;
    }
}

// The parts of a row tile added up: a workgroup has 4 values of lane rows of every 32-row
// tile, (wave, values) piece of 64 accumulators lanes each; its four waves take every
// fourth part and are added in their order.
template <int R>
__global__ __launch_bounds__(256) void latent_join_kernel(LatentDecodeArgs a, int64_t base) {
    __shared__ f4 acc[4][R][64];
    __shared__ float tops[4][R][32], sums[4][R][32];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, n32 = lane & 31;
    const int64_t unit = base + blockIdx.x, tile = unit >> 6;
    const int piece = (int)(unit & 63), pw = piece >> 4, pv = piece & 15;  // wave and group of values
    const int32_t head = a.seg[2 * tile];
    if (head == -1) return;
    const int64_t rows = a.T * a.H, n = tile / a.row_tiles, rt = tile - n * a.row_tiles;
    f4 o[R];
    float m[R], l[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        o[r] = f4{0.0f, 0.0f, 0.0f, 0.0f};
        m[r] = -INFINITY;
        l[r] = 0.0f;
    }
    if (head >= 0) {
        const int64_t w0 = head >> 1, w1 = a.seg[2 * tile + 1];
        const auto slot_of = [&](int64_t w) { return w == w0 ? (int64_t)head : 2 * w; };
#pragma unroll 4
        for (int64_t w = w0 + wave; w <= w1; w += 4)
#pragma unroll
            for (int r = 0; r < R; ++r) m[r] = fmaxf(m[r], a.part_stat[(slot_of(w) * R + r) * 64 + n32]);
        if (lane < 32)
#pragma unroll
            for (int r = 0; r < R; ++r) tops[wave][r][lane] = m[r];
        __syncthreads();
#pragma unroll
        for (int r = 0; r < R; ++r) m[r] = fmaxf(fmaxf(tops[0][r][n32], tops[1][r][n32]), fmaxf(tops[2][r][n32], tops[3][r][n32]));
#pragma unroll 4
        for (int64_t w = w0 + wave; w <= w1; w += 4)
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const int64_t s = slot_of(w);
                const float *st = a.part_stat + (s * R + r) * 64 + n32;
                const float f = m[r] == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(st[0] - m[r]);
                o[r] += reinterpret_cast<const f4 *>(a.part)[((s * 4 + pw) * R + r) * (kWaveDims / 8 * 64) + pv * 64 + lane] * f;
                l[r] += st[32] * f;
            }
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
        acc[wave][r][lane] = o[r];
        if (lane < 32) sums[wave][r][lane] = l[r];
    }
    __syncthreads();
    if (wave >= R) return;
    const int r = wave;
    const int64_t i = (rt * R + r) * 32 + n32;
    if (i >= rows) return;
    const f4 x = (acc[0][r][lane] + acc[1][r][lane]) + (acc[2][r][lane] + acc[3][r][lane]);
    const float z = (sums[0][r][n32] + sums[1][r][n32]) + (sums[2][r][n32] + sums[3][r][n32]);
    const float f = z == 0.0f ? 0.0f : 1.0f / z;
    uint16_t *out = a.out + (n * rows + i) * kLat + pw * kWaveDims + 32 * (pv >> 2) + 8 * (pv & 3) + 4 * (lane >> 5);
    *reinterpret_cast<u2v *>(out) = u2v{pack2(x[0] * f, x[1] * f), pack2(x[2] * f, x[3] * f)};
    float top = -INFINITY;
#pragma unroll
    for (int q = 0; q < R; ++q) top = q == r ? m[q] : top;
    if (a.lse && piece == 0 && lane < 32) a.lse[n * rows + i] = z == 0.0f ? -INFINITY : (top + __builtin_amdgcn_logf(z)) * kLn2;
}

}  // namespace

}  // namespace kda

using namespace kda;

hipError_t kda_launch_latent_decode(const LatentDecodeArgs &a, hipStream_t s) {
    const dim3 grid((unsigned)a.groups);
    if (a.rows32 == 1) hipLaunchKernelGGL(latent_decode_kernel<1>, grid, dim3(256), 0, s, a);
    else hipLaunchKernelGGL(latent_decode_kernel<2>, grid, dim3(256), 0, s, a);
    return hipGetLastError();
}

hipError_t kda_launch_latent_join(const LatentDecodeArgs &a, hipStream_t s) {
    return launch_groups(a.N * a.row_tiles * 64, 0, [&](int64_t base, dim3 grid) {
        if (a.rows32 == 1) hipLaunchKernelGGL(latent_join_kernel<1>, grid, dim3(256), 0, s, a, base);
        else hipLaunchKernelGGL(latent_join_kernel<2>, grid, dim3(256), 0, s, a, base);
    });
}
