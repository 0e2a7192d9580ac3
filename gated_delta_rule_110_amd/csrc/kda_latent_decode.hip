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
// Of a step, each of eight waves takes the scores of 16 rows (S^T = K Q^T, queries in
// registers) and a quarter or half of the keys, leaves their probabilities in LDS, and
// then takes 64 of the 512 values of all rows (O^T += V^T P^T).  The copies of the next 64
// rows run meanwhile.  (Four waves of larger tiles, or 32 rows a wave among the scores, need
// more than the 256 registers that matrix and vector instructions share: what moves
// between the halves of the file, or to memory and back, then costs more than the LDS reads
// it saves: 64 rows 12 and 5 us a step.)
//
// Precision: as in the expanded form, probabilities are rounded to bf16, all else is fp32.
#include "kda_latent_common.h"

namespace kda {

namespace {

constexpr int kSub = kKeys * 128;              // bytes of 64 values of a tile's rows
constexpr int kSubs = kRow / 64;
constexpr int kWaves = kLat / 64;              // each has 64 values among the outputs

struct DecodeSmem {
    uint16_t row[2][kSubs][kKeys * 64];
    uint16_t p[64 * kKeys];                    // [row][key], 16-byte chunk c of row r at c ^ (r % 8)
    float top[4][64], sum[4][64];              // [group of keys][row]
    int rise[2], odd;
    int64_t wave_sum[kWaves];
    int64_t begin_n, begin_rest;
};

// Copies 16 bytes a lane from p + OFF into LDS from lds on.
template <int OFF>
__device__ __forceinline__ void copy16_at(const uint16_t *p, uint32_t lds) {
    asm volatile("s_nop 0\n\tglobal_load_lds_dwordx4 %0, off offset:%c2" :: "v"(p), "{m0}"(lds - OFF), "i"(OFF) : "memory");
}

// This thread's row (tid / 8) of a tile, chunk tid % 8 of every 128 bytes.
__device__ __forceinline__ void copy_row(const uint16_t *p, uint32_t lds) {
    copy16_at<0>(p, lds);
    copy16_at<128>(p, lds + kSub);
    copy16_at<256>(p, lds + 2 * kSub);
    copy16_at<384>(p, lds + 3 * kSub);
    copy16_at<512>(p, lds + 4 * kSub);
    copy16_at<640>(p, lds + 5 * kSub);
    copy16_at<768>(p, lds + 6 * kSub);
    copy16_at<896>(p, lds + 7 * kSub);
    copy16_at<1024>(p, lds + 8 * kSub);
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

// R: 32-row tiles of the workgroup's rows, and 16-key tiles of a wave's.
template <int R>
__global__ __launch_bounds__(512, 2) void latent_decode_kernel(LatentDecodeArgs a) {
    __shared__ __attribute__((aligned(1024))) DecodeSmem sm;
    const int tid = threadIdx.x, lane = tid & 63, g = lane >> 5, n16 = lane & 15, g16 = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int64_t w = blockIdx.x;
    constexpr int kRowGroups = 2 * R, kKeyGroups = kWaves / kRowGroups;
    const int kg = wave / kRowGroups, k0 = kg * 16 * R, my_row = wave % kRowGroups * 16 + n16;  // the lane's among the scores
    const int64_t top_len = a.max_pages << a.page_shift;
    const auto length = [&](int64_t n) { return clamp64(a.len[n], 0, top_len); };
    const auto tiles_of = [&](int64_t n) { return (length(n) + kKeys - 1) / kKeys; };

    // The line of steps: sequence after sequence, row tile after row tile.  Thread t sums
    // up an even share of the sequences.
    const int64_t share = (a.N + 511) / 512, n0 = min(a.N, tid * share), n1 = min(a.N, n0 + share);
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
    for (int i = 0; i < kWaves; ++i) {
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
    const uint32_t lds = lds_addr(sm.row), lds_p = lds_addr(sm.p);
    // operands: a key's values 8 g16 .. of every 32; the values' columns of keys 8 g .. of every
    // 16 (two reads of 4 keys each); a row's probabilities of those keys
    const uint32_t at_k = lds + (k0 + n16) * 128 + ((g16 ^ swap(n16)) << 4);
    const int vr = 8 * g + (n16 >> 2);
    const uint32_t at_v = lds + wave * kSub + vr * 128 + (((2 * (g16 & 1) + ((n16 & 3) >> 1)) ^ swap(vr)) << 4) + (n16 & 1) * 8;
    const uint32_t at_p = lds_p + (lane & 31) * 128 + ((g ^ (lane & 7)) << 4);
    const uint32_t put_p = lds_p + my_row * 128 + (((2 * R * kg + (g16 >> 1)) ^ (n16 & 7)) << 4) + (g16 & 1) * 8;
    const uint32_t rows = (uint32_t)(a.T * a.H), H = (uint32_t)a.H;
    int64_t n = __builtin_amdgcn_readfirstlane((int)sm.begin_n), rest = sm.begin_rest, step = first;
    rest = ((int64_t)__builtin_amdgcn_readfirstlane((int)(rest >> 32)) << 32) | (uint32_t)__builtin_amdgcn_readfirstlane((int)rest);
    bool opening = true;
    while (step < end) {
        // A segment: tiles t0 .. t1 - 1 of row tile rt of sequence n.
        const int len = (int)length(n), tiles = (len + kKeys - 1) / kKeys;
        if (tiles * a.row_tiles <= rest) {
            ++n;
            rest = 0;
            continue;
        }
        const int rt = (uint64_t)rest >> 32 ? (int)(rest / tiles) : (int)((uint32_t)rest / (uint32_t)tiles);  // below 2^24 / 32
        const int t0 = (int)(rest - (int64_t)rt * tiles), t1 = (int)min((int64_t)tiles, t0 + (end - step));
        const bool alone = t0 == 0 && t1 == tiles;

        // Keys that a row sees; rows behind the last stand for it and are not stored.
        const auto seen_by = [&](int row) {
            const uint32_t i = min((uint32_t)(rt * R * 32 + row), rows - 1);
            return min(max(len - (int)a.T + 1 + (int)(i / H), 0), len);
        };
        const int all_see = seen_by(0);
        f16v o[R][2];
        // Maxima in use: of the row among the scores, and of those among the outputs (lane % 32 of
        // each 32-row tile).  l: the sum over this lane's keys.
        float ms, mo[R], l;

        // Where this thread's row of tile t lies; rows behind the length take the last one's place.
        int32_t page;
        const auto look_up = [&](int t) {
            const int pos = min(t * kKeys + (tid >> 3), len - 1);
            page = a.table[n * a.max_pages + (pos >> a.page_shift)];
        };
        const auto copy = [&](int t) {
            const int pos = min(t * kKeys + (tid >> 3), len - 1);
            const int64_t slot = (clamp64(page, 0, a.pages - 1) << a.page_shift) + (pos & ((1 << a.page_shift) - 1));
            copy_row(a.cache + slot * kRow + (((tid & 7) ^ swap(tid >> 3)) << 3),
                     lds + (uint32_t)(t & 1) * (uint32_t)sizeof(sm.row[0]) + wave * 1024);
        };

        look_up(t0);
        copies_done();  // the last segment's reads, too
        copy(t0);
        const int seen = seen_by(my_row);
        s8 q[kRow / 32];
        {
            const uint32_t i = min((uint32_t)(rt * R * 32 + my_row), rows - 1), tok = i / H, head = i - tok * H;
            const uint16_t *ql = a.ql + n * a.qln + (int64_t)tok * a.qlt + (int64_t)head * a.qlh + 8 * g16;
            const uint16_t *qp = a.qp + n * a.qpn + (int64_t)tok * a.qpt + (int64_t)head * a.qph + 8 * g16;
#pragma unroll
            for (int ks = 0; ks < kRow / 32; ++ks)
                q[ks] = ks < kLat / 32 ? *reinterpret_cast<const s8 *>(ql + 32 * ks) : *reinterpret_cast<const s8 *>(qp + 32 * ks - kLat);
        }

        // apart: hidden keys' NaNs and infinities are kept from the rows that do not see them
        // (as in the expanded form: the segment runs again with them added apart).
        for (int apart = 0; apart < 2; ++apart) {
#pragma unroll
            for (int r = 0; r < R; ++r) {
                mo[r] = -INFINITY;
                o[r][0] = o[r][1] = zero16();
            }
            ms = -INFINITY;
            l = 0.0f;
            if (apart) {
                look_up(t0);
                copies_done();
                copy(t0);
            }
            look_up(min(t0 + 1, tiles - 1));
#pragma unroll 1
            for (int t = t0; t < t1; ++t) {
                copies_done();
                if (t + 1 < t1) {
                    copy(t + 1);
                    look_up(min(t + 2, tiles - 1));
                }
                const uint32_t buf = (uint32_t)(t & 1) * (uint32_t)sizeof(sm.row[0]);
                // scores
                f4 s[R];
                {
                    // One tile of keys has two sums, two have one each: every second product waits for none.
                    constexpr int kAhead = 6;
                    const uint32_t k = at_k + buf;
                    const auto operand = [&](int i) { return read8((k ^ (((i / R) & 1) << 6)) + (i / R >> 1) * kSub + i % R * 16 * 128); };
                    s8 ring[kAhead];
                    f4 sums[2];
#pragma unroll
                    for (int i = 0; i < kAhead; ++i) ring[i] = operand(i);
                    sums[0] = sums[1] = f4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                    for (int i = 0; i < R * kRow / 32; ++i) {
                        sums[i & 1] = mfma16x16x32_bf16(ring[i % kAhead], q[i / R], sums[i & 1]);
                        if (i + kAhead < R * kRow / 32) ring[i % kAhead] = operand(i + kAhead);
                        __builtin_amdgcn_sched_barrier(0);
                    }
                    if (R == 1) s[0] = sums[0] + sums[1];
                    else {
                        s[0] = sums[0];
                        s[R - 1] = sums[1];
                    }
                }
                if ((t + 1) * kKeys > all_see) {
#pragma unroll
                    for (int r = 0; r < R; ++r)
#pragma unroll
                        for (int i = 0; i < 4; ++i) s[r][i] = t * kKeys + k0 + 16 * r + 4 * g16 + i < seen ? s[r][i] : -INFINITY;
                }
                // Probabilities by the maximum in use, which may stay 2^40 behind the true one (bf16
                // has fp32's exponents, so that nothing is lost): only a larger step, as in a segment's first
                // tile, makes the waves agree on new maxima first.
                constexpr float kSlack = 40.0f;
                float top = -INFINITY;
#pragma unroll
                for (int r = 0; r < R; ++r) top = fmaxf(top, fmaxf(fmaxf(s[r][0], s[r][1]), fmaxf(s[r][2], s[r][3])));
                top = quad_max(top) * c;
                if (g16 == 0) sm.top[kg][my_row] = top;
                if (__builtin_amdgcn_ballot_w64(top > ms + kSlack) != 0 && lane == 0) sm.rise[t & 1] = 1;
                float part;
                const auto probabilities = [&]() {
                    const float x = ms == -INFINITY ? 0.0f : ms;
                    part = 0.0f;
#pragma unroll
                    for (int r = 0; r < R; ++r) {
                        float e[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i) e[i] = __builtin_amdgcn_exp2f(fmaf(s[r][i], c, -x));
                        part += (e[0] + e[1]) + (e[2] + e[3]);
                        *reinterpret_cast<__attribute__((address_space(3))) u2v *>(put_p ^ (r << 5)) = u2v{pack2(e[0], e[1]), pack2(e[2], e[3])};
                    }
                };
                probabilities();
                lds_barrier();
                if (sm.rise[t & 1]) {
                    const auto risen = [&](float m, int row) {
#pragma unroll
                        for (int k = 0; k < kKeyGroups; ++k) m = fmaxf(m, sm.top[k][row]);
                        return m;
                    };
                    const auto factor = [](float from, float to) { return to == -INFINITY ? 1.0f : __builtin_amdgcn_exp2f(from - to); };
                    const float xs = risen(ms, my_row);
                    l *= factor(ms, xs);
                    ms = xs;
#pragma unroll
                    for (int r = 0; r < R; ++r) {
                        const float xo = risen(mo[r], 32 * r + (lane & 31)), f = factor(mo[r], xo);
                        mo[r] = xo;
#pragma unroll
                        for (int d = 0; d < 2; ++d)
#pragma unroll
                            for (int i = 0; i < 16; ++i) o[r][d][i] *= f;
                    }
                    probabilities();
                    lds_barrier();
                    if (tid == 0) sm.rise[t & 1] = 0;  // set again two tiles on
                }
                l += part;
                if (apart && (t + 1) * kKeys > all_see) {
                    int sees[R];
#pragma unroll
                    for (int r = 0; r < R; ++r) sees[r] = seen_by(32 * r + (lane & 31));
#pragma unroll 1
                    for (int i = 0; i < kKeys; ++i) {
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            const uint16_t *x = sm.row[t & 1][wave] + i * 64 + ((e ^ swap(i)) << 3) + 4 * g;
                            const u2v v = *reinterpret_cast<const u2v *>(x);
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                const uint32_t b = (v[j / 2] >> (16 * (j & 1))) & 0xffffu;
                                const float f = (b & 0x7f80u) == 0x7f80u ? bf16_bits_to_f32(b) : 0.0f;
#pragma unroll
                                for (int r = 0; r < R; ++r) o[r][e / 4][4 * (e % 4) + j] += t * kKeys + i < sees[r] ? f : 0.0f;
                            }
                        }
                    }
                    __syncthreads();
                    uint32_t *x = reinterpret_cast<uint32_t *>(sm.row[t & 1]);
                    for (int i = tid; i < kLat / 64 * kSub / 4; i += 512) {
                        uint32_t v = x[i];
                        if ((v & 0x7f80u) == 0x7f80u) v &= 0xffff0000u;
                        if ((v >> 16 & 0x7f80u) == 0x7f80u) v &= 0x0000ffffu;
                        x[i] = v;
                    }
                    __syncthreads();
                }
                // outputs
                {
                    constexpr int kAhead = 3;
                    const uint32_t v = at_v + buf;
                    const auto operand = [&](int i) {
                        const uint32_t x = (v ^ ((i & 1) << 6)) + (i >> 1) * 16 * 128;
                        const s4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16(reinterpret_cast<lds_s4>(x));
                        const s4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16(reinterpret_cast<lds_s4>((x ^ 16) + 4 * 128));
                        return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
                    };
                    s8 p[R][2], ring[kAhead];
#pragma unroll
                    for (int r = 0; r < R; ++r) p[r][0] = read8(at_p + r * 32 * 128);
#pragma unroll
                    for (int i = 0; i < kAhead; ++i) ring[i] = operand(i);
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        if ((i & 1) == 0 && i < 6)
#pragma unroll
                            for (int r = 0; r < R; ++r) p[r][(i >> 1) + 1 & 1] = read8((at_p ^ (((i >> 1) + 1) << 5)) + r * 32 * 128);
#pragma unroll
                        for (int r = 0; r < R; ++r) o[r][i & 1] = mfma32(ring[i % kAhead], p[r][i >> 1 & 1], o[r][i & 1]);
                        if (i + kAhead < 8) ring[i % kAhead] = operand(i + kAhead);
                        __builtin_amdgcn_sched_barrier(0);
                    }
                }
            }
            if (apart || t1 * kKeys <= all_see || a.T == 1) break;
            float odd = 0.0f;
#pragma unroll
            for (int r = 0; r < R; ++r)
#pragma unroll
                for (int d = 0; d < 2; ++d)
#pragma unroll
                    for (int i = 0; i < 16; ++i) odd = fmaf(o[r][d][i], 0.0f, odd);
            __syncthreads();
            if (tid == 0) sm.odd = 0;
            __syncthreads();
            if (!(odd == 0.0f)) sm.odd = 1;
            __syncthreads();
            if (!sm.odd) break;
        }

        // The sums over all keys.
        __syncthreads();
        const float mine = quad_sum(l);
        if (g16 == 0) sm.sum[kg][my_row] = mine;
        __syncthreads();
        float z[R];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int row = 32 * r + (lane & 31);
            z[r] = sm.sum[0][row] + sm.sum[1][row];
            if (kKeyGroups == 4) z[r] += sm.sum[2][row] + sm.sum[3][row];
        }
        if (alone) {
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const uint32_t i = (uint32_t)((rt * R + r) * 32 + (lane & 31));
                const float f = z[r] == 0.0f ? 0.0f : 1.0f / z[r];
                if (i >= rows) continue;
                uint16_t *out = a.out + (n * rows + i) * kLat + wave * 64 + 4 * g;
#pragma unroll
                for (int d = 0; d < 2; ++d)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const u2v x = {pack2(o[r][d][4 * e] * f, o[r][d][4 * e + 1] * f), pack2(o[r][d][4 * e + 2] * f, o[r][d][4 * e + 3] * f)};
                        *reinterpret_cast<u2v *>(out + 32 * d + 8 * e) = x;
                    }
                if (a.lse && g == 0 && wave == 0)
                    a.lse[n * rows + i] = z[r] == 0.0f ? -INFINITY : (mo[r] + __builtin_amdgcn_logf(z[r])) * kLn2;
            }
            if (tid == 0) a.seg[2 * (n * a.row_tiles + rt)] = -1;
        } else {
            const int64_t slot = 2 * w + (opening ? 0 : 1);
#pragma unroll
            for (int r = 0; r < R; ++r) {
                f4 *p = reinterpret_cast<f4 *>(a.part) + ((slot * kWaves + wave) * R + r) * (8 * 64) + lane;
#pragma unroll
                for (int d = 0; d < 2; ++d)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        p[(4 * d + e) * 64] = f4{o[r][d][4 * e], o[r][d][4 * e + 1], o[r][d][4 * e + 2], o[r][d][4 * e + 3]};
                if (g == 0 && wave == 0) {
                    float *st = a.part_stat + (slot * R + r) * 64 + lane;
                    st[0] = mo[r];
                    st[32] = z[r];
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

// The parts of a row tile added up: a workgroup has 8 of a wave's values of 32 rows, 4
// a lane; each of its waves takes every kJoinWaves-th part, with a running maximum, and
// the waves' sums are added in their order.
template <int R, int kJoinWaves>
__global__ __launch_bounds__(64 * kJoinWaves) void latent_join_kernel(LatentDecodeArgs a, int64_t base) {
    __shared__ f4 acc[kJoinWaves][64];
    __shared__ float tops[kJoinWaves][32], sums[kJoinWaves][32];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, n32 = lane & 31;
    const int64_t unit = base + blockIdx.x, tile = unit / (64 * R);
    const int piece = (int)(unit & 63), r = (int)(unit / 64 % R);
    const int pw = piece >> 3, pv = piece & 7;  // wave and group of values
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
        for (int w = w0 + wave; w <= w1; w += kJoinWaves) {
            const int64_t s = (int64_t)(w == w0 ? head : 2 * w) * R + r;
            const float *st = a.part_stat + s * 64 + n32;
            const f4 x = reinterpret_cast<const f4 *>(a.part)[((s / R * kWaves + pw) * R + r) * (8 * 64) + pv * 64 + lane];
            const float top = fmaxf(m, st[0]), f = factor(m, top), e = factor(st[0], top);
            o = o * f + x * e;
            l = l * f + st[32] * e;
            m = top;
        }
    }
    acc[wave][lane] = o;
    if (lane < 32) {
        tops[wave][lane] = m;
        sums[wave][lane] = l;
    }
    __syncthreads();
    if (wave > 0 || i >= rows) return;
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
    const float f = l == 0.0f ? 0.0f : 1.0f / l;
    uint16_t *out = a.out + (n * rows + i) * kLat + pw * 64 + 32 * (pv >> 2) + 8 * (pv & 3) + 4 * (lane >> 5);
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
    // A row tile has about groups / (N row_tiles) parts: with many, eight waves take them (128 parts of 64
    // rows: 8 us, with two waves 28), with few, two (64 row tiles of 5 parts: 8 us, with eight 12).
    const bool many = a.N * a.row_tiles * 16 <= a.groups;
    return launch_groups(a.N * a.row_tiles * a.rows32 * 64, 0, [&](int64_t base, dim3 grid) {
        if (a.rows32 == 1 && many) hipLaunchKernelGGL((latent_join_kernel<1, 8>), grid, dim3(512), 0, s, a, base);
        else if (a.rows32 == 1) hipLaunchKernelGGL((latent_join_kernel<1, 2>), grid, dim3(128), 0, s, a, base);
        else if (many) hipLaunchKernelGGL((latent_join_kernel<2, 8>), grid, dim3(512), 0, s, a, base);
        else hipLaunchKernelGGL((latent_join_kernel<2, 2>), grid, dim3(128), 0, s, a, base);
    });
}
