// kda_norm.hip -- RMS normalisation with the residual's addition (gfx950):
// bf16 output, e4m3 output with scales, and the gradient.
//
//   h = x + residual,  r = 1 / sqrt(mean(h^2) + eps),  y = h r weight
//
// and backwards, with n = h r and c = mean(weight d_out n),
//
//   dh = r (weight d_out - n c) + d_residual_out,   dweight = sum_rows d_out n.
//
// The row is read once and stays in registers between the reduction and the
// output, so the kernels are bound by the memory traffic of their inputs and
// outputs.  Everything between load and store is fp32.  With rows of 4096: 8191 rows
// and an fp32 residual 83 us (4.9 TB/s of what has to be read and written; the
// runtime's copy reaches 5.1, an elementwise one of a GiB 6.2), the gradient of 8192
// rows 49 us and 5 for the weight's sum (5.0 TB/s), 64 rows to e4m3 4.3 us, all of it
// latency.
#include "kda_layer_args.h"

using namespace kda;

namespace {

constexpr int kBlock = 256;
constexpr float kE4m3Max = 448.0f;
constexpr float kTiny = 1.17549435e-38f;  // 2^-126, the smallest normal fp32

// 8 consecutive values of a bf16 or fp32 row.
template <bool kF32>
__device__ __forceinline__ void load8(const void *p, int64_t i, float *o) {
    if constexpr (kF32) {
        const float4 a = *reinterpret_cast<const float4 *>(reinterpret_cast<const float *>(p) + i);
        const float4 b = *reinterpret_cast<const float4 *>(reinterpret_cast<const float *>(p) + i + 4);
        o[0] = a.x; o[1] = a.y; o[2] = a.z; o[3] = a.w;
        o[4] = b.x; o[5] = b.y; o[6] = b.z; o[7] = b.w;
    } else {
        unpack_bf16x8(*reinterpret_cast<const uint4 *>(reinterpret_cast<const uint16_t *>(p) + i), o);
    }
}
template <bool kF32>
__device__ __forceinline__ void store8(void *p, int64_t i, const float *v) {
    if constexpr (kF32) {
        float *q = reinterpret_cast<float *>(p) + i;
        *reinterpret_cast<float4 *>(q) = make_float4(v[0], v[1], v[2], v[3]);
        *reinterpret_cast<float4 *>(q + 4) = make_float4(v[4], v[5], v[6], v[7]);
    } else {
        *reinterpret_cast<uint4 *>(reinterpret_cast<uint16_t *>(p) + i) =
            make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
    }
}

// Sum over the kT lanes (a power of two, at most a wave) that share a row.
template <int kT>
__device__ __forceinline__ float lanes_sum(float v) {
#pragma unroll
    for (int m = kT / 2; m >= 1; m >>= 1) v += __shfl_xor(v, m);
    return v;
}
template <int kT>
__device__ __forceinline__ uint32_t lanes_max(uint32_t v) {
#pragma unroll
    for (int m = kT / 2; m >= 1; m >>= 1) {
        const uint32_t o = (uint32_t)__shfl_xor((int)v, m);
        v = o > v ? o : v;
    }
    return v;
}

// Sum over the kT threads of a row; with more than one wave through LDS.  Two
// calls in a row use different halves of `buf` (`phase`), so that one barrier a
// call is enough.
template <int kT>
__device__ __forceinline__ float row_sum(float v, float *buf, int phase) {
    if constexpr (kT <= 64) return lanes_sum<kT>(v);
    v = lanes_sum<64>(v);
    float *b = buf + phase * (kT / 64);
    if ((threadIdx.x & 63) == 0) b[threadIdx.x >> 6] = v;
    __syncthreads();
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < kT / 64; ++i) s += b[i];
    return s;
}
template <int kT>
__device__ __forceinline__ uint32_t row_max(uint32_t v, float *buf, int phase) {
    if constexpr (kT <= 64) return lanes_max<kT>(v);
    v = lanes_max<64>(v);
    float *b = buf + phase * (kT / 64);
    if ((threadIdx.x & 63) == 0) b[threadIdx.x >> 6] = __uint_as_float(v);
    __syncthreads();
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < kT / 64; ++i) {
        const uint32_t o = __float_as_uint(b[i]);
        m = o > m ? o : m;
    }
    return m;
}

// The scale of a group from the bits of its largest |y|: the bits of a NaN are
// above those of every number, so that the maximum over bits carries it along.
__device__ __forceinline__ float scale_of(uint32_t amax_bits) {
    const float s = __uint_as_float(amax_bits) / kE4m3Max;
    return s < kTiny ? kTiny : s;  // false for NaN
}
// Saturates to the largest e4m3 value (the largest entry's quotient may exceed
// 448 by a rounding) and keeps NaN.
__device__ __forceinline__ float sat(float v) { return fabsf(v) > kE4m3Max ? copysignf(kE4m3Max, v) : v; }
__device__ __forceinline__ uint32_t pack_e4m3(const float *v) {
    int r = __builtin_amdgcn_cvt_pk_fp8_f32(sat(v[0]), sat(v[1]), 0, false);
    r = __builtin_amdgcn_cvt_pk_fp8_f32(sat(v[2]), sat(v[3]), r, true);
    return (uint32_t)r;
}
__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7fffffffu; }

// kT threads per row, kV groups of 8 columns each: thread t holds the columns
// 8 (i kT + t) .. + 7, so that every access is 16 or 32 bytes per lane and a
// 128-column group is 16 neighbouring lanes.  Workgroups walk over rows, with
// the weight in registers.
template <int kT, int kV, int kRes, int kQuant>
__global__ __launch_bounds__(kT > kBlock ? kT : kBlock) void kda_rmsnorm_kernel(NormArgs a) {
    constexpr int kThreads = kT > kBlock ? kT : kBlock;
    constexpr int kRows = kThreads / kT;
    __shared__ float red[4 * (kT > 64 ? kT / 64 : 1)];
    const int t = threadIdx.x % kT;
    float w[kV][8];
#pragma unroll
    for (int i = 0; i < kV; ++i) {
        const int64_t c = 8 * ((int64_t)i * kT + t);
#pragma unroll
        for (int e = 0; e < 8; ++e) w[i][e] = 0.f;
        if (c < a.D) {
            if (a.w_f32) load8<true>(a.w, c, w[i]);
            else load8<false>(a.w, c, w[i]);
        }
    }
    const float inv_d = 1.0f / (float)a.D;
    int phase = 0;
    for (int64_t row = (int64_t)blockIdx.x * kRows + threadIdx.x / kT; row < a.rows;
         row += (int64_t)gridDim.x * kRows) {
        float h[kV][8];
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < kV; ++i) {
            const int64_t c = 8 * ((int64_t)i * kT + t);
#pragma unroll
            for (int e = 0; e < 8; ++e) h[i][e] = 0.f;
            if (c < a.D) {
                load8<false>(a.x, row * a.xs + c, h[i]);
                if constexpr (kRes != 0) {
                    float r[8];
                    load8<kRes == 2>(a.res, row * a.rs + c, r);
#pragma unroll
                    for (int e = 0; e < 8; ++e) h[i][e] += r[e];
                }
            }
        }
#pragma unroll
        for (int i = 0; i < kV; ++i)
#pragma unroll
            for (int e = 0; e < 8; ++e) ss += h[i][e] * h[i][e];
        ss = row_sum<kT>(ss, red, phase);
        const float r = fast_rsqrt(ss * inv_d + a.eps);
        uint32_t amax[kV] = {};
#pragma unroll
        for (int i = 0; i < kV; ++i) {
            const int64_t c = 8 * ((int64_t)i * kT + t);
            if constexpr (kRes != 0) {
                if (a.res_out && c < a.D) store8<kRes == 2>(a.res_out, row * a.D + c, h[i]);
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                h[i][e] = h[i][e] * r * w[i][e];
                if constexpr (kQuant != 0) {
                    const uint32_t b = abs_bits(h[i][e]);
                    if (c < a.D) amax[i] = b > amax[i] ? b : amax[i];
                }
            }
            if constexpr (kQuant == 0) {
                if (c < a.D) store8<false>(a.out, row * a.D + c, h[i]);
            }
        }
        if constexpr (kQuant == 1) {
            uint32_t m = 0;
#pragma unroll
            for (int i = 0; i < kV; ++i) m = amax[i] > m ? amax[i] : m;
            m = row_max<kT>(m, red, 2 + phase);
            const float s = scale_of(m), inv = 1.0f / s;
            if (t == 0) a.scales[row] = s;
#pragma unroll
            for (int i = 0; i < kV; ++i) {
                const int64_t c = 8 * ((int64_t)i * kT + t);
#pragma unroll
                for (int e = 0; e < 8; ++e) h[i][e] *= inv;
                if (c < a.D)
                    *reinterpret_cast<uint2 *>(reinterpret_cast<uint8_t *>(a.out) + row * a.D + c) =
                        make_uint2(pack_e4m3(h[i]), pack_e4m3(h[i] + 4));
            }
        }
        if constexpr (kQuant == 2) {
#pragma unroll
            for (int i = 0; i < kV; ++i) {
                const int64_t c = 8 * ((int64_t)i * kT + t);
                const float s = scale_of(lanes_max<16>(amax[i])), inv = 1.0f / s;
                if (c < a.D) {
                    if ((t & 15) == 0) a.scales[row * a.groups + c / 128] = s;
#pragma unroll
                    for (int e = 0; e < 8; ++e) h[i][e] *= inv;
                    *reinterpret_cast<uint2 *>(reinterpret_cast<uint8_t *>(a.out) + row * a.D + c) =
                        make_uint2(pack_e4m3(h[i]), pack_e4m3(h[i] + 4));
                }
            }
        }
        phase ^= 1;
    }
}

// Any width, stride and alignment: one value at a time, one workgroup per row,
// the row read again (from L2) for every pass over it.  x and the residual may
// be overwritten in place, since each entry is written by the thread that reads
// it, after its last read.
__device__ __forceinline__ float h_at(const NormArgs &a, int64_t row, int64_t c) {
    float v = bf16_bits_to_f32(a.x[row * a.xs + c]);
    if (a.res) v += load_any(a.res, row * a.rs + c, a.res_f32);
    return v;
}
__device__ __forceinline__ void norm_store(const NormArgs &a, int64_t row, int64_t c, float h, float v) {
    if (a.res_out) store_any(a.res_out, row * a.D + c, a.res_f32, h);
    if (a.quant == 0) reinterpret_cast<uint16_t *>(a.out)[row * a.D + c] = f32_to_bf16_bits(v);
    else
        reinterpret_cast<uint8_t *>(a.out)[row * a.D + c] =
            (uint8_t)(__builtin_amdgcn_cvt_pk_fp8_f32(sat(v), 0.f, 0, false) & 0xff);
}

__global__ __launch_bounds__(kBlock) void kda_rmsnorm_scalar_kernel(NormArgs a) {
    __shared__ float red[16];
    int phase = 0;
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        float ss = 0.f;
        for (int64_t c = threadIdx.x; c < a.D; c += kBlock) {
            const float v = h_at(a, row, c);
            ss += v * v;
        }
        ss = row_sum<kBlock>(ss, red, phase);
        const float r = fast_rsqrt(ss / (float)a.D + a.eps);
        if (a.quant == 2) {
            // a wave takes 128-column groups in turn
            for (int64_t g = threadIdx.x / 64; g < a.groups; g += kBlock / 64) {
                float h[2], y[2];
                uint32_t m = 0;
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const int64_t c = 128 * g + 64 * j + (threadIdx.x & 63);
                    h[j] = c < a.D ? h_at(a, row, c) : 0.f;
                    y[j] = c < a.D ? h[j] * r * load_any(a.w, c, a.w_f32) : 0.f;
                    m = abs_bits(y[j]) > m ? abs_bits(y[j]) : m;
                }
                const float s = scale_of(lanes_max<64>(m)), inv = 1.0f / s;
                if ((threadIdx.x & 63) == 0) a.scales[row * a.groups + g] = s;
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const int64_t c = 128 * g + 64 * j + (threadIdx.x & 63);
                    if (c < a.D) norm_store(a, row, c, h[j], y[j] * inv);
                }
            }
        } else {
            float inv = 1.0f;
            if (a.quant == 1) {
                uint32_t m = 0;
                for (int64_t c = threadIdx.x; c < a.D; c += kBlock) {
                    const uint32_t b = abs_bits(h_at(a, row, c) * r * load_any(a.w, c, a.w_f32));
                    m = b > m ? b : m;
                }
                const float s = scale_of(row_max<kBlock>(m, red, 2 + phase));
                inv = 1.0f / s;
                if (threadIdx.x == 0) a.scales[row] = s;
            }
            for (int64_t c = threadIdx.x; c < a.D; c += kBlock) {
                const float h = h_at(a, row, c);
                const float y = h * r * load_any(a.w, c, a.w_f32);
                norm_store(a, row, c, h, a.quant ? y * inv : y);
            }
        }
        phase ^= 1;
    }
}

// ---- gradient ----------------------------------------------------------------

// The same split of a row as the forward's.  A workgroup's rows add to one
// partial sum of dweight, held in registers, written once at the end.
template <int kT, int kV, bool kHF32>
__global__ __launch_bounds__(kT > kBlock ? kT : kBlock) void kda_rmsnorm_bwd_kernel(NormBwdArgs a) {
    constexpr int kThreads = kT > kBlock ? kT : kBlock;
    constexpr int kRows = kThreads / kT;
    __shared__ float red[4 * (kT > 64 ? kT / 64 : 1)];
    __shared__ float sdw[kRows > 1 ? kThreads * kV * 8 : 1];
    const int t = threadIdx.x % kT;
    float w[kV][8], dw[kV][8];
#pragma unroll
    for (int i = 0; i < kV; ++i) {
        const int64_t c = 8 * ((int64_t)i * kT + t);
#pragma unroll
        for (int e = 0; e < 8; ++e) w[i][e] = dw[i][e] = 0.f;
        if (c < a.D) {
            if (a.w_f32) load8<true>(a.w, c, w[i]);
            else load8<false>(a.w, c, w[i]);
        }
    }
    const float inv_d = 1.0f / (float)a.D;
    int phase = 0;
    for (int64_t row = (int64_t)blockIdx.x * kRows + threadIdx.x / kT; row < a.rows;
         row += (int64_t)gridDim.x * kRows) {
        float h[kV][8], g[kV][8], d[kV][8];
        float ss = 0.f, dot = 0.f;
#pragma unroll
        for (int i = 0; i < kV; ++i) {
            const int64_t c = 8 * ((int64_t)i * kT + t);
#pragma unroll
            for (int e = 0; e < 8; ++e) h[i][e] = g[i][e] = d[i][e] = 0.f;
            if (c < a.D) {
                load8<kHF32>(a.h, row * a.hs + c, h[i]);
                load8<false>(a.dy, row * a.ds + c, g[i]);
                if (a.dres) load8<kHF32>(a.dres, row * a.rs + c, d[i]);
            }
        }
#pragma unroll
        for (int i = 0; i < kV; ++i)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                ss += h[i][e] * h[i][e];
                dot += w[i][e] * g[i][e] * h[i][e];
            }
        ss = row_sum<kT>(ss, red, phase);
        dot = row_sum<kT>(dot, red, 2 + phase);
        const float r = fast_rsqrt(ss * inv_d + a.eps);
        const float c1 = dot * inv_d * r * r;  // n c = h r (mean(w dy h) r)
#pragma unroll
        for (int i = 0; i < kV; ++i) {
            const int64_t c = 8 * ((int64_t)i * kT + t);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                dw[i][e] += g[i][e] * (h[i][e] * r);
                d[i][e] += r * (w[i][e] * g[i][e] - h[i][e] * c1);
            }
            if (c < a.D) {
                store8<false>(a.dx, row * a.D + c, d[i]);
                if (kHF32 && a.dresidual) store8<true>(a.dresidual, row * a.D + c, d[i]);
            }
        }
        phase ^= 1;
    }
    if constexpr (kRows == 1) {
#pragma unroll
        for (int i = 0; i < kV; ++i) {
            const int64_t c = 8 * ((int64_t)i * kT + t);
            if (c < a.D) store8<true>(a.part, (int64_t)blockIdx.x * a.D + c, dw[i]);
        }
    } else {
        constexpr int kCols = kT * kV * 8;
#pragma unroll
        for (int i = 0; i < kV; ++i)
#pragma unroll
            for (int e = 0; e < 8; ++e) sdw[(threadIdx.x / kT) * kCols + 8 * (i * kT + t) + e] = dw[i][e];
        __syncthreads();
        for (int c = threadIdx.x; c < kCols && c < a.D; c += kThreads) {
            float s = 0.f;
#pragma unroll
            for (int q = 0; q < kRows; ++q) s += sdw[q * kCols + c];
            a.part[(int64_t)blockIdx.x * a.D + c] = s;
        }
    }
}

__global__ __launch_bounds__(kBlock) void kda_rmsnorm_bwd_scalar_kernel(NormBwdArgs a) {
    __shared__ float red[16];
    int phase = 0;
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        float ss = 0.f, dot = 0.f;
        for (int64_t c = threadIdx.x; c < a.D; c += kBlock) {
            const float h = load_any(a.h, row * a.hs + c, a.h_f32);
            ss += h * h;
            dot += load_any(a.w, c, a.w_f32) * bf16_bits_to_f32(a.dy[row * a.ds + c]) * h;
        }
        ss = row_sum<kBlock>(ss, red, phase);
        dot = row_sum<kBlock>(dot, red, 2 + phase);
        const float inv_d = 1.0f / (float)a.D;
        const float r = fast_rsqrt(ss * inv_d + a.eps);
        const float c1 = dot * inv_d * r * r;
        if (threadIdx.x == 0) a.rstd[row] = r;
        for (int64_t c = threadIdx.x; c < a.D; c += kBlock) {
            const float h = load_any(a.h, row * a.hs + c, a.h_f32);
            const float g = bf16_bits_to_f32(a.dy[row * a.ds + c]);
            float d = r * (load_any(a.w, c, a.w_f32) * g - h * c1);
            if (a.dres) d += load_any(a.dres, row * a.rs + c, a.h_f32);
            a.dx[row * a.D + c] = f32_to_bf16_bits(d);
            if (a.dresidual) a.dresidual[row * a.D + c] = d;
        }
        phase ^= 1;
    }
}

// dweight of the scalar path: a thread per column, blockIdx.y over shares of the rows.
__global__ __launch_bounds__(kBlock) void kda_rmsnorm_bwd_weight_kernel(NormBwdArgs a) {
    const int64_t c = (int64_t)blockIdx.x * kBlock + threadIdx.x;
    if (c >= a.D) return;
    for (int64_t p = blockIdx.y; p < a.parts; p += gridDim.y) {
        float s = 0.f;
        for (int64_t row = p; row < a.rows; row += a.parts)
            s += bf16_bits_to_f32(a.dy[row * a.ds + c]) * (load_any(a.h, row * a.hs + c, a.h_f32) * a.rstd[row]);
        a.part[p * a.D + c] = s;
    }
}

// dweight = the sum of the partial sums, in a fixed order: 16 columns per
// workgroup, 64 threads per column.
__global__ __launch_bounds__(1024) void kda_rmsnorm_bwd_sum_kernel(NormBwdArgs a) {
    __shared__ float s[64][17];
    const int col = threadIdx.x & 15, q = threadIdx.x >> 4;
    const int64_t c = (int64_t)blockIdx.x * 16 + col;
    float v = 0.f;
    if (c < a.D)
        for (int64_t p = q; p < a.parts; p += 64) v += a.part[p * a.D + c];
    s[q][col] = v;
    __syncthreads();
    if (q < 8) {
#pragma unroll
        for (int i = 1; i < 8; ++i) v += s[q + 8 * i][col];
        s[q][col] = v;
    }
    __syncthreads();
    if (q == 0 && c < a.D) {
#pragma unroll
        for (int i = 1; i < 8; ++i) v += s[i][col];
        a.dw[c] = v;
    }
}

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

// Workgroups: enough to fill the 256 CUs to their 2048 threads.
constexpr int64_t kMaxBlocks = 2048;
// The gradient's workgroups each write a partial dweight; 512 keep that to
// 1/16th of the traffic at 8192 rows.
constexpr int64_t kMaxParts = 512;

int64_t grid_of(int64_t rows, int64_t per, int64_t cap) {
    const int64_t n = (rows + per - 1) / per;
    return n < cap ? n : cap;
}

// Calls f(kT, kV) with the smallest split that holds D columns; false if none does.
template <int kTv, int kVv> struct Split { static constexpr int kT = kTv, kV = kVv; };
template <typename F>
bool with_split(int64_t D, F f) {
    if (D <= 128) f(Split<16, 1>());
    else if (D <= 256) f(Split<16, 2>());
    else if (D <= 512) f(Split<64, 1>());
    else if (D <= 1024) f(Split<64, 2>());
    else if (D <= 2048) f(Split<256, 1>());
    else if (D <= 4096) f(Split<256, 2>());
    else if (D <= 8192) f(Split<256, 4>());
    else if (D <= 16384) f(Split<512, 4>());
    else return false;
    return true;
}

template <typename Sp, int kRes, int kQuant>
void launch_norm(const NormArgs &a, hipStream_t s) {
    constexpr int threads = Sp::kT > kBlock ? Sp::kT : kBlock;
    const int64_t grid = grid_of(a.rows, threads / Sp::kT, kMaxBlocks * kBlock / threads);
    hipLaunchKernelGGL((kda_rmsnorm_kernel<Sp::kT, Sp::kV, kRes, kQuant>), dim3((unsigned)grid), dim3(threads), 0, s, a);
}
template <typename Sp, int kRes>
void launch_norm_quant(const NormArgs &a, hipStream_t s) {
    if (a.quant == 0) launch_norm<Sp, kRes, 0>(a, s);
    else if (a.quant == 1) launch_norm<Sp, kRes, 1>(a, s);
    else launch_norm<Sp, kRes, 2>(a, s);
}

bool vector_rows(int64_t D, int64_t s0, int64_t s1, int64_t s2) {
    return D % 8 == 0 && s0 % 8 == 0 && s1 % 8 == 0 && s2 % 8 == 0;
}

bool bwd_vector(const NormBwdArgs &a) {
    return a.D <= 16384 && vector_rows(a.D, a.hs, a.ds, a.dres ? a.rs : 0) && aligned16(a.h) && aligned16(a.w) &&
           aligned16(a.dy) && aligned16(a.dres) && aligned16(a.dx) && aligned16(a.dresidual);
}

}  // namespace

// Rows of 8-column groups at 16-byte aligned addresses take the register
// kernels (up to 16384 columns), all others the scalar one (8192 rows of 4096 columns
// 42 us, of 4097 186).
hipError_t kda_launch_rmsnorm(const NormArgs &a, hipStream_t s) {
    if (a.rows <= 0) return hipSuccess;
    const bool vec = vector_rows(a.D, a.xs, a.res ? a.rs : 0, 0) && aligned16(a.x) && aligned16(a.res) &&
                     aligned16(a.w) && aligned16(a.res_out) && aligned16(a.out);
    const bool done = vec && with_split(a.D, [&](auto sp) {
        using Sp = decltype(sp);
        if (!a.res) launch_norm_quant<Sp, 0>(a, s);
        else if (a.res_f32) launch_norm_quant<Sp, 2>(a, s);
        else launch_norm_quant<Sp, 1>(a, s);
    });
    if (!done)
        hipLaunchKernelGGL(kda_rmsnorm_scalar_kernel, dim3((unsigned)grid_of(a.rows, 1, kMaxBlocks)), dim3(kBlock), 0, s, a);
    return hipGetLastError();
}

int64_t kda_rmsnorm_parts(int64_t rows, int64_t D) {
    (void)D;
    return grid_of(rows, 1, kMaxParts);
}

hipError_t kda_launch_rmsnorm_bwd(const NormBwdArgs &a, hipStream_t s) {
    NormBwdArgs b = a;
    if (a.rows > 0) {
        const bool done = bwd_vector(a) && with_split(a.D, [&](auto sp) {
            using Sp = decltype(sp);
            constexpr int threads = Sp::kT > kBlock ? Sp::kT : kBlock;
            b.parts = grid_of(a.rows, threads / Sp::kT, a.parts);
            if (a.h_f32)
                hipLaunchKernelGGL((kda_rmsnorm_bwd_kernel<Sp::kT, Sp::kV, true>), dim3((unsigned)b.parts), dim3(threads), 0, s, b);
            else
                hipLaunchKernelGGL((kda_rmsnorm_bwd_kernel<Sp::kT, Sp::kV, false>), dim3((unsigned)b.parts), dim3(threads), 0, s, b);
        });
        if (!done) {
            hipLaunchKernelGGL(kda_rmsnorm_bwd_scalar_kernel, dim3((unsigned)grid_of(a.rows, 1, kMaxBlocks)), dim3(kBlock), 0, s, b);
            hipLaunchKernelGGL(kda_rmsnorm_bwd_weight_kernel, dim3((unsigned)((a.D + kBlock - 1) / kBlock), (unsigned)b.parts),
                               dim3(kBlock), 0, s, b);
        }
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    } else {
        b.parts = 0;
    }
    hipLaunchKernelGGL(kda_rmsnorm_bwd_sum_kernel, dim3((unsigned)((a.D + 15) / 16)), dim3(1024), 0, s, b);
    return hipGetLastError();
}
