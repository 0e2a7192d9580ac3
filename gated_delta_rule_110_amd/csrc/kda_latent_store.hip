// kda_latent_store.hip -- what the cache of latent attention needs: tokens' vectors
// into it (kda_latent_store), and the pages and slots of a serving step
// (kda_page_assign in include/kda_latent.h).
#include <algorithm>
#include "kda_latent_common.h"

namespace kda {

namespace {

// A wave takes a token: 8 values of the latent a lane, the 64 shared ones in lanes 0 to
// 7.  Sums of squares in fp32, n rounded once.  Memory-bound (32768 tokens with the
// normalised latents kept: 18 us, 5.8 TB/s); a wave goes on to further tokens so that the
// weights are read once.
constexpr int kStoreGroups = 2048;  // workgroups of four waves: 8 a CU
template <int NORM>  // 0: no weight, 1: bf16, 2: fp32
__global__ __launch_bounds__(256) void latent_store_kernel(LatentStoreArgs a) {
    const int lane = threadIdx.x & 63;
    float w[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) w[j] = NORM ? load_any(a.w, 8 * lane + j, NORM == 2) : 1.0f;
    for (int64_t t = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); t < a.tokens; t += (int64_t)gridDim.x * 4) {
        u4v x = *reinterpret_cast<const u4v *>(a.latent + t * a.ls + 8 * lane);
        u4v r;
        if (lane < 8) r = *reinterpret_cast<const u4v *>(a.pe + t * a.ps + 8 * lane);
        const int64_t slot = a.slots[t];
        if (NORM) {
            float v[8], s = 0.0f;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                v[j] = __uint_as_float(j & 1 ? x[j / 2] & 0xffff0000u : x[j / 2] << 16);
                s = fmaf(v[j], v[j], s);
            }
#pragma unroll
            for (int d = 1; d < 64; d <<= 1) s += __shfl_xor(s, d);
            const float f = fast_rsqrt(s * (1.0f / kLat) + a.eps);
#pragma unroll
            for (int j = 0; j < 4; ++j) x[j] = pack2(v[2 * j] * f * w[2 * j], v[2 * j + 1] * f * w[2 * j + 1]);
        }
        if (a.normed) *reinterpret_cast<u4v *>(a.normed + t * kLat + 8 * lane) = x;
        if (slot >= 0 && slot < a.num_slots) {
            uint16_t *row = a.cache + slot * kRow + 8 * lane;
            *reinterpret_cast<u4v *>(row) = x;
            if (lane < 8) *reinterpret_cast<u4v *>(row + kLat) = r;
        }
    }
}

// ---- pages ---------------------------------------------------------------------------

__device__ __forceinline__ int64_t least0(int64_t v) { return clamp64(v, 0, int64_t(1) << 40); }

// Exclusive sums over the 1024 threads of two numbers each, and the totals.
__device__ void scan1024(int64_t &u, int64_t &v, int64_t (*lds)[2], int64_t &all_u, int64_t &all_v) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    int64_t x = u, y = v;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int64_t p = __shfl_up(x, d), q = __shfl_up(y, d);
        if (lane >= d) {
            x += p;
            y += q;
        }
    }
    if (lane == 63) {
        lds[wave][0] = x;
        lds[wave][1] = y;
    }
    __syncthreads();
    all_u = all_v = 0;
    u = x - u;
    v = y - v;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        if (i < wave) {
            u += lds[i][0];
            v += lds[i][1];
        }
        all_u += lds[i][0];
        all_v += lds[i][1];
    }
}

// What a request's rows are found by: the running sums of new tokens, the tokens
// granted, those held before and the pages that the requests ahead take.
struct Found {
    const int64_t *cu, *granted, *len_out, *base;
};

// The slot of packed row i, and where it is the first of a new page, its table entry.
// have: pages on the stack; cu[lo] <= i < cu[hi] where i is a row of some request.
__device__ __forceinline__ void page_slot(const PageArgs &a, const Found &f, int64_t rows, int64_t have, int64_t i, int64_t lo, int64_t hi) {
    int64_t slot = -1;
    if (i < rows) {
        while (hi - lo > 1) {
            const int64_t mid = (lo + hi) >> 1;
            if (f.cu[mid] <= i) lo = mid;
            else hi = mid;
        }
        const int64_t got = f.granted[lo];
        if (got > 0) {
            const int64_t before = f.len_out[lo] - got, pos = before + i - f.cu[lo];
            const int64_t size = int64_t(1) << a.shift, held = (before + size - 1) >> a.shift, p = pos >> a.shift;
            int64_t page;
            if (p < held) {
                page = a.table[lo * a.max_pages + p];
            } else {
                page = a.free_pages[have - 1 - f.base[lo] - (p - held)];
                if ((pos & (size - 1)) == 0) a.table[lo * a.max_pages + p] = (int32_t)page;
            }
            slot = (page << a.shift) + (pos & (size - 1));
        }
    }
    a.slots[i] = slot;
}

// One workgroup runs through the requests.  With few of them (kNear: one a thread) their
// numbers stay in registers and LDS, and with few tokens (kFewTokens) it puts the pages
// back and finds the slots itself; otherwise those are launches of their own behind it,
// over all CUs (1024 requests, 131072 tokens, 33000 pages back: 47 -> 23 us).
constexpr int64_t kNear = 1024, kFewTokens = 2048;
__global__ __launch_bounds__(1024) void pages_kernel(PageArgs a, int further) {
    __shared__ int64_t lds[2][16][2];
    __shared__ unsigned long long taken;
    __shared__ int64_t s_cu[kNear + 1], s_granted[kNear], s_out[kNear], s_base[kNear];
    __shared__ int32_t s_give[kNear], s_to[kNear];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int64_t size = int64_t(1) << a.shift, most = a.max_pages << a.shift;
    const int64_t count = clamp64(*a.count, 0, a.stack);
    const auto pages = [&](int64_t v) { return (v + size - 1) >> a.shift; };
    struct Request {
        int64_t length, add, give;   // tokens held, to come; pages to give back
    };
    const auto request = [&](int64_t n) {
        Request r{clamp64(a.len[n], 0, most), least0(a.add[n]), 0};
        if (a.ended && a.ended[n]) {
            r.give = pages(r.length);
            r.length = 0;
        }
        return r;
    };
    // pages that a request needs whose rows begin at `row`; negative where it is refused in any case
    const auto needs = [&](const Request &r, int64_t row) {
        return r.add <= most - r.length && row + r.add <= a.tokens ? pages(r.length + r.add) - pages(r.length) : int64_t(-1);
    };
    const int64_t share = (a.N + 1023) / 1024, n0 = min(a.N, tid * share), n1 = min(a.N, n0 + share);
    const bool near = a.N <= kNear;

    // offsets of the new tokens, and of the pages that go back
    int64_t add = 0, give = 0, total, back;
    Request own{0, 0, 0};
    for (int64_t n = n0; n < n1; ++n) {
        own = request(n);
        add += own.add;
        give += own.give;
    }
    if (tid == 0) taken = 0;
    scan1024(add, give, lds[0], total, back);
    const int64_t have = min(count + back, a.stack), row0 = add, rows = min(total, a.tokens);
    if (tid == 0) {
        a.cu[a.N] = rows;
        *a.have = have;
        a.have[1] = count;
        if (further) a.back[a.N] = back;
        if (near) s_cu[a.N] = rows;
    }
    // the pages that are needed, and who gets them
    int64_t need = 0, none = 0, all, nothing;
    for (int64_t n = n0; n < n1; ++n) {
        if (!near) own = request(n);
        const int64_t k = needs(own, add);
        need += k > 0 ? k : 0;
        add += own.add;
    }
    scan1024(need, none, lds[1], all, nothing);
    add = row0;
    for (int64_t n = n0; n < n1; ++n) {
        if (!near) own = request(n);
        const int64_t k = needs(own, add), upto = need + (k > 0 ? k : 0);
        const bool ok = k == 0 || (k > 0 && upto <= have);
        const int64_t got = ok ? own.add : 0, first = min(add, a.tokens);
        a.cu[n] = first;
        a.granted[n] = got;
        a.len_out[n] = own.length + got;
        if (further) {
            a.base[n] = need;
            a.back[n] = give;
        }
        if (near) {
            s_cu[n] = first;
            s_granted[n] = got;
            s_out[n] = own.length + got;
            s_base[n] = need;
            s_give[n] = (int32_t)own.give;
            s_to[n] = (int32_t)min(count + give, a.stack);
        }
        if (ok && k > 0) atomicMax(&taken, (unsigned long long)upto);  // the granted ones are the first that need any
        need = upto;
        add += own.add;
        give += own.give;
    }
    __syncthreads();
    if (tid == 0) *a.count_out = have - (int64_t)taken;
    if (further) return;
    if (back > 0) {
        // a wave looks at 64 requests, and puts the pages of those that end on the stack
        for (int first = wave * 64; first < a.N; first += 1024) {
            uint64_t who = __builtin_amdgcn_ballot_w64(first + lane < a.N && s_give[first + lane] > 0);
            while (who) {
                const int n = first + __builtin_ctzll(who);
                who &= who - 1;
                for (int64_t i = lane, k = s_give[n], to = s_to[n]; i < k && to + i < a.stack; i += 64)
                    a.free_pages[to + i] = a.table[n * a.max_pages + i];
            }
        }
        __syncthreads();
    }
    const Found f = {s_cu, s_granted, s_out, s_base};
    for (int64_t i = tid; i < a.tokens; i += 1024) page_slot(a, f, rows, have, i, 0, a.N);
}

// A wave's request gives its pages back.
__global__ __launch_bounds__(256) void back_kernel(PageArgs a, int64_t base) {
    const int64_t n = (base + blockIdx.x) * 4 + (threadIdx.x >> 6);
    if (n >= a.N || !a.ended[n]) return;
    const int64_t k = a.back[n + 1] - a.back[n], to = a.have[1] + a.back[n];
    for (int64_t i = threadIdx.x & 63; i < k && to + i < a.stack; i += 64) a.free_pages[to + i] = a.table[n * a.max_pages + i];
}

__global__ __launch_bounds__(256) void slots_kernel(PageArgs a, int64_t base) {
    // The requests of the workgroup's first and last row: 64 places at a time.
    const int lane = threadIdx.x & 63;
    const int64_t i = (base + blockIdx.x) * 256 + threadIdx.x;
    const auto request = [&](int64_t row) {
        int64_t lo = 0, hi = a.N;
        while (hi - lo > 1) {
            const int64_t step = (hi - lo + 63) / 64, at = min(hi, lo + lane * step);
            const int k = __builtin_popcountll(__builtin_amdgcn_ballot_w64(at < hi && a.cu[at] <= row));  // at least lane 0
            lo += (int64_t)(k > 0 ? k - 1 : 0) * step;
            hi = min(hi, lo + step);
        }
        return lo;
    };
    const int64_t first = (base + blockIdx.x) * 256, lo = request(first), hi = request(min(first + 255, a.tokens - 1)) + 1;
    const Found f = {a.cu, a.granted, a.len_out, a.base};
    if (i < a.tokens) page_slot(a, f, a.cu[a.N], *a.have, i, lo, hi);
}

}  // namespace

}  // namespace kda

using namespace kda;

hipError_t kda_launch_latent_store(const LatentStoreArgs &a, hipStream_t s) {
    const dim3 grid((unsigned)std::min<int64_t>((a.tokens + 3) / 4, kStoreGroups)), block(256);
    if (!a.w) hipLaunchKernelGGL(latent_store_kernel<0>, grid, block, 0, s, a);
    else if (!a.w_f32) hipLaunchKernelGGL(latent_store_kernel<1>, grid, block, 0, s, a);
    else hipLaunchKernelGGL(latent_store_kernel<2>, grid, block, 0, s, a);
    return hipGetLastError();
}

hipError_t kda_launch_pages(const PageArgs &a, hipStream_t s) {
    const int further = a.N > kNear || a.tokens > kFewTokens;
    hipLaunchKernelGGL(pages_kernel, dim3(1), dim3(1024), 0, s, a, further);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || !further) return e;
    if (a.ended) {
        hipLaunchKernelGGL(back_kernel, dim3((unsigned)((a.N + 3) / 4)), dim3(256), 0, s, a, 0);
        e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return launch_groups((a.tokens + 255) / 256, 0, [&](int64_t base, dim3 grid) {
        hipLaunchKernelGGL(slots_kernel, grid, dim3(256), 0, s, a, base);
    });
}
