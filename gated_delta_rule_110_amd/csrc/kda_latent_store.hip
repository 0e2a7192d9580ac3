// kda_latent_store.hip -- what the cache of latent attention needs: tokens' vectors
// into it (kda_latent_store), and the pages and slots of a serving step
// (kda_page_assign in include/kda_latent.h).
#include <algorithm>
#include "kda_latent_common.h"

namespace kda {

namespace {

// A wave takes a token: 8 values of the latent a lane, the 64 shared ones in lanes 0 to
// 7.  Sums of squares in fp32, n rounded once.  Memory-bound; a wave goes on to further
// tokens so that the weights are read once.
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

// Exclusive sum over the 1024 threads, and the total.
__device__ int64_t scan1024(int64_t v, int64_t *lds, int64_t &total) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    int64_t s = v;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int64_t o = __shfl_up(s, d);
        if (lane >= d) s += o;
    }
    __syncthreads();
    if (lane == 63) lds[wave] = s;
    __syncthreads();
    total = 0;
    int64_t before = 0;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        if (i < wave) before += lds[i];
        total += lds[i];
    }
    return before + s - v;
}

// The slot of packed row i, and where it is the first of a new page, its table entry.
__device__ __forceinline__ void page_slot(const PageArgs &a, int64_t i, int64_t lo, int64_t hi) {
    int64_t slot = -1;
    if (i < a.cu[a.N]) {
        while (hi - lo > 1) {  // cu[lo] <= i < cu[hi]
            const int64_t mid = (lo + hi) >> 1;
            if (a.cu[mid] <= i) lo = mid;
            else hi = mid;
        }
        const int64_t got = a.granted[lo];
        if (got > 0) {
            const int64_t before = a.len_out[lo] - got, pos = before + i - a.cu[lo];
            const int64_t size = int64_t(1) << a.shift, held = (before + size - 1) >> a.shift, p = pos >> a.shift;
            int64_t page;
            if (p < held) {
                page = a.table[lo * a.max_pages + p];
            } else {
                page = a.free_pages[*a.have - 1 - a.base[lo] - (p - held)];
                if ((pos & (size - 1)) == 0) a.table[lo * a.max_pages + p] = (int32_t)page;
            }
            slot = (page << a.shift) + (pos & (size - 1));
        }
    }
    a.slots[i] = slot;
}

// One workgroup runs through the requests; with few tokens it finds their slots too.
constexpr int64_t kFewTokens = 4096;
__global__ __launch_bounds__(1024) void pages_kernel(PageArgs a) {
    __shared__ int64_t lds[16];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int64_t size = int64_t(1) << a.shift, most = a.max_pages << a.shift;
    const int64_t count = clamp64(*a.count, 0, a.stack);
    const auto pages = [&](int64_t v) { return (v + size - 1) >> a.shift; };
    const auto length = [&](int64_t n) { return clamp64(a.len[n], 0, most); };
    const auto gives = [&](int64_t n) { return a.ended && a.ended[n] ? pages(length(n)) : 0; };
    const int64_t share = (a.N + 1023) / 1024, n0 = min(a.N, tid * share), n1 = min(a.N, n0 + share);

    // offsets of the new tokens, and of the pages that go back
    int64_t add = 0, give = 0, total, back;
    for (int64_t n = n0; n < n1; ++n) {
        add += least0(a.add[n]);
        give += gives(n);
    }
    add = scan1024(add, lds, total);
    int64_t row = add;
    give = scan1024(give, lds, back);
    for (int64_t n = n0; n < n1; ++n) {
        a.cu[n] = min(add, a.tokens);
        add += least0(a.add[n]);
        a.base[n] = give;
        give += gives(n);
    }
    if (tid == 0) a.cu[a.N] = min(total, a.tokens);
    const int64_t have = min(count + back, a.stack);
    if (back > 0) {
        __syncthreads();
        for (int64_t first = wave * 64; first < a.N; first += 1024) {
            const int64_t n = first + lane;
            uint64_t who = __builtin_amdgcn_ballot_w64(n < a.N && gives(n) > 0);
            while (who) {
                const int64_t m = first + __builtin_ctzll(who);
                who &= who - 1;
                const int64_t k = gives(m), to = count + a.base[m];
                for (int64_t i = lane; i < k && to + i < a.stack; i += 64) a.free_pages[to + i] = a.table[m * a.max_pages + i];
            }
        }
        __syncthreads();
    }

    // the pages that are needed, and who gets them
    const auto needs = [&](int64_t n, int64_t at, int64_t &before, bool &fits) {
        before = a.ended && a.ended[n] ? 0 : length(n);
        const int64_t now = least0(a.add[n]);
        fits = now <= most - before && at + now <= a.tokens;
        return fits ? pages(before + now) - pages(before) : int64_t(0);
    };
    int64_t need = 0, used = 0, all, taken, before;
    bool fits;
    int64_t at = row;
    for (int64_t n = n0; n < n1; ++n) {
        need += needs(n, at, before, fits);
        at += least0(a.add[n]);
    }
    need = scan1024(need, lds, all);
    for (int64_t n = n0; n < n1; ++n) {
        const int64_t k = needs(n, row, before, fits), now = least0(a.add[n]);
        row += now;
        const bool ok = fits && (k == 0 || need + k <= have);
        a.base[n] = need;
        need += k;
        if (ok) used += k;
        a.granted[n] = ok ? now : 0;
        a.len_out[n] = before + (ok ? now : 0);
    }
    scan1024(used, lds, taken);
    if (tid == 0) {
        *a.have = have;
        *a.count_out = have - taken;
    }
    if (a.tokens <= kFewTokens) {
        __syncthreads();
        for (int64_t i = tid; i < a.tokens; i += 1024) page_slot(a, i, 0, a.N);
    }
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
    if (i < a.tokens) page_slot(a, i, lo, hi);
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
    hipLaunchKernelGGL(pages_kernel, dim3(1), dim3(1024), 0, s, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || a.tokens <= kFewTokens) return e;
    return launch_groups((a.tokens + 255) / 256, 0, [&](int64_t base, dim3 grid) {
        hipLaunchKernelGGL(slots_kernel, grid, dim3(256), 0, s, a, base);
    });
}
