// kda_latent_api.hip -- the C ABI of latent attention and its cache
// (include/kda_latent.h): validation, workspaces, launches.
#include <math.h>
#include <algorithm>
#include "kda_latent.h"
#include "kda_checks.h"
#include "kda_latent_args.h"

using namespace kda;

namespace {

constexpr int64_t kMaxAttention = (int64_t(1) << 31) - 512;  // tokens; positions are counted in 32 bits

bool scale_ok(float s) { return isfinite(s) && s > 0.0f; }

// Strides of an activation that is read 16 bytes at a time.
kda_status_t check_strides(int64_t b, int64_t t) {
    if (!stride_ok(b) || !stride_ok(t) || t >= kMaxTokenStride) return KDA_ERR_SHAPE;
    return b % 8 != 0 || t % 8 != 0 ? KDA_ERR_ALIGN : KDA_OK;
}

// ---- the expanded form ----

kda_status_t check_latent(const kda_latent_desc_t *d, bool packed) {
    if (d->B < 1 || d->T < 0 || d->Tk < 0 || d->H < 1 || d->num_seqs < 1) return KDA_ERR_SHAPE;
    if (d->H > 65535 || d->B > kMaxSeqs || d->num_seqs > kMaxSeqs) return KDA_ERR_SHAPE;
    if (d->T > kMaxAttention / d->B || d->Tk > kMaxAttention / d->B) return KDA_ERR_SHAPE;
    if (packed ? d->B != 1 : d->num_seqs != d->B) return KDA_ERR_SHAPE;
    const int64_t strides[][2] = {{d->q_stride_b, d->q_stride_t}, {d->kv_stride_b, d->kv_stride_t}, {d->pe_stride_b, d->pe_stride_t}};
    for (const auto &s : strides) {
        const kda_status_t st = check_strides(s[0], s[1]);
        if (st != KDA_OK) return st;
    }
    if (!scale_ok(d->scale) || (d->causal != 0 && d->causal != 1) || d->launch_piece < 0) return KDA_ERR_PARAM;
    return KDA_OK;
}

kda_status_t latent_args(const void *q, const void *kv, const void *pe, const int64_t *cu, const int64_t *cuk,
                         const kda_latent_desc_t *d, LatentArgs &a) {
    if (!d || (cuk && !cu)) return KDA_ERR_NULL;
    const kda_status_t st = check_latent(d, cu != nullptr);
    if (st != KDA_OK) return st;
    if (cu && !cuk && d->T != d->Tk) return KDA_ERR_SHAPE;
    if ((d->T > 0 && !q) || (d->Tk > 0 && (!kv || !pe))) return KDA_ERR_NULL;
    if (!aligned(q, 16) || !aligned(kv, 16) || !aligned(pe, 16) || !aligned(cu, 8) || !aligned(cuk, 8)) return KDA_ERR_ALIGN;
    a = LatentArgs{};
    a.q = static_cast<const uint16_t *>(q);
    a.kv = static_cast<const uint16_t *>(kv);
    a.pe = static_cast<const uint16_t *>(pe);
    a.qb = d->q_stride_b; a.qt = d->q_stride_t;
    a.kvb = d->kv_stride_b; a.kvt = d->kv_stride_t;
    a.peb = d->pe_stride_b; a.pet = d->pe_stride_t;
    a.cu = cu; a.cuk = cuk ? cuk : cu;
    a.B = d->B; a.T = d->T; a.Tk = d->Tk; a.H = d->H; a.seqs = d->num_seqs;
    a.scale = d->scale; a.causal = d->causal;
    a.launch_cap = d->launch_piece;
    return KDA_OK;
}

size_t latent_rows(const kda_latent_desc_t *d) { return (size_t)(d->B * d->T) * (size_t)d->H; }
size_t latent_keys(const kda_latent_desc_t *d) { return (size_t)(d->B * d->Tk); }

void latent_reads(Memory &m, const void *q, const void *kv, const void *pe, const int64_t *cu, const int64_t *cuk,
                  const kda_latent_desc_t *d) {
    m.read(q, extent(d->B, d->q_stride_b, d->T, d->q_stride_t, d->H * kQk, 2));
    m.read(kv, extent(d->B, d->kv_stride_b, d->Tk, d->kv_stride_t, d->H * kKvRow, 2));
    m.read(pe, extent(d->B, d->pe_stride_b, d->Tk, d->pe_stride_t, kPe, 2));
    m.read(cu, (size_t)(d->num_seqs + 1) * 8);
    m.read(cuk, (size_t)(d->num_seqs + 1) * 8);
}

// Blocks of `size` tokens: of a batch row, or at most of a packed batch.
int64_t blocks_of(int64_t T, int64_t size, int64_t seqs, bool packed) { return packed ? T / size + seqs : (T + size - 1) / size; }

// Packed: the table of blocks.
kda_status_t table_bytes(int64_t blocks, size_t &bytes) {
    if (blocks > kMaxSeqs) return KDA_ERR_SHAPE;
    bytes = align_up((size_t)(2 + 2 * blocks) * 4, 256);
    return KDA_OK;
}

}  // namespace

extern "C" size_t kda_latent_fwd_workspace_size(const kda_latent_desc_t *desc) {
    size_t need = 0;
    if (!desc || check_latent(desc, true) != KDA_OK) return 0;
    const int block = kda_latent_block(desc->B, desc->T, desc->H);
    return table_bytes(blocks_of(desc->T, block, desc->num_seqs, true), need) == KDA_OK ? need : 0;
}

extern "C" kda_status_t kda_latent_fwd(const void *q, const void *kv, const void *k_pe, const int64_t *cu_seqlens,
                                       const int64_t *cu_seqlens_k, void *out, float *lse, const kda_latent_desc_t *desc,
                                       hipStream_t stream) {
    LatentArgs a;
    kda_status_t st = latent_args(q, kv, k_pe, cu_seqlens, cu_seqlens_k, desc, a);
    if (st != KDA_OK) return st;
    if (desc->T > 0 && !out) return KDA_ERR_NULL;
    if (!aligned(out, 16) || !aligned(lse, 4)) return KDA_ERR_ALIGN;
    const bool packed = cu_seqlens != nullptr;
    const int block = kda_latent_block(desc->B, desc->T, desc->H);
    a.blocks = blocks_of(desc->T, block, desc->num_seqs, packed);
    size_t need = 0;
    if (packed) st = table_bytes(a.blocks, need);
    if (st != KDA_OK) return st;
    Memory m;
    latent_reads(m, q, kv, k_pe, cu_seqlens, cu_seqlens_k, desc);
    m.write(out, latent_rows(desc) * kVal * 2);
    m.write(lse, latent_rows(desc) * 4);
    m.write(desc->workspace, need);
    if (m.clash()) return KDA_ERR_OVERLAP;
    st = validate_cu(cu_seqlens, desc->num_seqs, desc->T, stream);
    if (st == KDA_OK) st = validate_cu(cu_seqlens_k, desc->num_seqs, desc->Tk, stream);
    if (st != KDA_OK) return st;
    if (desc->T == 0) return KDA_OK;
    Workspace ws(desc->workspace, desc->workspace_bytes, need, stream);
    if (ws.status() != KDA_OK) return ws.status();
    a.out = static_cast<uint16_t *>(out);
    a.lse = lse;
    hipError_t e = hipSuccess;
    if (packed) {
        int32_t *table = reinterpret_cast<int32_t *>(ws.at(0));
        e = kda_launch_latent_table(a, block, 0, table, stream);
        a.table = table;
    }
    if (e == hipSuccess) e = kda_launch_latent_fwd(a, block, stream);
    return of_hip(e);
}

namespace {
struct LatentBwdPlan {
    int64_t q_blocks, k_blocks;
    size_t off_qt, off_kt, off_stat, off_part, total;
};
kda_status_t plan_latent_bwd(const kda_latent_desc_t *d, bool packed, LatentBwdPlan &p) {
    p = LatentBwdPlan{};
    p.q_blocks = blocks_of(d->T, kLatentBwdBlock, d->num_seqs, packed);
    p.k_blocks = blocks_of(d->Tk, kLatentBwdBlock, d->num_seqs, packed);
    size_t qt = 0, kt = 0;
    if (packed) {
        kda_status_t st = table_bytes(p.q_blocks, qt);
        if (st == KDA_OK) st = table_bytes(p.k_blocks, kt);
        if (st != KDA_OK) return st;
    }
    p.off_qt = 0;
    p.off_kt = qt;
    p.off_stat = p.off_kt + kt;
    p.off_part = p.off_stat + align_up(latent_rows(d) * 8, 256);
    p.total = p.off_part + align_up(latent_keys(d) * (size_t)d->H * kPe * 4, 256);
    return KDA_OK;
}
}  // namespace

extern "C" size_t kda_latent_bwd_workspace_size(const kda_latent_desc_t *desc) {
    size_t best = 0;
    if (!desc) return 0;
    for (bool packed : {false, true}) {
        LatentBwdPlan p;
        if (check_latent(desc, packed) != KDA_OK || plan_latent_bwd(desc, packed, p) != KDA_OK) continue;
        best = p.total > best ? p.total : best;
    }
    return best;
}

extern "C" kda_status_t kda_latent_bwd(const void *q, const void *kv, const void *k_pe, const int64_t *cu_seqlens,
                                       const int64_t *cu_seqlens_k, const void *out, const float *lse, const void *d_out,
                                       void *dq, void *dkv, void *dk_pe, const kda_latent_desc_t *desc, hipStream_t stream) {
    LatentArgs a;
    kda_status_t st = latent_args(q, kv, k_pe, cu_seqlens, cu_seqlens_k, desc, a);
    if (st != KDA_OK) return st;
    if ((desc->T > 0 && (!out || !lse || !d_out || !dq)) || (desc->Tk > 0 && (!dkv || !dk_pe))) return KDA_ERR_NULL;
    st = check_strides(desc->out_stride_b, desc->out_stride_t);
    if (st == KDA_OK) st = check_strides(desc->d_out_stride_b, desc->d_out_stride_t);
    if (st != KDA_OK) return st;
    if (!aligned(out, 16) || !aligned(d_out, 16) || !aligned(dq, 16) || !aligned(dkv, 16) || !aligned(dk_pe, 16) || !aligned(lse, 4))
        return KDA_ERR_ALIGN;
    const bool packed = cu_seqlens != nullptr;
    LatentBwdPlan p;
    st = plan_latent_bwd(desc, packed, p);
    if (st != KDA_OK) return st;
    Memory m;
    latent_reads(m, q, kv, k_pe, cu_seqlens, cu_seqlens_k, desc);
    m.read(out, extent(desc->B, desc->out_stride_b, desc->T, desc->out_stride_t, desc->H * kVal, 2));
    m.read(d_out, extent(desc->B, desc->d_out_stride_b, desc->T, desc->d_out_stride_t, desc->H * kVal, 2));
    m.read(lse, latent_rows(desc) * 4);
    m.write(dq, latent_rows(desc) * kQk * 2);
    m.write(dkv, latent_keys(desc) * (size_t)desc->H * kKvRow * 2);
    m.write(dk_pe, latent_keys(desc) * kPe * 2);
    m.write(desc->workspace, p.total);
    if (m.clash()) return KDA_ERR_OVERLAP;
    st = validate_cu(cu_seqlens, desc->num_seqs, desc->T, stream);
    if (st == KDA_OK) st = validate_cu(cu_seqlens_k, desc->num_seqs, desc->Tk, stream);
    if (st != KDA_OK) return st;
    if (desc->T == 0 && desc->Tk == 0) return KDA_OK;
    Workspace ws(desc->workspace, desc->workspace_bytes, p.total, stream);
    if (ws.status() != KDA_OK) return ws.status();
    a.o = static_cast<const uint16_t *>(out); a.ob = desc->out_stride_b; a.ot = desc->out_stride_t;
    a.dy = static_cast<const uint16_t *>(d_out); a.yb = desc->d_out_stride_b; a.yt = desc->d_out_stride_t;
    a.lse_in = lse;
    a.stat = reinterpret_cast<float *>(ws.at(p.off_stat));
    a.dpe_part = reinterpret_cast<float *>(ws.at(p.off_part));
    a.dq = static_cast<uint16_t *>(dq);
    a.dkv = static_cast<uint16_t *>(dkv);
    a.dpe = static_cast<uint16_t *>(dk_pe);

    LatentArgs k = a;
    a.blocks = p.q_blocks;
    k.blocks = p.k_blocks;
    hipError_t e = hipSuccess;
    if (packed) {
        int32_t *qt = reinterpret_cast<int32_t *>(ws.at(p.off_qt)), *kt = reinterpret_cast<int32_t *>(ws.at(p.off_kt));
        e = kda_launch_latent_table(a, kLatentBwdBlock, 0, qt, stream);
        if (e == hipSuccess) e = kda_launch_latent_table(k, kLatentBwdBlock, 1, kt, stream);
        a.table = qt;
        k.table = kt;
    }
    if (e == hipSuccess) e = kda_launch_latent_dq(a, stream);
    if (e == hipSuccess) e = kda_launch_latent_dkv(k, stream);
    if (e == hipSuccess) e = kda_launch_latent_dpe(k, stream);
    return of_hip(e);
}
