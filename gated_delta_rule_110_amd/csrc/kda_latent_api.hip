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

struct LatentFwdPlan {
    int block, part_tiles;
    int64_t blocks, parts;
    size_t off_stat, off_part, total;
};
// Few blocks with many keys leave CUs idle: their keys are split into parts, of at least
// kPartTiles tiles, so that there are some 256 workgroups, and joined by a second kernel
// (512 tokens x 8 heads over 16384 keys 280 -> 62 us, 2048 x 2 over their own 41 -> 23; 512
// workgroups take 6% more or less).  A packed batch, whose lengths the host does not know, is
// planned as if every block saw all keys; the kernels size the parts by the sequence (part_tiles_of).
kda_status_t plan_latent_fwd(const kda_latent_desc_t *d, bool packed, LatentFwdPlan &p) {
    constexpr int64_t kFewUnits = 128, kUnits = 256;
    p = LatentFwdPlan{};
    p.block = kda_latent_block(d->B, d->T, d->H, d->num_seqs);
    p.blocks = blocks_of(d->T, p.block, d->num_seqs, packed);
    p.parts = 1;
    if (packed) {
        const kda_status_t st = table_bytes(p.blocks, p.off_stat);
        if (st != KDA_OK) return st;
    }
    p.off_part = p.total = p.off_stat;
    const int64_t units = p.blocks * d->B * d->H, tiles = (d->Tk + kKeys - 1) / kKeys;
    if (units > kFewUnits || tiles <= kFewTiles) return KDA_OK;
    const int64_t even = (units * tiles + kUnits - 1) / kUnits;
    p.part_tiles = (int)(std::max<int64_t>(kPartTiles, even) + 1) / 2 * 2;
    p.parts = (tiles + p.part_tiles - 1) / p.part_tiles;
    if (p.parts < 2) return KDA_OK;  // part_tiles may be all of them
    p.off_part = p.off_stat + align_up((size_t)(units * p.parts) * p.block * 8, 256);
    p.total = p.off_part + (size_t)(units * p.parts) * p.block * kVal * 4;
    return KDA_OK;
}

}  // namespace

extern "C" size_t kda_latent_fwd_workspace_size(const kda_latent_desc_t *desc) {
    size_t best = 0;
    if (!desc) return 0;
    for (bool packed : {false, true}) {
        LatentFwdPlan p;
        if (check_latent(desc, packed) != KDA_OK || plan_latent_fwd(desc, packed, p) != KDA_OK) continue;
        best = std::max(best, p.total);
    }
    return best;
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
    LatentFwdPlan p;
    st = plan_latent_fwd(desc, packed, p);
    if (st != KDA_OK) return st;
    a.blocks = p.blocks;
    a.parts = p.parts;
    a.part_tiles = p.part_tiles;
    const bool counted = packed && kda_latent_counted(desc->num_seqs, a.blocks * desc->H);
    Memory m;
    latent_reads(m, q, kv, k_pe, cu_seqlens, cu_seqlens_k, desc);
    m.write(out, latent_rows(desc) * kVal * 2);
    m.write(lse, latent_rows(desc) * 4);
    m.write(desc->workspace, p.total);
    if (m.clash()) return KDA_ERR_OVERLAP;
    st = validate_cu(cu_seqlens, desc->num_seqs, desc->T, stream);
    if (st == KDA_OK) st = validate_cu(cu_seqlens_k, desc->num_seqs, desc->Tk, stream);
    if (st != KDA_OK) return st;
    if (desc->T == 0) return KDA_OK;
    Workspace ws(desc->workspace, desc->workspace_bytes, p.total, stream);
    if (ws.status() != KDA_OK) return ws.status();
    a.out = static_cast<uint16_t *>(out);
    a.lse = lse;
    hipError_t e = hipSuccess;
    if (packed && !counted) {
        int32_t *table = reinterpret_cast<int32_t *>(ws.at(0));
        e = kda_launch_latent_table(a, p.block, table, a.blocks, nullptr, 0, stream);
        a.table = table;
    }
    if (p.parts > 1) {
        a.part_stat = reinterpret_cast<float *>(ws.at(p.off_stat));
        a.part = reinterpret_cast<float *>(ws.at(p.off_part));
    }
    if (e == hipSuccess) e = kda_launch_latent_fwd(a, p.block, stream);
    return of_hip(e);
}

namespace {
struct LatentBwdPlan {
    int64_t q_blocks, k_blocks, q_parts, k_parts;
    int part_tiles;
    size_t off_qt, off_kt, off_stat, off_part, off_q, off_k, total;
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
    p.off_q = p.off_k = p.total = p.off_part + align_up(latent_keys(d) * (size_t)d->H * kPe * 4, 256);
    p.q_parts = p.k_parts = 1;
    // Few blocks are split as in the forward, here by a common number of tiles of the other side, for some
    // 256 workgroups, all that run at once (4096 tokens x 2 heads 136 -> 90 us, with 512 of them 102; 512
    // tokens of one head over 8512 keys 209 -> 42).
    constexpr int64_t kFewUnits = 128, kUnits = 256;
    const int64_t q_units = p.q_blocks * d->B * d->H, k_units = p.k_blocks * d->B * d->H;
    const int64_t q_tiles = (d->T + kKeys - 1) / kKeys, k_tiles = (d->Tk + kKeys - 1) / kKeys;
    if (q_units + k_units > kFewUnits || std::max(q_tiles, k_tiles) <= kFewTiles) return KDA_OK;
    p.part_tiles = (int)std::max<int64_t>(kPartTiles, (q_units * k_tiles + k_units * q_tiles + kUnits - 1) / kUnits);
    p.q_parts = std::max<int64_t>(1, (k_tiles + p.part_tiles - 1) / p.part_tiles);
    p.k_parts = std::max<int64_t>(1, (q_tiles + p.part_tiles - 1) / p.part_tiles);
    p.off_k = p.off_q + (size_t)(q_units * p.q_parts) * kLatentBwdBlock * kQk * 4;
    p.total = p.off_k + (size_t)(k_units * p.k_parts) * kLatentBwdBlock * (kQk + kVal) * 4;
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
    a.parts = p.q_parts;
    k.parts = p.k_parts;
    a.part_tiles = k.part_tiles = p.part_tiles;
    a.part = reinterpret_cast<float *>(ws.at(p.off_q));
    k.part = reinterpret_cast<float *>(ws.at(p.off_k));
    hipError_t e = hipSuccess;
    if (packed && !kda_latent_counted(desc->num_seqs, std::max(p.q_blocks, p.k_blocks) * desc->H)) {
        int32_t *qt = reinterpret_cast<int32_t *>(ws.at(p.off_qt)), *kt = reinterpret_cast<int32_t *>(ws.at(p.off_kt));
        e = kda_launch_latent_table(a, kLatentBwdBlock, qt, p.q_blocks, kt, p.k_blocks, stream);
        a.table = qt;
        k.table = kt;
    }
    if (e == hipSuccess) e = kda_launch_latent_pairs(a, k, stream);
    if (e == hipSuccess) e = kda_launch_latent_dpe(k, stream);
    return of_hip(e);
}

// ---- the absorbed form ----

namespace {

struct DecodePlan {
    int rows32;
    int64_t row_tiles;
    size_t off_seg, off_stat, off_part, total;
};

bool page_ok(int64_t size) { return size >= 1 && size <= 65536 && (size & (size - 1)) == 0; }
int log2_of(int64_t v) {
    int s = 0;
    while ((int64_t(1) << s) < v) ++s;
    return s;
}

kda_status_t plan_decode(const kda_latent_decode_desc_t *d, DecodePlan &p) {
    if (d->N < 0 || d->T < 1 || d->H < 1 || d->pages < 0 || d->max_pages < 0) return KDA_ERR_SHAPE;
    if (!page_ok(d->page_size)) return KDA_ERR_UNSUPPORTED;
    constexpr int64_t kMaxRows = int64_t(1) << 24;
    if (d->H > 65535 || d->T > kMaxRows / d->H || d->N > kMaxRows / (d->T * d->H)) return KDA_ERR_SHAPE;
    if (d->pages > kMaxSeqs / d->page_size || d->max_pages > kMaxSeqs || d->max_pages > kMaxAttention / d->page_size) return KDA_ERR_SHAPE;
    const int64_t strides[] = {d->ql_stride_n, d->ql_stride_t, d->ql_stride_h, d->qp_stride_n, d->qp_stride_t, d->qp_stride_h};
    for (int64_t s : strides)
        if (!stride_ok(s)) return KDA_ERR_SHAPE;
    for (int64_t s : strides)
        if (s % 8 != 0) return KDA_ERR_ALIGN;
    if (!scale_ok(d->scale)) return KDA_ERR_PARAM;
    const int64_t rows = d->T * d->H;
    p.rows32 = rows <= 32 ? 1 : 2;
    p.row_tiles = (rows + 32 * p.rows32 - 1) / (32 * p.rows32);
    // a workgroup counts its steps of 32 cached rows in 32 bits
    if (d->N > 0 && d->max_pages * d->page_size > (int64_t(1) << 43) / (d->N * p.row_tiles)) return KDA_ERR_SHAPE;
    const size_t slots = 2 * (size_t)kLatentGroups, lanes = (size_t)p.rows32 * 32;
    p.off_seg = 0;
    p.off_stat = align_up((size_t)(d->N * p.row_tiles) * 8, 256);
    p.off_part = p.off_stat + align_up(slots * lanes * 8, 256);
    p.total = p.off_part + slots * lanes * kLat * 4;
    return KDA_OK;
}

// Elements from the first to behind the last of [n, t, h, inner].
size_t extent4(int64_t n, int64_t sn, int64_t t, int64_t st, int64_t h, int64_t sh, int64_t inner) {
    return n > 0 ? (size_t)((n - 1) * sn + (t - 1) * st + (h - 1) * sh + inner) * 2 : 0;
}

}  // namespace

extern "C" size_t kda_latent_decode_workspace_size(const kda_latent_decode_desc_t *desc) {
    DecodePlan p;
    return desc && plan_decode(desc, p) == KDA_OK ? p.total : 0;
}

extern "C" kda_status_t kda_latent_decode(const void *q_latent, const void *q_pe, const void *cache, const int64_t *lengths,
                                          const int32_t *block_table, void *out, float *lse,
                                          const kda_latent_decode_desc_t *desc, hipStream_t stream) {
    if (!desc) return KDA_ERR_NULL;
    DecodePlan p;
    const kda_status_t st = plan_decode(desc, p);
    if (st != KDA_OK) return st;
    const bool any = desc->N > 0;
    const bool keys = any && desc->pages > 0 && desc->max_pages > 0;
    if (any && (!q_latent || !q_pe || !lengths || !out)) return KDA_ERR_NULL;
    if (keys && (!cache || !block_table)) return KDA_ERR_NULL;
    if (!aligned(q_latent, 16) || !aligned(q_pe, 16) || !aligned(cache, 16) || !aligned(out, 16) || !aligned(lengths, 8) ||
        !aligned(block_table, 4) || !aligned(lse, 4))
        return KDA_ERR_ALIGN;
    const size_t rows = (size_t)(desc->N * desc->T) * (size_t)desc->H;
    Memory m;
    m.read(q_latent, extent4(desc->N, desc->ql_stride_n, desc->T, desc->ql_stride_t, desc->H, desc->ql_stride_h, kLat));
    m.read(q_pe, extent4(desc->N, desc->qp_stride_n, desc->T, desc->qp_stride_t, desc->H, desc->qp_stride_h, kPe));
    m.read(cache, (size_t)desc->pages * (size_t)desc->page_size * kRow * 2);
    m.read(lengths, (size_t)desc->N * 8);
    m.read(block_table, (size_t)(desc->N * desc->max_pages) * 4);
    m.write(out, rows * kLat * 2);
    m.write(lse, rows * 4);
    m.write(desc->workspace, p.total);
    if (m.clash()) return KDA_ERR_OVERLAP;
    if (!any) return KDA_OK;
    Workspace ws(desc->workspace, desc->workspace_bytes, p.total, stream);
    if (ws.status() != KDA_OK) return ws.status();
    LatentDecodeArgs a{};
    a.ql = static_cast<const uint16_t *>(q_latent);
    a.qp = static_cast<const uint16_t *>(q_pe);
    a.cache = static_cast<const uint16_t *>(cache);
    a.qln = desc->ql_stride_n; a.qlt = desc->ql_stride_t; a.qlh = desc->ql_stride_h;
    a.qpn = desc->qp_stride_n; a.qpt = desc->qp_stride_t; a.qph = desc->qp_stride_h;
    a.len = lengths; a.table = block_table;
    a.N = desc->N; a.T = desc->T; a.H = desc->H; a.pages = desc->pages;
    a.max_pages = keys ? desc->max_pages : 0;  // no cache: no sequence has keys
    a.page_shift = log2_of(desc->page_size);
    a.scale = desc->scale;
    a.out = static_cast<uint16_t *>(out);
    a.lse = lse;
    a.rows32 = p.rows32; a.row_tiles = p.row_tiles;
    a.groups = kLatentGroups;
    a.seg = reinterpret_cast<int32_t *>(ws.at(p.off_seg));
    a.part_stat = reinterpret_cast<float *>(ws.at(p.off_stat));
    a.part = reinterpret_cast<float *>(ws.at(p.off_part));
    hipError_t e = kda_launch_latent_decode(a, stream);
    if (e == hipSuccess) e = kda_launch_latent_join(a, stream);
    return of_hip(e);
}

// ---- the cache ----

extern "C" kda_status_t kda_latent_store(const void *latent, const void *k_pe, const void *weight, const int64_t *slots,
                                         void *cache, void *normed, const kda_latent_store_desc_t *desc, hipStream_t stream) {
    if (!desc) return KDA_ERR_NULL;
    if (desc->tokens < 0 || desc->num_slots < 0 || desc->tokens > kMaxTokens || desc->num_slots > kMaxTokens) return KDA_ERR_SHAPE;
    if (!stride_ok(desc->latent_stride) || !stride_ok(desc->pe_stride)) return KDA_ERR_SHAPE;
    if (weight && !dtype_ok(desc->weight_dtype)) return KDA_ERR_DTYPE;
    // a smaller eps is zero to the hardware's reciprocal root
    if (weight && (!(desc->eps >= 0x1p-126f) || !isfinite(desc->eps))) return KDA_ERR_PARAM;
    if (desc->latent_stride % 8 != 0 || desc->pe_stride % 8 != 0) return KDA_ERR_ALIGN;
    if (desc->tokens > 0 && (!latent || !k_pe || !slots || (desc->num_slots > 0 && !cache))) return KDA_ERR_NULL;
    if (!aligned(latent, 16) || !aligned(k_pe, 16) || !aligned(cache, 16) || !aligned(normed, 16) || !aligned(slots, 8) ||
        (weight && !aligned(weight, width(desc->weight_dtype))))
        return KDA_ERR_ALIGN;
    Memory m;
    m.read(latent, extent(1, 0, desc->tokens, desc->latent_stride, kLat, 2));
    m.read(k_pe, extent(1, 0, desc->tokens, desc->pe_stride, kPe, 2));
    if (weight) m.read(weight, kLat * width(desc->weight_dtype));
    m.read(slots, (size_t)desc->tokens * 8);
    m.write(cache, (size_t)desc->num_slots * kRow * 2);
    m.write(normed, (size_t)desc->tokens * kLat * 2);
    if (m.clash()) return KDA_ERR_OVERLAP;
    if (desc->tokens == 0) return KDA_OK;
    LatentStoreArgs a{};
    a.latent = static_cast<const uint16_t *>(latent); a.ls = desc->latent_stride;
    a.pe = static_cast<const uint16_t *>(k_pe); a.ps = desc->pe_stride;
    a.w = weight; a.w_f32 = desc->weight_dtype == KDA_FP32;
    a.slots = slots;
    a.cache = static_cast<uint16_t *>(cache);
    a.normed = static_cast<uint16_t *>(normed);
    a.tokens = desc->tokens; a.num_slots = desc->num_slots;
    a.eps = desc->eps;
    return of_hip(kda_launch_latent_store(a, stream));
}

namespace {
kda_status_t check_pages(const kda_page_desc_t *d) {
    if (d->N < 0 || d->max_pages < 0 || d->stack < 0 || d->tokens < 0) return KDA_ERR_SHAPE;
    if (d->N > int64_t(1) << 20 || d->max_pages > kMaxSeqs || d->stack > kMaxSeqs || d->tokens > kMaxSeqs) return KDA_ERR_SHAPE;
    if (d->N * d->max_pages > kMaxSeqs) return KDA_ERR_SHAPE;
    return page_ok(d->page_size) ? KDA_OK : KDA_ERR_UNSUPPORTED;
}
}  // namespace

extern "C" size_t kda_page_workspace_size(const kda_page_desc_t *desc) {
    return desc && check_pages(desc) == KDA_OK ? align_up((size_t)(2 * desc->N + 3) * 8, 256) : 0;
}

extern "C" kda_status_t kda_page_assign(const int64_t *lengths, const int64_t *new_tokens, const uint8_t *ended,
                                        int32_t *block_table, int32_t *free_pages, const int64_t *free_count, int64_t *slots,
                                        int64_t *cu_seqlens, int64_t *lengths_out, int64_t *granted, int64_t *free_count_out,
                                        const kda_page_desc_t *desc, hipStream_t stream) {
    if (!desc) return KDA_ERR_NULL;
    const kda_status_t st = check_pages(desc);
    if (st != KDA_OK) return st;
    if (!free_count || !free_count_out || !cu_seqlens) return KDA_ERR_NULL;
    if (desc->N > 0 && (!lengths || !new_tokens || !lengths_out || !granted || (desc->max_pages > 0 && !block_table)))
        return KDA_ERR_NULL;
    if ((desc->stack > 0 && !free_pages) || (desc->tokens > 0 && !slots)) return KDA_ERR_NULL;
    for (const void *q : {(const void *)lengths, (const void *)new_tokens, (const void *)free_count, (const void *)slots,
                          (const void *)cu_seqlens, (const void *)lengths_out, (const void *)granted, (const void *)free_count_out})
        if (!aligned(q, 8)) return KDA_ERR_ALIGN;
    if (!aligned(block_table, 4) || !aligned(free_pages, 4)) return KDA_ERR_ALIGN;
    const size_t n = (size_t)desc->N, need = kda_page_workspace_size(desc);
    Memory m;
    m.read(lengths, n * 8);
    m.read(new_tokens, n * 8);
    m.read(ended, n);
    m.read(free_count, 8);
    m.write(block_table, n * (size_t)desc->max_pages * 4);
    m.write(free_pages, (size_t)desc->stack * 4);
    m.write(slots, (size_t)desc->tokens * 8);
    m.write(cu_seqlens, (n + 1) * 8);
    m.write(lengths_out, n * 8, lengths);
    m.write(granted, n * 8);
    m.write(free_count_out, 8, free_count);
    m.write(desc->workspace, need);
    if (m.clash()) return KDA_ERR_OVERLAP;
    Workspace ws(desc->workspace, desc->workspace_bytes, need, stream);
    if (ws.status() != KDA_OK) return ws.status();
    PageArgs a{};
    a.len = lengths; a.add = new_tokens; a.ended = ended;
    a.table = block_table; a.free_pages = free_pages; a.count = free_count;
    a.slots = slots; a.cu = cu_seqlens; a.len_out = lengths_out; a.granted = granted; a.count_out = free_count_out;
    a.N = desc->N; a.max_pages = desc->max_pages; a.stack = desc->stack; a.tokens = desc->tokens;
    a.shift = log2_of(desc->page_size);
    a.have = reinterpret_cast<int64_t *>(ws.at(0));
    a.base = a.have + 2;
    a.back = a.base + a.N;
    return of_hip(kda_launch_pages(a, stream));
}
