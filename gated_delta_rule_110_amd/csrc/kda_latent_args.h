// kda_latent_args.h -- kernel arguments and launchers of latent attention and its
// cache (include/kda_latent.h).
#pragma once
#include "kda_layer_args.h"

namespace kda {

constexpr int kNope = 128, kPe = 64, kQk = kNope + kPe;   // a head's own key values, the shared ones, both
constexpr int kVal = 128, kKvRow = kNope + kVal;          // a head's values, its row of kv
constexpr int kLat = 512, kRow = kLat + kPe;              // the latent, a cached row
constexpr int kKeys = 64;                                 // keys (or queries) of a tile in LDS
// Few blocks have their tiles split into parts of at least kPartTiles; up to kFewTiles in all are
// not worth a second kernel (700 queries of one head over their own 11 tiles would take 21 us instead of 18).
constexpr int kPartTiles = 8, kFewTiles = 12;

struct LatentArgs {
    const uint16_t *q, *kv, *pe;
    int64_t qb, qt, kvb, kvt, peb, pet;
    const int64_t *cu, *cuk;   // packed: offsets of queries and keys, else nullptr
    int64_t B, T, Tk, H, seqs;
    int64_t blocks;            // blocks of queries (keys) per batch row; packed: at most, in all
    const int32_t *table;      // packed: their number, then (sequence, block) of each, longest first; or nullptr
    float scale;
    int causal;
    uint16_t *out;
    float *lse;
    int64_t launch_cap, base;  // base: first workgroup of this launch; set by the launcher
    // parts (1: none) of part_tiles tiles of the other side that a block's work may be split in (packed: as
    // many at most, of a number of tiles that goes by the sequence); what each leaves of its 128 tokens:
    // accumulators, and in the forward (maximum, sum)
    int64_t parts;
    int part_tiles;
    float *part, *part_stat;
    // gradient
    const uint16_t *o, *dy;    // out, d_out
    int64_t ob, ot, yb, yt;
    const float *lse_in;
    float *stat;               // [2][H][B T]: lse in log2 units (0 where no key is seen), d_out . out
    float *dpe_part;           // [H, B Tk, 64] fp32
    uint16_t *dq, *dkv, *dpe;
};

struct LatentDecodeArgs {
    const uint16_t *ql, *qp, *cache;
    int64_t qln, qlt, qlh, qpn, qpt, qph;
    const int64_t *len;
    const int32_t *table;
    int64_t N, T, H, pages, max_pages;
    int page_shift;
    float scale;
    uint16_t *out;
    float *lse;
    int rows32;                // 32-row tiles of a workgroup's rows, 1 or 2
    int64_t row_tiles;         // row tiles of a sequence
    int64_t groups;            // workgroups the steps are shared among
    // What a workgroup leaves of the first (slot 2 w) and the last (slot 2 w + 1) of its
    // row tiles where others have a part of it: accumulators, and (maximum, sum) of 64 rows.
    float *part, *part_stat;
    int32_t *seg;              // [N row_tiles][2]: first slot and last workgroup; (-1, 0): no part, nothing left to do,
                               // (-2, 0): no keys
};

struct LatentStoreArgs {
    const uint16_t *latent, *pe;
    int64_t ls, ps;            // elements between rows
    const void *w;             // [512] or nullptr
    const int64_t *slots;
    uint16_t *cache, *normed;
    int64_t tokens, num_slots;
    int w_f32;
    float eps;
};

struct PageArgs {
    const int64_t *len, *add;
    const uint8_t *ended;
    int32_t *table, *free_pages;
    const int64_t *count;
    int64_t *slots, *cu, *len_out, *granted, *count_out;
    int64_t N, max_pages, stack, tokens;
    int shift;                 // log2 of the page size
    // workspace
    int64_t *have;             // [2] pages on the stack once all are back, and before
    int64_t *base, *back;      // [N], [N + 1] pages that the requests before one take, and give back
};

}  // namespace kda

// Queries per workgroup of the forward (128 or 256), by which its table is made.
int kda_latent_block(int64_t B, int64_t T, int64_t H, int64_t seqs);
// Whether the workgroups (units: blocks times heads) of a packed batch count through its
// sequences themselves: one launch less where they all run at once, so that it does not matter which
// comes first (1000 tokens in 7 sequences x 32 heads: 30 -> 25 us).
bool kda_latent_counted(int64_t seqs, int64_t units);
// The tables of a packed batch: blocks of `size` queries and (where keys is given) keys of
// every sequence, those with the most tiles first.  int32 [2 + 2 blocks].
hipError_t kda_launch_latent_table(const kda::LatentArgs &a, int size, int32_t *queries, int64_t q_blocks, int32_t *keys,
                                   int64_t k_blocks, hipStream_t s);
// With parts (blocks of 128 queries only) their joining too.
hipError_t kda_launch_latent_fwd(const kda::LatentArgs &a, int block, hipStream_t s);
// The gradient: dq and `stat`, dkv and the heads' parts of dk_pe (q, k: the passes' blocks and
// tables); then their sum.
constexpr int kLatentBwdBlock = 128;  // queries or keys per workgroup
hipError_t kda_launch_latent_pairs(const kda::LatentArgs &q, const kda::LatentArgs &k, hipStream_t s);
hipError_t kda_launch_latent_dpe(const kda::LatentArgs &a, hipStream_t s);
// The absorbed form: the workgroups' parts, then their joining.
constexpr int64_t kLatentGroups = 256;
hipError_t kda_launch_latent_decode(const kda::LatentDecodeArgs &a, hipStream_t s);
hipError_t kda_launch_latent_join(const kda::LatentDecodeArgs &a, hipStream_t s);
hipError_t kda_launch_latent_store(const kda::LatentStoreArgs &a, hipStream_t s);
hipError_t kda_launch_pages(const kda::PageArgs &a, hipStream_t s);
