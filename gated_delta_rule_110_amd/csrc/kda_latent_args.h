// kda_latent_args.h -- kernel arguments and launchers of latent attention and its
// cache (include/kda_latent.h).
#pragma once
#include "kda_layer_args.h"

namespace kda {

constexpr int kNope = 128, kPe = 64, kQk = kNope + kPe;   // a head's own key values, the shared ones, both
constexpr int kVal = 128, kKvRow = kNope + kVal;          // a head's values, its row of kv
constexpr int kLat = 512, kRow = kLat + kPe;              // the latent, a cached row
constexpr int kKeys = 64;                                 // keys (or queries) of a tile in LDS

struct LatentArgs {
    const uint16_t *q, *kv, *pe;
    int64_t qb, qt, kvb, kvt, peb, pet;
    const int64_t *cu, *cuk;   // packed: offsets of queries and keys
    int64_t B, T, Tk, H, seqs;
    int64_t blocks;            // blocks of queries (keys) per batch row; packed: at most, in all
    const int32_t *table;      // packed: their number, then (sequence, block) of each, longest first
    float scale;
    int causal;
    uint16_t *out;
    float *lse;
    int64_t launch_cap, base;  // base: first workgroup of this launch; set by the launcher
    // gradient
    const uint16_t *o, *dy;    // out, d_out
    int64_t ob, ot, yb, yt;
    const float *lse_in;
    float *stat;               // [2][H][B T]: lse in log2 units (0 where no key is seen), d_out . out
    float *dpe_part;           // [H, B Tk, 64] fp32
    uint16_t *dq, *dkv, *dpe;
};

}  // namespace kda

// Queries per workgroup of the forward: the caller's table is made for them.
int kda_latent_block(int64_t B, int64_t T, int64_t H);
// The table of a packed batch: blocks of `size` queries (or keys, with by_keys) of every sequence, those with the
// most tiles first.  table: int32 [2 + 2 blocks].
hipError_t kda_launch_latent_table(const kda::LatentArgs &a, int size, int by_keys, int32_t *table, hipStream_t s);
hipError_t kda_launch_latent_fwd(const kda::LatentArgs &a, int block, hipStream_t s);
// The gradient: dq and `stat`, then dkv and the heads' parts of dk_pe, then their sum.
constexpr int kLatentBwdBlock = 128;  // queries or keys per workgroup
hipError_t kda_launch_latent_dq(const kda::LatentArgs &a, hipStream_t s);
hipError_t kda_launch_latent_dkv(const kda::LatentArgs &a, hipStream_t s);
hipError_t kda_launch_latent_dpe(const kda::LatentArgs &a, hipStream_t s);
