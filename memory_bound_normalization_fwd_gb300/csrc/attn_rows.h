// How a call of attention over the cache is dealt out to the row kernels (attn_rows.cuh), and
// their launches by format.
#pragma once

#include "ops.h"

namespace rmsn {

// The rows of a sequence that share a key head (queries times the query heads of a key
// head) are taken in blocks of 8 * NT, and the tokens in tiles. A slot is a block of a
// sequence; the CTAs of a head block take equal runs of all slots' tiles.
struct RowsPlan {
    int gd;           // groups of a head that the kernel is made for: 2, 3, 4, 6 or 8, at least the cache's
    int nt;           // 8 * nt rows a block: 1, 2, or 4 up to 3 groups
    int hb;           // key heads of a CTA
    int wph;          // warps a key head, which take turns at the tokens of a tile
    int head_blocks;  // heads / hb
    int slots;        // at least the slots of the call: rows * G / (8 nt) + sequences
    int gx;           // CTAs a head block
    int start_tiles;  // tiles that a slot's start counts as in the runs
    int split;        // 1: equal runs of tiles; 0: whole slots, one after another
    int tile_shift;   // tokens of a tile, as a power of two
    int most_tokens;  // that a row of the table has room for (below 2^31)
    int window;       // 0: none
    uint32_t g_mul;   // i / G = i * g_mul >> g_shift for i < 2^31
    int g_shift;
    uint32_t pages;
    uint32_t page_mul;  // t / page_size = t * page_mul >> page_shift for t < 2^31
    int page_shift;
    int narrow;       // 0, or the bytes that codes are copied by: 4 or 16 (heads that are not whole groups)
    int vec_scales;   // a head's scale bytes are read at once
    int vec_q;        // rows of q are read by vectors
    int vec_out;      // rows of out are written in pairs
    int ring;         // bytes of a warp's ring (also room for its results)
    int at_q, at_factors, at_ring, at_plan;  // offsets in shared memory
    int smem;
    // the workspace, of parts of slots that were split: two a CTA of a head block
    int4* entries;    // [slots]: the first CTA and (from bit 16) the last, -1 where one CTA took all of it;
                      // the sequence's first row, the block's first row and rows
    float2* ml;       // [2 gx][heads][rows of a block]: maximum, sum
    float* o;         // [2 gx][heads][rows of a block][gd * 32]
};

constexpr int kSplitSlots = 1024;  // most slots (and sequences) of a call that is dealt out evenly

// Allows a kernel `smem` bytes of shared memory on the current device, once.
cudaError_t allow_smem(const void* kernel, int smem);

// The row kernels by format and type; attn_join puts the parts of split slots together.
cudaError_t attn_rows_e2m1(const AttnP& p, const RowsPlan& r, const OpCfg& c);
cudaError_t attn_rows_e2m1_fp32(const AttnP& p, const RowsPlan& r, const OpCfg& c);
cudaError_t attn_rows_e4m3(const AttnP& p, const RowsPlan& r, const OpCfg& c);
cudaError_t attn_rows_e4m3_fp32(const AttnP& p, const RowsPlan& r, const OpCfg& c);
cudaError_t attn_join(const AttnP& p, const RowsPlan& r, const OpCfg& c);
// Prompts, on the tensor cores: 16-bit types, heads of 64, 96 or 128 values, vectors everywhere.
cudaError_t attn_tiles(const AttnP& p, const RowsPlan& r, const OpCfg& c);

// Bytes of a token's codes in a warp's ring: an odd number of 16 bytes, so that eight tokens'
// pieces of 16 bytes lie on different banks.
__host__ __device__ constexpr int rows_pitch(bool e4m3, int groups) {
    return ((e4m3 ? 2 * groups : groups) | 1) * 16;
}
// Floats a token in the factors' table.
__host__ __device__ constexpr int rows_factors(int groups) { return groups <= 2 ? 2 : groups <= 4 ? 4 : 8; }

}  // namespace rmsn
