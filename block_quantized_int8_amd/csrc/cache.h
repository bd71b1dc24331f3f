// cache.h - the block-quantised key/value cache: where a value of it lies, and the launchers that
// write, read and attend to it (cache.hip, cache_attn.hip; api.cpp).
#pragma once

#include "mmq_internal.h"
#include "rows.h"

namespace mmq {

constexpr int CACHE_TILE = 32;              // tokens of a record
constexpr int CACHE_MAX_SEQS = 4096;        // sequences of an attention call

inline bool cache_type(mmq_wtype t) { return t == MMQ_Q8_0 || t == MMQ_Q4_0; }

// A record (mmq.h, "Key/value cache") holds 32 tokens of one head: its values, then its scales. Values lie in
// the order of the matrix core's operands, so that a wave's 16-byte loads are whole lines and nothing
// moves between lanes:
//   keys: lane = token (16 of them) x four groups of 8 values of a block (k of q k^T),
//   values: lane = value (16 of them) x four groups of 8 tokens (k of p v).
// The tokens of group g are 4g..4g+3 and 16+4g..16+4g+3: those whose scores a lane of group g holds
// after the first product. The scales of a lane's 8 tokens are one 16-byte load a block, for keys
// and for values.
__host__ __device__ constexpr int cache_values(bool q8, int D) { return q8 ? 32 * D : 16 * D; }
__host__ __device__ constexpr int cache_record(bool q8, int D) { return cache_values(q8, D) + 2 * D; }

// Byte of the first of 8 key values 8g.. of block b of token t: 8 bytes (q8_0) or 4 (q4_0).
__host__ __device__ inline int key_at(bool q8, int D, int t, int b, int g) {
    const int lane = g * 16 + (t & 15), h = t >> 4;
    return q8 ? ((h * (D / 64) + b / 2) * 64 + lane) * 16 + (b & 1) * 8
              : (((b / 2) * 64 + lane) * 2 + h) * 8 + (b & 1) * 4;
}
// The nibble of value 8g + j (j < 8) in its 4 bytes: j and j + 1 (j even) lie 16 bits apart.
__host__ __device__ inline int key_nibble(int j) { return j / 2 + (j & 1) * 4; }

// Byte of value i (0..31) of block b of token t. q4_0: values i and i + 16 share a byte (low, high
// nibble), given by i < 16; a token's neighbour of the same pair lies two bytes on.
__host__ __device__ inline int value_at(bool q8, int t, int b, int i) {
    const int lane = ((t & 15) >> 2) * 16 + (i & 15), hi = t >> 4, lo = t & 3;
    return q8 ? (b * 64 + lane) * 16 + (i >> 4) * 8 + hi * 4 + lo
              : ((b / 2) * 64 + lane) * 16 + (b & 1) * 8 + hi * 4 + (lo >> 1) + (lo & 1) * 2;
}
// Byte, after the values, of the f16 scale of block b of token t.
__host__ __device__ inline int scale_at(int D, int t, int b) {
    return ((((t & 15) >> 2) * (D / 32) + b) * 8 + (t >> 4) * 4 + (t & 3)) * 2;
}

// A cache: pages of `tiles` records a head.
struct CacheShape {
    int pages, tiles, heads, D;
};

hipError_t launch_cache_write(mmq_otype o, const void* k, int64_t ldk, const void* v, int64_t ldv, const int32_t* slots,
                              int64_t rows, mmq_wtype tk, void* kcache, mmq_wtype tv, void* vcache, CacheShape c,
                              hipStream_t s);
hipError_t launch_cache_read(mmq_otype o, const int32_t* slots, int64_t rows, mmq_wtype tk, const void* kcache,
                             mmq_wtype tv, const void* vcache, CacheShape c, void* k, int64_t ldk, void* v, int64_t ldv,
                             hipStream_t s);

struct AttnShape {
    int64_t rows, B, max_q, width;
    int Hq;
};
bool cache_attn_grid_ok(const CacheShape& c, const AttnShape& a);
size_t cache_attn_workspace_bytes(const CacheShape& c, const AttnShape& a);
hipError_t launch_cache_attn(mmq_otype o, const void* q, int64_t ldq, mmq_wtype tk, const void* kcache, mmq_wtype tv,
                             const void* vcache, CacheShape c, const int32_t* table, int64_t ldt, const int32_t* lens,
                             const int32_t* starts, AttnShape a, const uint64_t* mask, float scale, void* out,
                             int64_t ldo, void* workspace, hipStream_t s);

}  // namespace mmq
