// What the paged key/value cache's kernels share: device views of the cache
// and of a step's batch, the search of a row's sequence, and the launchers.
// Semantics of the entry points: include/lora_mi355x.h.
#pragma once

#include "lora_internal.hpp"

namespace lora {

struct KvDev {
    void* k;
    void* v;
    int64_t page_stride, token_stride, head_stride;   // elements
    int32_t n_pages;
    int32_t page_shift;   // page_size = 1 << page_shift
    int32_t n_kv_heads;
};

struct KvBatchDev {
    const int32_t* row_off;   // [n_seqs + 1]
    const int32_t* kv_len;    // [n_seqs]
    const int32_t* pages;     // [n_seqs, ldp]
    int64_t ldp;
    int32_t n_seqs, n_rows;
    // groups of sequences behind one prefix (n_groups = 0: none)
    const int32_t* group_off;      // [n_groups + 1]
    const int32_t* prefix_len;     // [n_groups]
    const int32_t* prefix_pages;   // [n_groups, ldpp]
    int64_t ldpp;
    int32_t n_groups;
};

// Number of i in 1 .. n with off[i] <= key, off ascending: the run that `key`
// lies in when off holds run boundaries with off[0] = 0 (n: past the last).
// Called by one whole wave with a uniform key; 64 probes a round, so one
// round up to 64 runs and two up to 4096.  Any content of off ends it, with
// an answer in [0, n].
__device__ inline int wave_find_run(const int32_t* __restrict__ off, int n, int key, int lane) {
    int lo = 0, hi = n;
    while (lo < hi) {
        const int step = (hi - lo + 63) >> 6;
        const int i = lo + (lane + 1) * step;
        const bool le = i <= hi && off[i] <= key;
        const int c = __popcll(__ballot(le));
        hi = min(hi, lo + (c + 1) * step - 1);
        lo += c * step;
    }
    return lo;
}

struct AppendArgs {
    KvDev C;
    KvBatchDev B;
    const float* cos;   // null: no rotation
    const float* sin;
    int64_t ldr;
    int32_t n_pos, half;   // half: rotated pairs of a head
    int32_t interleaved;
    const void* q;
    const void* k;
    const void* v;
    int64_t ldq, ldk, ldv;
    int32_t n_q_heads;
    void* q_out;
    int64_t ldqo;
    int32_t* status;
};
hipError_t launch_kv_append(const AppendArgs& a, lora_dtype_t in, lora_dtype_t cache, int32_t head_dim,
                            hipStream_t stream);

// Attention over the pages.  A "problem" is a sequence over its own tokens
// (kind 0) or a group of sequences over their shared prefix (kind 1).  Its
// query columns are (row, query head of one key head) pairs, row-major; up to
// ATTN_FEW_COLS of them go to the few-column kernel, which splits keys over
// waves and workgroups, more to the tiled kernel, which splits columns.
constexpr int ATTN_FEW_COLS = 16;
constexpr int ATTN_FEW_KEYS = 128;     // keys of a few-column work unit
constexpr int ATTN_FEW_WGS = 512;      // workgroups that share the units
constexpr int ATTN_TILE_KEYS = 64;

struct AttnPart {       // one kind's kernels and where their partial results lie
    int32_t max_rows;   // host bounds that the sizes below rest on: a problem's rows
    int32_t max_len;    // and keys past them are not looked at
    int32_t few;        // 0: not launched, 1: a workgroup per (problem, head), 2: units shared
    int32_t few_grid;   // its workgroups
    int32_t spl;        // key tiles of a tiled item
    int32_t tile_grid;  // tiled items at most (0: no problem has that many columns)
    int32_t slots;      // tiled items write partial results (some problem may be split)
    int2* rec;          // few 2: first and last workgroup of each (problem, head)
    float* few_o;       // [2 * ATTN_FEW_WGS][16][head_dim], unnormalised
    float2* few_ml;     // [..][16] (largest score, sum)
    int4* item;         // tiled: first item, column tiles, splits of each problem
    float* tile_o;      // [tile_grid][tile_cols][head_dim]
    float2* tile_ml;
    float* row_o;       // [n_rows][n_q_heads][head_dim]: whole results that the join still needs
    float2* row_ml;
};

struct AttnArgs {
    KvDev C;
    KvBatchDev B;
    const void* q;
    int64_t ldq;
    int32_t n_q_heads, share;   // share: query heads per key head
    float scale;
    int32_t window, n_sink;     // window 0: none
    void* o;
    int64_t ldo;
    int32_t o_bf16;
    float* lse;                 // may be null
    int32_t* status;            // may be null
    int32_t join;               // outputs come from the join launch alone
    int32_t need_join;
    int32_t tile_cols;          // columns of a tiled item: 128 or 256
    int32_t together;           // both forms in one launch
    int32_t decode;             // every sequence has few columns
    AttnPart part[2];
};
struct AttnPlan {
    AttnArgs a;       // with part[] sized (pointers unset)
    size_t off[2][7]; // workspace offsets of part[].rec .. row_ml
    size_t bytes;
};
// max_rows, max_len: host bounds of a problem's rows and keys, per kind
void plan_attn(AttnPlan& P, int32_t head_dim, int32_t elem_bytes, const int32_t (&n_prob)[2], const int32_t (&max_rows)[2],
               const int32_t (&max_len)[2]);
hipError_t launch_attn(const AttnArgs& a, lora_dtype_t dt, int32_t head_dim, hipStream_t stream);

}  // namespace lora
