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

// The same search for a row's sequence s, or for what grows with it (at(i, off[i])
// ascending; s the last with at <= key), with its first row, the next one's and
// its length, which come with the last probes.  false: past the last sequence.
template <class AT>
__device__ inline bool wave_find_seq(const KvBatchDev& B, int key, int lane, AT at, int& s, int& r0, int& r1, int& len) {
    int lo = 0, hi = B.n_seqs;
    while (hi - lo > 63) {
        const int step = (hi - lo + 63) >> 6;
        const int i = lo + (lane + 1) * step;
        const bool le = i <= hi && at(i, B.row_off[i]) <= key;
        const int c = __popcll(__ballot(le));
        hi = min(hi, lo + (c + 1) * step - 1);
        lo += c * step;
    }
    const int i = min(lo + lane, B.n_seqs);
    const int off = B.row_off[i], n = i < B.n_seqs ? B.kv_len[i] : 0;
    const int c = __popcll(__ballot(lane > 0 && lo + lane <= hi && at(i, off) <= key));
    s = lo + c;
    if (s >= B.n_seqs) return false;
    r0 = __builtin_amdgcn_readlane(off, c);
    len = __builtin_amdgcn_readlane(n, c);
    r1 = c < 63 ? __builtin_amdgcn_readlane(off, c + 1) : B.row_off[s + 1];
    return true;
}

// What a cache in 8 bits has besides (KvDev's strides are then bytes).
constexpr int Q8_LEAST = -100, Q8_MOST = 100;   // exponents of a scale
struct Q8Dev {
    float* k_scale;
    float* v_scale;
    int64_t page_stride, block_stride, head_stride;   // of the scales
    int32_t block_shift;   // block_size = 1 << block_shift
    int32_t n_kv_heads;
    // append: room for a sequence's blocks beyond its rows / block_size, and
    // all (block, head, K or V) units
    int32_t per;
    int64_t units;
};

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
    Q8Dev S;
};
hipError_t launch_kv_append(const AppendArgs& a, lora_dtype_t in, lora_dtype_t cache, int32_t head_dim,
                            hipStream_t stream);
// C.n_kv_heads is 0 here (the rows' part is the queries'), S.n_kv_heads is not
hipError_t launch_kv_append_q8(const AppendArgs& a, lora_dtype_t in, int32_t head_dim, hipStream_t stream);

struct PlanArgs {   // lora_kv_plan_t, and where its workspace's parts lie
    const int32_t* new_rows;
    const int32_t* adapter;
    const int32_t* kv_len;
    int32_t* kv_len_out;
    int32_t* pages;
    int64_t ldp;
    int32_t* free_pages;
    const int32_t* n_free;
    int32_t* n_free_out;
    const int32_t* group_off;
    const int32_t* prefix_len;
    int32_t* row_off;
    int32_t* row_seq;
    int32_t* row_adapter;
    int32_t* row_pos;
    int64_t* row_slot;
    int32_t n_seqs, n_groups, page_shift, max_free, max_rows;
    int32_t* status;
    int32_t* take;   // [n_seqs + 1] granted pages before a sequence
    int32_t* back;   // [n_seqs + 1] returned pages
    int32_t* len;    // [n_seqs] tokens before the step
    int32_t* head;   // the stack's old height, and with the returned pages; granted rows and pages
};
size_t plan_bytes(int32_t n_seqs);
hipError_t launch_kv_plan(PlanArgs a, void* ws, hipStream_t stream);

// Attention over the pages.  A "problem" is a sequence over its own tokens
// (kind 0) or a group of sequences over their shared prefix (kind 1).  Its
// query columns are (row, query head of one key head) pairs, row-major; up to
// ATTN_FEW_COLS of them go to the few-column kernel, which splits keys over
// waves and workgroups, more to the tiled kernel, which splits columns.
constexpr int ATTN_FEW_COLS = 16;
constexpr int ATTN_FEW_KEYS = 128;     // keys of a few-column work unit
constexpr int ATTN_WAVE_KEYS_Q8 = 64;  // in 8 bits: of a wave
constexpr int ATTN_FEW_WGS = 512;      // workgroups that share the units
constexpr int ATTN_TILE_KEYS = 64;

// Waves of a few-column workgroup in 8 bits.  Beside tiles it has their four;
// alone eight, so that a (problem, key head) that has a workgroup to itself has
// a whole CU's waves.  Heads of 256 need the registers of two waves.
constexpr int few_waves_q8(int head_dim, bool together) { return together || head_dim > 128 ? 4 : 8; }

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
    Q8Dev S;                    // a cache in 8 bits
};
struct AttnPlan {
    AttnArgs a;       // with part[] sized (pointers unset)
    size_t off[2][7]; // workspace offsets of part[].rec .. row_ml
    size_t bytes;
};
// max_rows, max_len: host bounds of a problem's rows and keys, per kind
void plan_attn(AttnPlan& P, int32_t head_dim, int32_t elem_bytes, const int32_t (&n_prob)[2], const int32_t (&max_rows)[2],
               const int32_t (&max_len)[2], bool in_8_bits = false);
hipError_t launch_attn(const AttnArgs& a, lora_dtype_t dt, int32_t head_dim, hipStream_t stream);
hipError_t launch_attn_q8(const AttnArgs& a, int32_t head_dim, hipStream_t stream);

}  // namespace lora
