// A step's tables from its requests' rows (lora_kv_plan): who is served, the
// pages that are taken and given back, and each row's sequence, adapter,
// position and place.
//
// All of it follows from prefix sums over the sequences: of pages that come
// back, of rows and pages asked for (who is served), and of rows and pages
// granted (where they lie).  Page k of the granted ones is the k-th from the
// top of the stack with the returned pages on it; neither that stack nor the
// tables in between are ever built: an entry of it is read from the free stack
// or, above its old height, from the table of the sequence that returns it.
// The two parts do not meet: pushed entries lie above the old height, popped
// ones of the free stack below, and a sequence that returns pages takes none.
//
// The bytes (20 a sequence and a row, 8 a page) are nothing; the time is a
// launch and chains of dependent loads.
#include "kv_internal.hpp"

namespace lora {
namespace {

constexpr int PL_WAVES = 16;
constexpr int PL_ONE_SEQS = 1024, PL_ONE_ROWS = 4096;   // up to these, one launch
constexpr int PL_FILL = 256;                            // threads of a filling workgroup

__device__ __forceinline__ int pages_of(int tokens, int shift) { return (int)(((int64_t)tokens + (1 << shift) - 1) >> shift); }

// sums of what requests ask for may pass 32 bits; past 2^31 - 1 they stay there
__device__ __forceinline__ int sat_add(int a, int b) {
    return (int)min((uint32_t)a + (uint32_t)b, 0x7fffffffu);
}
// Inclusive sums of three counts over the workgroup; total: all of them.  sh: 3 * PL_WAVES ints.
__device__ inline void scan3(int (&v)[3], int (&total)[3], int tid, int* sh) {
    const int lane = tid & 63, wave = tid >> 6;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        int o[3];
#pragma unroll
        for (int i = 0; i < 3; ++i) o[i] = __shfl_up(v[i], d, 64);
#pragma unroll
        for (int i = 0; i < 3; ++i)
            if (lane >= d) v[i] = sat_add(v[i], o[i]);
    }
    __syncthreads();
    if (lane == 63) {
#pragma unroll
        for (int i = 0; i < 3; ++i) sh[i * PL_WAVES + wave] = v[i];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 3; ++i) {
        int before = 0;
        total[i] = 0;
        for (int w = 0; w < PL_WAVES; ++w) {
            const int x = sh[i * PL_WAVES + w];
            if (w < wave) before = sat_add(before, x);
            total[i] = sat_add(total[i], x);
        }
        v[i] = sat_add(v[i], before);
    }
}

// number of i in 1 .. n with off[i] <= key
__device__ __forceinline__ int run_of(const int32_t* off, int n, int key) {
    int lo = 0, hi = n;
    while (lo < hi) {
        const int m = (lo + hi + 1) >> 1;
        if (off[m] <= key) lo = m;
        else hi = m - 1;
    }
    return lo;
}

struct Sums {              // of the whole step
    const int32_t* row;    // granted rows before sequence s, [n_seqs + 1]
    const int32_t* take;   // granted pages
    const int32_t* back;   // returned pages
    int rows, taken, old_free, there;   // there: old_free and the returned ones
};

// Entry `at` of the stack with the returned pages on it.
__device__ __forceinline__ int stack_at(const PlanArgs& a, const Sums& S, int at) {
    if (at < S.old_free) return a.free_pages[max(at, 0)];
    const int s = min(run_of(S.back, a.n_seqs, at - S.old_free), a.n_seqs - 1);
    return a.pages[(int64_t)s * a.ldp + max(min((int64_t)(at - S.old_free - S.back[s]), a.ldp - 1), (int64_t)0)];
}

// The tables' new pages, the stack's new entries and the rows, by `threads` threads.
__device__ inline void fill(const PlanArgs& a, const Sums& S, int at, int threads) {
    const int left = S.there - S.taken;
    for (int r = at; r < a.max_rows; r += threads) {
        int s = -1, adapter = -1, pos = -1;
        int64_t slot = -1;
        if (r < S.rows) {
            s = min(run_of(S.row, a.n_seqs, r), a.n_seqs - 1);
            const int first = S.row[s], n = S.row[s + 1] - first;
            const int before = a.kv_len_out[s] - n;     // its tokens before the step
            const int t = before + (r - first), held = pages_of(before, a.page_shift), pg = t >> a.page_shift;
            if (a.adapter) adapter = a.adapter[s];
            pos = t;
            if (a.n_groups) {
                const int g = run_of(a.group_off, a.n_groups, s);
                if (g < a.n_groups && s >= a.group_off[0]) pos += max(a.prefix_len[g], 0);
            }
            if (a.row_slot) {
                const int page = pg < held ? a.pages[(int64_t)s * a.ldp + min((int64_t)pg, a.ldp - 1)]
                                           : stack_at(a, S, S.there - 1 - (S.take[s] + pg - held));
                slot = ((int64_t)page << a.page_shift) + (t & ((1 << a.page_shift) - 1));
            }
        }
        if (a.row_seq) a.row_seq[r] = s;
        if (a.row_adapter) a.row_adapter[r] = adapter;
        if (a.row_pos) a.row_pos[r] = pos;
        if (a.row_slot) a.row_slot[r] = slot;
    }
    for (int k = at; k < S.taken; k += threads) {
        const int s = min(run_of(S.take, a.n_seqs, k), a.n_seqs - 1);
        const int n = S.row[s + 1] - S.row[s];
        const int64_t pg = (int64_t)pages_of(a.kv_len_out[s] - n, a.page_shift) + (k - S.take[s]);
        const int page = stack_at(a, S, S.there - 1 - k);
        if (pg < a.ldp) a.pages[(int64_t)s * a.ldp + pg] = page;
    }
    for (int i = S.old_free + at; i < left; i += threads) a.free_pages[i] = stack_at(a, S, i);
}

// One workgroup: the sums and everything of a sequence; ONE: the rest too.
template <bool ONE>
__global__ __launch_bounds__(64 * PL_WAVES) void k_plan(PlanArgs a) {
    __shared__ int sh[3 * PL_WAVES];
    __shared__ int s_off[ONE ? 3 : 1][ONE ? PL_ONE_SEQS + 1 : 1];
    const int tid = threadIdx.x, n = a.n_seqs;
    int32_t* take = ONE ? s_off[0] : a.take;
    int32_t* back = ONE ? s_off[ONE ? 1 : 0] : a.back;
    int32_t* row = ONE ? s_off[ONE ? 2 : 0] : a.row_off;
    const int old_free = min(max(*a.n_free, 0), a.max_free);

    // a sequence's length, the rows and pages it asks for, the pages it returns
    struct Seq {
        int len, want, need, back;
        bool asks;
    };
    auto load = [&](int s) {
        Seq q{0, 0, 0, 0, false};
        if (s >= n) return q;
        const int w = a.new_rows[s];
        q.len = max(a.kv_len[s], 0);
        const int held = pages_of(q.len, a.page_shift);
        if (w < 0) q.back = (int)min((int64_t)held, a.ldp);
        q.asks = w > 0;
        if (q.asks && (int64_t)q.len + w <= min(a.ldp << a.page_shift, (int64_t)0x7fffff00)) {
            q.want = w;
            q.need = pages_of(q.len + w, a.page_shift) - held;
        }
        return q;
    };
    int all_back = 0;
    if (n > 64 * PL_WAVES) {   // who is served depends on all pages that come back
        for (int s0 = 0; s0 < n; s0 += 64 * PL_WAVES) {
            int v[3] = {load(s0 + tid).back, 0, 0}, total[3];
            scan3(v, total, tid, sh);
            all_back = sat_add(all_back, total[0]);
        }
    }
    int asked[3] = {0, 0, 0}, given[3] = {0, 0, 0};   // before this round's sequences
    bool refused = false;
    for (int s0 = 0; s0 < n; s0 += 64 * PL_WAVES) {
        const int s = s0 + tid;
        const Seq q = load(s);
        int v[3] = {q.want, q.need, q.back}, total[3];
        scan3(v, total, tid, sh);
        if (n <= 64 * PL_WAVES) all_back = total[2];
        const int there = min(sat_add(old_free, all_back), a.max_free);
        const bool served = q.want > 0 && sat_add(asked[0], v[0]) <= a.max_rows &&
                            (q.need == 0 || sat_add(asked[1], v[1]) <= there);
        refused = refused || (q.asks && !served);
        int g[3] = {served ? q.want : 0, served ? q.need : 0, 0}, sum[3];
        scan3(g, sum, tid, sh);
        if (s < n) {
            row[s + 1] = given[0] + g[0];
            take[s + 1] = given[1] + g[1];
            back[s + 1] = sat_add(asked[2], v[2]);
            if (ONE) a.row_off[s + 1] = given[0] + g[0];
            a.kv_len_out[s] = q.back || a.new_rows[s] < 0 ? 0 : q.len + (served ? q.want : 0);
        }
#pragma unroll
        for (int i = 0; i < 3; ++i) {
            asked[i] = sat_add(asked[i], total[i]);
            given[i] += sum[i];
        }
    }
    const int there = min(sat_add(old_free, all_back), a.max_free);
    if (tid == 0) {
        row[0] = take[0] = back[0] = 0;
        if (ONE) a.row_off[0] = 0;
        else {
            a.head[0] = old_free;
            a.head[1] = there;
        }
        *a.n_free_out = there - given[1];
    }
    if (a.status) {
        if (__ballot(refused) && (tid & 63) == 0) __hip_atomic_fetch_or(a.status, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        if (tid == 0 && sat_add(old_free, all_back) > a.max_free)
            __hip_atomic_fetch_or(a.status, 2, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
    if (ONE) {
        __syncthreads();
        fill(a, Sums{row, take, back, given[0], given[1], old_free, there}, tid, 64 * PL_WAVES);
    }
}

__global__ __launch_bounds__(PL_FILL) void k_plan_fill(PlanArgs a) {
    const Sums S{a.row_off, a.take, a.back, a.row_off[a.n_seqs], a.take[a.n_seqs], a.head[0], a.head[1]};
    fill(a, S, blockIdx.x * PL_FILL + threadIdx.x, gridDim.x * PL_FILL);
}

}  // namespace

size_t plan_bytes(int32_t n_seqs) { return align_up((size_t)(2 * ((int64_t)n_seqs + 1) + 2) * 4, 256); }

hipError_t launch_kv_plan(PlanArgs a, void* ws, hipStream_t stream) {
    if (a.n_seqs <= PL_ONE_SEQS && a.max_rows <= PL_ONE_ROWS) {
        hipLaunchKernelGGL((k_plan<true>), dim3(1), dim3(64 * PL_WAVES), 0, stream, a);
        return hipGetLastError();
    }
    a.take = (int32_t*)ws;
    a.back = a.take + a.n_seqs + 1;
    a.head = a.back + a.n_seqs + 1;
    hipLaunchKernelGGL((k_plan<false>), dim3(1), dim3(64 * PL_WAVES), 0, stream, a);
    const int grid = (int)std::max<int64_t>(64, std::min<int64_t>(2048, ceil_div(a.max_rows, PL_FILL)));
    hipLaunchKernelGGL(k_plan_fill, dim3(grid), dim3(PL_FILL), 0, stream, a);
    return hipGetLastError();
}

}  // namespace lora
