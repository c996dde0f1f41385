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
// launch and chains of dependent loads: the request's row count, the sums, the
// page of a row.  32 requests, one launch of one wave, 3.9 us; 776 with 37000
// rows behind eight prefixes, 5.2 us for the sums and 6.7 for the rows, which
// search what they need in LDS (in memory 9.4).
#include "kv_internal.hpp"

namespace lora {
namespace {

constexpr int PL_ONE_SEQS = 1024, PL_ONE_ROWS = 4096;   // up to these, one launch
constexpr int PL_FILL = 256;                            // threads of a filling workgroup
constexpr int PL_FILL_SEQS = 2048, PL_FILL_GROUPS = 512;   // up to these, what it searches lies in LDS

__device__ __forceinline__ int pages_of(int tokens, int shift) { return (int)(((int64_t)tokens + (1 << shift) - 1) >> shift); }

// sums of what requests ask for may pass 32 bits; past 2^31 - 1 they stay there
__device__ __forceinline__ int sat_add(int a, int b) {
    return (int)min((uint32_t)a + (uint32_t)b, 0x7fffffffu);
}
template <int N>
__device__ __forceinline__ void wave_scan(int (&v)[N], int lane, int lanes) {
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        if (d >= lanes) break;
        int o[N];
#pragma unroll
        for (int i = 0; i < N; ++i) o[i] = __shfl_up(v[i], d, 64);
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (lane >= d) v[i] = sat_add(v[i], o[i]);
    }
}
// Inclusive sums of N counts over the workgroup's NW waves; total: all of them.  sh: N * NW ints.
template <int NW, int N>
__device__ inline void scan(int (&v)[N], int (&total)[N], int tid, int* sh) {
    const int lane = tid & 63, wave = tid >> 6;
    wave_scan(v, lane, 64);
    if constexpr (NW == 1) {
#pragma unroll
        for (int i = 0; i < N; ++i) total[i] = __builtin_amdgcn_readlane(v[i], 63);
    } else {
        __syncthreads();
        if (lane == 63) {
#pragma unroll
            for (int i = 0; i < N; ++i) sh[i * NW + wave] = v[i];
        }
        __syncthreads();
        int w[N];   // every wave sums the waves' sums
#pragma unroll
        for (int i = 0; i < N; ++i) w[i] = sh[i * NW + (lane & (NW - 1))];
        wave_scan(w, lane & (NW - 1), NW);
#pragma unroll
        for (int i = 0; i < N; ++i) {
            total[i] = __builtin_amdgcn_readlane(w[i], NW - 1);
            const int before = __shfl(w[i], max(wave - 1, 0), 64);
            v[i] = sat_add(v[i], wave > 0 ? before : 0);
        }
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
    const int32_t* len;    // the sequence's tokens before the step, [n_seqs]
    const int32_t* group;  // group_off and prefix_len
    const int32_t* prefix;
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
            const int before = S.len[s], t = before + (r - S.row[s]);
            const int held = pages_of(before, a.page_shift), pg = t >> a.page_shift;
            if (a.adapter) adapter = a.adapter[s];
            pos = t;
            if (a.n_groups) {
                const int g = run_of(S.group, a.n_groups, s);
                if (g < a.n_groups && s >= S.group[0]) pos += max(S.prefix[g], 0);
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
    // (from the last thread on, which have the fewest rows)
    for (int k = threads - 1 - at; k < S.taken; k += threads) {
        const int s = min(run_of(S.take, a.n_seqs, k), a.n_seqs - 1);
        const int64_t pg = (int64_t)pages_of(S.len[s], a.page_shift) + (k - S.take[s]);
        const int page = stack_at(a, S, S.there - 1 - k);
        if (pg < a.ldp) a.pages[(int64_t)s * a.ldp + pg] = page;
    }
    for (int i = S.old_free + at; i < left; i += threads) a.free_pages[i] = stack_at(a, S, i);
}

// One workgroup of NW waves: the sums and everything of a sequence; ONE: the
// rest too.
template <bool ONE, int NW>
__global__ __launch_bounds__(64 * NW) void k_plan(PlanArgs a) {
    constexpr int T = 64 * NW, KEPT = NW == 16 ? PL_ONE_SEQS : T;
    __shared__ int sh[3 * NW];
    __shared__ int kept[ONE ? 4 : 1][ONE ? KEPT + 1 : 1];
    const int tid = threadIdx.x, n = a.n_seqs;
    int32_t* take = ONE ? kept[0] : a.take;
    int32_t* back = ONE ? kept[ONE ? 1 : 0] : a.back;
    int32_t* row = ONE ? kept[ONE ? 2 : 0] : a.row_off;
    int32_t* len = ONE ? kept[ONE ? 3 : 0] : a.len;
    const int old_free = min(max(*a.n_free, 0), a.max_free);

    // a sequence's length, the rows and pages it asks for, the pages it returns
    struct Seq {
        int len, want, need, back;
        bool asks, ends;
    };
    auto load = [&](int s) {
        Seq q{0, 0, 0, 0, false, false};
        if (s >= n) return q;
        const int w = a.new_rows[s];
        q.len = max(a.kv_len[s], 0);
        const int held = pages_of(q.len, a.page_shift);
        q.ends = w < 0;
        if (q.ends) q.back = (int)min((int64_t)held, a.ldp);
        q.asks = w > 0;
        if (q.asks && (int64_t)q.len + w <= min(a.ldp << a.page_shift, (int64_t)0x7fffff00)) {
            q.want = w;
            q.need = pages_of(q.len + w, a.page_shift) - held;
        }
        return q;
    };
    int all_back = 0;
    if (n > T) {   // who is served depends on all pages that come back
        for (int s0 = 0; s0 < n; s0 += T) {
            int v[1] = {load(s0 + tid).back}, total[1];
            scan<NW>(v, total, tid, sh);
            all_back = sat_add(all_back, total[0]);
        }
    }
    int asked[3] = {0, 0, 0}, given[2] = {0, 0};   // before this pass's sequences
    bool refused = false;
    for (int s0 = 0; s0 < n; s0 += T) {
        const int s = s0 + tid;
        const Seq q = load(s);
        int v[3] = {q.want, q.need, q.back}, total[3];
        scan<NW>(v, total, tid, sh);
        if (n <= T) all_back = total[2];
        const int there = min(sat_add(old_free, all_back), a.max_free);
        const bool served = q.want > 0 && sat_add(asked[0], v[0]) <= a.max_rows &&
                            (q.need == 0 || sat_add(asked[1], v[1]) <= there);
        refused = refused || (q.asks && !served);
        int g[2] = {served ? q.want : 0, served ? q.need : 0}, sum[2];
        scan<NW>(g, sum, tid, sh);
        if (s < n) {
            row[s + 1] = given[0] + g[0];
            take[s + 1] = given[1] + g[1];
            back[s + 1] = sat_add(asked[2], v[2]);
            len[s] = q.len;
            if (ONE) a.row_off[s + 1] = given[0] + g[0];
            a.kv_len_out[s] = q.ends ? 0 : q.len + (served ? q.want : 0);
        }
#pragma unroll
        for (int i = 0; i < 3; ++i) asked[i] = sat_add(asked[i], total[i]);
        given[0] += sum[0];
        given[1] += sum[1];
    }
    const int there = min(sat_add(old_free, all_back), a.max_free);
    if (tid == 0) {
        row[0] = take[0] = back[0] = 0;
        if (ONE) a.row_off[0] = 0;
        else {
            a.head[0] = old_free;
            a.head[1] = there;
            a.head[2] = given[0];
            a.head[3] = given[1];
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
        fill(a, Sums{row, take, back, len, a.group_off, a.prefix_len, given[0], given[1], old_free, there}, tid, T);
    }
}

__global__ __launch_bounds__(PL_FILL) void k_plan_fill(PlanArgs a) {
    __shared__ int32_t rows[PL_FILL_SEQS + 1], takes[PL_FILL_SEQS + 1], groups[PL_FILL_GROUPS + 1], prefixes[PL_FILL_GROUPS];
    Sums S{a.row_off, a.take, a.back, a.len, a.group_off, a.prefix_len, a.head[2], a.head[3], a.head[0], a.head[1]};
    if (a.n_seqs <= PL_FILL_SEQS) {
        for (int i = threadIdx.x; i <= a.n_seqs; i += PL_FILL) {
            rows[i] = a.row_off[i];
            takes[i] = a.take[i];
        }
        S.row = rows;
        S.take = takes;
    }
    if (a.n_groups > 0 && a.n_groups <= PL_FILL_GROUPS) {
        for (int i = threadIdx.x; i <= a.n_groups; i += PL_FILL) {
            groups[i] = a.group_off[i];
            if (i < a.n_groups) prefixes[i] = a.prefix_len[i];
        }
        S.group = groups;
        S.prefix = prefixes;
    }
    __syncthreads();
    fill(a, S, blockIdx.x * PL_FILL + threadIdx.x, gridDim.x * PL_FILL);
}

}  // namespace

size_t plan_bytes(int32_t n_seqs) { return align_up((size_t)(3 * ((int64_t)n_seqs + 1) + 4) * 4, 256); }

hipError_t launch_kv_plan(PlanArgs a, void* ws, hipStream_t stream) {
    if (a.n_seqs <= PL_ONE_SEQS && a.max_rows <= PL_ONE_ROWS) {
        // as many threads as sequences, and no more than four rows for each
        const int need = std::max(a.n_seqs, a.max_rows / 4);
        if (need <= 64) hipLaunchKernelGGL((k_plan<true, 1>), dim3(1), dim3(64), 0, stream, a);
        else if (need <= 256) hipLaunchKernelGGL((k_plan<true, 4>), dim3(1), dim3(256), 0, stream, a);
        else hipLaunchKernelGGL((k_plan<true, 16>), dim3(1), dim3(1024), 0, stream, a);
        return hipGetLastError();
    }
    a.take = (int32_t*)ws;
    a.back = a.take + a.n_seqs + 1;
    a.len = a.back + a.n_seqs + 1;
    a.head = a.len + a.n_seqs + 1;
    hipLaunchKernelGGL((k_plan<false, 16>), dim3(1), dim3(1024), 0, stream, a);
    const int grid = (int)std::max<int64_t>(64, std::min<int64_t>(2048, ceil_div(a.max_rows, PL_FILL) + 16));
    hipLaunchKernelGGL(k_plan_fill, dim3(grid), dim3(PL_FILL), 0, stream, a);
    return hipGetLastError();
}

}  // namespace lora
