// Appending a step's keys and values to a paged cache, with the rotary
// position rotation of queries and keys applied on the way:
//
//     (a, b) -> (a cos f - b sin f, a sin f + b cos f)   per rotated pair,
//     cos f, sin f = row `position` of the caller's tables
//
// Every element is read once and written once, in fp32 between, rounded once
// into the cache's type: 2 * rows * (heads of q, k and v) * head_dim elements
// plus 4 bytes per pair and row of the tables, 6 flop per pair.  Bytes bound
// for prompts (20304 rows of 64 heads on 8 of 128, bf16: 163 us, 5.1 TB/s, the
// rate of a plain copy); for one decode step the time is the chain of
// dependent loads (row's sequence -> its length -> its page -> the store): 32
// rows of 32 heads on 8, 4 us.
#include "kv_append.hpp"

namespace lora {
namespace {

template <typename TI, typename TO, int D>
__global__ __launch_bounds__(KA_WAVES * 64) void k_kv_append(AppendArgs a, int it) {
    append_row<TI, TO, D, false>(a, it, blockIdx.x, blockIdx.y);
}

template <typename TI, typename TO>
hipError_t launch_t(const AppendArgs& a, int32_t head_dim, hipStream_t stream) {
    const int chunks = (int)ceil_div((int64_t)(a.n_q_heads + 2 * a.C.n_kv_heads) * (head_dim / 16), 64);
    // a decode step spreads each row over as many waves as it has 64-item
    // runs; with many rows a wave keeps its row, so that the row's place is
    // looked up once
    const int it = (int)std::max<int64_t>(1, std::min<int64_t>(chunks, (int64_t)a.B.n_rows * chunks / 8192));
    dim3 grid((unsigned)ceil_div(a.B.n_rows, KA_WAVES), (unsigned)ceil_div(chunks, it));
    switch (head_dim) {
        case 64: hipLaunchKernelGGL((k_kv_append<TI, TO, 64>), grid, dim3(KA_WAVES * 64), 0, stream, a, it); break;
        case 128: hipLaunchKernelGGL((k_kv_append<TI, TO, 128>), grid, dim3(KA_WAVES * 64), 0, stream, a, it); break;
        default: hipLaunchKernelGGL((k_kv_append<TI, TO, 256>), grid, dim3(KA_WAVES * 64), 0, stream, a, it); break;
    }
    return hipGetLastError();
}

}  // namespace

hipError_t launch_kv_append(const AppendArgs& a, lora_dtype_t in, lora_dtype_t cache, int32_t head_dim,
                            hipStream_t stream) {
    if (in == LORA_BF16)
        return cache == LORA_BF16 ? launch_t<bf16, bf16>(a, head_dim, stream) : launch_t<bf16, float>(a, head_dim, stream);
    return cache == LORA_BF16 ? launch_t<float, bf16>(a, head_dim, stream) : launch_t<float, float>(a, head_dim, stream);
}

}  // namespace lora
