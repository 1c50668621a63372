// Grouped-head attention on the CUDA cores: one new token over the paged
// cache, and packed causal prompts.
//   l_i = scale * q.k_i ; out = sum e^(l_i - M) v_i / (sum e^(l_i - M) + e^(sink - M))
// One block of four warps per (query row, head); the warps take the visible
// keys in turn, each lane holding d / 32 dims, with a running maximum and sum
// per warp that are joined at the end.
#include "kernels.h"

namespace csa {

namespace {

constexpr int kWarps = 4;
constexpr float kLog2e = 1.4426950408889634f;

template <int ACT>
__device__ __forceinline__ float load_act(const void* p, int64_t off) {
    if constexpr (ACT == CSA_F32) return ((const float*)p)[off];
    else return bf16_bits_to_f32(((const uint16_t*)p)[off]);
}

// Join the warps' partials of one row and write it.
template <int ACT, int E>
__device__ __forceinline__ void join_row(float m, float l, const float (&o)[E], const float* sinks, int h,
                                         void* out, int64_t out_off, int lane, int warp) {
    __shared__ float sm[kWarps], sl[kWarps];
    __shared__ float so[kWarps][32 * E];
    if (lane == 0) { sm[warp] = m; sl[warp] = l; }
#pragma unroll
    for (int e = 0; e < E; ++e) so[warp][lane + 32 * e] = o[e];
    __syncthreads();
    float M = sinks ? sinks[h] * kLog2e : -INFINITY;
    const float sg = M;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) M = fmaxf(M, sm[w]);
    float den = sinks && M != -INFINITY ? exp2f(sg - M) : 0.f;
    float f[kWarps];
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        f[w] = sm[w] == -INFINITY ? 0.f : exp2f(sm[w] - M);
        den += f[w] * sl[w];
    }
    const float inv = den == 0.f ? 0.f : 1.f / den;
    for (int c = threadIdx.x; c < 32 * E; c += 32 * kWarps) {
        float x = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w)
            if (f[w] != 0.f) x += f[w] * so[w][c];
        x *= inv;
        if constexpr (ACT == CSA_F32) ((float*)out)[out_off + c] = x;
        else ((__nv_bfloat16*)out)[out_off + c] = __float2bfloat16_rn(x);
    }
}

// One key: its logit (log2 units) over the warp, then the running softmax.
template <int E, class KeyFn, class ValFn>
__device__ __forceinline__ void attend_key(const float (&q)[E], float (&o)[E], float& m, float& l, float sl2,
                                           KeyFn key, ValFn val) {
    float dot = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) dot += q[e] * key(e);
    dot = warp_sum(dot) * sl2;
    if (dot == -INFINITY) return;
    if (dot > m) {
        const float al = m == -INFINITY ? 0.f : exp2f(m - dot);
        l *= al;
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] = al == 0.f ? 0.f : o[e] * al;
        m = dot;
    }
    const float p = exp2f(dot - m);
    l += p;
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] += p * val(e);
}

}  // namespace

template <int ACT, int FMT, int E>
__global__ void __launch_bounds__(32 * kWarps) paged_decode_simt_kernel(const PagedDecodeArgs a) {
    constexpr int D = 32 * E;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int h = blockIdx.x % a.H;
    const int64_t b = blockIdx.x / a.H;
    const int hk = h / (a.H / a.HK);
    float q[E], o[E];
#pragma unroll
    for (int e = 0; e < E; ++e) {
        q[e] = load_act<ACT>(a.q, b * a.q_ld + int64_t(h) * D + lane + 32 * e);
        o[e] = 0.f;
    }
    const int64_t t = a.q_pos[b];
    int64_t hi = t + 1;
    if (hi > a.max_pages * a.page_size) {
        if (threadIdx.x == 0) flag_status(CSA_DEV_BAD_INDEX);
        hi = a.max_pages * a.page_size;
    }
    const int64_t lo = a.W > 0 ? max(t - a.W + 1, int64_t(0)) : 0;
    float m = -INFINITY, l = 0.f;
    const float sl2 = a.scale * kLog2e;
    for (int64_t i = lo + warp; i < hi; i += kWarps) {
        const int64_t id = a.block_table[b * a.max_pages + i / a.page_size];
        if (id < 0 || id >= a.n_pages) {
            if (lane == 0) flag_status(CSA_DEV_BAD_INDEX);
            continue;
        }
        const int64_t row = (id * a.HK + hk) * a.page_size + i % a.page_size;
        attend_key<E>(q, o, m, l, sl2,
                      [&](int e) { return load_elem<FMT>(a.k_cache, a.k_scales, row, D, lane + 32 * e); },
                      [&](int e) { return load_elem<FMT>(a.v_cache, a.v_scales, row, D, lane + 32 * e); });
    }
    join_row<ACT, E>(m, l, o, a.sinks, h, a.out, (b * a.H + h) * D, lane, warp);
}

template <int ACT, int E>
__global__ void __launch_bounds__(32 * kWarps) prompt_simt_kernel(const PromptArgs a) {
    constexpr int D = 32 * E;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int h = blockIdx.x % a.H;
    const int64_t i = blockIdx.x / a.H;
    const int hk = h / (a.H / a.HK);
    const int s = find_sequence(a.cu_q, a.n_seq, i, lane);
    if (s < 0) return;
    const int64_t k0 = max(int64_t(a.cu_k[s]), int64_t(0)), k1 = min(int64_t(a.cu_k[s + 1]), a.n_k);
    const int64_t t = (i - a.cu_q[s]) + (a.cu_k[s + 1] - a.cu_k[s]) - (a.cu_q[s + 1] - a.cu_q[s]);
    const int64_t lo = a.W > 0 ? max(t - a.W + 1, int64_t(0)) : 0;
    float q[E], o[E];
#pragma unroll
    for (int e = 0; e < E; ++e) {
        q[e] = load_act<ACT>(a.q, i * a.q_ld + int64_t(h) * D + lane + 32 * e);
        o[e] = 0.f;
    }
    float m = -INFINITY, l = 0.f;
    const float sl2 = a.scale * kLog2e;
    for (int64_t j = k0 + lo + warp; j <= k0 + t && j < k1; j += kWarps)
        attend_key<E>(q, o, m, l, sl2,
                      [&](int e) { return load_act<ACT>(a.k, j * a.k_ld + int64_t(hk) * D + lane + 32 * e); },
                      [&](int e) { return load_act<ACT>(a.v, j * a.v_ld + int64_t(hk) * D + lane + 32 * e); });
    join_row<ACT, E>(m, l, o, a.sinks, h, a.out, (i * a.H + h) * D, lane, warp);
}

template <int ACT, int FMT>
static cudaError_t launch_decode_fmt(const PagedDecodeArgs& a, cudaStream_t s) {
    const unsigned grid = unsigned(a.batch * a.H);
    switch (a.D) {
        case 64: paged_decode_simt_kernel<ACT, FMT, 2><<<grid, 32 * kWarps, 0, s>>>(a); break;
        case 128: paged_decode_simt_kernel<ACT, FMT, 4><<<grid, 32 * kWarps, 0, s>>>(a); break;
        case 192: paged_decode_simt_kernel<ACT, FMT, 6><<<grid, 32 * kWarps, 0, s>>>(a); break;
        default: paged_decode_simt_kernel<ACT, FMT, 8><<<grid, 32 * kWarps, 0, s>>>(a); break;
    }
    return cudaGetLastError();
}

template <int ACT>
static cudaError_t launch_decode_act(const PagedDecodeArgs& a, cudaStream_t s) {
    if (a.cache_fmt == CSA_F32) return launch_decode_fmt<ACT, CSA_F32>(a, s);
    if (a.cache_fmt == CSA_BF16) return launch_decode_fmt<ACT, CSA_BF16>(a, s);
    return launch_decode_fmt<ACT, CSA_FP8_S64>(a, s);
}

cudaError_t launch_paged_decode_simt(const PagedDecodeArgs& a, cudaStream_t s) {
    return a.act_fmt == CSA_F32 ? launch_decode_act<CSA_F32>(a, s) : launch_decode_act<CSA_BF16>(a, s);
}

template <int ACT>
static cudaError_t launch_prompt_act(const PromptArgs& a, cudaStream_t s) {
    const unsigned grid = unsigned(a.n_q * a.H);
    switch (a.D) {
        case 64: prompt_simt_kernel<ACT, 2><<<grid, 32 * kWarps, 0, s>>>(a); break;
        case 128: prompt_simt_kernel<ACT, 4><<<grid, 32 * kWarps, 0, s>>>(a); break;
        case 192: prompt_simt_kernel<ACT, 6><<<grid, 32 * kWarps, 0, s>>>(a); break;
        default: prompt_simt_kernel<ACT, 8><<<grid, 32 * kWarps, 0, s>>>(a); break;
    }
    return cudaGetLastError();
}

cudaError_t launch_prompt_simt(const PromptArgs& a, cudaStream_t s) {
    return a.act_fmt == CSA_F32 ? launch_prompt_act<CSA_F32>(a, s) : launch_prompt_act<CSA_BF16>(a, s);
}

}  // namespace csa
