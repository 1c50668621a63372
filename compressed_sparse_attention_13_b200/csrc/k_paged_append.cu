// Appending new tokens to the paged key / value cache, with the position
// rotation of queries and keys (and the cache's FP8 quantisation) on the way.
//
// Rotation of the pair (a, b) at position t with frequency f:
//   a' = a cos(t f) - b sin(t f),  b' = b cos(t f) + a sin(t f).
// The angle is formed in fp64 and reduced to a fraction of a turn there (at
// t = 10^6 an fp32 product would be off by 0.06 rad), the sine and cosine of
// the fraction are fp32.
//
// One block per token.  Its cosines and sines are computed once into shared
// memory and serve all H + HK rotated heads.  Bound by HBM: q, k and v are
// read once and q', k' and the cache rows written once.  A warp takes 32 / C
// whole head rows at a time (C = d / 8 chunks of eight elements, one lane
// each; 24 of 32 lanes for d = 192), so that a pair's partner chunk comes
// from another lane by shuffle, loads and stores are 16 bytes a lane for
// bf16, an FP8 scale group of 64 channels is eight neighbouring lanes, and a
// row is read completely before it is written (the outputs may be the
// inputs).
#include "kernels.h"

namespace csa {

namespace {

constexpr int kAppendThreads = 256;

struct Chunk { float v[8]; };

template <int ACT>
__device__ __forceinline__ Chunk load_chunk(const void* p, int64_t off) {
    Chunk c;
    if constexpr (ACT == CSA_F32) {
        const float4* s = reinterpret_cast<const float4*>((const float*)p + off);
        const float4 x = s[0], y = s[1];
        c.v[0] = x.x; c.v[1] = x.y; c.v[2] = x.z; c.v[3] = x.w;
        c.v[4] = y.x; c.v[5] = y.y; c.v[6] = y.z; c.v[7] = y.w;
    } else {
        const uint4 x = *reinterpret_cast<const uint4*>((const uint16_t*)p + off);
        const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            c.v[2 * i] = __uint_as_float(w[i] << 16);
            c.v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        }
    }
    return c;
}

template <int FMT>
__device__ __forceinline__ void store_chunk(void* p, int64_t off, const Chunk& c) {
    if constexpr (FMT == CSA_F32) {
        float4* d = reinterpret_cast<float4*>((float*)p + off);
        d[0] = make_float4(c.v[0], c.v[1], c.v[2], c.v[3]);
        d[1] = make_float4(c.v[4], c.v[5], c.v[6], c.v[7]);
    } else {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 b = __floats2bfloat162_rn(c.v[2 * i], c.v[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t*>(&b);
        }
        *reinterpret_cast<uint4*>((uint16_t*)p + off) = make_uint4(w[0], w[1], w[2], w[3]);
    }
}

// A chunk of a cache row (FP8: the group's scale is the amax of eight lanes
// over 448; every lane of the warp calls this).  row: the row's index in the
// cache; wr: this lane's row is to be written.
template <int FMT>
__device__ __forceinline__ void store_cache(void* cache, float* scales, int64_t row, int d, int c, const Chunk& x,
                                            bool wr) {
    if constexpr (FMT == CSA_FP8_S64) {
        float top = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) top = fmaxf(top, fabsf(x.v[i]));
#pragma unroll
        for (int o = 1; o < 8; o <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        float s = __fdiv_rn(top, 448.0f);
        if (!(s > 0.f)) s = 1.0f;  // an all-zero group (or one whose scale underflows): codes of 0
        uint32_t w[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            uint16_t lo, hi;
            asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;"
                : "=h"(lo) : "f"(__fdiv_rn(x.v[4 * h + 1], s)), "f"(__fdiv_rn(x.v[4 * h], s)));
            asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;"
                : "=h"(hi) : "f"(__fdiv_rn(x.v[4 * h + 3], s)), "f"(__fdiv_rn(x.v[4 * h + 2], s)));
            w[h] = uint32_t(lo) | (uint32_t(hi) << 16);
        }
        if (wr) {
            *reinterpret_cast<uint2*>((uint8_t*)cache + row * d + 8 * c) = make_uint2(w[0], w[1]);
            if ((c & 7) == 0) scales[row * (d / 64) + (c >> 3)] = s;
        }
    } else {
        if (wr) store_chunk<FMT>(cache, row * d + 8 * c, x);
    }
}

}  // namespace

// The sequence of packed row i: the last s with cu[s] <= i, or -1 for a row
// behind the last sequence.  One warp, 32 probes a step.
__device__ int find_sequence(const int32_t* cu, int n_seq, int64_t i, int lane) {
    int lo = 0, n = n_seq;  // the answer is in [lo, lo + n)
    if (i >= cu[n_seq] || i < cu[0]) return -1;
    while (n > 1) {
        const int step = (n + 31) / 32;
        const int at = min(lane * step, n);  // probes lo, lo + step, ...
        const unsigned le = __ballot_sync(0xffffffffu, at < n && int64_t(cu[lo + at]) <= i);
        const int last = le ? 31 - __clz(int(le)) : 0;
        lo += last * step;
        n = min(step, n - last * step);
    }
    return lo;
}

template <int ACT, int FMT>
__global__ void __launch_bounds__(kAppendThreads)
    paged_append_kernel(const PagedAppendArgs a) {
    __shared__ float2 turn[128];
    __shared__ int s_seq;
    __shared__ int64_t s_pos, s_row;
    const int64_t tok = blockIdx.x;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (warp == 0) {
        const int s = a.cu_q ? find_sequence(a.cu_q, a.n_seq, tok, lane) : int(tok);
        if (lane == 0) {
            int64_t pos = -1, row = -1;
            if (s >= 0 && a.pos0[s] >= 0) {
                pos = a.pos0[s] + (a.cu_q ? tok - a.cu_q[s] : 0);
                const int64_t pg = pos / a.page_size;
                const int64_t id = pg < a.max_pages ? a.block_table[int64_t(s) * a.max_pages + pg] : -1;
                if (id >= 0 && id < a.n_pages)
                    row = (id * a.HK) * a.page_size + pos % a.page_size;  // head 0's row; head h's is h * page_size on
                else
                    flag_status(CSA_DEV_BAD_INDEX);
            }
            s_seq = s;
            s_pos = pos;
            s_row = row;
        }
    }
    __syncthreads();
    const int64_t pos = s_pos, row0 = s_row;
    if (pos < 0) return;
    const int R = a.rot_dim, d = a.D;
    for (int j = threadIdx.x; j < R / 2; j += kAppendThreads) {
        const double turns = double(pos) * a.inv_freq[j] * 0.15915494309189533577;  // 1 / (2 pi)
        const float f = float(turns - rint(turns));
        float sn, cs;
        sincospif(2.f * f, &sn, &cs);
        turn[j] = make_float2(cs, sn);
    }
    __syncthreads();
    const int C = d / 8, rows_per_warp = 32 / C;  // d = 192: 24 lanes, one row
    const int sub = lane / C, c = lane % C;
    const bool live = sub < rows_per_warp;
    const int hq = a.q ? a.H : 0, total = hq + 2 * a.HK;
    const int half = R / 16;  // chunks in half of the rotated dims
    const int stride = (kAppendThreads / 32) * rows_per_warp;
    for (int r0 = warp * rows_per_warp; r0 < total; r0 += stride) {
        const int r = r0 + sub;
        const bool on = live && r < total;
        const bool isq = r < hq, isk = !isq && r < hq + a.HK;
        Chunk x;
#pragma unroll
        for (int i = 0; i < 8; ++i) x.v[i] = 0.f;
        if (on) {
            const void* src = isq ? a.q : isk ? a.k : a.v;
            const int64_t ld = isq ? a.q_ld : isk ? a.k_ld : a.v_ld;
            const int head = isq ? r : isk ? r - hq : r - hq - a.HK;
            x = load_chunk<ACT>(src, tok * ld + int64_t(head) * d + 8 * c);
        }
        if (R > 0) {
            Chunk y = x;
            if (a.rot_pairs) {
                if (c < 2 * half) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float2 t = turn[4 * c + i];
                        y.v[2 * i] = x.v[2 * i] * t.x - x.v[2 * i + 1] * t.y;
                        y.v[2 * i + 1] = x.v[2 * i + 1] * t.x + x.v[2 * i] * t.y;
                    }
                }
            } else {
                const bool lower = c < half;
                const int from = c < 2 * half ? (lower ? lane + half : lane - half) : lane;
                Chunk o;
#pragma unroll
                for (int i = 0; i < 8; ++i) o.v[i] = __shfl_sync(0xffffffffu, x.v[i], from);
                if (c < 2 * half) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float2 t = turn[8 * (lower ? c : c - half) + i];
                        y.v[i] = lower ? x.v[i] * t.x - o.v[i] * t.y : x.v[i] * t.x + o.v[i] * t.y;
                    }
                }
            }
            if (isq || isk) x = y;
        }
        if (on && isq) store_chunk<ACT>(a.q_out, (tok * a.H + r) * int64_t(d) + 8 * c, x);
        if (on && isk && a.k_out) store_chunk<ACT>(a.k_out, (tok * a.HK + (r - hq)) * int64_t(d) + 8 * c, x);
        const int h = isk ? r - hq : r - hq - a.HK;
        const bool wr = on && !isq && row0 >= 0;
        // (a warp may hold query, key and value rows at once: all lanes take part in the group reductions)
        if (r0 + rows_per_warp > hq)
            store_cache<FMT>(isk ? a.k_cache : a.v_cache, isk ? a.k_scales : a.v_scales,
                             row0 + int64_t(h) * a.page_size, d, c, x, wr);
    }
}

template <int ACT>
static cudaError_t launch_append_act(const PagedAppendArgs& a, cudaStream_t s) {
    const unsigned grid = unsigned(a.n_tokens);
    if (a.cache_fmt == CSA_F32) paged_append_kernel<ACT, CSA_F32><<<grid, kAppendThreads, 0, s>>>(a);
    else if (a.cache_fmt == CSA_BF16) paged_append_kernel<ACT, CSA_BF16><<<grid, kAppendThreads, 0, s>>>(a);
    else paged_append_kernel<ACT, CSA_FP8_S64><<<grid, kAppendThreads, 0, s>>>(a);
    return cudaGetLastError();
}

cudaError_t launch_paged_append(const PagedAppendArgs& a, cudaStream_t s) {
    return a.act_fmt == CSA_F32 ? launch_append_act<CSA_F32>(a, s) : launch_append_act<CSA_BF16>(a, s);
}

}  // namespace csa
