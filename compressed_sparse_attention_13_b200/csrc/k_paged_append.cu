// Appending new tokens to the paged key / value cache, with the position
// rotation of queries and keys (and the cache's FP8 quantisation) on the way.
//
// Rotation of the pair (a, b) at position t with frequency f:
//   a' = a cos(t f) - b sin(t f),  b' = b cos(t f) + a sin(t f).
// The angle is formed in fp64 and reduced to a fraction of a turn there (at
// t = 10^6 an fp32 product would be off by 0.06 rad), the sine and cosine of
// the fraction are fp32.
//
// A block has a few consecutive tokens (two of many, one of few: then the
// blocks' number counts).  Their cosines and sines are computed once into shared
// memory and serve all H + HK rotated heads.  Bound by HBM: q, k and v are
// read once and q', k' and the cache rows written once; what has to be kept
// small for that is the instructions a byte.  A lane takes two chunks of eight
// elements of a head row, those that are rotated into each other, so that eight
// cosines and sines serve sixteen elements and nothing is exchanged; loads and
// stores are 16 bytes a lane for bf16.  d / 16 lanes (16 for d = 192, four of
// them idle) hold a row, and a row is read completely before it is written
// (the outputs may be the inputs).  The loads of kAhead rows a lane are under way
// while the tokens' sequences, pages and angles are found.  8,192 tokens of 48
// head rows of 128: 46 us; with one chunk a lane and its partner by shuffle 69 us.
#include "kernels.h"

namespace csa {

namespace {

constexpr int kAppendThreads = 128;

constexpr int kAhead = 2;   // rows of a lane loaded together
constexpr int kTokens = 2;  // of a block, at most

struct Chunk { float v[8]; };

// Two chunks as they lie in memory.
template <int ACT>
struct Raw {
    uint4 w[2][ACT == CSA_F32 ? 2 : 1];
};
template <int ACT>
__device__ __forceinline__ void load_raw(uint4 (&w)[ACT == CSA_F32 ? 2 : 1], const uint8_t* p) {
    const uint4* s = reinterpret_cast<const uint4*>(p);
    w[0] = s[0];
    if constexpr (ACT == CSA_F32) w[1] = s[1];
}
template <int ACT>
__device__ __forceinline__ Chunk values_of(const uint4 (&u)[ACT == CSA_F32 ? 2 : 1]) {
    Chunk c;
    if constexpr (ACT == CSA_F32) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            c.v[4 * h] = __uint_as_float(u[h].x); c.v[4 * h + 1] = __uint_as_float(u[h].y);
            c.v[4 * h + 2] = __uint_as_float(u[h].z); c.v[4 * h + 3] = __uint_as_float(u[h].w);
        }
    } else {
        const uint32_t w[4] = {u[0].x, u[0].y, u[0].z, u[0].w};
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

__device__ __forceinline__ float amax(const Chunk& x) {
    float top = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) top = fmaxf(top, fabsf(x.v[i]));
    return top;
}
// Eight E4M3 codes of x / s.
__device__ __forceinline__ uint2 codes_of(const Chunk& x, float s) {
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
    return make_uint2(w[0], w[1]);
}

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

// Position of the token `i` behind a sequence's first one at `first` >= 0: the last
// there is where the sum would overflow (no table reaches it either).
__device__ __forceinline__ int64_t place_of(int64_t first, int64_t i) {
    return first > INT64_MAX - i ? INT64_MAX : first + i;
}

// Position of packed row tok and its sequence; -1 for a row of no sequence or of
// one that is left out.  Called by a whole warp.
__device__ __forceinline__ int64_t position_of(const PagedAppendArgs& a, int64_t tok, int lane, int& s) {
    if (!a.cu_q) {
        s = int(tok);
        return max(a.pos0[tok], int64_t(-1));
    }
    if (a.n_seq > 32) {
        s = find_sequence(a.cu_q, a.n_seq, tok, lane);
        return s >= 0 && a.pos0[s] >= 0 ? place_of(a.pos0[s], tok - a.cu_q[s]) : -1;
    }
    // up to 32 sequences: all loads at once
    const int32_t from = lane < a.n_seq ? a.cu_q[lane] : INT32_MAX, end = a.cu_q[a.n_seq];
    const int64_t first = lane < a.n_seq ? a.pos0[lane] : -1;
    const unsigned le = __ballot_sync(0xffffffffu, lane < a.n_seq && from <= tok);
    s = le && tok < end ? 31 - __clz(int(le)) : -1;
    const int64_t p = __shfl_sync(0xffffffffu, first, max(s, 0));
    const int32_t at = __shfl_sync(0xffffffffu, from, max(s, 0));
    return s >= 0 && p >= 0 ? place_of(p, tok - at) : -1;
}

}  // namespace

template <int ACT, int FMT>
__global__ void __launch_bounds__(kAppendThreads, ACT == CSA_F32 ? 5 : 7)
    paged_append_kernel(const PagedAppendArgs a, int tokens) {
    constexpr int AB = ACT == CSA_F32 ? 4 : 2;  // bytes of an element
    __shared__ float4 turn[kTokens][64];        // (cos, sin) of two pairs
    __shared__ int64_t s_pos[kTokens], s_row[kTokens];
    const int64_t tok0 = int64_t(blockIdx.x) * tokens;
    const int n = int(min(int64_t(tokens), a.n_tokens - tok0));
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int d = a.D, R = a.rot_dim, half = R / 16;        // chunks in half of the rotated dims
    const int width = d == 64 ? 4 : d == 128 ? 8 : 16;      // lanes of a row
    const int rows = 32 / width, sub = lane / width, u = lane % width;
    const bool live = u < d / 16;
    // this lane's chunks: the two halves' for a rotated pair of chunks, else neighbours
    const bool turns = u < half;                            // its elements are rotated
    const int ca = turns && !a.rot_pairs ? u : 2 * u, cb = turns && !a.rot_pairs ? u + half : 2 * u + 1;
    const int hq = a.q ? a.H : 0, total = hq + 2 * a.HK;    // rows of a token: queries, keys, values
    const int stride = (kAppendThreads / 32) * rows, own = warp * rows + sub;
    const int rounds = (total + stride - 1) / stride;       // of a token
    // Round x of the block: row own + (x % rounds) * stride of token x / rounds.
    Raw<ACT> raw[kAhead];
    auto load_ahead = [&](int x) {
#pragma unroll
        for (int i = 0; i < kAhead; ++i, ++x) {
            const int t = x / rounds, r = own + (x - t * rounds) * stride;
            if (t >= n || !live || r >= total) continue;
            const bool isq = r < hq, isk = r < hq + a.HK;
            const void* src = isq ? a.q : isk ? a.k : a.v;
            const int64_t ld = isq ? a.q_ld : isk ? a.k_ld : a.v_ld;
            const int head = isq ? r : isk ? r - hq : r - hq - a.HK;
            const uint8_t* p = (const uint8_t*)src + ((tok0 + t) * ld + head * d) * AB;
            load_raw<ACT>(raw[i].w[0], p + 8 * AB * ca);
            load_raw<ACT>(raw[i].w[1], p + 8 * AB * cb);
        }
    };
    load_ahead(0);
    // Places of the tokens, a warp each; the page's entry is looked at after the barrier.
    int64_t pos = -1, id = -1, off = 0;
    if (warp < n) {
        int s;
        pos = position_of(a, tok0 + warp, lane, s);
        if (lane == 0) {
            s_pos[warp] = pos;
            if (pos >= 0) {
                const bool small = pos <= INT32_MAX;  // (64-bit division: another 100 instructions)
                const int64_t pg = small ? uint32_t(pos) / uint32_t(a.page_size) : pos / a.page_size;
                off = pos - pg * a.page_size;
                if (pg < a.max_pages) id = a.block_table[int64_t(s) * a.max_pages + pg];
            }
        }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < n * (R / 2); i += kAppendThreads) {
        const int t = i / (R / 2), j = i - t * (R / 2);
        const double angle = double(s_pos[t]) * a.inv_freq[j] * 0.15915494309189533577;  // in turns: 1 / (2 pi)
        const float f = float(angle - rint(angle));
        float sn, cs;
        sincospif(2.f * f, &sn, &cs);
        // a lane's eight pairs j = 8 u + i: two by two, the lanes next to one another
        float2* w = reinterpret_cast<float2*>(&turn[t][(j >> 1 & 3) * half + (j >> 3)]);
        w[j & 1] = make_float2(cs, sn);
    }
    if (warp < n && lane == 0) {
        const bool held = id >= 0 && id < a.n_pages;
        if (pos >= 0 && !held) flag_status(CSA_DEV_BAD_INDEX);
        s_row[warp] = held ? id * a.HK * a.page_size + off : -1;  // head 0's row; head h's is h * page_size on
    }
    __syncthreads();
    for (int x0 = 0; x0 < n * rounds; x0 += kAhead) {
        if (x0 > 0) load_ahead(x0);
#pragma unroll
        for (int at = 0; at < kAhead; ++at) {
            const int t = (x0 + at) / rounds, r = own + (x0 + at - t * rounds) * stride;
            if (t >= n) break;
            if (r - sub >= total || s_pos[t] < 0) continue;  // (for the whole warp)
            const bool on = live && r < total;
            const bool isq = r < hq, isk = !isq && r < hq + a.HK;
            Chunk x = values_of<ACT>(raw[at].w[0]), y = values_of<ACT>(raw[at].w[1]);
            if (turns && (isq || isk)) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float4 w = turn[t][i * half + u];
                    if (a.rot_pairs) {
                        Chunk& z = i < 2 ? x : y;
                        const int e = 4 * (i & 1);
                        const float p0 = z.v[e], p1 = z.v[e + 1], p2 = z.v[e + 2], p3 = z.v[e + 3];
                        z.v[e] = p0 * w.x - p1 * w.y;
                        z.v[e + 1] = p1 * w.x + p0 * w.y;
                        z.v[e + 2] = p2 * w.z - p3 * w.w;
                        z.v[e + 3] = p3 * w.z + p2 * w.w;
                    } else {
                        const float x0_ = x.v[2 * i], x1_ = x.v[2 * i + 1];
                        x.v[2 * i] = x0_ * w.x - y.v[2 * i] * w.y;
                        y.v[2 * i] = y.v[2 * i] * w.x + x0_ * w.y;
                        x.v[2 * i + 1] = x1_ * w.z - y.v[2 * i + 1] * w.w;
                        y.v[2 * i + 1] = y.v[2 * i + 1] * w.z + x1_ * w.w;
                    }
                }
            }
            const int64_t tok = tok0 + t;
            if (on && (isq || (isk && a.k_out))) {
                void* out = isq ? a.q_out : a.k_out;
                const int64_t o = isq ? (tok * a.H + r) * d : (tok * a.HK + (r - hq)) * d;
                store_chunk<ACT>(out, o + 8 * ca, x);
                store_chunk<ACT>(out, o + 8 * cb, y);
            }
            if (r - sub + rows <= hq) continue;  // (query rows only)
            const bool wr = on && !isq && s_row[t] >= 0;
            const int64_t row = s_row[t] + int64_t(isk ? r - hq : r - hq - a.HK) * a.page_size;
            void* cache = isk ? a.k_cache : a.v_cache;
            if constexpr (FMT == CSA_FP8_S64) {
                // the scales of the row's groups of 64: amax over 448, 1 for an all-zero group (or one whose scale
                // underflows); all lanes of the warp take part
                const float ta = on ? amax(x) : 0.f, tb = on ? amax(y) : 0.f;
                float sa = 1.f, sb = 1.f;
                for (int g = 0; g < d / 64; ++g) {
                    float top = fmaxf(ca >> 3 == g ? ta : 0.f, cb >> 3 == g ? tb : 0.f);
                    for (int o = 1; o < width; o <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
                    float sc = __fdiv_rn(top, 448.0f);
                    if (!(sc > 0.f)) sc = 1.0f;
                    if (ca >> 3 == g) sa = sc;
                    if (cb >> 3 == g) sb = sc;
                    if (wr && u == 0) (isk ? a.k_scales : a.v_scales)[row * (d / 64) + g] = sc;
                }
                if (wr) {
                    *reinterpret_cast<uint2*>((uint8_t*)cache + row * d + 8 * ca) = codes_of(x, sa);
                    *reinterpret_cast<uint2*>((uint8_t*)cache + row * d + 8 * cb) = codes_of(y, sb);
                }
            } else {
                if (wr) {
                    store_chunk<FMT>(cache, row * d + 8 * ca, x);
                    store_chunk<FMT>(cache, row * d + 8 * cb, y);
                }
            }
        }
    }
}

template <int ACT>
static cudaError_t launch_append_act(const PagedAppendArgs& a, cudaStream_t s) {
    // two tokens a block once that leaves every SM four blocks
    const int tokens = a.n_tokens >= 4 * kTokens * kNumSMs ? kTokens : 1;
    const unsigned grid = unsigned(ceil_div(a.n_tokens, tokens));
    if (a.cache_fmt == CSA_F32) paged_append_kernel<ACT, CSA_F32><<<grid, kAppendThreads, 0, s>>>(a, tokens);
    else if (a.cache_fmt == CSA_BF16) paged_append_kernel<ACT, CSA_BF16><<<grid, kAppendThreads, 0, s>>>(a, tokens);
    else paged_append_kernel<ACT, CSA_FP8_S64><<<grid, kAppendThreads, 0, s>>>(a, tokens);
    return cudaGetLastError();
}

cudaError_t launch_paged_append(const PagedAppendArgs& a, cudaStream_t s) {
    return a.act_fmt == CSA_F32 ? launch_append_act<CSA_F32>(a, s) : launch_append_act<CSA_BF16>(a, s);
}

}  // namespace csa
