// Causal attention over packed prompts on the CUDA cores: full precision, and
// bf16 with a scale that the tensor-core kernel does not take.
//
//   l_j = scale q.k_j ; out = sum e^(l_j - M) v_j / (sum e^(l_j - M) + e^(sink - M))
//
// Bound by the fp32 pipes: 2 d multiply-adds a visible (query, key) pair and
// head.  A block has 32 query tokens of one head.  Its groups of four warps (two
// up to d = 128, one above) take the keys' tiles of 64 in turn, each with a
// running maximum and sum per row, and are joined at the end: the blocks of a
// short batch do not fill the GPU, and the longest one's time is the call's
// (1,024 tokens, 8 heads of 64: 57 us; one group: 62 us, and 74 to 104 us at d = 128).  A thread has 4 x 4
// scores (rows 4 ty + i, keys tx + 16 j) and 4 rows x d / 16 dims of the output:
// four 16-byte loads of either operand feed 64 multiply-adds, in packed pairs.
// Rows of q and K are padded by 16 bytes so that the loads of a quarter warp hit
// all banks.  The next tile's K is copied under the product with V, its V under
// the scores (one buffer each).
#include "gqa_tiles.cuh"
#include "kernels.h"

namespace csa {

namespace {

constexpr int kThreads = 128;  // of a group
constexpr int kRows = 32, kKeys = 64;
constexpr float kLog2e = 1.4426950408889634f;

template <int D>
struct Tile {
    static constexpr int kGroups = D <= 128 ? 2 : 1;
    static constexpr int kLdK = D + 4;  // q and K
    static constexpr int kGroup = kKeys * kLdK + kKeys * D + kRows * (kKeys + 4);  // floats of a group
    static constexpr int kFloats = kRows * kLdK + kGroups * kGroup;
};

__device__ __forceinline__ float4 bf16x4(uint2 u) {
    return make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xFFFF0000u), __uint_as_float(u.y << 16),
                       __uint_as_float(u.y & 0xFFFF0000u));
}

// Rows [row0, row0 + live) of one head as fp32 into a tile of N rows (rows from
// `live` on keep what they held: nothing of them reaches a result).  fp32 rows
// are copied asynchronously, in a group of their own; bf16 ones are converted.
template <int ACT, int D, int LD, int N>
__device__ __forceinline__ void load_rows(float* dst, const void* src, int64_t row0, int64_t ld, int64_t col, int live,
                                          int tid) {
    constexpr int per = D / 4, rows = kThreads / per;  // threads of a row, rows at a time
    int r = tid / per;
    const int d = tid % per * 4;
    live = r < rows ? min(live, N) : 0;
    dst += r * LD + d;
    int64_t at = (row0 + r) * ld + col + d;
    if constexpr (ACT == CSA_F32) {
        const float* p = (const float*)src + at;
        uint32_t to = static_cast<uint32_t>(__cvta_generic_to_shared(dst));
#pragma unroll 8
        for (; r < live; r += rows, p += rows * ld, to += rows * LD * 4)
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(p) : "memory");
        asm volatile("cp.async.commit_group;" ::: "memory");
    } else {
        for (; r < live; r += rows, at += rows * ld, dst += rows * LD)
            *reinterpret_cast<float4*>(dst) = bf16x4(*reinterpret_cast<const uint2*>((const uint16_t*)src + at));
    }
}
__device__ __forceinline__ void group_sync(int g) {
    asm volatile("bar.sync %0, %1;" ::"r"(1 + g), "n"(kThreads) : "memory");
}
// The copies but the last N are there, those of every thread of the group.
template <int N>
__device__ __forceinline__ void landed(int g) {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
    group_sync(g);
}

// packed fp32 pairs: half the instructions of the products
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ __forceinline__ uint64_t pack2(float x, float y) {
    uint64_t v;
    asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(x), "f"(y));
    return v;
}
__device__ __forceinline__ float lo2(uint64_t v) { return __uint_as_float(uint32_t(v)); }
__device__ __forceinline__ float hi2(uint64_t v) { return __uint_as_float(uint32_t(v >> 32)); }

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

}  // namespace

template <int ACT, int D>
__global__ void __launch_bounds__(kThreads * Tile<D>::kGroups, D == 64 ? 2 : 1) prompt_simt_kernel(const PromptArgs a) {
    constexpr int LDK = Tile<D>::kLdK, LDP = kKeys + 4, E = D / 64;  // E groups of four output dims a thread
    extern __shared__ __align__(16) float sm[];
    float* const sq = sm;
    const int g = threadIdx.x / kThreads, tid = threadIdx.x % kThreads;
    float* const sk = sq + kRows * LDK + g * Tile<D>::kGroup;
    float* const sv = sk + kKeys * LDK;
    float* const sp = sv + kKeys * D;
    __shared__ SeqTile tile;
    const int tx = tid & 15, ty = tid >> 4, lane = threadIdx.x & 31;
    if (threadIdx.x < 32) {
        const SeqTile t = find_tile(a.cu_q, a.cu_k, a.n_seq, kRows, int(blockIdx.x / unsigned(a.H)), lane);
        if (lane == 0) tile = t;
    }
    __syncthreads();
    if (tile.s < 0) return;
    const int h = int(blockIdx.x % unsigned(a.H)), hk = h / (a.H / a.HK);
    const int64_t q0 = tile.q0, k0 = tile.k0;
    const int full_q = tile.len_q, len_k = tile.len_k;
    const int len_q = int(min(int64_t(full_q), a.n_q - q0));
    const int nk = int(max(min(k0 + len_k, a.n_k) - k0, int64_t(0)));
    const int off = len_k - full_q, tok0 = tile.tile * kRows;
    const int tok_last = min(tok0 + kRows, len_q) - 1;
    const int t_first = min(tok0 + off, nk - 1), t_last = min(tok_last + off, nk - 1);
    const int lo_first = first_seen(tok0 + off, a.W), lo_last = first_seen(tok_last + off, a.W);
    const float sl2 = a.scale * kLog2e;
    uint64_t o[4][E][2];
    float m[4], l[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        m[i] = -INFINITY;
        l[i] = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) o[i][e][0] = o[i][e][1] = 0;
    }
    auto load_k = [&](int kb) { load_rows<ACT, D, LDK, kKeys>(sk, a.k, k0 + kb, a.k_ld, int64_t(hk) * D, t_last + 1 - kb, tid); };
    auto load_v = [&](int kb) { load_rows<ACT, D, D, kKeys>(sv, a.v, k0 + kb, a.v_ld, int64_t(hk) * D, t_last + 1 - kb, tid); };
    const int step = Tile<D>::kGroups * kKeys, first = lo_first + g * kKeys;
    if (g == 0) load_rows<ACT, D, LDK, kRows>(sq, a.q, q0 + tok0, a.q_ld, int64_t(h) * D, len_q - tok0, tid);
    load_k(first);
    load_v(first);
    asm volatile("cp.async.wait_group 2;" ::: "memory");  // q, the first group's third newest
    __syncthreads();
    for (int kb = first; kb <= t_last; kb += step) {
        landed<1>(g);  // K
        uint64_t s2[4][4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) s2[i][j] = 0;
#pragma unroll 4
        for (int d = 0; d < D; d += 4) {
            ulonglong2 q[4], k[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) q[i] = *reinterpret_cast<const ulonglong2*>(sq + (4 * ty + i) * LDK + d);
#pragma unroll
            for (int j = 0; j < 4; ++j) k[j] = *reinterpret_cast<const ulonglong2*>(sk + (tx + 16 * j) * LDK + d);
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) s2[i][j] = fma2(q[i].y, k[j].y, fma2(q[i].x, k[j].x, s2[i][j]));
        }
        group_sync(g);
        load_k(kb + step);  // (no rows behind the last tile)
        // a cut tile: some row does not see all of it
        const bool cut = kb + kKeys - 1 > t_first || kb < lo_last;
        float s[4][4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) s[i][j] = (lo2(s2[i][j]) + hi2(s2[i][j])) * sl2;
        if (cut) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int at = tok0 + 4 * ty + i + off, t = min(at, nk - 1), lo = first_seen(at, a.W);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int key = kb + tx + 16 * j;
                    s[i][j] = key > t || key < lo ? -INFINITY : s[i][j];
                }
            }
        }
        float mx[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) mx[i] = max_nan(max_nan(s[i][0], s[i][1]), max_nan(s[i][2], s[i][3]));
#pragma unroll
        for (int x = 8; x > 0; x >>= 1)  // over the 16 threads of the rows
#pragma unroll
            for (int i = 0; i < 4; ++i) mx[i] = max_nan(mx[i], __shfl_xor_sync(0xffffffffu, mx[i], x));
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (!(mx[i] < INFINITY)) l[i] = __int_as_float(0x7FFFFFFF);  // NaN or +inf among the logits: the row is NaN
            if (mx[i] > m[i]) {
                const float al = m[i] == -INFINITY ? 0.f : ex2(m[i] - mx[i]);
                const uint64_t al2 = pack2(al, al);
                m[i] = mx[i];
                l[i] *= al;
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    o[i][e][0] = fma2(o[i][e][0], al2, 0);
                    o[i][e][1] = fma2(o[i][e][1], al2, 0);
                }
            }
            const float ref = m[i] == -INFINITY ? 0.f : m[i];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float p = ex2(s[i][j] - ref);
                l[i] += p;
                sp[(4 * ty + i) * LDP + tx + 16 * j] = p;
            }
        }
        landed<1>(g);  // V
        if (!cut) {
#pragma unroll 2
            for (int j = 0; j < kKeys; j += 4) {
                float4 p[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) p[i] = *reinterpret_cast<const float4*>(sp + (4 * ty + i) * LDP + j);
#pragma unroll
                for (int y = 0; y < 4; ++y) {
                    uint64_t w[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) w[i] = pack2((&p[i].x)[y], (&p[i].x)[y]);
#pragma unroll
                    for (int e = 0; e < E; ++e) {
                        const ulonglong2 v = *reinterpret_cast<const ulonglong2*>(sv + (j + y) * D + 64 * e + 4 * tx);
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            o[i][e][0] = fma2(w[i], v.x, o[i][e][0]);
                            o[i][e][1] = fma2(w[i], v.y, o[i][e][1]);
                        }
                    }
                }
            }
        } else {
            // a probability of 0 does not keep out what its value holds (infinities, NaN): left out instead
            for (int j = 0; j < kKeys; ++j) {
                float w[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) w[i] = sp[(4 * ty + i) * LDP + j];
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    const ulonglong2 v = *reinterpret_cast<const ulonglong2*>(sv + j * D + 64 * e + 4 * tx);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        if (w[i] != 0.f) {
                            o[i][e][0] = fma2(pack2(w[i], w[i]), v.x, o[i][e][0]);
                            o[i][e][1] = fma2(pack2(w[i], w[i]), v.y, o[i][e][1]);
                        }
                    }
                }
            }
        }
        group_sync(g);
        load_v(kb + step);
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int x = 8; x > 0; x >>= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], x);
    if constexpr (Tile<D>::kGroups == 2) {
        // The second group hands its rows over in its own K and V tiles.
        float* const jo = sq + kRows * LDK + Tile<D>::kGroup;
        float2* const jml = reinterpret_cast<float2*>(jo + kRows * D);
        if (g == 1) {
            group_sync(g);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int r = 4 * ty + i;
                if (tx == 0) jml[r] = make_float2(m[i], l[i]);
#pragma unroll
                for (int e = 0; e < E; ++e)
                    *reinterpret_cast<ulonglong2*>(jo + r * D + 64 * e + 4 * tx) = make_ulonglong2(o[i][e][0], o[i][e][1]);
            }
        }
        __syncthreads();
        if (g == 1) return;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = 4 * ty + i;
            const float2 y = jml[r];
            const float M = fmaxf(m[i], y.x);
            const float f0 = m[i] == -INFINITY ? 0.f : ex2(m[i] - M), f1 = y.x == -INFINITY ? 0.f : ex2(y.x - M);
            m[i] = M;
            l[i] = l[i] * f0 + y.y * f1;  // (a NaN sum stays NaN)
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const ulonglong2 v = *reinterpret_cast<const ulonglong2*>(jo + r * D + 64 * e + 4 * tx);
                o[i][e][0] = fma2(o[i][e][0], pack2(f0, f0), fma2(v.x, pack2(f1, f1), 0));
                o[i][e][1] = fma2(o[i][e][1], pack2(f0, f0), fma2(v.y, pack2(f1, f1), 0));
            }
        }
    }
    const float sg = a.sinks ? a.sinks[h] * kLog2e : -INFINITY;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float M = fmaxf(m[i], sg);
        float f = m[i] == -INFINITY ? 0.f : ex2(m[i] - M);
        float den = l[i] * f + (M == -INFINITY ? 0.f : ex2(sg - M));
        f = den == 0.f ? 0.f : f / den;
        const int tok = tok0 + 4 * ty + i;
        if (tok >= len_q) continue;
        const int64_t at = ((q0 + tok) * a.H + h) * int64_t(D) + 4 * tx;
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const float x[4] = {lo2(o[i][e][0]) * f, hi2(o[i][e][0]) * f, lo2(o[i][e][1]) * f, hi2(o[i][e][1]) * f};
            if constexpr (ACT == CSA_F32) {
                *reinterpret_cast<float4*>((float*)a.out + at + 64 * e) = make_float4(x[0], x[1], x[2], x[3]);
            } else {
                const __nv_bfloat162 y0 = __floats2bfloat162_rn(x[0], x[1]), y1 = __floats2bfloat162_rn(x[2], x[3]);
                *reinterpret_cast<uint2*>((uint16_t*)a.out + at + 64 * e) =
                    make_uint2(*reinterpret_cast<const uint32_t*>(&y0), *reinterpret_cast<const uint32_t*>(&y1));
            }
        }
    }
}

template <int ACT, int D>
static cudaError_t launch_d(const PromptArgs& a, cudaStream_t s) {
    const size_t smem = Tile<D>::kFloats * sizeof(float);
    const cudaError_t e = ensure_smem(prompt_simt_kernel<ACT, D>, smem);
    if (e != cudaSuccess) return e;
    // an upper bound of the tiles: the lengths are on the device
    const int64_t tiles = a.n_q / kRows + std::min<int64_t>(a.n_seq, a.n_q);
    if (tiles * a.H > INT32_MAX) return cudaErrorInvalidValue;
    prompt_simt_kernel<ACT, D><<<unsigned(tiles * a.H), kThreads * Tile<D>::kGroups, smem, s>>>(a);
    return cudaGetLastError();
}

template <int ACT>
static cudaError_t launch_act(const PromptArgs& a, cudaStream_t s) {
    switch (a.D) {
        case 64: return launch_d<ACT, 64>(a, s);
        case 128: return launch_d<ACT, 128>(a, s);
        case 192: return launch_d<ACT, 192>(a, s);
        default: return launch_d<ACT, 256>(a, s);
    }
}

cudaError_t launch_prompt_simt(const PromptArgs& a, cudaStream_t s) {
    return a.act_fmt == CSA_F32 ? launch_act<CSA_F32>(a, s) : launch_act<CSA_BF16>(a, s);
}

}  // namespace csa
