// Attention of one new token per sequence over the paged cache on the CUDA
// cores: full-precision queries or a full-precision cache, where tensor-core
// products would round.
//
//   out = sum_i e^(l_i - M) v_i / (sum_i e^(l_i - M) + e^(sink - M)),  l_i = scale q.k_i
//
// Bound by HBM for few heads a key head (4 bytes of fp32 cache take G
// multiply-adds; at G = 8 the fp32 pipes are about half busy at the copy's
// rate).  The split over the blocks and the copies: paged_split.cuh, with
// tiles of 8 tokens.  In a warp four lanes share a token's dot products (16
// dims of theirs at a time, all NH heads, the query from shared memory), and
// for the values a lane owns the dims 2 lane + 64 j, j < d / 64, of all heads.
// All products are packed fp32 pairs.  The running maximum of a head is raised
// only when a tile exceeds it by more than 8 in log2 units.
//
// 16 sequences of up to 8,192 tokens in fp32, d = 128, 8 key heads (571 MB, a call
// from cold caches): 111 us with one query head a key head, 147 with four, 152 with
// eight; the bytes at the copy's rate take 88.  Two instances with eight heads spill
// registers: d = 256 with FP8 pages 24 bytes, d = 192 with fp32 pages 12.
#include "paged_split.cuh"

namespace csa {

namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kRescale = 8.0f;  // log2 units

template <int D, int FMT, int NH>
struct Dec {
    static constexpr bool FP8 = FMT == CSA_FP8_S64;
    static constexpr int kTok = 8, kStep = kNW * kTok;   // tokens of a warp's tile, of a step
    static constexpr int kRow = D * (FMT == CSA_F32 ? 4 : FMT == CSA_BF16 ? 2 : 1);
    static constexpr int kChunks = kRow / 16;
    static constexpr int kGroups = D / 64;
    static constexpr int kScaleBytes = FP8 ? kTok * kGroups * 4 : 0;
    static constexpr int kTile = 2 * (kTok * kRow + kScaleBytes);
    // Stages: two blocks of about 100 KB an SM for d <= 128, one above
    static constexpr int kBudget = (D <= 128 ? 96 : 144) * 1024;
    static constexpr int kStages = kBudget / (kNW * kTile) > 8 ? 8 : kBudget / (kNW * kTile);
    static constexpr int kRing = kNW * kStages * kTile;
    static constexpr int kJoinDims = D > 64 ? D / 2 : D;
    static constexpr int kSmem = kRing + (NH * D + kNW * NH * kJoinDims + kNW * kTok * NH) * 4;
    static constexpr int kCtas = 2 * (kSmem + 2048 + kAlignSmem) <= 228 * 1024 ? 2 : 1;  // per SM
};

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
__device__ __forceinline__ uint64_t bf16_pair(uint32_t w) {
    return pack2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}
__device__ __forceinline__ uint64_t e4m3_pair(uint32_t w) {  // two codes, exact
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(uint16_t(w)));
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
    return pack2(f.x, f.y);
}

// Dims [d, d + 4) / [d, d + 2) of row r of a tile at shared address `base` (without scales).
template <class C, int FMT>
__device__ __forceinline__ void load4(const uint8_t* base, int r, int d, uint64_t (&x)[2]) {
    if constexpr (FMT == CSA_F32) {
        const ulonglong2 y = *reinterpret_cast<const ulonglong2*>(base + place<C::kTok, C::kRow>(r, d / 4));
        x[0] = y.x;
        x[1] = y.y;
    } else if constexpr (FMT == CSA_BF16) {
        const uint2 y = *reinterpret_cast<const uint2*>(base + place<C::kTok, C::kRow>(r, d / 8) + d % 8 * 2);
        x[0] = bf16_pair(y.x);
        x[1] = bf16_pair(y.y);
    } else {
        const uint32_t y = *reinterpret_cast<const uint32_t*>(base + place<C::kTok, C::kRow>(r, d / 16) + d % 16);
        x[0] = e4m3_pair(y);
        x[1] = e4m3_pair(y >> 16);
    }
}
template <class C, int FMT>
__device__ __forceinline__ uint64_t load2(const uint8_t* base, int r, int d) {
    if constexpr (FMT == CSA_F32) return *reinterpret_cast<const uint64_t*>(base + place<C::kTok, C::kRow>(r, d / 4) + d % 4 * 4);
    else if constexpr (FMT == CSA_BF16) return bf16_pair(*reinterpret_cast<const uint32_t*>(base + place<C::kTok, C::kRow>(r, d / 8) + d % 8 * 2));
    else return e4m3_pair(*reinterpret_cast<const uint16_t*>(base + place<C::kTok, C::kRow>(r, d / 16) + d % 16));
}

}  // namespace

template <int D, int FMT, int NH>
__global__ void __launch_bounds__(32 * kNW, Dec<D, FMT, NH>::kCtas)
    paged_decode_simt_kernel(const PagedDecodeArgs a, int units, int hb, JoinRec* recs, float* slots) {
    using C = Dec<D, FMT, NH>;
    constexpr int kTok = C::kTok, JD = C::kJoinDims;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* const smem = aligned_smem(smem_raw);
    __shared__ Plan plan;
    __shared__ uint32_t vmask[kNW][8];
    __shared__ float2 jml[kNW][NH];
    float* const sq = reinterpret_cast<float*>(smem + C::kRing);  // [NH][D]; the scale is applied to the scores
    float* const jo = sq + NH * D;                                // [kNW][NH][JD]
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    float* const sp = jo + kNW * NH * JD + warp * kTok * NH;      // [kTok][NH]
    const int tok = lane >> 2, quarter = lane & 3;
    pdl_launch_dependents();
    make_plan<C::kStep>(a, units, &plan);
    if (!a.invariant && threadIdx.x == 0) recs[blockIdx.x].n = 0;
    if (plan.x0 >= plan.x1) return;
    const int G = a.H / a.HK;
    const float sl2 = a.scale * kLog2e;

    Cursor cur;
    cur.x = plan.x0; cur.x1 = plan.x1; cur.s = plan.s; cur.u = plan.u; cur.at = plan.at;
    cur.v = span_of<C::kStep>(a, cur.s);
    uint8_t* const ring = smem + warp * C::kStages * C::kTile;
    Copier<C, C::FP8> copier(a, units, hb, cur, smem_addr(ring), vmask[warp]);
#pragma unroll 1
    for (int i = 0; i < C::kStages - 1; ++i) copier.issue(i);

    int stage = 0;
#pragma unroll 1
    while (cur.x < cur.x1) {
        int b, e, dx;
        piece_of<C::kStep>(a, cur, b, e, dx);
        if (b >= e) {
            advance<C::kStep>(a, units, cur, dx);
            continue;
        }
        if (threadIdx.x == 0 && a.q_pos[cur.s] >= a.max_pages * a.page_size) flag_status(CSA_DEV_BAD_INDEX);
        const int hk = cur.u / hb, head0 = (cur.u % hb) * NH;  // within the group of G
        const int n_heads = min(NH, G - head0);
        const int64_t q_at = int64_t(cur.s) * a.q_ld + (int64_t(hk) * G + head0) * D;
        for (int i = threadIdx.x; i < NH * D; i += 32 * kNW) {
            float x = 0.f;
            if (i < n_heads * D)
                x = a.act_fmt == CSA_F32 ? ((const float*)a.q)[q_at + i] : bf16_bits_to_f32(((const uint16_t*)a.q)[q_at + i]);
            sq[i] = x;
        }
        __syncthreads();
        uint64_t o[NH][D / 64];
        float m[NH], l[NH];
#pragma unroll
        for (int h = 0; h < NH; ++h) {
            m[h] = -INFINITY;
            l[h] = 0.f;
#pragma unroll
            for (int j = 0; j < D / 64; ++j) o[h][j] = 0;
        }
#pragma unroll 1
        for (int st = b; st < e; ++st) {
            cp_wait<C::kStages - 2>();
            __syncwarp();
            copier.issue(stage == 0 ? C::kStages - 1 : stage - 1);  // into the stage consumed last
            const uint8_t* const kt = ring + stage * C::kTile;
            const uint8_t* const vt = kt + kTok * C::kRow;
            const float* const ksc = reinterpret_cast<const float*>(vt + kTok * C::kRow);
            const float* const vsc = ksc + C::kScaleBytes / 4;
            // ---- scores of this lane's token: the lane's dims first
            uint64_t s2[NH];
            float s[NH];
#pragma unroll
            for (int h = 0; h < NH; ++h) { s2[h] = 0; s[h] = 0.f; }
#pragma unroll
            for (int i = 0; i < D / 16; ++i) {
                const int d = 16 * i + 4 * quarter;
                uint64_t k[2];
                load4<C, FMT>(kt, tok, d, k);
#pragma unroll
                for (int h = 0; h < NH; ++h) {
                    const ulonglong2 q = *reinterpret_cast<const ulonglong2*>(sq + h * D + d);
                    s2[h] = fma2(q.y, k[1], fma2(q.x, k[0], s2[h]));
                }
                if (C::FP8 && (i & 3) == 3) {
                    const float x = ksc[tok * C::kGroups + i / 4];
#pragma unroll
                    for (int h = 0; h < NH; ++h) {
                        s[h] = fmaf(lo2(s2[h]) + hi2(s2[h]), x, s[h]);
                        s2[h] = 0;
                    }
                }
            }
            const bool seen = vmask[warp][stage] >> tok & 1;
            bool raise = false;
#pragma unroll
            for (int h = 0; h < NH; ++h) {
                if (!C::FP8) s[h] = lo2(s2[h]) + hi2(s2[h]);
                s[h] += __shfl_xor_sync(0xffffffffu, s[h], 1);
                s[h] += __shfl_xor_sync(0xffffffffu, s[h], 2);
                s[h] = seen ? s[h] * sl2 : -INFINITY;
                raise |= s[h] > m[h] + kRescale;
            }
            if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
                for (int h = 0; h < NH; ++h) {
                    float mx = s[h];
#pragma unroll
                    for (int z = 4; z < 32; z <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, z));
                    if (mx > m[h] + kRescale) {
                        const float al = m[h] == -INFINITY ? 0.f : ex2(m[h] - mx);
                        m[h] = mx;
                        l[h] *= al;
#pragma unroll
                        for (int j = 0; j < D / 64; ++j) o[h][j] = fma2(o[h][j], pack2(al, al), 0);
                    }
                }
            }
#pragma unroll
            for (int h = 0; h < NH; ++h) {
                s[h] = ex2(s[h] - (m[h] == -INFINITY ? 0.f : m[h]));
                l[h] += s[h];
                if (quarter == (h & 3)) sp[tok * NH + h] = s[h];
            }
            __syncwarp();
            // ---- values: all tokens, this lane's dims
#pragma unroll
            for (int t = 0; t < kTok; ++t) {
                float p[NH];
#pragma unroll
                for (int h = 0; h < NH; h += 2) {
                    const float2 y = *reinterpret_cast<const float2*>(sp + t * NH + h);
                    p[h] = y.x;
                    p[h + 1] = y.y;
                }
#pragma unroll
                for (int j = 0; j < D / 64; ++j) {
                    uint64_t v = load2<C, FMT>(vt, t, 64 * j + 2 * lane);
                    if constexpr (C::FP8) {
                        const float x = vsc[t * C::kGroups + j];
                        v = fma2(v, pack2(x, x), 0);
                    }
#pragma unroll
                    for (int h = 0; h < NH; ++h) o[h][j] = fma2(pack2(p[h], p[h]), v, o[h][j]);
                }
            }
            __syncwarp();
            stage = stage + 1 == C::kStages ? 0 : stage + 1;
        }

        // ---- the unit (or this block's part of it) is done: join the warps
#pragma unroll
        for (int h = 0; h < NH; ++h) {
#pragma unroll
            for (int z = 4; z < 32; z <<= 1) l[h] += __shfl_xor_sync(0xffffffffu, l[h], z);
            if (lane == 0) jml[warp][h] = make_float2(m[h], l[h]);
        }
        const bool whole = b == 0 && e == cur.v.steps;
        const int64_t slot = part_slot(a, plan, cur, units, weight<C::kStep>(a, cur.v), b == 0, whole, recs);
#pragma unroll
        for (int pass = 0; pass < D / JD; ++pass) {
            // the dims of this half: those of the lane's pairs that lie in it
#pragma unroll
            for (int j = 0; j < D / 64; ++j) {
                const int d = 64 * j + 2 * lane - pass * JD;
                if (d >= 0 && d < JD)
#pragma unroll
                    for (int h = 0; h < NH; ++h)
                        *reinterpret_cast<uint64_t*>(jo + (warp * NH + h) * JD + d) = o[h][j];
            }
            __syncthreads();
            for (int i = threadIdx.x; i < n_heads * JD; i += 32 * kNW) {
                const int head = i / JD, jd = i % JD, dim = pass * JD + jd, h = hk * G + head0 + head;
                float M = -INFINITY, L = 0.f, acc = 0.f;
#pragma unroll
                for (int w = 0; w < kNW; ++w) M = fmaxf(M, jml[w][head].x);
                const float sg = whole && a.sinks ? a.sinks[h] * kLog2e : -INFINITY;
                M = fmaxf(M, sg);
#pragma unroll
                for (int w = 0; w < kNW; ++w) {
                    const float2 v = jml[w][head];
                    const float wt = v.x == -INFINITY ? 0.f : ex2(v.x - M);
                    L += wt * v.y;  // (NaN logits leave m at -inf: they reach the result through l)
                    if (wt != 0.f) acc += wt * jo[(w * NH + head) * JD + jd];
                }
                if (whole) {
                    if (sg != -INFINITY) L += ex2(sg - M);
                    const float r = L == 0.f ? 0.f : acc / L;
                    const int64_t at = (int64_t(cur.s) * a.H + h) * D + dim;
                    if (a.act_fmt == CSA_F32) ((float*)a.out)[at] = r;
                    else ((__nv_bfloat16*)a.out)[at] = __float2bfloat16_rn(r);
                } else {
                    float* p = slots + slot * (NH * (D + 2));
                    if (dim == 0) { p[2 * head] = M; p[2 * head + 1] = L; }
                    p[2 * NH + head * D + dim] = acc;
                }
            }
            __syncthreads();
        }
        advance<C::kStep>(a, units, cur, dx);
    }
    cp_wait<0>();
}

// Heads of a unit: 8, or 2 where a key head has no more.
static int unit_heads(int H, int HK) { return H / HK <= 2 ? 2 : 8; }
constexpr int kStepSimt = 32;

size_t paged_decode_simt_workspace(int H, int HK, int D, int64_t batch, int64_t n_ctx, bool invariant) {
    return decode_layout(H, HK, D, batch, n_ctx, invariant, unit_heads(H, HK), kStepSimt).bytes;
}

template <int D, int FMT, int NH>
static cudaError_t launch_nh(PagedDecodeArgs a, void* ws, cudaStream_t s) {
    using C = Dec<D, FMT, NH>;
    static_assert(C::kStages >= 2 && C::kStages <= 8 && C::kStep == kStepSimt && C::kSmem <= 227 * 1024 - 2048 - kAlignSmem, "tile");
    const DecodeLayout w = decode_layout(a.H, a.HK, D, a.batch, a.max_pages * a.page_size, a.invariant, NH, C::kStep);
    const bool single = one_piece(a);
    if (single) a.invariant = 1;
    JoinRec* recs = single ? nullptr : (JoinRec*)ws;
    float* slots = (float*)((char*)ws + w.rec_bytes);
    const int hb = int(w.units / a.HK);
    cudaError_t e = ensure_smem(paged_decode_simt_kernel<D, FMT, NH>, C::kSmem + kAlignSmem);
    if (e != cudaSuccess) return e;
    paged_decode_simt_kernel<D, FMT, NH><<<C::kCtas * kNumSMs, 32 * kNW, C::kSmem + kAlignSmem, s>>>(a, int(w.units), hb, recs, slots);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    if (single) return cudaSuccess;
    return launch_paged_join(a, a.invariant ? w.recs : C::kCtas * kNumSMs, hb, NH, recs, slots, s);
}

template <int FMT>
static cudaError_t launch_fmt(const PagedDecodeArgs& a, void* ws, cudaStream_t s) {
    const bool few = unit_heads(a.H, a.HK) == 2;
    switch (a.D) {
        case 64: return few ? launch_nh<64, FMT, 2>(a, ws, s) : launch_nh<64, FMT, 8>(a, ws, s);
        case 128: return few ? launch_nh<128, FMT, 2>(a, ws, s) : launch_nh<128, FMT, 8>(a, ws, s);
        case 192: return few ? launch_nh<192, FMT, 2>(a, ws, s) : launch_nh<192, FMT, 8>(a, ws, s);
        default: return few ? launch_nh<256, FMT, 2>(a, ws, s) : launch_nh<256, FMT, 8>(a, ws, s);
    }
}

cudaError_t launch_paged_decode_simt(const PagedDecodeArgs& args, void* ws, cudaStream_t s) {
    PagedDecodeArgs a = args;
    set_page_division(&a);
    if (a.cache_fmt == CSA_F32) return launch_fmt<CSA_F32>(a, ws, s);
    if (a.cache_fmt == CSA_BF16) return launch_fmt<CSA_BF16>(a, ws, s);
    return launch_fmt<CSA_FP8_S64>(a, ws, s);
}

}  // namespace csa
