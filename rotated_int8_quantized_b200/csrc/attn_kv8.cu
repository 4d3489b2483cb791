// attn_kv8.cu -- attention of a step's queries over the paged INT8 cache.
//
//   s_ij = scale * q_i . (ks_j kq_j)      keys' codes kq, one scale a block
//   o_i  = sum_j softmax_j(s_ij) (vs_j vq_j)
//
// The codes are never dequantised one by one.  A code is exact in FP16, so
// the products run on codes: a key block's scale multiplies 16 columns of
// q . kq at once, and a value block's scale joins the exponent,
//   p'_ij = exp2(s_ij log2(e) + log2(vs_j) - m_i),   o_i = sum_j p'_ij vq_j / l_i,   l_i = sum_j p'_ij / vs_j,
// with m_i a running maximum of the exponents.  Queries become FP16 with a
// power of two per row that brings the row's largest element to [2^14, 2^15):
// exact for every element above 2^-28 of the largest, off by 2^-39 of the
// largest below that (a BF16 product would be no closer).  p' is held as FP16
// scaled by 2^4: 11 bits where BF16 keeps 8, nothing above 2^-29 of the row's
// maximum lost (fewer bits below 2^-18 of it), and room for 2^11 more, so that
// the running maximum (and with it all that was summed under it) is moved only
// when it falls behind: by a score 2^11 above it where rows are streamed, by a
// step of 128 weights that sums to more than 2^15 (one score 2^11 above, or all
// of them 2^4) in prompts.  Sums, maxima and accumulators are FP32.
#include <cstdint>
#include <type_traits>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "common.cuh"
#include "kv8.h"
#include "umma_f16.cuh"

namespace convrot {

constexpr int kStreamWarps = 4;
constexpr int kStreamUnit = 16 * kStreamWarps;      // tokens a CTA takes at a time: a block for each warp
constexpr int kJoin = 64;                           // parts of a tile joined at a time
constexpr float kPBias = 4.f;                       // p' is held times 2^4
constexpr float kLazy = 11.f;                       // the running maximum moves once it is exceeded by 2^11
// Whether a sequence's rows (tokens times queries a key head) are streamed
// (attn_stream_kernel) or go through tensor-core tiles (attn_prompt_kernel):
// up to 64 rows always streamed, above 512 never.  Between,
//   a sequence by itself goes by what either would take as measured at 64 / 8
// heads of 128 and 40 / 40 of 64: the streaming kernel works off 230 (head dim
// 64: 380) units of 16 rows x 64 tokens a microsecond after 4 us, the other
// takes 10 us and 2 us a step of 128 tokens, eight at the most (several CTAs
// share a pass).  96 rows on 512 tokens: 12.3 us streamed, 16.8 tiled; 512 rows
// on 2048: 41.1 and 28.5.
//   of several sequences all should go one way, or the step takes both times:
// where sequences times key heads leave SMs idle and the rows average at most
// 128, up to 256 are streamed.  Eight sequences at 8 key heads, up to 192 rows
// on up to 1024 tokens: 34.3 us streamed, 48.4 partly tiled; up to 256 rows:
// 54.7 and 34.7; at 40 key heads of 64, up to 128 rows: 62.7 and 50.8.
constexpr int kFewRows = 64, kManyRows = 512;

__host__ __device__ __forceinline__ bool few_rows(int64_t rows, int64_t len, const AttnArgs &a) {
    if (rows <= kFewRows) return true;
    if (rows > kManyRows) return false;
    const int64_t heads = a.c.heads, batch = a.s.batch;
    if (batch > 1) return rows <= 256 && batch * heads <= 148 && a.s.tokens * (a.q_heads / heads) <= 128 * batch;
    const int64_t units = heads * ((rows + 15) / 16) * ((len + 63) / 64), steps = (len + 127) / 128;
    return 4000 + units * (a.c.dim == 128 ? 4400 : 2600) / 1000 < 10000 + 2000 * (steps < 8 ? steps : 8);
}

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
// Value scales below this count as this (a block of zeros has scale 0); the
// values it stands for are below 2^-93.
constexpr float kLeastScale = 7.888609052210118e-31f;   // 2^-100

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Four codes to FP16 pairs: code + 128 is the low byte of the FP16 number
// 1024 + (code + 128), from which 1152 is taken; every step is exact.
__device__ __forceinline__ void codes_to_half(uint32_t w, uint32_t &lo, uint32_t &hi) {
    const uint32_t u = w ^ 0x80808080u;
    const uint32_t a = __byte_perm(u, 0x64646464u, 0x4140), b = __byte_perm(u, 0x64646464u, 0x4342);
    const __half2 k = __half2half2(__ushort_as_half((unsigned short)0x6480));
    const __half2 x = __hsub2(*reinterpret_cast<const __half2 *>(&a), k), y = __hsub2(*reinterpret_cast<const __half2 *>(&b), k);
    lo = *reinterpret_cast<const uint32_t *>(&x);
    hi = *reinterpret_cast<const uint32_t *>(&y);
}

__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}

__device__ __forceinline__ uint32_t movmatrix_trans(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

// d[16 x 8] += a[16 x 16] b[16 x 8], FP16 in, FP32 sums.
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint4 ld_stream16(const void *p) {
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}
// 32 bytes a lane, so that four lanes read a whole row of 128.
__device__ __forceinline__ void ld_stream32(const void *p, uint32_t (&v)[8]) {
    asm volatile("ld.global.nc.L1::no_allocate.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7])
                 : "l"(p));
}
__device__ __forceinline__ uint2 ld_stream8(const void *p) {
    uint2 v;
    asm volatile("ld.global.nc.L1::no_allocate.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p));
    return v;
}

// An atomic add that orders this thread's (and, behind a barrier, its CTA's)
// accesses on both sides of it.
__device__ __forceinline__ int add_acq_rel(int *p, int v) {
    int old;
    asm volatile("atom.acq_rel.gpu.global.add.s32 %0, [%1], %2;" : "=r"(old) : "l"(p), "r"(v) : "memory");
    return old;
}

// a / b for a >= 0 and b > 0, in 32 bits where they do (a 64-bit quotient is a
// quarter of a microsecond, and several stand between a small call and its end).
__device__ __forceinline__ long long quotient(long long a, int b) {
    return (a >> 32) == 0 ? (long long)((uint32_t)a / (uint32_t)b) : a / b;
}

// Rows, cached tokens and first row of a sequence, held to the step's bounds
// whatever the device arrays say.
struct SeqInfo {
    int64_t t0;
    int n, len;
    bool bad;
};

__device__ __forceinline__ SeqInfo seq_info(const KvSeqs &s, int b) {
    SeqInfo q;
    int64_t t0 = b, t1 = b + 1;
    if (s.cu) {
        t0 = __ldg(s.cu + b);
        t1 = __ldg(s.cu + b + 1);
    }
    const int64_t len = __ldg(s.kv_len + b), cap = (int64_t)s.max_pages << s.page_shift;
    q.bad = t0 < 0 || (b == 0 && t0 != 0) || t1 < t0 || t1 > s.tokens || len < 0 || len > cap;
    t0 = min(max(t0, (int64_t)0), s.tokens);
    t1 = min(max(t1, t0), s.tokens);
    q.t0 = t0;
    q.n = (int)(t1 - t0);
    q.len = (int)min(max(len, (int64_t)0), cap);
    return q;
}

// ------------------------------------------------------------ few rows a sequence
//
// The queries of one sequence that share a key head are the rows of a tile:
// row r is token r / group, head kv_head * group + r % group.  A CTA of four
// warps streams the cache through such tiles of 8 NT rows; warp w takes block
// w of every four blocks of 16 tokens, from global memory straight into the
// operand layout of mma.m16n8k16 (16 tokens x 16 dims of K as the first
// operand, 16 dims x 16 tokens of V; the sums run over dims, then tokens, in an
// order of our choosing, so a lane simply takes a quarter of a K row or an
// eighth of a V row and queries and outputs follow the same order).  The next
// block's K is in flight from the moment this one's is used up, its V likewise.
//
// Bound by memory, so the cache's blocks are dealt out evenly: all units (64
// tokens of a tile) of the step in one list, an equal range for each of the
// resident CTAs, whatever the lengths.  A tile that a range cuts leaves its
// parts (FP32 sums, maximum) in the workspace, and the CTA that finds itself
// last at the tile's counter joins them, in the order of the ranges, and sets
// the counter back to zero.
//
// Measured at 64 / 8 heads of 128: 64 sequences of 2048 .. 8192 tokens (675 MB)
// 134 .. 140 us, 3 of up to 131071 (694 MB) 136 .. 142 us, 75 .. 78 % of the copy
// rate; with the products left out the loads alone take 124 us, so about a
// third of the rest is conversion (some 300 instructions a block and warp) and
// the rest the start (5 us to the first block) and the join (4 us).  Four CTAs
// of 128 registers an SM beat three with the next block in registers (147 us)
// and five with spills (157 us); bulk prefetch into L2 five blocks ahead cost 9
// us, 16- or 32-byte loads of K made no difference.
template <int D, int NT>
struct StreamSmem {
    float o[kStreamWarps][8 * NT][D + 4];            // later the maxima and sums of a tile's parts, [kJoin][8 NT][2]
    float m[kStreamWarps][8 * NT], l[kStreamWarps][8 * NT];
    long long first[kStreamWarps];
    int seq, last;
    long long seq_unit;
};

// CTAs of the persistent grid on an SM; also what the registers are held to.
constexpr int kMostStreamCtas = 4;
__host__ __device__ constexpr int stream_ctas(int nt) { return nt == 1 ? kMostStreamCtas : 2; }

// Tile counters in front of the workspace, as many as the larger grid needs
// whichever is launched: calls of other shapes on the same workspace leave
// sums behind them, never in them.
__host__ __device__ constexpr int stream_counters(int grid, int nt) {
    return (grid / stream_ctas(nt) * kMostStreamCtas + 63) / 64 * 64;
}

// All: every sequence is this kernel's (the rule between the two kernels would
// cost a tile of 8 rows registers that it does not have: 96 bytes of spills, 6 us of 134).
template <int D, int NT, bool All>
__global__ void __launch_bounds__(kStreamWarps * 32, stream_ctas(NT)) attn_stream_kernel(const __grid_constant__ AttnArgs a) {
    constexpr int R = 8 * NT, T = kStreamWarps * 32;
    constexpr int VW = D / 32;                       // words of a V row a lane holds
    constexpr int MT = D / 16;                       // words of a K row a lane holds; 16-dim pieces of a row
    extern __shared__ __align__(16) uint8_t smem_raw[];
    StreamSmem<D, NT> &sm = *reinterpret_cast<StreamSmem<D, NT> *>(smem_raw);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t4 = lane & 3;
    const int H = a.c.heads, group = a.q_heads / H;
    const KvSeqs &S = a.s;

    // units of every sequence, summed; thread i holds sequences [i per, i per + per)
    const int per = (S.batch + T - 1) / T;
    auto seq_units = [&](const SeqInfo &q) {
        if (!All && !few_rows((int64_t)q.n * group, q.len, a)) return 0ll;       // attn_prompt_kernel's
        const int tiles = (q.n * group + R - 1) / R;
        const int units = q.len > 0 ? (q.len + kStreamUnit - 1) / kStreamUnit : 1;   // empty rows are written too
        return (long long)tiles * units * H;
    };
    long long mine = 0;
    for (int i = 0; i < per; ++i) {
        const int b = tid * per + i;
        if (b >= S.batch) break;
        const SeqInfo q = seq_info(S, b);
        if (q.bad && blockIdx.x == 0) report_invalid();
        mine += seq_units(q);
    }
    long long scan = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long v = __shfl_up_sync(0xffffffffu, scan, o);
        if (lane >= o) scan += v;
    }
    if (lane == 31) sm.first[warp] = scan;
    __syncthreads();
    long long before = 0, total = 0;
#pragma unroll
    for (int w = 0; w < kStreamWarps; ++w) {
        const long long v = sm.first[w];
        if (w < warp) before += v;
        total += v;
    }
    before += scan - mine;
    // range c holds `share` units, the first `more` ranges one more
    const int G = (int)min((long long)gridDim.x, total), c = blockIdx.x;
    if (c >= G) {
        pdl_wait();
        return;
    }
    const long long share = quotient(total, G);
    const int more = (int)(total - share * G);
    auto range_start = [&](int i) { return share * i + min(i, more); };
    auto range_of = [&](long long unit) {
        const long long head = (share + 1) * more;               // units of the longer ranges (share < 2^31: a range is below 2^37 tokens)
        return unit < head ? (int)quotient(unit, (int)share + 1) : more + (int)quotient(unit - head, (int)share);
    };
    const long long u0 = range_start(c), u1 = range_start(c + 1);
    long long u = u0;
    if (before <= u && u < before + mine) {
        long long x = before;
        int b = tid * per;
        for (; b + 1 < S.batch; ++b) {
            const long long n = seq_units(seq_info(S, b));
            if (u < x + n) break;
            x += n;
        }
        sm.seq = b;
        sm.seq_unit = x;
    }
    __syncthreads();
    int b = sm.seq;
    long long seq_unit = sm.seq_unit;
    SeqInfo q = seq_info(S, b);

    int *const counters = static_cast<int *>(a.ws);
    float *const parts = reinterpret_cast<float *>(counters + stream_counters((int)gridDim.x, NT));
    constexpr int kPart = R * (D + 2);

    while (u < u1) {
        // the tile of unit u
        long long n_units;
        while (u >= seq_unit + (n_units = seq_units(q)) && b + 1 < S.batch) {
            seq_unit += n_units;
            ++b;
            q = seq_info(S, b);
        }
        const int units = q.len > 0 ? (q.len + kStreamUnit - 1) / kStreamUnit : 1;
        const int rows = q.n * group, tiles = (rows + R - 1) / R;
        if (tiles == 0) break;                       // only if the lengths changed under the kernel
        const int tile_index = (int)quotient(u - seq_unit, units);           // < tiles * H
        const long long tile_unit = seq_unit + (long long)tile_index * units;
        const int h = tile_index / tiles, rt = tile_index - h * tiles;
        const int unit0 = (int)(u - tile_unit);
        const int unit1 = (int)min((long long)units, u1 - tile_unit);

        // what the tile's last and first row see
        auto sees = [&](int tok) { return a.causal ? min(max(q.len - q.n + tok + 1, 0), q.len) : q.len; };
        const int most = sees((min(rt * R + R, rows) - 1) / group), least = sees(rt * R / group);

        // this warp's blocks: warp, warp + 4, .. of [4 unit0, 4 unit1), as far as a row sees
        const int blk1 = min(unit1 * kStreamWarps, (most + 15) >> 4);
        const int32_t *pages = S.table + (int64_t)b * S.max_pages;
        const int bshift = S.page_shift - 4, bmask = (1 << bshift) - 1;
        uint32_t kr[2][MT];
        uint32_t vr[4][VW];
        // Where this warp's blocks lie (in blocks of the cache; -1: no such page, its tokens are not seen) and their
        // scales: a lane looks after one of the next 32.
        int sc = -1;
        float ks = 0.f, vs = 0.f, lv = 0.f, iv = 0.f;
        auto look_up = [&](int first) {
            const int blk = first + lane * kStreamWarps;
            sc = -1;
            if (blk >= blk1) return;
            const int page = __ldg(pages + (blk >> bshift));
            if (page < 0 || page >= S.pages) {
                report_invalid();
                return;
            }
            sc = ((page * H + h) << bshift) + (blk & bmask);         // < 2^31 (checked by the host)
            ks = __ldg(a.c.ks + sc);
            vs = __ldg(a.c.vs + sc);
        };
        // apart, so that nothing waits for them before the codes are asked for.  The quick logarithm (two units in its last
        // place) moves a weight by 2^-20 of itself at usual scales and 2^-16 at the ends of the range, the quick quotient by
        // 2^-22; a weight is rounded to 2^-12.
        auto scales = [&] {
            const float ve = fmaxf(vs, kLeastScale);
            lv = __log2f(ve);
            iv = __fdividef(1.f, ve);
        };
        const int8_t *const k0 = a.c.k + g * D + t4 * (D / 4), *const v0 = a.c.v + 2 * t4 * D + g * (D / 8);
        auto load_k = [&](int sc) {
            if (sc < 0) return;
            const int8_t *kp = k0 + (int64_t)sc * (16 * D);
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                if constexpr (MT == 8) {
                    ld_stream32(kp + 8 * r * D, kr[r]);
                } else {
                    const uint4 x = ld_stream16(kp + 8 * r * D);
                    kr[r][0] = x.x, kr[r][1] = x.y, kr[r][2] = x.z, kr[r][3] = x.w;
                }
            }
        };
        auto load_v = [&](int sc) {
            if (sc < 0) return;
            const int8_t *vp = v0 + (int64_t)sc * (16 * D);
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int8_t *p = vp + ((r & 1) + 8 * (r >> 1)) * D;
                if constexpr (VW == 4) {
                    const uint4 x = ld_stream16(p);
                    vr[r][0] = x.x, vr[r][1] = x.y, vr[r][2] = x.z, vr[r][3] = x.w;
                } else {
                    const uint2 x = ld_stream8(p);
                    vr[r][0] = x.x, vr[r][1] = x.y;
                }
            }
        };
        // the first block is on its way before the queries are looked at
        int blk = unit0 * kStreamWarps + warp;
        look_up(blk);
        int now = __shfl_sync(0xffffffffu, sc, 0);
        load_k(now);
        load_v(now);
        scales();

        // queries: row 8 nt + g, dims (D / 4) t4 .. + D / 4 - 1
        uint32_t qf[NT][MT][2];
        float f[NT][2];                              // rows 8 nt + 2 t4, + 1: log2(e) * softmax scale * row scale
        int vis[NT][2];                              // tokens they see
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const int row = rt * R + 8 * nt + g;
            const bool in = row < rows;
            const int tok = row / group, head = h * group + row - tok * group;
            const uint16_t *src = a.q.p + (q.t0 + tok) * a.q.ts + (int64_t)head * a.q.hs + t4 * (D / 4);
            uint32_t w[D / 8];
            float top = 0.f;
#pragma unroll
            for (int i = 0; i < D / 32; ++i) {
                const uint4 x = in ? __ldg(reinterpret_cast<const uint4 *>(src) + i) : make_uint4(0u, 0u, 0u, 0u);
                w[4 * i] = x.x, w[4 * i + 1] = x.y, w[4 * i + 2] = x.z, w[4 * i + 3] = x.w;
            }
#pragma unroll
            for (int i = 0; i < D / 8; ++i)
                top = fmaxf(top, fmaxf(fabsf(__uint_as_float(w[i] << 16)), fabsf(__uint_as_float(w[i] & 0xFFFF0000u))));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
            // 2^(14 - e), e the exponent of the row's largest element (held to what FP32 can scale by)
            int e = (int)(__float_as_uint(top) >> 23) - 127;
            const bool finite = e <= 127;                // a row with an infinity becomes NaN, whatever it meets
            e = e < -100 ? -100 : e;
            const float up = finite ? __int_as_float((127 + 14 - e) << 23) : __int_as_float(0x7FC00000);
#pragma unroll
            for (int i = 0; i < MT; ++i)
#pragma unroll
                for (int k = 0; k < 2; ++k)
                    qf[nt][i][k] = pack_half2(__uint_as_float(w[2 * i + k] << 16) * up, __uint_as_float(w[2 * i + k] & 0xFFFF0000u) * up);
            const float down = a.scale * kLog2e * __int_as_float((127 - 14 + e) << 23);
            const int v = in ? sees(tok) : most;                 // a row that is none only has to stay out of the way
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                f[nt][k] = __shfl_sync(0xffffffffu, down, (2 * t4 + k) * 4);
                vis[nt][k] = __shfl_sync(0xffffffffu, v, (2 * t4 + k) * 4);
            }
        }

        float o[NT][MT][4], m[NT][2], l[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int i = 0; i < MT; ++i)
#pragma unroll
                for (int k = 0; k < 4; ++k) o[nt][i][k] = 0.f;
            m[nt][0] = m[nt][1] = -INFINITY;
            l[nt][0] = l[nt][1] = 0.f;
        }

        {
            for (int at = 0; blk < blk1; blk += kStreamWarps) {
                const bool seen = now >= 0;
                const float kscale = __shfl_sync(0xffffffffu, ks, at), vlog = __shfl_sync(0xffffffffu, lv, at),
                            vinv = __shfl_sync(0xffffffffu, iv, at);
                if (++at == 32) {
                    at = 0;
                    look_up(blk + kStreamWarps);
                    scales();
                }
                const int next = __shfl_sync(0xffffffffu, sc, at);
                float s[NT][4];
                if (seen) {
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) s[nt][0] = s[nt][1] = s[nt][2] = s[nt][3] = 0.f;
#pragma unroll
                    for (int i = 0; i < MT; ++i) {
                        uint32_t a0, a1, a2, a3;
                        codes_to_half(kr[0][i], a0, a2);
                        codes_to_half(kr[1][i], a1, a3);
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) mma_f16(s[nt], a0, a1, a2, a3, qf[nt][i][0], qf[nt][i][1]);
                    }
                }
                load_k(next);
                if (seen) {
                    const int tok = blk * 16 + g;
                    const bool whole = blk * 16 + 16 <= least;
                    bool over = false;
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            s[nt][k] = fmaf(s[nt][k], f[nt][k & 1] * kscale, vlog);
                            if (!whole && tok + 8 * (k >> 1) >= vis[nt][k & 1]) s[nt][k] = -INFINITY;
                            over |= s[nt][k] > m[nt][k & 1] + kLazy;
                        }
                    if (__any_sync(0xffffffffu, over)) {
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                            for (int k = 0; k < 2; ++k) {
                                float x = fmaxf(s[nt][k], s[nt][k + 2]);
                                x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
                                x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
                                x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
                                // by this row alone: what a row gets does not depend on its neighbours
                                const float mn = x > m[nt][k] + kLazy ? x : m[nt][k];
                                const float al = m[nt][k] == mn ? 1.f : ex2(m[nt][k] - mn);
                                m[nt][k] = mn;
                                l[nt][k] *= al;
#pragma unroll
                                for (int i = 0; i < MT; ++i) o[nt][i][k] *= al, o[nt][i][k + 2] *= al;
                            }
                    }
                    uint32_t p0[NT], p1[NT];
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        float p[4];
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const float mm = m[nt][k & 1] == -INFINITY ? 0.f : m[nt][k & 1];
                            p[k] = ex2(s[nt][k] - mm + kPBias);
                        }
                        l[nt][0] = fmaf(p[0] + p[2], vinv, l[nt][0]);
                        l[nt][1] = fmaf(p[1] + p[3], vinv, l[nt][1]);
                        p0[nt] = movmatrix_trans(pack_half2(p[0], p[1]));
                        p1[nt] = movmatrix_trans(pack_half2(p[2], p[3]));
                    }
#pragma unroll
                    for (int w = 0; w < VW; ++w) {
                        // bytes of tokens (2 t4, 2 t4 + 1) and (2 t4 + 8, 2 t4 + 9) side by side, dims 4 w .. 4 w + 3
                        uint32_t x[2][4];
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            const uint32_t lo = __byte_perm(vr[2 * k][w], vr[2 * k + 1][w], 0x5140);
                            const uint32_t hi = __byte_perm(vr[2 * k][w], vr[2 * k + 1][w], 0x7362);
                            codes_to_half(lo, x[k][0], x[k][1]);
                            codes_to_half(hi, x[k][2], x[k][3]);
                        }
#pragma unroll
                        for (int d = 0; d < 2; ++d)
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt)
                                mma_f16(o[nt][2 * w + d], x[0][2 * d], x[0][2 * d + 1], x[1][2 * d], x[1][2 * d + 1], p0[nt], p1[nt]);
                    }
                }
                load_v(next);
                now = next;
            }
        }

        // the four warps' parts
        __syncthreads();
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                float x = l[nt][k];
                x += __shfl_xor_sync(0xffffffffu, x, 4);
                x += __shfl_xor_sync(0xffffffffu, x, 8);
                x += __shfl_xor_sync(0xffffffffu, x, 16);
                const int r = 8 * nt + 2 * t4 + k;
                if (g == 0) sm.m[warp][r] = m[nt][k], sm.l[warp][r] = x;
#pragma unroll
                for (int i = 0; i < MT; ++i) {
                    // fragment rows g and g + 8 of tile i are dims (D / 8) g + 2 i and + 1
                    *reinterpret_cast<float2 *>(&sm.o[warp][r][(D / 8) * g + 2 * i]) = make_float2(o[nt][i][k], o[nt][i][k + 2]);
                }
            }
        __syncthreads();
        const bool cut = unit0 > 0 || unit1 < units;
        float *part = parts + (2ll * c + (u == u0 ? 0 : 1)) * kPart;
        constexpr int PER = R * D / T;               // outputs of a thread, consecutive dims of one row
        const int r = tid * PER / D, d0 = tid * PER % D;
        auto write_out = [&](const float (&x)[PER], float M, float L) {
            const int row = rt * R + r;
            if (row >= rows) return;
            const int tok = row / group;
            const int64_t at = (q.t0 + tok) * a.q_heads + h * group + (row - tok * group);
            const float inv = L == 0.f ? 0.f : 1.f / L;             // nothing seen: zeros
            uint32_t w[PER / 2];
#pragma unroll
            for (int i = 0; i < PER / 2; ++i) w[i] = pack_bf16x2(x[2 * i] * inv, x[2 * i + 1] * inv);
            uint32_t *dst = reinterpret_cast<uint32_t *>(a.out + at * D + d0);
#pragma unroll
            for (int i = 0; i < PER / 2; ++i) dst[i] = w[i];
            if (a.lse && d0 == 0) a.lse[at] = L == 0.f ? -INFINITY : (M - kPBias + log2f(L)) * kLn2;
        };
        {
            float M = -INFINITY, L = 0.f, x[PER], wt[kStreamWarps];
#pragma unroll
            for (int w = 0; w < kStreamWarps; ++w) M = fmaxf(M, sm.m[w][r]);
#pragma unroll
            for (int w = 0; w < kStreamWarps; ++w) {
                wt[w] = sm.m[w][r] == -INFINITY ? (sm.l[w][r] != sm.l[w][r] ? sm.l[w][r] : 0.f) : ex2(sm.m[w][r] - M);
                L = fmaf(wt[w], sm.l[w][r], L);
            }
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                x[i] = 0.f;
#pragma unroll
                for (int w = 0; w < kStreamWarps; ++w) x[i] = fmaf(wt[w], sm.o[w][r][d0 + i], x[i]);
            }
            if (!cut) {
                write_out(x, M, L);
            } else {
#pragma unroll
                for (int i = 0; i < PER; i += 4)
                    __stcg(reinterpret_cast<float4 *>(part + r * D + d0 + i), make_float4(x[i], x[i + 1], x[i + 2], x[i + 3]));
                if (d0 == 0) __stcg(reinterpret_cast<float2 *>(part + R * D) + r, make_float2(M, L));
            }
        }
        if (cut) {
            __syncthreads();
            const int c0 = range_of(tile_unit), c1 = range_of(tile_unit + units - 1);      // the ranges that hold the tile
            if (tid == 0) {
                const int seen = add_acq_rel(counters + c0, 1);         // releases the whole CTA's part (barrier above)
                sm.last = seen == c1 - c0;
                if (sm.last) counters[c0] = 0;
            }
            __syncthreads();
            if (sm.last) {
                // the parts' maxima and sums first, all at once, then the sums in the order of the ranges, loads ahead
                float (*const pml)[2] = reinterpret_cast<float (*)[2]>(sm.o);
                const int n_parts = c1 - c0 + 1, first_slot = range_start(c0) != tile_unit ? 1 : 0;
                auto part_of = [&](int i) { return parts + (2ll * (c0 + i) + (i == 0 ? first_slot : 0)) * kPart; };
                float M = -INFINITY, L = 0.f, x[PER];
#pragma unroll
                for (int i = 0; i < PER; ++i) x[i] = 0.f;
                for (int p0 = 0; p0 < n_parts; p0 += kJoin) {
                    const int np = min(kJoin, n_parts - p0);
                    __syncthreads();
                    for (int i = tid; i < np * R; i += T) {
                        const float2 v = __ldcg(reinterpret_cast<const float2 *>(part_of(p0 + i / R) + R * D) + i % R);
                        pml[i][0] = v.x;
                        pml[i][1] = v.y;
                    }
                    __syncthreads();
                    float mn = M;
                    for (int i = 0; i < np; ++i) mn = fmaxf(mn, pml[i * R + r][0]);
                    const float wa = M == mn ? 1.f : ex2(M - mn);
                    L *= wa;
#pragma unroll
                    for (int i = 0; i < PER; ++i) x[i] *= wa;
                    M = mn;
#pragma unroll 4
                    for (int i = 0; i < np; ++i) {
                        const float pm = pml[i * R + r][0], pl = pml[i * R + r][1];
                        // nothing seen in a part: no weight, unless its sum says NaN
                        const float w = pm == -INFINITY ? (pl == 0.f ? 0.f : pl) : ex2(pm - mn);
                        const float4 *src = reinterpret_cast<const float4 *>(part_of(p0 + i) + r * D + d0);
                        L = fmaf(pl, w, L);
#pragma unroll
                        for (int k = 0; k < PER / 4; ++k) {
                            const float4 v = __ldcg(src + k);
                            x[4 * k] = fmaf(v.x, w, x[4 * k]);
                            x[4 * k + 1] = fmaf(v.y, w, x[4 * k + 1]);
                            x[4 * k + 2] = fmaf(v.z, w, x[4 * k + 2]);
                            x[4 * k + 3] = fmaf(v.w, w, x[4 * k + 3]);
                        }
                    }
                }
                write_out(x, M, L);
            }
        }
        u = tile_unit + unit1;
    }
    pdl_wait();
}

// ------------------------------------------------------------ many rows a sequence
//
// Prompts and chunks of them: two tiles of 128 rows (of one sequence and key
// head, rows as above) share a pass over the cache in tiles of 128 tokens, on
// the tcgen05 tensor cores.  Sixteen warps:
//   0-3, 4-7  softmax of the first and second tile, a thread for each row;
//   8-11      the cache's codes from global memory to FP16 operands in shared
//             memory (exact), the next tile's loads in flight meanwhile;
//   12-15     one thread that issues the products; the others only give their
//             registers away: a row's thread holds a step's 128 scores.
// S = Q K^T (FP32, tensor memory) is read by the row's thread, and the weights
// go back as FP16 over S and are the first operand of P V from there.  The
// second product sums in tensor memory; its scale (the running maximum) moves
// only when a step's weights sum to more than 2^15, and the row's thread then
// rescales it in place.  While one tile is in its softmax
// the tensor cores work on the other.
// K and V tiles are the same rows of 128 bytes (64 dims) in the 128-byte
// swizzle; K is read along the dims (K-major), V along the tokens (MN-major).
// Measured at 64 / 8 heads of 128: a prompt of 8192 tokens 1.20 .. 1.24 ms, 890 ..
// 915 TFLOP/s of what is visible (55 % of the cuBLAS rate).  Of a step's 3850
// clocks a tile spends 2100 in its softmax (of which 1024 are the exponentials'
// at 8 clocks a warp and instruction; two warps at once would need 1275 each),
// 1330 in its two products (1024 at full rate; the operands of Q K^T alone take
// all of the shared memory's bandwidth) and 400 between them, and the other tile
// fills the tensor cores only meanwhile: a second S buffer would decouple the
// two, but tensor memory is full at head dim 128.  Measured and dropped: two
// threads a row (1.45 ms: barriers and register spills), the maximum in a pass
// of its own (1.39 ms), a branch for every 32 columns (1.27 ms).
// The blocks' scales go through a ring of four, so that a step's are still
// there, and its barrier's phase still open to be seen, whatever the order in
// which the warps get on: step j + 4's are written after S of step j + 2,
// which is after every row's weights of step j + 1.
constexpr int kPromptWarps = 16;
constexpr int kPromptRows = 256;                     // two tiles
constexpr int kKvTile = 128;
constexpr int kInfoRing = 4;
// Where there are too few tile pairs for the GPU, several CTAs share a pair's
// pass over the cache, each a range of its steps (four at least: the join costs
// as much as three), and leave FP32 sums and maxima in the workspace for
// attn_join_kernel: 192 rows on 8192 tokens at 8 key heads are 8 pairs, 64 steps
// each, for 148 SMs.
constexpr int kMostSplit = 16;

// Ranges that a pass of `steps` is cut into, of `split` at the most.
__host__ __device__ __forceinline__ int prompt_ranges(int steps, int split) {
    const int n = steps / 4 < split ? steps / 4 : split;
    return n < 1 ? 1 : n;
}

// A tile pair: sequence, slot within it, rows, and the steps of its pass.
struct PromptTile {
    int b, steps;
    SeqInfo q;
    int64_t rows, row0;
};

// Where a range's part lies: [kPromptRows][D] sums, then [kPromptRows] pairs
// of maximum and weights' sum.
template <int D>
__device__ __forceinline__ float *prompt_part(float *parts, int64_t pair, int split, int range) {
    return parts + (pair * split + range) * (int64_t)(kPromptRows * (D + 2));
}

template <int D>
struct PromptSmem {
    uint8_t q[2][D / 64][128 * 128];
    uint8_t k[2][D / 64][128 * 128];
    uint8_t v[2][D / 64][128 * 128];
    // of a tile's blocks: key scale, log2 of the value scale, its inverse
    float4 info[kInfoRing][kKvTile / 16];
    unsigned long long q_full, k_full[2], k_empty[2], v_full[2], v_empty[2], s_full[2], p_full[2], o_full[2];
    unsigned long long info_full[kInfoRing], drain;
    uint32_t tmem;
    int abort, seq, slot;
};

__device__ __forceinline__ uint64_t add_f32x2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}

// True in one lane of a converged warp, the same one each time.
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "elect.sync _|p, 0xffffffff;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(p));
    return p != 0;
}

// Instructions that stay in the order written (volatile).
__device__ __forceinline__ float in_order_ex2(float x) {
    float y;
    asm volatile("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ uint64_t in_order_fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t d;
    asm volatile("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ __forceinline__ uint64_t in_order_add2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm volatile("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ uint32_t in_order_half2(float lo, float hi) {
    uint32_t d;
    asm volatile("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
    return d;
}

// The registers of a warpgroup.  512 threads are launched with 128 each, all
// there are; 2 x 128 x 184 + 128 x 104 + 128 x 40 are as many.
template <int N>
__device__ __forceinline__ void registers_up() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void registers_down() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// 32 columns of tensor memory, in registers when this returns (the empty
// statements keep their uses behind the wait).
__device__ __forceinline__ void tmem_read32(uint32_t taddr, uint32_t (&r)[32]) {
    tmem_ld_32x32b_x32(taddr, r);
    tmem_ld_wait();
#pragma unroll
    for (int i = 0; i < 32; ++i) asm volatile("" : "+r"(r[i]));
}

// Sequence b owns the slots from floor(cu[b] group / 256) + b on, at least as
// many as it has pairs of tiles.  Called by a whole warp; -1: none.  within < 0
// where cu decreases.
__device__ __forceinline__ int find_slot(const AttnArgs &a, int64_t slot, int &within) {
    const int group = a.q_heads / a.c.heads;
    auto first_slot = [&](int i) {
        const int64_t t0 = a.s.cu ? (int64_t)__ldg(a.s.cu + i) : i;
        return t0 * group / kPromptRows + i;
    };
    const int b = search_lanes<32>(a.s.batch, slot, first_slot);
    within = b < 0 ? 0 : (int)(slot - first_slot(b));
    return b;
}

__device__ __forceinline__ bool prompt_tile(const AttnArgs &a, int b, int slot, bool all, PromptTile &t) {
    const int group = a.q_heads / a.c.heads;
    t.b = b;
    t.q = seq_info(a.s, b);
    t.rows = (int64_t)t.q.n * group;
    t.row0 = (int64_t)slot * kPromptRows;
    if (slot < 0 || t.row0 >= t.rows || (!all && few_rows(t.rows, t.q.len, a))) return false;
    // what the last row sees is what any row sees
    const int64_t tok = (min(t.rows, t.row0 + kPromptRows) - 1) / group;
    const int64_t most = a.causal ? max((int64_t)0, min((int64_t)t.q.len, (int64_t)t.q.len - t.q.n + tok + 1)) : t.q.len;
    t.steps = (int)((most + kKvTile - 1) / kKvTile);
    return true;
}

template <int D>
__global__ void __launch_bounds__(kPromptWarps * 32, 1)
    attn_prompt_kernel(const __grid_constant__ AttnArgs a, bool all, int split, float *parts) {
    constexpr int DB = D / 64;                       // 128-byte row blocks of an operand
    constexpr uint32_t kBlockBytes = 128 * 128;
    extern __shared__ uint8_t smem_raw[];
    PromptSmem<D> &sm = *reinterpret_cast<PromptSmem<D> *>(smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u));
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int H = a.c.heads, group = a.q_heads / H;
    const KvSeqs &S = a.s;

    // The tile pair of this CTA.  Last ones first: under a causal mask they are the longest.
    pdl_launch_dependents();                         // attn_stream_kernel waits for this one at its end only
    const int64_t pairs = gridDim.x / split, pair = pairs - 1 - blockIdx.x / split;
    const int h = pair % H;
    if (warp == 0) {
        int slot;
        const int b = find_slot(a, pair / H, slot);
        if (lane == 0) sm.seq = b, sm.slot = slot;
    }
    __syncthreads();
    const int b = sm.seq;
    if (b < 0) {                                     // cu[0] > 0
        if (tid == 0) report_invalid();
        return;
    }
    PromptTile tile;
    const bool has_rows = prompt_tile(a, b, sm.slot, all, tile);
    const SeqInfo &q = tile.q;
    if (q.bad && tid == 0) report_invalid();         // also where no row is left of it
    if (!has_rows) return;
    const int64_t rows = tile.rows, row0 = tile.row0;
    const int tiles = rows - row0 > 128 ? 2 : 1;
    // this CTA's range of the pass
    const int ranges = prompt_ranges(tile.steps, split), range = blockIdx.x % split;
    if (range >= ranges) return;
    const int step0 = (int)((int64_t)tile.steps * range / ranges);
    const int steps = (int)((int64_t)tile.steps * (range + 1) / ranges) - step0;

    const uint32_t q_full = smem_addr(&sm.q_full), k_full = smem_addr(sm.k_full), k_empty = smem_addr(sm.k_empty),
                   v_full = smem_addr(sm.v_full), v_empty = smem_addr(sm.v_empty), s_full = smem_addr(sm.s_full),
                   p_full = smem_addr(sm.p_full), o_full = smem_addr(sm.o_full), info_full = smem_addr(sm.info_full), drain = smem_addr(&sm.drain);
    volatile int *abort_flag = &sm.abort;
    if (tid == 0) {
        mbar_init(q_full, 128 * tiles);
        for (int i = 0; i < 2; ++i) {
            mbar_init(k_full + 8 * i, 4);
            mbar_init(v_full + 8 * i, 4);
            mbar_init(k_empty + 8 * i, 1);
            mbar_init(v_empty + 8 * i, 1);
            mbar_init(s_full + 8 * i, 1);
            mbar_init(p_full + 8 * i, 128);
            mbar_init(o_full + 8 * i, 1);
        }
        for (int i = 0; i < kInfoRing; ++i) mbar_init(info_full + 8 * i, 4);
        mbar_init(drain, 1);
        sm.abort = 0;
        fence_mbar_init();
    }
    if (warp == 12) {
        tmem_alloc(smem_addr(&sm.tmem), 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = __shfl_sync(0xffffffffu, *(volatile uint32_t *)&sm.tmem, 0);
    const uint32_t tm_s = tmem, tm_o = tmem + 256;

    if (warp < 8) {
        registers_up<184>();
        // ------------------------------------------------ a row each: queries, softmax, output
        const int t = warp >> 2, r = tid & 127;
        if (t < tiles) {
            const int64_t row = row0 + 128 * t + r;
            const bool in = row < rows;
            const int64_t tok = in ? row / group : 0;
            const int head = h * group + (in ? (int)(row - tok * group) : 0);
            const uint16_t *src = a.q.p + (q.t0 + tok) * a.q.ts + (int64_t)head * a.q.hs;
            uint4 x[D / 8];
            float top = 0.f;
#pragma unroll
            for (int i = 0; i < D / 8; ++i) {
                x[i] = in ? __ldg(reinterpret_cast<const uint4 *>(src) + i) : make_uint4(0u, 0u, 0u, 0u);
                const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    top = fmaxf(top, fmaxf(fabsf(__uint_as_float(w[k] << 16)), fabsf(__uint_as_float(w[k] & 0xFFFF0000u))));
            }
            int e = (int)(__float_as_uint(top) >> 23) - 127;
            const bool finite = e <= 127;                // a row with an infinity becomes NaN, whatever it meets
            e = e < -100 ? -100 : e;
            const float up = finite ? __int_as_float((127 + 14 - e) << 23) : __int_as_float(0x7FC00000);
#pragma unroll
            for (int i = 0; i < D / 8; ++i) {
                const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
                uint32_t y[4];
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    y[k] = pack_half2(__uint_as_float(w[k] << 16) * up, __uint_as_float(w[k] & 0xFFFF0000u) * up);
                *reinterpret_cast<uint4 *>(&sm.q[t][i / 8][r * 128 + (((i & 7) ^ (r & 7)) << 4)]) = make_uint4(y[0], y[1], y[2], y[3]);
            }
            fence_proxy_async_shared();
            mbar_arrive(q_full);
            const float f = a.scale * kLog2e * __int_as_float((127 - 14 + e) << 23);
            const int64_t seen = !in ? 0 : (a.causal ? (int64_t)q.len - q.n + tok + 1 : q.len);
            // from the first token of this range on
            const int vis = (int)max((int64_t)0, min(seen, (int64_t)q.len)) - step0 * kKvTile;

            const uint32_t lanes = (uint32_t)(warp & 3) << 21;                // 32 lanes a warp, in bits 16 and up
            const uint32_t ts = tm_s + lanes + 128 * t, to = tm_o + lanes + D * t;
            float m = -INFINITY;
            uint64_t l2 = 0;
            bool ok = true;
            for (int j = 0; j < steps; ++j) {
                // the blocks' scales, on their way while S is computed
                ok = mbar_wait_bounded(info_full + 8 * (j & (kInfoRing - 1)), (j / kInfoRing) & 1, abort_flag);
                float fb[8], lv[8], iv[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float4 b4 = sm.info[j & (kInfoRing - 1)][i];
                    fb[i] = f * b4.x;
                    lv[i] = b4.y;
                    iv[i] = b4.z;
                }
                ok = ok && mbar_wait_bounded(s_full + 8 * t, j & 1, abort_flag);
                if (!__all_sync(0xffffffffu, ok)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const int limit = vis - j * kKvTile;
                const bool masked = __any_sync(0xffffffffu, limit < kKvTile);       // some row does not see all of the tile
                auto ready = [&](uint32_t (&s)[32], int c) {
                    tmem_ld_wait();
#pragma unroll
                    for (int i = 0; i < 32; ++i) asm volatile("" : "+r"(s[i]));     // behind the wait
                    if (masked) {
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            if (i >= limit - 32 * c) s[i] = 0xFF800000u;            // -inf
                    }
                };
                uint32_t s[2][32], p[4][16];
                // The weights are taken against the maximum so far without looking at the scores first: were one far above
                // it, their sum says so (beyond 2^15; 128 weights of 2^kPBias at a maximum that holds reach 2^11), and
                // the step is done again against the scores' own maximum.  By this row alone: what a row gets does not
                // depend on its neighbours.
                bool over = m == -INFINITY;          // the first step, or nothing seen so far
                uint64_t l_add = 0;
                for (int turn = 0;; ++turn) {
                    if (__any_sync(0xffffffffu, over)) {
                        float top = -INFINITY;
                        tmem_ld_32x32b_x32(ts, s[0]);
#pragma unroll
                        for (int c = 0; c < 4; ++c) {
                            ready(s[c & 1], c);
                            if (c < 3) tmem_ld_32x32b_x32(ts + 32 * (c + 1), s[(c + 1) & 1]);
#pragma unroll
                            for (int k = 0; k < 2; ++k) {
                                float y[4];
#pragma unroll
                                for (int i = 0; i < 16; ++i) {
                                    const float x = __uint_as_float(s[c & 1][16 * k + i]);
                                    y[i & 3] = i < 4 ? x : fmaxf(y[i & 3], x);
                                }
                                const float z = fmaxf(fmaxf(y[0], y[1]), fmaxf(y[2], y[3]));
                                // a block that is not seen: -inf times a key scale of zero would be NaN
                                top = fmaxf(top, z == -INFINITY ? z : fmaf(z, fb[2 * c + k], lv[2 * c + k]));
                            }
                        }
                        const float mn = over ? top : m;
                        const float al = m == mn ? 1.f : ex2(m - mn);
                        m = mn;
                        l2 = mul_f32x2(l2, pack_f32x2(al, al));
                        if (j > 0 && __any_sync(0xffffffffu, al != 1.f)) {
                            // what was summed so far: this step's S being complete, so is the product before it
#pragma unroll 1
                            for (int i = 0; i < D / 32; ++i) {
                                tmem_read32(to + 32 * i, s[0]);
#pragma unroll
                                for (int k = 0; k < 32; ++k) s[0][k] = __float_as_uint(__uint_as_float(s[0][k]) * al);
                                tmem_st_32x32b_x32(to + 32 * i, s[0]);
                            }
                        }
                    }
                    // Two columns at a time, in the order written: the exponentials are what bounds a row (8 clocks a warp
                    // and instruction), so the product of the next pair and the sum and packing of the pair before last
                    // stand between them.
                    const float base = kPBias - (m == -INFINITY ? 0.f : m);
                    uint64_t all = 0, sum[2], x[2], f2, a2;
                    float u[3], v[3];
                    l_add = 0;
                    tmem_ld_32x32b_x32(ts, s[0]);
#pragma unroll
                    for (int n = 0; n < 64 + 3; ++n) {
                        if (n < 64) {
                            if (n % 16 == 0) {
                                ready(s[n / 16 & 1], n / 16);
                                if (n < 48) tmem_ld_32x32b_x32(ts + 2 * n + 32, s[(n / 16 & 1) ^ 1]);
                            }
                            if (n % 8 == 0) {
                                // the smallest float instead of zero, so that a masked -inf stays -inf
                                const float fk = fmaxf(fb[n / 8], 1.1754944e-38f), ak = lv[n / 8] + base;
                                f2 = pack_f32x2(fk, fk);
                                a2 = pack_f32x2(ak, ak);
                            }
                            const uint32_t *d = s[n / 16 & 1] + 2 * (n % 16);
                            x[n & 1] = in_order_fma2(pack_f32x2(__uint_as_float(d[0]), __uint_as_float(d[1])), f2, a2);
                        }
                        if (n >= 1 && n < 65) {
                            float lo, hi;
                            unpack_f32x2(x[(n - 1) & 1], lo, hi);
                            u[(n - 1) % 3] = in_order_ex2(lo);
                            v[(n - 1) % 3] = in_order_ex2(hi);
                        }
                        if (n >= 3) {
                            const int q = n - 3;
                            const uint64_t uv = pack_f32x2(u[q % 3], v[q % 3]);
                            sum[q & 1] = q % 8 < 2 ? uv : in_order_add2(sum[q & 1], uv);
                            p[q / 16][q % 16] = in_order_half2(u[q % 3], v[q % 3]);
                            if (q % 8 == 7) {
                                const uint64_t block = in_order_add2(sum[0], sum[1]);
                                all = in_order_add2(all, block);
                                l_add = in_order_fma2(block, pack_f32x2(iv[q / 8], iv[q / 8]), l_add);
                            }
                        }
                    }
                    float lo, hi;
                    unpack_f32x2(all, lo, hi);
                    over = lo + hi > 32768.f;
                    // sums against the scores' own maximum stay small (and where scores are so large that FP32 no longer
                    // tells them apart, twice is enough)
                    if (turn == 2 || !__any_sync(0xffffffffu, over)) break;
                }
                l2 = add_f32x2(l2, l_add);
#pragma unroll
                for (int c = 0; c < 4; ++c) tmem_st_32x32b_x16(ts + 16 * c, p[c]);
                tmem_st_wait();
                tc_fence_before();
                mbar_arrive(p_full + 8 * t);
            }
            float l0, l1;
            unpack_f32x2(l2, l0, l1);
            const float l = l0 + l1;
            const float inv = l == 0.f ? 0.f : 1.f / l;              // nothing seen: zeros
            if (steps > 0 && ok) ok = __all_sync(0xffffffffu, mbar_wait_bounded(o_full + 8 * t, 0, abort_flag));
            tc_fence_after();
            const int64_t at = (q.t0 + tok) * a.q_heads + head;
            float *part = prompt_part<D>(parts, pair, split, range);
#pragma unroll
            for (int c = 0; c < D / 32; ++c) {
                uint32_t o[32];
                if (steps > 0 && ok) {
                    tmem_read32(to + 32 * c, o);
                } else {
#pragma unroll
                    for (int i = 0; i < 32; ++i) o[i] = 0u;
                }
                if (!in) continue;
                if (ranges > 1) {
                    uint4 *dst = reinterpret_cast<uint4 *>(part + (128 * t + r) * D + 32 * c);
#pragma unroll
                    for (int i = 0; i < 8; ++i) dst[i] = make_uint4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
                    continue;
                }
                uint4 *dst = reinterpret_cast<uint4 *>(a.out + at * D + 32 * c);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    uint32_t w[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        w[k] = pack_bf16x2(__uint_as_float(o[8 * i + 2 * k]) * inv, __uint_as_float(o[8 * i + 2 * k + 1]) * inv);
                    dst[i] = make_uint4(w[0], w[1], w[2], w[3]);
                }
            }
            if (in && ranges > 1)
                *reinterpret_cast<float2 *>(part + kPromptRows * D + 2 * (128 * t + r)) = make_float2(m, l);
            else if (in && a.lse)
                a.lse[at] = l == 0.f ? -INFINITY : (m - kPBias + log2f(l)) * kLn2;
        }
    } else if (warp < 12) {
        registers_down<104>();
        // ------------------------------------------------ codes to operands
        // Warp w converts tokens 32 w .. + 31 of a tile: eight rows by 64 codes a step, a lane 16 codes of a row, which
        // become two of the row's 16-byte chunks; the eight lanes that store together (two rows, even and odd) fill all
        // eight chunk positions.
        const int w = warp - 8, rr = lane >> 2, c4 = lane & 3;
        const int32_t *pages = S.table + (int64_t)b * S.max_pages;
        const int bshift = S.page_shift - 4, bmask = (1 << bshift) - 1;
        const int blocks = (q.len + 15) >> 4;
        uint4 kx[4][DB], vx[4][DB];
        // A lane looks after one of the warp's blocks of the next 16 steps: where it lies in the cache (-1: no token of it
        // is seen) and what the rows' threads need of it.
        int sc = -1;
        float4 about = make_float4(0.f, -INFINITY, 0.f, 0.f);
        auto look_up = [&](int j) {
            const int step = j + (lane >> 1), blk = (step0 + step) * 8 + 2 * w + (lane & 1);
            sc = -1;
            about = make_float4(0.f, -INFINITY, 0.f, 0.f);
            if (step >= steps || blk >= blocks) return;
            const int page = __ldg(pages + (blk >> bshift));
            if (page < 0 || page >= S.pages) {
                report_invalid();
                return;
            }
            sc = ((page * H + h) << bshift) + (blk & bmask);
            about.x = __ldg(a.c.ks + sc);
            about.y = __ldg(a.c.vs + sc);            // until finish()
        };
        auto finish = [&] {
            if (sc < 0) return;
            // finite even where the scale is not: a row that does not see the block has -infinity for its scores, and the
            // sum with an infinite logarithm would be NaN
            const float ve = fminf(fmaxf(about.y, kLeastScale), 3.40282347e38f);
            about.y = log2f(ve);
            about.z = 1.f / ve;
        };
        auto load = [&](const int8_t *base, int at, uint4 (&x)[4][DB]) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int b = __shfl_sync(0xffffffffu, sc, 2 * at + (i >> 1));
#pragma unroll
                for (int d = 0; d < DB; ++d)
                    x[i][d] = b < 0 ? make_uint4(0u, 0u, 0u, 0u)
                                    : ld_stream16(base + (int64_t)b * (16 * D) + (8 * (i & 1) + rr) * D + 64 * d + 16 * c4);
            }
        };
        auto store = [&](uint8_t (*dst)[128 * 128], const uint4 (&x)[4][DB]) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int d = 0; d < DB; ++d) {
                    const int row = 32 * w + 8 * i + rr;
                    uint32_t y[8];
                    codes_to_half(x[i][d].x, y[0], y[1]);
                    codes_to_half(x[i][d].y, y[2], y[3]);
                    codes_to_half(x[i][d].z, y[4], y[5]);
                    codes_to_half(x[i][d].w, y[6], y[7]);
                    uint8_t *p = dst[d] + row * 128;
                    *reinterpret_cast<uint4 *>(p + (((2 * c4) ^ (row & 7)) << 4)) = make_uint4(y[0], y[1], y[2], y[3]);
                    *reinterpret_cast<uint4 *>(p + (((2 * c4 + 1) ^ (row & 7)) << 4)) = make_uint4(y[4], y[5], y[6], y[7]);
                }
        };
        look_up(0);
        load(a.c.k, 0, kx);
        load(a.c.v, 0, vx);
        finish();
        for (int j = 0; j < steps; ++j) {
            const int st = j & 1;
            const uint32_t free_parity = ((j >> 1) & 1) ^ 1;
            if (!__all_sync(0xffffffffu, mbar_wait_bounded(k_empty + 8 * st, free_parity, abort_flag))) break;
            store(sm.k[st], kx);
            const int mine = 2 * (j & 15) + (lane & 1);
            const float4 now = make_float4(__shfl_sync(0xffffffffu, about.x, mine), __shfl_sync(0xffffffffu, about.y, mine),
                                           __shfl_sync(0xffffffffu, about.z, mine), 0.f);
            if (lane < 2) sm.info[j & (kInfoRing - 1)][2 * w + lane] = now;
            fence_proxy_async_shared();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(k_full + 8 * st);
                mbar_arrive(info_full + 8 * (j & (kInfoRing - 1)));
            }
            const bool refill = ((j + 1) & 15) == 0;
            if (refill) look_up(j + 1);
            load(a.c.k, (j + 1) & 15, kx);
            if (!__all_sync(0xffffffffu, mbar_wait_bounded(v_empty + 8 * st, free_parity, abort_flag))) break;
            store(sm.v[st], vx);
            fence_proxy_async_shared();
            __syncwarp();
            if (lane == 0) mbar_arrive(v_full + 8 * st);
            load(a.c.v, (j + 1) & 15, vx);
            if (refill) finish();
        }
    } else {
        registers_down<40>();
        if (warp == 12 && steps > 0) {
            // ------------------------------------------------ products
            // The whole warp goes through the loop and one lane issues: what the instructions take (descriptors, addresses)
            // is then the same for the warp and stays in uniform registers.
            constexpr uint32_t idesc_s = idesc_f16(128, kKvTile, false), idesc_o = idesc_f16(128, D, true);
            // operands' addresses count in 16 bytes in their descriptors' low bits
            constexpr uint32_t kStage = DB * kBlockBytes / 16;
            const uint64_t q_desc = smem_desc_k_sw128(smem_addr(sm.q)), k_desc = smem_desc_k_sw128(smem_addr(sm.k)),
                           v_desc = smem_desc_mn_sw128(smem_addr(sm.v), kBlockBytes);
            const bool one = elect_one();
            auto scores = [&](int t, int st) {
                const uint64_t qd = q_desc + t * kStage, kd = k_desc + st * kStage;
                const uint32_t d = tm_s + 128 * t;
                if (one) {
#pragma unroll
                    for (int i = 0; i < D / 16; ++i) {
                        const uint32_t off = ((i / 4) * kBlockBytes + (i % 4) * 32) / 16;
                        umma_f16(d, qd + off, kd + off, idesc_s, i > 0);
                    }
                    umma_commit(s_full + 8 * t);
                }
            };
            auto values = [&](int t, int st, bool first, bool last) {
                const uint64_t vd = v_desc + st * kStage;
                const uint32_t d = tm_o + D * t, p = tm_s + 128 * t;
                if (one) {
                    umma_f16_ts(d, p, vd, idesc_o, !first);
#pragma unroll
                    for (int i = 1; i < kKvTile / 16; ++i) umma_f16_ts(d, p + 8 * i, vd + i * (16 * 128 / 16), idesc_o, 1);
                    if (last) umma_commit(o_full + 8 * t);
                }
            };
            bool ok = mbar_wait_bounded(q_full, 0, abort_flag) && mbar_wait_bounded(k_full, 0, abort_flag);
            ok = __all_sync(0xffffffffu, ok);
            tc_fence_after();
            if (ok) {
                scores(0, 0);
                if (tiles > 1) scores(1, 0);
                if (one && steps > 2) umma_commit(k_empty);      // waited for by the stage's next use, where there is one
            }
            for (int j = 0; ok && j < steps; ++j) {
                const int st = j & 1, sn = st ^ 1;
                ok = mbar_wait_bounded(v_full + 8 * st, (j >> 1) & 1, abort_flag);
                if (ok && j + 1 < steps) ok = mbar_wait_bounded(k_full + 8 * sn, ((j + 1) >> 1) & 1, abort_flag);
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    if (t == 1 && tiles < 2) break;
                    if (ok) ok = mbar_wait_bounded(p_full + 8 * t, j & 1, abort_flag);
                    ok = __all_sync(0xffffffffu, ok);
                    if (!ok) break;
                    tc_fence_after();
                    values(t, st, j == 0, j + 1 == steps);
                    if (j + 1 < steps) scores(t, sn);
                }
                if (ok && one) {
                    if (j + 2 < steps) umma_commit(v_empty + 8 * st);
                    if (j + 3 < steps) umma_commit(k_empty + 8 * sn);
                }
            }
            if (one && *abort_flag) {
                // given up: what was issued still has to be complete before tensor memory goes (otherwise the rows' threads
                // have waited for the last products)
                umma_commit(drain);
                const unsigned long long start = global_timer_ns();
                while (!mbar_try_wait(drain, 0) && global_timer_ns() - start < 1000000000ull) {}
            }
            __syncwarp();
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 12) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// The parts of the tile pairs that several CTAs shared, a warp for each row,
// in the order of their ranges.
constexpr int kJoinWarps = 8;

template <int D>
__global__ void __launch_bounds__(kJoinWarps * 32) attn_join_kernel(const __grid_constant__ AttnArgs a, bool all, int split,
                                                                  float *parts) {
    constexpr int V = D / 32;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int H = a.c.heads, group = a.q_heads / H;
    const int64_t pair = blockIdx.x / (kPromptRows / kJoinWarps);
    const int r = (int)(blockIdx.x % (kPromptRows / kJoinWarps)) * kJoinWarps + warp, h = pair % H;
    int slot;
    const int b = find_slot(a, pair / H, slot);
    PromptTile tile;
    if (b < 0 || !prompt_tile(a, b, slot, all, tile)) return;
    const int ranges = prompt_ranges(tile.steps, split);
    const int64_t row = tile.row0 + r;
    if (ranges < 2 || row >= tile.rows) return;
    const int64_t tok = row / group, at = (tile.q.t0 + tok) * a.q_heads + h * group + (row - tok * group);
    // the ranges' maxima and sums: a lane each (kMostSplit <= 32)
    float m = -INFINITY, l = 0.f;
    if (lane < ranges) {
        const float2 v = *(reinterpret_cast<const float2 *>(prompt_part<D>(parts, pair, split, lane) + kPromptRows * D) + r);
        m = v.x;
        l = v.y;
    }
    float top = m;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    // nothing seen in a range: no weight, unless its sum says NaN
    const float w = m == -INFINITY ? (l == 0.f ? 0.f : l) : ex2(m - top);
    float total = 0.f, x[V];
#pragma unroll
    for (int k = 0; k < V; ++k) x[k] = 0.f;
#pragma unroll 4
    for (int i = 0; i < ranges; ++i) {
        const float wi = __shfl_sync(0xffffffffu, w, i), li = __shfl_sync(0xffffffffu, l, i);
        const float *src = prompt_part<D>(parts, pair, split, i) + r * D + lane * V;
        float y[V];
        if constexpr (V == 4) {
            const float4 v = *reinterpret_cast<const float4 *>(src);
            y[0] = v.x, y[1] = v.y, y[2] = v.z, y[3] = v.w;
        } else {
            const float2 v = *reinterpret_cast<const float2 *>(src);
            y[0] = v.x, y[1] = v.y;
        }
        total = fmaf(wi, li, total);
#pragma unroll
        for (int k = 0; k < V; ++k) x[k] = fmaf(wi, y[k], x[k]);
    }
    const float inv = total == 0.f ? 0.f : 1.f / total;
    uint32_t *dst = reinterpret_cast<uint32_t *>(a.out + at * D + lane * V);
#pragma unroll
    for (int k = 0; k < V / 2; ++k) dst[k] = pack_bf16x2(x[2 * k] * inv, x[2 * k + 1] * inv);
    if (a.lse && lane == 0) a.lse[at] = total == 0.f ? -INFINITY : (top - kPBias + log2f(total)) * kLn2;
}

// Rows of a tile: 8 where a sequence has no more, 16 otherwise (the next tile of
// the same head reads the cache again, mostly from L2).
static int stream_tiles(int64_t tokens, int32_t batch, int32_t q_heads, int32_t kv_heads) {
    const int64_t rows = (tokens + batch - 1) / batch * (q_heads / kv_heads);
    return rows <= 8 ? 1 : 2;
}

static int64_t prompt_pairs(int64_t tokens, int32_t batch, int32_t q_heads, int32_t kv_heads) {
    return (tokens * (q_heads / kv_heads) / kPromptRows + batch) * kv_heads;
}

// CTAs to a tile pair: as many as the SMs have room for, no more than the
// longest pass could feed.
static int prompt_split(int64_t pairs, int64_t most_tokens, int sms) {
    const int64_t room = sms / pairs, steps = (most_tokens + kKvTile - 1) / kKvTile;
    const int64_t split = room < kMostSplit ? room : kMostSplit;
    return prompt_ranges((int)(steps < 4096 ? steps : 4096), split < 1 ? 1 : (int)split);
}

// Which kernels a step takes.  A sequence's rows and length decide, on the
// device (few_rows); what the host can tell is the most rows that one may have
// and how long the page table lets it be.  Where the largest is streamed, all
// are: fewer rows never turn the rule, and in the length it holds a linear sum
// that starts below against a concave one.
struct AttnPlan {
    bool tiled, streamed;             // kernels to launch; with only one, it takes every sequence
    int nt, split;
    int64_t stream_floats, pairs;
};

static AttnPlan attn_plan(const AttnArgs &a, int sms) {
    AttnPlan p;
    const int group = a.q_heads / a.c.heads;
    const int64_t most = (a.s.cu ? a.s.tokens : 1) * group, longest = (int64_t)a.s.max_pages << a.s.page_shift;
    p.tiled = !few_rows(most, longest, a);
    p.streamed = !(p.tiled && a.s.batch == 1 && most > kManyRows);
    p.nt = stream_tiles(a.s.tokens, a.s.batch, a.q_heads, a.c.heads);
    const int64_t grid = (int64_t)sms * stream_ctas(p.nt);
    p.stream_floats = stream_counters((int)grid, p.nt) + 2 * grid * (8 * p.nt) * (a.c.dim + 2);
    p.pairs = prompt_pairs(a.s.tokens, a.s.batch, a.q_heads, a.c.heads);
    p.split = p.tiled ? prompt_split(p.pairs, longest, sms) : 1;
    return p;
}

// Counters and parts of the streamed tiles, then parts of the tile pairs.
int64_t attn_kv8_workspace_bytes(const AttnArgs &a, int sms) {
    const AttnPlan p = attn_plan(a, sms);
    return 4 * (p.stream_floats + (p.split > 1 ? p.pairs * p.split * kPromptRows * (a.c.dim + 2) : 0));
}

// Shared memory beyond the default, set once for a kernel and device.
template <typename Kernel>
static cudaError_t allow_smem(Kernel *kernel, int bytes, bool (&done)[64]) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess || (dev < 64 && done[dev])) return e;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess && dev < 64) done[dev] = true;
    return e;
}

// beside: launched behind attn_prompt_kernel and independent of it, so it may
// start while that one's last CTAs run (it ends after them: a kernel that
// follows on the stream finds both complete).
template <int D, int NT, bool All>
static cudaError_t launch_stream(const AttnArgs &a, int sms, bool beside, cudaStream_t stream) {
    static bool done[64] = {};
    const int bytes = (int)sizeof(StreamSmem<D, NT>);
    const cudaError_t e = allow_smem(attn_stream_kernel<D, NT, All>, bytes, done);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3((unsigned)(sms * stream_ctas(NT)));
    cfg.blockDim = dim3(kStreamWarps * 32);
    cfg.dynamicSmemBytes = (size_t)bytes;
    cfg.stream = stream;
    cfg.attrs = beside ? attr : nullptr;
    cfg.numAttrs = beside ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, attn_stream_kernel<D, NT, All>, a);
}

template <int D>
static cudaError_t launch_stream(const AttnArgs &a, const AttnPlan &p, int sms, cudaStream_t stream) {
    const bool beside = p.tiled && p.split == 1;     // directly behind attn_prompt_kernel
    if (p.nt == 1)
        return p.tiled ? launch_stream<D, 1, false>(a, sms, beside, stream) : launch_stream<D, 1, true>(a, sms, beside, stream);
    return p.tiled ? launch_stream<D, 2, false>(a, sms, beside, stream) : launch_stream<D, 2, true>(a, sms, beside, stream);
}

template <int D>
static cudaError_t launch_prompt(const AttnArgs &a, const AttnPlan &p, cudaStream_t stream) {
    static bool done[64] = {};
    const int bytes = (int)sizeof(PromptSmem<D>) + 1024;
    cudaError_t e = allow_smem(attn_prompt_kernel<D>, bytes, done);
    if (e != cudaSuccess) return e;
    float *parts = static_cast<float *>(a.ws) + p.stream_floats;
    attn_prompt_kernel<D><<<(unsigned)(p.pairs * p.split), kPromptWarps * 32, bytes, stream>>>(a, !p.streamed, p.split, parts);
    if ((e = cudaGetLastError()) != cudaSuccess || p.split == 1) return e;
    attn_join_kernel<D><<<(unsigned)(p.pairs * (kPromptRows / kJoinWarps)), kJoinWarps * 32, 0, stream>>>(a, !p.streamed, p.split, parts);
    return cudaGetLastError();
}

cudaError_t launch_attn_kv8(const AttnArgs &a, int sms, cudaStream_t stream) {
    const AttnPlan p = attn_plan(a, sms);
    if (p.tiled) {
        const cudaError_t e = a.c.dim == 128 ? launch_prompt<128>(a, p, stream) : launch_prompt<64>(a, p, stream);
        if (e != cudaSuccess || !p.streamed) return e;
    }
    return a.c.dim == 128 ? launch_stream<128>(a, p, sms, stream) : launch_stream<64>(a, p, sms, stream);
}

}  // namespace convrot
