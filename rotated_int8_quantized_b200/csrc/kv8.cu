// kv8.cu -- what stands between the q/k/v projections and attention: norms
// of queries and keys per head with the position rotation in the same pass,
// and the paged INT8 key/value cache (append, read).
//
//   norm    y_d = x_d * rsqrt(mean_d(x_d^2) + eps) * w_d          per head
//   rotate  (a, b) -> (a c - b s, b c + a s)      c, s = table[position][pair]
//   store   codes q = clamp(rne(x / s), +-127), one FP32 scale s for every
//           16 tokens of a page and head
//
// All of it is bound by memory: a value is loaded once as BF16, kept in
// FP32 registers through norm and rotation, and rounded once on its way out
// (to BF16, or to its INT8 code).
//
// A row (one head of one token) belongs to dim / 8 consecutive lanes, eight
// values each.  With the pairs (i, i + rot / 2) a lane holds dims 4i .. 4i+3
// and their partners, so the rotation needs no exchange between lanes and a
// lane needs four table entries (32 bytes) for all the heads it works on.
//
// The scale of a block that still has room.  A block of 16 tokens is filled
// by one call or, token by token, by sixteen.  Its first tokens set
// s = max|x| / 127; later tokens keep s while they fit (max|x| < 127.5 s: no
// code would round past 127), and double it as often as it takes when they do
// not, the older codes q becoming rne(q / 2^j).  Doubling, not max|x| / 127
// again, bounds what a value can lose to the block's history: roundings of
// 0.5 s, 0.5 s / 2, 0.5 s / 4 .. in units of the final scale s, less than one
// step in all however the tokens arrived, where rescaling to every new
// maximum could round sixteen times at full size.
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "common.cuh"
#include "kv8.h"

namespace convrot {

constexpr int kHeadThreads = 256;

// An invalid argument that only the device can see: recorded unless another
// error is (a warning gives way).
__device__ __forceinline__ void report_invalid() {
    if (atomicCAS(&g_device_status, 0, 1 /* CONVROT_ERR_INVALID_ARG */) == 8) atomicCAS(&g_device_status, 8, 1);
}

// ------------------------------------------------------------ sequences
// Token row t of a step belongs to sequence b with cu[b] <= t < cu[b + 1],
// at cache position kv_len[b] - (cu[b + 1] - t).
struct TokenPlace {
    int b;                // -1: behind the last sequence
    int64_t pos;          // < 0: padding, the sequence is shorter than its rows
};

// The last b in [0, batch) with key(b) <= x, for key monotone in b; -1 if
// there is none.  L consecutive lanes search together, L probes a step.
// Where key is not monotone (a cu that decreases) some b of [0, batch), whose
// key may be above x: callers that count from key(b) check that.
template <int L, typename Key>
__device__ __forceinline__ int search_lanes(int batch, int64_t x, Key key) {
    const int lane = threadIdx.x & (L - 1);
    const unsigned group = (L == 32) ? 0xffffffffu : (((1u << (L & 31)) - 1u) << (threadIdx.x & 31 & ~(L - 1)));
    int lo = 0, n = batch;
    while (true) {
        const int step = (n + L - 1) / L;
        const int i = lo + lane * step;
        const bool le = lane * step < n && key(i) <= x;
        const int c = __popc(__ballot_sync(group, le) & group);
        if (c == 0) return -1;
        const int end = lo + n;
        lo += (c - 1) * step;
        if (step == 1) return lo;
        n = end - lo < step ? end - lo : step;
    }
}

template <int L>
__device__ __forceinline__ TokenPlace place_token(const KvSeqs &s, int64_t t) {
    TokenPlace p;
    if (!s.cu) {
        p.b = (int)t;
        p.pos = (int64_t)__ldg(s.kv_len + t) - 1;
        return p;
    }
    const int b = search_lanes<L>(s.batch, t, [&](int i) { return (int64_t)__ldg(s.cu + i); });
    p.b = -1;
    p.pos = -1;
    if (b < 0) {                                     // cu[0] > 0
        if ((threadIdx.x & (L - 1)) == 0) report_invalid();
        return p;
    }
    const int64_t end = __ldg(s.cu + b + 1);
    if (t >= end) return p;
    p.b = b;
    p.pos = (int64_t)__ldg(s.kv_len + b) - (end - t);
    return p;
}

// ------------------------------------------------------------ head rows
// Where a lane's eight values lie in a row, and its rotation's coefficients.
struct LaneGeo {
    int a, b;             // dims a .. a+3 and b .. b+3
    bool rotated;
};

__device__ __forceinline__ LaneGeo lane_geo(int lane, const RopeArgs &r) {
    LaneGeo g;
    const int rl = r.cs ? r.rot / 8 : 0;
    g.rotated = lane < rl;
    if (g.rotated && !r.adjacent) {
        g.a = 4 * lane;
        g.b = r.rot / 2 + 4 * lane;
    } else {
        g.a = 8 * lane;
        g.b = 8 * lane + 4;
    }
    return g;
}

// Coefficients of pairs 4 lane .. 4 lane + 3 at token row t (cache position
// `pos` where the caller gives no positions).  False if a position lies
// outside the table or an axis outside the positions.
__device__ __forceinline__ bool load_rotation(const RopeArgs &r, const LaneGeo &g, int lane, int64_t t, int64_t tokens,
                                              int64_t pos, float (&c)[4], float (&s)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) c[i] = 1.f, s[i] = 0.f;
    if (!g.rotated) return true;
    const int half = r.rot / 2;
    if (!r.axis) {
        const int64_t p = r.pos ? (int64_t)__ldg(r.pos + t) : pos;
        if (p < 0 || p >= r.rows) return false;
        const float4 *e = reinterpret_cast<const float4 *>(r.cs + (p * half + 4 * lane) * 2);
        const float4 x = __ldg(e), y = __ldg(e + 1);
        c[0] = x.x, s[0] = x.y, c[1] = x.z, s[1] = x.w;
        c[2] = y.x, s[2] = y.y, c[3] = y.z, s[3] = y.w;
        return true;
    }
    bool ok = true;
    const uchar4 axes = __ldg(reinterpret_cast<const uchar4 *>(r.axis) + lane);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int ax = i == 0 ? axes.x : i == 1 ? axes.y : i == 2 ? axes.z : axes.w;
        const int64_t p = ax < r.axes ? (int64_t)__ldg(r.pos + ax * tokens + t) : -1;
        if (p < 0 || p >= r.rows) {
            ok = false;
            continue;
        }
        const float2 e = __ldg(reinterpret_cast<const float2 *>(r.cs) + p * half + 4 * lane + i);
        c[i] = e.x;
        s[i] = e.y;
    }
    return ok;
}

__device__ __forceinline__ void unpack_bf16x4(const uint2 &w, float *y) {
    y[0] = __uint_as_float(w.x << 16);
    y[1] = __uint_as_float(w.x & 0xFFFF0000u);
    y[2] = __uint_as_float(w.y << 16);
    y[3] = __uint_as_float(w.y & 0xFFFF0000u);
}

__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
    __nv_bfloat162 h = __halves2bfloat162(__float2bfloat16_rn(lo), __float2bfloat16_rn(hi));
    return *reinterpret_cast<uint32_t *>(&h);
}

// A lane's eight values as FP32 pairs: the even and odd elements of its two
// pieces, which is how they come apart from (and go back into) BF16 words.
struct Row8 {
    uint64_t e[2], o[2];                  // piece 0 (dims a ..): (0, 2) and (1, 3); piece 1 (dims b ..) likewise
};

__device__ __forceinline__ Row8 unpack_row(const uint2 &a, const uint2 &b) {
    Row8 r;
    r.e[0] = pack_f32x2(__uint_as_float(a.x << 16), __uint_as_float(a.y << 16));
    r.o[0] = pack_f32x2(__uint_as_float(a.x & 0xFFFF0000u), __uint_as_float(a.y & 0xFFFF0000u));
    r.e[1] = pack_f32x2(__uint_as_float(b.x << 16), __uint_as_float(b.y << 16));
    r.o[1] = pack_f32x2(__uint_as_float(b.x & 0xFFFF0000u), __uint_as_float(b.y & 0xFFFF0000u));
    return r;
}

__device__ __forceinline__ void row_piece(const Row8 &r, int piece, float (&y)[4]) {
    unpack_f32x2(r.e[piece], y[0], y[2]);
    unpack_f32x2(r.o[piece], y[1], y[3]);
}

__device__ __forceinline__ uint2 pack_piece(const Row8 &r, int piece) {
    float y[4];
    row_piece(r, piece, y);
    return make_uint2(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]));
}

// What a row is multiplied by, the norm's weights and the rotation's
// coefficients in one: with P and Q the two values of four rotated pairs (two
// at a time), P' = P c1 - Q s1 and Q' = Q c2 + P s2, where c1 = w_P cos, s1 = w_Q
// sin, c2 = w_Q cos, s2 = w_P sin.  P and Q are the pieces (Adjacent: the even
// and odd elements of a piece).  A lane whose dims are not rotated only
// multiplies by the weights (c1 and c2): 0 times an infinity in the partner
// would be NaN.
struct Turns {
    uint64_t c1[2], s1[2], c2[2], s2[2];
    bool rotated;
};

template <bool Adjacent>
__device__ __forceinline__ Turns make_turns(const float (&w)[8], const float (&c)[4], const float (&s)[4], bool rotated) {
    Turns t;
    t.rotated = rotated;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        // elements of P and Q, and their pairs' numbers
        const int p0 = Adjacent ? 4 * k : k, q0 = Adjacent ? 4 * k + 1 : 4 + k, f0 = Adjacent ? 2 * k : k, f1 = Adjacent ? f0 + 1 : f0 + 2;
        t.c1[k] = pack_f32x2(w[p0] * c[f0], w[p0 + 2] * c[f1]);
        t.s1[k] = pack_f32x2(-w[q0] * s[f0], -w[q0 + 2] * s[f1]);
        t.c2[k] = pack_f32x2(w[q0] * c[f0], w[q0 + 2] * c[f1]);
        t.s2[k] = pack_f32x2(w[p0] * s[f0], w[p0 + 2] * s[f1]);
    }
    return t;
}

// Norm and rotation of a row; its L lanes call it together.
template <int L, bool Adjacent>
__device__ __forceinline__ void norm_rotate(Row8 &x, const Turns &t, bool norm, float eps) {
    if (norm) {
        uint64_t q = mul_f32x2(x.e[0], x.e[0]);
        q = fma_f32x2(x.o[0], x.o[0], q);
        q = fma_f32x2(x.e[1], x.e[1], q);
        q = fma_f32x2(x.o[1], x.o[1], q);
        float a, b;
        unpack_f32x2(q, a, b);
        a += b;
        // lanes of other rows of the warp may have left: only this row's take part
        const unsigned group = ((1u << L) - 1u) << (threadIdx.x & 31 & ~(L - 1));
#pragma unroll
        for (int o = L / 2; o > 0; o >>= 1) a += __shfl_xor_sync(group, a, o);
        const float r = rsqrtf(fmaf(a, 1.f / (8 * L), eps));
        const uint64_t r2 = pack_f32x2(r, r);
#pragma unroll
        for (int k = 0; k < 2; ++k) x.e[k] = mul_f32x2(x.e[k], r2), x.o[k] = mul_f32x2(x.o[k], r2);
    }
    auto turn = [](uint64_t &p, uint64_t &q, const Turns &t, int k) {
        uint64_t u = mul_f32x2(p, t.c1[k]), v = mul_f32x2(q, t.c2[k]);
        if (t.rotated) u = fma_f32x2(q, t.s1[k], u), v = fma_f32x2(p, t.s2[k], v);
        p = u;
        q = v;
    };
    if (Adjacent) {
        turn(x.e[0], x.o[0], t, 0);
        turn(x.e[1], x.o[1], t, 1);
    } else {
        turn(x.e[0], x.e[1], t, 0);
        turn(x.o[0], x.o[1], t, 1);
    }
}

__device__ __forceinline__ void load_weight(const uint16_t *w, const LaneGeo &g, float (&out)[8]) {
    if (!w) {
#pragma unroll
        for (int i = 0; i < 8; ++i) out[i] = 1.f;
        return;
    }
    unpack_bf16x4(__ldg(reinterpret_cast<const uint2 *>(w + g.a)), out);
    unpack_bf16x4(__ldg(reinterpret_cast<const uint2 *>(w + g.b)), out + 4);
}

// Heads [h0, h1) of token row t: load, norm, rotate, round, store, two rows at
// a time and the next two in flight.  Next to memory it is bound by what it
// issues (one value at a time: 198 instructions a pair of rows, 79 % of the issue
// slots, 83 us for 8191 tokens of 84 heads), hence the FP32 pairs: 75 us, 4.76
// TB/s, 73 % of the copy rate.  `rotation` finds the coefficients once the first
// rows are on their way, and says what to write: the rows (1), zeros (0) or
// nothing (-1).  Rows may be rotated in place, so plain loads.
template <int L, bool Adjacent, typename Rotation>
__device__ __forceinline__ void head_rows(const HeadRows &in, const HeadRowsOut &out, int64_t t, int h0, int h1,
                                          const uint16_t *weight, float eps, const LaneGeo &g, Rotation rotation) {
    const uint16_t *src = in.p + t * in.ts + h0 * in.hs;
    uint16_t *dst = out.p + t * out.ts + h0 * out.hs;
    uint2 x[2][2];
    auto load = [&](int h) {
        if (h < h1) {
            x[0][0] = *reinterpret_cast<const uint2 *>(src + g.a);
            x[0][1] = *reinterpret_cast<const uint2 *>(src + g.b);
        }
        src += in.hs;
        if (h + 1 < h1) {
            x[1][0] = *reinterpret_cast<const uint2 *>(src + g.a);
            x[1][1] = *reinterpret_cast<const uint2 *>(src + g.b);
        }
        src += in.hs;
    };
    load(h0);
    float w[8], c[4], s[4];
    load_weight(weight, g, w);
    const int what = rotation(c, s);
    if (what < 0) return;
    const Turns turns = make_turns<Adjacent>(w, c, s, g.rotated);
    for (int h = h0; h < h1; h += 2) {
        Row8 y[2] = {unpack_row(x[0][0], x[0][1]), unpack_row(x[1][0], x[1][1])};
        load(h + 2);
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            if (h + u < h1) {
                norm_rotate<L, Adjacent>(y[u], turns, weight != nullptr, eps);
                uint2 lo = pack_piece(y[u], 0), hi = pack_piece(y[u], 1);
                if (what == 0) lo = hi = make_uint2(0u, 0u);
                *reinterpret_cast<uint2 *>(dst + g.a) = lo;
                *reinterpret_cast<uint2 *>(dst + g.b) = hi;
            }
            dst += out.hs;
        }
    }
}

template <int L>
__device__ __forceinline__ bool all_lanes(bool ok) {
    const unsigned group = ((1u << L) - 1u) << (threadIdx.x & 31 & ~(L - 1));
    return __all_sync(group, ok);
}

template <int L, bool Adjacent>
__global__ void __launch_bounds__(kHeadThreads, 4) norm_rope_kernel(const __grid_constant__ NormRopeArgs a, int per, int cq,
                                                               int chunks) {
    const int lane = threadIdx.x & (L - 1);
    const int64_t task = (int64_t)blockIdx.x * (kHeadThreads / L) + threadIdx.x / L;
    const int64_t t = task / chunks;
    if (t >= a.tokens) return;
    const int ch = (int)(task - t * chunks);
    const LaneGeo g = lane_geo(lane, a.rope);
    auto rotation = [&](float (&c)[4], float (&s)[4]) {
        const bool ok = all_lanes<L>(load_rotation(a.rope, g, lane, t, a.tokens, -1, c, s));
        if (!ok && lane == 0) report_invalid();
        return ok ? 1 : 0;
    };
    if (ch < cq) {
        const int h0 = ch * per;
        head_rows<L, Adjacent>(a.q, a.q_out, t, h0, min(h0 + per, a.q_heads), a.qw, a.eps, g, rotation);
    } else {
        const int h0 = (ch - cq) * per;
        head_rows<L, Adjacent>(a.k, a.k_out, t, h0, min(h0 + per, a.kv_heads), a.kw, a.eps, g, rotation);
    }
}

// Heads a lane group takes one after another: one while there are few rows
// (latency), up to eight once the GPU is full (the table entries and weights
// are then loaded once for eight heads).
constexpr int kMostPer = 8;
static int heads_per_group(int64_t tokens, int heads, int lanes, int sms) {
    const int64_t groups = (int64_t)sms * 2048 / lanes;
    int per = 1;
    while (per < kMostPer && tokens * heads > groups * per * 2) per *= 2;
    return per;
}

// The same for each of `heads`' chunks.
static int even(int heads, int per) {
    if (heads == 0) return 1;
    const int chunks = (heads + per - 1) / per;
    return (heads + chunks - 1) / chunks;
}

cudaError_t launch_norm_rope(const NormRopeArgs &a, int sms, cudaStream_t stream) {
    const int L = a.dim / 8;
    const int per = even(a.q_heads, heads_per_group(a.tokens, a.q_heads + a.kv_heads, L, sms));
    const int cq = (a.q_heads + per - 1) / per, chunks = cq + (a.kv_heads + per - 1) / per;
    const int64_t blocks = (a.tokens * chunks + kHeadThreads / L - 1) / (kHeadThreads / L);
    const auto kernel = L == 16 ? (a.rope.adjacent ? norm_rope_kernel<16, true> : norm_rope_kernel<16, false>)
                                : (a.rope.adjacent ? norm_rope_kernel<8, true> : norm_rope_kernel<8, false>);
    kernel<<<(unsigned)blocks, kHeadThreads, 0, stream>>>(a, per, cq, chunks);
    return cudaGetLastError();
}

// ------------------------------------------------------------ append
// Four codes on scale s (0: an all-zero block): clamp(rne(fl(y / s))).  The
// quotient itself is only needed near a half: with r = fl(1 / s), y r is within
// |y / s| 2^-22 < 3.1e-5 of it (|y / s| <= 127.5), so an integer that y r is less
// than 0.4999 from is the quotient's nearest.
__device__ __forceinline__ uint32_t codes4(const float *y, float s, float r) {
    constexpr float kMagic = 12582912.f;          // 1.5 * 2^23: the sum's low byte is the integer
    float e[4], off = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        e[i] = fmaf(y[i], r, kMagic);
        off = fmaxf(off, fabsf(fmaf(y[i], r, kMagic - e[i])));
    }
    // r: zero where 1 / s is no normal number
    if (r != 0.f && off < 0.4999f)
        return pack_low_bytes(__float_as_uint(e[0]), __float_as_uint(e[1]), __float_as_uint(e[2]), __float_as_uint(e[3]));
    uint32_t w = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float q = s > 0.f ? rintf(__fdiv_rn(y[i], s)) : 0.f;
        q = fminf(fmaxf(q, -127.f), 127.f);
        w |= ((uint32_t)(int)q & 0xFFu) << (8 * i);
    }
    return w;
}

__device__ __forceinline__ float code_factor(float s) {
    return s >= 1.17549435e-38f && s <= 8.5e37f ? __frcp_rn(s) : 0.f;
}

// rne(q * f) of four codes; f = 2^-j (or 0), so the product is exact.
__device__ __forceinline__ uint32_t rescale4(uint32_t w, float f) {
    uint32_t r = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float q = (float)(int8_t)(w >> (8 * i));
        r |= ((uint32_t)(int)rintf(q * f) & 0xFFu) << (8 * i);
    }
    return r;
}

// The block's scale once values up to `most` join it.  held: the block has
// older tokens, on scale old.  shrink: what their codes are multiplied by.
__device__ __forceinline__ float grow_scale(float most, bool held, float old, float &shrink) {
    shrink = 1.f;
    if (!held) return __fdiv_rn(most, 127.f);
    if (most == 0.f) return old;
    const float r = __fdiv_rn(most, 127.5f * old);
    if (!(old > 0.f) || !(r < 16777216.f)) {       // nothing of the older codes (all below half a step) is left
        shrink = 0.f;
        return __fdiv_rn(most, 127.f);
    }
    if (r < 1.f) return old;
    const int j = ilogbf(r) + 1;
    shrink = __int_as_float((127 - j) << 23);
    return old * __int_as_float((127 + j) << 23);
}

// CTA = 16 rows x L lanes: one block of 16 tokens of one head, keys and
// values together (blockIdx.x < kv_ctas), or chunks of the queries' heads.
// A block is one CTA's so that its scale needs no atomics and comes out the same
// each time.  Measured: 5134 tokens of 5 sequences, 64 / 8 heads of 128 (200 MB)
// 59 us, 52 % of the copy rate; no unit is at its limit (issue slots 66 % busy, DRAM
// 40 %): a CTA has one block of one head, and searches its sequence, length, page
// and coefficients and has every warp work out the block's scale for it.  One
// token for each of 64 sequences is all latency (13 us with the call that reads
// them back).
template <int L, bool Adjacent>
__global__ void __launch_bounds__(16 * L, 64 / L) kv8_append_kernel(const __grid_constant__ AppendArgs a, int64_t kv_ctas, int per,
                                                          int chunks) {
    const int lane = threadIdx.x & (L - 1), row = threadIdx.x / L;
    const LaneGeo g = lane_geo(lane, a.rope);
    const int64_t cap = (int64_t)a.s.max_pages << a.s.page_shift;
    if ((int64_t)blockIdx.x >= kv_ctas) {
        // ---------------------------------------------------- queries
        const int64_t task = ((int64_t)blockIdx.x - kv_ctas) * 16 + row;
        const int64_t t = task / chunks;
        if (t >= a.s.tokens) return;
        const int h0 = (int)(task - t * chunks) * per;
        head_rows<L, Adjacent>(a.q, a.q_out, t, h0, min(h0 + per, a.q_heads), a.qw, a.eps, g,
                     [&](float (&c)[4], float (&s)[4]) {
#pragma unroll
                         for (int i = 0; i < 4; ++i) c[i] = 1.f, s[i] = 0.f;
                         const TokenPlace p = place_token<L>(a.s, t);
                         if (p.b < 0) return -1;                            // behind the last sequence
                         if (p.pos < 0) return 0;                           // padding: zeros
                         const bool ok = all_lanes<L>(load_rotation(a.rope, g, lane, t, a.s.tokens, p.pos, c, s)) && p.pos < cap;
                         if (!ok && lane == 0) report_invalid();
                         return ok ? 1 : 0;
                     });
        return;
    }
    // -------------------------------------------------------- keys, values
    __shared__ float most_k[16], most_v[16];
    const int H = a.c.heads;
    const int64_t slot = blockIdx.x / H;
    const int h = (int)(blockIdx.x - slot * H);
    // sequence b owns the block slots from cu[b] / 16 + 2 b on: enough for
    // its n tokens wherever they start in a block
    int b;
    int64_t t0, n, j;
    if (!a.s.cu) {
        b = (int)slot;
        t0 = slot;
        n = 1;
        j = 0;
    } else {
        b = search_lanes<L>(a.s.batch, slot, [&](int i) { return (int64_t)(__ldg(a.s.cu + i) >> 4) + 2 * (int64_t)i; });
        if (b < 0) {                                 // cu[0] > 0
            if (threadIdx.x == 0) report_invalid();
            return;
        }
        t0 = __ldg(a.s.cu + b);
        n = (int64_t)__ldg(a.s.cu + b + 1) - t0;
        j = slot - ((t0 >> 4) + 2 * (int64_t)b);
        if (t0 < 0 || n < 0 || t0 + n > a.s.tokens || j < 0) {       // j < 0: cu decreases
            if (threadIdx.x == 0) report_invalid();
            return;
        }
    }
    const int64_t len = __ldg(a.s.kv_len + b);
    int64_t first = len - n;
    if (first < 0) first = 0;                               // padding rows in front
    if (first >= len) return;
    const int64_t blk = (first >> 4) + j;
    if (blk * kKvBlock >= len) return;
    if (len > cap) {
        if (threadIdx.x == 0) report_invalid();
        if (blk * kKvBlock >= cap) return;
    }
    const int64_t page = __ldg(a.s.table + (int64_t)b * a.s.max_pages + (blk * kKvBlock >> a.s.page_shift));
    const int64_t pos = blk * kKvBlock + row;
    const bool fresh = pos >= first && pos < len;
    const bool held = blk * kKvBlock < first;               // the block has older tokens
    const int64_t t = t0 + n - (len - pos);
    // the row's values and coefficients are on their way before the page is known
    float k[2][4], v[2][4], w[8], c[4], s[4], mk = 0.f, mv = 0.f;
    uint2 x[4];
    bool ok = true;
    if (fresh) {
        const uint16_t *kp = a.k.p + t * a.k.ts + h * a.k.hs, *vp = a.v.p + t * a.v.ts + h * a.v.hs;
        x[0] = __ldg(reinterpret_cast<const uint2 *>(kp + g.a)), x[1] = __ldg(reinterpret_cast<const uint2 *>(kp + g.b));
        x[2] = __ldg(reinterpret_cast<const uint2 *>(vp + g.a)), x[3] = __ldg(reinterpret_cast<const uint2 *>(vp + g.b));
        load_weight(a.kw, g, w);
        ok = load_rotation(a.rope, g, lane, t, a.s.tokens, pos, c, s);
    }
    if (page < 0 || page >= a.s.pages) {
        if (threadIdx.x == 0) report_invalid();
        return;
    }
    const int blocks = 1 << (a.s.page_shift - 4), in_page = (int)(blk & (blocks - 1));
    const int64_t sc = (page * H + h) * blocks + in_page;
    const float old_k = held ? a.c.ks[sc] : 0.f, old_v = held ? a.c.vs[sc] : 0.f;
    if (fresh) {
        ok = all_lanes<L>(ok);
        Row8 y = unpack_row(x[0], x[1]);
        norm_rotate<L, Adjacent>(y, make_turns<Adjacent>(w, c, s, g.rotated), a.kw != nullptr, a.eps);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            row_piece(y, i, k[i]);
            unpack_bf16x4(x[2 + i], v[i]);
        }
        if (!ok && lane == 0) report_invalid();
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if (!ok) k[i >> 2][i & 3] = 0.f;
            mk = fmaxf(mk, fabsf(k[i >> 2][i & 3]));
            mv = fmaxf(mv, fabsf(v[i >> 2][i & 3]));
        }
    }
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) {
        mk = fmaxf(mk, __shfl_xor_sync(0xffffffffu, mk, o));
        mv = fmaxf(mv, __shfl_xor_sync(0xffffffffu, mv, o));
    }
    if (lane == 0) most_k[row] = mk, most_v[row] = mv;
    __syncthreads();
    mk = most_k[threadIdx.x & 15];
    mv = most_v[threadIdx.x & 15];
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) {
        mk = fmaxf(mk, __shfl_xor_sync(0xffffffffu, mk, o));
        mv = fmaxf(mv, __shfl_xor_sync(0xffffffffu, mv, o));
    }
    float shrink_k, shrink_v;
    const float sk = grow_scale(mk, held, old_k, shrink_k), sv = grow_scale(mv, held, old_v, shrink_v);
    const int64_t at = (sc * kKvBlock + row) * a.c.dim;
    int8_t *kq = a.c.k + at, *vq = a.c.v + at;
    if (fresh) {
        const float rk = code_factor(sk), rv = code_factor(sv);
        *reinterpret_cast<uint32_t *>(kq + g.a) = codes4(k[0], sk, rk);
        *reinterpret_cast<uint32_t *>(kq + g.b) = codes4(k[1], sk, rk);
        *reinterpret_cast<uint32_t *>(vq + g.a) = codes4(v[0], sv, rv);
        *reinterpret_cast<uint32_t *>(vq + g.b) = codes4(v[1], sv, rv);
    } else if (pos < first) {
        if (shrink_k != 1.f) {
            uint2 *p = reinterpret_cast<uint2 *>(kq + 8 * lane);
            const uint2 w = *p;
            *p = make_uint2(rescale4(w.x, shrink_k), rescale4(w.y, shrink_k));
        }
        if (shrink_v != 1.f) {
            uint2 *p = reinterpret_cast<uint2 *>(vq + 8 * lane);
            const uint2 w = *p;
            *p = make_uint2(rescale4(w.x, shrink_v), rescale4(w.y, shrink_v));
        }
    }
    if (threadIdx.x == 0) a.c.ks[sc] = sk, a.c.vs[sc] = sv;
}

cudaError_t launch_kv8_append(const AppendArgs &a, int sms, cudaStream_t stream) {
    const int L = a.c.dim / 8;
    const int64_t slots = a.s.cu ? a.s.tokens / kKvBlock + 2 * (int64_t)a.s.batch : a.s.batch;
    const int64_t kv_ctas = slots * a.c.heads;
    const int per = even(a.q_heads, heads_per_group(a.s.tokens, a.q_heads, L, sms));
    const int chunks = (a.q_heads + per - 1) / per;
    const int64_t blocks = kv_ctas + (a.s.tokens * chunks + 15) / 16;
    const auto kernel = L == 16 ? (a.rope.adjacent ? kv8_append_kernel<16, true> : kv8_append_kernel<16, false>)
                                : (a.rope.adjacent ? kv8_append_kernel<8, true> : kv8_append_kernel<8, false>);
    kernel<<<(unsigned)blocks, 16 * L, 0, stream>>>(a, kv_ctas, per, chunks);
    return cudaGetLastError();
}

// ------------------------------------------------------------ read
// Eight codes to BF16: fl(q * s) rounded once more to BF16.
__device__ __forceinline__ uint4 dequant8(const uint2 &w, float s) {
    const uint32_t x[2] = {w.x, w.y};
    uint32_t r[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t b = x[i >> 1] >> (16 * (i & 1));
        r[i] = pack_bf16x2((float)(int8_t)b * s, (float)(int8_t)(b >> 8) * s);
    }
    return make_uint4(r[0], r[1], r[2], r[3]);
}

// Bound by memory: 8 sequences of up to 4096 tokens, 8 heads of 128 (150 MB) 29.7
// us, 77 % of the copy rate; one head at a time instead of four 34 us.
template <int L>
__global__ void __launch_bounds__(kHeadThreads) kv8_read_kernel(const __grid_constant__ ReadArgs a, int per, int chunks) {
    const int lane = threadIdx.x & (L - 1);
    const int64_t task = (int64_t)blockIdx.x * (kHeadThreads / L) + threadIdx.x / L;
    const int64_t t = task / chunks;
    if (t >= a.s.tokens) return;
    // cu that is no partition of the rows: seen by one thread, whether or not a row meets it
    if (a.s.cu && task == 0 && lane == 0 && (__ldg(a.s.cu) != 0 || __ldg(a.s.cu + a.s.batch) > a.s.tokens)) report_invalid();
    const TokenPlace p = place_token<L>(a.s, t);
    if (p.b < 0) return;
    const int H = a.c.heads, D = 8 * L;
    int64_t page = -1;
    if (p.pos >= 0) {
        if (p.pos < (int64_t)a.s.max_pages << a.s.page_shift)
            page = __ldg(a.s.table + (int64_t)p.b * a.s.max_pages + (p.pos >> a.s.page_shift));
        if (page < 0 || page >= a.s.pages) {
            if (lane == 0) report_invalid();
            page = -1;
        }
    }
    const int in_page = (int)(p.pos & ((1 << a.s.page_shift) - 1));
    const int h0 = (int)(task - t * chunks) * per, h1 = min(h0 + per, H);
    constexpr int U = 4;                  // heads in flight
    for (int h = h0; h < h1; h += U) {
        uint2 kc[U], vc[U];
        float ks[U], vs[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            kc[u] = vc[u] = make_uint2(0u, 0u);
            ks[u] = vs[u] = 0.f;
            if (page >= 0 && h + u < h1) {
                const int64_t r = ((page * H + h + u) << a.s.page_shift) + in_page;
                ks[u] = __ldg(a.c.ks + (r >> 4));
                vs[u] = __ldg(a.c.vs + (r >> 4));
                kc[u] = __ldg(reinterpret_cast<const uint2 *>(a.c.k + r * D) + lane);
                vc[u] = __ldg(reinterpret_cast<const uint2 *>(a.c.v + r * D) + lane);
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (h + u < h1) {
                const int64_t o = (t * H + h + u) * L + lane;
                if (a.k_out) reinterpret_cast<uint4 *>(a.k_out)[o] = dequant8(kc[u], ks[u]);
                if (a.v_out) reinterpret_cast<uint4 *>(a.v_out)[o] = dequant8(vc[u], vs[u]);
            }
    }
}

cudaError_t launch_kv8_read(const ReadArgs &a, int sms, cudaStream_t stream) {
    const int L = a.c.dim / 8;
    const int per = heads_per_group(a.s.tokens, a.c.heads, L, sms);
    const int chunks = (a.c.heads + per - 1) / per;
    const int64_t blocks = (a.s.tokens * chunks + kHeadThreads / L - 1) / (kHeadThreads / L);
    if (L == 16)
        kv8_read_kernel<16><<<(unsigned)blocks, kHeadThreads, 0, stream>>>(a, per, chunks);
    else
        kv8_read_kernel<8><<<(unsigned)blocks, kHeadThreads, 0, stream>>>(a, per, chunks);
    return cudaGetLastError();
}

}  // namespace convrot
