// Rotary positions, and per-head norms of queries and keys with the rotation in
// the same pass (into the caches, and backward).
//
// Pair i of a head at position p turns by theta_i = p * freq_i:
//     (a, b) -> mscale * (a cos - b sin, b cos + a sin)
// with (a, b) = dims (i, i + rot/2) of the head (half layout) or (2i, 2i + 1)
// (interleaved), i < rot/2; dims from rot on are left as they are.  Far positions
// need more than fp32: at p = 10^6 an fp32 product is off by up to 0.03 rad.  So
// the turns p * freq / 2 pi are formed and reduced to [-1/2, 1/2] in fp64 (two
// operations a pair, once for all heads of a token), and the sine and cosine are
// taken of the reduced fp32 value in half turns (about 1e-7 absolute).
//
// Everything here is bound by HBM: each element is read and written once.  A group
// of D / (2 VEC) lanes owns one token (and a run of its heads): a lane holds VEC
// pairs, i.e. two 16-byte vectors, chosen so that both halves of each pair are in
// its registers: no exchange, and the same VEC angles serve either layout and
// every head.  A head's sum of squares is log2(lanes) shuffles.
#include <math.h>

#include "qsa_common.cuh"
#include "qsa_launch.h"

namespace qsa {

namespace rope {

constexpr int THREADS = 256;
// The plain rotation: vectors of 4 (with 8, in bf16, 98 registers a thread left two blocks an SM:
// 8 x 900 tokens of 16 heads of 128 15.0 us, with 4 13.0), and head rows whose loads are issued
// together.  On tensors that are not in L2 that call is 14.4 us, 32K tokens are 47 us: 1.6 and
// 1.15 times the time of their bytes at a copy's rate; the short one's rest is its launch.
constexpr int ROPE_VEC = 4;
template <typename T>
constexpr int ROPE_ROWS = sizeof(T) == 4 ? 2 : 4;
constexpr double INV_2PI = 0.15915494309189533576888376337251;

template <typename T, int VEC>
struct Raw;
template <>
struct Raw<uint16_t, 4> {
    uint2 v;
    QSA_DEVICE void load(const uint16_t *p) { v = *reinterpret_cast<const uint2 *>(p); }
    QSA_DEVICE void store(uint16_t *p) const { *reinterpret_cast<uint2 *>(p) = v; }
    QSA_DEVICE void get(float (&f)[4]) const {
        f[0] = bf16_lo(v.x);
        f[1] = bf16_hi(v.x);
        f[2] = bf16_lo(v.y);
        f[3] = bf16_hi(v.y);
    }
    QSA_DEVICE void set(const float (&f)[4]) {
        v = make_uint2(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]));
    }
};
template <int VEC>
struct Raw<float, VEC> {
    float4 v[VEC / 4];
    QSA_DEVICE void load(const float *p) {
#pragma unroll
        for (int i = 0; i < VEC / 4; ++i) v[i] = reinterpret_cast<const float4 *>(p)[i];
    }
    QSA_DEVICE void store(float *p) const {
#pragma unroll
        for (int i = 0; i < VEC / 4; ++i) reinterpret_cast<float4 *>(p)[i] = v[i];
    }
    QSA_DEVICE void get(float (&f)[VEC]) const {
#pragma unroll
        for (int i = 0; i < VEC / 4; ++i) {
            f[4 * i] = v[i].x;
            f[4 * i + 1] = v[i].y;
            f[4 * i + 2] = v[i].z;
            f[4 * i + 3] = v[i].w;
        }
    }
    QSA_DEVICE void set(const float (&f)[VEC]) {
#pragma unroll
        for (int i = 0; i < VEC / 4; ++i)
            v[i] = make_float4(f[4 * i], f[4 * i + 1], f[4 * i + 2], f[4 * i + 3]);
    }
};

// What a lane of a head's group holds: vectors at dims da and db, pairs
// f0 .. f0 + VEC - 1 of the frequency table if `turns`.
template <int VEC, bool HALF>
struct Lane {
    int da, db, f0;
    bool turns;
    QSA_DEVICE Lane(int lane, int rot) {
        const int nr = rot / (2 * VEC);  // lanes that hold rotated pairs
        turns = lane < nr;
        f0 = lane * VEC;
        da = HALF && turns ? lane * VEC : 2 * lane * VEC;
        db = HALF && turns ? lane * VEC + rot / 2 : da + VEC;
    }
};

template <int VEC>
QSA_DEVICE void load_turns(const double *freq, int f0, bool turns, double (&tf)[VEC]) {
#pragma unroll
    for (int e = 0; e < VEC; ++e) tf[e] = turns ? freq[f0 + e] * INV_2PI : 0.0;
}

// cos and sin of this token's angles, times mscale; sin negated for the transpose.
template <int VEC>
QSA_DEVICE void angles(int64_t p, const double (&tf)[VEC], bool turns, float mscale, float sign,
                       float (&c)[VEC], float (&s)[VEC]) {
    const double dp = (double)p;
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
        const double t = dp * tf[e];
        const float r = (float)(t - rint(t));
        float sn, cs;
        sincospif(2.f * r, &sn, &cs);
        c[e] = turns ? cs * mscale : 1.f;
        s[e] = turns ? sn * mscale * sign : 0.f;
    }
}

template <int VEC, bool HALF>
QSA_DEVICE void rotate(float (&a)[VEC], float (&b)[VEC], const float (&c)[VEC],
                       const float (&s)[VEC]) {
    if (HALF) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            const float x = a[e], y = b[e];
            a[e] = x * c[e] - y * s[e];
            b[e] = y * c[e] + x * s[e];
        }
    } else {
#pragma unroll
        for (int e = 0; e < VEC / 2; ++e) {
            const float x = a[2 * e], y = a[2 * e + 1];
            a[2 * e] = x * c[e] - y * s[e];
            a[2 * e + 1] = y * c[e] + x * s[e];
            const float z = b[2 * e], w = b[2 * e + 1];
            b[2 * e] = z * c[VEC / 2 + e] - w * s[VEC / 2 + e];
            b[2 * e + 1] = w * c[VEC / 2 + e] + z * s[VEC / 2 + e];
        }
    }
}

template <int VEC>
QSA_DEVICE void load_weight(const float *w, int d, float (&f)[VEC]) {
#pragma unroll
    for (int i = 0; i < VEC / 4; ++i) {
        const float4 v = __ldg(reinterpret_cast<const float4 *>(w + d) + i);
        f[4 * i] = v.x;
        f[4 * i + 1] = v.y;
        f[4 * i + 2] = v.z;
        f[4 * i + 3] = v.w;
    }
}

struct Pos {
    const int64_t *pos;   // [B, T] or nullptr
    const int64_t *pos0;  // [B] or nullptr
    QSA_DEVICE int64_t at(int64_t tok, int64_t T) const {
        if (pos) return pos[tok];
        const int64_t b = tok / T;
        return (pos0 ? pos0[b] : 0) + (tok - b * T);
    }
};

// ------------------------------------------------------------- rotation --
struct RopeArgs {
    const void *x;
    void *y;
    int64_t xs, ys;  // elements between tokens
    int64_t T, n_tok;
    int H, D, rot, lanes;
    int hpg, n_hg;   // heads per item, items per token
    const double *freq;
    float mscale, sign;
    Pos pos;
};

template <typename T, bool HALF>
__global__ void __launch_bounds__(THREADS) rope_kernel(const RopeArgs a) {
    constexpr int VEC = ROPE_VEC, ROWS = ROPE_ROWS<T>;
    const int lane = threadIdx.x % a.lanes;
    const Lane<VEC, HALF> L(lane, a.rot);
    double tf[VEC];
    load_turns<VEC>(a.freq, L.f0, L.turns, tf);
    const int64_t per_block = blockDim.x / a.lanes;
    const int64_t items = a.n_tok * a.n_hg;
    for (int64_t it = blockIdx.x * per_block + threadIdx.x / a.lanes; it < items;
         it += gridDim.x * per_block) {
        const int64_t tok = it / a.n_hg;
        const int h0 = (int)(it - tok * a.n_hg) * a.hpg;
        const int h1 = min(h0 + a.hpg, a.H);
        float c[VEC], s[VEC];
        angles<VEC>(a.pos.at(tok, a.T), tf, L.turns, a.mscale, a.sign, c, s);
        const T *x = static_cast<const T *>(a.x) + tok * a.xs;
        T *y = static_cast<T *>(a.y) + tok * a.ys;
        for (int h = h0; h < h1; h += ROWS) {
            Raw<T, VEC> ra[ROWS], rb[ROWS];
#pragma unroll
            for (int r = 0; r < ROWS; ++r)
                if (h + r < h1) {
                    ra[r].load(x + (int64_t)(h + r) * a.D + L.da);
                    rb[r].load(x + (int64_t)(h + r) * a.D + L.db);
                }
#pragma unroll
            for (int r = 0; r < ROWS; ++r)
                if (h + r < h1) {
                    if (L.turns) {
                        float fa[VEC], fb[VEC];
                        ra[r].get(fa);
                        rb[r].get(fb);
                        rotate<VEC, HALF>(fa, fb, c, s);
                        ra[r].set(fa);
                        rb[r].set(fb);
                    }
                    ra[r].store(y + (int64_t)(h + r) * a.D + L.da);
                    rb[r].store(y + (int64_t)(h + r) * a.D + L.db);
                }
        }
    }
}

// ---------------------------------------------------- norm and rotation --
// Both kernels below stream rows (one head of one token): a group of lanes takes an item
// (a token, or a batch of its rows) and its batches of rows one after the other, so that
// one set of angles serves all of them.  Rows come through a ring in shared memory that
// belongs to the thread alone (cp.async, no barrier), STAGES batches deep: registers hold
// one batch, and enough bytes are in flight for HBM whatever the occupancy.  What bounds
// the kernels beyond that is the issue of instructions: so D is a template argument and
// the batches are unrolled (offsets are immediates), and the arithmetic is in packed pairs
// of fp32.  32K tokens, 16 + 2 heads of 128, forward / backward with fp32 gradients, a few
// calls at the full clock: rows from registers 84 / 195 us, a ring of single rows 66 / 164 us,
// this 62.5 / 134 us (5.4 and 5.6 TB/s of a copy's 6.5).  Call after call for a second, the power
// limit takes the clock to 1.85 / 1.75 GHz and the calls to 66 / 138 us.

// Packed fp32 pairs.
struct F2 {
    uint64_t v;
};
QSA_DEVICE F2 pack2(float a, float b) {
    F2 x;
    asm("mov.b64 %0, {%1, %2};\n" : "=l"(x.v) : "f"(a), "f"(b));
    return x;
}
QSA_DEVICE float2 unpack2(F2 x) {
    float2 f;
    asm("mov.b64 {%0, %1}, %2;\n" : "=f"(f.x), "=f"(f.y) : "l"(x.v));
    return f;
}
QSA_DEVICE F2 swap2(F2 x) {
    const float2 f = unpack2(x);
    return pack2(f.y, f.x);
}
QSA_DEVICE F2 fma2(F2 a, F2 b, F2 c) {
    F2 d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;\n" : "=l"(d.v) : "l"(a.v), "l"(b.v), "l"(c.v));
    return d;
}
QSA_DEVICE F2 mul2(F2 a, F2 b) {
    F2 d;
    asm("mul.rn.f32x2 %0, %1, %2;\n" : "=l"(d.v) : "l"(a.v), "l"(b.v));
    return d;
}
QSA_DEVICE float sum2(F2 x) {
    const float2 f = unpack2(x);
    return f.x + f.y;
}

// VEC elements as they lie in memory; cp.async into shared memory and back.
template <typename T, int VEC>
struct Line {
    static constexpr int BYTES = VEC * (int)sizeof(T);
    uint32_t w[BYTES / 4];
    QSA_DEVICE static void copy(uint32_t dst, const T *src) {
        if (BYTES == 8)
            asm volatile("cp.async.ca.shared.global [%0], [%1], 8;\n" ::"r"(dst), "l"(src)
                         : "memory");
        else
#pragma unroll
            for (int i = 0; i < BYTES / 16; ++i)
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16;\n" ::"r"(dst + i * 16),
                             "l"(src + i * (16 / (int)sizeof(T)))
                             : "memory");
    }
    QSA_DEVICE void fetch(const uint8_t *p) {
        if (BYTES == 8) {
            const uint2 v = *reinterpret_cast<const uint2 *>(p);
            w[0] = v.x;
            w[1] = v.y;
        } else {
#pragma unroll
            for (int i = 0; i < BYTES / 16; ++i) {
                const uint4 v = reinterpret_cast<const uint4 *>(p)[i];
                w[4 * i] = v.x;
                w[4 * i + 1] = v.y;
                w[4 * i + 2] = v.z;
                w[4 * i + 3] = v.w;
            }
        }
    }
    QSA_DEVICE void store(T *p) const {
        if (BYTES == 8)
            *reinterpret_cast<uint2 *>(p) = make_uint2(w[0], w[1]);
        else
#pragma unroll
            for (int i = 0; i < BYTES / 16; ++i)
                reinterpret_cast<uint4 *>(p)[i] =
                    make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
    }
    QSA_DEVICE F2 get(int i) const {  // elements 2 i and 2 i + 1
        if (sizeof(T) == 2) return pack2(bf16_lo(w[i]), bf16_hi(w[i]));
        return pack2(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1]));
    }
    QSA_DEVICE void set(int i, F2 x) {
        const float2 f = unpack2(x);
        if (sizeof(T) == 2) {
            w[i] = pack_bf16x2(f.x, f.y);
        } else {
            w[2 * i] = __float_as_uint(f.x);
            w[2 * i + 1] = __float_as_uint(f.y);
        }
    }
};

// A lane's turned pair of vectors: a' = k0 a + k1 x, b' = k2 b + k3 y, where (x, y) is
// (b, a) in the half layout and (a, b) with each pair swapped in the interleaved one.
// Lanes beyond the rotated dims only scale by k0 and k2: a zero times the other half's
// infinity must not reach them.
template <int VEC, bool HALF>
struct Turn {
    F2 k0[VEC / 2], k1[VEC / 2], k2[VEC / 2], k3[VEC / 2];
    // cosines and sines of the lane's pairs (sines negated for the transpose), times what
    // each element is scaled by before it is turned
    QSA_DEVICE void set(const float (&c)[VEC], const float (&s)[VEC], const float (&wa)[VEC],
                        const float (&wb)[VEC], bool turns) {
#pragma unroll
        for (int i = 0; i < VEC / 2; ++i) {
            const int e = 2 * i, f = 2 * i + 1;
            if (!turns) {
                k0[i] = pack2(wa[e], wa[f]);
                k2[i] = pack2(wb[e], wb[f]);
                k1[i] = k3[i] = pack2(0.f, 0.f);
            } else if (HALF) {
                k0[i] = pack2(c[e] * wa[e], c[f] * wa[f]);
                k1[i] = pack2(-s[e] * wb[e], -s[f] * wb[f]);
                k2[i] = pack2(c[e] * wb[e], c[f] * wb[f]);
                k3[i] = pack2(s[e] * wa[e], s[f] * wa[f]);
            } else {
                const float ca = c[i], sa = s[i], cb = c[VEC / 2 + i], sb = s[VEC / 2 + i];
                k0[i] = pack2(ca * wa[e], ca * wa[f]);
                k1[i] = pack2(-sa * wa[f], sa * wa[e]);
                k2[i] = pack2(cb * wb[e], cb * wb[f]);
                k3[i] = pack2(-sb * wb[f], sb * wb[e]);
            }
        }
    }
    QSA_DEVICE void apply(int i, F2 a, F2 b, bool turns, F2 &ya, F2 &yb) const {
        ya = mul2(k0[i], a);
        yb = mul2(k2[i], b);
        if (turns) {
            ya = fma2(k1[i], HALF ? b : swap2(a), ya);
            yb = fma2(k3[i], HALF ? a : swap2(b), yb);
        }
    }
};

// Sum over a group of LANES lanes; whole warps.
template <int LANES>
QSA_DEVICE float lanes_sum(float x) {
#pragma unroll
    for (int o = LANES / 2; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

// Batches of rows of a group in order: items it, it + stride, ..., batches 0 .. hpb - 1 of
// each, batch `at` of the token.
struct Batches {
    int64_t it, tok;
    int n, at;
    bool live;    // the item is one
    QSA_DEVICE void locate(int64_t items, int hpb, int n_hg) {
        live = it < items;
        n = at = 0;
        tok = it;
        if (n_hg > 1) {
            tok = it / n_hg;
            at = (int)(it - tok * n_hg) * hpb;
        }
    }
    QSA_DEVICE bool next(int64_t stride, int64_t items, int hpb, int n_hg) {
        ++at;
        if (++n < hpb) return false;
        it += stride;
        locate(items, hpb, n_hg);
        return true;
    }
};

// Turns per position of the frequency table, p * freq / 2 pi, once per block.
QSA_DEVICE void load_table(const double *freq, int rot, double *s_tf) {
    for (int i = threadIdx.x; i < rot / 2; i += blockDim.x) s_tf[i] = freq[i] * INV_2PI;
    __syncthreads();
}

template <int VEC>
QSA_DEVICE void table_angles(int64_t p, const double *s_tf, int f0, bool turns, float mscale,
                             float sign, float (&c)[VEC], float (&s)[VEC]) {
    double tf[VEC];
#pragma unroll
    for (int e = 0; e < VEC; ++e) tf[e] = turns ? s_tf[f0 + e] : 0.0;
    angles<VEC>(p, tf, turns, mscale, sign, c, s);
}

// Asks for a sector of an array (or of none) and does not wait for it.
QSA_DEVICE void warm(const float *p, int i) {
    if (p)
        asm volatile("{\n\t.reg .b32 x;\n\tld.global.ca.b32 x, [%0];\n\t}\n" ::"l"(p + i)
                     : "memory");
}

struct NormArgs {
    const uint16_t *x[3];        // queries, keys, values
    int64_t xs[3];               // elements between tokens
    uint16_t *y[3];
    const float *w[3];           // [D] or nullptr (no norm)
    int H[3], first[3];          // rows; first batch of a token
    const int64_t *slot;         // [B, T] cache rows, or nullptr (row = token)
    int64_t L;                   // cache rows per sequence
    int64_t T, n_tok;
    int rot;
    int batches, hpb, n_hg;      // batches of a token, per item, items of a token
    float eps;
    const double *freq;
    float mscale;
    Pos pos;
    void *status;
};

constexpr int NORM_ROWS = 4, NORM_STAGES = 3, NORM_CTAS = 2;  // rows of a batch

template <int D, int VEC, bool HALF>
__global__ void __launch_bounds__(THREADS, NORM_CTAS) norm_rope_kernel(const NormArgs a) {
    using X = Line<uint16_t, VEC>;
    constexpr int LANES = D / (2 * VEC), RB = NORM_ROWS, S = NORM_STAGES;
    constexpr int HB = X::BYTES * THREADS, STAGE = 2 * HB * RB;
    extern __shared__ __align__(16) uint8_t ring[];
    __shared__ double s_tf[128];
    const int lane = threadIdx.x % LANES;
    const Lane<VEC, HALF> L(lane, a.rot);
    const int per_block = blockDim.x / LANES;
    const int64_t stride = (int64_t)gridDim.x * per_block;
    const int64_t items = a.n_tok * a.n_hg;
    // the weights into L1, for when the first rows have come
    for (int i = threadIdx.x; i < D / 8; i += blockDim.x) {
        warm(a.w[0], i * 8);
        warm(a.w[1], i * 8);
    }
    // whole warps stay in the loop (the sums are shuffles): as long as their first group
    const int64_t wfirst = (int64_t)blockIdx.x * per_block + (threadIdx.x & ~31) / LANES;
    const int steps = wfirst < items ? (int)((items - wfirst + stride - 1) / stride) * a.hpb : 0;
    Batches in, out;
    in.it = (int64_t)blockIdx.x * per_block + threadIdx.x / LANES;
    in.locate(items, a.hpb, a.n_hg);
    out = in;
    uint8_t *mine = ring + threadIdx.x * X::BYTES;
    const uint32_t mine32 = smem_u32(mine);
    // which tensor a batch is of
    auto part = [&](int at) { return at < a.first[1] ? 0 : at < a.first[2] ? 1 : 2; };
    int fill = 0, fslot = 0;
    auto prefetch = [&]() {
        if (fill < steps && in.live && in.at < a.batches) {
            const int t = part(in.at), r0 = (in.at - a.first[t]) * RB, cnt = a.H[t] - r0;
            const uint16_t *x = a.x[t] + in.tok * a.xs[t] + r0 * D;
            const uint32_t d = mine32 + fslot;
#pragma unroll
            for (int r = 0; r < RB; ++r)
                if (r < cnt) {
                    X::copy(d + r * 2 * HB, x + r * D + L.da);
                    X::copy(d + r * 2 * HB + HB, x + r * D + L.db);
                }
        }
        cp_async_commit();
        ++fill;
        fslot = fslot == (S - 1) * STAGE ? 0 : fslot + STAGE;
        in.next(stride, items, a.hpb, a.n_hg);
    };
#pragma unroll
    for (int n = 0; n < S - 1; ++n) prefetch();
    auto position = [&](const Batches &w) { return w.live ? a.pos.at(w.tok, a.T) : 0; };
    auto slot = [&](const Batches &w) { return a.slot && w.live ? a.slot[w.tok] : 0; };
    // the next item's position and slot are read an item ahead
    int64_t p = position(out), sl = slot(out), orow = 0;
    load_table(a.freq, a.rot, s_tf);
    float c[VEC], s[VEC];
    Turn<VEC, HALF> turn;
    int of = -1;  // whose weight is in `turn`
    int at = 0;
    bool fresh = true;
    for (int n = 0; n < steps; ++n) {
        cp_async_wait<S - 2>();
        if (fresh) {
            table_angles<VEC>(p, s_tf, L.f0, L.turns, a.mscale, 1.f, c, s);
            orow = out.tok;  // row of the key and value outputs, or -1: not written
            if (a.slot) {
                orow = sl >= 0 && sl < a.L ? (a.n_tok == a.T ? 0 : out.tok / a.T * a.L) + sl : -1;
                if (sl >= a.L && lane == 0 && out.live) record_status(a.status, QSA_ERR_DEVICE);
            }
            of = -1;
            Batches w = out;
            w.it += stride;
            w.locate(items, a.hpb, a.n_hg);
            p = position(w);
            sl = slot(w);
        }
        const bool on = out.live && out.at < a.batches;
        const int t = on ? part(out.at) : 2;
        const int r0 = on ? (out.at - a.first[t]) * RB : 0;
        const int cnt = on && (t == 0 || orow >= 0) ? a.H[t] - r0 : 0;  // rows to write
        X xa[RB], xb[RB];
#pragma unroll
        for (int r = 0; r < RB; ++r) {
            xa[r].fetch(mine + at + r * 2 * HB);
            xb[r].fetch(mine + at + r * 2 * HB + HB);
        }
        const float *w = a.w[t];
        float rs[RB];
        if (__any_sync(0xffffffffu, w != nullptr)) {
#pragma unroll
            for (int r = 0; r < RB; ++r) {
                F2 ss = pack2(0.f, 0.f);
#pragma unroll
                for (int i = 0; i < VEC / 2; ++i) {
                    const F2 fa = xa[r].get(i), fb = xb[r].get(i);
                    ss = fma2(fa, fa, ss);
                    ss = fma2(fb, fb, ss);
                }
                rs[r] = rsqrtf(lanes_sum<LANES>(sum2(ss)) * (1.f / D) + a.eps);
            }
        }
        if (t != 2) {
            if (of != t) {
                of = t;
                float wa[VEC], wb[VEC];
#pragma unroll
                for (int e = 0; e < VEC; ++e) wa[e] = wb[e] = 1.f;
                if (w) {
                    load_weight<VEC>(w, L.da, wa);
                    load_weight<VEC>(w, L.db, wb);
                }
                turn.set(c, s, wa, wb, L.turns);
            }
#pragma unroll
            for (int r = 0; r < RB; ++r) {
                const float f = w ? rs[r] : 1.f;
                const F2 f2 = pack2(f, f);
#pragma unroll
                for (int i = 0; i < VEC / 2; ++i) {
                    F2 ya, yb;
                    turn.apply(i, xa[r].get(i), xb[r].get(i), L.turns, ya, yb);
                    xa[r].set(i, mul2(ya, f2));
                    xb[r].set(i, mul2(yb, f2));
                }
            }
        }
        uint16_t *y = a.y[t] + ((t == 0 ? out.tok : orow) * a.H[t] + r0) * D;
#pragma unroll
        for (int r = 0; r < RB; ++r)
            if (r < cnt) {
                xa[r].store(y + r * D + L.da);
                xb[r].store(y + r * D + L.db);
            }
        prefetch();
        at = at == (S - 1) * STAGE ? 0 : at + STAGE;
        fresh = out.next(stride, items, a.hpb, a.n_hg);
    }
    cp_async_wait<0>();
}

// ------------------------------------------------------------- backward --
// With z = x r w (r = 1 / sqrt(mean x^2 + eps)), y = mscale R z and u = w dz:
//   dz = mscale R^T dy,  dw = sum dz x r,  dx = r (u - x r mean(u x r)).
// Blocks belong to the queries or to the keys, so a thread keeps the sums of one
// weight in registers over all its rows; block partials go to the workspace and
// are added in a fixed order by weight_sum_kernel: the same bits on every run.
struct Side {
    const void *dy;
    const uint16_t *x;
    int64_t xs;
    void *dx;
    const float *w;
    int H, batches, hpb, n_hg;
};
struct GradArgs {
    Side side[2];        // queries, keys
    int n_blocks_q;      // blocks before this one work on the queries
    int64_t T, n_tok;
    int rot;
    float eps;
    const double *freq;
    float mscale;
    Pos pos;
    float *part;         // [blocks, D]
};

// Vectors of 4: fp32 gradients fill 16 bytes a lane (with 8 a lane's two loads would each
// touch half of every sector; 195 -> 176 us before the ring).
constexpr int GRAD_VEC = 4, GRAD_ROWS = 2, GRAD_STAGES = 4, GRAD_CTAS = 2;
template <typename TD>
constexpr int grad_stage() { return 2 * GRAD_VEC * ((int)sizeof(TD) + 2) * GRAD_ROWS * THREADS; }

template <int D, bool HALF, typename TD, typename TX>
__global__ void __launch_bounds__(THREADS, GRAD_CTAS) norm_rope_grad_kernel(const GradArgs a) {
    constexpr int VEC = GRAD_VEC, LANES = D / (2 * VEC), RB = GRAD_ROWS, S = GRAD_STAGES;
    using G = Line<TD, VEC>;
    using X = Line<uint16_t, VEC>;
    constexpr int GB = G::BYTES * THREADS, XB = X::BYTES * THREADS, ROW = 2 * (GB + XB);
    constexpr int STAGE = ROW * RB;
    extern __shared__ __align__(16) uint8_t ring[];
    __shared__ double s_tf[128];
    __shared__ float s_dw[THREADS / 32][D];
    const bool isq = (int)blockIdx.x < a.n_blocks_q;
    const Side &sd = a.side[isq ? 0 : 1];
    const int blk = isq ? blockIdx.x : blockIdx.x - a.n_blocks_q;
    const int n_blk = isq ? a.n_blocks_q : gridDim.x - a.n_blocks_q;
    const int lane = threadIdx.x % LANES;
    const Lane<VEC, HALF> L(lane, a.rot);
    float wa[VEC], wb[VEC];
#pragma unroll
    for (int e = 0; e < VEC; ++e) wa[e] = wb[e] = 0.f;
    const bool norm = sd.w != nullptr;
    if (norm) {
        load_weight<VEC>(sd.w, L.da, wa);
        load_weight<VEC>(sd.w, L.db, wb);
    }
    F2 ga[VEC / 2], gb[VEC / 2], w2a[VEC / 2], w2b[VEC / 2];
#pragma unroll
    for (int i = 0; i < VEC / 2; ++i) {
        ga[i] = gb[i] = pack2(0.f, 0.f);
        w2a[i] = pack2(wa[2 * i], wa[2 * i + 1]);
        w2b[i] = pack2(wb[2 * i], wb[2 * i + 1]);
    }
    constexpr int per_block = THREADS / LANES;
    const int64_t stride = (int64_t)n_blk * per_block;
    const int H = sd.H, hpb = sd.hpb, n_hg = sd.n_hg;
    const int64_t items = a.n_tok * n_hg;
    const int64_t wfirst = (int64_t)blk * per_block + (threadIdx.x & ~31) / LANES;
    const int steps = wfirst < items ? (int)((items - wfirst + stride - 1) / stride) * hpb : 0;
    Batches in, out;
    in.it = (int64_t)blk * per_block + threadIdx.x / LANES;
    in.locate(items, hpb, n_hg);
    out = in;
    uint8_t *mg = ring + threadIdx.x * G::BYTES, *mx = ring + 2 * GB + threadIdx.x * X::BYTES;
    const uint32_t mg32 = smem_u32(mg), mx32 = smem_u32(mx);
    int fill = 0, fslot = 0;
    auto prefetch = [&]() {
        if (fill < steps && in.live) {
            const int r0 = in.at * RB, cnt = H - r0;
            const TD *d = static_cast<const TD *>(sd.dy) + (in.tok * H + r0) * D;
            const uint16_t *x = sd.x + in.tok * sd.xs + r0 * D;
#pragma unroll
            for (int r = 0; r < RB; ++r)
                if (r < cnt) {
                    G::copy(mg32 + fslot + r * ROW, d + r * D + L.da);
                    G::copy(mg32 + fslot + r * ROW + GB, d + r * D + L.db);
                    X::copy(mx32 + fslot + r * ROW, x + r * D + L.da);
                    X::copy(mx32 + fslot + r * ROW + XB, x + r * D + L.db);
                }
        }
        cp_async_commit();
        ++fill;
        fslot = fslot == (S - 1) * STAGE ? 0 : fslot + STAGE;
        in.next(stride, items, hpb, n_hg);
    };
#pragma unroll
    for (int n = 0; n < S - 1; ++n) prefetch();
    auto position = [&](const Batches &w) { return w.live ? a.pos.at(w.tok, a.T) : 0; };
    int64_t p = position(out);
    load_table(a.freq, a.rot, s_tf);
    int at = 0;
    Turn<VEC, HALF> turn;
    bool fresh = true;
    for (int n = 0; n < steps; ++n) {
        cp_async_wait<S - 2>();
        if (fresh) {
            float c[VEC], s[VEC], one[VEC];
            table_angles<VEC>(p, s_tf, L.f0, L.turns, a.mscale, -1.f, c, s);
#pragma unroll
            for (int e = 0; e < VEC; ++e) one[e] = 1.f;
            turn.set(c, s, one, one, L.turns);
            Batches w = out;
            w.it += stride;
            w.locate(items, hpb, n_hg);
            p = position(w);
        }
        const int r0 = out.at * RB, cnt = out.live ? H - r0 : 0;
        F2 za[RB][VEC / 2], zb[RB][VEC / 2];
        X xa[RB], xb[RB];
        float ss[RB], mm[RB];
#pragma unroll
        for (int r = 0; r < RB; ++r) {
            G da, db;
            da.fetch(mg + at + r * ROW);
            db.fetch(mg + at + r * ROW + GB);
            xa[r].fetch(mx + at + r * ROW);
            xb[r].fetch(mx + at + r * ROW + XB);
            F2 s2 = pack2(0.f, 0.f), m2 = s2;
#pragma unroll
            for (int i = 0; i < VEC / 2; ++i) {
                turn.apply(i, da.get(i), db.get(i), L.turns, za[r][i], zb[r][i]);
                const F2 fa = xa[r].get(i), fb = xb[r].get(i);
                s2 = fma2(fa, fa, s2);
                s2 = fma2(fb, fb, s2);
                m2 = fma2(mul2(za[r][i], w2a[i]), fa, m2);
                m2 = fma2(mul2(zb[r][i], w2b[i]), fb, m2);
            }
            ss[r] = sum2(s2);
            mm[r] = sum2(m2);
        }
        if (norm) {
#pragma unroll
            for (int r = 0; r < RB; ++r) {
                ss[r] = lanes_sum<LANES>(ss[r]);
                mm[r] = lanes_sum<LANES>(mm[r]);
            }
#pragma unroll
            for (int r = 0; r < RB; ++r) {
                const float rs = rsqrtf(ss[r] * (1.f / D) + a.eps);
                const float m = mm[r] * rs * (1.f / D);
                const F2 rs2 = pack2(rs, rs), m2 = pack2(-m, -m);
                if (r < cnt) {
#pragma unroll
                    for (int i = 0; i < VEC / 2; ++i) {
                        const F2 ha = mul2(xa[r].get(i), rs2), hb = mul2(xb[r].get(i), rs2);
                        ga[i] = fma2(za[r][i], ha, ga[i]);
                        gb[i] = fma2(zb[r][i], hb, gb[i]);
                        za[r][i] = mul2(rs2, fma2(ha, m2, mul2(za[r][i], w2a[i])));
                        zb[r][i] = mul2(rs2, fma2(hb, m2, mul2(zb[r][i], w2b[i])));
                    }
                }
            }
        }
        TX *y = static_cast<TX *>(sd.dx) + (out.tok * H + r0) * D;
#pragma unroll
        for (int r = 0; r < RB; ++r)
            if (r < cnt) {
                Line<TX, VEC> oa, ob;
#pragma unroll
                for (int i = 0; i < VEC / 2; ++i) {
                    oa.set(i, za[r][i]);
                    ob.set(i, zb[r][i]);
                }
                oa.store(y + r * D + L.da);
                ob.store(y + r * D + L.db);
            }
        prefetch();
        at = at == (S - 1) * STAGE ? 0 : at + STAGE;
        fresh = out.next(stride, items, hpb, n_hg);
    }
    cp_async_wait<0>();
    if (!a.part) return;
    // groups of a warp, then warps, each in a fixed order
    const int warp = threadIdx.x >> 5;
    float fa[VEC], fb[VEC];
#pragma unroll
    for (int i = 0; i < VEC / 2; ++i) {
        const float2 u = unpack2(ga[i]), v = unpack2(gb[i]);
        fa[2 * i] = u.x;
        fa[2 * i + 1] = u.y;
        fb[2 * i] = v.x;
        fb[2 * i + 1] = v.y;
    }
#pragma unroll
    for (int e = 0; e < VEC; ++e)
        for (int o = LANES; o < 32; o <<= 1) {
            fa[e] += __shfl_xor_sync(0xffffffffu, fa[e], o);
            fb[e] += __shfl_xor_sync(0xffffffffu, fb[e], o);
        }
    if ((threadIdx.x & 31) < LANES) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            s_dw[warp][L.da + e] = fa[e];
            s_dw[warp][L.db + e] = fb[e];
        }
    }
    __syncthreads();
    for (int d = threadIdx.x; d < D; d += THREADS) {
        float t = 0.f;
#pragma unroll
        for (int w = 0; w < THREADS / 32; ++w) t += s_dw[w][d];
        a.part[(int64_t)blockIdx.x * D + d] = t;
    }
}

// dw[d] = sum of the partials of this weight's blocks: a warp takes every 32nd of
// the warp's blocks for 32 dims, the warps are added in order.
__global__ void __launch_bounds__(1024)
    weight_sum_kernel(const float *__restrict__ part, int n_q, int n_k, int D,
                      float *__restrict__ dqw, float *__restrict__ dkw) {
    griddep_wait();  // the partials
    __shared__ float s[32][33];
    const bool isq = blockIdx.y == 0;
    float *out = isq ? dqw : dkw;
    if (!out) return;
    const int n = isq ? n_q : n_k, b0 = isq ? 0 : n_q;
    const int w = threadIdx.x >> 5, l = threadIdx.x & 31;
    const int d = blockIdx.x * 32 + l;
    float t = 0.f;
    for (int i = w; i < n; i += 32) t += part[(int64_t)(b0 + i) * D + d];
    s[w][l] = t;
    __syncthreads();
    t = s[l][w];  // warp w adds dim w over the 32 warps
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
    if (l == 0) out[blockIdx.x * 32 + w] = t;
}

// ----------------------------------------------------------------- host --

// 16-bit rows take 16-byte vectors where the rotated part splits into them
// (rot a multiple of 16), else 8-byte ones; fp32 rows always take 16 bytes.
int pick_vec(int rot) { return rot % 16 == 0 ? 8 : 4; }

// Heads per item of the plain rotation: a token's heads share one set of angles, but at most
// `most` (2 x 4099 tokens of 16 heads of 128 in fp32: 31.0 us with 1, 25.1 with 2 and 4, 25.9
// with 8; 32K tokens in bf16 109 with 1, 64.6 with 2, 47.2 with 4, 45.7 with 8), and a small
// batch is spread over more lanes first.  (Through the ring below it took
// 37 us: without the norms' arithmetic there is nothing for a ring to hide.)
int heads_per_item(int64_t n_tok, int rows, int most, int lanes, int num_sms) {
    const int64_t want = (int64_t)num_sms * 1024 / lanes;  // groups that fill the GPU
    int hpg = rows < most ? rows : most;
    while (hpg > 1 && n_tok * ((rows + hpg - 1) / hpg) < want) hpg = (hpg + 1) / 2;
    return hpg;
}

// Batches of rows per item, up to three, which share one set of angles: what makes the fewest
// rounds of the resident groups, each as long as its batches and the angles (`angles`, in
// batches).  32K tokens of 6 batches: 62.5 us with 3, 67 with 2 (more angles) and 66 with all 6
// (a last round that is half empty), 81 with 1; 4000 tokens 14.9 us with 3, 18.5 with 1.
int batches_per_item(int64_t n_tok, int batches, int64_t groups, double angles) {
    int best = 1;
    double least = 0;
    for (int n = 1; n <= 3 && n <= batches; ++n) {
        const int64_t items = n_tok * ((batches + n - 1) / n);
        const double cost = (double)((items + groups - 1) / groups) * (n + angles);
        if (n == 1 || cost < least) {
            best = n;
            least = cost;
        }
    }
    return best;
}

// Threads of a block: 256, or fewer while that leaves SMs without one (64 sequences' decode
// step: 6.16 us with 64 or 128 threads a block, 6.42 with 256).
int block_of(int64_t items, int lanes, int num_sms) {
    int t = THREADS;
    while (t > 64 && items * lanes < (int64_t)num_sms * t) t /= 2;
    return t;
}

int grid_of(int64_t items, int lanes, int num_sms, int per_sm, int threads = THREADS) {
    const int64_t per_block = threads / lanes;
    const int64_t need = (items + per_block - 1) / per_block;
    const int64_t cap = (int64_t)num_sms * per_sm;
    return (int)(need < cap ? (need > 0 ? need : 1) : cap);
}

// Blocks of the backward: one wave, in proportion to the head counts, at least one each.
void grad_grid(int64_t n_tok, int Hq, int Hkv, int D, int num_sms, int *nq, int *nk) {
    const int total = num_sms * GRAD_CTAS;
    int64_t k = (int64_t)total * Hkv / (Hq + Hkv);
    if (k < 1) k = 1;
    const int64_t per_block = THREADS / (D / (2 * GRAD_VEC));
    const int64_t most_q = (n_tok * Hq + per_block - 1) / per_block;
    const int64_t most_k = (n_tok * Hkv + per_block - 1) / per_block;
    int64_t q = total - k;
    if (q > most_q) q = most_q;
    if (k > most_k) k = most_k;
    *nq = (int)(q < 1 ? 1 : q);
    *nk = (int)(k < 1 ? 1 : k);
}

template <typename T>
cudaError_t run_rope(const RopeArgs &a, bool half, int grid, int threads, cudaStream_t s) {
    if (half)
        rope_kernel<T, true><<<grid, threads, 0, s>>>(a);
    else
        rope_kernel<T, false><<<grid, threads, 0, s>>>(a);
    return cudaGetLastError();
}

template <int D, int VEC, bool HALF>
cudaError_t run_norm(const NormArgs &a, int grid, int threads, cudaStream_t s) {
    constexpr int bytes = 2 * VEC * 2 * NORM_ROWS * NORM_STAGES * THREADS;
    auto kern = norm_rope_kernel<D, VEC, HALF>;
    const cudaError_t e = ensure_smem(reinterpret_cast<const void *>(kern), bytes);
    if (e != cudaSuccess) return e;
    kern<<<grid, threads, bytes, s>>>(a);
    return cudaGetLastError();
}

template <int D>
cudaError_t run_norm(const NormArgs &a, int vec, bool half, int num_sms, cudaStream_t s) {
    const int64_t items = a.n_tok * a.n_hg;
    const int lanes = D / (2 * vec), t = block_of(items, lanes, num_sms);
    const int grid = grid_of(items, lanes, num_sms, NORM_CTAS, t);
    if (vec == 8)
        return half ? run_norm<D, 8, true>(a, grid, t, s) : run_norm<D, 8, false>(a, grid, t, s);
    return half ? run_norm<D, 4, true>(a, grid, t, s) : run_norm<D, 4, false>(a, grid, t, s);
}

template <int D, bool HALF, typename TD, typename TX>
cudaError_t run_grad(const GradArgs &a, int grid, cudaStream_t s) {
    constexpr int bytes = grad_stage<TD>() * GRAD_STAGES;
    auto kern = norm_rope_grad_kernel<D, HALF, TD, TX>;
    const cudaError_t e = ensure_smem(reinterpret_cast<const void *>(kern), bytes);
    if (e != cudaSuccess) return e;
    kern<<<grid, THREADS, bytes, s>>>(a);
    return cudaGetLastError();
}

template <int D, bool HALF>
cudaError_t run_grad(const GradArgs &a, bool d_fp32, bool dx_fp32, int grid, cudaStream_t s) {
    if (d_fp32)
        return dx_fp32 ? run_grad<D, HALF, float, float>(a, grid, s)
                       : run_grad<D, HALF, float, uint16_t>(a, grid, s);
    return dx_fp32 ? run_grad<D, HALF, uint16_t, float>(a, grid, s)
                   : run_grad<D, HALF, uint16_t, uint16_t>(a, grid, s);
}

template <int D>
cudaError_t run_grad(const GradArgs &a, bool half, bool d_fp32, bool dx_fp32, int grid,
                     cudaStream_t s) {
    return half ? run_grad<D, true>(a, d_fp32, dx_fp32, grid, s)
                : run_grad<D, false>(a, d_fp32, dx_fp32, grid, s);
}

}  // namespace rope

cudaError_t launch_rope(const void *x, int64_t xs, void *y, int64_t ys, bool fp32, int B,
                        int64_t T, int H, int D, const double *freq, int rot, bool half,
                        float mscale, bool transpose, const int64_t *pos, const int64_t *pos0,
                        int num_sms, cudaStream_t s) {
    using namespace rope;
    RopeArgs a{};
    a.x = x; a.y = y; a.xs = xs; a.ys = ys; a.T = T; a.n_tok = (int64_t)B * T;
    a.H = H; a.D = D; a.rot = rot; a.lanes = D / (2 * ROPE_VEC);
    a.hpg = heads_per_item(a.n_tok, H, fp32 ? ROPE_ROWS<float> : ROPE_ROWS<uint16_t>, a.lanes,
                           num_sms);
    a.n_hg = (H + a.hpg - 1) / a.hpg;
    a.freq = freq; a.mscale = mscale; a.sign = transpose ? -1.f : 1.f;
    a.pos = Pos{pos, pos0};
    const int64_t items = a.n_tok * a.n_hg;
    const int t = block_of(items, a.lanes, num_sms);
    const int grid = grid_of(items, a.lanes, num_sms, 8, t);
    return fp32 ? run_rope<float>(a, half, grid, t, s) : run_rope<uint16_t>(a, half, grid, t, s);
}

cudaError_t launch_norm_rope(const uint16_t *q, int64_t qs, const uint16_t *k, int64_t ks,
                             const uint16_t *v, int64_t vs, int B, int64_t T, int Hq, int Hkv,
                             int D, const float *qw, const float *kw, float eps,
                             const double *freq, int rot, bool half, float mscale,
                             const int64_t *pos, const int64_t *pos0, uint16_t *qo, uint16_t *ko,
                             uint16_t *vo, const int64_t *slot, int64_t L, void *status,
                             int num_sms, cudaStream_t s) {
    using namespace rope;
    const int vec = pick_vec(rot), lanes = D / (2 * vec);
    NormArgs a{};
    a.x[0] = q; a.x[1] = k; a.x[2] = v;
    a.xs[0] = qs; a.xs[1] = ks; a.xs[2] = vs;
    a.y[0] = qo; a.y[1] = ko; a.y[2] = vo;
    a.w[0] = qw; a.w[1] = kw;
    a.H[0] = Hq; a.H[1] = a.H[2] = Hkv;
    const int bk = (Hkv + NORM_ROWS - 1) / NORM_ROWS;
    a.first[1] = (Hq + NORM_ROWS - 1) / NORM_ROWS;
    a.first[2] = a.first[1] + bk;
    a.batches = a.first[2] + (v ? bk : 0);
    a.slot = slot; a.L = L; a.T = T; a.n_tok = (int64_t)B * T; a.rot = rot;
    a.hpb = batches_per_item(a.n_tok, a.batches, (int64_t)num_sms * NORM_CTAS * THREADS / lanes,
                             0.9);
    a.n_hg = (a.batches + a.hpb - 1) / a.hpb;
    a.eps = eps; a.freq = freq; a.mscale = mscale; a.pos = Pos{pos, pos0}; a.status = status;
    return D == 32    ? run_norm<32>(a, vec, half, num_sms, s)
           : D == 64  ? run_norm<64>(a, vec, half, num_sms, s)
           : D == 128 ? run_norm<128>(a, vec, half, num_sms, s)
                      : run_norm<256>(a, vec, half, num_sms, s);
}

// The grid depends on the device, so the workspace is sized for the largest one.
size_t norm_rope_grad_ws_bytes(int64_t n_tok, int Hq, int Hkv, int D) {
    int nq, nk;
    rope::grad_grid(n_tok, Hq, Hkv, D, 160, &nq, &nk);
    return kWsHeader + (size_t)(nq + nk) * D * sizeof(float);
}

cudaError_t launch_norm_rope_grad(const void *d_q, const void *d_k, bool d_fp32,
                                  const uint16_t *q, int64_t qs, const uint16_t *k, int64_t ks,
                                  int B, int64_t T, int Hq, int Hkv, int D, const float *qw,
                                  const float *kw, float eps, const double *freq, int rot,
                                  bool half, float mscale, const int64_t *pos,
                                  const int64_t *pos0, void *dq, void *dk, bool dx_fp32,
                                  float *dqw, float *dkw, void *ws, int num_sms,
                                  cudaStream_t s) {
    using namespace rope;
    const int lanes = D / (2 * GRAD_VEC);
    GradArgs a{};
    a.T = T; a.n_tok = (int64_t)B * T; a.rot = rot;
    a.eps = eps; a.freq = freq; a.mscale = mscale; a.pos = Pos{pos, pos0};
    const int sms = num_sms < 160 ? num_sms : 160;
    int nq, nk;
    grad_grid(a.n_tok, Hq, Hkv, D, sms, &nq, &nk);
    auto side = [&](const void *dy, const uint16_t *x, int64_t xs, void *dx, const float *w,
                    int H, int blocks) {
        const int n = (H + GRAD_ROWS - 1) / GRAD_ROWS;
        const int hpb = batches_per_item(a.n_tok, n, (int64_t)blocks * THREADS / lanes, 0.5);
        return Side{dy, x, xs, dx, w, H, n, hpb, (n + hpb - 1) / hpb};
    };
    a.side[0] = side(d_q, q, qs, dq, qw, Hq, nq);
    a.side[1] = side(d_k, k, ks, dk, kw, Hkv, nk);
    a.n_blocks_q = nq;
    a.part = dqw || dkw ? reinterpret_cast<float *>(static_cast<uint8_t *>(ws) + kWsHeader)
                        : nullptr;
    const int grid = nq + nk;
    const cudaError_t e = D == 32    ? run_grad<32>(a, half, d_fp32, dx_fp32, grid, s)
                          : D == 64  ? run_grad<64>(a, half, d_fp32, dx_fp32, grid, s)
                          : D == 128 ? run_grad<128>(a, half, d_fp32, dx_fp32, grid, s)
                                     : run_grad<256>(a, half, d_fp32, dx_fp32, grid, s);
    if (e != cudaSuccess || !a.part) return e;
    return launch_dependent(weight_sum_kernel, dim3(D / 32, 2), dim3(1024), 0, s,
                            (const float *)a.part, nq, nk, D, dqw, dkw);
}

}  // namespace qsa
