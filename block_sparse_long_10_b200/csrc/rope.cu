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
constexpr int ROWS = 4;  // head rows whose loads are issued together
constexpr double INV_2PI = 0.15915494309189533576888376337251;

template <typename T, int VEC>
struct Raw;
template <>
struct Raw<uint16_t, 8> {
    uint4 v;
    QSA_DEVICE void load(const uint16_t *p) { v = *reinterpret_cast<const uint4 *>(p); }
    QSA_DEVICE void store(uint16_t *p) const { *reinterpret_cast<uint4 *>(p) = v; }
    QSA_DEVICE void get(float (&f)[8]) const {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[2 * i] = bf16_lo(w[i]);
            f[2 * i + 1] = bf16_hi(w[i]);
        }
    }
    QSA_DEVICE void set(const float (&f)[8]) {
        v = make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]),
                       pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
    }
};
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

QSA_DEVICE float group_sum(float x, int lanes) {
    for (int o = lanes >> 1; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
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

template <typename T, int VEC, bool HALF>
__global__ void __launch_bounds__(THREADS) rope_kernel(const RopeArgs a) {
    const int lane = threadIdx.x % a.lanes;
    const Lane<VEC, HALF> L(lane, a.rot);
    double tf[VEC];
    load_turns<VEC>(a.freq, L.f0, L.turns, tf);
    const int64_t per_block = THREADS / a.lanes;
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
struct NormArgs {
    const uint16_t *q, *k, *v;
    int64_t qs, ks, vs;          // elements between tokens
    uint16_t *qo, *ko, *vo;
    const float *qw, *kw;        // [D] or nullptr (no norm)
    const int64_t *slot;         // [B, T] cache rows, or nullptr (row = token)
    int64_t L;                   // cache rows per sequence
    int64_t T, n_tok;
    int Hq, Hkv, D, rot, lanes;
    int rows, hpg, n_hg;         // head rows of a token (q, k and v), per item, items
    float eps;
    const double *freq;
    float mscale;
    Pos pos;
    void *status;
};

template <int VEC, bool HALF>
__global__ void __launch_bounds__(THREADS) norm_rope_kernel(const NormArgs a) {
    const int lane = threadIdx.x % a.lanes;
    const Lane<VEC, HALF> L(lane, a.rot);
    double tf[VEC];
    load_turns<VEC>(a.freq, L.f0, L.turns, tf);
    const int64_t per_block = THREADS / a.lanes;
    const int64_t items = a.n_tok * a.n_hg;
    const float inv_d = 1.f / (float)a.D;
    // whole warps stay in the loop (the sums are shuffles); `live` guards the memory
    const int64_t first = blockIdx.x * per_block;
    for (int64_t base = first; base < items; base += gridDim.x * per_block) {
        const int64_t it = base + threadIdx.x / a.lanes;
        const bool live = it < items;
        const int64_t tok = live ? it / a.n_hg : 0;
        const int r0 = live ? (int)(it - tok * a.n_hg) * a.hpg : 0;
        float c[VEC], s[VEC];
        angles<VEC>(a.pos.at(tok, a.T), tf, L.turns, a.mscale, 1.f, c, s);
        int64_t orow = tok;  // row of the key and value outputs, or -1: not written
        if (a.slot && live) {
            const int64_t sl = a.slot[tok];
            orow = sl >= 0 && sl < a.L ? tok / a.T * a.L + sl : -1;
            if (sl >= a.L && lane == 0) record_status(a.status, QSA_ERR_DEVICE);
        }
        for (int rr = 0; rr < a.hpg; rr += ROWS) {
            Raw<uint16_t, VEC> ra[ROWS], rb[ROWS];
            bool on[ROWS];
#pragma unroll
            for (int r = 0; r < ROWS; ++r) {
                const int row = r0 + rr + r;
                on[r] = live && rr + r < a.hpg && row < a.rows;
                if (on[r]) {
                    const uint16_t *x =
                        row < a.Hq ? a.q + tok * a.qs + (int64_t)row * a.D
                        : row < a.Hq + a.Hkv
                            ? a.k + tok * a.ks + (int64_t)(row - a.Hq) * a.D
                            : a.v + tok * a.vs + (int64_t)(row - a.Hq - a.Hkv) * a.D;
                    ra[r].load(x + L.da);
                    rb[r].load(x + L.db);
                }
            }
#pragma unroll
            for (int r = 0; r < ROWS; ++r) {
                const int row = r0 + rr + r;
                const bool isq = row < a.Hq, isv = row >= a.Hq + a.Hkv;
                float fa[VEC], fb[VEC];
                float ss = 0.f;
                if (on[r]) {
                    ra[r].get(fa);
                    rb[r].get(fb);
#pragma unroll
                    for (int e = 0; e < VEC; ++e) ss += fa[e] * fa[e] + fb[e] * fb[e];
                }
                ss = group_sum(ss, a.lanes);
                if (!on[r]) continue;
                if (!isv) {
                    const float *w = isq ? a.qw : a.kw;
                    if (w) {
                        const float rs = rsqrtf(ss * inv_d + a.eps);
                        float wa[VEC], wb[VEC];
                        load_weight<VEC>(w, L.da, wa);
                        load_weight<VEC>(w, L.db, wb);
#pragma unroll
                        for (int e = 0; e < VEC; ++e) {
                            fa[e] *= rs * wa[e];
                            fb[e] *= rs * wb[e];
                        }
                    }
                    rotate<VEC, HALF>(fa, fb, c, s);
                    ra[r].set(fa);
                    rb[r].set(fb);
                }
                if (!isq && orow < 0) continue;
                uint16_t *y = isq ? a.qo + (tok * a.Hq + row) * a.D
                              : !isv ? a.ko + (orow * a.Hkv + row - a.Hq) * a.D
                                     : a.vo + (orow * a.Hkv + row - a.Hq - a.Hkv) * a.D;
                ra[r].store(y + L.da);
                rb[r].store(y + L.db);
            }
        }
    }
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
    int H, hpg, n_hg;
};
struct GradArgs {
    Side side[2];        // queries, keys
    int n_blocks_q;      // blocks before this one work on the queries
    int64_t T, n_tok;
    int D, rot, lanes;
    float eps;
    const double *freq;
    float mscale;
    Pos pos;
    float *part;         // [blocks, D]
};

template <int VEC, bool HALF, typename TD, typename TX>
__global__ void __launch_bounds__(THREADS) norm_rope_grad_kernel(const GradArgs a) {
    constexpr int RB = 2;  // rows whose loads are issued together
    __shared__ float s_dw[THREADS / 32][256];
    const bool isq = (int)blockIdx.x < a.n_blocks_q;
    const Side &sd = a.side[isq ? 0 : 1];
    const int blk = isq ? blockIdx.x : blockIdx.x - a.n_blocks_q;
    const int n_blk = isq ? a.n_blocks_q : gridDim.x - a.n_blocks_q;
    const int lane = threadIdx.x % a.lanes;
    const Lane<VEC, HALF> L(lane, a.rot);
    double tf[VEC];
    load_turns<VEC>(a.freq, L.f0, L.turns, tf);
    float wa[VEC], wb[VEC], ga[VEC], gb[VEC];
#pragma unroll
    for (int e = 0; e < VEC; ++e) ga[e] = gb[e] = wa[e] = wb[e] = 0.f;
    if (sd.w) {
        load_weight<VEC>(sd.w, L.da, wa);
        load_weight<VEC>(sd.w, L.db, wb);
    }
    const int64_t per_block = THREADS / a.lanes;
    const int64_t items = a.n_tok * sd.n_hg;
    const float inv_d = 1.f / (float)a.D;
    for (int64_t base = blk * per_block; base < items; base += n_blk * per_block) {
        const int64_t it = base + threadIdx.x / a.lanes;
        const bool live = it < items;
        const int64_t tok = live ? it / sd.n_hg : 0;
        const int h0 = live ? (int)(it - tok * sd.n_hg) * sd.hpg : 0;
        float c[VEC], s[VEC];
        angles<VEC>(a.pos.at(tok, a.T), tf, L.turns, a.mscale, -1.f, c, s);
        for (int hh = 0; hh < sd.hpg; hh += RB) {
            Raw<TD, VEC> da[RB], db[RB];
            Raw<uint16_t, VEC> xa[RB], xb[RB];
            bool on[RB];
#pragma unroll
            for (int r = 0; r < RB; ++r) {
                const int h = h0 + hh + r;
                on[r] = live && hh + r < sd.hpg && h < sd.H;
                if (on[r]) {
                    const TD *d = static_cast<const TD *>(sd.dy) + (tok * sd.H + h) * a.D;
                    const uint16_t *x = sd.x + tok * sd.xs + (int64_t)h * a.D;
                    da[r].load(d + L.da);
                    db[r].load(d + L.db);
                    xa[r].load(x + L.da);
                    xb[r].load(x + L.db);
                }
            }
#pragma unroll
            for (int r = 0; r < RB; ++r) {
                const int h = h0 + hh + r;
                float za[VEC], zb[VEC], fa[VEC], fb[VEC];
                float ss = 0.f, m = 0.f;
#pragma unroll
                for (int e = 0; e < VEC; ++e) za[e] = zb[e] = fa[e] = fb[e] = 0.f;
                if (on[r]) {
                    da[r].get(za);
                    db[r].get(zb);
                    rotate<VEC, HALF>(za, zb, c, s);
                    xa[r].get(fa);
                    xb[r].get(fb);
                }
                if (sd.w) {
#pragma unroll
                    for (int e = 0; e < VEC; ++e) {
                        ss += fa[e] * fa[e] + fb[e] * fb[e];
                        m += za[e] * wa[e] * fa[e] + zb[e] * wb[e] * fb[e];
                    }
                    ss = group_sum(ss, a.lanes);
                    m = group_sum(m, a.lanes);
                    const float rs = rsqrtf(ss * inv_d + a.eps);
                    m = m * rs * inv_d;
#pragma unroll
                    for (int e = 0; e < VEC; ++e) {
                        const float ha = fa[e] * rs, hb = fb[e] * rs;
                        ga[e] += za[e] * ha;
                        gb[e] += zb[e] * hb;
                        za[e] = rs * (za[e] * wa[e] - ha * m);
                        zb[e] = rs * (zb[e] * wb[e] - hb * m);
                    }
                }
                if (on[r]) {
                    Raw<TX, VEC> oa, ob;
                    oa.set(za);
                    ob.set(zb);
                    TX *y = static_cast<TX *>(sd.dx) + (tok * sd.H + h) * a.D;
                    oa.store(y + L.da);
                    ob.store(y + L.db);
                }
            }
        }
    }
    if (!a.part) return;
    // groups of a warp, then warps, each in a fixed order
    const int warp = threadIdx.x >> 5;
#pragma unroll
    for (int e = 0; e < VEC; ++e)
        for (int o = a.lanes; o < 32; o <<= 1) {
            ga[e] += __shfl_xor_sync(0xffffffffu, ga[e], o);
            gb[e] += __shfl_xor_sync(0xffffffffu, gb[e], o);
        }
    if ((threadIdx.x & 31) < a.lanes) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            s_dw[warp][L.da + e] = ga[e];
            s_dw[warp][L.db + e] = gb[e];
        }
    }
    __syncthreads();
    for (int d = threadIdx.x; d < a.D; d += THREADS) {
        float t = 0.f;
#pragma unroll
        for (int w = 0; w < THREADS / 32; ++w) t += s_dw[w][d];
        a.part[(int64_t)blockIdx.x * a.D + d] = t;
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

// Heads per item: all of a token's rows share one set of angles, but a small batch
// is spread over more lanes first.  The rotation of a token's `rows` rows costs
// about as much as its angles at 4 rows, so items are cut to 4 rows only while the
// GPU has room for them, and to 1 when even those leave SMs idle.
int heads_per_item(int64_t n_tok, int rows, int lanes, int num_sms) {
    const int64_t want = (int64_t)num_sms * 1024 / lanes;  // groups that fill the GPU
    int hpg = rows;
    while (hpg > 1 && n_tok * ((rows + hpg - 1) / hpg) < want) hpg = (hpg + 1) / 2;
    return hpg;
}

int grid_of(int64_t items, int lanes, int num_sms, int per_sm) {
    const int64_t per_block = THREADS / lanes;
    const int64_t need = (items + per_block - 1) / per_block;
    const int64_t cap = (int64_t)num_sms * per_sm;
    return (int)(need < cap ? (need > 0 ? need : 1) : cap);
}

// Blocks of the backward: in proportion to the head counts, at least one each.
void grad_grid(int64_t n_tok, int Hq, int Hkv, int D, int num_sms, int *nq, int *nk) {
    const int lanes_min = D / 16;
    const int total = num_sms * 4;
    int64_t k = (int64_t)total * Hkv / (Hq + Hkv);
    if (k < 1) k = 1;
    const int64_t per_block = THREADS / lanes_min;
    const int64_t most_q = (n_tok * Hq + per_block - 1) / per_block;
    const int64_t most_k = (n_tok * Hkv + per_block - 1) / per_block;
    int64_t q = total - k;
    if (q > most_q) q = most_q;
    if (k > most_k) k = most_k;
    *nq = (int)(q < 1 ? 1 : q);
    *nk = (int)(k < 1 ? 1 : k);
}

template <typename T, int VEC>
cudaError_t run_rope(const RopeArgs &a, bool half, int grid, cudaStream_t s) {
    if (half)
        rope_kernel<T, VEC, true><<<grid, THREADS, 0, s>>>(a);
    else
        rope_kernel<T, VEC, false><<<grid, THREADS, 0, s>>>(a);
    return cudaGetLastError();
}

template <int VEC, typename TD, typename TX>
cudaError_t run_grad(const GradArgs &a, bool half, int grid, cudaStream_t s) {
    if (half)
        norm_rope_grad_kernel<VEC, true, TD, TX><<<grid, THREADS, 0, s>>>(a);
    else
        norm_rope_grad_kernel<VEC, false, TD, TX><<<grid, THREADS, 0, s>>>(a);
    return cudaGetLastError();
}

}  // namespace rope

cudaError_t launch_rope(const void *x, int64_t xs, void *y, int64_t ys, bool fp32, int B,
                        int64_t T, int H, int D, const double *freq, int rot, bool half,
                        float mscale, bool transpose, const int64_t *pos, const int64_t *pos0,
                        int num_sms, cudaStream_t s) {
    using namespace rope;
    const int vec = fp32 ? 4 : pick_vec(rot);
    RopeArgs a{};
    a.x = x; a.y = y; a.xs = xs; a.ys = ys; a.T = T; a.n_tok = (int64_t)B * T;
    a.H = H; a.D = D; a.rot = rot; a.lanes = D / (2 * vec);
    a.hpg = heads_per_item(a.n_tok, H, a.lanes, num_sms);
    a.n_hg = (H + a.hpg - 1) / a.hpg;
    a.freq = freq; a.mscale = mscale; a.sign = transpose ? -1.f : 1.f;
    a.pos = Pos{pos, pos0};
    const int grid = grid_of(a.n_tok * a.n_hg, a.lanes, num_sms, 8);
    if (fp32) return run_rope<float, 4>(a, half, grid, s);
    return vec == 8 ? run_rope<uint16_t, 8>(a, half, grid, s)
                    : run_rope<uint16_t, 4>(a, half, grid, s);
}

cudaError_t launch_norm_rope(const uint16_t *q, int64_t qs, const uint16_t *k, int64_t ks,
                             const uint16_t *v, int64_t vs, int B, int64_t T, int Hq, int Hkv,
                             int D, const float *qw, const float *kw, float eps,
                             const double *freq, int rot, bool half, float mscale,
                             const int64_t *pos, const int64_t *pos0, uint16_t *qo, uint16_t *ko,
                             uint16_t *vo, const int64_t *slot, int64_t L, void *status,
                             int num_sms, cudaStream_t s) {
    using namespace rope;
    const int vec = pick_vec(rot);
    NormArgs a{};
    a.q = q; a.k = k; a.v = v; a.qs = qs; a.ks = ks; a.vs = vs; a.qo = qo; a.ko = ko; a.vo = vo;
    a.qw = qw; a.kw = kw; a.slot = slot; a.L = L; a.T = T; a.n_tok = (int64_t)B * T;
    a.Hq = Hq; a.Hkv = Hkv; a.D = D; a.rot = rot; a.lanes = D / (2 * vec);
    a.rows = Hq + Hkv + (v ? Hkv : 0);
    a.hpg = heads_per_item(a.n_tok, a.rows, a.lanes, num_sms);
    a.n_hg = (a.rows + a.hpg - 1) / a.hpg;
    a.eps = eps; a.freq = freq; a.mscale = mscale; a.pos = Pos{pos, pos0}; a.status = status;
    const int grid = grid_of(a.n_tok * a.n_hg, a.lanes, num_sms, 8);
    if (vec == 8) {
        if (half)
            norm_rope_kernel<8, true><<<grid, THREADS, 0, s>>>(a);
        else
            norm_rope_kernel<8, false><<<grid, THREADS, 0, s>>>(a);
    } else {
        if (half)
            norm_rope_kernel<4, true><<<grid, THREADS, 0, s>>>(a);
        else
            norm_rope_kernel<4, false><<<grid, THREADS, 0, s>>>(a);
    }
    return cudaGetLastError();
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
    const int vec = pick_vec(rot);
    GradArgs a{};
    a.T = T; a.n_tok = (int64_t)B * T; a.D = D; a.rot = rot; a.lanes = D / (2 * vec);
    a.eps = eps; a.freq = freq; a.mscale = mscale; a.pos = Pos{pos, pos0};
    const int sms = num_sms < 160 ? num_sms : 160;
    auto side = [&](const void *dy, const uint16_t *x, int64_t xs, void *dx, const float *w,
                    int H) {
        Side d{dy, x, xs, dx, w, H, heads_per_item(a.n_tok, H, a.lanes, sms), 0};
        d.n_hg = (H + d.hpg - 1) / d.hpg;
        return d;
    };
    a.side[0] = side(d_q, q, qs, dq, qw, Hq);
    a.side[1] = side(d_k, k, ks, dk, kw, Hkv);
    int nq, nk;
    grad_grid(a.n_tok, Hq, Hkv, D, sms, &nq, &nk);
    a.n_blocks_q = nq;
    a.part = dqw || dkw ? reinterpret_cast<float *>(static_cast<uint8_t *>(ws) + kWsHeader)
                        : nullptr;
    cudaError_t e;
    const int grid = nq + nk;
#define QSA_GRAD(V_, TD_, TX_) run_grad<V_, TD_, TX_>(a, half, grid, s)
#define QSA_GRAD_T(V_)                                                              \
    (d_fp32 ? (dx_fp32 ? QSA_GRAD(V_, float, float) : QSA_GRAD(V_, float, uint16_t)) \
            : (dx_fp32 ? QSA_GRAD(V_, uint16_t, float) : QSA_GRAD(V_, uint16_t, uint16_t)))
    e = vec == 8 ? QSA_GRAD_T(8) : QSA_GRAD_T(4);
#undef QSA_GRAD_T
#undef QSA_GRAD
    if (e != cudaSuccess || !a.part) return e;
    return launch_dependent(weight_sum_kernel, dim3(D / 32, 2), dim3(1024), 0, s,
                            (const float *)a.part, nq, nk, D, dqw, dkw);
}

}  // namespace qsa
