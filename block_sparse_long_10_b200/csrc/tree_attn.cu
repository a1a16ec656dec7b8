// Attention for a tree of drafted tokens over the caches, dense and over selected
// micro-blocks: the decode step that verifies several drafted tokens at once.
//
// Sequence b holds seqlens[b] tokens, the last n of them (n = n_draft[b]) drafts:
// draft i lies in cache row P + i, P = seqlens[b] - n, whatever its depth.  Row i
// attends to the prefix u < P (dense) or to the prefix tokens of its selected
// blocks and the unpooled tail (sparse), and to its own chain i, parent[i],
// parent[parent[i]], ...: softmax over both parts together.
//
// What the cache rows of other branches hold (infinities, NaN) never enters a row, as a
// zero times it in a matrix product would, and does not change its bits.  Dense, the drafts
// lie behind the prefix in the same tiles: two matrix products (tree_dense_kernel) with a
// mask of ancestors, in which values of drafts that are not finite count as zeros; the
// merge adds them to the rows whose chains they are in.  Selections differ from row to row:
// they and the chains are gathered row by row (sparse_attn.cu).  All parts of a row are
// (max, sum, O) in base 2 and meet in tree_merge_kernel.
#include "qsa_common.cuh"
#include "qsa_launch.h"
#include "sm100.cuh"

namespace qsa {

namespace tree {

constexpr int MAX_N = TREE_DRAFTS;
constexpr float LOG2E = 1.4426950408889634f;
constexpr float LN2 = 0.6931471805599453f;

struct Seq {
    int64_t P;  // committed tokens
    int n;      // drafts
    bool bad;   // lengths out of range: every row of the sequence is empty
};

struct Lens {
    const int32_t *seqlens;  // [B]
    const int32_t *n_draft;  // [B] or nullptr (N drafts each)
    int N;
    int64_t L_max;
    QSA_DEVICE Seq at(int64_t b) const {
        const int64_t S = seqlens[b];
        const int n = n_draft ? n_draft[b] : N;
        Seq s{S - n, n, n < 0 || n > N || S < n || S > L_max};
        if (s.bad) s.P = s.n = 0;
        return s;
    }
};

constexpr int KT = 128;  // tokens per tile (dense)
constexpr int DRAFT_TILES = (MAX_N + KT - 2) / KT + 1;  // that drafts can lie in

// What the prefix kernel leaves of a unit for the merge.
struct UnitInfo {
    int32_t first, last;             // CTAs that have tiles of it
    int32_t cleared[DRAFT_TILES];    // dense: that tile has drafts' values that are not finite
};

struct Args {
    const uint16_t *q;   // [B, N, Hq, D]
    const uint16_t *k;   // [B, L_max, Hkv, D]
    const uint16_t *v;
    Lens lens;
    const int32_t *parent;  // [B, N]
    int B, N, Hq, Hkv, G, lg;  // lg: log2 G
    float scale_log2;
    // prefix parts: part x holds O[x * D ..] and (max, sum)[x * 2 ..]
    float *part, *ml;
    // Units: dense, `rows` (draft, head) pairs of a KV head, `units` to a (sequence, KV head);
    // sparse, the heads of a draft.  CTA c leaves unit u's row r in part (c + u) * rows + r.
    int units, rows;
    UnitInfo *info;
    uint16_t *o;
    float *lse;
    void *status;
};

// ------------------------------------------------------------ dense prefix --
// Rows of one KV head, (draft, head) pairs r = i * G + h, are cut into units of
// 128 * NT.  A unit times a run of 128-token tiles of its sequence is a flash attention
// on the tensor cores: S = Q K^T and O += P V with 128 x 128 x 16 MMAs (tcgen05), S, P
// and O in TMEM, a thread per row for the softmax.
//
// Work split: the units' tiles, in one row over all sequences, are cut into equal runs,
// one per SM, whatever the lengths (known on the device only).  A run may end one unit
// and begin another; each such segment leaves one part per row, in slot CTA + unit
// (every segment raises one of the two).
//
// Two softmax streams of 128 threads keep the tensor core busy: with NT = 2 they are
// two row tiles over the same K and V, with NT = 1 (at most 128 rows) even and odd
// token tiles of one row tile, merged at the end of the segment.  Step t of a segment is
// S(t), softmax, O += P V (t); the MMA warp issues S(t + 2) right after P V (t), so one
// stream's products run under the other's softmax.  P (bf16) overwrites the S it came
// from.  O is rescaled only when the running maximum has grown by more than 8 (a
// factor 256) since its last rescale: sums and O stay far inside fp32, and P keeps bf16's
// relative precision at any size.  P is rounded to bf16 for the matrix product, which takes
// both operands in V's type: at most 2^-8 of each weight, unbiased: the output is off by 0.0018 to
// 0.0026 of its size against 64 bits (2-norms), where its own rounding alone is 0.0017.  The sum
// is taken of the unrounded values, in fp32.
// (Two streams over one tensor core, rescaling past a threshold only and a polynomial for part of
// the exponentials are published ideas for attention on this architecture; layout, split,
// thresholds and coefficients are this file's.)
//
// What bounds it.  Up to 128 rows a unit: HBM (32 x 8 drafts over 8K to 16K: the CTAs' runs end
// 48 to 66 us in, 409 MB; a call is 77 us).  More: the chain of a stream's step,
// softmax about 1500 clocks, its own two products 1024, handing over about 400, against 2048
// of products for both streams (4 x 64 drafts over 64K: runs of 102 to 119 us, 137 GFLOP, the
// tensor pipe 58 % busy; a call is 139 us).  These are a few calls (or graph replays, which take
// as long) at 1.9 GHz; call after call for a second, the power limit takes the clock to 1.54
// and 1.40 GHz and the calls to 81 and 168 us.
constexpr int ATOM = KT * 128; // bytes of a 64-column half tile in shared memory
constexpr int SOFT = 256;      // softmax threads
constexpr int THREADS = SOFT + 96;   // and a producer, an MMA and a cleaning warp
constexpr float GROWTH = 8.f;
constexpr int MAX_CTAS = 160;  // what the workspace is sized for
constexpr uint64_t WAIT_NS = 2000000000ull;

template <int D, int NT>
struct Cfg {
    static constexpr int TILE = KT * D * 2;
    static constexpr int OFF_RING = NT * TILE;
    static constexpr int ROOM = 227 * 1024 - 1024 - 512;  // alignment; barriers
    static constexpr int FIT = (ROOM - OFF_RING) / TILE;
    static constexpr int SLOTS = FIT > 8 ? 8 : FIT;
    static constexpr int OFF_BAR = OFF_RING + SLOTS * TILE;
    static constexpr int BYTES = 1024 + OFF_BAR + 512;
    static_assert((4 * SLOTS + 8) * 8 + 16 <= 512, "barriers");
    static_assert(NT == 2 || 2 * 128 * 8 <= TILE, "the streams' sums fit in the query tile");
    // TMEM columns
    static constexpr int O_COL = 256;
    static constexpr uint32_t IDESC_S = sm100::idesc_bf16_f32(128, KT);
    static constexpr uint32_t IDESC_O = sm100::idesc_bf16_f32(128, D) | sm100::IDESC_B_MNMAJOR;
};

// A run of tiles of one unit.
struct Seg {
    int64_t b, t0, P;  // first tile; committed tokens
    int g, qt, nd, n;  // tiles
    bool begins, ends; // the unit's first (last) tile is in it
};

// The segments of this CTA, in order.  Each thread that asks walks by itself.  A unit counts
// START tiles more than it has, before its first: a CTA that goes on to another unit drains
// its pipeline, stores a part and loads queries, the time of about START tiles (without
// them such CTAs were the last by 8 us of 77, at 8 drafts over 32 prefixes of 8K to 16K).
constexpr int START = 5;
// (32 bits: a tile is 16 KB of caches and more, times at most 16 units.)
template <int NT>
struct Walk {
    int pos, hi, b, b0;  // b0: flat index of sequence b's first tile

    QSA_DEVICE static int tiles(const Seq &s) {
        return s.n > 0 ? (int)((s.P + s.n + KT - 1) / KT) + START : 0;
    }
    QSA_DEVICE static int units(const Args &a, const Seq &s) {
        return ((s.n << a.lg) + 128 * NT - 1) / (128 * NT);
    }
    QSA_DEVICE static int weight(const Args &a, int b) {
        const Seq s = a.lens.at(b);
        return tiles(s) * units(a, s) * a.Hkv;
    }
    // Whole warps; false: nothing for this CTA.
    QSA_DEVICE bool start(const Args &a, int lane) {
        int total = 0, w0 = 0;
        for (int i = 0; i < a.B; i += 32) {
            const int w = i + lane < a.B ? weight(a, i + lane) : 0;
            if (i == 0) w0 = w;
            total += w;
        }
        total = __reduce_add_sync(0xffffffffu, total);
        // no CTA without tiles between two of one unit: the merge reads every slot
        const int ctas = total < (int)gridDim.x ? total : gridDim.x, c = blockIdx.x;
        if (c >= ctas) return false;
        const int each = total / ctas, more = total - each * ctas;
        pos = each * c + min(c, more);
        hi = pos + each + (c < more);
        b0 = 0;
        for (int i = 0;; i += 32) {
            const int w = i == 0 ? w0 : i + lane < a.B ? weight(a, i + lane) : 0;
            int end = w;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, end, o);
                if (lane >= o) end += y;
            }
            const uint32_t past = __ballot_sync(0xffffffffu, b0 + end > pos);
            if (past) {
                const int f = __ffs(past) - 1;
                b = i + f;
                b0 += __shfl_sync(0xffffffffu, end - w, f);
                return true;
            }
            b0 += __shfl_sync(0xffffffffu, end, 31);
        }
    }
    QSA_DEVICE bool next(const Args &a, Seg &s) {
        while (pos < hi) {
            Seq sq = a.lens.at(b);
            int nt = tiles(sq), w = nt * units(a, sq) * a.Hkv;
            while (pos >= b0 + w) {
                b0 += w;
                sq = a.lens.at(++b);
                nt = tiles(sq);
                w = nt * units(a, sq) * a.Hkv;
            }
            const int u = (pos - b0) / nt, qn = units(a, sq);
            const int t = pos - b0 - u * nt, n = min(nt - t, hi - pos);
            pos += n;
            if (t + n <= START) continue;  // only tiles that stand for the start
            s.b = b;
            s.P = sq.P;
            s.nd = sq.n;
            s.g = u / qn;
            s.qt = u - s.g * qn;
            s.t0 = t > START ? t - START : 0;
            s.n = t + n - START - (int)s.t0;
            s.begins = s.t0 == 0;
            s.ends = t + n == nt;
            return true;
        }
        return false;
    }
};

// Order of a segment's 2 n tiles in the ring: K0, then (NT = 1) K(j + 1), V(j) by turns,
// or (NT = 2) V(j), K(j + 1): the order in which the MMAs want and free them.
template <int NT>
QSA_DEVICE uint32_t ring_k(uint32_t base, int j) {
    return NT == 2 ? base + 2 * j : base + (j == 0 ? 0 : 2 * j - 1);
}
template <int NT>
QSA_DEVICE uint32_t ring_v(uint32_t base, int j, int n) {
    return NT == 2 ? base + 2 * j + 1 : base + (j == n - 1 ? 2 * j + 1 : 2 * j + 2);
}

QSA_DEVICE void soft_sync() { asm volatile("bar.sync 1, %0;\n" ::"n"(SOFT) : "memory"); }

// A thread's 32-byte sector in one store (the parts start at a multiple of 32 bytes).
QSA_DEVICE void store_sector(float *p, const uint32_t *r) {
    asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};\n" ::"l"(p), "r"(r[0]),
                 "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
}

// Packed fp32 pairs.
QSA_DEVICE uint64_t pair(float a, float b) {
    uint64_t x;
    asm("mov.b64 %0, {%1, %2};\n" : "=l"(x) : "f"(a), "f"(b));
    return x;
}
QSA_DEVICE void unpair(uint64_t x, float &a, float &b) {
    asm("mov.b64 {%0, %1}, %2;\n" : "=f"(a), "=f"(b) : "l"(x));
}
QSA_DEVICE uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;\n" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
QSA_DEVICE uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;\n" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
// The largest of three, NaN if one is.
QSA_DEVICE float max3(float a, float b, float c) {
    float d;
    asm("max.NaN.f32 %0, %1, %2, %3;\n" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

// 2^x for two x <= 2^7 on the FMA pipe: x = j + f with j whole and |f| <= 1/2 (adding 1.5 * 2^23
// rounds to j and leaves it in the low bits), 2^f by a polynomial of degree 5 fitted to the
// least largest relative error with 2^0 = 1 exactly (below 2^-22.4 over every fp32 f; the
// exponential unit's is 2^-22), j added to the exponent.  From x = -126 down, where fp32 has no
// more exponents, some value up to 2^-126, and 0 from x = -127 on.
QSA_DEVICE void exp2_fma(uint64_t x2, float &p0, float &p1) {
    constexpr float SHIFT = 12582912.f;
    float x0, x1;
    unpair(x2, x0, x1);
    const uint64_t x = pair(fmaxf(x0, -127.f), fmaxf(x1, -127.f));
    const uint64_t t = add2(x, pair(SHIFT, SHIFT));
    const uint64_t f = fma2(add2(t, pair(-SHIFT, -SHIFT)), pair(-1.f, -1.f), x);
    uint64_t p = fma2(f, pair(0.001326472614891827f, 0.001326472614891827f),
                      pair(0.009671512991189957f, 0.009671512991189957f));
    p = fma2(p, f, pair(0.05550733581185341f, 0.05550733581185341f));
    p = fma2(p, f, pair(0.24022242426872253f, 0.24022242426872253f));
    p = fma2(p, f, pair(0.6931470036506653f, 0.6931470036506653f));
    p = fma2(p, f, pair(1.f, 1.f));
    float t0, t1;
    unpair(t, t0, t1);
    unpair(p, p0, p1);
    p0 = __uint_as_float(__float_as_uint(p0) + (__float_as_uint(t0) << 23));
    p1 = __uint_as_float(__float_as_uint(p1) + (__float_as_uint(t1) << 23));
}

// Scores without a bit in `ok` become -inf.  Whole warps.  A loop, not unrolled code: it runs
// once or twice in a kernel, and fetching its instructions was most of its time.
QSA_DEVICE void mask_tile(uint32_t s_tm, const uint32_t (&ok)[4]) {
#pragma unroll 1
    for (int c = 0; c < 4; ++c) {
        const uint32_t bits = c == 0 ? ok[0] : c == 1 ? ok[1] : c == 2 ? ok[2] : ok[3];
        if (__all_sync(0xffffffffu, bits == ~0u)) continue;
        uint32_t y[32];
        sm100::tmem_ld32(s_tm + c * 32, y);
#pragma unroll
        for (int e = 0; e < 32; ++e)
            if (!(bits >> e & 1)) y[e] = 0xff800000u;
        sm100::tmem_st32(s_tm + c * 32, y);
    }
    sm100::tmem_wait_st();
}

// Softmax of one row's 128 scores: scores in TMEM at s_tm become bf16 probabilities in its
// first 64 columns; the row's maximum, sum and (at o_tm, if there is one) O move along.
// `phalf` learns when the first 64 tokens' are there: their half of O += P V runs under the
// rest.  Whole warps.
//
// The exponential unit does 16 a clock and SM, so 128 x 128 of them take as long as the
// tile's two matrix products; POLY of every 8 pairs go to the FMA pipe instead.
// NaN (and an infinite maximum) must reach the row's output, and exp2_fma does not carry
// them: they turn the maximum, or what is subtracted, into NaN, and with it every other
// probability of the row.
constexpr int POLY = 3;
template <int D>
QSA_DEVICE void soft_tile(uint32_t s_tm, uint32_t o_tm, float sc, bool has_o, float &m, float &l,
                          uint64_t *phalf) {
    // The scores are read twice, 32 at a time: all 128 in registers would spill.
    uint32_t x[2][32];
    float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
    sm100::tmem_ld32_begin(s_tm, x[0]);
#pragma unroll
    for (int c = 0; c < KT; c += 32) {
        uint32_t(&y)[32] = x[(c >> 5) & 1];
        sm100::tmem_ld32_end(y);
        sm100::tmem_ld32_begin(s_tm + (c + 32) % KT, x[1 - ((c >> 5) & 1)]);
#pragma unroll
        for (int e = 0; e < 32; e += 2)
            mx[(e >> 1) & 3] =
                max3(mx[(e >> 1) & 3], __uint_as_float(y[e]), __uint_as_float(y[e + 1]));
    }
    const float mt = max3(max3(mx[0], mx[1], mx[2]), mx[3], mx[3]) * sc;
    const bool grow = !(mt <= m + GROWTH);  // or NaN
    if (__any_sync(0xffffffffu, grow)) {
        const float mn = grow ? mt : m;
        const float f = grow ? fast_exp2(m - mn) : 1.f;
        l *= f;
        m = mn;
        if (has_o) {
#pragma unroll 1
            for (int c = 0; c < D; c += 16) {
                uint32_t y[16];
                sm100::tmem_ld16(o_tm + c, y);
#pragma unroll
                for (int e = 0; e < 16; ++e) y[e] = __float_as_uint(__uint_as_float(y[e]) * f);
                sm100::tmem_st16(o_tm + c, y);
            }
        }
    }
    const float mu = m == -INFINITY ? 0.f : m + (m - m);
    const uint64_t sc2 = pair(sc, sc), mu2 = pair(-mu, -mu);
    uint64_t sum[2] = {0, 0};
#pragma unroll
    for (int c = 0; c < KT; c += 32) {
        uint32_t pk[16];
        uint32_t(&y)[32] = x[(c >> 5) & 1];
        sm100::tmem_ld32_end(y);
        if (c + 32 < KT) sm100::tmem_ld32_begin(s_tm + c + 32, x[1 - ((c >> 5) & 1)]);
#pragma unroll
        for (int e = 0; e < 32; e += 2) {
            float p0, p1;
            const uint64_t z =
                fma2(pair(__uint_as_float(y[e]), __uint_as_float(y[e + 1])), sc2, mu2);
            if ((e >> 1) % 8 * POLY % 8 < POLY) {
                exp2_fma(z, p0, p1);
            } else {
                unpair(z, p0, p1);
                p0 = fast_exp2(p0);
                p1 = fast_exp2(p1);
            }
            sum[(e >> 1) & 1] = add2(sum[(e >> 1) & 1], pair(p0, p1));
            pk[e / 2] = pack_bf16x2(p0, p1);
        }
        sm100::tmem_st16(s_tm + c / 2, pk);
        if (c + 32 == KT / 2) {
            sm100::tmem_wait_st();
            sm100::tc_fence_before();
            sm100::mbar_arrive(phalf);
        }
    }
    float a, b;
    unpair(add2(sum[0], sum[1]), a, b);
    l += a + b;
    sm100::tmem_wait_st();
}

// A pair of bf16 with what is not finite cleared; sets `some` if anything was.
QSA_DEVICE uint32_t finite_pair(uint32_t w, bool &some) {
    const bool lo = (w & 0x7F80u) == 0x7F80u, hi = (w & 0x7F800000u) == 0x7F800000u;
    some |= lo || hi;
    return w & (lo ? 0xFFFF0000u : ~0u) & (hi ? 0x0000FFFFu : ~0u);
}
// In a V tile, clears what is not finite in rows d0 .. d1 - 1 and all of the rows behind
// them.  One warp; true if this lane met something that was not finite.
template <int D>
QSA_DEVICE bool clean_rows(uint8_t *vt, int d0, int d1, int lane) {
    const uint4 zero = make_uint4(0, 0, 0, 0);
    bool some = false;
#pragma unroll 1
    for (int at = 0; at < D / 64; ++at) {
        uint4 *v = reinterpret_cast<uint4 *>(vt + at * ATOM);
#pragma unroll 4
        for (int i = d0 * 8 + lane; i < d1 * 8; i += 32) {
            uint4 x = v[i];
            bool bad = false;
            x.x = finite_pair(x.x, bad);
            x.y = finite_pair(x.y, bad);
            x.z = finite_pair(x.z, bad);
            x.w = finite_pair(x.w, bad);
            if (bad) v[i] = x;
            some |= bad;
        }
#pragma unroll 4
        for (int i = d1 * 8 + lane; i < KT * 8; i += 32) v[i] = zero;
    }
    return some;
}
// Tile j of the segment reaches behind the prefix.
QSA_DEVICE bool has_drafts(const Seg &sg, int j) { return (sg.t0 + j + 1) * KT > sg.P; }

// The tokens of a tile that draft i (-1: none) attends to: the pl (or, below 0, none) that
// are committed, and of the drafts, 0 being token pl, itself and its ancestors.  A parent
// must come before its child; any other value ends the chain.
QSA_DEVICE void visible(const Args &a, const Seg &sg, int i, int pl, uint32_t (&ok)[4]) {
    const int32_t *parent = a.parent + sg.b * a.N;
    int j = i;
#pragma unroll
    for (int w = 3; w >= 0; --w) {
        const int lo = 32 * w - pl;  // the draft at the word's first token
        // (from above the tile, too: a child may lie there)
        uint32_t m = lo >= 0 ? 0u : lo <= -32 ? ~0u : (1u << -lo) - 1;
        while (j >= max(lo, 0)) {
            if (j - lo < 32) m |= 1u << (j - lo);
            const int p = parent[j];
            const bool wrong = (uint32_t)(p + 1) > (uint32_t)j;
            if (wrong && j == i) record_status(a.status, QSA_ERR_DEVICE);
            j = wrong ? -1 : p;
        }
        ok[w] = m;
    }
}

template <int D, int NT>
__global__ void __launch_bounds__(THREADS, 1)
    tree_dense_kernel(const __grid_constant__ CUtensorMap tm_k,
                      const __grid_constant__ CUtensorMap tm_v, const Args a) {
    using C = Cfg<D, NT>;
    constexpr int SL = C::SLOTS;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *sm = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    uint64_t *full = reinterpret_cast<uint64_t *>(sm + C::OFF_BAR), *empty = full + SL;
    uint64_t *dfull = empty + SL, *clean = dfull + SL;  // drafts' values have come; are clean
    uint64_t *sfull = clean + SL, *phalf = sfull + 2, *pready = phalf + 2,
             *odone = pready + 2, *qready = odone + 1;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(qready + 1);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    // The merge may be launched now: its blocks (no room beside this CTA's registers) are handed
    // out as SMs fall free, and have their lengths and indices when the last run ends.
    asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
    Walk<NT> walk;
    if (!walk.start(a, lane)) return;
    if (tid == 0) {
        for (int i = 0; i < SL; ++i) {
            sm100::mbar_init(&full[i], 1);
            sm100::mbar_init(&empty[i], 1);
            sm100::mbar_init(&dfull[i], 1);
            sm100::mbar_init(&clean[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            sm100::mbar_init(&sfull[i], 1);
            sm100::mbar_init(&phalf[i], 128);
            sm100::mbar_init(&pready[i], 128);
        }
        sm100::mbar_init(odone, 1);
        sm100::mbar_init(qready, SOFT);
        *abort_flag = 0;
        sm100::fence_mbar_init();
    }
    if (warp == SOFT / 32 + 1) sm100::tmem_alloc(tmem_slot, 512);
    sm100::tc_fence_before();
    __syncthreads();
    sm100::tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const uint32_t ring = smem_u32(sm + C::OFF_RING);
    auto wait = [&](uint64_t *bar, uint32_t parity) {
        return sm100::mbar_wait(bar, parity & 1, abort_flag, WAIT_NS, a.status);
    };
    Seg sg;

    if (warp == SOFT / 32) {
        // ------------------------------------------------------ producer --
        if (lane == 0) {
            sm100::prefetch_tensormap(&tm_k);
            sm100::prefetch_tensormap(&tm_v);
            uint32_t it = 0, drafts = 0;
            bool dead = false;
            auto put = [&](const CUtensorMap *cache, int64_t tile, bool cleaned) {
                const uint32_t slot = it % SL;
                if (dead || !wait(&empty[slot], (it / SL) + 1)) {
                    dead = true;
                    return;
                }
                // values that are cleaned first complete a barrier of their own
                uint64_t *bar = &full[slot];
                if (cleaned) {
                    sm100::mbar_arrive(bar);
                    bar = &dfull[drafts++ % SL];
                }
                sm100::mbar_arrive_expect_tx(bar, C::TILE);
#pragma unroll
                for (int at = 0; at < D / 64; ++at)
                    sm100::tma_load_3d(ring + slot * C::TILE + at * ATOM, cache, sg.g * D + at * 64,
                                       (int32_t)(tile * KT), (int32_t)sg.b, bar);
                ++it;
            };
            while (walk.next(a, sg)) {
                put(&tm_k, sg.t0, false);
                for (int j = 0; j < sg.n; ++j) {
                    if (NT == 1 && j + 1 < sg.n) put(&tm_k, sg.t0 + j + 1, false);
                    put(&tm_v, sg.t0 + j, has_drafts(sg, j));
                    if (NT == 2 && j + 1 < sg.n) put(&tm_k, sg.t0 + j + 1, false);
                }
            }
            // no copy may land after the CTA has gone
            for (uint32_t i = it > SL ? it - SL : 0; i < it; ++i)
                sm100::mbar_wait_for(&full[i % SL], (i / SL) & 1, 100000000ull);
            for (uint32_t i = drafts > SL ? drafts - SL : 0; i < drafts; ++i)
                sm100::mbar_wait_for(&dfull[i % SL], (i / SL) & 1, 100000000ull);
        }
    } else if (warp == SOFT / 32 + 1) {
        // ----------------------------------------------------------- MMA --
        // The whole warp walks and waits, so that descriptors stay in uniform registers;
        // one lane issues.
        const bool leader = sm100::elect_one();
        const uint32_t qs = smem_u32(sm);
        uint32_t base = 0, done[2] = {0, 0}, segs = 0, cleaned = 0;
        while (walk.next(a, sg)) {
            const int n = __shfl_sync(0xffffffffu, sg.n, 0), steps = NT * n;
            wait(qready, segs);
            sm100::tc_fence_after();
            auto scores = [&](int t) {
                const int s = t & 1;
                const uint32_t idx = ring_k<NT>(base, NT == 2 ? t >> 1 : t), slot = idx % SL;
                if (NT == 1 || s == 0) wait(&full[slot], idx / SL);
                const uint64_t qa = sm100::smem_desc_kmajor(qs + (NT == 2 ? s * C::TILE : 0), 128);
                const uint64_t ka = sm100::smem_desc_kmajor(ring + slot * C::TILE, 128);
                if (leader) {
#pragma unroll
                    for (int k = 0; k < D / 16; ++k) {
                        const uint32_t off = ((k >> 2) * ATOM + (k & 3) * 32) >> 4;
                        sm100::mma_bf16(tmem + s * KT, qa + off, ka + off, C::IDESC_S, k > 0);
                    }
                    sm100::mma_commit(&sfull[s]);
                    if (NT == 1 || s == 1) sm100::mma_commit(&empty[slot]);
                }
            };
            scores(0);
            if (steps > 1) scores(1);
            for (int t = 0; t < steps; ++t) {
                const int s = t & 1;
                const uint32_t idx = ring_v<NT>(base, NT == 2 ? t >> 1 : t, n), slot = idx % SL;
                wait(&phalf[s], done[s]);
                if (NT == 1 || s == 0) {
                    wait(&full[slot], idx / SL);
                    if (has_drafts(sg, NT == 2 ? t >> 1 : t)) {
                        wait(&clean[cleaned % SL], cleaned / SL);
                        ++cleaned;
                    }
                }
                sm100::tc_fence_after();
                const uint64_t va = sm100::smem_desc_mnmajor(ring + slot * C::TILE, ATOM);
                auto weigh = [&](int k) {
                    sm100::mma_bf16_ta(tmem + C::O_COL + s * D, tmem + s * KT + k * 8,
                                       va + k * (2048 >> 4), C::IDESC_O, t > 1 || k > 0);
                };
                if (leader) {
#pragma unroll
                    for (int k = 0; k < KT / 32; ++k) weigh(k);
                }
                wait(&pready[s], done[s]++);
                sm100::tc_fence_after();
                if (leader) {
#pragma unroll
                    for (int k = KT / 32; k < KT / 16; ++k) weigh(k);
                    if (NT == 1 || s == 1) sm100::mma_commit(&empty[slot]);
                }
                if (t + 2 < steps) scores(t + 2);
            }
            if (leader) sm100::mma_commit(odone);
            base += 2 * n;
            ++segs;
        }
    } else if (warp == SOFT / 32 + 2) {
        // ---------------------------------------------------------- clean --
        // V rows of drafts, before they meet zeros: no infinity, no NaN; and none at all
        // behind the drafts.  Such tiles have barriers of their own, in their own order: a
        // wait for a ring slot's parity passes if the phase before has not ended either, and
        // this warp does not wait for the others' phases.  (No more than SLOTS are on their
        // way, so no barrier is a phase ahead.)
        uint32_t base = 0, drafts = 0;
        while (walk.next(a, sg)) {
            const int64_t u = (sg.b * a.Hkv + sg.g) * a.units + sg.qt;
            for (int j = 0; j < sg.n; ++j) {
                if (!has_drafts(sg, j)) continue;
                const int64_t pl = sg.P - (sg.t0 + j) * KT, sl = pl + sg.nd;
                const uint32_t slot = ring_v<NT>(base, j, sg.n) % SL, x = drafts % SL;
                wait(&dfull[x], drafts / SL);
                ++drafts;
                uint8_t *vt = sm + C::OFF_RING + slot * C::TILE;
                const bool some = clean_rows<D>(vt, pl > 0 ? (int)pl : 0, sl < KT ? (int)sl : KT,
                                                lane);
                sm100::fence_async_shared();
                const bool any = __any_sync(0xffffffffu, some);
                __syncwarp();  // a vote orders no memory: all lanes' stores before the arrival
                if (lane == 0) {
                    a.info[u].cleared[sg.t0 + j - sg.P / KT] = any;
                    sm100::mbar_arrive(&clean[x]);
                }
            }
            base += 2 * sg.n;
        }
    } else {
        // ------------------------------------------------------- softmax --
        const int s = warp >> 2, r = tid & 127;
        const uint32_t lanes = (uint32_t)(warp & 3) << 21;  // this warp's quarter of TMEM
        const uint32_t s_tm = tmem + lanes + s * KT, o_tm = tmem + lanes + C::O_COL + s * D;
        // at least FLT_MIN, so that a masked score's -inf stays one at a scale of 0
        const float sc = fmaxf(fabsf(a.scale_log2), 1.17549435e-38f);
        const uint32_t flip = a.scale_log2 < 0.f ? 0x80008000u : 0u;  // the sign moves into Q
        constexpr int QB = D / 16;  // loads in flight
        float2 *s_ml = reinterpret_cast<float2 *>(sm);  // [2][128]: the query tile, once done with
        uint32_t base = 0, got = 0, segs = 0;
        while (walk.next(a, sg)) {
            const int steps = NT * sg.n;
            const int R = sg.nd * a.G, r0 = sg.qt * 128 * NT;
            const uint16_t *qb = a.q + (sg.b * a.N * a.Hq + sg.g * a.G) * D;
            if (segs > 0) soft_sync();  // the sums have been read
            if (sg.ends && tid < sg.nd)  // into L1, for the masks
                asm volatile("{\n\t.reg .b32 x;\n\tld.global.ca.b32 x, [%0];\n\t}\n" ::"l"(
                                 a.parent + sg.b * a.N + tid)
                             : "memory");
            // all of a thread's loads at once: one after the other they took 7 us
#pragma unroll 1
            for (int i0 = tid; i0 < NT * 128 * (D / 8); i0 += SOFT * QB) {
                uint4 x[QB];
#pragma unroll
                for (int e = 0; e < QB; ++e) {
                    const int i = i0 + e * SOFT, rr = r0 + i / (D / 8);
                    x[e] = make_uint4(0, 0, 0, 0);
                    if (rr < R)
                        x[e] = *reinterpret_cast<const uint4 *>(
                            qb + ((int64_t)(rr >> a.lg) * a.Hq + (rr & (a.G - 1))) * D +
                            i % (D / 8) * 8);
                }
#pragma unroll
                for (int e = 0; e < QB; ++e) {
                    const int i = i0 + e * SOFT, row = i / (D / 8), ch = i % (D / 8);
                    x[e].x ^= flip; x[e].y ^= flip; x[e].z ^= flip; x[e].w ^= flip;
                    *reinterpret_cast<uint4 *>(sm + (row >> 7) * C::TILE + (ch >> 3) * ATOM +
                                               (row & 127) * 128 + (((ch ^ row) & 7) << 4)) = x[e];
                }
            }
            sm100::fence_async_shared();
            sm100::tc_fence_before();
            sm100::mbar_arrive(qready);
            if (tid == 0) {
                const int64_t u = (sg.b * a.Hkv + sg.g) * a.units + sg.qt;
                if (sg.begins) a.info[u].first = blockIdx.x;
                if (sg.ends) a.info[u].last = blockIdx.x;
            }
            const int row = r0 + (NT == 2 ? s * 128 : 0) + r;
            const bool on = __any_sync(0xffffffffu, row < R);  // a live row in this warp
            float m = -INFINITY, l = 0.f;
            for (int t = s; t < steps; t += 2) {
                const int j = NT == 2 ? t >> 1 : t;
                uint32_t ok[4];
                const bool drafts = has_drafts(sg, j);
                if (drafts)  // the mask while the tile is on its way
                    visible(a, sg, row < R ? row >> a.lg : -1, (int)(sg.P - (sg.t0 + j) * KT), ok);
                wait(&sfull[s], got++);
                sm100::tc_fence_after();
                if (on) {
                    if (drafts) mask_tile(s_tm, ok);
                    soft_tile<D>(s_tm, o_tm, sc, t > 1, m, l, &phalf[s]);
                } else {
                    sm100::mbar_arrive(&phalf[s]);
                }
                sm100::tc_fence_before();
                sm100::mbar_arrive(&pready[s]);
            }
            wait(odone, segs);
            sm100::tc_fence_after();
            const int64_t unit = (sg.b * a.Hkv + sg.g) * a.units + sg.qt;
            const int64_t slot_row = (blockIdx.x + unit) * a.rows;
            if (NT == 2) {
                if (on) {
                    float *out = a.part + (slot_row + s * 128 + r) * D;
#pragma unroll 1
                    for (int c = 0; c < D; c += 32) {
                        uint32_t y[32];
                        sm100::tmem_ld32(o_tm + c, y);
                        if (row < R)
#pragma unroll
                            for (int e = 0; e < 32; e += 8) store_sector(out + c + e, y + e);
                    }
                    if (row < R)
                        *reinterpret_cast<float2 *>(a.ml + (slot_row + s * 128 + r) * 2) =
                            make_float2(m, l);
                }
            } else {
                // the streams' parts become one; each writes half of the columns
                s_ml[s * 128 + r] = make_float2(m, l);
                soft_sync();
                if (on) {
                    const float2 w0 = s_ml[r], w1 = s_ml[128 + r];
                    const float M = fmaxf(w0.x, w1.x), Mu = M == -INFINITY ? 0.f : M;
                    const float f0 = fast_exp2(w0.x - Mu), f1 = fast_exp2(w1.x - Mu);
                    float *out = a.part + (slot_row + r) * D;
#pragma unroll 1
                    for (int c = s * (D / 2); c < (s + 1) * (D / 2); c += 32) {
                        uint32_t y[32], z[32];
                        sm100::tmem_ld32(tmem + lanes + C::O_COL + c, y);
                        if (steps > 1) {
                            sm100::tmem_ld32(tmem + lanes + C::O_COL + D + c, z);
                        } else {
#pragma unroll
                            for (int e = 0; e < 32; ++e) z[e] = 0;
                        }
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            y[e] = __float_as_uint(__uint_as_float(y[e]) * f0 +
                                                   __uint_as_float(z[e]) * f1);
                        if (row < R)
#pragma unroll
                            for (int e = 0; e < 32; e += 8) store_sector(out + c + e, y + e);
                    }
                    if (row < R && s == 0)
                        *reinterpret_cast<float2 *>(a.ml + (slot_row + r) * 2) =
                            make_float2(M, w0.y * f0 + w1.y * f1);
                }
            }
            base += 2 * sg.n;
            ++segs;
        }
    }
    sm100::tc_fence_before();
    __syncthreads();
    sm100::tc_fence_after();
    if (warp == SOFT / 32 + 1) sm100::tmem_dealloc(tmem, 512);
}

// ------------------------------------------------------------------ merge --
// A (row, head) in a group of LANES lanes, E dims a lane: running (max, sum, O).
template <int D, int LANES>
struct Row {
    static constexpr int E = D / LANES;
    float o[E];
    float m, l;

    struct Raw {
        uint4 v[E / 8];
        QSA_DEVICE void load(const uint16_t *p) {
#pragma unroll
            for (int i = 0; i < E / 8; ++i) v[i] = reinterpret_cast<const uint4 *>(p)[i];
        }
        QSA_DEVICE void get(float (&f)[E]) const {
#pragma unroll
            for (int i = 0; i < E / 8; ++i) {
                const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    f[8 * i + 2 * j] = bf16_lo(w[j]);
                    f[8 * i + 2 * j + 1] = bf16_hi(w[j]);
                }
            }
        }
    };
    QSA_DEVICE void start() {
        m = -INFINITY;
        l = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] = 0.f;
    }
    // (max, sum, O) of another part joins this one
    QSA_DEVICE void join(float m2, float l2, const float (&o2)[E]) {
        const float mn = fmaxf(m, m2);
        const float mu = mn == -INFINITY ? 0.f : mn;
        const float fa = fast_exp2(m - mu), fb = fast_exp2(m2 - mu);
        l = l * fa + l2 * fb;
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] = o[e] * fa + o2[e] * fb;
        m = mn;
    }
    // of a token that is in m and l already, the values that are not finite (all lanes call)
    QSA_DEVICE void patch(const Raw &q, const Raw &k, const Raw &v, bool on, float scale_log2) {
        float f[E], x = 0.f;
        {
            float g[E];
            q.get(g);
            k.get(f);
#pragma unroll
            for (int e = 0; e < E; ++e) x += g[e] * f[e];
        }
#pragma unroll
        for (int i = 1; i < LANES; i <<= 1) x += __shfl_xor_sync(0xffffffffu, x, i);
        const float p = fast_exp2(x * scale_log2 - (m == -INFINITY ? 0.f : m));
        v.get(f);
#pragma unroll
        for (int e = 0; e < E; ++e)
            if (on && !(fabsf(f[e]) < INFINITY)) o[e] += p * f[e];
    }
    // the parts of the warp's groups become one, in every lane
    QSA_DEVICE void join_groups() {
#pragma unroll
        for (int x = LANES; x < 32; x <<= 1) {
            float o2[E];
            const float m2 = __shfl_xor_sync(0xffffffffu, m, x);
            const float l2 = __shfl_xor_sync(0xffffffffu, l, x);
#pragma unroll
            for (int e = 0; e < E; ++e) o2[e] = __shfl_xor_sync(0xffffffffu, o[e], x);
            join(m2, l2, o2);
        }
    }
};

// The parts of a (row, head) are shared out over the groups of W warps, or (W = 0) are all
// one group's; the loads of U of them are issued together.  Groups of D / 8 lanes keep the
// registers down to 64, four blocks an SM.  A group of 8 lanes alone (W = 0) takes a part at a
// time: with a part or two to a pair what a warp does once is most of it (D = 64, 8192 pairs
// 21.2 us, with two together 22.7).
template <int D, bool SPARSE, int W, int LANES>
__global__ void __launch_bounds__(256, W == 1 || (W == 0 && LANES == 16) ? 4 : 3)
    tree_merge_kernel(const Args a) {
    constexpr int GROUPS = 32 / LANES;
    using R = Row<D, LANES>;
    constexpr int E = R::E, STEP = W == 0 ? 1 : GROUPS * W, U = W == 0 && LANES == 8 ? 1 : 2;
    __shared__ float s_o[W > 1 ? W : 1][W > 1 ? D : 1], s_m[W > 1 ? W : 1], s_l[W > 1 ? W : 1];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, li = lane % LANES;
    // (row, head) pairs: a block's (W > 1), a warp's, a group's
    const int64_t pairs = (int64_t)a.B * a.N * a.Hq;
    const int64_t pair = W > 1    ? blockIdx.x
                         : W == 1 ? (int64_t)blockIdx.x * 8 + warp
                                  : ((int64_t)blockIdx.x * 8 + warp) * GROUPS + lane / LANES;
    const int64_t row = pair / a.Hq, b = row / a.N;
    const int h = (int)(pair - row * a.Hq), i = (int)(row - b * a.N);
    const int first = W == 0 ? 0 : (W > 1 ? warp * GROUPS : 0) + lane / LANES;
    Seq sq{0, 0, false};
    if (pair < pairs) sq = a.lens.at(b);
    if (sq.bad && i == 0 && h == 0 && li == 0) record_status(a.status, QSA_ERR_DEVICE);
    const bool live = pair < pairs && (sq.bad || i < sq.n);
    R r;
    r.start();
    // The prefix kernel's parts; and without a row to write too: what follows in the stream
    // starts when this kernel has ended, and may change lengths that the prefix kernel still
    // reads.
    griddep_wait();
    if (W > 0 && !live) return;  // whole warps and blocks; groups stay for the shuffles
    int64_t x0 = 0;
    int parts = 0;
    bool patch = false;  // values of drafts were not finite
    if (live && !sq.bad) {
        // unit and row in it
        const int rr = SPARSE ? h : (i << a.lg) + (h & (a.G - 1)), qt = rr / a.rows;
        const int64_t u = SPARSE ? row : (b * a.Hkv + (h >> a.lg)) * a.units + qt;
        const UnitInfo &info = a.info[u];
        x0 = (info.first + u) * a.rows + (rr - qt * a.rows);
        parts = info.last - info.first + 1;
        if (!SPARSE)
            for (int k = 0; k <= (int)((sq.P + sq.n - 1) / KT - sq.P / KT); ++k)
                patch |= info.cleared[k] != 0;
    }
    for (int s = first; s < parts; s += U * STEP) {
        float2 ml[U];
        float4 f[U][E / 4];
#pragma unroll
        for (int n = 0; n < U; ++n) {
            if (s + n * STEP >= parts) continue;
            const int64_t x = x0 + (int64_t)(s + n * STEP) * a.rows;
            ml[n] = *reinterpret_cast<const float2 *>(a.ml + x * 2);
#pragma unroll
            for (int e = 0; e < E / 4; ++e)
                f[n][e] = reinterpret_cast<const float4 *>(a.part + x * D + li * E)[e];
        }
#pragma unroll
        for (int n = 0; n < U; ++n) {
            if (s + n * STEP >= parts) continue;
            float o2[E];
#pragma unroll
            for (int e = 0; e < E / 4; ++e) {
                o2[4 * e] = f[n][e].x;
                o2[4 * e + 1] = f[n][e].y;
                o2[4 * e + 2] = f[n][e].z;
                o2[4 * e + 3] = f[n][e].w;
            }
            r.join(ml[n].x, ml[n].y, o2);
        }
    }
    __syncwarp();
    if (W > 0) r.join_groups();
    if (W > 1) {
        if (lane < LANES) {
#pragma unroll
            for (int e = 0; e < E; ++e) s_o[warp][li * E + e] = r.o[e];
            if (li == 0) {
                s_m[warp] = r.m;
                s_l[warp] = r.l;
            }
        }
        __syncthreads();
        if (warp != 0) return;
        // group g of warp 0 takes the sums of warps g, g + GROUPS, ...
        r.start();
#pragma unroll
        for (int w = 0; w < W; w += GROUPS) {
            float o2[E];
            const int ww = w + lane / LANES;
#pragma unroll
            for (int e = 0; e < E; ++e) o2[e] = s_o[ww][li * E + e];
            r.join(s_m[ww], s_l[ww], o2);
        }
        r.join_groups();
    }
    // what was cleared in the chain's values (W > 0: all groups the same token)
    if (!SPARSE && __any_sync(0xffffffffu, patch)) {
        typename R::Raw q, k, v;
        const int64_t tok = (int64_t)a.Hkv * D;
        const int64_t base = (b * a.lens.L_max + sq.P) * tok + (h >> a.lg) * D + li * E;
        q.load(a.q + (patch ? pair : 0) * D + li * E);
        for (int j = patch ? i : -1; __any_sync(0xffffffffu, j >= 0);) {
            const int64_t at = j >= 0 ? base + j * tok : 0;
            k.load(a.k + at);
            v.load(a.v + at);
            r.patch(q, k, v, j >= 0, a.scale_log2);
            if (j >= 0) {
                const int p = a.parent[b * a.N + j];
                j = (uint32_t)(p + 1) > (uint32_t)j ? -1 : p;
            }
        }
    }
    if (live && (W == 0 || lane < LANES)) {
        const float inv = r.l == 0.f ? 0.f : 1.f / r.l;
        uint16_t *orow = a.o + pair * D + li * E;
#pragma unroll
        for (int e = 0; e < E; e += 8)
            *reinterpret_cast<uint4 *>(orow + e) =
                make_uint4(pack_bf16x2(r.o[e] * inv, r.o[e + 1] * inv),
                           pack_bf16x2(r.o[e + 2] * inv, r.o[e + 3] * inv),
                           pack_bf16x2(r.o[e + 4] * inv, r.o[e + 5] * inv),
                           pack_bf16x2(r.o[e + 6] * inv, r.o[e + 7] * inv));
        if (a.lse && li == 0)
            a.lse[pair] = r.l == 0.f ? -INFINITY : (r.m + __log2f(r.l)) * LN2;
    }
}

// ------------------------------------------------------------------- host --

// Rows of a unit, units of a (sequence, KV head).
int unit_tiles(int N, int G) { return N * G > 128 ? 2 : 1; }
int unit_rows(int N, int G) {
    const int most = 128 * unit_tiles(N, G);
    return N * G < most ? N * G : most;
}
int unit_count(int N, int G) { return (N * G + unit_rows(N, G) - 1) / unit_rows(N, G); }

// Offsets from the workspace's first multiple of 32 bytes: a caller's need only be aligned to
// 16, and the parts are stored by whole sectors.
struct Workspace {
    size_t info, part, ml, bytes;
    Workspace(size_t ctas, size_t units, size_t rows, size_t D) {
        info = kWsHeader;
        part = info + (units * sizeof(UnitInfo) + 255) / 256 * 256;
        ml = part + (ctas + units) * rows * D * 4;
        bytes = ml + (ctas + units) * rows * 8 + 16;
    }
    static uint8_t *base(void *ws) {
        return reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(ws) + 31) / 32 * 32);
    }
};
Workspace dense_ws(int B, int N, int Hkv, int G, int D) {
    return Workspace(MAX_CTAS, (size_t)B * Hkv * unit_count(N, G), unit_rows(N, G), D);
}
Workspace sparse_ws(int B, int N, int Hq, int D) {
    return Workspace(tree_sparse_ctas(MAX_CTAS), (size_t)B * N, Hq, D);
}

template <int D, int NT>
cudaError_t run_dense(const CUtensorMap &tk, const CUtensorMap &tv, const Args &a, int ctas,
                      cudaStream_t s) {
    auto kern = tree_dense_kernel<D, NT>;
    const cudaError_t e = ensure_smem(reinterpret_cast<const void *>(kern), Cfg<D, NT>::BYTES);
    if (e != cudaSuccess) return e;
    kern<<<ctas, THREADS, Cfg<D, NT>::BYTES, s>>>(tk, tv, a);
    return cudaGetLastError();
}

// 8 warps a (row, head) where all of them run at once (3 blocks on each SM), and in two rounds
// where a unit, as the grid is shared out, has 16 parts or more.  A group from two rounds of 24
// warps an SM on, a warp between.  The group has D / 8 lanes from two parts a unit on, else 8.
// Whole calls of dense trees, 16 heads, on three sets of tensors in turn (us; D = 128 / 64):
//   pairs of parts   8 warps      a warp       D / 8 lanes  8 lanes
//      112 of   8    12.3 / 11.2  12.6 / 11.3  13.0 / 12.3  14.8 / 12.3
//      448 of  37    28.9 / 22.6  33.8 / 24.2  39.8 / 28.9  57.6 / 28.9
//      768 of  18    17.5 / 16.4  19.0 / 14.5  22.3 / 18.1  32.5 / 18.1
//      640 of   5    22.5 / 18.5  20.9 / 16.4  21.9 / 16.6  24.2 / 16.7   (8 heads)
//     1280 of  18    22.6 / 20.5  22.5 / 18.5  26.5 / 20.5  37.0 / 20.5
//     4096 of   9                  162 / 113    166 / 114    176 / 114
//     8192 of   5                 38.7 / 39.7  35.5 / 33.9  38.2 / 33.6
//    32768 of   1                 38.9 / 34.8  30.5 / 22.6  29.2 / 22.6
// Sparse (a unit is a row, three CTAs an SM), D = 128: 256 pairs of 28 parts 12.7 us with 8 warps,
// 16.0 with one; 640 of 22 22.3 and 22.4, with a budget of 512 13.9 and 15.3; 1280 of 6 30.2 and
// 27.2.
template <int D, bool SPARSE>
cudaError_t run_merge(const Args &a, int ctas, int sms, cudaStream_t s) {
    const int64_t pairs = (int64_t)a.B * a.N * a.Hq;
    const int64_t units = (int64_t)a.B * (SPARSE ? a.N : a.Hkv * a.units);
    auto launch = [&](auto kern, int per) {
        return launch_dependent(kern, dim3((unsigned)((pairs + per - 1) / per)), dim3(256), 0, s, a);
    };
    constexpr int L = D / 8;
    if (pairs <= (int64_t)sms * (ctas >= 16 * units ? 6 : 3))
        return launch(tree_merge_kernel<D, SPARSE, 8, L>, 1);
    if (pairs <= (int64_t)sms * 48) return launch(tree_merge_kernel<D, SPARSE, 1, L>, 8);
    // (so many pairs of a sparse call have a part or two each)
    if constexpr (!SPARSE)
        if (ctas >= 2 * units) return launch(tree_merge_kernel<D, SPARSE, 0, L>, 8 * 32 / L);
    return launch(tree_merge_kernel<D, SPARSE, 0, 8>, 32);
}

}  // namespace tree

size_t tree_dense_ws_bytes(int B, int N, int Hq, int Hkv, int D) {
    return tree::dense_ws(B, N, Hkv, Hq / Hkv, D).bytes;
}

size_t tree_sparse_ws_bytes(int B, int N, int Hq, int D) {
    return tree::sparse_ws(B, N, Hq, D).bytes;
}

cudaError_t launch_tree_decode(const uint16_t *q, const uint16_t *k, const uint16_t *v,
                               const int32_t *seqlens, const int32_t *n_draft, int64_t L_max,
                               const int32_t *sel, int64_t sel_b, int64_t sel_n, int kb,
                               const int32_t *parent, int B, int N, int Hq, int Hkv, int D,
                               float scale, uint16_t *o, float *lse, void *ws, int num_sms,
                               cudaStream_t s) {
    tree::Args a{};
    uint8_t *w = tree::Workspace::base(ws);
    a.q = q; a.k = k; a.v = v; a.lens = tree::Lens{seqlens, n_draft, N, L_max};
    a.parent = parent; a.B = B; a.N = N; a.Hq = Hq; a.Hkv = Hkv; a.G = Hq / Hkv;
    while (1 << a.lg < a.G) ++a.lg;  // 1, 2, 4 or 8 heads to a KV head
    a.scale_log2 = scale * tree::LOG2E; a.o = o; a.lse = lse; a.status = ws;
    const tree::Workspace x =
        sel ? tree::sparse_ws(B, N, Hq, D) : tree::dense_ws(B, N, Hkv, a.G, D);
    a.info = reinterpret_cast<tree::UnitInfo *>(w + x.info);
    a.part = reinterpret_cast<float *>(w + x.part);
    a.ml = reinterpret_cast<float *>(w + x.ml);
    const int sms = num_sms < tree::MAX_CTAS ? num_sms : tree::MAX_CTAS;
    const int ctas = sel ? tree_sparse_ctas(sms) : sms;
    cudaError_t e;
    if (sel) {
        a.units = 1;
        a.rows = Hq;
        const TreePrefix t{seqlens, n_draft, parent, N, sel, sel_b, sel_n, kb, a.part, a.ml, &a.info->first, &a.info->last,
                           sizeof(tree::UnitInfo) / 4};
        e = launch_tree_sparse_prefix(q, k, v, t, L_max, B, Hq, Hkv, D, scale, ws,
                                      ctas, s);
    } else {
        a.units = tree::unit_count(N, a.G);
        a.rows = tree::unit_rows(N, a.G);
        CUtensorMap tk, tv;
        if (!tensor_map_cache_bf16(&tk, k, B, L_max, Hkv * D, tree::KT) ||
            !tensor_map_cache_bf16(&tv, v, B, L_max, Hkv * D, tree::KT))
            return cudaErrorInvalidValue;
        const bool two = tree::unit_tiles(N, a.G) == 2;
        if (D == 64)
            e = two ? tree::run_dense<64, 2>(tk, tv, a, ctas, s)
                    : tree::run_dense<64, 1>(tk, tv, a, ctas, s);
        else
            e = two ? tree::run_dense<128, 2>(tk, tv, a, ctas, s)
                    : tree::run_dense<128, 1>(tk, tv, a, ctas, s);
    }
    if (e != cudaSuccess) return e;
    if (sel) return D == 64 ? tree::run_merge<64, true>(a, ctas, sms, s)
                            : tree::run_merge<128, true>(a, ctas, sms, s);
    return D == 64 ? tree::run_merge<64, false>(a, ctas, sms, s)
                   : tree::run_merge<128, false>(a, ctas, sms, s);
}

}  // namespace qsa
