// Attention for a tree of drafted tokens over the caches, dense and over selected
// micro-blocks: the decode step that verifies several drafted tokens at once.
//
// Sequence b holds seqlens[b] tokens, the last n of them (n = n_draft[b]) drafts:
// draft i lies in cache row P + i, P = seqlens[b] - n, whatever its depth.  Row i
// attends to the prefix u < P (dense) or to the prefix tokens of its selected
// blocks and the unpooled tail (sparse), and to its own chain i, parent[i],
// parent[parent[i]], ...: softmax over both parts together.
//
// The two parts are kept apart.  The prefix has no mask that differs between rows.
// The chain is a handful of tokens with a mask of its own per row: it is walked
// token by token in fp32, so what a masked draft's cache rows hold (infinities,
// NaN) never enters another branch, as a zero times it in a matrix product would.
// Both parts leave (max, sum, O) and meet in tree_merge_kernel.
#include "qsa_common.cuh"
#include "qsa_launch.h"

namespace qsa {

namespace tree {

constexpr int MAX_N = 256;  // drafts per sequence
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

// One query head against single tokens: 4 groups of 8 lanes take a token each; a
// lane holds E = D / 8 dims.  Running (max, sum, O) per group, in base 2.
template <int D>
struct Row {
    static constexpr int E = D / 8;
    float q[E], o[E];
    float m, l;

    QSA_DEVICE static void load16(const uint16_t *p, float (&f)[E]) {
#pragma unroll
        for (int i = 0; i < E / 8; ++i) {
            const uint4 v = reinterpret_cast<const uint4 *>(p)[i];
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                f[8 * i + 2 * j] = bf16_lo(w[j]);
                f[8 * i + 2 * j + 1] = bf16_hi(w[j]);
            }
        }
    }
    QSA_DEVICE void start(const uint16_t *qrow, int li) {
        load16(qrow + li * E, q);
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
    // token with cache rows k and v; `on` false: the group sits out (all lanes call)
    QSA_DEVICE void token(const uint16_t *k, const uint16_t *v, bool on, int li,
                          float scale_log2) {
        float f[E];
        float x = 0.f;
        if (on) {
            load16(k + li * E, f);
#pragma unroll
            for (int e = 0; e < E; ++e) x += q[e] * f[e];
        }
        x += __shfl_xor_sync(0xffffffffu, x, 1);
        x += __shfl_xor_sync(0xffffffffu, x, 2);
        x += __shfl_xor_sync(0xffffffffu, x, 4);
        if (!on) return;
        load16(v + li * E, f);
        x *= scale_log2;
        const float mn = fmaxf(m, x);
        const float mu = mn == -INFINITY ? 0.f : mn;
        const float fa = fast_exp2(m - mu), p = fast_exp2(x - mu);
        l = l * fa + p;
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] = o[e] * fa + p * f[e];
        m = mn;
    }
    // the four groups' parts become one, in every lane
    QSA_DEVICE void join_groups() {
#pragma unroll
        for (int x = 8; x < 32; x <<= 1) {
            float o2[E];
            const float m2 = __shfl_xor_sync(0xffffffffu, m, x);
            const float l2 = __shfl_xor_sync(0xffffffffu, l, x);
#pragma unroll
            for (int e = 0; e < E; ++e) o2[e] = __shfl_xor_sync(0xffffffffu, o[e], x);
            join(m2, l2, o2);
        }
    }
};

struct Args {
    const uint16_t *q;   // [B, N, Hq, D]
    const uint16_t *k;   // [B, L_max, Hkv, D]
    const uint16_t *v;
    Lens lens;
    const int32_t *parent;  // [B, N]
    const int32_t *sel;     // selected blocks of row (b, i) at b * sel_b + i * sel_n
    int64_t sel_b, sel_n;
    int kb;
    int N, Hq, Hkv, G, nsplit;
    float scale_log2;
    float *part;            // [B * N, nsplit, Hq, D + 2]
    uint16_t *o;
    float *lse;
    void *status;
};

constexpr int WARPS = 4;

// Prefix part of row (b, i), heads in warps, one slice of its tokens per block.
template <int D, bool SPARSE>
__global__ void __launch_bounds__(WARPS * 32) tree_prefix_kernel(const Args a) {
    const int64_t row = blockIdx.x / a.nsplit;
    const int split = (int)(blockIdx.x - row * a.nsplit);
    const int64_t b = row / a.N;
    const int i = (int)(row - b * a.N);
    const Seq sq = a.lens.at(b);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, grp = lane >> 3, li = lane & 7;
    const int h = blockIdx.y * WARPS + warp;
    if (i >= sq.n || h >= a.Hq) return;
    const int64_t tok = (int64_t)a.Hkv * D;
    const uint16_t *k = a.k + b * a.lens.L_max * tok + (h / a.G) * D;
    const uint16_t *v = a.v + b * a.lens.L_max * tok + (h / a.G) * D;
    Row<D> r;
    r.start(a.q + (row * a.Hq + h) * D, li);
    if (SPARSE) {
        const int64_t whole = sq.P / 4;
        const int chunk = (a.kb + a.nsplit - 1) / a.nsplit;
        const int e1 = min((split + 1) * chunk, a.kb);
        const int32_t *sel = a.sel + b * a.sel_b + i * a.sel_n;
        for (int e = split * chunk; e < e1; ++e) {
            const int64_t j = sel[e];
            const bool on = j >= 0 && j < whole;
            const int64_t u = on ? j * 4 + grp : 0;
            r.token(k + u * tok, v + u * tok, on, li, a.scale_log2);
        }
        if (split == 0) {
            const int64_t u = whole * 4 + grp;
            const bool on = u < sq.P;
            r.token(k + (on ? u : 0) * tok, v + (on ? u : 0) * tok, on, li, a.scale_log2);
        }
    } else {
        const int64_t chunk = (sq.P + a.nsplit - 1) / a.nsplit;
        const int64_t u1 = min((split + 1) * chunk, sq.P);
        for (int64_t u0 = split * chunk; u0 < u1; u0 += 4) {
            const bool on = u0 + grp < u1;
            const int64_t u = on ? u0 + grp : 0;
            r.token(k + u * tok, v + u * tok, on, li, a.scale_log2);
        }
    }
    r.join_groups();
    float *pp = a.part + ((row * a.nsplit + split) * a.Hq + h) * (D + 2);
    if (grp == 0) {
#pragma unroll
        for (int e = 0; e < Row<D>::E; ++e) pp[li * Row<D>::E + e] = r.o[e];
        if (li == 0) {
            pp[D] = r.m;
            pp[D + 1] = r.l;
        }
    }
}

// Chain part and merge: a warp per (row, head).
template <int D>
__global__ void __launch_bounds__(WARPS * 32) tree_merge_kernel(const Args a) {
    constexpr int E = Row<D>::E;
    __shared__ int s_par[MAX_N];
    const int64_t row = blockIdx.x;
    const int64_t b = row / a.N;
    const int i = (int)(row - b * a.N);
    const Seq sq = a.lens.at(b);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, grp = lane >> 3, li = lane & 7;
    const int h = blockIdx.y * WARPS + warp;
    if (sq.bad) {
        if (i == 0 && blockIdx.y == 0 && threadIdx.x == 0) record_status(a.status, QSA_ERR_DEVICE);
    } else if (i >= sq.n) {
        return;
    }
    // a parent must come before its child; any other value ends the chain
    for (int j = threadIdx.x; j <= i && j < sq.n; j += WARPS * 32) {
        int p = a.parent[b * a.N + j];
        if (p < -1 || p >= j) {
            record_status(a.status, QSA_ERR_DEVICE);
            p = -1;
        }
        s_par[j] = p;
    }
    __syncthreads();
    griddep_wait();  // the prefix parts
    if (h >= a.Hq) return;
    Row<D> r;
    r.start(a.q + (row * a.Hq + h) * D, li);
    if (!sq.bad) {
        const int64_t tok = (int64_t)a.Hkv * D;
        const int64_t base = (b * a.lens.L_max + sq.P) * tok + (h / a.G) * D;
        for (int j = i; j >= 0;) {
            int mine = -1;  // four steps of the chain, one a group
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                if (s == grp) mine = j;
                if (j >= 0) j = s_par[j];
            }
            const int64_t at = base + (int64_t)(mine < 0 ? 0 : mine) * tok;
            r.token(a.k + at, a.v + at, mine >= 0, li, a.scale_log2);
        }
        for (int s = grp; s < a.nsplit; s += 4) {
            const float *pp = a.part + ((row * a.nsplit + s) * a.Hq + h) * (D + 2);
            float o2[E];
#pragma unroll
            for (int e = 0; e < E; ++e) o2[e] = pp[li * E + e];
            r.join(pp[D], pp[D + 1], o2);
        }
    }
    r.join_groups();
    if (grp == 0) {
        const float inv = r.l > 0.f ? 1.f / r.l : 0.f;
        uint16_t *orow = a.o + (row * a.Hq + h) * D + li * E;
#pragma unroll
        for (int e = 0; e < E; e += 2)
            reinterpret_cast<uint32_t *>(orow)[e / 2] = pack_bf16x2(r.o[e] * inv, r.o[e + 1] * inv);
        if (a.lse && li == 0)
            a.lse[row * a.Hq + h] = r.l > 0.f ? (r.m + __log2f(r.l)) * LN2 : -INFINITY;
    }
}

int splits(int B, int N, int Hq) {
    const int64_t blocks = (int64_t)B * N * ((Hq + WARPS - 1) / WARPS);
    int64_t ns = (148 * 8 + blocks - 1) / blocks;
    return (int)(ns < 1 ? 1 : ns > 32 ? 32 : ns);
}

template <int D>
cudaError_t run(const Args &a, int B, cudaStream_t s) {
    const int64_t rows = (int64_t)B * a.N;
    const unsigned hy = (a.Hq + WARPS - 1) / WARPS;
    const dim3 pg((unsigned)(rows * a.nsplit), hy);
    if (a.sel)
        tree_prefix_kernel<D, true><<<pg, WARPS * 32, 0, s>>>(a);
    else
        tree_prefix_kernel<D, false><<<pg, WARPS * 32, 0, s>>>(a);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    return launch_dependent(tree_merge_kernel<D>, dim3((unsigned)rows, hy), dim3(WARPS * 32), 0, s,
                            a);
}

}  // namespace tree

int tree_max_drafts() { return tree::MAX_N; }

size_t tree_ws_bytes(int B, int N, int Hq, int D) {
    return kWsHeader +
           (size_t)B * N * tree::splits(B, N, Hq) * Hq * (D + 2) * sizeof(float);
}

cudaError_t launch_tree_decode(const uint16_t *q, const uint16_t *k, const uint16_t *v,
                               const int32_t *seqlens, const int32_t *n_draft, int64_t L_max,
                               const int32_t *sel, int64_t sel_b, int64_t sel_n, int kb,
                               const int32_t *parent, int B, int N, int Hq, int Hkv, int D,
                               float scale, uint16_t *o, float *lse, void *ws, cudaStream_t s) {
    tree::Args a{};
    a.q = q; a.k = k; a.v = v; a.lens = tree::Lens{seqlens, n_draft, N, L_max};
    a.parent = parent; a.sel = sel; a.sel_b = sel_b; a.sel_n = sel_n; a.kb = kb;
    a.N = N; a.Hq = Hq; a.Hkv = Hkv; a.G = Hq / Hkv; a.nsplit = tree::splits(B, N, Hq);
    a.scale_log2 = scale * tree::LOG2E;
    a.part = reinterpret_cast<float *>(static_cast<uint8_t *>(ws) + kWsHeader);
    a.o = o; a.lse = lse; a.status = ws;
    return D == 64 ? tree::run<64>(a, B, s) : tree::run<128>(a, B, s);
}

}  // namespace qsa
