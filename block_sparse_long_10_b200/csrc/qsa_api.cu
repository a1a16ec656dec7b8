// libqsa C ABI: argument validation, device checks, workspace layout and
// launches.  Every entry point validates on the host first and returns before
// touching the CUDA runtime when an argument is wrong, so argument errors are
// reported identically with or without a GPU.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>
#include <string.h>

#include <atomic>
#include <mutex>

#include "../../include/qsa.h"
#include "qsa_launch.h"

namespace {

constexpr int kMaxDevices = 64;
constexpr size_t kHeader = 256;

struct DeviceInfo {
    std::atomic<int> state{0};  // 0 unknown, 1 sm_100, 2 other arch
    int num_sms = 0;
};
DeviceInfo g_dev[kMaxDevices];
std::mutex g_dev_mu;

// QSA_OK and the SM count of the current device, or an error.
qsa_status_t current_device(int *num_sms) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) {
        cudaGetLastError();
        return QSA_ERR_CUDA;
    }
    DeviceInfo &d = g_dev[dev];
    int st = d.state.load(std::memory_order_acquire);
    if (st == 0) {
        std::lock_guard<std::mutex> lk(g_dev_mu);
        st = d.state.load(std::memory_order_relaxed);
        if (st == 0) {
            int major = 0, minor = 0, sms = 0;
            if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) !=
                    cudaSuccess ||
                cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) !=
                    cudaSuccess ||
                cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) !=
                    cudaSuccess) {
                cudaGetLastError();
                return QSA_ERR_CUDA;
            }
            d.num_sms = sms;
            st = (major == 10 && minor == 0) ? 1 : 2;
            d.state.store(st, std::memory_order_release);
        }
    }
    if (st != 1) return QSA_ERR_ARCH;
    *num_sms = d.num_sms;
    return QSA_OK;
}

qsa_status_t from_cuda(cudaError_t e) { return e == cudaSuccess ? QSA_OK : QSA_ERR_CUDA; }

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

bool supported_attn(int Hq, int Hkv, int D) {
    if (D != 64 && D != 128) return false;
    if (Hkv != 1 && Hkv != 2 && Hkv != 4) return false;
    const int G = Hq / Hkv;
    return G == 1 || G == 2 || G == 4 || G == 8;
}

bool supported_indexer(int Hi, int Di) {
    return (Hi == 1 || Hi == 2 || Hi == 4) && (Di == 32 || Di == 64);
}

int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

// About one wave of slices (2 CTAs per SM on 148 SMs ~ 296 slots): at 64
// sequences, 4 slices of 128 blocks each.
int sparse_decode_nsplit(int B, int kb) {
    int ns = (int)cdiv(256, B > 0 ? B : 1);
    int max_ns = kb / 16 > 1 ? kb / 16 : 1;
    if (ns > max_ns) ns = max_ns;
    return ns < 1 ? 1 : ns;
}

constexpr int kDenseDecodeChunk = 512;  // blocks (2048 tokens) per split

int dense_decode_nsplit(int64_t L_max) {
    const int64_t n = cdiv(cdiv(L_max, 4), kDenseDecodeChunk);
    return (int)(n < 1 ? 1 : n);
}

size_t partial_bytes(int B, int ns, int Hq, int D) {
    return (size_t)B * ns * Hq * (D + 2) * sizeof(float);
}

}  // namespace

extern "C" {

const char *qsa_version(void) { return "0.1.0"; }

const char *qsa_status_string(qsa_status_t s) {
    switch (s) {
        case QSA_OK: return "ok";
        case QSA_ERR_INVALID_ARG: return "invalid argument";
        case QSA_ERR_UNSUPPORTED_SHAPE: return "shape not supported by the GPU kernels";
        case QSA_ERR_WORKSPACE: return "workspace missing or too small";
        case QSA_ERR_ARCH: return "current device is not sm_100 (B200)";
        case QSA_ERR_CUDA: return "CUDA runtime error";
        case QSA_ERR_TIMEOUT: return "bounded device-side wait timed out";
        case QSA_ERR_DEVICE: return "kernel met an out-of-range input value";
    }
    return "unknown status";
}

// ------------------------------------------------------------------ pool --
qsa_status_t qsa_pool(const qsa_bf16_t *k_idx, int B, int64_t T, int Di, int r,
                      int64_t blk_begin, int64_t blk_end, qsa_bf16_t *k_pooled, void *stream) {
    if (B < 0 || T < 0 || Di <= 0 || r <= 0) return QSA_ERR_INVALID_ARG;
    if (blk_begin < 0 || blk_end < blk_begin || blk_end > T / r) return QSA_ERR_INVALID_ARG;
    if (r != 4 || Di % 8 != 0) return QSA_ERR_UNSUPPORTED_SHAPE;
    if (B == 0 || blk_end == blk_begin) return QSA_OK;
    if (!k_idx || !k_pooled || !aligned16(k_idx) || !aligned16(k_pooled))
        return QSA_ERR_INVALID_ARG;
    int sms = 0;
    qsa_status_t st = current_device(&sms);
    if (st != QSA_OK) return st;
    return from_cuda(qsa::launch_pool(k_idx, B, T, Di, blk_begin, blk_end, k_pooled,
                                      static_cast<cudaStream_t>(stream), sms));
}

// --------------------------------------------------------- index top-k --
size_t qsa_index_topk_workspace_size(int B, int64_t Tq, int64_t n_blocks, int Hi, int Di, int r,
                                     int budget) {
    if (B < 1 || Tq < 0 || n_blocks < 0 || Hi < 1 || Di < 1 || r < 1 || budget < r ||
        budget % r != 0)
        return SIZE_MAX;
    (void)Di;
    return qsa::index_tc_ws_bytes(B, Tq, Hi);
}

qsa_status_t qsa_index_topk(const qsa_bf16_t *q_idx, const float *w, const qsa_bf16_t *k_pooled,
                            const int64_t *q_pos0, int B, int64_t Tq, int64_t n_blocks, int Hi,
                            int Di, int r, int budget, int32_t *sel, float *sel_score, void *ws,
                            size_t ws_bytes, void *stream) {
    if (B < 1 || Tq < 0 || n_blocks < 0 || Hi < 1 || Di < 1 || r < 1 || budget < r ||
        budget % r != 0)
        return QSA_ERR_INVALID_ARG;
    if (Tq == 0) return QSA_OK;
    if (!q_idx || !w || (!k_pooled && n_blocks > 0) || !sel) return QSA_ERR_INVALID_ARG;
    if (!q_pos0 && (Tq - 1) / r > n_blocks) return QSA_ERR_INVALID_ARG;
    const int kb = budget / r;
    if (r != 4 || !supported_indexer(Hi, Di) || kb - 1 > qsa::index_tc_max_keep())
        return QSA_ERR_UNSUPPORTED_SHAPE;
    if (!ws || ws_bytes < qsa::index_tc_ws_bytes(B, Tq, Hi) || !aligned16(ws))
        return QSA_ERR_WORKSPACE;
    if (!aligned16(q_idx) || !aligned16(k_pooled)) return QSA_ERR_INVALID_ARG;
    int sms = 0;
    qsa_status_t st = current_device(&sms);
    if (st != QSA_OK) return st;
    return from_cuda(qsa::launch_index_topk_tc(q_idx, w, k_pooled, q_pos0, B, Tq, n_blocks, Hi,
                                               Di, kb, sel, sel_score, ws, sms,
                                               static_cast<cudaStream_t>(stream)));
}

size_t qsa_index_topk_decode_workspace_size(int B, int64_t n_blocks, int r, int budget) {
    if (B < 1 || n_blocks < 0 || r < 1 || budget < r || budget % r != 0) return SIZE_MAX;
    return qsa::index_decode_ws_bytes(B, n_blocks, budget / r, 0);
}

qsa_status_t qsa_index_topk_decode(const qsa_bf16_t *q_idx, const float *w,
                                   const qsa_bf16_t *k_pooled, const int32_t *seqlens, int B,
                                   int64_t n_blocks, int Hi, int Di, int r, int budget,
                                   int32_t *sel, float *sel_score, void *ws, size_t ws_bytes,
                                   void *stream) {
    if (B < 1 || n_blocks < 0 || Hi < 1 || Di < 1 || r < 1 || budget < r || budget % r != 0)
        return QSA_ERR_INVALID_ARG;
    if (!q_idx || !w || (!k_pooled && n_blocks > 0) || !seqlens || !sel)
        return QSA_ERR_INVALID_ARG;
    const int kb = budget / r;
    if (r != 4 || !supported_indexer(Hi, Di) || kb - 1 > qsa::index_tc_max_keep() ||
        qsa::index_decode_merge_cap(n_blocks, kb) < 0)
        return QSA_ERR_UNSUPPORTED_SHAPE;
    if (!ws || ws_bytes < qsa::index_decode_ws_bytes(B, n_blocks, kb, 0) || !aligned16(ws))
        return QSA_ERR_WORKSPACE;
    if (!aligned16(q_idx) || !aligned16(k_pooled)) return QSA_ERR_INVALID_ARG;
    int sms = 0;
    qsa_status_t st = current_device(&sms);
    if (st != QSA_OK) return st;
    return from_cuda(qsa::launch_index_topk_decode(q_idx, w, k_pooled, seqlens, B, n_blocks, Hi,
                                                   Di, kb, sel, sel_score, ws, sms,
                                                   static_cast<cudaStream_t>(stream)));
}

// ------------------------------------------------------ sparse attention --
qsa_status_t qsa_sparse_attn_prefill(const qsa_bf16_t *q, const qsa_bf16_t *k,
                                     const qsa_bf16_t *v, const int32_t *sel,
                                     const int64_t *q_pos0, int B, int64_t Tq, int64_t Tk,
                                     int Hq, int Hkv, int D, int r, int budget, float scale,
                                     qsa_bf16_t *o, float *lse, void *stream) {
    if (B < 1 || Tq < 0 || Tk < 0 || Hq < 1 || Hkv < 1 || Hq % Hkv != 0 || D < 1 || r < 1 ||
        budget < r || budget % r != 0 || !(scale == scale))
        return QSA_ERR_INVALID_ARG;
    if (Tq == 0) return QSA_OK;
    if (Tk < 1 || !q || !k || !v || !sel || !o) return QSA_ERR_INVALID_ARG;
    if (!q_pos0 && Tq > Tk) return QSA_ERR_INVALID_ARG;
    const int kb = budget / r;
    if (r != 4 || !supported_attn(Hq, Hkv, D) || kb > 1024) return QSA_ERR_UNSUPPORTED_SHAPE;
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o))
        return QSA_ERR_INVALID_ARG;
    int sms = 0;
    qsa_status_t st = current_device(&sms);
    if (st != QSA_OK) return st;
    return from_cuda(qsa::launch_sparse_attn_prefill(q, k, v, sel, q_pos0, B, Tq, Tk, Hq, Hkv, D,
                                                     kb, scale, o, lse, sms,
                                                     static_cast<cudaStream_t>(stream)));
}

size_t qsa_sparse_attn_decode_workspace_size(int B, int Hq, int D, int r, int budget) {
    if (B < 1 || Hq < 1 || D < 1 || r < 1 || budget < r || budget % r != 0) return SIZE_MAX;
    return kHeader + partial_bytes(B, sparse_decode_nsplit(B, budget / r), Hq, D);
}

qsa_status_t qsa_sparse_attn_decode(const qsa_bf16_t *q, const qsa_bf16_t *k_cache,
                                    const qsa_bf16_t *v_cache, const int32_t *seqlens,
                                    int64_t L_max, const int32_t *sel, int B, int Hq, int Hkv,
                                    int D, int r, int budget, float scale, qsa_bf16_t *o,
                                    float *lse, void *ws, size_t ws_bytes, void *stream) {
    if (B < 1 || L_max < 1 || Hq < 1 || Hkv < 1 || Hq % Hkv != 0 || D < 1 || r < 1 ||
        budget < r || budget % r != 0 || !(scale == scale))
        return QSA_ERR_INVALID_ARG;
    if (!q || !k_cache || !v_cache || !seqlens || !sel || !o) return QSA_ERR_INVALID_ARG;
    const int kb = budget / r;
    if (r != 4 || !supported_attn(Hq, Hkv, D) || kb > 1024) return QSA_ERR_UNSUPPORTED_SHAPE;
    const int ns = sparse_decode_nsplit(B, kb);
    if (!ws || ws_bytes < kHeader + partial_bytes(B, ns, Hq, D) || !aligned16(ws))
        return QSA_ERR_WORKSPACE;
    if (!aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(o))
        return QSA_ERR_INVALID_ARG;
    int sms = 0;
    qsa_status_t st = current_device(&sms);
    if (st != QSA_OK) return st;
    float *part = reinterpret_cast<float *>(static_cast<uint8_t *>(ws) + kHeader);
    return from_cuda(qsa::launch_split_decode(q, k_cache, v_cache, seqlens, L_max, sel, kb, ns, B,
                                              Hq, Hkv, D, scale, o, lse, part, ws, sms,
                                              static_cast<cudaStream_t>(stream)));
}

// -------------------------------------------------------- dense baseline --
qsa_status_t qsa_dense_gqa_prefill(const qsa_bf16_t *q, const qsa_bf16_t *k, const qsa_bf16_t *v,
                                   int B, int64_t T, int Hq, int Hkv, int D, float scale,
                                   qsa_bf16_t *o, float *lse, void *stream) {
    if (B < 1 || T < 0 || Hq < 1 || Hkv < 1 || Hq % Hkv != 0 || D < 1 || !(scale == scale))
        return QSA_ERR_INVALID_ARG;
    if (T == 0) return QSA_OK;
    if (!q || !k || !v || !o) return QSA_ERR_INVALID_ARG;
    if (!supported_attn(Hq, Hkv, D)) return QSA_ERR_UNSUPPORTED_SHAPE;
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o))
        return QSA_ERR_INVALID_ARG;
    int sms = 0;
    qsa_status_t st = current_device(&sms);
    if (st != QSA_OK) return st;
    return from_cuda(qsa::launch_dense_prefill(q, k, v, B, T, Hq, Hkv, D, scale, o, lse,
                                               static_cast<cudaStream_t>(stream)));
}

size_t qsa_dense_gqa_decode_workspace_size(int B, int64_t L_max, int Hq, int D) {
    if (B < 1 || L_max < 1 || Hq < 1 || D < 1) return SIZE_MAX;
    return kHeader + partial_bytes(B, dense_decode_nsplit(L_max), Hq, D);
}

qsa_status_t qsa_dense_gqa_decode(const qsa_bf16_t *q, const qsa_bf16_t *k_cache,
                                  const qsa_bf16_t *v_cache, const int32_t *seqlens,
                                  int64_t L_max, int B, int Hq, int Hkv, int D, float scale,
                                  qsa_bf16_t *o, float *lse, void *ws, size_t ws_bytes,
                                  void *stream) {
    if (B < 1 || L_max < 1 || Hq < 1 || Hkv < 1 || Hq % Hkv != 0 || D < 1 || !(scale == scale))
        return QSA_ERR_INVALID_ARG;
    if (!q || !k_cache || !v_cache || !seqlens || !o) return QSA_ERR_INVALID_ARG;
    if (!supported_attn(Hq, Hkv, D)) return QSA_ERR_UNSUPPORTED_SHAPE;
    const int ns = dense_decode_nsplit(L_max);
    if (!ws || ws_bytes < kHeader + partial_bytes(B, ns, Hq, D) || !aligned16(ws))
        return QSA_ERR_WORKSPACE;
    if (!aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(o))
        return QSA_ERR_INVALID_ARG;
    int sms = 0;
    qsa_status_t st = current_device(&sms);
    if (st != QSA_OK) return st;
    float *part = reinterpret_cast<float *>(static_cast<uint8_t *>(ws) + kHeader);
    const int n_entries = (int)cdiv(L_max, 4);
    return from_cuda(qsa::launch_split_decode(q, k_cache, v_cache, seqlens, L_max, nullptr,
                                              n_entries, ns, B, Hq, Hkv, D, scale, o, lse, part,
                                              ws, sms, static_cast<cudaStream_t>(stream)));
}

// ------------------------------------------- sparse attention backward --
qsa_status_t qsa_sparse_attn_backward(const qsa_bf16_t *q, const qsa_bf16_t *k,
                                      const qsa_bf16_t *v, const int32_t *sel,
                                      const qsa_bf16_t *d_o, int B, int64_t T, int Hq, int Hkv,
                                      int D, int r, int budget, float scale, float *dq,
                                      float *dk, float *dv, void *stream) {
    if (B < 1 || T < 0 || Hq < 1 || Hkv < 1 || Hq % Hkv != 0 || D < 1 || r < 1 ||
        budget < r || budget % r != 0 || !(scale == scale))
        return QSA_ERR_INVALID_ARG;
    if (T == 0) return QSA_OK;
    if (!q || !k || !v || !sel || !d_o || !dq || !dk || !dv) return QSA_ERR_INVALID_ARG;
    const int kb = budget / r;
    if (r != 4 || !supported_attn(Hq, Hkv, D) || kb > 1024) return QSA_ERR_UNSUPPORTED_SHAPE;
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(d_o) || !aligned16(dq) ||
        !aligned16(dk) || !aligned16(dv))
        return QSA_ERR_INVALID_ARG;
    int sms = 0;
    qsa_status_t st = current_device(&sms);
    if (st != QSA_OK) return st;
    return from_cuda(qsa::launch_sparse_attn_backward(q, k, v, sel, d_o, B, T, Hq, Hkv, D, kb,
                                                      scale, dq, dk, dv,
                                                      static_cast<cudaStream_t>(stream)));
}

// ---------------------------------------------------- measurement aid --
qsa_status_t qsa_probe_l2_read(const void *buf, size_t bytes, int reps, void *sink,
                               void *stream) {
    if (!buf || !sink || reps < 1 || bytes < 16) return QSA_ERR_INVALID_ARG;
    if (!aligned16(buf) || (reinterpret_cast<uintptr_t>(sink) & 3u) != 0) return QSA_ERR_INVALID_ARG;
    int sms = 0;
    qsa_status_t st = current_device(&sms);
    if (st != QSA_OK) return st;
    return from_cuda(qsa::launch_l2_read_probe(buf, bytes, reps, static_cast<uint32_t *>(sink),
                                               sms, static_cast<cudaStream_t>(stream)));
}

// ------------------------------------------------------- Gated DeltaNet --
static bool supported_gdn(int dk, int dv) {
    return (dk == 64 || dk == 128) && (dv == 64 || dv == 128);
}

qsa_status_t qsa_gdn_prefill(const qsa_bf16_t *q, const qsa_bf16_t *k, const qsa_bf16_t *v,
                             const float *alpha, const float *beta, const float *state_in, int B,
                             int64_t T, int H, int dk, int dv, float *o, float *state_out,
                             void *stream) {
    if (B < 1 || T < 0 || H < 1 || dk < 1 || dv < 1) return QSA_ERR_INVALID_ARG;
    if (!state_out || (T > 0 && (!q || !k || !v || !alpha || !beta || !o)))
        return QSA_ERR_INVALID_ARG;
    if (!supported_gdn(dk, dv)) return QSA_ERR_UNSUPPORTED_SHAPE;
    if (!aligned16(state_out) || (state_in && !aligned16(state_in))) return QSA_ERR_INVALID_ARG;
    int sms = 0;
    qsa_status_t st = current_device(&sms);
    if (st != QSA_OK) return st;
    return from_cuda(qsa::launch_gdn_prefill(q, k, v, alpha, beta, state_in, B, T, H, dk, dv, o,
                                             state_out, static_cast<cudaStream_t>(stream)));
}

size_t qsa_gdn_prefill_chunked_workspace_size(int B, int64_t T, int H, int dk, int dv) {
    if (B < 1 || T < 0 || H < 1 || !supported_gdn(dk, dv)) return SIZE_MAX;
    return qsa::gdn_chunked_ws_bytes(B, T, H, dk, dv);
}

qsa_status_t qsa_gdn_prefill_chunked(const qsa_bf16_t *q, const qsa_bf16_t *k,
                                     const qsa_bf16_t *v, const float *alpha, const float *beta,
                                     const float *state_in, int B, int64_t T, int H, int dk,
                                     int dv, float *o, float *state_out, void *ws,
                                     size_t ws_bytes, void *stream) {
    if (B < 1 || T < 0 || H < 1 || dk < 1 || dv < 1) return QSA_ERR_INVALID_ARG;
    if (!state_out || (T > 0 && (!q || !k || !v || !alpha || !beta || !o)))
        return QSA_ERR_INVALID_ARG;
    if (!supported_gdn(dk, dv)) return QSA_ERR_UNSUPPORTED_SHAPE;
    if (!aligned16(state_out) || (state_in && !aligned16(state_in)) ||
        (T > 0 && (!aligned16(q) || !aligned16(k))))
        return QSA_ERR_INVALID_ARG;
    if (!ws || ws_bytes < qsa::gdn_chunked_ws_bytes(B, T, H, dk, dv) ||
        (reinterpret_cast<uintptr_t>(ws) & 255u) != 0)
        return QSA_ERR_WORKSPACE;
    int sms = 0;
    qsa_status_t st = current_device(&sms);
    if (st != QSA_OK) return st;
    return from_cuda(qsa::launch_gdn_prefill_chunked(q, k, v, alpha, beta, state_in, B, T, H, dk,
                                                     dv, o, state_out, ws,
                                                     static_cast<cudaStream_t>(stream)));
}

qsa_status_t qsa_gdn_decode(const qsa_bf16_t *q, const qsa_bf16_t *k, const qsa_bf16_t *v,
                            const float *alpha, const float *beta, float *state, int B, int H,
                            int dk, int dv, float *o, void *stream) {
    if (B < 1 || H < 1 || dk < 1 || dv < 1) return QSA_ERR_INVALID_ARG;
    if (!q || !k || !v || !alpha || !beta || !state || !o) return QSA_ERR_INVALID_ARG;
    if (!supported_gdn(dk, dv)) return QSA_ERR_UNSUPPORTED_SHAPE;
    if (!aligned16(state)) return QSA_ERR_INVALID_ARG;
    int sms = 0;
    qsa_status_t st = current_device(&sms);
    if (st != QSA_OK) return st;
    return from_cuda(qsa::launch_gdn_decode(q, k, v, alpha, beta, state, B, H, dk, dv, o,
                                            static_cast<cudaStream_t>(stream)));
}

// ------------------------------------------------- indexer distillation --
size_t qsa_index_distill_workspace_size(int B, int64_t T, int Hkv, int r) {
    if (B < 1 || T < 0 || Hkv < 1 || r != 4) return SIZE_MAX;
    return qsa::index_distill_ws_bytes(B, T, Hkv);
}

qsa_status_t qsa_index_distill(const qsa_bf16_t *q, const qsa_bf16_t *k, const float *lse,
                               const qsa_bf16_t *q_idx, const float *w,
                               const qsa_bf16_t *k_pooled, int B, int64_t T, int Hq, int Hkv,
                               int D, int Hi, int Di, int r, float scale, float *kl,
                               float *dq_idx, float *dw, float *dk_pooled, float *dk_idx,
                               void *ws, size_t ws_bytes, void *stream) {
    if (B < 1 || T < 0 || Hq < 1 || Hkv < 1 || Hq % Hkv != 0 || D < 1 || Hi < 1 || Di < 1 ||
        r < 1 || !(scale == scale))
        return QSA_ERR_INVALID_ARG;
    if (T == 0) return QSA_OK;
    const int64_t N = T / r;
    if (!q || !k || !lse || !q_idx || !w || !kl || !dq_idx || !dw ||
        (N > 0 && (!k_pooled || !dk_pooled)))
        return QSA_ERR_INVALID_ARG;
    if (r != 4 || !supported_attn(Hq, Hkv, D) || !supported_indexer(Hi, Di))
        return QSA_ERR_UNSUPPORTED_SHAPE;
    if (!ws || ws_bytes < qsa::index_distill_ws_bytes(B, T, Hkv) || !aligned16(ws))
        return QSA_ERR_WORKSPACE;
    if (!aligned16(q) || !aligned16(k) || !aligned16(q_idx) || !aligned16(k_pooled))
        return QSA_ERR_INVALID_ARG;
    int sms = 0;
    qsa_status_t st = current_device(&sms);
    if (st != QSA_OK) return st;
    return from_cuda(qsa::launch_index_distill(q, k, lse, q_idx, w, k_pooled, B, T, Hq, Hkv, D,
                                               Hi, Di, scale, kl, dq_idx, dw, dk_pooled, dk_idx,
                                               ws, static_cast<cudaStream_t>(stream)));
}

// ------------------------------------------- stage-2 indexer loss --
size_t qsa_index_distill_sparse_workspace_size(int B, int64_t T, int Hkv, int r, int budget) {
    if (B < 1 || T < 0 || Hkv < 1 || r != 4 || budget < r || budget % r != 0) return SIZE_MAX;
    return qsa::index_distill_sparse_ws_bytes(B, T, Hkv, budget / r);
}

qsa_status_t qsa_index_distill_sparse(const qsa_bf16_t *q, const qsa_bf16_t *k,
                                      const float *lse, const int32_t *sel,
                                      const qsa_bf16_t *q_idx, const float *w,
                                      const qsa_bf16_t *k_pooled, int B, int64_t T, int Hq,
                                      int Hkv, int D, int Hi, int Di, int r, int budget,
                                      float scale, float *kl, float *dq_idx, float *dw,
                                      float *dk_pooled, float *dk_idx, void *ws, size_t ws_bytes,
                                      void *stream) {
    if (B < 1 || T < 0 || Hq < 1 || Hkv < 1 || Hq % Hkv != 0 || D < 1 || Hi < 1 || Di < 1 ||
        r < 1 || budget < r || budget % r != 0 || !(scale == scale))
        return QSA_ERR_INVALID_ARG;
    if (T == 0) return QSA_OK;
    const int64_t N = T / r;
    if (!q || !k || !lse || !sel || !q_idx || !w || !kl || !dq_idx || !dw ||
        (N > 0 && (!k_pooled || !dk_pooled)))
        return QSA_ERR_INVALID_ARG;
    const int kb = budget / r;
    if (r != 4 || !supported_attn(Hq, Hkv, D) || !supported_indexer(Hi, Di) ||
        kb > qsa::index_distill_sparse_max_entries())
        return QSA_ERR_UNSUPPORTED_SHAPE;
    if (!ws || ws_bytes < qsa::index_distill_sparse_ws_bytes(B, T, Hkv, kb) || !aligned16(ws))
        return QSA_ERR_WORKSPACE;
    if (!aligned16(q) || !aligned16(k) || !aligned16(q_idx) || !aligned16(k_pooled))
        return QSA_ERR_INVALID_ARG;
    int sms = 0;
    qsa_status_t st = current_device(&sms);
    if (st != QSA_OK) return st;
    return from_cuda(qsa::launch_index_distill_sparse(
        q, k, lse, sel, q_idx, w, k_pooled, B, T, Hq, Hkv, D, Hi, Di, kb, scale, kl, dq_idx, dw,
        dk_pooled, dk_idx, ws, static_cast<cudaStream_t>(stream)));
}

// ------------------------------------- rotary positions, per-head norms --

static bool supported_head(int D) { return D == 32 || D == 64 || D == 128 || D == 256; }

static bool valid_dtype(int t) { return t == QSA_BF16 || t == QSA_F32; }

static bool valid_layout(int l) { return l == QSA_ROPE_HALF || l == QSA_ROPE_INTERLEAVED; }

// Rows of H heads of D elements every `stride`: 0 heads never reach here.
static bool valid_stride(int64_t stride, int H, int D, int esize) {
    return stride >= (int64_t)H * D && stride * esize % 16 == 0;
}

static bool aligned8(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 7u) == 0; }

qsa_status_t qsa_rope_frequencies(double base, int rot, int scaling, double factor,
                                  double orig_len, double beta_fast, double beta_slow,
                                  double *freq, float *mscale) {
    if (!freq || rot < 2 || rot % 2 != 0 || !(base > 1.0) || !isfinite(base) ||
        !(factor >= 1.0) || !isfinite(factor))
        return QSA_ERR_INVALID_ARG;
    if (scaling < QSA_ROPE_PLAIN || scaling > QSA_ROPE_BY_PARTS) return QSA_ERR_INVALID_ARG;
    if (scaling == QSA_ROPE_NTK && rot < 4) return QSA_ERR_INVALID_ARG;
    double lo = 0, hi = 0;
    if (scaling == QSA_ROPE_BY_PARTS) {
        if (!(orig_len > 0) || !isfinite(orig_len) || !(beta_slow > 0) ||
            !(beta_fast >= beta_slow) || !isfinite(beta_fast))
            return QSA_ERR_INVALID_ARG;
        const double two_pi = 6.283185307179586476925286766559;
        const double per = rot / (2 * log(base));
        lo = fmax(floor(per * log(orig_len / (two_pi * beta_fast))), 0.0);
        hi = fmin(ceil(per * log(orig_len / (two_pi * beta_slow))), (double)(rot - 1));
    }
    if (scaling == QSA_ROPE_NTK) base *= pow(factor, (double)rot / (rot - 2));
    for (int i = 0; i < rot / 2; ++i) {
        double f = pow(base, -2.0 * i / rot);
        if (scaling == QSA_ROPE_LINEAR) f /= factor;
        if (scaling == QSA_ROPE_BY_PARTS) {
            const double w = fmin(fmax((i - lo) / fmax(hi - lo, 0.001), 0.0), 1.0);
            f = f * (1 - w) + f / factor * w;
        }
        freq[i] = f;
    }
    if (mscale) *mscale = scaling == QSA_ROPE_BY_PARTS ? (float)(0.1 * log(factor) + 1.0) : 1.f;
    return QSA_OK;
}

qsa_status_t qsa_rope(const void *x, int64_t x_stride, void *y, int64_t y_stride, int dtype,
                      int B, int64_t T, int H, int D, const double *freq, int rot, int layout,
                      float mscale, int transpose, const int64_t *pos, const int64_t *pos0,
                      void *stream) {
    if (B < 1 || T < 0 || H < 1 || D < 1 || rot < 0 || rot > D || !valid_dtype(dtype) ||
        !valid_layout(layout) || !isfinite(mscale))
        return QSA_ERR_INVALID_ARG;
    if (!supported_head(D) || rot % 8 != 0) return QSA_ERR_UNSUPPORTED_SHAPE;
    if (T == 0) return QSA_OK;
    if (!x || !y || (rot > 0 && !freq)) return QSA_ERR_INVALID_ARG;
    const int es = dtype == QSA_F32 ? 4 : 2;
    if (!aligned16(x) || !aligned16(y) || !valid_stride(x_stride, H, D, es) ||
        !valid_stride(y_stride, H, D, es) || !aligned8(freq) || !aligned8(pos) ||
        !aligned8(pos0) || (x == y && x_stride != y_stride))
        return QSA_ERR_INVALID_ARG;
    int sms = 0;
    qsa_status_t st = current_device(&sms);
    if (st != QSA_OK) return st;
    return from_cuda(qsa::launch_rope(x, x_stride, y, y_stride, dtype == QSA_F32, B, T, H, D,
                                      freq, rot, layout == QSA_ROPE_HALF, mscale,
                                      transpose != 0, pos, pos0, sms,
                                      static_cast<cudaStream_t>(stream)));
}

qsa_status_t qsa_qk_norm_rope(const qsa_bf16_t *q, int64_t q_stride, const qsa_bf16_t *k,
                              int64_t k_stride, const qsa_bf16_t *v, int64_t v_stride, int B,
                              int64_t T, int Hq, int Hkv, int D, const float *q_weight,
                              const float *k_weight, float eps, const double *freq, int rot,
                              int layout, float mscale, const int64_t *pos, const int64_t *pos0,
                              qsa_bf16_t *q_out, qsa_bf16_t *k_out, qsa_bf16_t *v_out,
                              const int64_t *slot, int64_t L_max, void *ws, void *stream) {
    if (B < 1 || T < 0 || Hq < 1 || Hkv < 1 || D < 1 || rot < 0 || rot > D ||
        !valid_layout(layout) || !isfinite(mscale) || !(eps >= 0.f) || !isfinite(eps) ||
        L_max < 0)
        return QSA_ERR_INVALID_ARG;
    if (!supported_head(D) || rot % 8 != 0) return QSA_ERR_UNSUPPORTED_SHAPE;
    if (T == 0) return QSA_OK;
    if (!q || !k || !q_out || (rot > 0 && !freq) || (v == nullptr) != (v_out == nullptr) ||
        (!slot && L_max != T))
        return QSA_ERR_INVALID_ARG;
    if (L_max > 0 && !k_out) return QSA_ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(q_out) ||
        !aligned16(k_out) || !aligned16(v_out) || !aligned16(q_weight) || !aligned16(k_weight) ||
        !aligned8(freq) || !aligned8(pos) || !aligned8(pos0) || !aligned8(slot) ||
        !aligned16(ws) || !valid_stride(q_stride, Hq, D, 2) ||
        !valid_stride(k_stride, Hkv, D, 2) || (v && !valid_stride(v_stride, Hkv, D, 2)))
        return QSA_ERR_INVALID_ARG;
    // in place: a row is written where it was read, by those who read it
    const bool one = (int64_t)B * T == 1;
    if ((q == q_out && !one && q_stride != (int64_t)Hq * D) ||
        (k == k_out && (slot || (!one && k_stride != (int64_t)Hkv * D))) ||
        (v && v == v_out && (slot || (!one && v_stride != (int64_t)Hkv * D))))
        return QSA_ERR_INVALID_ARG;
    int sms = 0;
    qsa_status_t st = current_device(&sms);
    if (st != QSA_OK) return st;
    return from_cuda(qsa::launch_norm_rope(q, q_stride, k, k_stride, v, v_stride, B, T, Hq, Hkv,
                                           D, q_weight, k_weight, eps, freq, rot,
                                           layout == QSA_ROPE_HALF, mscale, pos, pos0, q_out,
                                           k_out, v_out, slot, L_max, ws, sms,
                                           static_cast<cudaStream_t>(stream)));
}

size_t qsa_qk_norm_rope_backward_workspace_size(int B, int64_t T, int Hq, int Hkv, int D) {
    if (B < 1 || T < 0 || Hq < 1 || Hkv < 1 || !supported_head(D)) return SIZE_MAX;
    return qsa::norm_rope_grad_ws_bytes((int64_t)B * T, Hq, Hkv, D);
}

qsa_status_t qsa_qk_norm_rope_backward(
    const void *d_q, const void *d_k, int d_dtype, const qsa_bf16_t *q, int64_t q_stride,
    const qsa_bf16_t *k, int64_t k_stride, int B, int64_t T, int Hq, int Hkv, int D,
    const float *q_weight, const float *k_weight, float eps, const double *freq, int rot,
    int layout, float mscale, const int64_t *pos, const int64_t *pos0, void *dq, void *dk,
    int dx_dtype, float *dq_weight, float *dk_weight, void *ws, size_t ws_bytes, void *stream) {
    if (B < 1 || T < 0 || Hq < 1 || Hkv < 1 || D < 1 || rot < 0 || rot > D ||
        !valid_layout(layout) || !valid_dtype(d_dtype) || !valid_dtype(dx_dtype) ||
        !isfinite(mscale) || !(eps >= 0.f) || !isfinite(eps))
        return QSA_ERR_INVALID_ARG;
    if ((dq_weight && !q_weight) || (dk_weight && !k_weight)) return QSA_ERR_INVALID_ARG;
    if (!supported_head(D) || rot % 8 != 0) return QSA_ERR_UNSUPPORTED_SHAPE;
    if (T == 0 && !dq_weight && !dk_weight) return QSA_OK;
    // (the table is read for T == 0 too: the kernel runs, to write zeros)
    if ((rot > 0 && !freq) || (T > 0 && (!d_q || !d_k || !q || !k || !dq || !dk)))
        return QSA_ERR_INVALID_ARG;
    if ((dq_weight || dk_weight) &&
        (!ws || !aligned16(ws) ||
         ws_bytes < qsa::norm_rope_grad_ws_bytes((int64_t)B * T, Hq, Hkv, D)))
        return QSA_ERR_WORKSPACE;
    if (!aligned16(d_q) || !aligned16(d_k) || !aligned16(q) || !aligned16(k) ||
        !aligned16(dq) || !aligned16(dk) || !aligned16(q_weight) || !aligned16(k_weight) ||
        !aligned8(freq) || !aligned8(pos) || !aligned8(pos0) ||
        (T > 0 && (!valid_stride(q_stride, Hq, D, 2) || !valid_stride(k_stride, Hkv, D, 2))))
        return QSA_ERR_INVALID_ARG;
    if (d_dtype != dx_dtype && T > 0 && (d_q == dq || d_k == dk)) return QSA_ERR_INVALID_ARG;
    int sms = 0;
    qsa_status_t st = current_device(&sms);
    if (st != QSA_OK) return st;
    return from_cuda(qsa::launch_norm_rope_grad(
        d_q, d_k, d_dtype == QSA_F32, q, q_stride, k, k_stride, B, T, Hq, Hkv, D, q_weight,
        k_weight, eps, freq, rot, layout == QSA_ROPE_HALF, mscale, pos, pos0, dq, dk,
        dx_dtype == QSA_F32, dq_weight, dk_weight, ws, sms, static_cast<cudaStream_t>(stream)));
}

// ------------------------------------------- trees of drafted tokens --

// Drafts that a call takes: a row index times 32 query heads fits 31 bits.
static bool tree_rows(int B, int N) {
    return N <= qsa::TREE_DRAFTS && (int64_t)B * N <= INT32_MAX / 32;
}

static qsa_status_t check_tree(const void *q, const void *k, const void *v, const void *seqlens,
                               int64_t L_max, const void *parent, int B, int N, int Hq, int Hkv,
                               int D, float scale, const void *o) {
    if (B < 1 || N < 1 || L_max < 1 || Hq < 1 || Hkv < 1 || Hq % Hkv != 0 || D < 1 ||
        !isfinite(scale))
        return QSA_ERR_INVALID_ARG;
    if (!q || !k || !v || !seqlens || !parent || !o) return QSA_ERR_INVALID_ARG;
    if (!supported_attn(Hq, Hkv, D) || !tree_rows(B, N) || L_max > INT32_MAX)
        return QSA_ERR_UNSUPPORTED_SHAPE;
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o))
        return QSA_ERR_INVALID_ARG;
    return QSA_OK;
}

size_t qsa_dense_tree_decode_workspace_size(int B, int N, int Hq, int Hkv, int D) {
    if (B < 1 || N < 1 || Hq < 1 || Hkv < 1 || Hq % Hkv != 0 || !tree_rows(B, N) ||
        !supported_attn(Hq, Hkv, D))
        return SIZE_MAX;
    return qsa::tree_dense_ws_bytes(B, N, Hq, Hkv, D);
}

qsa_status_t qsa_dense_tree_decode(const qsa_bf16_t *q, const qsa_bf16_t *k_cache,
                                   const qsa_bf16_t *v_cache, const int32_t *seqlens,
                                   int64_t L_max, const int32_t *parent, const int32_t *n_draft,
                                   int B, int N, int Hq, int Hkv, int D, float scale,
                                   qsa_bf16_t *o, float *lse, void *ws, size_t ws_bytes,
                                   void *stream) {
    qsa_status_t st = check_tree(q, k_cache, v_cache, seqlens, L_max, parent, B, N, Hq, Hkv, D,
                                 scale, o);
    if (st != QSA_OK) return st;
    if (!ws || ws_bytes < qsa::tree_dense_ws_bytes(B, N, Hq, Hkv, D) || !aligned16(ws))
        return QSA_ERR_WORKSPACE;
    int sms = 0;
    st = current_device(&sms);
    if (st != QSA_OK) return st;
    return from_cuda(qsa::launch_tree_decode(q, k_cache, v_cache, seqlens, n_draft, L_max,
                                             nullptr, 0, 0, 0, parent, B, N, Hq, Hkv, D, scale,
                                             o, lse, ws, sms, static_cast<cudaStream_t>(stream)));
}

// Sums of the rows' stages are 32-bit in the kernel.
static bool tree_stages(int B, int N, int Hkv, int kb) {
    return qsa::tree_sparse_stages(B, N, Hkv, kb) <= INT32_MAX;
}

size_t qsa_sparse_tree_decode_workspace_size(int B, int N, int Hq, int D, int r, int budget) {
    if (B < 1 || N < 1 || Hq < 1 || r < 1 || budget < r || budget % r != 0 ||
        !tree_rows(B, N) || Hq > 32 || (D != 64 && D != 128))
        return SIZE_MAX;
    // (the fewest key heads have the fewest stages)
    const int least = Hq <= 8 ? 1 : Hq <= 16 ? 2 : 4;
    if (!tree_stages(B, N, least, budget / r)) return SIZE_MAX;
    return qsa::tree_sparse_ws_bytes(B, N, Hq, D);
}

qsa_status_t qsa_sparse_tree_decode(const qsa_bf16_t *q, const qsa_bf16_t *k_cache,
                                    const qsa_bf16_t *v_cache, const int32_t *seqlens,
                                    int64_t L_max, const int32_t *sel, int64_t sel_batch_stride,
                                    int64_t sel_row_stride, const int32_t *parent,
                                    const int32_t *n_draft, int B, int N, int Hq, int Hkv, int D,
                                    int r, int budget, float scale, qsa_bf16_t *o, float *lse,
                                    void *ws, size_t ws_bytes, void *stream) {
    if (r < 1 || budget < r || budget % r != 0 || sel_batch_stride < 0 || sel_row_stride < 0)
        return QSA_ERR_INVALID_ARG;
    qsa_status_t st = check_tree(q, k_cache, v_cache, seqlens, L_max, parent, B, N, Hq, Hkv, D,
                                 scale, o);
    if (st != QSA_OK) return st;
    if (!sel) return QSA_ERR_INVALID_ARG;
    if (r != 4 || budget / r > 1024 || !tree_stages(B, N, Hkv, budget / r))
        return QSA_ERR_UNSUPPORTED_SHAPE;
    if (!ws || ws_bytes < qsa::tree_sparse_ws_bytes(B, N, Hq, D) || !aligned16(ws))
        return QSA_ERR_WORKSPACE;
    int sms = 0;
    st = current_device(&sms);
    if (st != QSA_OK) return st;
    return from_cuda(qsa::launch_tree_decode(q, k_cache, v_cache, seqlens, n_draft, L_max, sel,
                                             sel_batch_stride, sel_row_stride, budget / r,
                                             parent, B, N, Hq, Hkv, D, scale, o, lse, ws, sms,
                                             static_cast<cudaStream_t>(stream)));
}

// ---------------------------------------------------------------- status --
qsa_status_t qsa_check_device_status(void *ws, void *stream) {
    if (!ws) return QSA_ERR_INVALID_ARG;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (cudaStreamSynchronize(s) != cudaSuccess) {
        cudaGetLastError();
        return QSA_ERR_CUDA;
    }
    int word = 0;
    if (cudaMemcpy(&word, ws, sizeof(int), cudaMemcpyDeviceToHost) != cudaSuccess) {
        cudaGetLastError();
        return QSA_ERR_CUDA;
    }
    if (word != 0 && cudaMemset(ws, 0, sizeof(int)) != cudaSuccess) {
        cudaGetLastError();
        return QSA_ERR_CUDA;
    }
    return static_cast<qsa_status_t>(word);
}

}  // extern "C"
