// extern "C" entry points declared in include/qat.h: argument checks on the
// host, workspace carving, and the sequencing of quantizer and GEMM launches.
#include <algorithm>
#include <atomic>
#include <cmath>
#include <initializer_list>
#include <mutex>
#include <numeric>

#include "gemm_sm100.cuh"
#include "lm_ops.cuh"
#include "quant.cuh"

namespace qat {

// The one device-side error flag (per device, zero-initialised at load).
__device__ int g_device_error = 0;

// Per-device caches below are filled on first use with the device current;
// concurrent first calls from several host threads store the same value.
int* device_error_ptr() {
  static std::atomic<int*> cached[64] = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return nullptr;
  int* p = cached[dev].load(std::memory_order_acquire);
  if (!p) {
    void* a = nullptr;
    if (cudaGetSymbolAddress(&a, g_device_error) != cudaSuccess) return nullptr;
    p = static_cast<int*>(a);
    cached[dev].store(p, std::memory_order_release);
  }
  return p;
}

static std::atomic<int64_t> g_launches{0};
void count_launch() { g_launches.fetch_add(1, std::memory_order_relaxed); }

int sm_count() {
  static std::atomic<int> cached[64] = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 148;
  int n = cached[dev].load(std::memory_order_relaxed);
  if (n == 0) {
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0)
      n = 148;
    cached[dev].store(n, std::memory_order_relaxed);
  }
  return n;
}

bool device_flag_once(std::atomic<uint64_t>& done, int* dev_out) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) dev = 0;
  if (dev_out) *dev_out = dev;
  if (dev < 0 || dev >= 64) return false;
  return (done.load(std::memory_order_acquire) >> dev) & 1u;
}

void device_flag_set(std::atomic<uint64_t>& done, int dev) {
  if (dev >= 0 && dev < 64) done.fetch_or(uint64_t{1} << dev, std::memory_order_acq_rel);
}

namespace {

constexpr size_t kAlign = 256;
inline size_t align_up(size_t x) { return (x + kAlign - 1) / kAlign * kAlign; }

// Carves 256-byte aligned pieces from the caller's workspace.
struct Carver {
  uint8_t* base;
  size_t cap, used = 0;
  Carver(void* b, size_t c) : base(static_cast<uint8_t*>(b)), cap(c) {}
  void* take(size_t bytes) {
    const size_t at = used;
    used = align_up(used + bytes);
    return (base && used <= cap) ? base + at : nullptr;
  }
};

inline size_t operand_bytes(int64_t N, int64_t K) { return align_up(N * K * 2) + align_up(N * 4); }

bool bits_ok(int bits) { return bits == 5 || bits == 6 || bits == 8; }
bool act_ok(int act) { return act == QAT_ACT_RELU2 || act == QAT_ACT_LEAKY_RELU2; }
bool dim_ok(int64_t x) { return x > 0 && (x & 7) == 0 && x <= (1 << 20); }

// An argument's memory: `rows` runs of `run` bytes, `step` bytes apart (step >= run
// where there is more than one).  Null or empty ones share nothing.
struct Span {
  uintptr_t at;
  int64_t rows, step, run;
  Span(const void* p, int64_t n, int64_t step_bytes, int64_t run_bytes)
      : at(reinterpret_cast<uintptr_t>(p)), rows(n), step(step_bytes), run(run_bytes) {}
  Span(const void* p, int64_t bytes) : Span(p, 1, bytes, bytes) {}
  bool empty() const { return !at || rows <= 0 || run <= 0; }
  uintptr_t end() const { return at + static_cast<uintptr_t>((rows - 1) * step + run); }
};
Span rows_span(const qat_bf16* p, int64_t rows, int64_t ld, int64_t cols) { return Span(p, rows, ld * 2, cols * 2); }

// Whether both hold some byte.  Columns of one wider row lie between one another's
// runs and share none.
bool shares(const Span& a, const Span& b) {
  if (a.empty() || b.empty() || a.end() <= b.at || b.end() <= a.at) return false;
  // A row of a that starts within b hits by its offset modulo b's step, which repeats after
  // step / gcd rows of a; one that starts before b and reaches it hits.
  const int64_t first = a.at >= b.at ? 0 : static_cast<int64_t>(b.at - a.at) / a.step;
  const int64_t last = std::min(a.rows - 1, static_cast<int64_t>(b.end() - 1 - a.at) / a.step);
  auto hits = [&](int64_t i) {
    const int64_t lo = static_cast<int64_t>(a.at - b.at) + i * a.step, hi = lo + a.run;  // from b's start
    if (hi <= 0 || lo >= (b.rows - 1) * b.step + b.run) return false;
    if (lo < 0) return true;
    const int64_t in = lo % b.step;
    return in < b.run || in + a.run > b.step;
  };
  const int64_t period = b.rows > 1 ? b.step / std::gcd(a.step, b.step) : 1;
  for (int64_t i = first; i <= last && i <= first + period; ++i)
    if (hits(i)) return true;
  return false;
}

// Whether one of the `outputs` shares memory with an input or with another output.
bool outputs_shared(std::initializer_list<Span> outputs, std::initializer_list<Span> inputs) {
  for (const Span* o = outputs.begin(); o != outputs.end(); ++o) {
    for (const Span& in : inputs)
      if (shares(*o, in)) return true;
    for (const Span* other = outputs.begin(); other != o; ++other)
      if (shares(*o, *other)) return true;
  }
  return false;
}

// Exactly one of W / qw, of the expected shape.
int check_operand(const float* W, const qat_qweight* qw, int64_t N, int64_t K) {
  if ((W == nullptr) == (qw == nullptr)) return QAT_ERR_ARG;
  if (!qw) return aligned16(W) ? QAT_OK : QAT_ERR_ALIGN;
  if (!qw->operand || qw->N != N || qw->K != K) return QAT_ERR_ARG;
  return aligned16(qw->operand) ? QAT_OK : QAT_ERR_ALIGN;
}

// What get_operand reads.
Span words_span(const float* W, const qat_qweight* qw, int64_t N, int64_t K) {
  return W ? Span(W, N * K * 4) : Span(qw->operand, N * K * 2);
}

// The bf16 operand of a weight: taken from `qw`, or produced from fp32 `W`
// into the workspace.
int get_operand(const float* W, const qat_qweight* qw, int64_t N, int64_t K, int bits, Carver& ws,
                cudaStream_t s, const __nv_bfloat16** out) {
  if (const int rc = check_operand(W, qw, N, K)) return rc;
  if (qw) {
    *out = reinterpret_cast<const __nv_bfloat16*>(qw->operand);
    return QAT_OK;
  }
  void* op = ws.take(N * K * 2);
  void* sc = ws.take(N * 4);
  if (!op || !sc) return QAT_ERR_WORKSPACE;
  const int rc = launch_quantize_weights(W, static_cast<int>(N), static_cast<int>(K), bits, nullptr,
                                         static_cast<float*>(sc),
                                         static_cast<__nv_bfloat16*>(op), s);
  *out = static_cast<const __nv_bfloat16*>(op);
  return rc;
}

bool aligned_to(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// Longest row stride in bf16 elements (the tensor maps' stride field).
constexpr int64_t kMaxStride = 1ll << 38;

// ---- softmax cross entropy
constexpr int64_t kCeMaxVocab = 1 << 20;
constexpr int64_t kCeMaxTokens = (1ll << 31) - 256;

// Tokens that one accumulator of dW sums: the tensor core's fp32 accumulation truncates
// at every step, the runs are added rounded to nearest.  dW of the 8,192-word head over
// 65,536 tokens is off by (relative, against 64 bits) 1.1e-5 with runs of 9,472 and 3e-6
// to 5e-6 with these (4,099 tokens of 50,257 words: 3.5e-6, fp32 multiply-adds 1.1e-6).
constexpr int64_t kCeTokenRun = 2048;

// Row stride of the gradient pieces [rows, V]: 16-byte rows.
inline int64_t ce_ldg(int64_t V) { return (V + 7) / 8 * 8; }

// Tokens of one piece of the backward.  The product g . W has
// ceil(rows / 256) x ceil(d / 256) tiles and reduces over the whole vocabulary
// in each, so a piece takes as many tokens as fill the CTA pairs once (9,472 at
// d = 512), but at most 1 GiB of gradient, and at least one row of tiles.
int64_t ce_rows_wanted(int64_t V, int64_t d, int64_t T) {
  const int64_t n_blk = (d + 255) / 256, pairs = sm_count() / 2;
  int64_t rows = 256 * std::max<int64_t>(1, pairs / n_blk);
  rows = std::min<int64_t>(rows, (1ll << 30) / (4 * ce_ldg(V)) / 256 * 256);
  return std::min<int64_t>(std::max<int64_t>(rows, 256), T);
}

// (Fewer than 256 tokens may take narrower tiles, hence more statistics each: a workspace
// of the longest batch serves the shorter ones.)
size_t ce_fwd_bytes(int64_t V, int64_t T) {
  const int64_t few = std::min<int64_t>(T, 255);
  return align_up(std::max(ce_slots(T, V) * T, ce_slots(few, V) * few) * 8) + align_up(T * 4) +
         align_up(ce_parts_bytes(T));
}
size_t ce_bwd_bytes(int64_t V, int64_t rows) {
  return 2 * align_up(rows * ce_ldg(V) * 2) + align_up(rows * 4);
}
// The products of a piece of n tokens without their addresses: dZ = g . Wq, and dW = g^T . Z
// with both halves of g.
GemmDesc ce_dz_product(int64_t V, int64_t d, int64_t n) {
  GemmDesc x;
  x.M = n; x.N = d; x.K = V;
  x.b_mn = true;
  return x;
}
GemmDesc ce_dw_product(int64_t V, int64_t d, int64_t n, const void* half) {
  GemmDesc w;
  w.M = V; w.N = d; w.K = n;
  w.A2 = half;
  w.a_mn = w.b_mn = true;
  w.epi = EPI_F32;
  w.k_run = kCeTokenRun;
  return w;
}
// Partial products where the output tiles leave most of the GPU idle and the reduction is
// split (0: it is not): dZ of a piece of few tokens, over the vocabulary, and dW of a small
// head, over the tokens; both are joined in order, one after the other in the same place.
// Loss and gradients with dZ split (dW's two halves in one product and the joins
// included): one token of 50,000 words, d = 512, 361 -> 89 us; 300 of 20,001, d = 256,
// 165 -> 66 us; 1,500 of 50,257, d = 768, 689 -> 544 us.
size_t ce_slab_bytes(const GemmDesc& g) {
  if (g.M <= 0 || g.K <= 0) return 0;
  const Slabs s = f32_slabs(g);
  return s.count > 1 ? align_up(s.count * s.rows * g.N * 4) : 0;
}
size_t ce_slab_bytes(int64_t V, int64_t d, int64_t n, bool dz, bool dw) {
  const int half = 0;
  return std::max(dz ? ce_slab_bytes(ce_dz_product(V, d, n)) : 0,
                  dw ? ce_slab_bytes(ce_dw_product(V, d, n, &half)) : 0);
}
// What every piece of T tokens, `rows` at a time, can use.
size_t ce_slab_bytes_max(int64_t V, int64_t d, int64_t T, int64_t rows, bool dz, bool dw) {
  return std::max(ce_slab_bytes(V, d, rows, dz, dw), ce_slab_bytes(V, d, T % rows, dz, dw));
}

// ---- attention
// Longest sequence of keys under more than 128 queries.  The second tile of a piece of
// work may have no queries, and its warps then wait for the next piece while the first
// tile walks all keys: about 2 us a block of 128, 1.1 s of the 2 s after which a device-side
// wait gives up.  (The backward's grids end at 65,535 * 128 keys; up to 128 queries both
// tiles walk.)
constexpr int64_t kAttnMaxKeys = 1ll << 26;

// The checks that both directions share; fills the kernels' arguments.
int attn_args(const qat_attn* a, const qat_bf16* Q, const qat_bf16* K, const qat_bf16* V,
              const qat_bf16* O, const float* lse, AttnArgs* out) {
  if (!a || a->Tq < 0 || a->Tk < 0 || a->batch < 0 || a->max_q < 0 || a->max_k < 0) return QAT_ERR_ARG;
  if (a->heads <= 0 || a->kv_heads <= 0 || a->heads % a->kv_heads || a->window < 0)
    return QAT_ERR_ARG;
  if (a->window > 0 && !a->causal) return QAT_ERR_ARG;
  if (!std::isfinite(a->scale) || a->scale < 0.0f) return QAT_ERR_ARG;
  if (a->head_dim <= 0 || (a->head_dim & 7) || a->head_dim > QAT_ATTN_MAX_HEAD_DIM || a->heads > 65536)
    return QAT_ERR_SHAPE;
  if (a->Tq > (1ll << 31) - 512 || a->Tk > (1ll << 31) - 512) return QAT_ERR_SHAPE;
  if (!a->cu_q && a->Tq != static_cast<int64_t>(a->batch) * a->max_q) return QAT_ERR_ARG;
  if (!a->cu_k && a->Tk != static_cast<int64_t>(a->batch) * a->max_k) return QAT_ERR_ARG;
  if ((a->Tq > 0 && (!Q || !O || !lse)) || (a->Tk > 0 && (!K || !V))) return QAT_ERR_ARG;
  const int64_t wq = static_cast<int64_t>(a->heads) * a->head_dim;
  const int64_t wk = static_cast<int64_t>(a->kv_heads) * a->head_dim;
  const int64_t ldq = a->ldq ? a->ldq : wq, ldo = a->ldo ? a->ldo : wq;
  const int64_t ldk = a->ldk ? a->ldk : wk, ldv = a->ldv ? a->ldv : wk;
  if (ldq < wq || ldo < wq || ldk < wk || ldv < wk || ((ldq | ldo | ldk | ldv) & 7))
    return QAT_ERR_SHAPE;
  if (std::max({ldq, ldo, ldk, ldv}) > kMaxStride) return QAT_ERR_SHAPE;
  if (!aligned16(Q) || !aligned16(K) || !aligned16(V) || !aligned16(O)) return QAT_ERR_ALIGN;
  if (!aligned_to(lse, 4) || !aligned_to(a->cu_q, 4) || !aligned_to(a->cu_k, 4)) return QAT_ERR_ALIGN;
  AttnArgs p{};
  p.Tq = a->Tq; p.Tk = a->Tk;
  p.cu_q = a->cu_q; p.cu_k = a->cu_k;
  p.batch = a->batch; p.max_q = a->max_q; p.max_k = a->max_k;
  p.heads = a->heads; p.group = a->heads / a->kv_heads; p.hd = a->head_dim;
  p.causal = a->causal != 0; p.window = a->window;
  p.scale = a->scale != 0.0f ? a->scale : 1.0f / std::sqrt(static_cast<float>(a->head_dim));
  p.Q = Q; p.K = K; p.V = V;
  p.O = const_cast<qat_bf16*>(O);
  p.lse = const_cast<float*>(lse);
  p.ldq = ldq; p.ldk = ldk; p.ldv = ldv; p.ldo = ldo;
  if (a->Tk == 0) {  // no key is ever loaded, but the maps need an address
    p.K = p.V = Q;
    p.ldk = p.ldv = ldq;
  }
  *out = p;
  return QAT_OK;
}

// The memory of what both directions are given.
struct AttnSpans {
  Span Q, K, V, O, lse, cu_q, cu_k;
  AttnSpans(const AttnArgs& p, const qat_attn& a, const qat_bf16* q, const qat_bf16* k, const qat_bf16* v)
      : Q(rows_span(q, p.Tq, p.ldq, width(p.heads, p))),
        K(rows_span(k, p.Tk, p.ldk, width(p.heads / p.group, p))),
        V(rows_span(v, p.Tk, p.ldv, width(p.heads / p.group, p))),
        O(rows_span(static_cast<const qat_bf16*>(p.O), p.Tq, p.ldo, width(p.heads, p))),
        lse(p.lse, p.heads * p.Tq * 4),
        cu_q(a.cu_q, (static_cast<int64_t>(a.batch) + 1) * 4),
        cu_k(a.cu_k, (static_cast<int64_t>(a.batch) + 1) * 4) {}
  static int64_t width(int heads, const AttnArgs& p) { return static_cast<int64_t>(heads) * p.hd; }
};

}  // namespace
}  // namespace qat

using namespace qat;

extern "C" {

const char* qat_strerror(int code) {
  switch (code) {
    case QAT_OK: return "ok";
    case QAT_ERR_ARG: return "invalid argument";
    case QAT_ERR_ALIGN: return "pointer not 16-byte aligned";
    case QAT_ERR_SHAPE: return "unsupported shape (feature dims must be multiples of 8)";
    case QAT_ERR_WORKSPACE: return "workspace missing or too small";
    case QAT_ERR_CUDA: return "CUDA runtime error";
    case QAT_ERR_TIMEOUT: return "a bounded device wait timed out";
    case QAT_ERR_UNSUPPORTED: return "unsupported device or driver";
    default: return "unknown error";
  }
}

int64_t qat_launch_count(void) { return g_launches.load(std::memory_order_relaxed); }

int qat_device_error(qat_stream_t stream) {
  if (cudaStreamSynchronize(stream) != cudaSuccess) return QAT_ERR_CUDA;
  int v = 0, zero = 0;
  if (cudaMemcpyFromSymbol(&v, g_device_error, sizeof(int)) != cudaSuccess) return QAT_ERR_CUDA;
  if (v != 0 && cudaMemcpyToSymbol(g_device_error, &zero, sizeof(int)) != cudaSuccess)
    return QAT_ERR_CUDA;
  return v;
}

int qat_noisy_operand(const float* W, int32_t N, int32_t K, int32_t bits, uint64_t seed,
                      uint64_t offset, float* scales, qat_bf16* operand, qat_stream_t stream) {
  if (!W || !operand || N <= 0 || !bits_ok(bits)) return QAT_ERR_ARG;
  if (!dim_ok(K)) return QAT_ERR_SHAPE;
  if (!aligned16(W) || !aligned16(operand)) return QAT_ERR_ALIGN;
  return launch_noisy_operand(W, N, K, bits, seed, offset, scales,
                              reinterpret_cast<__nv_bfloat16*>(operand), stream);
}

size_t qat_workspace_size(int32_t op, int32_t N_or_d, int32_t K_or_H, int64_t T,
                          int32_t raw_weights) {
  const int64_t a = N_or_d, b = K_or_H;
  if (a <= 0 || b <= 0 || T < 0) return 0;
  switch (op) {
    case QAT_OP_LINEAR_FWD:
    case QAT_OP_LINEAR_BWD:
      return raw_weights ? operand_bytes(a, b) : 0;
    case QAT_OP_MLP_FWD:  // h [T,H] when not saved by the caller, + operands of fc [H,d], proj [d,H]
    case QAT_OP_MLP_BWD:  // dpre [T,H] + operands
      return align_up(static_cast<size_t>(T) * b * 2) +
             (raw_weights ? operand_bytes(b, a) + operand_bytes(a, b) : 0);
    case QAT_OP_CE_FWD:
    case QAT_OP_CE_BWD: {  // a = V, b = d; the backward's size serves the forward too
      if (a > kCeMaxVocab || T > kCeMaxTokens) return 0;
      size_t n = T > 0 ? ce_fwd_bytes(a, T) : 0;
      if (op == QAT_OP_CE_BWD && T > 0) {
        const int64_t rows = ce_rows_wanted(a, b, T);
        n = std::max(n, ce_bwd_bytes(a, rows) + ce_slab_bytes_max(a, b, T, rows, true, true));
      }
      return n + (raw_weights ? operand_bytes(a, b) : 0);
    }
    case QAT_OP_ATTN_BWD:  // a = heads: rowsum(dO * O) of every query and head
      return align_up(static_cast<size_t>(a) * T * 4);
    default:
      return 0;
  }
}

int qat_quantize_weights(const float* W, int32_t N, int32_t K, int32_t bits, int8_t* codes,
                         float* scales, qat_bf16* operand, qat_stream_t stream) {
  if (!W || !scales || N <= 0 || !bits_ok(bits)) return QAT_ERR_ARG;
  if (!dim_ok(K)) return QAT_ERR_SHAPE;
  if (!aligned16(W) || (codes && !aligned16(codes)) || (operand && !aligned16(operand)))
    return QAT_ERR_ALIGN;
  return launch_quantize_weights(W, N, K, bits, codes, scales,
                                 reinterpret_cast<__nv_bfloat16*>(operand), stream);
}

int qat_quantize_weights_batch(const qat_quant_desc* descs, int32_t n, qat_stream_t stream) {
  if (!descs || n <= 0 || n > QAT_QUANT_MAX_DESCS) return QAT_ERR_ARG;
  QuantBatch b;
  b.n = n;
  b.tile_begin[0] = 0;
  for (int i = 0; i < n; ++i) {
    const qat_quant_desc& s = descs[i];
    if (!s.W || !s.scales || s.N <= 0 || !bits_ok(s.bits)) return QAT_ERR_ARG;
    if (!dim_ok(s.K)) return QAT_ERR_SHAPE;
    if (!aligned16(s.W) || (s.codes && !aligned16(s.codes)) || (s.operand && !aligned16(s.operand)))
      return QAT_ERR_ALIGN;
    b.d[i] = QuantDescDev{s.W, s.codes, s.scales, reinterpret_cast<__nv_bfloat16*>(s.operand),
                          s.N, s.K, s.bits, 0};
    b.tile_begin[i + 1] = b.tile_begin[i] + quant_tiles(s.N, s.K);
  }
  return launch_quantize_batch(b, stream);
}

int qat_linear_fwd(const float* W, const qat_qweight* qw, int32_t N, int32_t K, int32_t bits,
                   const qat_bf16* X, int64_t ldx, int64_t T, const qat_bf16* residual,
                   qat_bf16* Y, void* workspace, size_t ws_bytes, qat_stream_t stream) {
  if ((T > 0 && (!X || !Y)) || T < 0 || !bits_ok(bits)) return QAT_ERR_ARG;
  if (!dim_ok(N) || !dim_ok(K)) return QAT_ERR_SHAPE;
  if (ldx == 0) ldx = K;
  if (ldx < K || (ldx & 7)) return QAT_ERR_SHAPE;
  if (T == 0) return ((W == nullptr) != (qw == nullptr)) ? QAT_OK : QAT_ERR_ARG;
  GemmDesc g;
  g.A = X; g.lda = ldx;
  g.M = T; g.N = N; g.K = K;
  g.epi = residual ? EPI_BF16_RESID : EPI_BF16;
  g.D = Y; g.ldd = N;
  g.R = residual; g.ldr = N;
  if (W && !qw && workspace == nullptr && fused_b_supported(T, N, K, g.epi)) {
    // no workspace: the GEMM quantizes W itself, the operand never reaches global memory
    if (!aligned16(W)) return QAT_ERR_ALIGN;
    g.Wraw = W;
    g.bits = bits;
    return launch_gemm(g, stream);
  }
  Carver ws(workspace, ws_bytes);
  const __nv_bfloat16* op = nullptr;
  int rc = get_operand(W, qw, N, K, bits, ws, stream, &op);
  if (rc) return rc;
  g.B = op; g.ldb = K;
  return launch_gemm(g, stream);
}

int qat_linear_bwd(const float* W, const qat_qweight* qw, int32_t N, int32_t K, int32_t bits,
                   const qat_bf16* X, int64_t ldx, const qat_bf16* dY, int64_t T,
                   const qat_bf16* dX_residual, qat_bf16* dX, float* dW, int32_t accumulate_dW,
                   void* workspace, size_t ws_bytes, qat_stream_t stream) {
  if ((T > 0 && !dY) || T < 0 || !bits_ok(bits)) return QAT_ERR_ARG;
  if (!dim_ok(N) || !dim_ok(K)) return QAT_ERR_SHAPE;
  if (T > 0 && dW && !X) return QAT_ERR_ARG;
  if (dX_residual && !dX) return QAT_ERR_ARG;
  if (ldx == 0) ldx = K;
  if (ldx < K || (ldx & 7)) return QAT_ERR_SHAPE;
  Carver ws(workspace, ws_bytes);
  if (dX) {
    const __nv_bfloat16* op = nullptr;
    int rc = get_operand(W, qw, N, K, bits, ws, stream, &op);
    if (rc) return rc;
    if (T > 0) {
      GemmDesc g;  // dX[T,K] = dY[T,N] . Wq[N,K] (+ residual): B = Wq read N-major along K
      g.A = dY; g.lda = N;
      g.B = op; g.ldb = K; g.b_mn = true;
      g.M = T; g.N = K; g.K = N;
      g.epi = dX_residual ? EPI_BF16_RESID : EPI_BF16;
      g.D = dX; g.ldd = K;
      g.R = dX_residual; g.ldr = K;
      rc = launch_gemm(g, stream);
      if (rc) return rc;
    }
  }
  if (dW) {
    if (T == 0) {
      if (!accumulate_dW) return cuda_status(cudaMemsetAsync(dW, 0, static_cast<size_t>(N) * K * 4, stream));
      return QAT_OK;
    }
    GemmDesc g;  // dW[N,K] = dY^T . X : both operands read along T
    g.A = dY; g.lda = N; g.a_mn = true;
    g.B = X; g.ldb = ldx; g.b_mn = true;
    g.M = N; g.N = K; g.K = T;
    g.epi = EPI_F32;
    g.D = dW; g.ldd = K;
    g.accumulate = accumulate_dW != 0;
    return launch_gemm(g, stream);
  }
  return QAT_OK;
}

int qat_mlp_fwd(const float* Wfc, const float* Wproj, const qat_qweight* qfc,
                const qat_qweight* qproj, int32_t d, int32_t H, int32_t bits, int32_t act,
                const qat_bf16* X, int64_t T, const qat_bf16* residual, qat_bf16* Y,
                qat_bf16* pre_save, qat_bf16* h_save, void* workspace, size_t ws_bytes,
                qat_stream_t stream) {
  if ((T > 0 && (!X || !Y)) || T < 0 || !bits_ok(bits) || !act_ok(act)) return QAT_ERR_ARG;
  if (!dim_ok(d) || !dim_ok(H)) return QAT_ERR_SHAPE;
  if ((pre_save && !aligned16(pre_save)) || (h_save && !aligned16(h_save))) return QAT_ERR_ALIGN;
  Carver ws(workspace, ws_bytes);
  const __nv_bfloat16 *op_fc = nullptr, *op_proj = nullptr;
  const int fc_epi = act == QAT_ACT_RELU2 ? EPI_RELU2 : EPI_LRELU2;
  // fc from fp32 weights and no workspace: the fc GEMM quantizes Wfc itself
  const bool fc_fused = Wfc && !qfc && !workspace && T > 0 && fused_b_supported(T, H, d, fc_epi);
  int rc = QAT_OK;
  if (fc_fused) {
    if (!aligned16(Wfc)) return QAT_ERR_ALIGN;
  } else {
    rc = get_operand(Wfc, qfc, H, d, bits, ws, stream, &op_fc);
    if (rc) return rc;
  }
  rc = get_operand(Wproj, qproj, d, H, bits, ws, stream, &op_proj);
  if (rc) return rc;
  if (T == 0) return QAT_OK;
  void* h = h_save;
  if (!h) {
    h = ws.take(static_cast<size_t>(T) * H * 2);
    if (!h) return QAT_ERR_WORKSPACE;
  }
  GemmDesc g1;  // pre = X . Wfc^T ; h = act(pre)
  g1.A = X; g1.lda = d;
  g1.B = op_fc; g1.ldb = d;
  if (fc_fused) {
    g1.Wraw = Wfc;
    g1.bits = bits;
  }
  g1.M = T; g1.N = H; g1.K = d;
  g1.epi = fc_epi;
  g1.D = pre_save; g1.ldd = H;
  g1.D2 = h; g1.ldd2 = H;
  rc = launch_gemm(g1, stream);
  if (rc) return rc;
  GemmDesc g2;  // Y = h . Wproj^T (+ residual)
  g2.A = h; g2.lda = H;
  g2.B = op_proj; g2.ldb = H;
  g2.M = T; g2.N = d; g2.K = H;
  g2.epi = residual ? EPI_BF16_RESID : EPI_BF16;
  g2.D = Y; g2.ldd = d;
  g2.R = residual; g2.ldr = d;
  return launch_gemm(g2, stream);
}

int qat_mlp_bwd(const float* Wfc, const float* Wproj, const qat_qweight* qfc,
                const qat_qweight* qproj, int32_t d, int32_t H, int32_t bits, int32_t act,
                const qat_bf16* X, const qat_bf16* pre, const qat_bf16* h, const qat_bf16* dY,
                int64_t T, const qat_bf16* dX_residual, qat_bf16* dX, qat_bf16* dpre_save,
                float* dWfc, float* dWproj, int32_t accumulate_dW, void* workspace,
                size_t ws_bytes, qat_stream_t stream) {
  if ((T > 0 && (!X || !pre || !h || !dY)) || T < 0 || !bits_ok(bits) || !act_ok(act))
    return QAT_ERR_ARG;
  if (dX_residual && !dX) return QAT_ERR_ARG;
  if (!dim_ok(d) || !dim_ok(H)) return QAT_ERR_SHAPE;
  Carver ws(workspace, ws_bytes);
  const __nv_bfloat16 *op_fc = nullptr, *op_proj = nullptr;
  int rc = get_operand(Wfc, qfc, H, d, bits, ws, stream, &op_fc);
  if (rc) return rc;
  rc = get_operand(Wproj, qproj, d, H, bits, ws, stream, &op_proj);
  if (rc) return rc;
  if (T == 0) {
    if (!accumulate_dW) {
      if (dWfc && cudaMemsetAsync(dWfc, 0, static_cast<size_t>(H) * d * 4, stream) != cudaSuccess)
        return QAT_ERR_CUDA;
      if (dWproj && cudaMemsetAsync(dWproj, 0, static_cast<size_t>(d) * H * 4, stream) != cudaSuccess)
        return QAT_ERR_CUDA;
    }
    return QAT_OK;
  }
  if (dpre_save && !aligned16(dpre_save)) return QAT_ERR_ALIGN;
  void* dpre = dpre_save ? static_cast<void*>(dpre_save) : ws.take(static_cast<size_t>(T) * H * 2);
  if (!dpre) return QAT_ERR_WORKSPACE;
  if (dWproj) {  // dWproj[d,H] = dY^T . h
    GemmDesc g;
    g.A = dY; g.lda = d; g.a_mn = true;
    g.B = h; g.ldb = H; g.b_mn = true;
    g.M = d; g.N = H; g.K = T;
    g.epi = EPI_F32;
    g.D = dWproj; g.ldd = H;
    g.accumulate = accumulate_dW != 0;
    rc = launch_gemm(g, stream);
    if (rc) return rc;
  }
  {  // dpre[T,H] = (dY . Wproj_q) * act'(pre)
    GemmDesc g;
    g.A = dY; g.lda = d;
    g.B = op_proj; g.ldb = H; g.b_mn = true;
    g.M = T; g.N = H; g.K = d;
    g.epi = act == QAT_ACT_RELU2 ? EPI_DRELU2 : EPI_DLRELU2;
    g.D = dpre; g.ldd = H;
    g.R = pre; g.ldr = H;
    rc = launch_gemm(g, stream);
    if (rc) return rc;
  }
  if (dWfc) {  // dWfc[H,d] = dpre^T . X
    GemmDesc g;
    g.A = dpre; g.lda = H; g.a_mn = true;
    g.B = X; g.ldb = d; g.b_mn = true;
    g.M = H; g.N = d; g.K = T;
    g.epi = EPI_F32;
    g.D = dWfc; g.ldd = d;
    g.accumulate = accumulate_dW != 0;
    rc = launch_gemm(g, stream);
    if (rc) return rc;
  }
  if (dX) {  // dX[T,d] = dpre . Wfc_q (+ residual)
    GemmDesc g;
    g.A = dpre; g.lda = H;
    g.B = op_fc; g.ldb = d; g.b_mn = true;
    g.M = T; g.N = d; g.K = H;
    g.epi = dX_residual ? EPI_BF16_RESID : EPI_BF16;
    g.D = dX; g.ldd = d;
    g.R = dX_residual; g.ldr = d;
    rc = launch_gemm(g, stream);
    if (rc) return rc;
  }
  return QAT_OK;
}

int quantize_rows_export(const float* W, int64_t rows, int64_t cols, int32_t bits, int8_t* codes,
                         qat_fp16* scales, qat_stream_t stream) {
  qat_export_desc d;
  d.src = W;
  d.rows = rows;
  d.cols = cols;
  d.mode = bits;
  d.flags = 0;
  d.dst = codes;
  d.scales = scales;
  if (!bits_ok(bits)) return QAT_ERR_ARG;
  return quantize_export_batch(&d, 1, stream);
}

int quantize_export_batch(const qat_export_desc* descs, int32_t n, qat_stream_t stream) {
  if (!descs || n <= 0 || n > QAT_EXPORT_MAX_DESCS) return QAT_ERR_ARG;
  static thread_local ExportBatch b;  // ~20 KB: kept off the stack
  b.n = n;
  b.total_units = 0;
  for (int i = 0; i < n; ++i) {
    const qat_export_desc& s = descs[i];
    ExportDescDev& d = b.d[i];
    if (!s.src || !s.dst || s.rows < 0 || s.cols < 0) return QAT_ERR_ARG;
    if (!aligned16(s.src) || !aligned16(s.dst)) return QAT_ERR_ALIGN;
    d.src = s.src;
    d.dst = s.dst;
    d.scales = reinterpret_cast<__half*>(s.scales);
    d.mode = s.mode;
    d.m = 1;
    d.frac = 0.0f;
    if (s.flags & ~(QAT_EXPORT_PACK6 | QAT_EXPORT_CLIP_SEARCH)) return QAT_ERR_ARG;
    d.pack6 = (s.flags & QAT_EXPORT_PACK6) != 0;
    d.search = (s.flags & QAT_EXPORT_CLIP_SEARCH) != 0;
    d.pad = 0;
    if (d.pack6 && s.mode != 5 && s.mode != 6) return QAT_ERR_ARG;
    if (d.search && !bits_ok(s.mode)) return QAT_ERR_ARG;
    if (d.search && !clip_search_supported(s.cols)) return QAT_ERR_SHAPE;
    d.unit_begin = b.total_units;
    if (s.mode == QAT_EXPORT_FP16) {
      d.numel = s.rows * s.cols;
      d.cols = kFp16Chunk;
      d.rows = (d.numel + kFp16Chunk - 1) / kFp16Chunk;
      d.unit_rows = 1;
    } else if (bits_ok(s.mode)) {
      if (!s.scales) return QAT_ERR_ARG;
      if (!dim_ok(s.cols)) return QAT_ERR_SHAPE;
      d.rows = s.rows;
      d.cols = s.cols;
      d.numel = s.rows * s.cols;
      // staged rows travel in units of as many rows as fit kExportUnitBytes
      d.unit_rows = (s.cols <= kExportMaxStagedCols)
                        ? std::max<int64_t>(1, kExportUnitBytes / (s.cols * 4))
                        : 1;
      const int rc = export_quantile_params(s.cols, &d.m, &d.frac);
      if (rc) return rc;
    } else {
      return QAT_ERR_ARG;
    }
    b.total_units += (d.rows + d.unit_rows - 1) / d.unit_rows;
  }
  return launch_export_batch(b, stream);
}

int unpack_codes6(const uint8_t* packed, int64_t n, int32_t bits, int8_t* codes,
                  qat_stream_t stream) {
  if (!packed || !codes || n < 0 || (bits != 5 && bits != 6)) return QAT_ERR_ARG;
  if (n % 8 != 0) return QAT_ERR_SHAPE;
  if (!aligned16(packed) || !aligned16(codes)) return QAT_ERR_ALIGN;
  return launch_unpack6(packed, n, bits, codes, stream);
}

int dequantize_rows(const int8_t* codes, const qat_fp16* scales, int64_t rows, int64_t cols,
                    int32_t out_dtype, void* out, qat_stream_t stream) {
  if (!codes || !scales || !out || rows < 0) return QAT_ERR_ARG;
  if (out_dtype != QAT_DTYPE_F32 && out_dtype != QAT_DTYPE_BF16) return QAT_ERR_ARG;
  if (!dim_ok(cols)) return QAT_ERR_SHAPE;
  if (!aligned16(codes) || !aligned16(out)) return QAT_ERR_ALIGN;
  return launch_dequant(codes, reinterpret_cast<const __half*>(scales), rows, cols,
                        out_dtype == QAT_DTYPE_BF16, out, stream);
}

int dequantize_rows_batch(const qat_dequant_desc* descs, int32_t n, qat_stream_t stream) {
  if (!descs || n <= 0 || n > QAT_DEQUANT_MAX_DESCS) return QAT_ERR_ARG;
  static thread_local DequantBatch b;  // ~14 KB: kept off the stack
  b.n = n;
  b.tile_begin[0] = 0;
  for (int i = 0; i < n; ++i) {
    const qat_dequant_desc& s = descs[i];
    if (!s.codes || !s.scales || !s.out || s.rows < 0) return QAT_ERR_ARG;
    if (s.out_dtype != QAT_DTYPE_F32 && s.out_dtype != QAT_DTYPE_BF16) return QAT_ERR_ARG;
    if (!dim_ok(s.cols)) return QAT_ERR_SHAPE;
    if (!aligned16(s.codes) || !aligned16(s.out)) return QAT_ERR_ALIGN;
    DequantDescDev& d = b.d[i];
    d.codes = s.codes;
    d.scales = reinterpret_cast<const __half*>(s.scales);
    d.out = s.out;
    d.items = s.rows * (s.cols >> 2);
    d.row_magic = dequant_row_magic(s.cols >> 2);
    d.out_bf16 = s.out_dtype == QAT_DTYPE_BF16;
    d.pad = 0;
    b.tile_begin[i + 1] = b.tile_begin[i] + (d.items + kDequantTile - 1) / kDequantTile;
  }
  return launch_dequant_batch(b, stream);
}

int qat_ce_fwd(const float* W, const qat_qweight* qw, int32_t V, int32_t d, int32_t bits,
               const qat_bf16* Z, int64_t ldz, int64_t T, const int64_t* targets, float* loss,
               float* lse, float* mean, void* workspace, size_t ws_bytes, qat_stream_t stream) {
  if (T < 0 || V <= 0 || !bits_ok(bits) || (T > 0 && (!Z || !targets || !loss || !lse)))
    return QAT_ERR_ARG;
  if ((W == nullptr) == (qw == nullptr)) return QAT_ERR_ARG;
  if (!dim_ok(d) || V > kCeMaxVocab || T > kCeMaxTokens) return QAT_ERR_SHAPE;
  if (ldz == 0) ldz = d;
  if (ldz < d || (ldz & 7) || ldz > kMaxStride) return QAT_ERR_SHAPE;
  if (!aligned_to(targets, 8) || !aligned_to(loss, 4) || !aligned_to(lse, 4) || !aligned_to(mean, 4))
    return QAT_ERR_ALIGN;
  if (T == 0)
    return mean ? cuda_status(cudaMemsetAsync(mean, 0, 8, stream)) : static_cast<int>(QAT_OK);
  if (!aligned16(Z) || !aligned16(workspace)) return QAT_ERR_ALIGN;
  Carver ws(workspace, ws_bytes);
  CeJoin j{};
  j.slots = static_cast<int>(ce_slots(T, V));
  float2* stats = static_cast<float2*>(ws.take(static_cast<size_t>(j.slots) * T * 8));
  float* tlogit = static_cast<float*>(ws.take(static_cast<size_t>(T) * 4));
  j.parts = ws.take(ce_parts_bytes(T));
  if (!stats || !tlogit || !j.parts) return QAT_ERR_WORKSPACE;
  int rc = check_operand(W, qw, V, d);
  if (rc) return rc;
  const size_t used = ws.used + (W ? operand_bytes(V, d) : 0);
  if (used > ws_bytes) return QAT_ERR_WORKSPACE;
  if (outputs_shared({Span(loss, T * 4), Span(lse, T * 4), Span(mean, 8), Span(workspace, used)},
                     {rows_span(Z, T, ldz, d), Span(targets, T * 8), words_span(W, qw, V, d)}))
    return QAT_ERR_ARG;
  const __nv_bfloat16* op = nullptr;
  rc = get_operand(W, qw, V, d, bits, ws, stream, &op);
  if (rc) return rc;
  GemmDesc g;  // logits = Z . Wq^T, as tiles that only the epilogue sees
  g.A = Z; g.lda = ldz;
  g.B = op; g.ldb = d;
  g.M = T; g.N = V; g.K = d;
  g.epi = EPI_CE_STATS;
  g.ce.targets = targets;
  g.ce.vocab = V;
  g.ce.stats = stats;
  g.ce.tlogit = tlogit;
  rc = launch_gemm(g, stream);
  if (rc) return rc;
  j.stats = stats;
  j.tlogit = tlogit;
  j.targets = targets;
  j.loss = loss;
  j.lse = lse;
  j.mean = mean;
  j.T = T;
  j.vocab = V;
  return launch_ce_join(j, stream);
}

int qat_ce_bwd(const float* W, const qat_qweight* qw, int32_t V, int32_t d, int32_t bits,
               const qat_bf16* Z, int64_t ldz, int64_t T, const int64_t* targets, const float* lse,
               const float* dloss, const float* gscale, qat_bf16* dZ, float* dW,
               int32_t accumulate_dW, void* workspace, size_t ws_bytes, qat_stream_t stream) {
  if (T < 0 || V <= 0 || !bits_ok(bits) || (T > 0 && (!Z || !targets || !lse))) return QAT_ERR_ARG;
  if ((W == nullptr) == (qw == nullptr)) return QAT_ERR_ARG;
  if (!dim_ok(d) || V > kCeMaxVocab || T > kCeMaxTokens) return QAT_ERR_SHAPE;
  if (ldz == 0) ldz = d;
  if (ldz < d || (ldz & 7) || ldz > kMaxStride) return QAT_ERR_SHAPE;
  if (!aligned_to(targets, 8) || !aligned_to(lse, 4) || !aligned_to(dloss, 4) ||
      !aligned_to(gscale, 4))
    return QAT_ERR_ALIGN;
  if ((dZ && !aligned16(dZ)) || (dW && !aligned16(dW))) return QAT_ERR_ALIGN;
  if (!dZ && !dW) return QAT_OK;
  if (T == 0) {
    if (dW && !accumulate_dW)
      return cuda_status(cudaMemsetAsync(dW, 0, static_cast<size_t>(V) * d * 4, stream));
    return QAT_OK;
  }
  if (!aligned16(Z) || !aligned16(workspace)) return QAT_ERR_ALIGN;
  int rc = check_operand(W, qw, V, d);
  if (rc) return rc;
  Carver ws(workspace, ws_bytes);
  Carver operand_ws = ws;  // its place comes first; it is filled once nothing is left to refuse
  if (W) ws.used += operand_bytes(V, d);
  // Tokens of a piece: what the operator asks for, or what the workspace holds
  // (whole row tiles), down to one of them.
  const int64_t ldg = ce_ldg(V);
  int64_t rows = ce_rows_wanted(V, d, T);
  const size_t left = ws_bytes > ws.used ? ws_bytes - ws.used : 0;
  if (ce_bwd_bytes(V, rows) > left) {
    rows = static_cast<int64_t>(left / (4 * static_cast<size_t>(ldg))) / 256 * 256;
    while (rows > 0 && ce_bwd_bytes(V, rows) > left) rows -= 256;
    if (rows <= 0) return QAT_ERR_WORKSPACE;
  }
  void* ghi = ws.take(static_cast<size_t>(rows) * ldg * 2);
  void* glo = ws.take(static_cast<size_t>(rows) * ldg * 2);
  float* rem = static_cast<float*>(ws.take(static_cast<size_t>(rows) * 4));
  if (!ghi || !glo || !rem) return QAT_ERR_WORKSPACE;
  // (a smaller workspace than asked for may leave no room for these: the product is then whole)
  const size_t slab_bytes = ce_slab_bytes_max(V, d, T, rows, dZ != nullptr, dW != nullptr);
  float* slabs = slab_bytes ? static_cast<float*>(ws.take(slab_bytes)) : nullptr;
  // (dW reads the rows of Z after their dZ is written)
  if (outputs_shared({Span(dZ, T * d * 2), Span(dW, static_cast<int64_t>(V) * d * 4),
                      Span(workspace, std::min(ws.used, ws_bytes))},
                     {rows_span(Z, T, ldz, d), Span(targets, T * 8), Span(lse, T * 4), Span(dloss, T * 4),
                      Span(gscale, 4), words_span(W, qw, V, d)}))
    return QAT_ERR_ARG;
  const __nv_bfloat16* op = nullptr;
  rc = get_operand(W, qw, V, d, bits, operand_ws, stream, &op);
  if (rc) return rc;
  for (int64_t t0 = 0; t0 < T; t0 += rows) {
    const int64_t n = std::min(rows, T - t0);
    const qat_bf16* Zp = Z + t0 * ldz;
    GemmDesc g;  // g = (softmax(Z . Wq^T) - [target]) * dloss, as bf16 and its remainder
    g.A = Zp; g.lda = ldz;
    g.B = op; g.ldb = d;
    g.M = n; g.N = V; g.K = d;
    g.epi = EPI_CE_GRAD;
    g.D = ghi; g.ldd = ldg;
    g.D2 = dW ? glo : nullptr; g.ldd2 = ldg;
    g.ce.targets = targets + t0;
    g.ce.vocab = V;
    g.ce.rem = dZ ? rem : nullptr;
    g.ce.lse = lse + t0;
    g.ce.dloss = dloss ? dloss + t0 : nullptr;
    g.ce.gscale = gscale;
    rc = launch_gemm(g, stream);
    if (rc) return rc;
    if (dZ) {  // dZ = g . Wq from g's bf16 half, the target's remainder added at the end
      GemmDesc x = ce_dz_product(V, d, n);
      x.A = ghi; x.lda = ldg;
      x.B = op; x.ldb = d;
      const Slabs sl = f32_slabs(x);
      if (slabs && sl.count > 1) {  // few tokens: over parts of the vocabulary, joined after
        x.epi = EPI_F32;
        x.slabs = true;
        x.D = slabs; x.ldd = d;
        rc = launch_gemm(x, stream);
        if (rc) return rc;
        CeDz j{};
        j.slabs = slabs;
        j.count = sl.count;
        j.rows = sl.rows;
        j.targets = targets + t0;
        j.rem = rem;
        j.words = op;
        j.dZ = reinterpret_cast<__nv_bfloat16*>(dZ + t0 * d);
        j.n = n;
        j.d = d;
        j.vocab = V;
        rc = launch_ce_dz_join(j, stream);
      } else {
        x.epi = EPI_CE_DZ;
        x.D = dZ + t0 * d; x.ldd = d;
        x.ce.targets = targets + t0;
        x.ce.vocab = V;
        x.ce.rem = rem;
        x.ce.words = op;
        rc = launch_gemm(x, stream);
      }
      if (rc) return rc;
    }
    // dW (+)= g^T . Z, kept in 32 bits: g's bf16 rounding alone would leave it
    // 1e-3 off, so its remainder is multiplied too (and first: it is small), in the same
    // pass: dW of a large vocabulary is written once, not written, read and written.
    if (dW) {
      GemmDesc w = ce_dw_product(V, d, n, ghi);
      w.A = glo; w.lda = ldg;
      w.B = Zp; w.ldb = ldz;
      w.D = dW; w.ldd = d;
      const bool add = accumulate_dW != 0 || t0 > 0;
      const Slabs sl = f32_slabs(w);
      if (slabs && sl.count > 1) {  // a small head: over parts of the tokens, joined after
        w.slabs = true;
        w.D = slabs;
        rc = launch_gemm(w, stream);
        if (rc) return rc;
        CeDw j{};
        j.slabs = slabs;
        j.count = sl.count;
        j.stride = sl.rows * d;
        j.dW = dW;
        j.n = static_cast<int64_t>(V) * d;
        j.add = add;
        rc = launch_ce_dw_join(j, stream);
      } else {
        w.accumulate = add;
        rc = launch_gemm(w, stream);
      }
      if (rc) return rc;
    }
  }
  return QAT_OK;
}

int qat_rope_freqs(int32_t rotary, double base, int32_t scaling, double factor,
                   int64_t trained_len, double beta_fast, double beta_slow, double* freqs,
                   double* scale) {
  if (!freqs || !scale || rotary <= 0 || (rotary & 1) || !(base > 1.0) || !std::isfinite(base))
    return QAT_ERR_ARG;
  if (scaling != QAT_ROPE_PLAIN && scaling != QAT_ROPE_LINEAR && scaling != QAT_ROPE_NTK &&
      scaling != QAT_ROPE_YARN)
    return QAT_ERR_ARG;
  if (scaling != QAT_ROPE_PLAIN && (!(factor >= 1.0) || !std::isfinite(factor))) return QAT_ERR_ARG;
  if (scaling == QAT_ROPE_YARN && (trained_len <= 0 || !(beta_slow > 0.0) || !(beta_fast > beta_slow)))
    return QAT_ERR_ARG;
  if (rotary > QAT_ROPE_MAX_DIMS) return QAT_ERR_SHAPE;
  const double two_pi = 6.283185307179586476925;
  const int n = rotary / 2;
  *scale = 1.0;
  if (scaling == QAT_ROPE_NTK && rotary > 2) base *= std::pow(factor, rotary / (rotary - 2.0));
  for (int i = 0; i < n; ++i) {
    freqs[i] = std::pow(base, -2.0 * i / rotary) / two_pi;
    if (scaling == QAT_ROPE_LINEAR) freqs[i] /= factor;
  }
  if (scaling == QAT_ROPE_YARN) {
    // the pair number that makes `turns` whole turns over the trained length
    auto pair_of = [&](double turns) {
      return rotary * std::log(trained_len / (turns * two_pi)) / (2.0 * std::log(base));
    };
    const double low = std::max(std::floor(pair_of(beta_fast)), 0.0);
    const double high = std::min(std::ceil(pair_of(beta_slow)), rotary - 1.0);
    for (int i = 0; i < n; ++i) {
      const double ramp =
          std::min(std::max((i - low) / std::max(high - low, 0.001), 0.0), 1.0);
      freqs[i] = freqs[i] * (1.0 - ramp) + freqs[i] / factor * ramp;
    }
    *scale = 0.1 * std::log(factor) + 1.0;
  }
  return QAT_OK;
}

int qat_rope(const void* X, int64_t ldx, void* Y, int64_t ldy, int32_t dtype, int64_t T,
             int32_t heads, int32_t head_dim, int32_t rotary, const double* freqs, float scale,
             const int64_t* positions, int64_t seq_len, int32_t interleaved, int32_t inverse,
             qat_stream_t stream) {
  if (T < 0 || heads <= 0 || seq_len < 0 || !freqs || (T > 0 && (!X || !Y))) return QAT_ERR_ARG;
  if (dtype != QAT_DTYPE_F32 && dtype != QAT_DTYPE_BF16) return QAT_ERR_ARG;
  if (!dim_ok(head_dim) || heads > (1 << 20) || rotary <= 0 || (rotary & 1) || rotary > head_dim ||
      rotary > QAT_ROPE_MAX_DIMS)
    return QAT_ERR_SHAPE;
  const int64_t width = static_cast<int64_t>(heads) * head_dim;
  if (ldx == 0) ldx = width;
  if (ldy == 0) ldy = width;
  if (width > (1 << 24) || ldx < width || ldy < width || (ldx & 7) || (ldy & 7)) return QAT_ERR_SHAPE;
  if (!aligned_to(freqs, 8) || !aligned_to(positions, 8)) return QAT_ERR_ALIGN;
  if (T == 0) return QAT_OK;
  if (!aligned16(X) || !aligned16(Y)) return QAT_ERR_ALIGN;
  if (X == Y && ldx != ldy) return QAT_ERR_ARG;
  const int64_t b = dtype == QAT_DTYPE_BF16 ? 2 : 4;
  const Span x(X, T, ldx * b, width * b), y(Y, T, ldy * b, width * b);
  if (outputs_shared({y}, {X == Y ? Span(nullptr, 0) : x, Span(freqs, rotary / 2 * 8), Span(positions, T * 8)}))
    return QAT_ERR_ARG;
  RopeArgs r{};
  r.X = X;
  r.Y = Y;
  r.ldx = ldx;
  r.ldy = ldy;
  r.T = T;
  r.positions = positions;
  r.seq_len = seq_len;
  r.freqs = freqs;
  r.scale = scale;
  r.heads = heads;
  r.head_dim = head_dim;
  r.rotary = rotary;
  r.interleaved = interleaved != 0;
  r.inverse = inverse != 0;
  r.copy_rest = X != Y;
  return launch_rope(r, dtype == QAT_DTYPE_BF16, stream);
}

int qat_attn_fwd(const qat_attn* a, const qat_bf16* Q, const qat_bf16* K, const qat_bf16* V,
                 qat_bf16* O, float* lse, qat_stream_t stream) {
  AttnArgs p;
  const int rc = attn_args(a, Q, K, V, O, lse, &p);
  if (rc) return rc;
  if (p.Tq == 0 || p.batch == 0 || p.max_q == 0) return QAT_OK;
  if (p.max_q > 128 && std::min<int64_t>(p.max_k, p.Tk) > kAttnMaxKeys) return QAT_ERR_SHAPE;
  const AttnSpans m(p, *a, Q, K, V);
  if (outputs_shared({m.O, m.lse}, {m.Q, m.K, m.V, m.cu_q, m.cu_k})) return QAT_ERR_ARG;
  return launch_attn_fwd(p, stream);
}

int qat_attn_bwd(const qat_attn* a, const qat_bf16* dO, int64_t lddo, const qat_bf16* Q,
                 const qat_bf16* K, const qat_bf16* V, const qat_bf16* O, const float* lse,
                 qat_bf16* dQ, int64_t lddq, qat_bf16* dK, int64_t lddk, qat_bf16* dV, int64_t lddv,
                 void* workspace, size_t ws_bytes, qat_stream_t stream) {
  AttnArgs p;
  const int rc = attn_args(a, Q, K, V, O, lse, &p);
  if (rc) return rc;
  if ((p.Tq > 0 && (!dO || !dQ)) || (p.Tk > 0 && (!dK || !dV))) return QAT_ERR_ARG;
  const int64_t wq = static_cast<int64_t>(p.heads) * p.hd, wk = wq / p.group;
  p.lddo = lddo ? lddo : wq;
  p.lddq = lddq ? lddq : wq;
  p.lddk = lddk ? lddk : wk;
  p.lddv = lddv ? lddv : wk;
  if (p.lddo < wq || p.lddq < wq || p.lddk < wk || p.lddv < wk ||
      ((p.lddo | p.lddq | p.lddk | p.lddv) & 7) || p.lddo > kMaxStride)
    return QAT_ERR_SHAPE;
  if (!aligned16(dO) || !aligned16(dQ) || !aligned16(dK) || !aligned16(dV) || !aligned16(workspace))
    return QAT_ERR_ALIGN;
  if (p.batch == 0 || (p.Tq == 0 && p.Tk == 0)) return QAT_OK;
  Carver ws(workspace, ws_bytes);
  p.delta = static_cast<float*>(ws.take(static_cast<size_t>(p.heads) * p.Tq * 4));
  if (p.Tq > 0 && !p.delta) return QAT_ERR_WORKSPACE;
  // the second kernel reads Q, K, V and dO when dQ is written already
  const AttnSpans m(p, *a, Q, K, V);
  if (outputs_shared({rows_span(dQ, p.Tq, p.lddq, wq), rows_span(dK, p.Tk, p.lddk, wk),
                      rows_span(dV, p.Tk, p.lddv, wk), Span(p.delta, p.Tq > 0 ? p.heads * p.Tq * 4 : 0)},
                     {m.Q, m.K, m.V, m.O, m.lse, m.cu_q, m.cu_k, rows_span(dO, p.Tq, p.lddo, wq)}))
    return QAT_ERR_ARG;
  p.dO = dO;
  p.dQ = dQ;
  p.dK = dK;
  p.dV = dV;
  if (p.Tq == 0) {  // no query is ever loaded, but the maps need an address
    p.Q = p.dO = K;
    p.ldq = p.lddo = p.ldk;
  }
  return launch_attn_bwd(p, stream);
}

}  // extern "C"
