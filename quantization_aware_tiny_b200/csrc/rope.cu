// Rotary positions: each pair (a, b) of a head's first `rotary` dimensions is
// turned by 2 pi * position * freqs[i] and scaled by m,
//   a' = m (a cos - b sin),  b' = m (a sin + b cos)   (inverse: -sin),
// the rest of the head is copied.  Bound by reading and writing the rows once.
//
// The angle is the same for all heads of a token, so a block computes the
// sines of its tokens once into shared memory (position * turns in 64 bits,
// only the fraction of a turn kept: exact to 2^-53 of the position, where an
// fp32 product is a whole turn off at two million) and then streams the rows.
#include <algorithm>
#include <type_traits>

#include "lm_ops.cuh"

namespace qat {

namespace {

constexpr int kThreads = 256;
constexpr int kMaxPairs = 512;       // rotary <= 1024
constexpr int kTablePairs = 2048;    // (cos, sin) pairs of a block: 16 KiB

template <class T>
__device__ __forceinline__ float to_f(T v) {
  if constexpr (std::is_same_v<T, float>) return v;
  else return __bfloat162float(v);
}
template <class T>
__device__ __forceinline__ T from_f(float v) {
  if constexpr (std::is_same_v<T, float>) return v;
  else return __float2bfloat16_rn(v);
}

// V consecutive elements of one row, moved at once where they are 16 bytes.
template <class T, int V>
struct alignas(V * sizeof(T) == 16 ? 16 : alignof(T)) Pack {
  T v[V];
};
template <class T, int V>
__device__ __forceinline__ Pack<T, V> load(const T* p) {
  Pack<T, V> r;
  if constexpr (V * sizeof(T) == 16) *reinterpret_cast<uint4*>(r.v) = *reinterpret_cast<const uint4*>(p);
  else {
#pragma unroll
    for (int i = 0; i < V; ++i) r.v[i] = p[i];
  }
  return r;
}
template <class T, int V>
__device__ __forceinline__ void store(T* p, const Pack<T, V>& r) {
  if constexpr (V * sizeof(T) == 16) *reinterpret_cast<uint4*>(p) = *reinterpret_cast<const uint4*>(r.v);
  else {
#pragma unroll
    for (int i = 0; i < V; ++i) p[i] = r.v[i];
  }
}

// A head's units: half layout P = rotary/2/V units of two packs (a at i, b at
// i + rotary/2), interleaved rotary/V (even V) packs of V/2 pairs; then
// (head_dim - rotary)/V packs to copy.
template <class T, int V, bool INTER>
__global__ void __launch_bounds__(kThreads) rope_kernel(const RopeArgs r, int tokens_per_block) {
  __shared__ float2 table[kTablePairs];
  const int pairs = r.rotary >> 1;
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * tokens_per_block;
  const int nt = static_cast<int>(min(static_cast<int64_t>(tokens_per_block), r.T - t0));
  for (int i = threadIdx.x; i < nt * pairs; i += kThreads) {
    const int t = i / pairs, k = i - t * pairs;
    const int64_t pos = r.positions ? r.positions[t0 + t] : (r.seq_len > 0 ? (t0 + t) % r.seq_len : t0 + t);
    const double turns = static_cast<double>(pos) * r.freqs[k];
    float s, c;
    sincospif(2.0f * static_cast<float>(turns - rint(turns)), &s, &c);
    table[i] = make_float2(c * r.scale, (r.inverse ? -s : s) * r.scale);
  }
  __syncthreads();
  const int rot_units = INTER ? r.rotary / V : pairs / V;
  const int units = rot_units + (r.copy_rest ? (r.head_dim - r.rotary) / V : 0);
  const int per_token = units * r.heads;
  const T* X = static_cast<const T*>(r.X);
  T* Y = static_cast<T*>(r.Y);
  for (int i = threadIdx.x; i < nt * per_token; i += kThreads) {
    const int t = i / per_token, j = i - t * per_token;
    const int h = j / units, u = j - h * units;
    const int64_t row = t0 + t;
    const T* x = X + row * r.ldx + h * r.head_dim;
    T* y = Y + row * r.ldy + h * r.head_dim;
    const float2* tab = table + t * pairs;
    if (u >= rot_units) {
      const int at = r.rotary + (u - rot_units) * V;
      store<T, V>(y + at, load<T, V>(x + at));
    } else if constexpr (INTER) {
      static_assert(!INTER || V % 2 == 0, "an interleaved unit holds whole pairs");
      Pack<T, V> a = load<T, V>(x + u * V);
#pragma unroll
      for (int e = 0; e < V; e += 2) {
        const float2 cs = tab[(u * V + e) >> 1];
        const float p = to_f(a.v[e]), q = to_f(a.v[e + 1]);
        a.v[e] = from_f<T>(p * cs.x - q * cs.y);
        a.v[e + 1] = from_f<T>(p * cs.y + q * cs.x);
      }
      store<T, V>(y + u * V, a);
    } else {
      Pack<T, V> a = load<T, V>(x + u * V), b = load<T, V>(x + pairs + u * V);
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const float2 cs = tab[u * V + e];
        const float p = to_f(a.v[e]), q = to_f(b.v[e]);
        a.v[e] = from_f<T>(p * cs.x - q * cs.y);
        b.v[e] = from_f<T>(p * cs.y + q * cs.x);
      }
      store<T, V>(y + u * V, a);
      store<T, V>(y + pairs + u * V, b);
    }
  }
}

template <class T, int V, bool INTER>
int launch(const RopeArgs& r, cudaStream_t s) {
  const int pairs = r.rotary / 2;
  // enough rows for a few packs per thread, a table that fits, and blocks for every SM
  const int64_t row_units = static_cast<int64_t>(r.heads) * r.head_dim / V;
  int64_t tok = std::max<int64_t>(1, 4 * kThreads / std::max<int64_t>(1, row_units));
  tok = std::min<int64_t>(tok, std::max(1, kTablePairs / std::max(1, pairs)));
  const int64_t blocks = (r.T + tok - 1) / tok;
  if (blocks > (1ll << 31) - 1) return QAT_ERR_SHAPE;
  rope_kernel<T, V, INTER><<<static_cast<unsigned>(blocks), kThreads, 0, s>>>(r, static_cast<int>(tok));
  count_launch();
  return cuda_status(cudaGetLastError());
}

template <class T>
int dispatch(const RopeArgs& r, cudaStream_t s) {
  constexpr int W = 16 / sizeof(T);
  const int half = r.rotary / 2;
  // 16-byte packs where every part of a head starts on a pack's boundary
  // (rows and heads do: head_dim and the row strides are multiples of 8 elements).
  // (65,536 tokens of 12 heads of 64 bf16: 37 us, 5.4 TB/s; more packs of a thread in
  // flight, 2 to 8, gave 38 to 53 us.)
  if (r.interleaved) {
    if (r.rotary % W == 0) return launch<T, W, true>(r, s);
    return launch<T, 2, true>(r, s);
  }
  if (half % W == 0) return launch<T, W, false>(r, s);
  return launch<T, 1, false>(r, s);
}

}  // namespace

int launch_rope(const RopeArgs& r, bool bf16, cudaStream_t stream) {
  if (r.rotary / 2 > kMaxPairs) return QAT_ERR_SHAPE;
  return bf16 ? dispatch<__nv_bfloat16>(r, stream) : dispatch<float>(r, stream);
}

}  // namespace qat
