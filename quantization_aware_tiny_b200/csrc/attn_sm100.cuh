// What the attention kernels share: arguments, sequences, masks, and the
// tcgen05 forms beside the GEMM's (operand A in tensor memory, TMEM stores).
#pragma once

#include "lm_ops.cuh"
#include "sm100_ptx.cuh"

namespace qat {

constexpr float kAttnLog2e = 1.4426950408889634f;

// 2^x to about 2^-22 relative (the special-function unit; 0 for x = -inf).
__device__ __forceinline__ float attn_exp2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float y;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
  return y;
}

__device__ __forceinline__ uint32_t pack2(float a, float b) {
  __nv_bfloat162 v = __floats2bfloat162_rn(a, b);  // .x = a (low half), .y = b
  return *reinterpret_cast<uint32_t*>(&v);
}

// 3-D tiled load {64 dims, 1 head, box rows} of a [token][head][dim] tensor.
__device__ __forceinline__ void tma_load_3d(const CUtensorMap* map, uint64_t* bar, void* dst,
                                            int32_t c0, int32_t c1, int32_t c2) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(smem_u32(dst)),
      "l"(map), "r"(smem_u32(bar)), "r"(c0), "r"(c1), "r"(c2)
      : "memory");
}

// The MMA forms below are executed by a whole warp, with `issue` set in one lane
// (the same one throughout): the code around them stays convergent, so the
// descriptors live in uniform registers.  Issued from a branch of one lane, with
// the descriptors built on the spot, an MMA took 90 to 180 cycles to issue,
// longer than the 64 it runs for, and the issue bound every attention kernel
// (dq, head size 64: 2,250 of 2,900 cycles a block).
__device__ __forceinline__ uint32_t elect_lane() {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}\n"
      : "=r"(r));
  return r;
}
// D[tmem] (+)= A[smem] * B[smem]^T
__device__ __forceinline__ void mma_ss(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc,
                                       uint32_t idesc, uint32_t accumulate, uint32_t issue) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "setp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate), "r"(issue));
}
// D[tmem] (+)= A[tmem] * B[smem]^T: A's rows are TMEM lanes, two bf16 per column.
__device__ __forceinline__ void mma_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc,
                                       uint32_t idesc, uint32_t accumulate, uint32_t issue) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "setp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}\n" ::"r"(d_tmem),
      "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate), "r"(issue));
}
// Arrive once on `bar` when every MMA issued so far by the issuing lane completes.
__device__ __forceinline__ void mma_commit(uint64_t* bar, uint32_t issue) {
  asm volatile(
      "{\n\t.reg .pred q;\n\t"
      "setp.ne.b32 q, %1, 0;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}\n" ::"r"(
          smem_u32(bar)),
      "r"(issue)
      : "memory");
}

// Each lane of the warp writes 16 consecutive columns of its own TMEM lane.
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]),
      "r"(r[15])
      : "memory");
}
// Each lane reads 16 consecutive columns of its own TMEM lane.
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_st_wait() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

// A warp's bounded wait: the same answer in every lane, so a wait that runs out
// never leaves part of a warp behind.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort_flag,
                                          int* err) {
  return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort_flag, err));
}

// Register split of a warpgroup (all its warps call it).
template <int N>
__device__ __forceinline__ void set_regs_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void set_regs_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}

// ---- work stealing.  A kernel is launched with one block per piece of work; a
// running block takes over pieces whose blocks have not started, so its set-up is
// paid once and the next piece's loads run below this one's last products.  The
// hardware hands pieces out in launch order, longest first here.
struct Work {
  int list, block;  // blockIdx.x, blockIdx.y of the piece
};
// Asks for a piece; the answer (16 bytes) completes on `bar`.  One thread.
__device__ __forceinline__ void work_ask(uint32_t answer, uint64_t* bar) {
  mbar_arrive_expect_tx(bar, 16);
  asm volatile(
      "clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(
          answer),
      "r"(smem_u32(bar))
      : "memory");
}
// Whether the answer is a piece, and which.
__device__ __forceinline__ bool work_read(uint32_t answer, Work& w) {
  uint32_t x = 0, y = 0, ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b128 r;\n\t"
      "ld.shared.b128 r, [%3];\n\t"
      "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, r;\n\t"
      "selp.u32 %2, 1, 0, p;\n\t"
      "@p clusterlaunchcontrol.query_cancel.get_first_ctaid.v4.b32.b128 {%0, %1, _, _}, r;\n\t}\n"
      : "+r"(x), "+r"(y), "=r"(ok)
      : "r"(answer)
      : "memory");
  w.list = static_cast<int>(x);
  w.block = static_cast<int>(y);
  return ok != 0;
}
// The answers' two slots: 32 bytes, and a full and an empty barrier each.
struct WorkQueue {
  uint32_t answers;
  uint64_t *full, *empty;  // [2]

  // Slot of the n-th answer is read by `readers` warps.
  __device__ void init(int readers) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], readers);
    }
  }
  // Asks for the (n + 1)-th piece (one thread, at the start of the n-th).
  __device__ bool ask(int n, volatile int* abort_flag, int* err) {
    if (n >= 2 && !mbar_wait(&empty[n & 1], ((n >> 1) & 1) ^ 1, abort_flag, err)) return false;
    work_ask(answers + (n & 1) * 16, &full[n & 1]);
    return true;
  }
  // The piece after the n-th; false: there is none (or a wait ran out).  A whole warp.
  __device__ bool next(int n, Work& w, int lane, volatile int* abort_flag, int* err) {
    if (!warp_wait(&full[n & 1], (n >> 1) & 1, abort_flag, err)) return false;
    const bool ok = work_read(answers + (n & 1) * 16, w);
    fence_proxy_async_smem();  // read before the slot is written again
    __syncwarp();
    if (lane == 0) mbar_arrive(&empty[n & 1]);
    return ok;
  }
};

// ---- sequences
struct Seq {
  int64_t q0, k0;  // first query / key row
  int nq, nk;      // rows
};

// Sequence b: [cu[b], cu[b+1]) of the packed rows, or rows of equal length.
// Offsets outside the tensor are cut to it, and lengths to max_q / max_k, so no
// table makes a kernel leave the tensors or read what no block computed.
__device__ __forceinline__ Seq seq_of(const AttnArgs& p, int b) {
  Seq s;
  if (p.cu_q) {
    const int64_t a = min(max(static_cast<int64_t>(p.cu_q[b]), int64_t{0}), p.Tq);
    const int64_t e = min(max(static_cast<int64_t>(p.cu_q[b + 1]), a), p.Tq);
    s.q0 = a;
    s.nq = min(static_cast<int>(e - a), p.max_q);
  } else {
    s.q0 = static_cast<int64_t>(b) * p.max_q;
    s.nq = p.max_q;
  }
  if (p.cu_k) {
    const int64_t a = min(max(static_cast<int64_t>(p.cu_k[b]), int64_t{0}), p.Tk);
    const int64_t e = min(max(static_cast<int64_t>(p.cu_k[b + 1]), a), p.Tk);
    s.k0 = a;
    s.nk = min(static_cast<int>(e - a), p.max_k);
  } else {
    s.k0 = static_cast<int64_t>(b) * p.max_k;
    s.nk = p.max_k;
  }
  return s;
}

// Keys [lo, hi) that query i of a sequence sees: all of them, or with `causal`
// those up to its own place (the last query is at the last key), at most the
// last `window` of these.
__device__ __forceinline__ void keys_of(const AttnArgs& p, const Seq& s, int i, int& lo, int& hi) {
  lo = 0;
  hi = s.nk;
  if (p.causal) {
    const int64_t last = static_cast<int64_t>(i) + s.nk - s.nq;  // negative: no key at all
    hi = static_cast<int>(min(static_cast<int64_t>(hi), max(last + 1, int64_t{0})));
    if (p.window > 0)
      lo = static_cast<int>(min(max(last - p.window + 1, int64_t{0}), static_cast<int64_t>(hi)));
  }
}

// Queries [lo, hi) of a sequence that see key j (the same rule, read the other way).
__device__ __forceinline__ void queries_of(const AttnArgs& p, const Seq& s, int j, int& lo, int& hi) {
  lo = 0;
  hi = s.nq;
  if (p.causal) {
    const int64_t same = static_cast<int64_t>(j) + s.nq - s.nk;  // the query at this key's place
    lo = static_cast<int>(min(max(same, int64_t{0}), static_cast<int64_t>(s.nq)));
    if (p.window > 0)
      hi = static_cast<int>(min(max(same + p.window, int64_t{0}), static_cast<int64_t>(s.nq)));
  }
  lo = min(lo, hi);
}

// Key blocks [b0, b1) that ROWS queries from i0 on see; none: b1 = b0.
template <int ROWS, int KEYS>
__device__ __forceinline__ void key_blocks(const AttnArgs& p, const Seq& s, int i0, int& b0, int& b1) {
  b0 = b1 = 0;
  if (i0 >= s.nq) return;
  int lo, hi, lo2, hi2;
  keys_of(p, s, i0, lo, hi);
  keys_of(p, s, min(i0 + ROWS, s.nq) - 1, lo2, hi2);
  // the last row sees furthest; where the first sees nothing, a later one starts at key 0
  b0 = hi > lo ? lo / KEYS : 0;
  b1 = hi2 > lo2 ? (hi2 + KEYS - 1) / KEYS : b0;
}

// Scores of 32 neighbouring places of a row, of which [a, a + n) are seen (n = 0:
// none): the others become -inf.  Rows of a warp lie next to one another, so most
// such pieces of a masked block are seen by all of them and left alone.
__device__ __forceinline__ void mask_scores(uint32_t (&s)[32], int a, int n) {
  const int lo = min(max(a, 0), 32), hi = min(max(a + n, 0), 32);
  const uint32_t seen = hi > lo ? (0xffffffffu >> (32 - hi + lo)) << lo : 0u;  // bit k: place k
  if (__any_sync(0xffffffffu, ~seen)) {
#pragma unroll
    for (int k = 0; k < 32; ++k) s[k] = (seen & (1u << k)) ? s[k] : 0xff800000u;
  }
}

// Bytes of a tile of `rows` rows and NC 64-dim chunks; chunk c starts at c * rows * 128.
__host__ __device__ constexpr int tile_bytes(int rows, int nc) { return rows * 128 * nc; }

// Clears rows [from, rows) of a staged tile (every 128-byte row lies in one
// swizzle line, so whole rows need no unswizzling); all lanes of one warp.
// Rows behind a sequence's end hold other sequences' values, or anything, and
// a zero probability does not cancel a NaN there.
template <int NC>
__device__ __forceinline__ void clear_rows(uint8_t* tile, int rows, int from, int lane) {
  const uint32_t base = smem_u32(tile);
  const int n = (rows - from) * 8;
#pragma unroll
  for (int c = 0; c < NC; ++c)
    for (int i = lane; i < n; i += 32)
      st_shared_v4(base + c * rows * 128 + from * 128 + i * 16, 0, 0, 0, 0);
  fence_proxy_async_smem();
  __syncwarp();
}

// bf16(v * f) of N (16 or 32) accumulator columns of the warp's 32 rows (a row per
// lane) to global rows ld apart, columns [0, cols) of the piece and rows [0, live):
// through 64 N bytes of shared memory, so that a store instruction covers whole
// sectors of several rows.  (Each lane storing its own row in 16-byte pieces took
// 3,700 cycles for dK and dV of a 128-key tile.)
template <int N>
__device__ __forceinline__ void store_piece(__nv_bfloat16* out, int64_t ld, const uint32_t (&v)[N],
                                            float f, int cols, int live, uint32_t stage, int lane) {
  constexpr int G = N / 8;  // 16-byte groups of a row
  const uint32_t mine = stage + lane * 2 * N;
  const int sw = (lane * G >> 3) & (G - 1);  // keeps 8 neighbouring lanes off one another's banks
#pragma unroll
  for (int g = 0; g < G; ++g) {
    uint32_t o[4];
#pragma unroll
    for (int k = 0; k < 4; ++k)
      o[k] = pack2(__uint_as_float(v[g * 8 + 2 * k]) * f, __uint_as_float(v[g * 8 + 2 * k + 1]) * f);
    st_shared_v4(mine + ((g ^ sw) << 4), o[0], o[1], o[2], o[3]);
  }
  __syncwarp();
  const int g = lane & (G - 1);
#pragma unroll
  for (int n = 0; n < G; ++n) {
    const int r = n * (32 / G) + lane / G;
    const uint4 x = ld_shared_v4(stage + r * 2 * N + ((g ^ ((r * G >> 3) & (G - 1))) << 4));
    if (r < live && g * 8 < cols) *reinterpret_cast<uint4*>(out + r * ld + g * 8) = x;
  }
  __syncwarp();
}

// Descriptors of staged tiles of ROWS rows.  K-major: the contraction runs over a
// row's dims, k-step kk (16 dims) adds kmajor_step(kk).  By rows: it runs over the
// tile's rows, k-step kk (rows 16 kk .. 16 kk + 15) adds rows_step(kk).  (The address
// sits in the descriptor's low bits in units of 16 bytes.)
template <int ROWS>
__device__ __forceinline__ uint64_t kmajor_desc(const uint8_t* tile) {
  return sw128_desc(smem_u32(tile), 16, 1024);
}
template <int ROWS>
__device__ __forceinline__ constexpr uint32_t kmajor_step(int kk) {
  return ((kk >> 2) * ROWS * 128 + (kk & 3) * 32) >> 4;
}
template <int ROWS>
__device__ __forceinline__ uint64_t rows_desc(const uint8_t* tile) {
  return sw128_desc(smem_u32(tile), ROWS * 128, 1024);
}
__device__ __forceinline__ constexpr uint32_t rows_step(int kk) { return (kk * 2048) >> 4; }

// D = A B^T over the 16-dim steps of the head (at most 4 NC), both operands K-major tiles.
template <int NC, int ROWS>
__device__ __forceinline__ void product(uint32_t d_tmem, uint64_t a, uint64_t b, uint32_t idesc,
                                        int ks, uint32_t issue) {
#pragma unroll
  for (int kk = 0; kk < 4 * NC; ++kk)
    if (kk < ks) mma_ss(d_tmem, a + kmajor_step<ROWS>(kk), b + kmajor_step<ROWS>(kk), idesc, kk > 0, issue);
}

}  // namespace qat
