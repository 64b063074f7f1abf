// Attention backward on tcgen05.  With P recomputed from Q, K and the forward's
// lse, and delta = rowsum(dO * O):
//   dP = dO V^T,  dS = P * (dP - delta),
//   dV = P^T dO,  dK = scale dS^T Q,  dQ = scale dS K.
//
// Two kernels, each with its sums in tensor memory from first to last:
//   attn_dq_kernel   a block owns 128 queries of a head and walks the keys
//   attn_dkv_kernel  a block owns 128 keys of a key head and walks the queries of
//                    all heads of its group (their gradients meet in the sum)
// S and dP are thus formed twice, 7 products instead of 5; in return no partial
// sum ever leaves a block: no fp32 copy of dQ in memory, no atomics, and the same
// inputs give the same bits.
//
// Bound by the chain of hand-overs from a block's S to its dS (about 2,500 cycles a
// 128 x 128 block in dq and 3,300 in dkv at head size 64, where the products take
// 768 and 1,024 and the exponentials 1,024): tensor memory loads and stores, and
// barriers, each some 150 to 400 cycles with 16 warps at them.  4 sequences of 4,096
// tokens, 8 heads of 64 over 4: dq 154 us and dkv 190 us (344 us together, 500 TFLOP/s
// of the 5 products that have to be); 8,192 tokens of 128, 8 over 2: 182 and 512 us,
// 695 together (a key tile's block walks all 4 heads of its group).  Exponentials
// partly on the multiply-add units, two issuing warps, and P and dS handed over together
// gained nothing or lost.
//
// P and dS are rounded to bf16 for the second products, as P is in the forward: each
// off by at most 2^-8 of itself, which leaves dQ, dK and dV 2.4e-3 off in the 2-norm
// where their own rounding alone gives 1.7e-3; second halves would be three products
// more.  delta, lse and all sums are fp32.  P and dS go back to tensor memory and are
// read from there as operand A.  Both kernels form P as soon as S is there and dS once
// dP is, so that the products of the next block (and the sums of this one) run below
// the exponentials; four math warpgroups share a block, 32 of its 128 columns each.
#include <algorithm>
#include <atomic>

#include "attn_maps.cuh"
#include "attn_sm100.cuh"

namespace qat {

namespace {

constexpr int BT = 128;  // rows of the stationary tile and of a streamed block

template <int NC>
struct Cfg {
  // 16 math warps, four to a scheduler: with 8 (64 columns per thread) the waits for
  // tensor memory and for the exponentials lay bare, 3,700 cycles a block instead of
  // about 2,000 (dq, head size 64)
  static constexpr int GROUPS = 4;                  // math warpgroups
  static constexpr int MC = BT / GROUPS;            // columns of a block per thread
  static constexpr int THREADS = 128 * (1 + GROUPS);
  // registers per thread: 96 at launch (65,536 / 640), 56 + 4 * 104 <= 5 * 96 after the split
  // (dkv keeps 28 to 40 bytes a thread in local memory, dq none)
  static constexpr int REGS_ISSUE = 56, REGS_MATH = 104;
  static constexpr int TILE = tile_bytes(BT, NC);
  static constexpr int ST = NC == 1 ? 4 : 2;        // stages of either ring
  // dkv: lse and delta, per warp; dq: delta of the rows, and its parts per warpgroup
  static constexpr int ROWS_BYTES = 4 * GROUPS * 2 * MC * 4;
  static_assert((1 + GROUPS) * BT * 4 <= ROWS_BYTES, "dq's rows");
  static constexpr int OUT_BYTES = 4 * GROUPS * 1024;  // the gradient rows' way out, per warp
  static constexpr int SMEM = (2 + 2 * ST) * TILE + ROWS_BYTES + OUT_BYTES + 1024 + 512;
  static constexpr int COLS = 64 * NC;              // tensor-memory columns of an accumulator
};

// The rings and barriers of both kernels: two stationary tiles, two rings.
template <int NC>
struct Smem {
  using C = Cfg<NC>;
  uint8_t *fix_a, *fix_b, *ring_a, *ring_b, *out;
  float* rows;
  uint64_t *fix_full, *fix_empty, *a_full, *a_empty, *b_full, *b_empty;
  uint64_t *s_full, *dp_full, *s_read, *p_full, *p_free, *ds_full, *acc_full, *delta_full, *mma_done;
  uint32_t* tmem_slot;
  volatile int* abort_flag;

  __device__ explicit Smem(uint8_t* raw) {
    fix_a = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~static_cast<uintptr_t>(1023));
    fix_b = fix_a + C::TILE;
    ring_a = fix_b + C::TILE;
    ring_b = ring_a + C::ST * C::TILE;
    rows = reinterpret_cast<float*>(ring_b + C::ST * C::TILE);
    out = reinterpret_cast<uint8_t*>(rows) + C::ROWS_BYTES;
    fix_full = reinterpret_cast<uint64_t*>(out + C::OUT_BYTES);
    fix_empty = fix_full + 1;
    a_full = fix_empty + 1;
    a_empty = a_full + C::ST;
    b_full = a_empty + C::ST;
    b_empty = b_full + C::ST;
    s_full = b_empty + C::ST;
    dp_full = s_full + 1;
    s_read = dp_full + 1;
    p_full = s_read + 1;
    p_free = p_full + 1;
    ds_full = p_free + 1;
    acc_full = ds_full + 1;
    delta_full = acc_full + 1;
    mma_done = delta_full + 1;
    tmem_slot = reinterpret_cast<uint32_t*>(mma_done + 5);
    abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    static_assert((2 + 4 * C::ST + 13) * 8 + 8 <= 512 - 32, "barrier block overflow");
  }
  __device__ WorkQueue queue() const {
    return WorkQueue{smem_u32(fix_full) + 512 - 32, mma_done + 1, mma_done + 3};
  }
  __device__ void init() {
    queue().init(2 + 4 * C::GROUPS);  // producer, MMA, math warps
    mbar_init(fix_empty, 1);
    mbar_init(fix_full, 1);
    for (int i = 0; i < C::ST; ++i) {
      mbar_init(&a_full[i], 1);
      mbar_init(&a_empty[i], 1);
      mbar_init(&b_full[i], 1);
      mbar_init(&b_empty[i], 1);
    }
    mbar_init(s_full, 1);
    mbar_init(dp_full, 1);
    mbar_init(s_read, 4 * C::GROUPS);  // the math warps
    mbar_init(p_full, 4 * C::GROUPS);
    mbar_init(p_free, 1);
    mbar_init(ds_full, 4 * C::GROUPS);
    mbar_init(acc_full, 1);
    mbar_init(delta_full, 4 * C::GROUPS);
    mbar_init(mma_done, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
};

// One staged tile of `head`, rows from `row` on.
template <int NC>
__device__ __forceinline__ void load_tile(const CUtensorMap* map, uint64_t* bar, uint8_t* dst, int head, int row) {
#pragma unroll
  for (int c = 0; c < NC; ++c) tma_load_3d(map, bar, dst + c * BT * 128, c * 64, head, row);
}

// The warp's 32 rows of an accumulator (at t) times f, as bf16, to `out` (its first
// row and the head's first column): the 16-column pieces from, from + step, ...
__device__ __forceinline__ void store_rows(__nv_bfloat16* out, int64_t ld, uint32_t t, int hd, float f,
                                           bool any, int live, int from, int step, uint8_t* stage, int lane) {
  for (int c = from; c < (hd + 15) / 16; c += step) {
    uint32_t o[16] = {};
    if (any) {
      tmem_ld16(t + c * 16, o);
      tmem_ld_wait();
    }
    store_piece(out + c * 16, ld, o, f, hd - c * 16, live, smem_u32(stage), lane);
  }
}

// Producer of both kernels (lane 0 of a warp that walks together): per piece of
// work the fixed tiles, then the rings; `fixed` and `ring` issue the loads.
template <int NC, class PieceT, class Fixed, class Ring>
__device__ __forceinline__ void produce(const Smem<NC>& m, const AttnArgs& p, Work work, int lane, Fixed fixed,
                                        Ring ring) {
  using C = Cfg<NC>;
  constexpr int ST = C::ST;
  WorkQueue queue = m.queue();
  int na = 0, nb = 0, loads = 0, asked = 0;
  bool ok = true;
  for (int pieces = 0;; ++pieces) {
    if (lane == 0) {
      const PieceT x(p, work);
      if (x.steps > 0) {
        ok = loads == 0 || mbar_wait(m.fix_empty, (loads - 1) & 1, m.abort_flag, p.err);
        if (ok) {
          mbar_arrive_expect_tx(m.fix_full, 2 * C::TILE);
          fixed(x);
          ++loads;
        }
        for (int n = 0; ok && n < x.steps; ++n) {
          const int st = na % ST;
          const uint32_t free = ((na / ST) & 1) ^ 1;
          ok = mbar_wait(&m.a_empty[st], free, m.abort_flag, p.err);
          if (!ok) break;
          mbar_arrive_expect_tx(&m.a_full[st], C::TILE);
          ring(x, n, false, &m.a_full[st], m.ring_a + st * C::TILE);
          ++na;
          ok = mbar_wait(&m.b_empty[st], free, m.abort_flag, p.err);
          if (!ok) break;
          mbar_arrive_expect_tx(&m.b_full[st], C::TILE);
          ring(x, n, true, &m.b_full[st], m.ring_b + st * C::TILE);
          ++nb;
        }
      }
      // (only now: a block that asked early would hold a piece that an idle one could start)
      ok = ok && queue.ask(pieces, m.abort_flag, p.err);
      asked += ok;
    }
    __syncwarp();
    if (!__all_sync(0xffffffffu, ok) || !queue.next(pieces, work, lane, m.abort_flag, p.err)) break;
  }
  if (lane == 0) {  // every copy has landed before the block may exit (at once, unless a wait ran out)
    if (loads > 0) mbar_drain(m.fix_full, (loads - 1) & 1);
    for (int n = max(0, na - ST); n < na; ++n) mbar_drain(&m.a_full[n % ST], (n / ST) & 1);
    for (int n = max(0, nb - ST); n < nb; ++n) mbar_drain(&m.b_full[n % ST], (n / ST) & 1);
    if (asked > 0) mbar_drain(&queue.full[(asked - 1) & 1], ((asked - 1) >> 1) & 1);
  }
}

// ------------------------------------------------------------------------ dQ

// delta = rowsum(dO * O) comes from the O that was rounded to bf16, and dP - delta
// takes two near numbers apart where a row's softmax rests on few keys: with two keys
// dQ and dK were 0.004 to 0.02 off (and anything where one of the two has nearly all the
// weight), where their roundings leave 0.0024.  By its definition delta is sum(P * dP):
// sum(P * (dP - delta)) is what it lacks.  A row whose keys lie in one block gets it
// before its dS is formed (all rows of few keys, but for small windows: those tiles are
// walked twice, the first time for the sum alone); the others take delta as it came,
// which costs nothing at scores of unit spread (0.0024), up to 0.0036 at four times that
// and 0.0065 where every row is nearly one-hot (simulated, 300 to 1,000 keys).  dK always
// gets the mended delta: the sum goes along with dS.  The sums take 3 % of this kernel
// (150 -> 154 us at 4 x 4,096 tokens of 8 heads of 64); tiles walked twice are a kernel
// of their own, since the branch around the products that a common one needs took 9 %
// more.  At windows past 16 keys dQ is 0.0025 off as it is.
constexpr int kFewKeys = 16;

// A CTA owns 128 queries of a head.  Tensor memory: S, dP (128 columns each), dS
// (bf16, 64), dQ.  Issue order: S(n + 1) once S(n) is read; then, once dS(n) is
// written, dQ += dS(n) K(n) and dP(n + 1) -- whose arrival thus also says that
// dS(n) has been read.
template <bool TWICE>
struct DqPiece {
  Seq sq;
  int head, kv_head, i0, j0, blocks;  // queries from i0 on, key blocks j0 .. j0 + blocks - 1
  int steps;                          // blocks walked, all times taken together
  bool live;

  __device__ DqPiece(const AttnArgs& p, const Work& w) {
    head = w.list % p.heads;
    kv_head = head / p.group;
    sq = seq_of(p, w.list / p.heads);
    i0 = (static_cast<int>(gridDim.y) - 1 - w.block) * BT;  // longest rows first
    live = i0 < sq.nq;
    int j1;
    key_blocks<BT, BT>(p, sq, i0, j0, j1);
    blocks = live ? j1 - j0 : 0;
    steps = TWICE && blocks > 1 ? 2 * blocks : blocks;
  }
  __device__ int first() const { return TWICE ? steps - blocks : 0; }  // steps taken for delta alone
  __device__ int key0(int n) const { return (j0 + (n < first() ? n : n - first())) * BT; }
};

template <int NC, bool TWICE>
__global__ void __launch_bounds__(Cfg<NC>::THREADS, 1)
    attn_dq_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmdO,
                   const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                   const AttnArgs p) {
  using C = Cfg<NC>;
  using PieceT = DqPiece<TWICE>;
  constexpr int ST = C::ST;
  constexpr uint32_t T_DP = BT, T_DS = 2 * BT, T_DQ = 2 * BT + BT / 2;
  static_assert(T_DQ + C::COLS <= 512, "tensor memory");
  extern __shared__ uint8_t smem_raw[];
  const Smem<NC> m(smem_raw);  // fixed: Q, dO; rings: K, V

  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  Work work{static_cast<int>(blockIdx.x), static_cast<int>(blockIdx.y)};
  WorkQueue queue = m.queue();

  if (threadIdx.x == 0) {
    Smem<NC>(smem_raw).init();
    tma_prefetch_desc(&tmQ);
    tma_prefetch_desc(&tmdO);
    tma_prefetch_desc(&tmK);
    tma_prefetch_desc(&tmV);
  }
  if (warp == 1) {
    tmem_alloc(m.tmem_slot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *m.tmem_slot;

  if (warp < 4) {
    set_regs_dec<C::REGS_ISSUE>();
    if (warp == 0) {
      produce<NC, PieceT>(
          m, p, work, lane,
          [&](const PieceT& x) {
            const int row = static_cast<int>(x.sq.q0) + x.i0;
            load_tile<NC>(&tmQ, m.fix_full, m.fix_a, x.head, row);
            load_tile<NC>(&tmdO, m.fix_full, m.fix_b, x.head, row);
          },
          [&](const PieceT& x, int n, bool second, uint64_t* bar, uint8_t* dst) {
            load_tile<NC>(second ? &tmV : &tmK, bar, dst, x.kv_head, static_cast<int>(x.sq.k0) + x.key0(n));
          });
    } else if (warp == 1) {
      // ------------------------------------------------ MMA issuer
      const int ks = (p.hd + 15) / 16;
      const uint32_t id_s = idesc_bf16(BT, BT, false, false);
      const uint32_t id_q = idesc_bf16(BT, ks * 16, false, true);
      const uint32_t issue = elect_lane();
      const uint64_t fix_a = kmajor_desc<BT>(m.fix_a), fix_b = kmajor_desc<BT>(m.fix_b);
      const uint64_t ring_a = kmajor_desc<BT>(m.ring_a), ring_b = kmajor_desc<BT>(m.ring_b);
      const uint64_t rows_a = rows_desc<BT>(m.ring_a);
      constexpr uint32_t STAGE = C::TILE >> 4;
      bool ok = true;
      int base = 0, loads = 0;  // blocks and fixed tiles of the pieces before
      for (int pieces = 0;; ++pieces) {
        const PieceT x(p, work);
        // X = fixed streamed^T of block n
        auto scores = [&](int n, uint64_t* full, uint8_t* ring, uint64_t b, uint64_t fix, uint32_t t, uint64_t* done) {
          const int g = base + n, st = g % ST;
          ok = ok && warp_wait(&full[st], (g / ST) & 1, m.abort_flag, p.err);
          if (!ok) return;
          const int rows = x.sq.nk - x.key0(n);
          if (rows < BT) clear_rows<NC>(ring + st * C::TILE, BT, rows, lane);
          tc_fence_after();
          product<NC, BT>(tmem + t, fix, b + st * STAGE, id_s, ks, issue);
          mma_commit(done, issue);
        };
        if (x.steps > 0) {
          ok = warp_wait(m.fix_full, loads & 1, m.abort_flag, p.err);
          ++loads;
          scores(0, m.a_full, m.ring_a, ring_a, fix_a, 0, m.s_full);
          scores(0, m.b_full, m.ring_b, ring_b, fix_b, T_DP, m.dp_full);
          if (ok) mma_commit(&m.b_empty[base % ST], issue);
          if (x.steps == 1) mma_commit(m.fix_empty, issue);  // Q and dO: the next piece's may come
          for (int n = 0; ok && n < x.steps; ++n) {
            const int g = base + n;
            const bool more = n + 1 < x.steps;
            if (more) {
              ok = warp_wait(m.s_read, g & 1, m.abort_flag, p.err);
              scores(n + 1, m.a_full, m.ring_a, ring_a, fix_a, 0, m.s_full);
            }
            ok = ok && warp_wait(m.ds_full, g & 1, m.abort_flag, p.err);
            if (!ok) break;
            tc_fence_after();
            const uint64_t k = rows_a + g % ST * STAGE;
            if (!TWICE || n >= x.first()) {
#pragma unroll
              for (int kk = 0; kk < BT / 16; ++kk)
                mma_ts(tmem + T_DQ, tmem + T_DS + kk * 8, k + rows_step(kk), id_q, (kk > 0) | (n > x.first()), issue);
            }
            mma_commit(&m.a_empty[g % ST], issue);
            if (more) {
              scores(n + 1, m.b_full, m.ring_b, ring_b, fix_b, T_DP, m.dp_full);
              if (ok) mma_commit(&m.b_empty[(g + 1) % ST], issue);
              if (n + 2 == x.steps) mma_commit(m.fix_empty, issue);
            } else {
              mma_commit(m.acc_full, issue);
            }
          }
          base += x.steps;
        }
        if (!ok || !queue.next(pieces, work, lane, m.abort_flag, p.err)) break;
      }
      mma_commit(m.mma_done, issue);
      warp_wait(m.mma_done, 0, m.abort_flag, p.err);  // before tensor memory is freed
    }
  } else {
    set_regs_inc<C::REGS_MATH>();
    // ------------------------------------------------ dS: a thread holds 32 keys of a query row
    const int w = (warp - 4) >> 2;
    const int quarter = warp & 3;  // tensor-memory lanes this warp may access
    const uint32_t t = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
    const float c2 = p.scale * kAttnLog2e;
    bool ok = true;
    int base = 0, accs = 0;  // blocks of the pieces before, and pieces that had any
    for (int pieces = 0;; ++pieces) {
      const PieceT x(p, work);
      const int i = x.i0 + quarter * 32 + lane;
      const int64_t at = x.sq.q0 + i;
      int lo, hi;
      keys_of(p, x.sq, i, lo, hi);
      int full0, full1, unused;  // keys that every row of the tile sees
      keys_of(p, x.sq, x.i0, unused, full1);
      keys_of(p, x.sq, x.i0 + BT - 1, full0, unused);
      float lse2 = 0.0f;
      if (i < x.sq.nq) {
        const float l = p.lse[x.head * p.Tq + at];
        lse2 = l == -INFINITY ? 0.0f : l * kAttnLog2e;  // (no key: every place is masked below)
      }
      // delta = rowsum(dO * O): a warp takes 8 of the tile's rows, half a warp a row, all
      // loads first; shared memory (and p_full, otherwise unused here) hands them round.
      // (A thread per row, 16 bytes at a time, took 20,000 cycles.)
      {
        const int r0 = (warp - 4) * 8 + (lane >> 4), e = (lane & 15) * 8;
        uint4 o[4], d[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          o[k] = d[k] = make_uint4(0, 0, 0, 0);
          const int64_t row = x.sq.q0 + x.i0 + r0 + 2 * k;
          if (x.i0 + r0 + 2 * k < x.sq.nq && e < p.hd) {
            o[k] = __ldg(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.O) + row * p.ldo + x.head * p.hd + e));
            d[k] = __ldg(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.dO) + row * p.lddo + x.head * p.hd + e));
          }
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const __nv_bfloat162* a = reinterpret_cast<const __nv_bfloat162*>(&o[k]);
          const __nv_bfloat162* b = reinterpret_cast<const __nv_bfloat162*>(&d[k]);
          float sum = 0.0f;
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const float2 u = __bfloat1622float2(a[c]), v = __bfloat1622float2(b[c]);
            sum = fmaf(u.x, v.x, fmaf(u.y, v.y, sum));
          }
#pragma unroll
          for (int b = 8; b > 0; b >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, b);
          const int r = r0 + 2 * k;
          if ((lane & 15) == 0) {
            m.rows[r] = sum;
            // for the other kernel (rows that see no key; the others' is mended first)
            if (x.steps == 0 && x.i0 + r < x.sq.nq) p.delta[x.head * p.Tq + x.sq.q0 + x.i0 + r] = sum;
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(m.p_full);
      }
      ok = warp_wait(m.p_full, pieces & 1, m.abort_flag, p.err);
      const float delta = m.rows[quarter * 32 + lane];
      const float2 cc = make_float2(c2, c2), nl = make_float2(-lse2, -lse2);
      float2 nd = make_float2(-delta, -delta), lacks = make_float2(0.0f, 0.0f);
      // -delta with what it lacks: the warpgroups' shares of a row meet in shared memory
      // (read before any warp leaves this piece's p_full behind again)
      auto settle = [&]() {
        float* part = m.rows + BT + quarter * 32 + lane;
        part[w * BT] = lacks.x + lacks.y;
        __syncwarp();
        if (lane == 0) mbar_arrive(m.delta_full);
        ok = warp_wait(m.delta_full, accs & 1, m.abort_flag, p.err);
        const float d = delta + ((part[0] + part[BT]) + (part[2 * BT] + part[3 * BT]));
        if (ok && w == 0 && i < x.sq.nq) p.delta[x.head * p.Tq + at] = d;  // for the other kernel
        nd = make_float2(-d, -d);
      };
      const bool open = x.steps > 1 && x.first() == 0;  // dS is formed before delta is mended
      for (int n = 0; ok && n < x.steps; ++n) {
        if (!warp_wait(m.s_full, (base + n) & 1, m.abort_flag, p.err)) { ok = false; break; }
        tc_fence_after();
        uint32_t s[32];
        tmem_ld32(t + w * 32, s);
        tmem_ld_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(m.s_read);
        const int key0 = x.key0(n);
        // (a query of a single key has no gradient: dS is 0, where dP and delta differ by roundings)
        if (key0 < full0 || key0 + BT > full1) mask_scores(s, lo - key0 - w * 32, hi - lo == 1 ? 0 : hi - lo);
        float2 pr[16];
#pragma unroll
        for (int k = 0; k < 16; ++k) {
          const float2 e = fma2(make_float2(__uint_as_float(s[2 * k]), __uint_as_float(s[2 * k + 1])), cc, nl);
          pr[k] = make_float2(attn_exp2(e.x), attn_exp2(e.y));
        }
        if (!warp_wait(m.dp_full, (base + n) & 1, m.abort_flag, p.err)) { ok = false; break; }
        tc_fence_after();
        tmem_ld32(t + T_DP + w * 32, s);
        tmem_ld_wait();
        if (x.steps == 1 || (TWICE && n < x.first())) {
#pragma unroll
          for (int k = 0; k < 16; ++k)
            lacks = fma2(pr[k], add2(make_float2(__uint_as_float(s[2 * k]), __uint_as_float(s[2 * k + 1])), nd), lacks);
          if (!TWICE || x.steps == 1 || n + 1 == x.first()) {
            settle();
            if (!ok) break;
          }
        }
        if (!TWICE || n >= x.first()) {
          uint32_t pk[16];
#pragma unroll
          for (int k = 0; k < 16; ++k) {
            pr[k] = mul2(pr[k], add2(make_float2(__uint_as_float(s[2 * k]), __uint_as_float(s[2 * k + 1])), nd));
            pk[k] = pack2(pr[k].x, pr[k].y);
          }
          tmem_st16(t + T_DS + w * 16, pk);
          tmem_st_wait();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(m.ds_full);
        if (open) {  // (below the next block's products)
#pragma unroll
          for (int k = 0; k < 16; k += 4)
            lacks = add2(lacks, add2(add2(pr[k], pr[k + 1]), add2(pr[k + 2], pr[k + 3])));
        }
      }
      if (ok && open) settle();
      if (ok && x.steps > 0) ok = warp_wait(m.acc_full, accs & 1, m.abort_flag, p.err);
      accs += x.steps > 0;
      base += x.steps;
      tc_fence_after();
      if (ok) {  // the warpgroups store a quarter of the row each
        const int r0 = x.i0 + quarter * 32;
        store_rows(static_cast<__nv_bfloat16*>(p.dQ) + (x.sq.q0 + r0) * p.lddq + x.head * p.hd, p.lddq, t + T_DQ, p.hd,
                   p.scale, x.steps > 0, x.sq.nq - r0, w, C::GROUPS, m.out + (warp - 4) * 1024, lane);
      }
      tc_fence_before();
      if (!ok || !queue.next(pieces, work, lane, m.abort_flag, p.err)) break;
    }
  }
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// -------------------------------------------------------------------- dK, dV

// A CTA owns 128 keys of a key head.  Tensor memory: S^T and dP^T (128 columns
// each; dS^T replaces dP^T as bf16, each warpgroup within the columns it reads),
// P^T, dV, dK.  Issue order: S^T(n + 1) once S^T(n) is read; dV += P^T(n) dO(n)
// once P(n) is written; dK += dS^T(n) Q(n) and dP^T(n + 1) once dS(n) is.
// Heads of more than 96 dims leave no columns for P^T: it then replaces S^T, and
// S^T(n + 1) waits for dV's product.
struct DkvPiece {
  Seq sq;
  int kv_head, key0;       // keys from key0 on
  int full0, full1;        // queries that see every key of the tile
  int j0, nb, steps;       // the steps: query blocks j0 .. j0 + nb - 1 of each head of the group
  bool live;

  __device__ DkvPiece(const AttnArgs& p, const Work& w) {
    const int kv_heads = p.heads / p.group;
    kv_head = w.list % kv_heads;
    sq = seq_of(p, w.list / kv_heads);
    key0 = w.block * BT;  // early keys are seen by most queries: first
    live = key0 < sq.nk;
    int qa, qb;  // queries that see some key of it
    queries_of(p, sq, key0, qa, full1);
    queries_of(p, sq, min(key0 + BT, sq.nk) - 1, full0, qb);
    j0 = qa / BT;
    nb = live && qb > qa ? (qb + BT - 1) / BT - j0 : 0;
    steps = nb * p.group;
  }
};

// Head (within the group) and block of a step, counted along: divided out of the
// step's number by the one issuing warp they cost 800 of a step's 3,500 cycles.
struct Step {
  int head = 0, block = 0;
  __device__ void advance(int nb) {
    if (++block == nb) {
      block = 0;
      ++head;
    }
  }
};

template <int NC>
__global__ void __launch_bounds__(Cfg<NC>::THREADS, 1)
    attn_dkv_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmdO,
                    const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                    const AttnArgs p) {
  using C = Cfg<NC>;
  constexpr int ST = C::ST;
  constexpr uint32_t T_DP = BT;
  const int ks = (p.hd + 15) / 16;
  const bool apart = ks <= 6;  // 2 * 128 + 64 + 2 * 96 = 512 columns
  const uint32_t t_p = apart ? 2 * BT : 0, p_step = apart ? 16 : C::MC;  // a warpgroup's P^T columns
  const uint32_t t_dv = apart ? 2 * BT + BT / 2 : 2 * BT, t_dk = t_dv + (apart ? ks * 16 : C::COLS);
  extern __shared__ uint8_t smem_raw[];
  const Smem<NC> m(smem_raw);  // fixed: K, V; rings: Q, dO

  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  Work work{static_cast<int>(blockIdx.x), static_cast<int>(blockIdx.y)};
  WorkQueue queue = m.queue();

  if (threadIdx.x == 0) {
    Smem<NC>(smem_raw).init();
    tma_prefetch_desc(&tmQ);
    tma_prefetch_desc(&tmdO);
    tma_prefetch_desc(&tmK);
    tma_prefetch_desc(&tmV);
  }
  if (warp == 1) {
    tmem_alloc(m.tmem_slot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *m.tmem_slot;

  if (warp < 4) {
    set_regs_dec<C::REGS_ISSUE>();
    if (warp == 0) {
      Step at;
      produce<NC, DkvPiece>(
          m, p, work, lane,
          [&](const DkvPiece& x) {
            const int row = static_cast<int>(x.sq.k0) + x.key0;
            load_tile<NC>(&tmK, m.fix_full, m.fix_a, x.kv_head, row);
            load_tile<NC>(&tmV, m.fix_full, m.fix_b, x.kv_head, row);
          },
          [&](const DkvPiece& x, int n, bool second, uint64_t* bar, uint8_t* dst) {
            if (n == 0) at = Step();
            load_tile<NC>(second ? &tmdO : &tmQ, bar, dst, x.kv_head * p.group + at.head,
                          static_cast<int>(x.sq.q0) + (x.j0 + at.block) * BT);
            if (second) at.advance(x.nb);
          });
    } else if (warp == 1) {
      // ------------------------------------------------ MMA issuer
      const uint32_t id_s = idesc_bf16(BT, BT, false, false);
      const uint32_t id_a = idesc_bf16(BT, ks * 16, false, true);
      const uint32_t issue = elect_lane();
      const uint64_t fix_a = kmajor_desc<BT>(m.fix_a), fix_b = kmajor_desc<BT>(m.fix_b);
      const uint64_t ring_a = kmajor_desc<BT>(m.ring_a), ring_b = kmajor_desc<BT>(m.ring_b);
      const uint64_t rows_a = rows_desc<BT>(m.ring_a), rows_b = rows_desc<BT>(m.ring_b);
      constexpr uint32_t STAGE = C::TILE >> 4;
      bool ok = true;
      int base = 0, loads = 0;  // steps and fixed tiles of the pieces before
      for (int pieces = 0;; ++pieces) {
        const DkvPiece x(p, work);
        const int tail = x.sq.nq - x.j0 * BT;  // rows from the first block on
        Step at_s, at_dp;                      // of the next S^T and dP^T
        // X^T = fixed streamed^T of step n
        auto scores = [&](int n, Step& at, uint64_t* full, uint8_t* ring, uint64_t b, uint64_t fix, uint32_t t, uint64_t* done) {
          const int g = base + n, st = g % ST;
          ok = ok && warp_wait(&full[st], (g / ST) & 1, m.abort_flag, p.err);
          if (!ok) return;
          const int rows = tail - at.block * BT;
          at.advance(x.nb);
          if (rows < BT) clear_rows<NC>(ring + st * C::TILE, BT, rows, lane);
          tc_fence_after();
          product<NC, BT>(tmem + t, fix, b + st * STAGE, id_s, ks, issue);
          mma_commit(done, issue);
        };
        // accumulator += (bf16 probabilities at t) . streamed rows of step n
        auto add = [&](int n, uint64_t* ready, uint32_t t, uint32_t t_step, uint32_t acc, uint64_t rows,
                       uint64_t* empty) {
          const int g = base + n;
          ok = ok && warp_wait(ready, g & 1, m.abort_flag, p.err);
          if (!ok) return;
          tc_fence_after();
          const uint64_t b = rows + g % ST * STAGE;
#pragma unroll
          for (int kk = 0; kk < BT / 16; ++kk)
            mma_ts(tmem + acc, tmem + t + (kk >> 1) * t_step + (kk & 1) * 8, b + rows_step(kk), id_a,
                   (kk > 0) | (n > 0), issue);
          mma_commit(&empty[g % ST], issue);
        };
        if (x.steps > 0) {
          ok = warp_wait(m.fix_full, loads & 1, m.abort_flag, p.err);
          ++loads;
          scores(0, at_s, m.a_full, m.ring_a, ring_a, fix_a, 0, m.s_full);
          scores(0, at_dp, m.b_full, m.ring_b, ring_b, fix_b, T_DP, m.dp_full);
          if (x.steps == 1) mma_commit(m.fix_empty, issue);  // K and V: the next piece's may come
          for (int n = 0; ok && n < x.steps; ++n) {
            const bool more = n + 1 < x.steps;
            if (apart && more) {
              ok = warp_wait(m.s_read, (base + n) & 1, m.abort_flag, p.err);
              scores(n + 1, at_s, m.a_full, m.ring_a, ring_a, fix_a, 0, m.s_full);
            }
            add(n, m.p_full, t_p, p_step, t_dv, rows_b, m.b_empty);
            if (ok) mma_commit(m.p_free, issue);
            if (!apart && more) scores(n + 1, at_s, m.a_full, m.ring_a, ring_a, fix_a, 0, m.s_full);
            add(n, m.ds_full, T_DP, C::MC, t_dk, rows_a, m.a_empty);
            if (more) scores(n + 1, at_dp, m.b_full, m.ring_b, ring_b, fix_b, T_DP, m.dp_full);
            if (n + 2 == x.steps) mma_commit(m.fix_empty, issue);
          }
          if (ok) mma_commit(m.acc_full, issue);
          base += x.steps;
        }
        if (!ok || !queue.next(pieces, work, lane, m.abort_flag, p.err)) break;
      }
      mma_commit(m.mma_done, issue);
      warp_wait(m.mma_done, 0, m.abort_flag, p.err);  // before tensor memory is freed
    }
  } else {
    set_regs_inc<C::REGS_MATH>();
    // ------------------------------------------------ P^T, dS^T: a thread holds 32 queries of a key row
    const int w = (warp - 4) >> 2;
    const int quarter = warp & 3;
    const int r = quarter * 32 + lane;
    const uint32_t lanes = static_cast<uint32_t>(quarter * 32) << 16;
    const uint32_t t = tmem + lanes + w * 32;
    const float c2 = p.scale * kAttnLog2e;
    bool ok = true;
    int base = 0, accs = 0;  // steps of the pieces before, and pieces that had any
    for (int pieces = 0;; ++pieces) {
      const DkvPiece x(p, work);
      int lo, hi;  // queries that see this thread's key
      queries_of(p, x.sq, x.key0 + r, lo, hi);
      // lse and delta of the warp's 32 queries, a copy per warp: warps wait for nothing but
      // their barriers; the next block's values are on their way while this one is worked on
      float* buf = m.rows + (warp - 4) * 2 * C::MC;
      float l = 0.0f, d = 0.0f;  // as loaded: nothing waits for them before the next block
      Step next;  // of the next fetch
      auto fetch = [&]() {
        const int i = (x.j0 + next.block) * BT + w * 32 + lane;
        if (i < x.sq.nq) {
          const int64_t at = (x.kv_head * p.group + next.head) * p.Tq + x.sq.q0 + i;
          l = p.lse[at];
          d = p.delta[at];
        }
        next.advance(x.nb);
      };
      if (x.steps > 0) fetch();
      int block = 0;  // of the step
      const float2 cc = make_float2(c2, c2);
      const bool single = x.sq.nk == 1 || p.window == 1;  // every query sees one key at most
      // under a causal mask the query at key 0's place sees that key alone
      const int lone = p.causal && x.key0 == 0 ? x.sq.nq - x.sq.nk : -1;
      for (int n = 0; ok && n < x.steps; ++n) {
        const int i0 = (x.j0 + block) * BT;
        if (++block == x.nb) block = 0;
        __syncwarp();  // the previous block's values are read
        // (behind the last query the rows are cleared, whatever lse and delta hold there;
        // lse = -inf, no key: every place is masked below)
        const bool there = i0 + w * 32 + lane < x.sq.nq;
        buf[lane] = there && l != -INFINITY ? -l * kAttnLog2e : 0.0f;
        buf[C::MC + lane] = there ? -d : 0.0f;
        __syncwarp();
        if (n + 1 < x.steps) fetch();
        if (!warp_wait(m.s_full, (base + n) & 1, m.abort_flag, p.err)) { ok = false; break; }
        tc_fence_after();
        uint32_t s[32], pk[16];
        tmem_ld32(t, s);
        tmem_ld_wait();
        if (apart) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(m.s_read);
        }
        if (i0 < x.full0 || i0 + BT > x.full1) mask_scores(s, lo - i0 - w * 32, hi - lo);
        float2 pr[16];
#pragma unroll
        for (int k = 0; k < 16; k += 2) {
          const float4 l = *reinterpret_cast<const float4*>(buf + 2 * k);
          const float2 u = fma2(make_float2(__uint_as_float(s[2 * k]), __uint_as_float(s[2 * k + 1])), cc,
                                make_float2(l.x, l.y));
          const float2 v = fma2(make_float2(__uint_as_float(s[2 * k + 2]), __uint_as_float(s[2 * k + 3])), cc,
                                make_float2(l.z, l.w));
          pr[k] = make_float2(attn_exp2(u.x), attn_exp2(u.y));
          pr[k + 1] = make_float2(attn_exp2(v.x), attn_exp2(v.y));
          pk[k] = pack2(pr[k].x, pr[k].y);
          pk[k + 1] = pack2(pr[k + 1].x, pr[k + 1].y);
        }
        // (P of the block before has been multiplied long since)
        if (base + n > 0 && !warp_wait(m.p_free, (base + n - 1) & 1, m.abort_flag, p.err)) { ok = false; break; }
        tc_fence_after();
        tmem_st16(tmem + lanes + t_p + w * p_step, pk);
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(m.p_full);
        if (!warp_wait(m.dp_full, (base + n) & 1, m.abort_flag, p.err)) { ok = false; break; }
        tc_fence_after();
        tmem_ld32(t + T_DP, s);
        tmem_ld_wait();
        if (single || (lone >= i0 && lone < i0 + BT)) {
          // a query of a single key has no gradient: dP is delta (rounded another way)
          const int at0 = r == 0 ? lone - i0 - w * 32 : -1;
#pragma unroll
          for (int k = 0; k < 32; ++k)
            if (single || k == at0) s[k] = __float_as_uint(-buf[C::MC + k]);
        }
#pragma unroll
        for (int k = 0; k < 16; k += 2) {
          const float4 d = *reinterpret_cast<const float4*>(buf + C::MC + 2 * k);
          const float2 u = mul2(pr[k], add2(make_float2(__uint_as_float(s[2 * k]), __uint_as_float(s[2 * k + 1])),
                                            make_float2(d.x, d.y)));
          const float2 v = mul2(pr[k + 1], add2(make_float2(__uint_as_float(s[2 * k + 2]), __uint_as_float(s[2 * k + 3])),
                                                make_float2(d.z, d.w)));
          pk[k] = pack2(u.x, u.y);
          pk[k + 1] = pack2(v.x, v.y);
        }
        tmem_st16(t + T_DP, pk);
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(m.ds_full);
      }
      if (ok && x.steps > 0) ok = warp_wait(m.acc_full, accs & 1, m.abort_flag, p.err);
      accs += x.steps > 0;
      base += x.steps;
      tc_fence_after();
      if (ok) {  // the even warpgroups write dV, the odd ones dK, half a row each
        const int r0 = x.key0 + quarter * 32;
        const int64_t at = x.sq.k0 + r0;
        uint8_t* stage = m.out + (warp - 4) * 1024;
        if ((w & 1) == 0)
          store_rows(static_cast<__nv_bfloat16*>(p.dV) + at * p.lddv + x.kv_head * p.hd, p.lddv, tmem + lanes + t_dv, p.hd,
                     1.0f, x.steps > 0, x.sq.nk - r0, w >> 1, 2, stage, lane);
        else
          store_rows(static_cast<__nv_bfloat16*>(p.dK) + at * p.lddk + x.kv_head * p.hd, p.lddk, tmem + lanes + t_dk, p.hd,
                     p.scale, x.steps > 0, x.sq.nk - r0, w >> 1, 2, stage, lane);
      }
      tc_fence_before();
      if (!ok || !queue.next(pieces, work, lane, m.abort_flag, p.err)) break;
    }
  }
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <int NC>
int launch(const AttnArgs& a, cudaStream_t s) {
  using C = Cfg<NC>;
  const int kv_heads = a.heads / a.group;
  static std::atomic<uint64_t> dq_done{0}, dq_twice_done{0}, dkv_done{0};
  const bool twice = a.window > 1 && a.window <= kFewKeys;
  const auto dq = twice ? attn_dq_kernel<NC, true> : attn_dq_kernel<NC, false>;
  int rc = allow_smem(reinterpret_cast<const void*>(dq), C::SMEM, twice ? dq_twice_done : dq_done);
  if (!rc) rc = allow_smem(reinterpret_cast<const void*>(attn_dkv_kernel<NC>), C::SMEM, dkv_done);
  if (rc) return rc;
  CUtensorMap mq, mo, mk, mv;
  const int64_t lists = static_cast<int64_t>(a.heads) * a.batch;
  const int64_t qb = (static_cast<int64_t>(a.max_q) + BT - 1) / BT;
  const int64_t kb = (static_cast<int64_t>(a.max_k) + BT - 1) / BT;
  if (qb > 65535 || kb > 65535 || lists > (1ll << 31) - 1) return QAT_ERR_SHAPE;
  if ((rc = make_head_map(&mq, a.Q, a.hd, a.heads, std::max<int64_t>(a.Tq, 1), a.ldq, BT))) return rc;
  if ((rc = make_head_map(&mo, a.dO, a.hd, a.heads, std::max<int64_t>(a.Tq, 1), a.lddo, BT))) return rc;
  if ((rc = make_head_map(&mk, a.K, a.hd, kv_heads, std::max<int64_t>(a.Tk, 1), a.ldk, BT))) return rc;
  if ((rc = make_head_map(&mv, a.V, a.hd, kv_heads, std::max<int64_t>(a.Tk, 1), a.ldv, BT))) return rc;
  if (a.Tq > 0 && qb > 0) {
    dq<<<dim3(static_cast<unsigned>(lists), static_cast<unsigned>(qb)), C::THREADS, C::SMEM, s>>>(mq, mo, mk, mv, a);
    count_launch();
    if (cudaGetLastError() != cudaSuccess) return QAT_ERR_CUDA;
  }
  if (a.Tk > 0 && kb > 0) {
    attn_dkv_kernel<NC><<<dim3(static_cast<unsigned>(lists / a.group), static_cast<unsigned>(kb)), C::THREADS,
                          C::SMEM, s>>>(mq, mo, mk, mv, a);
    count_launch();
    if (cudaGetLastError() != cudaSuccess) return QAT_ERR_CUDA;
  }
  return QAT_OK;
}

}  // namespace

int launch_attn_bwd(AttnArgs a, cudaStream_t stream) {
  a.err = device_error_ptr();
  return a.hd <= 64 ? launch<1>(a, stream) : launch<2>(a, stream);
}

}  // namespace qat
