// t3_linear_tc.cu -- linear attention with a decay for each head, by chunks of 128
// tokens on the tensor cores (sm_103a: tcgen05, TMEM, TMA, mbarrier).
//
// What it computes: the recurrence of t3_linear.cuh over bf16 rows.  For a chunk of n tokens that
// begins with the state S, row i at place pos(i) in the order the tokens are taken:
//   o_i = out_scale (sum over pos(j) <= pos(i) of in_scale g^(pos(i) - pos(j)) (q_i . k_j) v_j
//                    + g^(pos(i) + e) S^T q_i)
//   S  <- g^(n - 1 + e) S + sum_j in_scale g^(n - 1 - pos(j)) k_j v_j^T
// e is 1, or 0 where a reversed pass begins.  Four products of 128 x 128 x d: P = Q K^T, masked, decayed and
// rounded to bf16; P V; Q S with S rounded to bf16; and K'^T V with K' = decayed K as the sum of two bf16,
// so that the state, which lives on, keeps 2^-17 of each term.  S itself stays float, in TMEM.
//
// What bounds it: memory, q, k, v in and o out once.  A chunk of a head of 128 moves 128 KB, some 5600 clocks of an
// SM's share of the memory's rate; its five products take 1300 of the tensor pipe.  The rest is latency: P
// waits for Q K^T, the state for the product before.  So every step has warps of its own, handing over through
// mbarriers, K and V come two chunks ahead and Q one:
//   warp 0 TMA; warp 1 issues the products; warps 4-7 P; 8-11 K'; 12-15 the state; 16-19 o.
// Each group's thread owns a TMEM lane: a token's row of P and o, a row of the state (dk), and for K' a
// token's row in shared memory.  TMEM columns: Q K^T 128, with P over its first 64; P V; Q S; the state.
//
// Decays.  A thread of P has one row; in a block of 32 columns next to it the coefficient is a power of its own
// times one of a table of 32 that all rows share, and where the block meets the diagonal the
// table read at the distance: two products an element, no exponential, and none of them above 1.
#include <cudaTypedefs.h>

#include <cstring>

#include "t3_internal.h"
#include "t3_linear.cuh"

namespace t3 {

PFN_cuTensorMapEncodeTiled_v12000 encode_fn();

namespace lin {

constexpr int kChunk = 128;
constexpr int kGroup = 4;  // warps of a group
constexpr int kWarpP = 4, kWarpK = 8, kWarpS = 12, kWarpO = 16;
constexpr int kTcThreads = 32 * 20;
constexpr int kColS = 0, kColPV = 128, kColQS = 256, kColState = 384;  // TMEM columns
constexpr int kCode = 12 << 8;

template <int DK, int DV> struct Smem {
  static constexpr int half = kChunk * 128;  // a tile's 64 columns
  static constexpr int tile_k = DK / 64 * half, tile_v = DV / 64 * half;
  static constexpr int state = DK * DV * 2;
  static constexpr int q = 0;
  static constexpr int k = q + tile_k;         // two
  static constexpr int v = k + 2 * tile_k;     // two
  static constexpr int k_low = v + 2 * tile_v; // what K' leaves behind its first bf16
  static constexpr int s = k_low + tile_k;     // the state as bf16, [DK][64] halves
  static constexpr int tables = s + state;     // a warp of P each: g^0 .. g^31, and backwards
  static constexpr int bars = tables + 4 * 2 * 32 * 4;
  static constexpr int n_bars = 2 + 8 + 7;
  static constexpr int misc = bars + 8 * n_bars;
  static constexpr int bytes = misc + 16 + 1024;
  static_assert(bytes <= 227 * 1024, "shared memory budget");
  // 64 rows of the state: its product is taken with 128, of which the upper half reads whatever lies
  // 64 columns on
  static_assert(k_low + tile_k + half <= tables || DK == 128, "inside the buffers");
};

__device__ __forceinline__ uint32_t idesc_bf16(int n, bool a_mn, bool b_mn) {
  return (1u << 4) | (1u << 7) | (1u << 10) | (a_mn ? 1u << 15 : 0u) | (b_mn ? 1u << 16 : 0u) |
         (static_cast<uint32_t>(n >> 3) << 17) | (128u >> 4 << 24);
}

__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t add) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(add)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t add) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(add)
      : "memory");
}
__device__ __forceinline__ void mma_commit(uint64_t* bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_addr(bar))
               : "memory");
}

__device__ __forceinline__ void tma_load_4d(void* dst, const CUtensorMap* map, uint64_t* bar, int x, int head, int token,
                                            int batch) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(smem_addr(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_addr(bar)), "r"(x), "r"(head), "r"(token), "r"(batch)
      : "memory");
}

__device__ __forceinline__ void tmem_st_x16(uint32_t taddr, const uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16};" ::"r"(taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
      "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
}

// g^n from log2 g, 1 for n = 0 whatever g.
__device__ __forceinline__ float power(float log2_decay, int n) {
  return n == 0 ? 1.0f : exp2f(log2_decay * static_cast<float>(n));
}

// A CTA's chunks, in the order they are taken.  Every role walks the same ones.
struct Walk {
  int64_t at, end;
  int64_t pair, block;
  int count = 0;  // chunks taken before this one
  __device__ __forceinline__ void next(const Args& p) {
    ++at;
    ++count;
    if (++block == p.blocks) {
      block = 0;
      ++pair;
    }
  }
  __device__ __forceinline__ bool more() const { return at < end; }
  __device__ __forceinline__ uint32_t parity() const { return count & 1; }
};

template <bool kReverse, bool kStates>
__device__ __forceinline__ Walk walk(const Args& p) {
  Walk w;
  w.at = part_begin(p, blockIdx.x);
  w.end = part_begin(p, blockIdx.x + 1);
  if (kStates) {
    int64_t b0, b1;
    if (!cut_piece(p, blockIdx.x, w.pair, b0, b1)) {
      w.at = w.end;
      return w;
    }
    w.block = b0;
    w.at = w.end - (b1 - b0);
  } else {
    w.pair = w.at / p.blocks;
    w.block = w.at - w.pair * p.blocks;
  }
  return w;
}

// A chunk: its first token, tokens, and whether it begins a reversed pass.
struct Chunk {
  int64_t t0;
  int n, e;
  template <bool kReverse>
  static __device__ __forceinline__ Chunk of(const Args& p, int64_t block) {
    Chunk c;
    c.t0 = (kReverse ? p.blocks - 1 - block : block) * kChunk;
    c.n = static_cast<int>(p.length - c.t0 < kChunk ? p.length - c.t0 : kChunk);
    c.e = kReverse && block == 0 ? 0 : 1;
    return c;
  }
};

// The marks of a chunk's tokens, a bit each; the whole warp calls.
struct Marks {
  uint32_t w[4];
  __device__ __forceinline__ Marks(const Args& p, int64_t batch, const Chunk& c) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      w[i] = 0u;
      if (p.resets) {
        const int j = 32 * i + lane;
        w[i] = __ballot_sync(0xffffffffu, j < c.n && p.resets[batch * p.length + c.t0 + j] != 0);
      }
    }
  }
  __device__ __forceinline__ bool any() const { return (w[0] | w[1] | w[2] | w[3]) != 0u; }
  // the last mark at or in front of token i, -1 if none; the first at or behind it, 128 if none
  __device__ __forceinline__ int last(int i) const {
    int r = -1;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int in = i - 32 * k;  // bits 0 .. in count
      const uint32_t m = in < 0 ? 0u : in >= 31 ? w[k] : w[k] & ((2u << in) - 1u);
      if (m) r = 32 * k + 31 - __clz(m);
    }
    return r;
  }
  __device__ __forceinline__ int first(int i) const {
    int r = 128;
#pragma unroll
    for (int k = 3; k >= 0; --k) {
      const int from = i - 32 * k;  // bits from .. 31 count
      const uint32_t m = from > 31 ? 0u : from <= 0 ? w[k] : w[k] & (0xFFFFFFFFu << from);
      if (m) r = 32 * k + __ffs(m) - 1;
    }
    return r;
  }
};

// kStates: only what each part's last piece adds to the state (Args::local).
template <int DK, int DV, bool kReverse, bool kStates>
__global__ void __launch_bounds__(kTcThreads, 1)
    linear_tc_kernel(const Args p, const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
                     const __grid_constant__ CUtensorMap map_v, int* err) {
  using L = Smem<DK, DV>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + (((smem_addr(smem_raw) + 1023u) & ~1023u) - smem_addr(smem_raw));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::bars);
  uint64_t *q_full = bars, *q_empty = bars + 1, *k_full = bars + 2, *k_empty = bars + 4, *v_full = bars + 6,
           *v_empty = bars + 8, *s_full = bars + 10, *p_full = bars + 11, *kp_full = bars + 12, *st_full = bars + 13,
           *upd_done = bars + 14, *o_full = bars + 15, *o_empty = bars + 16;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(smem + L::misc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::misc + 4);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int i = 0; i < L::n_bars; ++i) {
      const uint64_t* b = bars + i;
      mbar_init(bars + i, b == p_full || b == kp_full || b == st_full || b == o_empty ? kGroup : 1);
    }
    *abort_flag = 0;
    fence_mbarrier_init();
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_addr(tmem_holder)) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_holder;
  launch_dependents();
  grid_dependency_wait();

  Walk w = walk<kReverse, kStates>(p);
  bool ok = true;
  if (warp == 0) {
    // ---------------------------------------------------------------- loads
    if (lane == 0) {
      prefetch_tensormap(&map_k);
      prefetch_tensormap(&map_v);
      if (!kStates) prefetch_tensormap(&map_q);
      int q_loads = 0, kv_loads = 0, v_loads = 0;
      for (; ok && w.more(); w.next(p)) {
        const Chunk c = Chunk::of<kReverse>(p, w.block);
        const int head = static_cast<int>(w.pair % p.heads), batch = static_cast<int>(w.pair / p.heads);
        const int slot = w.count & 1, t0 = static_cast<int>(c.t0);
        const uint32_t free = ((w.count >> 1) & 1) ^ 1u;
        ok = mbar_wait(&k_empty[slot], free, abort_flag, err, kCode | 1);
        if (!ok) break;
        mbar_arrive_expect_tx(&k_full[slot], L::tile_k);
        for (int h = 0; h < DK / 64; ++h)
          tma_load_4d(smem + L::k + slot * L::tile_k + h * L::half, &map_k, &k_full[slot], 64 * h, head, t0, batch);
        ++kv_loads;
        ok = mbar_wait(&v_empty[slot], free, abort_flag, err, kCode | 1);
        if (!ok) break;
        mbar_arrive_expect_tx(&v_full[slot], L::tile_v);
        for (int h = 0; h < DV / 64; ++h)
          tma_load_4d(smem + L::v + slot * L::tile_v + h * L::half, &map_v, &v_full[slot], 64 * h, head, t0, batch);
        ++v_loads;
        if (kStates) continue;
        ok = mbar_wait(q_empty, w.parity() ^ 1u, abort_flag, err, kCode | 1);
        if (!ok) break;
        mbar_arrive_expect_tx(q_full, L::tile_k);
        for (int h = 0; h < DK / 64; ++h)
          tma_load_4d(smem + L::q + h * L::half, &map_q, q_full, 64 * h, head, t0, batch);
        ++q_loads;
      }
      if (!ok) {  // giving up: the copies in flight land before this CTA leaves
        const uint64_t t = global_timer_ns();
        auto landed = [&](uint64_t* bar, int loads) {
          if (loads > 0)
            while (!mbar_try_wait(bar, (loads - 1) & 1) && global_timer_ns() - t < kWaitLimitNs) {
            }
        };
        for (int s = 0; s < 2; ++s) {
          landed(&k_full[s], (kv_loads + 1 - s) / 2);
          landed(&v_full[s], (v_loads + 1 - s) / 2);
        }
        landed(q_full, q_loads);
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------------------- products
    if (lane == 0) {
      const uint32_t base = smem_addr(smem);
      bool issued = false;
      for (; ok && w.more(); w.next(p)) {
        const int slot = w.count & 1;
        const uint32_t par = w.parity(), par2 = (w.count >> 1) & 1;
        const uint32_t q = base + L::q, k = base + L::k + slot * L::tile_k, v = base + L::v + slot * L::tile_v;
        if (!kStates) {
          // Q K^T, over the columns that the product before reads P from
          if (w.count > 0) ok = mbar_wait(o_full, par ^ 1u, abort_flag, err, kCode | 3);
          ok = ok && mbar_wait(q_full, par, abort_flag, err, kCode | 3);
          ok = ok && mbar_wait(&k_full[slot], par2, abort_flag, err, kCode | 3);
          if (!ok) break;
          tc_fence_after();
#pragma unroll
          for (int j = 0; j < DK / 16; ++j)
            mma_ss(tmem + kColS, smem_desc_k_sw128(q + (j >> 2) * L::half + 32 * (j & 3)),
                   smem_desc_k_sw128(k + (j >> 2) * L::half + 32 * (j & 3)), idesc_bf16(128, false, false), j > 0);
          issued = true;
          mma_commit(s_full);
        }
        ok = mbar_wait(st_full, par, abort_flag, err, kCode | 3);
        if (!kStates && ok) {
          // Q S
          ok = w.count == 0 || mbar_wait(o_empty, par ^ 1u, abort_flag, err, kCode | 3);
          if (!ok) break;
          tc_fence_after();
#pragma unroll
          for (int j = 0; j < DK / 16; ++j)
            mma_ss(tmem + kColQS, smem_desc_k_sw128(q + (j >> 2) * L::half + 32 * (j & 3)),
                   smem_desc_mn_sw128(base + L::s + j * 2048, DK * 128, 1024), idesc_bf16(DV, false, true), j > 0);
          mma_commit(q_empty);
        }
        // S += K'^T V
        ok = ok && mbar_wait(kp_full, par, abort_flag, err, kCode | 3);
        ok = ok && mbar_wait(&v_full[slot], par2, abort_flag, err, kCode | 3);
        if (!ok) break;
        tc_fence_after();
#pragma unroll
        for (int j = 0; j < kChunk / 16; ++j) {
          const uint64_t vd = smem_desc_mn_sw128(v + j * 2048, L::half, 1024);
          mma_ss(tmem + kColState, smem_desc_mn_sw128(k + j * 2048, L::half, 1024), vd, idesc_bf16(DV, true, true), 1u);
          mma_ss(tmem + kColState, smem_desc_mn_sw128(base + L::k_low + j * 2048, L::half, 1024), vd,
                 idesc_bf16(DV, true, true), 1u);
        }
        issued = true;
        mma_commit(upd_done);
        mma_commit(&k_empty[slot]);
        if (kStates) {
          mma_commit(&v_empty[slot]);
          continue;
        }
        // P V
        ok = mbar_wait(p_full, par, abort_flag, err, kCode | 3);
        if (!ok) break;
        tc_fence_after();
#pragma unroll
        for (int j = 0; j < kChunk / 16; ++j)
          mma_ts(tmem + kColPV, tmem + kColS + 8 * j, smem_desc_mn_sw128(v + j * 2048, L::half, 1024),
                 idesc_bf16(DV, false, true), j > 0);
        mma_commit(o_full);
        mma_commit(&v_empty[slot]);
      }
      if (!ok && issued) {  // the products in flight end before their operands go
        uint64_t* drain = reinterpret_cast<uint64_t*>(smem + L::tables);
        mbar_init(drain, 1);
        fence_mbarrier_init();
        mma_commit(drain);
        const uint64_t t = global_timer_ns();
        while (!mbar_try_wait(drain, 0) && global_timer_ns() - t < kWaitLimitNs) {
        }
      }
    }
    __syncwarp();
  } else if (warp >= kWarpP && warp < kWarpK) {
    // --------------------------------------------------------------------- P
    const int q = warp - kWarpP, row = 32 * q + lane;
    const uint32_t at = tmem + (static_cast<uint32_t>(32 * q) << 16) + kColS;
    float* up = reinterpret_cast<float*>(smem + L::tables) + q * 64;  // g^t
    float* down = up + 32;                                             // g^(31 - t)
    int64_t head_of_table = -1;
    float log2_decay = 0.0f;
    for (; !kStates && w.more(); w.next(p)) {
      const Chunk c = Chunk::of<kReverse>(p, w.block);
      const int64_t head = w.pair % p.heads;
      if (head != head_of_table) {
        head_of_table = head;
        log2_decay = p.log_decay[head] * kLog2e;
        __syncwarp();
        up[lane] = power(log2_decay, lane);
        down[lane] = power(log2_decay, 31 - lane);
        __syncwarp();
      }
      const Marks marks(p, w.pair / p.heads, c);
      // the columns that count: in time lo .. row, against it row .. hi
      const int lo = kReverse ? row : max(marks.last(row), 0), hi = kReverse ? marks.first(row + 1) - 1 : row;
      const bool marked = marks.any();
      ok = mbar_wait(s_full, w.parity(), abort_flag, err, kCode | 2);
      if (!__all_sync(0xffffffffu, ok)) break;
      tc_fence_after();
#pragma unroll 1
      for (int b = 0; b < 4; ++b) {
        uint32_t out[16];
        if (kReverse ? b < q : b > q) {
#pragma unroll
          for (int i = 0; i < 16; ++i) out[i] = 0u;
        } else {
          uint32_t s[32];
          tmem_ld_32x32b_x32(at + 32 * b, s);
          tmem_wait_ld();
          float2 x[16];
          if (b == q) {
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const int d0 = kReverse ? 2 * i - lane : lane - 2 * i, d1 = kReverse ? 2 * i + 1 - lane : lane - 2 * i - 1;
              x[i].x = d0 >= 0 ? up[d0] * p.in_scale * __uint_as_float(s[2 * i]) : 0.0f;
              x[i].y = d1 >= 0 ? up[d1] * p.in_scale * __uint_as_float(s[2 * i + 1]) : 0.0f;
            }
          } else {
            // in time g^(row - 32 b - 31) g^(31 - t), against it g^(32 b - row) g^t
            const float f = p.in_scale * power(log2_decay, kReverse ? 32 * b - row : row - 32 * b - 31);
            const float4* table = reinterpret_cast<const float4*>(kReverse ? up : down);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const float4 t = table[i];
              const float2 f2 = make_float2(f, f);
              x[2 * i] = __fmul2_rn(make_float2(__uint_as_float(s[4 * i]), __uint_as_float(s[4 * i + 1])),
                                    __fmul2_rn(make_float2(t.x, t.y), f2));
              x[2 * i + 1] = __fmul2_rn(make_float2(__uint_as_float(s[4 * i + 2]), __uint_as_float(s[4 * i + 3])),
                                        __fmul2_rn(make_float2(t.z, t.w), f2));
            }
          }
          if (marked) {
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const int j = 32 * b + 2 * i;
              if (j < lo || j > hi) x[i].x = 0.0f;
              if (j + 1 < lo || j + 1 > hi) x[i].y = 0.0f;
            }
          }
#pragma unroll
          for (int i = 0; i < 16; ++i) out[i] = pack(x[i].x, x[i].y);
        }
        tmem_st_x16(at + 16 * b, out);  // over columns that this row's thread has read
      }
      tc2::tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(p_full);
    }
  } else if (warp >= kWarpK && warp < kWarpS) {
    // -------------------------------------------------------------------- K'
    const int row = 32 * (warp - kWarpK) + lane;
    for (; w.more(); w.next(p)) {
      const Chunk c = Chunk::of<kReverse>(p, w.block);
      const Marks marks(p, w.pair / p.heads, c);
      // whether this token's row is still in the state when the chunk ends
      const bool alive = row < c.n && (kReverse ? marks.first(0) > row : marks.last(127) <= row);
      const float f = alive ? p.in_scale * power(p.log_decay[w.pair % p.heads] * kLog2e, kReverse ? row : c.n - 1 - row) : 0.0f;
      const int slot = w.count & 1;
      ok = mbar_wait(&k_full[slot], (w.count >> 1) & 1, abort_flag, err, kCode | 2);
      if (!kStates && ok) ok = mbar_wait(s_full, w.parity(), abort_flag, err, kCode | 2);  // K has been read as it came
      if (w.count > 0 && ok) ok = mbar_wait(upd_done, w.parity() ^ 1u, abort_flag, err, kCode | 2);
      if (!__all_sync(0xffffffffu, ok)) break;
      uint8_t* high = smem + L::k + slot * L::tile_k;
      uint8_t* low = smem + L::k_low;
#pragma unroll
      for (int h = 0; h < DK / 64; ++h) {
#pragma unroll 4
        for (int g = 0; g < 8; ++g) {
          const int o = h * L::half + tc::sw128(row, g);
          const uint4 x = *reinterpret_cast<const uint4*>(high + o);
          const uint32_t in[4] = {x.x, x.y, x.z, x.w};
          uint32_t a[4], b[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            float u0, u1, h0, h1;
            unpack(in[i], u0, u1);
            u0 = f == 0.0f ? 0.0f : u0 * f;
            u1 = f == 0.0f ? 0.0f : u1 * f;
            a[i] = pack(u0, u1);
            unpack(a[i], h0, h1);
            b[i] = pack(u0 - h0, u1 - h1);
          }
          sts128(high + o, a[0], a[1], a[2], a[3]);
          sts128(low + o, b[0], b[1], b[2], b[3]);
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(kp_full);
    }
  } else if (warp >= kWarpS && warp < kWarpO) {
    // ------------------------------------------------------------- the state
    const int q = warp - kWarpS, row = 32 * q + lane;
    const uint32_t at = tmem + (static_cast<uint32_t>(32 * q) << 16) + kColState;
    const bool mine = 32 * q < DK;  // this warp has rows of it
    const int64_t size = static_cast<int64_t>(p.dk) * p.dv;
    int64_t decays = 0;
    bool cut_off = false;
    // the state behind a piece, to the caller or to the next part
    auto put = [&](int64_t pair, float* to, float f) {
      if (!mine) return;
      const bool wide = (reinterpret_cast<uintptr_t>(to) & 15) == 0;  // rows are multiples of 32 bytes
#pragma unroll 1
      for (int b = 0; b < DV / 32; ++b) {
        uint32_t s[32];
        __syncwarp();
        tmem_ld_32x32b_x32(at + 32 * b, s);
        tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int col = 32 * b + 4 * i;
          if (row >= p.dk || col >= p.dv) break;
          float x[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) x[j] = f == 0.0f ? 0.0f : f * __uint_as_float(s[4 * i + j]);
          float* o = to + static_cast<int64_t>(row) * p.dv + col;
          if (wide) {
            *reinterpret_cast<float4*>(o) = make_float4(x[0], x[1], x[2], x[3]);
          } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) o[j] = x[j];
          }
        }
      }
    };
    auto ended = [&](int64_t pair) {  // a sequence has
      if (kStates || !p.last) return;
      const bool cut = kReverse && p.resets && p.resets[pair / p.heads * p.length] != 0;
      put(pair, p.last + pair * size, cut ? 0.0f : kReverse ? expf(p.log_decay[pair % p.heads]) : 1.0f);
    };
    for (; w.more(); w.next(p)) {
      const Chunk c = Chunk::of<kReverse>(p, w.block);
      const Marks marks(p, w.pair / p.heads, c);
      const float log_decay = p.log_decay[w.pair % p.heads];
      __syncwarp();
      const float f = marks.any() ? 0.0f : power(log_decay * kLog2e, c.n - 1 + c.e);
      decays += c.n - 1 + c.e;
      cut_off |= marks.any();
      if (w.count > 0) {
        ok = mbar_wait(upd_done, w.parity() ^ 1u, abort_flag, err, kCode | 4);
        if (!__all_sync(0xffffffffu, ok)) break;
        tc_fence_after();
        if (w.block == 0) ended(w.pair - 1);
      }
      const bool fresh = w.block == 0 || w.count == 0;
      const float* from = nullptr;
      bool transposed = false;
      if (fresh && !kStates) {
        from = w.block > 0 ? p.local + blockIdx.x * size : p.init ? p.init + w.pair * size : nullptr;
        transposed = w.block == 0 && p.init_transposed;
      }
      if (mine) {
#pragma unroll 1
        for (int b = 0; b < DV / 32; ++b) {
          uint32_t s[32];
          if (fresh) {
#pragma unroll
            for (int i = 0; i < 32; ++i) {
              const int col = 32 * b + i;
              float x = 0.0f;
              if (from && row < p.dk && col < p.dv)
                x = from[transposed ? static_cast<int64_t>(col) * p.dk + row : static_cast<int64_t>(row) * p.dv + col];
              s[i] = __float_as_uint(x);
            }
          } else {
            tmem_ld_32x32b_x32(at + 32 * b, s);
            tmem_wait_ld();
          }
          if (!kStates) {
            uint8_t* to = smem + L::s + (b >> 1) * DK * 128;
#pragma unroll
            for (int g = 0; g < 4; ++g) {
              uint32_t o[4];
#pragma unroll
              for (int i = 0; i < 4; ++i) o[i] = pack(__uint_as_float(s[8 * g + 2 * i]), __uint_as_float(s[8 * g + 2 * i + 1]));
              sts128(to + tc::sw128(row, 4 * (b & 1) + g), o[0], o[1], o[2], o[3]);
            }
          }
#pragma unroll
          for (int i = 0; i < 32; ++i) s[i] = f == 0.0f ? 0u : __float_as_uint(f * __uint_as_float(s[i]));
          __syncwarp();
          tc2::tmem_st_32x32b_x32(at + 32 * b, s);
        }
      }
      tc2::tmem_wait_st();
      fence_proxy_async_smem();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(st_full);
    }
    if (ok && w.count > 0) {
      ok = mbar_wait(upd_done, w.parity() ^ 1u, abort_flag, err, kCode | 4);
      if (__all_sync(0xffffffffu, ok)) {
        tc_fence_after();
        if (kStates) {
          put(w.pair, p.local + (blockIdx.x + 1) * size, 1.0f);
          if (threadIdx.x == 32 * kWarpS) {
            const float g = p.log_decay[(w.at - 1) / p.blocks % p.heads];
            p.pass[blockIdx.x + 1] = cut_off ? 0.0f : decays == 0 ? 1.0f : expf(g * static_cast<float>(decays));
          }
        } else if (w.block == 0) {
          ended(w.pair - 1);
        }
      }
    }
  } else if (warp >= kWarpO) {
    // --------------------------------------------------------------------- o
    const int q = warp - kWarpO, row = 32 * q + lane;
    const uint32_t at = tmem + (static_cast<uint32_t>(32 * q) << 16);
    for (; !kStates && w.more(); w.next(p)) {
      const Chunk c = Chunk::of<kReverse>(p, w.block);
      const int64_t head = w.pair % p.heads, batch = w.pair / p.heads;
      const Marks marks(p, batch, c);
      // what the state that the chunk begins with has left at this token
      const bool alive = kReverse ? marks.first(row + 1) >= 128 : marks.last(row) < 0;
      const int pos = kReverse ? c.n - 1 - row : row;
      const float f = alive && pos >= 0 ? p.out_scale * power(p.log_decay[head] * kLog2e, pos + c.e) : 0.0f;
      bf16* out = static_cast<bf16*>(p.o) + (batch * p.length + c.t0 + row) * p.ldo + head * p.dv;
      ok = mbar_wait(o_full, w.parity(), abort_flag, err, kCode | 4);
      if (!__all_sync(0xffffffffu, ok)) break;
      tc_fence_after();
#pragma unroll 1
      for (int b = 0; b < DV / 32; ++b) {
        uint32_t x[32], y[32];
        __syncwarp();
        tmem_ld_32x32b_x32(at + kColPV + 32 * b, x);
        tmem_ld_32x32b_x32(at + kColQS + 32 * b, y);
        tmem_wait_ld();
        if (b + 1 == DV / 32) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(o_empty);
        }
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          const int col = 32 * b + 8 * g;
          if (row >= c.n || col >= p.dv) break;
          uint32_t o[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int j = 8 * g + 2 * i;
            float z[2];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const float s = p.out_scale * __uint_as_float(x[j + k]);
              z[k] = f == 0.0f ? s : fmaf(f, __uint_as_float(y[j + k]), s);
            }
            o[i] = pack(z[0], z[1]);
          }
          *reinterpret_cast<uint4*>(out + col) = make_uint4(o[0], o[1], o[2], o[3]);
        }
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
}

// Rows of a head's 64 columns and 128 tokens of [batch][length][heads][d], 128-byte swizzle, zeros outside.
bool make_map(CUtensorMap* map, const void* base, const Args& p, int64_t ld, int d) {
  std::memset(map, 0, sizeof(*map));
  auto fn = encode_fn();
  if (!fn) return false;
  cuuint64_t dims[4] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(p.heads), static_cast<cuuint64_t>(p.length),
                        static_cast<cuuint64_t>(p.pairs / p.heads)};
  cuuint64_t strides[3] = {static_cast<cuuint64_t>(d) * 2, static_cast<cuuint64_t>(ld) * 2,
                           static_cast<cuuint64_t>(p.length) * ld * 2};
  cuuint32_t box[4] = {64, 1, kChunk, 1};
  cuuint32_t estr[4] = {1, 1, 1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(base), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int DK, int DV, bool kReverse>
int run_tc(const Args& p, const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mv, int* err, cudaStream_t s) {
  int dev = 0, st;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return T3_EDEVICE;
  constexpr int kBytes = Smem<DK, DV>::bytes;
  if ((st = allow_smem<linear_tc_kernel<DK, DV, kReverse, false>>(dev, kBytes)) != T3_OK) return st;
  if (p.local) {
    if ((st = allow_smem<linear_tc_kernel<DK, DV, kReverse, true>>(dev, kBytes)) != T3_OK) return st;
    st = launch(linear_tc_kernel<DK, DV, kReverse, true>, p.parts, kTcThreads, kBytes, s, 1, p, mq, mk, mv, err);
    if (st == T3_OK) st = launch_join(p, s);
    if (st != T3_OK) return st;
  }
  return launch(linear_tc_kernel<DK, DV, kReverse, false>, p.parts, kTcThreads, kBytes, s, 1, p, mq, mk, mv, err);
}

template <int DK, int DV>
int run_tc(const Args& p, bool reverse, const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mv, int* err,
           cudaStream_t s) {
  return reverse ? run_tc<DK, DV, true>(p, mq, mk, mv, err, s) : run_tc<DK, DV, false>(p, mq, mk, mv, err, s);
}

}  // namespace lin

// More tokens than one block of the other kernel takes as fast; rows and heads that TMA can address, and
// outputs that take 16-byte stores.
bool linear_tc_fits(const lin::Args& p, int dtype) {
  auto rows = [](const void* base, int64_t ld) { return vec::aligned(base, 16) && ld % 8 == 0; };
  return dtype == T3_OUT_BF16 && p.length > 16 && p.dk % 8 == 0 && p.dv % 8 == 0 && rows(p.q, p.ldq) &&
         rows(p.k, p.ldk) && rows(p.v, p.ldv) && rows(p.o, p.ldo) && p.ldq >= p.heads * p.dk &&
         p.ldk >= p.heads * p.dk && p.ldv >= p.heads * p.dv &&
         p.length * std::max(p.ldq, std::max(p.ldk, p.ldv)) < (int64_t{1} << 38);
}

int launch_linear_tc(lin::Args p, bool reverse, float* workspace, int sms, int* err, cudaStream_t s) {
  CUtensorMap mq, mk, mv;
  if (!lin::make_map(&mq, p.q, p, p.ldq, p.dk) || !lin::make_map(&mk, p.k, p, p.ldk, p.dk) ||
      !lin::make_map(&mv, p.v, p, p.ldv, p.dv))
    return T3_ECUDA;
  p.blocks = (p.length + lin::kChunk - 1) / lin::kChunk;
  const int st = lin::cut(&p, sms, workspace, s);
  if (st != T3_OK) return st;
  return lin::run_tc<128, 128>(p, reverse, mq, mk, mv, err, s);
}

}  // namespace t3
