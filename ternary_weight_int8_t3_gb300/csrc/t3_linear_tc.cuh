// t3_linear_tc.cuh -- linear attention with a decay for each head, by chunks of 128
// tokens on the tensor cores (sm_103a: tcgen05, TMEM, TMA, mbarrier).
//
// What it computes: the recurrence of t3_linear.cuh over bf16 rows.  For a chunk of n tokens that
// begins with the state S, row i at place pos(i) in the order the tokens are taken:
//   o_i = out_scale (sum over pos(j) <= pos(i) of in_scale g^(pos(i) - pos(j)) (q_i . k_j) v_j
//                    + g^(pos(i) + e) S^T q_i)
//   S  <- g^(n - 1 + e) S + sum_j in_scale g^(n - 1 - pos(j)) k_j v_j^T
// e is 1, or 0 where a reversed pass begins.  Four products of 128 x 128 x d: P = Q K^T, masked, decayed and
// rounded to bf16; P V; Q S with S rounded to bf16; and K'^T V with K' = decayed K as the sum of two bf16,
// so that the state, which lives on, keeps 2^-17 of each term (2.5e-6 relative).  S itself stays float, in TMEM, whose sums
// are cut off behind 24 bits: 16 additions a chunk, 6e-7 at a memory of 400 tokens.
//
// What bounds it: memory, q, k, v in and o out once.  A chunk of a head of 128 moves 128 KB, some 5600 clocks of an
// SM's share of the memory's rate; its five products take 1300 of the tensor pipe.  The rest is latency: P
// waits for Q K^T, the state for the product before.  So every step has warps of its own, handing over through
// mbarriers, and the two chains have an issuer each; Q and K, which a chunk begins with, come a chunk ahead:
//   warp 0 TMA; warp 1 issues Q K^T, Q S and P V, warp 2 K'^T V; warps 4-7 P; 8-15 K'; 16-23 the state; 24-27 o.
// Where rows of K have 64 elements warps 4-11 take P and 12-15 K': a chunk waits for P longest (132 us -> 127; with 128, where K'
// is as long, 125 -> 128).
// Each group's thread owns a TMEM lane: a token's row of P and o, half a row of the state (dk), and for K' half a
// token's row in shared memory.  TMEM columns: Q K^T 128, with P over its first 64; P V; Q S; the state.
//
// Decays.  A thread of P has one row; in a block of 32 columns next to it the coefficient is a power of its own
// times one of a table of 32 that all rows share, and where the block meets the diagonal the
// table read at the distance, zeros where it is negative: no exponential an element, and no coefficient above 1.
// The pass for the states alone takes K' decayed to the end of the piece, so that it is one long product.
//
// Measured (bf16, replays of a graph).  8 x 2048 tokens of 27 heads of 128: forward 127 us, 3.8 TB/s: 100 us of it this kernel, 19
// the states of the ranges that the last 64 of 216 sequences are cut into, the rest joining those;
// gradient 371, three such passes.  54 heads of 64: 130 and 395.  1 x 16384 of 10 heads of 128: 74 (states 23, join 8, this 47)
// and 213.  In the middle of a sequence a chunk takes 6500 clocks, where memory's rate allows 6000; what is
// lost lies at the ends: a sequence's begin and end cost 4000 to 10000 clocks more, a kernel's begin
// as much.  A state on its way through shared memory in whole lines instead of a row a lane took 5 % longer,
// and so did P by eight warps (K' by four), 32 warps with 64 registers 15 %.
// The roles' code together is more than the instruction cache next to a scheduler holds: with every wait, mark and division
// written out at its place and the products' loops unrolled (82 KB instead of 51) the first case took 148 us.
//
// Marks.  Where a chunk has any, documents meet in it, and zero times a value that is not finite would pass from one to
// another: P is masked by selection, K' by bits, and rows of V are looked through (by the warps of K') and cleared,
// with NaN in P and K' in their place.  Documents of 300 tokens on average: the first case 168 us (139 without the look at V, which waits for
// V's one place) and gradient 508, heads of 64 186 and 551.
//
// Without marks a value that is not finite meets P's zeros in the rows in front of it: the warps of o look whether P V is finite
// and take such rows again (take_again).  Without ever being run this costs up to 3 % (54 heads of 64 127 us -> 131, 27 of 128 none); as a
// call, or with more loads on their way, 3 to 6 %.
//
// Heads are taken as 64 or 128 elements, zeros behind their own (DK, DV; a file for each pair of them, so that they compile
// in parallel).
#pragma once
#include "t3_internal.h"
#include "t3_linear.cuh"

namespace t3 {
namespace lin {

constexpr int kChunk = 128;
constexpr int kWarpP = 4, kWarpS = 16, kWarpO = 24;
constexpr int kTcThreads = 32 * 28;
constexpr int kColS = 0, kColPV = 128, kColQS = 256, kColState = 384;  // TMEM columns
constexpr int kCode = 12 << 8;
constexpr float kInfinity = __builtin_huge_valf();
constexpr int kTable = 96;  // floats: 32 zeros, g^0 .. g^31 (times both scales), and those backwards

template <int DK, int DV> struct Smem {
  static constexpr int half = kChunk * 128;  // a tile's 64 columns
  static constexpr int tile_k = DK / 64 * half, tile_v = DV / 64 * half;
  static constexpr int state = DK * DV * 2;
  static constexpr int k = 0;                  // two
  static constexpr int v = k + 2 * tile_k;
  static constexpr int k_low = v + tile_v;     // what K' leaves behind its first bf16
  static constexpr int q = k_low + tile_k;     // two; for the states alone a second k_low and V
  static constexpr int s = q + 2 * tile_k;     // the state as bf16, [DK][64] halves
  static constexpr int warps_p = DK == 64 ? 8 : 4;  // half the row's terms of K' leave warps to P
  static constexpr int tables = s + state;     // a warp of P each: see kTable
  static constexpr int bars = tables + warps_p * kTable * 4;
  static constexpr int n_bars = 27;
  static constexpr int misc = bars + 8 * n_bars;
  static constexpr int bad = (misc + 8 + 15) / 16 * 16;  // a bit a token, for each half of its row of V; one marked chunk's and the next's
  static constexpr int bytes = bad + 64 + 1024;
  static_assert(bytes <= 227 * 1024, "shared memory budget");
  // 64 rows of the state: its product is taken with 128, of which the upper half reads whatever lies
  // 64 columns on
  static_assert(DK == 128 || q + 2 * half <= tables, "inside the buffers");  // K's last place is q
  static_assert(tile_k + tile_v <= 2 * tile_k + state, "the states' second V");
};

__device__ __forceinline__ uint32_t idesc_bf16(int n, bool a_mn, bool b_mn) {
  return (1u << 4) | (1u << 7) | (1u << 10) | (a_mn ? 1u << 15 : 0u) | (b_mn ? 1u << 16 : 0u) |
         (static_cast<uint32_t>(n >> 3) << 17) | (128u >> 4 << 24);
}

// Issued by the thread whose `lead` is set; the whole warp comes here, so that descriptors stay in uniform
// registers (issued from a branch of one thread, a product took 110 clocks instead of the tensor pipe's 64).
__device__ __forceinline__ void mma_ss(uint32_t lead, uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t add) {
  asm volatile(
      "{\n\t.reg .pred p, l;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 l, %5, 0;\n\t"
      "@l tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(add), "r"(lead)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t lead, uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t add) {
  asm volatile(
      "{\n\t.reg .pred p, l;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 l, %5, 0;\n\t"
      "@l tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(add), "r"(lead)
      : "memory");
}
__device__ __forceinline__ void mma_commit(uint32_t lead, uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .pred l;\n\tsetp.ne.b32 l, %1, 0;\n\t"
      "@l tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_addr(bar)),
      "r"(lead)
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

__device__ __forceinline__ void tmem_st_x8(uint32_t taddr, const uint32_t (&v)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr), "r"(v[0]),
               "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
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

// One column, and eight, of the rows' own; loaded on return.
__device__ __forceinline__ void tmem_st_x1(uint32_t taddr, float v) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x1.b32 [%0], {%1};" ::"r"(taddr), "r"(__float_as_uint(v)) : "memory");
}
__device__ __forceinline__ float tmem_ld_x1(uint32_t taddr) {
  uint32_t v;
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];\n\ttcgen05.wait::ld.sync.aligned;" : "=r"(v) : "r"(taddr) : "memory");
  return __uint_as_float(v);
}
__device__ __forceinline__ void tmem_ld_x8(uint32_t taddr, uint32_t (&v)[8]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];\n\ttcgen05.wait::ld.sync.aligned;"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7])
      : "r"(taddr)
      : "memory");
}

// `bytes` of memory on their way to L2, multiples of 16 at a multiple of 16.
__device__ __forceinline__ void prefetch_l2(const void* p, int bytes) {
  asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(p), "r"(bytes) : "memory");
}

// 32 bytes at once: a row a lane, so that each takes a whole sector.
__device__ __forceinline__ void load8(const float* p, uint32_t* v) {
  asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7])
               : "l"(p)
               : "memory");
}
__device__ __forceinline__ void store8(void* p, const uint32_t* v) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(v[0]), "r"(v[1]), "r"(v[2]),
               "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}

// The loads so far are in; what was loaded cannot be used in front of this.
__device__ __forceinline__ void loaded(uint32_t (&v)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(v[0]), "+r"(v[1]), "+r"(v[2]), "+r"(v[3]), "+r"(v[4]), "+r"(v[5]), "+r"(v[6]), "+r"(v[7]), "+r"(v[8]),
                 "+r"(v[9]), "+r"(v[10]), "+r"(v[11]), "+r"(v[12]), "+r"(v[13]), "+r"(v[14]), "+r"(v[15])::"memory");
}

// What a wait does when its barrier keeps it, once in the code: the roles together would not fit the
// instruction cache with a copy at each wait.
static __device__ __noinline__ bool keep_waiting(uint64_t* bar, uint32_t parity, volatile int* abort_flag, int* err, int code) {
  return mbar_wait(bar, parity, abort_flag, err, code);
}
__device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity, volatile int* abort_flag, int* err, int code) {
  return mbar_try_wait(bar, parity) || keep_waiting(bar, parity, abort_flag, err, code);
}
static __device__ __noinline__ int quotient(int a, int b) { return static_cast<int>(static_cast<uint32_t>(a) / static_cast<uint32_t>(b)); }

// g^n from log2 g, 1 for n = 0 whatever g.
__device__ __forceinline__ float power(float log2_decay, int n) {
  return n == 0 ? 1.0f : exp2f(log2_decay * static_cast<float>(n));
}

// log2 of the decay of the head at hand.
struct Decay {
  int head = -1;
  float log2 = 0.0f;
  __device__ __forceinline__ bool go(const Args& p, int to) {
    if (to == head) return false;
    head = to;
    log2 = p.log_decay[to] * kLog2e;
    return true;
  }
};

// A CTA's chunks, in the order they are taken: those of its whole sequences, then those of its range of the
// others.  Every role walks the same ones.
struct Walk {
  int left;              // chunks still to take
  int turn = -1;         // of which so many are of the second kind, which begins at
  int then = 0;          // this block
  int count = 0;         // and taken
  int pair, head, batch;
  int block;             // in the sequence
  __device__ __forceinline__ void next(const Args& p) {
    --left;
    ++count;
    if (left == turn) {
      go(p, then);
    } else if (++block == static_cast<int>(p.blocks)) {
      block = 0;
      ++pair;
      if (++head == static_cast<int>(p.heads)) {
        head = 0;
        ++batch;
      }
    }
  }
  // to a block among those of all sequences
  __device__ __forceinline__ void go(const Args& p, int at) {
    pair = quotient(at, static_cast<int>(p.blocks));
    block = at - pair * static_cast<int>(p.blocks);
    batch = quotient(pair, static_cast<int>(p.heads));
    head = pair - batch * static_cast<int>(p.heads);
  }
  // The state comes from memory: at a sequence's begin, and at that of the range
  __device__ __forceinline__ bool fresh() const { return block == 0 || count == 0 || left == turn; }
  __device__ __forceinline__ bool more() const { return left > 0; }
  __device__ __forceinline__ uint32_t parity() const { return count & 1; }
};

template <bool kStates>
__device__ __forceinline__ Walk walk(const Args& p) {
  Walk w;
  int at = 0;
  if (kStates) {
    int pair, b0, b1;
    w.left = cut_piece(p, blockIdx.x, pair, b0, b1) ? b1 - b0 : 0;
    if (w.left > 0) at = pair * static_cast<int>(p.blocks) + b0;
  } else {
    w.then = part_begin(p, blockIdx.x);
    w.turn = part_begin(p, blockIdx.x + 1) - w.then;
    w.left = p.whole * static_cast<int>(p.blocks) + w.turn;
    at = p.whole > 0 ? static_cast<int>(blockIdx.x) * p.whole * static_cast<int>(p.blocks) : w.then;
    if (w.turn == 0 || p.whole == 0) w.turn = -1;
  }
  w.go(p, w.left > 0 ? at : 0);
  return w;
}

// The state that a walk's chunk takes from memory; null: zeros.
__device__ __forceinline__ const float* state_from(const Args& p, const Walk& w) {
  const int64_t size = static_cast<int64_t>(p.dk) * p.dv;
  return w.block > 0 ? p.local + blockIdx.x * size : p.init ? p.init + w.pair * size : nullptr;
}

// A chunk: its first token, tokens, and whether it begins a reversed pass.
struct Chunk {
  int t0, n, e;
};
template <bool kReverse>
__device__ __forceinline__ Chunk chunk(const Args& p, int block) {
  Chunk c;
  c.t0 = (kReverse ? static_cast<int>(p.blocks) - 1 - block : block) * kChunk;
  c.n = min(static_cast<int>(p.length) - c.t0, kChunk);
  c.e = kReverse && block == 0 ? 0 : 1;
  return c;
}

// The marks of n tokens, a bit each; the whole warp calls.
static __device__ __noinline__ uint4 read_marks(const uint8_t* resets, int n) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int j = 32 * i + (threadIdx.x & 31);
    w[i] = __ballot_sync(0xffffffffu, j < n && resets[j] != 0);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}
// The last mark at or in front of token i, -1 if none.
static __device__ __noinline__ int last_mark(uint4 marks, int i) {
  const uint32_t w[4] = {marks.x, marks.y, marks.z, marks.w};
  int r = -1;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int in = i - 32 * k;  // bits 0 .. in count
    const uint32_t m = in < 0 ? 0u : in >= 31 ? w[k] : w[k] & ((2u << in) - 1u);
    if (m) r = 32 * k + 31 - __clz(m);
  }
  return r;
}
// The first mark at or behind token i, 128 if none.
static __device__ __noinline__ int first_mark(uint4 marks, int i) {
  const uint32_t w[4] = {marks.x, marks.y, marks.z, marks.w};
  int r = 128;
#pragma unroll
  for (int k = 3; k >= 0; --k) {
    const int from = i - 32 * k;  // bits from .. 31 count
    const uint32_t m = from > 31 ? 0u : from <= 0 ? w[k] : w[k] & (0xFFFFFFFFu << from);
    if (m) r = 32 * k + __ffs(m) - 1;
  }
  return r;
}

struct Marks {
  uint4 w;
  __device__ __forceinline__ Marks(const Args& p, int batch, const Chunk& c) : w(read_marks(p.resets + batch * p.length + c.t0, c.n)) {}
  __device__ __forceinline__ bool any() const { return (w.x | w.y | w.z | w.w) != 0u; }
  __device__ __forceinline__ int last(int i) const { return last_mark(w, i); }
  __device__ __forceinline__ int first(int i) const { return first_mark(w, i); }
};

// Whether `pieces` of 16 bytes of a row of V hold a value that is not finite; they are cleared then.  Zero times it would be
// NaN in the rows of other documents: what it spoils of its own is marked in P and K' instead.
static __device__ __noinline__ bool clear_bad(uint8_t* row, int pieces) {
  bool bad = false;
#pragma unroll 4
  for (int g = 0; g < pieces; ++g) {
    const uint4 x = *reinterpret_cast<const uint4*>(row + 16 * g);
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) bad |= (w[i] & 0x7F80u) == 0x7F80u || (w[i] & 0x7F800000u) == 0x7F800000u;
  }
  if (bad)
    for (int g = 0; g < pieces; ++g) *reinterpret_cast<uint4*>(row + 16 * g) = make_uint4(0u, 0u, 0u, 0u);
  return bad;
}

// Rows of o that P V left not finite, taken again from memory over their own tokens alone: P's zeros on the other side of a
// row's place leave out what is finite, but zero times a value that is not is NaN.  Written small, since the roles' code has to fit: 0.7 ms a chunk that has one.
struct Again {
  const bf16 *q, *k, *v;  // the row's q, the chunk's first k and v
  int64_t ldk, ldv;
  bf16* out;
  int dk, dv, n, row;
  uint32_t at;            // this lane's TMEM
  float state, scale, log2;  // coefficients of Q S and of P, and the decay's logarithm
  bool bad;               // this row is one of them; the whole warp calls
};
template <bool kReverse>
__device__ __forceinline__ void take_again(const Again a) {
  auto dot8 = [](const bf16* x, const bf16* y, float sum) {
    const uint4 u = *reinterpret_cast<const uint4*>(x), t = *reinterpret_cast<const uint4*>(y);
    const uint32_t us[4] = {u.x, u.y, u.z, u.w}, ts[4] = {t.x, t.y, t.z, t.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float2 c, d;
      unpack(us[i], c.x, c.y);
      unpack(ts[i], d.x, d.y);
      sum = fmaf(c.x, d.x, fmaf(c.y, d.y, sum));
    }
    return sum;
  };
  auto counts = [&](int j) { return a.bad && (kReverse ? j >= a.row : j <= a.row); };
  // the row of P over that of P V
#pragma unroll 1
  for (int j = 0; j < a.n; ++j) {
    float x = 0.0f;
    if (counts(j)) {
#pragma unroll 1
      for (int d = 0; d < a.dk; d += 8) x = dot8(a.q + d, a.k + j * a.ldk + d, x);
      x *= a.scale * power(a.log2, kReverse ? j - a.row : a.row - j);
    }
    __syncwarp();
    tmem_st_x1(a.at + kColPV + j, x);
  }
  tc2::tmem_wait_st();
#pragma unroll 1
  for (int b = 0; b < a.dv; b += 8) {
    uint32_t y[8], o[4];
    float z[8];
    __syncwarp();
    tmem_ld_x8(a.at + kColQS + b, y);
#pragma unroll
    for (int i = 0; i < 8; ++i) z[i] = a.state * __uint_as_float(y[i]);
#pragma unroll 1
    for (int j = 0; j < a.n; ++j) {
      __syncwarp();
      const float x = tmem_ld_x1(a.at + kColPV + j);
      if (!counts(j)) continue;
      const uint4 v = *reinterpret_cast<const uint4*>(a.v + j * a.ldv + b);
      const uint32_t vs[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float2 t;
        unpack(vs[i], t.x, t.y);
        z[2 * i] = fmaf(x, t.x, z[2 * i]);
        z[2 * i + 1] = fmaf(x, t.y, z[2 * i + 1]);
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = pack(z[2 * i], z[2 * i + 1]);
    if (a.bad) *reinterpret_cast<uint4*>(a.out + b) = make_uint4(o[0], o[1], o[2], o[3]);
  }
  __syncwarp();
}

// kStates: only what each part's last piece adds to the state (Args::local).  kMarks: with resets, whose code the others
// are faster without (8 x 2048 tokens of 54 heads of 64 11 % so).
template <int DK, int DV, bool kReverse, bool kStates, bool kMarks>
__global__ void __launch_bounds__(kTcThreads, 1)
    linear_tc_kernel(const Args p, const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
                     const __grid_constant__ CUtensorMap map_v, int* err) {
  using L = Smem<DK, DV>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + (((smem_addr(smem_raw) + 1023u) & ~1023u) - smem_addr(smem_raw));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::bars);
  uint64_t *k_full = bars + 1, *v_full = bars + 3, *k_empty = bars + 5, *s_full = bars + 7,
           *pv_done = bars + 8, *upd_done = bars + 9, *end_bar = bars + 10,
           *o_full = bars + 12;                                           // one arrival each
  uint64_t* v_empty = bars + 13;                                          // both issuers; two, of which without kStates one is used
  uint64_t *p_full = bars + 15, *o_empty = bars + 16, *kp_full = bars + 17, *st_full = bars + 19;  // a group's warps, kp_full two
  uint64_t* drain = bars + 20;                                            // one for each issuer
  uint64_t *q_full = bars + 22, *q_empty = bars + 24;                     // one arrival, two of each
  uint64_t* v_seen = bars + 26;                                           // the warps of K', where a chunk has marks
  uint32_t* bad = reinterpret_cast<uint32_t*>(smem + L::bad);
  int marked_chunks = 0;                                                  // so far
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(smem + L::misc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::misc + 4);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // the first warp of K'; how many warps share a row of P (by halves of its columns) and of K' (by halves of it)
  constexpr int kWarpK = kStates ? 8 : kWarpP + L::warps_p, kShareP = (kWarpK - kWarpP) / 4, kShareK = (kWarpS - kWarpK) / 4;
  constexpr int kGapP = kShareP == 2 ? 32 : 0;  // between the halves of P, each of which lies over its own half of Q K^T

  if (threadIdx.x == 0) {
    for (int i = 0; i < L::n_bars; ++i)
      mbar_init(bars + i, i < 13 ? 1 : i < 15 ? (kStates ? 1 : 2) : i == 15 ? 4 * kShareP : i == 16 ? 4 : i < 19 || i == 26 ? 4 * kShareK : i == 19 ? 8 : 1);
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

  Walk w = walk<kStates>(p);
  bool ok = true;
  if (warp == 0) {
    // ---------------------------------------------------------------- loads
    if (lane == 0) {
      prefetch_tensormap(&map_k);
      prefetch_tensormap(&map_v);
      if (!kStates) prefetch_tensormap(&map_q);
      int q_loads = 0, k_loads = 0, v_loads = 0;
      auto load_q = [&](const Walk& at) {
        const int slot = at.count & 1;
        ok = wait(&q_empty[slot], ((at.count >> 1) & 1) ^ 1u, abort_flag, err, kCode | 1);
        if (!ok) return;
        mbar_arrive_expect_tx(&q_full[slot], L::tile_k);
        for (int h = 0; h < DK / 64; ++h)
          tma_load_4d(smem + L::q + slot * L::tile_k + h * L::half, &map_q, &q_full[slot], 64 * h, at.head,
                      chunk<kReverse>(p, at.block).t0, at.batch);
        ++q_loads;
      };
      auto load_k = [&](const Walk& at) {
        const int slot = at.count & 1;
        ok = wait(&k_empty[slot], ((at.count >> 1) & 1) ^ 1u, abort_flag, err, kCode | 1);
        if (!ok) return;
        mbar_arrive_expect_tx(&k_full[slot], L::tile_k);
        for (int h = 0; h < DK / 64; ++h)
          tma_load_4d(smem + L::k + slot * L::tile_k + h * L::half, &map_k, &k_full[slot], 64 * h, at.head,
                      chunk<kReverse>(p, at.block).t0, at.batch);
        ++k_loads;
      };
      auto load_v = [&](const Walk& at) {
        const int slot = kStates ? at.count & 1 : 0;
        const uint32_t round = kStates ? at.count >> 1 : at.count;
        ok = wait(&v_empty[slot], (round & 1) ^ 1u, abort_flag, err, kCode | 1);
        if (!ok) return;
        mbar_arrive_expect_tx(&v_full[slot], L::tile_v);
        for (int h = 0; h < DV / 64; ++h)
          tma_load_4d(smem + (slot ? L::q + L::tile_k : L::v) + h * L::half, &map_v, &v_full[slot], 64 * h, at.head,
                      chunk<kReverse>(p, at.block).t0, at.batch);
        ++v_loads;
      };
      if (kStates) {
        for (; ok && w.more(); w.next(p)) {
          load_k(w);
          if (ok) load_v(w);
        }
      } else {
        // Q and K of a chunk in front of V of the one before: V's place is free later
        Walk before = w;
        while (ok) {
          const bool more = w.more();
          if (more) {
            const float* state = state_from(p, w);
            if (w.fresh() && (reinterpret_cast<uintptr_t>(state) & 15) == 0 && state) prefetch_l2(state, p.dk * p.dv * 4);
            load_q(w);
            if (ok) load_k(w);
          }
          if (ok && w.count > 0) load_v(before);
          if (!more) break;
          before = w;
          w.next(p);
        }
      }
      if (!ok) {  // giving up: the copies in flight land before this CTA leaves
        const uint64_t t = global_timer_ns();
        auto landed = [&](uint64_t* bar, int loads) {
          if (loads > 0)
            while (!mbar_try_wait(bar, (loads - 1) & 1) && global_timer_ns() - t < kWaitLimitNs) {
            }
        };
        for (int s = 0; s < 2; ++s) {
          landed(&k_full[s], (k_loads + 1 - s) / 2);
          landed(&q_full[s], (q_loads + 1 - s) / 2);
          landed(&v_full[s], kStates ? (v_loads + 1 - s) / 2 : s ? 0 : v_loads);
        }
      }
    }
    __syncwarp();
  } else if (warp == 1 || warp == 2) {
    // ------------------------------------------------------------- products
    const uint32_t lead = lane == 0;
    const uint32_t base = smem_addr(smem);
    const uint64_t q_rows = smem_desc_k_sw128(base + L::q), k_rows = smem_desc_k_sw128(base + L::k);
    const uint64_t k_cols = smem_desc_mn_sw128(base + L::k, L::half, 1024), v1_cols = smem_desc_mn_sw128(base + L::v, L::half, 1024);
    const uint64_t low_cols = smem_desc_mn_sw128(base + L::k_low, L::half, 1024);
    const uint64_t low2_cols = smem_desc_mn_sw128(base + L::q, L::half, 1024);
    const uint64_t v2_cols = smem_desc_mn_sw128(base + L::q + L::tile_k, L::half, 1024);
    const uint64_t s_cols = smem_desc_mn_sw128(base + L::s, DK * 128, 1024);
    // step j of 16 along a product's sum: rows of 128 bytes hold 64 of it, 32 bytes a step; columns
    // go on by two groups of eight rows
    auto along = [](int j) { return static_cast<uint64_t>((j >> 2) * L::half + 32 * (j & 3)) >> 4; };
    auto down = [](int j) { return static_cast<uint64_t>(2048 * j) >> 4; };
    bool issued = false;
    auto seen = [&](uint64_t* bar, uint32_t parity) {
      ok = ok && wait(bar, parity, abort_flag, err, kCode | 3);
    };
    for (; w.more(); w.next(p)) {
      const int slot = w.count & 1;
      const uint32_t par = w.parity(), par2 = (w.count >> 1) & 1;
      const uint64_t k_at = static_cast<uint64_t>(slot * L::tile_k) >> 4;  // of Q's and K's slot
      const int v_slot = kStates ? slot : 0;
      const uint32_t v_par = kStates ? par2 : par;
      const uint64_t v_cols = v_slot ? v2_cols : v1_cols;
      if (warp == 1) {
        if (kStates) break;
        // Q K^T, over the columns that the product before reads P from, and not before the warps of K' have seen
        // that one's end: a barrier that moves on twice is missed
        if (w.count > 0) {
          seen(pv_done, par ^ 1u);
          seen(&kp_full[slot ^ 1], ((w.count - 1) >> 1) & 1);
        }
        seen(&q_full[slot], par2);
        seen(&k_full[slot], par2);
        if (!__all_sync(0xffffffffu, ok)) break;
        tc_fence_after();
#pragma unroll 4
        for (int j = 0; j < DK / 16; ++j)
          mma_ss(lead, tmem + kColS, q_rows + k_at + along(j), k_rows + k_at + along(j), idesc_bf16(128, false, false), j > 0);
        issued = true;
        mma_commit(lead, s_full);
        // Q S
        if (w.count > 0) seen(o_empty, par ^ 1u);
        seen(st_full, par);
        if (!__all_sync(0xffffffffu, ok)) break;
        tc_fence_after();
#pragma unroll 4
        for (int j = 0; j < DK / 16; ++j)
          mma_ss(lead, tmem + kColQS, q_rows + k_at + along(j), s_cols + down(j), idesc_bf16(DV, false, true), j > 0);
        mma_commit(lead, &q_empty[slot]);
        // P V
        seen(&v_full[v_slot], v_par);
        seen(p_full, par);
        if (!__all_sync(0xffffffffu, ok)) break;
        tc_fence_after();
#pragma unroll 4
        for (int j = 0; j < kChunk / 16; ++j)
          mma_ts(lead, tmem + kColPV, tmem + kColS + 8 * j + kGapP * (j >> 2), v_cols + down(j), idesc_bf16(DV, false, true), j > 0);
        mma_commit(lead, pv_done);
        mma_commit(lead, o_full);
        mma_commit(lead, &v_empty[v_slot]);
      } else {
        // S += K'^T V
        if (!kStates) seen(st_full, par);
        seen(&v_full[v_slot], v_par);
        seen(&kp_full[slot], par2);
        if (!__all_sync(0xffffffffu, ok)) break;
        tc_fence_after();
        const uint64_t low = kStates && slot ? low2_cols : low_cols;
#pragma unroll 4
        for (int j = 0; j < kChunk / 16; ++j) {
          mma_ss(lead, tmem + kColState, k_cols + k_at + down(j), v_cols + down(j), idesc_bf16(DV, true, true),
                 !kStates || j > 0 || w.count > 0);
          mma_ss(lead, tmem + kColState, low + down(j), v_cols + down(j), idesc_bf16(DV, true, true), 1u);
        }
        issued = true;
        if (!kStates) mma_commit(lead, upd_done);
        mma_commit(lead, &k_empty[slot]);
        mma_commit(lead, &v_empty[v_slot]);
      }
    }
    if (kStates && warp == 2 && ok && issued) mma_commit(lead, end_bar);
    if (!__all_sync(0xffffffffu, ok) && issued && lead) {  // the products in flight end before their operands go
      mma_commit(1u, drain + warp - 1);
      const uint64_t t = global_timer_ns();
      while (!mbar_try_wait(drain + warp - 1, 0) && global_timer_ns() - t < kWaitLimitNs) {
      }
    }
    __syncwarp();
  } else if (warp >= kWarpP && warp < kWarpK) {
    // --------------------------------------------------------------------- P
    const int q = warp & 3, row = 32 * q + lane, group = (warp - kWarpP) >> 2;
    const uint32_t at = tmem + (static_cast<uint32_t>(32 * q) << 16) + kColS;
    const uint32_t to = at + kGapP * group;
    float* up = reinterpret_cast<float*>(smem + L::tables) + (warp - kWarpP) * kTable + 32;  // g^t, zeros for t < 0
    float* back = up + 32;                                                      // g^(31 - t)
    const float* mine = kReverse ? up - lane : up + lane;  // g^distance at [t] against time, at [-t] in time
    Decay decay;
    float near = 0.0f, over32 = 0.0f;  // a row's power for the next block, and from block to block
    for (; !kStates && w.more(); w.next(p)) {
      if (decay.go(p, w.head)) {
        __syncwarp();
        up[lane - 32] = 0.0f;
        up[lane] = p.in_scale * p.out_scale * power(decay.log2, lane);
        back[lane] = p.in_scale * p.out_scale * power(decay.log2, 31 - lane);
        near = power(decay.log2, kReverse ? 32 - lane : lane + 1);
        over32 = power(decay.log2, 32);
        __syncwarp();
      }
      // the columns that count where not all do that the table leaves (zeros there for those on the row's other side)
      int lo = 0, hi = kChunk - 1;
      bool marked = false, some = false;
      if (kReverse) {  // none lies behind the sequence's end, where a power of a growing state may be infinite
        const int n = chunk<kReverse>(p, w.block).n;
        some = n < kChunk;
        hi = n - 1;
      }
      if (kMarks) {
        const Marks marks(p, w.batch, chunk<kReverse>(p, w.block));
        marked = marks.any();
        if (marked) {
          some = true;
          if (kReverse)
            lo = row, hi = min(hi, marks.first(row + 1) - 1);
          else
            lo = max(marks.last(row), 0), hi = row;
        }
      }
      ok = wait(s_full, w.parity(), abort_flag, err, kCode | 2);
      if (!__all_sync(0xffffffffu, ok)) break;
      tc_fence_after();
      // 16 columns at a time: units 0 .. 2 q + 1 in time, 2 q .. 7 against it; the next one's on their way
      const int first = 8 / kShareP * group, end = first + 8 / kShareP;  // this warp's
      const int u0 = max(kReverse ? 2 * q : 0, first), u1 = min(kReverse ? 8 : 2 * q + 2, end);
      uint32_t s[16];
      if (u0 < u1) tmem_ld_32x32b_x16(at + 16 * u0, s);
#pragma unroll 1
      for (int u = u0; u < u1; ++u) {
        const int b = u >> 1;
        float2 x[8];
        if (b == q) {
          const float* m = mine + (kReverse ? 16 : -16) * (u & 1);
#pragma unroll
          for (int i = 0; i < 8; ++i) x[i] = make_float2(m[kReverse ? 2 * i : -2 * i], m[kReverse ? 2 * i + 1 : -2 * i - 1]);
        } else {
          // in time g^(row - 32 b - 31) g^(31 - t), against it g^(32 b - row) g^t
          const int blocks = kReverse ? b - q : q - b;
          float f = blocks > 2 ? near * over32 : near;
          if (blocks > 1) f *= over32;
          const float4* table = reinterpret_cast<const float4*>((kReverse ? up : back) + 16 * (u & 1));
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float4 t = table[i];
            x[2 * i] = __fmul2_rn(make_float2(t.x, t.y), make_float2(f, f));
            x[2 * i + 1] = __fmul2_rn(make_float2(t.z, t.w), make_float2(f, f));
          }
        }
        loaded(s);
#pragma unroll
        for (int i = 0; i < 8; ++i)
          x[i] = __fmul2_rn(x[i], make_float2(__uint_as_float(s[2 * i]), __uint_as_float(s[2 * i + 1])));
        __syncwarp();
        if (u + 1 < u1) tmem_ld_32x32b_x16(at + 16 * (u + 1), s);
        if (some) {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int j = 16 * u + 2 * i;
            if (j < lo || j > hi) x[i].x = 0.0f;
            if (j + 1 < lo || j + 1 > hi) x[i].y = 0.0f;
          }
        }
        uint32_t out[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) out[i] = pack(x[i].x, x[i].y);
        __syncwarp();
        tmem_st_x8(to + 8 * u, out);  // over columns that this thread has read
      }
      const uint32_t none[8] = {};
      for (int u = first; u < end; ++u)
        if (u < u0 || u >= u1) tmem_st_x8(to + 8 * u, none);
      tc2::tmem_wait_st();
      if (marked) {  // what V holds that is not finite spoils the rows of its document
        ok = wait(v_seen, marked_chunks & 1, abort_flag, err, kCode | 2);
        if (!__all_sync(0xffffffffu, ok)) break;
        const uint32_t* words = bad + 8 * (marked_chunks & 1);
        ++marked_chunks;
#pragma unroll 1
        for (int b = first / 2; b < end / 2; ++b) {
          const uint32_t spoilt = words[b] | words[4 + b];
          if (spoilt == 0u) continue;
          uint32_t v[16];
          __syncwarp();
          tmem_ld_32x32b_x16(to + 16 * b, v);
          loaded(v);
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const int j = 32 * b + 2 * i;
            if (spoilt >> (2 * i) & 1 && j >= lo && j <= hi) v[i] |= 0x7FFFu;
            if (spoilt >> (2 * i + 1) & 1 && j + 1 >= lo && j + 1 <= hi) v[i] |= 0x7FFF0000u;
          }
          __syncwarp();
          tmem_st_x16(to + 16 * b, v);
        }
        tc2::tmem_wait_st();
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(p_full);
    }
  } else if (warp >= kWarpK && warp < kWarpS) {
    // -------------------------------------------------------------------- K'
    const int row = 32 * (warp & 3) + lane, part = (warp - kWarpK) >> 2;  // of the row's 16-byte pieces
    constexpr int kPieces = DK / 8 / kShareK;
    // kStates: decayed to the end of the piece, tokens of which those from `edge` on count (against
    // time those in front of it); the others are cut off by a mark behind them
    int behind = 0, edge = kReverse ? 0x7FFFFFFF : -1;
    Decay decay;
    if (kStates && w.more()) {
      const Chunk first = chunk<kReverse>(p, w.block), end = chunk<kReverse>(p, w.block + w.left - 1);
      const int t0 = kReverse ? end.t0 : first.t0, t1 = kReverse ? first.t0 + first.n : end.t0 + end.n;
      behind = t1 - t0;
      if (kMarks) {
        for (int t = t0 + lane; t < t1; t += 32)
          if (p.resets[w.batch * p.length + t] != 0) edge = kReverse ? min(edge, t) : max(edge, t);
        edge = kReverse ? __reduce_min_sync(0xffffffffu, edge) : __reduce_max_sync(0xffffffffu, edge);
      }
    }
    for (; w.more(); w.next(p)) {
      const Chunk c = chunk<kReverse>(p, w.block);
      // whether this token's row is still in the state in the end, and behind how many tokens
      bool alive = row < c.n, marked = false;
      int away = kReverse ? row : c.n - 1 - row;
      if (kStates) {
        behind -= c.n;
        away += behind;
        alive = alive && (kReverse ? c.t0 + row < edge : c.t0 + row >= edge);
      } else if (kMarks) {
        const Marks marks(p, w.batch, c);
        marked = marks.any();
        if (marked) alive = alive && (kReverse ? marks.first(0) > row : marks.last(kChunk - 1) <= row);
      }
      decay.go(p, w.head);
      const float f = alive ? p.in_scale * power(decay.log2, away) : 0.0f;
      const uint32_t keep = alive ? 0xFFFFFFFFu : 0u;  // whatever a row that is cut off holds
      const float2 f2 = make_float2(f, f);
      const int slot = w.count & 1;
      ok = wait(&k_full[slot], (w.count >> 1) & 1, abort_flag, err, kCode | 2);
      if (!kStates && ok) ok = wait(s_full, w.parity(), abort_flag, err, kCode | 2);  // K has been read as it came
      if (!kStates && w.count > 0 && ok) ok = wait(upd_done, w.parity() ^ 1u, abort_flag, err, kCode | 2);
      if (kStates && (kReverse ? c.t0 + c.n > edge : c.t0 < edge)) {  // nor may what V holds in rows that are cut off count
        ok = ok && wait(&v_full[slot], (w.count >> 1) & 1, abort_flag, err, kCode | 2);
        if (ok && !alive)
          for (int i = part * (DV / 16); i < (part + 1) * (DV / 16); ++i)
            *reinterpret_cast<uint4*>(smem + (slot ? L::q + L::tile_k : L::v) + (i >> 3) * L::half + row * 128 + 16 * (i & 7)) =
                make_uint4(0u, 0u, 0u, 0u);
      }
      if (!__all_sync(0xffffffffu, ok)) break;
      uint8_t* high = smem + L::k + slot * L::tile_k + row * 128;
      uint8_t* low = smem + (kStates && slot ? L::q : L::k_low) + row * 128;
#pragma unroll 4
      for (int i0 = 0; i0 < kPieces; ++i0) {
        const int g = part * kPieces + i0;
        const int o = (g >> 3) * L::half + (((g ^ row) & 7) << 4);  // the 128-byte swizzle
        const uint4 x = *reinterpret_cast<const uint4*>(high + o);
        const uint32_t in[4] = {x.x & keep, x.y & keep, x.z & keep, x.w & keep};
        uint32_t a[4], b[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float2 u, t;
          unpack(in[i], u.x, u.y);
          u = __fmul2_rn(u, f2);
          a[i] = pack(u.x, u.y);
          unpack(a[i], t.x, t.y);
          u = __ffma2_rn(t, make_float2(-1.0f, -1.0f), u);
          b[i] = pack(u.x, u.y);
        }
        sts128(high + o, a[0], a[1], a[2], a[3]);
        sts128(low + o, b[0], b[1], b[2], b[3]);
      }
      if (!kStates && marked) {
        ok = wait(v_full, w.parity(), abort_flag, err, kCode | 2);
        if (!__all_sync(0xffffffffu, ok)) break;
        uint32_t* words = bad + 8 * (marked_chunks & 1) + (warp & 3);
        for (int h = part; h < 2; h += kShareK) {  // by halves of the row
          const uint32_t found = __ballot_sync(
              0xffffffffu, clear_bad(smem + L::v + (DV == 128 ? h * L::half : h * 64) + row * 128, DV / 16));
          if (lane == 0) words[4 * h] = found;
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(v_seen);
        ok = wait(v_seen, marked_chunks & 1, abort_flag, err, kCode | 2);
        if (!__all_sync(0xffffffffu, ok)) break;
        ++marked_chunks;
        if (alive && (words[0] | words[4]) >> lane & 1)
          for (int g = part * kPieces; g < (part + 1) * kPieces; ++g)
            sts128(high + (g >> 3) * L::half + ((g & 7) << 4), 0x7FFF7FFFu, 0x7FFF7FFFu, 0x7FFF7FFFu, 0x7FFF7FFFu);
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&kp_full[slot]);
    }
    if (kStates && w.count > 0 && threadIdx.x == 32 * kWarpK) {
      // what a state in front of the piece has left behind it; the first token of a reversed pass takes it whole
      const bool cut = kReverse ? edge != 0x7FFFFFFF : edge >= 0;
      const int begun = w.block - w.count;  // its first block: the piece ends inside the sequence
      int tokens = 0;
      for (int i = 0; i < w.count; ++i) tokens += chunk<kReverse>(p, begun + i).n;
      if (kReverse && begun == 0) --tokens;
      p.pass[blockIdx.x + 1] = cut ? kCutOff : tokens == 0 ? 1.0f : expf(p.log_decay[w.head] * static_cast<float>(tokens));
    }
  } else if (warp >= kWarpS && warp < kWarpO) {
    // ------------------------------------------------------------- the state
    const int q = warp & 3, row = 32 * q + lane;
    const int col0 = ((warp - kWarpS) >> 2) * (DV / 2);  // half of the columns
    const uint32_t at = tmem + (static_cast<uint32_t>(32 * q) << 16) + kColState + col0;
    const bool mine = 32 * q < DK;  // this warp has rows of it
    Decay decay;
    const int64_t size = static_cast<int64_t>(p.dk) * p.dv;
    // the state behind a piece, to the caller or to the next part
    auto put = [&](float* to, bool cut, float f) {
      if (!mine) return;
      const bool wide = (reinterpret_cast<uintptr_t>(to) & 31) == 0;  // rows are multiples of 32 bytes
#pragma unroll 1
      for (int b = 0; b < DV / 32; ++b) {
        uint32_t s[16];
        __syncwarp();
        tmem_ld_32x32b_x16(at + 16 * b, s);
        loaded(s);
#pragma unroll
        for (int i = 0; i < 16; ++i) s[i] = cut ? 0u : __float_as_uint(f * __uint_as_float(s[i]));
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int col = col0 + 16 * b + 8 * i;
          if (row >= p.dk || col >= p.dv) break;
          float* o = to + row * p.dv + col;
          if (wide) {
            store8(o, s + 8 * i);
          } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) o[j] = __uint_as_float(s[8 * i + j]);
          }
        }
      }
    };
    // the sequence that the chunk before was the last of has ended
    int last_pair = -1;
    auto ended = [&]() {
      const int pair = last_pair;
      last_pair = -1;
      if (pair < 0 || !p.last) return;
      const int batch = quotient(pair, static_cast<int>(p.heads)), head = pair - batch * static_cast<int>(p.heads);
      const bool cut = kReverse && kMarks && p.resets[batch * p.length] != 0;
      put(p.last + pair * size, cut, kReverse ? expf(p.log_decay[head]) : 1.0f);
    };
    // one turn behind the last chunk, for the state behind it
    for (; !kStates; w.next(p)) {
      const bool more = w.more();
      float f = 0.0f;
      bool cut = false;
      if (more) {
        const Chunk c = chunk<kReverse>(p, w.block);
        decay.go(p, w.head);
        f = power(decay.log2, c.n - 1 + c.e);
        if (kMarks) cut = Marks(p, w.batch, c).any();
      }
      // a state that comes from memory, 16 columns ahead
      const bool fresh = more && w.fresh();
      const bool transposed = w.block == 0 && p.init_transposed;
      const float* from = state_from(p, w);
      const bool wide = !transposed && (reinterpret_cast<uintptr_t>(from) & 31) == 0;
      uint32_t next[16];
#pragma unroll 1
      for (int b = fresh ? -1 : 0; b < DV / 32; ++b) {
        if (b == 0) {
          if (w.count > 0) {
            ok = wait(upd_done, w.parity() ^ 1u, abort_flag, err, kCode | 4);
            // and Q S has read the bf16 state: the two products have an issuer each, and it may be the later one
            ok = ok && wait(&q_empty[(w.count - 1) & 1], ((w.count - 1) >> 1) & 1, abort_flag, err, kCode | 4);
            if (!__all_sync(0xffffffffu, ok)) break;
            tc_fence_after();
            ended();
          }
          if (!more) break;
          if (w.block + 1 == static_cast<int>(p.blocks)) last_pair = w.pair;
        }
        if (!mine) continue;
        uint32_t s[16];
        __syncwarp();
        if (fresh) {
#pragma unroll
          for (int i = 0; i < 16; ++i) s[i] = next[i];
          if (b + 1 < DV / 32) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const int col = col0 + 16 * (b + 1) + 8 * i;
#pragma unroll
              for (int j = 0; j < 8; ++j) next[8 * i + j] = 0u;
              if (!from || row >= p.dk || col >= p.dv) continue;
              if (wide) {
                load8(from + row * p.dv + col, next + 8 * i);
              } else {
                const int step = transposed ? p.dk : 1;
                const float* at8 = from + (transposed ? col * p.dk + row : row * p.dv + col);
#pragma unroll
                for (int j = 0; j < 8; ++j) next[8 * i + j] = __float_as_uint(at8[j * step]);
              }
            }
          }
          if (b < 0) continue;
          __syncwarp();
        } else {
          tmem_ld_32x32b_x16(at + 16 * b, s);
          loaded(s);
        }
        const int col = col0 + 16 * b;
        uint8_t* to = smem + L::s + (col >> 6) * DK * 128;
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          uint32_t o[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) o[i] = pack(__uint_as_float(s[8 * g + 2 * i]), __uint_as_float(s[8 * g + 2 * i + 1]));
          sts128(to + tc::sw128(row, (col >> 3 & 7) + g), o[0], o[1], o[2], o[3]);
        }
        if (kMarks && cut) {  // whatever it holds
#pragma unroll
          for (int i = 0; i < 16; ++i) s[i] = 0u;
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float2 x = __fmul2_rn(make_float2(__uint_as_float(s[2 * i]), __uint_as_float(s[2 * i + 1])), make_float2(f, f));
            s[2 * i] = __float_as_uint(x.x);
            s[2 * i + 1] = __float_as_uint(x.y);
          }
        }
        __syncwarp();
        tmem_st_x16(at + 16 * b, s);
      }
      if (!__all_sync(0xffffffffu, ok) || !more) break;
      tc2::tmem_wait_st();
      fence_proxy_async_smem();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(st_full);
    }
    if (kStates && w.more()) {
      ok = wait(end_bar, 0, abort_flag, err, kCode | 4);
      if (__all_sync(0xffffffffu, ok)) {
        tc_fence_after();
        put(p.local + (blockIdx.x + 1) * size, false, 1.0f);
      }
    }
  } else if (warp >= kWarpO) {
    // --------------------------------------------------------------------- o
    const int q = warp - kWarpO, row = 32 * q + lane;
    const uint32_t at = tmem + (static_cast<uint32_t>(32 * q) << 16);
    Decay decay;
    const bool wide = ((reinterpret_cast<uintptr_t>(p.o) | (p.ldo * 2) | (p.dv * 2)) & 31) == 0;
    for (; !kStates && w.more(); w.next(p)) {
      const Chunk c = chunk<kReverse>(p, w.block);
      // what the state that the chunk begins with has left at this token
      const int pos = kReverse ? c.n - 1 - row : row;
      bool alive = pos >= 0, marked = false;
      if (kMarks) {
        const Marks marks(p, w.batch, c);
        marked = marks.any();
        if (marked) alive = alive && (kReverse ? marks.first(row + 1) >= kChunk : marks.last(row) < 0);
      }
      decay.go(p, w.head);
      const float f = alive ? p.out_scale * power(decay.log2, pos + c.e) : 0.0f;
      bf16* out = static_cast<bf16*>(p.o) + (w.batch * p.length + c.t0 + row) * p.ldo + w.head * p.dv;
      ok = wait(o_full, w.parity(), abort_flag, err, kCode | 4);
      if (!__all_sync(0xffffffffu, ok)) break;
      tc_fence_after();
      float top = 0.0f;  // of P V, or NaN
      bool again = false;
      auto release = [&]() {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(o_empty);
      };
#pragma unroll 1
      for (int b = 0; b < DV / 16; ++b) {
        uint32_t x[16], y[16], o[8];
        __syncwarp();
        tmem_ld_32x32b_x16(at + kColPV + 16 * b, x);
        tmem_ld_32x32b_x16(at + kColQS + 16 * b, y);
        loaded(x);
        loaded(y);
#pragma unroll
        for (int i = 0; i < 8; ++i)
          asm("max.NaN.abs.f32 %0, %0, %1, %2;" : "+f"(top) : "f"(__uint_as_float(x[2 * i])), "f"(__uint_as_float(x[2 * i + 1])));
        if (b + 1 == DV / 16) {
          again = !marked && __any_sync(0xffffffffu, row < c.n && !(top < kInfinity));
          if (__builtin_expect(!again, 1)) release();
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          // P has out_scale in it
          const float2 z = __ffma2_rn(make_float2(__uint_as_float(y[2 * i]), __uint_as_float(y[2 * i + 1])), make_float2(f, f),
                                      make_float2(__uint_as_float(x[2 * i]), __uint_as_float(x[2 * i + 1])));
          o[i] = pack(z.x, z.y);
        }
        if (marked && !alive) {  // whatever a state that is cut off holds
#pragma unroll
          for (int i = 0; i < 8; ++i) o[i] = pack(__uint_as_float(x[2 * i]), __uint_as_float(x[2 * i + 1]));
        }
        if (row < c.n && 16 * b < p.dv) {
          if (wide) {
            store8(out + 16 * b, o);
          } else {
            *reinterpret_cast<uint4*>(out + 16 * b) = make_uint4(o[0], o[1], o[2], o[3]);
            if (16 * b + 8 < p.dv) *reinterpret_cast<uint4*>(out + 16 * b + 8) = make_uint4(o[4], o[5], o[6], o[7]);
          }
        }
      }
      if (__builtin_expect(again, 0)) {
        const int64_t first = w.batch * p.length + c.t0;
        take_again<kReverse>({static_cast<const bf16*>(p.q) + (first + row) * p.ldq + w.head * p.dk,
                              static_cast<const bf16*>(p.k) + first * p.ldk + w.head * p.dk,
                              static_cast<const bf16*>(p.v) + first * p.ldv + w.head * p.dv, p.ldk, p.ldv, out, p.dk, p.dv, c.n, row,
                              at, f, p.in_scale * p.out_scale, decay.log2, row < c.n && !(top < kInfinity)});
        release();
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
}

template <int DK, int DV, bool kReverse, bool kMarks>
int run_tc(const Args& p, const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mv, int* err, cudaStream_t s) {
  int dev = 0, st;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return T3_EDEVICE;
  constexpr int kBytes = Smem<DK, DV>::bytes;
  if ((st = allow_smem<linear_tc_kernel<DK, DV, kReverse, false, kMarks>>(dev, kBytes)) != T3_OK) return st;
  if (p.local) {
    if ((st = allow_smem<linear_tc_kernel<DK, DV, kReverse, true, kMarks>>(dev, kBytes)) != T3_OK) return st;
    st = launch(linear_tc_kernel<DK, DV, kReverse, true, kMarks>, p.parts, kTcThreads, kBytes, s, 1, p, mq, mk, mv, err);
    if (st == T3_OK) st = launch_join(p, s);
    if (st != T3_OK) return st;
  }
  return launch(linear_tc_kernel<DK, DV, kReverse, false, kMarks>, p.parts, kTcThreads, kBytes, s, 1, p, mq, mk, mv, err);
}

template <int DK, int DV>
int run_tc(const Args& p, bool reverse, const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mv, int* err,
           cudaStream_t s) {
  if (p.resets)
    return reverse ? run_tc<DK, DV, true, true>(p, mq, mk, mv, err, s) : run_tc<DK, DV, false, true>(p, mq, mk, mv, err, s);
  return reverse ? run_tc<DK, DV, true, false>(p, mq, mk, mv, err, s) : run_tc<DK, DV, false, false>(p, mq, mk, mv, err, s);
}

// One pass for heads of up to DK and DV elements.
#define T3_LINEAR_TC(DK, DV)                                                                                       \
  template int run_tc<DK, DV>(const Args& p, bool reverse, const CUtensorMap& mq, const CUtensorMap& mk,          \
                              const CUtensorMap& mv, int* err, cudaStream_t s)

}  // namespace lin
}  // namespace t3
