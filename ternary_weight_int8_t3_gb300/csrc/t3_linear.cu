// t3_linear.cu -- linear attention with a decay for each head, token by token: single
// tokens, float rows, short sequences, heads and strides of any size.
//
// What it computes: the recurrence of t3_linear.cuh.
//
// What bounds it: a single token reads and writes its state, dk dv floats each way: memory. Longer
// sequences, three packed instructions for two elements of the state a token.  A CTA holds
// 32 columns of a state in registers, 16 rows of a column a thread, so that S stays where it is from
// token to token; a block of tokens' rows is staged in shared memory as floats, where a warp reads
// q and k as broadcasts, and o is summed over the rows by the warps, each leaving its part in
// shared memory until the block ends.  A step with g above a half is taken as S + (g - 1) S + k v^T with g - 1 =
// expm1(log_decay): g itself, rounded, would be off by as much at every step, and a memory of n tokens by n
// times that (512 tokens: the state 2e-4).  Below, g S keeps its own relative precision.  The states alone take
// the decays up to their end in v, and one instruction for three.
//
// The next block's rows are on their way in registers while one is taken: fetched behind the block
// before, with nothing under way meanwhile, 3 x 1782 tokens of 9 float heads of 81 took 631 us.  As many parts as
// CTAs run at once: two more, which ran behind the others, made it 262 for 181.
// Measured: that case 167 us forward and 500 backward (twelve warps an SM that read q and k four rows at a time: shared memory
// is in use 60 % of the time, the float units 50 %); 2 x 2048 of 8 float heads of 128 175 and 532.  Decays kept out of the inner
// loop, in v and o, as for the states alone: 1.05 times as fast in parts of sequences, 0.93 in whole ones.
// One token of 27 sequences and 64 heads of 128 x 128: 40.6 us, 5.6 TB/s (eight CTAs an SM, 8 rows of 16 bytes a
// thread on their way; whole states a CTA and 16 rows a thread 48, 4 rows 59, one element a thread and row 77).  Where rows of a
// state are no 16-byte pieces (dv off multiples of 4) the blocks' kernel takes it: 128 x 126 94 us.
#include <type_traits>

#include "t3_linear.cuh"

namespace t3 {
namespace lin {

constexpr int kCols = 32;   // columns of a state a CTA holds, one a lane
constexpr int kRows = 16;   // rows of it a warp
constexpr int kTokens = 16; // tokens of a block
constexpr float kLn2 = 0.69314718f;

__device__ __forceinline__ float as_float(float x) { return x; }
__device__ __forceinline__ float as_float(bf16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void store1(float* p, float x) { *p = x; }
__device__ __forceinline__ void store1(bf16* p, float x) { *p = __float2bfloat16_rn(x); }

// Rows a CTA holds: whole warps, two at least (so that a thread fetches half a block's v at most).
constexpr int padded(int d) { return d <= 2 * kRows ? 2 * kRows : (d + kRows - 1) / kRows * kRows; }
constexpr int smem_floats(int dk) {
  return 2 * kTokens * (2 * padded(dk) + kCols + 1) + 2 * padded(dk) / kRows * kTokens * kCols;
}

// A token whose state starts anew, among the factors: expm1 and exp of a decay are -1 and 0 at least.
constexpr float kCut = -2.0f;

// How a token is taken: S = S + c S + k v^T, or S = c S + k v^T; for the states alone S = S + k v^T, with
// the decays up to the end in v.
enum Take { kSlow, kFast, kStates };

// One token, and this warp's part of S^T q.
template <Take kTake>
__device__ __forceinline__ float token(float2 (&S)[kRows / 2], float c, float v, const float4* k, const float4* q) {
  if (kTake != kStates && c == kCut) {  // whatever the state held
    c = 0.0f;
#pragma unroll
    for (int i = 0; i < kRows / 2; ++i) S[i] = make_float2(0.0f, 0.0f);
  }
  const float2 c2 = make_float2(c, c), v2 = make_float2(v, v);
  float2 sum = make_float2(0.0f, 0.0f), sum2 = sum;
#pragma unroll
  for (int i = 0; i < kRows / 4; ++i) {
    const float4 k4 = k[i];
    float2 &a = S[2 * i], &b = S[2 * i + 1];
    a = __ffma2_rn(make_float2(k4.x, k4.y), v2, kTake == kSlow ? __ffma2_rn(a, c2, a) : kTake == kFast ? __fmul2_rn(a, c2) : a);
    b = __ffma2_rn(make_float2(k4.z, k4.w), v2, kTake == kSlow ? __ffma2_rn(b, c2, b) : kTake == kFast ? __fmul2_rn(b, c2) : b);
    if (kTake != kStates) {
      const float4 q4 = q[i];
      sum = __ffma2_rn(make_float2(q4.x, q4.y), a, sum);
      sum2 = __ffma2_rn(make_float2(q4.z, q4.w), b, sum2);
    }
  }
  return (sum.x + sum.y) + (sum2.x + sum2.y);
}

// A block of a sequence's tokens.
struct Where {
  int pair, block;
  int64_t batch, head, t0;
  int n;
};

template <bool kReverse>
__device__ __forceinline__ Where locate(const Args& p, int pair, int block) {
  Where w;
  w.pair = pair, w.block = block;
  w.batch = pair / static_cast<int>(p.heads), w.head = pair - w.batch * p.heads;
  w.t0 = static_cast<int64_t>(kReverse ? static_cast<int>(p.blocks) - 1 - block : block) * kTokens;
  w.n = static_cast<int>(p.length - w.t0 < kTokens ? p.length - w.t0 : kTokens);
  return w;
}

// A block's rows on their way, in the order the tokens are taken: half the CTA's threads hold an element
// of each k, the others of each q; each warp every `warps`th v.
template <class T>
struct Rows {
  T kq[kTokens], v[kTokens / 2];
  uint8_t mark;
};

template <class T, bool kReverse, bool kStates>
__device__ __forceinline__ void fetch(const Args& p, const Where& w, int rows, int col, Rows<T>& x) {
  const int warp = threadIdx.x >> 5, warps = rows / kRows, tid = threadIdx.x;
  const bool is_q = tid >= rows;
  const int r = is_q ? tid - rows : tid;
  const int64_t ld = is_q ? p.ldq : p.ldk, row0 = w.batch * p.length + w.t0 + (kReverse ? w.n - 1 : 0);
  const T zero = T(0.0f);
  if (!(kStates && is_q)) {
    const T* from = static_cast<const T*>(is_q ? p.q : p.k) + row0 * ld + w.head * p.dk + r;
#pragma unroll
    for (int j = 0; j < kTokens; ++j) {
      x.kq[j] = j < w.n && r < p.dk ? *from : zero;
      from += kReverse ? -ld : ld;
    }
  }
  const T* from = static_cast<const T*>(p.v) + (row0 + (kReverse ? -warp : warp)) * p.ldv + w.head * p.dv + col;
#pragma unroll
  for (int i = 0; i < kTokens / 2; ++i) {
    x.v[i] = i * warps + warp < w.n && col < p.dv ? *from : zero;
    from += (kReverse ? -warps : warps) * p.ldv;
  }
  x.mark = 0;
  if (p.resets && tid < w.n) {
    // what cuts a token off from the one taken before it: in time its own mark, against time
    // that of the token taken before it, which is the next one
    const int64_t mark = kReverse ? w.t0 + w.n - tid : w.t0 + tid;
    if (mark < p.length) x.mark = p.resets[w.batch * p.length + mark];
  }
}

// kAlone: only what each part's last piece adds to the state (Args::local).
template <class T, bool kReverse, bool kAlone>
__global__ void __launch_bounds__(kMaxHead / kRows * 32, 2) linear_tokens_kernel(const Args p, int col_blocks) {
  extern __shared__ __align__(16) float sm[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  const int part = blockIdx.x / col_blocks, col = (blockIdx.x - part * col_blocks) * kCols + lane;
  const int rows = warps * kRows;
  // twice: k and q [tokens][rows], v [tokens][kCols], the factors [tokens]; twice the sums [warps][tokens][kCols]
  const int block_floats = kTokens * (2 * rows + kCols + 1);
  float* sums = sm + 2 * block_floats;
  launch_dependents();
  grid_dependency_wait();
  const int blocks = static_cast<int>(p.blocks);
  int at = part_begin(p, part), end = part_begin(p, part + 1);
  if (kAlone) {
    int pair, b0, b1;
    if (!cut_piece(p, part, pair, b0, b1)) return;
    at = pair * blocks + b0;
  } else if (p.whole > 0) {  // whole sequences: then there are no others
    at = part * p.whole * blocks;
    end = at + p.whole * blocks;
  }
  if (at >= end) return;
  const bool has_col = col < p.dv;
  float2 S[kRows / 2];
  bool fresh = true;  // the state is still to be loaded

  Where w = locate<kReverse>(p, at / blocks, at % blocks), next = w;
  // kAlone: the piece's tokens, counted in the order they are taken, and the last one of them that is cut off from the one
  // in front: those in front of it are not in the state
  int tau0 = 0, tau1 = 0, edge = -1;
  auto tau = [&](const Where& x) { return static_cast<int>(kReverse ? p.length - x.t0 - x.n : x.t0); };
  if (kAlone) {
    const Where last = locate<kReverse>(p, w.pair, w.block + (end - at) - 1);
    tau0 = tau(w);
    tau1 = tau(last) + last.n;
    if (p.resets) {
      const uint8_t* marks = p.resets + w.batch * p.length;
      for (int i = tau0 + lane; i < tau1; i += 32)
        if (kReverse ? i > 0 && marks[p.length - i] != 0 : marks[i] != 0) edge = max(edge, i);
      edge = __reduce_max_sync(0xffffffffu, edge);
    }
  }
  Rows<T> x;
  float log_decay = 0.0f;
  auto put = [&](float* to) {
    const bool slow = log_decay > -kLn2;
    const int r = threadIdx.x;  // k's rows, then q's
    const int dead = kAlone ? edge - tau(next) : 0;  // so many of the block's first tokens
    if (!(kAlone && r >= rows)) {
      float* kq = to + (r >= rows ? kTokens * rows + r - rows : r);
#pragma unroll
      for (int j = 0; j < kTokens; ++j) kq[j * rows] = kAlone && j < dead ? 0.0f : as_float(x.kq[j]);
    }
    float* vs = to + 2 * kTokens * rows;
    const int behind = tau1 - 1 - tau(next);
#pragma unroll
    for (int i = 0; i < kTokens / 2; ++i) {
      const int j = i * warps + warp;
      if (j >= kTokens) break;
      float f = p.in_scale;
      if (kAlone && j < behind) f *= expf(log_decay * static_cast<float>(behind - j));
      vs[j * kCols + lane] = kAlone && j < dead ? 0.0f : f * as_float(x.v[i]);
    }
    if (!kAlone && threadIdx.x < kTokens)  // of the state from token to token, and where it comes from behind the last token
      vs[kTokens * kCols + threadIdx.x] = x.mark ? kCut
                                          : kReverse && next.t0 + next.n - threadIdx.x == p.length ? (slow ? 0.0f : 1.0f)
                                          : slow ? expm1f(log_decay) : expf(log_decay);
  };
  fetch<T, kReverse, kAlone>(p, w, rows, col, x);
  log_decay = p.log_decay[w.head];
  put(sm);
  __syncthreads();
  for (int turn = 0; at < end; ++at, turn ^= 1) {
    const bool slow = log_decay > -kLn2;
    const float log_decay_now = log_decay;
    if (at + 1 < end) {
      const bool ends = w.block + 1 == blocks;
      next = locate<kReverse>(p, ends ? w.pair + 1 : w.pair, ends ? 0 : w.block + 1);
      fetch<T, kReverse, kAlone>(p, next, rows, col, x);
      log_decay = p.log_decay[next.head];
    }
    const int64_t state_at = static_cast<int64_t>(w.pair) * p.dk * p.dv;
    if (fresh || w.block == 0) {
      fresh = false;
      const bool inside = w.block > 0 && !kAlone;  // behind a cut
      const float* from = inside ? p.local + static_cast<int64_t>(part) * p.dk * p.dv : p.init ? p.init + state_at : nullptr;
      const bool transposed = !inside && p.init_transposed;
      const bool there = from && has_col && !kAlone;
#pragma unroll
      for (int i = 0; i < kRows; ++i) {
        const int r = warp * kRows + i;
        const float y = there && r < p.dk ? from[transposed ? col * p.dk + r : r * p.dv + col] : 0.0f;
        if (i & 1)
          S[i / 2].y = y;
        else
          S[i / 2].x = y;
      }
    }
    const float* ks = sm + turn * block_floats;
    const float* vs = ks + 2 * kTokens * rows + lane;
    const float* cs = ks + 2 * kTokens * rows + kTokens * kCols;
    const float4* kp = reinterpret_cast<const float4*>(ks + warp * kRows);
    const float4* qp = reinterpret_cast<const float4*>(ks + kTokens * rows + warp * kRows);
    float* os = sums + (turn * warps + warp) * kTokens * kCols + lane;
    auto take = [&](auto how) {
      constexpr Take kTake = decltype(how)::value;
#pragma unroll 2
      for (int j = 0; j < w.n; ++j) {
        const float y = token<kTake>(S, kTake == kStates ? 0.0f : cs[j], vs[j * kCols], kp + j * (rows / 4), qp + j * (rows / 4));
        if (kTake != kStates) os[j * kCols] = y;
      }
    };
    if (kAlone) {
      take(std::integral_constant<Take, kStates>());
    } else if (slow) {
      take(std::integral_constant<Take, kSlow>());
    } else {
      take(std::integral_constant<Take, kFast>());
    }
    if (at + 1 < end) put(sm + (turn ^ 1) * block_floats);
    __syncthreads();
    if (!kAlone && has_col) {
      const float* from = sums + turn * warps * kTokens * kCols + lane;
      for (int j = warp; j < w.n; j += warps) {
        float y = 0.0f;
        for (int u = 0; u < warps; ++u) y += from[(u * kTokens + j) * kCols];
        const int64_t row = w.batch * p.length + w.t0 + (kReverse ? w.n - 1 - j : j);
        store1(static_cast<T*>(p.o) + row * p.ldo + w.head * p.dv + col, p.out_scale * y);
      }
    }
    const bool behind = !kAlone && w.block + 1 == blocks && p.last;  // the sequence ends
    if ((behind || (kAlone && at + 1 == end)) && has_col) {
      float* to = kAlone ? p.local + static_cast<int64_t>(part + 1) * p.dk * p.dv : p.last + state_at;
      // against time what is left is the gradient of the state in front of the first token
      const bool cut = kReverse && behind && p.resets && p.resets[w.batch * p.length] != 0;
      const float f = kReverse && behind ? expf(log_decay_now) : 1.0f;
#pragma unroll
      for (int i = 0; i < kRows; ++i) {
        const int r = warp * kRows + i;
        const float y = i & 1 ? S[i / 2].y : S[i / 2].x;
        if (r < p.dk) to[r * p.dv + col] = cut ? 0.0f : f * y;
      }
      if (kAlone && threadIdx.x == 0 && col == 0) {
        const int decays = tau1 - tau0 - (kReverse && tau0 == 0 ? 1 : 0);
        p.pass[part + 1] = edge >= 0 ? kCutOff : decays == 0 ? 1.0f : expf(log_decay_now * static_cast<float>(decays));
      }
    }
    w = next;
  }
}

// One token a sequence, its state read once and written once, 16 bytes a thread and row, all of a thread's 8 rows on
// their way at a time.  A CTA takes 32 columns of a state; `lanes` lanes (a power of two, 4 columns each) share a row.
constexpr int kStepRows = 8, kStepCols = 32;
constexpr int kStepWarps = kMaxHead / (kStepRows * 32 / (kStepCols / 4));

template <class T>
__global__ void __launch_bounds__(kStepWarps * 32, 8) linear_step_kernel(const Args p, int lanes, int col_blocks) {
  __shared__ float4 sums[kStepWarps][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  const int pair = blockIdx.x / col_blocks, col0 = (blockIdx.x - pair * col_blocks) * kStepCols;
  const int sub = lane / lanes, c = (lane - sub * lanes) * 4, col = col0 + c, step = 32 / lanes;
  const int row0 = warp * kStepRows * step + sub;
  const bool has_col = col < p.dv;
  const int64_t batch = pair / static_cast<int>(p.heads), head = pair - batch * p.heads;
  const int64_t at = static_cast<int64_t>(pair) * p.dk * p.dv + static_cast<int64_t>(row0) * p.dv + col;
  launch_dependents();
  grid_dependency_wait();
  float4 S[kStepRows];
#pragma unroll
  for (int i = 0; i < kStepRows; ++i)
    S[i] = p.init && has_col && row0 + i * step < p.dk ? *reinterpret_cast<const float4*>(p.init + at + i * step * p.dv)
                                                       : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  const float log_decay = p.log_decay[head];
  const bool cut = p.resets && p.resets[batch] != 0, slow = log_decay > -kLn2;
  const float f = cut ? 0.0f : slow ? expm1f(log_decay) : expf(log_decay);
  float v[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    v[i] = has_col ? p.in_scale * as_float(static_cast<const T*>(p.v)[batch * p.ldv + head * p.dv + col + i]) : 0.0f;
  const T* kp = static_cast<const T*>(p.k) + batch * p.ldk + head * p.dk + row0;
  const T* qp = static_cast<const T*>(p.q) + batch * p.ldq + head * p.dk + row0;
  float4 sum = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
  for (int i = 0; i < kStepRows; ++i) {
    const bool in = row0 + i * step < p.dk;
    const float k = in ? as_float(kp[i * step]) : 0.0f, q = in ? as_float(qp[i * step]) : 0.0f;
    auto one = [&](float s, float x) {
      return fmaf(k, x, cut ? 0.0f : slow ? fmaf(s, f, s) : s * f);
    };
    S[i] = make_float4(one(S[i].x, v[0]), one(S[i].y, v[1]), one(S[i].z, v[2]), one(S[i].w, v[3]));
    sum = make_float4(fmaf(q, S[i].x, sum.x), fmaf(q, S[i].y, sum.y), fmaf(q, S[i].z, sum.z), fmaf(q, S[i].w, sum.w));
    if (p.last && has_col && in) *reinterpret_cast<float4*>(p.last + at + i * step * p.dv) = S[i];
  }
  sums[warp][lane] = sum;
  __syncthreads();
  // o: over the warps and the rows of each
  for (int i = threadIdx.x; i < kStepCols && col0 + i < p.dv; i += blockDim.x) {
    float y = 0.0f;
    for (int w = 0; w < warps; ++w)
      for (int u = 0; u < step; ++u) y += reinterpret_cast<const float*>(&sums[w][u * lanes])[i];
    store1(static_cast<T*>(p.o) + batch * p.ldo + head * p.dv + col0 + i, p.out_scale * y);
  }
}

template <class T>
int run_step(const Args& p, cudaStream_t s) {
  int lanes = 1;
  while (4 * lanes < kStepCols && 4 * lanes < p.dv) lanes *= 2;
  const int rows = kStepRows * (32 / lanes), warps = (p.dk + rows - 1) / rows, col_blocks = (p.dv + kStepCols - 1) / kStepCols;
  return launch(linear_step_kernel<T>, p.pairs * col_blocks, warps * 32, 0, s, 1, p, lanes, col_blocks);
}

// The states in front of the ranges that begin inside a sequence: what the piece before adds, plus what is left
// of the state in front of that.  A CTA takes 512 elements of the states of one of the sequences that are cut,
// eight ranges' pieces on their way at a time, or four where there are no more (with two or three, room for eight
// cost 4 us more; with fifteen, four at a time 3 us).
__global__ void __launch_bounds__(256) linear_join_kernel(const Args p, int element_blocks) {
  constexpr int kEach = 2;
  const int slot = blockIdx.x / element_blocks, size = p.dk * p.dv, blocks = static_cast<int>(p.blocks);
  const int e0 = (blockIdx.x - slot * element_blocks) * (256 * kEach) + threadIdx.x;
  const int first = p.first + slot * blocks, pair = first / blocks;
  launch_dependents();
  // the ranges that begin inside the sequence: about the slot's share of all of them
  __shared__ int found[2];
  if (threadIdx.x < 32) {
    const float share = static_cast<float>(p.ranges) / static_cast<float>(static_cast<int>(p.pairs) * blocks - p.first);
    int j = min(static_cast<int>(static_cast<float>(slot * blocks) * share), p.ranges);
    while (j > 0 && part_begin(p, j) > first) --j;
    while (j < p.ranges && part_begin(p, j) <= first) ++j;
    int end = min(j + static_cast<int>(static_cast<float>(blocks) * share), p.ranges);
    while (end > j && part_begin(p, end - 1) >= first + blocks) --end;
    while (end < p.ranges && part_begin(p, end) < first + blocks) ++end;
    found[0] = j;
    found[1] = end;
  }
  __syncthreads();
  int j = found[0];
  const int end = found[1];
  grid_dependency_wait();
  if (j >= end) return;
  float x[kEach];
#pragma unroll
  for (int k = 0; k < kEach; ++k) {
    const int e = e0 + 256 * k;
    x[k] = 0.0f;
    if (p.init && e < size) x[k] = p.init[static_cast<int64_t>(pair) * size + (p.init_transposed ? e % p.dv * p.dk + e / p.dv : e)];
  }
  auto join = [&](auto ahead) {
    constexpr int kAhead = decltype(ahead)::value;
#pragma unroll 1
    for (; j < end; j += kAhead) {
      float* at = p.local + static_cast<int64_t>(j) * size + e0;
      float piece[kAhead][kEach], pass[kAhead];
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        pass[i] = j + i < end ? p.pass[j + i] : 0.0f;
#pragma unroll
        for (int k = 0; k < kEach; ++k)
          piece[i][k] = j + i < end && e0 + 256 * k < size ? at[static_cast<int64_t>(i) * size + 256 * k] : 0.0f;
      }
#pragma unroll
      for (int i = 0; i < kAhead; ++i)
#pragma unroll
        for (int k = 0; k < kEach; ++k) {
          x[k] = pass[i] == kCutOff ? piece[i][k] : fmaf(pass[i], x[k], piece[i][k]);
          if (j + i < end && e0 + 256 * k < size) at[static_cast<int64_t>(i) * size + 256 * k] = x[k];
        }
    }
  };
  if (end - j > 4)
    join(std::integral_constant<int, 8>());
  else
    join(std::integral_constant<int, 4>());
}

int cut(Args* p, int64_t parts, float* workspace, cudaStream_t s) {
  const int64_t total = p->pairs * p->blocks;
  const bool in_place = p->init && p->last == p->init;
  p->local = p->pass = nullptr;
  auto deal = [&](int64_t n) {
    p->parts = static_cast<int>(n);
    p->whole = static_cast<int>(p->pairs / n);
    p->first = static_cast<int>(p->whole * n * p->blocks);
    const int64_t left = total - p->first;
    p->ranges = static_cast<int>(std::min(left, n));
    p->each = left > 0 ? static_cast<int>(left / p->ranges) : 0;
    p->rest = left > 0 ? static_cast<int>(left % p->ranges) : 0;
  };
  deal(std::min(parts, total));
  if (p->first == total || p->blocks == 1) return T3_OK;  // nothing is cut
  // tenths of a block's time
  const int64_t longest = p->each + (p->rest > 0 ? 1 : 0);
  const bool pays = 10 * p->whole * p->blocks + 16 * longest + 30 < 10 * (p->whole + 1) * p->blocks;
  if (!workspace || !pays || p->parts > kMaxLinearParts || (in_place && p->pairs >= kMaxLinearParts)) {
    deal(p->pairs);
    return T3_OK;
  }
  const int64_t size = static_cast<int64_t>(p->dk) * p->dv;
  p->local = workspace;
  p->pass = workspace + kMaxLinearParts * size;
  if (in_place) {  // one range may end a sequence before another has begun it
    float* copy = workspace + kMaxLinearParts * (size + 1);
    if (cudaMemcpyAsync(copy, p->init, p->pairs * size * sizeof(float), cudaMemcpyDeviceToDevice, s) != cudaSuccess)
      return T3_ECUDA;
    p->init = copy;
  }
  return T3_OK;
}

int launch_join(const Args& p, cudaStream_t s) {
  const int blocks = (p.dk * p.dv + 511) / 512;
  return launch(linear_join_kernel, (p.pairs - p.first / p.blocks) * blocks, 256, 0, s, 1, p, blocks);
}

template <class T, bool kReverse>
int run(const Args& p, cudaStream_t s) {
  const int col_blocks = (p.dv + kCols - 1) / kCols, threads = padded(p.dk) / kRows * 32;
  const size_t smem = smem_floats(p.dk) * sizeof(float);
  int dev = 0, st;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return T3_EDEVICE;
  constexpr int kMost = smem_floats(kMaxHead) * 4;
  if ((st = allow_smem<linear_tokens_kernel<T, kReverse, false>>(dev, kMost)) != T3_OK) return st;
  if (p.local) {
    if ((st = allow_smem<linear_tokens_kernel<T, kReverse, true>>(dev, kMost)) != T3_OK) return st;
    st = launch(linear_tokens_kernel<T, kReverse, true>, static_cast<int64_t>(p.parts) * col_blocks, threads, smem, s, 1, p,
                col_blocks);
    if (st == T3_OK) st = launch_join(p, s);
    if (st != T3_OK) return st;
  }
  return launch(linear_tokens_kernel<T, kReverse, false>, static_cast<int64_t>(p.parts) * col_blocks, threads, smem, s, 1,
                p, col_blocks);
}

}  // namespace lin

int launch_linear_tokens(lin::Args p, bool reverse, int dtype, float* workspace, int sms, cudaStream_t s) {
  const auto aligned = [](const void* x) { return reinterpret_cast<uintptr_t>(x) % 16 == 0; };
  if (p.length == 1 && !reverse && !p.init_transposed && p.dv % 4 == 0 && aligned(p.init) && aligned(p.last))
    return dtype == T3_OUT_BF16 ? lin::run_step<vec::bf16>(p, s) : lin::run_step<float>(p, s);
  p.blocks = (p.length + lin::kTokens - 1) / lin::kTokens;
  // as many CTAs as run at once (16 warps an SM): whole sequences where there are as many, else cuts
  const int64_t col_blocks = (p.dv + lin::kCols - 1) / lin::kCols, warps = lin::padded(p.dk) / lin::kRows;
  const int64_t want = std::min<int64_t>(sms * (16 / warps) / col_blocks, kMaxLinearParts);
  const int st = lin::cut(&p, std::max(p.pairs, want), workspace, s);
  if (st != T3_OK) return st;
  if (dtype == T3_OUT_BF16)
    return reverse ? lin::run<vec::bf16, true>(p, s) : lin::run<vec::bf16, false>(p, s);
  return reverse ? lin::run<float, true>(p, s) : lin::run<float, false>(p, s);
}

}  // namespace t3
