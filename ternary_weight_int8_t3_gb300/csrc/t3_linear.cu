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
// times that (512 tokens: the state 2e-4).  Below, g S keeps its own relative precision.
#include "t3_linear.cuh"

namespace t3 {
namespace lin {

constexpr int kCols = 32;   // columns of a state a CTA holds, one a lane
constexpr int kRows = 16;   // rows of it a warp
constexpr int kTokens = 32; // tokens of a block
constexpr float kLn2 = 0.69314718f;

__device__ __forceinline__ float load1(const float* p) { return *p; }
__device__ __forceinline__ float load1(const bf16* p) { return __bfloat162float(*p); }
__device__ __forceinline__ void store1(float* p, float x) { *p = x; }
__device__ __forceinline__ void store1(bf16* p, float x) { *p = __float2bfloat16_rn(x); }

constexpr int padded(int d) { return (d + kRows - 1) / kRows * kRows; }
constexpr int smem_floats(int tokens, int dk) {
  return tokens * (2 * padded(dk) + kCols + 1) + padded(dk) / kRows * tokens * kCols;
}

constexpr float kCut = 2.0f;  // a token whose state starts anew, among the factors

// One token: S = S + c S (kSlow) or c S, plus k v^T, and this warp's part of S^T q.
template <bool kSlow, bool kStates>
__device__ __forceinline__ float token(float2 (&S)[kRows / 2], float c, float v, const float4* k, const float4* q) {
  if (c == kCut) {  // whatever the state held
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
    a = __ffma2_rn(make_float2(k4.x, k4.y), v2, kSlow ? __ffma2_rn(a, c2, a) : __fmul2_rn(a, c2));
    b = __ffma2_rn(make_float2(k4.z, k4.w), v2, kSlow ? __ffma2_rn(b, c2, b) : __fmul2_rn(b, c2));
    if (!kStates) {
      const float4 q4 = q[i];
      sum = __ffma2_rn(make_float2(q4.x, q4.y), a, sum);
      sum2 = __ffma2_rn(make_float2(q4.z, q4.w), b, sum2);
    }
  }
  return (sum.x + sum.y) + (sum2.x + sum2.y);
}

// kStates: only what each part's last piece adds to the state (Args::local).
template <class T, bool kReverse, bool kStates>
__global__ void __launch_bounds__(kMaxHead / kRows * 32) linear_tokens_kernel(const Args p, int col_blocks) {
  extern __shared__ __align__(16) float sm[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5, threads = blockDim.x;
  const int part = blockIdx.x / col_blocks, col = (blockIdx.x - part * col_blocks) * kCols + lane;
  const int rows = warps * kRows;
  const int tokens = p.length < kTokens ? static_cast<int>(p.length) : kTokens;
  float* qs = sm;                         // [tokens][rows]
  float* ks = qs + tokens * rows;         // [tokens][rows]
  float* vs = ks + tokens * rows;         // [tokens][kCols]
  float* os = vs + tokens * kCols;        // [warps][tokens][kCols]
  float* cs = os + warps * tokens * kCols;  // [tokens]
  launch_dependents();
  grid_dependency_wait();
  const int blocks = static_cast<int>(p.blocks);
  int at = part_begin(p, part), end = part_begin(p, part + 1);
  if (kStates) {
    int pair, b0, b1;
    if (!cut_piece(p, part, pair, b0, b1)) return;
    at = pair * blocks + b0;
  } else if (p.whole > 0) {  // whole sequences: then there are no others
    at = part * p.whole * blocks;
    end = at + p.whole * blocks;
  }
  const bool has_col = col < p.dv;
  float2 S[kRows / 2];
  bool fresh = true;  // the state is still to be loaded
  int64_t decays = 0;  // of a state that passes this piece, and whether something cuts it off
  bool cut_off = false;
  for (; at < end; ++at) {
    const int pair = at / blocks, block = at - pair * blocks, tb = kReverse ? blocks - 1 - block : block;
    const int64_t batch = pair / static_cast<int>(p.heads), head = pair - batch * p.heads, t0 = static_cast<int64_t>(tb) * kTokens;
    const int n = static_cast<int>(p.length - t0 < kTokens ? p.length - t0 : kTokens);
    const float log_decay = p.log_decay[head];
    const bool slow = log_decay > -kLn2;
    // of the state from token to token, and where it comes from behind the last token
    const float factor = slow ? expm1f(log_decay) : expf(log_decay), whole = slow ? 0.0f : 1.0f;
    const int64_t state_at = static_cast<int64_t>(pair) * p.dk * p.dv;
    if (fresh || block == 0) {
      fresh = false;
      const bool inside = block > 0 && !kStates;  // behind a cut
      const float* from = inside ? p.local + static_cast<int64_t>(part) * p.dk * p.dv : p.init ? p.init + state_at : nullptr;
      const bool transposed = !inside && p.init_transposed;
      const bool there = from && has_col && !kStates;
#pragma unroll
      for (int i = 0; i < kRows; ++i) {
        const int r = warp * kRows + i;
        const float x = there && r < p.dk ? from[transposed ? col * p.dk + r : r * p.dv + col] : 0.0f;
        if (i & 1)
          S[i / 2].y = x;
        else
          S[i / 2].x = x;
      }
    }
    // the block's rows, in the order they are taken
    const int64_t row0 = batch * p.length + t0;
    for (int i = threadIdx.x; i < n * rows; i += threads) {
      const int j = i / rows, r = i - j * rows;
      const int64_t row = row0 + (kReverse ? n - 1 - j : j);
      const bool in = r < p.dk;
      ks[i] = in ? p.in_scale * load1(static_cast<const T*>(p.k) + row * p.ldk + head * p.dk + r) : 0.0f;
      if (!kStates) qs[i] = in ? load1(static_cast<const T*>(p.q) + row * p.ldq + head * p.dk + r) : 0.0f;
    }
    for (int i = threadIdx.x; i < n * kCols; i += threads) {
      const int j = i / kCols, c = col - lane + i % kCols;
      const int64_t row = row0 + (kReverse ? n - 1 - j : j);
      vs[i] = c < p.dv ? load1(static_cast<const T*>(p.v) + row * p.ldv + head * p.dv + c) : 0.0f;
    }
    for (int j = threadIdx.x; j < n; j += threads) {
      const int64_t t = t0 + (kReverse ? n - 1 - j : j);
      // what cuts a token off from the one taken before it: in time its own mark, against time
      // that of the token taken before it, which is the next one
      const int64_t mark = kReverse ? t + 1 : t;
      const bool cut = p.resets && mark < p.length && p.resets[batch * p.length + mark] != 0;
      cs[j] = cut ? kCut : kReverse && t + 1 == p.length ? whole : factor;
    }
    __syncthreads();
    for (int j = 0; j < n; ++j) {
      const float c = cs[j], v = vs[j * kCols + lane];
      if (kStates) {
        decays += c != whole;
        cut_off |= c == kCut;
      }
      const float4* kp = reinterpret_cast<const float4*>(ks + j * rows + warp * kRows);
      const float4* qp = reinterpret_cast<const float4*>(qs + j * rows + warp * kRows);
      const float x = slow ? token<true, kStates>(S, c, v, kp, qp) : token<false, kStates>(S, c, v, kp, qp);
      if (!kStates) os[(warp * tokens + j) * kCols + lane] = x;
    }
    __syncthreads();
    if (!kStates)
      for (int i = threadIdx.x; i < n * kCols; i += threads) {
        const int j = i / kCols, c = col - lane + i % kCols;
        if (c >= p.dv) continue;
        float x = 0.0f;
        for (int w = 0; w < warps; ++w) x += os[w * tokens * kCols + i];
        const int64_t row = row0 + (kReverse ? n - 1 - j : j);
        store1(static_cast<T*>(p.o) + row * p.ldo + head * p.dv + c, p.out_scale * x);
      }
    const bool behind = !kStates && block + 1 == blocks && p.last;  // the sequence ends
    if ((behind || (kStates && at + 1 == end)) && has_col) {
      float* to = kStates ? p.local + static_cast<int64_t>(part + 1) * p.dk * p.dv : p.last + state_at;
      // against time what is left is the gradient of the state in front of the first token
      const bool cut = kReverse && behind && p.resets && p.resets[batch * p.length] != 0;
      const float f = kReverse && behind ? expf(log_decay) : 1.0f;
#pragma unroll
      for (int i = 0; i < kRows; ++i) {
        const int r = warp * kRows + i;
        const float x = i & 1 ? S[i / 2].y : S[i / 2].x;
        if (r < p.dk) to[r * p.dv + col] = cut || f == 0.0f ? 0.0f : f * x;
      }
      if (kStates && threadIdx.x == 0 && col == 0)
        p.pass[part + 1] = cut_off ? 0.0f : decays == 0 ? 1.0f : expf(log_decay * static_cast<float>(decays));
    }
  }
}

// The states in front of the ranges that begin inside a sequence: what the piece before adds, plus what is left
// of the state in front of that.  A CTA takes 1024 elements of one sequence's states, and goes with the
// first range that begins inside the sequence; four ranges' pieces are on their way at a time.
__global__ void __launch_bounds__(256) linear_join_kernel(const Args p, int element_blocks) {
  constexpr int kAhead = 4, kEach = 4;
  const int slot = blockIdx.x / element_blocks, size = p.dk * p.dv, blocks = static_cast<int>(p.blocks);
  const int e0 = (blockIdx.x - slot * element_blocks) * 1024 + threadIdx.x;
  int j = slot + 1;
  const int begin = part_begin(p, j), pair = begin / blocks, first = pair * blocks;
  launch_dependents();
  if (begin == first || part_begin(p, j - 1) > first) return;
  int end = j + 1;
  while (end < p.ranges && part_begin(p, end) < first + blocks) ++end;
  grid_dependency_wait();
  float x[kEach];
#pragma unroll
  for (int k = 0; k < kEach; ++k) {
    const int e = e0 + 256 * k;
    x[k] = 0.0f;
    if (p.init && e < size) x[k] = p.init[static_cast<int64_t>(pair) * size + (p.init_transposed ? e % p.dv * p.dk + e / p.dv : e)];
  }
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
        x[k] = pass[i] == 0.0f ? piece[i][k] : fmaf(pass[i], x[k], piece[i][k]);
        if (j + i < end && e0 + 256 * k < size) at[static_cast<int64_t>(i) * size + 256 * k] = x[k];
      }
  }
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
  const int blocks = (p.dk * p.dv + 1023) / 1024;
  return launch(linear_join_kernel, static_cast<int64_t>(p.ranges - 1) * blocks, 256, 0, s, 1, p, blocks);
}

template <class T, bool kReverse>
int run(const Args& p, cudaStream_t s) {
  const int col_blocks = (p.dv + kCols - 1) / kCols, threads = padded(p.dk) / kRows * 32;
  const int tokens = p.length < kTokens ? static_cast<int>(p.length) : kTokens;
  const size_t smem = smem_floats(tokens, p.dk) * sizeof(float);
  int dev = 0, st;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return T3_EDEVICE;
  constexpr int kMost = smem_floats(kTokens, kMaxHead) * 4;
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
  p.blocks = (p.length + lin::kTokens - 1) / lin::kTokens;
  // about two CTAs an SM: whole sequences where there are as many, else cuts
  const int64_t col_blocks = (p.dv + lin::kCols - 1) / lin::kCols, want = (2 * sms + col_blocks - 1) / col_blocks;
  const int st = lin::cut(&p, p.pairs < want ? std::min<int64_t>(want, kMaxLinearParts) : p.pairs, workspace, s);
  if (st != T3_OK) return st;
  if (dtype == T3_OUT_BF16)
    return reverse ? lin::run<vec::bf16, true>(p, s) : lin::run<vec::bf16, false>(p, s);
  return reverse ? lin::run<float, true>(p, s) : lin::run<float, false>(p, s);
}

}  // namespace t3
