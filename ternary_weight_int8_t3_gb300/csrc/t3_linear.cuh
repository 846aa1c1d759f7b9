// t3_linear.cuh -- what the kernels of linear attention share (t3_linear.cu token by token,
// t3_linear_tc.cu by chunks on the tensor cores).
//
// One recurrence serves the forward and all of the gradient.  For a head with decay g = exp(log_decay),
// rows q_t, k_t of dk and v_t of dv elements, in the order the tokens are taken:
//   S = c_t S + in_scale k_t v_t^T,   o_t = out_scale S^T q_t
// with c_t = g, or 0 where the token in front is cut off (a reset), or 1 at the first token of a
// reversed pass.  With G_t = dL/dS_t the gradients are the same recurrence over other operands:
//   o  = (q, k, v)    in time, in_scale 1, out_scale scale, from the state
//   dq = (do, v, k)   in time, the same scales, from the state transposed
//   dv = (k, q, do)   against time, in_scale scale, out_scale 1, from dstate_last; leaves G_0
//   dk = (v, do, q)   the same, from dstate_last transposed
//
// Parts.  Every sequence and head is `blocks` blocks of tokens in the order they are taken.  Each of `parts` CTAs
// (or groups of CTAs that share a state's columns) takes as many whole sequences as there are for all of them; the
// blocks of the sequences left, one after the other, are cut into equal ranges, one for each, so that few long
// sequences fill the GPU as many short ones do.  Where a cut falls inside a sequence, a first kernel takes the state that the range in front of the cut
// adds, a second joins those along the sequence, and the ranges then begin with the state they need.
#pragma once
#include <algorithm>

#include "t3_vec.cuh"

namespace t3 {
namespace lin {

using namespace vec;

constexpr int kMaxHead = 128;   // elements of a head's row

struct Args {
  const void *q, *k, *v;
  int64_t ldq, ldk, ldv;  // elements from token to token; heads lie one after the other
  void* o;
  int64_t ldo;
  const float* log_decay;  // [heads]
  const float* init;       // [batch][heads] states [dk][dv], or [dv][dk] (init_transposed); null: zeros
  int init_transposed;
  const uint8_t* resets;   // [batch][length] or null
  float in_scale, out_scale;
  float* last;             // the state behind the last token, [dk][dv]; null: not wanted
  int64_t length, heads, pairs;  // pairs: batch * heads
  int dk, dv;
  int64_t blocks;          // blocks of tokens a sequence
  int parts;
  int whole;               // sequences a part takes as wholes
  int first;               // the first block of the others
  int ranges;              // parts that have some of them: so many each, and one more for some
  int each, rest;
  float* local;            // [parts][dk * dv]: the state in front of each range that begins inside a sequence
  float* pass;             // [parts]: what is left of a state across the piece in front of such a range, or kCutOff
};
// A mark lies in between: nothing, whatever the state holds (a decay of 0 times what is not finite is NaN).
constexpr float kCutOff = -1.0f;

// Blocks are counted in 32 bits (2^36 tokens of all heads would not fit the memory).
__host__ __device__ __forceinline__ int part_begin(const Args& p, int i) {
  return i >= p.ranges ? static_cast<int>(p.pairs * p.blocks)
                       : p.first + p.each * i + static_cast<int>(static_cast<uint32_t>(p.rest * i) / static_cast<uint32_t>(p.ranges));
}

// A sequence's first block of the piece that part i computes last, and the end of it; false
// where the part ends with a sequence.
__device__ __forceinline__ bool cut_piece(const Args& p, int part, int& pair, int& b0, int& b1) {
  const int begin = part_begin(p, part), end = part_begin(p, part + 1), blocks = static_cast<int>(p.blocks);
  pair = end / blocks;
  b1 = end - pair * blocks;
  b0 = begin > pair * blocks ? begin - pair * blocks : 0;
  return b1 > 0;
}

// Deals the sequences to so many parts at most, cutting those left over into ranges where there is a workspace for
// their states and it pays: a range's blocks are taken once more for the states, at 0.6 of the time (by chunks;
// 0.5 token by token), and two more kernels cost some three blocks' time.  Else a part for each sequence and
// head.  A pass that replaces the states it begins with takes a copy of them.
int cut(Args* p, int64_t parts, float* workspace, cudaStream_t s);
int launch_join(const Args& p, cudaStream_t s);

}  // namespace lin

// Ranges a pass is cut into at most: a workspace's size does not depend on the device.
constexpr int kMaxLinearParts = 304;
// Floats of workspace for a pass: `local` and `pass` of the ranges, and a copy of the first states for a
// pass that replaces them (few sequences: kMaxLinearParts at most; more are not cut then).
inline int64_t linear_workspace(int64_t pairs, int64_t length, int64_t dk, int64_t dv) {
  if (pairs <= 0 || length <= 32 || dk <= 0 || dv <= 0) return 0;
  return kMaxLinearParts * (dk * dv + 1) + std::min<int64_t>(pairs, kMaxLinearParts) * dk * dv;
}

// One pass of the recurrence above, by chunks on the tensor cores (bf16, rows of 16-byte
// pieces, t3_linear_tc.cu) and token by token (t3_linear.cu).  workspace: linear_workspace()
// floats, or null.
bool linear_tc_fits(const lin::Args& p, int dtype);
int launch_linear_tc(lin::Args p, bool reverse, float* workspace, int sms, int* err, cudaStream_t s);
int launch_linear_tokens(lin::Args p, bool reverse, int dtype, float* workspace, int sms, cudaStream_t s);

}  // namespace t3
