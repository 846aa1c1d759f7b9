// t3_scan.cu -- the gated linear recurrence over a sequence, and its gradient.
//
// What it computes, per sequence and channel, with the gate's logit f_t and
// the candidate c_t:
//   k_t = sigmoid(-f_t)                        (how much of the candidate is taken)
//   h_t = (1 - k_t) h'_{t-1} + k_t c_t = h' + k_t (c_t - h'),
//   h'_{t-1} = h_{t-1}, or 0 where a reset starts a new document at t.
// Backward, with G_t the whole gradient of h_t:
//   G_t = dh_t + (1 - k_{t+1}) G_{t+1}        (without the second term at a reset)
//   dc_t = k_t G_t,   df_t = G_t (h'_{t-1} - c_t) k_t (1 - k_t)
//   dh0 = (1 - k_0) G_0.
// Backward, h' comes from the forward's output: 2 bytes an element for bf16 rows, where a float
// copy for the gradient would add 6 to the 18 of both directions.  The
// rounding costs dgate half of what its own costs (8 x 2048 x 3456, gates around 1.5:
// relative norm 8.2e-4 for h', 1.66e-3 for dgate's bf16, 1.85e-3 together); a user who needs
// more keeps gate, candidate and h in float.
// The state is float.  The step is taken as h' + k (c - h'): k = sigmoid(-f)
// keeps its relative precision as the gate closes, where 1 - k would not, so a
// long memory is not lost to rounding.  Where k is exactly 0 (f = +inf, or a gate
// closed below the float range) the candidate is not looked at: f = +inf masks a
// token whatever its candidate holds.
//
// What bounds it: memory (bf16: 6 bytes an element forward, 12 backward), once
// there is enough work in flight; a few sequences have few channels, so time
// is split.  A step is the linear map h -> (h - R h) + H, and maps compose (R
// and not 1 - R is what is kept: products of factors near 1 would lose the
// same long memory), so:
//   * a lane holds two channels over a run of S steps in registers (neighbours,
//     worked on with packed instructions; half a tile apart where rows go element
//     by element), a warp 64 channels over S steps or 32 over 2 S, a CTA of 8
//     warps 8 times as many consecutive steps, a cluster up to 8 CTAs;
//   * each lane composes its run's map; warp 0 composes the CTA's, which travel to
//     the cluster's other CTAs by asynchronous stores that complete on the
//     receiver's barrier (so that nobody waits for its own output stores), and
//     steps the carried state from warp to warp; each lane then runs its steps
//     again from registers, this time from the true state;
//   * the cluster walks along the sequence, a round at a time.
// More tiles of channels than are resident at once need no split in time; forward, a
// cluster's CTAs then share several tiles evenly (scan_fwd_shared_kernel).
// Each direction reads its operands once (the backward gate, candidate and h anew) and
// writes once, in a fixed order: the result does not change from call to call.  Sequences of a few tokens take one thread per
// channel pair and no exchange.
//
// Operands arrive by asynchronous copies, a round ahead, in a stage of the warp's
// own; k stays in registers between the two passes over a run, the candidate is
// read from the stage again.
//
// Measured (GB300; bytes of the formulas, of the measured 6784 GB/s): bf16 8 x 2048 x
// 3456 forward 55 to 56 us (90 %), with resets 57; backward 109 us (92 %) to 129, by how the
// arrays happen to lie in memory, with resets 111; 8 x 2048 x 2560 forward 42.5 us (87 %),
// backward 96 (77 %); 1 x 16384 x 1280 forward 33 us (57 %) and backward 64 us (58 %),
// with resets 37 and 70; 27 single tokens of 8192 channels 2 us.  Float 6 x 1000 x 4096
// 48 us (91 %) and 91 us (95 %), with resets 49 and 93.
// Rows of 4-byte pieces take 1.2 to 1.5 times as long as aligned ones, odd rows of
// 2-byte elements, copied one by one, twice (11 x 1500 x 1101 bf16: 52 and 101 us;
// 3 x 1782 x 729 float with resets 12.8 and 21.8).
// The long sequence is held up by no one thing (left out one at a time, of 33 us: the
// exchange 9, the first pass 7, the second 4.5, the copies 4): four warps a scheduler
// do not overlap them all.  Trading the maps behind the next round's first pass, in a
// warp of its own and with shorter runs, takes 35 us; runs of 8 and 12 steps in three or
// four CTAs an SM 45 to 63; of 20 and 24 steps 34 and 42.
#include <algorithm>
#include <type_traits>

#include "t3_vec.cuh"

namespace t3 {
namespace sc {

using namespace vec;

constexpr int kWarps = 8;
// CTAs that share an SM.  Their 64 KB of stages would let three; but the 16
// steps a lane holds spill at the 80 registers that leaves, and two balance better over
// the SMs (8 x 2048 x 3456 forward: 57 us with three and 12 steps, 55 with two and
// 16; 1 x 16384 x 1280: 45 and 33).
constexpr int kPerSm = 2;

struct FwdArgs {
  const void *gate, *cand;
  int64_t ldg, ldc, ldh;
  const float* h0;
  const uint8_t* resets;
  void* h;
  float* h_last;
  int64_t length, width, tiles;  // tiles: of a sequence
  int64_t all_tiles;  // of all (shared tiles)
  int64_t channels;  // batch * width (short sequences)
  int* err;
};

struct BwdArgs {
  const void *gate, *cand, *h, *dh;
  int64_t ldg, ldc, ldh, lddh, lddg, lddc;
  const float* h0;
  const uint8_t* resets;
  const float* dh_last;
  void *dgate, *dcand;
  float* dh0;
  int64_t length, width, tiles;
  int* err;
};

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}
// All threads of the cluster arrive; nothing is ordered by it (a release here
// would wait for every output store in flight).
__device__ __forceinline__ void cluster_meet() {
  asm volatile("barrier.cluster.arrive.relaxed.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
}
// The address in CTA `rank` of the cluster of a shared variable of this one.
__device__ __forceinline__ uint32_t peer(const void* p, int rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(smem_addr(p)), "r"(rank));
  return r;
}

// Where a CTA waits for its cluster's maps; `failed` once a wait ran out, after which no wait
// is made and the results are not valid (the error word says so).
struct Waits {
  int* err;
  volatile int* abort_flag;
  bool failed;
};
constexpr int kWaitCode = (11 << 8) | 7;

// Waits for a phase of `bar` that peers complete with st.async; bounded like
// mbar_wait, with the acquire at cluster scope.
__device__ __forceinline__ void wait_peers(uint64_t* bar, uint32_t parity, Waits& w,
                                           uint64_t limit_ns = kWaitLimitNs) {
  if (w.failed) return;
  uint64_t t0 = 0;
  for (uint32_t spin = 0;; ++spin) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2, %3;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_addr(bar)), "r"(parity), "r"(1000000u)
        : "memory");
    if (ok) return;
    if (spin == 0) t0 = global_timer_ns();
    if (*w.abort_flag || global_timer_ns() - t0 > limit_ns) {
      atomicCAS(w.err, 0, kWaitCode);
      *w.abort_flag = 1;
      w.failed = true;
      return;
    }
  }
}

// One CTA waits for peers that it does not have: the wait gives up, and so does the
// next one at once.
__global__ void wait_peers_selftest_kernel(int* err, uint64_t limit_ns) {
  __shared__ uint64_t bar;
  __shared__ int aborted;
  if (threadIdx.x == 0) {
    mbar_init(&bar, 1);
    aborted = 0;
    fence_mbarrier_init();
  }
  __syncthreads();
  Waits waits{err, &aborted, false};
  wait_peers(&bar, 0, waits, limit_ns);
  wait_peers(&bar, 0, waits, limit_ns);
}

// k = sigmoid(-f) = 1 / (1 + e) with e = exp(f), 0 once e is infinite.  Both ways
// from zero it keeps its relative precision.  With e held below infinity,
// k (1 - k) = e k^2 is 0 where k is.
__device__ __forceinline__ float ex2_approx(float x) {
  float e;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(x));
  return e;
}
__device__ __forceinline__ float rcp_approx(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float below_inf(float e) {
  asm("min.NaN.f32 %0, %0, %1;" : "+f"(e) : "f"(3.402823466e38f));
  return e;
}
__device__ __forceinline__ float take_of(float f) { return rcp_approx(1.0f + ex2_approx(1.4426950408889634f * f)); }

// (1 - k) g, with slope = k (1 - k): to a few roundings however near k is to 1.
__device__ __forceinline__ float past(float k, float slope, float g) {
  return k < 0.5f ? fmaf(-k, g, g) : slope / k * g;
}

// One step of the state.
__device__ __forceinline__ float step(float h, float k, float c) { return fmaf(k, c - h, h); }

// Two channels at once: a packed instruction takes the place of two.
__device__ __forceinline__ float2 sub2(float2 a, float2 b) { return __ffma2_rn(b, make_float2(-1.0f, -1.0f), a); }
__device__ __forceinline__ float2 step2(float2 h, float2 k, float2 c) { return __ffma2_rn(k, sub2(c, h), h); }
// R of a step after R: R + k (1 - R).
__device__ __forceinline__ float2 join2(float2 R, float2 k) {
  return __ffma2_rn(k, sub2(make_float2(1.0f, 1.0f), R), R);
}
__device__ __forceinline__ float2 take2(float2 f) {
  const float2 x = __fmul2_rn(f, make_float2(1.4426950408889634f, 1.4426950408889634f));
  const float2 e = __fadd2_rn(make_float2(ex2_approx(x.x), ex2_approx(x.y)), make_float2(1.0f, 1.0f));
  return make_float2(rcp_approx(e.x), rcp_approx(e.y));
}
__device__ __forceinline__ float2 take2(float2 f, float2& slope) {
  const float2 x = __fmul2_rn(f, make_float2(1.4426950408889634f, 1.4426950408889634f));
  const float2 e = make_float2(below_inf(ex2_approx(x.x)), below_inf(ex2_approx(x.y)));
  const float2 d = __fadd2_rn(e, make_float2(1.0f, 1.0f));
  const float2 k = make_float2(rcp_approx(d.x), rcp_approx(d.y));
  slope = __fmul2_rn(__fmul2_rn(e, k), k);
  return k;
}

// A lane's mark of a round: whether a reset stands at step t0 + lane (lane < n <= 32).
// Loaded a round ahead and in front of that round's copies, behind which it would
// come back late (8 x 2048 x 3456 backward: 132 us, against 109); the ballot of all
// lanes' is the round's resets.
__device__ __forceinline__ uint32_t reset_mark(const uint8_t* resets, int64_t at, int64_t t0, int64_t length, int n,
                                               int lane) {
  return lane < n && t0 + lane < length ? resets[at + t0 + lane] : 0u;
}

// A map (R, H) applied to a state, and the map of first (a, b), then (R, H).
// kMarks: a run that holds a reset has R = NaN, which stays NaN through every
// product and composition, and its map gives H whatever the state holds: R = 1 would
// carry an infinite or NaN state of one document into the next (0 times it), and
// is what a long run without a reset rounds to.  A gate of NaN makes H NaN too.
template <bool kMarks>
__device__ __forceinline__ float apply(float R, float H, float h) {
  const float y = fmaf(-R, h, h) + H;
  return kMarks && R != R ? H : y;
}
template <bool kMarks>
__device__ __forceinline__ void compose(float R, float H, float& a, float& b) {
  b = apply<kMarks>(R, H, b);
  a = fmaf(R, 1.0f - a, a);
}
__device__ __forceinline__ float2 forget() {
  return make_float2(__int_as_float(0x7fffffff), __int_as_float(0x7fffffff));
}

// What a CTA's warps exchange, two channels an entry: their maps (R0, H0, R1,
// H1) and the states in front of their steps.  The cluster's maps, [2][CTAs][LPR] in
// two copies used in turn, lie behind the operands' stages in dynamic shared
// memory.  A copy is free again two rounds later: a CTA sends its map of the
// round in between only behind its reads of the first, and nobody sends for the
// third without having received that.
template <int LPR>
struct Maps {
  float4 map[kWarps][LPR];
  float2 state[kWarps][LPR];
  uint64_t full[2];  // a round's maps of all the cluster's CTAs have arrived
  int aborted;
};

// Sets the barriers up; every thread of the cluster calls it.
template <int LPR>
__device__ __forceinline__ void open_maps(Maps<LPR>& m) {
  if (threadIdx.x == 0) {
    mbar_init(&m.full[0], 1);
    mbar_init(&m.full[1], 1);
    m.aborted = 0;
    fence_mbarrier_init();
  }
  __syncthreads();
  cluster_meet();  // the peers run, with their barriers, before anything is sent to them
}

// LPR lanes (two channels each) share a row of the tile, and the 32 / LPR groups
// of lanes take consecutive runs of steps; each lane has the map (R, H) of its
// run.  Returns the state in front of (behind, for kReverse) this lane's run.
// `carry`, kept by warp 0, is the state in front of the whole cluster's steps and
// becomes the state past them.  Warp 0 composes the CTA's maps, trades them
// with the cluster and steps the state from warp to warp; the others only hand
// their map in and take their state out.
template <int LPR, bool kReverse, bool kMarks>
__device__ __forceinline__ float2 exchange(Maps<LPR>& m, float4* cta, int round, int size, int rank, Waits& waits,
                                           float2 R2, float2 H2, float (&carry)[2]) {
  const float R[2] = {R2.x, R2.y}, H[2] = {H2.x, H2.y};
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int col = lane % LPR, phase = round & 1;
  // over the groups of this warp: the map before this lane's run, and of all
  float gr[2] = {}, gh[2] = {}, tr[2], th[2];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    tr[j] = R[j];
    th[j] = H[j];
    if constexpr (LPR == 16) {
      const float r2 = __shfl_xor_sync(0xffffffffu, R[j], 16), h2 = __shfl_xor_sync(0xffffffffu, H[j], 16);
      if ((lane >= 16) != kReverse) {  // the other group comes first
        gr[j] = r2;
        gh[j] = h2;
        tr[j] = r2;
        th[j] = h2;
        compose<kMarks>(R[j], H[j], tr[j], th[j]);
      } else {
        compose<kMarks>(r2, h2, tr[j], th[j]);
      }
    }
  }
  if (lane < LPR) m.map[warp][col] = make_float4(tr[0], th[0], tr[1], th[1]);
  __syncthreads();
  if (warp == 0) {
    float4 e[kWarps];
#pragma unroll
    for (int i = 0; i < kWarps; ++i) e[i] = m.map[kReverse ? kWarps - 1 - i : i][col];
    float s[2] = {carry[0], carry[1]};  // the state in front of this CTA
    if (size > 1) {
      float ar[2] = {}, ah[2] = {};
#pragma unroll
      for (int i = 0; i < kWarps; ++i) {
        compose<kMarks>(e[i].x, e[i].y, ar[0], ah[0]);
        compose<kMarks>(e[i].z, e[i].w, ar[1], ah[1]);
      }
      if (lane == 0) mbar_arrive_expect_tx(&m.full[phase], size * LPR * 16);
      float4* slots = cta + phase * size * LPR + col;
      if (lane < LPR) {
#pragma unroll
        for (int r = 0; r < kMaxCluster; ++r)
          if (r < size)
            st_async_v4(peer(slots + rank * LPR, r), __float_as_uint(ar[0]), __float_as_uint(ah[0]),
                        __float_as_uint(ar[1]), __float_as_uint(ah[1]), peer(&m.full[phase], r));
      }
      __syncwarp();
      wait_peers(&m.full[phase], (round >> 1) & 1, waits);
      float4 c[kMaxCluster];
#pragma unroll
      for (int i = 0; i < kMaxCluster; ++i)
        if (i < size) c[i] = slots[(kReverse ? size - 1 - i : i) * LPR];
#pragma unroll
      for (int i = 0; i < kMaxCluster; ++i) {
        if (i >= size) break;
        if ((kReverse ? size - 1 - i : i) == rank) {
          s[0] = carry[0];
          s[1] = carry[1];
        }
        carry[0] = apply<kMarks>(c[i].x, c[i].y, carry[0]);
        carry[1] = apply<kMarks>(c[i].z, c[i].w, carry[1]);
      }
    }
#pragma unroll
    for (int i = 0; i < kWarps; ++i) {
      if (lane < LPR) m.state[kReverse ? kWarps - 1 - i : i][col] = make_float2(s[0], s[1]);
      s[0] = apply<kMarks>(e[i].x, e[i].y, s[0]);
      s[1] = apply<kMarks>(e[i].z, e[i].w, s[1]);
    }
    if (size == 1) {
      carry[0] = s[0];
      carry[1] = s[1];
    }
  }
  __syncthreads();
  const float2 v = m.state[warp][col];
  return make_float2(apply<kMarks>(gr[0], gh[0], v.x), apply<kMarks>(gr[1], gh[1], v.y));
}

// v where the candidate or gradient of a taken token counts: 0 for k = 0.
__device__ __forceinline__ float2 masked2(float2 k, float2 v) {
  return make_float2(k.x == 0.0f ? 0.0f : v.x, k.y == 0.0f ? 0.0f : v.y);
}

// One stage of a warp's operands in shared memory: NA arrays, each the warp's
// 32 / LPR * S rows of 2 * LPR channels, copied asynchronously in pieces of CH
// bytes.  Rows and channels outside the sequence are filled with zeros.
template <class T, int LPR, int S, int NA>
struct Slab {
  static constexpr int kRow = 2 * LPR * static_cast<int>(sizeof(T));
  static constexpr int kRows = 32 / LPR * S;
  // the second group's rows lie one row further on, so that both groups' reads
  // of a step meet all banks once
  static constexpr int kSkip = LPR == 16 ? kRow : 0;
  static constexpr int kBytes = kRow * kRows + kSkip;
  uint8_t a[NA][kBytes];
};

template <int CH>
__device__ __forceinline__ void copy_async(uint8_t* dst, const void* src, bool valid) {
  const int n = valid ? CH : 0;
  if constexpr (CH == 2)  // rows of 2-byte elements on odd boundaries: a plain copy
    *reinterpret_cast<uint16_t*>(dst) = valid ? *static_cast<const uint16_t*>(src) : 0;
  else if constexpr (CH == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_addr(dst)), "l"(src), "r"(n) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(smem_addr(dst)), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Rows t0 .. of one array (row t at base + t * ld, its first channel ch0 of
// `width`) into a slab; rows outside [0, length) become zeros.
// kBare: without checks where every row and channel exists, which pays for many
// small copies (11 x 1500 x 1100 forward 35.6 us for 40.1; but 4 copies of single
// elements, 11 x 1500 x 1101 backward: 115 for 100).
template <class T, int LPR, int S, int CH, bool kBare>
__device__ __forceinline__ void load_rows(uint8_t* slab, const T* base, int64_t ld, int64_t t0, int64_t length,
                                          int64_t ch0, int64_t width, int lane) {
  constexpr int kRow = 2 * LPR * static_cast<int>(sizeof(T));
  constexpr int kPieces = (32 / LPR * S) * kRow / CH;
  static_assert(kPieces % 32 == 0, "whole rounds of pieces");
  constexpr int kEach = 32 * CH >= kRow ? 32 * CH / kRow : 1;  // rows a round of the warp's copies covers
  constexpr int kPer = 32 * CH >= kRow ? 1 : kRow / (32 * CH);  // rounds a row takes
  const int row = lane * CH / kRow, c = lane * CH % kRow / static_cast<int>(sizeof(T));
  const T* src = base + (t0 + row) * ld + c;
  if constexpr (kBare) {
    if (t0 >= 0 && t0 + 32 / LPR * S <= length && ch0 + 2 * LPR <= width) {
#pragma unroll
      for (int i = 0; i < kPieces / 32; ++i) {
        const int r = row + i / kPer * kEach;
        uint8_t* dst = slab + (i * 32 + lane) * CH + (r >= S ? kRow : 0);
        copy_async<CH>(dst, src + i % kPer * (32 * CH / static_cast<int>(sizeof(T))), true);
        if (i % kPer == kPer - 1) src += kEach * ld;
      }
      return;
    }
  }
#pragma unroll
  for (int i = 0; i < kPieces / 32; ++i) {
    const int r = row + i / kPer * kEach;
    uint8_t* dst = slab + (i * 32 + lane) * CH + (r >= S ? kRow : 0);  // r >= S: the second group
    const int64_t t = t0 + r;
    const int at = i % kPer * (32 * CH / static_cast<int>(sizeof(T)));  // channels along the row
    const bool ok = t >= 0 && t < length && ch0 + c + at < width;
    copy_async<CH>(dst, ok ? src + at : base, ok);
    if (i % kPer == kPer - 1) src += kEach * ld;
  }
}

// A lane's two channels of a tile: neighbours where one access takes both, else
// `col` and `col + LPR`, so that each access of a warp covers neighbouring elements.
template <class T, int CH> constexpr bool kPair = CH >= 2 * static_cast<int>(sizeof(T));
template <int LPR, bool kTwo> __device__ __forceinline__ int first_channel(int col) { return kTwo ? 2 * col : col; }
template <int LPR, bool kTwo> constexpr int kApart = kTwo ? 1 : LPR;

// This lane's pair of a row; `slab` is where its group's rows begin.
template <class T, int LPR, bool kTwo>
__device__ __forceinline__ float2 read_pair(const uint8_t* slab, int row, int col) {
  const T* p = reinterpret_cast<const T*>(slab) + row * (2 * LPR);
  if constexpr (kTwo) {
    float f[2];
    to_float(load<T, 2>(p + 2 * col), f);
    return make_float2(f[0], f[1]);
  } else {
    float x[1], y[1];
    to_float(load<T, 1>(p + col), x);
    to_float(load<T, 1>(p + col + LPR), y);
    return make_float2(x[0], y[0]);
  }
}

// The pair to memory, p at its first channel.
template <class T, int LPR, bool kTwo>
__device__ __forceinline__ void write_pair(T* p, float2 v, bool second) {
  if constexpr (kTwo) {
    const float f[2] = {v.x, v.y};
    store<T, 2>(p, from_float(f, T()));
  } else {
    const float lo[1] = {v.x}, hi[1] = {v.y};
    store<T, 1>(p, from_float(lo, T()));
    if (second) store<T, 1>(p + LPR, from_float(hi, T()));
  }
}

// What the steps of a lane's run have to look at.  Resets alone are common (a
// packed batch) and cost a few predicated moves a step; with everything looked at, the one
// slow warp in many rounds holds its CTA's others.
enum { kPlain, kResets, kCareful };

// A round of this lane's steps: `stage` holds them, t0 is the first, o its output.
template <class T, int LPR, int S, int CH, bool kMarks>
__device__ __forceinline__ void forward_round(const Slab<T, LPR, S, 2>& stage, int64_t t0, int64_t length, uint32_t resets,
                                              T* o, int64_t ldh, bool live, bool second, Maps<LPR>& maps,
                                              float4* cta_maps, int round, int size, int rank, Waits& waits,
                                              float (&carry)[2]) {
  using Stage = Slab<T, LPR, S, 2>;
  const int col = (threadIdx.x & 31) % LPR, group = (threadIdx.x & 31) / LPR;
  const uint8_t* sf = stage.a[0] + group * (S * Stage::kRow + Stage::kSkip);
  const uint8_t* sc = stage.a[1] + group * (S * Stage::kRow + Stage::kSkip);
  const int n = length - t0 < S ? static_cast<int>(length - t0) : S;  // steps here (may be negative)
  // A run is plain, or has resets; one that reaches past the sequence's end, or has masked
  // tokens (k = 0) whose candidate is not finite, takes the careful form.  Such a candidate
  // shows in H, at the run's end or (`gone`, their sum) where a reset clears it.
  const float2 none = make_float2(0.0f, 0.0f);
  float2 k[S], R = none, H = none, gone = none, h;
  int form = n < S ? kCareful : kMarks && resets != 0 ? kResets : kPlain;
  auto first = [&](auto how) {
    R = H = none;
#pragma unroll
    for (int i = 0; i < S; ++i) {
      const float2 f = read_pair<T, LPR, kPair<T, CH>>(sf, i, col);
      float2 c = read_pair<T, LPR, kPair<T, CH>>(sc, i, col);
      k[i] = how.value < kCareful || i < n ? take2(f) : none;
      if (how.value >= kResets && (resets >> i & 1)) {
        if (how.value == kResets) gone = __fadd2_rn(gone, H);
        R = forget();
        H = none;
      }
      if (how.value == kCareful) c = masked2(k[i], c);
      R = join2(R, k[i]);
      H = step2(H, k[i], c);
    }
  };
  if (form == kPlain)
    first(std::integral_constant<int, kPlain>());
  else if (kMarks && form == kResets)
    first(std::integral_constant<int, kResets>());
  const float2 seen = __fadd2_rn(gone, H);
  if (!(fabsf(seen.x) + fabsf(seen.y) < __int_as_float(0x7f800000))) form = kCareful;
  if (form == kCareful) first(std::integral_constant<int, kCareful>());
  h = exchange<LPR, false, kMarks>(maps, cta_maps, round, size, rank, waits, R, H, carry);
  // a masked candidate near the float limit overflows c - h where h is large, which H (from a
  // state of 0) did not show
  if (!(fabsf(h.x) + fabsf(h.y) < 1e30f)) form = kCareful;
  auto second_pass = [&](auto how) {
#pragma unroll
    for (int i = 0; i < S; ++i, o += ldh) {
      float2 c = read_pair<T, LPR, kPair<T, CH>>(sc, i, col);
      if (how.value >= kResets && (resets >> i & 1)) h = none;
      if (how.value == kCareful) c = masked2(k[i], c);
      h = step2(h, k[i], c);
      if (live && (how.value < kCareful || i < n)) write_pair<T, LPR, kPair<T, CH>>(o, h, second);
    }
  };
  if (form == kPlain)
    second_pass(std::integral_constant<int, kPlain>());
  else if (kMarks && form == kResets)
    second_pass(std::integral_constant<int, kResets>());
  else
    second_pass(std::integral_constant<int, kCareful>());
}

// CH: bytes a copy (16: rows of whole 16-byte pieces, outputs on pairs).  kMarks:
// there are resets (looking whether there are costs a call without them 1 to 4 %).  A launch
// without a cluster (size 1) executes no cluster instruction.
template <class T, int LPR, int S, int CH, bool kMarks>
__global__ void __launch_bounds__(32 * kWarps, kPerSm) scan_fwd_kernel(const FwdArgs p) {
  using Stage = Slab<T, LPR, S, 2>;
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ Maps<LPR> maps;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int col = lane % LPR, group = lane / LPR;
  const int size = static_cast<int>(cluster_size()), rank = static_cast<int>(cluster_rank());
  const int64_t tile = blockIdx.x / size;
  const int64_t b = tile / p.tiles, ch0 = (tile - b * p.tiles) * (2 * LPR), ch = ch0 + first_channel<LPR, kPair<T, CH>>(col);
  constexpr int kNext = kApart<LPR, kPair<T, CH>>;  // to the lane's second channel
  const bool live = ch < p.width, second = ch + kNext < p.width;
  const T* gate = static_cast<const T*>(p.gate) + b * p.length * p.ldg + ch0;
  const T* cand = static_cast<const T*>(p.cand) + b * p.length * p.ldc + ch0;
  T* out = static_cast<T*>(p.h) + b * p.length * p.ldh + ch;
  Stage* stages = reinterpret_cast<Stage*>(smem) + warp * 2;  // this warp's
  float4* cta_maps = reinterpret_cast<float4*>(smem + 2 * kWarps * sizeof(Stage));
  float carry[2] = {};
  launch_dependents();
  grid_dependency_wait();
  const int64_t span = static_cast<int64_t>(size) * kWarps * Stage::kRows;
  const int64_t mine = (rank * kWarps + warp) * Stage::kRows;  // this warp's rows in a span
  auto issue = [&](int64_t base, int st) {
    load_rows<T, LPR, S, CH, CH < 16>(stages[st].a[0], gate, p.ldg, base + mine, p.length, ch0, p.width, lane);
    load_rows<T, LPR, S, CH, CH < 16>(stages[st].a[1], cand, p.ldc, base + mine, p.length, ch0, p.width, lane);
    copy_commit();
  };
  issue(0, 0);
  uint32_t mark = kMarks ? reset_mark(p.resets, b * p.length, mine, p.length, Stage::kRows, lane) : 0u;
  if (p.h0 && live) {  // plain loads: h_last may be the same array
    carry[0] = p.h0[b * p.width + ch];
    if (second) carry[1] = p.h0[b * p.width + ch + kNext];
  }
  if (size > 1) open_maps(maps);
  Waits waits{p.err, &maps.aborted, false};
  int round = 0;
  for (int64_t base = 0; base < p.length; base += span, ++round) {
    const int phase = round & 1;
    const uint32_t next_mark =
        kMarks ? reset_mark(p.resets, b * p.length, base + span + mine, p.length, Stage::kRows, lane) : 0u;
    if (base + span < p.length)
      issue(base + span, phase ^ 1);
    else
      copy_commit();  // an empty group, so that waiting for all but one still means this stage
    copy_wait<1>();
    __syncwarp();
    const uint32_t resets = kMarks ? __ballot_sync(0xffffffffu, mark != 0) >> (group * S) : 0u;
    mark = next_mark;
    const int64_t t0 = base + mine + group * S;
    forward_round<T, LPR, S, CH, kMarks>(stages[phase], t0, p.length, resets, out + t0 * p.ldh, p.ldh, live, second,
                                         maps, cta_maps, round, size, rank, waits, carry);
    __syncwarp();  // this stage is read: the next round copies into it
  }
  copy_wait<0>();
  if (size > 1) cluster_meet();  // nothing is on its way to a CTA that has left
  // the carried state is past the last step; every CTA has read h0 by now
  if (p.h_last && live && rank == 0 && warp == 0 && group == 0) {
    p.h_last[b * p.width + ch] = carry[0];
    if (second) p.h_last[b * p.width + ch + kNext] = carry[1];
  }
}

// What a CTA works through: tiles `last` down to `first`, in rounds of a tile's
// [0, rounds), where the last ends in front of round `to` and the first begins
// with round `from`.
struct Work {
  int64_t first, last;
  int from, to, rounds;
};

__device__ __forceinline__ Work work_of(int64_t tiles, int64_t length, int64_t span, int size, int rank) {
  Work w;
  w.rounds = static_cast<int>((length + span - 1) / span);
  const int64_t cluster = blockIdx.x / size, clusters = gridDim.x / size;
  const int64_t t0 = tiles * cluster / clusters, n = (tiles * (cluster + 1) / clusters - t0) * w.rounds;
  const int64_t u0 = n * rank / size, u1 = n * (rank + 1) / size;
  w.first = t0 + u0 / w.rounds;
  w.last = t0 + (u1 - 1) / w.rounds;
  w.from = static_cast<int>(u0 % w.rounds);
  w.to = static_cast<int>((u1 - 1) % w.rounds) + 1;
  return w;
}

// The state at the end of a CTA's first piece to the CTA behind it, and at the
// beginning of its last piece from the one in front; warp 0, each lane its channels.
template <int LPR>
__device__ __forceinline__ void send_state(Maps<LPR>& m, float4* slots, int rank, const float (&carry)[2]) {
  const int col = (threadIdx.x & 31) % LPR;
  st_async_v4(peer(slots + col, rank + 1), __float_as_uint(carry[0]), __float_as_uint(carry[1]), 0u, 0u,
              peer(&m.full[0], rank + 1));
}
template <int LPR>
__device__ __forceinline__ void receive_state(Maps<LPR>& m, const float4* slots, Waits& waits, float (&carry)[2]) {
  if ((threadIdx.x & 31) == 0) mbar_arrive_expect_tx(&m.full[0], LPR * 16);
  __syncwarp();
  wait_peers(&m.full[0], 0, waits);
  const float4 v = slots[(threadIdx.x & 31) % LPR];
  carry[0] = v.x;
  carry[1] = v.y;
}

// For many tiles: a cluster takes consecutive tiles, at least as many as it has CTAs, and
// each of its CTAs an equal part of all their rounds: the end of one tile, whole ones, the
// beginning of another.  The beginning comes first, and its state travels once to
// the next CTA, which needs it at its own end only: nobody waits, there is no
// exchange in between, and no last wave in which most of the GPU idles (8 x 2048 x
// 2560: 42.6 us, against 53.9 with a CTA a tile).  The backward, nearer to its limit of
// instructions, loses by it (8 x 2048 x 3456: 131 us, against 108).
template <class T, int S, bool kMarks>
__global__ void __launch_bounds__(32 * kWarps, kPerSm) scan_fwd_shared_kernel(const FwdArgs p) {
  constexpr int kLanes = 32;  // tiles of 64 channels, whole 16-byte pieces
  using Stage = Slab<T, kLanes, S, 2>;
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ Maps<kLanes> maps;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int size = static_cast<int>(cluster_size()), rank = static_cast<int>(cluster_rank());
  Stage* stages = reinterpret_cast<Stage*>(smem) + warp * 2;  // this warp's
  float4* slots = reinterpret_cast<float4*>(smem + 2 * kWarps * sizeof(Stage));
  constexpr int64_t span = kWarps * Stage::kRows;
  const int64_t mine = warp * Stage::kRows;  // this warp's rows in a span
  const Work w = work_of(p.all_tiles, p.length, span, size, rank);
  int64_t b, ch0;  // of the tile
  auto issue = [&](int64_t b, int64_t ch0, int64_t base, int st) {
    const int64_t row0 = b * p.length;
    load_rows<T, kLanes, S, 16, false>(stages[st].a[0], static_cast<const T*>(p.gate) + row0 * p.ldg + ch0, p.ldg, base + mine,
                             p.length, ch0, p.width, lane);
    load_rows<T, kLanes, S, 16, false>(stages[st].a[1], static_cast<const T*>(p.cand) + row0 * p.ldc + ch0, p.ldc, base + mine,
                             p.length, ch0, p.width, lane);
    copy_commit();
  };
  auto mark_of = [&](int64_t b, int64_t base) {
    return kMarks ? reset_mark(p.resets, b * p.length, base + mine, p.length, Stage::kRows, lane) : 0u;
  };
  launch_dependents();
  grid_dependency_wait();
  int64_t tile = w.last;
  b = tile / p.tiles;
  ch0 = (tile - b * p.tiles) * (2 * kLanes);
  int r = w.first == w.last ? w.from : 0, end = w.to;
  uint32_t mark = mark_of(b, r * span);
  issue(b, ch0, r * span, 0);
  open_maps(maps);
  Waits waits{p.err, &maps.aborted, false};
  float carry[2] = {};
  int round = 0;  // of all
  for (;;) {  // a piece of a tile
    const int64_t ch = ch0 + 2 * lane;
    const bool live = ch < p.width, second = ch + 1 < p.width;
    T* out = static_cast<T*>(p.h) + b * p.length * p.ldh + ch;
    carry[0] = carry[1] = 0.0f;
    if (r > 0) {
      if (warp == 0) receive_state(maps, slots, waits, carry);
    } else if (p.h0 && live) {  // plain loads: h_last may be the same array
      carry[0] = p.h0[b * p.width + ch];
      if (second) carry[1] = p.h0[b * p.width + ch + 1];
    }
    int64_t next_b = b, next_ch0 = ch0;
    for (; r < end; ++r, ++round) {
      const int phase = round & 1;
      const int64_t base = r * span;
      uint32_t next_mark = 0;
      if (r + 1 < end) {
        next_mark = mark_of(b, base + span);
        issue(b, ch0, base + span, phase ^ 1);
      } else if (tile != w.first) {
        const bool first_of = ch0 == 0;  // of the sequence's tiles
        next_b = first_of ? b - 1 : b;
        next_ch0 = first_of ? (p.tiles - 1) * (2 * kLanes) : ch0 - 2 * kLanes;
        const int64_t next = (tile - 1 == w.first ? w.from : 0) * span;
        next_mark = mark_of(next_b, next);
        issue(next_b, next_ch0, next, phase ^ 1);
      } else {
        copy_commit();  // an empty group, so that waiting for all but one still means this stage
      }
      copy_wait<1>();
      __syncwarp();
      const uint32_t resets = kMarks ? __ballot_sync(0xffffffffu, mark != 0) : 0u;
      mark = next_mark;
      const int64_t t0 = base + mine;
      forward_round<T, kLanes, S, 16, kMarks>(stages[phase], t0, p.length, resets, out + t0 * p.ldh, p.ldh, live, second,
                                              maps, slots, round, 1, rank, waits, carry);
      __syncwarp();  // this stage is read: the next round copies into it
    }
    if (end < w.rounds) {
      if (warp == 0) send_state(maps, slots, rank, carry);
    } else if (p.h_last && live && warp == 0) {
      // the carried state is past the last step, and h0 has been read
      p.h_last[b * p.width + ch] = carry[0];
      if (second) p.h_last[b * p.width + ch + 1] = carry[1];
    }
    if (tile == w.first) break;
    --tile;
    b = next_b;
    ch0 = next_ch0;
    r = tile == w.first ? w.from : 0;
    end = w.rounds;
  }
  copy_wait<0>();
  cluster_meet();  // nothing is on its way to a CTA that has left
}

// A few tokens per sequence: a thread takes CPL channels through all of them.
template <class T, int CPL>
__global__ void __launch_bounds__(128) scan_fwd_short_kernel(const FwdArgs p) {
  const int64_t at = (static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x) * CPL;
  launch_dependents();
  grid_dependency_wait();
  if (at >= p.channels) return;
  const int64_t b = at / p.width, ch = at - b * p.width;
  const T* gate = static_cast<const T*>(p.gate) + b * p.length * p.ldg + ch;
  const T* cand = static_cast<const T*>(p.cand) + b * p.length * p.ldc + ch;
  T* out = static_cast<T*>(p.h) + b * p.length * p.ldh + ch;
  float h[CPL] = {}, k[CPL], c[CPL];
  if (p.h0) {
#pragma unroll
    for (int j = 0; j < CPL; ++j) h[j] = p.h0[at + j];
  }
#pragma unroll 4
  for (int64_t t = 0; t < p.length; ++t) {
    to_float(load<T, CPL>(gate + t * p.ldg), k);
    to_float(load<T, CPL>(cand + t * p.ldc), c);
    const bool reset = p.resets && p.resets[b * p.length + t];
#pragma unroll
    for (int j = 0; j < CPL; ++j) {
      k[j] = take_of(k[j]);
      h[j] = step(reset ? 0.0f : h[j], k[j], k[j] == 0.0f ? 0.0f : c[j]);
    }
    store<T, CPL>(out + t * p.ldh, from_float(h, T()));
  }
  if (p.h_last) {
#pragma unroll
    for (int j = 0; j < CPL; ++j) p.h_last[at + j] = h[j];
  }
}

template <class T, int LPR, int S, int CH, bool kMarks>
__global__ void __launch_bounds__(32 * kWarps, kPerSm) scan_bwd_kernel(const BwdArgs p) {
  using Stage = Slab<T, LPR, S, 4>;
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ Maps<LPR> maps;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int col = lane % LPR, group = lane / LPR;
  const int size = static_cast<int>(cluster_size()), rank = static_cast<int>(cluster_rank());
  constexpr int kNext = kApart<LPR, kPair<T, CH>>;  // to the lane's second channel
  Stage* stages = reinterpret_cast<Stage*>(smem) + warp * 2;
  float4* cta_maps = reinterpret_cast<float4*>(smem + 2 * kWarps * sizeof(Stage));
  const int64_t span = static_cast<int64_t>(size) * kWarps * Stage::kRows;
  const int64_t mine = (rank * kWarps + warp) * Stage::kRows;
  const int rounds = static_cast<int>((p.length + span - 1) / span);
  const int64_t tile = blockIdx.x / size;
  const int64_t b = tile / p.tiles, ch0 = (tile - b * p.tiles) * (2 * LPR), ch = ch0 + first_channel<LPR, kPair<T, CH>>(col);
  const bool live = ch < p.width, second = ch + kNext < p.width;
  auto issue = [&](int64_t base, int st) {  // rows in front of the sequence: zeros
    const int64_t t = base + mine, row0 = b * p.length;
    load_rows<T, LPR, S, CH, CH == 4>(stages[st].a[0], static_cast<const T*>(p.gate) + row0 * p.ldg + ch0, p.ldg, t, p.length,
                             ch0, p.width, lane);
    load_rows<T, LPR, S, CH, CH == 4>(stages[st].a[1], static_cast<const T*>(p.cand) + row0 * p.ldc + ch0, p.ldc, t, p.length,
                             ch0, p.width, lane);
    load_rows<T, LPR, S, CH, CH == 4>(stages[st].a[2], static_cast<const T*>(p.dh) + row0 * p.lddh + ch0, p.lddh, t, p.length,
                             ch0, p.width, lane);
    load_rows<T, LPR, S, CH, CH == 4>(stages[st].a[3], static_cast<const T*>(p.h) + row0 * p.ldh + ch0, p.ldh, t - 1, p.length,
                             ch0, p.width, lane);
    copy_commit();
  };
  auto mark_of = [&](int64_t base) {
    return kMarks ? reset_mark(p.resets, b * p.length, base + mine, p.length, Stage::kRows, lane) : 0u;
  };
  launch_dependents();
  grid_dependency_wait();
  const int64_t last = (rounds - 1) * span;  // round r is the r-th from the sequence's end
  uint32_t mark = 0;
  if (rounds > 0) {
    mark = mark_of(last);
    issue(last, 0);
  }
  if (size > 1) open_maps(maps);
  Waits waits{p.err, &maps.aborted, false};
  T* dgate = static_cast<T*>(p.dgate) + b * p.length * p.lddg + ch;
  T* dcand = static_cast<T*>(p.dcand) + b * p.length * p.lddc + ch;
  float carry[2] = {}, start[2] = {};
  if (live) {
    if (p.dh_last) {
      carry[0] = p.dh_last[b * p.width + ch];
      if (second) carry[1] = p.dh_last[b * p.width + ch + kNext];
    }
    if (p.h0) {
      start[0] = p.h0[b * p.width + ch];
      if (second) start[1] = p.h0[b * p.width + ch + kNext];
    }
  }
  for (int round = 0; round < rounds; ++round) {
    const int phase = round & 1;
    const int64_t base = last - round * span;
    uint32_t next_mark = 0;
    if (round + 1 < rounds) {
      next_mark = mark_of(base - span);
      issue(base - span, phase ^ 1);
    } else {
      copy_commit();  // an empty group, so that waiting for all but one still means this stage
    }
    copy_wait<1>();
    __syncwarp();
    const uint32_t resets = kMarks ? __ballot_sync(0xffffffffu, mark != 0) >> (group * S) : 0u;
    mark = next_mark;
    const int64_t t0 = base + mine + group * S;
    const Stage& st = stages[phase];
    const int at = group * (S * Stage::kRow + Stage::kSkip);
    const int n = p.length - t0 < S ? static_cast<int>(p.length - t0) : S;
    const float2 none = make_float2(0.0f, 0.0f);
    float2 k[S], slope[S], R = none, Q = none, v;
    const int form = n < S || t0 == 0 ? kCareful : kMarks && resets != 0 ? kResets : kPlain;  // either end
    // the map of (1 - k) G past these steps to the same in front of them
    auto fold = [&](auto how) {
#pragma unroll
      for (int i = S - 1; i >= 0; --i) {
        k[i] = take2(read_pair<T, LPR, kPair<T, CH>>(st.a[0] + at, i, col), slope[i]);
        if (how.value == kCareful && i >= n) k[i] = none;
        const float2 g = __fadd2_rn(read_pair<T, LPR, kPair<T, CH>>(st.a[2] + at, i, col), Q);
        R = join2(R, k[i]);
        Q = sub2(g, __fmul2_rn(k[i], g));
        if (how.value >= kResets && (resets >> i & 1)) {
          R = forget();
          Q = none;
        }
      }
    };
    if (form == kPlain)
      fold(std::integral_constant<int, kPlain>());
    else if (kMarks && form == kResets)
      fold(std::integral_constant<int, kResets>());
    else
      fold(std::integral_constant<int, kCareful>());
    v = exchange<LPR, true, kMarks>(maps, cta_maps, round, size, rank, waits, R, Q, carry);
    auto put = [&](auto how) {
      T* og = dgate + (t0 + S - 1) * p.lddg;
      T* oc = dcand + (t0 + S - 1) * p.lddc;
#pragma unroll
      for (int i = S - 1; i >= 0; --i, og -= p.lddg, oc -= p.lddc) {
        const float2 g = __fadd2_rn(read_pair<T, LPR, kPair<T, CH>>(st.a[2] + at, i, col), v);
        float2 before = read_pair<T, LPR, kPair<T, CH>>(st.a[3] + at, i, col);
        const bool reset = how.value >= kResets && (resets >> i & 1);
        if (how.value == kCareful && t0 + i == 0) before = make_float2(start[0], start[1]);
        if (reset) before = none;
        const float2 dc = __fmul2_rn(k[i], g);
        const float2 diff = sub2(before, read_pair<T, LPR, kPair<T, CH>>(st.a[1] + at, i, col));
        const float2 df = masked2(slope[i], __fmul2_rn(__fmul2_rn(g, slope[i]), diff));
        v = reset ? none : sub2(g, dc);
        if (how.value == kCareful && t0 + i == 0 && p.dh0 && live) {
          // a G leaves the sequence: with a = slope / k where 1 - k would cancel
          p.dh0[b * p.width + ch] = reset ? 0.0f : past(k[i].x, slope[i].x, g.x);
          if (second) p.dh0[b * p.width + ch + kNext] = reset ? 0.0f : past(k[i].y, slope[i].y, g.y);
        }
        if (live && (how.value < kCareful || i < n)) {
          write_pair<T, LPR, kPair<T, CH>>(og, df, second);
          write_pair<T, LPR, kPair<T, CH>>(oc, dc, second);
        }
      }
    };
    if (form == kPlain)
      put(std::integral_constant<int, kPlain>());
    else if (kMarks && form == kResets)
      put(std::integral_constant<int, kResets>());
    else
      put(std::integral_constant<int, kCareful>());
    __syncwarp();  // this stage is read: the next round copies into it
  }
  copy_wait<0>();
  if (size > 1) cluster_meet();  // nothing is on its way to a CTA that has left
  if (rounds == 0 && p.dh0 && live && rank == 0 && warp == 0 && group == 0) {  // no tokens
    p.dh0[b * p.width + ch] = carry[0];
    if (second) p.dh0[b * p.width + ch + kNext] = carry[1];
  }
}

constexpr int64_t kShort = 8;  // tokens up to which a sequence is not split
// Steps a lane holds: the operands of a stage are 2 KB an array and warp
// forward, 1 KB backward.
template <class T> constexpr int kFwdSteps = 32 / sizeof(T);
template <class T> constexpr int kBwdSteps = 16 / sizeof(T);

// By how much an estimate has to win before its kernel is taken, from 728 measurements of all
// that could run (150 sizes of 2 to 60 million elements, most drawn at random, 1 to 64 sequences of 64 to 16384
// tokens, both directions and types; a third of them again in odd rows).  Tiles of 32 channels
// fetch rows half as long, which costs most where those are 64 bytes of 16-byte copies: the
// mean time lost against the best choice is 1.8 to 2.0 % for any factor from 1.16 to 1.2
// there (4.6 % at 1, 2.7 at 1.3), and elsewhere least at 1.03 to 1.12 (1.1 %; 2.2 at 1, 3.8 at 1.3).
// Shared tiles, whose pieces depend on one another, lose 2.3 % at 1 (12 x 967 x 3464: 74 us
// for 50), 0.8 at 1.2 and 1.0 where they are never taken.
template <class T, int CH> constexpr double kNarrowGain = sizeof(T) == 2 && CH == 16 ? 1.18 : 1.08;
constexpr double kSharedGain = 1.2;

// A launch: CTAs a cluster, and its estimated time in rounds of one CTA.  All
// clusters of a wave walk their sequences side by side, `rows` steps a CTA and
// round; a round that ends in an exchange across the cluster is counted 1.15
// times one that does not, or 1.4 times where later waves keep the SMs full: how far
// the choice is off with these is said at kNarrowGain.
struct Plan {
  int cluster;
  double cost;
  int64_t clusters = 0;  // shared tiles: how many there are
};

template <auto Fn>
Plan plan(int dev, int64_t tiles, int64_t length, int rows, int smem, int per_cta) {
  Plan best{0, 0.0};
  for (int c = 1; c <= kMaxCluster; ++c) {
    if (c > 1 && (c - 1) * static_cast<int64_t>(rows) >= length) break;  // CTAs without steps
    const int n = max_clusters<Fn>(dev, c, 32 * kWarps, smem + (c > 1 ? c * per_cta : 0));
    if (n < 1) continue;
    const int64_t full = tiles / n, left = tiles % n, rounds = (length + c * rows - 1) / (c * rows);
    // a last wave that is not full has the SMs more to itself
    const double waves = static_cast<double>(full) + (left ? 0.5 + 0.5 * left / n : 0.0);
    const double cost = waves * rounds * (c == 1 ? 1.0 : waves <= 1.0 ? 1.15 : 1.4);
    if (best.cluster == 0 || cost < best.cost) best = {c, cost};
  }
  return best;
}

// The same for shared tiles, each of whose CTAs has its part of the cluster's rounds.
template <auto Fn>
Plan plan_shared(int dev, int64_t tiles, int64_t length, int rows, int smem, int per_cta) {
  Plan best{0, 0.0};
  const int64_t rounds = (length + rows - 1) / rows;
  for (int c = 2; c <= kMaxCluster; ++c) {
    const int64_t n = std::min<int64_t>(max_clusters<Fn>(dev, c, 32 * kWarps, smem + c * per_cta), tiles / c);
    if (n < 1) continue;
    const double cost = static_cast<double>((tiles + n - 1) / n) * rounds / c;
    if (best.cluster == 0 || cost < best.cost) best = {c, cost, n};
  }
  return best;
}

template <class T, int CH, bool kMarks>
struct Fwd {
  template <int LPR> struct Kernel;
};
template <class T, int CH, bool kMarks>
struct Bwd {
  template <int LPR> struct Kernel;
};
template <class T, int CH, bool kMarks>
template <int LPR>
struct Fwd<T, CH, kMarks>::Kernel {
  using Type = T;
  static constexpr bool marks = kMarks;
  static constexpr double gain = kNarrowGain<T, CH>;
  static constexpr int S = kFwdSteps<T>, rows = kWarps * (32 / LPR) * S;
  static constexpr int smem = 2 * kWarps * sizeof(Slab<T, LPR, S, 2>), per_cta = 2 * LPR * sizeof(float4);
  static constexpr auto fn = scan_fwd_kernel<T, LPR, S, CH, kMarks>;
};
template <class T, int CH, bool kMarks>
template <int LPR>
struct Bwd<T, CH, kMarks>::Kernel {
  static constexpr double gain = kNarrowGain<T, CH>;
  static constexpr int S = kBwdSteps<T>, rows = kWarps * (32 / LPR) * S;
  static constexpr int smem = 2 * kWarps * sizeof(Slab<T, LPR, S, 4>), per_cta = 2 * LPR * sizeof(float4);
  static constexpr auto fn = scan_bwd_kernel<T, LPR, S, CH, kMarks>;
};

template <class K, int LPR, class Args>
int run_plan(Args p, int64_t batch, int cluster, cudaStream_t s) {
  p.tiles = (p.width + 2 * LPR - 1) / (2 * LPR);
  return launch(K::fn, batch * p.tiles * cluster, 32 * kWarps,
                K::smem + (cluster > 1 ? cluster * K::per_cta : 0), s, cluster, p);
}

// Tiles of 64 channels, or of 32 where that is estimated to be faster: few
// channels leave the GPU short of CTAs.
template <template <int> class K, bool kTryShared, class Args>
int run(const Args& p, int64_t batch, cudaStream_t s) {
  using Wide = K<32>;
  using Narrow = K<16>;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return T3_ECUDA;
  if (dev < 0 || dev >= 64) return T3_EDEVICE;
  int st = allow_smem<Wide::fn>(dev, Wide::smem + kMaxCluster * Wide::per_cta);
  if (st == T3_OK) st = allow_smem<Narrow::fn>(dev, Narrow::smem + kMaxCluster * Narrow::per_cta);
  if (st != T3_OK) return st;
  const Plan w = plan<Wide::fn>(dev, batch * ((p.width + 63) / 64), p.length, Wide::rows, Wide::smem, Wide::per_cta);
  const Plan n = plan<Narrow::fn>(dev, batch * ((p.width + 31) / 32), p.length, Narrow::rows, Narrow::smem, Narrow::per_cta);
  if (w.cluster == 0 && n.cluster == 0) return T3_ECUDA;
  if constexpr (kTryShared) {
    constexpr auto fn = scan_fwd_shared_kernel<typename Wide::Type, Wide::S, Wide::marks>;
    st = allow_smem<fn>(dev, Wide::smem + kMaxCluster * Wide::per_cta);
    if (st != T3_OK) return st;
    Args q = p;
    q.tiles = (p.width + 63) / 64;
    q.all_tiles = batch * q.tiles;
    const Plan h = plan_shared<fn>(dev, q.all_tiles, p.length, Wide::rows, Wide::smem, Wide::per_cta);
    if (h.cluster > 0 && h.cost * kSharedGain < std::min(w.cost, n.cost * Wide::gain))
      return launch(fn, h.clusters * h.cluster, 32 * kWarps, Wide::smem + h.cluster * Wide::per_cta, s, h.cluster, q);
  }
  if (n.cluster == 0 || (w.cluster > 0 && w.cost <= Wide::gain * n.cost)) return run_plan<Wide, 32>(p, batch, w.cluster, s);
  return run_plan<Narrow, 16>(p, batch, n.cluster, s);
}

// CH 16: rows of whole 16-byte pieces; otherwise pieces of 4 bytes, or of one
// element where rows of 2-byte elements start on odd boundaries.
template <class T, bool kMarks, class Args>
int run_rows(const Args& p, int64_t batch, int ch, cudaStream_t s) {
  constexpr bool kFwd = std::is_same_v<Args, FwdArgs>;
  constexpr int kOdd = sizeof(T) == 4 ? 4 : 2;
  if constexpr (kFwd) {
    if (ch == 16) return run<Fwd<T, 16, kMarks>::template Kernel, true>(p, batch, s);
    if (ch == 4) return run<Fwd<T, 4, kMarks>::template Kernel, false>(p, batch, s);
    return run<Fwd<T, kOdd, kMarks>::template Kernel, false>(p, batch, s);
  } else {
    if (ch == 16) return run<Bwd<T, 16, kMarks>::template Kernel, false>(p, batch, s);
    if (ch == 4) return run<Bwd<T, 4, kMarks>::template Kernel, false>(p, batch, s);
    return run<Bwd<T, kOdd, kMarks>::template Kernel, false>(p, batch, s);
  }
}

template <class Args>
int run_any(const Args& p, int64_t batch, int ch, int dtype, cudaStream_t s) {
  if (dtype == T3_OUT_BF16)
    return p.resets ? run_rows<vec::bf16, true>(p, batch, ch, s) : run_rows<vec::bf16, false>(p, batch, ch, s);
  return p.resets ? run_rows<float, true>(p, batch, ch, s) : run_rows<float, false>(p, batch, ch, s);
}

// Whether every row of `width` elements at `p` with stride ld starts and ends
// on a boundary of `bytes`.
bool rows_on(const void* p, int64_t ld, int64_t width, int es, int bytes) {
  return aligned(p, bytes) && ld * es % bytes == 0 && width * es % bytes == 0;
}

}  // namespace sc

int launch_scan_wait_selftest(int* err, uint64_t limit_ns, cudaStream_t s) {
  sc::wait_peers_selftest_kernel<<<1, 32, 0, s>>>(err, limit_ns);
  return cudaGetLastError() == cudaSuccess ? T3_OK : T3_ECUDA;
}

int launch_scan_fwd(const void* gate, int64_t ldg, const void* cand, int64_t ldc, const float* h0,
                    const uint8_t* resets, void* h, int64_t ldh, float* h_last, int64_t batch,
                    int64_t length, int64_t width, int dtype, int* err, cudaStream_t s) {
  const sc::FwdArgs p{gate, cand, ldg, ldc, ldh, h0, resets, h, h_last, length, width, 0, 0, batch * width, err};
  const int es = dtype == T3_OUT_BF16 ? 2 : 4;
  auto on = [&](int n) { return sc::rows_on(gate, ldg, width, es, n) && sc::rows_on(cand, ldc, width, es, n); };
  const bool pair = sc::rows_on(h, ldh, width, es, 2 * es);
  if (length <= sc::kShort) {
    const bool two = pair && on(2 * es);
    const int64_t n = p.channels / (two ? 2 : 1);
    auto fn = dtype == T3_OUT_BF16
                  ? (two ? sc::scan_fwd_short_kernel<vec::bf16, 2> : sc::scan_fwd_short_kernel<vec::bf16, 1>)
                  : (two ? sc::scan_fwd_short_kernel<float, 2> : sc::scan_fwd_short_kernel<float, 1>);
    return vec::launch(fn, (n + 127) / 128, 128, 0, s, 1, p);
  }
  const int ch = pair && on(16) ? 16 : (pair || es == 4) && on(4) ? 4 : 2;
  return sc::run_any(p, batch, ch, dtype, s);
}

int launch_scan_bwd(const void* gate, int64_t ldg, const void* cand, int64_t ldc, const void* h,
                    int64_t ldh, const void* dh, int64_t lddh, const float* h0, const uint8_t* resets,
                    const float* dh_last, void* dgate, int64_t lddg, void* dcand, int64_t lddc,
                    float* dh0, int64_t batch, int64_t length, int64_t width, int dtype, int* err,
                    cudaStream_t s) {
  const sc::BwdArgs p{gate, cand, h, dh, ldg, ldc, ldh, lddh, lddg, lddc, h0, resets, dh_last,
                      dgate, dcand, dh0, length, width, 0, err};
  const int es = dtype == T3_OUT_BF16 ? 2 : 4;
  auto on = [&](int n) {
    return sc::rows_on(gate, ldg, width, es, n) && sc::rows_on(cand, ldc, width, es, n) &&
           sc::rows_on(h, ldh, width, es, n) && sc::rows_on(dh, lddh, width, es, n);
  };
  const bool pair = sc::rows_on(dgate, lddg, width, es, 2 * es) && sc::rows_on(dcand, lddc, width, es, 2 * es);
  const int ch = pair && on(16) ? 16 : (pair || es == 4) && on(4) ? 4 : 2;
  return sc::run_any(p, batch, ch, dtype, s);
}

}  // namespace t3
