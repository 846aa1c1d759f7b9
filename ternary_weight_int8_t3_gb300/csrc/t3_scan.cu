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
// The state is float.  The step is taken as h' + k (c - h'): k = sigmoid(-f)
// keeps its relative precision as the gate closes, where 1 - k would not, so a
// long memory is not lost to rounding.  Where k is exactly 0 (f = +inf, or a gate
// closed below the float range) the candidate is not looked at: f = +inf masks a token
// whatever its candidate holds.
//
// What bounds it: memory (bf16: 6 bytes an element forward, 12 backward), once
// there is enough work in flight; a few sequences have few channels, so time
// is split.  A step is the linear map h -> (h - R h) + H, and maps compose (R
// and not 1 - R is what is kept: products of factors near 1 would lose the
// same long memory), so:
//   * a lane holds two neighbouring channels (one where rows do not allow) over
//     S steps in registers, a warp 64 channels, a CTA of 8 warps 8 S
//     consecutive steps, and a cluster of up to 8 CTAs 64 S consecutive steps;
//   * each warp composes its S steps, the CTA's maps meet in shared memory, the
//     cluster's in every CTA's shared memory (stores to the peers, one cluster
//     barrier), each warp applies the maps before it to the carried state and
//     runs its S steps again from registers, this time with the true state;
//   * the cluster walks along the sequence; every thread carries the state.
// Everything is read once and written once, in a fixed order: the result does
// not change from call to call.  Sequences of a few tokens take one thread per
// channel pair and no exchange.
#include "t3_vec.cuh"

namespace t3 {
namespace sc {

using namespace vec;

constexpr int kWarps = 8;
constexpr int kMaxCluster = 8;

struct FwdArgs {
  const void *gate, *cand;
  int64_t ldg, ldc, ldh;
  const float* h0;
  const uint8_t* resets;
  void* h;
  float* h_last;
  int64_t length, width, tiles;
  int64_t channels;  // batch * width (short sequences)
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
  int64_t channels;
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
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// Stores two floats at `p` in the shared memory of CTA `rank` of the cluster.
__device__ __forceinline__ void store_peer(float2* p, uint32_t rank, float a, float b) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(smem_addr(p)), "r"(rank));
  asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(r), "f"(a), "f"(b) : "memory");
}

// k = sigmoid(-f) and, where asked for, k (1 - k).
__device__ __forceinline__ float take_of(float f) { return logistic(f).neg; }

// One step of the state.
__device__ __forceinline__ float step(float h, float k, float c) { return fmaf(k, c - h, h); }

// Bit i of the result: whether a reset stands at step t0 + i (i < n <= 32).
__device__ __forceinline__ uint32_t reset_bits(const uint8_t* resets, int64_t at, int64_t t0, int64_t length,
                                               int n, int lane) {
  if (!resets) return 0;
  const bool r = lane < n && t0 + lane < length && resets[at + t0 + lane] != 0;
  return __ballot_sync(0xffffffffu, r);
}

// A map (R, H) applied to a state, and the map of first (a, b), then (R, H).
__device__ __forceinline__ float apply(float R, float H, float h) { return fmaf(-R, h, h) + H; }
__device__ __forceinline__ void compose(float R, float H, float& a, float& b) {
  b = apply(R, H, b);
  a = fmaf(R, 1.0f - a, a);
}

// The maps of a CTA's warps and of the cluster's CTAs.
template <int CPL>
struct Maps {
  float2 warp[2][kWarps][32 * CPL];      // this CTA's warps
  float2 cta[2][kMaxCluster][32 * CPL];  // the cluster's CTAs
};

// Hands this warp's maps (R, H) to the cluster, applies the maps of all warps
// before this one (after it when kReverse) to `carry` and returns that state in `in`; carry
// becomes the state past the whole cluster's steps.
template <int CPL, bool kReverse>
__device__ __forceinline__ void exchange(Maps<CPL>& m, int phase, const float (&R)[CPL], const float (&H)[CPL],
                                         float (&carry)[CPL], float (&in)[CPL]) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int rank = static_cast<int>(cluster_rank()), size = static_cast<int>(cluster_size());
#pragma unroll
  for (int j = 0; j < CPL; ++j) m.warp[phase][warp][lane * CPL + j] = make_float2(R[j], H[j]);
  __syncthreads();
  if (size > 1) {
    if (warp == 0) {
#pragma unroll
      for (int j = 0; j < CPL; ++j) {
        float a = 0.0f, h = 0.0f;
#pragma unroll
        for (int i = 0; i < kWarps; ++i) {
          const float2 w = m.warp[phase][kReverse ? kWarps - 1 - i : i][lane * CPL + j];
          compose(w.x, w.y, a, h);
        }
        for (int r = 0; r < size; ++r) store_peer(&m.cta[phase][rank][lane * CPL + j], r, a, h);
      }
    }
    cluster_sync();
  }
#pragma unroll
  for (int j = 0; j < CPL; ++j) {
    float h = carry[j], mine = h;
    if (size > 1) {
      for (int i = 0; i < size; ++i) {
        const int r = kReverse ? size - 1 - i : i;
        if (r == rank) mine = h;
        const float2 w = m.cta[phase][r][lane * CPL + j];
        h = apply(w.x, w.y, h);
      }
      carry[j] = h;
      h = mine;
    }
#pragma unroll
    for (int i = 0; i < kWarps; ++i) {
      const int w = kReverse ? kWarps - 1 - i : i;
      if (w == warp) in[j] = h;
      const float2 v = m.warp[phase][w][lane * CPL + j];
      h = apply(v.x, v.y, h);
    }
    if (size == 1) carry[j] = h;
  }
}

template <class T, int CPL, int S>
__global__ void __launch_bounds__(32 * kWarps) scan_fwd_kernel(const FwdArgs p) {
  __shared__ Maps<CPL> maps;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int size = static_cast<int>(cluster_size()), rank = static_cast<int>(cluster_rank());
  const int64_t tile = blockIdx.x / size;
  const int64_t b = tile / p.tiles, ch = (tile - b * p.tiles) * (32 * CPL) + lane * CPL;
  const bool live = ch < p.width;
  const T* gate = static_cast<const T*>(p.gate) + b * p.length * p.ldg + ch;
  const T* cand = static_cast<const T*>(p.cand) + b * p.length * p.ldc + ch;
  T* out = static_cast<T*>(p.h) + b * p.length * p.ldh + ch;
  float carry[CPL] = {};
  launch_dependents();
  grid_dependency_wait();
  if (p.h0 && live) {  // plain loads: h_last may be the same array
#pragma unroll
    for (int j = 0; j < CPL; ++j) carry[j] = p.h0[b * p.width + ch + j];
  }
  if (size > 1) cluster_sync();  // the peers run before anything is stored to them
  int phase = 0;
  for (int64_t base = 0; base < p.length; base += static_cast<int64_t>(size) * kWarps * S, phase ^= 1) {
    const int64_t t0 = base + (rank * kWarps + warp) * S;
    const int n = p.length - t0 < S ? static_cast<int>(p.length - t0) : S;  // steps here (may be negative)
    Raw<T, CPL> f[S], c[S];
#pragma unroll
    for (int i = 0; i < S; ++i) {
      f[i] = zero<T, CPL>();
      c[i] = zero<T, CPL>();
      if (live && i < n) {
        f[i] = load<T, CPL>(gate + (t0 + i) * p.ldg);
        c[i] = load<T, CPL>(cand + (t0 + i) * p.ldc);
      }
    }
    const uint32_t resets = reset_bits(p.resets, b * p.length, t0, p.length, S, lane);
    float k[S][CPL], cv[CPL], R[CPL], H[CPL], h[CPL];
#pragma unroll
    for (int j = 0; j < CPL; ++j) {
      R[j] = 0.0f;
      H[j] = 0.0f;
    }
#pragma unroll
    for (int i = 0; i < S; ++i) {
      to_float(f[i], k[i]);
      to_float(c[i], cv);
#pragma unroll
      for (int j = 0; j < CPL; ++j) {
        k[i][j] = i < n ? take_of(k[i][j]) : 0.0f;
        if (resets >> i & 1) {
          R[j] = 1.0f;
          H[j] = 0.0f;
        }
        R[j] = fmaf(k[i][j], 1.0f - R[j], R[j]);
        H[j] = step(H[j], k[i][j], k[i][j] == 0.0f ? 0.0f : cv[j]);
      }
    }
    exchange<CPL, false>(maps, phase, R, H, carry, h);
#pragma unroll
    for (int i = 0; i < S; ++i) {
      to_float(c[i], cv);
#pragma unroll
      for (int j = 0; j < CPL; ++j) {
        if (resets >> i & 1) h[j] = 0.0f;
        h[j] = step(h[j], k[i][j], k[i][j] == 0.0f ? 0.0f : cv[j]);
      }
      if (live && i < n) store<T, CPL>(out + (t0 + i) * p.ldh, from_float(h, T()));
    }
  }
  // the carried state is past the last step; every CTA has read h0 by now
  if (p.h_last && live && rank == 0 && warp == 0) {
#pragma unroll
    for (int j = 0; j < CPL; ++j) p.h_last[b * p.width + ch + j] = carry[j];
  }
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

template <class T, int CPL, int S>
__global__ void __launch_bounds__(32 * kWarps) scan_bwd_kernel(const BwdArgs p) {
  __shared__ Maps<CPL> maps;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int size = static_cast<int>(cluster_size()), rank = static_cast<int>(cluster_rank());
  const int64_t tile = blockIdx.x / size;
  const int64_t b = tile / p.tiles, ch = (tile - b * p.tiles) * (32 * CPL) + lane * CPL;
  const bool live = ch < p.width;
  const int64_t row0 = b * p.length;
  const T* gate = static_cast<const T*>(p.gate) + row0 * p.ldg + ch;
  const T* cand = static_cast<const T*>(p.cand) + row0 * p.ldc + ch;
  const T* hs = static_cast<const T*>(p.h) + row0 * p.ldh + ch;
  const T* dh = static_cast<const T*>(p.dh) + row0 * p.lddh + ch;
  T* dgate = static_cast<T*>(p.dgate) + row0 * p.lddg + ch;
  T* dcand = static_cast<T*>(p.dcand) + row0 * p.lddc + ch;
  float carry[CPL] = {}, first[CPL] = {};
  launch_dependents();
  grid_dependency_wait();
  if (live) {
    if (p.dh_last) load_floats<CPL>(p.dh_last + b * p.width + ch, carry);
    if (p.h0) load_floats<CPL>(p.h0 + b * p.width + ch, first);
  }
  if (size > 1) cluster_sync();  // the peers run before anything is stored to them
  const int64_t span = static_cast<int64_t>(size) * kWarps * S;
  int phase = 0;
  for (int64_t base = (p.length - 1) / span * span; base >= 0; base -= span, phase ^= 1) {
    const int64_t t0 = base + (rank * kWarps + warp) * S;
    const int n = p.length - t0 < S ? static_cast<int>(p.length - t0) : S;
    Raw<T, CPL> f[S], c[S], hp[S], d[S];
#pragma unroll
    for (int i = 0; i < S; ++i) {
      f[i] = zero<T, CPL>();
      c[i] = zero<T, CPL>();
      hp[i] = zero<T, CPL>();
      d[i] = zero<T, CPL>();
      if (live && i < n) {
        f[i] = load<T, CPL>(gate + (t0 + i) * p.ldg);
        c[i] = load<T, CPL>(cand + (t0 + i) * p.ldc);
        d[i] = load<T, CPL>(dh + (t0 + i) * p.lddh);
        if (t0 + i > 0) hp[i] = load<T, CPL>(hs + (t0 + i - 1) * p.ldh);
      }
    }
    const uint32_t resets = reset_bits(p.resets, row0, t0, p.length, S, lane);
    float R[CPL], Q[CPL], v[CPL], fv[CPL], cv[CPL], dv[CPL], hv[CPL];
#pragma unroll
    for (int j = 0; j < CPL; ++j) {
      R[j] = 0.0f;
      Q[j] = 0.0f;
    }
    // the map of (1 - k_{t1}) G_{t1} at the end of these steps to the same at their start
#pragma unroll
    for (int i = S - 1; i >= 0; --i) {
      to_float(f[i], fv);
      to_float(d[i], dv);
#pragma unroll
      for (int j = 0; j < CPL; ++j) {
        const float k = i < n ? take_of(fv[j]) : 0.0f;
        const float g = dv[j] + Q[j];
        R[j] = fmaf(k, 1.0f - R[j], R[j]);
        Q[j] = fmaf(-k, g, g);
        if (resets >> i & 1) {
          R[j] = 1.0f;
          Q[j] = 0.0f;
        }
      }
    }
    exchange<CPL, true>(maps, phase, R, Q, carry, v);
#pragma unroll
    for (int i = S - 1; i >= 0; --i) {
      to_float(f[i], fv);
      to_float(c[i], cv);
      to_float(d[i], dv);
      to_float(hp[i], hv);
      float df[CPL], dc[CPL];
#pragma unroll
      for (int j = 0; j < CPL; ++j) {
        const Logistic s = logistic(fv[j]);
        const float k = i < n ? s.neg : 0.0f;
        const float g = dv[j] + v[j];
        const bool reset = resets >> i & 1;
        const float before = reset ? 0.0f : (t0 + i == 0 ? first[j] : hv[j]);
        dc[j] = k * g;
        df[j] = s.slope == 0.0f ? 0.0f : g * s.slope * (before - cv[j]);
        v[j] = reset ? 0.0f : fmaf(-k, g, g);
      }
      if (live && i < n) {
        store<T, CPL>(dgate + (t0 + i) * p.lddg, from_float(df, T()));
        store<T, CPL>(dcand + (t0 + i) * p.lddc, from_float(dc, T()));
      }
    }
  }
  if (p.dh0 && live && rank == 0 && warp == 0) {
#pragma unroll
    for (int j = 0; j < CPL; ++j) p.dh0[b * p.width + ch + j] = carry[j];
  }
}

// CTAs in a cluster: enough that the grid has about four CTAs an SM (the
// registers hold that many), none of them without steps.
int cluster_for(int64_t tiles, int64_t length, int steps, int sms) {
  int c = 1;
  while (c < kMaxCluster && tiles * c < 4ll * sms && length > static_cast<int64_t>(c) * kWarps * steps) c *= 2;
  return c;
}

constexpr int64_t kShort = 8;  // tokens up to which a sequence is not split
constexpr int kFwdSteps = 16, kBwdSteps = 8;

template <class T, int CPL>
int fwd(FwdArgs p, int64_t batch, int sms, cudaStream_t s) {
  if (p.length <= kShort) {
    const int64_t n = p.channels / CPL;
    return launch(scan_fwd_short_kernel<T, CPL>, (n + 127) / 128, 128, 0, s, 1, p);
  }
  p.tiles = (p.width + 32 * CPL - 1) / (32 * CPL);
  const int64_t tiles = batch * p.tiles;
  const int c = cluster_for(tiles, p.length, kFwdSteps, sms);
  return launch(scan_fwd_kernel<T, CPL, kFwdSteps>, tiles * c, 32 * kWarps, 0, s, c, p);
}

template <class T, int CPL>
int bwd(BwdArgs p, int64_t batch, int sms, cudaStream_t s) {
  p.tiles = (p.width + 32 * CPL - 1) / (32 * CPL);
  const int64_t tiles = batch * p.tiles;
  const int c = cluster_for(tiles, p.length, kBwdSteps, sms);
  return launch(scan_bwd_kernel<T, CPL, kBwdSteps>, tiles * c, 32 * kWarps, 0, s, c, p);
}

}  // namespace sc

namespace {
// Rows of pairs: every row starts on a boundary of two elements.
bool pair_rows(const void* p, int64_t ld, int es) { return ld % 2 == 0 && vec::aligned(p, 2 * es); }
}  // namespace

int launch_scan_fwd(const void* gate, int64_t ldg, const void* cand, int64_t ldc, const float* h0,
                    const uint8_t* resets, void* h, int64_t ldh, float* h_last, int64_t batch,
                    int64_t length, int64_t width, int dtype, int sms, cudaStream_t s) {
  const sc::FwdArgs p{gate, cand, ldg, ldc, ldh, h0, resets, h, h_last, length, width, 0, batch * width};
  const int es = dtype == T3_OUT_BF16 ? 2 : 4;
  const bool pairs = width % 2 == 0 && pair_rows(gate, ldg, es) && pair_rows(cand, ldc, es) && pair_rows(h, ldh, es);
  if (dtype == T3_OUT_BF16)
    return pairs ? sc::fwd<vec::bf16, 2>(p, batch, sms, s) : sc::fwd<vec::bf16, 1>(p, batch, sms, s);
  return pairs ? sc::fwd<float, 2>(p, batch, sms, s) : sc::fwd<float, 1>(p, batch, sms, s);
}

int launch_scan_bwd(const void* gate, int64_t ldg, const void* cand, int64_t ldc, const void* h,
                    int64_t ldh, const void* dh, int64_t lddh, const float* h0, const uint8_t* resets,
                    const float* dh_last, void* dgate, int64_t lddg, void* dcand, int64_t lddc,
                    float* dh0, int64_t batch, int64_t length, int64_t width, int dtype, int sms,
                    cudaStream_t s) {
  const sc::BwdArgs p{gate, cand, h, dh, ldg, ldc, ldh, lddh, lddg, lddc, h0, resets, dh_last,
                      dgate, dcand, dh0, length, width, 0, batch * width};
  const int es = dtype == T3_OUT_BF16 ? 2 : 4;
  const bool pairs = width % 2 == 0 && pair_rows(gate, ldg, es) && pair_rows(cand, ldc, es) &&
                     pair_rows(h, ldh, es) && pair_rows(dh, lddh, es) && pair_rows(dgate, lddg, es) &&
                     pair_rows(dcand, lddc, es);
  if (dtype == T3_OUT_BF16)
    return pairs ? sc::bwd<vec::bf16, 2>(p, batch, sms, s) : sc::bwd<vec::bf16, 1>(p, batch, sms, s);
  return pairs ? sc::bwd<float, 2>(p, batch, sms, s) : sc::bwd<float, 1>(p, batch, sms, s);
}

}  // namespace t3
