// t3_api.cu -- the C ABI: argument checks, the host packer, TMA descriptors,
// launches and the device error word.  See include/t3.h for the contract.
#include <cudaTypedefs.h>

#include <algorithm>
#include <atomic>
#include <cstring>
#include <mutex>

#include "t3.h"
#include "t3_internal.h"
#include "t3_linear.cuh"

namespace t3 {

// One error word per device (a __device__ variable has one instance per
// device context).  Kernels receive its address; t3_last_device_error reads
// and clears it.
__device__ int g_error_word;

PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static std::once_flag once;
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                         &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  });
  return fn;
}


bool make_u8_map_tiled(CUtensorMap* map, const void* base, int64_t rows, int64_t cols, int64_t ld,
                       int box_rows, int box_cols, bool swizzle128) {
  std::memset(map, 0, sizeof(*map));
  if (reinterpret_cast<uintptr_t>(base) % 16 != 0 || ld % 16 != 0) return false;
  auto fn = encode_fn();
  if (!fn) return false;
  cuuint64_t dims[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows)};
  cuuint64_t strides[1] = {static_cast<cuuint64_t>(ld)};
  cuuint32_t box[2] = {static_cast<cuuint32_t>(box_cols), static_cast<cuuint32_t>(box_rows)};
  cuuint32_t estr[2] = {1, 1};
  CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides,
                  box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  swizzle128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) std::memset(map, 0, sizeof(*map));
  return r == CUDA_SUCCESS;
}

bool make_i32_map_tiled(CUtensorMap* map, const void* base, int64_t rows, int64_t cols,
                        int box_rows, int box_cols, bool swizzle128) {
  std::memset(map, 0, sizeof(*map));
  if (reinterpret_cast<uintptr_t>(base) % 16 != 0 || (cols * 4) % 16 != 0) return false;
  auto fn = encode_fn();
  if (!fn) return false;
  cuuint64_t dims[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows)};
  cuuint64_t strides[1] = {static_cast<cuuint64_t>(cols * 4)};
  cuuint32_t box[2] = {static_cast<cuuint32_t>(box_cols), static_cast<cuuint32_t>(box_rows)};
  cuuint32_t estr[2] = {1, 1};
  CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_INT32, 2, const_cast<void*>(base), dims, strides,
                  box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  swizzle128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) std::memset(map, 0, sizeof(*map));
  return r == CUDA_SUCCESS;
}

// bf16 matrix [rows][cols] (cols elements of 2 bytes per row) as 16-bit
// elements, boxes of box_cols x box_rows in the 128-byte swizzle.
bool make_u16_map_tiled(CUtensorMap* map, const void* base, int64_t rows, int64_t cols,
                        int box_rows, int box_cols) {
  std::memset(map, 0, sizeof(*map));
  if (reinterpret_cast<uintptr_t>(base) % 16 != 0 || (cols * 2) % 16 != 0) return false;
  auto fn = encode_fn();
  if (!fn) return false;
  cuuint64_t dims[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows)};
  cuuint64_t strides[1] = {static_cast<cuuint64_t>(cols * 2)};
  cuuint32_t box[2] = {static_cast<cuuint32_t>(box_cols), static_cast<cuuint32_t>(box_rows)};
  cuuint32_t estr[2] = {1, 1};
  CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT16, 2, const_cast<void*>(base), dims, strides,
                  box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) std::memset(map, 0, sizeof(*map));
  return r == CUDA_SUCCESS;
}

// Output tensor map of the pair pipeline for output kind `kind` (tc2::kOutI32
// or a T3_OUT_* kind): boxes of 32 columns x 128 rows; int32 and float rows
// in the 128-byte swizzle, bf16 rows (64 bytes) unswizzled.
// per_warp: boxes of 32 x 32 as a layer's epilogue takes them, bf16 rows in the
// 64-byte swizzle (no int32 there).
// box_cols 16: boxes of 16 x 32 for two products' epilogue, float rows in the 64-byte swizzle,
// bf16 rows in the 32-byte one.
bool make_out_map(CUtensorMap* map, const void* base, int64_t rows, int64_t cols, int kind,
                  bool per_warp = false, uint32_t box_cols = 32) {
  if (kind == tc2::kOutI32) return make_i32_map_tiled(map, base, rows, cols, 128, 32, true);
  std::memset(map, 0, sizeof(*map));
  const int64_t esize = (kind == T3_OUT_BF16) ? 2 : 4;
  if (reinterpret_cast<uintptr_t>(base) % 16 != 0 || (cols * esize) % 16 != 0) return false;
  auto fn = encode_fn();
  if (!fn) return false;
  cuuint64_t dims[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows)};
  cuuint64_t strides[1] = {static_cast<cuuint64_t>(cols * esize)};
  cuuint32_t box[2] = {box_cols, per_warp ? 32u : 128u};
  cuuint32_t estr[2] = {1, 1};
  CUresult r = fn(map,
                  kind == T3_OUT_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32,
                  2, const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  box_cols == 16      ? (kind != T3_OUT_BF16 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_32B)
                  : kind != T3_OUT_BF16 ? CU_TENSOR_MAP_SWIZZLE_128B
                  : per_warp          ? CU_TENSOR_MAP_SWIZZLE_64B
                                      : CU_TENSOR_MAP_SWIZZLE_NONE,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) std::memset(map, 0, sizeof(*map));
  return r == CUDA_SUCCESS;
}

namespace {

constexpr int kMaxDevices = 64;
constexpr int64_t kMaxDim = 2147483647LL;           // TMA coordinates are int32
constexpr int64_t kMaxTernaryReduction = 16777215;  // 128 * K <= INT32_MAX
constexpr int64_t kMaxInt8Reduction = 131071;       // 16384 * M <= INT32_MAX
// What splitting a pair pipeline's last wave costs, in stages of one pair
// (~0.7 us each), fitted to measurements: the split kernel runs ~5 % slower
// per stage than the whole-tile one, and each piece ends in an accumulator
// flush that adds rather than stores, which short pieces cannot hide.  The
// zeroing grid and the dependent launch before it cost nothing measurable.
constexpr int64_t kSplitCostStages = 8;
constexpr int64_t kSmallM = 32;                     // forward rows served by the small-M path
constexpr int64_t kGemvM = 8;                       // of those, at most the rows the CUDA cores serve
constexpr int64_t kGemvSmallBytes = 4 << 20;        // packed weights up to which they serve 3..8 rows

struct DeviceInfo {
  bool ready = false;
  int status = T3_OK;
  int sms = 0;
  int* err_word = nullptr;
};

std::mutex g_mu;
DeviceInfo g_dev[kMaxDevices];

int device_info(const DeviceInfo** out) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return T3_ECUDA;
  if (dev < 0 || dev >= kMaxDevices) return T3_EDEVICE;
  std::lock_guard<std::mutex> lock(g_mu);
  DeviceInfo& d = g_dev[dev];
  if (!d.ready) {
    int major = 0, minor = 0;
    if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&d.sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
      return T3_ECUDA;
    if (major != 10 || minor != 3) {
      d.status = T3_EDEVICE;  // built for sm_103a only
    } else if (cudaGetSymbolAddress(reinterpret_cast<void**>(&d.err_word), g_error_word) !=
               cudaSuccess) {
      return T3_ECUDA;
    }
    d.ready = true;
  }
  *out = &d;
  return d.status;
}

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// One CTA waits on a barrier that nothing completes, with the pipelines' wait
// (suspend hints, abort flag, error word) but a limit of limit_ns: it must
// give up, record (10 << 8) | 2 in the error word and return.
__global__ void wait_selftest_kernel(int* err, uint64_t limit_ns) {
  __shared__ uint64_t bar;
  __shared__ int abort_flag;
  if (threadIdx.x == 0) {
    mbar_init(&bar, 1);
    abort_flag = 0;
    fence_mbarrier_init();
  }
  __syncthreads();
  if (threadIdx.x == 0)
    mbar_wait_limit(&bar, 0, &abort_flag, err, (10 << 8) | 2, limit_ns);
}

// The CTA-pair pipeline for the forward (OP = kOpFwd: act = A [M][K], weights
// packed along K) or dX (act = dY [M][N], reduction N), for operands of any
// alignment.  A scaled output kind needs bulk stores and the reduction in one
// exact chunk: otherwise it returns T3_EINVAL without launching, and the
// caller computes the exact int32 product and then t3_dequant_i32.
template <int OP>
int run_tc2(const int8_t* act, const uint8_t* Wp, void* out, int64_t M, int64_t N, int64_t K,
            cudaStream_t stream, int out_kind = tc2::kOutI32, const float* row_scale = nullptr,
            const float* col_scale = nullptr, const EpilogueArgs* epi = nullptr) {
  const DeviceInfo* dev = nullptr;
  int st = device_info(&dev);
  if (st != T3_OK) return st;
  const int64_t KB = (K + 3) / 4;
  const int64_t act_cols = (OP == kOpFwd) ? K : N;
  const int64_t out_cols = (OP == kOpFwd) ? N : K;
  CUtensorMap ma, mw, mo;
  // Operands TMA cannot address (row strides or bases not 16-byte aligned)
  // are loaded by their converters from global memory instead; an int32
  // output that cannot take bulk stores is written with plain stores.
  const bool a_ok = make_u8_map_tiled(&ma, act, M, act_cols, act_cols, 128, tc2::BK, true);
  const bool w_ok = (OP == kOpFwd)
                        ? make_u8_map_tiled(&mw, Wp, N, KB, KB, tc2::BNH, tc2::BK / 4)
                        : make_u8_map_tiled(&mw, Wp, N, KB, KB, tc2::BK, tc2::BN / 4);
  const bool out_ok = make_out_map(&mo, out, M, out_cols, out_kind, epi != nullptr);
  if (!out_ok && out_kind != tc2::kOutI32) return T3_EINVAL;  // scaled output needs bulk stores
  // a layer's epilogue also wants TMA operands, and maps of the pre-activation
  // and the residual
  tc2::ActMaps more;
  if (epi) {
    if (!a_ok || !w_ok) return T3_EINVAL;
    more.pre = more.res = mo;  // unused copies: any initialised map
    if (epi->pre && !make_out_map(&more.pre, epi->pre, M, out_cols, out_kind, true)) return T3_EINVAL;
    if (epi->residual && !make_out_map(&more.res, epi->residual, M, out_cols, out_kind, true)) return T3_EINVAL;
  }
  if (!a_ok) ma = w_ok ? mw : mo;  // unused copies: any initialised map
  if (!w_ok) mw = ma;
  if (out_kind != tc2::kOutI32 && ceil_div(act_cols, tc2::BK) > tc2::kChunkStages) return T3_EINVAL;
  tc2::Params p{};
  p.M = M;
  p.N = N;
  p.K = K;
  p.out_rows = M;
  p.out_cols = out_cols;
  p.num_stages = ceil_div(act_cols, tc2::BK);
  const int64_t tiles_r = ceil_div(M, tc2::BMP), tiles_c = ceil_div(out_cols, tc2::BN);
  if (tiles_r * tiles_c > kMaxDim) return T3_EINVAL;
  p.tiles_r = static_cast<int>(tiles_r);
  p.tiles_c = static_cast<int>(tiles_c);
  p.out = static_cast<int32_t*>(out);
  p.use_tma_out = out_ok ? 1 : 0;
  p.out_kind = out_kind;
  p.row_scale = row_scale;
  p.col_scale = col_scale;
  p.wp = Wp;
  p.kb_bytes = KB;
  p.w_tma = w_ok ? 1 : 0;
  p.w_vec4 = (KB % 4 == 0) && (reinterpret_cast<uintptr_t>(Wp) % 4 == 0);
  p.act = act;
  p.act_rows = M;
  p.act_cols = act_cols;
  p.act_vec4 = (act_cols % 4 == 0) && (reinterpret_cast<uintptr_t>(act) % 4 == 0);
  p.a_tma = a_ok ? 1 : 0;
  // the weights-from-global instantiation loads whole words only
  p.mode = (a_ok && w_ok) ? tc2::kModeTma
           : (a_ok && p.w_vec4) ? tc2::kModeWGlobal
                                : tc2::kModeAGlobal;
  p.err = dev->err_word;
  // Schedule.  Whole tiles dealt round-robin keep the busiest pair busy for
  // ceil(T / P) tiles of S stages.  Dealing only the full waves that way and
  // splitting the stages of the remaining tiles evenly over all pairs
  // (stream-K) takes floor(T / P) tiles plus ceil(rem * S / P) stages, and
  // costs the zeroing of those tiles' rows and one more partial-tile flush
  // per pair, counted as kSplitCostStages.  A scaled epilogue needs a tile's
  // whole sum, so it keeps whole tiles, and so do the global-load modes.
  const int64_t num_tiles = tiles_r * tiles_c;
  const int64_t max_pairs = std::max(dev->sms / 2, 1);
  const int64_t waves = num_tiles / max_pairs, rem = num_tiles % max_pairs;
  int64_t dp_tiles = num_tiles;
  if (out_kind == tc2::kOutI32 && p.mode == tc2::kModeTma && rem != 0) {
    const int64_t t_whole = (waves + 1) * p.num_stages;
    const int64_t t_split =
        (waves * p.num_stages + ceil_div(rem * p.num_stages, max_pairs)) * 21 / 20 +
        kSplitCostStages;
    if (t_split < t_whole) dp_tiles = waves * max_pairs;
  }
  p.dp_tiles = static_cast<int>(dp_tiles);
  const bool split = dp_tiles < num_tiles;
  if (split) {
    // the split kernel's attributes first, so that a failure there leaves the
    // output untouched
    st = (OP == kOpFwd) ? prepare_tc2_fwd() : prepare_tc2_dx();
    if (st != T3_OK) return st;
    // from the first tile row that holds a split tile to the end
    const int64_t row0 = (dp_tiles / tiles_c) * tc2::BMP;
    st = launch_zero_pdl(static_cast<int32_t*>(out) + row0 * out_cols, (M - row0) * out_cols,
                         dev->sms, stream);
    if (st != T3_OK) return st;
  }
  const int64_t pairs = split ? max_pairs : std::min(num_tiles, max_pairs);
  const int grid = static_cast<int>(2 * pairs);
  if (epi) {
    p.mode = tc2::kModeAct;
    p.epi = *epi;
    return launch_tc2_fwd_act(p, ma, mw, mo, more, grid, stream);
  }
  return (OP == kOpFwd) ? launch_tc2_fwd(p, ma, mw, mo, grid, stream)
                        : launch_tc2_dx(p, ma, mw, mo, grid, stream);
}

// Two forwards with their product in the epilogue on the CTA pairs (tc2::kModeGlu), for
// operands and outputs that TMA can address; T3_EINVAL, with nothing launched, for others.
int run_tc2_glu(const int8_t* A, const uint8_t* Wg, const uint8_t* Wu, void* C, int64_t M, int64_t N, int64_t K,
                const GluArgs& e, int out_kind, const DeviceInfo* dev, cudaStream_t stream) {
  const int64_t KB = (K + 3) / 4;
  const int64_t tiles_r = ceil_div(M, tc2::BMP), tiles_c = ceil_div(N, tc2::BNH), tiles = tiles_r * tiles_c;
  if (ceil_div(K, tc2::BK) > tc2::kChunkStages || tiles > kMaxDim) return T3_EINVAL;
  CUtensorMap ma, mw, mo;
  tc2::GluMaps more;
  if (!make_u8_map_tiled(&ma, A, M, K, K, 128, tc2::BK, true) ||
      !make_u8_map_tiled(&mw, Wg, N, KB, KB, tc2::BNH, tc2::BK / 4) ||
      !make_u8_map_tiled(&more.w2, Wu, N, KB, KB, tc2::BNH, tc2::BK / 4) ||
      !make_out_map(&mo, C, M, N, out_kind, true, 16))
    return T3_EINVAL;
  for (int i = 0; i < 2; ++i) {
    more.pre[i] = mo;  // an unused copy: any initialised map
    if (e.pre[i] && !make_out_map(&more.pre[i], e.pre[i], M, N, out_kind, true, 16)) return T3_EINVAL;
  }
  tc2::Params p{};
  p.M = M;
  p.N = N;
  p.K = K;
  p.out_rows = M;
  p.out_cols = N;
  p.num_stages = ceil_div(K, tc2::BK);
  p.tiles_r = static_cast<int>(tiles_r);
  p.tiles_c = static_cast<int>(tiles_c);
  p.use_tma_out = 1;
  p.out_kind = out_kind;
  p.row_scale = e.row_scale;
  p.w_tma = 1;
  p.a_tma = 1;
  p.mode = tc2::kModeGlu;
  p.dp_tiles = static_cast<int>(tiles);
  p.glu = e;
  p.err = dev->err_word;
  const int64_t pairs = std::min<int64_t>(tiles, std::max(dev->sms / 2, 1));
  return launch_tc2_fwd_glu(p, ma, mw, mo, more, static_cast<int>(2 * pairs), stream);
}

// The CTA-pair dW pipeline, for operands and output of any alignment.
int run_dw2(const int8_t* A, const int8_t* dY, int32_t* dW, int64_t M, int64_t N, int64_t K,
            cudaStream_t stream) {
  const DeviceInfo* dev = nullptr;
  int st = device_info(&dev);
  if (st != T3_OK) return st;
  CUtensorMap ma, mdy, mo;
  // operands TMA cannot address are loaded by the converters themselves, and
  // a dW that cannot take bulk adds gets per-element atomic adds
  const bool a_ok = make_u8_map_tiled(&ma, A, M, K, K, dw2::BK, 128);
  const bool dy_ok = make_u8_map_tiled(&mdy, dY, M, N, N, dw2::BK, 128);
  const bool out_ok = make_i32_map_tiled(&mo, dW, K, N, 128, 32, true);
  if (!a_ok) ma = dy_ok ? mdy : mo;  // unused copies: any initialised map
  if (!dy_ok) mdy = ma;
  if (!out_ok) mo = ma;
  dw2::Params p{};
  p.a = A;
  p.dy = dY;
  p.a_vec4 = (K % 4 == 0) && (reinterpret_cast<uintptr_t>(A) % 4 == 0);
  p.dy_vec4 = (N % 4 == 0) && (reinterpret_cast<uintptr_t>(dY) % 4 == 0);
  p.out = dW;
  p.use_tma_out = out_ok ? 1 : 0;
  p.global_ops = (a_ok && dy_ok) ? 0 : 1;
  p.M = M;
  p.N = N;
  p.K = K;
  p.num_stages = ceil_div(M, dw2::BK);
  const int64_t tiles_r = ceil_div(K, dw2::BMP), tiles_c = ceil_div(N, dw2::BN);
  if (tiles_r * tiles_c > kMaxDim) return T3_EINVAL;
  p.tiles_r = static_cast<int>(tiles_r);
  p.tiles_c = static_cast<int>(tiles_c);
  p.num_chunks = static_cast<int>(ceil_div(M, dw2::kChunkElems));
  p.err = dev->err_word;
  // (tile, chunk) units, dealt evenly to at most one pair per two SMs
  const int64_t units = tiles_r * tiles_c * p.num_chunks;
  const int64_t pairs = std::min<int64_t>(units, std::max(dev->sms / 2, 1));
  st = launch_zero_pdl(dW, K * N, dev->sms, stream);
  if (st != T3_OK) return st;
  return launch_dw2(p, ma, mdy, mo, static_cast<int>(2 * pairs), stream);
}

bool valid_out_kind(int kind) {
  return kind == T3_OUT_F32 || kind == T3_OUT_BF16 || kind == T3_OUT_F32_ADD;
}

// The scaled products where the pair pipeline cannot scale in its epilogue:
// the exact int32 product into `workspace` (or, for float output without
// accumulation, into the output buffer itself, converted in place), then
// the dequantization.  bf16 and "+=" outputs need the workspace.
template <class Product>
int scaled_two_pass(Product product, void* out, int64_t rows, int64_t cols, const float* row_scale,
                    const float* col_scale, int kind, int32_t* workspace, cudaStream_t stream) {
  int32_t* x = workspace ? workspace : (kind == T3_OUT_F32 ? static_cast<int32_t*>(out) : nullptr);
  if (!x) return T3_EINVAL;
  int st = product(x);
  if (st != T3_OK) return st;
  const DeviceInfo* dev = nullptr;
  st = device_info(&dev);
  if (st != T3_OK) return st;
  return launch_dequant(x, out, rows, cols, row_scale, col_scale, kind, dev->sms, stream);
}

// Products of at most this many multiply-adds run on the CUDA cores
// (t3_small.cu) when an operand's rows are not 4-byte aligned, and of at most
// an eighth of it otherwise: the CTA-pair pipelines load rows that are not
// even word-aligned byte by byte (the pages' HSLM layers, widths 243 and 729
// at 1782 rows: 15-26 us on the CUDA cores against 21-74 us), while with TMA
// or word loads they stay ahead down to a few 10^7 (the same layers padded to
// 256 and 736: 8.5-14.6 against 13-18 us).  Set with
// t3_set_small_product_limit.
std::atomic<int64_t> g_small_macs{int64_t{1} << 29};

bool small_product(int64_t a, int64_t b, int64_t c, bool aligned) {
  int64_t lim = g_small_macs.load(std::memory_order_relaxed);
  if (aligned) lim /= 8;
  return static_cast<__int128>(a) * b * c <= static_cast<__int128>(lim);
}

// Rows of `len` bytes from `base`, every one starting on a 4-byte boundary.
bool word_rows(const void* base, int64_t len) {
  return len % 4 == 0 && reinterpret_cast<uintptr_t>(base) % 4 == 0;
}

// Forwards of few rows that run on the CUDA cores: one or two rows, or up to
// eight over few weights (measured: they beat the tensor cores there; the
// tensor cores win from four rows at N = K = 8192).
bool gemv_rows(int64_t M, int64_t N, int64_t K) {
  return M <= 2 || (M <= kGemvM && N * ((K + 3) / 4) <= kGemvSmallBytes);
}

int run_small(int op, const int8_t* x, const int8_t* y, const uint8_t* wp, int32_t* out, int64_t M,
              int64_t N, int64_t K, cudaStream_t stream) {
  const DeviceInfo* dev = nullptr;
  const int st = device_info(&dev);
  if (st != T3_OK) return st;
  return launch_small(op, x, y, wp, out, M, N, K, dev->sms, stream);
}

bool bad_dims(int64_t M, int64_t N, int64_t K) {
  return M < 0 || N < 0 || K < 0 || M > kMaxDim || N > kMaxDim || K > kMaxDim;
}

// Where t3_gemm_fwd_act lays out operands whose rows are not 16-byte pieces:
// A [M][K'] and Wp [N'][K' / 4] with K' = K rounded up to 64 and N' = N to 4, and an
// int32 result [M][N'].
struct AlignedLayout {
  int64_t K, N;              // the padded sizes
  int64_t a, w, x, bytes;    // byte offsets, and all of it
};
AlignedLayout aligned_layout(int64_t M, int64_t N, int64_t K) {
  AlignedLayout l;
  l.K = ceil_div(K, 64) * 64;
  l.N = ceil_div(N, 4) * 4;
  l.a = 0;
  l.w = M * l.K;
  l.x = l.w + l.N * (l.K / 4);
  const __int128 bytes = static_cast<__int128>(l.x) + static_cast<__int128>(M) * l.N * 4;
  l.bytes = bytes > INT64_MAX ? INT64_MAX : static_cast<int64_t>(bytes);  // never fits, instead of a negative count
  return l;
}

// How t3_gemm_fwd_act takes a product: in one kernel of the routes of t3_gemm_fwd that
// can end in its epilogue; on the CTA pairs behind a layout in scratch (`room`); or as the
// int32 product in a workspace and the epilogue behind it.
enum class ActRoute { kGemv, kSmall, kFew, kPairs, kAligned, kTwoKernels };

ActRoute act_route(const int8_t* A, const uint8_t* Wp, const void* C, int64_t M, int64_t N, int64_t K,
                   const void* residual, const void* pre, int out_kind, bool room, int sms) {
  if (K == 0) return ActRoute::kTwoKernels;
  if (M <= kSmallM) {
    if (gemv_rows(M, N, K) && gemv_fits(M, N, K)) return ActRoute::kGemv;
    return small_product(M, N, K, false) && few_act_fits(M, N, K, sms) ? ActRoute::kFew : ActRoute::kTwoKernels;
  }
  const bool words = word_rows(A, K) && word_rows(Wp, (K + 3) / 4);
  if (small_product(M, N, K, words || room)) {
    if (small_act_fits(M, N, sms)) return ActRoute::kSmall;
    return few_act_fits(M, N, K, sms) ? ActRoute::kFew : ActRoute::kTwoKernels;
  }
  auto bulk = [](const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; };
  const int64_t es = out_kind == T3_OUT_BF16 ? 2 : 4;
  if (K % 64 == 0 && bulk(A) && bulk(Wp) && bulk(C) && bulk(residual) && bulk(pre) && N * es % 16 == 0 &&
      ceil_div(K, tc2::BK) <= tc2::kChunkStages && ceil_div(M, tc2::BMP) * ceil_div(N, tc2::BN) <= kMaxDim)
    return ActRoute::kPairs;
  return room ? ActRoute::kAligned : ActRoute::kTwoKernels;
}

// How t3_gemm_fwd_glu takes a product, and where its workspace holds what: operands laid out aligned
// (A [M][K'] and both weights [N'][K' / 4], K' = K rounded up to 64 and N' = N to 4) and
// the int32 results [M][N'].  An offset below 0: as the caller has it, or not needed.
struct GluPlan {
  enum Route { kGemv, kSmall, kFew, kPairs, kTwoKernels } route;
  bool aligned = false;           // kPairs: operands laid out first
  int64_t K = 0, N = 0;           // the padded sizes (kTwoKernels: the caller's)
  int64_t a = -1, w[2] = {-1, -1}, x[2] = {-1, -1};
  int64_t bytes = 0;
};

GluPlan glu_plan(const int8_t* A, const uint8_t* Wg, const uint8_t* Wu, const void* C, int64_t M, int64_t N, int64_t K,
                 const void* pre_gate, const void* pre_up, int out_kind, int sms) {
  GluPlan p;
  p.K = K;
  p.N = N;
  auto take = [&p](int64_t rows, int64_t pitch) {
    const int64_t at = p.bytes;
    const __int128 end = static_cast<__int128>(rows) * pitch + at + 255;
    p.bytes = end > INT64_MAX ? INT64_MAX : static_cast<int64_t>(end) / 256 * 256;  // never fits, instead of a negative count
    return at;
  };
  auto results = [&] {
    for (int i = 0; i < 2; ++i) p.x[i] = take(M, p.N * 4);
  };
  auto bulk = [](const void* q) { return reinterpret_cast<uintptr_t>(q) % 16 == 0; };
  const int64_t twice = 2 * N;  // columns of both products
  p.route = GluPlan::kTwoKernels;
  if (K == 0) {
    results();
    return p;
  }
  if (M <= kSmallM) {
    if (gemv_rows(M, twice, K) && gemv_fits(M, N, K))
      p.route = GluPlan::kGemv;
    else if (small_product(M, twice, K, false) && few_act_fits(M, twice, K, sms))
      p.route = GluPlan::kFew;
    else
      results();
    return p;
  }
  const int64_t KB = (K + 3) / 4, es = out_kind == T3_OUT_BF16 ? 2 : 4;
  const bool a_ok = K % 16 == 0 && bulk(A), w_ok = KB % 16 == 0 && bulk(Wg) && bulk(Wu);
  const bool out_ok = bulk(C) && bulk(pre_gate) && bulk(pre_up) && N * es % 16 == 0;
  const bool one_chunk = ceil_div(K, tc2::BK) <= tc2::kChunkStages;
  if (small_product(M, twice, K, true)) {
    if (small_act_fits(M, twice, sms)) {
      p.route = GluPlan::kSmall;
      return p;
    }
    if (few_act_fits(M, twice, K, sms))
      p.route = GluPlan::kFew;
    else
      results();
    return p;
  }
  // rows that TMA cannot address cost the pipelines several times as much as
  // laying them out once (4096 x 3456 x 1281 75 us, with K = 1280 64).  Few tiles over a long reduction are better off
  // as two split products (40 x 1280 x 16384 85 us here, 21 each), which this plan does not know.
  p.route = GluPlan::kPairs;
  p.aligned = !a_ok || !w_ok || !out_ok || !one_chunk;
  if (!p.aligned) return p;
  if (!a_ok || !w_ok) p.K = ceil_div(K, 64) * 64;
  p.N = ceil_div(N, 4) * 4;
  if (!a_ok || p.K != K) p.a = take(M, p.K);
  if (!w_ok || p.K != K)
    for (int i = 0; i < 2; ++i) p.w[i] = take(p.N, p.K / 4);
  if (!out_ok || !one_chunk) results();
  return p;
}

// Activations' element types are the output kinds that store them.
bool valid_dtype(int dtype) { return dtype == T3_OUT_F32 || dtype == T3_OUT_BF16; }
bool valid_act(int act) { return act >= T3_ACT_NONE && act <= T3_ACT_GELU; }
// Row strides so large that a row's offset in bytes could pass 63 bits.
bool bad_ld(int64_t ld) { return ld < 0 || ld > kMaxDim; }

// Sizes of linear attention: heads of 1 to kMaxHead elements, tokens of all heads countable.
bool bad_linear(int64_t batch, int64_t length, int64_t heads, int64_t dk, int64_t dv, int dtype) {
  return bad_dims(batch, length, heads) || !valid_dtype(dtype) || dk < 1 || dv < 1 || dk > lin::kMaxHead ||
         dv > lin::kMaxHead || static_cast<__int128>(batch) * heads > kMaxDim ||
         static_cast<__int128>(batch) * heads * ceil_div(length, 16) > kMaxDim;
}

// One pass of the recurrence on the kernels that take it.
int linear_pass(const lin::Args& p, bool reverse, int dtype, float* workspace, const DeviceInfo* dev, cudaStream_t s) {
  if (linear_tc_fits(p, dtype)) return launch_linear_tc(p, reverse, workspace, dev->sms, dev->err_word, s);
  return launch_linear_tokens(p, reverse, dtype, workspace, dev->sms, s);
}

// Empty reduction: the output is all zeros.
int zero_fill(int32_t* out, int64_t rows, int64_t cols, cudaStream_t s) {
  if (!out) return T3_EINVAL;
  return cudaMemsetAsync(out, 0, static_cast<size_t>(rows) * cols * sizeof(int32_t), s) ==
                 cudaSuccess
             ? T3_OK
             : T3_ECUDA;
}

}  // namespace
}  // namespace t3

using namespace t3;

extern "C" {

int t3_pack_ternary(const int8_t* w, uint8_t* wp, int64_t K, int64_t N) {
  if (K < 0 || N < 0) return T3_EINVAL;
  if (K == 0 || N == 0) return T3_OK;
  if (!w || !wp) return T3_EINVAL;
  const int64_t total = K * N;
  for (int64_t i = 0; i < total; ++i)
    if (w[i] < -1 || w[i] > 1) return T3_EVALUE;
  const int64_t KB = (K + 3) / 4;
  for (int64_t kb = 0; kb < KB; ++kb) {
    const int64_t k0 = 4 * kb;
    const int nk = static_cast<int>(K - k0 < 4 ? K - k0 : 4);
    for (int64_t n = 0; n < N; ++n) {
      uint32_t byte = 0;
      for (int j = 0; j < nk; ++j) {
        const int8_t v = w[(k0 + j) * N + n];
        const uint32_t code = v == 1 ? 1u : (v == -1 ? 2u : 0u);
        byte |= code << (2 * j);
      }
      wp[n * KB + kb] = static_cast<uint8_t>(byte);
    }
  }
  return T3_OK;
}

int t3_gemm_fwd(const int8_t* A, const uint8_t* Wp, int32_t* C, int64_t M, int64_t N, int64_t K,
                t3_stream_t stream) {
  if (bad_dims(M, N, K)) return T3_EINVAL;
  if (M == 0 || N == 0) return T3_OK;
  if (K == 0) return zero_fill(C, M, N, stream);
  if (!A || !Wp || !C) return T3_EINVAL;
  if (K > kMaxTernaryReduction) return T3_EOVERFLOW;
  if (M <= kSmallM) {
    const DeviceInfo* dev = nullptr;
    int st = device_info(&dev);
    if (st != T3_OK) return st;
    if (gemv_rows(M, N, K)) {
      st = launch_gemv_fwd(A, Wp, C, M, N, K, dev->sms, stream);
      if (st != T3_EINVAL) return st;
    }
    // packed rows the small-M kernel's TMA cannot address: it would load them
    // byte by byte in one warp
    const bool wp_tma =
        ((K + 3) / 4) % 16 == 0 && reinterpret_cast<uintptr_t>(Wp) % 16 == 0;
    if (!wp_tma && small_product(M, N, K, false))
      return run_small(1, A, nullptr, Wp, C, M, N, K, stream);
    return launch_skinny_fwd(A, Wp, C, M, N, K, dev->sms, dev->err_word, stream);
  }
  if (small_product(M, N, K, word_rows(A, K) && word_rows(Wp, (K + 3) / 4)))
    return run_small(1, A, nullptr, Wp, C, M, N, K, stream);
  return run_tc2<kOpFwd>(A, Wp, C, M, N, K, stream);
}

int t3_gemm_bwd_dx(const int8_t* dY, const uint8_t* Wp, int32_t* dX, int64_t M, int64_t N,
                   int64_t K, t3_stream_t stream) {
  if (bad_dims(M, N, K)) return T3_EINVAL;
  if (M == 0 || K == 0) return T3_OK;
  if (N == 0) return zero_fill(dX, M, K, stream);
  if (!dY || !Wp || !dX) return T3_EINVAL;
  if (N > kMaxTernaryReduction) return T3_EOVERFLOW;
  if (small_product(M, N, K, word_rows(dY, N) && word_rows(Wp, (K + 3) / 4)))
    return run_small(2, dY, nullptr, Wp, dX, M, N, K, stream);
  return run_tc2<kOpDx>(dY, Wp, dX, M, N, K, stream);
}

int t3_gemm_bwd_dw(const int8_t* A, const int8_t* dY, int32_t* dW, int64_t M, int64_t N,
                   int64_t K, t3_stream_t stream) {
  if (bad_dims(M, N, K)) return T3_EINVAL;
  if (K == 0 || N == 0) return T3_OK;
  if (M == 0) return zero_fill(dW, K, N, stream);
  if (!A || !dY || !dW) return T3_EINVAL;
  if (M > kMaxInt8Reduction) return T3_EOVERFLOW;
  if (small_product(M, N, K, word_rows(A, K) && word_rows(dY, N)))
    return run_small(3, A, dY, nullptr, dW, M, N, K, stream);
  return run_dw2(A, dY, dW, M, N, K, stream);
}

int t3_pack_ternary_device(const int8_t* w, uint8_t* wp, int64_t K, int64_t N,
                           t3_stream_t stream) {
  if (K < 0 || N < 0 || K > kMaxDim || N > kMaxDim) return T3_EINVAL;
  if (K == 0 || N == 0) return T3_OK;
  if (!w || !wp) return T3_EINVAL;
  const DeviceInfo* dev = nullptr;
  const int st = device_info(&dev);
  if (st != T3_OK) return st;
  return launch_pack_device(w, wp, K, N, dev->sms, dev->err_word, stream);
}

int t3_quantize_rows_bf16(const void* x, int8_t* q, float* row_scale, int64_t M, int64_t K,
                          t3_stream_t stream) {
  if (M < 0 || K < 0 || M > kMaxDim || K > kMaxDim) return T3_EINVAL;
  if (M == 0) return T3_OK;
  if (!row_scale || (K > 0 && (!x || !q))) return T3_EINVAL;
  const DeviceInfo* dev = nullptr;
  const int st = device_info(&dev);
  if (st != T3_OK) return st;
  return launch_quant_rows(x, q, row_scale, M, K, dev->sms, stream);
}

int t3_dequant_i32(const int32_t* x, void* out, int64_t rows, int64_t cols,
                   const float* row_scale, const float* col_scale, int out_kind,
                   t3_stream_t stream) {
  if (rows < 0 || cols < 0 || !valid_out_kind(out_kind)) return T3_EINVAL;
  if (rows == 0 || cols == 0) return T3_OK;
  if (!x || !out) return T3_EINVAL;
  if (out_kind != T3_OUT_F32 && static_cast<const void*>(x) == out) return T3_EINVAL;
  const DeviceInfo* dev = nullptr;
  const int st = device_info(&dev);
  if (st != T3_OK) return st;
  return launch_dequant(x, out, rows, cols, row_scale, col_scale, out_kind, dev->sms, stream);
}

int t3_gemm_fwd_scaled(const int8_t* A, const uint8_t* Wp, void* C, int64_t M, int64_t N,
                       int64_t K, const float* row_scale, const float* col_scale, int out_kind,
                       int32_t* workspace, t3_stream_t stream) {
  if (bad_dims(M, N, K) || !valid_out_kind(out_kind)) return T3_EINVAL;
  if (M == 0 || N == 0) return T3_OK;
  if (!C) return T3_EINVAL;
  if (K > 0 && (!A || !Wp)) return T3_EINVAL;
  if (K > kMaxTernaryReduction) return T3_EOVERFLOW;
  if (M > kSmallM && K > 0) {
    const int st = run_tc2<kOpFwd>(A, Wp, C, M, N, K, stream, out_kind, row_scale, col_scale);
    if (st != T3_EINVAL) return st;
  }
  return scaled_two_pass(
      [&](int32_t* x) { return t3_gemm_fwd(A, Wp, x, M, N, K, stream); }, C, M, N, row_scale,
      col_scale, out_kind, workspace, stream);
}

int t3_gemm_bwd_dx_scaled(const int8_t* dY, const uint8_t* Wp, void* dX, int64_t M, int64_t N,
                          int64_t K, const float* row_scale, const float* col_scale, int out_kind,
                          int32_t* workspace, t3_stream_t stream) {
  if (bad_dims(M, N, K) || !valid_out_kind(out_kind)) return T3_EINVAL;
  if (M == 0 || K == 0) return T3_OK;
  if (!dX) return T3_EINVAL;
  if (N > 0 && (!dY || !Wp)) return T3_EINVAL;
  if (N > kMaxTernaryReduction) return T3_EOVERFLOW;
  if (N > 0) {
    const int st = run_tc2<kOpDx>(dY, Wp, dX, M, N, K, stream, out_kind, row_scale, col_scale);
    if (st != T3_EINVAL) return st;
  }
  return scaled_two_pass(
      [&](int32_t* x) { return t3_gemm_bwd_dx(dY, Wp, x, M, N, K, stream); }, dX, M, K,
      row_scale, col_scale, out_kind, workspace, stream);
}

int t3_gemm_bwd_dw_scaled(const int8_t* A, const int8_t* dY, void* dW, int64_t M, int64_t N,
                          int64_t K, const float* row_scale, const float* col_scale, int out_kind,
                          int32_t* workspace, t3_stream_t stream) {
  if (bad_dims(M, N, K) || !valid_out_kind(out_kind)) return T3_EINVAL;
  if (K == 0 || N == 0) return T3_OK;
  if (!dW) return T3_EINVAL;
  if (M > 0 && (!A || !dY)) return T3_EINVAL;
  if (M > kMaxInt8Reduction) return T3_EOVERFLOW;
  return scaled_two_pass(
      [&](int32_t* x) { return t3_gemm_bwd_dw(A, dY, x, M, N, K, stream); }, dW, K, N, row_scale,
      col_scale, out_kind, workspace, stream);
}

int64_t t3_colsum_workspace(int64_t rows, int64_t cols) {
  if (rows <= 0 || cols <= 0 || rows > kMaxDim || cols > kMaxDim) return 0;
  return std::min<int64_t>(rows, kMaxColParts) * cols;
}

int t3_rmsnorm_quant(const void* x, int64_t ldx, const void* residual, int64_t ldr,
                     const float* gamma, float eps, int8_t* q, float* row_scale, float* rstd,
                     void* sum_out, int64_t lds, int64_t rows, int64_t cols, int dtype,
                     t3_stream_t stream) {
  if (bad_dims(rows, cols, 0) || !valid_dtype(dtype) || bad_ld(ldx) || (residual && bad_ld(ldr)) ||
      (sum_out && (bad_ld(lds) || lds < cols)) || !(eps > 0.0f) || !(eps <= 3.4028234e38f))
    return T3_EINVAL;
  if (rows == 0) return T3_OK;
  if (!row_scale || (cols > 0 && (!x || !q))) return T3_EINVAL;
  const DeviceInfo* dev = nullptr;
  const int st = device_info(&dev);
  if (st != T3_OK) return st;
  return launch_norm_fwd(x, ldx, residual, ldr, gamma, eps, q, row_scale, rstd, sum_out, lds, rows, cols,
                         dtype, dev->sms, stream);
}

int t3_rmsnorm_bwd(const void* dy, int64_t lddy, const void* s, int64_t lds, const float* rstd,
                   const float* gamma, const void* dsum, int64_t lddsum, void* dx, int64_t lddx,
                   float* dgamma, int64_t rows, int64_t cols, int dtype, float* workspace,
                   t3_stream_t stream) {
  if (bad_dims(rows, cols, 0) || !valid_dtype(dtype) || bad_ld(lddy) || bad_ld(lds) ||
      (dsum && bad_ld(lddsum)) || bad_ld(lddx) || (rows > 1 && lddx < cols))
    return T3_EINVAL;
  if (cols == 0) return T3_OK;
  if (rows == 0) return dgamma ? zero_fill(reinterpret_cast<int32_t*>(dgamma), 1, cols, stream) : T3_OK;
  if (!dy || !s || !rstd || !dx || (dgamma && !workspace)) return T3_EINVAL;
  const DeviceInfo* dev = nullptr;
  const int st = device_info(&dev);
  if (st != T3_OK) return st;
  return launch_norm_bwd(dy, lddy, s, lds, rstd, gamma, dsum, lddsum, dx, lddx, dgamma, rows, cols, dtype,
                         workspace, dev->sms, stream);
}

int t3_layernorm_quant(const void* x, int64_t ldx, const void* residual, int64_t ldr, const float* gamma,
                       const float* beta, float eps, int8_t* q, float* row_scale, float* mean, float* rstd,
                       void* sum_out, int64_t lds, int64_t rows, int64_t cols, int dtype, t3_stream_t stream) {
  if (bad_dims(rows, cols, 0) || !valid_dtype(dtype) || bad_ld(ldx) || (residual && bad_ld(ldr)) ||
      (sum_out && (bad_ld(lds) || lds < cols)) || !(eps > 0.0f) || !(eps <= 3.4028234e38f))
    return T3_EINVAL;
  if (rows == 0) return T3_OK;
  if (!row_scale || (cols > 0 && (!x || !q))) return T3_EINVAL;
  const DeviceInfo* dev = nullptr;
  const int st = device_info(&dev);
  if (st != T3_OK) return st;
  return launch_layernorm_fwd(x, ldx, residual, ldr, gamma, beta, eps, q, row_scale, mean, rstd, sum_out, lds, rows,
                              cols, dtype, dev->sms, stream);
}

int t3_layernorm_bwd(const void* dy, int64_t lddy, const void* s, int64_t lds, const float* mean, const float* rstd,
                     const float* gamma, const void* dsum, int64_t lddsum, void* dx, int64_t lddx, float* dgamma,
                     float* dbeta, int64_t rows, int64_t cols, int dtype, float* workspace, t3_stream_t stream) {
  if (bad_dims(rows, cols, 0) || !valid_dtype(dtype) || bad_ld(lddy) || bad_ld(lds) ||
      (dsum && bad_ld(lddsum)) || bad_ld(lddx) || (rows > 1 && lddx < cols) || (dgamma && dgamma == dbeta))
    return T3_EINVAL;
  if (cols == 0) return T3_OK;
  if (rows == 0) {
    const int st = dgamma ? zero_fill(reinterpret_cast<int32_t*>(dgamma), 1, cols, stream) : T3_OK;
    return st == T3_OK && dbeta ? zero_fill(reinterpret_cast<int32_t*>(dbeta), 1, cols, stream) : st;
  }
  if (!dy || !s || !mean || !rstd || !dx || ((dgamma || dbeta) && !workspace)) return T3_EINVAL;
  const DeviceInfo* dev = nullptr;
  const int st = device_info(&dev);
  if (st != T3_OK) return st;
  return launch_layernorm_bwd(dy, lddy, s, lds, mean, rstd, gamma, dsum, lddsum, dx, lddx, dgamma, dbeta, rows, cols,
                              dtype, workspace, dev->sms, stream);
}

int t3_gated_scan_fwd(const void* gate, int64_t ldg, const void* cand, int64_t ldc,
                      const float* h0, const uint8_t* resets, void* h, int64_t ldh, float* h_last,
                      int64_t batch, int64_t length, int64_t width, int dtype, t3_stream_t stream) {
  if (bad_dims(batch, length, width) || !valid_dtype(dtype) || bad_ld(ldg) || bad_ld(ldc) || bad_ld(ldh) ||
      ldh < width)
    return T3_EINVAL;
  if (batch == 0 || width == 0) return T3_OK;
  if (length > 0 && (!gate || !cand || !h)) return T3_EINVAL;
  if (length == 0 && !h_last) return T3_OK;
  const DeviceInfo* dev = nullptr;
  const int st = device_info(&dev);
  if (st != T3_OK) return st;
  return launch_scan_fwd(gate, ldg, cand, ldc, h0, resets, h, ldh, h_last, batch, length, width, dtype,
                         dev->err_word, stream);
}

int t3_gated_scan_bwd(const void* gate, int64_t ldg, const void* cand, int64_t ldc, const void* h,
                      int64_t ldh, const void* dh, int64_t lddh, const float* h0,
                      const uint8_t* resets, const float* dh_last, void* dgate, int64_t lddg,
                      void* dcand, int64_t lddc, float* dh0, int64_t batch, int64_t length,
                      int64_t width, int dtype, t3_stream_t stream) {
  if (bad_dims(batch, length, width) || !valid_dtype(dtype) || bad_ld(ldg) || bad_ld(ldc) || bad_ld(ldh) ||
      bad_ld(lddh) || bad_ld(lddg) || bad_ld(lddc) || lddg < width || lddc < width)
    return T3_EINVAL;
  if (batch == 0 || width == 0) return T3_OK;
  if (length > 0 && (!gate || !cand || !h || !dh || !dgate || !dcand)) return T3_EINVAL;
  if (length == 0 && !dh0) return T3_OK;
  const DeviceInfo* dev = nullptr;
  const int st = device_info(&dev);
  if (st != T3_OK) return st;
  return launch_scan_bwd(gate, ldg, cand, ldc, h, ldh, dh, lddh, h0, resets, dh_last, dgate, lddg, dcand, lddc,
                         dh0, batch, length, width, dtype, dev->err_word, stream);
}

int64_t t3_gemm_fwd_act_scratch(int64_t M, int64_t N, int64_t K) {
  if (bad_dims(M, N, K) || M <= kSmallM || N == 0 || K == 0 || (K % 64 == 0 && N % 8 == 0)) return 0;
  return aligned_layout(M, N, K).bytes;
}

int64_t t3_gemm_fwd_act_workspace(const int8_t* A, const uint8_t* Wp, const void* C, int64_t M, int64_t N,
                                  int64_t K, const void* residual, const void* pre, int out_kind,
                                  int64_t scratch_bytes) {
  if (bad_dims(M, N, K) || M == 0 || N == 0 || out_kind != T3_OUT_BF16) return 0;
  const DeviceInfo* dev = nullptr;
  const int st = device_info(&dev);
  if (st != T3_OK) return st;
  const bool room = scratch_bytes >= aligned_layout(M, N, K).bytes;
  return act_route(A, Wp, C, M, N, K, residual, pre, out_kind, room, dev->sms) == ActRoute::kTwoKernels ? M * N : 0;
}

int64_t t3_gemm_fwd_act_scratch_now(int64_t M, int64_t N, int64_t K) {
  const int64_t bytes = t3_gemm_fwd_act_scratch(M, N, K);
  return bytes > 0 && small_product(M, N, K, true) ? 0 : bytes;
}

int t3_gemm_fwd_act(const int8_t* A, const uint8_t* Wp, void* C, int64_t M, int64_t N, int64_t K,
                    const float* row_scale, const float* col_scale, const float* bias, int act,
                    const void* residual, void* pre, int out_kind, int32_t* workspace, void* scratch,
                    int64_t scratch_bytes, t3_stream_t stream) {
  if (bad_dims(M, N, K) || !valid_dtype(out_kind) || !valid_act(act) || scratch_bytes < 0) return T3_EINVAL;
  if (M == 0 || N == 0) return T3_OK;
  if (!C || (K > 0 && (!A || !Wp)) || C == residual || C == pre || (pre && pre == residual) ||
      (out_kind == T3_OUT_BF16 && workspace == C))
    return T3_EINVAL;
  if (K > kMaxTernaryReduction) return T3_EOVERFLOW;
  const EpilogueArgs e{row_scale, col_scale, bias, residual, pre, act};
  const DeviceInfo* dev = nullptr;
  int st = device_info(&dev);
  if (st != T3_OK) return st;
  const AlignedLayout lay = aligned_layout(M, N, K);
  const bool room = scratch && scratch_bytes >= lay.bytes && reinterpret_cast<uintptr_t>(scratch) % 16 == 0;
  st = T3_EINVAL;
  switch (act_route(A, Wp, C, M, N, K, residual, pre, out_kind, room, dev->sms)) {
    case ActRoute::kGemv: st = launch_gemv_fwd_act(A, Wp, C, e, out_kind, M, N, K, dev->sms, stream); break;
    case ActRoute::kSmall: st = launch_small_act(A, Wp, C, e, out_kind, M, N, K, stream); break;
    case ActRoute::kFew: st = launch_few_act(A, Wp, C, e, out_kind, M, N, K, stream); break;
    case ActRoute::kPairs:
      st = run_tc2<kOpFwd>(A, Wp, C, M, N, K, stream, out_kind, row_scale, col_scale, &e);
      break;
    case ActRoute::kAligned: {
      // rows that TMA cannot address cost the pipelines several times as much as
      // laying them out once: operands padded with zeros to whole 64-element
      // groups, and an int32 result of whole 16-byte rows where C, residual or pre are not
      const bool tma = K % 64 == 0 && reinterpret_cast<uintptr_t>(A) % 16 == 0 && reinterpret_cast<uintptr_t>(Wp) % 16 == 0;
      uint8_t* base = static_cast<uint8_t*>(scratch);
      const int8_t* A2 = tma ? A : reinterpret_cast<int8_t*>(base + lay.a);
      uint8_t* W2 = base + lay.w;
      st = launch_align_rows(tma ? nullptr : reinterpret_cast<const uint8_t*>(A), M, K, base + lay.a, M, lay.K, Wp, N,
                             (K + 3) / 4, W2, lay.N, lay.K / 4, stream);
      if (st != T3_OK) return st;
      st = tma ? T3_EINVAL : run_tc2<kOpFwd>(A2, W2, C, M, N, lay.K, stream, out_kind, row_scale, col_scale, &e);
      if (st == T3_EINVAL) {
        int32_t* x = reinterpret_cast<int32_t*>(base + lay.x);
        st = run_tc2<kOpFwd>(A2, W2, x, M, lay.N, lay.K, stream);
        if (st == T3_OK) st = launch_epilogue(x, lay.N, C, e, M, N, out_kind, dev->sms, stream);
      }
      break;
    }
    case ActRoute::kTwoKernels: break;
  }
  if (st != T3_EINVAL) return st;
  int32_t* x = workspace ? workspace : (out_kind == T3_OUT_F32 ? static_cast<int32_t*>(C) : nullptr);
  if (!x) return T3_EINVAL;
  st = t3_gemm_fwd(A, Wp, x, M, N, K, stream);
  if (st != T3_OK) return st;
  return launch_epilogue(x, N, C, e, M, N, out_kind, dev->sms, stream);
}

int t3_act_bwd(const void* dy, const void* z, int act, void* dz, float* dbias, int64_t rows,
               int64_t cols, int dtype, float* workspace, t3_stream_t stream) {
  if (bad_dims(rows, cols, 0) || !valid_dtype(dtype) || !valid_act(act)) return T3_EINVAL;
  if (cols == 0 || (!dz && !dbias)) return T3_OK;
  if (rows == 0) return dbias ? zero_fill(reinterpret_cast<int32_t*>(dbias), 1, cols, stream) : T3_OK;
  if (!dy || (act != T3_ACT_NONE && !z) || (dbias && !workspace)) return T3_EINVAL;
  const DeviceInfo* dev = nullptr;
  const int st = device_info(&dev);
  if (st != T3_OK) return st;
  return launch_act_bwd(dy, z, act, dz, dbias, rows, cols, dtype, workspace, dev->sms, stream);
}

int64_t t3_gemm_fwd_glu_workspace(const int8_t* A, const uint8_t* Wg, const uint8_t* Wu, const void* C, int64_t M,
                                  int64_t N, int64_t K, const void* pre_gate, const void* pre_up, int out_kind) {
  if (bad_dims(M, N, K) || M == 0 || N == 0 || !valid_dtype(out_kind)) return 0;
  const DeviceInfo* dev = nullptr;
  const int st = device_info(&dev);
  if (st != T3_OK) return st;
  return glu_plan(A, Wg, Wu, C, M, N, K, pre_gate, pre_up, out_kind, dev->sms).bytes;
}

int t3_gemm_fwd_glu(const int8_t* A, const uint8_t* Wg, const uint8_t* Wu, void* C, int64_t M, int64_t N, int64_t K,
                    const float* row_scale, const float* gate_scale, const float* up_scale, const float* gate_bias,
                    const float* up_bias, int act, void* pre_gate, void* pre_up, int out_kind, void* workspace,
                    int64_t workspace_bytes, t3_stream_t stream) {
  if (bad_dims(M, N, K) || !valid_dtype(out_kind) || !valid_act(act) || workspace_bytes < 0) return T3_EINVAL;
  if (M == 0 || N == 0) return T3_OK;
  if (!C || (K > 0 && (!A || !Wg || !Wu)) || C == pre_gate || C == pre_up || (pre_gate && pre_gate == pre_up) ||
      (workspace && (workspace == C || workspace == pre_gate || workspace == pre_up)))
    return T3_EINVAL;
  if (K > kMaxTernaryReduction) return T3_EOVERFLOW;
  const GluArgs e{row_scale, {gate_scale, up_scale}, {gate_bias, up_bias}, {pre_gate, pre_up}, act};
  const DeviceInfo* dev = nullptr;
  int st = device_info(&dev);
  if (st != T3_OK) return st;
  const GluPlan p = glu_plan(A, Wg, Wu, C, M, N, K, pre_gate, pre_up, out_kind, dev->sms);
  if (p.bytes > 0 && (!workspace || workspace_bytes < p.bytes || reinterpret_cast<uintptr_t>(workspace) % 16 != 0))
    return T3_EINVAL;
  uint8_t* base = static_cast<uint8_t*>(workspace);
  int32_t* x[2] = {nullptr, nullptr};
  for (int i = 0; i < 2; ++i)
    if (p.x[i] >= 0) x[i] = reinterpret_cast<int32_t*>(base + p.x[i]);
  switch (p.route) {
    case GluPlan::kGemv: return launch_gemv_fwd_glu(A, Wg, Wu, C, e, out_kind, M, N, K, dev->sms, stream);
    case GluPlan::kSmall: return launch_small_glu(A, Wg, Wu, C, e, out_kind, M, N, K, stream);
    case GluPlan::kFew: return launch_few_glu(A, Wg, Wu, C, e, out_kind, M, N, K, stream);
    case GluPlan::kPairs: {
      const int8_t* A2 = p.a >= 0 ? reinterpret_cast<const int8_t*>(base + p.a) : A;
      const uint8_t* w[2] = {p.w[0] >= 0 ? base + p.w[0] : Wg, p.w[1] >= 0 ? base + p.w[1] : Wu};
      if (p.w[0] >= 0) {
        const int64_t KB = (K + 3) / 4;
        st = launch_align_rows(p.a >= 0 ? reinterpret_cast<const uint8_t*>(A) : nullptr, M, K, base + p.a, M, p.K, Wg,
                               N, KB, base + p.w[0], p.N, p.K / 4, stream);
        if (st == T3_OK)
          st = launch_align_rows(nullptr, 0, 0, nullptr, 0, 16, Wu, N, KB, base + p.w[1], p.N, p.K / 4, stream);
      } else if (p.a >= 0) {
        st = launch_align_rows(nullptr, 0, 0, nullptr, 0, 16, reinterpret_cast<const uint8_t*>(A), M, K, base + p.a, M,
                               p.K, stream);
      }
      if (st != T3_OK) return st;
      if (!x[0]) return run_tc2_glu(A2, w[0], w[1], C, M, N, p.K, e, out_kind, dev, stream);
      // weights laid out have rows of zeros up to N'; the caller's have N
      const int64_t n = p.w[0] >= 0 ? p.N : N;
      for (int i = 0; i < 2 && st == T3_OK; ++i) st = run_tc2<kOpFwd>(A2, w[i], x[i], M, n, p.K, stream);
      return st != T3_OK ? st : launch_glu_epilogue(x[0], x[1], n, C, e, M, N, out_kind, dev->sms, stream);
    }
    case GluPlan::kTwoKernels: break;
  }
  st = t3_gemm_fwd(A, Wg, x[0], M, N, K, stream);
  if (st == T3_OK) st = t3_gemm_fwd(A, Wu, x[1], M, N, K, stream);
  return st != T3_OK ? st : launch_glu_epilogue(x[0], x[1], N, C, e, M, N, out_kind, dev->sms, stream);
}

int t3_glu_bwd(const void* dy, const void* gate, const void* up, int act, void* dgate, void* dup, float* dgate_bias,
               float* dup_bias, int64_t rows, int64_t cols, int dtype, float* workspace, t3_stream_t stream) {
  if (bad_dims(rows, cols, 0) || !valid_dtype(dtype) || !valid_act(act) || (dgate && dgate == dup) ||
      (dgate_bias && dgate_bias == dup_bias))
    return T3_EINVAL;
  if (cols == 0 || (!dgate && !dup && !dgate_bias && !dup_bias)) return T3_OK;
  if (rows == 0) {
    const int st = dgate_bias ? zero_fill(reinterpret_cast<int32_t*>(dgate_bias), 1, cols, stream) : T3_OK;
    return st == T3_OK && dup_bias ? zero_fill(reinterpret_cast<int32_t*>(dup_bias), 1, cols, stream) : st;
  }
  if (!dy || !gate || !up || ((dgate_bias || dup_bias) && !workspace)) return T3_EINVAL;
  const DeviceInfo* dev = nullptr;
  const int st = device_info(&dev);
  if (st != T3_OK) return st;
  return launch_glu_bwd(dy, gate, up, act, dgate, dup, dgate_bias, dup_bias, rows, cols, dtype, workspace, dev->sms,
                        stream);
}

int64_t t3_linear_attn_workspace(int64_t batch, int64_t length, int64_t heads, int64_t dk, int64_t dv) {
  return bad_linear(batch, length, heads, dk, dv, T3_OUT_BF16) ? 0 : linear_workspace(batch * heads, length, dk, dv);
}

int t3_linear_attn_fwd(const void* q, int64_t ldq, const void* k, int64_t ldk, const void* v, int64_t ldv,
                       const float* log_decay, const float* state, const uint8_t* resets, float scale, void* o,
                       int64_t ldo, float* state_last, int64_t batch, int64_t length, int64_t heads, int64_t dk,
                       int64_t dv, int dtype, float* workspace, t3_stream_t stream) {
  if (bad_linear(batch, length, heads, dk, dv, dtype) || bad_ld(ldq) || bad_ld(ldk) || bad_ld(ldv) || bad_ld(ldo) ||
      ldo < heads * dv)
    return T3_EINVAL;
  if (batch == 0 || heads == 0) return T3_OK;
  const int64_t state_bytes = batch * heads * dk * dv * static_cast<int64_t>(sizeof(float));
  if (length > 0 && (!q || !k || !v || !o || !log_decay || o == q || o == k || o == v)) return T3_EINVAL;
  const DeviceInfo* dev = nullptr;
  const int st = device_info(&dev);
  if (st != T3_OK) return st;
  if (length == 0) {  // the state stays
    if (!state_last || state_last == state) return T3_OK;
    const cudaError_t e = state ? cudaMemcpyAsync(state_last, state, state_bytes, cudaMemcpyDeviceToDevice, stream)
                                : cudaMemsetAsync(state_last, 0, state_bytes, stream);
    return e == cudaSuccess ? T3_OK : T3_ECUDA;
  }
  lin::Args p{};
  p.q = q, p.k = k, p.v = v, p.o = o;
  p.ldq = ldq, p.ldk = ldk, p.ldv = ldv, p.ldo = ldo;
  p.log_decay = log_decay;
  p.init = state;
  p.resets = resets;
  p.in_scale = 1.0f, p.out_scale = scale;
  p.last = state_last;
  p.length = length, p.heads = heads, p.pairs = batch * heads;
  p.dk = static_cast<int>(dk), p.dv = static_cast<int>(dv);
  return linear_pass(p, false, dtype, workspace, dev, stream);
}

int t3_linear_attn_bwd(const void* q, int64_t ldq, const void* k, int64_t ldk, const void* v, int64_t ldv,
                       const void* dout, int64_t lddo, const float* log_decay, const float* state,
                       const uint8_t* resets, float scale, const float* dstate_last, void* dq, int64_t lddq, void* dk_out,
                       int64_t lddk, void* dv_out, int64_t lddv, float* dstate, int64_t batch, int64_t length,
                       int64_t heads, int64_t dk, int64_t dv, int dtype, float* workspace, t3_stream_t stream) {
  if (bad_linear(batch, length, heads, dk, dv, dtype) || bad_ld(ldq) || bad_ld(ldk) || bad_ld(ldv) || bad_ld(lddo) ||
      bad_ld(lddq) || bad_ld(lddk) || bad_ld(lddv) || lddq < heads * dk || lddk < heads * dk || lddv < heads * dv)
    return T3_EINVAL;
  if (batch == 0 || heads == 0) return T3_OK;
  if (length > 0) {
    if (!q || !k || !v || !dout || !log_decay || !dq || !dk_out || !dv_out) return T3_EINVAL;
    for (const void* g : {dq, dk_out, dv_out})  // each pass reads what another one's gradient would lie over
      if (g == q || g == k || g == v || g == dout) return T3_EINVAL;
    if (dq == dk_out || dq == dv_out || dk_out == dv_out) return T3_EINVAL;
  }
  const DeviceInfo* dev = nullptr;
  int st = device_info(&dev);
  if (st != T3_OK) return st;
  const int64_t state_bytes = batch * heads * dk * dv * static_cast<int64_t>(sizeof(float));
  if (length == 0) {
    if (!dstate || dstate == dstate_last) return T3_OK;
    const cudaError_t e = dstate_last ? cudaMemcpyAsync(dstate, dstate_last, state_bytes, cudaMemcpyDeviceToDevice, stream)
                                      : cudaMemsetAsync(dstate, 0, state_bytes, stream);
    return e == cudaSuccess ? T3_OK : T3_ECUDA;
  }
  lin::Args p{};
  p.log_decay = log_decay;
  p.resets = resets;
  p.length = length, p.heads = heads, p.pairs = batch * heads;
  lin::Args a = p;  // dq: in time, from the state transposed
  a.q = dout, a.k = v, a.v = k, a.o = dq;
  a.ldq = lddo, a.ldk = ldv, a.ldv = ldk, a.ldo = lddq;
  a.init = state, a.init_transposed = 1;
  a.in_scale = 1.0f, a.out_scale = scale;
  a.dk = static_cast<int>(dv), a.dv = static_cast<int>(dk);
  st = linear_pass(a, false, dtype, workspace, dev, stream);
  if (st != T3_OK) return st;
  a.q = v, a.k = dout, a.v = q, a.o = dk_out;  // dk: against time, from dstate_last transposed
  a.ldq = ldv, a.ldk = lddo, a.ldv = ldq, a.ldo = lddk;
  a.init = dstate_last;
  a.in_scale = scale, a.out_scale = 1.0f;
  st = linear_pass(a, true, dtype, workspace, dev, stream);
  if (st != T3_OK) return st;
  // dv, and dstate, which may lie over dstate_last: the last to read it
  p.q = k, p.k = q, p.v = dout, p.o = dv_out;
  p.ldq = ldk, p.ldk = ldq, p.ldv = lddo, p.ldo = lddv;
  p.init = dstate_last;
  p.in_scale = scale, p.out_scale = 1.0f;
  p.last = dstate;
  p.dk = static_cast<int>(dk), p.dv = static_cast<int>(dv);
  return linear_pass(p, true, dtype, workspace, dev, stream);
}

int64_t t3_set_small_product_limit(int64_t macs) {
  return g_small_macs.exchange(macs < 0 ? 0 : macs);
}

}  // extern "C"

extern "C" {

const char* t3_status_string(int status) {
  switch (status) {
    case T3_OK: return "T3_OK: success";
    case T3_EINVAL: return "T3_EINVAL: null pointer or invalid size";
    case T3_EVALUE: return "T3_EVALUE: weight outside {-1, 0, +1}";
    case T3_EOVERFLOW: return "T3_EOVERFLOW: reduction too long for an exact int32 result";
    case T3_ECUDA: return "T3_ECUDA: a CUDA call failed";
    case T3_ETIMEOUT: return "T3_ETIMEOUT: a bounded device wait gave up";
    case T3_EDEVICE: return "T3_EDEVICE: no usable sm_103 device";
    default: return "unknown t3 status";
  }
}

int t3_last_device_error(t3_stream_t stream, int32_t* detail) {
  if (detail) *detail = 0;
  const DeviceInfo* dev = nullptr;
  int st = device_info(&dev);
  if (st != T3_OK) return st;
  if (cudaStreamSynchronize(stream) != cudaSuccess) return T3_ECUDA;
  int value = 0;
  if (cudaMemcpy(&value, dev->err_word, sizeof(int), cudaMemcpyDeviceToHost) != cudaSuccess)
    return T3_ECUDA;
  if (value != 0) {
    const int zero = 0;
    if (cudaMemcpy(dev->err_word, &zero, sizeof(int), cudaMemcpyHostToDevice) != cudaSuccess)
      return T3_ECUDA;
  }
  if (detail) *detail = value;
  if (value == 0) return T3_OK;
  return (value & 0xFF) == 6 ? T3_EVALUE : T3_ETIMEOUT;  // role 6: an invalid input value
}

int t3_gemm_fwd_bf16(const void* X, const uint8_t* Wp, int32_t* C, float* row_scale,
                     float* row_inv, int64_t M, int64_t N, int64_t K, t3_stream_t stream) {
  if (bad_dims(M, N, K)) return T3_EINVAL;
  if (M == 0) return T3_OK;
  if (!row_scale || !row_inv || (K > 0 && !X)) return T3_EINVAL;
  if (K > kMaxTernaryReduction) return T3_EOVERFLOW;
  // the fused kernel's shapes, checked before any CUDA call
  if (N > 0 && K > 0 &&
      (M <= kSmallM || K % 64 != 0 || reinterpret_cast<uintptr_t>(X) % 16 != 0 ||
       reinterpret_cast<uintptr_t>(Wp) % 16 != 0))
    return T3_EINVAL;
  const DeviceInfo* dev = nullptr;
  int st = device_info(&dev);
  if (st != T3_OK) return st;
  if (K == 0) {  // zero rows: scales 0, and the empty reduction writes zeros
    if (cudaMemsetAsync(row_scale, 0, M * sizeof(float), stream) != cudaSuccess ||
        cudaMemsetAsync(row_inv, 0, M * sizeof(float), stream) != cudaSuccess)
      return T3_ECUDA;
    return N == 0 ? T3_OK : zero_fill(C, M, N, stream);
  }
  if (N > 0 && (!Wp || !C)) return T3_EINVAL;
  // the fused kernel's shapes: checked before anything is launched
  const int64_t KB = (K + 3) / 4;
  CUtensorMap ma, mw, mo;
  if (N > 0) {
    if (!make_u16_map_tiled(&ma, X, M, K, 128, tc2::BK / 2)) return T3_EINVAL;
    if (!make_u8_map_tiled(&mw, Wp, N, KB, KB, tc2::BNH, tc2::BK / 4)) return T3_EINVAL;
    if (!make_out_map(&mo, C, M, N, tc2::kOutI32)) mo = mw;  // plain stores
  }
  st = launch_row_scales(X, row_scale, row_inv, M, K, dev->sms, stream);
  if (st != T3_OK || N == 0) return st;
  tc2::Params p{};
  p.M = M;
  p.N = N;
  p.K = K;
  p.out_rows = M;
  p.out_cols = N;
  p.num_stages = ceil_div(K, tc2::BK);
  const int64_t tiles_r = ceil_div(M, tc2::BMP), tiles_c = ceil_div(N, tc2::BN);
  if (tiles_r * tiles_c > kMaxDim) return T3_EINVAL;
  p.tiles_r = static_cast<int>(tiles_r);
  p.tiles_c = static_cast<int>(tiles_c);
  p.out = C;
  p.use_tma_out = (reinterpret_cast<uintptr_t>(C) % 16 == 0 && (N * 4) % 16 == 0) ? 1 : 0;
  p.out_kind = tc2::kOutI32;
  p.wp = Wp;
  p.kb_bytes = KB;
  p.w_tma = 1;
  p.w_vec4 = 1;
  p.act = nullptr;
  p.act_rows = M;
  p.act_cols = K;
  p.a_tma = 1;
  p.mode = tc2::kModeBf16;
  p.dp_tiles = static_cast<int>(tiles_r * tiles_c);
  p.row_inv = row_inv;
  p.err = dev->err_word;
  const int64_t pairs = std::min<int64_t>(tiles_r * tiles_c, std::max(dev->sms / 2, 1));
  return launch_tc2_fwd_bf16(p, ma, mw, mo, static_cast<int>(2 * pairs), stream);
}

int t3_selftest_scan_wait_timeout(int64_t limit_ns, t3_stream_t stream) {
  if (limit_ns < 1000 || limit_ns > static_cast<int64_t>(kWaitLimitNs)) return T3_EINVAL;
  const DeviceInfo* dev = nullptr;
  const int st = device_info(&dev);
  if (st != T3_OK) return st;
  return launch_scan_wait_selftest(dev->err_word, static_cast<uint64_t>(limit_ns), stream);
}

int t3_selftest_wait_timeout(int64_t limit_ns, t3_stream_t stream) {
  if (limit_ns < 1000 || limit_ns > static_cast<int64_t>(kWaitLimitNs)) return T3_EINVAL;
  const DeviceInfo* dev = nullptr;
  const int st = device_info(&dev);
  if (st != T3_OK) return st;
  wait_selftest_kernel<<<1, 32, 0, stream>>>(dev->err_word, static_cast<uint64_t>(limit_ns));
  return cudaGetLastError() == cudaSuccess ? T3_OK : T3_ECUDA;
}

int t3_version(void) { return 200; }

}  // extern "C"
