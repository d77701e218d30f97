// Host side of the C ABI declared in include/ep_combine.h: argument
// validation, handle state, tile-configuration choice and kernel launches.
// No device memory is allocated here; every buffer belongs to the caller,
// except the small library-held counter array of the allocation-free GEMM
// entry point below.
#include "ep_combine.h"

#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstring>
#include <mutex>
#include <new>

#include "combine_common.h"
#include "ep_kernels.h"
#include "layer_kernels.h"

// Counters of ep_grouped_gemm_scatter_noalloc: R election counters, then E_l
// per-expert tile counters (the roles of ep_combine_buffers.rank_counter and
// .tile_counter), at most EP_MAX_RANKS + EP_MAX_LOCAL_EXPERTS words.  Every GPU
// the library runs on holds its own copy until the process ends.  In host
// code this name is not a device address: kernels and copies get the address
// that hipGetSymbolAddress returned for the current device (scratch_on()).
constexpr int kScratchWords = EP_MAX_RANKS + EP_MAX_LOCAL_EXPERTS;
static __device__ __align__(256) int32_t scratch[kScratchWords];

struct ep_combine_handle {
  ep_combine_params p;
  ep_combine_buffers b;
  int device;
  int num_cus;
  int tile;                 // ep::GemmTile used for this geometry
};

namespace {

constexpr int64_t kDefaultSpinLimit = int64_t(1) << 22;

// Device address of `scratch` on each device, looked up once per device by
// ep_combine_init with that device current.
constexpr int kMaxDevices = 64;
std::mutex g_scratch_mu;
int32_t* g_scratch[kMaxDevices];

// Looks up (once) the address of `scratch` on device `dev`, which must be the
// current device.  Returns EP_OK or EP_ERR_HIP.
int resolve_scratch(int dev) {
  if (dev < 0 || dev >= kMaxDevices) return EP_ERR_UNSUPPORTED;
  std::lock_guard<std::mutex> lock(g_scratch_mu);
  if (g_scratch[dev]) return EP_OK;
  void* p = nullptr;
  if (hipGetSymbolAddress(&p, HIP_SYMBOL(scratch)) != hipSuccess || !p) return EP_ERR_HIP;
  g_scratch[dev] = static_cast<int32_t*>(p);
  return EP_OK;
}

int32_t* scratch_on(int dev) {
  if (dev < 0 || dev >= kMaxDevices) return nullptr;
  std::lock_guard<std::mutex> lock(g_scratch_mu);
  return g_scratch[dev];
}

// Zeroes n words (a kernel, not a memset node: callers may capture the
// allocation-free entry point in a graph).
__global__ void zero_words_kernel(int32_t* p, int n) {
  const int i = blockIdx.x * blockDim.x + threadIdx.x;
  if (i < n) p[i] = 0;
}
// at most this many rows per local expert on average: bf16 GEMMs use the
// decode tile below
constexpr int kDecodeRowsPerExpert = 48;
constexpr int kDecodeTile = ep::kTileDecode64x128;

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Bytes of `experts` down-projections in the handle's dtype.
uint64_t weight_bytes(const ep_combine_params& p, int experts) {
  return uint64_t(experts) * p.hidden_n * p.hidden_k * (p.dtype == EP_DTYPE_BF16 ? 2 : 1);
}

int validate_params(const ep_combine_params* p) {
  if (!p) return EP_ERR_INVALID_ARG;
  if (p->n_ranks < 1 || p->n_ranks > EP_MAX_RANKS) return EP_ERR_INVALID_ARG;
  // Only ranks reachable by direct stores are supported (no SHMEM path).
  if (p->p2p_world_size != p->n_ranks) return EP_ERR_UNSUPPORTED;
  if (p->my_rank < 0 || p->my_rank >= p->n_ranks) return EP_ERR_INVALID_ARG;
  if (p->top_k < 1 || p->top_k > 64) return EP_ERR_INVALID_ARG;
  if (p->n_experts_per_device < 1 || p->n_experts_per_device > EP_MAX_LOCAL_EXPERTS)
    return EP_ERR_INVALID_ARG;
  if (p->max_tokens_per_rank < 1) return EP_ERR_INVALID_ARG;
  if (p->hidden_k < 1 || p->hidden_n < 1) return EP_ERR_INVALID_ARG;
  if (p->msg_bytes < 2 * p->hidden_n || p->msg_bytes % 16) return EP_ERR_INVALID_ARG;
  if (p->hidden_n % 128) return EP_ERR_UNSUPPORTED;
  if (p->dtype == EP_DTYPE_BF16) {
    if (p->hidden_k % 64) return EP_ERR_UNSUPPORTED;
  } else if (p->dtype == EP_DTYPE_FP8_E4M3_B128) {
    if (p->hidden_k % 128) return EP_ERR_UNSUPPORTED;
  } else {
    return EP_ERR_UNSUPPORTED;
  }
  if (p->flags &
      ~uint32_t(EP_FLAG_SYSTEM_SCOPE | EP_FLAG_PER_EXPERT_RELEASE | EP_FLAG_EPILOGUE_ONLY |
                EP_FLAG_TRACE | EP_FLAG_W_SLICE_MAJOR | EP_FLAG_DEVICE_EPOCH |
                EP_FLAG_SEND_TILE))
    return EP_ERR_INVALID_ARG;
  if ((p->flags & EP_FLAG_W_SLICE_MAJOR) && p->dtype != EP_DTYPE_BF16) return EP_ERR_UNSUPPORTED;
  if (p->send_waves != 0 && p->send_waves != 4) return EP_ERR_INVALID_ARG;
  if (p->send_waves || (p->flags & EP_FLAG_SEND_TILE)) {
    // the send-wave kernel: bf16, no measurement modes
    if (p->dtype != EP_DTYPE_BF16) return EP_ERR_UNSUPPORTED;
    if (p->flags & (EP_FLAG_EPILOGUE_ONLY | EP_FLAG_TRACE)) return EP_ERR_UNSUPPORTED;
  }
  if (p->flag_spin_limit < 0) return EP_ERR_INVALID_ARG;
  // 32-bit offsets inside one expert's weights
  if (weight_bytes(*p, 1) >= (uint64_t(1) << 32)) return EP_ERR_UNSUPPORTED;
  return EP_OK;
}

// The products of weights in the handle's dtype (not those of 4-bit weights) take a stack
// below 4 GiB.
bool stack_ok(const ep_combine_handle* h) {
  return weight_bytes(h->p, h->p.n_experts_per_device) < (uint64_t(1) << 32);
}

ep::SinkState sink_state(const ep_combine_handle* h, uint64_t epoch) {
  ep::SinkState s{};
  for (int i = 0; i < EP_MAX_RANKS; ++i)
    s.recv[i] = i < h->p.n_ranks ? static_cast<uint8_t*>(h->b.recv_buf[i]) : nullptr;
  s.words = h->b.recv_count;
  s.rank_counter = h->b.rank_counter;
  s.tile_counter = h->b.tile_counter;
  s.err = h->b.error_word;
  s.epoch_ptr = (h->p.flags & EP_FLAG_DEVICE_EPOCH) ? h->b.epoch_word : nullptr;
  s.epoch = epoch;
  s.n_ranks = h->p.n_ranks;
  s.n_experts = h->p.n_experts_per_device;
  s.top_k = h->p.top_k;
  s.msg_bytes = h->p.msg_bytes;
  s.max_tokens = h->p.max_tokens_per_rank;
  s.system_scope = (h->p.flags & EP_FLAG_SYSTEM_SCOPE) ? 1 : 0;
  s.per_expert = (h->p.flags & EP_FLAG_PER_EXPERT_RELEASE) ? 1 : 0;
  return s;
}

// A step's epoch is nonzero.  With per-expert completion the count words
// carry its low 32 bits as their tag and start out zero, so those bits must be
// nonzero as well (epochs then only need to differ modulo 2^32).  A handle
// that keeps the epoch in device memory takes 0 here: the kernels read the word.
bool epoch_ok(const ep_combine_handle* h, uint64_t epoch) {
  if (h->p.flags & EP_FLAG_DEVICE_EPOCH) return epoch == 0;
  if (epoch == 0) return false;
  if ((h->p.flags & EP_FLAG_PER_EXPERT_RELEASE) && (epoch & 0xffffffffull) == 0) return false;
  return true;
}

// Checks and fills the consumer combine's arguments (ep_combine_reduce and the
// consumer side of ep_grouped_gemm_scatter_combine).  tokens_per_rank > 0.
int combine_args(const ep_combine_handle* h, const int32_t* topk_ids, const float* topk_w,
                 int32_t tokens_per_rank, void* out, uint64_t epoch, ep::CombineArgs* a) {
  if (!topk_ids || !topk_w || !out || !aligned16(out)) return EP_ERR_INVALID_ARG;
  *a = ep::CombineArgs{};
  a->topk_ids = topk_ids;
  a->topk_w = topk_w;
  a->out = static_cast<uint8_t*>(out);
  a->flags = h->b.recv_count + size_t(h->p.n_experts_per_device) * h->p.n_ranks;
  for (int i = 0; i < EP_MAX_RANKS; ++i)
    a->recv[i] = i < h->p.n_ranks ? static_cast<uint8_t*>(h->b.recv_buf[i]) : nullptr;
  a->err = h->b.error_word;
  a->epoch = epoch;
  a->epoch_ptr = (h->p.flags & EP_FLAG_DEVICE_EPOCH) ? h->b.epoch_word : nullptr;
  a->spin_limit = h->p.flag_spin_limit;
  a->n_ranks = h->p.n_ranks;
  a->tokens = tokens_per_rank;
  a->top_k = h->p.top_k;
  a->N = h->p.hidden_n;
  a->msg_bytes = h->p.msg_bytes;
  a->expert_lo = h->p.my_rank * h->p.n_experts_per_device;
  a->n_experts = h->p.n_experts_per_device;
  a->system_scope = (h->p.flags & EP_FLAG_SYSTEM_SCOPE) ? 1 : 0;
  a->per_expert = (h->p.flags & EP_FLAG_PER_EXPERT_RELEASE) ? 1 : 0;
  a->words = h->b.recv_count;
  return EP_OK;
}

int pick_tile(const ep_combine_params* p) {
  if (p->dtype == EP_DTYPE_FP8_E4M3_B128)
    return (p->hidden_n % 256 == 0) ? ep::kTile256x256 : ep::kTile256x128;
  if (p->send_waves) return ep::kTileSend128x128;
  if (p->flags & EP_FLAG_SEND_TILE) return ep::kTileSendNone128x128;
  return (p->hidden_n % 256 == 0) ? ep::kTile256x256 : ep::kTile128x128;
}

// Tile of one grouped-GEMM call: small row groups (decode: a few dozen rows
// per local expert) stream W_e with the decode tile, which keeps several K
// slices in flight.
int call_tile(const ep_combine_handle* h, int32_t m_total) {
  const bool fp8 = h->p.dtype == EP_DTYPE_FP8_E4M3_B128;
  return (!fp8 && h->tile == ep::kTile256x256 &&
          int64_t(m_total) <= int64_t(kDecodeRowsPerExpert) * h->p.n_experts_per_device)
             ? kDecodeTile
             : h->tile;
}

}  // namespace

extern "C" {

int ep_combine_version(void) { return 300; }

const char* ep_combine_strerror(int code) {
  switch (code) {
    case EP_OK: return "ok";
    case EP_ERR_INVALID_ARG: return "invalid argument";
    case EP_ERR_UNSUPPORTED: return "unsupported shape or dtype";
    case EP_ERR_HIP: return "HIP runtime error";
    case EP_ERR_SLOT_OOB: return "device: receive slot out of bounds";
    case EP_ERR_FLAG_TIMEOUT: return "device: timed out waiting for a rank flag";
    case EP_ERR_BAD_GROUP: return "device: inconsistent group offsets or signal coordinates";
    default: return code > 0 ? "device: several error bits" : "unknown error";
  }
}

int ep_combine_init(const ep_combine_params* params, const ep_combine_buffers* bufs,
                    ep_combine_t* out) {
  if (!out) return EP_ERR_INVALID_ARG;
  *out = nullptr;
  int rc = validate_params(params);
  if (rc != EP_OK) return rc;
  if (!bufs || !bufs->recv_count || !bufs->rank_counter || !bufs->tile_counter ||
      !bufs->error_word)
    return EP_ERR_INVALID_ARG;
  for (int i = 0; i < params->n_ranks; ++i)
    if (!bufs->recv_buf[i] || !aligned16(bufs->recv_buf[i])) return EP_ERR_INVALID_ARG;
  if ((params->flags & EP_FLAG_TRACE) &&
      (!bufs->trace || !aligned16(bufs->trace) || bufs->trace_records <= 0))
    return EP_ERR_INVALID_ARG;
  if ((params->flags & EP_FLAG_DEVICE_EPOCH) &&
      (!bufs->epoch_word || reinterpret_cast<uintptr_t>(bufs->epoch_word) % 8))
    return EP_ERR_INVALID_ARG;
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess) return EP_ERR_HIP;
  int cus = 0;
  if (hipDeviceGetAttribute(&cus, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess)
    return EP_ERR_HIP;
  // the allocation-free GEMM's counters on this device; a failed lookup only
  // makes that one entry point unavailable (it then returns EP_ERR_HIP)
  (void)resolve_scratch(dev);
  auto* h = new (std::nothrow) ep_combine_handle;
  if (!h) return EP_ERR_INVALID_ARG;
  h->p = *params;
  if (h->p.flag_spin_limit == 0) h->p.flag_spin_limit = kDefaultSpinLimit;
  h->b = *bufs;
  h->device = dev;
  h->num_cus = cus > 0 ? cus : 256;
  h->tile = pick_tile(params);
  *out = h;
  return EP_OK;
}

void ep_combine_destroy(ep_combine_t h) { delete h; }

}  // extern "C"

namespace {

// ep_grouped_gemm_scatter with its election and tile counters at
// rank_counter / tile_counter (the caller's, or the library's scratch).
int gemm_scatter(ep_combine_t h, const void* x, const void* w, const float* x_scale,
                 const float* w_scale, const int32_t* offsets, const int32_t* src_info,
                 int32_t m_total, int32_t p3_control, void* c_local, uint64_t epoch,
                 void* stream, int32_t* rank_counter, int32_t* tile_counter,
                 const ep::CombineArgs* comb = nullptr) {
  if (!h || !w || !offsets) return EP_ERR_INVALID_ARG;
  if (m_total < 0) return EP_ERR_INVALID_ARG;
  if (m_total > 0 && (!x || !src_info)) return EP_ERR_INVALID_ARG;
  const bool sink_on = p3_control >= 0;
  if (!sink_on && m_total > 0 && (!c_local || !aligned16(c_local))) return EP_ERR_INVALID_ARG;
  if (sink_on && !epoch_ok(h, epoch)) return EP_ERR_INVALID_ARG;
  const bool fp8 = h->p.dtype == EP_DTYPE_FP8_E4M3_B128;
  if (fp8 && ((m_total > 0 && !x_scale) || !w_scale)) return EP_ERR_INVALID_ARG;
  if (!stack_ok(h)) return EP_ERR_UNSUPPORTED;
  const int elt = fp8 ? 1 : 2;
  if (uint64_t(m_total) * h->p.hidden_k * elt >= (uint64_t(1) << 32)) return EP_ERR_UNSUPPORTED;
  if ((x && !aligned16(x)) || !aligned16(w)) return EP_ERR_INVALID_ARG;

  ep::GemmArgs a{};
  a.x = static_cast<const uint8_t*>(x);
  a.w = static_cast<const uint8_t*>(w);
  a.x_scale = x_scale;
  a.w_scale = w_scale;
  a.offsets = offsets;
  a.src_info = src_info;
  a.c_local = static_cast<uint8_t*>(c_local);
  a.m_total = m_total;
  a.K = h->p.hidden_k;
  a.N = h->p.hidden_n;
  a.sink_on = sink_on ? 1 : 0;
  a.epilogue_only = (h->p.flags & EP_FLAG_EPILOGUE_ONLY) ? 1 : 0;
  a.w_slice_major = (h->p.flags & EP_FLAG_W_SLICE_MAJOR) ? 1 : 0;
  a.s = sink_state(h, epoch);
  a.s.rank_counter = rank_counter;
  a.s.tile_counter = tile_counter;
  if ((h->p.flags & EP_FLAG_TRACE) && !a.epilogue_only) {
    a.trace = h->b.trace;
    a.trace_records = h->b.trace_records;
  }

  const int El = h->p.n_experts_per_device;
  const int tile = call_tile(h, m_total);
  const int bm = ep::gemm_tile_rows(tile), bn = ep::gemm_tile_cols(tile);
  const int64_t nt = h->p.hidden_n / bn;
  const int64_t items = (int64_t(m_total) / bm + El) * nt + El;     // upper bound
  const int64_t resident = int64_t(h->num_cus) * ep::gemm_blocks_per_cu(tile);
  int64_t grid = std::min(items, resident);
  grid = (grid + 7) / 8 * 8;
  if (comb) {
    // fused launch: every workgroup turns consumer after its tiles, and a
    // consumer waits for workgroups that are still producing, so the whole grid
    // must be resident at once: at most `resident` workgroups, a multiple of 8
    if (a.epilogue_only || a.trace || !sink_on || tile >= ep::kTileSend128x128)
      return EP_ERR_UNSUPPORTED;
    grid = std::max<int64_t>(8, resident / 8 * 8);   // the launcher sizes it from occupancy
    a.fused = 1;
    a.num_cus = h->num_cus;
    a.comb = *comb;
    int tpr = 0, rpr = 0;
    // about four runs per workgroup
    ep::combine_split(comb->n_ranks, comb->tokens, 4 * grid, &tpr, &rpr);
    a.comb_tokens_per_run = tpr;
    a.comb_runs_per_rank = rpr;
    a.comb_chunks = ep::combine_chunks(comb->N);
  }
  hipStream_t st = static_cast<hipStream_t>(stream);
  hipError_t err = fp8 ? ep::launch_gemm_fp8(a, tile, int(grid), st)
                  : tile >= ep::kTileSend128x128
                      ? ep::launch_gemm_send(a, tile == ep::kTileSend128x128 ? 4 : 0, int(grid), st)
                      : ep::launch_gemm_bf16(a, tile, int(grid), st);
  return err == hipSuccess ? EP_OK : (err == hipErrorNotSupported ? EP_ERR_UNSUPPORTED : EP_ERR_HIP);
}

}  // namespace

extern "C" {

int ep_grouped_gemm_scatter(ep_combine_t h, const void* x, const void* w, const float* x_scale,
                            const float* w_scale, const int32_t* offsets,
                            const int32_t* src_info, int32_t m_total, int32_t p3_control,
                            void* c_local, uint64_t epoch, void* stream) {
  if (!h) return EP_ERR_INVALID_ARG;
  return gemm_scatter(h, x, w, x_scale, w_scale, offsets, src_info, m_total, p3_control,
                      c_local, epoch, stream, h->b.rank_counter, h->b.tile_counter);
}

int ep_grouped_gemm_scatter_noalloc(ep_combine_t h, const void* x, const void* w,
                                    const float* x_scale, const float* w_scale,
                                    const int32_t* offsets, const int32_t* src_info,
                                    int32_t m_total, int32_t p3_control, void* c_local,
                                    uint64_t epoch, void* stream) {
  if (!h) return EP_ERR_INVALID_ARG;
  const int R = h->p.n_ranks, El = h->p.n_experts_per_device;
  if (R > EP_MAX_RANKS || El > EP_MAX_LOCAL_EXPERTS || R + El > kScratchWords)
    return EP_ERR_UNSUPPORTED;
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess) return EP_ERR_HIP;
  int32_t* ws = scratch_on(dev);
  if (!ws) return EP_ERR_HIP;        // no handle was initialised on this device
  hipStream_t st = static_cast<hipStream_t>(stream);
  if (p3_control >= 0) {
    // the counters start each call at zero, whatever an earlier call left
    const int n = R + El;
    hipLaunchKernelGGL(zero_words_kernel, dim3((n + 255) / 256), dim3(256), 0, st, ws, n);
    if (hipGetLastError() != hipSuccess) return EP_ERR_HIP;
  }
  return gemm_scatter(h, x, w, x_scale, w_scale, offsets, src_info, m_total, p3_control,
                      c_local, epoch, stream, ws, ws + R);
}

int ep_gemm_tile(ep_combine_t h, int32_t m_total, int32_t* tile_rows, int32_t* tile_cols) {
  if (!h || m_total < 0 || !tile_rows || !tile_cols) return EP_ERR_INVALID_ARG;
  const int tile = call_tile(h, m_total);
  const bool fp8 = h->p.dtype == EP_DTYPE_FP8_E4M3_B128;
  // the bf16 256-column tile takes up to nine 32-row blocks (rows spread
  // evenly over an expert's tiles)
  *tile_rows = (!fp8 && tile == ep::kTile256x256) ? 288 : ep::gemm_tile_rows(tile);
  *tile_cols = ep::gemm_tile_cols(tile);
  return tile;
}

int ep_group_local_picks(ep_combine_t h, const int32_t* topk_ids, int32_t tokens_per_rank,
                         int32_t* offsets, int32_t* src_info, void* stream) {
  if (!h || !offsets) return EP_ERR_INVALID_ARG;
  if (tokens_per_rank < 0 || tokens_per_rank > h->p.max_tokens_per_rank) return EP_ERR_INVALID_ARG;
  if (tokens_per_rank > 0 && (!topk_ids || !src_info)) return EP_ERR_INVALID_ARG;
  const int R = h->p.n_ranks, El = h->p.n_experts_per_device;
  // row indices and src_info word offsets stay in 32 bits
  if (int64_t(2) * R * tokens_per_rank * h->p.top_k >= (int64_t(1) << 31)) return EP_ERR_UNSUPPORTED;
  ep::GroupArgs a{};
  a.topk_ids = topk_ids;
  a.offsets = offsets;
  a.src_info = src_info;
  a.n_ranks = R;
  a.n_experts = El;
  a.expert_lo = h->p.my_rank * El;
  a.tokens = tokens_per_rank;
  a.top_k = h->p.top_k;
  const hipError_t err = ep::launch_grouping(a, static_cast<hipStream_t>(stream));
  return err == hipSuccess ? EP_OK : EP_ERR_HIP;
}

int ep_dispatch_rows(ep_combine_t h, const void* tokens_x, int32_t tokens_per_rank,
                     int32_t row_bytes, const int32_t* offsets, const int32_t* src_info,
                     int32_t m_total, void* x_out, void* stream) {
  if (!h || !offsets || m_total < 0) return EP_ERR_INVALID_ARG;
  if (tokens_per_rank < 0 || tokens_per_rank > h->p.max_tokens_per_rank) return EP_ERR_INVALID_ARG;
  if (row_bytes < 16 || row_bytes % 16) return EP_ERR_INVALID_ARG;
  if (m_total == 0) return EP_OK;
  if (!tokens_x || !src_info || !x_out || !aligned16(tokens_x) || !aligned16(x_out))
    return EP_ERR_INVALID_ARG;
  ep::DispatchArgs a{};
  a.tokens_x = static_cast<const uint8_t*>(tokens_x);
  a.offsets = offsets;
  a.src_info = src_info;
  a.x_out = static_cast<uint8_t*>(x_out);
  a.err = h->b.error_word;
  a.m_total = m_total;
  a.row_bytes = row_bytes;
  a.tokens = tokens_per_rank;
  a.n_ranks = h->p.n_ranks;
  a.n_experts = h->p.n_experts_per_device;
  const hipError_t err = ep::launch_dispatch(a, h->num_cus, static_cast<hipStream_t>(stream));
  return err == hipSuccess ? EP_OK : EP_ERR_HIP;
}

int ep_pack_weights(ep_combine_t h, const void* w, void* w_out, void* stream) {
  if (!h || !w || !w_out || !aligned16(w) || !aligned16(w_out)) return EP_ERR_INVALID_ARG;
  if (h->p.dtype != EP_DTYPE_BF16 || !stack_ok(h)) return EP_ERR_UNSUPPORTED;
  const uint64_t bytes = weight_bytes(h->p, h->p.n_experts_per_device);
  const uintptr_t a = reinterpret_cast<uintptr_t>(w), b = reinterpret_cast<uintptr_t>(w_out);
  if (a < b + bytes && b < a + bytes) return EP_ERR_INVALID_ARG;
  const hipError_t err = ep::launch_pack_slice_major(
      static_cast<const uint8_t*>(w), static_cast<uint8_t*>(w_out), h->p.n_experts_per_device,
      h->p.hidden_n, h->p.hidden_k, h->num_cus, static_cast<hipStream_t>(stream));
  return err == hipSuccess ? EP_OK : EP_ERR_HIP;
}

int ep_grouped_gemm_swiglu(ep_combine_t h, const void* x1, const void* w1,
                           const int32_t* offsets, int32_t m_total, void* h_out, void* stream) {
  if (!h || !w1 || !offsets || m_total < 0) return EP_ERR_INVALID_ARG;
  if (m_total > 0 && (!x1 || !h_out)) return EP_ERR_INVALID_ARG;
  if ((x1 && !aligned16(x1)) || !aligned16(w1) || (h_out && !aligned16(h_out)))
    return EP_ERR_INVALID_ARG;
  if (h->p.dtype != EP_DTYPE_BF16) return EP_ERR_UNSUPPORTED;
  const int hidden = h->p.hidden_n, inter = h->p.hidden_k;
  // 2I GEMM columns in whole 256-column tiles; 32-bit offsets inside X1 and W1_e
  if (inter % 128 || !stack_ok(h)) return EP_ERR_UNSUPPORTED;
  if (uint64_t(m_total) * hidden * 2 >= (uint64_t(1) << 32)) return EP_ERR_UNSUPPORTED;
  if (uint64_t(2) * inter * hidden * 2 >= (uint64_t(1) << 32)) return EP_ERR_UNSUPPORTED;

  ep::GemmArgs a{};
  a.x = static_cast<const uint8_t*>(x1);
  a.w = static_cast<const uint8_t*>(w1);
  a.offsets = offsets;
  a.c_local = static_cast<uint8_t*>(h_out);
  a.m_total = m_total;
  a.K = hidden;
  a.N = 2 * inter;
  a.sink_on = 0;
  a.s = sink_state(h, 1);     // rank / expert counts and the error word only

  const int El = h->p.n_experts_per_device;
  const int64_t nt = a.N / ep::gemm_tile_cols(ep::kTile256x256);
  const int64_t items = (int64_t(m_total) / ep::gemm_tile_rows(ep::kTile256x256) + El) * nt + El;
  const int64_t resident = int64_t(h->num_cus) * ep::gemm_blocks_per_cu(ep::kTile256x256);
  int64_t grid = std::min(items, resident);
  grid = (grid + 7) / 8 * 8;
  hipError_t err = ep::launch_swiglu_bf16(a, int(grid), static_cast<hipStream_t>(stream));
  return err == hipSuccess ? EP_OK : EP_ERR_HIP;
}

int ep_grouped_gemm_swiglu_fp8(ep_combine_t h, const void* x1, const float* x1_scale,
                               const void* w1, const float* w1_scale, const int32_t* offsets,
                               int32_t m_total, void* h_out, float* h_scale, void* stream) {
  if (!h || !w1 || !w1_scale || !offsets || m_total < 0) return EP_ERR_INVALID_ARG;
  if (m_total > 0 && (!x1 || !x1_scale || !h_out || !h_scale)) return EP_ERR_INVALID_ARG;
  if ((x1 && !aligned16(x1)) || !aligned16(w1) || (h_out && !aligned16(h_out)))
    return EP_ERR_INVALID_ARG;
  if (h->p.dtype != EP_DTYPE_FP8_E4M3_B128) return EP_ERR_UNSUPPORTED;
  const int hidden = h->p.hidden_n, inter = h->p.hidden_k;
  // the handle's fp8 rules give hidden and I multiples of 128: 2I GEMM columns in
  // whole 256-column tiles; 32-bit offsets inside X1 and W1_e
  if (!stack_ok(h)) return EP_ERR_UNSUPPORTED;
  if (uint64_t(m_total) * hidden >= (uint64_t(1) << 32)) return EP_ERR_UNSUPPORTED;
  if (uint64_t(2) * inter * hidden >= (uint64_t(1) << 32)) return EP_ERR_UNSUPPORTED;

  ep::GemmArgs a{};
  a.x = static_cast<const uint8_t*>(x1);
  a.w = static_cast<const uint8_t*>(w1);
  a.x_scale = x1_scale;
  a.w_scale = w1_scale;
  a.offsets = offsets;
  a.c_local = static_cast<uint8_t*>(h_out);
  a.c_scale = h_scale;
  a.m_total = m_total;
  a.K = hidden;
  a.N = 2 * inter;
  a.sink_on = 0;
  a.s = sink_state(h, 1);     // rank / expert counts and the error word only

  const int El = h->p.n_experts_per_device;
  const int64_t nt = a.N / ep::gemm_tile_cols(ep::kTile256x256);
  const int64_t items = (int64_t(m_total) / ep::gemm_tile_rows(ep::kTile256x256) + El) * nt + El;
  const int64_t resident = int64_t(h->num_cus) * ep::gemm_blocks_per_cu(ep::kTile256x256);
  int64_t grid = std::min(items, resident);
  grid = (grid + 7) / 8 * 8;
  hipError_t err = ep::launch_swiglu_fp8(a, int(grid), static_cast<hipStream_t>(stream));
  return err == hipSuccess ? EP_OK : EP_ERR_HIP;
}

int ep_signal_completion(ep_combine_t h, const int32_t* expert, const int32_t* dst_rank,
                         const uint64_t* signal, int32_t n, uint64_t epoch, void* stream) {
  if (!h || n < 0 || !epoch_ok(h, epoch)) return EP_ERR_INVALID_ARG;
  if (n == 0) return EP_OK;
  if (!expert || !dst_rank || !signal) return EP_ERR_INVALID_ARG;
  hipError_t err = ep::launch_signal(sink_state(h, epoch), expert, dst_rank, signal, n,
                                     static_cast<hipStream_t>(stream));
  return err == hipSuccess ? EP_OK : EP_ERR_HIP;
}

int ep_combine_reduce(ep_combine_t h, const int32_t* topk_ids, const float* topk_w,
                      int32_t tokens_per_rank, void* out, uint64_t epoch, void* stream) {
  if (!h || !epoch_ok(h, epoch)) return EP_ERR_INVALID_ARG;
  if (tokens_per_rank < 0 || tokens_per_rank > h->p.max_tokens_per_rank) return EP_ERR_INVALID_ARG;
  if (tokens_per_rank == 0) return EP_OK;
  ep::CombineArgs a{};
  const int rc = combine_args(h, topk_ids, topk_w, tokens_per_rank, out, epoch, &a);
  if (rc != EP_OK) return rc;
  hipError_t err = ep::launch_combine(a, h->num_cus, static_cast<hipStream_t>(stream));
  return err == hipSuccess ? EP_OK : EP_ERR_HIP;
}

int ep_grouped_gemm_scatter_combine(ep_combine_t h, const void* x, const void* w,
                                    const float* x_scale, const float* w_scale,
                                    const int32_t* offsets, const int32_t* src_info,
                                    int32_t m_total, const int32_t* topk_ids,
                                    const float* topk_w, int32_t tokens_per_rank, void* out,
                                    uint64_t epoch, void* stream) {
  if (!h || !epoch_ok(h, epoch)) return EP_ERR_INVALID_ARG;
  if (tokens_per_rank < 1 || tokens_per_rank > h->p.max_tokens_per_rank) return EP_ERR_INVALID_ARG;
  if (h->p.flags & (EP_FLAG_EPILOGUE_ONLY | EP_FLAG_TRACE)) return EP_ERR_UNSUPPORTED;
  ep::CombineArgs c{};
  const int rc = combine_args(h, topk_ids, topk_w, tokens_per_rank, out, epoch, &c);
  if (rc != EP_OK) return rc;
  return gemm_scatter(h, x, w, x_scale, w_scale, offsets, src_info, m_total, 0, nullptr, epoch,
                      stream, h->b.rank_counter, h->b.tile_counter, &c);
}

}  // extern "C"

namespace {

// Whether the handle's device is the current one (its buffers, and the caller's,
// live there).
bool on_device(const ep_combine_handle* h) {
  int dev = -1;
  return hipGetDevice(&dev) == hipSuccess && dev == h->device;
}

// Checks a router call and fills its common arguments.
int route_args(const ep_combine_handle* h, const ep_route_params* p, const void* logits,
               int32_t tokens_per_rank, ep::RouteArgs* a) {
  if (!h || !p) return EP_ERR_INVALID_ARG;
  if (tokens_per_rank < 0 || tokens_per_rank > h->p.max_tokens_per_rank) return EP_ERR_INVALID_ARG;
  if (p->n_experts < h->p.top_k || p->n_groups < 1) return EP_ERR_INVALID_ARG;
  if (p->n_experts > EP_MAX_ROUTED_EXPERTS || p->n_groups > EP_MAX_ROUTE_GROUPS)
    return EP_ERR_UNSUPPORTED;
  if (p->n_experts % p->n_groups || p->topk_groups < 1 || p->topk_groups > p->n_groups)
    return EP_ERR_INVALID_ARG;
  if (p->score != EP_SCORE_SOFTMAX && p->score != EP_SCORE_SIGMOID) return EP_ERR_INVALID_ARG;
  if (p->group_score != EP_GROUP_MAX && p->group_score != EP_GROUP_TOP2) return EP_ERR_INVALID_ARG;
  if (p->renormalize != 0 && p->renormalize != 1) return EP_ERR_INVALID_ARG;
  if (p->logits_dtype < EP_LOGITS_F32 || p->logits_dtype > EP_LOGITS_F16) return EP_ERR_INVALID_ARG;
  if (!std::isfinite(p->scale)) return EP_ERR_INVALID_ARG;
  if (tokens_per_rank > 0 && (!logits || !aligned16(logits))) return EP_ERR_INVALID_ARG;
  if (!on_device(h)) return EP_ERR_INVALID_ARG;
  *a = ep::RouteArgs{};
  a->logits = static_cast<const uint8_t*>(logits);
  a->tokens = int64_t(h->p.n_ranks) * tokens_per_rank;
  a->n_experts = p->n_experts;
  a->n_groups = p->n_groups;
  a->topk_groups = p->topk_groups;
  a->top_k = h->p.top_k;
  a->score = p->score;
  a->group_score = p->group_score;
  a->renormalize = p->renormalize;
  a->dtype = p->logits_dtype;
  a->scale = p->scale;
  return EP_OK;
}

bool w4_format_ok(const ep_w4_format* f) {
  return f && (f->codes == EP_W4_INT4 || f->codes == EP_W4_E2M1) &&
         (f->group == 32 || f->group == 64 || f->group == 128) &&
         (f->scales == EP_W4_SCALE_BF16 || f->scales == EP_W4_SCALE_F16);
}

// Whether np bytes at p and nq bytes at q meet.
bool overlap(const void* p, uint64_t np, const void* q, uint64_t nq) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(q);
  return np && nq && a < b + nq && b < a + np;
}

// Whether `out` meets what a product of 4-bit weights (rows x k an expert) reads.
bool w4_output_overlaps(const ep_combine_handle* h, const ep_w4_format* f, const void* x,
                        const void* w, const void* scales, uint64_t rows, uint64_t k,
                        const int32_t* offsets, int32_t m_total, const void* out,
                        uint64_t out_bytes) {
  const uint64_t El = h->p.n_experts_per_device;
  return overlap(x, uint64_t(m_total) * k * 2, out, out_bytes) ||
         overlap(w, El * rows * k / 2, out, out_bytes) ||
         overlap(scales, El * rows * (k / f->group) * 2, out, out_bytes) ||
         overlap(offsets, (El * h->p.n_ranks + 1) * 4, out, out_bytes);
}

}  // namespace

extern "C" {

int ep_route_topk(ep_combine_t h, const ep_route_params* params, const void* logits,
                  const float* bias, int32_t tokens_per_rank, int32_t* topk_ids, float* topk_w,
                  void* stream) {
  ep::RouteArgs a{};
  const int rc = route_args(h, params, logits, tokens_per_rank, &a);
  if (rc != EP_OK) return rc;
  if (tokens_per_rank == 0) return EP_OK;
  if (!topk_ids || !topk_w) return EP_ERR_INVALID_ARG;
  const uint64_t in = uint64_t(a.tokens) * a.n_experts * (a.dtype == EP_LOGITS_F32 ? 4 : 2);
  const uint64_t out = uint64_t(a.tokens) * a.top_k * 4;
  if (overlap(logits, in, topk_ids, out) || overlap(logits, in, topk_w, out) ||
      overlap(topk_ids, out, topk_w, out))
    return EP_ERR_INVALID_ARG;
  // every token reads the bias, and a second launch reads it again
  const uint64_t bias_bytes = bias ? uint64_t(a.n_experts) * 4 : 0;
  if (overlap(bias, bias_bytes, topk_ids, out) || overlap(bias, bias_bytes, topk_w, out))
    return EP_ERR_INVALID_ARG;
  a.bias = bias;
  a.topk_ids = topk_ids;
  a.topk_w = topk_w;
  const hipError_t err = ep::launch_route(a, h->num_cus, static_cast<hipStream_t>(stream));
  return err == hipSuccess ? EP_OK : EP_ERR_HIP;
}

int ep_route_topk_backward(ep_combine_t h, const ep_route_params* params, const void* logits,
                           const int32_t* topk_ids, const float* grad_w, int32_t tokens_per_rank,
                           void* grad_logits, void* stream) {
  ep::RouteArgs a{};
  const int rc = route_args(h, params, logits, tokens_per_rank, &a);
  if (rc != EP_OK) return rc;
  if (tokens_per_rank == 0) return EP_OK;
  if (!topk_ids || !grad_w || !grad_logits || !aligned16(grad_logits)) return EP_ERR_INVALID_ARG;
  const uint64_t bytes =
      uint64_t(a.tokens) * a.n_experts * (a.dtype == EP_LOGITS_F32 ? 4 : 2);
  const uint64_t picks = uint64_t(a.tokens) * a.top_k * 4;
  if (overlap(logits, bytes, grad_logits, bytes) || overlap(topk_ids, picks, grad_logits, bytes) ||
      overlap(grad_w, picks, grad_logits, bytes))
    return EP_ERR_INVALID_ARG;
  a.topk_ids = const_cast<int32_t*>(topk_ids);
  a.grad_w = grad_w;
  a.grad_logits = static_cast<uint8_t*>(grad_logits);
  const hipError_t err = ep::launch_route_backward(a, h->num_cus, static_cast<hipStream_t>(stream));
  return err == hipSuccess ? EP_OK : EP_ERR_HIP;
}

int ep_combine_backward(ep_combine_t h, const void* grad_out, const int32_t* topk_ids,
                        const float* topk_w, int32_t tokens_per_rank, const int32_t* offsets,
                        const int32_t* src_info, int32_t m_total, void* grad_rows, float* grad_w,
                        void* stream) {
  if (!h || m_total < 0) return EP_ERR_INVALID_ARG;
  if (tokens_per_rank < 0 || tokens_per_rank > h->p.max_tokens_per_rank) return EP_ERR_INVALID_ARG;
  if (!on_device(h)) return EP_ERR_INVALID_ARG;
  if (tokens_per_rank == 0) return EP_OK;
  if (!grad_out || !aligned16(grad_out) || !topk_ids || !topk_w || !grad_w)
    return EP_ERR_INVALID_ARG;
  if (grad_rows && (!aligned16(grad_rows) || !offsets || (m_total > 0 && !src_info)))
    return EP_ERR_INVALID_ARG;
  const uint64_t tokens = uint64_t(h->p.n_ranks) * tokens_per_rank;
  const uint64_t go_bytes = tokens * h->p.hidden_n * 2, w_bytes = tokens * h->p.top_k * 4;
  const uint64_t rows_bytes = grad_rows ? uint64_t(m_total) * h->p.hidden_n * 2 : 0;
  if (overlap(grad_w, w_bytes, grad_rows, rows_bytes)) return EP_ERR_INVALID_ARG;
  // every other workgroup still reads these while rows and weights' gradients are stored
  auto meets_output = [&](const void* p, uint64_t n) {
    return overlap(p, n, grad_w, w_bytes) || overlap(p, n, grad_rows, rows_bytes);
  };
  if (meets_output(grad_out, go_bytes) || meets_output(topk_ids, w_bytes) ||
      meets_output(topk_w, w_bytes))
    return EP_ERR_INVALID_ARG;
  const uint64_t runs = uint64_t(h->p.n_experts_per_device) * h->p.n_ranks + 1;
  if (grad_rows && (meets_output(offsets, runs * 4) || meets_output(src_info, uint64_t(m_total) * 8)))
    return EP_ERR_INVALID_ARG;
  const uint64_t slots = uint64_t(tokens_per_rank) * h->p.top_k * h->p.msg_bytes;
  for (int i = 0; i < h->p.n_ranks; ++i)
    if (meets_output(h->b.recv_buf[i], slots)) return EP_ERR_INVALID_ARG;
  ep::CombineBackwardArgs a{};
  a.grad_out = static_cast<const uint8_t*>(grad_out);
  a.topk_ids = topk_ids;
  a.topk_w = topk_w;
  for (int i = 0; i < h->p.n_ranks; ++i) a.recv[i] = static_cast<const uint8_t*>(h->b.recv_buf[i]);
  a.offsets = offsets;
  a.src_info = src_info;
  a.grad_rows = static_cast<uint8_t*>(grad_rows);
  a.grad_w = grad_w;
  a.err = h->b.error_word;
  a.m_total = m_total;
  a.n_ranks = h->p.n_ranks;
  a.tokens = tokens_per_rank;
  a.top_k = h->p.top_k;
  a.N = h->p.hidden_n;
  a.msg_bytes = h->p.msg_bytes;
  a.expert_lo = h->p.my_rank * h->p.n_experts_per_device;
  a.n_experts = h->p.n_experts_per_device;
  const hipError_t err =
      ep::launch_combine_backward(a, h->num_cus, static_cast<hipStream_t>(stream));
  return err == hipSuccess ? EP_OK : EP_ERR_HIP;
}

int ep_pack_weights_w4(ep_combine_t h, const ep_w4_format* format, const void* codes,
                       const void* scales, int32_t rows, int32_t k, void* codes_out,
                       void* scales_out, void* stream) {
  if (!h || !w4_format_ok(format) || rows < 1 || k < 1) return EP_ERR_INVALID_ARG;
  if (h->p.dtype != EP_DTYPE_BF16 || rows % 16 || k % 128) return EP_ERR_UNSUPPORTED;
  for (const void* p : {codes, scales, const_cast<const void*>(codes_out),
                        const_cast<const void*>(scales_out)})
    if (!p || !aligned16(p)) return EP_ERR_INVALID_ARG;
  const int64_t experts = h->p.n_experts_per_device;
  const uint64_t nc = uint64_t(experts) * rows * k / 2;
  const uint64_t ns = uint64_t(experts) * rows * (k / format->group) * 2;
  if (overlap(codes, nc, codes_out, nc) || overlap(codes, nc, scales_out, ns) ||
      overlap(scales, ns, codes_out, nc) || overlap(scales, ns, scales_out, ns) ||
      overlap(codes_out, nc, scales_out, ns))
    return EP_ERR_INVALID_ARG;
  if (!on_device(h)) return EP_ERR_INVALID_ARG;
  const hipError_t err = ep::launch_pack_w4(
      static_cast<const uint8_t*>(codes), static_cast<const uint16_t*>(scales),
      static_cast<uint8_t*>(codes_out), static_cast<uint16_t*>(scales_out), experts, rows, k,
      format->group, format->codes == EP_W4_INT4, h->num_cus, static_cast<hipStream_t>(stream));
  return err == hipSuccess ? EP_OK : EP_ERR_HIP;
}

int ep_grouped_gemm_swiglu_w4(ep_combine_t h, const ep_w4_format* format, const void* x1,
                              const void* w1, const void* w1_scale, const int32_t* offsets,
                              int32_t m_total, void* h_out, void* stream) {
  if (!h || !w4_format_ok(format) || !w1 || !w1_scale || !offsets || m_total < 0)
    return EP_ERR_INVALID_ARG;
  if (m_total > 0 && (!x1 || !h_out)) return EP_ERR_INVALID_ARG;
  if ((x1 && !aligned16(x1)) || !aligned16(w1) || !aligned16(w1_scale) ||
      (h_out && !aligned16(h_out)))
    return EP_ERR_INVALID_ARG;
  if (h->p.dtype != EP_DTYPE_BF16) return EP_ERR_UNSUPPORTED;
  const int hidden = h->p.hidden_n, inter = h->p.hidden_k;
  if (inter % 128) return EP_ERR_UNSUPPORTED;
  if (w4_output_overlaps(h, format, x1, w1, w1_scale, 2 * uint64_t(inter), hidden, offsets,
                         m_total, h_out, uint64_t(m_total) * inter * 2))
    return EP_ERR_INVALID_ARG;
  if (!on_device(h)) return EP_ERR_INVALID_ARG;

  ep::W4Args a{};
  a.g.x = static_cast<const uint8_t*>(x1);
  a.g.w = static_cast<const uint8_t*>(w1);
  a.g.offsets = offsets;
  a.g.c_local = static_cast<uint8_t*>(h_out);
  a.g.m_total = m_total;
  a.g.K = hidden;
  a.g.N = 2 * inter;
  a.g.s = sink_state(h, 1);     // rank / expert counts and the error word only
  a.scales = static_cast<const uint16_t*>(w1_scale);
  a.codes = format->codes;
  a.group = format->group;
  a.scale_f16 = format->scales == EP_W4_SCALE_F16;
  const hipError_t err = ep::launch_gemm_w4(a, true, h->num_cus, static_cast<hipStream_t>(stream));
  return err == hipSuccess ? EP_OK : EP_ERR_HIP;
}

int ep_grouped_gemm_scatter_w4(ep_combine_t h, const ep_w4_format* format, const void* x,
                               const void* w, const void* w_scale, const int32_t* offsets,
                               const int32_t* src_info, int32_t m_total, int32_t p3_control,
                               void* c_local, uint64_t epoch, void* stream) {
  if (!h || !w4_format_ok(format) || !w || !w_scale || !offsets || m_total < 0)
    return EP_ERR_INVALID_ARG;
  if (m_total > 0 && (!x || !src_info)) return EP_ERR_INVALID_ARG;
  const bool sink_on = p3_control >= 0;
  if (!sink_on && m_total > 0 && (!c_local || !aligned16(c_local))) return EP_ERR_INVALID_ARG;
  if (sink_on && !epoch_ok(h, epoch)) return EP_ERR_INVALID_ARG;
  if ((x && !aligned16(x)) || !aligned16(w) || !aligned16(w_scale)) return EP_ERR_INVALID_ARG;
  if (h->p.dtype != EP_DTYPE_BF16 || h->p.hidden_k % 128 || h->p.send_waves ||
      (h->p.flags & (EP_FLAG_EPILOGUE_ONLY | EP_FLAG_TRACE | EP_FLAG_SEND_TILE)))
    return EP_ERR_UNSUPPORTED;
  if (!sink_on &&
      w4_output_overlaps(h, format, x, w, w_scale, h->p.hidden_n, h->p.hidden_k, offsets,
                         m_total, c_local, uint64_t(m_total) * h->p.hidden_n * 2))
    return EP_ERR_INVALID_ARG;
  if (!on_device(h)) return EP_ERR_INVALID_ARG;

  ep::W4Args a{};
  a.g.x = static_cast<const uint8_t*>(x);
  a.g.w = static_cast<const uint8_t*>(w);
  a.g.offsets = offsets;
  a.g.src_info = src_info;
  a.g.c_local = static_cast<uint8_t*>(c_local);
  a.g.m_total = m_total;
  a.g.K = h->p.hidden_k;
  a.g.N = h->p.hidden_n;
  a.g.sink_on = sink_on ? 1 : 0;
  a.g.s = sink_state(h, epoch);
  a.scales = static_cast<const uint16_t*>(w_scale);
  a.codes = format->codes;
  a.group = format->group;
  a.scale_f16 = format->scales == EP_W4_SCALE_F16;
  const hipError_t err =
      ep::launch_gemm_w4(a, false, h->num_cus, static_cast<hipStream_t>(stream));
  return err == hipSuccess ? EP_OK : EP_ERR_HIP;
}

}  // extern "C"

namespace {

struct Range {
  const void* p;
  uint64_t bytes;
};

// Whether an output meets another output or an input, but for the input of the same place
// in `same` where it is exactly that memory.
template <size_t O, size_t I>
bool outputs_meet(const Range (&out)[O], const Range (&in)[I], const Range (&same)[O]) {
  for (size_t i = 0; i < O; ++i) {
    for (size_t j = 0; j < O; ++j)
      if (i != j && overlap(out[i].p, out[i].bytes, out[j].p, out[j].bytes)) return true;
    for (const Range& r : in)
      if (overlap(out[i].p, out[i].bytes, r.p, r.bytes) &&
          !(same[i].p && r.p == same[i].p && out[i].p == r.p && out[i].bytes == r.bytes))
        return true;
  }
  return false;
}

bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

uint64_t row_type_bytes(int dtype) { return dtype == EP_ROWS_F32 ? 4 : 2; }

// Checks what the norm and its gradient share and fills it in.
int norm_args(const ep_combine_handle* h, const ep_norm_params* p, const void* weight,
              int32_t tokens_per_rank, ep::NormArgs* a) {
  if (!h || !p) return EP_ERR_INVALID_ARG;
  if (tokens_per_rank < 0 || tokens_per_rank > h->p.max_tokens_per_rank) return EP_ERR_INVALID_ARG;
  if (p->dtype < EP_ROWS_F32 || p->dtype > EP_ROWS_F16) return EP_ERR_INVALID_ARG;
  if (p->residual_dtype != p->dtype && p->residual_dtype != EP_ROWS_F32) return EP_ERR_INVALID_ARG;
  if (p->weight_dtype != p->dtype && p->weight_dtype != EP_ROWS_F32) return EP_ERR_INVALID_ARG;
  if (!std::isfinite(p->eps) || p->eps < 0.f) return EP_ERR_INVALID_ARG;
  if (!weight || !aligned16(weight) || !on_device(h)) return EP_ERR_INVALID_ARG;
  *a = ep::NormArgs{};
  a->weight = static_cast<const uint8_t*>(weight);
  a->rows = int64_t(h->p.n_ranks) * tokens_per_rank;
  a->N = h->p.hidden_n;
  a->dtype = p->dtype;
  a->sum_dtype = p->residual_dtype;
  a->weight_f32 = p->weight_dtype == EP_ROWS_F32;
  a->eps = p->eps;
  return EP_OK;
}

bool moe_tokens_ok(const ep_combine_handle* h, int32_t tokens_per_rank) {
  const int64_t tokens = int64_t(h->p.n_ranks) * tokens_per_rank;
  return tokens <= EP_MOE_MAX_TOKENS && tokens * h->p.top_k <= EP_MOE_MAX_PICKS;
}

uint64_t moe_workspace(const ep_combine_handle* h, int32_t tokens_per_rank) {
  // two bf16 parts of each hidden value
  return uint64_t(h->p.n_ranks) * tokens_per_rank * h->p.top_k * h->p.hidden_k * 2 * 2;
}

// One product's weights of `rows` x k an expert: bytes of an expert's weights, of the
// stack's and of its scales.
struct MoeStack {
  uint64_t expert, w, scales;
};

MoeStack moe_stack(const ep_combine_handle* h, const ep_w4_format* f, uint64_t rows, uint64_t k) {
  const uint64_t El = h->p.n_experts_per_device;
  if (f) return {rows * k / 2, El * rows * k / 2, El * rows * (k / f->group) * 2};
  if (h->p.dtype == EP_DTYPE_BF16) return {rows * k * 2, El * rows * k * 2, 0};
  return {rows * k, El * rows * k, El * (rows / 128) * (k / 128) * 4};
}

ep::MoeWeights moe_weights(const ep_w4_format* f, const void* w, const void* scales) {
  ep::MoeWeights m{};
  m.w = static_cast<const uint8_t*>(w);
  m.scales = scales;
  if (f) {
    m.codes = f->codes;
    m.group = f->group;
    m.scale_f16 = f->scales == EP_W4_SCALE_F16;
  }
  return m;
}

}  // namespace

static_assert(EP_MOE_MAX_TOKENS == ep::kMoeTokens && EP_MOE_MAX_PICKS == ep::kMoePicks,
              "limits of the kernels");

extern "C" {

int ep_rms_norm(ep_combine_t h, const ep_norm_params* params, const void* x, const void* residual,
                const void* weight, int32_t tokens_per_rank, void* residual_out, void* out,
                void* codes, float* scales, void* stream) {
  ep::NormArgs a{};
  const int rc = norm_args(h, params, weight, tokens_per_rank, &a);
  if (rc != EP_OK) return rc;
  if (tokens_per_rank == 0) return EP_OK;
  if (!x || !codes != !scales || (!out && !codes)) return EP_ERR_INVALID_ARG;
  for (const void* p : {x, residual, const_cast<const void*>(residual_out),
                        const_cast<const void*>(out), const_cast<const void*>(codes)})
    if (!aligned16(p)) return EP_ERR_INVALID_ARG;
  if (!aligned4(scales)) return EP_ERR_INVALID_ARG;
  const uint64_t values = uint64_t(a.rows) * a.N;
  const uint64_t xb = values * row_type_bytes(a.dtype), rb = values * row_type_bytes(a.sum_dtype);
  const Range outs[] = {{residual_out, residual_out ? rb : 0}, {out, out ? xb : 0},
                        {codes, codes ? values : 0}, {scales, scales ? values / 32 : 0}};
  const Range ins[] = {{x, xb}, {residual, residual ? rb : 0},
                       {weight, uint64_t(a.N) * row_type_bytes(params->weight_dtype)}};
  const Range same[] = {{residual, 0}, {x, 0}, {nullptr, 0}, {nullptr, 0}};
  if (outputs_meet(outs, ins, same)) return EP_ERR_INVALID_ARG;
  a.x = static_cast<const uint8_t*>(x);
  a.residual = static_cast<const uint8_t*>(residual);
  a.residual_out = static_cast<uint8_t*>(residual_out);
  a.out = static_cast<uint8_t*>(out);
  a.codes = static_cast<uint8_t*>(codes);
  a.scales = scales;
  const hipError_t err = ep::launch_rms_norm(a, h->num_cus, static_cast<hipStream_t>(stream));
  return err == hipSuccess ? EP_OK : EP_ERR_HIP;
}

int64_t ep_rms_norm_backward_workspace(ep_combine_t h, int32_t tokens_per_rank) {
  if (!h || tokens_per_rank < 0 || tokens_per_rank > h->p.max_tokens_per_rank)
    return EP_ERR_INVALID_ARG;
  const int64_t rows = int64_t(h->p.n_ranks) * tokens_per_rank;
  return int64_t(ep::norm_backward_parts(rows, h->p.hidden_n, h->num_cus)) * h->p.hidden_n * 4;
}

int ep_rms_norm_backward(ep_combine_t h, const ep_norm_params* params, const void* grad_out,
                         const void* grad_residual_out, const void* sums, const void* weight,
                         int32_t tokens_per_rank, void* grad_x, void* grad_residual,
                         float* grad_weight, void* workspace, int64_t workspace_bytes,
                         void* stream) {
  ep::NormArgs a{};
  const int rc = norm_args(h, params, weight, tokens_per_rank, &a);
  if (rc != EP_OK) return rc;
  if (!grad_weight || !aligned16(grad_weight)) return EP_ERR_INVALID_ARG;
  const int64_t need = ep_rms_norm_backward_workspace(h, tokens_per_rank);
  if (tokens_per_rank > 0) {
    if (!grad_out || !sums || (!grad_x && !grad_residual) || !workspace || workspace_bytes < need)
      return EP_ERR_INVALID_ARG;
    for (const void* p : {grad_out, grad_residual_out, sums, const_cast<const void*>(grad_x),
                          const_cast<const void*>(grad_residual),
                          const_cast<const void*>(workspace)})
      if (!aligned16(p)) return EP_ERR_INVALID_ARG;
  }
  const uint64_t values = uint64_t(a.rows) * a.N;
  const uint64_t xb = values * row_type_bytes(a.dtype), rb = values * row_type_bytes(a.sum_dtype);
  const Range outs[] = {{grad_x, grad_x ? xb : 0}, {grad_residual, grad_residual ? rb : 0},
                        {grad_weight, uint64_t(a.N) * 4}, {workspace, uint64_t(need)}};
  const Range ins[] = {{grad_out, xb}, {grad_residual_out, grad_residual_out ? rb : 0},
                       {sums, rb}, {weight, uint64_t(a.N) * row_type_bytes(params->weight_dtype)}};
  const Range same[] = {{grad_out, 0}, {grad_residual_out, 0}, {nullptr, 0}, {nullptr, 0}};
  if (outputs_meet(outs, ins, same)) return EP_ERR_INVALID_ARG;
  a.grad_out = static_cast<const uint8_t*>(grad_out);
  a.grad_residual = static_cast<const uint8_t*>(grad_residual_out);
  a.x = static_cast<const uint8_t*>(sums);
  a.grad_x = static_cast<uint8_t*>(grad_x);
  a.grad_sum = static_cast<uint8_t*>(grad_residual);
  a.grad_weight = grad_weight;
  a.partial = static_cast<float*>(workspace);
  const hipError_t err =
      ep::launch_rms_norm_backward(a, h->num_cus, static_cast<hipStream_t>(stream));
  return err == hipSuccess ? EP_OK : EP_ERR_HIP;
}

int64_t ep_moe_layer_workspace(ep_combine_t h, int32_t tokens_per_rank) {
  if (!h || tokens_per_rank < 0 || tokens_per_rank > h->p.max_tokens_per_rank)
    return EP_ERR_INVALID_ARG;
  if (!moe_tokens_ok(h, tokens_per_rank)) return EP_ERR_UNSUPPORTED;
  return int64_t(moe_workspace(h, tokens_per_rank));
}

int ep_moe_layer(ep_combine_t h, const ep_w4_format* format1, const ep_w4_format* format2,
                 const void* x, const float* x_scale, const void* w1, const void* w1_scale,
                 const void* w2, const void* w2_scale, const int32_t* topk_ids,
                 const float* topk_w, int32_t tokens_per_rank, void* out, void* workspace,
                 int64_t workspace_bytes, void* stream) {
  if (!h || !format1 != !format2) return EP_ERR_INVALID_ARG;
  if (format1 && (!w4_format_ok(format1) || !w4_format_ok(format2))) return EP_ERR_INVALID_ARG;
  if (tokens_per_rank < 0 || tokens_per_rank > h->p.max_tokens_per_rank) return EP_ERR_INVALID_ARG;
  const bool fp8 = h->p.dtype == EP_DTYPE_FP8_E4M3_B128;
  const uint64_t hidden = h->p.hidden_n, inter = h->p.hidden_k;
  if ((fp8 && format1) || inter % 128 || !moe_tokens_ok(h, tokens_per_rank))
    return EP_ERR_UNSUPPORTED;
  const MoeStack s1 = moe_stack(h, format1, 2 * inter, hidden);
  const MoeStack s2 = moe_stack(h, format2, hidden, inter);
  const uint64_t tokens = uint64_t(h->p.n_ranks) * tokens_per_rank;
  const uint64_t x_bytes = tokens * hidden * (fp8 ? 1 : 2), out_bytes = tokens * hidden * 2;
  const uint64_t need = moe_workspace(h, tokens_per_rank);
  constexpr uint64_t k4G = uint64_t(1) << 32;      // 32-bit offsets inside each
  if (s1.expert >= k4G || s2.expert >= k4G || x_bytes >= k4G || need >= k4G)
    return EP_ERR_UNSUPPORTED;
  if (!on_device(h)) return EP_ERR_INVALID_ARG;
  if (tokens_per_rank == 0) return EP_OK;
  if (!x || !w1 || !w2 || !topk_ids || !topk_w || !out || !workspace ||
      workspace_bytes < int64_t(need))
    return EP_ERR_INVALID_ARG;
  if ((fp8 && !x_scale) || ((fp8 || format1) && (!w1_scale || !w2_scale)))
    return EP_ERR_INVALID_ARG;
  for (const void* p : {x, w1, w2, const_cast<const void*>(out),
                        const_cast<const void*>(workspace)})
    if (!aligned16(p)) return EP_ERR_INVALID_ARG;
  if (!aligned4(topk_ids) || !aligned4(topk_w)) return EP_ERR_INVALID_ARG;
  if (fp8 && (!aligned4(x_scale) || !aligned4(w1_scale) || !aligned4(w2_scale)))
    return EP_ERR_INVALID_ARG;
  if (format1 && (!aligned16(w1_scale) || !aligned16(w2_scale))) return EP_ERR_INVALID_ARG;
  const uint64_t pick_bytes = tokens * h->p.top_k * 4;
  const Range outs[] = {{out, out_bytes}, {workspace, need}};
  const Range ins[] = {{x, x_bytes}, {x_scale, fp8 ? tokens * (hidden / 128) * 4 : 0},
                       {w1, s1.w}, {w1_scale, s1.scales}, {w2, s2.w}, {w2_scale, s2.scales},
                       {topk_ids, pick_bytes}, {topk_w, pick_bytes}};
  const Range same[] = {{nullptr, 0}, {nullptr, 0}};
  if (outputs_meet(outs, ins, same)) return EP_ERR_INVALID_ARG;
  ep::MoeArgs a{};
  a.x = static_cast<const uint8_t*>(x);
  a.x_scale = x_scale;
  a.topk_ids = topk_ids;
  a.topk_w = topk_w;
  a.h = static_cast<uint8_t*>(workspace);
  a.out = static_cast<uint8_t*>(out);
  a.w1 = moe_weights(format1, w1, w1_scale);
  a.w2 = moe_weights(format2, w2, w2_scale);
  a.w2.slice_major = (h->p.flags & EP_FLAG_W_SLICE_MAJOR) ? 1 : 0;
  a.fp8 = fp8;
  a.tokens = int(tokens);
  a.top_k = h->p.top_k;
  a.expert_lo = h->p.my_rank * h->p.n_experts_per_device;
  a.n_experts = h->p.n_experts_per_device;
  a.hidden = h->p.hidden_n;
  a.inter = h->p.hidden_k;
  const hipError_t err = ep::launch_moe(a, h->num_cus, static_cast<hipStream_t>(stream));
  return err == hipSuccess ? EP_OK : EP_ERR_HIP;
}

int ep_advance_epoch(ep_combine_t h, void* stream) {
  if (!h) return EP_ERR_INVALID_ARG;
  if (!(h->p.flags & EP_FLAG_DEVICE_EPOCH)) return EP_ERR_UNSUPPORTED;
  const hipError_t err = ep::launch_advance_epoch(h->b.epoch_word, static_cast<hipStream_t>(stream));
  return err == hipSuccess ? EP_OK : EP_ERR_HIP;
}

int ep_combine_query_error(ep_combine_t h, void* stream) {
  if (!h) return EP_ERR_INVALID_ARG;
  hipStream_t st = static_cast<hipStream_t>(stream);
  int32_t v = 0;
  if (hipMemcpyAsync(&v, h->b.error_word, sizeof(v), hipMemcpyDeviceToHost, st) != hipSuccess)
    return EP_ERR_HIP;
  if (hipStreamSynchronize(st) != hipSuccess) return EP_ERR_HIP;
  if (v != 0) {
    const int32_t zero = 0;
    if (hipMemcpyAsync(h->b.error_word, &zero, sizeof(zero), hipMemcpyHostToDevice, st) !=
            hipSuccess ||
        hipStreamSynchronize(st) != hipSuccess)
      return EP_ERR_HIP;
  }
  return v;
}

}  // extern "C"
