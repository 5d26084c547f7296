// block_api.cu -- host side of the layer operators (include/replayssm_block.h):
// argument validation, choice of kernel, launch.  Nothing here reads device
// memory, allocates or synchronizes.
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdarg>
#include <cstdio>
#include <mutex>

#include "norm_params.h"
#include "ssm_params.h"
#include "ssm_tc_params.h"

namespace {

thread_local char g_error[512];

int fail(int code, const char* fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(g_error, sizeof g_error, fmt, ap);
  va_end(ap);
  return code;
}

int done() {
  g_error[0] = '\0';
  return RSM_OK;
}

struct Named {
  const void* p;
  const char* name;
};

template <int K>
int need(const Named (&list)[K]) {
  for (const Named& n : list)
    if (n.p == nullptr) return fail(RSM_EINVAL, "%s is NULL", n.name);
  return RSM_OK;
}

bool is_state(int dt, bool one_byte) {
  return dt == RSM_F32 || dt == RSM_BF16 || dt == RSM_F16 || (one_byte && (dt == RSM_I8 || dt == RSM_FP8_E4M3));
}

template <typename A>
int check_sizes(const A* a) {
  if (a->num_heads <= 0 || a->num_groups <= 0 || a->num_heads % a->num_groups != 0)
    return fail(RSM_EINVAL, "num_groups (%d) must divide num_heads (%d)", a->num_groups, a->num_heads);
  if (a->dim <= 0 || a->dstate <= 0) return fail(RSM_EINVAL, "dim and dstate must be positive");
  if (a->num_slots < 0) return fail(RSM_EINVAL, "num_slots must be >= 0 (got %d)", a->num_slots);
  if (a->input_dtype != RSM_BF16 && a->input_dtype != RSM_F32)
    return fail(RSM_EINVAL, "input_dtype must be BF16 or F32 (got %d)", a->input_dtype);
  return RSM_OK;
}

int launch(const void* fn, int64_t grid, int threads, const void* params, void* stream, size_t smem = 0) {
  if (grid > 0x7FFFFFFFLL) return fail(RSM_EINVAL, "the call needs %lld blocks, more than 2^31-1", static_cast<long long>(grid));
  void* kargs[] = {const_cast<void*>(params)};
  const cudaError_t e = cudaLaunchKernel(fn, dim3(static_cast<unsigned>(grid)), dim3(threads), kargs, smem,
                                         static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return fail(RSM_ECUDA, "launch failed: %s", cudaGetErrorString(e));
  return done();
}

int validate(const rsm_ssm_prefill_args* a, bool pointers) {
  if (a == nullptr) return fail(RSM_EINVAL, "args is NULL");
  if (a->num_seqs < 0 || a->tokens < 0) return fail(RSM_EINVAL, "num_seqs and tokens must be >= 0");
  int rc = check_sizes(a);
  if (rc != RSM_OK) return rc;
  if (!is_state(a->state_dtype, false)) return fail(RSM_EINVAL, "state_dtype must be F32, BF16 or F16 (got %d)", a->state_dtype);
  if (pointers && a->num_seqs > 0) {
    rc = need({{a->A, "A"}, {a->cu_seqlens, "cu_seqlens"}});
    if (rc != RSM_OK) return rc;
    if (a->tokens > 0) {
      rc = need({{a->x, "x"}, {a->B, "B"}, {a->C, "C"}, {a->dt, "dt"}, {a->out, "out"}});
      if (rc != RSM_OK) return rc;
    }
    if ((a->initial_slots != nullptr || a->final_slots != nullptr) && a->state == nullptr)
      return fail(RSM_EINVAL, "state is NULL and slots are given");
  }
  int threads;
  if (ssm::seq_kernel(a->input_dtype, a->dim, a->dstate, &threads) == nullptr)
    return fail(RSM_ENOTSUP, "no kernel compiled for dim %d, dstate %d", a->dim, a->dstate);
  return RSM_OK;
}

template <typename A>
int check_batch(const A* a) {
  if (a->batch < 0) return fail(RSM_EINVAL, "batch must be >= 0 (got %d)", a->batch);
  if (a->window < 1) return fail(RSM_EINVAL, "window must be >= 1 (got %d)", a->window);
  const int rc = check_sizes(a);
  if (rc != RSM_OK) return rc;
  int threads;
  if (ssm::seq_kernel(a->input_dtype, a->dim, a->dstate, &threads) == nullptr)
    return fail(RSM_ENOTSUP, "no kernel compiled for dim %d, dstate %d", a->dim, a->dstate);
  return a->batch == 0 ? RSM_OK
                       : need({{a->x, "x"}, {a->B, "B"}, {a->C, "C"}, {a->dt, "dt"}, {a->A, "A"}, {a->out, "out"},
                               {a->state, "state"}});
}

template <typename A>
void fill_batch(const A* a, ssm::Params* p) {
  p->x = a->x;
  p->B = a->B;
  p->C = a->C;
  p->dt = a->dt;
  p->A = a->A;
  p->D = a->D;
  p->out = a->out;
  p->status = a->device_status;
  p->x_bs = a->x_batch_stride;
  p->x_ts = a->x_stride;
  p->B_bs = a->B_batch_stride;
  p->B_ts = a->B_stride;
  p->C_bs = a->C_batch_stride;
  p->C_ts = a->C_stride;
  p->dt_bs = a->dt_batch_stride;
  p->dt_ts = a->dt_stride;
  p->out_ts = static_cast<int64_t>(a->num_heads) * a->dim;
  p->out_bs = p->out_ts * a->window;
  p->state_ss = a->state_slot_stride;
  p->units = a->batch;
  p->window = a->window;
  p->num_slots = a->num_slots;
  p->H = a->num_heads;
  p->G = a->num_groups;
  p->pad = a->pad_slot_id;
  p->state_dtype = a->state_dtype;
}

int launch_seq(const ssm::Params& p, int input_dtype, int dim, int dstate, void* stream) {
  int threads = 0;
  const void* fn = ssm::seq_kernel(input_dtype, dim, dstate, &threads);
  return launch(fn, static_cast<int64_t>(p.units) * p.H, threads, &p, stream);
}

// ---------------------------------------------------------------------------
// prompts on the tensor cores
// ---------------------------------------------------------------------------
constexpr int kMaxDevices = 64;
std::mutex g_mu;
int g_sms[kMaxDevices];
bool g_tc_ready[kMaxDevices][4];
bool g_token_ready[kMaxDevices][2][5][6];  // input type, state type, mode

// Lets a kernel take up to `bytes` of dynamic shared memory: once, since the limit is the
// kernel's and not the call's, and calls come from several threads.
int allow_smem(bool* ready, const void* fn, int bytes) {
  std::lock_guard<std::mutex> lk(g_mu);
  if (*ready) return RSM_OK;
  const cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e != cudaSuccess) return fail(RSM_ECUDA, "cudaFuncSetAttribute: %s", cudaGetErrorString(e));
  *ready = true;
  return RSM_OK;
}

int device_sms(int* dev, int* sms) {
  cudaError_t e = cudaGetDevice(dev);
  if (e != cudaSuccess) return fail(RSM_ECUDA, "cudaGetDevice: %s", cudaGetErrorString(e));
  if (*dev < 0 || *dev >= kMaxDevices) return fail(RSM_ECUDA, "device ordinal %d out of range", *dev);
  std::lock_guard<std::mutex> lk(g_mu);
  if (g_sms[*dev] == 0) {
    e = cudaDeviceGetAttribute(&g_sms[*dev], cudaDevAttrMultiProcessorCount, *dev);
    if (e != cudaSuccess) return fail(RSM_ECUDA, "device query failed: %s", cudaGetErrorString(e));
  }
  *sms = g_sms[*dev];
  return RSM_OK;
}

using TensorMapEncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                       const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                       CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

TensorMapEncodeFn tensor_map_encoder() {
  static const TensorMapEncodeFn fn = [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q = cudaDriverEntryPointSymbolNotFound;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      return static_cast<TensorMapEncodeFn>(nullptr);
    return reinterpret_cast<TensorMapEncodeFn>(f);
  }();
  return fn;
}

// A [tokens, cols] bf16 tensor in boxes of rows x columns, swizzled over a box's row (64 or 32 columns).
int token_map(CUtensorMap* map, const void* base, int64_t cols, int64_t tokens, int64_t stride, unsigned box_cols,
              unsigned box_rows, const char* name) {
  const TensorMapEncodeFn encode = tensor_map_encoder();
  if (encode == nullptr) return fail(RSM_ECUDA, "cuTensorMapEncodeTiled is not available from the driver");
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(tokens)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(tokens == 1 ? cols : stride) * 2u};
  const cuuint32_t box[2] = {box_cols, box_rows}, ones[2] = {1u, 1u};
  const CUresult cr = encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2u, const_cast<void*>(base), dims, strides, box, ones,
                             CU_TENSOR_MAP_INTERLEAVE_NONE,
                             box_cols == 64 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                             CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (cr != CUDA_SUCCESS) return fail(RSM_ECUDA, "cuTensorMapEncodeTiled failed for %s (%d)", name, static_cast<int>(cr));
  return RSM_OK;
}

// Tensor-map rows, and the output's, start on 16 bytes.
bool rows_aligned(const void* base, int64_t stride, int64_t cols, int64_t tokens) {
  return reinterpret_cast<uintptr_t>(base) % 16 == 0 &&
         (tokens == 1 || (stride >= cols && stride < (int64_t{1} << 38) && stride % 8 == 0));
}

// bf16 prompts with 64 x 128 states whose rows the tensor maps can address; the rest
// runs on the sequential kernel, and so do the fewest tokens, which it has done before a
// chunk has gone round.  (One sequence, 80 heads: 1, 4, 8, 16 and 2048 tokens take 6.1, 8.2,
// 11.1, 17 and 1561 us there, 10.5 to 11.6 and 42 on the tensor cores.)
bool uses_tensor_cores(const rsm_ssm_prefill_args* a) {
  return a->input_dtype == RSM_BF16 && a->dim == ssm::kDim && a->dstate == ssm::kState && a->tokens > 7 &&
         a->tokens < 0x7FFFFF00LL && static_cast<int64_t>(a->num_heads) * ssm::kState <= 0x7FFFFFFFLL;
}
bool tensor_maps_fit(const rsm_ssm_prefill_args* a) {
  const int64_t xc = static_cast<int64_t>(a->num_heads) * a->dim, bc = static_cast<int64_t>(a->num_groups) * a->dstate;
  return rows_aligned(a->x, a->x_stride, xc, a->tokens) && rows_aligned(a->B, a->B_stride, bc, a->tokens) &&
         rows_aligned(a->C, a->C_stride, bc, a->tokens) && rows_aligned(a->out, a->out_stride, xc, a->tokens);
}

struct PrefillPlan {
  int heads;       // of a CTA
  int pairs;       // CTAs' head groups in all
  uint32_t seg;    // tokens of a segment
  int64_t segs;    // segments at most; 0: nothing is split
};

// Segment states and decays, the states first.
int64_t workspace_bytes(const PrefillPlan& pl, int H) {
  return pl.segs * H * (ssm::kDim * ssm::kState + 1) * 4;
}

// How many heads a CTA takes, and whether the sequences are cut into segments, whose
// states then come from a pass of their own (x and B read twice, no outputs) and a join.
// Lengths are on the device, so sequences are taken as equally long.  Times are in chunks
// of a CTA with two heads, about 3 us, and measured: a chunk of one head 0.83; a
// states-only chunk half of a whole one; a unit (a segment of a head group) one to begin
// and end; the two launches more about four.  80 heads, cut into 1, 3, 7, 11 and 19
// segments: one sequence of 32768 tokens takes 719, 414, 381, 377 and 390 us, one of 4096
// 102, 78, 82, 84 and 94 (L2 flushed before each); one of 1024 takes 23 us with a head a CTA and 31 with two.
PrefillPlan plan_prefill(const rsm_ssm_prefill_args* a, int sms) {
  PrefillPlan pl{};
  const int64_t chunks = (a->tokens + static_cast<int64_t>(a->num_seqs) * ssm::kChunk - 1) /
                         (static_cast<int64_t>(a->num_seqs) * ssm::kChunk);
  double best = 1e300;
  for (int heads = a->num_heads / a->num_groups % 2 == 0 ? 2 : 1; heads >= 1; --heads) {
    const int pairs = a->num_heads / heads;
    const int64_t units = static_cast<int64_t>(a->num_seqs) * pairs;
    const double chunk = heads == 2 ? 1.0 : 0.83;
    auto pass = [&](int64_t n, double per) { return static_cast<double>((n + sms - 1) / sms) * (per + 1.0); };
    for (int64_t n = 1; n <= 64 && n <= std::max<int64_t>(chunks, 1); ++n) {
      const int64_t per = (chunks + n - 1) / n;
      double t = pass(units * n, chunk * static_cast<double>(per));
      if (n > 1) t += pass(units * (n - 1), 0.5 * chunk * static_cast<double>(per)) + 4.0;
      if (t >= best) continue;
      best = t;
      pl.heads = heads;
      pl.pairs = pairs;
      pl.seg = n == 1 ? 0x7FFFFF80u : static_cast<uint32_t>(per * ssm::kChunk);
      pl.segs = n == 1 ? 0 : ssm::segments_at_most(a->tokens, pl.seg, a->num_seqs);
    }
  }
  return pl;
}

int launch_tc(const rsm_ssm_prefill_args* a, const ssm::Params& p, void* stream) {
  int dev = 0, sms = 0;
  int rc = device_sms(&dev, &sms);
  if (rc != RSM_OK) return rc;
  const PrefillPlan pl = plan_prefill(a, sms);
  ssm::TcParams tp{};
  const int64_t xc = static_cast<int64_t>(a->num_heads) * ssm::kDim, bc = static_cast<int64_t>(a->num_groups) * ssm::kState;
  rc = token_map(&tp.x_map, a->x, xc, a->tokens, a->x_stride, 64, ssm::kChunk, "x");
  if (rc == RSM_OK) rc = token_map(&tp.B_map, a->B, bc, a->tokens, a->B_stride, 64, ssm::kChunk, "B");
  if (rc == RSM_OK) rc = token_map(&tp.C_map, a->C, bc, a->tokens, a->C_stride, 64, ssm::kChunk, "C");
  if (rc == RSM_OK) rc = token_map(&tp.y_map, a->out, xc, a->tokens, a->out_stride, 32, 32, "out");
  if (rc != RSM_OK) return rc;
  tp.p = p;
  tp.seg = pl.seg;
  tp.pairs = pl.pairs;
  int64_t units = static_cast<int64_t>(a->num_seqs) * pl.pairs;
  if (pl.segs > 0) {
    const int64_t need_bytes = workspace_bytes(pl, a->num_heads);
    if (a->workspace == nullptr || a->workspace_bytes < need_bytes || reinterpret_cast<uintptr_t>(a->workspace) % 256 != 0)
      return fail(RSM_EINVAL, "workspace of %lld bytes, 256-byte aligned, is needed", static_cast<long long>(need_bytes));
    tp.seg_state = static_cast<float*>(a->workspace);
    tp.seg_decay = tp.seg_state + pl.segs * a->num_heads * (ssm::kDim * ssm::kState);
    units = pl.segs * pl.pairs;
  }
  // the state's terms keep 16 bits where the state that is kept has more than bf16's 8
  const bool lo = a->final_slots != nullptr && a->state_dtype != RSM_BF16;
  const void* fn = ssm::tc_kernel(pl.heads, lo);
  const int ki = (pl.heads - 1) * 2 + (lo ? 1 : 0);
  rc = allow_smem(&g_tc_ready[dev][ki], fn, static_cast<int>(ssm::kTcSmem));
  if (rc != RSM_OK) return rc;
  // (a unit's number and the next one's after it stay below 2^32)
  if (units > 0x7FFFFFFFLL) return fail(RSM_EINVAL, "%lld units of work, more than 2^31-1", static_cast<long long>(units));
  const unsigned grid = static_cast<unsigned>(std::min<int64_t>(units, sms));
  auto run = [&](bool states_only) {
    tp.states_only = states_only ? 1 : 0;
    void* kargs[] = {&tp};
    return cudaLaunchKernel(fn, dim3(grid), dim3(ssm::kTcThreads), kargs, ssm::kTcSmem, static_cast<cudaStream_t>(stream));
  };
  if (pl.segs > 0) {
    cudaError_t e = run(true);
    if (e != cudaSuccess) return fail(RSM_ECUDA, "launch failed: %s", cudaGetErrorString(e));
    rc = launch(ssm::join_kernel(), static_cast<int64_t>(a->num_seqs) * a->num_heads * (ssm::kDim * ssm::kState) / (4 * ssm::kJoinThreads),
                ssm::kJoinThreads, &tp, stream);
    if (rc != RSM_OK) return rc;
  }
  const cudaError_t e = run(false);
  if (e != cudaSuccess) return fail(RSM_ECUDA, "launch failed: %s", cudaGetErrorString(e));
  return done();
}

// New tokens: the token kernel for 64 x 128 states on 16 bytes and up to 16 new tokens, the sequential
// kernel for the rest.  (Ring of 16, 4 new tokens, 64 requests of 256 heads, bf16: 52 us
// and 603; one token to the state itself: 93 and 578; one request of 80 heads, fp32: 6.7
// and 8.7.)  With bf16 inputs the products go to the tensor cores, but for a single
// token of the recurrent form, whose lanes keep up with the memory, or after a ring on
// fp16 states, which cost more to split than they save.  (64 requests of 256 heads, 4
// tokens after a ring of 16, fp16: 58 us and 108; 32 requests, fp32, 4 tokens: 51 and
// 118, one after a ring of 8: 48 and 63; 64 requests, fp16, one after a ring of 8: 55
// and 48; to the states: 4 tokens, bf16, 116 and 190, one, fp16, 136 and 94.)
int launch_tokens(ssm::Params& p, int input_dtype, int dim, int dstate, void* stream) {
  const int es = p.state_dtype == RSM_F32 ? 4 : p.state_dtype == RSM_BF16 || p.state_dtype == RSM_F16 ? 2 : 1;
  const bool fits = dim == ssm::kDim && dstate == ssm::kState && p.window <= ssm::kTokenMaxNew &&
                    reinterpret_cast<uintptr_t>(p.state) % 16 == 0 && p.state_ss * es % 16 == 0;
  if (!fits) return launch_seq(p, input_dtype, dim, dstate, stream);
  int dev = 0, sms = 0;
  int rc = device_sms(&dev, &sms);
  if (rc != RSM_OK) return rc;
  const bool step = p.mode == ssm::kStep;
  const int ie = input_dtype == RSM_F32 ? 4 : 2, hpg = p.H / p.G;
  p.tokens_max = step ? p.window : std::min(p.R, ssm::kTokenMaxAll);
  const bool tc = input_dtype == RSM_BF16 && (step ? p.window > 1 && p.window <= 8 : p.window > 1 || p.state_dtype != RSM_F16);
  const int mode = step ? (tc ? 5 : p.window == 1 ? 1 : 2) : !tc ? 0 : p.window <= 8 ? 3 : 4;
  // rows of a head's x or a group's B start on 16 bytes wherever they are
  auto even = [&](const void* base, int64_t bs, int64_t ts) {
    return reinterpret_cast<uintptr_t>(base) % 16 == 0 && (p.units == 1 || bs * ie % 16 == 0) && (p.window == 1 || ts * ie % 16 == 0);
  };
  p.wide = even(p.x, p.x_bs, p.x_ts) &&
           ((step && !tc) || (even(p.B, p.B_bs, p.B_ts) && even(p.C, p.C_bs, p.C_ts))) &&
           (step || (reinterpret_cast<uintptr_t>(p.x_cache) % 16 == 0 && p.xc_ss * ie % 16 == 0 &&
                     reinterpret_cast<uintptr_t>(p.B_cache) % 16 == 0 && p.Bc_ss * ie % 16 == 0));
  // A CTA works on two heads at a time.  Many heads in all: as many a CTA as leave four
  // CTAs an SM, eight for sixteen heads, since a CTA's first loads wait for nothing to do
  // meanwhile, and two for one-byte states, whose heads take little time beside them; few:
  // two a CTA, to spread over the SMs.  (After a ring of 16, left with 2, 4 and 8: int8, 16
  // requests of 256 heads, 4 tokens: 16.7, 19.6 and 19.8 us; bf16, 32 requests, one: -, 29.9
  // and 33.  64 requests, 4 tokens, with 16 heads and 8: int8 44 and 51, bf16 54 and 52, to
  // bf16 states 124 and 116.)  Long rings take fewer, to leave three CTAs an SM.
  int per = 2;
  while (per < ssm::kTokenMaxHeads &&
         static_cast<int64_t>(p.units) * p.H / (2 * per) >= static_cast<int64_t>(es == 1 ? 2 : per < 8 ? 4 : 8) * sms)
    per *= 2;
  per = std::min(per, hpg);
  auto smem = [&](int n) { return ssm::token_smem(mode, ie, n, p.window, p.tokens_max); };
  while (per > 1 && smem(per) > ssm::kTokenMaxSmem) per = (per + 1) / 2;
  p.heads_per_cta = per;
  const int64_t parts = (hpg + per - 1) / per, grid = static_cast<int64_t>(p.units) * p.G * parts;
  const void* fn = ssm::token_kernel(input_dtype, p.state_dtype, mode);
  if (smem(per) > 48 * 1024) {
    rc = allow_smem(&g_token_ready[dev][input_dtype == RSM_F32 ? 1 : 0][p.state_dtype][mode], fn, ssm::kTokenMaxSmem);
    if (rc != RSM_OK) return rc;
  }
  return launch(fn, grid, ssm::kTokenThreads, &p, stream, smem(per));
}

// ---------------------------------------------------------------------------
// norms
// ---------------------------------------------------------------------------
bool is_input(int dt) { return dt == RSM_F32 || dt == RSM_BF16; }

// Eight columns at a time: every row of a tensor starts on 16 bytes (32 hold the eight of fp32).
bool vectors_fit(const void* base, int64_t stride, int64_t rows, int dt) {
  return reinterpret_cast<uintptr_t>(base) % 16 == 0 && (rows == 1 || stride * (dt == RSM_F32 ? 4 : 2) % 16 == 0);
}

int launch_norm(int kind, int input_dtype, int other_dtype, const rmsnorm::Params& p, void* stream) {
  const bool fits = p.group % 8 == 0 && vectors_fit(p.x, p.x_rs, p.rows, input_dtype) &&
                    vectors_fit(p.other, p.other_rs, p.rows, other_dtype) &&
                    vectors_fit(p.out, p.out_rs, p.rows, input_dtype) &&
                    (kind != 0 || vectors_fit(p.residual_out, p.res_rs, p.rows, other_dtype)) &&
                    reinterpret_cast<uintptr_t>(p.weight) % 16 == 0;
  const int64_t units = p.rows * p.groups;
  const int vecs = p.group / 8;
  if (!fits || vecs > 4096) return launch(rmsnorm::kernel(kind, input_dtype, other_dtype, 0, false, false), units, 256, &p, stream);
  int dev = 0, sms = 0;
  const int rc = device_sms(&dev, &sms);
  if (rc != RSM_OK) return rc;
  // Few groups: as many threads as there are vectors, for the shortest way
  // through; many: two vectors a thread, for more bytes in flight, and CTAs that stay,
  // 1024 threads an SM.
  const bool many = units >= 4 * static_cast<int64_t>(sms);
  const bool warp = vecs <= (many ? 64 : 32);
  const int v = warp ? (vecs <= 32 ? 1 : 2) : vecs > 2048 ? 4 : vecs > 1024 || many ? 2 : 1;
  const int threads = warp ? (many ? 128 : 32) : ((vecs + v - 1) / v + 31) / 32 * 32;
  const int64_t per = warp ? threads / 32 : 1, ctas = (units + per - 1) / per;
  const int64_t stay = static_cast<int64_t>(sms) * (1024 / threads);
  const bool loop = ctas > stay && many && rmsnorm::can_loop(kind, input_dtype == RSM_BF16, v);
  return launch(rmsnorm::kernel(kind, input_dtype, other_dtype, v, warp, loop), loop ? stay : ctas, threads, &p, stream);
}

}  // namespace

extern "C" {

int rsm_ssm_prefill(const rsm_ssm_prefill_args* a, void* stream) {
  int rc = validate(a, true);
  if (rc != RSM_OK) return rc;
  if (a->num_seqs == 0) return done();
  ssm::Params p{};
  p.x = a->x;
  p.B = a->B;
  p.C = a->C;
  p.dt = a->dt;
  p.A = a->A;
  p.D = a->D;
  p.cu_seqlens = a->cu_seqlens;
  p.state = a->state;
  p.src = a->initial_slots;
  p.dst = a->final_slots;
  p.out = a->out;
  p.status = a->device_status;
  p.tokens = a->tokens;
  p.x_ts = a->x_stride;
  p.B_ts = a->B_stride;
  p.C_ts = a->C_stride;
  p.dt_ts = a->dt_stride;
  p.out_ts = a->out_stride;
  p.state_ss = a->state_slot_stride;
  p.units = a->num_seqs;
  p.num_slots = a->num_slots;
  p.H = a->num_heads;
  p.G = a->num_groups;
  p.pad = a->pad_slot_id;
  p.mode = ssm::kPrefill;
  p.state_dtype = a->state_dtype;
  if (uses_tensor_cores(a) && tensor_maps_fit(a)) return launch_tc(a, p, stream);
  return launch_seq(p, a->input_dtype, a->dim, a->dstate, stream);
}

int64_t rsm_ssm_prefill_workspace(const rsm_ssm_prefill_args* a) {
  int rc = validate(a, false);
  if (rc != RSM_OK) return rc;
  int64_t bytes = 0;
  if (a->num_seqs > 0 && uses_tensor_cores(a)) {
    int dev = 0, sms = 0;
    rc = device_sms(&dev, &sms);
    if (rc != RSM_OK) return rc;
    bytes = workspace_bytes(plan_prefill(a, sms), a->num_heads);
  }
  done();
  return bytes;
}

int rsm_ssm_step(const rsm_ssm_step_args* a, void* stream) {
  if (a == nullptr) return fail(RSM_EINVAL, "args is NULL");
  if (!is_state(a->state_dtype, false))
    return fail(RSM_EINVAL, "state_dtype must be F32, BF16 or F16 (got %d): one-byte states are read by rsm_replayssm_decode and committed by rsm_materialize", a->state_dtype);
  int rc = check_batch(a);
  if (rc != RSM_OK) return rc;
  if (a->batch == 0) return done();
  rc = need({{a->src_slots, "src_slots"}});
  if (rc != RSM_OK) return rc;
  ssm::Params p{};
  fill_batch(a, &p);
  p.state = a->state;
  p.src = a->src_slots;
  p.dst = a->dst_slots;
  p.mode = ssm::kStep;
  return launch_tokens(p, a->input_dtype, a->dim, a->dstate, stream);
}

int rsm_replayssm_decode(const rsm_replayssm_decode_args* a, void* stream) {
  if (a == nullptr) return fail(RSM_EINVAL, "args is NULL");
  if (!is_state(a->state_dtype, true)) return fail(RSM_EINVAL, "unknown state_dtype %d", a->state_dtype);
  int rc = check_batch(a);
  if (rc != RSM_OK) return rc;
  const bool one_byte = a->state_dtype == RSM_I8 || a->state_dtype == RSM_FP8_E4M3;
  if (one_byte && (a->dim != 64 || a->dstate != 128))
    return fail(RSM_EINVAL, "one-byte state requires dim=64 and dstate=128 (got %d, %d)", a->dim, a->dstate);
  if (a->ring_buffer_len < 1) return fail(RSM_EINVAL, "ring_buffer_len must be >= 1 (got %d)", a->ring_buffer_len);
  if (a->window > a->ring_buffer_len || a->window > 64)
    return fail(RSM_EINVAL, "window (%d) must not exceed ring_buffer_len (%d) and 64", a->window, a->ring_buffer_len);
  if (a->batch == 0) return done();
  rc = need({{a->slots, "slots"}, {a->ring_start, "ring_start"}, {a->ring_len, "ring_len"}, {a->x_cache, "x_cache"},
             {a->B_cache, "B_cache"}, {a->dt_cache, "dt_cache"}});
  if (rc != RSM_OK) return rc;
  if (one_byte && a->state_scale == nullptr) return fail(RSM_EINVAL, "one-byte state needs state_scale");
  ssm::Params p{};
  fill_batch(a, &p);
  p.state = const_cast<void*>(a->state);
  p.scale = one_byte ? a->state_scale : nullptr;
  p.x_cache = a->x_cache;
  p.B_cache = a->B_cache;
  p.dt_cache = a->dt_cache;
  p.src = a->slots;
  p.ring_start = a->ring_start;
  p.ring_len = a->ring_len;
  p.scale_ss = a->scale_slot_stride;
  p.xc_ss = a->x_cache_slot_stride;
  p.Bc_ss = a->B_cache_slot_stride;
  p.dtc_ss = a->dt_cache_slot_stride;
  p.R = a->ring_buffer_len;
  p.mode = ssm::kDecode;
  return launch_tokens(p, a->input_dtype, a->dim, a->dstate, stream);
}

int rsm_add_rms_norm(const rsm_add_rms_norm_args* a, void* stream) {
  if (a == nullptr) return fail(RSM_EINVAL, "args is NULL");
  if (a->rows < 0) return fail(RSM_EINVAL, "rows must be >= 0");
  if (a->dim <= 0) return fail(RSM_EINVAL, "dim must be positive (got %d)", a->dim);
  if (!is_input(a->input_dtype) || !is_input(a->residual_dtype))
    return fail(RSM_EINVAL, "input_dtype and residual_dtype must be BF16 or F32 (got %d, %d)", a->input_dtype, a->residual_dtype);
  if (a->rows == 0) return done();
  const int rc = need({{a->x, "x"}, {a->residual, "residual"}, {a->weight, "weight"}, {a->out, "out"}, {a->residual_out, "residual_out"}});
  if (rc != RSM_OK) return rc;
  const rmsnorm::Params p{a->x, a->residual, a->weight, a->out, a->residual_out, a->rows, a->x_stride, a->residual_stride,
                          a->out_stride, a->residual_out_stride, a->dim, a->dim, 1, a->residual_scale, a->eps};
  return launch_norm(0, a->input_dtype, a->residual_dtype, p, stream);
}

int rsm_gated_rms_norm(const rsm_gated_rms_norm_args* a, void* stream) {
  if (a == nullptr) return fail(RSM_EINVAL, "args is NULL");
  if (a->rows < 0) return fail(RSM_EINVAL, "rows must be >= 0");
  if (a->dim <= 0) return fail(RSM_EINVAL, "dim must be positive (got %d)", a->dim);
  if (a->group_size <= 0 || a->dim % a->group_size != 0)
    return fail(RSM_EINVAL, "group_size (%d) must divide dim (%d)", a->group_size, a->dim);
  if (!is_input(a->input_dtype)) return fail(RSM_EINVAL, "input_dtype must be BF16 or F32 (got %d)", a->input_dtype);
  if (a->rows == 0) return done();
  const int rc = need({{a->x, "x"}, {a->z, "z"}, {a->weight, "weight"}, {a->out, "out"}});
  if (rc != RSM_OK) return rc;
  const rmsnorm::Params p{a->x, a->z, a->weight, a->out, nullptr, a->rows, a->x_stride, a->z_stride, a->out_stride, 0,
                          a->dim, a->group_size, a->dim / a->group_size, 1.0f, a->eps};
  return launch_norm(a->norm_before_gate ? 2 : 1, a->input_dtype, a->input_dtype, p, stream);
}

const char* rsm_block_last_error(void) { return g_error; }

int rsm_block_args_size(int index) {
  switch (index) {
    case 0: return static_cast<int>(sizeof(rsm_ssm_prefill_args));
    case 1: return static_cast<int>(sizeof(rsm_ssm_step_args));
    case 2: return static_cast<int>(sizeof(rsm_replayssm_decode_args));
    case 3: return static_cast<int>(sizeof(rsm_add_rms_norm_args));
    case 4: return static_cast<int>(sizeof(rsm_gated_rms_norm_args));
    default: return 0;
  }
}

}  // extern "C"
