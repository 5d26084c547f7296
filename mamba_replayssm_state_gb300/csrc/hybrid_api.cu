// hybrid_api.cu -- host side of the operators of hybrid stacks
// (include/replayssm_hybrid.h): argument validation, choice of kernel, launch.
// Nothing here reads device memory, allocates or synchronizes.
#include <cuda_runtime.h>

#include <algorithm>
#include <cfloat>
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <mutex>

#include "hybrid_params.h"

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

// Requests, sequences, windows and a token's or request's rows are counted in 32 bits on the device,
// with room for the step of a loop.
constexpr int64_t kMost = int64_t{1} << 30;
int at_most(int64_t n, const char* name) {
  return n <= kMost ? RSM_OK : fail(RSM_ENOTSUP, "%s (%lld) must be at most 2^30", name, static_cast<long long>(n));
}

bool is_input(int dt) { return dt == RSM_F32 || dt == RSM_BF16; }
int input_size(int dt) { return dt == RSM_F32 ? 4 : 2; }

int launch(const void* fn, int64_t grid, int threads, const void* params, void* stream, size_t smem = 0) {
  if (grid > 0x7FFFFFFFLL) return fail(RSM_EINVAL, "the call needs %lld blocks, more than 2^31-1", static_cast<long long>(grid));
  void* kargs[] = {const_cast<void*>(params)};
  const cudaError_t e = cudaLaunchKernel(fn, dim3(static_cast<unsigned>(grid)), dim3(threads), kargs, smem,
                                         static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return fail(RSM_ECUDA, "launch failed: %s", cudaGetErrorString(e));
  return done();
}

constexpr int kMaxDevices = 64;
std::mutex g_mu;
int g_sms[kMaxDevices];
bool g_attn_ready[kMaxDevices][2][3][33][2][2][3];  // input type, dim 64, 128, 256, rows, three CTAs an SM, low, loads

bool g_rotary_ready[kMaxDevices][2][2];  // input type, 16 bytes at a time

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

// Rows of a tensor start on 16 bytes; a stride that no second row needs is not looked at.
bool rows_fit(const void* base, int es, int64_t n0, int64_t s0, int64_t n1 = 1, int64_t s1 = 0, int64_t n2 = 1, int64_t s2 = 0) {
  return reinterpret_cast<uintptr_t>(base) % 16 == 0 && (n0 <= 1 || s0 * es % 16 == 0) && (n1 <= 1 || s1 * es % 16 == 0) &&
         (n2 <= 1 || s2 * es % 16 == 0);
}

// ---------------------------------------------------------------------------
// convolution
// ---------------------------------------------------------------------------
template <typename A>
int check_conv(const A* a) {
  if (a->channels <= 0) return fail(RSM_EINVAL, "channels must be positive (got %d)", a->channels);
  if (a->width < 2 || a->width > 4) return fail(RSM_ENOTSUP, "no kernel compiled for width %d: 2, 3 or 4", a->width);
  if (!is_input(a->input_dtype)) return fail(RSM_EINVAL, "input_dtype must be BF16 or F32 (got %d)", a->input_dtype);
  if (a->num_slots < 0) return fail(RSM_EINVAL, "num_slots must be >= 0 (got %d)", a->num_slots);
  return RSM_OK;
}

template <typename A>
hybrid::ConvParams conv_params(const A* a) {
  hybrid::ConvParams p{};
  p.x = a->x;
  p.weight = a->weight;
  p.bias = a->bias;
  p.cache = a->cache;
  p.slots = a->slots;
  p.positions = a->positions;
  p.out = a->out;
  p.status = a->device_status;
  p.x_ts = a->x_stride;
  p.cache_ss = a->cache_slot_stride;
  p.num_slots = a->num_slots;
  p.C = a->channels;
  p.R = a->cache_rows;
  p.silu = a->silu != 0;
  p.pad = a->pad_slot_id;
  return p;
}

// Eight bf16 or four fp32 channels at a time: every row, and the weights', starts on 16 bytes.
bool conv_vec(const hybrid::ConvParams& p, int dt, int width) {
  const int es = input_size(dt), v = 16 / es;
  return p.C % v == 0 && reinterpret_cast<uintptr_t>(p.weight) % 16 == 0 && width * v % 4 == 0 &&
         rows_fit(p.x, es, p.seqs, p.x_bs, 2, p.x_ts) && rows_fit(p.out, es, 2, p.out_ts) &&
         (p.cache == nullptr || rows_fit(p.cache, es, 2, p.C, p.num_slots, p.cache_ss));
}

// ---------------------------------------------------------------------------
// pages
// ---------------------------------------------------------------------------
int check_pages(const rsm_pages& pg, int heads, int kv_heads, int dim, int dt) {
  if (kv_heads <= 0 || heads <= 0 || heads % kv_heads != 0)
    return fail(RSM_EINVAL, "num_kv_heads (%d) must divide num_heads (%d)", kv_heads, heads);
  if (dim <= 0) return fail(RSM_EINVAL, "dim must be positive (got %d)", dim);
  if (dim > 256) return fail(RSM_ENOTSUP, "no kernel compiled for dim %d: at most 256", dim);
  if (!is_input(dt)) return fail(RSM_EINVAL, "input_dtype must be BF16 or F32 (got %d)", dt);
  if (pg.requests < 0) return fail(RSM_EINVAL, "requests must be >= 0 (got %d)", pg.requests);
  if (pg.page_size < 1) return fail(RSM_EINVAL, "page_size must be >= 1 (got %d)", pg.page_size);
  if (pg.num_pages < 0 || pg.table_width < 0) return fail(RSM_EINVAL, "num_pages and table_width must be >= 0");
  return at_most(pg.requests, "requests");
}

int need_pages(const rsm_pages& pg) {
  const int rc = need({{pg.lengths, "lengths"}});
  return rc != RSM_OK || pg.table_width == 0 ? rc : need({{pg.k, "k pages"}, {pg.v, "v pages"}, {pg.page_table, "page_table"}});
}

bool pages_fit(const rsm_pages& pg, int es, int kv_heads) {
  return rows_fit(pg.k, es, pg.num_pages, pg.k_page_stride, pg.page_size, pg.k_row_stride, kv_heads, pg.k_head_stride) &&
         rows_fit(pg.v, es, pg.num_pages, pg.v_page_stride, pg.page_size, pg.v_row_stride, kv_heads, pg.v_head_stride);
}

int validate(const rsm_paged_attention_args* a, bool pointers) {
  if (a == nullptr) return fail(RSM_EINVAL, "args is NULL");
  if (a->window < 1) return fail(RSM_EINVAL, "window must be >= 1 (got %d)", a->window);
  int rc = check_pages(a->pages, a->num_heads, a->num_kv_heads, a->dim, a->input_dtype);
  if (rc == RSM_OK) rc = at_most(static_cast<int64_t>(a->num_heads) * a->window, "num_heads * window");
  if (rc == RSM_OK && pointers && a->pages.requests > 0) {
    rc = need({{a->q, "q"}, {a->out, "out"}});
    if (rc == RSM_OK) rc = need_pages(a->pages);
  }
  return rc;
}

// How a call runs on the tiled kernel.
struct AttnPlan {
  int dim;        // columns that the kernel is compiled for
  int rows;       // of a unit
  int row_tiles;  // units of a key head
  int ctas;
  int64_t units;
  bool three;     // CTAs an SM
  bool low;       // bf16 weights as two values
  bool split;     // units may have more than one tile, so the join has to run
  int64_t bytes;  // of workspace
};

// Rows of the caches and heads are whole 16-byte vectors.
bool uses_tiles(const rsm_paged_attention_args* a) { return a->dim * input_size(a->input_dtype) % 16 == 0; }

// A unit has as many rows as the kernel takes, or the fewest that hold them all (bf16: in eights;
// fp32: 1, 2, 4 or 8): more than it takes are several units, which read the same keys and values
// (from the L2).
AttnPlan plan_attention(const rsm_paged_attention_args* a, int sms) {
  AttnPlan pl{};
  const int es = input_size(a->input_dtype);
  pl.dim = hybrid::attn_dim(a->dim);
  const int most_rows = hybrid::attn_rows(es, pl.dim);
  const int64_t rows = static_cast<int64_t>(a->num_heads / a->num_kv_heads) * a->window;
  const int64_t row_tiles = (rows + most_rows - 1) / most_rows, each = (rows + row_tiles - 1) / row_tiles;
  pl.row_tiles = static_cast<int>(row_tiles);
  pl.rows = es == 2 ? static_cast<int>((each + 7) / 8 * 8) : each > 4 ? 8 : each > 2 ? 4 : static_cast<int>(each);
  pl.units = row_tiles * a->num_kv_heads * a->pages.requests;
  pl.three = hybrid::attn_three(es, pl.dim, pl.rows, pl.units >= 2 * sms);
  pl.low = hybrid::attn_low(pl.dim, rows);
  const int64_t longest = static_cast<int64_t>(a->pages.table_width) * a->pages.page_size, tile = 4 * hybrid::attn_step(es, pl.dim, pl.three);
  const int64_t most = std::max<int64_t>((longest + tile - 1) / tile, 1);
  pl.split = most > 1;
  const int64_t resident = std::min<int64_t>(static_cast<int64_t>(sms) * hybrid::attn_ctas_per_sm(es, pl.dim, pl.three), 2 * hybrid::kAttnJoinThreads);
  pl.ctas = static_cast<int>(most >= resident ? resident : std::min(resident, pl.units * most));
  if (pl.split) pl.bytes = 2LL * pl.ctas * pl.rows * (pl.dim + 2) * 4;
  return pl;
}

hybrid::AttnKernels attention_kernels(int input_dtype, const AttnPlan& pl) {
  if (input_dtype == RSM_F32) return pl.dim == 64 ? hybrid::attn_f32_64(pl.rows) : pl.dim == 128 ? hybrid::attn_f32_128(pl.rows) : hybrid::attn_f32_256(pl.rows);
  return pl.dim == 64    ? hybrid::attn_bf16_64(pl.rows, pl.low)
         : pl.dim == 128 ? hybrid::attn_bf16_128(pl.rows, pl.three, pl.low)
                         : hybrid::attn_bf16_256(pl.rows);
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

// Tensor maps take strides from 16 bytes to 2^40; a stride that no second element needs is put at the least.
bool box_stride(int64_t n, int64_t stride, int es, cuuint64_t* out) {
  *out = n <= 1 ? 16 : static_cast<cuuint64_t>(stride) * es;
  return n <= 1 || (stride > 0 && stride < (int64_t{1} << 37));
}

// What the L2 fetches for a row of a head: no more than the row, behind which lies another head's
// (400000 tokens of 8 heads of 64, bf16, whose rows are 128 bytes: 150 us, 184 by 256 bytes).
CUtensorMapL2promotion row_promotion(int dim, int es) {
  return dim * es % 256 == 0 ? CU_TENSOR_MAP_L2_PROMOTION_L2_256B : dim * es % 128 == 0 ? CU_TENSOR_MAP_L2_PROMOTION_L2_128B : CU_TENSOR_MAP_L2_PROMOTION_L2_64B;
}

// The boxes of `rows` rows of one head, 128 bytes of columns each; false where a map cannot be made.
bool page_map(CUtensorMap* map, const void* base, const rsm_pages& pg, int es, int rows, int kv_heads, int dim, int64_t page, int64_t row,
              int64_t head) {
  const TensorMapEncodeFn encode = tensor_map_encoder();
  const cuuint64_t dims[4] = {static_cast<cuuint64_t>(dim), static_cast<cuuint64_t>(kv_heads), static_cast<cuuint64_t>(pg.page_size),
                              static_cast<cuuint64_t>(pg.num_pages)};
  cuuint64_t strides[3];
  if (encode == nullptr || pg.num_pages < 1 || !box_stride(kv_heads, head, es, &strides[0]) ||
      !box_stride(pg.page_size, row, es, &strides[1]) || !box_stride(pg.num_pages, page, es, &strides[2]))
    return false;
  const cuuint32_t box[4] = {128u / es, 1, static_cast<cuuint32_t>(rows), 1}, ones[4] = {1, 1, 1, 1};
  return encode(map, es == 2 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 4u, const_cast<void*>(base), dims, strides, box, ones,
                CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, row_promotion(dim, es),
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Rows from anywhere: the pages as one matrix of rows, of which a token's is page * page_rows + row
// + head * head_rows, its columns from head * head_columns on.
struct RowGrid {
  int64_t pitch, rows, columns, page_rows, head_rows, head_columns;
  bool operator==(const RowGrid& o) const {
    return pitch == o.pitch && rows == o.rows && columns == o.columns && page_rows == o.page_rows && head_rows == o.head_rows &&
           head_columns == o.head_columns;
  }
};

// False where the strides do not make one.
bool row_grid(RowGrid* r, const rsm_pages& pg, int kv_heads, int dim, int64_t page, int64_t row, int64_t head) {
  *r = {pg.page_size > 1 ? row : pg.num_pages > 1 ? page : dim, 0, dim, 0, 0, 0};
  if (r->pitch < dim || pg.num_pages < 1) return false;
  if (pg.num_pages > 1) {
    if (page % r->pitch != 0) return false;
    r->page_rows = page / r->pitch;
  }
  if (kv_heads > 1) {
    if (head >= dim && head < r->pitch)
      r->head_columns = head, r->columns = (kv_heads - 1) * head + dim;
    else if (head >= r->pitch && head % r->pitch == 0)
      r->head_rows = head / r->pitch;
    else
      return false;
  }
  if (r->columns > r->pitch || r->page_rows < 0 || r->page_rows > 0x7FFFFFFF || r->head_rows > 0x7FFFFFFF) return false;
  const int64_t pages = pg.num_pages - 1, heads = kv_heads - 1;  // (each product < 2^62)
  r->rows = pages * r->page_rows;
  if (r->rows > 0x7FFFFFFF || heads * r->head_rows > 0x7FFFFFFF) return false;
  r->rows += heads * r->head_rows + pg.page_size;
  return r->rows <= 0x7FFFFFFF;
}

bool row_map(CUtensorMap* map, const void* base, const RowGrid& r, int es, int dim) {
  const TensorMapEncodeFn encode = tensor_map_encoder();
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(r.columns), static_cast<cuuint64_t>(r.rows)};
  cuuint64_t stride;
  if (encode == nullptr || !box_stride(2, r.pitch, es, &stride)) return false;
  const cuuint32_t box[2] = {128u / es, 1}, ones[2] = {1, 1};
  return encode(map, es == 2 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 2u, const_cast<void*>(base), dims, &stride, box, ones,
                CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, row_promotion(dim, es),
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// How a call's keys and values are loaded, and its maps.
hybrid::AttnLoads choose_loads(const rsm_paged_attention_args* a, const AttnPlan& pl, hybrid::AttnTileParams* tp) {
  const rsm_pages& pg = a->pages;
  const int es = input_size(a->input_dtype), box = hybrid::attn_box(es, pl.dim), G = a->num_kv_heads;
  if (pg.page_size % box == 0 && page_map(&tp->k_map, pg.k, pg, es, box, G, a->dim, pg.k_page_stride, pg.k_row_stride, pg.k_head_stride) &&
      page_map(&tp->v_map, pg.v, pg, es, box, G, a->dim, pg.v_page_stride, pg.v_row_stride, pg.v_head_stride))
    return hybrid::AttnLoads::kBoxes;
  // (columns behind a padded head would be the next one's)
  RowGrid k, v;
  if (a->dim == pl.dim && row_grid(&k, pg, G, a->dim, pg.k_page_stride, pg.k_row_stride, pg.k_head_stride) &&
      row_grid(&v, pg, G, a->dim, pg.v_page_stride, pg.v_row_stride, pg.v_head_stride) && k == v && row_map(&tp->k_map, pg.k, k, es, a->dim) &&
      row_map(&tp->v_map, pg.v, v, es, a->dim)) {
    tp->p.page_rows = static_cast<int32_t>(k.page_rows);
    tp->p.head_rows = static_cast<int32_t>(k.head_rows);
    tp->p.head_columns = static_cast<int32_t>(k.head_columns);
    return hybrid::AttnLoads::kGather;
  }
  return hybrid::AttnLoads::kRows;
}

int launch_tiles(const rsm_paged_attention_args* a, const hybrid::AttnParams& base, const AttnPlan& pl, int dev, void* stream) {
  if (pl.split && (a->workspace == nullptr || a->workspace_bytes < pl.bytes || reinterpret_cast<uintptr_t>(a->workspace) % 256 != 0))
    return fail(RSM_EINVAL, "workspace of %lld bytes, 256-byte aligned, is needed", static_cast<long long>(pl.bytes));
  const int es = input_size(a->input_dtype), smem = hybrid::attn_smem(es, pl.dim, pl.rows, pl.three), step = hybrid::attn_step(es, pl.dim, pl.three);
  hybrid::AttnTileParams tp{};
  tp.p = base;
  hybrid::AttnParams& p = tp.p;
  p.part = static_cast<float*>(a->workspace);
  p.hidden = p.scale_log2 < 0.0f ? INFINITY : -INFINITY;
  if (p.scale_log2 == 0.0f) p.scale_log2 = FLT_MIN;  // (infinity times it stays infinity)
  p.row_tiles = pl.row_tiles;
  p.unit_end = hybrid::attn_unit_end(es, pl.dim, pl.rows);
  p.ctas = pl.ctas;
  p.tile_shift = step == 8 ? 5 : step == 16 ? 6 : 7;
  p.page_shift = -1;
  for (int k = 0; k < 31; ++k)
    if (a->pages.page_size == 1 << k) p.page_shift = k;
  p.q_pairs = reinterpret_cast<uintptr_t>(a->q) % 4 == 0 && (a->pages.requests == 1 || a->q_batch_stride % 2 == 0) &&
              (a->window == 1 || a->q_stride % 2 == 0);
  const hybrid::AttnLoads loads = choose_loads(a, pl, &tp);
  p.q_wide = rows_fit(a->q, es, a->pages.requests, a->q_batch_stride, a->window, a->q_stride);
  p.out_wide = reinterpret_cast<uintptr_t>(a->out) % 16 == 0;  // (a head is whole 16-byte vectors)
  const hybrid::AttnKernels kernels = attention_kernels(a->input_dtype, pl);
  const void* fn = kernels.tiles[static_cast<int>(loads)];
  int rc = allow_smem(&g_attn_ready[dev][a->input_dtype == RSM_F32][pl.dim / 128][pl.rows][pl.three][pl.low][static_cast<int>(loads)], fn, smem);
  if (rc != RSM_OK) return rc;
  rc = launch(fn, pl.ctas, hybrid::kAttnThreads, &tp, stream, smem);
  if (rc != RSM_OK || !pl.split) return rc;
  // The join's CTAs come while the first kernel's finish, and wait for it.  Where few units
  // are in many pieces each, their rows are shared out.
  const int64_t pieces = pl.ctas / pl.units + 1;
  const int rows = static_cast<int>(std::min<int64_t>(pl.rows, static_cast<int64_t>(p.per) * p.window));
  int parts = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(rows, pieces / 4))), by_unit = pl.units <= pl.ctas;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>((by_unit ? pl.units : pl.ctas) * parts));
  cfg.blockDim = dim3(hybrid::kAttnJoinThreads);
  cfg.dynamicSmemBytes = pl.ctas * sizeof(float);
  cfg.stream = static_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  void* kargs[] = {&p, &parts, &by_unit};
  const cudaError_t e = cudaLaunchKernelExC(&cfg, kernels.join, kargs);
  if (e != cudaSuccess) return fail(RSM_ECUDA, "launch failed: %s", cudaGetErrorString(e));
  return done();
}

}  // namespace

extern "C" {

int rsm_causal_conv(const rsm_causal_conv_args* a, void* stream) {
  if (a == nullptr) return fail(RSM_EINVAL, "args is NULL");
  if (a->num_seqs < 0 || a->tokens < 0) return fail(RSM_EINVAL, "num_seqs and tokens must be >= 0");
  int rc = check_conv(a);
  if (rc == RSM_OK) rc = at_most(a->num_seqs, "num_seqs");
  if (rc != RSM_OK) return rc;
  if (a->cache != nullptr && a->cache_rows < a->width - 1)
    return fail(RSM_EINVAL, "cache_rows (%d) must be at least width - 1 (%d)", a->cache_rows, a->width - 1);
  if (a->num_seqs == 0 || a->tokens == 0) return done();
  rc = need({{a->x, "x"}, {a->weight, "weight"}, {a->out, "out"}, {a->cu_seqlens, "cu_seqlens"}});
  if (rc != RSM_OK) return rc;
  if ((a->cache == nullptr) != (a->slots == nullptr)) return fail(RSM_EINVAL, "cache and slots go together");
  if (a->cache == nullptr && a->positions != nullptr) return fail(RSM_EINVAL, "positions need a cache");
  if (a->out == a->x) return fail(RSM_EINVAL, "out must not be x");
  hybrid::ConvParams p = conv_params(a);
  p.cu = a->cu_seqlens;
  p.tokens = a->tokens;
  p.out_ts = a->out_stride;
  p.seqs = a->num_seqs;
  const bool vec = conv_vec(p, a->input_dtype, a->width);
  const int per = hybrid::kConvThreads * hybrid::conv_channels(a->input_dtype, vec);
  p.cblocks = (a->channels + per - 1) / per;
  int dev = 0, sms = 0;
  rc = device_sms(&dev, &sms);
  if (rc != RSM_OK) return rc;
  // As many tokens a CTA as leave four CTAs an SM, in fours: at least four, for the shortest way through (37
  // tokens of 5376 channels: 4.9 us, 5.3 of eight, 6.3 of 16), at most 48, of which three rows are read
  // twice (8192 tokens of 18432 channels: 96.2 us, 96.3 of 32, 97.0 of 64).  In between (1024 and 4096 tokens of
  // 5376 channels) 12 and 44 take 9.7 and 22.6 us, four 14.2 and 43.9.
  p.block = static_cast<int>(std::min<int64_t>(48, std::max<int64_t>(1, (a->tokens * p.cblocks / (4 * sms) + 3) / 4) * 4));
  const int64_t blocks = (a->tokens + p.block - 1) / p.block;
  return launch(hybrid::conv_kernel(a->input_dtype, a->width, vec), blocks * p.cblocks, hybrid::kConvThreads, &p, stream);
}

int rsm_causal_conv_step(const rsm_causal_conv_step_args* a, void* stream) {
  if (a == nullptr) return fail(RSM_EINVAL, "args is NULL");
  if (a->batch < 0) return fail(RSM_EINVAL, "batch must be >= 0 (got %d)", a->batch);
  if (a->window < 1) return fail(RSM_EINVAL, "window must be >= 1 (got %d)", a->window);
  int rc = check_conv(a);
  if (rc != RSM_OK) return rc;
  if (a->cache_rows < static_cast<int64_t>(a->width) - 1 + a->window)
    return fail(RSM_EINVAL, "cache_rows (%d) must be at least width - 1 + window (%lld)", a->cache_rows,
                static_cast<long long>(a->width) - 1 + a->window);
  rc = at_most(a->window, "window");
  if (rc != RSM_OK) return rc;
  if (a->batch == 0) return done();
  rc = need({{a->x, "x"}, {a->weight, "weight"}, {a->out, "out"}, {a->cache, "cache"}, {a->slots, "slots"}, {a->positions, "positions"}});
  if (rc != RSM_OK) return rc;
  if (a->out == a->x) return fail(RSM_EINVAL, "out must not be x");
  hybrid::ConvParams p = conv_params(a);
  p.x_bs = a->x_batch_stride;
  if (a->window == 1) p.x_ts = 0;
  p.out_ts = a->channels;
  p.seqs = a->batch;
  p.window = a->window;
  const bool vec = conv_vec(p, a->input_dtype, a->width);
  const int per = hybrid::kConvThreads * hybrid::conv_channels(a->input_dtype, vec);
  p.cblocks = (a->channels + per - 1) / per;
  int dev = 0, sms = 0;
  rc = device_sms(&dev, &sms);
  if (rc != RSM_OK) return rc;
  // as many requests a CTA as bring all CTAs onto the SMs at once, four each
  p.block = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(hybrid::kConvStepRequests, (static_cast<int64_t>(a->batch) * p.cblocks + 4 * sms - 1) / (4 * sms))));
  const int64_t groups = (a->batch + p.block - 1) / p.block;
  return launch(hybrid::conv_step_kernel_of(a->input_dtype, a->width, vec), groups * p.cblocks, hybrid::kConvThreads, &p, stream);
}

// Tokens an SM up to which each has a CTA of its own; us so and in rings, 32 heads and 8 of 128:
//   bf16, turned whole, halves           2432 tokens 18.8 and 20.1, 3648 23.7 and 24.4, 6000 36.0 and 33.8
//   the same, heads of 72 (by fours)     912 6.5 and 9.1, 2000 13.2 and 14.5, 4000 21.9 and 22.2
//   the same, neighbours                 2000 17.7 and 18.5, 2432 20.9 and 20.3, 6000 42.0 and 34.0
//   64 of 128, either                    608 6.2 and 7.5, 760 7.2 and 8.5, 800 9.5 and 8.5, 2000 17.3 and 15.5
//   24 of 128, by fours (halves)         300 6.8 and 6.7, 450 7.3 and 7.2, 608 8.2 and 7.3, 2000 24.3 and 15.0
//   fp32, turned whole, halves           760 10.4 and 14.2, 3000 27.4 and 30.8, 16000 120.6 and 138.4 (rings of few tokens)
//   the same, neighbours                 760 12.2 and 13.4, 800 15.7 and 13.4, 2432 30.8 and 25.7, 16000 160.0 and 132.2
//   64 of 128, either                    608 10.5 and 10.7, 760 11.4 and 12.1, 800 14.6 and 12.4, 2000 23.8 and 21.9
// Five an SM are as many CTAs as it takes at once.
int64_t rotary_few(bool whole, bool by_fours, bool interleaved, int es) {
  if (!whole) return es == 2 && by_fours ? 3 : 5;
  if (es == 4) return interleaved ? 5 : INT32_MAX;
  return interleaved ? 14 : 24;
}

int rsm_rotary_append(const rsm_rotary_append_args* a, void* stream) {
  if (a == nullptr) return fail(RSM_EINVAL, "args is NULL");
  const bool packed = a->cu_seqlens != nullptr;
  if (!packed && a->window < 1) return fail(RSM_EINVAL, "window must be >= 1 (got %d)", a->window);
  if (packed && a->tokens < 0) return fail(RSM_EINVAL, "tokens must be >= 0");
  int rc = check_pages(a->pages, a->num_heads, a->num_kv_heads, a->dim, a->input_dtype);
  if (rc != RSM_OK) return rc;
  if (a->rotary_dim < 0 || a->rotary_dim % 2 != 0 || a->rotary_dim > a->dim)
    return fail(RSM_EINVAL, "rotary_dim (%d) must be even and at most dim (%d)", a->rotary_dim, a->dim);
  rc = at_most((static_cast<int64_t>(a->num_heads) + 2LL * a->num_kv_heads) * a->dim, "a token's values");
  if (rc == RSM_OK && !packed) rc = at_most(a->window, "window");
  if (rc != RSM_OK) return rc;
  if (a->pages.requests == 0 || (packed && a->tokens == 0)) return done();
  rc = need({{a->q, "q"}, {a->k, "k"}, {a->v, "v"}, {a->q_out, "q_out"}});
  if (rc == RSM_OK && a->rotary_dim > 0) rc = need({{a->inv_freq, "inv_freq"}});
  if (rc == RSM_OK) rc = need_pages(a->pages);
  if (rc != RSM_OK) return rc;
  const int64_t b = packed ? 1 : a->pages.requests, n = packed ? a->tokens : a->window;
  hybrid::RotaryParams p{};
  p.q = a->q;
  p.k = a->k;
  p.v = a->v;
  p.inv_freq = a->inv_freq;
  p.cu = a->cu_seqlens;
  p.q_out = a->q_out;
  p.status = a->device_status;
  p.pages = a->pages;
  p.tokens = b * n;
  p.q_bs = a->q_batch_stride;
  p.q_ts = a->q_stride;
  p.k_bs = a->k_batch_stride;
  p.k_ts = a->k_stride;
  p.v_bs = a->v_batch_stride;
  p.v_ts = a->v_stride;
  p.out_bs = a->out_batch_stride;
  p.out_ts = a->out_stride;
  p.window = a->window;
  p.H = a->num_heads;
  p.G = a->num_kv_heads;
  p.dim = a->dim;
  p.half = a->rotary_dim / 2;
  p.interleaved = a->interleaved != 0;
  p.amplitude = a->amplitude;
  const int es = input_size(a->input_dtype), v = 16 / es;
  const bool aligned = rows_fit(p.q, es, b, p.q_bs, n, p.q_ts) && rows_fit(p.k, es, b, p.k_bs, n, p.k_ts) && rows_fit(p.v, es, b, p.v_bs, n, p.v_ts) &&
                       rows_fit(p.q_out, es, b, p.out_bs, n, p.out_ts) && pages_fit(p.pages, es, a->num_kv_heads) && a->dim % v == 0;
  // 16 bytes of pairs at a time; bf16 halves that are not whole 16 bytes, as 24 turned columns', 8 (4 values); else one,
  // without rings (8 and 8000 tokens of 56 heads of 128, 24 turned columns: 5.5 and 45 us by fours, 12.6 and 209 by one)
  const int turned = a->interleaved ? a->rotary_dim : p.half;
  const int at_once = !aligned ? 1 : turned % v == 0 ? v : turned % 4 == 0 ? 4 : 1;
  const int64_t token = (static_cast<int64_t>(a->num_heads) + 2LL * a->num_kv_heads) * a->dim * es, place = token + 8 * p.half;
  int dev = 0, sms = 0;
  rc = device_sms(&dev, &sms);
  if (rc != RSM_OK) return rc;
  if (at_once == 1 || p.tokens <= rotary_few(a->rotary_dim == a->dim, at_once == 4, a->interleaved != 0, es) * sms || 2 * place > hybrid::kRotaryRingAlone)
    return launch(hybrid::rotary_token_kernel_of(a->input_dtype, at_once), p.tokens, hybrid::kRotaryPlainThreads, &p, stream);
  const bool alone = 3 * place > hybrid::kRotaryRing;  // (three places: one in, one turned, one out)
  p.stages = static_cast<int>(std::min<int64_t>(hybrid::kRotaryMaxStages, (alone ? hybrid::kRotaryRingAlone : hybrid::kRotaryRing) / place));
  const void* fn = hybrid::rotary_kernel(a->input_dtype, at_once);
  rc = allow_smem(&g_rotary_ready[dev][a->input_dtype == RSM_F32][at_once == v], fn, hybrid::kRotaryRingAlone);
  if (rc != RSM_OK) return rc;
  return launch(fn, std::min<int64_t>(p.tokens, (alone ? 1 : 2) * sms), hybrid::kRotaryThreads, &p, stream, p.stages * place);
}

int64_t rsm_paged_attention_workspace(const rsm_paged_attention_args* a) {
  int rc = validate(a, false);
  if (rc != RSM_OK) return rc;
  int64_t bytes = 0;
  if (a->pages.requests > 0) {
    int dev = 0, sms = 0;
    rc = device_sms(&dev, &sms);
    if (rc != RSM_OK) return rc;
    if (uses_tiles(a)) bytes = plan_attention(a, sms).bytes;
  }
  done();
  return bytes;
}

int rsm_paged_attention(const rsm_paged_attention_args* a, void* stream) {
  int rc = validate(a, true);
  if (rc != RSM_OK) return rc;
  if (a->pages.requests == 0) return done();
  hybrid::AttnParams p{};
  p.q = a->q;
  p.out = a->out;
  p.status = a->device_status;
  p.pages = a->pages;
  p.q_bs = a->q_batch_stride;
  p.q_ts = a->q_stride;
  p.window = a->window;
  p.H = a->num_heads;
  p.G = a->num_kv_heads;
  p.per = a->num_heads / a->num_kv_heads;
  p.dim = a->dim;
  p.scale_log2 = a->scale * 1.44269504088896340736f;
  if (uses_tiles(a) && pages_fit(a->pages, input_size(a->input_dtype), a->num_kv_heads)) {
    int dev = 0, sms = 0;
    rc = device_sms(&dev, &sms);
    if (rc != RSM_OK) return rc;
    return launch_tiles(a, p, plan_attention(a, sms), dev, stream);
  }
  return launch(hybrid::attn_plain_kernel(a->input_dtype), static_cast<int64_t>(a->pages.requests) * a->window * a->num_heads,
                hybrid::kAttnPlainThreads, &p, stream);
}

int rsm_copy_pages(const rsm_copy_pages_args* a, void* stream) {
  if (a == nullptr) return fail(RSM_EINVAL, "args is NULL");
  if (a->num_pools < 0 || a->num_pairs < 0 || a->num_pages < 0) return fail(RSM_EINVAL, "num_pools, num_pairs and num_pages must be >= 0");
  if (a->page_elements < 1) return fail(RSM_EINVAL, "page_elements must be >= 1 (got %lld)", static_cast<long long>(a->page_elements));
  if (a->dtype < RSM_F32 || a->dtype > RSM_FP8_E4M3) return fail(RSM_EINVAL, "unknown dtype %d", a->dtype);
  if (a->num_pools == 0 || a->num_pairs == 0) return done();
  const int rc = need({{a->page_ptrs, "page_ptrs"}, {a->page_strides, "page_strides"}, {a->src_pages, "src_pages"}, {a->dst_pages, "dst_pages"}});
  if (rc != RSM_OK) return rc;
  hybrid::CopyParams p{};
  p.ptrs = a->page_ptrs;
  p.strides = a->page_strides;
  p.src = a->src_pages;
  p.dst = a->dst_pages;
  p.status = a->device_status;
  p.esize = a->dtype == RSM_F32 ? 4 : a->dtype == RSM_BF16 || a->dtype == RSM_F16 ? 2 : 1;
  if (a->page_elements > (int64_t{1} << 40)) return fail(RSM_EINVAL, "page_elements must be at most 2^40");
  p.page_bytes = a->page_elements * p.esize;
  p.pools = a->num_pools;
  p.pairs = a->num_pairs;
  p.pages = a->num_pages;
  const int64_t pieces = (p.page_bytes + hybrid::kCopyBytes - 1) / hybrid::kCopyBytes;
  const int64_t units = static_cast<int64_t>(a->num_pools) * a->num_pairs;  // < 2^62; the product below could pass 2^63
  if (units > 0x7FFFFFFFLL || units * pieces > 0x7FFFFFFFLL) return fail(RSM_EINVAL, "the call needs more than 2^31-1 blocks");
  return launch(hybrid::copy_kernel(), units * pieces, hybrid::kCopyThreads, &p, stream);
}

const char* rsm_hybrid_last_error(void) { return g_error; }

int rsm_hybrid_args_size(int index) {
  switch (index) {
    case 0: return static_cast<int>(sizeof(rsm_causal_conv_args));
    case 1: return static_cast<int>(sizeof(rsm_causal_conv_step_args));
    case 2: return static_cast<int>(sizeof(rsm_rotary_append_args));
    case 3: return static_cast<int>(sizeof(rsm_paged_attention_args));
    case 4: return static_cast<int>(sizeof(rsm_copy_pages_args));
    default: return 0;
  }
}

}  // extern "C"
