// libspecverify C ABI, the drafter's side: drawing tokens, the top logits of a row, and the
// distillation loss on them with its gradient (include/specverify.h). Argument checks,
// workspace layout and kernel launches.
#include <algorithm>
#include <cmath>

#include "distill.cuh"
#include "sample.cuh"
#include "specverify.h"

namespace {

using sv::kThreads;
static_assert(SPEC_MAX_TOP_LOGITS <= kThreads, "finish_row: one of the k largest to a thread");
static_assert(SPEC_MAX_TOP_LOGITS <= sv::kMaxTeacher, "a list's entries");

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
size_t up256(size_t b) { return (b + 255) / 256 * 256; }
int elem_bytes(spec_dtype dt) { return dt == SPEC_BF16 ? 2 : 4; }
spec_status check_launch(cudaError_t e) { return e == cudaSuccess ? SPEC_OK : SPEC_ERR_CUDA; }

// Tiles of a row of V entries wherever it starts: a row off the 16-byte grid touches one vector
// more. Workspace sizes are those of the larger element type.
int tiles_of(int V, int elem) {
  const int per = 16 / elem;
  const int vecs = (V + 2 * per - 2) / per;
  return (vecs + sv::kTileVectors - 1) / sv::kTileVectors;
}

// The logit rows every call takes.
spec_status check_rows(const void* logits, spec_dtype dtype, int rows, int V,
                       long long row_stride) {
  if (!logits || rows <= 0 || V <= 0 || row_stride < V ||
      (dtype != SPEC_F32 && dtype != SPEC_BF16))
    return SPEC_ERR_INVALID_ARG;
  if (reinterpret_cast<uintptr_t>(logits) % size_t(elem_bytes(dtype)) != 0)
    return SPEC_ERR_INVALID_ARG;
  if (V > SPEC_MAX_VOCAB) return SPEC_ERR_UNSUPPORTED;
  if ((long long)rows * tiles_of(V, elem_bytes(dtype)) > 0x7fffffffLL) return SPEC_ERR_UNSUPPORTED;
  return SPEC_OK;
}

struct TileLayout {
  size_t left, parts, lists, total;
};
TileLayout tile_layout(int rows, int n, int cap) {
  const size_t tiles = size_t(rows) * n;
  TileLayout l;
  l.left = 0;
  l.parts = up256(size_t(rows) * sizeof(sv::RowLeft));
  l.lists = l.parts + up256(tiles * sv::kWarps * sizeof(sv::WarpPart));
  l.total = l.lists + up256(tiles * size_t(cap) * sizeof(unsigned long long));
  return l;
}

// Blocks of a row's cluster: one per tile up to eight (the portable most), else the fewest that
// keep the busiest block's tiles down.
int blocks_of(int n) {
  const int each = (n + 7) / 8;
  return (n + each - 1) / each;
}

// (a list never holds more than the row)
int sample_cap(int V, int n) { return std::min(V, sv::list_cap(sv::kMaxJ, n)); }
int top_cap(int k, int V, int n) { return std::min(V, sv::list_cap(sv::list_aim(k, n), n)); }

sv::TileJob tile_job(const void* logits, long long stride, int rows, int V, int n, int cap,
                     int pool, void* workspace) {
  const TileLayout l = tile_layout(rows, n, cap);
  char* ws = static_cast<char*>(workspace);
  return sv::TileJob{logits, stride, rows, V, n, blocks_of(n), cap, pool,
                     reinterpret_cast<sv::WarpPart*>(ws + l.parts),
                     reinterpret_cast<unsigned long long*>(ws + l.lists),
                     reinterpret_cast<sv::RowLeft*>(ws + l.left)};
}

bool bad_temp(float t) { return !(t >= 0.0f && t < INFINITY); }

// Clusters of `ctas` blocks (1: none). A launch `after` another of its call is let in as that one's
// last blocks start, and waits (griddepcontrol.wait) where it needs what they leave.
template <typename K, typename Job>
cudaError_t launch(K kernel, const Job& j, unsigned clusters, int ctas, int threads, size_t smem,
                   bool after, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(clusters * unsigned(ctas), 1, 1);
  cfg.blockDim = dim3(unsigned(threads), 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  unsigned n = 0;
  if (ctas > 1) {
    attr[n].id = cudaLaunchAttributeClusterDimension;
    attr[n].val.clusterDim.x = unsigned(ctas);
    attr[n].val.clusterDim.y = 1;
    attr[n++].val.clusterDim.z = 1;
  }
  if (after) {
    attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[n++].val.programmaticStreamSerializationAllowed = 1;
  }
  cfg.attrs = attr;
  cfg.numAttrs = n;
  return cudaLaunchKernelEx(&cfg, kernel, j);
}

// More than the default 48 KB of shared memory for a kernel, its own included, asked for on every
// launch: the attribute belongs to the current device. Always for `most`, the most that any launch of
// the kernel takes: another thread's call with a smaller pool must not lower it between this and a
// launch, nor below what a captured one takes.
template <typename K>
cudaError_t allow_smem(K kernel, size_t bytes, size_t most) {
  if (bytes <= 40 * 1024) return cudaSuccess;
  return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, int(most));
}

// Entries that top-k keeps of every row, where that is known here (V: all, or not known).
int kept_by_all(const sv::TopJob& j) { return j.k; }
int kept_by_all(const sv::SampleJob& j) {
  const bool draws = j.row_temp || j.temp > 0.0f;
  return draws && !j.row_top_k && j.top_k > 1 && j.top_k < j.t.V ? j.top_k : j.t.V;
}

// One launch while all blocks fit on 148 SMs, two to each; else the tiles, the finishing, and the
// rows that it leaves (a cluster per row, a block per SM).
template <typename T, typename Job, typename Deep>
cudaError_t launch_rows(Job j, Deep deep, cudaStream_t s) {
  static_assert(sizeof(sv::DeepSmem) <= sizeof(sv::PoolSmem) + 2 * 1024 * 8, "one memory for both");
  const size_t pool = sv::pool_bytes(j.t.pool), most_pool = sv::pool_bytes(sv::kPoolCap);
  // a few rows get eight blocks each whatever their tiles: a row that its pool does not settle is
  // gone over by all of them (48,288 entries: 110 -> 84 us, against 2 to 4 blocks)
  if (j.t.rows <= 148 / 8) j.t.blocks = 8;
  if ((long long)j.t.rows * j.t.blocks <= 148LL * 2) {
    auto kernel = sv::row_kernel<T, Job>;
    const size_t smem = std::max(pool, sizeof(sv::TileSmem));
    const cudaError_t e = allow_smem(kernel, smem, std::max(most_pool, sizeof(sv::TileSmem)));
    if (e != cudaSuccess) return e;
    return launch(kernel, j, unsigned(j.t.rows), j.t.blocks, kThreads, smem, false, s);
  }
  sv::row_tile_kernel<T, Job><<<unsigned(j.t.rows * (long long)j.t.n), kThreads, 0, s>>>(j);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const bool brief = j.t.rows >= sv::kShortRows && kept_by_all(j) <= sv::kShortK;
  auto finish = brief ? sv::row_short_kernel<T, Job> : sv::row_finish_kernel<T, Job>;
  const size_t smem = brief ? sv::short_bytes(j.t.pool) : pool;
  const int blocks = brief ? (j.t.rows + sv::kWarps - 1) / sv::kWarps : j.t.rows;
  e = allow_smem(finish, smem, brief ? sv::short_bytes(sv::kPoolCap) : most_pool);
  if (e != cudaSuccess) return e;
  // (let in early, a few blocks would share the SMs that are free first, and each takes longer: 64
  // rows of 128,256 57 us instead of 51; many gain, 2,048 rows 152 instead of 158)
  e = launch(finish, j, unsigned(blocks), 1, kThreads, smem, j.t.rows > 148, s);
  if (e != cudaSuccess) return e;
  const int most = 148 / sv::kDeepCtas;
  return launch(deep, j, unsigned(j.t.rows < most ? j.t.rows : most), sv::kDeepCtas,
                sv::kDeepThreads, 0, true, s);
}

template <typename T>
cudaError_t launch_sample(const sv::SampleJob& j, cudaStream_t s) {
  return launch_rows<T>(j, sv::sample_deep_kernel<T>, s);
}

template <typename T>
cudaError_t launch_top(const sv::TopJob& j, cudaStream_t s) {
  return launch_rows<T>(j, sv::top_deep_kernel<T>, s);
}

// Rows of up to sixteen tiles: a cluster per row (more than eight blocks are not portable, and asked
// for), after, or beside, the lists' kernel.
template <typename T, bool kGrad, bool kList>
cudaError_t launch_distill_row(const sv::DistillRowJob& j, cudaStream_t s) {
  if (!kList) {
    sv::distill_list_kernel<T>
        <<<unsigned((j.rows + sv::kWarps - 1) / sv::kWarps), kThreads, 0, s>>>(j);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  auto kernel = sv::distill_row_kernel<T, kGrad, kList>;
  if (j.n > 8) {
    const cudaError_t e =
        cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
  }
  return launch(kernel, j, unsigned(j.rows), j.n, kThreads, 0, !kList, s);
}
// Calls of up to a block per SM: one launch, the list's side done by the rows' own blocks.
bool small_call(int rows, int n) { return (long long)rows * n <= 148; }

cudaError_t launch_distill_both(spec_dtype dt, const sv::DistillRowJob& j, cudaStream_t s) {
  const bool small = small_call(j.rows, j.n);
  if (dt == SPEC_BF16)
    return small ? launch_distill_row<__nv_bfloat16, true, true>(j, s)
                 : launch_distill_row<__nv_bfloat16, true, false>(j, s);
  return small ? launch_distill_row<float, true, true>(j, s)
               : launch_distill_row<float, true, false>(j, s);
}

// The loss in two kernels, the second let in as the first ends.
template <typename T>
cudaError_t launch_distill_loss(const sv::DistillJob& j, cudaStream_t s) {
  sv::distill_tile_kernel<T><<<unsigned(j.rows * (long long)j.n), kThreads, 0, s>>>(j);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  return launch(sv::distill_finish_kernel<T>, j, unsigned((j.rows + sv::kWarps - 1) / sv::kWarps),
                1, kThreads, 0, true, s);
}

template <typename T>
cudaError_t launch_distill_grad(const sv::DistillGradJob& j, cudaStream_t s) {
  sv::distill_grad_kernel<T><<<unsigned(j.rows * (long long)j.n), kThreads, 0, s>>>(j);
  return cudaGetLastError();
}

spec_status check_teacher(const int32_t* ids, const float* values, int k, float temp) {
  if (!ids || !values || k <= 0 || !(temp > 0.0f && temp < INFINITY)) return SPEC_ERR_INVALID_ARG;
  if (k > SPEC_MAX_TOP_LOGITS) return SPEC_ERR_UNSUPPORTED;
  return SPEC_OK;
}

// The gradient's rows: in their place, over the logits themselves or clear of them.
spec_status check_grad(const void* logits, spec_dtype dt, int rows, int V, long long row_stride,
                       const void* grad, long long grad_stride) {
  const long long e = elem_bytes(dt);
  if (!grad || grad_stride < V || reinterpret_cast<uintptr_t>(grad) % size_t(e) != 0)
    return SPEC_ERR_INVALID_ARG;
  const long long d = (long long)(reinterpret_cast<uintptr_t>(grad)) -
                      (long long)(reinterpret_cast<uintptr_t>(logits));
  const bool alike = rows == 1 || row_stride == grad_stride;
  if (d == 0) return alike ? SPEC_OK : SPEC_ERR_INVALID_ARG;
  using Wide = __int128;  // (a stride may be anything)
  if (d >= (Wide(rows - 1) * row_stride + V) * e || -d >= (Wide(rows - 1) * grad_stride + V) * e)
    return SPEC_OK;
  if (rows == 1 || !alike) return SPEC_ERR_INVALID_ARG;
  // side by side in one buffer's rows
  const Wide period = Wide(row_stride) * e, at = (d % period + period) % period;
  return at >= V * e && at <= period - V * e ? SPEC_OK : SPEC_ERR_INVALID_ARG;
}

struct DistillLayout {
  size_t stats, parts, total;
};
DistillLayout distill_layout(int rows, int n) {
  DistillLayout l;
  l.stats = 0;
  // (the same place holds the lists' side in calls on shorter rows)
  l.parts = up256(size_t(rows) * sizeof(sv::ListSide));
  l.total = l.parts + up256(size_t(rows) * n * sv::kWarps * sizeof(sv::DistillPart));
  return l;
}

}  // namespace

extern "C" {

size_t spec_sample_workspace_size(int rows, int V) {
  if (rows <= 0 || V <= 0 || V > SPEC_MAX_VOCAB) return 0;
  const int n2 = tiles_of(V, 2), n4 = tiles_of(V, 4);
  const size_t a = tile_layout(rows, n2, sample_cap(V, n2)).total;
  const size_t b = tile_layout(rows, n4, sample_cap(V, n4)).total;
  return a > b ? a : b;
}

spec_status spec_sample(const void* logits, spec_dtype dtype, int rows, int V, int64_t row_stride,
                        const float* uniforms, float temp, int top_k, float top_p, float min_p,
                        const float* row_temp, const int32_t* row_top_k, const float* row_top_p,
                        const float* row_min_p, int32_t* tokens, float* probs, void* workspace,
                        size_t workspace_bytes, void* stream) {
  if (!uniforms || !tokens) return SPEC_ERR_INVALID_ARG;
  if ((!row_temp && bad_temp(temp)) || (!row_top_p && !(top_p > 0.0f)) ||
      (!row_min_p && !(min_p >= 0.0f && min_p <= 1.0f)))
    return SPEC_ERR_INVALID_ARG;
  const spec_status st = check_rows(logits, dtype, rows, V, row_stride);
  if (st != SPEC_OK) return st;
  if (!workspace || !aligned16(workspace) ||
      workspace_bytes < spec_sample_workspace_size(rows, V))
    return SPEC_ERR_WORKSPACE;
  const int n = tiles_of(V, elem_bytes(dtype));
  // a top_k that holds for every row tells the pool's size
  const int want = !row_top_k && top_k >= 1 && top_k < V ? top_k : -1;
  sv::SampleJob j = {tile_job(logits, row_stride, rows, V, n, sample_cap(V, n),
                              sv::pool_cap(want, n), workspace),
                     uniforms, temp, top_p, min_p, top_k,
                     row_temp, row_top_k, row_top_p, row_min_p, tokens, probs};
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return check_launch(dtype == SPEC_BF16 ? launch_sample<__nv_bfloat16>(j, s)
                                         : launch_sample<float>(j, s));
}

size_t spec_top_logits_workspace_size(int rows, int V, int k) {
  if (rows <= 0 || V <= 0 || V > SPEC_MAX_VOCAB || k <= 0 || k > V || k > SPEC_MAX_TOP_LOGITS)
    return 0;
  const int n2 = tiles_of(V, 2), n4 = tiles_of(V, 4);
  const size_t a = tile_layout(rows, n2, top_cap(k, V, n2)).total;
  const size_t b = tile_layout(rows, n4, top_cap(k, V, n4)).total;
  return a > b ? a : b;
}

spec_status spec_top_logits(const void* logits, spec_dtype dtype, int rows, int V,
                            int64_t row_stride, int k, float temp, int32_t* ids, float* values,
                            float* lse, void* workspace, size_t workspace_bytes, void* stream) {
  if (!ids || !values || k <= 0 || k > V || !(temp > 0.0f && temp < INFINITY))
    return SPEC_ERR_INVALID_ARG;
  const spec_status st = check_rows(logits, dtype, rows, V, row_stride);
  if (st != SPEC_OK) return st;
  if (k > SPEC_MAX_TOP_LOGITS) return SPEC_ERR_UNSUPPORTED;
  if (!workspace || !aligned16(workspace) ||
      workspace_bytes < spec_top_logits_workspace_size(rows, V, k))
    return SPEC_ERR_WORKSPACE;
  const int n = tiles_of(V, elem_bytes(dtype));
  sv::TopJob j = {tile_job(logits, row_stride, rows, V, n, top_cap(k, V, n), sv::pool_cap(k, n),
                           workspace),
                  k, temp, sv::log2_scale(double(temp)), ids, values, lse};
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return check_launch(dtype == SPEC_BF16 ? launch_top<__nv_bfloat16>(j, s)
                                         : launch_top<float>(j, s));
}

size_t spec_distill_workspace_size(int rows, int V) {
  if (rows <= 0 || V <= 0 || V > SPEC_MAX_VOCAB) return 0;
  return distill_layout(rows, tiles_of(V, 4)).total;
}

spec_status spec_distill_loss(const void* logits, spec_dtype dtype, int rows, int V,
                              int64_t row_stride, const int32_t* teacher_ids,
                              const float* teacher_logits, const float* teacher_lse, int k,
                              float temp, float* loss, float* stats, void* workspace,
                              size_t workspace_bytes, void* stream) {
  if (!loss || !stats || !aligned16(stats)) return SPEC_ERR_INVALID_ARG;
  spec_status st = check_teacher(teacher_ids, teacher_logits, k, temp);
  if (st != SPEC_OK) return st;
  st = check_rows(logits, dtype, rows, V, row_stride);
  if (st != SPEC_OK) return st;
  if (!workspace || !aligned16(workspace) ||
      workspace_bytes < spec_distill_workspace_size(rows, V))
    return SPEC_ERR_WORKSPACE;
  const int n = tiles_of(V, elem_bytes(dtype));
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (n <= sv::kMaxRowBlocks && small_call(rows, n)) {
    sv::DistillRowJob r = {logits, row_stride, rows, V, n, k, 1.0 / double(temp),
                           sv::log2_scale(double(temp)),
                           teacher_ids, teacher_logits, teacher_lse, nullptr, loss, stats,
                           nullptr, 0, static_cast<sv::ListSide*>(workspace)};
    return check_launch(dtype == SPEC_BF16 ? launch_distill_row<__nv_bfloat16, false, true>(r, s)
                                           : launch_distill_row<float, false, true>(r, s));
  }
  char* ws = static_cast<char*>(workspace);
  sv::DistillJob j = {logits, row_stride, rows, V, n, k, 1.0 / double(temp),
                      sv::log2_scale(double(temp)), teacher_ids, teacher_logits, teacher_lse,
                      reinterpret_cast<sv::DistillPart*>(ws + distill_layout(rows, n).parts),
                      loss, stats};
  return check_launch(dtype == SPEC_BF16 ? launch_distill_loss<__nv_bfloat16>(j, s)
                                         : launch_distill_loss<float>(j, s));
}

spec_status spec_distill_grad(const void* logits, spec_dtype dtype, int rows, int V,
                              int64_t row_stride, const int32_t* teacher_ids,
                              const float* teacher_logits, const float* teacher_lse, int k,
                              float temp, const float* stats, const float* grad_loss, void* grad,
                              int64_t grad_stride, void* stream) {
  if (!stats || !aligned16(stats)) return SPEC_ERR_INVALID_ARG;
  spec_status st = check_teacher(teacher_ids, teacher_logits, k, temp);
  if (st != SPEC_OK) return st;
  st = check_rows(logits, dtype, rows, V, row_stride);
  if (st != SPEC_OK) return st;
  st = check_grad(logits, dtype, rows, V, row_stride, grad, grad_stride);
  if (st != SPEC_OK) return st;
  const int n = tiles_of(V, elem_bytes(dtype));
  sv::DistillGradJob j = {logits, row_stride, rows, V, n, k, temp, sv::log2_scale(double(temp)),
                          teacher_ids, teacher_logits, teacher_lse, stats, grad_loss, grad,
                          grad_stride};
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return check_launch(dtype == SPEC_BF16 ? launch_distill_grad<__nv_bfloat16>(j, s)
                                         : launch_distill_grad<float>(j, s));
}

spec_status spec_distill_loss_grad(const void* logits, spec_dtype dtype, int rows, int V,
                                   int64_t row_stride, const int32_t* teacher_ids,
                                   const float* teacher_logits, const float* teacher_lse, int k,
                                   float temp, const float* grad_loss, float* loss, void* grad,
                                   int64_t grad_stride, void* workspace, size_t workspace_bytes,
                                   void* stream) {
  if (!loss) return SPEC_ERR_INVALID_ARG;
  spec_status st = check_teacher(teacher_ids, teacher_logits, k, temp);
  if (st != SPEC_OK) return st;
  st = check_rows(logits, dtype, rows, V, row_stride);
  if (st != SPEC_OK) return st;
  st = check_grad(logits, dtype, rows, V, row_stride, grad, grad_stride);
  if (st != SPEC_OK) return st;
  if (!workspace || !aligned16(workspace) ||
      workspace_bytes < spec_distill_workspace_size(rows, V))
    return SPEC_ERR_WORKSPACE;
  const int n = tiles_of(V, elem_bytes(dtype));
  if (n <= sv::kMaxRowBlocks) {
    sv::DistillRowJob r = {logits, row_stride, rows, V, n, k, 1.0 / double(temp),
                           sv::log2_scale(double(temp)),
                           teacher_ids, teacher_logits, teacher_lse, grad_loss, loss, nullptr,
                           grad, grad_stride, static_cast<sv::ListSide*>(workspace)};
    return check_launch(launch_distill_both(dtype, r, static_cast<cudaStream_t>(stream)));
  }
  // longer rows, in two passes, the statistics at the head of the workspace (the tiles behind them)
  float* stats = static_cast<float*>(workspace);
  st = spec_distill_loss(logits, dtype, rows, V, row_stride, teacher_ids, teacher_logits,
                         teacher_lse, k, temp, loss, stats, workspace, workspace_bytes, stream);
  if (st != SPEC_OK) return st;
  return spec_distill_grad(logits, dtype, rows, V, row_stride, teacher_ids, teacher_logits,
                           teacher_lse, k, temp, stats, grad_loss, grad, grad_stride, stream);
}

}  // extern "C"
