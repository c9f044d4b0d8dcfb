// C ABI of liblocks.so: argument validation, workspace carving and launches
// on the caller's stream.  No allocation, no synchronisation (except
// locks_read_status, which documents it).
#include <math.h>
#include <stdio.h>

#include <initializer_list>

#include "common.cuh"
#include "launch.h"

using namespace locks;

namespace locks {
std::atomic<long long> g_kernel_launches{0};
}

static thread_local int g_last_cuda = 0;

static locks_status_t fail_cuda(cudaError_t e) {
  g_last_cuda = (int)e;
  return LOCKS_ERR_CUDA;
}

static size_t round_up(size_t x, size_t a) { return (x + a - 1) / a * a; }

// bytes of the scoring region: s_hat [batch][h_kv][G][max_pages] float and
// selection keys [batch][h_kv][max_pages] u32
static size_t score_region(int batch, int h_q, int h_kv, int max_pages) {
  const size_t G = (size_t)(h_q / h_kv);
  return round_up((size_t)batch * h_kv * G * max_pages * 4, 256) +
         round_up((size_t)batch * h_kv * max_pages * 4, 256);
}

// Decode partials: one slot per (unit, warp) piece, slot index unit + warp,
// so units + (warps launched) slots suffice.  The grid never has more warps
// than list positions nor more than kDecMaxWarps.
constexpr long long kDecMaxWarps = 8192;

static long long decode_warps_cap(int batch, int h_kv, int list_len) {
  long long w = (long long)batch * h_kv * list_len;
  if (w > kDecMaxWarps) w = kDecMaxWarps;
  return w < 1 ? 1 : w;
}

// bytes of the decode region: the unit layout written by the decode kernel
// (int meta[batch + 2]), o_part [slots][G][128] float and lse_part
// [slots][G] float
static size_t decode_meta_bytes(int batch) {
  return round_up(((size_t)batch + 2) * 4, 256);
}
static size_t decode_slots(int batch, int h_kv, int list_len) {
  return (size_t)batch * h_kv + (size_t)decode_warps_cap(batch, h_kv, list_len);
}
static size_t decode_region(int batch, int h_q, int h_kv, int list_len) {
  const size_t rows = decode_slots(batch, h_kv, list_len) * (size_t)(h_q / h_kv);
  return decode_meta_bytes(batch) + round_up(rows * kDim * 4, 256) +
         round_up(rows * 4, 256);
}

// the same region as the quantised cache's decode lays it out
struct DecodeRegion {
  int *meta;
  float *o_part;
  float2 *ml_part;
  size_t bytes;
};
// partials hold 128 sums, a reference and a sum of weights per head
static DecodeRegion qdecode_region(uint8_t *at, int batch, int h_q, int h_kv,
                                   int list_len) {
  const size_t rows = decode_slots(batch, h_kv, list_len) * (size_t)(h_q / h_kv);
  const size_t meta = decode_meta_bytes(batch);
  const size_t sums = round_up(rows * kDim * 4, 256);
  return {reinterpret_cast<int *>(at), reinterpret_cast<float *>(at + meta),
          reinterpret_cast<float2 *>(at + meta + sums),
          meta + sums + round_up(rows * 8, 256)};
}

static bool heads_ok(int h_q, int h_kv) {
  return h_kv >= 1 && h_q >= h_kv && h_q % h_kv == 0;
}

static locks_status_t check_select_args(int batch, int h_q, int h_kv,
                                        int max_pages, int k,
                                        const int32_t *seq_lens,
                                        int32_t *idx_out, void *workspace) {
  if (batch < 0 || max_pages < 1 || k < 2 || !heads_ok(h_q, h_kv))
    return LOCKS_ERR_INVALID_ARG;
  if (h_q / h_kv > kMaxGroup) return LOCKS_ERR_UNSUPPORTED;
  if (batch > 65535 || h_kv > 65535) return LOCKS_ERR_UNSUPPORTED;
  if ((long long)max_pages * kPage > 0x7fffffffLL) return LOCKS_ERR_UNSUPPORTED;
  if (batch > 0 && (!seq_lens || !idx_out || !workspace))
    return LOCKS_ERR_INVALID_ARG;
  return LOCKS_OK;
}

locks_status_t locks::score_select(const void *q, const void *summaries,
                                   const int32_t *seq_lens, int batch, int h_q,
                                   int h_kv, int max_pages, int k,
                                   int32_t *idx_out, void *workspace,
                                   size_t workspace_bytes, cudaStream_t stream,
                                   bool after_query) {
  locks_status_t st = check_select_args(batch, h_q, h_kv, max_pages, k,
                                        seq_lens, idx_out, workspace);
  if (st != LOCKS_OK) return st;
  if (batch == 0) return LOCKS_OK;
  if (!q || !summaries) return LOCKS_ERR_INVALID_ARG;
  if (batch > score_max_batch()) return LOCKS_ERR_UNSUPPORTED;
  if (workspace_bytes < kWsHeader + score_region(batch, h_q, h_kv, max_pages))
    return LOCKS_ERR_WORKSPACE;
  const int G = h_q / h_kv;
  uint8_t *ws = static_cast<uint8_t *>(workspace);
  int32_t *status = reinterpret_cast<int32_t *>(ws);
  float *s_hat = reinterpret_cast<float *>(ws + kWsHeader);
  uint32_t *keys = reinterpret_cast<uint32_t *>(
      ws + kWsHeader + round_up((size_t)batch * h_kv * G * max_pages * 4, 256));
  // short page lists on fewer units than SMs: one launch, the selection
  // done by the cluster that scored the unit
  const int cluster = fused_cluster_size(batch, h_kv, G, max_pages);
  if (cluster > 0) {
    const cudaError_t e = launch_score_select_fused(
        q, summaries, seq_lens, batch, h_kv, G, max_pages, k, cluster, s_hat,
        idx_out, status, stream, after_query);
    return e == cudaSuccess ? LOCKS_OK : fail_cuda(e);
  }
  cudaError_t e = launch_score(q, summaries, seq_lens, batch, h_kv, G,
                               max_pages, s_hat, status, stream, after_query);
  if (e != cudaSuccess) return fail_cuda(e);
  e = launch_select(s_hat, seq_lens, batch, h_kv, G, max_pages, k,
                    LOCKS_MERGE_SHARE_AVERAGE, idx_out, keys, status, stream);
  return e == cudaSuccess ? LOCKS_OK : fail_cuda(e);
}

locks_status_t locks::sparse_decode(
    const void *q, const void *k_cache, const void *v_cache,
    int64_t num_phys_pages, const int32_t *page_table,
    const int32_t *seq_lens, const int32_t *idx, int k, int batch, int h_q,
    int h_kv, int max_pages, void *o_out, float *lse_out, void *workspace,
    size_t workspace_bytes, cudaStream_t stream, int32_t *status_mirror) {
  if (batch < 0 || max_pages < 1 || num_phys_pages < 1 || !heads_ok(h_q, h_kv))
    return LOCKS_ERR_INVALID_ARG;
  if (idx && k < 1) return LOCKS_ERR_INVALID_ARG;
  if (h_q / h_kv > kMaxGroup) return LOCKS_ERR_UNSUPPORTED;
  if (batch > 65535 || h_kv > 65535) return LOCKS_ERR_UNSUPPORTED;
  if ((long long)max_pages * kPage > 0x7fffffffLL) return LOCKS_ERR_UNSUPPORTED;
  if (batch == 0) return LOCKS_OK;
  if (!q || !k_cache || !v_cache || !page_table || !seq_lens || !o_out ||
      !lse_out || !workspace)
    return LOCKS_ERR_INVALID_ARG;
  const int list_len = idx ? k : max_pages;
  // every list entry of every (sequence, KV head) is one int32 position
  if ((long long)batch * h_kv * list_len > 0x7fffffffLL)
    return LOCKS_ERR_UNSUPPORTED;
  if (batch > decode_max_batch()) return LOCKS_ERR_UNSUPPORTED;
  if (workspace_bytes < kWsHeader + decode_region(batch, h_q, h_kv, list_len))
    return LOCKS_ERR_WORKSPACE;
  const int G = h_q / h_kv;
  uint8_t *ws = static_cast<uint8_t *>(workspace);
  int32_t *status = reinterpret_cast<int32_t *>(ws);
  const size_t rows = decode_slots(batch, h_kv, list_len) * (size_t)G;
  int *meta = reinterpret_cast<int *>(ws + kWsHeader);
  float *o_part =
      reinterpret_cast<float *>(ws + kWsHeader + decode_meta_bytes(batch));
  float *lse_part = reinterpret_cast<float *>(
      ws + kWsHeader + decode_meta_bytes(batch) + round_up(rows * kDim * 4, 256));
  const int max_warps = (int)decode_warps_cap(batch, h_kv, list_len);
  cudaError_t e = launch_decode(
      q, k_cache, v_cache, num_phys_pages, page_table, seq_lens, idx, k, batch,
      h_kv, G, max_pages, max_warps, o_out, lse_out, o_part, lse_part, meta,
      status, stream, status_mirror);
  return e == cudaSuccess ? LOCKS_OK : fail_cuda(e);
}

extern "C" {

const char *locks_status_string(locks_status_t s) {
  switch (s) {
    case LOCKS_OK: return "ok";
    case LOCKS_ERR_INVALID_ARG: return "invalid argument";
    case LOCKS_ERR_UNSUPPORTED: return "unsupported size";
    case LOCKS_ERR_WORKSPACE: return "workspace too small";
    case LOCKS_ERR_CUDA: return "CUDA error";
  }
  return "unknown status";
}

int locks_last_cuda_error(void) { return g_last_cuda; }

long long locks_kernel_launches(void) {
  return g_kernel_launches.load(std::memory_order_relaxed);
}

size_t locks_summary_record_bytes(void) { return (size_t)kRec; }

locks_status_t locks_workspace_size(int batch, int h_q, int h_kv,
                                    int max_pages, int k, size_t *bytes) {
  if (!bytes || batch < 0 || max_pages < 1 || k < 1 || !heads_ok(h_q, h_kv))
    return LOCKS_ERR_INVALID_ARG;
  if (h_q / h_kv > kMaxGroup) return LOCKS_ERR_UNSUPPORTED;
  const size_t a = score_region(batch, h_q, h_kv, max_pages);
  const size_t b = decode_region(batch, h_q, h_kv, k);
  const size_t c = qdecode_region(nullptr, batch, h_q, h_kv, k).bytes;
  size_t most = a > b ? a : b;
  if (c > most) most = c;
  *bytes = kWsHeader + most;
  return LOCKS_OK;
}

static bool build_flags_ok(int flags) {
  return (flags & ~LOCKS_BUILD_VSCALE_PER_PAGE) == 0;
}

locks_status_t locks_build_summaries(
    const void *k_cache, int64_t num_phys_pages, int h_kv,
    const int32_t *page_table, int batch, int max_pages,
    const int32_t *seq_ids, const int32_t *page_ids, int n_pairs,
    void *summaries, float *tau_out, float *unquantised_out, int32_t *status,
    locks_stream_t stream) {
  return locks_build_summaries_ex(k_cache, num_phys_pages, h_kv, page_table,
                                  batch, max_pages, seq_ids, page_ids, n_pairs,
                                  summaries, tau_out, unquantised_out, 0,
                                  status, stream);
}

locks_status_t locks_build_summaries_ex(
    const void *k_cache, int64_t num_phys_pages, int h_kv,
    const int32_t *page_table, int batch, int max_pages,
    const int32_t *seq_ids, const int32_t *page_ids, int n_pairs,
    void *summaries, float *tau_out, float *unquantised_out, int flags,
    int32_t *status, locks_stream_t stream) {
  if (n_pairs < 0 || h_kv < 1 || batch < 1 || max_pages < 1 ||
      num_phys_pages < 1 || !build_flags_ok(flags))
    return LOCKS_ERR_INVALID_ARG;
  if (n_pairs == 0) return LOCKS_OK;
  if (!k_cache || !page_table || !seq_ids || !page_ids || !summaries)
    return LOCKS_ERR_INVALID_ARG;
  cudaError_t e = launch_build(k_cache, num_phys_pages, h_kv, page_table,
                               batch, max_pages, seq_ids, page_ids, n_pairs,
                               summaries, tau_out, unquantised_out, flags,
                               status, (cudaStream_t)stream);
  return e == cudaSuccess ? LOCKS_OK : fail_cuda(e);
}

static bool variant_ok(int rank, int vbits) {
  return (rank == 4 || rank == 8 || rank == 12 || rank == 15) &&
         (vbits == 2 || vbits == 4 || vbits == 8);
}

size_t locks_variant_record_bytes(int rank, int vbits) {
  return variant_ok(rank, vbits) ? variant_record_bytes(rank, vbits) : 0;
}

locks_status_t locks_build_variant(
    const void *k_cache, int64_t num_phys_pages, int h_kv,
    const int32_t *page_table, int batch, int max_pages,
    const int32_t *seq_ids, const int32_t *page_ids, int n_pairs, int rank,
    int vbits, void *records, float *tau_out, int32_t *status,
    locks_stream_t stream) {
  if (!variant_ok(rank, vbits)) return LOCKS_ERR_INVALID_ARG;
  if (n_pairs < 0 || h_kv < 1 || batch < 1 || max_pages < 1 ||
      num_phys_pages < 1)
    return LOCKS_ERR_INVALID_ARG;
  if (n_pairs == 0) return LOCKS_OK;
  if (!k_cache || !page_table || !seq_ids || !page_ids || !records)
    return LOCKS_ERR_INVALID_ARG;
  cudaError_t e = launch_build_variant(
      k_cache, num_phys_pages, h_kv, page_table, batch, max_pages, seq_ids,
      page_ids, n_pairs, rank, vbits, records, tau_out, status,
      (cudaStream_t)stream);
  return e == cudaSuccess ? LOCKS_OK : fail_cuda(e);
}

locks_status_t locks_score_variant(const void *q, const void *records,
                                   int rank, int vbits,
                                   const int32_t *seq_lens, int batch,
                                   int h_q, int h_kv, int max_pages,
                                   float *scores_out, int32_t *status,
                                   locks_stream_t stream) {
  if (!variant_ok(rank, vbits)) return LOCKS_ERR_INVALID_ARG;
  if (batch < 0 || max_pages < 1 || !heads_ok(h_q, h_kv))
    return LOCKS_ERR_INVALID_ARG;
  if (h_q / h_kv > kMaxGroup) return LOCKS_ERR_UNSUPPORTED;
  if (batch > variant_max_batch(rank, vbits) || h_kv > 65535 ||
      (long long)max_pages * kPage > 0x7fffffffLL)
    return LOCKS_ERR_UNSUPPORTED;
  if (batch == 0) return LOCKS_OK;
  if (!q || !records || !seq_lens || !scores_out) return LOCKS_ERR_INVALID_ARG;
  if (reinterpret_cast<uintptr_t>(records) & 15u) return LOCKS_ERR_INVALID_ARG;
  cudaError_t e = launch_score_variant(q, records, rank, vbits, seq_lens,
                                       batch, h_kv, h_q / h_kv, max_pages,
                                       scores_out, status,
                                       (cudaStream_t)stream);
  return e == cudaSuccess ? LOCKS_OK : fail_cuda(e);
}

locks_status_t locks_pack_summaries(const float *mu, const float *basis,
                                    const float *coeffs, int n, void *records,
                                    locks_stream_t stream) {
  return locks_pack_summaries_ex(mu, basis, coeffs, n, records, 0, stream);
}

locks_status_t locks_pack_summaries_ex(const float *mu, const float *basis,
                                       const float *coeffs, int n,
                                       void *records, int flags,
                                       locks_stream_t stream) {
  if (n < 0 || !build_flags_ok(flags)) return LOCKS_ERR_INVALID_ARG;
  if (n == 0) return LOCKS_OK;
  if (!mu || !basis || !coeffs || !records) return LOCKS_ERR_INVALID_ARG;
  cudaError_t e = launch_pack(mu, basis, coeffs, n, records, flags,
                              (cudaStream_t)stream);
  return e == cudaSuccess ? LOCKS_OK : fail_cuda(e);
}

locks_status_t locks_score_select(const void *q, const void *summaries,
                                  const int32_t *seq_lens, int batch, int h_q,
                                  int h_kv, int max_pages, int k,
                                  int32_t *idx_out, void *workspace,
                                  size_t workspace_bytes,
                                  locks_stream_t stream) {
  return locks::score_select(q, summaries, seq_lens, batch, h_q, h_kv,
                             max_pages, k, idx_out, workspace, workspace_bytes,
                             (cudaStream_t)stream, false);
}

locks_status_t locks_score_pages(const void *q, const void *summaries,
                                 const int32_t *seq_lens, int batch, int h_q,
                                 int h_kv, int max_pages, float *scores_out,
                                 int32_t *status, locks_stream_t stream) {
  if (batch < 0 || max_pages < 1 || !heads_ok(h_q, h_kv))
    return LOCKS_ERR_INVALID_ARG;
  if (h_q / h_kv > kMaxGroup) return LOCKS_ERR_UNSUPPORTED;
  if ((long long)max_pages * kPage > 0x7fffffffLL) return LOCKS_ERR_UNSUPPORTED;
  if (batch == 0) return LOCKS_OK;
  if (!q || !summaries || !seq_lens || !scores_out)
    return LOCKS_ERR_INVALID_ARG;
  if (batch > score_max_batch()) return LOCKS_ERR_UNSUPPORTED;
  cudaError_t e = launch_score(q, summaries, seq_lens, batch, h_kv,
                               h_q / h_kv, max_pages, scores_out, status,
                               (cudaStream_t)stream);
  return e == cudaSuccess ? LOCKS_OK : fail_cuda(e);
}

locks_status_t locks_exact_page_scores(
    const void *q, const void *k_cache, int64_t num_phys_pages,
    const int32_t *page_table, const int32_t *seq_lens, int batch, int h_q,
    int h_kv, int max_pages, float *scores_out, int32_t *status,
    locks_stream_t stream) {
  if (batch < 0 || max_pages < 1 || num_phys_pages < 1 || !heads_ok(h_q, h_kv))
    return LOCKS_ERR_INVALID_ARG;
  if (h_q / h_kv > kMaxGroup) return LOCKS_ERR_UNSUPPORTED;
  if ((long long)max_pages * kPage > 0x7fffffffLL ||
      (long long)batch * h_kv * max_pages > 0x7fffffffLL)
    return LOCKS_ERR_UNSUPPORTED;
  if (batch == 0) return LOCKS_OK;
  if (!q || !k_cache || !page_table || !seq_lens || !scores_out)
    return LOCKS_ERR_INVALID_ARG;
  if (batch > exact_max_batch()) return LOCKS_ERR_UNSUPPORTED;
  cudaError_t e = launch_exact(q, k_cache, num_phys_pages, page_table,
                               seq_lens, batch, h_kv, h_q / h_kv, max_pages,
                               scores_out, status, (cudaStream_t)stream);
  return e == cudaSuccess ? LOCKS_OK : fail_cuda(e);
}

locks_status_t locks_select_pages_merge(const float *scores,
                                        const int32_t *seq_lens, int batch,
                                        int h_q, int h_kv, int max_pages,
                                        int k, int rule, int32_t *idx_out,
                                        void *workspace,
                                        size_t workspace_bytes,
                                        locks_stream_t stream) {
  if (rule != LOCKS_MERGE_SHARE_AVERAGE && rule != LOCKS_MERGE_GROUP_MAX &&
      rule != LOCKS_MERGE_GROUP_MASS)
    return LOCKS_ERR_INVALID_ARG;
  locks_status_t st = check_select_args(batch, h_q, h_kv, max_pages, k,
                                        seq_lens, idx_out, workspace);
  if (st != LOCKS_OK) return st;
  if (batch == 0) return LOCKS_OK;
  if (!scores) return LOCKS_ERR_INVALID_ARG;
  if (workspace_bytes < kWsHeader + score_region(batch, h_q, h_kv, max_pages))
    return LOCKS_ERR_WORKSPACE;
  const int G = h_q / h_kv;
  uint8_t *ws = static_cast<uint8_t *>(workspace);
  int32_t *status = reinterpret_cast<int32_t *>(ws);
  uint32_t *keys = reinterpret_cast<uint32_t *>(
      ws + kWsHeader + round_up((size_t)batch * h_kv * G * max_pages * 4, 256));
  cudaError_t e =
      launch_select(scores, seq_lens, batch, h_kv, G, max_pages, k, rule,
                    idx_out, keys, status, (cudaStream_t)stream);
  return e == cudaSuccess ? LOCKS_OK : fail_cuda(e);
}

locks_status_t locks_select_pages(const float *scores, const int32_t *seq_lens,
                                  int batch, int h_q, int h_kv, int max_pages,
                                  int k, int32_t *idx_out, void *workspace,
                                  size_t workspace_bytes,
                                  locks_stream_t stream) {
  return locks_select_pages_merge(scores, seq_lens, batch, h_q, h_kv,
                                  max_pages, k, LOCKS_MERGE_SHARE_AVERAGE,
                                  idx_out, workspace, workspace_bytes, stream);
}

locks_status_t locks_sparse_decode(
    const void *q, const void *k_cache, const void *v_cache,
    int64_t num_phys_pages, const int32_t *page_table,
    const int32_t *seq_lens, const int32_t *idx, int k, int batch, int h_q,
    int h_kv, int max_pages, void *o_out, float *lse_out, void *workspace,
    size_t workspace_bytes, locks_stream_t stream) {
  return locks::sparse_decode(q, k_cache, v_cache, num_phys_pages, page_table,
                              seq_lens, idx, k, batch, h_q, h_kv, max_pages,
                              o_out, lse_out, workspace, workspace_bytes,
                              (cudaStream_t)stream, nullptr);
}

locks_status_t locks_append_kv(const void *k_new, const void *v_new,
                               void *k_cache, void *v_cache,
                               int64_t num_phys_pages, int h_kv,
                               const int32_t *page_table, int batch,
                               int max_pages, int32_t *seq_lens,
                               void *summaries, float *tau_out,
                               int32_t *status, locks_stream_t stream) {
  return locks_append_kv_ex(k_new, v_new, k_cache, v_cache, num_phys_pages,
                            h_kv, page_table, batch, max_pages, seq_lens,
                            summaries, tau_out, 0, status, stream);
}

static bool aligned16(const void *p) {
  return (reinterpret_cast<uintptr_t>(p) & 15u) == 0;
}

// what an append loads and stores: 8 bytes a lane of a row, 16 of a record
static bool append_aligned(const void *k_new, const void *v_new,
                           const void *k_cache, const void *v_cache,
                           const void *summaries) {
  for (const void *p : {k_new, v_new, k_cache, v_cache})
    if (reinterpret_cast<uintptr_t>(p) & 7u) return false;
  return aligned16(summaries);
}

locks_status_t locks_append_kv_ex(const void *k_new, const void *v_new,
                                  void *k_cache, void *v_cache,
                                  int64_t num_phys_pages, int h_kv,
                                  const int32_t *page_table, int batch,
                                  int max_pages, int32_t *seq_lens,
                                  void *summaries, float *tau_out, int flags,
                                  int32_t *status, locks_stream_t stream) {
  if (batch < 0 || h_kv < 1 || max_pages < 1 || num_phys_pages < 1 ||
      !build_flags_ok(flags))
    return LOCKS_ERR_INVALID_ARG;
  if (h_kv > 32) return LOCKS_ERR_UNSUPPORTED;
  if (batch == 0) return LOCKS_OK;
  if (!k_new || !v_new || !k_cache || !v_cache || !page_table || !seq_lens ||
      !summaries || !append_aligned(k_new, v_new, k_cache, v_cache, summaries))
    return LOCKS_ERR_INVALID_ARG;
  cudaError_t e = launch_append(k_new, v_new, k_cache, v_cache, num_phys_pages,
                                h_kv, page_table, batch, max_pages, seq_lens,
                                summaries, tau_out, flags, status,
                                (cudaStream_t)stream);
  return e == cudaSuccess ? LOCKS_OK : fail_cuda(e);
}

// ---------------------------------------------------------------------------
// quantised KV cache
// ---------------------------------------------------------------------------
static bool type_ok(int type) {
  return type == LOCKS_TYPE_BF16 || type == LOCKS_TYPE_FP16 ||
         type == LOCKS_TYPE_FP32;
}

locks_status_t locks_quantise_kv(
    const void *k_new, const void *v_new, int type, int64_t k_token_stride,
    int64_t k_head_stride, int64_t v_token_stride, int64_t v_head_stride,
    const int32_t *seq_ids, const int32_t *positions, int n_tokens,
    void *records, int64_t num_phys_pages, int h_kv,
    const int32_t *page_table, int batch, int max_pages, int32_t *status,
    locks_stream_t stream) {
  if (!type_ok(type) || n_tokens < 0 || h_kv < 1 || batch < 1 ||
      max_pages < 1 || num_phys_pages < 1)
    return LOCKS_ERR_INVALID_ARG;
  if ((long long)n_tokens * h_kv > 0x7fffffffLL ||
      (long long)max_pages * kPage > 0x7fffffffLL)
    return LOCKS_ERR_UNSUPPORTED;
  if (n_tokens == 0) return LOCKS_OK;
  if (!k_new || !v_new || !seq_ids || !positions || !records || !page_table)
    return LOCKS_ERR_INVALID_ARG;
  // 16 bytes of elements
  const int64_t step = type == LOCKS_TYPE_FP32 ? 4 : 8;
  if (!aligned16(k_new) || !aligned16(v_new) || !aligned16(records) ||
      k_token_stride % step || k_head_stride % step || v_token_stride % step ||
      v_head_stride % step)
    return LOCKS_ERR_INVALID_ARG;
  cudaError_t e = launch_quantise(
      k_new, v_new, type, k_token_stride, k_head_stride, v_token_stride,
      v_head_stride, seq_ids, positions, n_tokens, records, num_phys_pages,
      h_kv, page_table, batch, max_pages, status, (cudaStream_t)stream);
  return e == cudaSuccess ? LOCKS_OK : fail_cuda(e);
}

locks_status_t locks_dequantise_kv(
    const void *records, int64_t num_phys_pages, int h_kv,
    const int32_t *page_table, int batch, int max_pages,
    const int32_t *seq_ids, const int32_t *page_ids, int n_pairs,
    const int32_t *seq_lens, int type, void *k_out, void *v_out,
    int32_t *status, locks_stream_t stream) {
  if (!type_ok(type) || n_pairs < 0 || h_kv < 1 || batch < 1 ||
      max_pages < 1 || num_phys_pages < 1)
    return LOCKS_ERR_INVALID_ARG;
  if ((long long)n_pairs * h_kv > 0x7fffffffLL ||
      (long long)max_pages * kPage > 0x7fffffffLL)
    return LOCKS_ERR_UNSUPPORTED;
  if (n_pairs == 0) return LOCKS_OK;
  if (!records || !page_table || !seq_ids || !page_ids || (!k_out && !v_out))
    return LOCKS_ERR_INVALID_ARG;
  if (!aligned16(records) || !aligned16(k_out) || !aligned16(v_out))
    return LOCKS_ERR_INVALID_ARG;
  cudaError_t e = launch_dequantise(
      records, num_phys_pages, h_kv, page_table, batch, max_pages, seq_ids,
      page_ids, n_pairs, seq_lens, type, k_out, v_out, status,
      (cudaStream_t)stream);
  return e == cudaSuccess ? LOCKS_OK : fail_cuda(e);
}

// checks shared by the two attention calls (pointers after the empty batch)
static locks_status_t check_qdecode(const void *q, const void *records,
                                    int64_t num_phys_pages,
                                    const int32_t *page_table,
                                    const int32_t *seq_lens, int list_len,
                                    int batch, int h_q, int h_kv,
                                    int max_pages, const void *o_out,
                                    const float *lse_out,
                                    const void *workspace) {
  if (batch < 0 || max_pages < 1 || num_phys_pages < 1 || !heads_ok(h_q, h_kv))
    return LOCKS_ERR_INVALID_ARG;
  if (list_len < 1) return LOCKS_ERR_INVALID_ARG;
  if (h_q / h_kv > kMaxGroup) return LOCKS_ERR_UNSUPPORTED;
  if (batch > qdecode_max_batch() || h_kv > 65535) return LOCKS_ERR_UNSUPPORTED;
  // list entries are int32 positions, and a warp's run and window end past its
  // last one, by up to a window and a run's rounding
  if ((long long)max_pages * kPage > 0x7fffffffLL ||
      (long long)batch * h_kv * list_len > 0x7fffffffLL - 0xffffLL ||
      (long long)batch * h_q > 0x7fffffffLL)
    return LOCKS_ERR_UNSUPPORTED;
  if (batch == 0) return LOCKS_OK;
  if (!q || !records || !page_table || !seq_lens || !o_out || !lse_out ||
      !workspace)
    return LOCKS_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(records) || !aligned16(o_out) ||
      !aligned16(workspace))
    return LOCKS_ERR_INVALID_ARG;
  return LOCKS_OK;
}

locks_status_t locks_quantised_decode(
    const void *q, const void *records, int64_t num_phys_pages,
    const int32_t *page_table, const int32_t *seq_lens, const int32_t *idx,
    int k, int batch, int h_q, int h_kv, int max_pages, void *o_out,
    float *lse_out, void *workspace, size_t workspace_bytes,
    locks_stream_t stream) {
  const int list_len = idx ? k : max_pages;
  locks_status_t st =
      check_qdecode(q, records, num_phys_pages, page_table, seq_lens, list_len,
                    batch, h_q, h_kv, max_pages, o_out, lse_out, workspace);
  if (st != LOCKS_OK || batch == 0) return st;
  uint8_t *ws = static_cast<uint8_t *>(workspace);
  const DecodeRegion r =
      qdecode_region(ws + kWsHeader, batch, h_q, h_kv, list_len);
  if (workspace_bytes < kWsHeader + r.bytes) return LOCKS_ERR_WORKSPACE;
  cudaError_t e = launch_qdecode(
      q, records, num_phys_pages, page_table, seq_lens, idx, k, batch, h_kv,
      h_q / h_kv, max_pages, nullptr, 0,
      (int)decode_warps_cap(batch, h_kv, list_len), o_out, lse_out, r.o_part,
      r.ml_part, r.meta, nullptr, nullptr, 0, reinterpret_cast<int32_t *>(ws),
      (cudaStream_t)stream);
  return e == cudaSuccess ? LOCKS_OK : fail_cuda(e);
}

// the partials of the shared pages
struct PrefixRegion {
  PrefixPlan plan;
  float *o_part;
  float2 *ml_part;
  size_t bytes;
};
static PrefixRegion prefix_region(uint8_t *at, int batch, int h_q, int h_kv,
                                  int pages) {
  if (pages == 0 || batch == 0) return {{0, false}, nullptr, nullptr, 0};
  const PrefixPlan plan = prefix_plan(batch, h_kv, h_q / h_kv, pages);
  if (plan.splits == 0) return {plan, nullptr, nullptr, 0};
  const size_t rows = prefix_rows(batch, h_kv, h_q / h_kv, pages);
  const size_t sums = round_up(rows * kDim * 4, 256);
  return {plan, reinterpret_cast<float *>(at),
          reinterpret_cast<float2 *>(at + sums),
          sums + round_up(rows * 8, 256)};
}

locks_status_t locks_prefix_workspace_size(int batch, int h_q, int h_kv,
                                           int max_pages, int prefix_pages,
                                           size_t *bytes) {
  if (!bytes || batch < 0 || max_pages < 1 || prefix_pages < 0 ||
      prefix_pages > max_pages || !heads_ok(h_q, h_kv))
    return LOCKS_ERR_INVALID_ARG;
  if (h_q / h_kv > kMaxGroup) return LOCKS_ERR_UNSUPPORTED;
  *bytes =
      kWsHeader + qdecode_region(nullptr, batch, h_q, h_kv, max_pages).bytes +
      prefix_region(nullptr, batch, h_q, h_kv, prefix_pages).bytes;
  return LOCKS_OK;
}

locks_status_t locks_prefix_decode(
    const void *q, const void *records, int64_t num_phys_pages,
    const int32_t *prefix_table, int prefix_pages, const int32_t *page_table,
    const int32_t *seq_lens, int batch, int h_q, int h_kv, int max_pages,
    void *o_out, float *lse_out, void *workspace, size_t workspace_bytes,
    locks_stream_t stream) {
  if (prefix_pages < 0 || prefix_pages > max_pages)
    return LOCKS_ERR_INVALID_ARG;
  locks_status_t st =
      check_qdecode(q, records, num_phys_pages, page_table, seq_lens,
                    max_pages, batch, h_q, h_kv, max_pages, o_out, lse_out,
                    workspace);
  if (st != LOCKS_OK || batch == 0) return st;
  if (prefix_pages > 0 && !prefix_table) return LOCKS_ERR_INVALID_ARG;
  uint8_t *ws = static_cast<uint8_t *>(workspace);
  const DecodeRegion r =
      qdecode_region(ws + kWsHeader, batch, h_q, h_kv, max_pages);
  const PrefixRegion p = prefix_region(ws + kWsHeader + r.bytes, batch, h_q,
                                       h_kv, prefix_pages);
  if (workspace_bytes < kWsHeader + r.bytes + p.bytes)
    return LOCKS_ERR_WORKSPACE;
  const int G = h_q / h_kv;
  int32_t *status = reinterpret_cast<int32_t *>(ws);
  cudaError_t e = cudaSuccess;
  if (p.plan.splits > 0)
    e = launch_prefix(q, records, num_phys_pages, prefix_table, prefix_pages,
                      batch, h_kv, G, p.plan, p.o_part, p.ml_part, status,
                      (cudaStream_t)stream);
  if (e == cudaSuccess)
    e = launch_qdecode(q, records, num_phys_pages, page_table, seq_lens,
                       nullptr, 0, batch, h_kv, G, max_pages, prefix_table,
                       prefix_pages,
                       (int)decode_warps_cap(batch, h_kv, max_pages), o_out,
                       lse_out, r.o_part, r.ml_part, r.meta, p.o_part,
                       p.ml_part, p.plan.splits, status, (cudaStream_t)stream);
  return e == cudaSuccess ? LOCKS_OK : fail_cuda(e);
}

// ---------------------------------------------------------------------------
// rotary positions
// ---------------------------------------------------------------------------
locks_status_t locks_rotation_init(const double *frequencies,
                                   const int32_t *axes, int dim, int pairs,
                                   int n_axes, float amplitude,
                                   locks_rotation_t *out) {
  if (!frequencies || !out || dim < 16 || dim > kDim || dim % 16 ||
      (pairs != 0 && pairs != 1) || n_axes < 1 ||
      n_axes > LOCKS_ROTARY_AXES || !isfinite(amplitude))
    return LOCKS_ERR_INVALID_ARG;
  for (int j = 0; j < dim / 2; ++j)
    if (!(fabs(frequencies[j]) <= 0x1p20) ||
        (axes && (axes[j] < 0 || axes[j] >= n_axes)))
      return LOCKS_ERR_INVALID_ARG;
  locks_rotation_t r = {};
  // 1 / 2 pi as the sum of two doubles; the product's rounding is kept, so
  // that the fraction is good to the last of its 64 bits
  const double inv = 0x1.45f306dc9c883p-3, rest = -0x1.6b01ec5417056p-57;
  for (int j = 0; j < dim / 2; ++j) {
    const double f = fabs(frequencies[j]);
    const double hi = f * inv;
    const double lo = fma(f, inv, -hi) + f * rest;
    const double units = ldexp(hi - floor(hi), 64);  // exact, below 2^64
    const double whole = floor(units);
    const uint64_t t = (uint64_t)whole +
                       (uint64_t)llrint(units - whole + ldexp(lo, 64));
    r.turns[j] = frequencies[j] < 0 ? 0 - t : t;
    r.axes[j] = axes ? (uint8_t)axes[j] : 0;
  }
  r.dim = dim;
  r.pairs = pairs;
  r.n_axes = n_axes;
  r.amplitude = amplitude;
  *out = r;
  return LOCKS_OK;
}

// a struct that locks_rotation_init has filled, as far as kernels rely on it
static bool rotation_ok(const locks_rotation_t *r) {
  if (!r || r->dim < 16 || r->dim > kDim || r->dim % 16 ||
      (r->pairs != 0 && r->pairs != 1) || r->n_axes < 1 ||
      r->n_axes > LOCKS_ROTARY_AXES)
    return false;
  for (int j = 0; j < r->dim / 2; ++j)
    if (r->axes[j] >= r->n_axes) return false;
  return true;
}

static locks_status_t rotate(const locks_rotation_t *rotation, int type,
                             bool quantised, RotateArgs a,
                             cudaStream_t stream) {
  if (!rotation_ok(rotation) || !type_ok(type) || a.n_tokens < 0 ||
      a.h_kv < 1 || a.batch < 1 || a.max_pages < 1 || a.num_phys < 1 ||
      (a.q && a.h_q < 1))
    return LOCKS_ERR_INVALID_ARG;
  if (!a.q) a.h_q = 0;
  if ((long long)a.n_tokens * (a.h_q + 2LL * a.h_kv) > 0x7fffffffLL ||
      (long long)a.max_pages * kPage > 0x7fffffffLL)
    return LOCKS_ERR_UNSUPPORTED;
  if (a.n_tokens == 0) return LOCKS_OK;
  if (!a.k_new || !a.v_new || !a.seq_ids || !a.positions || !a.k_cache ||
      (!quantised && !a.v_cache) || !a.pt || (a.q && !a.q_out))
    return LOCKS_ERR_INVALID_ARG;
  // 16 bytes of elements
  const int64_t step = type == LOCKS_TYPE_FP32 ? 4 : 8;
  if (!aligned16(a.q) || !aligned16(a.k_new) || !aligned16(a.v_new) ||
      !aligned16(a.k_cache) || !aligned16(a.v_cache) ||
      (a.q && (!aligned16(a.q_out) || a.q_token % step || a.q_head % step)) ||
      a.k_token % step || a.k_head % step || a.v_token % step ||
      a.v_head % step)
    return LOCKS_ERR_INVALID_ARG;
  cudaError_t e = launch_rotate(a, type, quantised, *rotation, stream);
  return e == cudaSuccess ? LOCKS_OK : fail_cuda(e);
}

locks_status_t locks_rotate_kv(
    const void *q, const void *k_new, const void *v_new, int type,
    int64_t q_token_stride, int64_t q_head_stride, int64_t k_token_stride,
    int64_t k_head_stride, int64_t v_token_stride, int64_t v_head_stride,
    const locks_rotation_t *rotation, const int32_t *rotary_positions,
    const int32_t *seq_ids, const int32_t *positions, int n_tokens, int h_q,
    void *q_out, void *k_cache, void *v_cache, int64_t num_phys_pages,
    int h_kv, const int32_t *page_table, int batch, int max_pages,
    int32_t *status, locks_stream_t stream) {
  return rotate(rotation, type, false,
                {q, k_new, v_new, q_token_stride, q_head_stride,
                 k_token_stride, k_head_stride, v_token_stride, v_head_stride,
                 rotary_positions, seq_ids, positions, n_tokens, h_q, h_kv,
                 batch, max_pages, static_cast<__nv_bfloat16 *>(q_out),
                 k_cache, v_cache, num_phys_pages, page_table, status},
                (cudaStream_t)stream);
}

locks_status_t locks_rotate_quantise_kv(
    const void *q, const void *k_new, const void *v_new, int type,
    int64_t q_token_stride, int64_t q_head_stride, int64_t k_token_stride,
    int64_t k_head_stride, int64_t v_token_stride, int64_t v_head_stride,
    const locks_rotation_t *rotation, const int32_t *rotary_positions,
    const int32_t *seq_ids, const int32_t *positions, int n_tokens, int h_q,
    void *q_out, void *records, int64_t num_phys_pages, int h_kv,
    const int32_t *page_table, int batch, int max_pages, int32_t *status,
    locks_stream_t stream) {
  return rotate(rotation, type, true,
                {q, k_new, v_new, q_token_stride, q_head_stride,
                 k_token_stride, k_head_stride, v_token_stride, v_head_stride,
                 rotary_positions, seq_ids, positions, n_tokens, h_q, h_kv,
                 batch, max_pages, static_cast<__nv_bfloat16 *>(q_out),
                 records, nullptr, num_phys_pages, page_table, status},
                (cudaStream_t)stream);
}

locks_status_t locks_append_rotated_kv(
    const void *q, const void *k_new, const void *v_new,
    const locks_rotation_t *rotation, const int32_t *rotary_positions,
    int h_q, void *q_out, void *k_cache, void *v_cache,
    int64_t num_phys_pages, int h_kv, const int32_t *page_table, int batch,
    int max_pages, int32_t *seq_lens, void *summaries, float *tau_out,
    int flags, int32_t *status, locks_stream_t stream) {
  if (!rotation_ok(rotation) || batch < 0 || !heads_ok(h_q, h_kv) ||
      max_pages < 1 || num_phys_pages < 1 || !build_flags_ok(flags))
    return LOCKS_ERR_INVALID_ARG;
  // (a warp to a head: beyond 20 the append's form with 64 registers a thread would
  // have to turn rows as well)
  if (h_kv > 16) return LOCKS_ERR_UNSUPPORTED;
  if (batch == 0) return LOCKS_OK;
  if (!q || !q_out || !k_new || !v_new || !k_cache || !v_cache ||
      !page_table || !seq_lens || !summaries)
    return LOCKS_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(q_out) ||
      !append_aligned(k_new, v_new, k_cache, v_cache, summaries))
    return LOCKS_ERR_INVALID_ARG;
  cudaError_t e = launch_append_rotated(
      {q, q_out, h_q, rotary_positions, *rotation}, k_new, v_new, k_cache,
      v_cache, num_phys_pages, h_kv, page_table, batch, max_pages, seq_lens,
      summaries, tau_out, flags, status, (cudaStream_t)stream);
  return e == cudaSuccess ? LOCKS_OK : fail_cuda(e);
}

// ---------------------------------------------------------------------------
// attention over a window
// ---------------------------------------------------------------------------
static locks_status_t check_window(const void *q, const void *k_cache,
                                   const void *v_cache, int64_t num_phys_pages,
                                   const int32_t *page_table,
                                   const int32_t *seq_lens, int window,
                                   int sinks, int n_tokens, int batch, int h_q,
                                   int h_kv, int max_pages, const void *o_out,
                                   const float *lse_out,
                                   const void *workspace) {
  if (n_tokens < 0 || batch < 0 || max_pages < 1 || num_phys_pages < 1 ||
      window < 1 || sinks < 0 || !heads_ok(h_q, h_kv))
    return LOCKS_ERR_INVALID_ARG;
  if (h_q / h_kv > kMaxGroup || h_kv > 65535) return LOCKS_ERR_UNSUPPORTED;
  if ((long long)max_pages * kPage > 1LL << 30 ||
      (long long)n_tokens * h_q > 0x7fffffffLL)
    return LOCKS_ERR_UNSUPPORTED;
  if (batch == 0 || n_tokens == 0) return LOCKS_OK;
  if (!q || !k_cache || !v_cache || !page_table || !seq_lens || !o_out ||
      !lse_out || !workspace)
    return LOCKS_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache) ||
      !aligned16(o_out) || !aligned16(workspace))
    return LOCKS_ERR_INVALID_ARG;
  return LOCKS_OK;
}

// bytes of `rows` partials
static size_t window_region(size_t rows) {
  return round_up(rows * kDim * 4, 256) + round_up(rows * 8, 256);
}

locks_status_t locks_window_workspace_size(int n_tokens, int batch, int h_q,
                                           int h_kv, int max_pages, int window,
                                           int sinks, size_t *bytes) {
  if (!bytes || n_tokens < 0 || batch < 0 || max_pages < 1 || window < 1 ||
      sinks < 0 || !heads_ok(h_q, h_kv))
    return LOCKS_ERR_INVALID_ARG;
  if (h_q / h_kv > kMaxGroup || (long long)max_pages * kPage > 1LL << 30)
    return LOCKS_ERR_UNSUPPORTED;
  const size_t one = decode_region(batch, h_q, h_kv,
                                   window_list(max_pages, window, sinks));
  const size_t many = window_region(window_part_rows(
      n_tokens, h_kv, h_q / h_kv, max_pages, window, sinks));
  *bytes = kWsHeader + (one > many ? one : many);
  return LOCKS_OK;
}

// no sequence is longer than its table: what a window or a number of first
// tokens has beyond that says nothing
static int at_most_table(int tokens, int max_pages) {
  const int top = max_pages * kPage;
  return tokens < top ? tokens : top;
}

locks_status_t locks_window_decode(
    const void *q, const void *k_cache, const void *v_cache,
    int64_t num_phys_pages, const int32_t *page_table,
    const int32_t *seq_lens, int window, int sinks, int batch, int h_q,
    int h_kv, int max_pages, void *o_out, float *lse_out, void *workspace,
    size_t workspace_bytes, locks_stream_t stream) {
  locks_status_t st = check_window(q, k_cache, v_cache, num_phys_pages,
                                   page_table, seq_lens, window, sinks, batch,
                                   batch, h_q, h_kv, max_pages, o_out, lse_out,
                                   workspace);
  if (st != LOCKS_OK || batch == 0) return st;
  window = at_most_table(window, max_pages);
  sinks = at_most_table(sinks, max_pages);
  const int list = window_list(max_pages, window, sinks);
  // list entries are int32 positions, and a warp's run and window of entries
  // end past the last one, by up to a window and a run's rounding
  if ((long long)batch * h_kv * list > 0x7fffffffLL - 0xffffLL ||
      batch > decode_max_batch())
    return LOCKS_ERR_UNSUPPORTED;
  if (workspace_bytes < kWsHeader + decode_region(batch, h_q, h_kv, list))
    return LOCKS_ERR_WORKSPACE;
  uint8_t *ws = static_cast<uint8_t *>(workspace);
  const size_t rows = decode_slots(batch, h_kv, list) * (size_t)(h_q / h_kv);
  uint8_t *part = ws + kWsHeader + decode_meta_bytes(batch);
  cudaError_t e = launch_window_decode(
      q, k_cache, v_cache, num_phys_pages, page_table, seq_lens, window, sinks,
      batch, h_kv, h_q / h_kv, max_pages,
      (int)decode_warps_cap(batch, h_kv, list), o_out, lse_out,
      reinterpret_cast<float *>(part),
      reinterpret_cast<float *>(part + round_up(rows * kDim * 4, 256)),
      reinterpret_cast<int *>(ws + kWsHeader), reinterpret_cast<int32_t *>(ws),
      (cudaStream_t)stream);
  return e == cudaSuccess ? LOCKS_OK : fail_cuda(e);
}

locks_status_t locks_window_attention(
    const void *q, const void *k_cache, const void *v_cache,
    int64_t num_phys_pages, const int32_t *page_table,
    const int32_t *q_starts, const int32_t *seq_lens, int n_tokens,
    int window, int sinks, int batch, int h_q, int h_kv, int max_pages,
    void *o_out, float *lse_out, void *workspace, size_t workspace_bytes,
    locks_stream_t stream) {
  locks_status_t st = check_window(q, k_cache, v_cache, num_phys_pages,
                                   page_table, seq_lens, window, sinks,
                                   n_tokens, batch, h_q, h_kv, max_pages,
                                   o_out, lse_out, workspace);
  if (st != LOCKS_OK || batch == 0 || n_tokens == 0) return st;
  if (!q_starts) return LOCKS_ERR_INVALID_ARG;
  window = at_most_table(window, max_pages);
  sinks = at_most_table(sinks, max_pages);
  const int G = h_q / h_kv;
  // rows of a cache are int32 coordinates of its tensor map
  if (num_phys_pages > 0x7fffffffLL / (kPage * h_kv) ||
      ((long long)n_tokens * G / 128 + batch) * h_kv > 0x7fffffffLL)
    return LOCKS_ERR_UNSUPPORTED;
  const int splits =
      window_splits(n_tokens, batch, h_kv, G, max_pages, window, sinks);
  if (((long long)n_tokens * G / 128 + batch) * h_kv * splits > 0x7fffffffLL)
    return LOCKS_ERR_UNSUPPORTED;
  const size_t rows = splits > 1 ? (size_t)splits * n_tokens * h_q : 0;
  if (workspace_bytes < kWsHeader + window_region(rows))
    return LOCKS_ERR_WORKSPACE;
  uint8_t *ws = static_cast<uint8_t *>(workspace);
  cudaError_t e = launch_window(
      {static_cast<const __nv_bfloat16 *>(q),
       static_cast<const __nv_bfloat16 *>(k_cache),
       static_cast<const __nv_bfloat16 *>(v_cache), num_phys_pages, page_table,
       q_starts, seq_lens, n_tokens, window, sinks, batch, h_kv, G, max_pages,
       static_cast<__nv_bfloat16 *>(o_out), lse_out,
       reinterpret_cast<int32_t *>(ws), splits,
       reinterpret_cast<float *>(ws + kWsHeader),
       reinterpret_cast<float2 *>(ws + kWsHeader +
                                  round_up(rows * kDim * 4, 256)),
       0, false},
      (cudaStream_t)stream);
  return e == cudaSuccess ? LOCKS_OK : fail_cuda(e);
}

locks_status_t locks_clear_status(void *status_word, locks_stream_t stream) {
  if (!status_word) return LOCKS_ERR_INVALID_ARG;
  cudaError_t e =
      cudaMemsetAsync(status_word, 0, sizeof(int32_t), (cudaStream_t)stream);
  return e == cudaSuccess ? LOCKS_OK : fail_cuda(e);
}

locks_status_t locks_read_status(const void *status_word, int32_t *host_out,
                                 locks_stream_t stream) {
  if (!status_word || !host_out) return LOCKS_ERR_INVALID_ARG;
  cudaError_t e = cudaMemcpyAsync(host_out, status_word, sizeof(int32_t),
                                  cudaMemcpyDeviceToHost, (cudaStream_t)stream);
  if (e != cudaSuccess) return fail_cuda(e);
  e = cudaStreamSynchronize((cudaStream_t)stream);
  return e == cudaSuccess ? LOCKS_OK : fail_cuda(e);
}

}  // extern "C"
