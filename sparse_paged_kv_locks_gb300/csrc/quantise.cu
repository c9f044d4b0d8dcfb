// Writing rows into the quantised KV cache, and reading pages back.
//
// quantise: a row x of 128 numbers becomes codes e4m3(x / 2^e) and the byte
// e + 127, e from the row's largest magnitude (q_exponent).  Eight lanes take
// a row, 16 numbers each, so the maximum needs three shuffles and a lane's 16
// codes are one aligned group of the record; a warp holds four (token, head)
// rows at a time.  Reads and writes are each done once; both kernels are
// bound by memory: four prompts of 101K tokens and 8 heads 110 us (5.8 TB/s;
// 125 us before the rows were loaded ahead of their places; from fp32 150 us),
// two prompts of 32K read back 66 us (6.1 TB/s; as fp32 134 us, 5.0 TB/s); one
// token per sequence, or a page, 2 us among others and 8-9 us alone on cold data,
// by the launch and three dependent loads.
#include "launch.h"
#include "quantised.cuh"

namespace locks {

constexpr int kQThreads = 256;
constexpr int kQRowsPerBlock = kQThreads / 8;

// ---------------------------------------------------------------------------
// 16 consecutive numbers <-> registers
// ---------------------------------------------------------------------------
template <int TYPE>
__device__ __forceinline__ void load16(const void *base, int64_t at,
                                       float (&x)[16]) {
  if constexpr (TYPE == LOCKS_TYPE_FP32) {
    const float4 *p = reinterpret_cast<const float4 *>(
        static_cast<const float *>(base) + at);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float4 v = __ldg(p + i);
      x[4 * i] = v.x;
      x[4 * i + 1] = v.y;
      x[4 * i + 2] = v.z;
      x[4 * i + 3] = v.w;
    }
  } else {
    const uint4 *p = reinterpret_cast<const uint4 *>(
        static_cast<const uint16_t *>(base) + at);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint4 v = __ldg(p + i);
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        float2 f;
        if constexpr (TYPE == LOCKS_TYPE_BF16)
          f = make_float2(bf16_lo(w[j]), bf16_hi(w[j]));
        else
          f = __half22float2(u32_as_h2(w[j]));
        x[8 * i + 2 * j] = f.x;
        x[8 * i + 2 * j + 1] = f.y;
      }
    }
  }
}

template <int TYPE>
__device__ __forceinline__ void store16(void *base, size_t at,
                                        const float (&x)[16]) {
  if constexpr (TYPE == LOCKS_TYPE_FP32) {
    float4 *p = reinterpret_cast<float4 *>(static_cast<float *>(base) + at);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      p[i] = make_float4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
  } else {
    uint4 *p = reinterpret_cast<uint4 *>(static_cast<uint16_t *>(base) + at);
    uint32_t w[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if constexpr (TYPE == LOCKS_TYPE_BF16) {
        const __nv_bfloat162 v = __floats2bfloat162_rn(x[2 * j], x[2 * j + 1]);
        w[j] = *reinterpret_cast<const uint32_t *>(&v);
      } else {
        w[j] = h2_as_u32(__floats2half2_rn(x[2 * j], x[2 * j + 1]));
      }
    }
    p[0] = make_uint4(w[0], w[1], w[2], w[3]);
    p[1] = make_uint4(w[4], w[5], w[6], w[7]);
  }
}

// ---------------------------------------------------------------------------
// write
// ---------------------------------------------------------------------------
// one row (eight lanes, lane `j` its dims 16j .. 16j + 15) into slot s of a
// record's codes at `codes`, its exponent byte at `exps`
__device__ __forceinline__ void quantise_row(const float (&x)[16], int j,
                                             int s, uint8_t *codes,
                                             uint8_t *exps, bool live) {
  float m = 0.f;  // fmaxf drops NaN: a row's scale comes from its numbers
#pragma unroll
  for (int i = 0; i < 16; ++i) m = fmaxf(m, fabsf(x[i]));
#pragma unroll
  for (int o = 1; o < 8; o <<= 1)
    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  const int e = q_exponent(m);
  const float r = exp2_int(-e);
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    w[i] = e4m3x2_from(x[4 * i] * r, x[4 * i + 1] * r) |
           e4m3x2_from(x[4 * i + 2] * r, x[4 * i + 3] * r) << 16;
  if (!live) return;
  *reinterpret_cast<uint4 *>(codes + s * kDim + 16 * q_group(j, s)) =
      make_uint4(w[0], w[1], w[2], w[3]);
  if (j == 0) exps[s] = (uint8_t)(e + 127);
}

template <int TYPE>
__global__ void __launch_bounds__(kQThreads)
    quantise_kernel(const void *__restrict__ k_new,
                    const void *__restrict__ v_new, int64_t k_token,
                    int64_t k_head, int64_t v_token, int64_t v_head,
                    const int32_t *__restrict__ seq_ids,
                    const int32_t *__restrict__ positions, int n_tokens,
                    uint8_t *__restrict__ records, int64_t num_phys, int h_kv,
                    const int32_t *__restrict__ pt, int batch, int max_pages,
                    int32_t *status) {
  pdl_wait();
  // four tokens, then heads, then the next four: a warp has one head's rows of
  // four tokens, mostly neighbours in a page, so that their scale bytes are
  // one access
  const int64_t row =
      (int64_t)blockIdx.x * kQRowsPerBlock + (threadIdx.x >> 3);
  const int j = threadIdx.x & 7;
  const int64_t four = row / (4 * h_kv);
  const int rest = (int)(row - four * (4 * h_kv));
  const int64_t i = 4 * four + (rest & 3);  // token
  const int h = rest >> 2;
  bool live = i < n_tokens;
  // the rows are on their way while their places are looked up
  float x[16], y[16];
  int b = -1, pos = 0;
  if (live) {
    b = __ldg(seq_ids + i);
    pos = __ldg(positions + i);
    load16<TYPE>(k_new, i * k_token + h * k_head + 16 * j, x);
    load16<TYPE>(v_new, i * v_token + h * v_head + 16 * j, y);
  } else {
#pragma unroll
    for (int t = 0; t < 16; ++t) x[t] = y[t] = 0.f;
  }
  int64_t phys = 0;
  int slot = 0;
  if (b < 0) {  // padding
    live = false;
  } else if (b >= batch || pos < 0 || (pos >> 4) >= max_pages) {
    if (j == 0) set_status(status, LOCKS_DEV_BAD_PAIR);
    live = false;
  } else {
    phys = __ldg(pt + (size_t)b * max_pages + (pos >> 4));
    slot = pos & 15;
    if (phys < 0 || phys >= num_phys) {
      if (j == 0) set_status(status, LOCKS_DEV_BAD_PAGE_ID);
      live = false;
    }
  }
  uint8_t *rec = records + ((size_t)(live ? phys : 0) * h_kv + h) * kQRec;
  quantise_row(x, j, slot, rec, rec + kQOffKE, live);
  quantise_row(y, j, slot, rec + kQOffV, rec + kQOffVE, live);
}

// ---------------------------------------------------------------------------
// read
// ---------------------------------------------------------------------------
// Sixteen rows of a (pair, head) take 128 lanes, so a block reads two records
// at a time; outputs are page-shaped, [pair][h_kv][16][128].
template <int TYPE>
__global__ void __launch_bounds__(kQThreads)
    dequantise_kernel(const uint8_t *__restrict__ records, int64_t num_phys,
                      int h_kv, const int32_t *__restrict__ pt, int batch,
                      int max_pages, const int32_t *__restrict__ seq_ids,
                      const int32_t *__restrict__ page_ids, int n_pairs,
                      const int32_t *__restrict__ seq_lens, void *k_out,
                      void *v_out, int32_t *status) {
  pdl_wait();
  const int64_t unit = (int64_t)blockIdx.x * 2 + (threadIdx.x >> 7);
  const int64_t i = unit / h_kv;
  if (i >= n_pairs) return;
  const int h = (int)(unit - i * h_kv);
  const int s = (threadIdx.x >> 3) & 15, j = threadIdx.x & 7;
  const int b = __ldg(seq_ids + i), pg = __ldg(page_ids + i);
  int64_t phys = -1;
  bool live = false;
  if (b < 0 || b >= batch || pg < 0 || pg >= max_pages) {
    if (s == 0 && j == 0) set_status(status, LOCKS_DEV_BAD_PAIR);
  } else {
    phys = __ldg(pt + (size_t)b * max_pages + pg);
    if (phys < 0 || phys >= num_phys) {
      if (s == 0 && j == 0) set_status(status, LOCKS_DEV_BAD_PAGE_ID);
    } else {
      live = !seq_lens ||
             pg * kPage + s < checked_len(seq_lens, b, max_pages, status);
    }
  }
  const uint8_t *rec = records + ((size_t)(live ? phys : 0) * h_kv + h) * kQRec;
  const size_t at = ((size_t)unit * kPage + s) * kDim + 16 * j;
  uint4 c[2];
  int e[2];
#pragma unroll
  for (int kv = 0; kv < 2; ++kv) {
    c[kv] = make_uint4(0u, 0u, 0u, 0u);
    e[kv] = 127;
    if (!live || !(kv ? v_out : k_out)) continue;
    c[kv] = __ldg(reinterpret_cast<const uint4 *>(
        rec + kv * kQOffV + s * kDim + 16 * q_group(j, s)));
    e[kv] = __ldg(rec + kQOffKE + kv * kPage + s);
  }
#pragma unroll
  for (int kv = 0; kv < 2; ++kv) {
    void *out = kv ? v_out : k_out;
    if (!out) continue;
    const float scale = exp2_int(e[kv] - 127);
    const uint32_t w[4] = {c[kv].x, c[kv].y, c[kv].z, c[kv].w};
    float x[16];
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      const float2 lo = __half22float2(u32_as_h2(e4m3x2_lo(w[t])));
      const float2 hi = __half22float2(u32_as_h2(e4m3x2_hi(w[t])));
      x[4 * t] = lo.x * scale;
      x[4 * t + 1] = lo.y * scale;
      x[4 * t + 2] = hi.x * scale;
      x[4 * t + 3] = hi.y * scale;
    }
    store16<TYPE>(out, at, x);
  }
}

// ---------------------------------------------------------------------------
// launchers
// ---------------------------------------------------------------------------
cudaError_t launch_quantise(const void *k_new, const void *v_new, int type,
                            int64_t k_token, int64_t k_head, int64_t v_token,
                            int64_t v_head, const int32_t *seq_ids,
                            const int32_t *positions, int n_tokens,
                            void *records, int64_t num_phys, int h_kv,
                            const int32_t *pt, int batch, int max_pages,
                            int32_t *status, cudaStream_t stream) {
  auto *kern = type == LOCKS_TYPE_BF16   ? quantise_kernel<LOCKS_TYPE_BF16>
               : type == LOCKS_TYPE_FP16 ? quantise_kernel<LOCKS_TYPE_FP16>
                                         : quantise_kernel<LOCKS_TYPE_FP32>;
  const long long rows = ((long long)n_tokens + 3) / 4 * 4 * h_kv;
  const unsigned grid =
      (unsigned)((rows + kQRowsPerBlock - 1) / kQRowsPerBlock);
  return launch_pdl(kern, dim3(grid), dim3(kQThreads), 0, stream, k_new,
                    v_new, k_token, k_head, v_token, v_head, seq_ids,
                    positions, n_tokens, static_cast<uint8_t *>(records),
                    num_phys, h_kv, pt, batch, max_pages, status);
}

cudaError_t launch_dequantise(const void *records, int64_t num_phys, int h_kv,
                              const int32_t *pt, int batch, int max_pages,
                              const int32_t *seq_ids, const int32_t *page_ids,
                              int n_pairs, const int32_t *seq_lens, int type,
                              void *k_out, void *v_out, int32_t *status,
                              cudaStream_t stream) {
  auto *kern = type == LOCKS_TYPE_BF16   ? dequantise_kernel<LOCKS_TYPE_BF16>
               : type == LOCKS_TYPE_FP16 ? dequantise_kernel<LOCKS_TYPE_FP16>
                                         : dequantise_kernel<LOCKS_TYPE_FP32>;
  const long long units = (long long)n_pairs * h_kv;
  return launch_pdl(kern, dim3((unsigned)((units + 1) / 2)), dim3(kQThreads),
                    0, stream, static_cast<const uint8_t *>(records),
                    num_phys, h_kv, pt, batch, max_pages, seq_ids, page_ids,
                    n_pairs, seq_lens, k_out, v_out, status);
}

}  // namespace locks
