// Attention of one new token per sequence over the quantised KV cache: for
// every query head, x_t = q . k_t / sqrt(128), o = sum softmax(x)_t v_t and
// lse = ln sum exp(x_t), over the tokens of the listed pages (or of all).
//
// With keys k = 2^ek * c, values v = 2^ev * d (codes c, d), f = log2(e) /
// sqrt(128) and E the largest ev so far,
//   w_t = 2^(f 2^ek_t (q . c_t) - m + 8)
//   o   = 2^E sum w_t 2^(ev_t - E) d_t / sum w_t
//   lse = ln 2 * (log2(sum w_t) + m - 8)
// so a value's scale is part of its factor in the product.  The reference m
// follows scores alone and is taken off scores rounded like itself, which leaves
// equal scores equal however large they are.  m is raised, and
// the sums rescaled, only when a score passes it by more than 2^7: factors stay
// below 2^15 and, in fp16, keep full precision down to 2^-22 of the largest
// weight and some down to 2^-32.  A row whose scale lies far below E gets its
// factor in a bin of its own (kQdBins), with full precision down to 2^-118: the
// larger rows may be zero in the dims that this one fills.  Codes are exact in
// fp16, and so is the query after a power-of-two scale per head (elements 2^-22
// below its largest lose bits); products, sums and references are fp32.
//
// Bound: memory, 4128 bytes per listed page and KV head.  One bulk copy
// brings a record into a warp's private ring in shared memory, so the warps
// run free of one another.  256 lists of 128 pages (135 MB): 29-30 us, 4.5-4.7
// TB/s; copies of the same records in the same numbers that nothing uses take
// 24.5 us, this kernel without its arithmetic 29 us: what is left is the
// look-ups before the first copy and the merge after the last.  Two units of
// warps and stages were tried, 4 x 4 at three CTAs an SM and 8 x 3 at two: the
// same for lists, 72 against 92 us for a dense ragged batch.
//
// Tokens (then dims) are the M dimension of mma.m16n8k16 and the query heads
// the N dimension: a group of up to 8 heads is one column tile, and the page's
// 16 tokens fill M.  The order of dims in
// the products is free, so a lane's A fragments are whole 16-byte groups of a
// key row, and for the second product the 16 dims of one group.
#include "launch.h"
#include "quantised.cuh"

namespace locks {

constexpr int kQdWarps = 4;
constexpr int kQdThreads = 32 * kQdWarps;
constexpr int kQdStages = 4;
constexpr int kQdStride = 4224;  // ring stage: a record, 128-byte aligned
constexpr int kQdWarpRing = kQdStages * kQdStride;
constexpr int kQdRing = kQdWarps * kQdWarpRing;
// Split form: fewest list entries to a warp, so that a unit is not cut into
// more pieces than its merge is worth (2 units of 2,500 pages: 3 entries 39
// us, 6 28 us, 12 24 us).  Beside the prefix kernel, after which this one
// mostly runs and whose partials are merged anyhow, 2 (32K prefix for 32
// sequences: 12 entries 65 us, 2 51 us).
constexpr int kQdMinRun = 12, kQdMinRunBeside = 2;
// unit form for lists that are not given: tables of at most this many pages
// per CTA (a short sequence leaves its CTA idle, a long one would keep it)
constexpr int kQdUnitPages = 64;
constexpr float kQdLn2 = 0.69314718055994531f;
// Factors below fp16's normal numbers, of rows whose value scale is more than
// 2^kQSpread below the largest so far, are taken in bins of 24 powers of two
// each.  Ordinary pages pay two comparisons; with an infinity in every
// sequence's first page, 256 lists of 128 pages take 44 us instead of 29 and a
// dense ragged batch 82 instead of 70.
constexpr float kQdNormal = -14.f, kQdBin = 24.f;
constexpr int kQdBins = 4;

// One lane's entry of a window of 32 positions.
struct QEntry {
  const uint8_t *record;  // null: nothing to read
  int ntok, u;
};

struct QdArgs {
  const __nv_bfloat16 *q;
  const uint8_t *records;
  int64_t num_phys;
  const int32_t *pt, *seq_lens, *idx;
  int k, batch, h_kv, G, max_pages, n_warps;
  // pages that every sequence begins with (null, 0: none)
  const int32_t *prefix;
  int prefix_pages;
  __nv_bfloat16 *o_out;
  float *lse_out;
  float *o_part;     // [slot][G][128], sums not divided
  float2 *ml_part;   // [slot][G] (m, sum of weights)
  int *meta;         // run length, then the sequences' first positions
  int32_t *status;
  // launched beside the kernel that takes those pages: sequences at least as
  // long as they are leave them out of their lists, and this kernel waits for
  // that one only at its end.  What it reads until then was written by kernels
  // before both.  Every CTA of that kernel waits for those, which makes their
  // writes visible in L2, before it lets this one start, and none of the reads
  // goes through an L1 that could hold older values: queries, lengths and
  // tables by loads that bypass it, records by bulk copies.
  bool beside;
};

// pages of sequence b's own list, for lists that are not given
__device__ __forceinline__ int own_pages(const QdArgs &a, int L) {
  const int n = (L + kPage - 1) / kPage;
  return a.beside && L >= a.prefix_pages * kPage ? n - a.prefix_pages : n;
}

__device__ __forceinline__ QEntry q_resolve(const QdArgs &a,
                                            const PageLists &lists, int p,
                                            int pe) {
  QEntry e{nullptr, 0, 0};
  if (p >= pe) return e;
  const int b = lists.sequence(p);
  const int len = lists.length(b);
  const int r = p - lists.first(b);
  const int h = r / len;
  int pg = r - h * len;
  e.u = b * lists.h_kv + h;
  const int32_t *table = a.pt + (size_t)b * a.max_pages;
  int ph = 0;
  if (a.idx) {
    // the table entry is read beside the length it is checked against, where
    // the table has one
    pg = __ldcg(a.idx + (size_t)e.u * a.k + pg);
    if (pg < 0) return e;
    ph = pg < a.max_pages ? __ldcg(table + pg) : -1;
  }
  const int L = checked_len(a.seq_lens, b, a.max_pages, a.status);
  const int n = (L + kPage - 1) / kPage;
  if (a.idx) {
    if (pg >= n) {
      set_status(a.status, LOCKS_DEV_BAD_INDEX);
      return e;
    }
  } else {
    if (a.beside && L >= a.prefix_pages * kPage) pg += a.prefix_pages;
    if (pg >= n) return e;  // (unit form: lists as long as the table)
    if (pg < a.prefix_pages) table = a.prefix;
  }
  if (!a.idx) ph = __ldcg(table + pg);
  if (ph < 0 || ph >= a.num_phys) {
    set_status(a.status, LOCKS_DEV_BAD_PAGE_ID);
    return e;
  }
  e.record = a.records + ((size_t)ph * lists.h_kv + h) * kQRec;
  e.ntok = min(kPage, L - pg * kPage);
  return e;
}

__device__ __forceinline__ uint32_t pack_h2(float lo, float hi) {
  return h2_as_u32(__floats2half2_rn(lo, hi));
}
__device__ __forceinline__ uint32_t pack_bf2q(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t *>(&v);
}

// NT: column tiles of 8 query heads (1: G <= 8, 2: G <= 16).
// UNIT: lists of k entries each (the given ones, or k = max_pages), one unit
// to a CTA or cluster, merged on chip; otherwise every warp takes a run of
// positions and units that span runs are merged by merge_kernel.
template <int NT, bool UNIT>
__global__ void __launch_bounds__(kQdThreads, NT == 1 ? 3 : 2)
    qdecode_kernel(const QdArgs a) {
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ uint64_t s_bar[kQdWarps][kQdStages];
  int *s_pre = reinterpret_cast<int *>(smem + kQdRing);  // [batch + 1]
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
  const int g = lane >> 2, t = lane & 3;
  const int h_q = a.h_kv * a.G;
  const PageLists lists{s_pre, a.batch, a.h_kv,
                        UNIT || a.idx ? a.h_kv * a.k : 0};
  uint64_t *bar = s_bar[wid];
  if (lane == 0) {
#pragma unroll
    for (int i = 0; i < kQdStages; ++i) mbar_init(bar + i, 1);
    fence_mbar_init();
  }
  __syncwarp();
  if (UNIT || !a.beside) pdl_wait();
  pdl_trigger();

  int total = 0;
  if (UNIT || a.idx) {
    total = a.batch * a.h_kv * a.k;
  } else {
    for (int b = threadIdx.x; b < a.batch; b += kQdThreads)
      s_pre[b + 1] =
          a.h_kv * own_pages(a, checked_len(a.seq_lens, b, a.max_pages,
                                            blockIdx.x ? nullptr : a.status));
    if (threadIdx.x == 0) s_pre[0] = 0;
    __syncthreads();
    if (wid == 0) {
      int run = 0;  // of the entries before this block of 32
      for (int b0 = 1; b0 <= a.batch; b0 += 32) {
        int v = b0 + lane <= a.batch ? s_pre[b0 + lane] : 0;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int w = __shfl_up_sync(0xffffffffu, v, o);
          if (lane >= o) v += w;
        }
        if (b0 + lane <= a.batch) s_pre[b0 + lane] = run + v;
        run += __shfl_sync(0xffffffffu, v, 31);
      }
    }
    __syncthreads();
    total = s_pre[a.batch];
  }

  // this warp's run of positions [pb, pe)
  const int gw = blockIdx.x * kQdWarps + wid;
  const int ucl = UNIT ? (int)cluster_nctarank() : 1;
  const int urank = UNIT && ucl > 1 ? (int)cluster_ctarank() : 0;
  const int unit0 = UNIT ? (int)blockIdx.x / ucl : 0;
  int pb, pe, chunk = 0;
  if constexpr (UNIT) {
    const int sl = urank * kQdWarps + wid, nsl = ucl * kQdWarps;
    pb = unit0 * a.k + (int)((long long)sl * a.k / nsl);
    pe = unit0 * a.k + (int)((long long)(sl + 1) * a.k / nsl);
  } else {
    chunk = (int)max((long long)(a.beside ? kQdMinRunBeside : kQdMinRun),
                     ((long long)total + a.n_warps - 1) / a.n_warps);
    if (blockIdx.x == 0) {  // for the merge
      if (threadIdx.x == 0) a.meta[0] = chunk;
      if (!a.idx)
        for (int b = threadIdx.x; b <= a.batch; b += kQdThreads)
          a.meta[1 + b] = s_pre[b];
    }
    const long long from = (long long)gw * chunk;
    if (gw >= a.n_warps || from >= total) {
      if (a.beside) pdl_wait();
      return;
    }
    pb = (int)from;
    pe = min(total, pb + chunk);
  }

  uint8_t *ring = smem + wid * kQdWarpRing;
  const uint32_t ring_s = smem_u32(ring);

  // window of 32 positions: this lane's entry, and those not yet copied
  int win = pb - 32;
  uint32_t left = 0;
  QEntry we{nullptr, 0, 0};
  // has the next entry copied to stage st; its tokens (0: none left), unit
  auto issue = [&](int st, int &ntok, int &u) {
    while (left == 0) {
      win += 32;
      if (win >= pe) {
        ntok = 0;
        return;
      }
      we = q_resolve(a, lists, win + lane, pe);
      left = __ballot_sync(0xffffffffu, we.record != nullptr);
    }
    const int j = __ffs(left) - 1;
    left &= left - 1;
    if (lane == j) {
      mbar_arrive_tx(bar + st, kQRec);
      bulk_g2s(ring + st * kQdStride, we.record, kQRec, bar + st);
    }
    ntok = __shfl_sync(0xffffffffu, we.ntok, j);
    u = UNIT ? 0 : __shfl_sync(0xffffffffu, we.u, j);
  };
  // copies in flight, oldest first
  int fn[kQdStages], fu[kQdStages];
#pragma unroll
  for (int i = 0; i < kQdStages; ++i) {
    fn[i] = fu[i] = 0;
    issue(i, fn[i], fu[i]);
  }

  // query B fragments of a unit: column n = head 8 nt + g of the group,
  // k-step 4 j + w of the product over dims 16 (t + 4 j) + 4 w .. + 3; f:
  // factors of the scores of heads 8 nt + 2t, 2t + 1
  uint32_t qb[NT][8][2];
  float f[NT][2];
  auto load_q = [&](int u) {
    const int b = u / a.h_kv, h = u - b * a.h_kv;
    const __nv_bfloat16 *qu = a.q + ((size_t)b * h_q + (size_t)h * a.G) * kDim;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const bool in = 8 * nt + g < a.G;
      uint32_t raw[16];
      float top = 0.f;
#pragma unroll
      for (int i = 0; i < 4; ++i) {  // 16-byte loads: group t + 4 (i / 2)
        const uint4 v =
            in ? __ldcg(reinterpret_cast<const uint4 *>(
                     qu + (8 * nt + g) * kDim + 16 * (t + 4 * (i >> 1)) +
                     8 * (i & 1)))
               : make_uint4(0u, 0u, 0u, 0u);
        raw[4 * i] = v.x;
        raw[4 * i + 1] = v.y;
        raw[4 * i + 2] = v.z;
        raw[4 * i + 3] = v.w;
      }
#pragma unroll
      for (int i = 0; i < 16; ++i)
        top = fmaxf(top, fmaxf(fabsf(bf16_lo(raw[i])), fabsf(bf16_hi(raw[i]))));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
      // largest magnitude to [2^7, 2^8)
      const int e = max(-100, (int)(__float_as_uint(top) >> 23) - 127) - 7;
      const float down = exp2_int(-e);
#pragma unroll
      for (int i = 0; i < 16; ++i)
        qb[nt][i >> 1][i & 1] =
            pack_h2(bf16_lo(raw[i]) * down, bf16_hi(raw[i]) * down);
      const float fe = exp2_int(e) * kQScale;
      f[nt][0] = __shfl_sync(0xffffffffu, fe, 8 * t);
      f[nt][1] = __shfl_sync(0xffffffffu, fe, 8 * t + 4);
    }
  };

  // sums: tile i holds dims 16 g + 2 i (elements 0, 1) and 16 g + 2 i + 1
  // (2, 3) of heads 8 nt + 2t (0, 2) and 8 nt + 2t + 1 (1, 3)
  float o[NT][8][4], m[NT][2], l[NT][2];
  uint32_t e_top = 0;  // largest value scale so far: the sums' unit, E + 127
  auto reset = [&]() {
    e_top = 0;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        o[nt][i][0] = o[nt][i][1] = o[nt][i][2] = o[nt][i][3] = 0.f;
      m[nt][0] = m[nt][1] = -INFINITY;
      l[nt][0] = l[nt][1] = 0.f;
    }
  };
  reset();

  // the unit's sums so far: the result where the unit lies in this run
  // alone, else a partial (slot unit + warp, distinct for distinct pieces
  // because both grow along the positions; UNIT: this warp's ring)
  auto flush = [&](int u) {
    const int b = u / a.h_kv, h = u - b * a.h_kv;
    bool whole = false;
    if constexpr (!UNIT) {
      const int2 sp = lists.span(u);
      whole = !a.beside && sp.x >= pb && sp.y <= pe;
    }
    const float unit = exp2_int((int)e_top - 127);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        float ls = l[nt][c];
        ls += __shfl_xor_sync(0xffffffffu, ls, 4);
        ls += __shfl_xor_sync(0xffffffffu, ls, 8);
        ls += __shfl_xor_sync(0xffffffffu, ls, 16);
        const int hd = 8 * nt + 2 * t + c;
        if (hd >= a.G) continue;
        if (whole) {
          const size_t row = (size_t)b * h_q + (size_t)h * a.G + hd;
          const float inv = ls == 0.f ? 0.f : unit / ls;
          uint4 *dst = reinterpret_cast<uint4 *>(a.o_out + row * kDim + 16 * g);
          uint32_t w[8];
#pragma unroll
          for (int i = 0; i < 8; ++i)
            w[i] = pack_bf2q(o[nt][i][c] * inv, o[nt][i][2 + c] * inv);
          dst[0] = make_uint4(w[0], w[1], w[2], w[3]);
          dst[1] = make_uint4(w[4], w[5], w[6], w[7]);
          if (g == 0)
            a.lse_out[row] = ls == 0.f
                                 ? -INFINITY
                                 : (log2f(ls) + (m[nt][c] - kQLift)) * kQdLn2;
        } else {
          float *po = UNIT ? reinterpret_cast<float *>(ring) + hd * kDim
                           : a.o_part + (((size_t)u + gw) * a.G + hd) * kDim;
          float2 *ml =
              UNIT ? reinterpret_cast<float2 *>(ring + 8 * NT * kDim * 4) + hd
                   : a.ml_part + ((size_t)u + gw) * a.G + hd;
          float4 *dst = reinterpret_cast<float4 *>(po + 16 * g);
#pragma unroll
          for (int i = 0; i < 4; ++i)
            dst[i] = make_float4(
                o[nt][2 * i][c] * unit, o[nt][2 * i][2 + c] * unit,
                o[nt][2 * i + 1][c] * unit, o[nt][2 * i + 1][2 + c] * unit);
          if (g == 0) *ml = make_float2(m[nt][c], ls);
        }
      }
  };

  int cur = UNIT ? unit0 : lists.unit(pb);
  bool q_ready = false, dead = false;
  auto advance = [&](int u) {  // close the units before u
    while (cur < u) {
      const int2 sp = lists.span(cur);
      if (sp.y > sp.x) {
        flush(cur);
        reset();
      }
      ++cur;
      q_ready = false;
    }
  };

  // where this lane reads in a record: key codes of tokens g, g + 8, groups
  // t, t + 4; value codes of tokens 2t, 2t + 1, 2t + 8, 2t + 9, group g; the
  // scales of tokens g, g + 8
  const uint32_t k_at = ring_s + g * kDim + 16 * q_group(t, g);
  const uint32_t k_at4 = ring_s + g * kDim + 16 * q_group(t + 4, g);
  const uint32_t v_at = ring_s + kQOffV + 2 * t * kDim + 16 * q_group(g, 2 * t);
  const uint32_t v_at1 =
      ring_s + kQOffV + (2 * t + 1) * kDim + 16 * q_group(g, 2 * t + 1);
  const uint32_t e_at = ring_s + kQOffKE + g;

  // The factors of a page below fp16's normal numbers, in bins b = 1 .. 4 of
  // 2^(-14 - 24 b) <= w < 2^(-14 - 24 (b - 1)): a bin's factors times 2^(24 b)
  // have all their bits, its products are added with 2^(-24 b).  What is left
  // out is 2^-118 of the largest contribution.  Their y become -infinity, as
  // of places without a token: nothing is left of them for the page's products.
  auto binned_weights = [&](float (&y)[NT][4], const uint32_t (&e2)[2],
                            const uint4 (&vc)[4]) {
    const float unit[2] = {(float)((int)e2[0] - (int)e_top),
                           (float)((int)e2[1] - (int)e_top)};
#pragma unroll 1
    for (int b = 1; b <= kQdBins; ++b) {
      uint32_t pb0[NT], pb1[NT];
      bool some = false;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float at = y[nt][i] + unit[i >> 1] + kQdBin * (float)b;
          const bool here = at >= kQdNormal && at < kQdNormal + kQdBin;
          w[i] = here ? ex2_fast(at) : 0.f;
          some |= here;
        }
        pb0[nt] = movmatrix_trans(pack_h2(w[0], w[1]));
        pb1[nt] = movmatrix_trans(pack_h2(w[2], w[3]));
      }
      if (!__any_sync(0xffffffffu, some)) continue;
      const float down = exp2_int(-(int)kQdBin * b);
      const uint32_t *v0 = &vc[0].x, *v1 = &vc[1].x, *v2 = &vc[2].x,
                     *v3 = &vc[3].x;
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const uint32_t a01 = __byte_perm(v0[w], v1[w], 0x5140);
        const uint32_t a23 = __byte_perm(v2[w], v3[w], 0x5140);
        const uint32_t b01 = __byte_perm(v0[w], v1[w], 0x7362);
        const uint32_t b23 = __byte_perm(v2[w], v3[w], 0x7362);
        const uint32_t fa[4] = {e4m3x2_lo(a01), e4m3x2_hi(a01), e4m3x2_lo(a23),
                                e4m3x2_hi(a23)};
        const uint32_t fb[4] = {e4m3x2_lo(b01), e4m3x2_hi(b01), e4m3x2_lo(b23),
                                e4m3x2_hi(b23)};
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float t0[4] = {0.f, 0.f, 0.f, 0.f}, t1[4] = {0.f, 0.f, 0.f, 0.f};
          mma_f16(t0, fa, pb0[nt], pb1[nt]);
          mma_f16(t1, fb, pb0[nt], pb1[nt]);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            o[nt][2 * w][i] = fmaf(t0[i], down, o[nt][2 * w][i]);
            o[nt][2 * w + 1][i] = fmaf(t1[i], down, o[nt][2 * w + 1][i]);
          }
        }
      }
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (y[nt][i] + unit[i >> 1] < kQdNormal) {
          l[nt][i & 1] += ex2_fast(y[nt][i]);
          y[nt][i] = -INFINITY;
        }
  };

  uint32_t phase = 0;
  int st = 0;
  while (fn[0] > 0) {
    const int ntok = fn[0];
    if (!UNIT && fu[0] != cur) advance(fu[0]);
    if (!q_ready) {
      load_q(cur);
      q_ready = true;
    }
    // one verdict for the warp: its lanes' waits may end on either side of the
    // limit, and what follows either way takes all of them
    if (!__all_sync(0xffffffffu, q_wait(bar + st, phase))) {
      dead = true;
      break;
    }
    const uint32_t off = st * kQdStride;
    uint4 kc[2][2], vc[4];
    kc[0][0] = lds128(k_at + off);
    kc[1][0] = lds128(k_at + off + 8 * kDim);
    kc[0][1] = lds128(k_at4 + off);
    kc[1][1] = lds128(k_at4 + off + 8 * kDim);
    uint32_t ek[2], e2[2];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      asm volatile("ld.shared.u8 %0, [%1];\n"
                   : "=r"(ek[r])
                   : "r"(e_at + off + 8 * r));
      asm volatile("ld.shared.u8 %0, [%1];\n"
                   : "=r"(e2[r])
                   : "r"(e_at + off + kPage + 8 * r));
    }
    vc[0] = lds128(v_at + off);
    vc[1] = lds128(v_at1 + off);
    vc[2] = lds128(v_at + off + 8 * kDim);
    vc[3] = lds128(v_at1 + off + 8 * kDim);
    float ks[2];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      ks[r] = __uint_as_float(ek[r] << 23);
      e2[r] = q_scale_byte(e2[r]);
    }
    if (ntok < kPage) {  // rows past the end hold anything
#pragma unroll
      for (int r = 0; r < 4; ++r)
        if (2 * t + (r & 1) + 8 * (r >> 1) >= ntok)
          vc[r] = make_uint4(0u, 0u, 0u, 0u);
    }

    // scores: rows = tokens, columns = heads
    float s[NT][4], s2[NT][4];  // two chains of four products
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < 4; ++i) s[nt][i] = s2[nt][i] = 0.f;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const uint32_t k0[4] = {kc[0][j].x, kc[0][j].y, kc[0][j].z, kc[0][j].w};
      const uint32_t k1[4] = {kc[1][j].x, kc[1][j].y, kc[1][j].z, kc[1][j].w};
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const uint32_t fa[4] = {e4m3x2_lo(k0[w]), e4m3x2_lo(k1[w]),
                                e4m3x2_hi(k0[w]), e4m3x2_hi(k1[w])};
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
          mma_f16(w & 1 ? s2[nt] : s[nt], fa, qb[nt][4 * j + w][0],
                  qb[nt][4 * j + w][1]);
      }
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < 4; ++i) s[nt][i] += s2[nt][i];

    // weights
    const bool in[2] = {g < ntok, g + 8 < ntok};
    float y[NT][4];  // log2 of a weight
    // a scale above all before (the sums' unit follows it), or far below them
    bool rare = (in[0] && e_top - e2[0] > kQSpread) ||
                (in[1] && e_top - e2[1] > kQSpread);
    auto score = [&](int nt, int i) -> float {
      return __fmul_rn(s[nt][i], f[nt][i & 1] * ks[i >> 1]);
    };
    auto log_weights = [&]() {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          y[nt][i] = in[i >> 1] ? score(nt, i) - (m[nt][i & 1] - kQLift)
                                : -INFINITY;
    };
    log_weights();
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int c = 0; c < 2; ++c)
        rare |= fmaxf(y[nt][c], y[nt][2 + c]) > kQLift + kQSlack;
    if (__any_sync(0xffffffffu, rare)) {
      const uint32_t e_was = e_top;
      e_top = max(e_top, __reduce_max_sync(0xffffffffu,
                                           max(in[0] ? e2[0] : 0u,
                                               in[1] ? e2[1] : 0u)));
      const float unit = exp2_int(max(-126, (int)e_was - (int)e_top));
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          float top = fmaxf(in[0] ? score(nt, c) : -INFINITY,
                            in[1] ? score(nt, 2 + c) : -INFINITY);
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 4));
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 8));
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 16));
          top = fmaxf(top, m[nt][c]);
          const float fall = m[nt][c] == top ? 1.f : ex2_fast(m[nt][c] - top);
          m[nt][c] = top;
          l[nt][c] *= fall;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            o[nt][i][c] *= fall * unit;
            o[nt][i][2 + c] *= fall * unit;
          }
        }
      log_weights();
      // rows far below the largest scale whose weight fp16 would round to fewer
      // bits, or to nothing, although the larger rows may hold zeros in the
      // dims that these do not
      bool low = false;
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const float least = kQdNormal + (float)((int)e_top - (int)e2[r]);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int c = 0; c < 2; ++c)
            low |= in[r] && e_top - e2[r] > kQSpread &&
                   y[nt][2 * r + c] < least;
      }
      if (__any_sync(0xffffffffu, low)) binned_weights(y, e2, vc);
    }
    float v_unit[2];
#pragma unroll
    for (int r = 0; r < 2; ++r)
      v_unit[r] = in[r] ? exp2_int((int)e2[r] - (int)e_top) : 0.f;
    uint32_t pb0[NT], pb1[NT];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      float w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        w[i] = ex2_fast(y[nt][i]);
        l[nt][i & 1] += w[i];
        w[i] *= v_unit[i >> 1];
      }
      pb0[nt] = movmatrix_trans(pack_h2(w[0], w[1]));
      pb1[nt] = movmatrix_trans(pack_h2(w[2], w[3]));
    }

    // sums: rows = dims, columns = heads, k = tokens
    const uint32_t *v0 = &vc[0].x, *v1 = &vc[1].x, *v2 = &vc[2].x,
                   *v3 = &vc[3].x;
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      const uint32_t a01 = __byte_perm(v0[w], v1[w], 0x5140);
      const uint32_t a23 = __byte_perm(v2[w], v3[w], 0x5140);
      const uint32_t b01 = __byte_perm(v0[w], v1[w], 0x7362);
      const uint32_t b23 = __byte_perm(v2[w], v3[w], 0x7362);
      const uint32_t fa[4] = {e4m3x2_lo(a01), e4m3x2_hi(a01), e4m3x2_lo(a23),
                              e4m3x2_hi(a23)};
      const uint32_t fb[4] = {e4m3x2_lo(b01), e4m3x2_hi(b01), e4m3x2_lo(b23),
                              e4m3x2_hi(b23)};
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        mma_f16(o[nt][2 * w], fa, pb0[nt], pb1[nt]);
        mma_f16(o[nt][2 * w + 1], fb, pb0[nt], pb1[nt]);
      }
    }

    // the stage is read, by the fence's word and not by chance: refill it
    // (costs nothing: 30.8 us at 32 sequences of 128 pages with and without)
    fence_to_async();
    __syncwarp();
#pragma unroll
    for (int i = 0; i + 1 < kQdStages; ++i) {
      fn[i] = fn[i + 1];
      fu[i] = fu[i + 1];
    }
    issue(st, fn[kQdStages - 1], fu[kQdStages - 1]);
    if (++st == kQdStages) {
      st = 0;
      phase ^= 1;
    }
  }
  if (dead) {  // give the copies in flight a last, bounded chance to land
    if (lane == 0) set_status(a.status, LOCKS_DEV_TIMEOUT);
    for (int i = 0; i < kQdStages; ++i)
      if (fn[i] > 0) {
        const int at = st + i < kQdStages ? st + i : st + i - kQdStages;
        q_wait(bar + at, phase ^ (st + i < kQdStages ? 0u : 1u));
      }
  }
  __syncwarp();

  if constexpr (!UNIT) {
    const int last = lists.unit(pe - 1);
    advance(last);
    flush(last);
    if (a.beside) pdl_wait();
  } else {
    // the 4 C slices of the unit, merged head by head: CTA r of the cluster
    // takes heads r, r + C, .., its warp w every fourth of those; a lane
    // four dims
    flush(unit0);
    if (ucl > 1)
      cluster_sync();
    else
      __syncthreads();
    const int b = unit0 / a.h_kv, h = unit0 - b * a.h_kv;
    const int nsl = ucl * kQdWarps;
    const uint32_t base = smem_u32(smem);
    auto part = [&](int sl, int byte) -> uint32_t {
      const uint32_t at =
          base + (uint32_t)((sl % kQdWarps) * kQdWarpRing + byte);
      return ucl > 1 ? mapa_shared(at, (uint32_t)(sl / kQdWarps)) : at;
    };
    constexpr int kOffMl = 8 * NT * kDim * 4;
    for (int hd = urank + ucl * wid; hd < a.G; hd += ucl * kQdWarps) {
      // lane sl holds slice sl's reference and sum (at most 32 slices)
      float pm = -INFINITY, pl = 0.f;
      if (lane < nsl) {
        const uint32_t at = part(lane, kOffMl + 8 * hd);
        pm = ld_cluster_f32(at);
        pl = ld_cluster_f32(at + 4);
      }
      float M = pm;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1)
        M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, d));
      // a slice without tokens weighs nothing; one whose scores are not
      // numbers carries that on
      const float wt = pl == 0.f || pm == M ? (pl == 0.f ? 0.f : 1.f)
                                            : ex2_fast(pm - M);
      float sum = pl * wt;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1)
        sum += __shfl_xor_sync(0xffffffffu, sum, d);
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int s0 = 0; s0 < nsl; s0 += 4) {
        float4 v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          v[i] = ld_cluster_v4f(part(s0 + i, (hd * kDim + 4 * lane) * 4));
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float x = __shfl_sync(0xffffffffu, wt, s0 + i);
          if (x == 0.f) continue;
          acc.x = fmaf(x, v[i].x, acc.x);
          acc.y = fmaf(x, v[i].y, acc.y);
          acc.z = fmaf(x, v[i].z, acc.z);
          acc.w = fmaf(x, v[i].w, acc.w);
        }
      }
      const float inv = sum == 0.f ? 0.f : 1.f / sum;
      const size_t row = (size_t)b * h_q + (size_t)h * a.G + hd;
      reinterpret_cast<uint2 *>(a.o_out + row * kDim)[lane] =
          make_uint2(pack_bf2q(acc.x * inv, acc.y * inv),
                     pack_bf2q(acc.z * inv, acc.w * inv));
      if (lane == 0)
        a.lse_out[row] = sum == 0.f
                             ? -INFINITY
                             : (log2f(sum) + (M - kQLift)) * kQdLn2;
    }
    if (ucl > 1) cluster_sync();  // no CTA leaves while its slices are read
  }
}

// ---------------------------------------------------------------------------
// merge of partials
// ---------------------------------------------------------------------------
// W warps to a (sequence, query head) row, each every W-th partial, four dims
// to a lane: the pieces that the runs left of the row's unit, and before them
// the partials of the shared prefix where there is one (`shared` of them,
// [split][batch * h_q], skipped by sequences shorter than the prefix).  The
// references come first, all at once (a thread each), so that the sums' loads
// depend on nothing and are in flight together.  Bound by the latency of these
// three rounds of loads, and by the partials' bytes where rows are many: W is
// the most that keeps all rows' warps resident in two waves (4,096 rows of some
// 23 partials, caches cold: 8 warps 28 us, 2 warps 25 us; 16 rows of 200, as
// part of their call: 4 warps 39 us, 8 warps 28 us).
constexpr int kMergeWarps = 8;

template <int W>
__global__ void __launch_bounds__(32 * kMergeWarps)
    merge_kernel(const QdArgs a, const float *__restrict__ shared_o,
                 const float2 *__restrict__ shared_ml, int shared) {
  constexpr int kAtOnce = 32 * W;  // partials weighed at a time
  __shared__ float s_weight[32 * kMergeWarps], s_red[2][kMergeWarps];
  __shared__ float4 s_acc[kMergeWarps][32];
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int group = warp / W, wid = warp % W, first = group * W;
  const int in_group = wid * 32 + lane;
  const int rows = a.batch * a.h_kv * a.G;
  const int row = blockIdx.x * (kMergeWarps / W) + group;
  if (row >= rows) return;
  auto sync = [&]() {  // the row's warps
    if constexpr (W == 1)
      __syncwarp();
    else
      asm volatile("bar.sync %0, %1;\n" ::"r"(1 + group), "n"(32 * W)
                   : "memory");
  };
  const int u = row / a.G, hd = row - u * a.G;
  const int b = u / a.h_kv;
  const PageLists lists{a.meta + 1, a.batch, a.h_kv,
                        a.idx ? a.h_kv * a.k : 0};
  const int chunk = a.meta[0];
  const int2 sp = lists.span(u);
  const int L = shared ? checked_len(a.seq_lens, b, a.max_pages, nullptr) : 0;
  int w0 = 0, own = 0;
  if (sp.y > sp.x) {
    w0 = sp.x / chunk;
    own = (sp.y - 1) / chunk - w0 + 1;
    if (own == 1 && !a.beside) return;  // written by its warp
  }
  if (L < a.prefix_pages * kPage) shared = 0;
  const int n = shared + own;
  auto place = [&](int s) -> size_t {
    return s < shared ? (size_t)s * rows + row
                      : ((size_t)u + w0 + (s - shared)) * a.G + hd;
  };
  float M = -INFINITY, sum = 0.f;  // the same in all threads
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);  // this warp's share
  for (int s0 = 0; s0 < n; s0 += kAtOnce) {
    const int s = s0 + in_group;
    float2 ml = make_float2(-INFINITY, 0.f);
    if (s < n) ml = (s < shared ? shared_ml : a.ml_part)[place(s)];
    float top = ml.x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1)
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    if (W > 1) {
      if (lane == 0) s_red[0][warp] = top;
      sync();
#pragma unroll
      for (int w = 0; w < W; ++w) top = fmaxf(top, s_red[0][first + w]);
    }
    top = fmaxf(top, M);
    const float fall = M == top ? 1.f : ex2_fast(M - top);
    M = top;
    // nothing from a partial without tokens; one whose scores are not
    // numbers carries that on
    const float x = ml.y == 0.f ? 0.f : ml.x == M ? 1.f : ex2_fast(ml.x - M);
    float part = x * ml.y;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1)
      part += __shfl_xor_sync(0xffffffffu, part, o);
    if (W > 1 && lane == 0) s_red[1][warp] = part;
    s_weight[first * 32 + in_group] = x;
    sync();
    if (W > 1) {
      part = 0.f;
#pragma unroll
      for (int w = 0; w < W; ++w) part += s_red[1][first + w];
    }
    sum = sum * fall + part;
    acc.x *= fall;
    acc.y *= fall;
    acc.z *= fall;
    acc.w *= fall;
    const int m = min(n - s0, kAtOnce);
#pragma unroll 8
    for (int i = wid; i < m; i += W) {
      const float wt = s_weight[first * 32 + i];
      const int si = s0 + i;
      const float4 v =
          reinterpret_cast<const float4 *>(si < shared ? shared_o : a.o_part)
              [place(si) * (kDim / 4) + lane];
      if (wt == 0.f) continue;
      acc.x = fmaf(wt, v.x, acc.x);
      acc.y = fmaf(wt, v.y, acc.y);
      acc.z = fmaf(wt, v.z, acc.z);
      acc.w = fmaf(wt, v.w, acc.w);
    }
    if (s0 + kAtOnce < n) sync();  // weights read
  }
  if (W > 1) {
    s_acc[warp][lane] = acc;
    sync();
    if (wid != 0) return;
#pragma unroll
    for (int w = 1; w < W; ++w) {
      const float4 v = s_acc[first + w][lane];
      acc.x += v.x;
      acc.y += v.y;
      acc.z += v.z;
      acc.w += v.w;
    }
  }
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  reinterpret_cast<uint2 *>(a.o_out + (size_t)row * kDim)[lane] = make_uint2(
      pack_bf2q(acc.x * inv, acc.y * inv), pack_bf2q(acc.z * inv, acc.w * inv));
  if (lane == 0)
    a.lse_out[row] =
        sum == 0.f ? -INFINITY : (log2f(sum) + (M - kQLift)) * kQdLn2;
}

// ---------------------------------------------------------------------------
// launchers
// ---------------------------------------------------------------------------
// dynamic shared memory: what a CTA may have without its barriers, and the
// largest batch whose positions fit beside the ring
constexpr size_t kQdSmemMost = 227 * 1024 - 256;
constexpr int kQdMaxBatch = 41088;
static_assert(sizeof(uint64_t) * kQdWarps * kQdStages <= 256, "barriers");
static_assert(kQdRing + sizeof(int) * (kQdMaxBatch + 1) <= kQdSmemMost,
              "ring and positions");

static size_t qdecode_smem(bool unit, int batch) {
  return (size_t)kQdRing + (unit ? 0 : sizeof(int) * ((size_t)batch + 1));
}

int qdecode_max_batch() { return kQdMaxBatch; }

template <int NT, bool UNIT>
static cudaError_t qdecode_ready() {
  static DeviceFlags done;
  return once_per_device(done, [] {
    return cudaFuncSetAttribute(qdecode_kernel<NT, UNIT>,
                                cudaFuncAttributeMaxDynamicSharedMemorySize,
                                (int)kQdSmemMost);
  });
}

// The cluster size of the unit form, 0 for the split form.
static int unit_cluster(long long units, int k) {
  const int sms = device_sm_count();
  if (units > 0x7fffffffLL / (8 * kQdWarps)) return 0;
  if (units >= sms) return 1;
  for (int c = 8; c >= 2; c >>= 1)
    if (units * c <= 2LL * sms && k >= c * kQdWarps) return c;
  return k <= 2 * kQdWarps ? 1 : 0;
}

cudaError_t launch_qdecode(const void *q, const void *records,
                           int64_t num_phys, const int32_t *pt,
                           const int32_t *seq_lens, const int32_t *idx, int k,
                           int batch, int h_kv, int G, int max_pages,
                           const int32_t *prefix, int prefix_pages,
                           int max_warps, void *o_out, float *lse_out,
                           float *o_part, float2 *ml_part, int *meta,
                           const float *shared_o, const float2 *shared_ml,
                           int shared, int32_t *status, cudaStream_t stream) {
  QdArgs a{static_cast<const __nv_bfloat16 *>(q),
           static_cast<const uint8_t *>(records),
           num_phys, pt, seq_lens, idx, k, batch, h_kv, G, max_pages, 0,
           prefix, prefix_pages, static_cast<__nv_bfloat16 *>(o_out), lse_out,
           o_part, ml_part, meta, status, shared > 0};
  const bool wide = G > 8;
  const long long units = (long long)batch * h_kv;
  if (!idx) a.k = max_pages;
  int ucl = shared > 0 ? 0 : unit_cluster(units, a.k);
  if (!idx && max_pages > kQdUnitPages * ucl) ucl = 0;
  if (ucl > 0) {
    cudaError_t e = wide ? qdecode_ready<2, true>() : qdecode_ready<1, true>();
    if (e != cudaSuccess) return e;
    auto *kern = wide ? qdecode_kernel<2, true> : qdecode_kernel<1, true>;
    const dim3 grid((unsigned)(units * ucl));
    const size_t smem = qdecode_smem(true, batch);
    return ucl > 1 ? launch_pdl_cluster(kern, grid, dim3(kQdThreads), smem,
                                        stream, ucl, a)
                   : launch_pdl(kern, grid, dim3(kQdThreads), smem, stream, a);
  }
  cudaError_t e = wide ? qdecode_ready<2, false>() : qdecode_ready<1, false>();
  if (e != cudaSuccess) return e;
  // a grid that fills the GPU, at most one warp per list entry
  long long warps = (long long)(wide ? 2 : 3) * device_sm_count() * kQdWarps;
  if (warps > max_warps) warps = max_warps;
  a.n_warps = (int)warps;
  auto *kern = wide ? qdecode_kernel<2, false> : qdecode_kernel<1, false>;
  e = launch_pdl(kern, dim3((a.n_warps + kQdWarps - 1) / kQdWarps),
                 dim3(kQdThreads), qdecode_smem(false, batch), stream, a);
  if (e != cudaSuccess) return e;
  const long long rows = units * G;
  const long long room = 32LL * device_sm_count();
  auto merge = [&](auto *kern, int w) {
    const int per = kMergeWarps / w;
    return launch_pdl(kern, dim3((unsigned)((rows + per - 1) / per)),
                      dim3(32 * kMergeWarps), 0, stream, a, shared_o,
                      shared_ml, shared);
  };
  if (rows * 8 <= 2 * room) return merge(merge_kernel<8>, 8);
  if (rows * 4 <= 2 * room) return merge(merge_kernel<4>, 4);
  if (rows * 2 <= 2 * room) return merge(merge_kernel<2>, 2);
  return merge(merge_kernel<1>, 1);
}

}  // namespace locks
