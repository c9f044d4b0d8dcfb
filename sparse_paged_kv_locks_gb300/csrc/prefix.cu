// Attention of a batch's queries over pages that all its sequences share,
// read once for all: per KV head, the batch * G query rows against the prefix
// (the mathematics and the partials are those of the single-token kernel,
// qdecode.cu; the sequences' own pages and the merge are its work).
//
// A CTA takes 128 query rows of a KV head and a range of 128-token tiles.
// Both products are tcgen05 matrix products with fp32 accumulators in tensor
// memory: S = Q K^T from shared memory, O += W V with the weights W in fp16
// in tensor memory over the scores they came from.  Codes are exact in fp16;
// a page's rows are scaled there by 2^(e - E), E the largest exponent of the
// page, which is exact for rows within 2^15 of the page's largest (and below
// that off by 2^-25 of the page's largest code).  2^E of the keys multiplies
// a page's scores, E of the values joins the weights' exponent.
//
// Eight warps: 0-3 softmax, a query row to a thread, so that maxima and sums
// need no exchange; 4-7 bring records from memory and lay the fp16 tiles out
// for the tensor core, and one thread of theirs issues the products.  K and
// V have one tile buffer each: the values of tile j and the keys of j + 1 are
// laid out while the softmax of tile j runs.  Two CTAs fit an SM, and one's
// softmax runs under the other's products.
#include "launch.h"
#include "quantised.cuh"

namespace locks {

constexpr int kPfRows = 128;   // query rows of a CTA
constexpr int kPfTile = 128;   // tokens of a tile
constexpr int kPfPages = kPfTile / kPage;
constexpr int kPfThreads = 256;
constexpr int kPfOperand = kPfRows * kDim * 2;  // an fp16 tile, 32 KB
constexpr int kPfBlock = kPfOperand / 2;        // its half of 64 dims
constexpr int kPfSmem = 3 * kPfOperand + 1024;
constexpr int kPfColumns = 256;                 // tensor memory: S, O
constexpr int kPfColO = 128;
constexpr float kPfScale = 0.12751743074602467f;  // log2(e) / sqrt(128)
constexpr float kPfLift = 8.f;   // as in the single-token kernel
constexpr float kPfSlack = 7.f;
constexpr uint32_t kPfSpin = 1u << 21;  // tries before a wait gives up

// ---------------------------------------------------------------------------
// tcgen05
// ---------------------------------------------------------------------------
// Shared-memory matrix descriptor: 128-byte swizzle, 8-row groups 1024 bytes
// apart.  For keys and queries a row is a token and K runs along it; for
// values N runs along the row, and `lead` is the distance of the two blocks
// of 64 dims.
__device__ __forceinline__ uint64_t mat_desc(uint32_t addr, uint32_t lead) {
  return (uint64_t)((addr & 0x3FFFFu) >> 4) | (uint64_t)(lead >> 4) << 16 |
         (uint64_t)(1024u >> 4) << 32 | (uint64_t)1 << 46 | (uint64_t)2 << 61;
}
// fp16 x fp16 -> fp32, M = N = 128; bit 16: B runs along N
constexpr uint32_t kPfDescS =
    1u << 4 | (128u >> 3) << 17 | (128u >> 4) << 24;
constexpr uint32_t kPfDescO = kPfDescS | 1u << 16;

__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b,
                                       uint32_t desc, bool add) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.u32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
      "l"(a), "l"(b), "r"(desc), "r"((uint32_t)add)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b,
                                       uint32_t desc, bool add) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.u32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(
          d),
      "r"(a), "l"(b), "r"(desc), "r"((uint32_t)add)
      : "memory");
}
// the barrier completes when this thread's products so far have
__device__ __forceinline__ void mma_commit(uint64_t *bar) {
  asm volatile(
      "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 "
      "[%0];\n" ::"r"(smem_u32(bar))
      : "memory");
}
__device__ __forceinline__ void tm_fence_before() {
  asm volatile("tcgen05.fence::before_thread_sync;\n" ::: "memory");
}
__device__ __forceinline__ void tm_fence_after() {
  asm volatile("tcgen05.fence::after_thread_sync;\n" ::: "memory");
}
__device__ __forceinline__ void tm_wait_ld() {
  asm volatile("tcgen05.wait::ld.sync.aligned;\n" ::: "memory");
}
__device__ __forceinline__ void tm_wait_st() {
  asm volatile("tcgen05.wait::st.sync.aligned;\n" ::: "memory");
}
// 32 columns of this warp's 32 lanes
__device__ __forceinline__ void tm_ld32(uint32_t (&r)[32], uint32_t addr) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,"
      "%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]),
        "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]),
        "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]),
        "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]),
        "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]),
        "=r"(r[30]), "=r"(r[31])
      : "r"(addr)
      : "memory");
}
__device__ __forceinline__ void tm_st32(uint32_t addr,
                                        const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
      "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};\n" ::"r"(addr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]),
      "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]),
      "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]),
      "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]),
      "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]),
      "r"(r[30]), "r"(r[31])
      : "memory");
}
// 16 columns
__device__ __forceinline__ void tm_st16(uint32_t addr,
                                        const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};\n" ::"r"(
          addr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]),
      "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]),
      "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
// shared-memory writes of this thread, seen by the tensor core
__device__ __forceinline__ void fence_to_async() {
  asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory");
}
__device__ __forceinline__ void mbar_arrive(uint64_t *bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];\n" ::"r"(
                   smem_u32(bar))
               : "memory");
}
__device__ __forceinline__ void st_shared_v4(uint32_t a, uint4 v) {
  asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};\n" ::"r"(a), "r"(v.x),
               "r"(v.y), "r"(v.z), "r"(v.w)
               : "memory");
}

// byte offset of 16-byte chunk c (0..15, 8 fp16 each) of row r in a tile:
// two blocks of 64 dims, rows of 128 bytes, chunks swizzled by the row
__device__ __forceinline__ uint32_t tile_at(int r, int c) {
  return (uint32_t)((c >> 3) * kPfBlock + r * 128 +
                    (((c & 7) ^ (r & 7)) << 4));
}

struct PfArgs {
  const __nv_bfloat16 *q;
  const uint8_t *records;
  int64_t num_phys;
  const int32_t *table;   // [pages]
  int pages, batch, h_kv, G, row_tiles, splits;
  float *o_part;          // [split][batch * h_q][128], sums not divided
  float2 *ml_part;        // [split][batch * h_q] (m, sum of weights)
  int32_t *status;
};

struct PfShared {
  uint64_t k_full, v_full, p_full, qk_done, pv_done, drain;
  uint32_t tmem;
  int dead;
  // per tile parity and page: 2^E of the keys, E and 2^-E of the values,
  // and which pages are there
  float k_scale[2][kPfPages], v_exp[2][kPfPages], v_inv[2][kPfPages];
  uint32_t there[2];
};

// false when the wait gave up, or some other thread's did
__device__ __forceinline__ bool pf_wait(PfShared &sh, uint64_t *bar,
                                        uint32_t phase) {
  for (uint32_t i = 0; i < kPfSpin; ++i) {
    if (mbar_try_wait(bar, phase)) return true;
    if ((i & 255u) == 255u && *(volatile int *)&sh.dead) return false;
  }
  *(volatile int *)&sh.dead = 1;
  return false;
}

__global__ void __launch_bounds__(kPfThreads, 2)
    prefix_kernel(const PfArgs a) {
  extern __shared__ uint8_t raw_smem[];
  __shared__ PfShared sh;
  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
  // swizzled tiles start at multiples of 1024 bytes
  const uint32_t q_s = (smem_u32(raw_smem) + 1023u) & ~1023u;
  const uint32_t k_s = q_s + kPfOperand, v_s = k_s + kPfOperand;

  // this CTA's KV head, query rows and tiles
  const int tiles = (a.pages + kPfPages - 1) / kPfPages;
  const int rt = blockIdx.x % a.row_tiles;
  const int rest = blockIdx.x / a.row_tiles;
  const int h = rest % a.h_kv, split = rest / a.h_kv;
  const int t0 = (int)((long long)split * tiles / a.splits);
  const int t1 = (int)((long long)(split + 1) * tiles / a.splits);
  const int n = t1 - t0;
  const int rows = a.batch * a.G;
  const int row = rt * kPfRows + tid;  // softmax warps

  if (wid == 4) {
    asm volatile(
        "tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;\n"
        " tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;\n" ::"r"(
            smem_u32(&sh.tmem)),
        "r"(kPfColumns)
        : "memory");
    if (lane == 0) {
      mbar_init(&sh.k_full, 4);
      mbar_init(&sh.v_full, 4);
      mbar_init(&sh.p_full, 4);
      mbar_init(&sh.qk_done, 1);
      mbar_init(&sh.pv_done, 1);
      mbar_init(&sh.drain, 1);
      sh.dead = 0;
      fence_mbar_init();
    }
  }
  pdl_wait();
  pdl_trigger();

  // the query rows, fp16, each scaled so that its largest magnitude lies in
  // [2^7, 2^8)
  float f = 0.f;
  if (wid < 4) {
    uint32_t w[64];
    if (row < rows) {
      const uint4 *src = reinterpret_cast<const uint4 *>(
          a.q + ((size_t)(row / a.G) * a.h_kv * a.G + (size_t)h * a.G +
                 row % a.G) * kDim);
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const uint4 v = __ldg(src + i);
        w[4 * i] = v.x;
        w[4 * i + 1] = v.y;
        w[4 * i + 2] = v.z;
        w[4 * i + 3] = v.w;
      }
    } else {
#pragma unroll
      for (int i = 0; i < 64; ++i) w[i] = 0u;
    }
    float top = 0.f;
#pragma unroll
    for (int i = 0; i < 64; ++i)
      top = fmaxf(top, fmaxf(fabsf(bf16_lo(w[i])), fabsf(bf16_hi(w[i]))));
    const int e = max(-100, (int)(__float_as_uint(top) >> 23) - 127) - 7;
    const float down = exp2_int(-e);
    f = exp2_int(e) * kPfScale;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      uint32_t x[4];
#pragma unroll
      for (int j = 0; j < 4; ++j)
        x[j] = h2_as_u32(__floats2half2_rn(bf16_lo(w[4 * i + j]) * down,
                                           bf16_hi(w[4 * i + j]) * down));
      st_shared_v4(q_s + tile_at(tid, i), make_uint4(x[0], x[1], x[2], x[3]));
    }
    fence_to_async();
  }
  tm_fence_before();
  __syncthreads();
  tm_fence_after();
  const uint32_t tm = sh.tmem;

  if (wid < 4) {
    // ------------------------------------------------------------- softmax
    const uint32_t mine = tm + ((uint32_t)(wid * 32) << 16);
    float m = -INFINITY, l = 0.f;
    bool ok = true;
    for (int j = 0; j < n && ok; ++j) {
      ok = pf_wait(sh, &sh.qk_done, j & 1);
      // all products before S(j), among them O(j - 1), are done
      if (ok && j > 0) ok = pf_wait(sh, &sh.pv_done, (j - 1) & 1);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      tm_fence_after();
      const int par = j & 1;
      const uint32_t there = sh.there[par];
      // largest score plus value exponent of the row
      float top = -INFINITY;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        uint32_t s[32];
        tm_ld32(s, mine + 32 * c);
        tm_wait_ld();
#pragma unroll
        for (int p = 0; p < 2; ++p) {
          float x = __uint_as_float(s[16 * p]);
#pragma unroll
          for (int i = 1; i < 16; ++i)
            x = fmaxf(x, __uint_as_float(s[16 * p + i]));
          const int pg = 2 * c + p;
          if (there >> pg & 1)
            top = fmaxf(top, fmaf(x, f * sh.k_scale[par][pg],
                                  sh.v_exp[par][pg]));
        }
      }
      const bool raise = top > m + kPfSlack;
      if (__any_sync(0xffffffffu, raise)) {
        const float to = raise ? top : m;
        const float fall = to == m ? 1.f : ex2_fast(m - to);
        m = to;
        l *= fall;
        if (j > 0) {
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            uint32_t o[32];
            tm_ld32(o, mine + kPfColO + 32 * c);
            tm_wait_ld();
#pragma unroll
            for (int i = 0; i < 32; ++i)
              o[i] = __float_as_uint(__uint_as_float(o[i]) * fall);
            tm_st32(mine + kPfColO + 32 * c, o);
          }
        }
      }
      // weights, over the scores they come from
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        uint32_t s[32], w[16];
        tm_ld32(s, mine + 32 * c);
        tm_wait_ld();
#pragma unroll
        for (int p = 0; p < 2; ++p) {
          const int pg = 2 * c + p;
          if (there >> pg & 1) {
            const float mul = f * sh.k_scale[par][pg];
            const float add = sh.v_exp[par][pg] - (m - kPfLift);
            float sum = 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const float x = ex2_fast(
                  fmaf(__uint_as_float(s[16 * p + 2 * i]), mul, add));
              const float y = ex2_fast(
                  fmaf(__uint_as_float(s[16 * p + 2 * i + 1]), mul, add));
              sum += x + y;
              w[8 * p + i] = h2_as_u32(__floats2half2_rn(x, y));
            }
            l = fmaf(sum, sh.v_inv[par][pg], l);
          } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) w[8 * p + i] = 0u;
          }
        }
        tm_st16(mine + 16 * c, w);
      }
      tm_wait_st();
      tm_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.p_full);
    }
    if (ok) ok = pf_wait(sh, &sh.pv_done, (n - 1) & 1);
    ok = __all_sync(0xffffffffu, ok);
    tm_fence_after();
    const size_t all = (size_t)rows * a.h_kv;
    const size_t at = (size_t)split * all +
                      (size_t)(row / a.G) * a.h_kv * a.G + (size_t)h * a.G +
                      row % a.G;
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      uint32_t o[32];
      tm_ld32(o, mine + kPfColO + 32 * c);
      tm_wait_ld();
      if (row < rows && ok) {
        float4 *dst =
            reinterpret_cast<float4 *>(a.o_part + at * kDim) + 8 * c;
#pragma unroll
        for (int i = 0; i < 8; ++i)
          dst[i] = make_float4(
              __uint_as_float(o[4 * i]), __uint_as_float(o[4 * i + 1]),
              __uint_as_float(o[4 * i + 2]), __uint_as_float(o[4 * i + 3]));
      }
    }
    if (row < rows) a.ml_part[at] = make_float2(m, ok ? l : 0.f);
  } else {
    // --------------------------------------------- fp16 operands, products
    // thread i moves the 16-byte group i of every page's key or value codes:
    // slot s, dims 16 c .. 16 c + 15
    const int i = tid - 128, s = i >> 3, warp = wid - 4;
    const int c = q_group(i & 7, s);
    uint4 kraw[kPfPages], vraw[kPfPages];
    uint4 ksc, vsc, vsc_next;  // scale bytes of page lane & 7
    bool there = false;
    auto page = [&](int t) -> int {  // page lane & 7 of tile t
      const int pg = t * kPfPages + (lane & 7);
      if (t >= t1 || pg >= a.pages) return -1;
      const int ph = __ldg(a.table + pg);
      if (ph >= 0 && ph < a.num_phys) return ph;
      set_status(a.status, LOCKS_DEV_BAD_PAGE_ID);
      return -1;
    };
    auto load = [&](int ph, int off, uint4 (&raw)[kPfPages]) {
#pragma unroll
      for (int p = 0; p < kPfPages; ++p) {
        const int php = __shfl_sync(0xffffffffu, ph, p);
        raw[p] = make_uint4(0u, 0u, 0u, 0u);
        if (php >= 0)
          raw[p] = __ldg(reinterpret_cast<const uint4 *>(
              a.records + ((size_t)php * a.h_kv + h) * kQRec + off + 16 * i));
      }
    };
    auto load_scales = [&](int ph, uint4 &ks, uint4 &vs) {
      ks = vs = make_uint4(0x7f7f7f7fu, 0x7f7f7f7fu, 0x7f7f7f7fu, 0x7f7f7f7fu);
      if (ph >= 0) {
        const uint4 *sc = reinterpret_cast<const uint4 *>(
            a.records + ((size_t)ph * a.h_kv + h) * kQRec + kQOffKE);
        ks = __ldg(sc);
        vs = __ldg(sc + 1);
      }
    };
    auto top_byte = [&](uint4 x) -> uint32_t {
      uint32_t b = __vmaxu4(__vmaxu4(x.x, x.y), __vmaxu4(x.z, x.w));
      b = __vmaxu4(b, b >> 16);
      return max(b & 0xffu, b >> 8 & 0xffu);
    };
    auto store = [&](const uint4 (&raw)[kPfPages], uint4 sc, uint32_t ref,
                     uint32_t base) {
      // the scale bytes of slots 4 warp .. 4 warp + 3
      const uint32_t four = warp == 0 ? sc.x : warp == 1 ? sc.y
                            : warp == 2 ? sc.z : sc.w;
#pragma unroll
      for (int p = 0; p < kPfPages; ++p) {
        const uint32_t er = __shfl_sync(0xffffffffu, ref, p);
        const uint32_t e =
            __shfl_sync(0xffffffffu, four, p) >> (8 * (lane >> 3)) & 0xffu;
        // 2^(e - E): exact down to 2^-24, zero below
        const __half2 x =
            __float2half2_rn(exp2_int(max(-126, (int)e - (int)er)));
        const uint32_t w[4] = {raw[p].x, raw[p].y, raw[p].z, raw[p].w};
        uint32_t y[8];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          y[2 * k] = h2_as_u32(__hmul2(u32_as_h2(e4m3x2_lo(w[k])), x));
          y[2 * k + 1] = h2_as_u32(__hmul2(u32_as_h2(e4m3x2_hi(w[k])), x));
        }
        const int r = p * kPage + s;
        st_shared_v4(base + tile_at(r, 2 * c),
                     make_uint4(y[0], y[1], y[2], y[3]));
        st_shared_v4(base + tile_at(r, 2 * c + 1),
                     make_uint4(y[4], y[5], y[6], y[7]));
      }
    };
    const bool issuer = warp == 0 && lane == 0;
    // keys of tile j from kraw, with the tile's scale references
    auto store_keys = [&](int j) {
      const uint32_t kref = top_byte(ksc), vref = top_byte(vsc_next);
      store(kraw, ksc, kref, k_s);
      const uint32_t mask = __ballot_sync(0xffffffffu, there) & 0xffu;
      if (warp == 0) {
        const int par = j & 1;
        if (lane < kPfPages) {
          sh.k_scale[par][lane] = exp2_int((int)kref - 127);
          sh.v_exp[par][lane] = (float)((int)vref - 127);
          sh.v_inv[par][lane] = exp2_int(127 - (int)vref);
        }
        if (lane == 0) sh.there[par] = mask;
      }
      fence_to_async();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.k_full);
    };
    int ph = page(t0);
    load(ph, 0, kraw);
    load(ph, kQOffV, vraw);
    load_scales(ph, ksc, vsc_next);
    there = ph >= 0;
    store_keys(0);
    bool ok = true;
    for (int j = 0; j < n; ++j) {
      if (issuer) {
        ok = pf_wait(sh, &sh.k_full, j & 1);
        if (ok) {
          tm_fence_after();
#pragma unroll
          for (int kk = 0; kk < 8; ++kk) {
            const uint32_t off = (kk >> 2) * kPfBlock + (kk & 3) * 32;
            mma_ss(tm, mat_desc(q_s + off, 16), mat_desc(k_s + off, 16),
                   kPfDescS, kk > 0);
          }
          mma_commit(&sh.qk_done);
        }
      }
      if (!__shfl_sync(0xffffffffu, ok, 0)) break;
      vsc = vsc_next;
      const uint32_t vref = top_byte(vsc);
      ph = page(t0 + j + 1);
      load(ph, 0, kraw);
      load_scales(ph, ksc, vsc_next);
      there = ph >= 0;
      ok = j == 0 || pf_wait(sh, &sh.pv_done, (j - 1) & 1);
      if (!__all_sync(0xffffffffu, ok)) break;
      store(vraw, vsc, vref, v_s);
      fence_to_async();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.v_full);
      load(ph, kQOffV, vraw);
      if (j + 1 < n) {
        ok = pf_wait(sh, &sh.qk_done, j & 1);
        if (!__all_sync(0xffffffffu, ok)) break;
        store_keys(j + 1);
      }
      if (issuer) {
        ok = pf_wait(sh, &sh.v_full, j & 1) && pf_wait(sh, &sh.p_full, j & 1);
        if (ok) {
          tm_fence_after();
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)
            mma_ts(tm + kPfColO, tm + 8 * kk,
                   mat_desc(v_s + kk * kPage * 128, kPfBlock), kPfDescO,
                   j > 0 || kk > 0);
          mma_commit(&sh.pv_done);
        }
      }
      if (!__shfl_sync(0xffffffffu, ok, 0)) break;
    }
    if (issuer && *(volatile int *)&sh.dead) {
      // give what was issued a last, bounded chance to finish
      set_status(a.status, LOCKS_DEV_TIMEOUT);
      mma_commit(&sh.drain);
      for (uint32_t i2 = 0; i2 < kPfSpin; ++i2)
        if (mbar_try_wait(&sh.drain, 0)) break;
    }
  }
  __syncwarp();
  tm_fence_before();
  __syncthreads();
  if (wid == 4)
    asm volatile(
        "tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;\n" ::"r"(tm),
        "r"(kPfColumns)
        : "memory");
}

// ---------------------------------------------------------------------------
// launcher
// ---------------------------------------------------------------------------
// How many ranges the prefix's tiles are cut into: enough CTAs for two to an
// SM, and no more waves of them than pay.  A tile costs a CTA about 1.2 us,
// its start and end 4 us, a split of one row 1 KB of traffic.  A rule on
// sizes alone (152 SMs), so that the workspace's size needs no GPU.
int prefix_splits(int batch, int h_kv, int G, int pages) {
  const long long slots = 304;
  const long long row_tiles =
      ((long long)batch * G + kPfRows - 1) / kPfRows;
  const long long base = row_tiles * h_kv;
  const long long tiles = (pages + kPfPages - 1) / kPfPages;
  double best = 1e30;
  int splits = 1;
  for (long long s = 1; s <= tiles && s <= 64; ++s) {
    const double waves = (double)((base * s + slots - 1) / slots);
    const double us = waves * (1.2 * (double)((tiles + s - 1) / s) + 4.0) +
                      1.6e-4 * (double)(s * batch * h_kv * G);
    if (us < best * 0.999) {
      best = us;
      splits = (int)s;
    }
  }
  return splits;
}

cudaError_t launch_prefix(const void *q, const void *records,
                          int64_t num_phys, const int32_t *table, int pages,
                          int batch, int h_kv, int G, int splits,
                          float *o_part, float2 *ml_part, int32_t *status,
                          cudaStream_t stream) {
  static DeviceFlags done;
  cudaError_t e = once_per_device(done, [] {
    return cudaFuncSetAttribute(prefix_kernel,
                                cudaFuncAttributeMaxDynamicSharedMemorySize,
                                kPfSmem);
  });
  if (e != cudaSuccess) return e;
  const int row_tiles = (int)(((long long)batch * G + kPfRows - 1) / kPfRows);
  const PfArgs a{static_cast<const __nv_bfloat16 *>(q),
                 static_cast<const uint8_t *>(records),
                 num_phys, table, pages, batch, h_kv, G, row_tiles, splits,
                 o_part, ml_part, status};
  return launch_pdl(prefix_kernel,
                    dim3((unsigned)((long long)row_tiles * h_kv * splits)),
                    dim3(kPfThreads), kPfSmem, stream, a);
}

}  // namespace locks
