// Attention of a batch's queries over pages that all its sequences share,
// read once for all: per KV head, the batch * G query rows against the prefix
// (the mathematics and the partials are those of the single-token kernel,
// qdecode.cu; the sequences' own pages and the merge are its work).
//
// A CTA takes one or two tiles of 128 query rows of a KV head and a range of
// 128-token tiles.  Both products are tcgen05 matrix products with fp32
// accumulators in tensor memory: S = Q K^T, O += W V with the weights W in
// fp16 in tensor memory over the scores they came from.
//
// Keys take part as they are stored: the e4m3 rows are copied to shared
// memory, and the query row is the sum of two rows of codes, hi in e4m3 and lo
// in e5m2, after a power-of-two scale that puts its largest magnitude in (224,
// 448].  A bf16 number has 8 significant bits, hi 4, lo 3: hi is the nearest
// code, lo the rest, at most 8 of the last places (9 to 15 would need 4 bits).
// So hi + lo is exact from 2^-6 on, 2^-13 of the row's largest element; below,
// hi's step is 2^-9 and lo, whose own goes down to 2^-16, is off by at most
// 2^-14, 2^-21 of the row's largest element.  A row with an outlier, 64 times its
// mean and more, whose other elements would be there, is scaled to [2^11,
// 2^12): beyond 448 lo is the nearest code and hi the rest, at most 16 places and 256,
// and the others lose 2^-25 of the largest, less than fp32 products with it do.
//
// A key's scale multiplies its column of scores.  Value codes are widened to
// fp16, scaled by 2^(e - E), E the largest exponent so far, in whose unit the
// sums are: exact, since a tile with rows more than 2^8 below E takes another
// form (far_tile: codes and weights in bf16, the weights as hi + lo).
//
// Rows of a record are swizzled by f(s) = (s & 6) ^ 5 (s & 1), rows of the
// tensor core's operand by s & 7.  The two agree on even rows; an odd row's
// halves trade places in shared memory before its product.
//
// Four warps per row tile do its softmax, a query row to a thread, so that
// maxima and sums need no exchange; one warp issues the products; one has the
// keys copied and mends them; two have the values (with all scales) copied,
// and widen them, four pages of a tile each.  With one row tile two CTAs fit an
// SM, with their columns of tensor memory fill it, and one's softmax runs under
// the other's products; a buffer's next copy starts when it has been read.
// With two row tiles a CTA has an SM to itself, two buffers of everything, and
// its keys and values serve both tiles, whose softmax and products take turns.
//
// Bound: for many rows, the chain scores -> softmax -> weights -> products of
// a tile: some 2,150 cycles of softmax and as many from its weights to its next
// scores, in which the tensor core is busy with both row tiles for about 2,650
// of 4,300.  The product of keys and query reads shared memory at 122 bytes a
// cycle of 128 and runs at 70% of its rate.  A 128K prefix for 64 sequences and
// 64 query heads takes 270 us in this form (300 with one row tile to a CTA);
// with half of that product left out 24 us less, of the other 18, without the
// exponentials 18, without the loads of key scales 19; without the stores of
// widened values or of mended keys the same.  For few rows, the start and end
// of a CTA and the bytes of the records.
//
// What was slower on that prefix, with two row tiles: the products of a tile's
// first half under the softmax of its second (307 us), the second half's
// scores loaded under the first half's exponentials (285 us), key scales in
// bf16 (283 us); three buffers of keys took as long as two.  With one row tile
// (then 303 us): loads to registers instead of bulk copies (the pages lie far
// apart, and the proxy fence before a product waits for its thread's loads;
// 610 us), copies of single rows to their swizzled places (850 us), three warps
// that each do a third of everything (348 us), tiles of 64 tokens with two or
// three buffers of everything (335 us: a product then reads the query from
// shared memory for half as many columns), two threads to a row in eight
// softmax warps of 96 registers (347 us), the scores of the next tile's first
// half under the softmax of this one's second (323 us).
#include "launch.h"
#include "quantised.cuh"

namespace locks {

constexpr int kPfRows = 128;   // query rows of a row tile
constexpr int kPfTile = 128;   // tokens of a tile
constexpr int kPfPages = kPfTile / kPage;
constexpr int kPfWiden = 2;    // warps that widen values
constexpr int kPfOwn = kPfPages / kPfWiden;  // pages of each of them
constexpr int kPfQuery = kPfRows * kDim;    // hi or lo of the query, 16 KB
constexpr int kPfCodes = kPfTile * kDim;    // a tile of e4m3 keys, 16 KB
constexpr int kPfBlock = kPfTile * 128;     // 64 dims of fp16 values, 16 KB
constexpr int kPfRest = kQRec - kQOffV;     // values and scales of a record
constexpr int kPfRaw = kPfPages * kPfRest;  // a tile of them
// per row tile of a CTA: its query, and one more buffer of all the rest
constexpr int kPfPart = 2 * kPfQuery + kPfCodes + 2 * kPfBlock + kPfRaw;
constexpr int kPfColumns = 256;             // tensor memory: S, then O
constexpr int kPfColO = kPfTile;
template <int R>
constexpr int kPfThreads = 32 * (4 * R + 2 + kPfWiden);
template <int R>
constexpr int kPfSmem = R * kPfPart + 1024;
// fewest (sequence, KV head, page) triples that are worth the kernel
constexpr long long kPfMinShared = 12288;
// A tile with value rows more than 2^kQSpread below the largest scale so far
// takes its weights and values in bf16 (far_tile).  Twice the time, for tiles
// after an outlier's alone: with an infinity in its first page a 128K prefix for
// 64 sequences takes 502-508 us instead of 270 (the range that holds it is the
// last to end), one of 32K for 32 47 us either way.

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
// fp32 accumulators, operands of format 0 (e4m3 of kind::f8f6f4, fp16 of
// kind::f16), M = 128, N = a tile's tokens or the dims; bit 16: B runs along N
constexpr uint32_t kPfDescS =
    1u << 4 | ((uint32_t)kPfTile >> 3) << 17 | (128u >> 4) << 24;
// .. A in e5m2, the query's lo
constexpr uint32_t kPfDescLo = kPfDescS | 1u << 7;
constexpr uint32_t kPfDescO =
    1u << 4 | 1u << 16 | ((uint32_t)kDim >> 3) << 17 | (128u >> 4) << 24;
// .. both operands bf16
constexpr uint32_t kPfDescFar = kPfDescO | 1u << 7 | 1u << 10;

__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b,
                                       uint32_t desc, bool add) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.u32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
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
// 32 columns of 16 lanes, as matrix fragments
__device__ __forceinline__ void tm_ld16x256(uint32_t (&r)[16],
                                            uint32_t addr) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]),
        "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]),
        "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]),
        "=r"(r[15])
      : "r"(addr)
      : "memory");
}
// 16 columns
__device__ __forceinline__ void tm_ld16(uint32_t (&r)[16], uint32_t addr) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]),
        "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]),
        "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]),
        "=r"(r[15])
      : "r"(addr)
      : "memory");
}
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

// two numbers -> two e5m2 codes (low byte: lo), as e4m3x2_from
__device__ __forceinline__ uint32_t e5m2x2_from(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e5m2x2.f32 %0, %1, %2;\n"
      : "=h"(r)
      : "f"(hi), "f"(lo));
  return r;
}

// .. and back: an e5m2 code is the high byte of the fp16 number
__device__ __forceinline__ float2 e5m2x2_to(uint32_t codes) {
  return __half22float2(u32_as_h2(__byte_perm(codes, 0u, 0x1404)));
}

// two fp32 numbers in one 64-bit register pair
__device__ __forceinline__ uint64_t pack2(uint32_t lo, uint32_t hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};\n" : "=l"(r) : "r"(lo), "r"(hi));
  return r;
}
__device__ __forceinline__ uint64_t pack2(float lo, float hi) {
  return pack2(__float_as_uint(lo), __float_as_uint(hi));
}
__device__ __forceinline__ float2 unpack2(uint64_t x) {
  uint32_t lo, hi;
  asm("mov.b64 {%0, %1}, %2;\n" : "=r"(lo), "=r"(hi) : "l"(x));
  return make_float2(__uint_as_float(lo), __uint_as_float(hi));
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;\n" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;\n" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;\n" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;\n" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
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

template <int R>
struct PfShared {
  // of tile j, at j & 1: scales of the keys, the largest value scale so far,
  // which pages are there (a widening warp's each)
  float k_scale[2][kPfTile];
  uint32_t v_top[2], there[2][kPfWiden];
  // whether the tile is a far one, then the scales of its values by token; the
  // widening warps' largest and least of them
  alignas(16) uint8_t v_token[2][kPfTile];
  int far[2];
  uint2 range[2][kPfWiden];
  uint32_t tmem;
  int dead;
  uint64_t q_full[R], qk_done[R], p_full[R], o_done[R];      // of a row tile
  uint64_t k_raw[R], k_full[R], k_free[R];                   // of a buffer
  uint64_t v_raw[kPfWiden][R], v_full[R], v_free[R];
  uint64_t info[2], ranges[2], drain;
};

// one lane of the warp, for what a warp does once
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile(
      "{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n"
      " selp.b32 %0, 1, 0, p;\n}\n"
      : "=r"(r));
  return r != 0;
}

// false when the wait gave up, or some other thread's did
template <int R>
__device__ __forceinline__ bool pf_wait(PfShared<R> &sh, uint64_t *bar,
                                        uint32_t phase) {
  if (mbar_try_wait(bar, phase)) return true;
  const long long t0 = clock64();
  while (!*(volatile int *)&sh.dead) {
    if (mbar_try_wait(bar, phase)) return true;
    if (clock64() - t0 > kQWaitCycles) {
      *(volatile int *)&sh.dead = 1;
      break;
    }
  }
  return false;
}

// tile j's use of a ring of R
template <int R>
__device__ __forceinline__ bool pf_wait_ring(PfShared<R> &sh,
                                             uint64_t (&bars)[R], int j) {
  return pf_wait(sh, bars + j % R, j / R & 1);
}

template <int R>
__global__ void __launch_bounds__(kPfThreads<R>, 3 - R)
    prefix_kernel(const PfArgs a) {
  extern __shared__ uint8_t raw_smem[];
  __shared__ PfShared<R> sh;
  // the same for all of a warp, and known to be: products and copies take
  // their operands from uniform registers
  const int tid = threadIdx.x, lane = tid & 31;
  const int wid = __shfl_sync(0xffffffffu, tid >> 5, 0);
  // swizzled tiles start at multiples of 1024 bytes
  const uint32_t q_s = (smem_u32(raw_smem) + 1023u) & ~1023u;
  const uint32_t k_s = q_s + R * 2 * kPfQuery;
  const uint32_t v_s = k_s + R * kPfCodes;
  const uint32_t raw_s = v_s + R * 2 * kPfBlock;  // [buffer][page][kPfRest]
  constexpr int kProducts = 4 * R, kKeys = kProducts + 1;  // warps

  // this CTA's KV head, row tiles and tiles
  const int tiles = (a.pages + kPfPages - 1) / kPfPages;
  const int rts = (a.row_tiles + R - 1) / R;
  const int rt = blockIdx.x % rts * R;
  const int rest = blockIdx.x / rts;
  const int h = rest % a.h_kv, split = rest / a.h_kv;
  const int t0 = (int)((long long)split * tiles / a.splits);
  const int t1 = (int)((long long)(split + 1) * tiles / a.splits);
  const int n = t1 - t0;
  const int nt = min(R, a.row_tiles - rt);
  const int rows = a.batch * a.G;

  if (wid == kProducts && lane == 0) {
    for (int i = 0; i < R; ++i) {
      mbar_init(sh.q_full + i, 4);
      mbar_init(sh.qk_done + i, 1);
      mbar_init(sh.p_full + i, 4);
      mbar_init(sh.o_done + i, 1);
      mbar_init(sh.k_raw + i, 1);
      mbar_init(sh.k_full + i, 1);
      mbar_init(sh.k_free + i, 1);
      for (int w = 0; w < kPfWiden; ++w) mbar_init(sh.v_raw[w] + i, 1);
      mbar_init(sh.v_full + i, kPfWiden);
      mbar_init(sh.v_free + i, 1);
    }
    mbar_init(sh.info, kPfWiden);
    mbar_init(sh.info + 1, kPfWiden);
    mbar_init(sh.ranges, kPfWiden);
    mbar_init(sh.ranges + 1, kPfWiden);
    mbar_init(&sh.drain, 1);
    sh.dead = 0;
    fence_mbar_init();
  }
  __syncwarp();
  // Tensor memory is taken after the kernels before this one have ended: a
  // kernel that let this one start early and then takes its own, on an SM that
  // both fit, would wait for columns that are held here until it has ended.
  pdl_wait();
  if (wid == kProducts)
    asm volatile(
        "tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;\n"
        " tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;\n" ::"r"(
            smem_u32(&sh.tmem)),
        "r"(R * kPfColumns)
        : "memory");
  tm_fence_before();
  __syncthreads();
  tm_fence_after();
  const uint32_t tm = sh.tmem;
  // after the wait, never before: the kernel of the sequences' own pages starts
  // here and does not wait for the kernels before this one by itself
  pdl_trigger();

  const int tile = wid >> 2;  // row tile of a softmax warp
  if (wid < kProducts && tile >= nt) {
    // no rows
  } else if (wid < kProducts) {
    const int row = rt * kPfRows + tid;
    // the query rows: hi and lo codes, the scale that they leave to scores
    const uint4 *src = reinterpret_cast<const uint4 *>(
        a.q + ((size_t)(row / a.G) * a.h_kv * a.G + (size_t)h * a.G +
               row % a.G) * kDim);
    const bool in = row < rows;
    // The largest magnitude and, roughly, the sum of all.  (Loops of the start
    // and of rare paths are kept short: unrolled, their instructions come from
    // far, 1 us of 15 for 8 sequences and 256 pages.)
    const __nv_bfloat162 none = __floats2bfloat162_rn(0.f, 0.f);
    __nv_bfloat162 most[2] = {none, none}, sums[4] = {none, none, none, none};
#pragma unroll 8
    for (int i = 0; i < 16; ++i) {
      const uint4 v = in ? __ldg(src + i) : make_uint4(0u, 0u, 0u, 0u);
      const uint32_t x[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const uint32_t size = x[k] & 0x7fff7fffu;
        const __nv_bfloat162 a =
            *reinterpret_cast<const __nv_bfloat162 *>(&size);
        most[k & 1] = __hmax2(most[k & 1], a);
        sums[k] = __hadd2(sums[k], a);
      }
    }
    const float2 m0 = __bfloat1622float2(__hmax2(most[0], most[1]));
    const float top = fmaxf(m0.x, m0.y);
    float sum = 0.f;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float2 t = __bfloat1622float2(sums[k]);
      sum += t.x + t.y;
    }
    // largest magnitude to (224, 448], with an outlier to [2^11, 2^12)
    const bool outlier = top + top > sum;
    const uint32_t tb = __float_as_uint(top);
    const int less = outlier ? 11 : 8 - ((tb & 0x7fffffu) > 0x600000u);
    const int e = max(-100, (int)(tb >> 23) - 127 - less);
    const float down = exp2_int(-e);
    // codes have no infinity: a row that holds one has scores that are not
    // numbers
    const float f = isinf(top) ? top - top : exp2_int(e) * kQScale;
    // what lo has to take first of a number beyond hi's largest: its nearest
    // number of 3 bits
    auto beyond = [](float a) -> float {
      const uint32_t near = __float_as_uint(a) + 0x100000u;
      return fabsf(a) > 448.f ? __uint_as_float(near & 0xffe00000u) : 0.f;
    };
    auto codes = [&](auto first) {
#pragma unroll 2
      for (int i = 0; i < 8; ++i) {  // 16 dims
        uint32_t hi[4], lo[4];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const uint4 v =
              in ? __ldg(src + 2 * i + k) : make_uint4(0u, 0u, 0u, 0u);
          const uint32_t x[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
          for (int n2 = 0; n2 < 2; ++n2) {
            const float a0 = bf16_lo(x[2 * n2]) * down;
            const float a1 = bf16_hi(x[2 * n2]) * down;
            const float a2 = bf16_lo(x[2 * n2 + 1]) * down;
            const float a3 = bf16_hi(x[2 * n2 + 1]) * down;
            const uint32_t c =
                e4m3x2_from(a0 - first(a0), a1 - first(a1)) |
                e4m3x2_from(a2 - first(a2), a3 - first(a3)) << 16;
            const float2 h0 = __half22float2(u32_as_h2(e4m3x2_lo(c)));
            const float2 h1 = __half22float2(u32_as_h2(e4m3x2_hi(c)));
            hi[2 * k + n2] = c;
            lo[2 * k + n2] = e5m2x2_from(a0 - h0.x, a1 - h0.y) |
                             e5m2x2_from(a2 - h1.x, a3 - h1.y) << 16;
          }
        }
        const uint32_t at = q_s + tile * 2 * kPfQuery + (tid & 127) * 128 +
                            ((i ^ (tid & 7)) << 4);
        st_shared_v4(at, make_uint4(hi[0], hi[1], hi[2], hi[3]));
        st_shared_v4(at + kPfQuery, make_uint4(lo[0], lo[1], lo[2], lo[3]));
      }
    };
    if (__any_sync(0xffffffffu, outlier))
      codes(beyond);
    else
      codes([](float) -> float { return 0.f; });
    fence_to_async();
    __syncwarp();
    if (lane == 0) mbar_arrive(sh.q_full + tile);
    // ------------------------------------------------------------- softmax
    const uint32_t mine =
        tm + tile * kPfColumns + ((uint32_t)((wid & 3) * 32) << 16);
    float m = -INFINITY, l = 0.f;
    uint32_t e_top = 0;  // unit of the sums
    // a zero that the compiler does not know: mul.rn and add.rn of two numbers
    // at once are made one fma with one rounding, an fma and an add are not
    const float zero = __int_as_float(*(volatile int *)&sh.dead);
    bool ok = true;
    // rescales the sums in tensor memory
    auto rescale = [&](float fall) {
      tm_wait_st();
#pragma unroll 1
      for (int k = 0; k < 8; ++k) {
        uint32_t o[16];
        tm_ld16(o, mine + kPfColO + 16 * k);
        tm_wait_ld();
#pragma unroll
        for (int i = 0; i < 16; ++i)
          o[i] = __float_as_uint(__uint_as_float(o[i]) * fall);
        tm_st16(mine + kPfColO + 16 * k, o);
      }
    };
    // raises the reference to `top` in lanes whose scores pass it by too much
    auto raise = [&](float top, bool sums) -> float {
      const float to = top > m + kQSlack ? top : m;
      const float fall = to == m ? 1.f : ex2_fast(m - to);
      m = to;
      l *= fall;
      if (sums) rescale(fall);
      return fall;
    };
    // A far tile: a token's value scale in its factor, the factors as hi + lo in
    // bf16, whose range is fp32's: 16 bits at any size.  Hi and lo of a page lie
    // over the 16 columns of its scores, 8 columns each.
    auto far_tile = [&](int par, uint32_t there, bool sums) {
      float top = -INFINITY;
#pragma unroll 1
      for (int pg = 0; pg < kPfPages; ++pg) {
        uint32_t s[16];
        tm_ld16(s, mine + 16 * pg);
        tm_wait_ld();
        if (there >> pg & 1) {
#pragma unroll
          for (int i = 0; i < 16; ++i)
            top = fmaxf(top, __uint_as_float(s[i]) *
                                 sh.k_scale[par][kPage * pg + i]);
        }
      }
      top *= f;
      if (__any_sync(0xffffffffu, top > m + kQSlack)) raise(top, sums);
#pragma unroll 1
      for (int pg = 0; pg < kPfPages; ++pg) {
        uint32_t s[16], w[16];
        tm_ld16(s, mine + 16 * pg);
        tm_wait_ld();
        const uint4 e4 = reinterpret_cast<const uint4 *>(sh.v_token[par])[pg];
        const uint32_t e[4] = {e4.x, e4.y, e4.z, e4.w};
        const bool here = there >> pg & 1;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          float u[2];
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const int t = 2 * i + k;
            const uint32_t ev = e[t >> 2] >> 8 * (t & 3) & 255u;
            const float x = __uint_as_float(s[t]) *
                            sh.k_scale[par][kPage * pg + t];
            const float v =
                here ? ex2_fast(__fmul_rn(x, f) - (m - kQLift)) : 0.f;
            l += v;
            u[k] = here ? v * exp2_int((int)ev - (int)e_top) : 0.f;
          }
          const __nv_bfloat162 hi = __floats2bfloat162_rn(u[0], u[1]);
          const __nv_bfloat162 lo = __floats2bfloat162_rn(
              u[0] - __low2float(hi), u[1] - __high2float(hi));
          w[i] = *reinterpret_cast<const uint32_t *>(&hi);
          w[8 + i] = *reinterpret_cast<const uint32_t *>(&lo);
        }
        tm_st16(mine + 16 * pg, w);
      }
    };
    for (int j = 0; j < n; ++j) {
      const int par = j & 1;
      // with S(j) all products before it, among them O(j - 1), are done
      ok = pf_wait(sh, sh.info + par, j >> 1 & 1) &&
           pf_wait(sh, sh.qk_done + tile, j & 1);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      tm_fence_after();
      const uint32_t there = sh.there[par][0] | sh.there[par][1];
      const bool far = sh.far[par];
      if (sh.v_top[par] != e_top) {  // larger values than before
        if (j > 0)
          rescale(exp2_int(max(-126, (int)e_top - (int)sh.v_top[par])));
        e_top = sh.v_top[par];
      }
      if (far) {
        far_tile(par, there, j > 0);
      } else {
        // 64 columns at a time: their weights go over the scores they come
        // from, in columns that have been read
        for (int c = 0; c < 2; ++c) {
          uint64_t x[32];
          {
            uint32_t s0[32], s1[32];
            tm_ld32(s0, mine + 64 * c);
            tm_ld32(s1, mine + 64 * c + 32);
            tm_wait_ld();
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              x[i] = pack2(s0[2 * i], s0[2 * i + 1]);
              x[16 + i] = pack2(s1[2 * i], s1[2 * i + 1]);
            }
          }
          float top = -INFINITY;
#pragma unroll
          for (int p = 0; p < 4; ++p) {
            const int pg = 4 * c + p;
            float t4[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float4 k4 =
                  reinterpret_cast<const float4 *>(sh.k_scale[par])[4 * pg + i];
              uint64_t &x0 = x[8 * p + 2 * i], &x1 = x[8 * p + 2 * i + 1];
              x0 = mul2(x0, pack2(k4.x, k4.y));
              x1 = mul2(x1, pack2(k4.z, k4.w));
              const float2 u = unpack2(x0), v = unpack2(x1);
              t4[i] = fmaxf(max3(u.x, u.y, v.x), v.y);
            }
            const float t1 = fmaxf(max3(t4[0], t4[1], t4[2]), t4[3]);
            if (there >> pg & 1) top = fmaxf(top, t1);
          }
          top *= f;
          if (__any_sync(0xffffffffu, top > m + kQSlack)) {
            // rare after the first tiles
            const float fall = raise(top, j > 0);
            tm_wait_st();
            // this tile's weights so far, rounded a second time
#pragma unroll 1
            for (int k = 0; k < 2 * c; ++k) {
              uint32_t w[16];
              tm_ld16(w, mine + 16 * k);
              tm_wait_ld();
#pragma unroll
              for (int i = 0; i < 16; ++i) {
                const float2 v = __half22float2(u32_as_h2(w[i]));
                w[i] = h2_as_u32(__floats2half2_rn(v.x * fall, v.y * fall));
              }
              tm_st16(mine + 16 * k, w);
            }
          }
          uint32_t w[32];
          const uint64_t ff = pack2(f, f);
          // scores rounded before the reference is taken off, as it was: equal
          // ones stay equal and the largest differs from it by nothing, where a
          // difference rounded alone holds the reference's own rounding (at
          // 10^11 up to 4096; 3 us of 270)
          const float ref = kQLift - m;
          const uint64_t aa = pack2(ref, ref), zz = pack2(zero, zero);
#pragma unroll
          for (int p = 0; p < 4; ++p) {
            const int pg = 4 * c + p;
            uint64_t sum[2] = {0, 0};
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const float2 z = unpack2(add2(fma2(x[8 * p + i], ff, zz), aa));
              const float u = ex2_fast(z.x), v = ex2_fast(z.y);
              sum[i & 1] = add2(sum[i & 1], pack2(u, v));
              w[8 * p + i] = h2_as_u32(__floats2half2_rn(u, v));
            }
            if (there >> pg & 1) {
              const float2 t2 = unpack2(add2(sum[0], sum[1]));
              l += t2.x + t2.y;
            } else {
#pragma unroll
              for (int i = 0; i < 8; ++i) w[8 * p + i] = 0u;
            }
          }
          tm_st32(mine + 32 * c, w);
        }
      }
      tm_wait_st();
      tm_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(sh.p_full + tile);
    }
    if (ok) ok = pf_wait(sh, sh.o_done + tile, 0);
    ok = __all_sync(0xffffffffu, ok);
    tm_fence_after();
    // partials: 16 rows at a time as matrix fragments (row lane / 4 and + 8,
    // columns 2 (lane % 4), + 1 of every 8), so that four lanes write a whole
    // memory sector
    auto place = [&](int r) -> size_t {
      return (size_t)split * rows * a.h_kv +
             (size_t)(r / a.G) * a.h_kv * a.G + (size_t)h * a.G + r % a.G;
    };
    const float unit = exp2_int((int)e_top - 127);
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const int r0 = row - lane + 16 * half + (lane >> 2);
      float *d0 = a.o_part + place(r0) * kDim + 2 * (lane & 3);
      float *d1 = a.o_part + place(r0 + 8) * kDim + 2 * (lane & 3);
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        uint32_t o[16];
        tm_ld16x256(o, mine + ((uint32_t)(16 * half) << 16) + kPfColO + 32 * c);
        tm_wait_ld();
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (r0 < rows && ok)
            *reinterpret_cast<float2 *>(d0 + 32 * c + 8 * i) =
                make_float2(__uint_as_float(o[4 * i]) * unit,
                            __uint_as_float(o[4 * i + 1]) * unit);
          if (r0 + 8 < rows && ok)
            *reinterpret_cast<float2 *>(d1 + 32 * c + 8 * i) =
                make_float2(__uint_as_float(o[4 * i + 2]) * unit,
                            __uint_as_float(o[4 * i + 3]) * unit);
        }
      }
    }
    if (row < rows) a.ml_part[place(row)] = make_float2(m, ok ? l : 0.f);
  } else {
    auto good = [&](int ph) -> bool { return ph >= 0 && ph < a.num_phys; };
    // page `pg` of tile j as the table has it, -1 past the end
    auto page = [&](int j, int pg) -> int {
      pg += (t0 + j) * kPfPages;
      return j < n && pg < a.pages ? __ldg(a.table + pg) : -1;
    };
    // a part of the records of `pages` pages (ph: page of the lane); one
    // arrival for all, a lane to a page; which were there
    auto copy = [&](int ph, int pages, int off, uint32_t bytes, uint32_t to,
                    uint64_t *bar) -> uint32_t {
      const bool here = lane < pages && good(ph);
      const uint32_t there = __ballot_sync(0xffffffffu, here);
      if (lane == 0) mbar_arrive_tx(bar, __popc(there) * bytes);
      __syncwarp();
      if (here)
        bulk_g2s(to + lane * bytes,
                 a.records + ((size_t)ph * a.h_kv + h) * kQRec + off, bytes,
                 bar);
      __syncwarp();
      return there;
    };
    bool ok = true;
    if (wid == kProducts) {
      // -------------------------------------------------------- products
      const uint64_t dq = mat_desc(q_s, 16), dk = mat_desc(k_s, 16);
      const uint64_t dv = mat_desc(v_s, kPfBlock);
      // S(j) of row tile t, and after the last one its keys may go
      auto scores = [&](int t, int j) {
        if (elect_one()) {
          const uint64_t q = dq + t * (2 * kPfQuery >> 4);
          const uint64_t k = dk + j % R * (kPfCodes >> 4);
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)  // hi, then lo
            mma_ss(tm + t * kPfColumns,
                   q + ((kk >> 2) * (kPfQuery >> 4) + (kk & 3) * 2),
                   k + (kk & 3) * 2, kk < 4 ? kPfDescS : kPfDescLo, kk > 0);
          mma_commit(sh.qk_done + t);
          if (t == nt - 1) mma_commit(sh.k_free + j % R);
        }
        __syncwarp();
      };
      auto weighted = [&](int t, int j, int far) {
        if (elect_one()) {
          const uint64_t v = dv + j % R * (2 * kPfBlock >> 4);
          const uint32_t at = tm + t * kPfColumns;
          if (far) {  // hi and lo of each page
#pragma unroll 1
            for (int kk = 0; kk < 2 * kPfTile / 16; ++kk)
              mma_ts(at + kPfColO, at + 8 * kk,
                     v + (kk >> 1) * (kPage * 128 >> 4), kPfDescFar,
                     j > 0 || kk > 0);
          } else {
#pragma unroll
            for (int kk = 0; kk < kPfTile / 16; ++kk)
              mma_ts(at + kPfColO, at + 8 * kk, v + kk * (kPage * 128 >> 4),
                     kPfDescO, j > 0 || kk > 0);
          }
          if (t == nt - 1) mma_commit(sh.v_free + j % R);
          if (j == n - 1) mma_commit(sh.o_done + t);
        }
        __syncwarp();
      };
      for (int j = -1; j < n && ok; ++j)
        for (int t = 0; t < nt; ++t) {
          if (j >= 0) {
            ok = t > 0 || pf_wait_ring(sh, sh.v_full, j);
            // (under the wait for the weights: 2 us of 276)
            const int far = sh.far[j & 1];
            ok = ok && pf_wait(sh, sh.p_full + t, j & 1);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            tm_fence_after();
            weighted(t, j, far);
          }
          if (j + 1 < n) {
            ok = (t > 0 || pf_wait_ring(sh, sh.k_full, j + 1)) &&
                 (j >= 0 || pf_wait(sh, sh.q_full + t, 0));
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            tm_fence_after();
            scores(t, j + 1);
          }
        }
    } else if (wid == kKeys) {
      // ------------------------------------------------------------ keys
      int copied = 0;  // tiles
      auto copy_keys = [&](int ph) {
        const int j = copied++;
        if (lane < kPfPages && !good(ph) &&
            (t0 + j) * kPfPages + lane < a.pages)
          set_status(a.status, LOCKS_DEV_BAD_PAGE_ID);
        copy(ph, kPfPages, 0, kQCodes, k_s + j % R * kPfCodes,
             sh.k_raw + j % R);
      };
      for (int j = 0; j < R && j < n; ++j) copy_keys(page(j, lane));
      int ph = page(R, lane);
      for (int j = 0; j < n; ++j) {
        ok = pf_wait_ring(sh, sh.k_raw, j);
        if (!__all_sync(0xffffffffu, ok)) break;
        // the halves of odd key rows trade places
#pragma unroll
        for (int h2 = 0; h2 < 2; ++h2) {
          const uint32_t at = k_s + j % R * kPfCodes + h2 * 4 * kQCodes +
                              (2 * (lane >> 2) + 1) * 128 + 16 * (lane & 3);
          // rows that are read together start with different halves
          const uint32_t a0 = at + (lane & 4 ? 64 : 0);
          const uint32_t a1 = at + (lane & 4 ? 0 : 64);
          uint4 x[4], y[4];
#pragma unroll
          for (int p = 0; p < 4; ++p) {
            x[p] = lds128(a0 + p * kQCodes);
            y[p] = lds128(a1 + p * kQCodes);
          }
#pragma unroll
          for (int p = 0; p < 4; ++p) {
            st_shared_v4(a0 + p * kQCodes, y[p]);
            st_shared_v4(a1 + p * kQCodes, x[p]);
          }
        }
        fence_to_async();
        __syncwarp();
        if (lane == 0) mbar_arrive(sh.k_full + j % R);
        if (copied < n && copied == j + 1) {
          // the scores of the tile before in this buffer done: it may go
          ok = pf_wait_ring(sh, sh.k_free, copied - R);
          if (!__all_sync(0xffffffffu, ok)) break;
          copy_keys(ph);
          ph = page(copied, lane);
        }
      }
      if (*(volatile int *)&sh.dead)
        for (int j = max(0, copied - R); j < copied; ++j)
          q_wait(sh.k_raw + j % R, j / R & 1);
    } else {
      // ---------------------------------------------------------- values
      // A warp takes kPfOwn pages of a tile, four slots at a time, and has
      // them copied itself.  Eight lanes that read and store a 16-byte group
      // each have the same half of the dims of slots s and s + 1, which
      // either swizzle keeps in different banks.
      const int own = wid - kKeys - 1, first = own * kPfOwn;
      const int s4 = (lane >> 4) * 2 + (lane >> 2 & 1);
      const int c = (lane & 3) | (lane >> 1 & 4);
      const uint32_t mine = raw_s + first * kPfRest;
      int copied = 0;  // tiles
      auto copy_values = [&](int ph) -> uint32_t {
        const int b = copied++ % R;
        const uint32_t to = mine + b * kPfRaw;
        const uint32_t there =
            copy(ph, kPfOwn, kQOffV, kPfRest, to, sh.v_raw[own] + b);
        // a page that is not there reads as zeros
        for (uint32_t gone = ~there & ((1u << kPfOwn) - 1); gone;
             gone &= gone - 1)
          for (int i = lane; i < kPfRest / 16; i += 32)
            st_shared_v4(to + (__ffs(gone) - 1) * kPfRest + 16 * i,
                         make_uint4(0u, 0u, 0u, 0u));
        __syncwarp();
        return there;
      };
      uint32_t there[R];  // of tiles j to j + R - 1
#pragma unroll
      for (int j = 0; j < R; ++j)
        there[j] = j < n ? copy_values(page(j, first + lane)) : 0u;
      int ph = page(R, first + lane);
      uint32_t top_e = 0;  // largest scale so far
      for (int j = 0; j < n; ++j) {
        ok = pf_wait_ring(sh, sh.v_raw[own], j);
        if (!__all_sync(0xffffffffu, ok)) break;
        const uint32_t from = mine + j % R * kPfRaw;
        // lane 16 i + slot: exponents of rows of pages i and 2 + i
        uint32_t ke[kPfOwn / 2], ve[kPfOwn / 2];
#pragma unroll
        for (int i = 0; i < kPfOwn / 2; ++i) {
          const uint32_t at =
              from + (2 * i + (lane >> 4)) * kPfRest + (lane & 15);
          asm volatile("ld.shared.u8 %0, [%1];\n"
                       : "=r"(ke[i])
                       : "r"(at + (kQOffKE - kQOffV)));
          asm volatile("ld.shared.u8 %0, [%1];\n"
                       : "=r"(ve[i])
                       : "r"(at + (kQOffVE - kQOffV)));
          ve[i] = q_scale_byte(ve[i]);
        }
        // The largest and the least scale of these pages, for both warps.  (The
        // place of j - 2: the other warp has read it, or it had not come to the
        // range of j - 1.)
        const uint32_t now = there[0];
        uint32_t most = 0, least = 255;
#pragma unroll
        for (int i = 0; i < kPfOwn / 2; ++i)
          if (now >> (2 * i + (lane >> 4)) & 1) {
            most = max(most, ve[i]);
            least = min(least, ve[i]);
          }
        most = __reduce_max_sync(0xffffffffu, most);
        least = __reduce_min_sync(0xffffffffu, least);
        if (lane == 0) {
          sh.range[j & 1][own] = make_uint2(most, least);
          mbar_arrive(sh.ranges + (j & 1));
        }
        uint4 raw[4 * kPfOwn];
#pragma unroll
        for (int u = 0; u < 4 * kPfOwn; ++u) {
          const int sl = 4 * (u & 3) + s4;
          raw[u] = lds128(from + (u >> 2) * kPfRest + sl * kDim +
                          16 * q_group(c, sl));
        }
        // all has been read before the next copy is written there
        fence_to_async();
        __syncwarp();
        if (copied < n) {
          if (R > 1) there[0] = there[R - 1];
          there[R - 1] = copy_values(ph);
          ph = page(copied, first + lane);
        } else if (R > 1) {
          there[0] = there[R - 1];
        }
        // The largest scale so far and the least of this tile decide its form.
        ok = pf_wait(sh, sh.ranges + (j & 1), j >> 1 & 1);
        if (!__all_sync(0xffffffffu, ok)) break;
#pragma unroll
        for (int w = 0; w < kPfWiden; ++w) {
          const uint2 r = sh.range[j & 1][w];
          top_e = max(top_e, r.x);
          least = min(least, r.y);
        }
        const bool far = least + kQSpread < top_e;
        // what softmax needs to know of the tile, in the place of j - 2's:
        // O(j - 2) is done
        if (R == 2 && j >= 2) {
          ok = pf_wait_ring(sh, sh.v_free, j - R);
          if (!__all_sync(0xffffffffu, ok)) break;
        }
        // factor: 2^(e - E), 2^-8 or more (in a far tile it is not used)
        uint32_t factor[kPfOwn / 2];
#pragma unroll
        for (int i = 0; i < kPfOwn / 2; ++i) {
          const int at = kPage * (first + 2 * i + (lane >> 4)) + (lane & 15);
          sh.k_scale[j & 1][at] = __uint_as_float(ke[i] << 23);
          if (far) sh.v_token[j & 1][at] = (uint8_t)ve[i];
          factor[i] = h2_as_u32(__float2half2_rn(
              exp2_int(max(-126, min(0, (int)ve[i] - (int)top_e)))));
        }
        if (lane == 0) sh.there[j & 1][own] = now << first;
        if (lane == 0 && own == 0) {
          sh.far[j & 1] = far;
          sh.v_top[j & 1] = top_e;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(sh.info + (j & 1));
        // O(j - 1) done: its values may go
        if (R == 1 && j >= 1) {
          ok = pf_wait_ring(sh, sh.v_free, j - R);
          if (!__all_sync(0xffffffffu, ok)) break;
        }
        const uint32_t to = v_s + j % R * 2 * kPfBlock;
        auto widen = [&](auto number) {
#pragma unroll
          for (int u = 0; u < 4 * kPfOwn; ++u) {
            const int sl = 4 * (u & 3) + s4;
            const __half2 x = u32_as_h2(__shfl_sync(
                0xffffffffu, factor[u >> 3], 16 * (u >> 2 & 1) + sl));
            const uint32_t w[4] = {raw[u].x, raw[u].y, raw[u].z, raw[u].w};
            uint32_t y[8];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              y[2 * k] = number(u32_as_h2(e4m3x2_lo(w[k])), x);
              y[2 * k + 1] = number(u32_as_h2(e4m3x2_hi(w[k])), x);
            }
            const int r = (first + (u >> 2)) * kPage + sl;
            st_shared_v4(to + tile_at(r, 2 * c),
                         make_uint4(y[0], y[1], y[2], y[3]));
            st_shared_v4(to + tile_at(r, 2 * c + 1),
                         make_uint4(y[4], y[5], y[6], y[7]));
          }
        };
        if (far)  // the codes themselves
          widen([](__half2 code, __half2) -> uint32_t {
            const __nv_bfloat162 y =
                __float22bfloat162_rn(__half22float2(code));
            return *reinterpret_cast<const uint32_t *>(&y);
          });
        else
          widen([](__half2 code, __half2 x) -> uint32_t {
            return h2_as_u32(__hmul2(code, x));
          });
        fence_to_async();
        __syncwarp();
        if (lane == 0) mbar_arrive(sh.v_full + j % R);
      }
      if (*(volatile int *)&sh.dead)
        for (int j = max(0, copied - R); j < copied; ++j)
          q_wait(sh.v_raw[own] + j % R, j / R & 1);
    }
  }
  __syncwarp();
  tm_fence_before();
  __syncthreads();
  if (wid == kProducts) {
    // some role's wait gave up, the last of them that for the last products:
    // say so, and give what is in flight a last, bounded chance to finish
    if (*(volatile int *)&sh.dead && elect_one()) {
      set_status(a.status, LOCKS_DEV_TIMEOUT);
      mma_commit(&sh.drain);
      q_wait(&sh.drain, 0);
    }
    __syncwarp();
    asm volatile(
        "tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;\n" ::"r"(tm),
        "r"(R * kPfColumns)
        : "memory");
  }
}

// ---------------------------------------------------------------------------
// launcher
// ---------------------------------------------------------------------------
// How many ranges the prefix's tiles are cut into, and whether a CTA takes two
// row tiles.  A rule on sizes alone (152 SMs), so that the workspace's size
// needs no GPU.
//
// The estimate (us) that picks among them: a tile of a CTA 1.6 alone on its
// SM, 2.4 with another beside it, 2.0 of two row tiles; 6 for a CTA's start
// and end, a row's partial 1 KB of traffic; and the sequences' own pages,
// whose kernel finds room on SMs that the grid leaves free, or waits for its
// end.  Of 190 measured splits of 16 shapes it picks ones 2.4% from the best
// (worst 21%, 128 short sequences).  Two row tiles to a CTA pay for long
// prefixes of many rows, where keys and values are prepared once for both:
// 64, 8, 8192, G = 8: 265 us in 9 ranges, one row tile 285; 32, 8, 512, G = 8:
// 34.2 and 33.1; 40, 2, 4096, G = 8: 51.2 and 47.4.
//
// 0 ranges: too little to share, every sequence reads the pages itself.
// (Sequences, KV heads, pages, G = 4 unless given: read by each against once,
// us, replayed back to back.)
//   triples below the limit: 8, 8, 128: 12.2 and 13.5; 2, 8, 256: 10.6 and
//     13.9; 32, 8, 32: 11.1 and 16.2; 64, 8, 16, G = 8: 15.6 and 18.0; 16, 8,
//     64, G = 16: 13.9 and 20.8; 128, 1, 64, G = 8: 12.5 and 16.6; but 256, 8,
//     4, G = 1: 23.4 and 17.7
//   above: 8, 8, 256: 20.4 and 15.0; 2, 8, 1024: 20.5 and 21.0; 2, 8, 2048:
//     27.8 and 28.4; 32, 8, 64: 22.2 and 16.5; 64, 8, 32, G = 8: 20.3 and 20.1;
//     64, 8, 64, G = 8: 30.1 and 20.9; 16, 8, 128, G = 16: 26.6 and 21.8; 256,
//     8, 8, G = 1: 27.1 and 17.7; 128, 1, 128, G = 8: 23.4 and 18.0
// One sequence shares nothing (1, 8, 8192: 64 and 77).  The numbers of SMs and
// of CTAs that fit on them are this GPU's, written out.
PrefixPlan prefix_plan(int batch, int h_kv, int G, int pages) {
  PrefixPlan plan{0, false};
  if (batch < 2 || (long long)batch * h_kv * pages < kPfMinShared) return plan;
  const long long row_tiles =
      ((long long)batch * G + kPfRows - 1) / kPfRows;
  const long long tiles = (pages + kPfPages - 1) / kPfPages;
  double best = 1e30;
  for (int r = 1; r <= 2 && r <= row_tiles; ++r) {
    const long long slots = r == 1 ? 304 : 152;  // CTAs that run at once
    const long long base = (row_tiles + r - 1) / r * h_kv;
    for (long long s = 1, t = tiles;;) {  // s ranges of up to t tiles
      const long long ctas = base * s, waves = (ctas + slots - 1) / slots;
      const double tile = r == 2 ? 2.0 : ctas > 152 ? 2.4 : 1.6;
      const double room = (double)(waves * slots - ctas) / 88.0;
      const double us = (double)waves * (tile * (double)t + 6.0) +
                        1.6e-4 * (double)(s * batch * h_kv * G) +
                        (room < 1.0 ? 2.0 * r * (1.0 - room) : 0.0);
      if (us < best) {
        best = us;
        plan = {(int)s, r == 2};
      }
      if (t == 1) break;
      s = (tiles + t - 2) / (t - 1);  // the fewest of fewer tiles
      if (base * s > 2 * slots) break;
      t = (tiles + s - 1) / s;
    }
  }
  return plan;
}

// Rows of partials that the workspace has room for: no plan up to these sizes
// has more, whatever its number of ranges, so that a workspace of one batch and
// prefix serves all smaller ones.  A plan of more than one range has at most
// 2 * 304 (or 152) CTAs of 128 (256) rows each, and never more ranges than
// tiles.
size_t prefix_rows(int batch, int h_kv, int G, int pages) {
  if (batch < 2 || (long long)batch * h_kv * pages < kPfMinShared) return 0;
  const size_t rows = (size_t)batch * h_kv * G;
  const size_t tiles = ((size_t)pages + kPfPages - 1) / kPfPages;
  const size_t most = 2 * 304 * kPfRows;
  return tiles * rows < most ? tiles * rows : rows > most ? rows : most;
}

template <int R>
static cudaError_t launch_tiles(const PfArgs &a, cudaStream_t stream) {
  static DeviceFlags done;
  cudaError_t e = once_per_device(done, [] {
    return cudaFuncSetAttribute(prefix_kernel<R>,
                                cudaFuncAttributeMaxDynamicSharedMemorySize,
                                kPfSmem<R>);
  });
  if (e != cudaSuccess) return e;
  const long long ctas =
      (long long)((a.row_tiles + R - 1) / R) * a.h_kv * a.splits;
  return launch_pdl(prefix_kernel<R>, dim3((unsigned)ctas),
                    dim3(kPfThreads<R>), kPfSmem<R>, stream, a);
}

cudaError_t launch_prefix(const void *q, const void *records,
                          int64_t num_phys, const int32_t *table, int pages,
                          int batch, int h_kv, int G, PrefixPlan plan,
                          float *o_part, float2 *ml_part, int32_t *status,
                          cudaStream_t stream) {
  const int row_tiles = (int)(((long long)batch * G + kPfRows - 1) / kPfRows);
  const PfArgs a{static_cast<const __nv_bfloat16 *>(q),
                 static_cast<const uint8_t *>(records),
                 num_phys, table, pages, batch, h_kv, G, row_tiles, plan.splits,
                 o_part, ml_part, status};
  return plan.wide ? launch_tiles<2>(a, stream) : launch_tiles<1>(a, stream);
}

}  // namespace locks
