// Attention of many query tokens per sequence over the bf16 cache, causal with
// a sliding window and first tokens that stay visible (include/locks.h).
//
// A unit is two tiles of 128 query rows of one (sequence, KV head), the heads of
// the group side by side for each token, so that a key serves them all, over the
// 128-token tiles that any of its rows sees.  Both products are tcgen05 matrix
// products with fp32 accumulators in tensor memory: S = Q K^T, O += W V with the
// weights W in bf16 over the scores they came from (bf16 since both operands of
// a product have one type, and V is bf16).  Pages come by tensor copies, a page's
// rows of a head in one, straight to their swizzled places in a ring of five
// 32 KB buffers that keys and values take in turn.
//
// Eight warps per row tile do its softmax, two threads to a query row, half of
// the columns each, which need no word with each other between a unit's first
// tile and its end: a row's reference is its first tile's largest score (so that
// the weight of a token that has it all is 1) and stays, since bf16 weights and
// fp32 sums keep their bits at any size.  One thread issues the products, one
// warp the copies.
// One row tile's softmax runs under the other's products.  A CTA stays on its SM
// and takes further units from those that have no CTA yet; the next unit is
// loaded and its first scores computed under the end of the one before.
//
// Tiles that all rows see whole have no masks.  In the others a token that no
// row sees has its value row cleared, whatever it holds, and a value that is
// not finite, which a weight of zero would spread to rows that do not see it,
// sends the row tile to the plain form (plain_rows), in fp32, where a token that a
// row does not see is not touched for it.
//
// Few rows over many tokens (drafted tokens, short parts of long prompts): the
// tiles of a unit are cut into ranges, whose partials a second kernel joins.
//
// Bound: a prompt of 8192 tokens, 32 query and 8 KV heads, takes 343 us, 1600
// TFLOP/s, in bursts of a replayed graph (calls one after the other 366, 1503: the
// board's power), a tile of both row tiles some 2,700 cycles: 2 * 684 for the scores
// (64 in theory for each of 8 products of 16 dims; they read shared memory at all
// of its 128 bytes a cycle and take 85), 2 * 533 for the weighted values, the
// rest between them.  The tensor core is busy for 68% of the time, and the board
// draws the 1,400 W that it may (1.9 GHz).  A unit's
// start and end cost 9,000 cycles, the time of 3.5 tiles: 32768 tokens with a
// window of 4096 (34 tiles a unit) 1345 to 1410 us, 1480 to 1550 TFLOP/s; eight
// prompts of 100 to 2500 tokens and 5 heads to a group (6.5 tiles a unit) 128 us.
// (For the softmax of a row tile, one after the other: outputs 3,300 cycles, what
// the row tile's warps tell each other at the end 1,900, the next unit's fields
// 1,500, its first tile 2,600 where later ones take 1,000 and masked ones 1,900
// to 2,500; the copies' warp: 3,000 from the answer to the rows, 2,700 more to the
// first copy.)  Few rows: 4 tokens of 16 sequences of 32K 335 us, 6.4 TB/s.
//
// What was slower, for 8192 tokens: a warp that votes and elects between its
// products 440 us; two copies of 2 KB to a page 465 (the copies alone 453); a
// CTA to a unit 355; first tiles without masks where they need none 346; lone row
// tiles in both places in turn 345 (5% less for drafted tokens over a window of
// 256); three units under way 349.  What made no difference: four buffers instead
// of five; rows written by four lanes each; a first reference from 32 columns.
// Registers are short (96 with 18 warps): a variant that spills in the softmax
// takes 366 (outputs 32 columns at a time) to 510 us.  A search by all lanes for a
// unit's rows: 256 prompts of 16 to 100 tokens 98 us (one lane's bisection 111).
#include <cuda.h>

#include <type_traits>

#include "launch.h"
#include "quantised.cuh"
#include "tensor.cuh"

namespace locks {

constexpr int kWinRows = 128;   // query rows of a row tile
constexpr int kWinTile = 128;   // tokens of a tile
constexpr int kWinPages = kWinTile / kPage;
constexpr int kWinStages = 5;   // buffers of keys or values
constexpr int kWinPage = kPage * kDim * 2;       // 4 KB
constexpr int kWinBuffer = kWinTile * kDim * 2;  // a tile, or its query
constexpr int kWinQHalf = kWinBuffer / 2;        // 64 dims of a query tile
// barriers and the like, then the tiles, at multiples of 1024 bytes: all of
// the 227 KB that a CTA can have
constexpr int kWinHeader = 3 * 1024;
constexpr int kWinSmem = kWinHeader + (2 + kWinStages) * kWinBuffer;
static_assert(kWinSmem <= 227 * 1024, "shared memory");
constexpr int kWinProducts = 16;  // the softmax's warps, then one, then copies
constexpr int kWinThreads = 32 * 18;
constexpr float kWinScale = 0.12751743074602467f;  // log2(e) / sqrt(128)
constexpr float kWinMost = 0x1p64f;       // sum of 32 weights
constexpr int kWinPasses = 8;  // then the plain way
constexpr float kWinLargest = 1048576.f;  // reference, 2^20
constexpr float kWinLn2 = 0.69314718055994531f;
// bf16 operands, fp32 sums, M = N = 128; bit 16: B runs along N
constexpr uint32_t kWinDescS =
    1u << 4 | 1u << 7 | 1u << 10 | (128u >> 3) << 17 | (128u >> 4) << 24;
constexpr uint32_t kWinDescO = kWinDescS | 1u << 16;

// Tokens of a row tile: as many as fit with all heads of the group.
__host__ __device__ __forceinline__ int tile_tokens(int G) {
  return kWinRows / G;
}

// The rows of a CTA, two row tiles: `tokens` new tokens of sequence b from
// q row `q0`, at positions from p0; of those the first that sees anything and
// the last; and the tiles that any of them sees: the first `head`, then those
// from `from`, `tiles` in all.
struct WinRows {
  int b, tokens, q0, p0, p_min, p_max, from, head, tiles;

  __device__ __forceinline__ int tile(int j) const {
    return j < head ? j : from + j - head;
  }
  // whether any row sees a token of page pg
  __device__ __forceinline__ bool sees_page(const WinArgs &a, int pg) const {
    const int t = pg * kPage;
    return t <= p_max && (t < a.sinks || t + kPage - 1 > p_min - a.window);
  }
  __device__ __forceinline__ bool sees(const WinArgs &a, int t) const {
    return t <= p_max && (t < a.sinks || t > p_min - a.window);
  }
  // whether all rows do
  __device__ __forceinline__ bool all_see(const WinArgs &a, int t) const {
    return t <= p0 && (t < a.sinks || t > p_max - a.window);
  }
  // whether all rows see all tokens of a tile
  __device__ __forceinline__ bool whole(const WinArgs &a, int tile) const {
    const int t = tile * kWinTile;
    return t + kWinTile - 1 <= p0 &&
           (t + kWinTile <= a.sinks || t > p_max - a.window);
  }
};

// Slots of 2 * tile_tokens(G) tokens: sequence b's begin at slot
// floor(q_starts[b] / that) + b, which leaves room for all of them, whatever
// the lengths.
__device__ __forceinline__ long long first_slot(const WinArgs &a, int b) {
  return (long long)(__ldg(a.q_starts + b) / (2 * tile_tokens(a.G))) + b;
}

// The last of n things that x says yes to, which it does to the first ones; all
// of a warp, 32 candidates at a time.
template <class F>
__device__ __forceinline__ int last_where(int n, F x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) >> 5;
    const int b = min(lo + (int)(threadIdx.x & 31) * step, hi - 1);
    const int yes = __popc(__ballot_sync(0xffffffffu, x(b)));
    lo = min(lo + max(yes - 1, 0) * step, hi - 1);
    hi = min(hi, lo + step);
  }
  return lo;
}

// All of a warp; false: no rows
__device__ __forceinline__ bool find_rows(const WinArgs &a, long long slot,
                                          WinRows &r) {
  const int lo =
      last_where(a.batch, [&](int b) { return first_slot(a, b) <= slot; });
  const int s = __ldg(a.q_starts + lo), e = __ldg(a.q_starts + lo + 1);
  int L = __ldg(a.seq_lens + lo);
  if (s < 0 || e <= s || e > a.n_tokens) return false;
  const int most = 2 * tile_tokens(a.G);
  const long long first = (slot - (s / most) - lo) * most;
  if (first < 0 || first >= e - s) return false;
  L = max(0, min(L, a.max_pages * kPage));
  r.b = lo;
  r.q0 = s + (int)first;
  r.tokens = min(most, e - r.q0);
  r.p0 = L - (e - r.q0);
  r.p_min = max(0, r.p0);  // (positions below 0 see nothing)
  r.p_max = r.p0 + r.tokens - 1;
  const int start = max(0, r.p_min - (a.window - 1));
  r.from = start / kWinTile;
  r.head = min((min(a.sinks, start) + kWinTile - 1) / kWinTile, r.from);
  r.tiles = r.p_max < 0 ? 0 : r.head + r.p_max / kWinTile + 1 - r.from;
  return true;
}

// output row of head g of the group, token i of the CTA
__device__ __forceinline__ int out_row(const WinArgs &a, const WinRows &r,
                                       int h, int i, int g) {
  return (r.q0 + i) * (a.h_kv * a.G) + h * a.G + g;
}

// bad lengths and row starts, by one warp for all
__device__ __forceinline__ void report(const WinArgs &a) {
  for (int b = threadIdx.x & 31; b < a.batch; b += 32) {
    const int s = __ldg(a.q_starts + b), e = __ldg(a.q_starts + b + 1);
    const int L = __ldg(a.seq_lens + b);
    if (s < 0 || e < s || e > a.n_tokens)
      set_status(a.status, LOCKS_DEV_BAD_ROWS);
    if (L < 0 || L > a.max_pages * kPage)
      set_status(a.status, LOCKS_DEV_BAD_SEQ_LEN);
  }
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t *>(&v);
}

// What a CTA works on at a time: rows of a (sequence, KV head), the row tiles of
// them (bits), and a range of their tiles.
struct WinUnit {
  WinRows r;
  int id, live, h, split, j0, n, mask, pass;
  int again;  // row tiles to be gone over once more
};

struct WinShared {
  uint4 answer;  // which unit comes next
  WinUnit unit[2];
  uint32_t tmem, there[4];  // which pages of tile j are there, at j & 3
  int dead;
  uint32_t moved;  // when the CTA was last seen to move (win_wait)
  float other[2][2][kWinRows];  // what the halves of a row tell each other
  // of a unit's place; of a row tile; of a buffer; of `there`
  uint64_t unit_full[2], unit_free[2];
  uint64_t q_full[2], q_free[2], qk_done[2], p_full[2], o_done[2], o_free[2];
  uint64_t full[kWinStages], free[kWinStages], info[4];
  uint64_t answered, drain;
};

static_assert(sizeof(WinShared) <= kWinHeader, "shared memory");

// Time on an SM in 2^16 cycles, and the CTA's sign that it moves.
__device__ __forceinline__ uint32_t win_time() {
  return (uint32_t)(clock64() >> 16);
}
__device__ __forceinline__ void win_moves(WinShared &sh) {
  *(volatile uint32_t *)&sh.moved = win_time();
}

// False when the wait gave up, or some other thread's did.  The copies' warp, whose
// waits end with the tiles and with the units before, gives up after some time in
// which no tile was taken up in the plain way either.  The others may wait for as
// long as a unit takes, whose tiles are not theirs or in that way; they leave it to
// the copies' warp, which has a wait of its own until the last unit's end, and to a
// limit beyond any unit (2^30 tokens in the plain way take some 2^43 cycles).  (The
// same look at `moved` in the softmax's waits: eight ragged prompts 137 us instead
// of 129.)
constexpr long long kWinUnitCycles = 1LL << 45;
template <bool COPIES = false>
__device__ __forceinline__ bool win_wait(WinShared &sh, uint64_t *bar,
                                         uint32_t phase) {
  if (mbar_try_wait(bar, phase)) return true;
  const long long t0 = clock64();
  while (!*(volatile int *)&sh.dead) {
    if (mbar_try_wait(bar, phase)) return true;
    const long long t = clock64();
    // (a move may be later than the clock that was read)
    if (COPIES ? t - t0 > kQWaitCycles &&
                     (int)((uint32_t)(t >> 16) -
                           *(volatile uint32_t *)&sh.moved) >
                         (int)(kQWaitCycles >> 16)
               : t - t0 > kWinUnitCycles) {
      *(volatile int *)&sh.dead = 1;
      break;
    }
  }
  return false;
}

// The sums over a warp of kPlainTokens numbers a lane: that of x[i] in the lanes
// whose upper bits are i.
constexpr int kPlainTokens = 8;
__device__ __forceinline__ float sum_of_each(float (&x)[kPlainTokens]) {
  const int lane = threadIdx.x & 31;
  constexpr int kSame = 32 / kPlainTokens;  // lanes that end with the same sum
#pragma unroll
  for (int n = kPlainTokens / 2; n; n >>= 1) {  // n sums each
    const bool up = lane & kSame * n;
#pragma unroll
    for (int i = 0; i < n; ++i) {
      const float other =
          __shfl_xor_sync(0xffffffffu, up ? x[i] : x[i + n], kSame * n);
      x[i] = (up ? x[i + n] : x[i]) + other;
    }
  }
#pragma unroll
  for (int d = kSame / 2; d; d >>= 1)
    x[0] += __shfl_xor_sync(0xffffffffu, x[0], d);
  return x[0];
}

// A row tile's rows over a unit's tiles in the plain way, a row to a warp, lane l
// dims 4l .. 4l + 3, kPlainTokens tokens at a time: tokens that a row does not see
// are not touched for it.  For 128 rows 2.0 us a token (65536 tokens 130 ms), 3.2
// where keys and values come from memory (1M tokens 3.4 s), bound by the latency of
// what eight warps load and exchange; a token at a time took 10.7.
__device__ __noinline__ void plain_rows(const WinArgs &a, WinShared &sh, int u,
                                        int tile) {
  // (read where it is, again and again: the caller keeps its registers)
  const volatile WinUnit &un = sh.unit[u & 1];
  const int lane = threadIdx.x & 31;
  constexpr int kSame = 32 / kPlainTokens;
  int i = tile * tile_tokens(a.G) * a.G + (threadIdx.x >> 5 & 7);
  for (; i < min((tile + 1) * tile_tokens(a.G), un.r.tokens) * a.G; i += 8) {
    const int p = un.r.p0 + i / a.G;
    const size_t row = (size_t)(un.r.q0 + i / a.G) * (a.h_kv * a.G) +
                       un.h * a.G + i % a.G;
    const uint2 q = reinterpret_cast<const uint2 *>(a.q + row * kDim)[lane];
    // l: of the tokens whose number mod kPlainTokens is lane / kSame
    float m = -INFINITY, l = 0.f, o[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
    for (int j = un.j0; j < un.j0 + un.n; ++j) {
      if (lane == 0) win_moves(sh);
      const int first = (j < un.r.head ? j : un.r.from + j - un.r.head) * kWinTile;
      const int end = min(p + 1, first + kWinTile);
      int ids = -1;  // of the tile's pages, a lane each
      if (lane < kWinPages && first + lane * kPage < end)
        ids = __ldg(a.pt + (size_t)un.r.b * a.max_pages + first / kPage + lane);
#pragma unroll 1
      for (int t0 = first; t0 < end; t0 += kPlainTokens) {
        const int ph =
            __shfl_sync(0xffffffffu, ids, (t0 - first) / kPage);
        if (ph < 0 || ph >= a.num_phys) continue;
        auto sees = [&](int t) -> bool {
          return t <= p && (t < a.sinks || t > p - a.window);
        };
        const bool my_token = sees(t0 + lane / kSame);
        const uint32_t seen = __ballot_sync(0xffffffffu, my_token);
        if (seen == 0) continue;
        const size_t at =
            ((((size_t)ph * a.h_kv + un.h) * kPage + t0 % kPage) * kDim) / 4 +
            lane;
        uint2 v[kPlainTokens];
        auto load = [&](const __nv_bfloat16 *cache) {
          const uint2 *from = reinterpret_cast<const uint2 *>(cache) + at;
#pragma unroll
          for (int u = 0; u < kPlainTokens; ++u)
            v[u] = seen >> kSame * u & 1 ? from[u * (kDim / 4)]
                                         : make_uint2(0u, 0u);
        };
        load(a.k);
        float part[kPlainTokens];
#pragma unroll
        for (int u = 0; u < kPlainTokens; ++u)
          part[u] = bf16_lo(q.x) * bf16_lo(v[u].x) +
                    bf16_hi(q.x) * bf16_hi(v[u].x) +
                    bf16_lo(q.y) * bf16_lo(v[u].y) +
                    bf16_hi(q.y) * bf16_hi(v[u].y);
        asm volatile("" ::: "memory");
        load(a.v);  // under the sums and exponentials
        float x = sum_of_each(part);
        if (!my_token) x = -INFINITY;
        float top = fmaxf(m, x);
#pragma unroll
        for (int d = kSame; d < 32; d <<= 1)
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
        const float ref = top == -INFINITY ? 0.f : top;
        const float c = exp2f((m - ref) * kWinScale);
        const float weight = exp2f((x - ref) * kWinScale);
        m = top;
        l = l * c + weight;
#pragma unroll
        for (int d = 0; d < 4; ++d) o[d] *= c;
#pragma unroll
        for (int u = 0; u < kPlainTokens; ++u) {
          const float wu = __shfl_sync(0xffffffffu, weight, kSame * u);
          o[0] += wu * bf16_lo(v[u].x);
          o[1] += wu * bf16_hi(v[u].x);
          o[2] += wu * bf16_lo(v[u].y);
          o[3] += wu * bf16_hi(v[u].y);
        }
      }
    }
#pragma unroll
    for (int d = kSame; d < 32; d <<= 1)
      l += __shfl_xor_sync(0xffffffffu, l, d);
    if (a.splits > 1) {
      const size_t part = (size_t)un.split * a.n_tokens * a.h_kv * a.G + row;
      reinterpret_cast<float4 *>(a.o_part + part * kDim)[lane] =
          make_float4(o[0], o[1], o[2], o[3]);
      if (lane == 0) a.ml_part[part] = make_float2(m * kWinScale, l);
      continue;
    }
    const float inv = l != 0.f ? 1.f / l : 0.f;
    reinterpret_cast<uint2 *>(a.o + row * kDim)[lane] =
        make_uint2(pack_bf16(o[0] * inv, o[1] * inv),
                   pack_bf16(o[2] * inv, o[3] * inv));
    if (lane == 0)
      a.lse[row] =
          l != 0.f ? (m * kWinScale + log2f(l)) * kWinLn2 : -INFINITY;
  }
}

// A page's 16 rows of one head, 4 KB, to [8-row group][64 dims][row][128 bytes]:
// group `row8` of a cache and the next.
__device__ __forceinline__ void copy_page(uint32_t to, const CUtensorMap *map,
                                          int row8, uint64_t *bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile"
      ".mbarrier::complete_tx::bytes [%0], [%1, {%2, %2, %2, %3}], [%4];\n" ::
          "r"(to),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(row8),
      "r"(smem_u32(bar))
      : "memory");
}
// 64 dims from dim x of a row tile's query, heads from `head`, tokens from `t`
__device__ __forceinline__ void copy_query(uint32_t to, const CUtensorMap *map,
                                           int x, int head, int t,
                                           uint64_t *bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile"
      ".mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];\n" ::"r"(
          to),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(head), "r"(t),
      "r"(smem_u32(bar))
      : "memory");
}

// byte offset of 16-byte chunk c (0..15, 8 numbers each) of row r: rows of 128
// bytes, chunks swizzled by the row; 8-row groups of a tile of keys or values
// hold both blocks of 64 dims, a query's blocks lie one after the other
__device__ __forceinline__ uint32_t kv_at(int r, int c) {
  return (uint32_t)((r >> 3) * 2048 + (c >> 3) * 1024 + (r & 7) * 128 +
                    (((c & 7) ^ (r & 7)) << 4));
}
__device__ __forceinline__ uint32_t q_at(int r, int c) {
  return (uint32_t)((c >> 3) * kWinQHalf + r * 128 +
                    (((c & 7) ^ (r & 7)) << 4));
}

// 32 bytes: a whole memory sector where addresses allow it (`wide`; such a store
// to another address is a fault), else 16 and 16
__device__ __forceinline__ void store32(void *to, const uint32_t *w,
                                        bool wide) {
  if (wide)
    asm volatile(
        "st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};\n" ::"l"(to),
        "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]),
        "r"(w[6]), "r"(w[7])
        : "memory");
  else
    for (int i = 0; i < 2; ++i)
      static_cast<uint4 *>(to)[i] =
          make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
}

// Whether the values of a page of a unit's tile j take part in its product: of
// those that are there, and of its very first, which begins the sums.
__device__ __forceinline__ bool takes_part(uint32_t there, int j, int page) {
  return there >> page & 1 || (j == 0 && page == 0);
}

// whether any of two bf16 numbers in each word is not finite
__device__ __forceinline__ bool not_finite(uint4 v) {
  auto bad = [](uint32_t x) -> uint32_t {
    return ((x & 0x7f807f80u) + 0x00800080u) & 0x80008000u;
  };
  return (bad(v.x) | bad(v.y) | bad(v.z) | bad(v.w)) != 0;
}

// The next unit, taken from those that no CTA has been started for: the answer
// comes to sh.answer.
__device__ __forceinline__ void ask(WinShared &sh) {
  mbar_arrive_tx(&sh.answered, 16);
  asm volatile(
      "clusterlaunchcontrol.try_cancel.async.shared::cta"
      ".mbarrier::complete_tx::bytes.b128 [%0], [%1];\n" ::"r"(
          smem_u32(&sh.answer)),
      "r"(smem_u32(&sh.answered))
      : "memory");
}
// its number, -1: there is none
__device__ __forceinline__ int answer(WinShared &sh) {
  uint32_t id, some;
  asm volatile(
      "{\n .reg .b128 x;\n .reg .pred p;\n ld.shared.b128 x, [%2];\n"
      " clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, x;\n"
      " selp.u32 %1, 1, 0, p;\n mov.u32 %0, 0;\n"
      " @p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %0, "
      "x;\n}\n"
      : "=r"(id), "=r"(some)
      : "r"(smem_u32(&sh.answer))
      : "memory");
  return some ? (int)id : -1;
}

__global__ void __launch_bounds__(kWinThreads, 1)
    window_kernel(const WinArgs a, const __grid_constant__ CUtensorMap q_map,
                  const __grid_constant__ CUtensorMap k_map,
                  const __grid_constant__ CUtensorMap v_map) {
  extern __shared__ __align__(1024) uint8_t win_smem[];
  WinShared &sh = *reinterpret_cast<WinShared *>(win_smem);
  const int tid = threadIdx.x, lane = tid & 31;
  // the same for all of a warp, and known to be
  const int wid = __shfl_sync(0xffffffffu, tid >> 5, 0);
  const uint32_t q_s = smem_u32(win_smem) + kWinHeader;
  const uint32_t ring_s = q_s + 2 * kWinBuffer;
  if (wid == kWinProducts && lane == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(sh.unit_full + i, 1);
      mbar_init(sh.unit_free + i, 17);
      mbar_init(sh.q_full + i, 1);
      mbar_init(sh.q_free + i, 1);
      mbar_init(sh.qk_done + i, 1);
      mbar_init(sh.p_full + i, 8);
      mbar_init(sh.o_done + i, 1);
      mbar_init(sh.o_free + i, 8);
    }
    for (int i = 0; i < kWinStages; ++i) {
      mbar_init(sh.full + i, 1);
      mbar_init(sh.free + i, 1);
    }
    for (int i = 0; i < 4; ++i) mbar_init(sh.info + i, 1);
    mbar_init(&sh.answered, 1);
    mbar_init(&sh.drain, 1);
    sh.dead = 0;
    win_moves(sh);
    fence_mbar_init();
  }
  __syncwarp();
  // Tensor memory is taken after the kernels before this one have ended, so that
  // no kernel that starts under another's end holds columns which that waits for.
  pdl_wait();
  if (wid == kWinProducts)
    asm volatile(
        "tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;\n"
        " tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;\n" ::"r"(
            smem_u32(&sh.tmem))
        : "memory");
  tm_fence_before();
  __syncthreads();
  tm_fence_after();
  // after the wait: a kernel that starts here has all before this one done
  pdl_trigger();
  // columns: scores of the two row tiles, then their sums
  const uint32_t tm = sh.tmem;
  const int T = tile_tokens(a.G);
  auto unit_full = [&](int u) {
    return win_wait(sh, sh.unit_full + (u & 1), u >> 1 & 1);
  };

  // A softmax warp: row tile, half of the columns, and the thread's row.
  auto do_softmax = [&]() {
    const int tile = wid >> 3, half = wid >> 2 & 1;
    const int mine = (wid & 3) * 32 + lane;
    const int my_token = tile * T + mine / a.G, my_head = mine % a.G;
    const uint32_t lanes = (uint32_t)((wid & 3) * 32) << 16;
    const uint32_t s_at = tm + tile * 128 + 64 * half + lanes;
    const uint32_t o_at = s_at + 256;
    // whether any thread of the row tile's warps says so
    auto any_of_tile = [&](bool x) -> bool {
      uint32_t r2;
      asm volatile(
          "{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n"
          " barrier.cta.red.or.pred q, %2, 256, p;\n selp.u32 %0, 1, 0, q;\n}\n"
          : "=r"(r2)
          : "r"((uint32_t)x), "r"(9 + tile)
          : "memory");
      return r2 != 0;
    };
    // The other half's x.  (It has been read there before the next one is
    // written: between two of these calls lies a product that wants both
    // halves' weights, or a barrier of the row tile's warps.)
    auto others = [&](float x) -> float {
      sh.other[tile][half][mine] = x;
      asm volatile("barrier.cta.sync %0, 64;\n" ::"r"(1 + 4 * tile + (wid & 3))
                   : "memory");
      return *(volatile float *)&sh.other[tile][half ^ 1][mine];
    };
    // tiles so far: of all units, of those with this row tile, and their number
    int all = 0, steps = 0, units = 0;
    for (int u = 0;; ++u) {
      bool ok = unit_full(u);
      if (any_of_tile(!ok)) break;
      const WinUnit &un = sh.unit[u & 1];
      if (!un.live) break;
      const WinRows &r = un.r;
      const int n = un.n, j0 = un.j0, pass = un.pass;
      if (!(un.mask >> tile & 1)) {
        __syncwarp();
        if (lane == 0) mbar_arrive(sh.unit_free + (u & 1));
        all += n;
        continue;
      }
      auto in = [&]() -> bool {  // whether the row is there
        return mine < T * a.G && my_token < r.tokens;
      };
      // A row's reference, the same in both halves, is its first tile's largest
      // score; rows that are not there want none.  Should weights outgrow it
      // beyond all measure (2^64), the unit comes once more, with the reference
      // that they ask for.  `l`: the sum of this half's weights.
      float m = in() ? -INFINITY : 0.f, l = 0.f, next = -INFINITY;
      if (in() && pass > 0) {
        const int at = out_row(a, r, un.h, my_token, my_head);
        m = a.splits > 1 ? __ldcg(&a.ml_part[(size_t)un.split * a.n_tokens *
                                                 a.h_kv * a.G +
                                             at].x)
                         : __ldcg(a.lse + at);
      }
      // (Row starts that descend can give a row to two units; its halves have
      // to agree all the same, since they meet at barriers.)
      if (pass > 0) {
        m = fmaxf(m, others(m));
        any_of_tile(false);
      }
      // Beyond 2^24 a reference and a score's product with the scale differ by
      // more than the numbers nearby do: those rows go the plain way, as those
      // that a value that is no number could reach unseen.
      // (m is 0 where there is no row)
      bool bad = fabsf(m) > kWinLargest && m > -INFINITY;
      uint32_t seen[2];  // tokens of a tile's half that the row sees
      bool whole = true;
      // Weights 2^(x scale - m) of 32 scores, rounded once (equal scores have
      // equal weights), over the scores of columns that have been read.
      auto weigh = [&](const uint32_t (&s)[32], int c) {
        const float ref = m == -INFINITY ? 0.f : -m;
        const uint64_t rr = pack2(ref, ref), ff = pack2(kWinScale, kWinScale);
        uint64_t sum[2] = {0, 0};
        uint32_t w[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const float2 y =
              unpack2(fma2(pack2(s[2 * i], s[2 * i + 1]), ff, rr));
          const float e0 = ex2_fast(y.x), e1 = ex2_fast(y.y);
          sum[i & 1] = add2(sum[i & 1], pack2(e0, e1));
          w[i] = pack_bf16(e0, e1);
        }
        const float2 t2 = unpack2(add2(sum[0], sum[1]));
        const float t = t2.x + t2.y;
        l += t;
        // (32 weights' sum is near their largest; beyond fp32's range, as far
        // on as that goes)
        if (t > kWinMost)
          next = fmaxf(next, m + (t < INFINITY ? rintf(lg2_fast(t)) : 120.f));
        tm_st16(s_at + 16 * c, w);
      };
#pragma unroll 1
      for (int j = 0; j < n; ++j) {
        // (after a wait that gave up nothing is right, but all goes on to the
        // unit's end, so that all come to the same barriers)
        const int ja = all + j;
        ok = win_wait(sh, sh.info + (ja & 3), ja >> 2 & 1) && ok;
        const uint32_t there = sh.there[ja & 3];
        const int tl = r.tile(j0 + j);
        whole = there == (1u << kWinPages) - 1 && r.whole(a, tl);
        // with S(j) all products before it, among them O(j - 1), are done
        ok = win_wait(sh, sh.qk_done + tile, (steps + j) & 1) && ok;
        tm_fence_after();
        if (!whole || __any_sync(0xffffffffu, m == -INFINITY)) {
          // tokens [from, to] and those below `first` are seen
          const int t0 = tl * kWinTile;
          const int p = r.p0 + my_token;
          const int to = p - t0, from = max(p, -1) - a.window + 1 - t0;
          const int first = min(a.sinks - t0, to + 1);
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const int at = 2 * half + c;
            auto below = [at](int x) -> uint32_t {  // bits of tokens before x
              x = max(0, min(x - 32 * at, 32));
              return x == 32 ? 0xffffffffu : (1u << x) - 1;
            };
            seen[c] = (below(to + 1) & ~below(from)) | below(first);
            const uint32_t pages = there >> (2 * at);
            if (!(pages & 1)) seen[c] &= 0xffff0000u;
            if (!(pages & 2)) seen[c] &= 0x0000ffffu;
          }
          if (!whole) {
            // Half a value row to a thread (of either row tile's: what the
            // other does is the same): one that no row sees is cleared, in the
            // pages that take part, one that some rows see is looked at.
            const int sv = 2 * ja + 1;
            ok = win_wait(sh, sh.full + sv % kWinStages, sv / kWinStages & 1) &&
                 ok;
            const uint32_t v_at = ring_s + sv % kWinStages * kWinBuffer;
            if (!(there >> (mine / kPage) & 1) || !r.sees(a, t0 + mine)) {
              if (takes_part(there, j, mine / kPage)) {
#pragma unroll 4
                for (int c = 0; c < 8; ++c)
                  st_shared_v4(v_at + kv_at(mine, 8 * half + c),
                               make_uint4(0u, 0u, 0u, 0u));
              }
            } else if (!r.all_see(a, t0 + mine)) {
#pragma unroll 4
              for (int c = 0; c < 8; ++c)
                bad |= not_finite(lds128(v_at + kv_at(mine, 8 * half + c)));
            }
            fence_to_async();
            __syncwarp();
          }
          // rows that have seen nothing so far: their first scores' largest
          if (__any_sync(0xffffffffu, m == -INFINITY)) {
            float top = -INFINITY;
#pragma unroll 1
            for (int c = 0; c < 2; ++c) {
              uint32_t s[32];
              tm_ld32(s, s_at + 32 * c);
              tm_wait_ld();
              const uint32_t bits = c ? seen[1] : seen[0];
#pragma unroll
              for (int i = 0; i < 32; ++i)
                if (bits >> i & 1) top = fmaxf(top, __uint_as_float(s[i]));
            }
            top *= kWinScale;
            const float both = fmaxf(top, others(top));
            if (m == -INFINITY) {
              m = both;
              bad |= fabsf(m) > kWinLargest && m > -INFINITY;
            }
          }
          uint32_t s0[32], s1[32];
          tm_ld32(s0, s_at);
          tm_wait_ld();
          tm_ld32(s1, s_at + 32);
#pragma unroll
          for (int i = 0; i < 32; ++i)
            if (!(seen[0] >> i & 1)) s0[i] = 0xff800000u;
          weigh(s0, 0);
          tm_wait_ld();
#pragma unroll
          for (int i = 0; i < 32; ++i)
            if (!(seen[1] >> i & 1)) s1[i] = 0xff800000u;
          weigh(s1, 1);
        } else {
          uint32_t s0[32], s1[32];
          tm_ld32(s0, s_at);
          tm_wait_ld();
          tm_ld32(s1, s_at + 32);
          weigh(s0, 0);
          tm_wait_ld();
          weigh(s1, 1);
        }
        tm_wait_st();
        tm_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(sh.p_full + tile);
      }
      all += n;
      steps += n;
      // ------------------------------------------------------------- output
      const int my_row = in() ? out_row(a, r, un.h, my_token, my_head) : -1;
      const size_t split0 = (size_t)un.split * a.n_tokens * a.h_kv * a.G;
      if (n > 0) ok = win_wait(sh, sh.o_done + tile, units & 1) && ok;
      tm_fence_after();
      l += others(l);  // (after products that want both halves' weights)
      const bool none = n == 0 || l == 0.f;
      const float inv = none ? 0.f : 1.f / l;
      bool large = false;
#pragma unroll 1
      for (int c = 0; c < 4; ++c) {  // 16 dims
        uint32_t o[16];
        if (n > 0) {
          tm_ld16(o, o_at + 16 * c);
          tm_wait_ld();
          if (c == 3) {  // the next unit's products may come
            tm_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(sh.o_free + tile);
          }
        }
        float most = 0.f;  // (NaN has no part: the weights' sum shows it)
#pragma unroll
        for (int i = 0; i < 16; i += 2) {
          if (none) o[i] = o[i + 1] = 0u;
          most = max3(most, fabsf(__uint_as_float(o[i])),
                      fabsf(__uint_as_float(o[i + 1])));
        }
        large |= most == INFINITY;
        if (my_row >= 0) {
          const int at = 64 * half + 16 * c;
          if (a.splits > 1) {
            float *to = a.o_part + (split0 + my_row) * kDim + at;
            store32(to, o, a.wide);
            store32(to + 8, o + 8, a.wide);
          } else {
            uint32_t w[8];
#pragma unroll
            for (int i = 0; i < 8; ++i)
              w[i] = pack_bf16(__uint_as_float(o[2 * i]) * inv,
                               __uint_as_float(o[2 * i + 1]) * inv);
            store32(a.o + (size_t)my_row * kDim + at, w, a.wide);
          }
        }
        __syncwarp();
      }
      if (my_row >= 0 && half == 0) {
        if (a.splits > 1)
          a.ml_part[split0 + my_row] = make_float2(m, none ? 0.f : l);
        else
          a.lse[my_row] = none ? -INFINITY : (m + log2f(l)) * kWinLn2;
      }
      if (n > 0) ++units;
      // (weights up to 2^64 may have made large values' sums infinite)
      const bool again = my_row >= 0 && next > -INFINITY;
      // (a value that is no number has been met by the thread of its place, which
      // may have no row)
      bad |= (my_row >= 0 && large && l < INFINITY) ||
             (again && pass == kWinPasses);
      if (any_of_tile(bad || again || !ok)) {
        if (any_of_tile(!ok)) break;
        if (any_of_tile(bad)) {
          plain_rows(a, sh, u, tile);
        } else {
          // (a row that asks for nothing keeps the reference that it has)
          const float both = fmaxf(fmaxf(m, next), others(next));
          if (my_row >= 0 && half == 0) {
            if (a.splits > 1)
              a.ml_part[split0 + my_row].x = both;
            else
              a.lse[my_row] = both;
          }
          if (mine == 0 && half == 0) atomicOr(&sh.unit[u & 1].again, 1 << tile);
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(sh.unit_free + (u & 1));
    }
  };

  // One thread issues all products: between them it has no time for its warp
  // (with votes and a new election each, 440 us for 8192 tokens instead of 355).
  auto do_products = [&]() {
    const uint64_t dq = mat_desc(q_s, 16), dk = mat_desc(ring_s, 16, 2048);
    const uint64_t dv = mat_desc(ring_s, 1024, 2048);
    int all = 0, steps[2] = {0, 0}, units[2] = {0, 0};
    for (int u = 0;; ++u) {
      if (!unit_full(u)) return;
      const WinUnit &un = sh.unit[u & 1];
      const int live = un.live, n = un.n, mask = un.mask;
      mbar_arrive(sh.unit_free + (u & 1));
      if (!live) return;
      if (n == 0) continue;
      const int last = mask >> 1;  // the last row tile
      // S(j) of row tile t, and after the last one its keys may go, after the
      // last tile's its query
      auto scores = [&](int t, int j) {
        const int b = 2 * (all + j) % kWinStages;
        const uint64_t q = dq + t * (kWinBuffer >> 4);
        const uint64_t k = dk + b * (kWinBuffer >> 4);
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)
          mma_ss_f16(tm + t * 128,
                     q + (kk >> 2) * (kWinQHalf >> 4) + (kk & 3) * 2,
                     k + (kk >> 2) * (1024 >> 4) + (kk & 3) * 2, kWinDescS,
                     kk > 0);
        mma_commit(sh.qk_done + t);
        if (t == last) mma_commit(sh.free + b);
        if (j == n - 1) mma_commit(sh.q_free + t);
      };
      // O += W V, and after the last one its values may go
      auto weighted = [&](int t, int j) {
        const int b = (2 * (all + j) + 1) % kWinStages;
        const uint64_t v = dv + b * (kWinBuffer >> 4);
        // (the softmax has seen this before its weights)
        const uint32_t there = *(volatile uint32_t *)&sh.there[(all + j) & 3];
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)  // a page each
          if (takes_part(there, j, kk))
            mma_ts(tm + 256 + t * 128,
                   tm + t * 128 + (kk >> 2) * 64 + (kk & 3) * 8,
                   v + kk * (kWinPage >> 4), kWinDescO, j > 0 || kk > 0);
        if (t == last) mma_commit(sh.free + b);
        if (j == n - 1) mma_commit(sh.o_done + t);
      };
      auto wait_full = [&](int s) {
        return win_wait(sh, sh.full + s % kWinStages, s / kWinStages & 1);
      };
      for (int j = -1; j < n; ++j)
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          if (!(mask >> t & 1)) continue;
          if (j >= 0) {
            if (!wait_full(2 * (all + j) + 1) ||
                !win_wait(sh, sh.p_full + t, (steps[t] + j) & 1))
              return;
            // the unit before's sums have been read
            if (j == 0 && units[t] > 0 &&
                !win_wait(sh, sh.o_free + t, (units[t] - 1) & 1))
              return;
            tm_fence_after();
            weighted(t, j);
          }
          if (j + 1 < n) {
            if (!wait_full(2 * (all + j + 1)) ||
                (j < 0 && !win_wait(sh, sh.q_full + t, units[t] & 1)))
              return;
            tm_fence_after();
            scores(t, j + 1);
          }
        }
      all += n;
#pragma unroll
      for (int t = 0; t < 2; ++t)
        if (mask >> t & 1) {
          steps[t] += n;
          ++units[t];
        }
    }
  };

  auto do_copies = [&]() {
    constexpr int64_t kNone = 0x7fffffffffffffffLL;
    int s = 0, all = 0, queries[2] = {0, 0};
    // units to be gone over again (id, row tiles, pass); whether more may come
    int redo[2][3], redos = 0;
    bool first = true, more = true, asked = false, ok = true;
    bool reports = false;  // the warp that has the first unit, whosever it was
    int asks = 0;
    // a unit's place is free; what it wants again
    auto collect = [&](int u) {
      ok = win_wait<true>(sh, sh.unit_free + (u & 1), u >> 1 & 1);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) return;
      WinUnit &un = sh.unit[u & 1];
      const int again = *(volatile int *)&un.again;
      __syncwarp();
      if (again) {
        redo[redos][0] = un.id;
        redo[redos][1] = again;
        redo[redos++][2] = un.pass + 1;
        if (lane == 0) un.again = 0;
      }
      __syncwarp();
    };
    for (int u = 0; ok;) {
      if (u >= 2) collect(u - 2);
      int id = -1, pass = 0, mask = 0;
      WinRows r = {};
      while (ok) {
        if (redos > 0) {
          id = redo[--redos][0];
          mask = redo[redos][1];
          pass = redo[redos][2];
        } else if (first) {
          id = blockIdx.x;
          first = false;
        } else if (more) {
          if (!asked && lane == 0) ask(sh);
          asked = false;
          ok = win_wait<true>(sh, &sh.answered, asks++ & 1);
          ok = __all_sync(0xffffffffu, ok);
          id = answer(sh);
          // (read before the next answer is written there)
          fence_to_async();
          __syncwarp();
          more = id >= 0;
        }
        if (id < 0 && u >= 1 && ok) {
          // the unit before this one may still come again
          collect(u - 1);
          if (redos > 0) continue;
        }
        if (id < 0) break;
        reports |= id == 0;
        // the longest rows, a sequence's last, first
        if (find_rows(a, a.slots - 1 - id / a.splits / a.h_kv, r)) break;
        id = -1;
      }
      if (!ok) break;
      WinUnit un;
      un.r = r;
      un.id = id;
      un.live = id >= 0;
      un.split = id % a.splits;
      un.h = id / a.splits % a.h_kv;
      un.j0 = un.split * r.tiles / a.splits;  // (at most 2^23 tiles, 64 ranges)
      un.n = (un.split + 1) * r.tiles / a.splits - un.j0;
      un.mask = mask ? mask : r.tokens > T ? 3 : 1;
      un.pass = pass;
      un.again = 0;
      if (lane == 0) {
        sh.unit[u & 1] = un;
        mbar_arrive(sh.unit_full + (u & 1));
      }
      __syncwarp();
      ++u;
      if (!un.live) break;
      if (more && !asked) {  // the answer comes meanwhile
        if (lane == 0) ask(sh);
        asked = true;
      }
      const int32_t *table = a.pt + (size_t)r.b * a.max_pages;
      // physical page of the lane's page of tile j, 2^63 - 1 where none is seen
      auto page = [&](int j) -> int64_t {
        if (j >= un.n || lane >= kWinPages) return kNone;
        const int pg = r.tile(un.j0 + j) * kWinPages + lane;
        return r.sees_page(a, pg) ? __ldg(table + pg) : kNone;
      };
      int64_t ahead = page(0);
      for (int j = 0; j < un.n && ok; ++j) {
        const int64_t ph = ahead;
        ahead = page(j + 1);
        const bool good = ph >= 0 && ph < a.num_phys;
        if (!good && ph != kNone) set_status(a.status, LOCKS_DEV_BAD_PAGE_ID);
        const uint32_t there = __ballot_sync(0xffffffffu, good);
        // (in the place of the tile four before: its softmax is done, since
        // the keys after it, whose buffer the tile before this one got, are
        // behind its weights)
        if (lane == 0) {
          sh.there[(all + j) & 3] = there;
          mbar_arrive(sh.info + ((all + j) & 3));
        }
#pragma unroll 1
        for (int kv = 0; kv < 2; ++kv, ++s) {
          const int b = s % kWinStages;
          if (s >= kWinStages)
            ok = win_wait<true>(sh, sh.free + b, (s / kWinStages - 1) & 1);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          if (lane == 0) mbar_arrive_tx(sh.full + b, __popc(there) * kWinPage);
          __syncwarp();
          if (good)
            copy_page(ring_s + b * kWinBuffer + lane * kWinPage,
                      kv ? &v_map : &k_map, 2 * ((int)ph * a.h_kv + un.h),
                      sh.full + b);
          __syncwarp();
          if (j > 0 || kv > 0) continue;
          // the query, a lane to a row tile's, in the place of the unit
          // before's
          for (int t = 0; t < 2; ++t) {
            if (!(un.mask >> t & 1)) continue;
            if (queries[t] > 0)
              ok = win_wait<true>(sh, sh.q_free + t, (queries[t] - 1) & 1);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            ++queries[t];
            if (lane == 0) {
              mbar_arrive_tx(sh.q_full + t, 2 * T * a.G * 128);
              for (int i = 0; i < 2; ++i)
                copy_query(q_s + t * kWinBuffer + i * kWinQHalf, &q_map, 64 * i,
                           un.h * a.G, r.q0 + t * T, sh.q_full + t);
            }
            __syncwarp();
          }
        }
      }
      all += un.n;
    }
    if (reports) report(a);
    // what is in flight ends before the CTA does
    if (asked) q_wait(&sh.answered, asks & 1);
    if (*(volatile int *)&sh.dead) {
      for (int t = 0; t < 2; ++t)
        if (queries[t] > 0) q_wait(sh.q_full + t, (queries[t] - 1) & 1);
      for (int i = max(0, s - kWinStages); i < s; ++i)
        q_wait(sh.full + i % kWinStages, i / kWinStages & 1);
    }
  };

  if (wid < kWinProducts) {
    do_softmax();
  } else if (wid == kWinProducts) {
    if (elect_one()) do_products();
  } else {
    do_copies();
  }
  __syncwarp();
  tm_fence_before();
  __syncthreads();
  if (wid == kWinProducts) {
    // some role's wait gave up: say so, and give what is in flight a last,
    // bounded chance to finish
    if (*(volatile int *)&sh.dead && elect_one()) {
      set_status(a.status, LOCKS_DEV_TIMEOUT);
      mma_commit(&sh.drain);
      q_wait(&sh.drain, 0);
    }
    __syncwarp();
    asm volatile(
        "tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;\n" ::"r"(tm)
        : "memory");
  }
}

// Joins the ranges' partials of a token's heads, a warp to a row, lane l dims
// 4l .. 4l + 3; eight ranges' loads at a time.  (64 tokens behind 2000 take 18 us;
// with a unit's rows to a block, 32 to a warp, one after the other, 75.)
constexpr int kWinMergeWarps = 8;

__global__ void __launch_bounds__(32 * kWinMergeWarps)
    window_merge_kernel(const WinArgs a) {
  pdl_wait();
  const int lane = threadIdx.x & 31, token = blockIdx.x;
  const int h_q = a.h_kv * a.G;
  const int head = blockIdx.y * kWinMergeWarps + (threadIdx.x >> 5);
  if (head >= h_q) return;
  // the sequence that has the token, if there is one
  const int b = last_where(
      a.batch, [&](int x) { return __ldg(a.q_starts + x) <= token; });
  const int begin = __ldg(a.q_starts + b), end = __ldg(a.q_starts + b + 1);
  if (begin < 0 || end > a.n_tokens || token < begin || token >= end) return;
  const size_t all = (size_t)a.n_tokens * h_q;
  const size_t row = (size_t)token * h_q + head;
  constexpr int kAtOnce = 8;  // ranges
  float m = -INFINITY, l = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int s0 = 0; s0 < a.splits; s0 += kAtOnce) {
    float2 ml[kAtOnce];
    float4 v[kAtOnce];
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k) {
      const bool in = s0 + k < a.splits;
      ml[k] = in ? a.ml_part[(s0 + k) * all + row] : make_float2(0.f, 0.f);
      v[k] = in ? reinterpret_cast<const float4 *>(
                      a.o_part + ((s0 + k) * all + row) * kDim)[lane]
                : make_float4(0.f, 0.f, 0.f, 0.f);
    }
    float top = m;
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k)
      if (ml[k].y != 0.f) top = fmaxf(top, ml[k].x);
    const float ref = top == -INFINITY ? 0.f : top;
    const float c = exp2f(m - ref);
    m = top;
    l *= c;
    o.x *= c;
    o.y *= c;
    o.z *= c;
    o.w *= c;
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k) {
      if (ml[k].y == 0.f) continue;  // nothing seen
      const float w = exp2f(ml[k].x - ref);
      l += w * ml[k].y;
      o.x += w * v[k].x;
      o.y += w * v[k].y;
      o.z += w * v[k].z;
      o.w += w * v[k].w;
    }
  }
  const float inv = l != 0.f ? 1.f / l : 0.f;
  reinterpret_cast<uint2 *>(a.o + row * kDim)[lane] = make_uint2(
      pack_bf16(o.x * inv, o.y * inv), pack_bf16(o.z * inv, o.w * inv));
  if (lane == 0) a.lse[row] = l != 0.f ? (m + log2f(l)) * kWinLn2 : -INFINITY;
}

// ---------------------------------------------------------------------------
// launcher
// ---------------------------------------------------------------------------
static bool tensor_map(const void *base, int dims, const cuuint64_t *size,
                       const cuuint64_t *stride, const cuuint32_t *box,
                       CUtensorMap *map) {
  static const auto encode = [] {
    void *f = nullptr;
    cudaDriverEntryPointQueryResult found;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000,
                                         cudaEnableDefault, &found) !=
            cudaSuccess ||
        found != cudaDriverEntryPointSuccess)
      f = nullptr;
    return reinterpret_cast<decltype(&cuTensorMapEncodeTiled)>(f);
  }();
  const cuuint32_t step[4] = {1, 1, 1, 1};
  return encode &&
         encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, dims,
                const_cast<void *>(base), size, stride, box, step,
                CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// A cache as [8-row group][64 dims][row][dim], a box two groups: a page's rows
// of a head in one copy, their groups 2 KB apart and both blocks of dims in
// them (two copies of 2 KB a page took 1.3 times as long as the products).
static bool cache_map(const WinArgs &a, const void *cache, CUtensorMap *map) {
  const cuuint64_t size[4] = {64, 8, 2, (cuuint64_t)a.num_phys * a.h_kv * 2};
  const cuuint64_t stride[3] = {kDim * 2, 128, 8 * kDim * 2};
  const cuuint32_t box[4] = {64, 8, 2, 2};
  return tensor_map(cache, 4, size, stride, box, map);
}

// The query, a box the heads of a group for a row tile's tokens.
static bool query_map(const WinArgs &a, CUtensorMap *map) {
  const cuuint64_t h_q = (cuuint64_t)a.h_kv * a.G;
  const cuuint64_t size[3] = {kDim, h_q, (cuuint64_t)a.n_tokens};
  const cuuint64_t stride[2] = {kDim * 2, h_q * kDim * 2};
  const cuuint32_t box[3] = {64, (cuuint32_t)a.G, (cuuint32_t)tile_tokens(a.G)};
  return tensor_map(a.q, 3, size, stride, box, map);
}

static long long window_slots(int n_tokens, int batch, int G) {
  return (long long)n_tokens / (2 * tile_tokens(G)) + batch;
}

// Most tiles that a CTA's rows can see.
static int window_tiles(int n_tokens, int G, int max_pages, int window,
                        int sinks) {
  const long long rows = 2 * tile_tokens(G);  // tokens of a CTA
  const long long span = (rows < n_tokens ? rows : n_tokens) + (long long)window;
  const long long t = (span + kWinTile - 2) / kWinTile + 1 +
                      ((long long)sinks + kWinTile - 1) / kWinTile;
  const long long top = ((long long)max_pages * kPage + kWinTile - 1) / kWinTile;
  return (int)(t < top ? t : top);
}

// Ranges that the tiles of each unit are cut into: the number with the least
// estimate, in times of a tile (1.4 us), for 152 SMs.  A unit's start and end
// take 3.5 tiles, the kernel that joins ranges 3, and a range's row 1 KB of
// traffic.  (4 drafted tokens of 16 sequences of 32K, 128 units of 257 tiles: one
// range 364 us, 2 to 6 ranges 372-377, 7 334, 8 338, 9 345, 12 358; 64 tokens
// behind 2000, 8 units of 17 tiles: one 33, 3 22, 9 17.8; 1000 tokens behind 8000,
// one KV head of 8 query heads: one 106, 3 49, 4 41, 5 58, since a fifth range
// takes a second round.)  A sequence without rows counts as a unit too, which is far
// off where few of many have some: 4 tokens of one sequence of 32K 35 us in a table
// of one (19 ranges), 65 in a table of 16, 190 of 64, 358 of 128 (one range).
int window_splits(int n_tokens, int batch, int h_kv, int G, int max_pages,
                  int window, int sinks) {
  const long long T2 = 2 * tile_tokens(G);
  const long long least = (n_tokens + T2 - 1) / T2;
  const long long units = (least > batch ? least : batch) * h_kv;
  const int tiles = window_tiles(n_tokens, G, max_pages, window, sinks);
  const long long rows = (long long)n_tokens * h_kv * G;
  int best = 1;
  double cost = 1e30;
  for (int s = 1; s <= kWinSplits && s <= tiles; ++s) {
    if (s > 1 && rows * s > kWinPartRows) break;
    const long long waves = (units * s + 151) / 152;
    const double c = (double)waves * ((tiles + s - 1) / s + 3.5) +
                     (s > 1 ? 3.0 + 1.2e-4 * (double)(rows * s) : 0.0);
    if (c < cost) {
      cost = c;
      best = s;
    }
  }
  return best;
}

// Rows of partials that any call up to these sizes stays within.
size_t window_part_rows(int n_tokens, int h_kv, int G, int max_pages,
                        int window, int sinks) {
  const size_t tiles = window_tiles(n_tokens, G, max_pages, window, sinks);
  const size_t rows = (size_t)n_tokens * h_kv * G *
                      (tiles < kWinSplits ? tiles : kWinSplits);
  return rows < kWinPartRows ? rows : kWinPartRows;
}

cudaError_t launch_window(WinArgs a, cudaStream_t stream) {
  static DeviceFlags done;
  cudaError_t e = once_per_device(done, [] {
    return cudaFuncSetAttribute(
        window_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kWinSmem);
  });
  if (e != cudaSuccess) return e;
  CUtensorMap q_map, k_map, v_map;
  if (!query_map(a, &q_map) || !cache_map(a, a.k, &k_map) ||
      !cache_map(a, a.v, &v_map))
    return cudaErrorInvalidValue;
  a.slots = window_slots(a.n_tokens, a.batch, a.G);
  // what the softmax's warps write to, rows of 256 or 512 bytes
  a.wide = reinterpret_cast<uintptr_t>(
               a.splits > 1 ? static_cast<void *>(a.o_part) : a.o) % 32 == 0;
  const long long base = a.slots * a.h_kv;
  e = launch_pdl(window_kernel, dim3((unsigned)(base * a.splits)),
                 dim3(kWinThreads), kWinSmem, stream, a, q_map, k_map,
                 v_map);
  if (e != cudaSuccess || a.splits == 1) return e;
  const int h_q = a.h_kv * a.G;
  return launch_pdl(window_merge_kernel,
                    dim3((unsigned)a.n_tokens,
                         (unsigned)((h_q + kWinMergeWarps - 1) / kWinMergeWarps)),
                    dim3(32 * kWinMergeWarps), 0, stream, a);
}

}  // namespace locks
