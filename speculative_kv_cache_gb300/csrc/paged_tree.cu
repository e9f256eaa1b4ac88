// Attention of a tree of drafted tokens per request over a paged KV cache.
//
// Mathematics.  Request b has L tokens, the last n of them drafted.  Drafted token t sees key j when j < L - n, or when bit
// j - (L - n) of its mask is set (its ancestors and itself); for each of the G = Hq / Hkv query heads of a key head
//   z_j = scale q . K_j,  o = sum_j e^(z_j) V_j / sum_j e^(z_j)  over the keys it sees,
// in one pass over the tokens: every part keeps a reference m, l = sum 2^(z - m) and o = sum 2^(z - m) V (log2(e) is in
// the scale), and two parts join as m = max(m1, m2), l = sum l_i 2^(m_i - m), o likewise.
//
// What bounds it.  The n G rows of a key head share its keys and values: 4 d n G flop for 4 d bytes, so HBM up to about
// 280 rows and the tensor cores beyond.  Rows are the M = 128 of tcgen05.mma, tokens its N and the second product's K:
//   S[rows][128 tokens] = Q K^T (both in shared memory),  O[rows][d] += P V (P in tensor memory, where S was).
//
// A CTA (one an SM): a warp moves keys with TMA, 128 tokens a tile, through a ring, a warp values through a ring of theirs; a warp
// issues the MMAs; a warp fetches the units' queries; two groups of four warps turn S into P, a row a thread, each with S and
// O columns of its own, so that one works on its logits while the tensor cores work for the other.  Up to 128 rows the
// groups take tiles in turn and join their parts at the end (SPLIT); with more, a unit is 256 rows, and each group has
// 128 of them and every tile (PAIR), which halves what is read.
//
// Precision.  Weights are rounded to the type for the second product.  Fp16 has few exponents: the reference lies 10 (log2) below the
// largest logit that it was set by, so that weights keep their 11 bits down to 2^-24 of the largest, and moves (and O is
// scaled by the factor) only when one is more than 5.75 above that (bf16: 8).  (With 14 and 1, a warp's 32 rows move in one
// tile of three: two trees of 512 rows on 65536 tokens 149 us instead of 137.)  Sums of weights are fp32, unrounded.
//
// What is not attended.  Logits of tokens that a row does not see are left out by bits (the tile's tokens that hold
// anything, the row's mask), whatever they are.  A value of zero weight must not be NaN in an MMA: rows without a token are
// cleared in shared memory, and in drafted rows, which only some see, elements that are not finite; the rows that
// see them get them at the end.
//
// Work split.  As in the attention of one token: all tiles of all units in order, cut in equal shares, one a CTA; a unit in
// several CTAs leaves partials in the workspace (two slots a CTA: the unit it starts with, the unit it ends with), joined in
// order by a second kernel.  No atomics: the result does not depend on timing.
//
// Measured (device time; the copy rate of HBM is 6.75 TB/s; rows: queries of a key head).
//   One request of 131072 tokens, 8 key heads of 128, 537 MB, pages of 64: 86 us with 16 rows (0.92 of the copy rate), 87 with
//   64, 89 with 128, 110 with 256 (PAIR), 192 with 512.  64 rows in pages of 16: 89, of 8: 90.  Heads of 64, 268 MB: 51 us with 64
//   rows, 53 with 128, 92 with 256.
//   32 requests of 64 to 8192 tokens, 1 to 16 drafted, 558 MB, pages of 32: 98 us, 0.84; 4 are the join, of 150 cuts, 6 the plan
//   and the first tile, and without any arithmetic of the softmax the rest takes as long.
//   Two requests of 65536 tokens, 64 drafted, 512 rows, 136 Gflop: 110 us, 1.24 Pflop/s; a tile takes 3100 cycles, of which the
//   products are 2048.  The rest is a group's chain, 1240 cycles for a tile's values and the next one's logits and some 1900 for
//   its weights, which two groups cannot hide in each other altogether: with an eighth of the products 88 us, without
//   exponentials no less than with them.
//   8 drafted tokens on 256, 4 key heads of 64: 7.7 us: a chain of the plan, a page's number, the first tile, its weights.
// Tried and left out: a row in two threads (16 softmax warps), 155 -> 167 us; weights announced in halves, and rings of two keys and
// three values, no gain; tiles in two pieces, whose logits are there ahead, 135 -> 151 (a product of 64 tokens takes as
// long as one of 128, as its queries are read from shared memory again); the page table's entries fetched by the plan, no gain.
#include <cuda_bf16.h>
#include <math.h>

#include "ig_common.cuh"
#include "tc_common.cuh"

namespace ig {
namespace {

constexpr int kTreeMost = 64;  // drafted tokens of a request

struct TreeShape {
  int B, T, T_max, Hq, Hkv, G, page, n_pages, seqs, max_pages;
  float scale2;  // scale * log2(e)
  const int32_t *table, *L, *seq, *first;
  const unsigned long long* masks;
};

struct TreeRequest {
  int f, n, L, s;  // first drafted token in the packed order, their number, all tokens, sequence
};

// Early: read before the kernel has waited for the one before it, so not from an L1 that may hold older numbers.
template <bool Early = false>
__device__ __forceinline__ bool tree_request(const TreeShape& a, int r, TreeRequest& x) {
  auto get = [](const int32_t* p) { return Early ? __ldcg(p) : __ldca(p); };
  x.f = get(a.first + r);
  x.n = get(a.first + r + 1) - x.f;
  x.s = a.seq ? get(a.seq + r) : r;
  x.L = x.s >= 0 && x.s < a.seqs ? get(a.L + x.s) : -1;
  return x.f >= 0 && x.n >= 0 && x.n <= a.T_max && x.f <= a.T - x.n && x.L >= x.n && x.L <= a.max_pages * a.page;
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

template <bool BF>
__device__ __forceinline__ float to_float(uint16_t v) {
  if constexpr (BF) return __uint_as_float((uint32_t)v << 16);
  else return __half2float(__ushort_as_half(v));
}
template <bool BF>
__device__ __forceinline__ uint16_t from_float(float v) {
  if constexpr (BF) return __bfloat16_as_ushort(__float2bfloat16_rn(v));
  else return __half_as_ushort(__float2half_rn(v));
}

constexpr int kTreeTile = 128;                 // tokens of a tile, rows of a block
// Warps 4 .. 11 are the softmax groups, warp w with the rows of quarter w % 4, which also is the quarter of the SM it runs on.  The
// warp of the MMAs, which sets the pace, shares its own with the rows that are there last, as the TMA's nearly does.
constexpr int kTreeThreads = 384;
constexpr int kTreeTmaV = 0, kTreeQueries = 1, kTreeTmaK = 2, kTreeMma = 3, kTreeSoftmax = 4;
constexpr int kMaxTreeCtas = 160;              // upper bound of the grid (sizes the workspace)
constexpr int kTreePartHead = 8;               // a partial: [m, l, -.., o[D]] (o in whole sectors)
constexpr uint32_t kTreeTmem = 512;            // columns: S of either group, then O of either
// Units that could have a CTA each are not cut where the longest has at most kTreeWhole tiles, or where there are enough
// of them to keep HBM busy and the longest is at most kTreeEven tiles above the mean.
constexpr int kTreeWhole = 4;
constexpr int kTreeEven = 3;

// slots of the rings of keys and of values
template <int D>
__host__ __device__ constexpr int tree_k_slots() { return D == 128 ? 3 : 4; }
template <int D>
__host__ __device__ constexpr int tree_v_slots() { return D == 128 ? 2 : 4; }
template <int D>
__host__ __device__ constexpr int tree_slots() { return tree_k_slots<D>() + tree_v_slots<D>(); }
template <int D>
__host__ __device__ constexpr uint32_t tree_slot_bytes() { return kTreeTile * D * 2; }

struct TreeShared {
  // A tile's keys and values are there (by tile, as the groups each see every other tile of SPLIT, and a barrier's phases
  // can be told by their parity only by one that follows them all); a slot of the rings is free.
  uint64_t k_full[8], v_full[8], empty[8];  // (keys' slots, then values')
  uint64_t s_full[2], p_full[2];    // a group's logits are there, its weights are
  uint64_t o_done[2];               // its last product of a unit
  uint64_t q_full[2], q_empty[2];   // queries
  uint64_t half[2], o_free[2];      // a group's part of a unit is there for the other, has been taken
  uint64_t clean[8];                // values that had to be cleared, and that both groups use, are (by their count)
  uint64_t drain;
  uint32_t valid[8][4];             // tokens of a tile that hold anything
  float2 ml[kTreeTile];
  int poison[8];                    // by unit: 1 + its number, if it has drafted values that are not finite
  int scan[kTreeThreads / 32][3];
  uint32_t tmem;
  int start[10];                    // where this CTA's share begins
  int abort;
};

template <int D>
constexpr size_t tree_smem() {
  return 1024 + 2 * tree_slot_bytes<D>() + tree_slots<D>() * tree_slot_bytes<D>() + sizeof(TreeShared);
}
static_assert(tree_smem<128>() <= 232448, "more shared memory than a CTA can have");

// Words of a 128B-swizzled tile's descriptor, but for its address: 64-column halves `lead` bytes apart (read for an MN-major tile, as
// the values are: rows are tokens, the product's K), groups of 8 rows `stride` bytes apart; version 1, SWIZZLE_128B.
__device__ __forceinline__ uint32_t desc_low(uint32_t lead) { return (lead >> 4) << 16; }
__device__ __forceinline__ uint32_t desc_high(uint32_t stride) { return stride >> 4 | 1u << 14 | 2u << 29; }

__device__ __forceinline__ void tm_ld32(uint32_t (&r)[32], uint32_t addr) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]),
        "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]),
        "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(addr));
}
__device__ __forceinline__ void tm_st32(uint32_t addr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
      "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(addr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
      "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]),
      "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]),
      "r"(r[31])
      : "memory");
}
__device__ __forceinline__ void tm_st16(uint32_t addr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(addr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
      "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tm_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ float max3(float x, float y, float z) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(x), "f"(y), "f"(z));
  return r;
}
// A number that is the same in every lane, as one the compiler knows to be so (and may keep in a uniform register).
__device__ __forceinline__ int uniform(int x) { return (int)__reduce_max_sync(0xffffffffu, (unsigned)x); }
__device__ __forceinline__ uint32_t elected() {
  uint32_t y;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(y));
  return y;
}
__device__ __forceinline__ void tree_commit(uint64_t* bar, uint32_t lead) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.u32 p, %1, 0;\n"
      " @p tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}\n" ::"r"(smem_addr(bar)), "r"(lead)
      : "memory");
}
__device__ __forceinline__ void tree_arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_addr(bar)) : "memory");
}

// A bounded wait that ends together with the CTA's other waits; one verdict for the warp.  What is there already costs one look.
__device__ __noinline__ bool tree_wait_on(uint64_t* bar, uint32_t parity, volatile int* abort, uint32_t limit, int* err) {
  bool ok = false;
  for (uint32_t i = 0; i < limit && !*abort && !ok; ++i) ok = mbar_try_wait(bar, parity);
  ok = __all_sync(0xffffffffu, ok);
  if (!ok && (threadIdx.x & 31) == 0 && !atomicExch(const_cast<int*>(abort), 1)) raise_error(err, IG_DEVERR_TIMEOUT);
  return ok;
}
__device__ __forceinline__ bool tree_wait(uint64_t* bar, uint32_t parity, volatile int* abort, uint32_t limit, int* err) {
  if (limit > 0 && __all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
  return tree_wait_on(bar, parity, abort, limit, err);
}

// The units of a CTA's share, in order: of each request its key heads, of each key head its blocks of rows.
struct TreeWalk {
  int RU;        // rows of a unit
  bool whole;    // shares of whole units
  int team, member;  // CTAs that go side by side, one a block of rows (0: one after the other); the block of this one
  int r, left;   // request; tiles (whole units) left
  TreeRequest x;
  int blocks, units, nt, u, tile;  // blocks of rows of a key head, units of the request, tiles of a unit; unit and tile in it

  __device__ bool enter(const TreeShape& a) {
    if (!tree_request(a, r, x) || x.n == 0) return false;
    blocks = team ? 1 : (x.n * a.G + RU - 1) / RU;  // (a walk's own)
    units = blocks * a.Hkv;
    nt = (x.L + kTreeTile - 1) / kTreeTile;
    return true;
  }
  // One thread finds the beginning, and the others take it from shared memory: `off` into request r, which it has entered.
  __device__ void put(int* to, int off) const {
    const int v[10] = {r, x.f, x.n, x.L, x.s, blocks, units, nt, whole ? off : off / nt, whole ? 0 : off % nt};
#pragma unroll
    for (int i = 0; i < 10; ++i) to[i] = v[i];
  }
  __device__ void get(const int* from, int n) {
    r = from[0], x = {from[1], from[2], from[3], from[4]}, blocks = from[5], units = from[6], nt = from[7], u = from[8], tile = from[9];
    left = n;
  }
  __device__ int head() const { return u / blocks; }
  __device__ int block() const { return member + u % blocks; }
  __device__ int run() const { return whole ? nt : min(nt - tile, left); }
  __device__ void next(const TreeShape& a) {
    left -= whole ? 1 : run();
    tile = 0;
    if (left <= 0 || ++u < units) return;
    u = 0;
    do ++r;
    while (r < a.B && !enter(a));
    if (r >= a.B) left = 0;
  }
};

// Bits of the 32 tokens from `off` on (counted from the first drafted one) that a row with this mask sees.
__device__ __forceinline__ uint32_t seen_bits(unsigned long long mask, int off) {
  if (off >= 64) return 0u;
  if (off >= 0) return (uint32_t)(mask >> off);
  if (off <= -32) return ~0u;
  return (uint32_t)(mask << -off) | ((1u << -off) - 1);
}

// 16-bit pairs: whether either is not finite
template <bool BF>
__device__ __forceinline__ uint32_t odd_pair(uint32_t v) {
  return BF ? ((v & 0x7f807f80u) + 0x00800080u) & 0x80008000u : ((v & 0x7c007c00u) + 0x04000400u) & 0x80008000u;
}

template <bool BF>
__device__ __forceinline__ uint32_t pack2(float x, float y) {
  if constexpr (BF) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
    return *reinterpret_cast<const uint32_t*>(&h);
  } else {
    const __half2 h = __floats2half2_rn(x, y);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
}

template <bool BF, int D, bool PAIR>
__global__ void __launch_bounds__(kTreeThreads, 1) k_tree_attend(
    const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v, const __grid_constant__ CUtensorMap map_q,
    const uint16_t* __restrict__ q, const uint16_t* __restrict__ V, const TreeShape a, const int box, const int fat,
    const int q_rows, const int most_blocks,
    uint16_t* __restrict__ out, float* __restrict__ lse, float* __restrict__ part, int4* __restrict__ info, int* err) {
  constexpr int NS = tree_slots<D>(), RU = PAIR ? 2 * kTreeTile : kTreeTile;
  constexpr uint32_t kSlot = tree_slot_bytes<D>(), kHalf = kTreeTile * 128;
  // kind::f16, D fp32, A and B of the type; N >> 3 at bits 17-22, M >> 4 at bits 24-28; bit 16: B is MN-major
  constexpr uint32_t kType = (1u << 4) | (BF ? (1u << 7) | (1u << 10) : 0u) | ((uint32_t)(kTreeTile >> 4) << 24);
  constexpr uint32_t kIdS = kType | ((uint32_t)(kTreeTile >> 3) << 17);
  constexpr uint32_t kIdO = kType | (1u << 16) | ((uint32_t)(D >> 3) << 17);
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  unsigned char* sq = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  unsigned char* ring = sq + 2 * kSlot;
  TreeShared& sh = *reinterpret_cast<TreeShared*>(ring + NS * kSlot);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 32) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&map_k)) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&map_v)) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&map_q)) : "memory");
  }
  if (threadIdx.x == 0) {
    for (int i = 0; i < 8; ++i) {
      mbar_init(&sh.k_full[i], 1);
      mbar_init(&sh.v_full[i], 1);
      mbar_init(&sh.empty[i], 1);
      mbar_init(&sh.clean[i], 4);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh.s_full[i], 1);
      mbar_init(&sh.p_full[i], 4);
      mbar_init(&sh.o_done[i], 1);
      mbar_init(&sh.q_full[i], 1);
      mbar_init(&sh.q_empty[i], 1);
      mbar_init(&sh.half[i], 4);
      mbar_init(&sh.o_free[i], 4);
    }
    mbar_init(&sh.drain, 1);
    for (int i = 0; i < 8; ++i) sh.poison[i] = 0;
    sh.abort = 0;
    fence_mbar_init();
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  }
  // Tensor memory is taken when the kernels before have ended and before the next may start: none of them waits for
  // columns that another holds while it waits.
  pdl_wait();
  if (warp == kTreeMma) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(&sh.tmem)), "r"(kTreeTmem));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }

  // ---- this CTA's share of all tiles, and the request it starts in
  TreeWalk w;
  w.RU = RU;
  w.team = w.member = 0;
  const int per = (a.B + kTreeThreads - 1) / kTreeThreads;
  const int b0 = min(a.B, (int)threadIdx.x * per), b1 = min(a.B, b0 + per);
  int tiles = 0, units = 0, longest = 0;
  const int most = (a.T_max * a.G + RU - 1) / RU;
  bool alike = true;  // all requests have that many blocks of rows
  for (w.r = b0; w.r < b1; ++w.r) {
    if (w.enter(a)) {
      tiles += w.units * w.nt;
      units += w.units;
      longest = max(longest, w.nt);
      alike &= w.blocks == most;
    } else if (blockIdx.x == 0 && !tree_request(a, w.r, w.x)) {
      raise_error(err, IG_DEVERR_INDEX);
    }
  }
  int tiles_in = tiles, units_in = units;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, tiles_in, o), y2 = __shfl_up_sync(0xffffffffu, units_in, o);
    if (lane >= o) {
      tiles_in += y;
      units_in += y2;
    }
    longest = max(longest, __shfl_xor_sync(0xffffffffu, longest, o));
  }
  if (lane == 31) {
    sh.scan[warp][0] = tiles_in;
    sh.scan[warp][1] = units_in;
    sh.scan[warp][2] = longest;
  }
  if (threadIdx.x == 0 && !most_blocks) info[2 * blockIdx.x] = make_int4(-1, 0, 0, 0);
  tc_fence_before();
  alike = __syncthreads_and(alike);
  tc_fence_after();
  pdl_trigger();
  const uint32_t tmem = sh.tmem;
  int tiles_before = tiles_in - tiles, units_before = units_in - units, all_tiles = 0, all_units = 0;
  const int full = per == 1 ? (a.B + 31) / 32 : kTreeThreads / 32;  // warps that have requests
#pragma unroll 1
  for (int i = 0; i < full; ++i) {
    tiles_before += i < warp ? sh.scan[i][0] : 0;
    units_before += i < warp ? sh.scan[i][1] : 0;
    all_tiles += sh.scan[i][0];
    all_units += sh.scan[i][1];
    longest = max(longest, sh.scan[i][2]);
  }
  w.whole = all_units <= (int)gridDim.x &&
            (longest <= kTreeWhole ||
             (2 * all_units >= (int)gridDim.x && (long long)longest * all_units <= (long long)all_tiles + kTreeEven * all_units));
  // Where all requests have the same few blocks of rows, a team of CTAs takes the blocks of the same tiles side by side, which
  // then come from HBM once and else from L2 (two trees of 512 rows on 65536 tokens: 135 -> 130 us; with heads of 64, which
  // need half as much a tile, 182 -> 187, so not there).
  if (PAIR && D == 128 && !w.whole && alike && most > 1 && (int)gridDim.x / most * most * 20 >= (int)gridDim.x * 19) {
    w.team = most;
    w.member = blockIdx.x % most;
    tiles /= most;
    tiles_before /= most;
    all_tiles /= most;
  }
  const int stride = max(w.team, 1), cta = blockIdx.x / stride, places = (int)gridDim.x / stride;
  const int total = w.whole ? all_units : all_tiles, before = w.whole ? units_before : tiles_before,
            mine = w.whole ? units : tiles, ctas = min(places, total);
  const unsigned each = ctas ? (unsigned)total / ctas : 0, rest = ctas ? (unsigned)total % ctas : 0;
  auto first_of = [&](unsigned c) -> int { return (int)(each * c + rest * c / (unsigned)ctas); };  // CTA c's first share
  const int r0 = cta < ctas ? first_of(cta) : 0, r1 = cta < ctas ? first_of(cta + 1) : 0;
  if (r1 > r0 && r0 >= before && r0 < before + mine) {
    int at = before;
    if (per == 1 && !w.team) {  // (this thread's one request, which it has entered)
      w.r = b0;
      w.put(sh.start, r0 - at);
    } else {
      for (w.r = b0; w.r < b1; ++w.r) {
        const int n = w.enter(a) ? w.units * (w.whole ? 1 : w.nt) : 0;
        if (r0 < at + n) {
          w.put(sh.start, r0 - at);
          break;
        }
        at += n;
      }
    }
  }
  __syncthreads();
  w.get(sh.start, r1 - r0);
  const uint32_t most_iters = (uint32_t)kDefaultWaitIters;
  uint32_t sent = 0;  // tiles whose keys (or values) have been sent for, units whose queries have

  if (warp == kTreeTmaK || warp == kTreeTmaV) {
    // ---- tiles, a warp the keys and a warp the values (a copy's issue takes 130 cycles, whatever it moves: pages of 16 rows
    // 112 -> 97 us, of 8 rows 159 -> 99, for 131072 tokens, 64 rows).  A lane moves a box; a page's number is read a tile ahead.
    const bool values = warp == kTreeTmaV, thin = values || fat;
    constexpr int kCols = D / 64;
    const int box_at = (thin ? lane : lane / kCols) * box, col = thin ? 0 : lane % kCols;
    const uint32_t box_bytes = (uint32_t)box * (thin ? D * 2 : 128);
    const int slots = values ? tree_v_slots<D>() : tree_k_slots<D>();
    uint64_t* bars = values ? sh.v_full : sh.k_full;
    uint64_t* free_bars = values ? sh.empty + tree_k_slots<D>() : sh.empty;
    unsigned char* at_ring = ring + (values ? tree_k_slots<D>() * kSlot : 0u);
    at_ring += thin ? box_at * D * 2 : col * kHalf + box_at * 128;
    struct Tile {
      int token0, L, hk, id, row;
      bool is;
    };
    // the box's page and its row there, from tile to tile without a division
    const int pages = kTreeTile / a.page, rest_rows = kTreeTile % a.page, pg0 = box_at / a.page, row0 = box_at % a.page;
    int at = 0, run = w.left > 0 ? w.run() : 0, hk = 0, pg = pg0, row = row0;
    if (w.left > 0) {
      hk = w.head();
      if (w.tile > 0) {
        const int token = w.tile * kTreeTile + box_at;
        pg = token / a.page;
        row = token % a.page;
      }
    }
    auto fetch = [&]() -> Tile {
      Tile t{0, 0, 0, -1, 0, false};
      if (w.left <= 0) return t;
      t.is = true;
      t.token0 = (w.tile + at) * kTreeTile;
      t.L = w.x.L;
      t.hk = hk;
      t.row = row;
      if (box_at < kTreeTile && t.token0 + box_at < t.L) t.id = __ldca(a.table + (size_t)w.x.s * a.max_pages + pg);
      if (++at == run) {
        w.next(a);
        at = 0;
        pg = pg0;
        row = row0;
        if (w.left > 0) {
          run = w.run();
          hk = w.head();
        }
      } else {
        pg += pages;
        row += rest_rows;
        if (row >= a.page) {
          row -= a.page;
          ++pg;
        }
      }
      return t;
    };
    int slot = 0, round = 0;
    Tile t = fetch();
    while (t.is) {
      const Tile next = fetch();
      if (round > 0 && !tree_wait(&free_bars[slot], (round - 1) & 1, &sh.abort, most_iters, err)) break;
      const int token = t.token0 + box_at;
      const bool want = box_at < kTreeTile && token < t.L, ok = want && t.id >= 0 && t.id < a.n_pages;
      const unsigned moving = __ballot_sync(0xffffffffu, ok), bad = __ballot_sync(0xffffffffu, want && !ok);
      if (lane == 0) {
        if (!values) {
          const int live = min(t.L - t.token0, kTreeTile);
          uint32_t v[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) v[i] = live >= 32 * i + 32 ? ~0u : live <= 32 * i ? 0u : (1u << (live - 32 * i)) - 1;
          if (bad) {
            raise_error(err, IG_DEVERR_INDEX);
            for (unsigned m = bad; m; m &= m - 1) {
              const int b = (thin ? __ffs(m) - 1 : (__ffs(m) - 1) / kCols) * box;
              for (int i = 0; i < box; i += 8) v[(b + i) >> 5] &= ~(0xffu << ((b + i) & 31));
            }
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) sh.valid[sent & 7][i] = v[i];
        }
        mbar_arrive_expect_tx(&bars[sent & 7], (uint32_t)__popc(moving) * box_bytes);
      }
      __syncwarp();
      if (ok) {
        const int y = (t.id * a.Hkv + t.hk) * a.page + t.row;
        if (thin) tma_load_3d(at_ring + slot * kSlot, values ? &map_v : &map_k, 0, y, 0, &bars[sent & 7]);
        else tma_load_2d(at_ring + slot * kSlot, &map_k, col * 64, y, &bars[sent & 7]);
      }
      ++sent;
      if (++slot == slots) {
        slot = 0;
        ++round;
      }
      t = next;
    }
  } else if (warp == kTreeMma) {
    // ---- the MMAs.  The warp goes together, and one lane issues, by predicate: what the products take is then known to be the same
    // in every lane and stays in uniform registers, where the instructions want it.  An issue returns about when its
    // product begins, so the tensor cores wait for whatever is done between two products, and 170 cycles more to begin
    // again: with two blocks a group's values and its next logits are issued in one go, with all that they need in hand.
    // (Two issuing threads, one a group, whose products come mixed: 158 -> 190 us for two trees of 64 tokens on 65536.)
    const uint32_t lead = elected();
    uint32_t p_seen0 = 0, p_seen1 = 0;
    bool ok = true;
    const uint32_t ring_at = smem_addr(ring), q_at = smem_addr(sq);
    // queries lie by halves; keys too, or box by box (boxes of 8: a group of rows a box); values box by box
    const uint32_t q_high = desc_high(1024), low = desc_low(16);
    const uint32_t k_high = desc_high(fat && box == 8 ? 16 * D : 1024), k_half = fat ? (uint32_t)box * 128 >> 4 : kHalf >> 4;
    const uint32_t v_high = desc_high(box == 8 ? 16 * D : 1024), v_low = desc_low((uint32_t)box * 128);
    uint32_t v_step[kTreeTile / 16];  // where 16 tokens begin
#pragma unroll
    for (int ks = 0; ks < kTreeTile / 16; ++ks) v_step[ks] = (16 * ks / box * box * D * 2 + 16 * ks % box * 128) >> 4;
    const uint32_t tm = (uint32_t)uniform((int)tmem);
    auto wait = [&](uint64_t* bar, uint32_t parity) -> bool { return tree_wait(bar, parity, &sh.abort, most_iters, err); };
    // S of group g from queries at qa and the keys in a slot
    auto logits = [&](uint32_t g, uint32_t qa, uint32_t slot) {
      const uint32_t ad = low + (qa >> 4), bd = low + ((ring_at + slot * kSlot) >> 4);
#pragma unroll
      for (int ks = 0; ks < D / 16; ++ks)
        asm volatile(
            "{\n .reg .pred p, q;\n .reg .b64 da, db;\n mov.b64 da, {%1, %5};\n mov.b64 db, {%2, %7};\n setp.ne.b32 p, %4, 0;\n"
            " setp.ne.b32 q, %6, 0;\n @q tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %3, p;\n}\n" ::"r"(tm + g * kTreeTile),
            "r"(ad + ks / 4 * (kHalf >> 4) + ks % 4 * 2), "r"(bd + ks / 4 * k_half + ks % 4 * 2), "r"(kIdS), "r"(ks), "r"(q_high),
            "r"(lead), "r"(k_high));
      tree_commit(&sh.s_full[g], lead);
    };
    // O of group g, from its weights and the values in a slot
    auto values = [&](uint32_t g, uint32_t slot, uint32_t more) {
      const uint32_t bd = v_low + ((ring_at + (tree_k_slots<D>() + slot) * kSlot) >> 4);
#pragma unroll
      for (int ks = 0; ks < kTreeTile / 16; ++ks)
        asm volatile(
            "{\n .reg .pred p, q;\n .reg .b64 db;\n mov.b64 db, {%2, %5};\n setp.ne.b32 p, %4, 0;\n"
            " setp.ne.b32 q, %6, 0;\n @q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], db, %3, p;\n}\n" ::"r"(
                tm + (2 + g) * kTreeTile),
            "r"(tm + g * kTreeTile + ks * 8), "r"(bd + v_step[ks]), "r"(kIdO), "r"(more | (uint32_t)ks), "r"(v_high), "r"(lead));
    };
    auto weights = [&](uint32_t g) -> bool {
      const uint32_t parity = (g ? p_seen1++ : p_seen0++) & 1;
      return wait(&sh.p_full[g], parity);
    };
    constexpr uint32_t NK = tree_k_slots<D>(), NV = tree_v_slots<D>();
    uint64_t* v_empty = sh.empty + NK;
    uint32_t k_slot = 0, v_slot = 0;  // of the next keys and values
    auto step = [](uint32_t& slot, uint32_t n) { slot = slot + 1 < n ? slot + 1 : 0; };
    if constexpr (!PAIR) {
      // logits of a tile ahead of the values of the one before; tile i is of group i & 1
      uint32_t i = 0, seg = 0, j = 0;       // tile whose logits are next, its unit; tile whose values are
      TreeWalk v = w;                       // of the values
      int left = uniform(w.left), v_left = left;
      int seg_run = left > 0 ? uniform(w.run()) : 0, seg_at = 0, run = seg_run, k = 0;
      for (bool first = true; ok && v_left > 0;) {
        if (left > 0) {  // the next tile's logits
          const uint32_t buf = seg & 1;
          if (seg_at == 0) ok = wait(&sh.q_full[buf], seg >> 1 & 1);
          ok = ok && wait(&sh.k_full[i & 7], i >> 3 & 1);
          if (!ok) break;
          tc_fence_after();
          logits(i & 1, q_at + buf * kSlot, k_slot);
          tree_commit(&sh.empty[k_slot], lead);
          step(k_slot, NK);
          ++i;
          if (++seg_at == seg_run) {
            tree_commit(&sh.q_empty[buf], lead);
            ++seg;
            w.next(a);
            left = uniform(w.left);
            seg_at = 0;
            seg_run = left > 0 ? uniform(w.run()) : 0;
          }
        }
        if (first) {
          first = false;
          continue;
        }
        const uint32_t g = j & 1;
        ok = wait(&sh.v_full[j & 7], j >> 3 & 1) && weights(g);
        if (!ok) break;
        tc_fence_after();
        values(g, v_slot, k >= 2);
        tree_commit(&v_empty[v_slot], lead);
        if (k >= run - 2) tree_commit(&sh.o_done[g], lead);
        step(v_slot, NV);
        ++j;
        if (++k == run) {
          v.next(a);
          v_left = uniform(v.left);
          k = 0;
          run = v_left > 0 ? uniform(v.run()) : 0;
        }
      }
    } else {
      // a tile's values and the next tile's logits, group by group; a unit begins with logits alone
      uint32_t j = 0;
      for (uint32_t seg = 0; ok && uniform(w.left) > 0; w.next(a), ++seg) {
        const int run = uniform(w.run()), rows = uniform(w.x.n * a.G - w.block() * RU);
        const uint32_t groups = rows > kTreeTile ? 2 : 1;
        ok = wait(&sh.q_full[0], seg & 1) && wait(&sh.k_full[j & 7], j >> 3 & 1);
        if (!ok) break;
        tc_fence_after();
        for (uint32_t g = 0; g < groups; ++g) logits(g, q_at + g * kSlot, k_slot);
        tree_commit(&sh.empty[k_slot], lead);
        step(k_slot, NK);
        if (run == 1) tree_commit(&sh.q_empty[0], lead);
        for (int k = 0; k < run; ++k, ++j) {
          const bool next = k < run - 1;
          ok = wait(&sh.v_full[j & 7], j >> 3 & 1) && (!next || wait(&sh.k_full[(j + 1) & 7], (j + 1) >> 3 & 1));
          for (uint32_t g = 0; ok && g < groups; ++g) {
            ok = weights(g);
            if (!ok) break;
            tc_fence_after();
            values(g, v_slot, k > 0);
            if (next) {
              logits(g, q_at + g * kSlot, k_slot);
            } else {
              if (g == groups - 1) tree_commit(&v_empty[v_slot], lead);
              tree_commit(&sh.o_done[g], lead);  // (the unit's last: what comes before it has come when it is seen)
            }
          }
          if (!ok) break;
          if (next) {
            tree_commit(&v_empty[v_slot], lead);
            tree_commit(&sh.empty[k_slot], lead);
            if (k == run - 2) tree_commit(&sh.q_empty[0], lead);
            step(k_slot, NK);
          }
          step(v_slot, NV);
        }
      }
    }
    __syncwarp();
  } else if (warp == kTreeQueries) {
    // ---- queries, rows in the order (token, head); rows behind the last one hold anything.  By TMA where the group is a power of
    // two, so that 128 rows are a box of tokens and heads (a warp takes 5 us for 256 rows, and twice that beside the
    // others' work: 512 rows on 2 x 65536 tokens 129 -> 115 us).
    for (uint32_t seg = 0; w.left > 0; ++seg, w.next(a)) {
      const uint32_t buf = PAIR ? 0 : seg & 1, round = PAIR ? seg : seg >> 1;
      if (round > 0 && !tree_wait(&sh.q_empty[buf], (round - 1) & 1, &sh.abort, most_iters, err)) break;
      const int row0 = w.block() * RU, rows = min(RU, w.x.n * a.G - row0), hk = w.head();
      if (q_rows) {
        const int parts = rows > kTreeTile ? 2 : 1;
        if (lane == 0) mbar_arrive_expect_tx(&sh.q_full[buf], (uint32_t)(parts * (D / 64) * q_rows) * 128);
        __syncwarp();
        if (lane < parts * (D / 64)) {
          const int part = lane / (D / 64), col = lane % (D / 64), at = row0 + part * kTreeTile;
          tma_load_3d(sq + (buf + part) * kSlot + col * kHalf, &map_q, col * 64, hk * a.G + at % a.G, w.x.f + at / a.G,
                      &sh.q_full[buf]);
        }
        ++sent;
        continue;
      }
      constexpr int kRows = 32 / (D / 8);  // of the warp at a time
      const int ch = lane % (D / 8), at = row0 + lane / (D / 8), i = at / a.G;
      int g = at % a.G;
      const uint16_t* p = q + ((size_t)(w.x.f + i) * a.Hq + (size_t)hk * a.G + g) * D + ch * 8;
      const int heads = kRows % a.G, token = a.Hq * D, step = kRows / a.G * token + heads * D, wrap = token - a.G * D;
      const uint32_t to = smem_addr(sq + buf * kSlot + ch / 8 * kHalf);
#pragma unroll 4
      for (int row = lane / (D / 8); row < rows; row += kRows) {
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to + row / kTreeTile * kSlot + row % kTreeTile * 128 +
                                                                      (((ch & 7) ^ (row & 7)) << 4)),
                     "l"(p)
                     : "memory");
        g += heads;
        p += g >= a.G ? step + wrap : step;
        g -= g >= a.G ? a.G : 0;
      }
      asm volatile("cp.async.wait_all;" ::: "memory");
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncwarp();
      if (lane == 0) tree_arrive(&sh.q_full[buf]);
    }
  } else if (warp >= kTreeSoftmax) {
    // ---- softmax: group gs, a row a thread
    const int gs = (warp - kTreeSoftmax) >> 2, quarter = warp & 3;  // a warp reads the tensor memory lanes of its quarter
    const int row = quarter * 32 + lane;
    const uint32_t lanes = (uint32_t)(quarter * 32) << 16;
    const uint32_t s_at = tmem + lanes + gs * kTreeTile, o_at = s_at + 2 * kTreeTile;
    const uint32_t o_other = tmem + lanes + (3 - gs) * kTreeTile;
    const uint32_t limit = wait_limit(err);
    constexpr float kBelow = BF ? 0.f : 10.f, kAbove = BF ? 8.f : 15.75f;  // of the reference: the largest weight, and what moves it
    const float sc = a.scale2 == 0.f ? 1.f : fabsf(a.scale2), sgn = a.scale2 > 0.f ? 1.f : a.scale2 < 0.f ? -1.f : 0.f;
    uint32_t dirty = 0, at_tile = 0, s_seen = 0, o_seen = 0, half_seen = 0, free_seen = 0;
    bool ok = true, lent = false, cut = false;  // lent: the other group still reads this one's O
    for (uint32_t seg = 0; ok && w.left > 0; ++seg) {
      const int run = w.run(), tile0 = w.tile, nt = w.nt, hk = w.head(), block = w.block();
      const TreeRequest x = w.x;
      const int unit_r = w.r, left = w.left;
      const int rows_all = min(RU, x.n * a.G - block * RU);
      const int my_row = PAIR ? gs * kTreeTile + row : row;  // in the unit
      const bool live = my_row < rows_all, warp_live = my_row - lane < rows_all;
      const int rr = block * RU + my_row, node = live ? rr / a.G : 0, head = live ? rr % a.G : 0;
      const bool done = tile0 == 0 && run == nt;
      cut = tile0 == 0 && !done;
      w.next(a);
      const unsigned long long mask = live ? __ldca(a.masks + x.f + node) : 0;
      const int k0 = PAIR ? 0 : (int)((at_tile & 1) ^ (uint32_t)gs);  // this group's first tile of the run
      if (k0 >= run || (PAIR && gs * kTreeTile >= rows_all)) {
        at_tile += run;
        continue;
      }
      float m = -INFINITY, l = 0.f;
      for (int k = k0; ok && k < run; k += PAIR ? 1 : 2) {
        const uint32_t j = at_tile + k;  // tile of the CTA
        ok = tree_wait(&sh.s_full[gs], s_seen++ & 1, &sh.abort, limit, err);
        if (!ok) break;
        tc_fence_after();
        const int t0 = (tile0 + k) * kTreeTile, drafted = x.L - x.n;
        const volatile uint32_t* va = sh.valid[j & 7];
        const bool plain = (va[0] & va[1] & va[2] & va[3]) == ~0u && t0 + kTreeTile <= drafted;
        if (warp_live && (!plain || sgn != 1.f)) {  // the row's logits put right where they are: what it does not see is -inf
#pragma unroll 1
          for (int c = 0; c < 4; ++c) {
            const uint32_t vis = va[c] & seen_bits(mask, t0 + 32 * c - drafted);
            uint32_t y[32];
            tm_ld32(y, s_at + 32 * c);
            tm_wait_ld32(y);
#pragma unroll
            for (int i = 0; i < 32; ++i) y[i] = vis >> i & 1 ? __float_as_uint(__uint_as_float(y[i]) * sgn) : 0xff800000u;
            tm_st32(s_at + 32 * c, y);
          }
          tm_wait_st();
        }
        if (warp_live) {
          // (Loops over 32 logits at a time, read twice, keep the code small: unrolled over the row, all roles' code is more
          // than the instruction caches hold, and every instruction takes several times as long.)
          uint32_t ya[32], yb[32];  // 32 logits are on their way while 32 are worked on
          float top, sum[4], mx[4];
          auto none = [&]() {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              sum[i] = 0.f;
              mx[i] = -INFINITY;
            }
          };
          auto largest = [&](const uint32_t (&y)[32]) {
#pragma unroll
            for (int i = 0; i < 32; i += 2) mx[i / 2 % 4] = max3(mx[i / 2 % 4], __uint_as_float(y[i]), __uint_as_float(y[i + 1]));
          };
          auto weigh = [&](const uint32_t (&y)[32], uint32_t (&p)[16], float m0) {
#pragma unroll
            for (int i = 0; i < 32; i += 2) {
              const float y0 = ex2(fmaf(__uint_as_float(y[i]), sc, -m0)), y1 = ex2(fmaf(__uint_as_float(y[i + 1]), sc, -m0));
              sum[i / 2 % 4] += y0;
              sum[i / 2 % 4] += y1;
              p[i / 2] = pack2<BF>(y0, y1);
            }
          };
          bool again = true;
          none();
          tm_ld32(ya, s_at);
          if (k > k0) {
            // Weights by the reference that there is, and the largest logit with them: mostly it stays, and one look at the logits
            // is enough (8 trees of 256 to 512 rows 181 -> 174 us; 64 rows, heads of 64, 131072 tokens 54 -> 51; no gain where HBM
            // is waited for).  They stay where they are until that is known.
            const float m0 = m == -INFINITY ? 0.f : m;
            uint32_t p0[16], p1[16], p2[16], p3[16];
            tm_wait_ld32(ya);
            tm_ld32(yb, s_at + 32);
            largest(ya);
            weigh(ya, p0, m0);
            tm_wait_ld32(yb);
            tm_ld32(ya, s_at + 64);
            largest(yb);
            weigh(yb, p1, m0);
            tm_wait_ld32(ya);
            tm_ld32(yb, s_at + 96);
            largest(ya);
            weigh(ya, p2, m0);
            tm_wait_ld32(yb);
            largest(yb);
            top = fmaxf(max3(mx[0], mx[1], mx[2]), mx[3]) * sc;
            again = __any_sync(0xffffffffu, live && top > m + kAbove);
            if (!again) {
              tm_st16(s_at, p0);
              tm_st16(s_at + 16, p1);
              tm_st16(s_at + 32, p2);
              weigh(yb, p3, m0);
              tm_st16(s_at + 48, p3);
            } else {
              none();
              tm_ld32(ya, s_at);
            }
          }
          if (again) {
#pragma unroll 1
            for (int c = 0; c < 4; c += 2) {
              tm_wait_ld32(ya);
              tm_ld32(yb, s_at + 32 * c + 32);
              largest(ya);
              tm_wait_ld32(yb);
              tm_ld32(ya, s_at + (32 * c + 64) % 128);  // (at the end the first ones, for the weights)
              largest(yb);
            }
            top = fmaxf(max3(mx[0], mx[1], mx[2]), mx[3]) * sc;
            const bool move = live && top > m + kAbove;  // (from -inf on: whenever there is anything)
            if (__any_sync(0xffffffffu, move)) {
              const float to = move ? top - kBelow : m, f = move ? ex2(m - to) : 1.f;
              m = to;
              l *= f;
              if (k > k0) {
#pragma unroll 1
                for (int c = 0; c < D / 32; ++c) {
                  uint32_t o[32];
                  tm_ld32(o, o_at + 32 * c);
                  tm_wait_ld32(o);
#pragma unroll
                  for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
                  tm_st32(o_at + 32 * c, o);
                }
              }
            }
            const float m0 = m == -INFINITY ? 0.f : m;
            uint32_t p[16];
#pragma unroll 1
            for (int c = 0; c < 4; c += 2) {  // weights go where logits were that have been read
              tm_wait_ld32(ya);
              tm_ld32(yb, s_at + 32 * c + 32);
              weigh(ya, p, m0);
              tm_st16(s_at + 16 * c, p);
              tm_wait_ld32(yb);
              if (c == 0) tm_ld32(ya, s_at + 64);
              weigh(yb, p, m0);
              tm_st16(s_at + 16 * c + 16, p);
            }
          }
          tm_wait_st();
          l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
        }
        if (!plain && (!PAIR || gs == 0)) {
          // values without a token are cleared, and what is not finite in drafted ones: a row of the tile a thread
          ok = tree_wait(&sh.v_full[j & 7], j >> 3 & 1, &sh.abort, most_iters, err);
          if (!ok) break;
          uint4* vr = reinterpret_cast<uint4*>(ring + (tree_k_slots<D>() + j % tree_v_slots<D>()) * kSlot + row / box * box * D * 2 +
                                               row % box * 128);
          const int vh = box * 8;  // to the row's other half
          if (!(va[quarter] >> lane & 1)) {
#pragma unroll
            for (int c = 0; c < D / 8; ++c) vr[c / 8 * vh + c % 8] = make_uint4(0, 0, 0, 0);
          } else if (t0 + row >= drafted) {
            uint32_t odd = 0;
#pragma unroll
            for (int c = 0; c < D / 8; ++c) {
              const uint4 y = vr[c / 8 * vh + c % 8];
              odd |= odd_pair<BF>(y.x) | odd_pair<BF>(y.y) | odd_pair<BF>(y.z) | odd_pair<BF>(y.w);
            }
            if (odd) {
              uint16_t* e = reinterpret_cast<uint16_t*>(vr);
              for (int c = 0; c < D; ++c) {
                uint16_t& y = e[c / 64 * vh * 8 + c % 64];
                if (odd_pair<BF>(y)) y = 0;
              }
              *(volatile int*)&sh.poison[seg & 7] = (int)seg + 1;
            }
          }
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        }
        if (PAIR && !plain && rows_all > kTreeTile) {
          if (gs == 0) {
            __syncwarp();
            if (lane == 0) tree_arrive(&sh.clean[dirty & 7]);
          } else {
            ok = tree_wait(&sh.clean[dirty & 7], dirty >> 3 & 1, &sh.abort, most_iters, err);
            if (!ok) break;
          }
          ++dirty;
        }
        if (lent) {  // O is free again once the other group has taken what it needs
          ok = tree_wait(&sh.o_free[gs], free_seen++ & 1, &sh.abort, most_iters, err);
          if (!ok) break;
          lent = false;
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) tree_arrive(&sh.p_full[gs]);
      }
      if (!ok) break;
      // ---- the unit's end in this CTA
      ok = tree_wait(&sh.o_done[gs], o_seen++ & 1, &sh.abort, most_iters, err);
      if (!ok) break;
      tc_fence_after();
      const bool joined = !PAIR && run >= 2;
      const int last_of = (int)((at_tile + run - 1) & 1);  // the group of the run's last tile writes
      if (joined && gs != last_of) {
        sh.ml[row] = make_float2(m, l);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) tree_arrive(&sh.half[gs]);
        lent = true;
        at_tile += run;
        continue;
      }
      float f = 1.f, f2 = 0.f;
      if (joined) {
        ok = tree_wait(&sh.half[1 - gs], half_seen++ & 1, &sh.abort, most_iters, err);
        if (!ok) break;
        tc_fence_after();
        const float2 y = sh.ml[row];
        const float M = fmaxf(m, y.x), m0 = M == -INFINITY ? 0.f : M;
        f = ex2(m - m0);
        f2 = ex2(y.x - m0);
        l = l * f + y.y * f2;
        m = M;
      }
      const bool poisoned = *(volatile int*)&sh.poison[seg & 7] == (int)seg + 1;
      const size_t at = live ? (size_t)(x.f + node) * a.Hq + (size_t)hk * a.G + head : 0;
      // the unit it starts with, begun by an earlier CTA, to slot 0; one it begins to slot 1
      float* wp = part + ((size_t)(2 * blockIdx.x + (tile0 == 0 ? 1 : 0)) * RU + my_row) * (D + kTreePartHead);
      const float inv = l == 0.f ? 0.f : 1.f / l;
      if (warp_live) {
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c) {
          uint32_t o[32];
          __syncwarp();
          tm_ld32(o, o_at + 32 * c);
          if (joined) {
            uint32_t o2[32];
            tm_ld32(o2, o_other + 32 * c);
            tm_wait_ld32(o, o2);
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f + __uint_as_float(o2[i]) * f2);
          } else {
            tm_wait_ld32(o);
          }
          if (poisoned && live) {
            // drafted values that are not finite, of the tiles here: to the rows that see them
            for (int d = 0; d < x.n; ++d) {
              const int token = x.L - x.n + d;
              if (!(mask >> d & 1) || token < tile0 * kTreeTile || token >= (tile0 + run) * kTreeTile) continue;
              const int id = __ldca(a.table + (size_t)x.s * a.max_pages + token / a.page);
              if (id < 0 || id >= a.n_pages) continue;
              const uint16_t* vp = V + ((size_t)(id * a.Hkv + hk) * a.page + token % a.page) * D + 32 * c;
#pragma unroll
              for (int i = 0; i < 32; ++i) {
                const uint16_t y = __ldca(vp + i);
                if (odd_pair<BF>(y)) o[i] = __float_as_uint(__uint_as_float(o[i]) + to_float<BF>(y));
              }
            }
          }
          if (live && done) {
            uint4* to = reinterpret_cast<uint4*>(out + at * D + 32 * c);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              uint32_t h[4];
#pragma unroll
              for (int y = 0; y < 4; ++y)
                h[y] = pack2<BF>(__uint_as_float(o[8 * i + 2 * y]) * inv, __uint_as_float(o[8 * i + 2 * y + 1]) * inv);
              to[i] = make_uint4(h[0], h[1], h[2], h[3]);
            }
          } else if (live) {
            float* to = wp + kTreePartHead + 32 * c;  // (a row a thread, so a sector at a time: 115 -> 111 us)
#pragma unroll
            for (int i = 0; i < 32; i += 8)
              asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(to + i), "r"(o[i]), "r"(o[i + 1]), "r"(o[i + 2]),
                           "r"(o[i + 3]), "r"(o[i + 4]), "r"(o[i + 5]), "r"(o[i + 6]), "r"(o[i + 7])
                           : "memory");
          }
        }
        if (live) {
          if (done) {
            if (lse) lse[at] = (m + log2f(l)) * 0.6931471805599453f;
          } else {
            *reinterpret_cast<float2*>(wp) = make_float2(m, l);
          }
        }
      }
      if (joined) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) tree_arrive(&sh.o_free[1 - gs]);
      }
      // what the second kernel joins: a unit that begins here and goes on in later CTAs (listed by unit, where there are fewer
      // than CTAs, finished ones too; else by the CTA that it begins in)
      if ((cut || (most_blocks && done)) && row == 0 && (!PAIR || gs == 0)) {
        int last = cta;
        if (cut) {
          const int end = r1 - left + nt - 1;  // its last tile: a cut unit is this CTA's last, `left` tiles long here
          last = min(ctas - 1, (int)((float)end * ((float)ctas / (float)total)));  // within 1
          while (last + 1 < ctas && first_of(last + 1) <= end) ++last;
          while (first_of(last) > end) --last;
        }
        last = last * stride + w.member;
        const int at = most_blocks ? (unit_r * a.Hkv + hk) * most_blocks + block : blockIdx.x;
        info[2 * at] = make_int4(cut ? blockIdx.x : -1, last, stride, 0);
        info[2 * at + 1] = make_int4(x.f, x.n, hk, block);
      }
      at_tile += run;
    }
  }
  tc_fence_before();
  __syncthreads();
  // Where a wait ran out (only here, where every role is done, is it known), copies and products may be in flight: they end
  // before the CTA gives back its shared and its tensor memory.  (Else the last commit of all has been waited for.)
  if (*(volatile int*)&sh.abort) {
    if (warp == kTreeMma) {
      tree_commit(&sh.drain, elected());
      __syncwarp();
      mbar_wait_bounded(&sh.drain, 0);
    }
    if (warp == kTreeTmaK || warp == kTreeTmaV)
      for (uint32_t x = sent > 8 ? sent - 8 : 0; x < sent; ++x)
        mbar_wait_bounded(warp == kTreeTmaV ? &sh.v_full[x & 7] : &sh.k_full[x & 7], x >> 3 & 1);
    if (warp == kTreeQueries)
      for (uint32_t x = sent > 2 ? sent - 2 : 0; x < sent; ++x)
        mbar_wait_bounded(&sh.q_full[PAIR ? 0 : x & 1], (PAIR ? x : x >> 1) & 1);
    __syncthreads();
  }
  if (warp == kTreeMma) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTreeTmem));
  }
}

// Joins the partials of the units that were cut: block (x, y) takes unit x (or the one that CTA x began) and rows y * RB ... of it,
// WPR warps a row; a warp takes every WPR-th partial in order, and the warps join in order.  (Listed by CTA, 8 units of 128 rows
// in 152 CTAs take 19456 blocks, of which 1024 have anything to do: 12 us more.)
template <bool BF, int D, int WPR, int RB>
__global__ void __launch_bounds__(WPR * RB * 32) k_tree_join(const float* __restrict__ part, const int4* __restrict__ info,
                                                            const TreeShape a, int RU, int most_blocks, uint16_t* __restrict__ out,
                                                            float* __restrict__ lse) {
  constexpr int VEC = D / 32;
  __shared__ float sm[WPR * RB], sl[WPR * RB], so[WPR * RB][WPR > 1 ? D : 1];
  pdl_trigger();
  // Listed by unit, a unit that there is has an entry, but for those of CTAs whose waits ran out.  (What the first kernel was given
  // is there already: it lets this one start only when those before it have ended.)
  TreeRequest x;
  int f = 0, rows = 0, hk = 0, block = 0;
  if (most_blocks) {
    block = blockIdx.x % most_blocks, hk = blockIdx.x / most_blocks % a.Hkv;
    if (tree_request<true>(a, blockIdx.x / most_blocks / a.Hkv, x)) f = x.f, rows = x.n * a.G;
  }
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int4 e = __ldca(info + 2 * blockIdx.x), unit = __ldca(info + 2 * blockIdx.x + 1);
  const int c0 = e.x, last = e.y, stride = e.z;
  if (c0 < 0 || last < c0 || last >= kMaxTreeCtas || stride < 1) return;
  if (!most_blocks) f = unit.x, rows = unit.y * a.G, hk = unit.z, block = unit.w;
  const int n = (last - c0) / stride + 1, row = blockIdx.y * RB + warp / WPR, rr = block * RU + row;
  const bool live = row < RU && rr < rows;
  float m = -INFINITY, l = 0.f, o[VEC];
#pragma unroll
  for (int i = 0; i < VEC; ++i) o[i] = 0.f;
  if (live) {
    // this warp's partials are w0, w0 + WPR, ...: 32 references and sums at a time (one a lane), outputs U at a time,
    // the first U on their way before the references are there
    constexpr int U = 8;
    const int w0 = warp % WPR, mine = (n - w0 + WPR - 1) / WPR;
    auto at = [&](int i) -> const float* {
      const int j = w0 + i * WPR;
      return part + ((size_t)(2 * (c0 + j * stride) + (j == 0 ? 1 : 0)) * RU + row) * (D + kTreePartHead);
    };
    auto load = [&](int i0, float (&v)[U][VEC]) {
#pragma unroll
      for (int x = 0; x < U; ++x) {
        if (i0 + x < mine) {
          const float* p = at(i0 + x) + kTreePartHead + lane * VEC;
          if constexpr (VEC == 4) {
            const float4 y = __ldca(reinterpret_cast<const float4*>(p));
            v[x][0] = y.x, v[x][1] = y.y, v[x][2] = y.z, v[x][3] = y.w;
          } else {
            const float2 y = __ldca(reinterpret_cast<const float2*>(p));
            v[x][0] = y.x, v[x][1] = y.y;
          }
        } else {
#pragma unroll
          for (int i = 0; i < VEC; ++i) v[x][i] = 0.f;
        }
      }
    };
    float v[U][VEC];
    for (int b0 = 0; b0 < mine; b0 += 32) {
      load(b0, v);
      const float2 h = b0 + lane < mine ? __ldca(reinterpret_cast<const float2*>(at(b0 + lane))) : make_float2(-INFINITY, 0.f);
      float mx = h.x;
#pragma unroll
      for (int x = 16; x; x >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, x));
      const float mn = fmaxf(m, mx), m0 = mn == -INFINITY ? 0.f : mn;
      const float fo = ex2(m - m0), g = ex2(h.x - m0);
      float sum = h.y * g;
#pragma unroll
      for (int x = 16; x; x >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, x);
      l = l * fo + sum;
#pragma unroll
      for (int i = 0; i < VEC; ++i) o[i] *= fo;
      m = mn;
      for (int i0 = 0; i0 < 32 && b0 + i0 < mine; i0 += U) {
        if (i0) load(b0 + i0, v);
#pragma unroll
        for (int x = 0; x < U; ++x) {
          const float gx = __shfl_sync(0xffffffffu, g, i0 + x);
          // (a partial past the end has weight 0 and values 0)
#pragma unroll
          for (int i = 0; i < VEC; ++i) o[i] = fmaf(v[x][i], gx, o[i]);
        }
      }
    }
  }
  if constexpr (WPR > 1) {
    if (lane == 0) {
      sm[warp] = m;
      sl[warp] = l;
    }
#pragma unroll
    for (int i = 0; i < VEC; ++i) so[warp][lane * VEC + i] = o[i];
    __syncthreads();
    if (warp % WPR) return;
    m = -INFINITY;
#pragma unroll
    for (int x = 0; x < WPR; ++x) m = fmaxf(m, sm[warp + x]);
    const float m0 = m == -INFINITY ? 0.f : m;
    l = 0.f;
#pragma unroll
    for (int i = 0; i < VEC; ++i) o[i] = 0.f;
#pragma unroll
    for (int x = 0; x < WPR; ++x) {
      const float fx = ex2(sm[warp + x] - m0);
      l += sl[warp + x] * fx;
#pragma unroll
      for (int i = 0; i < VEC; ++i) o[i] += so[warp + x][lane * VEC + i] * fx;
    }
  }
  if (!live) return;
  const size_t at = (size_t)(f + rr / a.G) * a.Hq + (size_t)hk * a.G + rr % a.G;
  const float inv = l == 0.f ? 0.f : 1.f / l;
  uint32_t h[VEC / 2];
#pragma unroll
  for (int i = 0; i < VEC / 2; ++i) h[i] = pack2<BF>(o[2 * i] * inv, o[2 * i + 1] * inv);
  if constexpr (VEC == 4) *reinterpret_cast<uint2*>(out + at * D + lane * VEC) = make_uint2(h[0], h[1]);
  else *reinterpret_cast<uint32_t*>(out + at * D + lane * VEC) = h[0];
  if (lse && lane == 0) lse[at] = (m + log2f(l)) * 0.6931471805599453f;
}

// rows of a unit
inline int tree_rows(int T_max, int G) { return (long long)T_max * G > kTreeTile ? 2 * kTreeTile : kTreeTile; }

// workspace: two partials per CTA, then the join's list
inline size_t tree_part_bytes(int rows, int d) {
  return round_up((size_t)2 * kMaxTreeCtas * rows * (d + kTreePartHead) * sizeof(float), 256);
}

template <bool BF, int D, bool PAIR>
ig_status launch_tree(cudaStream_t st, const TreeShape& a, const uint16_t* q, const uint16_t* K, const uint16_t* V, uint16_t* out,
                      float* lse, void* ws) {
  constexpr int RU = PAIR ? 2 * kTreeTile : kTreeTile;
  const long long tiles = ((long long)a.max_pages * a.page + kTreeTile - 1) / kTreeTile;
  const long long blocks = ((long long)a.T_max * a.G + RU - 1) / RU;
  const double most = (double)a.B * a.Hkv * blocks * tiles;
  IG_REQUIRE(most < 2147483648.0, "n*max_pages*page*Hq is too large: %.0f tiles", most);
  int box = kTreeTile;
  while (a.page % box) box >>= 1;
  // Values lie box by box, both halves of its columns in one copy: their product takes 16 rows at a time, wherever they are.  Keys' 128
  // rows have to lie evenly, so theirs do so where a box is a tile or a group of 8 rows, else a half a copy.
  const int fat = D == 64 || box == 8 || box == kTreeTile ? 1 : 0, rows = a.n_pages * a.Hkv * a.page;
  // queries, 128 rows a box of whole tokens (or of a token's heads)
  const bool even = (a.G & (a.G - 1)) == 0;
  const int heads = a.G < kTreeTile ? a.G : kTreeTile, tokens = kTreeTile / heads < a.T_max ? kTreeTile / heads : a.T_max;
  CUtensorMap mk, mv, mq;
  ig_status r = fat ? make_map_halves(&mk, K, rows, D, box) : make_map(&mk, K, rows, D, box);
  if (r == IG_OK) r = make_map_halves(&mv, V, rows, D, box);
  if (r == IG_OK && even) r = make_map_heads(&mq, q, a.T, a.Hq, D, tokens, heads);
  if (r != IG_OK) return r;
  if (!even) mq = mk;  // (not used)
  constexpr size_t smem = tree_smem<D>();
  cudaError_t e = cudaFuncSetAttribute(k_tree_attend<BF, D, PAIR>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return cuda_fail(e, "tree attention smem attribute");
  int grid = sm_count(st);
  if (grid > kMaxTreeCtas) grid = kMaxTreeCtas;
  if (grid > most) grid = (int)most;
  const double units = (double)a.B * a.Hkv * blocks;  // at most
  const int most_blocks = units <= grid ? (int)blocks : 0;
  float* part = static_cast<float*>(ws);
  int4* info = reinterpret_cast<int4*>(static_cast<char*>(ws) + tree_part_bytes(RU, D));
  e = launch_pdl(k_tree_attend<BF, D, PAIR>, dim3(grid), dim3(kTreeThreads), smem, st, mk, mv, mq, q, V, a, box, fat,
                 even ? tokens * heads : 0, most_blocks, out, lse, part, info, error_word());
  if (e != cudaSuccess) return cuda_fail(e, "tree attention launch");
  IG_CHECK_LAUNCH("tree attention launch");
  if (grid == 1 || (most_blocks && tiles <= kTreeWhole)) return IG_OK;  // nothing can have been cut
  const int used = (long long)a.T_max * a.G < RU ? a.T_max * a.G : RU;
  const float* cpart = part;
  const int4* cinfo = info;
  const double partials = grid / units;  // of a unit, about
  const int list = most_blocks ? (int)units : grid;
#define IG_TJ(WPR, RB)                                                                                                     \
  e = launch_pdl(k_tree_join<BF, D, WPR, RB>, dim3(list, (used + RB - 1) / RB), dim3(WPR * RB * 32), 0, st, cpart, cinfo, a, RU, \
                 most_blocks, out, lse)
  if (partials >= 16) IG_TJ(4, 1);
  else IG_TJ(1, 4);
#undef IG_TJ
  if (e != cudaSuccess) return cuda_fail(e, "tree attention join launch");
  IG_CHECK_LAUNCH("tree attention join launch");
  return IG_OK;
}

template <bool BF, int D>
ig_status launch_rows(cudaStream_t st, const TreeShape& a, const uint16_t* q, const uint16_t* K, const uint16_t* V, uint16_t* out,
                      float* lse, void* ws) {
  return tree_rows(a.T_max, a.G) == kTreeTile ? launch_tree<BF, D, false>(st, a, q, K, V, out, lse, ws)
                                              : launch_tree<BF, D, true>(st, a, q, K, V, out, lse, ws);
}

}  // namespace
}  // namespace ig

using namespace ig;

extern "C" size_t ig_paged_tree_attend_workspace_bytes(int n, int T_max, int Hq, int Hkv, int d) {
  if (n <= 0 || T_max <= 0 || T_max > kTreeMost || Hq <= 0 || Hkv <= 0 || Hq % Hkv || (d != 64 && d != 128)) return 0;
  return tree_part_bytes(tree_rows(T_max, Hq / Hkv), d) + round_up(2 * kMaxTreeCtas * sizeof(int4), 256);
}

extern "C" ig_status ig_paged_tree_attend(void* stream, int dtype, int n, int T, int T_max, int Hq, int Hkv, int d, int page,
                                          int n_pages, int seqs, int max_pages, float scale, const uint16_t* q,
                                          const uint16_t* K, const uint16_t* V, const int32_t* page_table,
                                          const int32_t* L_valid, const int32_t* seq, const int32_t* first,
                                          const uint64_t* masks, uint16_t* out, float* lse, void* workspace,
                                          size_t workspace_bytes) {
  IG_REQUIRE(dtype == IG_F16 || dtype == IG_BF16, "dtype must be IG_F16 or IG_BF16 (got %d)", dtype);
  IG_REQUIRE(n > 0 && Hq > 0 && Hkv > 0 && seqs > 0, "n, Hq, Hkv, seqs must be positive");
  IG_REQUIRE(T >= 0, "T must not be negative");
  IG_REQUIRE(T_max > 0 && T_max <= kTreeMost, "T_max must be in [1, %d] (got %d)", kTreeMost, T_max);
  IG_REQUIRE(seq || n <= seqs, "%d requests for %d sequences: name them", n, seqs);
  IG_REQUIRE(Hq % Hkv == 0, "Hq = %d is not a multiple of Hkv = %d", Hq, Hkv);
  IG_REQUIRE(d == 64 || d == 128, "d must be 64 or 128 (got %d)", d);
  IG_REQUIRE(page > 0 && page % 8 == 0, "page must be a positive multiple of 8 (got %d)", page);
  IG_REQUIRE(n_pages > 0 && max_pages > 0, "n_pages and max_pages must be positive");
  IG_REQUIRE(Hq <= 65536 && (long long)T * Hq < (1ll << 31), "Hq at most 65536, T*Hq below 2^31");
  IG_REQUIRE((long long)max_pages * page < (1ll << 30), "max_pages*page must stay below 2^30");
  IG_REQUIRE((double)n_pages * Hkv * page < 2147483648.0, "n_pages*Hkv*page must stay below 2^31 rows");
  IG_REQUIRE(isfinite(scale) && fabsf(scale) < 1e38f, "scale must be finite (and below 1e38)");
  if (T == 0) return IG_OK;
  IG_REQUIRE(q && K && V && page_table && L_valid && first && masks && out, "null pointer argument");
  IG_REQUIRE(aligned(q, 16) && aligned(K, 16) && aligned(V, 16) && aligned(out, 16), "q, K, V, out must be 16-byte aligned");
  IG_REQUIRE(aligned(page_table, 4) && aligned(L_valid, 4) && aligned(seq, 4) && aligned(first, 4) && aligned(lse, 4) &&
                 aligned(masks, 8),
             "misaligned buffer");
  const size_t need = ig_paged_tree_attend_workspace_bytes(n, T_max, Hq, Hkv, d);
  if (!workspace || workspace_bytes < need)
    return fail(IG_ERR_CAPACITY, "tree attention needs %zu workspace bytes", need);
  IG_REQUIRE(aligned(workspace, 256), "workspace must be 256-byte aligned");
  const TreeShape a{n, T, T_max, Hq, Hkv, Hq / Hkv, page, n_pages, seqs, max_pages, scale * 1.4426950408889634f, page_table, L_valid,
                    seq, first, reinterpret_cast<const unsigned long long*>(masks)};
  cudaStream_t st = as_stream(stream);
  if (dtype == IG_F16)
    return d == 128 ? launch_rows<false, 128>(st, a, q, K, V, out, lse, workspace)
                    : launch_rows<false, 64>(st, a, q, K, V, out, lse, workspace);
  return d == 128 ? launch_rows<true, 128>(st, a, q, K, V, out, lse, workspace)
                  : launch_rows<true, 64>(st, a, q, K, V, out, lse, workspace);
}
