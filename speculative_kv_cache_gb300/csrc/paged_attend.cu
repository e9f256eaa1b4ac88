// Attention of one new token per sequence over a paged KV cache.
//
// Mathematics.  For a key/value head and the G = Hq / Hkv query heads that read it,
//   z_t = scale q . K_t,  o = sum_t e^(z_t) V_t / sum_t e^(z_t)
// in one pass over the tokens: every part of the tokens keeps its maximum m, l = sum e^(z - m) and
// o = sum e^(z - m) V, and two parts join as m = max(m1, m2), l = sum l_i e^(m_i - m), o likewise.
// Exponents are taken to base 2, with log2(e) folded into the scale.
//
// What bounds it.  Every key and value is read once from HBM and used by G queries (once per 64 queries where
// G is larger): 4 d G flop for 4 d bytes.  From G = 8 on that is more than the fp32 units do at HBM speed, so the products run
// on the tensor cores.  Tokens are the 16 rows of an MMA (mma.sync), queries its 8 columns: S^T = K Q^T,
// then O^T = V^T P^T, which costs no padding at G = 8 and at G = 1 leaves the tensor cores far from
// full (13 % busy at G = 5).  A tcgen05 kernel with the queries as M (at most 64 of them, twice, in its M = 128;
// 72 cycles an MMA whether N is 64 or 128, and 500 more of waits for a tile's two dependent batches) was about
// equal: 26.5 to 27.5 us where this takes 23 (fp16) to 27 (bf16) (16 sequences of about 4050 tokens, G = 56), and
// 34 where this takes 35 (fp16) to 40 (bf16) (4 x 32768 tokens, G = 64).  Tokens as M were not tried on tcgen05.
//
// Precision.  K, V, q enter as they are.  A weight in fp16 or bf16 alone would cost 2^-11 or 2^-8, so
// it is split into 16-bit parts that are multiplied in turn: two for fp16 (20 bits or more), three for bf16 (24 bits).
// fp16 has few exponents: scaled by 2^15, two parts hold weights from 1 down to 2^-19.  Smaller ones must keep their
// bits too, as a large weight's value may be zero (a sink).  So the reference that weights are taken against need
// not be the largest logit: it follows a tile down, by a power of two, which fp32 sums stand (kPaHigh) and
// the next tiles then have for nothing; and the few weights of a tile that spans more go token by token
// in fp32.  (It costs nothing at 16 x 4050 tokens, 56 heads, 23.1 us; 64 x 2048 tokens, 20 heads 27.7 -> 28.7
// us; 16 x 4050 tokens, 33 heads of 64 15.1 -> 16.6 us.)  Sums over the
// tokens of one tile run in the tensor cores, whose adds need not round to nearest; those over tiles in
// fp32 adds that do, so that long sequences collect no bias.  (2-norm error against 64 bits 3e-7 to 6e-7,
// plain fp32 torch operations 2e-7 to 1.2e-6.)
//
// Work split.  The tokens of every (sequence, key head) are cut into tiles of 16 KB of keys and values,
// and CTA c of G takes tiles [R c / G, R (c+1) / G) of all R, in sequence and head order: equal shares
// whatever the lengths.  A head whose tiles lie in one CTA is finished there; a head cut by a CTA
// boundary leaves one partial per CTA in the workspace (two slots per CTA: the head it starts with
// and the head it ends with), joined in order by a second kernel, a programmatic dependent launch.
// No atomics: the result does not depend on timing.
//
// A CTA is one producer warp and three or four consumer warps, two CTAs to an SM.  The producer walks the
// tiles, looks the pages up a window of 32 ahead, and moves each tile with TMA (a page's rows of one head
// are contiguous; a box is their two 64-column halves, 128-byte swizzle) into a ring of stages; a stage is
// consumed by one warp (or, for more than 16 queries, by as many warps as it takes, each with its own
// queries), the stages in turn.  A warp folds its tiles into its own (m, l, o); the warps join where a
// head ends.
//
// Measured (device time, HBM copy rate 6.79 TB/s): 64 sequences of 0 to 8192 tokens, 8 key heads of 128, 1.08
// GB, bf16: 167 us, 6.4 TB/s, 0.95 of the copy rate; one of 131071 tokens, 537 MB, fp16: 85 us, 0.93; 8 of 2000
// tokens, 32 key heads, 260 MB, fp16: 43.4 us, 0.88 (47 us where its 256 heads were cut); heads of 64, 64 of 4096
// tokens, 32 heads on 8, 537 MB: 87 us, 0.91, either type; a launch costs 5 us beside its bytes (launch 2, first
// loads 2, tail 1) and the join 3; 4 heads of 256 tokens: 6.0 us.  16 of 4050 tokens, 56 heads on one key head, 33
// MB: 27 us in bf16, 23 in fp16, bound by the products (three and two parts of a weight) of one or two warps per
// scheduler, as 64 of 2048 tokens with 16 heads on one key head, 67 MB: 26 us, floor 10.  What the steps
// gave: page numbers in windows instead of per tile 190 -> 165 us and 58 -> 47 us (one producer warp had
// set the pace); four products side by side instead of one accumulator after the other 1550 -> 1150 cycles
// a tile; heads of a few tiles to one warp each 22.5 -> 13.9 us (104 x 17 heads of 3 tokens).
#include <cuda_bf16.h>
#include <math.h>

#include "ig_common.cuh"
#include "tc_common.cuh"

namespace ig {
namespace {

constexpr int kPaCtasPerSm = 2;
constexpr int kMaxPaCtas = 320;                   // upper bound of the grid (sizes the workspace)
constexpr int kPaStageBytes = 16384;              // keys and values of one tile
// Tiles of a head that one warp takes alone, where its CTA has other heads for the other warps (149 x 11
// heads of 106 to 212 tokens: 42.3 us at 2, 39.7 at 4, 38.2 at 8, where 167 x 6 heads of 397 lose 10 %).
constexpr int kPaSolo = 4;
// Heads that could have a CTA each are not cut where the longest has at most kPaWhole tiles (the join costs
// 2 us, a tile 0.8 us: 4 heads of 256 tokens take 7.4 us cut, 6.2 us whole), or where there are enough of
// them to keep HBM busy (one per SM) and the longest is at most kPaEven tiles above the mean.
constexpr int kPaWhole = 6;
constexpr int kPaEven = 3;
// Powers of two of fp16 weights that two 16-bit parts cover: 22 bits of the upper 17, 20 of all.  (17 in all, so that
// more tiles leave them: 16.3 -> 18.9 us for 16 x 4050 tokens, 33 heads of 64 on one key head.)
constexpr int kPaBand = 19;
constexpr float kPaLeast = -126.f;                // weights below 2^kPaLeast of the reference are zero, as ex2 has them
constexpr int kPaHigh = 95;                       // weights and their sums, times 2^15, stay near or below 2^kPaHigh
constexpr int kPaPartHead = 4;                    // a partial: [max, sum, -, -, output[D]]

template <int D>
__host__ __device__ constexpr int pa_tokens() { return kPaStageBytes / (4 * D); }  // tokens of a tile: 32 or 64
// warps that take stages in turn, and stages
__host__ __device__ constexpr int pa_turns(int WQ) { return WQ == 1 ? 3 : WQ == 2 ? 2 : 1; }
__host__ __device__ constexpr int pa_stages(int WQ) { return WQ == 1 ? 6 : WQ == 2 ? 4 : 5; }  // two CTAs per SM
__host__ __device__ constexpr int pa_threads(int WQ) { return (pa_turns(WQ) * WQ + 1) * 32; }
// joining warps' outputs held at once, per group of queries
__host__ __device__ constexpr int pa_slots(int NQ, int WQ) { return pa_turns(WQ) == 1 ? 0 : NQ == 1 ? 2 : 1; }

// Where the work is: everything the kernels need beside the pointers.
struct PaShape {
  int B, Hq, Hkv, G, QT;   // G query heads per key head, in QT groups of the unit's rows
  int page, n_pages, max_pages;
  int box;                 // rows of a TMA box, a power of two that divides page
  float scale2;            // scale * log2(e)
  int by_unit;             // info is indexed by unit (units <= CTAs) or by CTA
};

// shared memory behind the ring
template <int D, int NQ, int WQ>
struct PaShared {
  // joining warps' outputs, a lane's registers apart
  float merge[pa_slots(NQ, WQ) ? pa_slots(NQ, WQ) * WQ : 1][pa_slots(NQ, WQ) ? D / 16 * NQ * 4 : 1][32];
  // the warps' queries, where they would not fit the registers (rows 16 bytes apart in the banks)
  uint4 q[WQ > 1 ? WQ * pa_turns(WQ) : 1][WQ > 1 ? NQ * 8 : 1][WQ > 1 ? D / 8 + 1 : 1];
  float m[pa_turns(WQ) * WQ][NQ * 8], l[pa_turns(WQ) * WQ][NQ * 8];
  unsigned long long valid[pa_stages(WQ)];  // tokens of the stage that count
  uint32_t tile[pa_stages(WQ)];             // the tile (of the CTA's) it is for
  uint64_t full[pa_stages(WQ)], empty[pa_stages(WQ)];
  int scan[pa_threads(WQ) / 32][3];
  int start_b, start_off;
  int abort;
};

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// c += a b, 16 x 8 x 16
template <bool BF>
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if constexpr (BF)
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ float lds_half(uint32_t addr) {
  uint16_t v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(addr) : "memory");
  return __half2float(__ushort_as_half(v));
}

__device__ __forceinline__ float power_of_two(int e) { return __int_as_float((127 + e) << 23); }  // -126 <= e <= 127

// m += by, and the factor 2^(m before - m after) that keeps sums right: what the addition rounds off (Knuth's two-sum) is in it.
__device__ __forceinline__ float pa_move(float& m, int by) {
  const float b = (float)by, s = m + b, c = s - m, lost = (m - (s - c)) + (b - c);
  m = s;
  return power_of_two(-by) * fmaf(lost, 0.6931471805599453f, 1.f);
}

// Two fp32 as a pair of 16-bit values (x in the low half), and what the rounding left of them.
template <bool BF>
__device__ __forceinline__ uint32_t split2(float& x, float& y) {
  if constexpr (BF) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
    x -= __low2float(h);
    y -= __high2float(h);
    return *reinterpret_cast<const uint32_t*>(&h);
  } else {
    const __half2 h = __floats2half2_rn(x, y);
    x -= __low2float(h);
    y -= __high2float(h);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
}

template <int THREADS>
__device__ __forceinline__ void consumer_sync() {
  asm volatile("bar.sync 1, %0;" ::"n"(THREADS) : "memory");
}

// The producer's wait for a free stage; gives up together with the CTA's other waits.  A consumer that gave
// up frees stages whose copies it did not wait for, but sets `abort` first: the flag is read again after
// the wait, so that no such stage is filled while its copies are still in flight.
__device__ __forceinline__ bool pa_wait(uint64_t* bar, uint32_t parity, volatile int* abort, uint32_t limit) {
  for (uint32_t i = 0; i < limit && !*abort; ++i)
    if (mbar_try_wait(bar, parity)) return !*abort;
  return false;
}

// The same for tile x of a stage's barrier.  A stage's phases go to different warps, and a warp that has
// not followed them all cannot tell them by their parity; so the producer writes the tile's number
// once the phase before is over.
__device__ __forceinline__ bool pa_wait_tile(const volatile uint32_t* tile, uint32_t x, uint64_t* bar, uint32_t parity,
                                             volatile int* abort, uint32_t limit) {
  for (uint32_t i = 0; i < limit && !*abort; ++i)
    if (*tile == x && mbar_try_wait(bar, parity)) return true;
  return false;
}

// (The kernels here start before the ones before them have ended, so what those write is read by plain
// (ld.ca) loads, not by the read-only path, which asks for data that stay as they are for a kernel's whole life.)
//
// The tiles of a CTA's share, in order, head by head; all lanes of a warp walk together.
template <int TT>
struct PaWalk {
  const int32_t* L_valid;
  int B, per_seq, max_len;  // heads (times query groups) of a sequence; the table's length
  int whole;                // shares of whole heads
  int b, off, nt, L, left;  // sequence, tile in its work, tiles of a head, its length; tiles (heads) left
  int base, len_here, len_next;

  __device__ int bounded(int i) const {
    const int v = i < B ? __ldca(L_valid + i) : 0;
    return v < 0 ? 0 : v > max_len ? max_len : v;
  }
  __device__ void enter(int seq) {
    b = seq;
    L = __shfl_sync(0xffffffffu, len_here, seq - base);
    nt = (L + TT - 1) / TT;
  }
  __device__ void start(int seq, int offset, int tiles) {
    const int lane = threadIdx.x & 31;
    base = seq;
    len_here = bounded(base + lane);
    len_next = bounded(base + 32 + lane);
    start_here(seq, offset, tiles);
  }
  __device__ void start_here(int seq, int offset, int tiles) {  // with the lengths in hand
    left = tiles;
    enter(seq);
    off = whole ? offset * nt : offset;
  }
  // the head that the walk stands in
  __device__ int unit() const { return off / nt; }
  __device__ int tile() const { return off % nt; }
  __device__ int run() const { return whole ? nt - off % nt : min(nt - off % nt, left); }
  __device__ void advance(int n) {  // n <= run()
    off += n;
    left -= whole ? (off % nt == 0 ? 1 : 0) : n;
    if (left <= 0 || off < nt * per_seq) return;
    off = 0;
    const int lane = threadIdx.x & 31;
    unsigned more = __ballot_sync(0xffffffffu, len_here > 0 && base + lane > b);
    while (!more) {  // tiles are left, so a sequence with tokens follows
      base += 32;
      len_here = len_next;
      len_next = bounded(base + 32 + lane);
      more = __ballot_sync(0xffffffffu, len_here > 0);
      if (base >= B) break;
    }
    if (more) enter(base + __ffs(more) - 1);
    else left = 0;
  }
};

template <bool BF, int D, int NQ, int WQ>
__global__ void __launch_bounds__(pa_threads(WQ), kPaCtasPerSm) k_paged_attend(
    const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v,
    const uint16_t* __restrict__ q, const int32_t* __restrict__ table, const int32_t* __restrict__ L_valid,
    const PaShape s, float* __restrict__ out, float* __restrict__ lse, float* __restrict__ part,
    int2* __restrict__ info, int* err) {
  constexpr int TT = pa_tokens<D>(), MT = TT / 16, NS = pa_stages(WQ);
  constexpr int RU = 8 * NQ * WQ;          // query rows of a unit
  constexpr int TG = pa_turns(WQ);         // warps that take stages in turn
  constexpr int kPaThreads = pa_threads(WQ), kPaWarps = TG * WQ, SLOTS = pa_slots(NQ, WQ);
  constexpr bool QS = WQ > 1;              // queries in shared memory
  static_assert(!QS || NQ == 2, "ldmatrix takes the queries 16 at a time");
  constexpr int PARTS = BF ? 3 : 2;        // 16-bit parts of a weight
  constexpr uint32_t kKvBytes = kPaStageBytes / 2;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  unsigned char* ring = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                                         ~static_cast<uintptr_t>(1023));
  auto& sh = *reinterpret_cast<PaShared<D, NQ, WQ>*>(ring + NS * kPaStageBytes);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int per_seq = s.Hkv * s.QT, max_len = s.max_pages * s.page;
  pdl_trigger();

  // ---- this CTA's share of all tiles, and the sequence it starts in
  if (threadIdx.x == 0) {
    for (int i = 0; i < NS; ++i) {
      mbar_init(&sh.full[i], 1);
      mbar_init(&sh.empty[i], WQ);
      sh.tile[i] = ~0u;
    }
    sh.abort = 0;
    fence_mbar_init();
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  }
  pdl_wait();
  auto length = [&](int b) -> int {
    int L = __ldca(L_valid + b);
    if (L < 0 || L > max_len) {
      raise_error(err, IG_DEVERR_INDEX);
      L = L < 0 ? 0 : max_len;
    }
    return L;
  };
  // the sums before each thread's sequences (of tiles, and of sequences that have any): a sequence per lane
  // of every warp, or, for more than 32, a run of sequences per thread
  const bool few = s.B <= 32;
  const int per = few ? 1 : (s.B + kPaThreads - 1) / kPaThreads;
  const int b0 = min(s.B, (few ? lane : (int)threadIdx.x) * per), b1 = min(s.B, b0 + per);
  int tiles = 0, used = 0, longest = 0, len = 0;
  for (int b = b0; b < b1; ++b) {
    len = length(b);
    const int n = (len + TT - 1) / TT;
    tiles += n;
    used += n > 0;
    longest = max(longest, n);
  }
  int tiles_in = tiles, used_in = used;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, tiles_in, o), y2 = __shfl_up_sync(0xffffffffu, used_in, o);
    if (lane >= o) {
      tiles_in += y;
      used_in += y2;
    }
    longest = max(longest, __shfl_xor_sync(0xffffffffu, longest, o));
  }
  int tiles_before = tiles_in - tiles, used_before = used_in - used;
  int all_tiles = __shfl_sync(0xffffffffu, tiles_in, 31), all_used = __shfl_sync(0xffffffffu, used_in, 31);
  if (!few) {
    if (lane == 31) {
      sh.scan[warp][0] = tiles_in;
      sh.scan[warp][1] = used_in;
      sh.scan[warp][2] = longest;
    }
    __syncthreads();
    all_tiles = all_used = 0;
#pragma unroll
    for (int w = 0; w < kPaThreads / 32; ++w) {
      tiles_before += w < warp ? sh.scan[w][0] : 0;
      used_before += w < warp ? sh.scan[w][1] : 0;
      all_tiles += sh.scan[w][0];
      all_used += sh.scan[w][1];
      longest = max(longest, sh.scan[w][2]);
    }
  }
  // heads are cut, and shares counted in tiles; or not, and shares counted in heads
  const bool uncut = s.by_unit && (longest <= kPaWhole || (2 * all_used * per_seq >= (int)gridDim.x &&
                                                           (long long)longest * all_used <= all_tiles + kPaEven * all_used));
  auto share_of = [&](int L) -> int { return (uncut ? min(L, 1) : (L + TT - 1) / TT) * per_seq; };
  const int before = (uncut ? used_before : tiles_before) * per_seq, mine = (uncut ? used : tiles) * per_seq;
  const int total = (uncut ? all_used : all_tiles) * per_seq;
  // with fewer shares than CTAs the first `ctas` get one each
  const int ctas = min((int)gridDim.x, total), cta = blockIdx.x;
  int r0 = 0, r1 = 0;
  // CTA c's first share, total c / ctas, without a 64-bit division
  const unsigned each = ctas ? (unsigned)total / ctas : 0, rest = ctas ? (unsigned)total % ctas : 0;
  auto first_of = [&](unsigned c) -> int { return (int)(each * c + rest * c / (unsigned)ctas); };
  if (cta < ctas) {
    r0 = first_of(cta);
    r1 = first_of(cta + 1);
  }
  const bool here = r1 > r0 && r0 >= before && r0 < before + mine;  // it starts in this thread's sequences
  PaWalk<TT> w;
  w.L_valid = L_valid;
  w.B = s.B;
  w.per_seq = per_seq;
  w.max_len = max_len;
  w.whole = uncut;
  w.b = w.off = w.L = w.left = 0;
  w.nt = 1;
  if (few) {
    const unsigned at = __ballot_sync(0xffffffffu, here);
    w.base = 0;
    w.len_here = len;
    w.len_next = 0;
    if (at) {
      const int seq = __ffs(at) - 1;
      w.start_here(seq, r0 - __shfl_sync(0xffffffffu, before, seq), r1 - r0);
    }
    __syncthreads();  // the barriers are set up
  } else {
    if (here) {
      int at = before;
      for (int b = b0; b < b1; ++b) {
        const int n = share_of(length(b));
        if (r0 < at + n) {
          sh.start_b = b;
          sh.start_off = r0 - at;
          break;
        }
        at += n;
      }
    }
    __syncthreads();
    if (r1 > r0) w.start(sh.start_b, sh.start_off, r1 - r0);
  }

  uint32_t sent = 0;  // the producer's tiles
  if (warp == kPaWarps) {
    // ---- producer.  The tiles of a head are taken in windows of 32 pages, a page number per lane;
    // the next window's numbers are loaded while this one's tiles go out.  Of a tile, lane i moves
    // box i / 2 of the keys (even i) or values.
    const int boxes = TT / s.box, box_at = lane / 2 * s.box, is_v = lane & 1;
    const int jump = TT / s.page, step = TT % s.page;  // a tile further: pages and rows
    const uint32_t box_bytes = (uint32_t)s.box * D * 2;
    // tiles from where `at` stands that 32 pages cover, and the lane's page number
    auto window = [&](const PaWalk<TT>& at, int& first, int& id) -> int {
      const int tile = at.tile();
      first = tile * TT / s.page;
      const long long covered = ((long long)first + 32) * s.page / TT - tile;
      const bool in = (long long)(first + lane) * s.page < at.L;
      id = in ? __ldca(table + (size_t)at.b * s.max_pages + first + lane) : -1;
      const int run = at.run();
      return covered < run ? (int)covered : run;
    };
    uint32_t st = 0, round = 0, it = 0;
    int first = 0, ids = -1, n = w.left > 0 ? window(w, first, ids) : 0;
    bool going = true;
    while (n > 0 && going) {
      const int tile = w.tile(), hk = w.unit() / s.QT, L = w.L;
      w.advance(n);
      int first2 = 0, ids2 = -1;
      const int n2 = w.left > 0 ? window(w, first2, ids2) : 0;
      int tokens = L - tile * TT;                  // from this tile on
      int pg = (tile * TT + box_at) / s.page;      // this lane's page and row in it
      int row = (tile * TT + box_at) - pg * s.page;
      pg -= first;
      for (int i = 0; i < n; ++i) {
        const int g = __shfl_sync(0xffffffffu, ids, pg & 31);
        const bool want = lane < 2 * boxes && box_at < tokens;
        const bool ok = want && g >= 0 && g < s.n_pages;
        const unsigned moving = __ballot_sync(0xffffffffu, ok), bad = __ballot_sync(0xffffffffu, want && !ok);
        const bool freed = round == 0 || pa_wait(&sh.empty[st], (round - 1) & 1, &sh.abort, (uint32_t)kDefaultWaitIters);
        if (!__all_sync(0xffffffffu, freed)) {  // one verdict for the warp
          if (lane == 0) {
            sh.abort = 1;
            raise_error(err, IG_DEVERR_TIMEOUT);
          }
          going = false;
          break;
        }
        if (lane == 0) {
          const int live = min(tokens, TT);
          unsigned long long v = live >= 64 ? ~0ull : (1ull << live) - 1;
          if (bad) {
            raise_error(err, IG_DEVERR_INDEX);
            for (unsigned m = bad & 0x55555555u; m; m &= m - 1)
              v &= ~((s.box >= 64 ? ~0ull : (1ull << s.box) - 1) << ((__ffs(m) - 1) / 2 * s.box));
          }
          sh.valid[st] = v;
          *(volatile uint32_t*)&sh.tile[st] = it;
          mbar_arrive_expect_tx(&sh.full[st], (uint32_t)__popc(moving) * box_bytes);
        }
        __syncwarp();
        if (ok)
          tma_load_3d(ring + st * kPaStageBytes + is_v * kKvBytes + box_at * (D * 2), is_v ? &map_v : &map_k, 0,
                      (g * s.Hkv + hk) * s.page + row, 0, &sh.full[st]);
        ++it;
        if (++st == NS) {
          st = 0;
          ++round;
        }
        tokens -= TT;
        pg += jump;
        row += step;
        if (row >= s.page) {
          row -= s.page;
          ++pg;
        }
      }
      n = n2;
      first = first2;
      ids = ids2;
    }
    sent = it;
  } else {
    // ---- consumers: warp = tg + TG * wq takes stages tg, tg + TG, ... for query rows wq
    const int tg = warp % TG, wq = warp / TG;
    const int gl = lane >> 2, tl = lane & 3;  // fragment row and column pair
    const uint32_t limit = wait_limit(err);
    // ldmatrix rows of this lane: keys (16 tokens x 16 columns), values transposed
    const uint32_t k_chunk = lane >> 4, v_chunk = (lane >> 3) & 1, swz = lane & 7, half_bytes = s.box * 128;
    uint32_t k_row[MT], v_row[MT];  // where one box after the other puts them
#pragma unroll
    for (int i = 0; i < MT; ++i) {
      auto at = [&](int r) -> uint32_t { return r / s.box * (s.box * D * 2) + r % s.box * 128; };
      k_row[i] = at(i * 16 + (lane & 7) + ((lane >> 3) & 1) * 8);
      v_row[i] = at(i * 16 + (lane & 7) + (lane >> 4) * 8);
    }
    const uint32_t q_row = QS ? smem_addr(&sh.q[warp][(lane & 7) + (lane >> 4) * 8][(lane >> 3) & 1]) : 0u;
    uint32_t it = 0;  // tile of this CTA
    bool cut = false;
    for (uint32_t seg = 0; w.left > 0; ++seg) {
      const int u_in = w.unit(), hk = u_in / s.QT, qt = u_in % s.QT, b = w.b;
      const int tile0 = w.tile(), nt = w.nt, run = w.run();
      const bool done = tile0 == 0 && run == nt;  // all of the head is here
      cut = tile0 == 0 && !done;                  // it goes on in later CTAs
      w.advance(run);
      // a few tiles are one warp's own (warps then work on different heads and need not meet)
      const bool solo = TG > 1 && run <= kPaSolo && (seg > 0 || w.left > 0);
      const int owner = solo ? seg % TG : 0;
      if (solo && tg != owner) {
        it += run;
        continue;
      }
      const int qrow = qt * RU + wq * 8 * NQ;  // of this warp, within the key head's G
      const uint16_t* qp = q + ((size_t)b * s.Hq + (size_t)hk * s.G + qrow) * D;
      uint32_t qf[QS ? 1 : D / 16][NQ][2];
      if constexpr (QS) {
        uint4 v[NQ * D / 32];  // all on their way before the first is put down
#pragma unroll
        for (int i = 0; i < NQ * D / 32; ++i) {
          const int r = (i * 32 + lane) / (D / 8), c = (i * 32 + lane) % (D / 8);
          v[i] = qrow + r < s.G ? __ldca(reinterpret_cast<const uint4*>(qp + (size_t)r * D) + c) : make_uint4(0, 0, 0, 0);
        }
        __syncwarp();
#pragma unroll
        for (int i = 0; i < NQ * D / 32; ++i) sh.q[warp][(i * 32 + lane) / (D / 8)][(i * 32 + lane) % (D / 8)] = v[i];
        __syncwarp();
      } else {
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks)
#pragma unroll
          for (int j = 0; j < NQ; ++j) {
            const bool in = qrow + j * 8 + gl < s.G;
            const uint16_t* p = qp + (size_t)(j * 8 + gl) * D + ks * 16 + tl * 2;
            qf[ks][j][0] = in ? __ldca(reinterpret_cast<const uint32_t*>(p)) : 0u;
            qf[ks][j][1] = in ? __ldca(reinterpret_cast<const uint32_t*>(p + 8)) : 0u;
          }
      }
      float m[NQ][2], l[NQ][2], o[D / 16][NQ][4];
#pragma unroll
      for (int j = 0; j < NQ; ++j) {
        m[j][0] = m[j][1] = -INFINITY;
        l[j][0] = l[j][1] = 0.f;
#pragma unroll
        for (int i = 0; i < D / 16; ++i) o[i][j][0] = o[i][j][1] = o[i][j][2] = o[i][j][3] = 0.f;
      }
      // this warp's stages of the run
      for (uint32_t x = solo ? it : it + (tg + TG - it % TG) % TG; x < it + run; x += solo ? 1 : TG) {
        const uint32_t st = x % NS;
        if (!pa_wait_tile(&sh.tile[st], x, &sh.full[st], (x / NS) & 1, &sh.abort, limit)) {
          if (lane == 0 && !atomicExch(&sh.abort, 1)) raise_error(err, IG_DEVERR_TIMEOUT);
          // the walk goes on without waiting, so that every warp meets the others' barriers
        }
        __syncwarp();
        const uint32_t kb = smem_addr(ring + st * kPaStageBytes), vb = kb + kKvBytes;
        const unsigned long long valid = sh.valid[st];
        const bool whole = valid == (TT == 64 ? ~0ull : (1ull << TT) - 1);
        // (a product depends on the one before it in its accumulator: at least four accumulators in turn)
        constexpr int ZC = MT * NQ >= 4 ? 1 : 2;
        float zc[ZC][MT][NQ][4];
#pragma unroll
        for (int c = 0; c < ZC; ++c)
#pragma unroll
          for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int j = 0; j < NQ; ++j) zc[c][i][j][0] = zc[c][i][j][1] = zc[c][i][j][2] = zc[c][i][j][3] = 0.f;
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
          uint32_t b[4];
          if constexpr (QS) {
            ldsm4(b, q_row + ks * 32);
          } else {
#pragma unroll
            for (int j = 0; j < NQ; ++j) {
              b[2 * j] = qf[ks][j][0];
              b[2 * j + 1] = qf[ks][j][1];
            }
          }
#pragma unroll
          for (int i = 0; i < MT; ++i) {
            uint32_t a[4];
            ldsm4(a, kb + (ks / 4) * half_bytes + k_row[i] + ((((ks % 4) * 2 + k_chunk) ^ swz) << 4));
#pragma unroll
            for (int j = 0; j < NQ; ++j) mma16816<BF>(zc[ks % ZC][i][j], a, b[2 * j], b[2 * j + 1]);
          }
        }
        float z[MT][NQ][4];
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
          for (int j = 0; j < NQ; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) z[i][j][e] = (ZC == 2 ? zc[0][i][j][e] + zc[ZC - 1][i][j][e] : zc[0][i][j][e]) * s.scale2;
        if (!whole) {
#pragma unroll
          for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const bool in = (valid >> (i * 16 + gl + (e >> 1) * 8)) & 1;
#pragma unroll
              for (int j = 0; j < NQ; ++j) z[i][j][e] = in ? z[i][j][e] : -INFINITY;
            }
        }
        // The running maximum; most tiles of a long sequence leave it as it is.  For fp16 it is a reference, that
        // follows the tiles down too where their weights would fall below what the parts hold.
        float tm[NQ][2], ym[NQ][2];
        bool look = false;
#pragma unroll
        for (int j = 0; j < NQ; ++j)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float x2 = fmaxf(z[0][j][e], z[0][j][e + 2]), y2 = fminf(z[0][j][e], z[0][j][e + 2]);
#pragma unroll
            for (int i = 1; i < MT; ++i) {
              x2 = fmaxf(x2, fmaxf(z[i][j][e], z[i][j][e + 2]));
              y2 = fminf(y2, fminf(z[i][j][e], z[i][j][e + 2]));
            }
            tm[j][e] = x2;
            ym[j][e] = y2;
            look |= x2 > m[j][e];
          }
        if constexpr (!BF) {
#pragma unroll
          for (int j = 0; j < NQ; ++j)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              if (!whole) {  // (of the tokens that count)
                float y2 = INFINITY;
#pragma unroll
                for (int i = 0; i < 2 * MT; ++i) {
                  const float v = z[i / 2][j][i % 2 * 2 + e];
                  y2 = fminf(y2, v > -INFINITY ? v : INFINITY);
                }
                ym[j][e] = y2;
              }
              look |= ym[j][e] < m[j][e] - kPaBand;
            }
        }
        float corr[NQ][2];
#pragma unroll
        for (int j = 0; j < NQ; ++j) corr[j][0] = corr[j][1] = 1.f;
        if (__any_sync(0xffffffffu, look)) {
          bool low = false;
#pragma unroll
          for (int j = 0; j < NQ; ++j)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              float x2 = tm[j][e];
#pragma unroll
              for (int sh2 = 4; sh2 < 32; sh2 <<= 1) x2 = fmaxf(x2, __shfl_xor_sync(0xffffffffu, x2, sh2));
              const float mn = fmaxf(m[j][e], x2);
              corr[j][e] = mn == -INFINITY ? 1.f : ex2(m[j][e] - mn);
              m[j][e] = mn;
              l[j][e] *= corr[j][e];
              if constexpr (!BF) {
                tm[j][e] = x2;
                low |= ym[j][e] < mn - kPaBand;
              }
            }
          if constexpr (!BF) {
            if (__any_sync(0xffffffffu, low)) {
              bool far = false;
#pragma unroll
              for (int j = 0; j < NQ; ++j)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                  float y2 = INFINITY, sum = l[j][e];  // the least logit whose weight is not zero
#pragma unroll
                  for (int i = 0; i < 2 * MT; ++i) {
                    const float v = z[i / 2][j][i % 2 * 2 + e];
                    y2 = fminf(y2, v - m[j][e] > kPaLeast ? v : INFINITY);
                  }
#pragma unroll
                  for (int sh2 = 4; sh2 < 32; sh2 <<= 1) {
                    y2 = fminf(y2, __shfl_xor_sync(0xffffffffu, y2, sh2));
                    sum += __shfl_xor_sync(0xffffffffu, sum, sh2);
                  }
                  // The reference goes down by a power of two.  Where the column's logits fit the parts, they come to lie
                  // in the middle; else it goes next to the largest, or, where more of them are in the lower half (a
                  // sink's tile), so far that the least fits.
                  const float span = tm[j][e] - y2, half = 0.5f * (tm[j][e] + y2);
                  int upper = 0;
#pragma unroll
                  for (int i = 0; i < 2 * MT; ++i) {
                    const float v = z[i / 2][j][i % 2 * 2 + e];
                    upper += v > half ? 1 : v >= y2 ? -1 : 0;
                  }
#pragma unroll
                  for (int sh2 = 4; sh2 < 32; sh2 <<= 1) upper += __shfl_xor_sync(0xffffffffu, upper, sh2);
                  if (y2 < m[j][e] - kPaBand) {
                    const float to = span < kPaBand - 1 ? fminf(half + 0.5f * kPaBand, y2 + (kPaBand - 1))
                                     : upper >= 0       ? tm[j][e]
                                                        : y2 + (kPaBand - 1);
                    const float room = (float)(kPaHigh + min(-16, 127 - (__float_as_int(sum) >> 23)));
                    const float down = fminf(floorf(m[j][e] - to), room);
                    if (down > 0.f && fabsf(m[j][e]) < 0x1p22f) {  // (where a float still tells one power from the next)
                      const float up = pa_move(m[j][e], -(int)down);
                      l[j][e] *= up;
                      corr[j][e] *= up;
                    }
                    far |= y2 < m[j][e] - kPaBand || tm[j][e] > m[j][e];
                  }
                }
              if (__any_sync(0xffffffffu, far)) {
                // weights that stay outside the parts: token by token, in fp32, and then as zeros
#pragma unroll
                for (int i = 0; i < D / 16; ++i)
#pragma unroll
                  for (int j = 0; j < NQ; ++j)
#pragma unroll
                    for (int e = 0; e < 4; ++e) o[i][j][e] *= corr[j][e & 1];
#pragma unroll
                for (int j = 0; j < NQ; ++j) corr[j][0] = corr[j][1] = 1.f;
                auto outside = [&](float v, float r) { return (v < r - kPaBand || v > r) && v - r > kPaLeast; };
                unsigned groups = 0;  // of eight tokens
#pragma unroll
                for (int i = 0; i < 2 * MT; ++i)
#pragma unroll
                  for (int j = 0; j < NQ; ++j)
#pragma unroll
                    for (int e = 0; e < 2; ++e) groups |= outside(z[i / 2][j][i % 2 * 2 + e], m[j][e]) ? 1u << i : 0u;
                for (groups = __reduce_or_sync(0xffffffffu, groups); groups; groups &= groups - 1) {
                  const int r8 = __ffs(groups) - 1;
                  float wt[NQ][2];
                  bool some = false;
#pragma unroll
                  for (int j = 0; j < NQ; ++j)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                      float v = z[0][j][e];
#pragma unroll
                      for (int i = 1; i < 2 * MT; ++i) v = i == r8 ? z[i / 2][j][i % 2 * 2 + e] : v;
                      const bool it_is = outside(v, m[j][e]);
                      wt[j][e] = it_is ? ex2(v - m[j][e]) * 32768.f : 0.f;
                      l[j][e] += wt[j][e];
                      some |= it_is;
                    }
                  for (unsigned left = __ballot_sync(0xffffffffu, some); left;) {
                    const int g = (__ffs(left) - 1) >> 2, r = r8 * 8 + g;
                    left &= ~(15u << (4 * g));
                    float wg[NQ][2];
#pragma unroll
                    for (int j = 0; j < NQ; ++j)
#pragma unroll
                      for (int e = 0; e < 2; ++e) wg[j][e] = __shfl_sync(0xffffffffu, wt[j][e], 4 * g + tl);
                    const uint32_t row = vb + r / s.box * (s.box * D * 2) + r % s.box * 128 + gl * 2;
#pragma unroll
                    for (int dt = 0; dt < D / 16; ++dt)
#pragma unroll
                      for (int hh = 0; hh < 2; ++hh) {
                        const float v = lds_half(row + (dt / 4) * half_bytes + ((((dt % 4) * 2 + hh) ^ g) << 4));
#pragma unroll
                        for (int j = 0; j < NQ; ++j)
#pragma unroll
                          for (int e = 0; e < 2; ++e) o[dt][j][2 * hh + e] = fmaf(wg[j][e], v, o[dt][j][2 * hh + e]);
                      }
                  }
                }
#pragma unroll
                for (int i = 0; i < MT; ++i)
#pragma unroll
                  for (int j = 0; j < NQ; ++j)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                      const float v = z[i][j][e], r = m[j][e & 1];
                      z[i][j][e] = v < r - kPaBand || (v > r && r > -INFINITY) ? -INFINITY : v;
                    }
              }
            }
          }
        }
        // the weights, as 16-bit parts in the layout of the second product's operand
        uint32_t p[PARTS][MT][NQ][2];
#pragma unroll
        for (int j = 0; j < NQ; ++j) {
          const float m0 = m[j][0] == -INFINITY ? 0.f : m[j][0], m1 = m[j][1] == -INFINITY ? 0.f : m[j][1];
#pragma unroll
          for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int hh = 0; hh < 2; ++hh) {
              float x0 = ex2(z[i][j][2 * hh] - m0), x1 = ex2(z[i][j][2 * hh + 1] - m1);
              if constexpr (!BF) {
                x0 *= 32768.f;
                x1 *= 32768.f;
              }
              l[j][0] += x0;
              l[j][1] += x1;
#pragma unroll
              for (int pp = 0; pp < PARTS; ++pp) p[pp][i][j][hh] = transpose8(split2<BF>(x0, x1));
            }
        }
        // DG column tiles side by side, for the same reason (four of 16 queries where registers allow: 27.2 ->
        // 26 us for 64 x 2048 tokens, 16 heads, bf16)
        constexpr int DG = WQ == 1 ? 4 : 2;
#pragma unroll
        for (int d0 = 0; d0 < D / 16; d0 += DG) {
          float acc[DG][NQ][4];
#pragma unroll
          for (int x = 0; x < DG; ++x)
#pragma unroll
            for (int j = 0; j < NQ; ++j) acc[x][j][0] = acc[x][j][1] = acc[x][j][2] = acc[x][j][3] = 0.f;
#pragma unroll
          for (int i = 0; i < MT; ++i) {
            uint32_t a[DG][4];
#pragma unroll
            for (int x = 0; x < DG; ++x) {
              const int dt = d0 + x;
              ldsm4_t(a[x], vb + (dt / 4) * half_bytes + v_row[i] + ((((dt % 4) * 2 + v_chunk) ^ swz) << 4));
            }
            if (!whole) {  // rows that do not count may hold anything: zero times NaN is NaN
              const unsigned v0 = (unsigned)(valid >> (i * 16 + tl * 2)) & 3u, v1 = (unsigned)(valid >> (i * 16 + 8 + tl * 2)) & 3u;
              const uint32_t k0 = (v0 & 1 ? 0xffffu : 0u) | (v0 & 2 ? 0xffff0000u : 0u);
              const uint32_t k1 = (v1 & 1 ? 0xffffu : 0u) | (v1 & 2 ? 0xffff0000u : 0u);
#pragma unroll
              for (int x = 0; x < DG; ++x) {
                a[x][0] &= k0;
                a[x][1] &= k0;
                a[x][2] &= k1;
                a[x][3] &= k1;
              }
            }
#pragma unroll
            for (int pp = 0; pp < PARTS; ++pp)
#pragma unroll
              for (int x = 0; x < DG; ++x)
#pragma unroll
                for (int j = 0; j < NQ; ++j) mma16816<BF>(acc[x][j], a[x], p[pp][i][j][0], p[pp][i][j][1]);
          }
#pragma unroll
          for (int x = 0; x < DG; ++x)
#pragma unroll
            for (int j = 0; j < NQ; ++j)
#pragma unroll
              for (int e = 0; e < 4; ++e) o[d0 + x][j][e] = fmaf(o[d0 + x][j][e], corr[j][e & 1], acc[x][j][e]);
        }
        __syncwarp();
        if (lane == 0)
          asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_addr(&sh.empty[st])) : "memory");
      }
      it += run;
      // ---- the head's end in this CTA: the sums of a query's lanes, then the warps
#pragma unroll
      for (int j = 0; j < NQ; ++j)
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
          for (int sh2 = 4; sh2 < 32; sh2 <<= 1) l[j][e] += __shfl_xor_sync(0xffffffffu, l[j][e], sh2);
      // A reference that followed the tiles down goes back to about the largest logit, so that other warps' and CTAs'
      // are not so far above it that the factor between them is zero.  (2^20: more than a sum of weights
      // of at most 1 usually is.)
      if constexpr (!BF) {
#pragma unroll
        for (int j = 0; j < NQ; ++j)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int up = (__float_as_int(l[j][e]) >> 23) - 127 - 15;
            if (up > 20 && up < kPaHigh) {
              const float f = pa_move(m[j][e], up);
              l[j][e] *= f;
#pragma unroll
              for (int i = 0; i < D / 16; ++i) {
                o[i][j][e] *= f;
                o[i][j][e + 2] *= f;
              }
            }
          }
      }
      if (TG > 1 && !solo) {
        if (gl == 0)
#pragma unroll
          for (int j = 0; j < NQ; ++j)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              sh.m[warp][j * 8 + tl * 2 + e] = m[j][e];
              sh.l[warp][j * 8 + tl * 2 + e] = l[j][e];
            }
        consumer_sync<kPaWarps * 32>();
#pragma unroll
        for (int j = 0; j < NQ; ++j)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int c = j * 8 + tl * 2 + e;
            float M = -INFINITY, Ls = 0.f;
#pragma unroll
            for (int x = 0; x < TG; ++x) M = fmaxf(M, sh.m[wq * TG + x][c]);
            const float m0 = M == -INFINITY ? 0.f : M;
#pragma unroll
            for (int x = 0; x < TG; ++x) Ls += sh.l[wq * TG + x][c] * ex2(sh.m[wq * TG + x][c] - m0);
            const float f = ex2(m[j][e] - m0);
#pragma unroll
            for (int i = 0; i < D / 16; ++i) {
              o[i][j][e] *= f;
              o[i][j][e + 2] *= f;
            }
            m[j][e] = M;
            l[j][e] = Ls;
          }
        // into warp tg = 0, in the warps' order
#pragma unroll
        for (int from = 1; from < TG; from += SLOTS) {
          if (tg >= from && tg < from + SLOTS)
#pragma unroll
            for (int i = 0; i < D / 16; ++i)
#pragma unroll
              for (int j = 0; j < NQ; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) sh.merge[wq * SLOTS + tg - from][(i * NQ + j) * 4 + e][lane] = o[i][j][e];
          consumer_sync<kPaWarps * 32>();
          if (tg == 0)
#pragma unroll
            for (int x = 0; x < SLOTS && from + x < TG; ++x)
#pragma unroll
              for (int i = 0; i < D / 16; ++i)
#pragma unroll
                for (int j = 0; j < NQ; ++j)
#pragma unroll
                  for (int e = 0; e < 4; ++e) o[i][j][e] += sh.merge[wq * SLOTS + x][(i * NQ + j) * 4 + e][lane];
          if (from + SLOTS < TG) consumer_sync<kPaWarps * 32>();
        }
      }
      const int unit = b * per_seq + u_in;
      if (tg == owner) {
#pragma unroll
        for (int j = 0; j < NQ; ++j)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int row = wq * 8 * NQ + j * 8 + tl * 2 + e, qi = qt * RU + row;
            if (qi >= s.G) continue;
            if (done) {
              const size_t at = (size_t)b * s.Hq + (size_t)hk * s.G + qi;
              const float inv = l[j][e] == 0.f ? 0.f : 1.f / l[j][e];
#pragma unroll
              for (int i = 0; i < D / 16; ++i) {
                out[at * D + i * 16 + gl] = o[i][j][e] * inv;
                out[at * D + i * 16 + 8 + gl] = o[i][j][e + 2] * inv;
              }
              if (lse && gl == 0) lse[at] = (m[j][e] + log2f(l[j][e]) - (BF ? 0.f : 15.f)) * 0.6931471805599453f;
            } else {
              // the head it starts with, begun by an earlier CTA, to slot 0; one it begins to slot 1
              float* wp = part + ((size_t)(2 * cta + (tile0 == 0 ? 1 : 0)) * RU + row) * (D + kPaPartHead);
#pragma unroll
              for (int i = 0; i < D / 16; ++i) {
                wp[kPaPartHead + i * 16 + gl] = o[i][j][e];
                wp[kPaPartHead + i * 16 + 8 + gl] = o[i][j][e + 2];
              }
              if (gl == 0) {
                wp[0] = m[j][e];
                wp[1] = l[j][e];
              }
            }
          }
      }
      // what the second kernel joins: a head that begins here and goes on in later CTAs
      if (tg == owner && wq == 0 && lane == 0 && (cut || (s.by_unit && done))) {
        int last = cta;  // the CTA that holds the head's last tile
        if (cut) {
          const int end = r1 - run + nt - 1;  // its last tile: a cut head is this CTA's last
          last = min(ctas - 1, (int)((float)end * ((float)ctas / (float)total)));  // within 1
          while (last + 1 < ctas && first_of(last + 1) <= end) ++last;
          while (first_of(last) > end) --last;
        }
        if (s.by_unit) info[unit] = make_int2(cut ? cta : -1, last);
        else info[cta] = make_int2(unit, last);
      }
    }
    if (threadIdx.x == 0 && !s.by_unit && !cut) info[cta] = make_int2(-1, 0);
    // sequences without a token
    for (int b = cta; b < s.B; b += gridDim.x) {
      if (__ldca(L_valid + b) > 0) continue;
      for (int i = threadIdx.x; i < s.Hq * D / 4; i += kPaWarps * 32)
        reinterpret_cast<float4*>(out + (size_t)b * s.Hq * D)[i] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (lse)
        for (int i = threadIdx.x; i < s.Hq; i += kPaWarps * 32) lse[(size_t)b * s.Hq + i] = -INFINITY;
      if (s.by_unit)
        for (int i = threadIdx.x; i < per_seq; i += kPaWarps * 32) info[b * per_seq + i] = make_int2(-1, 0);
    }
  }
  __syncthreads();
  // Where a wait ran out, copies may be in flight that no consumer waited for: they land before the CTA leaves,
  // and its shared memory is another's.  Only here, where every consumer is done, is it known whether one gave up.
  if (warp == kPaWarps && *(volatile int*)&sh.abort)
    for (uint32_t x = 0; x < NS && x < sent; ++x) mbar_wait_bounded(&sh.full[x], ((sent - 1 - x) / NS) & 1);
}

// Joins the partials of the heads that were cut: block (x, y) takes unit x (or the head that CTA x
// began) and rows y * RB ... of it, WPR warps a row; a warp takes every WPR-th partial in order, and the
// warps join in order.  A warp a row where a head would have few partials if every slot of the batch had
// tokens (blocks of four warps, which fit beside the attention's: 1 us less than eight); with about 16 or more,
// four warps, with 64 or more, sixteen.  (The host does not know the lengths: few long sequences in many
// slots have more partials than that, joined by one warp a row.)
template <int D, int WPR, int RB>
__global__ void __launch_bounds__(WPR * RB * 32) k_paged_join(const float* __restrict__ part, const int2* __restrict__ info,
                                                             const PaShape s, int RU, float scale_bits,
                                                             float* __restrict__ out, float* __restrict__ lse) {
  constexpr int VEC = D / 32;
  __shared__ float sm[WPR * RB], sl[WPR * RB], so[WPR * RB][WPR > 1 ? D : 1];
  pdl_trigger();
  pdl_wait();
  const int2 e = __ldca(info + blockIdx.x);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (e.x < 0) return;
  const int unit = s.by_unit ? (int)blockIdx.x : e.x, c0 = s.by_unit ? e.x : (int)blockIdx.x;
  const int per_seq = s.Hkv * s.QT, b = unit / per_seq, hk = unit % per_seq / s.QT, qt = unit % s.QT;
  const int row = blockIdx.y * RB + warp / WPR, qi = qt * RU + row, n = e.y - c0 + 1;
  const bool live = row < RU && qi < s.G;
  float m = -INFINITY, l = 0.f, o[VEC];
#pragma unroll
  for (int i = 0; i < VEC; ++i) o[i] = 0.f;
  if (live) {
    // this warp's partials are w0, w0 + WPR, ...: 32 maxima and sums at a time (one per lane), outputs U at
    // a time, the first U on their way before the maxima are there
    constexpr int U = 8;
    const int w0 = warp % WPR, mine = (n - w0 + WPR - 1) / WPR;
    auto at = [&](int i) -> const float* {
      const int j = w0 + i * WPR;
      return part + ((size_t)(2 * (c0 + j) + (j == 0 ? 1 : 0)) * RU + row) * (D + kPaPartHead);
    };
    auto load = [&](int i0, float (&v)[U][VEC]) {
#pragma unroll
      for (int x = 0; x < U; ++x) {
        if (i0 + x < mine) {
          const float* p = at(i0 + x) + kPaPartHead + lane * VEC;
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
      const float f = ex2(m - m0), g = ex2(h.x - m0);
      float sum = h.y * g;
#pragma unroll
      for (int x = 16; x; x >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, x);
      l = l * f + sum;
#pragma unroll
      for (int i = 0; i < VEC; ++i) o[i] *= f;
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
      const float f = ex2(sm[warp + x] - m0);
      l += sl[warp + x] * f;
#pragma unroll
      for (int i = 0; i < VEC; ++i) o[i] += so[warp + x][lane * VEC + i] * f;
    }
  }
  if (!live) return;
  const size_t at = (size_t)b * s.Hq + (size_t)hk * s.G + qi;
  const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
  for (int i = 0; i < VEC; ++i) out[at * D + lane * VEC + i] = o[i] * inv;
  if (lse && lane == 0) lse[at] = (m + log2f(l) - scale_bits) * 0.6931471805599453f;
}

// query rows of a unit: 8 per MMA column tile, up to two tiles a warp, then more warps
inline int pa_rows(int G) { return G <= 8 ? 8 : G <= 16 ? 16 : G <= 32 ? 32 : 64; }

// workspace: two partials per CTA, then the join's list
inline size_t pa_part_bytes(int G, int d) {
  return round_up((size_t)2 * kMaxPaCtas * pa_rows(G) * (d + kPaPartHead) * sizeof(float), 256);
}
inline size_t pa_info_bytes() { return round_up((size_t)kMaxPaCtas * sizeof(int2), 256); }

template <bool BF, int D, int NQ, int WQ>
ig_status launch_paged(cudaStream_t st, PaShape s, const uint16_t* q, const uint16_t* K, const uint16_t* V,
                       const int32_t* table, const int32_t* L, float* out, float* lse, void* ws) {
  constexpr int RU = 8 * NQ * WQ, TT = pa_tokens<D>();
  s.QT = (s.G + RU - 1) / RU;
  s.box = TT;
  while (s.page % s.box) s.box >>= 1;
  const long long most = (long long)s.B * ((s.max_pages * s.page + TT - 1) / TT) * s.Hkv * s.QT;
  IG_REQUIRE(most < (1ll << 31), "B*max_pages*page*Hkv is too large: %lld tiles", most);
  const int rows = s.n_pages * s.Hkv * s.page;
  CUtensorMap mk, mv;
  ig_status r = make_map_halves(&mk, K, rows, D, s.box);
  if (r == IG_OK) r = make_map_halves(&mv, V, rows, D, s.box);
  if (r != IG_OK) return r;
  constexpr size_t smem = 1024 + (size_t)pa_stages(WQ) * kPaStageBytes + sizeof(PaShared<D, NQ, WQ>);
  cudaError_t e = cudaFuncSetAttribute(k_paged_attend<BF, D, NQ, WQ>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       (int)smem);
  if (e != cudaSuccess) return cuda_fail(e, "paged attention smem attribute");
  int grid = kPaCtasPerSm * sm_count(st);
  if (grid > kMaxPaCtas) grid = kMaxPaCtas;
  if (grid > most) grid = (int)most;
  const long long units = (long long)s.B * s.Hkv * s.QT;
  s.by_unit = units <= grid ? 1 : 0;
  float* part = static_cast<float*>(ws);
  int2* info = reinterpret_cast<int2*>(static_cast<char*>(ws) + pa_part_bytes(s.G, D));
  // a programmatic dependent launch: its CTAs set up while the kernel before it in the stream drains
  e = launch_pdl(k_paged_attend<BF, D, NQ, WQ>, dim3(grid), dim3(pa_threads(WQ)), smem, st, mk, mv, q, table, L, s, out,
                 lse, part, info, error_word());
  if (e != cudaSuccess) return cuda_fail(e, "paged attention launch");
  IG_CHECK_LAUNCH("paged attention launch");
  if (grid == 1 || (s.by_unit && most <= units * kPaWhole)) return IG_OK;  // nothing can have been cut
  const int rows_used = s.G < RU ? s.G : RU, list = s.by_unit ? (int)units : grid;
  const float bits = BF ? 0.f : 15.f;
  const float* cpart = part;
  const int2* cinfo = info;
  const long long partials = grid / units;  // of a head, about
#define IG_PJ(WPR, RB)                                                                                            \
  e = launch_pdl(k_paged_join<D, WPR, RB>, dim3(list, (rows_used + RB - 1) / RB), dim3(WPR * RB * 32), 0, st, cpart, \
                 cinfo, s, RU, bits, out, lse)
  if (partials >= 64) IG_PJ(16, 1);
  else if (partials >= 16) IG_PJ(4, 1);
  else IG_PJ(1, 4);
#undef IG_PJ
  if (e != cudaSuccess) return cuda_fail(e, "paged attention join launch");
  IG_CHECK_LAUNCH("paged attention join launch");
  return IG_OK;
}

template <bool BF, int D>
ig_status launch_rows(cudaStream_t st, const PaShape& s, const uint16_t* q, const uint16_t* K, const uint16_t* V,
                      const int32_t* table, const int32_t* L, float* out, float* lse, void* ws) {
  switch (pa_rows(s.G)) {
    case 8: return launch_paged<BF, D, 1, 1>(st, s, q, K, V, table, L, out, lse, ws);
    case 16: return launch_paged<BF, D, 2, 1>(st, s, q, K, V, table, L, out, lse, ws);
    case 32: return launch_paged<BF, D, 2, 2>(st, s, q, K, V, table, L, out, lse, ws);
    default: return launch_paged<BF, D, 2, 4>(st, s, q, K, V, table, L, out, lse, ws);
  }
}

}  // namespace
}  // namespace ig

using namespace ig;

extern "C" size_t ig_paged_attend_workspace_bytes(int B, int Hq, int Hkv, int d) {
  if (B <= 0 || Hq <= 0 || Hkv <= 0 || Hq % Hkv || (d != 64 && d != 128)) return 0;
  return pa_part_bytes(Hq / Hkv, d) + pa_info_bytes();
}

extern "C" ig_status ig_paged_attend(void* stream, int dtype, int B, int Hq, int Hkv, int d, int page, int n_pages,
                                     int max_pages, float scale, const uint16_t* q, const uint16_t* K,
                                     const uint16_t* V, const int32_t* page_table, const int32_t* L_valid, float* out,
                                     float* lse, void* workspace, size_t workspace_bytes) {
  IG_REQUIRE(dtype == IG_F16 || dtype == IG_BF16, "dtype must be IG_F16 or IG_BF16 (got %d)", dtype);
  IG_REQUIRE(B > 0 && Hq > 0 && Hkv > 0, "B, Hq, Hkv must be positive");
  IG_REQUIRE(Hq % Hkv == 0, "Hq = %d is not a multiple of Hkv = %d", Hq, Hkv);
  IG_REQUIRE(d == 64 || d == 128, "d must be 64 or 128 (got %d)", d);
  IG_REQUIRE(page > 0 && page % 8 == 0, "page must be a positive multiple of 8 (got %d)", page);
  IG_REQUIRE(n_pages > 0 && max_pages > 0, "n_pages and max_pages must be positive");
  IG_REQUIRE(Hq <= 65536 && (long long)B * Hq < (1ll << 31), "Hq at most 65536, B*Hq below 2^31");
  IG_REQUIRE((long long)max_pages * page < (1ll << 30), "max_pages*page must stay below 2^30");
  IG_REQUIRE((double)n_pages * Hkv * page < 2147483648.0, "n_pages*Hkv*page must stay below 2^31 rows");
  IG_REQUIRE(isfinite(scale) && fabsf(scale) < 1e38f, "scale must be finite (and below 1e38)");
  IG_REQUIRE(q && K && V && page_table && L_valid && out, "null pointer argument");
  IG_REQUIRE(aligned(q, 16) && aligned(K, 16) && aligned(V, 16), "q, K, V must be 16-byte aligned");
  IG_REQUIRE(aligned(out, 16), "out must be 16-byte aligned");
  IG_REQUIRE(aligned(page_table, 4) && aligned(L_valid, 4) && aligned(lse, 4),
             "page_table, L_valid, lse must be 4-byte aligned");
  const size_t need = ig_paged_attend_workspace_bytes(B, Hq, Hkv, d);
  if (!workspace || workspace_bytes < need)
    return fail(IG_ERR_CAPACITY, "paged attention needs %zu workspace bytes", need);
  IG_REQUIRE(aligned(workspace, 256), "workspace must be 256-byte aligned");
  cudaStream_t st = as_stream(stream);
  PaShape s{};
  s.B = B;
  s.Hq = Hq;
  s.Hkv = Hkv;
  s.G = Hq / Hkv;
  s.page = page;
  s.n_pages = n_pages;
  s.max_pages = max_pages;
  s.scale2 = scale * 1.4426950408889634f;
  if (dtype == IG_F16)
    return d == 128 ? launch_rows<false, 128>(st, s, q, K, V, page_table, L_valid, out, lse, workspace)
                    : launch_rows<false, 64>(st, s, q, K, V, page_table, L_valid, out, lse, workspace);
  return d == 128 ? launch_rows<true, 128>(st, s, q, K, V, page_table, L_valid, out, lse, workspace)
                  : launch_rows<true, 64>(st, s, q, K, V, page_table, L_valid, out, lse, workspace);
}
