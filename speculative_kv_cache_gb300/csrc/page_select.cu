// The pages of a paged cache that a query's attention is worth: bounds of each page's keys, kept in 8 bits, and the
// choice of the pages whose bounds allow the largest logits.
//
// Mathematics.  For the keys of a page and head, lo_c <= K_tc <= hi_c, so for a query
//   q . K_t <= sum_c max(q_c lo_c, q_c hi_c) = sum_c (min(q_c, 0) lo_c + max(q_c, 0) hi_c).
// The bounds are kept as whole numbers of -127 .. 127 in units of a power of two (lo rounded down, hi up, so that they
// stay bounds), and the query is rounded to whole numbers in a power-of-two unit of its own.  Then every product
// and sum is a whole number below 2^24 and a score is that number times two powers of two: exact in
// fp32, whatever the order of the sum.  Which pages are chosen does not depend on rounding, ties go to the lower page.
#include <cuda_bf16.h>

#include "ig_common.cuh"

namespace ig {
namespace {

// Exponent e of the unit of numbers of magnitude up to `most` (finite, >= 0): the least e >= -126 with most <= 127 * 2^e.
__device__ __forceinline__ int unit_exponent(float most) {
  const int b = __float_as_int(most), x = (b >> 23) - 126;  // most = m 2^x with m in [1/2, 1), for a normal number
  const int e = (b & 0x7fffff) > 0x7e0000 ? x - 6 : x - 7;  // m > 127/128
  return max(e, -126);  // (a number that is not normal lies far below 127 * 2^-126)
}
__device__ __forceinline__ float power_of_two(int e) { return __int_as_float((127 + e) << 23); }  // -126 <= e <= 127
// x in units of 2^e, exact but for what lies below a float's range (e <= 122)
__device__ __forceinline__ float in_units(float x, int e) { return x * power_of_two(-e); }

template <bool BF>
__device__ __forceinline__ uint32_t min2(uint32_t a, uint32_t b) {
  if constexpr (BF) {
    const __nv_bfloat162 r = __hmin2_nan(*reinterpret_cast<__nv_bfloat162*>(&a), *reinterpret_cast<__nv_bfloat162*>(&b));
    return *reinterpret_cast<const uint32_t*>(&r);
  } else {
    const __half2 r = __hmin2_nan(*reinterpret_cast<__half2*>(&a), *reinterpret_cast<__half2*>(&b));
    return *reinterpret_cast<const uint32_t*>(&r);
  }
}
template <bool BF>
__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
  if constexpr (BF) {
    const __nv_bfloat162 r = __hmax2_nan(*reinterpret_cast<__nv_bfloat162*>(&a), *reinterpret_cast<__nv_bfloat162*>(&b));
    return *reinterpret_cast<const uint32_t*>(&r);
  } else {
    const __half2 r = __hmax2_nan(*reinterpret_cast<__half2*>(&a), *reinterpret_cast<__half2*>(&b));
    return *reinterpret_cast<const uint32_t*>(&r);
  }
}
template <bool BF>
__device__ __forceinline__ float2 unpack2(uint32_t v) {
  if constexpr (BF) return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u));
  else return h2_to_f2(v);
}

// ---------------------------------------------------------------------------------------
// bounds
// ---------------------------------------------------------------------------------------
constexpr int kBoundsThreads = 256;
constexpr int kBoundsFly = 4;  // rows of a lane in flight

// A warp a page and head: D/8 lanes hold a row's 16-byte pieces, so that 2 (or 4) rows go at a time; minima and
// maxima in packed 16-bit form, exact.  Bound by HBM, the keys once: 4000 pages of 16 rows, 8 heads of 128 (139 MB) 24.2 us,
// 5.75 TB/s, 0.85 of the copy rate; 64 pages of 32 rows 3.4 us.
template <bool BF, int D>
__global__ void __launch_bounds__(kBoundsThreads) k_page_bounds(const uint4* __restrict__ K, int n_pages, int Hkv, int page, int n,
                                                               const int32_t* __restrict__ list, uint2* __restrict__ codes,
                                                               float* __restrict__ scales, int* err) {
  constexpr int LR = D / 8, RW = 32 / LR;  // lanes of a row, rows of a warp's load
  pdl_trigger();
  pdl_wait();
  const long long task = (long long)blockIdx.x * (kBoundsThreads / 32) + (threadIdx.x >> 5);
  if (task >= (long long)n * Hkv) return;
  const int i = (int)(task / Hkv), h = (int)(task % Hkv), lane = threadIdx.x & 31, col = lane % LR;
  const int g = __ldca(list + 2 * (size_t)i), rows = __ldca(list + 2 * (size_t)i + 1);
  if (g < 0) return;
  if (g >= n_pages || rows < 0 || rows > page) {
    if (lane == 0) raise_error(err, IG_DEVERR_INDEX);
    return;
  }
  const size_t head = (size_t)g * Hkv + h;
  const uint4* p = K + head * page * LR + col;
  constexpr uint32_t kTop = BF ? 0x7f807f80u : 0x7c007c00u;  // +inf, twice
  uint32_t lo[4], hi[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    lo[j] = kTop;
    hi[j] = kTop | 0x80008000u;
  }
  for (int r0 = lane / LR; r0 < rows; r0 += RW * kBoundsFly) {
    uint4 v[kBoundsFly];
#pragma unroll
    for (int x = 0; x < kBoundsFly; ++x) {  // (a row past the end is the first one again)
      const int r = r0 + x * RW;
      v[x] = p[(size_t)(r < rows ? r : r0) * LR];
    }
#pragma unroll
    for (int x = 0; x < kBoundsFly; ++x) {
      const uint32_t w[4] = {v[x].x, v[x].y, v[x].z, v[x].w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        lo[j] = min2<BF>(lo[j], w[j]);
        hi[j] = max2<BF>(hi[j], w[j]);
      }
    }
  }
#pragma unroll
  for (int o = LR; o < 32; o <<= 1)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      lo[j] = min2<BF>(lo[j], __shfl_xor_sync(0xffffffffu, lo[j], o));
      hi[j] = max2<BF>(hi[j], __shfl_xor_sync(0xffffffffu, hi[j], o));
    }
  float a[8], b[8], most = 0.f;
  bool finite = true;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 x = unpack2<BF>(lo[j]), y = unpack2<BF>(hi[j]);
    a[2 * j] = x.x, a[2 * j + 1] = x.y;
    b[2 * j] = y.x, b[2 * j + 1] = y.y;
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    if (rows == 0) a[j] = b[j] = 0.f;
    finite &= isfinite(a[j]) && isfinite(b[j]);
    most = fmaxf(most, fmaxf(fabsf(a[j]), fabsf(b[j])));
  }
#pragma unroll
  for (int o = 1; o < LR; o <<= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
  finite = __all_sync(0xffffffffu, finite);
  const int e = finite ? unit_exponent(most) : 0;
  uint32_t cl[2] = {0, 0}, ch[2] = {0, 0};
  if (finite) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float x = in_units(a[j], e), y = in_units(b[j], e);
      const int l = x == 0.f && a[j] < 0.f ? -1 : (int)floorf(x), u = y == 0.f && b[j] > 0.f ? 1 : (int)ceilf(y);
      cl[j / 4] |= ((uint32_t)l & 0xffu) << (8 * (j % 4));
      ch[j / 4] |= ((uint32_t)u & 0xffu) << (8 * (j % 4));
    }
  }
  if (lane < LR) {
    codes[head * (2 * LR) + col] = make_uint2(cl[0], cl[1]);
    codes[head * (2 * LR) + LR + col] = make_uint2(ch[0], ch[1]);
  }
  if (lane == 0) scales[head] = finite ? power_of_two(e) : INFINITY;
}

// ---------------------------------------------------------------------------------------
// choice
// ---------------------------------------------------------------------------------------
constexpr int kSelThreads = 256;
constexpr int kMaxCluster = 16, kPortableCluster = 8;
constexpr int kMaxGroup = 256;        // queries of a key head
constexpr int kSelKeyBytes = 128 << 10;  // keys of a CTA's share, at most
constexpr int kSelHalfBytes = 100 << 10; // what a CTA can have (beside 10 KB of its own) that shares an SM with another
constexpr float kMostScore = 3.402823466e38f;

struct SelArgs {
  int B, Hq, Hkv, G, page, n_pages, max_pages, picks, first, last;
  const uint16_t* q;
  const uint4* codes;
  const float* scales;
  const int32_t *table, *L;
  int32_t *chosen, *tokens;
};

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.aligned;\n barrier.cluster.wait.aligned;" ::: "memory");
}
// Sums and maxima into a word of another CTA's shared memory.  (Each CTA sends what the others need before a barrier of the cluster,
// rather than fetch theirs after it: a trip less, and none may leave late.)
__device__ __forceinline__ void peer_add(void* p, uint32_t rank, uint32_t v) {
  uint32_t at;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_addr(p)), "r"(rank));
  asm volatile("red.relaxed.cluster.shared::cluster.add.u32 [%0], %1;" ::"r"(at), "r"(v) : "memory");
}
__device__ __forceinline__ void peer_max(void* p, uint32_t rank, uint32_t v) {
  uint32_t at;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_addr(p)), "r"(rank));
  asm volatile("red.relaxed.cluster.shared::cluster.max.u32 [%0], %1;" ::"r"(at), "r"(v) : "memory");
}

// Scores in the order of whole numbers; a page that is always taken is above them all.
__device__ __forceinline__ uint32_t score_key(float s) {
  const uint32_t b = __float_as_uint(s + 0.f);
  return (int)b < 0 ? ~b : b | 0x80000000u;
}
constexpr uint32_t kAlways = 0xffffffffu;

// One cluster of CL CTAs a sequence and key head, each with a run of its pages: scores into shared memory, then the least key
// that is taken, eight bits at a time from the first one in which the keys differ (histograms in shared memory, summed
// over the cluster) until its bin is taken whole, then the pages above it, and of those equal to it the first, in
// order.  Bound by latency: a page's number, its bounds, a few rounds through the cluster (1600 cycles each); U pages a lane's
// loads ahead.  8 rows of 8192 pages with 5 queries 13.7 us (17 MB of bounds, floor 2.5: 9100 cycles of 22500 are the
// scores, 7300 the radix passes); 512 rows of up to 512 pages with 4 queries 14.6 us (floor 5); 64 pages of one sequence
// 3.6 us.  Scores by mma.sync in fp16, exact as well, took longer (20.9 and 21.8 us), as did all keys sent to one CTA of the
// cluster (20.4, beside an earlier form of this kernel that took 17).
template <bool BF, int D, int U>
__global__ void __launch_bounds__(kSelThreads) k_page_select(const SelArgs a, int CL, int* err) {
  constexpr int LP = D / 32, PW = 32 / LP;  // lanes of a page (4 pieces of 16 bytes each), pages of a warp
  constexpr int NC = D / 8;                 // 16-byte pieces of a page's bounds: lo, then hi
  constexpr int NW = kSelThreads / 32;
  extern __shared__ __align__(16) unsigned char smem_raw[];
  uint4* qs = reinterpret_cast<uint4*>(smem_raw);              // [G][NC]: min(q, 0), then max(q, 0)
  float* unit = reinterpret_cast<float*>(qs + (size_t)a.G * NC);  // [G]
  uint32_t* key = reinterpret_cast<uint32_t*>(unit + a.G);     // [share]
  __shared__ uint32_t hist[4][256], sum[4][256];  // digits of this CTA's keys, and of the cluster's
  __shared__ uint32_t count[2], ahead[2];  // keys above the threshold, and equal to it: this CTA's, and those of the CTAs before it
  __shared__ uint32_t range[2], all[2];    // the keys' complement's largest, and their largest: this CTA's, the cluster's
  __shared__ uint32_t found[3], warp_sum[2][NW];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = CL > 1 ? (int)cluster_rank() : 0;
  const int row = blockIdx.x / CL, b = row / a.Hkv, h = row % a.Hkv;
  pdl_trigger();
  for (int i = tid; i < 4 * 256; i += kSelThreads) (&hist[0][0])[i] = (&sum[0][0])[i] = 0;
  if (tid < 2) count[tid] = ahead[tid] = range[tid] = all[tid] = 0;
  pdl_wait();
  int L = __ldca(a.L + b);
  if (L < 0 || L > a.max_pages * a.page) {
    if (tid == 0 && rank == 0) raise_error(err, IG_DEVERR_INDEX);
    L = L < 0 ? 0 : a.max_pages * a.page;
  }
  const int P = (L + a.page - 1) / a.page, take = min(P, a.picks);
  const int32_t* table = a.table + (size_t)b * a.max_pages;
  int32_t* chosen = a.chosen + (size_t)row * a.picks;
  for (int i = take + rank * kSelThreads + tid; i < a.picks; i += CL * kSelThreads) chosen[i] = -1;
  if (rank == 0 && tid == 0) a.tokens[row] = P ? (take - 1) * a.page + L - (P - 1) * a.page : 0;
  if (P <= a.picks) {  // all of them (the same for the whole cluster)
    for (int i = rank * kSelThreads + tid; i < P; i += CL * kSelThreads) {
      const int id = __ldca(table + i);
      chosen[i] = id;
      if (id < 0 || id >= a.n_pages) raise_error(err, IG_DEVERR_INDEX);
    }
    return;
  }
  if (CL > 1) asm volatile("barrier.cluster.arrive.aligned;" ::: "memory");  // this CTA is there, its sums begin at zero
  // this CTA's pages; the first ones' numbers are on their way while the queries are prepared
  const int each = (P + CL - 1) / CL, p0 = min(P, rank * each), p1 = min(P, p0 + each), mine = p1 - p0;
  const int sub = lane % LP;
  int id[U];
  auto numbers = [&](int at) {
#pragma unroll
    for (int x = 0; x < U; ++x) id[x] = at + x * NW * PW < p1 ? __ldca(table + min(at + x * NW * PW + lane / LP, p1 - 1)) : 0;
  };
  numbers(p0 + warp * PW);
  // ---- the queries as whole numbers, a warp each
  for (int g = warp; g < a.G; g += NW) {
    const uint16_t* q = a.q + ((size_t)b * a.Hq + (size_t)h * a.G + g) * D;
    float x[D / 32], most = 0.f;
    bool finite = true;
    if constexpr (D == 128) {
      const uint2 v = __ldca(reinterpret_cast<const uint2*>(q) + lane);
      const float2 y = unpack2<BF>(v.x), z = unpack2<BF>(v.y);
      x[0] = y.x, x[1] = y.y, x[2] = z.x, x[3] = z.y;
    } else {
      const float2 y = unpack2<BF>(__ldca(reinterpret_cast<const uint32_t*>(q) + lane));
      x[0] = y.x, x[1] = y.y;
    }
#pragma unroll
    for (int j = 0; j < D / 32; ++j) {
      finite &= isfinite(x[j]);
      most = fmaxf(most, fabsf(x[j]));
    }
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
    finite = __all_sync(0xffffffffu, finite);
    const int e = finite ? unit_exponent(most) : 0;
    int8_t* neg = reinterpret_cast<int8_t*>(qs + (size_t)g * NC) + lane * (D / 32);
#pragma unroll
    for (int j = 0; j < D / 32; ++j) {
      const int c = finite ? __float2int_rn(in_units(x[j], e)) : 0;
      neg[j] = (int8_t)min(c, 0);
      neg[D + j] = (int8_t)max(c, 0);
    }
    if (lane == 0) unit[g] = power_of_two(e);
  }
  __syncthreads();
  // ---- scores of this CTA's pages, U pages of a lane at a time
  uint32_t low = 0, high = 0;  // of the keys that are compared: their complement's largest, their largest
  for (int at = p0 + warp * PW; at < p1; at += U * NW * PW) {
    uint4 v[U][4];
    float scale[U];
    bool bad[U];
#pragma unroll
    for (int x = 0; x < U; ++x) {
      bad[x] = id[x] < 0 || id[x] >= a.n_pages;
      if (at + x * NW * PW >= p1) continue;  // (the same for the warp)
      const size_t head = (size_t)(bad[x] ? 0 : id[x]) * a.Hkv + h;
#pragma unroll
      for (int k = 0; k < 4; ++k) v[x][k] = __ldca(a.codes + head * NC + sub + k * LP);
      scale[x] = __ldca(a.scales + head);
    }
    numbers(at + U * NW * PW);
    float best[U];
#pragma unroll
    for (int x = 0; x < U; ++x) best[x] = -INFINITY;
    for (int g = 0; g < a.G; ++g) {
      int dot[U];
#pragma unroll
      for (int x = 0; x < U; ++x) dot[x] = 0;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const uint4 w = qs[(size_t)g * NC + sub + k * LP];
#pragma unroll
        for (int x = 0; x < U; ++x) {
          dot[x] = __dp4a((int)v[x][k].x, (int)w.x, dot[x]);
          dot[x] = __dp4a((int)v[x][k].y, (int)w.y, dot[x]);
          dot[x] = __dp4a((int)v[x][k].z, (int)w.z, dot[x]);
          dot[x] = __dp4a((int)v[x][k].w, (int)w.w, dot[x]);
        }
      }
      const float u = unit[g];
#pragma unroll
      for (int x = 0; x < U; ++x) {
#pragma unroll
        for (int o = 1; o < LP; o <<= 1) dot[x] += __shfl_xor_sync(0xffffffffu, dot[x], o);
        best[x] = fmaxf(best[x], (float)dot[x] * u);
      }
    }
#pragma unroll
    for (int x = 0; x < U; ++x) {
      const int p = at + x * NW * PW + lane / LP;
      if (p >= p1 || sub) continue;
      const float s = scale[x] == INFINITY ? kMostScore : fminf(best[x] * scale[x], kMostScore);
      uint32_t k = kAlways;
      if (p >= a.first && p < P - a.last) {
        k = bad[x] ? 0u : score_key(s);
        low = max(low, ~k);
        high = max(high, k);
      }
      key[p - p0] = k;
      if (bad[x]) raise_error(err, IG_DEVERR_INDEX);
    }
  }
  low = __reduce_max_sync(0xffffffffu, low);
  high = __reduce_max_sync(0xffffffffu, high);
  if (lane == 0) {
    atomicMax(&range[0], low);
    atomicMax(&range[1], high);
  }
  __syncthreads();
  if (CL > 1) {
    asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
    if (tid < 2 * CL) peer_max(&all[tid & 1], (uint32_t)tid >> 1, range[tid & 1]);
    cluster_sync();
    low = all[0];
    high = all[1];
  } else {
    low = range[0];
    high = range[1];
  }
  // ---- of the pages that are not always taken, the `want`-th largest key; keys agree from bit `top` on
  uint32_t want = (uint32_t)(a.picks - a.first - a.last);
  int top = 32 - __clz(high ^ ~low), shift = top;
  uint32_t prefix = top < 32 ? high >> top : 0u;  // keys >> shift that decide: above it taken, equal to it the first `want`
  auto begins = [&](uint32_t k, int s) -> uint32_t { return s < 32 ? k >> s : 0u; };
  for (int pass = 0; want > 0 && shift > 0; ++pass) {
    const int next = max(shift - 8, 0);
    const uint32_t mask = (1u << (shift - next)) - 1;
    for (int i = tid; i < mine; i += kSelThreads) {
      const uint32_t k = key[i];
      if (k != kAlways && begins(k, shift) == prefix) atomicAdd(&hist[pass][(k >> next) & mask], 1u);
    }
    __syncthreads();
    uint32_t n = hist[pass][255 - tid];  // thread t: the keys with digit 255 - t
    if (CL > 1) {
      for (int r = 0; n && r < CL; ++r) peer_add(&sum[pass][255 - tid], (uint32_t)r, n);
      cluster_sync();
      n = sum[pass][255 - tid];
    }
    uint32_t in = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t y = __shfl_up_sync(0xffffffffu, in, o);
      if (lane >= o) in += y;
    }
    if (lane == 31) warp_sum[pass & 1][warp] = in;
    __syncthreads();
    for (int w = 0; w < warp; ++w) in += warp_sum[pass & 1][w];
    if (in - n < want && want <= in) {
      found[0] = (uint32_t)(255 - tid);
      found[1] = want - (in - n);
      found[2] = n;
    }
    __syncthreads();
    prefix = prefix << (shift - next) | found[0];
    want = found[1];
    shift = next;
    if (want == found[2]) break;  // all that begin so are taken
  }
  // (the next write to `found` or `warp_sum` comes after a barrier that follows every read of them)
  __syncthreads();
  // ---- keys above the threshold are taken, and the first `want` of those equal to it
  auto place = [&](int i, bool& gt, bool& eq) {
    const uint32_t k = i < mine ? key[i] : 0u, y = begins(k, shift);
    gt = i < mine && (k == kAlways || y > prefix);
    eq = i < mine && k != kAlways && y == prefix;
  };
  uint32_t pos = 0, ties = 0;  // taken, and equal ones seen, before this share (nothing is sent after the last barrier)
  if (CL > 1) {
    uint32_t above = 0, equal = 0;
    for (int i = tid; i < mine; i += kSelThreads) {
      bool gt, eq;
      place(i, gt, eq);
      above += gt;
      equal += eq;
    }
    above = __reduce_add_sync(0xffffffffu, above);
    equal = __reduce_add_sync(0xffffffffu, equal);
    if (lane == 0) {
      atomicAdd(&count[0], above);
      atomicAdd(&count[1], equal);
    }
    __syncthreads();
    if (tid < 2 * CL && tid >> 1 > rank) peer_add(&ahead[tid & 1], (uint32_t)tid >> 1, count[tid & 1]);
    cluster_sync();
    ties = ahead[1];
    pos = ahead[0] + min(ties, want);
  }
  int turn = 0;
  for (int i0 = 0; i0 < mine; i0 += kSelThreads, turn ^= 1) {
    const int i = i0 + tid;
    bool gt, eq;
    place(i, gt, eq);
    const unsigned bg = __ballot_sync(0xffffffffu, gt), be = __ballot_sync(0xffffffffu, eq), lt = (1u << lane) - 1;
    if (lane == 0) warp_sum[turn][warp] = __popc(bg) | __popc(be) << 16;
    __syncthreads();
    uint32_t before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < NW; ++w) {
      before += w < warp ? warp_sum[turn][w] : 0;
      all += warp_sum[turn][w];
    }
    const uint32_t g_at = (before & 0xffff) + __popc(bg & lt), e_at = (before >> 16) + __popc(be & lt);
    // equal ones taken before this page: of those in this turn, as many as the first `want` reach
    const uint32_t e_taken = min(ties + e_at, want) - min(ties, want);
    if (gt || (eq && ties + e_at < want)) chosen[pos + g_at + e_taken] = __ldca(table + p0 + i);
    pos += (all & 0xffff) + min(ties + (all >> 16), want) - min(ties, want);
    ties += all >> 16;
  }
}

// U: with many rows two pages a lane, so that three CTAs share an SM (64 sequences of up to 512 pages, 8 key heads: 14.7 us, with
// four 18.2); with few four, so that more is on its way (8 rows of 8192: 13.7 us, with two 17.4).
template <bool BF, int D, int U>
ig_status launch_select_u(cudaStream_t st, const SelArgs& a, int CL, size_t smem) {
  cudaError_t e = cudaFuncSetAttribute(k_page_select<BF, D, U>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e == cudaSuccess && CL > kPortableCluster)
    e = cudaFuncSetAttribute(k_page_select<BF, D, U>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e != cudaSuccess) return cuda_fail(e, "page select attributes");
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((long long)a.B * a.Hkv * CL));
  cfg.blockDim = dim3(kSelThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = (unsigned)CL;
  at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = CL > 1 ? 2 : 1;
  e = cudaLaunchKernelEx(&cfg, k_page_select<BF, D, U>, a, CL, error_word());
  if (e != cudaSuccess) return cuda_fail(e, "page select launch");
  IG_CHECK_LAUNCH("page select launch");
  return IG_OK;
}

template <bool BF, int D>
ig_status launch_select(cudaStream_t st, SelArgs a) {
  // CTAs of a cluster: more where there are few rows, as long as each has 256 pages or more (not on a partition of the SMs,
  // which need not have room for clusters side by side; more than the portable number only where two CTAs share an SM, so that
  // half as many SMs are enough); and as many as the keys need
  const long long rows = (long long)a.B * a.Hkv;
  auto share = [&](int CL) -> size_t { return (size_t)((a.max_pages + CL - 1) / CL); };
  auto bytes = [&](int CL) -> size_t { return (size_t)a.G * (2 * D + 4) + share(CL) * 4; };
  int CL = 1;
  while (CL < kMaxCluster && stream_sms(st) == 0 && rows * CL < sm_count(st) && a.max_pages / (2 * CL) >= 256 &&
         (CL < kPortableCluster || bytes(2 * CL) <= (size_t)kSelHalfBytes))
    CL *= 2;
  while (CL < kPortableCluster && share(CL) * 4 > (size_t)kSelKeyBytes) CL *= 2;
  const size_t smem = bytes(CL);
  return rows * CL > sm_count(st) ? launch_select_u<BF, D, 2>(st, a, CL, smem) : launch_select_u<BF, D, 4>(st, a, CL, smem);
}

}  // namespace
}  // namespace ig

using namespace ig;

extern "C" ig_status ig_page_bounds(void* stream, int dtype, int n_pages, int Hkv, int page, int d, const uint16_t* K, int n,
                                    const int32_t* list, int8_t* codes, float* scales) {
  IG_REQUIRE(dtype == IG_F16 || dtype == IG_BF16, "dtype must be IG_F16 or IG_BF16 (got %d)", dtype);
  IG_REQUIRE(n_pages > 0 && Hkv > 0 && n >= 0, "n_pages, Hkv must be positive, n not negative");
  IG_REQUIRE(page > 0 && page % 8 == 0, "page must be a positive multiple of 8 (got %d)", page);
  IG_REQUIRE(d == 64 || d == 128, "d must be 64 or 128 (got %d)", d);
  IG_REQUIRE((double)n_pages * Hkv * page < 2147483648.0, "n_pages*Hkv*page must stay below 2^31 rows");
  IG_REQUIRE((double)n * Hkv < 2147483648.0, "n*Hkv must stay below 2^31");
  IG_REQUIRE(K && codes && scales, "null pointer argument");
  IG_REQUIRE(aligned(K, 16) && aligned(codes, 16) && aligned(scales, 4), "K, codes must be 16-byte aligned, scales 4-byte");
  if (n == 0) return IG_OK;
  IG_REQUIRE(list && aligned(list, 4), "null or misaligned list");
  const long long warps = (long long)n * Hkv, per = kBoundsThreads / 32;
  const dim3 grid((unsigned)((warps + per - 1) / per));
  auto kern = dtype == IG_BF16 ? (d == 128 ? k_page_bounds<true, 128> : k_page_bounds<true, 64>)
                               : (d == 128 ? k_page_bounds<false, 128> : k_page_bounds<false, 64>);
  const cudaError_t e = launch_pdl(kern, grid, dim3(kBoundsThreads), 0, as_stream(stream), reinterpret_cast<const uint4*>(K), n_pages,
                                   Hkv, page, n, list, reinterpret_cast<uint2*>(codes), scales, error_word());
  if (e != cudaSuccess) return cuda_fail(e, "page bounds launch");
  IG_CHECK_LAUNCH("page bounds launch");
  return IG_OK;
}

extern "C" ig_status ig_page_select(void* stream, int dtype, int B, int Hq, int Hkv, int d, int page, int n_pages, int max_pages,
                                    int picks, int first, int last, const uint16_t* q, const int8_t* codes,
                                    const float* scales, const int32_t* page_table, const int32_t* L_valid, int32_t* chosen,
                                    int32_t* tokens) {
  IG_REQUIRE(dtype == IG_F16 || dtype == IG_BF16, "dtype must be IG_F16 or IG_BF16 (got %d)", dtype);
  IG_REQUIRE(B > 0 && Hq > 0 && Hkv > 0, "B, Hq, Hkv must be positive");
  IG_REQUIRE(Hq % Hkv == 0, "Hq = %d is not a multiple of Hkv = %d", Hq, Hkv);
  IG_REQUIRE(Hq / Hkv <= kMaxGroup, "at most %d queries to a key head", kMaxGroup);
  IG_REQUIRE(d == 64 || d == 128, "d must be 64 or 128 (got %d)", d);
  IG_REQUIRE(page > 0 && page % 8 == 0, "page must be a positive multiple of 8 (got %d)", page);
  IG_REQUIRE(n_pages > 0 && max_pages > 0, "n_pages and max_pages must be positive");
  IG_REQUIRE((long long)max_pages * page < (1ll << 30), "max_pages*page must stay below 2^30");
  IG_REQUIRE(max_pages <= kPortableCluster * kSelKeyBytes / 4, "max_pages at most %d", kPortableCluster * kSelKeyBytes / 4);
  IG_REQUIRE((double)n_pages * Hkv * page < 2147483648.0, "n_pages*Hkv*page must stay below 2^31 rows");
  IG_REQUIRE((double)B * Hq < 134217728.0, "B*Hq must stay below 2^27");
  IG_REQUIRE(first >= 0 && last >= 1 && (long long)first + last <= picks,
             "the page written last is always picked, and first + last pages are at most picks (got %d + %d, %d)", first, last, picks);
  IG_REQUIRE((long long)picks * page < (1ll << 30), "picks*page must stay below 2^30");
  IG_REQUIRE(q && codes && scales && page_table && L_valid && chosen && tokens, "null pointer argument");
  IG_REQUIRE(aligned(q, 16) && aligned(codes, 16), "q, codes must be 16-byte aligned");
  IG_REQUIRE(aligned(scales, 4) && aligned(page_table, 4) && aligned(L_valid, 4) && aligned(chosen, 4) && aligned(tokens, 4),
             "misaligned buffer");
  const SelArgs a{B, Hq, Hkv, Hq / Hkv, page, n_pages, max_pages, picks, first, last, q, reinterpret_cast<const uint4*>(codes),
                  scales, page_table, L_valid, chosen, tokens};
  cudaStream_t st = as_stream(stream);
  if (dtype == IG_F16) return d == 128 ? launch_select<false, 128>(st, a) : launch_select<false, 64>(st, a);
  return d == 128 ? launch_select<true, 128>(st, a) : launch_select<true, 64>(st, a);
}
