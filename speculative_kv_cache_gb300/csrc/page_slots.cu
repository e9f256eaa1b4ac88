// Where the new tokens of a batch of requests go in a paged cache, and which of a tree's drafted tokens stay.
#include "ig_common.cuh"

namespace ig {
namespace {

constexpr int kMaxRequests = 8192;  // prefix sums in shared memory
constexpr int kMaxTree = 64;        // drafted tokens of a request: bits of a mask
constexpr int kSlotThreads = 256;

struct SlotArgs {
  int n, seqs, page, n_pages, max_pages, T;
  const int32_t *table, *L, *seq, *counts, *parents;
  int32_t *first, *slots, *positions;
  unsigned long long* masks;
};

// A request's sequence and the place of its first new token; false where it cannot be.
__device__ __forceinline__ bool slot_request(const SlotArgs& a, int r, int count, int& s, int& base) {
  s = a.seq ? __ldca(a.seq + r) : r;
  if (s < 0 || s >= a.seqs) return false;
  const int L = __ldca(a.L + s);
  base = L - count;
  return L >= 0 && L <= a.max_pages * a.page && base >= 0;
}

__device__ __forceinline__ int slot_of(const SlotArgs& a, int s, int at, int* err) {
  const int pg = at / a.page, g = __ldca(a.table + (size_t)s * a.max_pages + pg);
  if (g < 0 || g >= a.n_pages) {
    raise_error(err, IG_DEVERR_INDEX);
    return -1;
  }
  return g * a.page + (at - pg * a.page);
}

// Every CTA sums up all counts by itself (a few loads a thread, against another launch).  Without trees the tokens
// are spread over the threads, which find their request by bisection of the sums; with trees (at most 64 tokens a
// request) a warp has a request, a lane the tokens lane and lane + 32: their ancestors' bits double with
// every look at the parent's parent, six at most, all in registers.  Bound by latency: the counts, the sequence's
// length, its page's number, one after the other: 64 trees of up to 16 tokens 3.3 us, 48 prompts of 100 000 tokens in all
// 3.9 us (a thread has a token, as long as four CTAs an SM have room; with four, one after the other, 6.1).
template <bool TREE>
__global__ void __launch_bounds__(kSlotThreads) k_page_slots(const SlotArgs a, int* err) {
  __shared__ int first[kMaxRequests + 1];
  __shared__ long long warp_sum[kSlotThreads / 32];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  pdl_trigger();
  pdl_wait();
  bool bad = false;
  for (int i = tid; i < a.n; i += kSlotThreads) {
    int c = __ldca(a.counts + i);
    bad |= c < 0;
    first[i + 1] = c < 0 ? 0 : c;
  }
  __syncthreads();
  const int per = (a.n + kSlotThreads - 1) / kSlotThreads, i0 = min(a.n, tid * per), i1 = min(a.n, i0 + per);
  long long mine = 0;
  for (int i = i0; i < i1; ++i) mine += first[i + 1];
  long long in = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, in, o);
    if (lane >= o) in += y;
  }
  if (lane == 31) warp_sum[warp] = in;
  __syncthreads();
  long long at = in - mine;
  for (int w = 0; w < warp; ++w) at += warp_sum[w];
  for (int i = i0; i < i1; ++i) {
    at += first[i + 1];
    first[i + 1] = (int)(at < a.T ? at : a.T);
  }
  bad |= at > a.T;
  if (tid == 0) first[0] = 0;
  if (bad && blockIdx.x == 0) raise_error(err, IG_DEVERR_INDEX);
  __syncthreads();
  const int threads = gridDim.x * kSlotThreads, me = blockIdx.x * kSlotThreads + tid;
  for (int i = me; i <= a.n; i += threads) a.first[i] = first[i];
  // a request that the buffers cut off is left out as a whole
  auto whole = [&](int r, int c) -> bool { return c == first[r + 1] - first[r]; };
  const int total = first[a.n];
  if constexpr (!TREE) {
    for (int t = me; t < a.T; t += threads) {
      int slot = -1, pos = 0;
      if (t < total) {
        int lo = 0, hi = a.n;  // first[lo] <= t < first[hi]
        while (hi - lo > 1) {
          const int mid = (lo + hi) >> 1;
          if (first[mid] <= t) lo = mid;
          else hi = mid;
        }
        const int c = __ldca(a.counts + lo);
        int s, base;
        if (whole(lo, c) && slot_request(a, lo, c, s, base)) {
          pos = base + t - first[lo];
          slot = slot_of(a, s, pos, err);
        } else {
          raise_error(err, IG_DEVERR_INDEX);
        }
      }
      a.slots[t] = slot;
      a.positions[t] = pos;
    }
  } else {
    for (int r = blockIdx.x * (kSlotThreads / 32) + warp; r < a.n; r += gridDim.x * (kSlotThreads / 32)) {
      const int f = first[r], held = first[r + 1] - f, c = __ldca(a.counts + r);
      if (held == 0) continue;
      int s = 0, base = 0;
      if (c > kMaxTree || !whole(r, c) || !slot_request(a, r, c, s, base)) {
        if (lane == 0) raise_error(err, IG_DEVERR_INDEX);
        for (int i = lane; i < held; i += 32) {
          a.slots[f + i] = -1;
          a.positions[f + i] = 0;
          if (a.masks) a.masks[f + i] = 0;
        }
        continue;
      }
      unsigned long long m[2];
      int up[2];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int i = lane + 32 * k;
        up[k] = i >= c ? -1 : a.parents ? __ldca(a.parents + f + i) : i - 1;
        if (up[k] < -1 || up[k] >= i) {
          up[k] = -1;
          if (i < c) raise_error(err, IG_DEVERR_INDEX);
        }
        m[k] = 1ull << i;
      }
      while (__any_sync(0xffffffffu, up[0] >= 0 || up[1] >= 0)) {
        unsigned long long m2[2];
        int up2[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const int p = up[k];
          const unsigned long long x = __shfl_sync(0xffffffffu, m[0], p & 31), y = __shfl_sync(0xffffffffu, m[1], p & 31);
          const int u = __shfl_sync(0xffffffffu, up[0], p & 31), v = __shfl_sync(0xffffffffu, up[1], p & 31);
          m2[k] = p < 0 ? m[k] : m[k] | (p < 32 ? x : y);
          up2[k] = p < 0 ? -1 : p < 32 ? u : v;
        }
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          m[k] = m2[k];
          up[k] = up2[k];
        }
      }
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int i = lane + 32 * k;
        if (i >= c) continue;
        a.slots[f + i] = slot_of(a, s, base + i, err);
        a.positions[f + i] = base + __popcll(m[k]) - 1;
        if (a.masks) a.masks[f + i] = m[k];
      }
    }
    for (int t = total + me; t < a.T; t += threads) {
      a.slots[t] = -1;
      a.positions[t] = 0;
      if (a.masks) a.masks[t] = 0;
    }
  }
}

constexpr int kMaxKeepLayers = 128;
struct KeepLayers {
  uint4* p[2 * kMaxKeepLayers];  // K of every layer, then V
};
struct KeepArgs {
  int n_pages, Hkv, page, vpr, seqs, max_pages, T;
  const int32_t *table, *L, *seq, *first, *path, *kept;
};

// One CTA per (request, K or V of a layer).  The kept rows ascend, so row i comes from row path[i] >= i and no row
// that is still to be read has been written: a thread moves the same 16 bytes of every row, and needs no other's.  HBM-bound where
// there is much to move (64 requests, 8 of 32 tokens, 32 layers of 8 heads of 128: 130 MB read and written in 23.7 us, 5.5 TB/s,
// 0.81 of the copy rate: rows of 256 bytes), else a launch and three round trips (2.5 us).
constexpr int kKeepThreads = 128;
constexpr int kKeepFly = 8;
__global__ void __launch_bounds__(kKeepThreads) k_tree_keep(const KeepLayers P, const KeepArgs a, int* err) {
  __shared__ int src[kMaxTree], dst[kMaxTree];  // rows of the first head
  __shared__ int path[kMaxTree];
  const int r = blockIdx.x, tid = threadIdx.x;
  pdl_trigger();
  pdl_wait();
  const int s = a.seq ? __ldca(a.seq + r) : r, f = __ldca(a.first + r), n = __ldca(a.first + r + 1) - f, kept = __ldca(a.kept + r);
  const int L = s >= 0 && s < a.seqs ? __ldca(a.L + s) : -1;
  bool ok = f >= 0 && n >= 0 && n <= kMaxTree && f <= a.T - n && kept >= 0 && kept <= n && L >= n && L <= a.max_pages * a.page;
  if (ok && tid < kept) {
    const int p = __ldca(a.path + f + tid);
    ok = p >= 0 && p < n && (tid == 0 || __ldca(a.path + f + tid - 1) < p);
    path[tid] = p;
    if (ok) {
      const int from = L - n + p, to = L - n + tid;
      const int32_t* row = a.table + (size_t)s * a.max_pages;
      const int x = __ldca(row + from / a.page), y = __ldca(row + to / a.page);
      ok = x >= 0 && x < a.n_pages && y >= 0 && y < a.n_pages;
      src[tid] = x * a.Hkv * a.page + from % a.page;
      dst[tid] = y * a.Hkv * a.page + to % a.page;
    }
  }
  if (!__syncthreads_and(ok)) {
    if (tid == 0) raise_error(err, IG_DEVERR_INDEX);
    return;
  }
  int i0 = 0;  // rows that are where they belong
  while (i0 < kept && path[i0] == i0) ++i0;
  if (i0 >= kept) return;
  uint4* base = P.p[blockIdx.y];
  for (int c = tid; c < a.Hkv * a.vpr; c += kKeepThreads) {
    uint4* col = base + (size_t)(c / a.vpr) * a.page * a.vpr + c % a.vpr;
    for (int i = i0; i < kept; i += kKeepFly) {
      uint4 v[kKeepFly];
#pragma unroll
      for (int x = 0; x < kKeepFly; ++x)
        if (i + x < kept) v[x] = col[(size_t)src[i + x] * a.vpr];
#pragma unroll
      for (int x = 0; x < kKeepFly; ++x)
        if (i + x < kept) col[(size_t)dst[i + x] * a.vpr] = v[x];
    }
  }
}

}  // namespace
}  // namespace ig

using namespace ig;

extern "C" ig_status ig_page_slots(void* stream, int n, int seqs, int page, int n_pages, int max_pages, int T,
                                   const int32_t* page_table, const int32_t* L_valid, const int32_t* seq,
                                   const int32_t* counts, const int32_t* parents, int32_t* first, int32_t* slots,
                                   int32_t* positions, uint64_t* masks) {
  IG_REQUIRE(n > 0 && n <= kMaxRequests, "n must be in [1, %d] (got %d)", kMaxRequests, n);
  IG_REQUIRE(seqs > 0 && T >= 0 && T < (1 << 30), "seqs must be positive, T in [0, 2^30)");
  IG_REQUIRE(seq || n <= seqs, "%d requests for %d sequences: name them", n, seqs);
  IG_REQUIRE(page > 0 && page % 8 == 0, "page must be a positive multiple of 8 (got %d)", page);
  IG_REQUIRE(n_pages > 0 && max_pages > 0, "n_pages and max_pages must be positive");
  IG_REQUIRE((long long)max_pages * page < (1ll << 30), "max_pages*page must stay below 2^30");
  IG_REQUIRE((long long)n_pages * page < (1ll << 31), "n_pages*page must stay below 2^31");
  IG_REQUIRE(page_table && L_valid && counts && first, "null pointer argument");
  IG_REQUIRE(T == 0 || (slots && positions), "null pointer argument");
  IG_REQUIRE(aligned(page_table, 4) && aligned(L_valid, 4) && aligned(seq, 4) && aligned(counts, 4) && aligned(parents, 4) &&
                 aligned(first, 4) && aligned(slots, 4) && aligned(positions, 4) && aligned(masks, 8),
             "misaligned buffer");
  const bool tree = parents || masks;
  const SlotArgs a{n, seqs, page, n_pages, max_pages, T, page_table, L_valid, seq, counts, parents, first, slots, positions,
                   reinterpret_cast<unsigned long long*>(masks)};
  const long long work = tree ? (long long)n * 32 : T;
  long long grid = (work + kSlotThreads - 1) / kSlotThreads;
  const long long most = 4ll * sm_count(as_stream(stream));
  grid = grid < 1 ? 1 : grid > most ? most : grid;
  const cudaError_t e = launch_pdl(tree ? k_page_slots<true> : k_page_slots<false>, dim3((unsigned)grid), dim3(kSlotThreads), 0,
                                   as_stream(stream), a, error_word());
  if (e != cudaSuccess) return cuda_fail(e, "page slots launch");
  IG_CHECK_LAUNCH("page slots launch");
  return IG_OK;
}

extern "C" ig_status ig_tree_keep(void* stream, int layers, int n_pages, int Hkv, int page, int d, uint16_t* const* K,
                                  uint16_t* const* V, int n, int seqs, int max_pages, int T, const int32_t* page_table,
                                  const int32_t* L_valid, const int32_t* seq, const int32_t* first, const int32_t* path,
                                  const int32_t* kept) {
  IG_REQUIRE(layers > 0 && layers <= kMaxKeepLayers, "layers must be in [1, %d]", kMaxKeepLayers);
  IG_REQUIRE(n_pages > 0 && Hkv > 0 && n >= 0, "n_pages, Hkv must be positive, n not negative");
  IG_REQUIRE(page > 0 && page % 8 == 0, "page must be a positive multiple of 8 (got %d)", page);
  IG_REQUIRE(d > 0 && d % 8 == 0, "d must be a positive multiple of 8 (got %d)", d);
  IG_REQUIRE(seqs > 0 && max_pages > 0 && T >= 0, "seqs, max_pages must be positive, T not negative");
  IG_REQUIRE(seq || n <= seqs, "%d requests for %d sequences: name them", n, seqs);
  IG_REQUIRE((long long)max_pages * page < (1ll << 30), "max_pages*page must stay below 2^30");
  IG_REQUIRE((double)n_pages * Hkv * page < 2147483648.0, "n_pages*Hkv*page must stay below 2^31 rows");
  IG_REQUIRE((double)Hkv * (d / 8) < 1073741824.0, "Hkv*d is too large");
  IG_REQUIRE(K && V, "null pointer argument");
  KeepLayers P{};
  for (int l = 0; l < layers; ++l) {
    IG_REQUIRE(K[l] && V[l], "null pages of layer %d", l);
    IG_REQUIRE(aligned(K[l], 16) && aligned(V[l], 16), "the pages must be 16-byte aligned");
    P.p[l] = reinterpret_cast<uint4*>(K[l]);
    P.p[layers + l] = reinterpret_cast<uint4*>(V[l]);
  }
  if (n == 0) return IG_OK;
  IG_REQUIRE(page_table && L_valid && first && path && kept, "null pointer argument");
  IG_REQUIRE(aligned(page_table, 4) && aligned(L_valid, 4) && aligned(seq, 4) && aligned(first, 4) && aligned(path, 4) &&
                 aligned(kept, 4),
             "misaligned buffer");
  const KeepArgs a{n_pages, Hkv, page, d / 8, seqs, max_pages, T, page_table, L_valid, seq, first, path, kept};
  const cudaError_t e = launch_pdl(k_tree_keep, dim3((unsigned)n, (unsigned)(2 * layers)), dim3(kKeepThreads), 0,
                                   as_stream(stream), P, a, error_word());
  if (e != cudaSuccess) return cuda_fail(e, "tree keep launch");
  IG_CHECK_LAUNCH("tree keep launch");
  return IG_OK;
}
