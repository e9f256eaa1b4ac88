// Attention of a tree of drafted tokens per request over a paged KV cache.
//
// Mathematics.  Request b has L tokens, the last n of them drafted.  Drafted token t sees key j when j < L - n, or when bit
// j - (L - n) of its mask is set (its ancestors and itself); for each query head
//   z_j = scale q . K_j,  o = sum_j e^(z_j) V_j / sum_j e^(z_j)  over the keys it sees.
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

__device__ __forceinline__ bool tree_request(const TreeShape& a, int r, TreeRequest& x) {
  x.f = __ldca(a.first + r);
  x.n = __ldca(a.first + r + 1) - x.f;
  x.s = a.seq ? __ldca(a.seq + r) : r;
  x.L = x.s >= 0 && x.s < a.seqs ? __ldca(a.L + x.s) : -1;
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

// A block a token and key head, a warp a query; a lane a key for the logits, a lane D/32 columns for the sums.
template <bool BF, int D>
__global__ void __launch_bounds__(128) k_tree_simple(const uint16_t* __restrict__ q, const uint16_t* __restrict__ K,
                                                     const uint16_t* __restrict__ V, const TreeShape a, uint16_t* __restrict__ out,
                                                     float* __restrict__ lse, int* err) {
  __shared__ float sq[4][D];
  const int t = blockIdx.x, h = blockIdx.y, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int r = 0;
  while (r < a.B && __ldca(a.first + r + 1) <= t) ++r;
  if (r >= a.B || __ldca(a.first + r) > t) return;
  TreeRequest x;
  if (!tree_request(a, r, x)) {
    if (threadIdx.x == 0) raise_error(err, IG_DEVERR_INDEX);
    return;
  }
  const unsigned long long mask = __ldca(a.masks + t);
  for (int g = warp; g < a.G; g += 4) {
    const size_t at = (size_t)t * a.Hq + (size_t)h * a.G + g;
    for (int i = lane; i < D; i += 32) sq[warp][i] = to_float<BF>(q[at * D + i]);
    __syncwarp();
    float m = -INFINITY, l = 0.f, o[D / 32];
    for (int i = 0; i < D / 32; ++i) o[i] = 0.f;
    for (int j0 = 0; j0 < x.L; j0 += 32) {
      const int j = j0 + lane, bit = j - (x.L - x.n);
      bool seen = j < x.L && (bit < 0 || (mask >> bit & 1));
      int row = 0;
      if (seen) {
        const int pg = __ldca(a.table + (size_t)x.s * a.max_pages + j / a.page);
        if (pg < 0 || pg >= a.n_pages) {
          raise_error(err, IG_DEVERR_INDEX);
          seen = false;
        } else {
          row = (pg * a.Hkv + h) * a.page + j % a.page;
        }
      }
      float z = -INFINITY;
      if (seen) {
        float acc = 0.f;
        for (int i = 0; i < D; ++i) acc = fmaf(sq[warp][i], to_float<BF>(K[(size_t)row * D + i]), acc);
        z = acc * a.scale2;
      }
      float mx = z;
      for (int s = 16; s; s >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, s));
      const float mn = fmaxf(m, mx), m0 = mn == -INFINITY ? 0.f : mn;
      const float c = ex2(m - m0), p = seen ? ex2(z - m0) : 0.f;
      l = l * c + p;
      for (int i = 0; i < D / 32; ++i) o[i] *= c;
      for (unsigned left = __ballot_sync(0xffffffffu, seen); left; left &= left - 1) {
        const int k = __ffs(left) - 1;
        const float pk = __shfl_sync(0xffffffffu, p, k);
        const int rk = __shfl_sync(0xffffffffu, row, k);
        for (int i = 0; i < D / 32; ++i) o[i] = fmaf(pk, to_float<BF>(V[(size_t)rk * D + i * 32 + lane]), o[i]);
      }
      m = mn;
    }
    for (int s = 16; s; s >>= 1) l += __shfl_xor_sync(0xffffffffu, l, s);
    const float inv = l == 0.f ? 0.f : 1.f / l;
    for (int i = 0; i < D / 32; ++i) out[at * D + i * 32 + lane] = from_float<BF>(o[i] * inv);
    if (lse && lane == 0) lse[at] = (m + log2f(l)) * 0.6931471805599453f;
    __syncwarp();
  }
}

template <bool BF, int D>
ig_status launch_tree(cudaStream_t st, const TreeShape& a, const uint16_t* q, const uint16_t* K, const uint16_t* V, uint16_t* out,
                      float* lse, void* ws) {
  k_tree_simple<BF, D><<<dim3((unsigned)a.T, (unsigned)a.Hkv), 128, 0, st>>>(q, K, V, a, out, lse, error_word());
  IG_CHECK_LAUNCH("tree attention launch");
  return IG_OK;
}

}  // namespace
}  // namespace ig

using namespace ig;

extern "C" size_t ig_paged_tree_attend_workspace_bytes(int n, int T_max, int Hq, int Hkv, int d) {
  if (n <= 0 || T_max <= 0 || T_max > kTreeMost || Hq <= 0 || Hkv <= 0 || Hq % Hkv || (d != 64 && d != 128)) return 0;
  return 256;
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
    return d == 128 ? launch_tree<false, 128>(st, a, q, K, V, out, lse, workspace)
                    : launch_tree<false, 64>(st, a, q, K, V, out, lse, workspace);
  return d == 128 ? launch_tree<true, 128>(st, a, q, K, V, out, lse, workspace)
                  : launch_tree<true, 64>(st, a, q, K, V, out, lse, workspace);
}
