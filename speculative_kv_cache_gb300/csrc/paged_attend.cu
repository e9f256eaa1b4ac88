// Attention of one new token over a paged KV cache.
#include <cuda_bf16.h>
#include <math.h>

#include "ig_common.cuh"

namespace ig {
namespace {

constexpr int kPaThreads = 128;

template <typename T>
__device__ __forceinline__ float to_f(T x);
template <>
__device__ __forceinline__ float to_f(__half x) { return __half2float(x); }
template <>
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }

// One CTA per (sequence, query head): thread i takes tokens i, i + kPaThreads, ... with a
// running maximum, sum and output of its own, merged at the end.
template <typename T, int D>
__global__ void __launch_bounds__(kPaThreads) k_paged_attend(
    const T* __restrict__ q, const T* __restrict__ K, const T* __restrict__ V, const int32_t* __restrict__ table,
    const int32_t* __restrict__ L_valid, int Hq, int Hkv, int page, int n_pages, int max_pages, float scale,
    float* __restrict__ out, float* __restrict__ lse, int* err) {
  __shared__ float sm_m[kPaThreads], sm_l[kPaThreads], sm_o[kPaThreads];
  const int b = blockIdx.x / Hq, h = blockIdx.x % Hq, hk = h / (Hq / Hkv);
  int L = L_valid[b];
  if (L < 0 || L > max_pages * page) {
    if (threadIdx.x == 0) raise_error(err, IG_DEVERR_INDEX);
    L = L < 0 ? 0 : max_pages * page;
  }
  const T* qr = q + ((size_t)b * Hq + h) * D;
  float m = -INFINITY, l = 0.f, acc[D];
#pragma unroll
  for (int i = 0; i < D; ++i) acc[i] = 0.f;
  for (int t = threadIdx.x; t < L; t += kPaThreads) {
    const int g = table[(size_t)b * max_pages + t / page];
    if (g < 0 || g >= n_pages) {
      raise_error(err, IG_DEVERR_INDEX);
      continue;
    }
    const size_t row = (((size_t)g * Hkv + hk) * page + t % page) * D;
    float z = 0.f;
    for (int i = 0; i < D; ++i) z = fmaf(to_f(qr[i]), to_f(K[row + i]), z);
    z *= scale;
    const float mn = fmaxf(m, z);
    if (mn == -INFINITY) continue;
    const float c = expf(m - mn), p = expf(z - mn);
    l = l * c + p;
#pragma unroll
    for (int i = 0; i < D; ++i) acc[i] = fmaf(p, to_f(V[row + i]), acc[i] * c);
    m = mn;
  }
  sm_m[threadIdx.x] = m;
  sm_l[threadIdx.x] = l;
  __syncthreads();
  float M = -INFINITY, S = 0.f;
  for (int i = 0; i < kPaThreads; ++i) M = fmaxf(M, sm_m[i]);
  const float base = M == -INFINITY ? 0.f : M;
  for (int i = 0; i < kPaThreads; ++i) S += sm_l[i] * expf(sm_m[i] - base);
  const float f = expf(m - base);
  float* o = out + ((size_t)b * Hq + h) * D;
#pragma unroll
  for (int i = 0; i < D; ++i) {
    sm_o[threadIdx.x] = acc[i] * f;
    __syncthreads();
    for (int w = kPaThreads / 2; w; w >>= 1) {
      if (threadIdx.x < w) sm_o[threadIdx.x] += sm_o[threadIdx.x + w];
      __syncthreads();
    }
    if (threadIdx.x == 0) o[i] = S == 0.f ? 0.f : sm_o[0] / S;
    __syncthreads();
  }
  if (threadIdx.x == 0 && lse) lse[(size_t)b * Hq + h] = M + logf(S);
}

template <typename T, int D>
ig_status launch_paged(cudaStream_t st, int B, int Hq, int Hkv, int page, int n_pages, int max_pages, float scale,
                       const uint16_t* q, const uint16_t* K, const uint16_t* V, const int32_t* table,
                       const int32_t* L, float* out, float* lse) {
  k_paged_attend<T, D><<<B * Hq, kPaThreads, 0, st>>>(
      reinterpret_cast<const T*>(q), reinterpret_cast<const T*>(K), reinterpret_cast<const T*>(V), table, L, Hq, Hkv,
      page, n_pages, max_pages, scale, out, lse, error_word());
  IG_CHECK_LAUNCH("paged attention launch");
  return IG_OK;
}

}  // namespace
}  // namespace ig

using namespace ig;

extern "C" size_t ig_paged_attend_workspace_bytes(int B, int Hq, int Hkv, int d) {
  if (B <= 0 || Hq <= 0 || Hkv <= 0 || Hq % Hkv || (d != 64 && d != 128)) return 0;
  return 256;
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
  IG_REQUIRE((long long)B * Hq < (1ll << 31), "B*Hq must stay below 2^31");
  IG_REQUIRE((long long)max_pages * page < (1ll << 30), "max_pages*page must stay below 2^30");
  IG_REQUIRE((double)n_pages * Hkv * page < 2147483648.0, "n_pages*Hkv*page must stay below 2^31 rows");
  IG_REQUIRE(isfinite(scale), "scale must be finite");
  IG_REQUIRE(q && K && V && page_table && L_valid && out, "null pointer argument");
  IG_REQUIRE(aligned(q, 16) && aligned(K, 16) && aligned(V, 16), "q, K, V must be 16-byte aligned");
  IG_REQUIRE(aligned(out, 16), "out must be 16-byte aligned");
  IG_REQUIRE(aligned(page_table, 4) && aligned(L_valid, 4) && aligned(lse, 4),
             "page_table, L_valid, lse must be 4-byte aligned");
  const size_t need = ig_paged_attend_workspace_bytes(B, Hq, Hkv, d);
  if (!workspace || workspace_bytes < need)
    return fail(IG_ERR_CAPACITY, "paged attention needs %zu workspace bytes", need);
  IG_REQUIRE(aligned(workspace, 256), "workspace must be 256-byte aligned");
  cudaStream_t s = as_stream(stream);
#define IG_PA(T, D) \
  return launch_paged<T, D>(s, B, Hq, Hkv, page, n_pages, max_pages, scale, q, K, V, page_table, L_valid, out, lse)
  if (dtype == IG_F16) {
    if (d == 128) IG_PA(__half, 128);
    IG_PA(__half, 64);
  }
  if (d == 128) IG_PA(__nv_bfloat16, 128);
  IG_PA(__nv_bfloat16, 64);
#undef IG_PA
}
