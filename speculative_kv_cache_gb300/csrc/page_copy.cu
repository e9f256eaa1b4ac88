// Page moves of a paged KV cache: every layer's K and V in one launch.
#include "ig_common.cuh"

namespace ig {
namespace {

constexpr int kMaxCopyLayers = 128;
struct CopyLayers {
  uint4* p[2 * kMaxCopyLayers];  // K of every layer, then V
};

// One CTA per (move, K or V of a layer).  The rows to copy are one run of 16-byte pieces (every head's first
// `rows` rows; with whole pages, contiguous memory), kFly of them in flight per thread.  HBM-bound where
// pages are many: 500 pages of 128 KB in the K and V of 16 layers (2.1 GB read and written) take 609 us, 6.9
// TB/s, as a plain copy does; eight moves of 1 to 16 rows in 32 layers (15.7 MB) 5.0 us, one alone 1.6 us.
constexpr int kCopyThreads = 256;
constexpr int kCopyFly = 4;
__global__ void __launch_bounds__(kCopyThreads) k_page_copy(const CopyLayers P, int n_pages, int Hkv, int page, int vpr,
                                                           const int32_t* __restrict__ moves, int* err) {
  pdl_trigger();
  pdl_wait();
  const int32_t* mv = moves + 3 * (size_t)blockIdx.x;
  const int src = __ldca(mv), dst = __ldca(mv + 1), rows = __ldca(mv + 2);
  if (src < 0) return;
  if (src >= n_pages || dst < 0 || dst >= n_pages || rows < 0 || rows > page) {
    if (threadIdx.x == 0) raise_error(err, IG_DEVERR_INDEX);
    return;
  }
  const int head = page * vpr, part = rows * vpr, total = Hkv * part;
  const uint4* s = P.p[blockIdx.y] + (size_t)src * Hkv * head;
  uint4* d = P.p[blockIdx.y] + (size_t)dst * Hkv * head;
  for (int i0 = threadIdx.x; i0 < total; i0 += kCopyThreads * kCopyFly) {
    uint4 v[kCopyFly];
    int at[kCopyFly];
#pragma unroll
    for (int x = 0; x < kCopyFly; ++x) {
      const int i = i0 + x * kCopyThreads;
      at[x] = -1;
      if (i < total) {
        at[x] = part == head ? i : i / part * head + i % part;
        v[x] = s[at[x]];
      }
    }
#pragma unroll
    for (int x = 0; x < kCopyFly; ++x)
      if (at[x] >= 0) d[at[x]] = v[x];
  }
}

}  // namespace
}  // namespace ig

using namespace ig;

extern "C" ig_status ig_page_copy(void* stream, int layers, int n_pages, int Hkv, int page, int d,
                                  uint16_t* const* K, uint16_t* const* V, int n, const int32_t* moves) {
  IG_REQUIRE(layers > 0 && layers <= kMaxCopyLayers, "layers must be in [1, %d]", kMaxCopyLayers);
  IG_REQUIRE(n_pages > 0 && Hkv > 0 && n >= 0, "n_pages, Hkv must be positive, n not negative");
  IG_REQUIRE(page > 0 && page % 8 == 0, "page must be a positive multiple of 8 (got %d)", page);
  IG_REQUIRE(d > 0 && d % 8 == 0, "d must be a positive multiple of 8 (got %d)", d);
  IG_REQUIRE((double)n_pages * Hkv * page < 2147483648.0, "n_pages*Hkv*page must stay below 2^31 rows");
  IG_REQUIRE((double)Hkv * page * (d / 8) < 1073741824.0, "a page must stay below 2^30 pieces of 16 bytes");
  IG_REQUIRE(K && V, "null pointer argument");
  CopyLayers P{};
  for (int l = 0; l < layers; ++l) {
    IG_REQUIRE(K[l] && V[l], "null pages of layer %d", l);
    IG_REQUIRE(aligned(K[l], 16) && aligned(V[l], 16), "the pages must be 16-byte aligned");
    P.p[l] = reinterpret_cast<uint4*>(K[l]);
    P.p[layers + l] = reinterpret_cast<uint4*>(V[l]);
  }
  if (n == 0) return IG_OK;
  IG_REQUIRE(moves && aligned(moves, 4), "null or misaligned moves");
  dim3 grid((unsigned)n, (unsigned)(2 * layers));
  const cudaError_t e = launch_pdl(k_page_copy, grid, dim3(kCopyThreads), 0, as_stream(stream), P, n_pages, Hkv, page, d / 8,
                                   moves, error_word());
  if (e != cudaSuccess) return cuda_fail(e, "page copy launch");
  IG_CHECK_LAUNCH("page copy launch");
  return IG_OK;
}
