// Page moves of a paged KV cache: every layer's K and V in one launch.
#include "ig_common.cuh"

namespace ig {
namespace {

constexpr int kMaxCopyLayers = 128;
struct CopyLayers {
  uint4* p[2 * kMaxCopyLayers];  // K of every layer, then V
};

// One CTA per (move, K or V of a layer).
__global__ void __launch_bounds__(256) k_page_copy(const CopyLayers P, int n_pages, int Hkv, int page, int vpr,
                                                  const int32_t* __restrict__ moves, int* err) {
  const int src = moves[3 * blockIdx.x], dst = moves[3 * blockIdx.x + 1], rows = moves[3 * blockIdx.x + 2];
  if (src < 0) return;
  if (src >= n_pages || dst < 0 || dst >= n_pages || rows < 0 || rows > page) {
    if (threadIdx.x == 0) raise_error(err, IG_DEVERR_INDEX);
    return;
  }
  uint4* base = P.p[blockIdx.y];
  for (int h = 0; h < Hkv; ++h) {
    const uint4* s = base + ((size_t)src * Hkv + h) * page * vpr;
    uint4* d = base + ((size_t)dst * Hkv + h) * page * vpr;
    for (int i = threadIdx.x; i < rows * vpr; i += blockDim.x) d[i] = s[i];
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
  IG_REQUIRE((double)Hkv * page * (d / 8) < 2147483648.0, "a page must stay below 2^31 pieces of 16 bytes");
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
  k_page_copy<<<grid, 256, 0, as_stream(stream)>>>(P, n_pages, Hkv, page, d / 8, moves, error_word());
  IG_CHECK_LAUNCH("page copy launch");
  return IG_OK;
}
