// Queries and keys on their way from the projections: per-head RMS norm, rotation, and the keys
// and values into the pages of a paged cache; and the rotary frequencies on the host.
#include <cuda_bf16.h>
#include <math.h>

#include "ig_common.cuh"

namespace ig {
namespace {

template <typename T>
__device__ __forceinline__ float to_f(T x);
template <>
__device__ __forceinline__ float to_f(__half x) { return __half2float(x); }
template <>
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
template <typename T>
__device__ __forceinline__ T from_f(float x);
template <>
__device__ __forceinline__ __half from_f(float x) { return __float2half_rn(x); }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f(float x) { return __float2bfloat16_rn(x); }

struct RopeArgs {
  const void *q, *k, *v, *wq, *wk;
  int64_t sq, sk, sv;
  const int32_t *pos, *slot;
  const uint64_t* turns;
  void *qo, *ko, *vo;
  int T, Hq, Hkv, rot, layout, page, n_pages;
  float eps, rscale;
};

// One warp per row (token, head), q heads first, then k, then v.
template <typename T, int D>
__global__ void __launch_bounds__(128) k_qk_norm_rope(const RopeArgs a, int* err) {
  const int heads = a.Hq + (a.vo ? 2 : 1) * a.Hkv;
  const long long r = (long long)blockIdx.x * 4 + (threadIdx.x >> 5);
  if (r >= (long long)a.T * heads) return;
  const int t = (int)(r / heads), h = (int)(r % heads), lane = threadIdx.x & 31;
  const int kind = h < a.Hq ? 0 : h < a.Hq + a.Hkv ? 1 : 2;
  const int hh = kind == 0 ? h : (h - a.Hq) % a.Hkv;
  const T* x = kind == 0 ? (const T*)a.q + t * a.sq + hh * D
                         : kind == 1 ? (const T*)a.k + t * a.sk + hh * D : (const T*)a.v + t * a.sv + hh * D;
  T* y;
  if (kind == 0) {
    y = (T*)a.qo + ((size_t)t * a.Hq + hh) * D;
  } else {
    T* o = (T*)(kind == 1 ? a.ko : a.vo);
    if (a.page) {
      const int s = a.slot[t];
      if (s < 0) return;
      if (s / a.page >= a.n_pages) {
        if (lane == 0) raise_error(err, IG_DEVERR_INDEX);
        return;
      }
      y = o + (((size_t)(s / a.page) * a.Hkv + hh) * a.page + s % a.page) * D;
    } else {
      y = o + ((size_t)t * a.Hkv + hh) * D;
    }
  }
  if (kind == 2) {
    for (int i = lane; i < D; i += 32) y[i] = x[i];
    return;
  }
  const T* w = (const T*)(kind == 0 ? a.wq : a.wk);
  float v[D / 32];
  float ss = 0.f;
#pragma unroll
  for (int i = 0; i < D / 64; ++i) {  // pairs j = lane + 32 i of the rotated part, then the rest
    const int j = lane + 32 * i;
    int e0, e1;
    if (j < a.rot / 2) {
      e0 = a.layout == IG_ROPE_HALF ? j : 2 * j;
      e1 = a.layout == IG_ROPE_HALF ? j + a.rot / 2 : 2 * j + 1;
    } else {
      e0 = 2 * j;
      e1 = 2 * j + 1;
    }
    v[2 * i] = to_f(x[e0]);
    v[2 * i + 1] = to_f(x[e1]);
    ss += v[2 * i] * v[2 * i] + v[2 * i + 1] * v[2 * i + 1];
  }
  for (int o = 16; o; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
  const float rn = w ? 1.f / sqrtf(ss / D + a.eps) : 1.f;
#pragma unroll
  for (int i = 0; i < D / 64; ++i) {
    const int j = lane + 32 * i;
    const bool turn = j < a.rot / 2;
    const int e0 = turn && a.layout == IG_ROPE_HALF ? j : 2 * j;
    const int e1 = turn && a.layout == IG_ROPE_HALF ? j + a.rot / 2 : 2 * j + 1;
    float p = v[2 * i], n = v[2 * i + 1];
    if (w) {
      p *= rn * to_f(w[e0]);
      n *= rn * to_f(w[e1]);
    }
    if (turn) {
      // the angle in turns is the low 64 bits of position * turns; its top 32 bits, rounded, in
      // half turns
      const uint64_t at = (uint64_t)(int64_t)a.pos[t] * a.turns[j];
      float sn, cs;
      sincospif((float)(int32_t)((at + 0x80000000ull) >> 32) * 4.656612873077393e-10f, &sn, &cs);
      sn *= a.rscale;
      cs *= a.rscale;
      const float u = p * cs - n * sn;
      n = p * sn + n * cs;
      p = u;
    }
    y[e0] = from_f<T>(p);
    y[e1] = from_f<T>(n);
  }
}

template <typename T, int D>
ig_status launch_rope(cudaStream_t st, const RopeArgs& a) {
  const long long rows = (long long)a.T * (a.Hq + (a.vo ? 2 : 1) * a.Hkv);
  k_qk_norm_rope<T, D><<<(unsigned)((rows + 3) / 4), 128, 0, st>>>(a, error_word());
  IG_CHECK_LAUNCH("norm and rotation launch");
  return IG_OK;
}

// whether [p, p + n) and [r, r + m) share bytes
bool overlap(const void* p, size_t n, const void* r, size_t m) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(r);
  return p && r && a < b + m && b < a + n;
}

}  // namespace
}  // namespace ig

using namespace ig;

extern "C" ig_status ig_rope_turns(int rot, double theta, int scaling, double factor, int context, double p0,
                                   double p1, uint64_t* turns, float* rot_scale) {
  IG_REQUIRE(turns && rot_scale, "null argument");
  IG_REQUIRE(rot > 0 && rot % 2 == 0, "rot must be a positive multiple of 2 (got %d)", rot);
  IG_REQUIRE(theta > 0.0 && isfinite(theta), "theta must be positive");
  IG_REQUIRE(scaling >= IG_ROPE_PLAIN && scaling <= IG_ROPE_BANDS, "unknown scaling %d", scaling);
  IG_REQUIRE(scaling == IG_ROPE_PLAIN || (factor >= 1.0 && isfinite(factor)), "factor must be at least 1");
  IG_REQUIRE(scaling != IG_ROPE_BASE || rot > 2, "IG_ROPE_BASE needs rot > 2");
  const bool ranged = scaling == IG_ROPE_YARN || scaling == IG_ROPE_BANDS;
  IG_REQUIRE(!ranged || context > 0, "the trained context must be positive");
  IG_REQUIRE(scaling != IG_ROPE_YARN || (theta > 1.0 && p1 > 0.0 && p0 > p1 && isfinite(p0)),
             "IG_ROPE_YARN needs theta > 1 and p0 > p1 > 0");
  IG_REQUIRE(scaling != IG_ROPE_BANDS || (p0 > 0.0 && p1 > p0 && isfinite(p1)), "IG_ROPE_BANDS needs p1 > p0 > 0");
  const double two_pi = 6.283185307179586476925286766559;
  double lo = 0.0, hi = 0.0;
  if (scaling == IG_ROPE_BASE) theta *= pow(factor, (double)rot / (rot - 2));
  if (scaling == IG_ROPE_YARN) {
    auto at = [&](double n) { return rot * log(context / (two_pi * n)) / (2.0 * log(theta)); };
    lo = fmax(floor(at(p0)), 0.0);
    hi = fmin(ceil(at(p1)), rot - 1.0);
  }
  for (int j = 0; j < rot / 2; ++j) {
    double f = pow(theta, -2.0 * j / rot);
    if (scaling == IG_ROPE_LINEAR) {
      f /= factor;
    } else if (scaling == IG_ROPE_YARN) {
      const double r = fmin(fmax((j - lo) / fmax(hi - lo, 0.001), 0.0), 1.0);
      f = f / factor * r + f * (1.0 - r);
    } else if (scaling == IG_ROPE_BANDS) {
      const double w = two_pi / f;
      if (w > context / p0) {
        f /= factor;
      } else if (w >= context / p1) {
        const double s = (context / w - p0) / (p1 - p0);
        f *= (1.0 - s) / factor + s;
      }
    }
    const double turn = f / two_pi;
    turns[j] = (uint64_t)ldexp(turn - floor(turn), 64);  // below 2^64: the fraction is below 1
  }
  *rot_scale = scaling == IG_ROPE_YARN && factor > 1.0 ? (float)(0.1 * log(factor) + 1.0) : 1.f;
  return IG_OK;
}

extern "C" ig_status ig_qk_norm_rope(void* stream, int dtype, int T, int Hq, int Hkv, int d, int rot, int layout,
                                     const uint16_t* q, int64_t q_stride, const uint16_t* k, int64_t k_stride,
                                     const uint16_t* v, int64_t v_stride, const uint16_t* q_weight,
                                     const uint16_t* k_weight, float eps, const int32_t* positions,
                                     const uint64_t* turns, float rot_scale, uint16_t* q_out, int page, int n_pages,
                                     const int32_t* slot, uint16_t* k_out, uint16_t* v_out) {
  IG_REQUIRE(dtype == IG_F16 || dtype == IG_BF16, "dtype must be IG_F16 or IG_BF16 (got %d)", dtype);
  IG_REQUIRE(T >= 0 && Hq > 0 && Hkv > 0, "T must not be negative, Hq and Hkv positive");
  IG_REQUIRE(d == 64 || d == 128, "d must be 64 or 128 (got %d)", d);
  IG_REQUIRE(rot >= 0 && rot <= d && rot % 16 == 0, "rot must be 0 or a multiple of 16 up to d (got %d)", rot);
  IG_REQUIRE(layout == IG_ROPE_HALF || layout == IG_ROPE_PAIRS, "unknown layout %d", layout);
  if (T == 0) return IG_OK;
  IG_REQUIRE(q && k && q_out && k_out, "null pointer argument");
  IG_REQUIRE((v == nullptr) == (v_out == nullptr), "v and v_out go together");
  IG_REQUIRE(page == 0 || v, "pages take keys and values");
  IG_REQUIRE(rot == 0 || (positions && turns), "a rotation needs positions and turns");
  IG_REQUIRE(page >= 0 && page % 8 == 0, "page must be 0 or a positive multiple of 8 (got %d)", page);
  IG_REQUIRE(page > 0 ? n_pages > 0 && slot : n_pages == 0 && !slot, "page, n_pages and slot go together");
  IG_REQUIRE((double)n_pages * Hkv * page < 2147483648.0, "n_pages*Hkv*page must stay below 2^31 rows");
  IG_REQUIRE((long long)Hq + 2ll * Hkv < (1 << 24) && (double)T * ((double)Hq + 2.0 * Hkv) < 2147483648.0,
             "T*(Hq + 2 Hkv) must stay below 2^31 rows");
  IG_REQUIRE(q_stride >= (int64_t)Hq * d && k_stride >= (int64_t)Hkv * d && (!v || v_stride >= (int64_t)Hkv * d),
             "a stride is less than a token's heads");
  IG_REQUIRE(q_stride % 8 == 0 && k_stride % 8 == 0 && (!v || v_stride % 8 == 0), "strides must be multiples of 8");
  IG_REQUIRE(q_stride < (1ll << 40) && k_stride < (1ll << 40) && (!v || v_stride < (1ll << 40)), "stride too large");
  IG_REQUIRE(aligned(q, 16) && aligned(k, 16) && aligned(v, 16) && aligned(q_out, 16) && aligned(k_out, 16) &&
                 aligned(v_out, 16) && aligned(q_weight, 16) && aligned(k_weight, 16) && aligned(turns, 16),
             "q, k, v, weights, turns and outputs must be 16-byte aligned");
  IG_REQUIRE(aligned(positions, 4) && aligned(slot, 4), "positions and slot must be 4-byte aligned");
  IG_REQUIRE(!(q_weight || k_weight) || (eps >= 0.f && isfinite(eps)), "eps must not be negative");
  IG_REQUIRE(isfinite(rot_scale), "rot_scale must be finite");
  const size_t qb = ((size_t)(T - 1) * q_stride + (size_t)Hq * d) * 2, kb = ((size_t)(T - 1) * k_stride + (size_t)Hkv * d) * 2;
  const size_t vb = v ? ((size_t)(T - 1) * v_stride + (size_t)Hkv * d) * 2 : 0;
  const size_t qo = (size_t)T * Hq * d * 2, ko = (page ? (size_t)n_pages * page : (size_t)T) * Hkv * d * 2;
  IG_REQUIRE(!overlap(q_out, qo, q, qb) || (q_out == q && q_stride == (int64_t)Hq * d),
             "q_out may be q itself when its rows are dense, and must not overlap it otherwise");
  IG_REQUIRE(!overlap(q_out, qo, k, kb) && !overlap(q_out, qo, v, vb) && !overlap(k_out, ko, q, qb) &&
                 !overlap(k_out, ko, k, kb) && !overlap(k_out, ko, v, vb) && !overlap(v_out, ko, q, qb) &&
                 !overlap(v_out, ko, k, kb) && !overlap(v_out, ko, v, vb) && !overlap(q_out, qo, k_out, ko) &&
                 !overlap(q_out, qo, v_out, ko) && !overlap(k_out, ko, v_out, ko),
             "outputs must not overlap the inputs or each other");
  const RopeArgs a{q, k, v, q_weight, k_weight, q_stride, k_stride, v_stride, positions, slot, turns, q_out, k_out,
                   v_out, T, Hq, Hkv, rot, layout, page, n_pages, eps, rot_scale};
  cudaStream_t s = as_stream(stream);
  if (dtype == IG_F16) return d == 128 ? launch_rope<__half, 128>(s, a) : launch_rope<__half, 64>(s, a);
  return d == 128 ? launch_rope<__nv_bfloat16, 128>(s, a) : launch_rope<__nv_bfloat16, 64>(s, a);
}
