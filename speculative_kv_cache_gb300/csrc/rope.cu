// Queries and keys on their way from the projections: per-head RMS norm, rotation, and the keys
// and values into the pages of a paged cache; and the rotary frequencies on the host.
#include <cuda_bf16.h>
#include <math.h>

#include "ig_common.cuh"

namespace ig {
namespace {

// Eight 16-bit values in a uint4.
template <bool BF>
__device__ __forceinline__ void unpack8(const uint4& r, float (&f)[8]) {
  const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float2 v;
    if constexpr (BF) v = make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
    else v = h2_to_f2(w[i]);
    f[2 * i] = v.x;
    f[2 * i + 1] = v.y;
  }
}
template <bool BF>
__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (BF) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&h);
    } else {
      const __half2 h = __floats2half2_rn(f[2 * i], f[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// 16-byte load past L1 (every row is read once); not the read-only path, q may be written in place
__device__ __forceinline__ uint4 ld_once(const uint16_t* p) {
  uint4 r;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
               : "l"(p));
  return r;
}

struct RopeArgs {
  const uint16_t *q, *k, *v, *wq, *wk;
  int64_t sq, sk, sv;
  const int32_t *pos, *slot;
  const uint64_t* turns;
  uint16_t *qo, *ko, *vo;
  int T, Hq, Hkv, rot, layout, page, n_pages;
  float eps, rscale;
  int heads, chunk, chunks;  // rows of a token; rows of a work item, items of a token
};

constexpr int kRopeThreads = 128;
constexpr int kRopeFly = 2;  // rows per batch of a lane group; two batches in flight
constexpr int kRopeWarpsPerSm = 32;

// A row (one head of one token) is taken by D / 16 lanes with two 16-byte pieces each, chosen so
// that a lane holds both elements of its eight pairs: no exchange but the norm's sum.  A warp takes
// a work item: `chunk` of a token's rows (q heads, then k, then v), 32 / (D / 16) of them side by
// side; its lanes' sines and cosines are computed once per item.
//
// The angle of pair j at position p, in turns, is the low 64 bits of p * turns[j]: whole turns fall
// off the top of the integer, so a far position costs no precision.  Its top 32 bits, rounded, are
// the half turns that sincospif takes.
//
// HBM-bound where there are many tokens: every row is read and written once.  Measured (4 x 3968
// tokens of 32 + 64 heads of 128 fp16 into pages, 780 MB): 125 us, 6.2 TB/s, 0.92 of the copy rate; 4097
// tokens of 40 + 16 normed bf16 heads (117 MB): 22.2 us, 5.3 TB/s; one launch alone 2.8 us.  The next
// batch of rows is loaded before the last is worked on (without: 29 us for the second), five CTAs
// per SM (4: 25.2, 6: 24.1, 8 with one row per batch: 23.3 us).
template <bool BF, int D>
__global__ void __launch_bounds__(kRopeThreads, 5) k_qk_norm_rope(const RopeArgs a, int* err) {
  constexpr int GL = D / 16, RPW = 32 / GL;
  pdl_trigger();  // the attention that reads the pages may set up meanwhile
  pdl_wait();
  const long long item = (long long)blockIdx.x * (kRopeThreads / 32) + (threadIdx.x >> 5);
  if (item >= (long long)a.T * a.chunks) return;
  const int t = (int)(item / a.chunks), h0 = (int)(item % a.chunks) * a.chunk, h1 = min(a.heads, h0 + a.chunk);
  const int lane = threadIdx.x & 31, g = lane / GL, i = lane % GL;
  const unsigned group = (GL == 8 ? 0xffu : 0xfu) << (g * GL);
  // this lane's pieces (of 8 elements) and whether they are rotated
  int c0, c1;
  bool r0, r1;
  if (a.layout == IG_ROPE_HALF) {
    const int hc = a.rot / 16;
    r0 = r1 = i < hc;
    c0 = r0 ? i : 2 * i;  // 2 hc + 2 (i - hc)
    c1 = r0 ? i + hc : 2 * i + 1;
  } else {
    c0 = i;
    c1 = i + GL;
    r0 = c0 * 8 < a.rot;
    r1 = c1 * 8 < a.rot;
  }
  // where the token's key and value go; the row of head hk is hk * step further
  size_t row = (size_t)t * a.Hkv, step = 1;
  bool put = true;
  if (a.page && h1 > a.Hq) {
    const int sl = __ldca(a.slot + t), at = sl / a.page;
    if (sl < 0 || at >= a.n_pages) {
      put = false;
      if (sl >= 0 && lane == 0) raise_error(err, IG_DEVERR_INDEX);
    } else {
      row = (size_t)at * a.Hkv * a.page + sl % a.page;
      step = a.page;
    }
  }
  auto load = [&](int hb, uint4 (&raw)[kRopeFly][2]) {
#pragma unroll
    for (int x = 0; x < kRopeFly; ++x) {
      const int h = hb + x * RPW;
      if (h < h1) {
        const uint16_t* src = h < a.Hq ? a.q + t * a.sq + (int64_t)h * D
                              : h < a.Hq + a.Hkv ? a.k + t * a.sk + (int64_t)(h - a.Hq) * D
                                                 : a.v + t * a.sv + (int64_t)(h - a.Hq - a.Hkv) * D;
        raw[x][0] = ld_once(src + c0 * 8);
        raw[x][1] = ld_once(src + c1 * 8);
      }
    }
  };
  uint4 raw[kRopeFly][2], next[kRopeFly][2];
  load(h0 + g, raw);
  // (the angles while the first rows are on their way)
  float cs[8], sn[8];
  if (r0 && h0 < a.Hq + a.Hkv) {
    const uint64_t p = (uint64_t)(int64_t)__ldca(a.pos + t);
#pragma unroll
    for (int x = 0; x < 8; ++x) {
      const int j = a.layout == IG_ROPE_HALF ? 8 * i + x : 4 * (x < 4 ? c0 : c1) + (x & 3);
      if (a.layout == IG_ROPE_PAIRS && x >= 4 && !r1) continue;
      const uint64_t at = p * __ldca(reinterpret_cast<const unsigned long long*>(a.turns) + j);
      sincospif((float)(int32_t)((at + 0x80000000ull) >> 32) * 4.656612873077393e-10f, &sn[x], &cs[x]);
      sn[x] *= a.rscale;
      cs[x] *= a.rscale;
    }
  }
  for (int hb = h0 + g; hb - g < h1; hb += RPW * kRopeFly) {
    load(hb + RPW * kRopeFly, next);
#pragma unroll
    for (int x = 0; x < kRopeFly; ++x) {
      const int h = hb + x * RPW;
      if (h >= h1) continue;
      if (h < a.Hq + a.Hkv) {
        const uint16_t* w = h < a.Hq ? a.wq : a.wk;
        float e[8], f[8];
        unpack8<BF>(raw[x][0], e);
        unpack8<BF>(raw[x][1], f);
        if (w) {
          float ss = 0.f, w0[8], w1[8];
#pragma unroll
          for (int y = 0; y < 8; ++y) ss = fmaf(e[y], e[y], fmaf(f[y], f[y], ss));
#pragma unroll
          for (int o = GL / 2; o; o >>= 1) ss += __shfl_xor_sync(group, ss, o);
          const float rn = rsqrtf(ss * (1.f / D) + a.eps);
          unpack8<BF>(__ldca(reinterpret_cast<const uint4*>(w) + c0), w0);
          unpack8<BF>(__ldca(reinterpret_cast<const uint4*>(w) + c1), w1);
#pragma unroll
          for (int y = 0; y < 8; ++y) {
            e[y] *= rn * w0[y];
            f[y] *= rn * w1[y];
          }
        }
        if (a.layout == IG_ROPE_HALF) {
          if (r0)
#pragma unroll
            for (int y = 0; y < 8; ++y) {
              const float u = e[y] * cs[y] - f[y] * sn[y];
              f[y] = e[y] * sn[y] + f[y] * cs[y];
              e[y] = u;
            }
        } else {
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            if (r0) {
              const float u = e[2 * y] * cs[y] - e[2 * y + 1] * sn[y];
              e[2 * y + 1] = e[2 * y] * sn[y] + e[2 * y + 1] * cs[y];
              e[2 * y] = u;
            }
            if (r1) {
              const float u = f[2 * y] * cs[4 + y] - f[2 * y + 1] * sn[4 + y];
              f[2 * y + 1] = f[2 * y] * sn[4 + y] + f[2 * y + 1] * cs[4 + y];
              f[2 * y] = u;
            }
          }
        }
        raw[x][0] = pack8<BF>(e);
        raw[x][1] = pack8<BF>(f);
      }
      uint16_t* dst;
      if (h < a.Hq) {
        dst = a.qo + ((size_t)t * a.Hq + h) * D;
      } else {
        if (!put) continue;
        const bool isk = h < a.Hq + a.Hkv;
        dst = (isk ? a.ko : a.vo) + (row + step * (isk ? h - a.Hq : h - a.Hq - a.Hkv)) * D;
      }
      *reinterpret_cast<uint4*>(dst + c0 * 8) = raw[x][0];
      *reinterpret_cast<uint4*>(dst + c1 * 8) = raw[x][1];
    }
#pragma unroll
    for (int x = 0; x < kRopeFly; ++x) {
      raw[x][0] = next[x][0];
      raw[x][1] = next[x][1];
    }
  }
}

template <bool BF, int D>
ig_status launch_rope(cudaStream_t st, RopeArgs a) {
  constexpr int RPW = 32 / (D / 16);
  a.heads = a.Hq + (a.vo ? 2 : 1) * a.Hkv;
  // A work item is as many rows as leave kRopeWarpsPerSm items per SM, from one step of a warp up to
  // the whole token: few tokens spread over the SMs, many share each angle among their rows.  (64 items
  // per SM: 23.9 -> 25.0 us at 4097 tokens.)
  const long long rows = (long long)a.T * a.heads, want = (long long)sm_count(st) * kRopeWarpsPerSm;
  const long long per = (rows + want - 1) / want;
  a.chunks = per < a.heads ? (int)((a.heads + per - 1) / per) : 1;
  a.chunk = ((a.heads + a.chunks - 1) / a.chunks + RPW - 1) / RPW * RPW;
  a.chunks = (a.heads + a.chunk - 1) / a.chunk;
  const long long items = (long long)a.T * a.chunks, ctas = (items + kRopeThreads / 32 - 1) / (kRopeThreads / 32);
  const cudaError_t e = launch_pdl(k_qk_norm_rope<BF, D>, dim3((unsigned)ctas), dim3(kRopeThreads), 0, st, a, error_word());
  if (e != cudaSuccess) return cuda_fail(e, "norm and rotation launch");
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
  // (frequencies grow or shrink with j, so the first and last bound them)
  IG_REQUIRE(isfinite(theta) && isfinite(pow(theta, -2.0 * (rot / 2 - 1) / rot)), "a frequency or the base overflows");
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
                   v_out, T, Hq, Hkv, rot, layout, page, n_pages, eps, rot_scale, 0, 0, 0};
  cudaStream_t s = as_stream(stream);
  if (dtype == IG_F16) return d == 128 ? launch_rope<false, 128>(s, a) : launch_rope<false, 64>(s, a);
  return d == 128 ? launch_rope<true, 128>(s, a) : launch_rope<true, 64>(s, a);
}
