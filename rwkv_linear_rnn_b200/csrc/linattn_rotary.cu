// linattn_rotary.cu -- rotary positions of queries and keys (C ABI in
// include/linattn.h).
//
// Pair i of a head at position p turns by the angle p inv_freq[i].  The
// angle's turns are formed and reduced in float64 (p reaches 2^53 and float32
// would lose whole radians from about 2^20 on), the remainder goes to
// sincospi in float32.  A block takes a few positions and all their heads, so
// each sine and cosine is computed once for q and k together (R / 2 of them
// against (Hq + Hk) D elements read and written) and the kernel is bound by
// HBM: every element is read once and written once, 16 bytes at a time when
// the layout allows.
#include <algorithm>
#include <utility>

#include "../../include/linattn.h"
#include "../../include/wkv.h"
#include "wkv_internal.cuh"

namespace wkv {
namespace rotary {

struct View {
  const void *p;
  int64_t sb, st, sh;
};
struct Args {
  int64_t B, T;
  int D, R, Hq, Hk;
  View q, k, oq, ok;
  int copy_q, copy_k;  // elements from R on are to be copied (out of place)
  const void *pos;
  int pos64;
  int64_t pos_sb;
  const double *inv_freq;
  float mscale;
  int inverse;
  int tokens;  // per block
};

constexpr int kThreads = 256;

__device__ __forceinline__ float lo16(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi16(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}

// V elements of a tensor as float32: 16 bytes (VEC), or one.
template <typename E, int V>
struct Pack;
template <>
struct Pack<float, 4> {
  static __device__ __forceinline__ void ld(const void *p, int64_t i, float (&x)[4]) {
    const float4 v = *reinterpret_cast<const float4 *>(static_cast<const float *>(p) + i);
    x[0] = v.x, x[1] = v.y, x[2] = v.z, x[3] = v.w;
  }
  static __device__ __forceinline__ void st(const void *p, int64_t i, const float (&x)[4]) {
    *reinterpret_cast<float4 *>(static_cast<float *>(const_cast<void *>(p)) + i) = make_float4(x[0], x[1], x[2], x[3]);
  }
};
template <>
struct Pack<uint16_t, 8> {
  static __device__ __forceinline__ void ld(const void *p, int64_t i, float (&x)[8]) {
    const uint4 v = *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(p) + i);
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) x[2 * k] = lo16(w[k]), x[2 * k + 1] = hi16(w[k]);
  }
  static __device__ __forceinline__ void st(const void *p, int64_t i, const float (&x)[8]) {
    *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(const_cast<void *>(p)) + i) =
        make_uint4(pack2(x[0], x[1]), pack2(x[2], x[3]), pack2(x[4], x[5]), pack2(x[6], x[7]));
  }
};
template <>
struct Pack<float, 1> {
  static __device__ __forceinline__ void ld(const void *p, int64_t i, float (&x)[1]) {
    x[0] = static_cast<const float *>(p)[i];
  }
  static __device__ __forceinline__ void st(const void *p, int64_t i, const float (&x)[1]) {
    static_cast<float *>(const_cast<void *>(p))[i] = x[0];
  }
};
template <>
struct Pack<uint16_t, 1> {
  static __device__ __forceinline__ void ld(const void *p, int64_t i, float (&x)[1]) {
    x[0] = lo16(static_cast<const uint16_t *>(p)[i]);
  }
  static __device__ __forceinline__ void st(const void *p, int64_t i, const float (&x)[1]) {
    static_cast<uint16_t *>(const_cast<void *>(p))[i] = (uint16_t)(pack2(x[0], 0.f) & 0xFFFFu);
  }
};

// One item of a head: V pairs in the half layout (elements V j.. and
// V j + R/2..); V/2 pairs in the interleaved one (2 V elements there when
// V = 1); or, behind the pairs, V elements to copy.
template <typename E, int V, bool INTER>
__global__ void __launch_bounds__(kThreads) rotary_kernel(Args a) {
  extern __shared__ float2 cs[];  // [tokens][R / 2]: cos, sin, times mscale
  const int64_t all = a.B * a.T, first = (int64_t)blockIdx.x * a.tokens;
  const int m = (int)min((int64_t)a.tokens, all - first);
  const int half = a.R / 2;
  for (int e = threadIdx.x; e < m * half; e += kThreads) {
    const int64_t tok = first + e / half;
    const int i = e % half;
    const int64_t at = tok / a.T * a.pos_sb + tok % a.T;
    const double p = a.pos64 ? (double)static_cast<const int64_t *>(a.pos)[at] : (double)static_cast<const int32_t *>(a.pos)[at];
    const double turns = p * a.inv_freq[i] * 0.15915494309189533577;  // 1 / (2 pi)
    float sn, c;
    sincospif(2.f * (float)(turns - rint(turns)), &sn, &c);
    cs[e] = make_float2(a.mscale * c, a.inverse ? -a.mscale * sn : a.mscale * sn);
  }
  __syncthreads();
  constexpr int W = INTER && V == 1 ? 2 : V;  // elements of an interleaved item
  const int pairs = INTER ? a.R / W : half / V, tail = (a.D - a.R) / V;
  const int items = pairs + (a.copy_q || a.copy_k ? tail : 0);
  const int per_tok = (a.Hq + a.Hk) * items;
  for (int e = threadIdx.x; e < m * per_tok; e += kThreads) {
    const int i = e / per_tok, f = e % per_tok, hh = f / items, j = f % items;
    const int64_t tok = first + i, b = tok / a.T, t = tok % a.T;
    const bool is_q = hh < a.Hq;
    const View &in = is_q ? a.q : a.k, &out = is_q ? a.oq : a.ok;
    const int h = is_q ? hh : hh - a.Hq;
    const int64_t src = b * in.sb + t * in.st + h * in.sh, dst = b * out.sb + t * out.st + h * out.sh;
    if (j >= pairs) {
      if (is_q ? a.copy_q : a.copy_k) {
        const int64_t x = a.R + (int64_t)V * (j - pairs);
        float v[V];
        Pack<E, V>::ld(in.p, src + x, v);
        Pack<E, V>::st(out.p, dst + x, v);
      }
      continue;
    }
    const float2 *w = cs + i * half;
    if (INTER && V > 1) {
      float v[V];
      Pack<E, V>::ld(in.p, src + (int64_t)V * j, v);
#pragma unroll
      for (int r = 0; r < V / 2; ++r) {
        const float2 z = w[V / 2 * j + r];
        const float x = v[2 * r], y = v[2 * r + 1];
        v[2 * r] = x * z.x - y * z.y;
        v[2 * r + 1] = x * z.y + y * z.x;
      }
      Pack<E, V>::st(out.p, dst + (int64_t)V * j, v);
    } else {
      const int64_t x0 = INTER ? 2 * (int64_t)j : (int64_t)V * j, x1 = INTER ? x0 + 1 : x0 + half;
      float v[V], u[V];
      Pack<E, V>::ld(in.p, src + x0, v);
      Pack<E, V>::ld(in.p, src + x1, u);
#pragma unroll
      for (int r = 0; r < V; ++r) {
        const float2 z = w[V * j + r];
        const float x = v[r], y = u[r];
        v[r] = x * z.x - y * z.y;
        u[r] = x * z.y + y * z.x;
      }
      Pack<E, V>::st(out.p, dst + x0, v);
      Pack<E, V>::st(out.p, dst + x1, u);
    }
  }
}

}  // namespace rotary
}  // namespace wkv

namespace {
using namespace wkv;
using namespace wkv::rotary;

template <typename E, int V>
cudaError_t launch(Args a, bool inter, cudaStream_t st) {
  // about 1024 items per block: enough loads in flight, and the sines shared
  const int64_t items = std::max<int64_t>(1, (int64_t)(a.Hq + a.Hk) * (inter ? a.R / V : a.R / 2 / V));
  a.tokens = (int)std::min<int64_t>(std::max<int64_t>(1, 1024 / items), 16);
  const unsigned grid = (unsigned)((a.B * a.T + a.tokens - 1) / a.tokens);
  const size_t smem = sizeof(float2) * a.tokens * (a.R / 2);
  return inter ? launch_kernel(rotary_kernel<E, V, true>, dim3(grid), dim3(kThreads), smem, st, a)
               : launch_kernel(rotary_kernel<E, V, false>, dim3(grid), dim3(kThreads), smem, st, a);
}

bool aligned(const void *p, size_t n) { return ((uintptr_t)p & (n - 1)) == 0; }
constexpr int64_t kMostStride = int64_t(1) << 40;
// An output's elements must not overlap each other (as linattn_decay's).
int check(const linattn_view *v, const Args &a, int H, size_t es, bool output) {
  if (!v || !v->ptr || v->stride_b < 0 || v->stride_t < 0 || v->stride_h < 0 || (a.B > 1 && v->stride_b > kMostStride) ||
      (a.T > 1 && v->stride_t > kMostStride) || (H > 1 && v->stride_h > kMostStride))
    return WKV_ERR_INVALID_ARG;
  if (!aligned(v->ptr, es)) return WKV_ERR_UNSUPPORTED;
  if (output) {
    std::pair<int64_t, int64_t> d[3] = {{v->stride_b, a.B}, {v->stride_t, a.T}, {v->stride_h, H}};
    std::sort(d, d + 3);
    int64_t span = a.D;
    for (const auto &x : d) {
      if (x.second <= 1) continue;
      if (x.first < span) return WKV_ERR_INVALID_ARG;
      span += x.first * (x.second - 1);
    }
  }
  return WKV_OK;
}
View view(const linattn_view *v) { return View{v->ptr, v->stride_b, v->stride_t, v->stride_h}; }
bool same(const linattn_view *x, const linattn_view *y) {
  return x->ptr == y->ptr && x->stride_b == y->stride_b && x->stride_t == y->stride_t && x->stride_h == y->stride_h;
}
// 16-byte accesses: every row of every head starts on 16 bytes.
bool fits16(const View &v, int V) { return aligned(v.p, 16) && v.sb % V == 0 && v.st % V == 0 && v.sh % V == 0; }
}  // namespace

extern "C" int linattn_rotary(int64_t B, int64_t T, int D, int R, int dtype, int64_t Hq, const linattn_view *q,
                              int64_t Hk, const linattn_view *k, const void *positions, int pos_bytes,
                              int64_t pos_stride_b, const double *inv_freq, float mscale, int interleaved, int inverse,
                              const linattn_view *out_q, const linattn_view *out_k, void *stream) {
  constexpr int64_t kMostHeads = int64_t(1) << 15;  // items of one position fit 32 bits
  if (B < 1 || T < 0 || B >= (int64_t(1) << 31) || T >= (int64_t(1) << 31) || B * T >= (int64_t(1) << 31) || D < 1 ||
      D > 1024 || R < 2 || R > D || (R & 1) || (dtype != WKV_F32 && dtype != WKV_BF16) || Hq < 1 || Hq > kMostHeads ||
      Hk < 0 || Hk > kMostHeads || (Hk == 0) != (k == nullptr) || (Hk == 0) != (out_k == nullptr) ||
      (pos_bytes != 4 && pos_bytes != 8) || pos_stride_b < 0)
    return WKV_ERR_INVALID_ARG;
  if (T == 0) return WKV_OK;
  if (!positions || !inv_freq) return WKV_ERR_INVALID_ARG;
  const size_t es = dtype == WKV_F32 ? 4 : 2;
  Args a{};
  a.B = B, a.T = T, a.D = D, a.R = R, a.Hq = (int)Hq, a.Hk = (int)Hk;
  const linattn_view *v[4] = {q, out_q, k, out_k};
  for (int i = 0; i < (Hk ? 4 : 2); ++i) {
    const int rc = check(v[i], a, i < 2 ? a.Hq : a.Hk, es, i & 1);
    if (rc != WKV_OK) return rc;
  }
  if (!aligned(positions, pos_bytes) || !aligned(inv_freq, 8)) return WKV_ERR_UNSUPPORTED;
  if (out_q->ptr == q->ptr && !same(out_q, q)) return WKV_ERR_INVALID_ARG;
  if (Hk && ((out_k->ptr == k->ptr && !same(out_k, k)) || out_q->ptr == k->ptr || out_k->ptr == q->ptr ||
             out_q->ptr == out_k->ptr))
    return WKV_ERR_INVALID_ARG;
  a.q = view(q), a.oq = view(out_q);
  a.k = Hk ? view(k) : a.q, a.ok = Hk ? view(out_k) : a.oq;
  a.copy_q = a.q.p != a.oq.p, a.copy_k = Hk && a.k.p != a.ok.p;
  a.pos = positions, a.pos64 = pos_bytes == 8, a.pos_sb = pos_stride_b;
  a.inv_freq = inv_freq, a.mscale = mscale, a.inverse = inverse;
  const int V = dtype == WKV_F32 ? 4 : 8;
  bool vec = D % V == 0 && R % (interleaved ? V : 2 * V) == 0;
  for (const View *x : {&a.q, &a.oq, &a.k, &a.ok}) vec = vec && fits16(*x, V);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const bool inter = interleaved != 0;
  const cudaError_t e = dtype == WKV_F32 ? (vec ? launch<float, 4>(a, inter, st) : launch<float, 1>(a, inter, st))
                                         : (vec ? launch<uint16_t, 8>(a, inter, st) : launch<uint16_t, 1>(a, inter, st));
  return e == cudaSuccess ? WKV_OK : WKV_ERR_CUDA;
}
