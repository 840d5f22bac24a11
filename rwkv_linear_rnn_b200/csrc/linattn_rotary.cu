// linattn_rotary.cu -- rotary positions of queries and keys (C ABI in
// include/linattn.h).
//
// Pair i of a head at position p turns by the angle p inv_freq[i].  The
// angle's turns are formed and reduced in float64 pairs, each product with the
// remainder that an FMA gives (Dekker's product; p reaches 2^53, where float64
// alone is off by a radian, as float32 is from about 2^20 on), and what is left
// of a turn goes to sincospi in float32.  Every element is read once and written once, 16 bytes
// at a time when the layout allows: the kernel is bound by HBM.  A block has up
// to 512 items of one or a few positions, so that a sine and cosine serve all
// heads of q and k; a thread's four items are on their way before the sines are
// computed, and everything per item is 32-bit arithmetic without a division.
// 8 x 4096 positions of 32 heads of 128 in bfloat16: 88 us (6.1 TB/s), with half
// of each head turned 86 us; blocks of 256 threads 91, one item a thread 95.
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
  int pairs, items;   // of a head: items that turn, all items
  int tail;           // elements that an item behind the pairs copies
  int tokens, parts;  // positions of a block, or blocks of a position's items
  int share;          // items of such a block
  uint32_t by_tok, by_head;  // for divisions by a position's and a head's items
};

constexpr int kThreads = 128, kItems = 4;
// 1 / (2 pi) as a float64 and what is left of it.
constexpr double kTurn = 0x1.45f306dc9c883p-3, kTurnLow = -0x1.6b01ec5417056p-57;
// The part of p f / (2 pi) beyond whole turns, within half a turn of 0.
__device__ __forceinline__ float part_of_turn(double p, double f) {
  const double angle = p * f, t = angle * kTurn;
  const double low = fma(angle, kTurn, -t) + fma(angle, kTurnLow, fma(p, f, -angle) * kTurn);
  const double r = t - rint(t) + low;
  return (float)(r - rint(r));
}
// e / d for e d < 2^32 with m = ceil(2^32 / d); 0 stands for d = 1.
__device__ __forceinline__ uint32_t divide(uint32_t e, uint32_t m) { return m ? __umulhi(e, m) : e; }

__device__ __forceinline__ float lo16(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi16(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}

// V elements of a tensor: as they are stored (16 bytes, or one element), and as
// float32.
template <typename E, int V>
struct Pack;
template <>
struct Pack<float, 4> {
  typedef uint4 Raw;
  static __device__ __forceinline__ void get(const Raw &v, float (&x)[4]) {
    x[0] = __uint_as_float(v.x), x[1] = __uint_as_float(v.y), x[2] = __uint_as_float(v.z), x[3] = __uint_as_float(v.w);
  }
  static __device__ __forceinline__ Raw put(const float (&x)[4]) {
    return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
  }
};
template <>
struct Pack<uint16_t, 8> {
  typedef uint4 Raw;
  static __device__ __forceinline__ void get(const Raw &v, float (&x)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) x[2 * k] = lo16(w[k]), x[2 * k + 1] = hi16(w[k]);
  }
  static __device__ __forceinline__ Raw put(const float (&x)[8]) {
    return make_uint4(pack2(x[0], x[1]), pack2(x[2], x[3]), pack2(x[4], x[5]), pack2(x[6], x[7]));
  }
};
template <>
struct Pack<uint16_t, 4> {
  typedef uint2 Raw;
  static __device__ __forceinline__ void get(const Raw &v, float (&x)[4]) {
    x[0] = lo16(v.x), x[1] = hi16(v.x), x[2] = lo16(v.y), x[3] = hi16(v.y);
  }
  static __device__ __forceinline__ Raw put(const float (&x)[4]) { return make_uint2(pack2(x[0], x[1]), pack2(x[2], x[3])); }
};
template <>
struct Pack<float, 1> {
  typedef float Raw;
  static __device__ __forceinline__ void get(const Raw &v, float (&x)[1]) { x[0] = v; }
  static __device__ __forceinline__ Raw put(const float (&x)[1]) { return x[0]; }
};
template <>
struct Pack<uint16_t, 1> {
  typedef uint16_t Raw;
  static __device__ __forceinline__ void get(const Raw &v, float (&x)[1]) { x[0] = lo16(v); }
  static __device__ __forceinline__ Raw put(const float (&x)[1]) { return (uint16_t)(pack2(x[0], 0.f) & 0xFFFFu); }
};

// One item of a head: V pairs in the half layout (elements V j.. and
// V j + R/2..); V/2 pairs in the interleaved one (2 elements there when V = 1);
// or, behind the pairs, V elements to copy (2 V if the item's registers and the
// head's size allow).
template <typename E, int V, bool INTER>
__global__ void __launch_bounds__(kThreads) rotary_kernel(const __grid_constant__ Args a) {
  typedef Pack<E, V> P;
  typedef typename P::Raw Raw;
  constexpr bool TWO = !(INTER && V > 1);     // an item's pairs lie in two places
  constexpr int W = INTER && V == 1 ? 2 : V;  // elements of an interleaved item
  extern __shared__ float2 cs[];              // [tokens][R / 2]: cos, sin, times mscale
  const uint32_t half = a.R / 2, per_tok = (uint32_t)(a.Hq + a.Hk) * a.items;
  const uint32_t part = blockIdx.x % (uint32_t)a.parts;
  const int64_t first = (int64_t)(blockIdx.x / (uint32_t)a.parts) * a.tokens, all = a.B * a.T;
  const uint32_t m = (uint32_t)min((int64_t)a.tokens, all - first);
  const uint32_t T = (uint32_t)a.T, b0 = (uint32_t)first / T, t0 = (uint32_t)first % T;
  // items [from, to) of the block's m positions
  const uint32_t from = part * a.share, to = a.parts > 1 ? min(from + a.share, per_tok) : m * per_tok;

  Raw x[kItems][TWO ? 2 : 1];
  E *dst[kItems];
  uint32_t wi[kItems];  // the item's first entry of cs, or a mark
  constexpr uint32_t kNone = ~0u, kCopy = ~1u, kCopy2 = ~2u;
#pragma unroll
  for (int n = 0; n < kItems; ++n) {
    const uint32_t e = from + n * kThreads + threadIdx.x;
    wi[n] = kNone;
    if (e >= to) continue;
    const uint32_t i = a.parts > 1 ? 0u : divide(e, a.by_tok), f = e - i * per_tok;
    const uint32_t hh = V > 1 ? divide(f, a.by_head) : f / (uint32_t)a.items, j = f - hh * a.items;
    uint32_t b = b0, t = t0 + i;
    while (t >= T) t -= T, ++b;
    const bool is_q = hh < (uint32_t)a.Hq;
    const View &in = is_q ? a.q : a.k, &out = is_q ? a.oq : a.ok;
    const uint32_t h = is_q ? hh : hh - a.Hq;
    const E *src = static_cast<const E *>(in.p) + (b * in.sb + t * in.st + h * in.sh);
    dst[n] = static_cast<E *>(const_cast<void *>(out.p)) + (b * out.sb + t * out.st + h * out.sh);
    if (j < (uint32_t)a.pairs) {
      const uint32_t x0 = INTER ? W * j : V * j;
      wi[n] = i * half + (INTER ? x0 / 2 : x0);
      x[n][0] = *reinterpret_cast<const Raw *>(src + x0);
      if constexpr (TWO) x[n][1] = *reinterpret_cast<const Raw *>(src + (INTER ? x0 + 1 : x0 + half));
      dst[n] += x0;
    } else if (is_q ? a.copy_q : a.copy_k) {
      const uint32_t x0 = a.R + a.tail * (j - a.pairs);
      wi[n] = a.tail > V ? kCopy2 : kCopy;
      x[n][0] = *reinterpret_cast<const Raw *>(src + x0);
      if constexpr (TWO)
        if (a.tail > V) x[n][1] = *reinterpret_cast<const Raw *>(src + x0 + V);
      dst[n] += x0;
    }
  }
  for (uint32_t e = threadIdx.x; e < m * half; e += kThreads) {
    const uint32_t i = e / half;
    uint32_t b = b0, t = t0 + i;
    while (t >= T) t -= T, ++b;
    const int64_t at = b * a.pos_sb + t;
    const double p = a.pos64 ? (double)static_cast<const int64_t *>(a.pos)[at] : (double)static_cast<const int32_t *>(a.pos)[at];
    float sn, c;
    sincospif(2.f * part_of_turn(p, a.inv_freq[e - i * half]), &sn, &c);
    cs[e] = make_float2(a.mscale * c, a.inverse ? -a.mscale * sn : a.mscale * sn);
  }
  __syncthreads();
#pragma unroll
  for (int n = 0; n < kItems; ++n) {
    if (wi[n] == kNone) continue;
    if (wi[n] == kCopy || wi[n] == kCopy2) {
      *reinterpret_cast<Raw *>(dst[n]) = x[n][0];
      if constexpr (TWO)
        if (wi[n] == kCopy2) *reinterpret_cast<Raw *>(dst[n] + V) = x[n][1];
      continue;
    }
    const float2 *w = cs + wi[n];
    float v[V];
    P::get(x[n][0], v);
    if constexpr (!TWO) {
#pragma unroll
      for (int r = 0; r < V / 2; ++r) {
        const float2 z = w[r];
        const float p = v[2 * r], q = v[2 * r + 1];
        v[2 * r] = p * z.x - q * z.y;
        v[2 * r + 1] = p * z.y + q * z.x;
      }
    } else {
      float u[V];
      P::get(x[n][1], u);
#pragma unroll
      for (int r = 0; r < V; ++r) {
        const float2 z = w[r];
        const float p = v[r], q = u[r];
        v[r] = p * z.x - q * z.y;
        u[r] = p * z.y + q * z.x;
      }
      *reinterpret_cast<Raw *>(dst[n] + (INTER ? 1 : half)) = P::put(u);
    }
    *reinterpret_cast<Raw *>(dst[n]) = P::put(v);
  }
}

}  // namespace rotary
}  // namespace wkv

namespace {
using namespace wkv;
using namespace wkv::rotary;

uint32_t reciprocal(uint32_t d) { return d <= 1 ? 0u : 0xFFFFFFFFu / d + 1u; }
template <typename E, int V>
cudaError_t launch(Args a, bool inter, cudaStream_t st) {
  const int W = inter ? (V == 1 ? 2 : V) : V;
  a.pairs = inter ? a.R / W : a.R / 2 / V;
  a.tail = (!inter || V == 1) && (a.D - a.R) % (2 * V) == 0 ? 2 * V : V;
  a.items = a.pairs + (a.copy_q || a.copy_k ? (a.D - a.R) / a.tail : 0);
  const int64_t per_tok = (int64_t)(a.Hq + a.Hk) * a.items, most = kThreads * kItems, half = a.R / 2;
  // few positions: fewer items each, over more blocks, to shorten the call
  int64_t want = most;
  while (want > kThreads && a.B * a.T * ((per_tok + want - 1) / want) < 592) want /= 2;
  a.parts = (int)((per_tok + want - 1) / want);
  a.share = (int)((per_tok + a.parts - 1) / a.parts);
  a.tokens = a.parts > 1 ? 1 : (int)std::max<int64_t>(1, std::min({want / per_tok, int64_t(16), 4096 / half}));
  a.by_tok = reciprocal((uint32_t)per_tok), a.by_head = reciprocal((uint32_t)a.items);
  const int64_t blocks = (a.B * a.T + a.tokens - 1) / a.tokens * a.parts;
  const size_t smem = sizeof(float2) * a.tokens * half;
  return inter ? launch_kernel(rotary_kernel<E, V, true>, dim3((unsigned)blocks), dim3(kThreads), smem, st, a)
               : launch_kernel(rotary_kernel<E, V, false>, dim3((unsigned)blocks), dim3(kThreads), smem, st, a);
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
// Pieces of V elements: every row of every head starts on their bytes.
bool fits(const View &v, int V, size_t es) { return aligned(v.p, V * es) && v.sb % V == 0 && v.st % V == 0 && v.sh % V == 0; }
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
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const bool inter = interleaved != 0;
  auto pieces = [&](int V) {
    bool ok = D % V == 0 && R % (inter ? V : 2 * V) == 0;
    for (const View *x : {&a.q, &a.oq, &a.k, &a.ok}) ok = ok && fits(*x, V, es);
    return ok;
  };
  // 16 bytes, else 8 of bfloat16 (R / 2 an odd multiple of 4, as in 40 of 80), else one element
  cudaError_t e;
  if (dtype == WKV_F32) e = pieces(4) ? launch<float, 4>(a, inter, st) : launch<float, 1>(a, inter, st);
  else e = pieces(8) ? launch<uint16_t, 8>(a, inter, st) : pieces(4) ? launch<uint16_t, 4>(a, inter, st) : launch<uint16_t, 1>(a, inter, st);
  return cuda_status(e);
}
