// linattn_decay_rec.cu -- linear attention with a decay for each head on the
// CUDA cores: the recurrence itself, the single-token step, and the scan that
// joins the segments of a long sequence.
//
// The recurrence R_t = lam R_{t-1} + b_t c_t^T, o_t = a_t^T R_t costs two FMAs
// per state element and position and the decay.  The decay leaves the inner
// loop: over a batch of 8 positions the kernel holds R / lam^k instead of R
// (b enters divided by lam^k, o is multiplied by it: scalings, which round no
// more than the products they replace) and multiplies R by lam^8 once.  Where
// lam^8 < 2^-16 that would cost range, and R is multiplied at each position.
// (8 x 1024 x 12 heads of 64, forward: 469 us with three FMAs, one at a time;
// 188 with two-wide ones; 86 with fetches and strides that cost no arithmetic.)
//
// The kernel is bound by the FMA pipes: it serves float32 tensors (which the
// tensor cores' bfloat16 products would round), heads and strides that TMA
// cannot describe, and sequences of a few positions.
//
// Layout: a warp owns 64 rows (32 if X <= 32) and 32 columns of the state;
// lane (lane / 8, lane % 8) holds 4 columns of 16 (8) rows, as pairs of rows
// for the two-wide FMAs.  Per position a lane reads a and b of its rows as
// float4s that 8 lanes share and its 4 columns of c: 9 loads for 128 FMAs.
// The products' sums over the 4 lanes of a column are taken for four
// positions at a time (12 shuffles, one float4 stored), over the two warps of
// a column's rows when they are written out.
#include <algorithm>
#include <type_traits>

#include "linattn_decay.cuh"

namespace wkv {
namespace decay {

constexpr int kTB = 16;       // positions staged in shared memory at a time
constexpr int kStepWarps = 8; // most warps per block of the step: 128 columns

template <typename E>
__device__ __forceinline__ float load1(const void *p, int64_t i);
template <>
__device__ __forceinline__ float load1<float>(const void *p, int64_t i) {
  return static_cast<const float *>(p)[i];
}
template <>
__device__ __forceinline__ float load1<uint16_t>(const void *p, int64_t i) {
  return __uint_as_float((uint32_t) static_cast<const uint16_t *>(p)[i] << 16);
}
template <typename E>
__device__ __forceinline__ void store1(const void *p, int64_t i, float x);
template <>
__device__ __forceinline__ void store1<float>(const void *p, int64_t i, float x) {
  static_cast<float *>(const_cast<void *>(p))[i] = x;
}
template <>
__device__ __forceinline__ void store1<uint16_t>(const void *p, int64_t i, float x) {
  unsigned short h;
  asm("cvt.rn.bf16.f32 %0, %1;" : "=h"(h) : "f"(x));
  static_cast<uint16_t *>(const_cast<void *>(p))[i] = h;
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, bool real) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(real ? 16 : 0) : "memory");
}

template <int V>
__device__ __forceinline__ void ldv(float (&x)[V], const float *p) {
  if constexpr (V == 4) {
    const float4 f = *reinterpret_cast<const float4 *>(p);
    x[0] = f.x, x[1] = f.y, x[2] = f.z, x[3] = f.w;
  } else {
    x[0] = *p;
  }
}
template <int V>
__device__ __forceinline__ void stv(float *p, const float (&x)[V]) {
  if constexpr (V == 4) *reinterpret_cast<float4 *>(p) = make_float4(x[0], x[1], x[2], x[3]);
  else *p = x[0];
}

// Batches of 8 positions are taken relative to their start unless lam^8 is
// below 2^-16.
constexpr int kBatch = 8;
constexpr float kSlowest = -16.f * 0.69314718f / kBatch;

// One pass of the recurrence over a segment of a head (blockIdx.x: head and
// segment, blockIdx.y: pass, blockIdx.z: 32 nwy columns).  OUT: outputs, from
// the segment's start state; otherwise the segment's sum alone, from zero.
// VEC: float32 in 16-byte pieces, fetched one batch ahead.  168 registers let
// three warps share a scheduler.
template <typename E, int TX, int NX, bool OUT, bool VEC>
__global__ void __maxnreg__(168) rec_kernel(const __grid_constant__ Group g, int nwy) {
  const Pass &p = g.p[blockIdx.y];
  extern __shared__ __align__(16) float rec_smem[];
  constexpr int QX = TX / 4;  // a lane's float4s of rows, 16 rows apart
  constexpr int XS = 4 * TX * NX;
  const int YS = 32 * nwy;
  constexpr int NBUF = VEC ? 2 : 1;
  float *sb = rec_smem, *sc = sb + NBUF * kTB * XS, *sa = sc + NBUF * kTB * YS;  // sa, so: OUT only
  float *so = sa + NBUF * kTB * XS;                                           // [NX][kTB][YS]
  __shared__ __align__(16) float wk[kBatch], uk[kBatch];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, wx = warp % NX;
  const int rg = lane >> 3, x0 = 4 * TX * wx + 4 * rg, yl = 32 * (warp / NX) + 4 * (lane & 7);
  const int yt = blockIdx.z * YS, y0 = yt + yl;  // the block's first column, this lane's
  const int64_t bh = blockIdx.x / p.nseg, sg = blockIdx.x % p.nseg;
  const bool last = sg == (p.reverse ? 0 : p.nseg - 1);  // of the pass's segments
  if (!OUT && last) return;                              // no state starts from its sum
  const int64_t b = bh / p.H, h = bh % p.H;
  const int64_t n = row_len(p, b);
  const int64_t t0 = sg * p.seg_len, tz = min(t0 + p.seg_len, p.T), t1 = max(t0, min(tz, n));
  const float gd = p.log_decay[h];
  const bool slow = !(gd >= kSlowest);
  const E *pa = static_cast<const E *>(p.a.p) + (b * p.a.sb + h * p.a.sh),
          *pb = static_cast<const E *>(p.b.p) + (b * p.b.sb + h * p.b.sh),
          *pc = static_cast<const E *>(p.c.p) + (b * p.c.sb + h * p.c.sh);
  E *po = static_cast<E *>(const_cast<void *>(p.o.p)) + (b * p.o.sb + h * p.o.sh);
  const int64_t XY = (int64_t)p.X * p.Y;
  const int64_t count = t1 - t0, step = p.reverse ? -1 : 1;
  const int64_t t_first = p.reverse ? t1 - 1 : t0;  // row i of the segment is position t_first + step i

  if (tid < kBatch) {  // reverse: the state handed in meets the first position undecayed
    const float e = slow ? 0.f : gd * (float)(tid + (p.reverse ? 0 : 1));
    wk[tid] = p.sk * expf(-e);
    uk[tid] = p.si * expf(e);
  }

  // rows 16 q + x0 + (0..3), as two pairs each
  f2 S[2 * QX][4];
  const float *s0 = !OUT ? nullptr : p.nseg > 1 ? p.seg + blockIdx.x * XY : p.s_in ? p.s_in + bh * XY : nullptr;
  const bool s0_t = p.nseg == 1 && p.s_in_t;
#pragma unroll
  for (int r = 0; r < 2 * QX; ++r) {
    float v[2][4];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int x = x0 + 16 * (r >> 1) + 2 * (r & 1) + i;
      if (s0 && !s0_t && (p.Y & 3) == 0 && x < p.X && y0 < p.Y) {
        const float4 f = __ldcs(reinterpret_cast<const float4 *>(s0 + (int64_t)x * p.Y + y0));
        v[i][0] = f.x, v[i][1] = f.y, v[i][2] = f.z, v[i][3] = f.w;
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          v[i][e] = s0 && x < p.X && y0 + e < p.Y ? s0[s0_t ? (int64_t)(y0 + e) * p.X + x : (int64_t)x * p.Y + y0 + e] : 0.f;
      }
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) S[r][e] = pair(v[0][e], v[1][e]);
  }
  auto decay = [&](Decay d) {
    const f2 m = both(d.m);
    if (d.near_one) {
#pragma unroll
      for (int r = 0; r < 2 * QX; ++r)
#pragma unroll
        for (int e = 0; e < 4; ++e) S[r][e] = fma2(S[r][e], m, S[r][e]);
    } else {
#pragma unroll
      for (int r = 0; r < 2 * QX; ++r)
#pragma unroll
        for (int e = 0; e < 4; ++e) S[r][e] = mul2(S[r][e], m);
    }
  };
  const Decay lam = decay_of(gd, 1), lam_batch = decay_of(gd, kBatch);

  // rows s.. of the segment (m of them) into buffer `buf`.  A thread's pieces
  // of a and b are one column's, every rx-th row; of c every ry-th.
  constexpr int ux = XS / 4;
  const int uy = YS / 4, rx = blockDim.x / ux, ry = blockDim.x / uy;
  const int ix = tid / ux, px = 4 * (tid % ux), iy = tid / uy, py = 4 * (tid % uy);
  auto fetch = [&](int64_t s, int m, int buf) {
    float *db = sb + buf * kTB * XS, *dc = sc + buf * kTB * YS, *da = sa + buf * kTB * XS;
    const int64_t t = t_first + step * s;
    if constexpr (VEC) {
      const bool xr = px < p.X, yr = yt + py < p.Y;
      const E *fb = pb + (t + step * ix) * p.b.st + (xr ? px : 0), *fa = OUT ? pa + (t + step * ix) * p.a.st + (xr ? px : 0) : nullptr;
      const int64_t jb = step * rx * p.b.st, ja = step * rx * p.a.st;
      uint32_t ub = smem_addr(db + 4 * tid), ua = smem_addr(da + 4 * tid);
      for (int i = ix; i < m; i += rx, fb += jb, ub += 16 * blockDim.x) {
        cp_async16(ub, fb, xr);
        if (OUT) cp_async16(ua, fa, xr), fa += ja, ua += 16 * blockDim.x;
      }
      const E *fc = pc + (t + step * iy) * p.c.st + (yr ? yt + py : 0);
      const int64_t jc = step * ry * p.c.st;
      uint32_t uc = smem_addr(dc + 4 * tid);
      for (int i = iy; i < m; i += ry, fc += jc, uc += 16 * blockDim.x) cp_async16(uc, fc, yr);
    } else {
      for (int e = tid; e < m * XS; e += blockDim.x) {
        const int i = e / XS, x = e % XS;
        db[e] = x < p.X ? load1<E>(pb, (t + step * i) * p.b.st + x) : 0.f;
        if (OUT) da[e] = x < p.X ? load1<E>(pa, (t + step * i) * p.a.st + x) : 0.f;
      }
      for (int e = tid; e < m * YS; e += blockDim.x) {
        const int i = e / YS, y = yt + e % YS;
        dc[e] = y < p.Y ? load1<E>(pc, (t + step * i) * p.c.st + y) : 0.f;
      }
    }
  };

  int buf = 0;
  if (VEC && count > 0) {
    fetch(0, (int)min((int64_t)kTB, count), 0);
    asm volatile("cp.async.commit_group;" ::: "memory");
  }
  for (int64_t s = 0; s < count; s += kTB) {
    const int m = (int)min((int64_t)kTB, count - s);
    if constexpr (VEC) {
      if (s + kTB < count) fetch(s + kTB, (int)min((int64_t)kTB, count - s - kTB), buf ^ 1);
      asm volatile("cp.async.commit_group;" ::: "memory");
      asm volatile("cp.async.wait_group 1;" ::: "memory");
    } else {
      fetch(s, m, 0);
    }
    __syncthreads();
    const float *cb = sb + buf * kTB * XS + x0, *cc = sc + buf * kTB * YS + yl, *ca = sa + buf * kTB * XS + x0;
    // Four positions from i0; PLAIN: all of them there, and no decay between them.
    auto four = [&](int i0, auto plain) {
      constexpr bool PLAIN = decltype(plain)::value;
      f2 y[4][4];
      const float4 w4 = *reinterpret_cast<const float4 *>(wk + (i0 & (kBatch - 1)));
      const float w[4] = {w4.x, w4.y, w4.z, w4.w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
#pragma unroll
        for (int e = 0; e < 4; ++e) y[k][e] = 0ull;
        const int i = i0 + k;
        if (!PLAIN && i >= m) continue;
        if (!PLAIN && slow && !p.reverse) decay(lam);
        const float4 cv = *reinterpret_cast<const float4 *>(cc + i * YS);
        const f2 c[4] = {both(cv.x * w[k]), both(cv.y * w[k]), both(cv.z * w[k]), both(cv.w * w[k])};
#pragma unroll
        for (int q = 0; q < QX; ++q) {
          const ulonglong2 bv = *reinterpret_cast<const ulonglong2 *>(cb + i * XS + 16 * q);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            S[2 * q][e] = fma2(bv.x, c[e], S[2 * q][e]);
            S[2 * q + 1][e] = fma2(bv.y, c[e], S[2 * q + 1][e]);
          }
          if (OUT) {
            const ulonglong2 av = *reinterpret_cast<const ulonglong2 *>(ca + i * XS + 16 * q);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              y[k][e] = fma2(av.x, S[2 * q][e], y[k][e]);
              y[k][e] = fma2(av.y, S[2 * q + 1][e], y[k][e]);
            }
          }
        }
        if (!PLAIN && slow && p.reverse) decay(lam);
      }
      if (OUT) {
        // 16 sums over the lanes rg = 0..3: lane rg ends with those of position i0 + rg
        float z[8], o[4];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float2 lo = unpair(y[e >> 2][e & 3]), hi = unpair(y[2 + (e >> 2)][e & 3]);
          const float l = lo.x + lo.y, u = hi.x + hi.y;
          z[e] = (rg & 2 ? u : l) + __shfl_xor_sync(~0u, rg & 2 ? l : u, 16);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e)
          o[e] = (rg & 1 ? z[4 + e] : z[e]) + __shfl_xor_sync(~0u, rg & 1 ? z[e] : z[4 + e], 8);
        const float u = uk[(i0 + rg) & (kBatch - 1)];
        *reinterpret_cast<float4 *>(so + (wx * kTB + i0 + rg) * YS + yl) = make_float4(u * o[0], u * o[1], u * o[2], u * o[3]);
      }
    };
    if (slow) {
#pragma unroll 1
      for (int i0 = 0; i0 < m; i0 += 4) four(i0, std::false_type());
    } else {
      const int full = m & ~3;
#pragma unroll 1
      for (int i0 = 0; i0 < full; i0 += 4) {
        four(i0, std::true_type());
        if (i0 & 4) decay(lam_batch);
      }
      if (full < m) four(full, std::false_type());
      if (m & (kBatch - 1)) decay(decay_of(gd, m & (kBatch - 1)));
    }
    __syncthreads();
    if (OUT) {
      const int64_t t = t_first + step * s;
      if constexpr (VEC) {
        float *fo = po + (t + step * iy) * p.o.st + yt + py;
        const int64_t jo = step * ry * p.o.st;
        const float *uo = so + 4 * tid;
        if (yt + py < p.Y)
          for (int i = iy; i < m; i += ry, fo += jo, uo += 4 * blockDim.x) {
            float4 v = *reinterpret_cast<const float4 *>(uo);
            if (NX == 2) {
              const float4 u = *reinterpret_cast<const float4 *>(uo + kTB * YS);
              v.x += u.x, v.y += u.y, v.z += u.z, v.w += u.w;
            }
            *reinterpret_cast<float4 *>(fo) = v;
          }
      } else {
        for (int e = tid; e < m * YS; e += blockDim.x) {
          const int i = e / YS, y = yt + e % YS;
          if (y < p.Y) store1<E>(po, (t + step * i) * p.o.st + y, NX == 2 ? so[e] + so[kTB * YS + e] : so[e]);
        }
      }
    }
    buf ^= VEC ? 1 : 0;
  }
  float *dst = !OUT ? p.seg + blockIdx.x * XY : last && p.s_out ? p.s_out + bh * XY : nullptr;
  if (dst) {
#pragma unroll
    for (int r = 0; r < 2 * QX; ++r) {
      float2 v[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = unpair(S[r][e]);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int x = x0 + 16 * (r >> 1) + 2 * (r & 1) + i;
        if (x >= p.X) continue;
        float *d = dst + (int64_t)x * p.Y + y0;
        const float f[4] = {i ? v[0].y : v[0].x, i ? v[1].y : v[1].x, i ? v[2].y : v[2].x, i ? v[3].y : v[3].x};
        if ((p.Y & 3) == 0 && y0 < p.Y) {
          *reinterpret_cast<float4 *>(d) = make_float4(f[0], f[1], f[2], f[3]);
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (y0 + e < p.Y) d[e] = f[e];
        }
      }
    }
  }
  if (OUT)
    for (int64_t t = t1; t < tz; ++t)  // padding
      for (int y = yt + tid; y < min(p.Y, yt + YS); y += blockDim.x) store1<E>(po, t * p.o.st + y, 0.f);
}

// Joins the segments of every head in time order (or reverse): p.seg holds
// the segments' sums and receives the states at their starts.  blockIdx.y is the
// head, blockIdx.z the pass; V state elements per thread.  Eight segments' loads
// are in flight at a time, and the sum goes through them in order.
template <int V>
__global__ void __launch_bounds__(256) decay_scan_kernel(const __grid_constant__ Group g) {
  const Pass &p = g.p[blockIdx.z];
  const int XY = p.X * p.Y, f = ((int)blockIdx.x * 256 + (int)threadIdx.x) * V;
  if (f >= XY) return;
  const int64_t bh = blockIdx.y;
  const int64_t n = row_len(p, bh / p.H);
  const float gd = p.log_decay[bh % p.H];
  const Decay whole = decay_of(gd, p.seg_len);
  float run[V] = {};
  if (p.s_in) {
    const float *s = p.s_in + bh * XY;
    if (!p.s_in_t) ldv(run, s + f);
    else {
#pragma unroll
      for (int i = 0; i < V; ++i) run[i] = s[(f + i) % p.Y * p.X + (f + i) / p.Y];
    }
  }
  float *base = p.seg + bh * p.nseg * XY + f;
  constexpr int kAhead = 8;
  for (int s0 = 0; s0 < p.nseg; s0 += kAhead) {
    float v[kAhead][V] = {};
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int s = p.reverse ? p.nseg - 1 - (s0 + i) : s0 + i;
      if (s0 + i < p.nseg - 1) ldv(v[i], base + (int64_t)s * XY);
    }
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      if (s0 + i < p.nseg) {
        const int s = p.reverse ? p.nseg - 1 - (s0 + i) : s0 + i;
        const int64_t len = max((int64_t)0, min(p.seg_len, n - s * p.seg_len));
        stv(base + (int64_t)s * XY, run);
        const Decay d = len == p.seg_len ? whole : decay_of(gd, len);
#pragma unroll
        for (int e = 0; e < V; ++e) run[e] = decayed(run[e], d) + v[i][e];
      }
    }
  }
}

// Sum over the 8 lanes of equal lane % 4 of four columns each: afterwards a
// lane holds column 4 (lane % 4) + 2 bit4 + bit3 (twice, over bit 2).
__device__ __forceinline__ float reduce_columns(const float (&y)[4], int lane) {
  const bool h4 = lane & 16, h3 = lane & 8;
  const float r0 = __shfl_xor_sync(~0u, h4 ? y[0] : y[2], 16), r1 = __shfl_xor_sync(~0u, h4 ? y[1] : y[3], 16);
  const float k0 = (h4 ? y[2] : y[0]) + r0, k1 = (h4 ? y[3] : y[1]) + r1;
  const float r2 = __shfl_xor_sync(~0u, h3 ? k0 : k1, 8);
  const float z = (h3 ? k1 : k0) + r2;
  return z + __shfl_xor_sync(~0u, z, 4);
}
__device__ __forceinline__ int reduced_column(int lane) {
  return 4 * (lane & 3) + ((lane & 16) ? 2 : 0) + ((lane & 8) ? 1 : 0);
}

// A lane's RX x 4 part of a state of X x Y at `s`.
template <int RX>
__device__ __forceinline__ void load_state(float (&S)[RX][4], const float *s, int X, int Y, int x0, int y0) {
  const bool vec = (Y & 3) == 0;
#pragma unroll
  for (int r = 0; r < RX; ++r) {
    const int x = x0 + r;
    if (vec && x < X && y0 < Y) {
      const float4 v = __ldcs(reinterpret_cast<const float4 *>(s + (int64_t)x * Y + y0));
      S[r][0] = v.x, S[r][1] = v.y, S[r][2] = v.z, S[r][3] = v.w;
    } else {
#pragma unroll
      for (int q = 0; q < 4; ++q)
        S[r][q] = (x < X && y0 + q < Y) ? s[(int64_t)x * Y + y0 + q] : 0.f;
    }
  }
}
template <int RX>
__device__ __forceinline__ void store_state(const float (&S)[RX][4], float *s, int X, int Y, int x0, int y0) {
  const bool vec = (Y & 3) == 0;
#pragma unroll
  for (int r = 0; r < RX; ++r) {
    const int x = x0 + r;
    if (x >= X) continue;
    if (vec && y0 < Y) {
      __stcs(reinterpret_cast<float4 *>(s + (int64_t)x * Y + y0), make_float4(S[r][0], S[r][1], S[r][2], S[r][3]));
    } else {
#pragma unroll
      for (int q = 0; q < 4; ++q)
        if (y0 + q < Y) s[(int64_t)x * Y + y0 + q] = S[r][q];
    }
  }
}

// One token: the state read once and written once, 8 N H D M bytes, which is
// all there is to it (a few FMAs per 8 bytes).  A block is one sequence and
// head, a warp 16 columns; each lane has its RX float4s of state in flight
// before anything else.  Three blocks on an SM keep HBM busy while one stores:
// 512 x 40 heads of 128 x 128 take 447 us (6.1 TB/s), with two blocks 540.
template <typename E, int RX>
__global__ void __launch_bounds__(32 * kStepWarps, 3) decay_step_kernel(StepArgs s) {
  constexpr int XP = 8 * RX;
  __shared__ __align__(16) float sv[16 * kStepWarps];  // read four at a time
  __shared__ float sq[XP], sk[XP];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int x0 = (lane >> 2) * RX, y0 = 16 * warp + 4 * (lane & 3);
  const int64_t nh = blockIdx.x, n = nh / s.H, h = nh % s.H;
  const int64_t DM = (int64_t)s.D * s.M;
  float S[RX][4];
  load_state<RX>(S, s.s_in + nh * DM, s.D, s.M, x0, y0);
  const Decay lam = decay_of(s.log_decay[h], 1);
  for (int x = threadIdx.x; x < XP; x += blockDim.x) {
    sq[x] = x < s.D ? load1<E>(s.q.p, n * s.q.sb + h * s.q.sh + x) : 0.f;
    sk[x] = x < s.D ? load1<E>(s.k.p, n * s.k.sb + h * s.k.sh + x) : 0.f;
  }
  for (int y = threadIdx.x; y < 16 * (int)(blockDim.x >> 5); y += blockDim.x)
    sv[y] = y < s.M ? load1<E>(s.v.p, n * s.v.sb + h * s.v.sh + y) : 0.f;
  __syncthreads();
  const float4 c = *reinterpret_cast<const float4 *>(sv + y0);
  float y[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int r = 0; r < RX; ++r) {
    const float kr = sk[x0 + r], qr = sq[x0 + r];
    S[r][0] = fmaf(kr, c.x, decayed(S[r][0], lam));
    S[r][1] = fmaf(kr, c.y, decayed(S[r][1], lam));
    S[r][2] = fmaf(kr, c.z, decayed(S[r][2], lam));
    S[r][3] = fmaf(kr, c.w, decayed(S[r][3], lam));
#pragma unroll
    for (int q = 0; q < 4; ++q) y[q] = fmaf(qr, S[r][q], y[q]);
  }
  store_state<RX>(S, s.s_out + nh * DM, s.D, s.M, x0, y0);
  const float z = reduce_columns(y, lane);
  const int yc = 16 * warp + reduced_column(lane);
  if (!(lane & 4) && yc < s.M) store1<E>(s.o.p, n * s.o.sb + h * s.o.sh + yc, s.scale * z);
}

namespace {
// Warps of 32 columns in a block; 128 columns are two blocks of two, so that
// 12 warps fit an SM with two warps of rows as well.
int rec_warps_y(int Y) { return Y > 96 ? 2 : (Y + 31) / 32; }
template <typename E, int TX, int NX, bool VEC>
cudaError_t rec_t(const Group &g, int nwy, int ytiles, bool sums_only, cudaStream_t st) {
  const Pass &p = g.p[0];
  const dim3 grid((unsigned)(p.B * p.H * p.nseg), (unsigned)g.n, (unsigned)ytiles), block(32 * NX * nwy);
  const size_t rows = sizeof(float) * (VEC ? 2 : 1) * kTB * 4 * TX * NX, cols = sizeof(float) * kTB * 32 * nwy;
  const size_t smem = sums_only ? rows + (VEC ? 2 : 1) * cols : 2 * rows + (VEC ? 2 : 1) * cols + NX * cols;
  const auto kern = sums_only ? rec_kernel<E, TX, NX, false, VEC> : rec_kernel<E, TX, NX, true, VEC>;
  int blocks = 0;  // raises the kernel's shared-memory limit
  const cudaError_t e = blocks_per_sm((const void *)kern, (int)block.x, (int)smem, &blocks);
  return e == cudaSuccess ? launch_kernel(kern, grid, block, smem, st, g, nwy) : e;
}
bool pieces16(const View &v, const Pass &p) {
  auto fits = [](int64_t s, int64_t n) { return n <= 1 || s % 4 == 0; };
  return ((uintptr_t)v.p & 15u) == 0 && fits(v.sb, p.B) && fits(v.st, p.T) && fits(v.sh, p.H);
}
template <typename E, bool VEC>
cudaError_t rec_v(const Group &g, bool sums_only, cudaStream_t st) {
  int y = 0;
  for (int i = 0; i < g.n; ++i) y = std::max(y, g.p[i].Y);
  const int nwy = rec_warps_y(y), tiles = (y + 32 * nwy - 1) / (32 * nwy), cls = rec_class(g.p[0].X);
  return cls == 0   ? rec_t<E, 8, 1, VEC>(g, nwy, tiles, sums_only, st)
         : cls == 1 ? rec_t<E, 16, 1, VEC>(g, nwy, tiles, sums_only, st)
                    : rec_t<E, 16, 2, VEC>(g, nwy, tiles, sums_only, st);
}
template <typename E>
cudaError_t step_e(const StepArgs &s, cudaStream_t st) {
  const dim3 grid((unsigned)(s.N * s.H)), block(32 * ((s.M + 15) / 16));
  return s.D <= 32   ? launch_kernel(decay_step_kernel<E, 4>, grid, block, 0, st, s)
         : s.D <= 64 ? launch_kernel(decay_step_kernel<E, 8>, grid, block, 0, st, s)
                     : launch_kernel(decay_step_kernel<E, 16>, grid, block, 0, st, s);
}
}  // namespace

// Rows in one warp (32 or 64), or two warps of 64.
int rec_class(int X) { return X <= 32 ? 0 : X <= 64 ? 1 : 2; }
int64_t rec_segments(int64_t BH, int64_t T, int X, int Y, int npass, int sms) {
  // In cycles, measured: a position takes a warp of 64 rows about 290 of its
  // scheduler's, and at least 330 from one to the next; 12 warps fit an SM at
  // a time.  A head in several segments costs its sums (half of that again),
  // the scan and a launch more.  (8 x 1024 x 12 heads of 64: forward 174 us in
  // one segment, 86 in the 6 that this gives, 87 with states in and out;
  // backward 175 us in the one that it gives, 224 in 2.)
  const int64_t warps = npass * BH * ((Y + 31) / 32) * (X <= 64 ? 1 : 2);
  const double each = X <= 32 ? 160. : 290., chain = X <= 32 ? 220. : 330.;
  int64_t best = 1;
  double least = 1e300;
  for (int64_t n = 1; n <= std::max<int64_t>(1, std::min<int64_t>(T / 32, 12 * sms)); ++n) {
    const int64_t len = (T + n - 1) / n, per_sm = (warps * n + sms - 1) / sms;
    if (n > 1 && (T + len - 1) / len != n) continue;
    const double full = (double)(per_sm / 12), rest = (double)((per_sm % 12 + 3) / 4);
    const double pos = full * std::max(chain, 3 * each) + (rest > 0 ? std::max(chain, rest * each) : 0.);
    const double t = (n > 1 ? 1.5 : 1.) * pos * (double)len + (n > 1 ? 15000. + 400. * (double)n : 0.);
    if (t < least) least = t, best = n;
    if (per_sm > 48) break;
  }
  return best;
}
cudaError_t launch_rec(const Group &g, int dtype, bool sums_only, cudaStream_t st) {
  if (dtype != 0) return rec_v<uint16_t, false>(g, sums_only, st);
  bool vec = true;
  for (int i = 0; i < g.n; ++i) {
    const Pass &p = g.p[i];
    vec = vec && p.X % 4 == 0 && p.Y % 4 == 0 && pieces16(p.a, p) && pieces16(p.b, p) && pieces16(p.c, p) && pieces16(p.o, p);
  }
  return vec ? rec_v<float, true>(g, sums_only, st) : rec_v<float, false>(g, sums_only, st);
}
cudaError_t launch_scan(const Group &g, cudaStream_t st) {
  const Pass &p = g.p[0];
  const int n = p.X * p.Y, v = n % 4 == 0 ? 4 : 1;
  const dim3 grid((unsigned)((n / v + 255) / 256), (unsigned)(p.B * p.H), (unsigned)g.n);
  return v == 4 ? launch_kernel(decay_scan_kernel<4>, grid, dim3(256), 0, st, g)
                : launch_kernel(decay_scan_kernel<1>, grid, dim3(256), 0, st, g);
}
cudaError_t launch_step(const StepArgs &s, int dtype, cudaStream_t st) {
  return dtype == 0 ? step_e<float>(s, st) : step_e<uint16_t>(s, st);
}

}  // namespace decay
}  // namespace wkv
