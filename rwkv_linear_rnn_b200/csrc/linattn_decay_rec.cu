// linattn_decay_rec.cu -- linear attention with a decay for each head on the
// CUDA cores: the recurrence itself, the single-token step, and the scan that
// joins the segments of a long sequence.
//
// The recurrence R_t = lam R_{t-1} + b_t c_t^T, o_t = a_t^T R_t costs three
// FMAs per state element and position (the two of the update, one of the
// product), so it is bound by the FMA pipes: it serves float32 tensors (which
// the tensor cores' bfloat16 products would round), heads and strides that
// TMA cannot describe, and sequences of a few positions.
//
// Layout: a warp owns 16 columns of Y and all rows of X; lane (xl, yl) =
// (lane / 4, lane % 4) holds rows xl * RX .. + RX - 1 of columns
// 4 yl .. + 3, so a state row is read as 64-byte segments, a and b come from
// shared memory as broadcast float4s, and the product needs one reduction
// over the 8 lanes that share columns: 4 shuffles and no block barrier.
#include <algorithm>

#include "linattn_decay.cuh"

namespace wkv {
namespace decay {

constexpr int kTB = 16;     // positions staged in shared memory at a time
constexpr int kRecWarps = 8;  // most warps per block: 128 columns of Y

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

// A lane's RX x 4 part of a state of X x Y at `s` (or Y x X, transposed).
template <int RX>
__device__ __forceinline__ void load_state(float (&S)[RX][4], const float *s, int X, int Y, int x0, int y0,
                                           bool transposed) {
  const bool vec = !transposed && (Y & 3) == 0;
#pragma unroll
  for (int r = 0; r < RX; ++r) {
    const int x = x0 + r;
    if (vec && x < X && y0 < Y) {
      const float4 v = __ldcs(reinterpret_cast<const float4 *>(s + (int64_t)x * Y + y0));
      S[r][0] = v.x, S[r][1] = v.y, S[r][2] = v.z, S[r][3] = v.w;
    } else {
#pragma unroll
      for (int q = 0; q < 4; ++q)
        S[r][q] = (x < X && y0 + q < Y) ? s[transposed ? (int64_t)(y0 + q) * X + x : (int64_t)x * Y + y0 + q] : 0.f;
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

// One pass of the recurrence over a segment of a head (blockIdx.x: head and
// segment, blockIdx.y: 16 columns per warp).  OUT: outputs, from the
// segment's start state; otherwise the segment's sum alone, from zero.
template <typename E, int RX, bool OUT>
__global__ void __launch_bounds__(32 * kRecWarps) rec_kernel(Pass p) {
  constexpr int XP = 8 * RX;
  extern __shared__ float rec_smem[];
  const int nw = blockDim.x >> 5, YB = 16 * nw;
  float *sb = rec_smem, *sc = sb + kTB * XP, *sa = sc + kTB * YB, *so = sa + kTB * XP;  // sa, so: OUT only
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int x0 = (lane >> 2) * RX, yw = 16 * warp + 4 * (lane & 3), yb = blockIdx.y * YB;
  const int64_t bh = blockIdx.x / p.nseg, sg = blockIdx.x % p.nseg;
  const int64_t b = bh / p.H, h = bh % p.H;
  const int64_t n = row_len(p, b);
  const int64_t t0 = sg * p.seg_len, tz = min(t0 + p.seg_len, p.T), t1 = max(t0, min(tz, n));
  const Decay lam = decay_of(p.log_decay[h], 1);
  const int64_t oa = b * p.a.sb + h * p.a.sh, ob = b * p.b.sb + h * p.b.sh, oc = b * p.c.sb + h * p.c.sh,
                oo = b * p.o.sb + h * p.o.sh;
  const int64_t XY = (int64_t)p.X * p.Y;

  float S[RX][4];
  const float *s0 = !OUT ? nullptr : p.nseg > 1 ? p.seg + blockIdx.x * XY : p.s_in ? p.s_in + bh * XY : nullptr;
  if (s0) {
    load_state<RX>(S, s0, p.X, p.Y, x0, yb + yw, p.nseg == 1 && p.s_in_t);
  } else {
#pragma unroll
    for (int r = 0; r < RX; ++r) S[r][0] = S[r][1] = S[r][2] = S[r][3] = 0.f;
  }

  const int64_t count = t1 - t0;
  for (int64_t s = 0; s < count; s += kTB) {
    const int m = (int)min((int64_t)kTB, count - s);
    // row i of this batch is position t0 + s + i, or t1 - 1 - s - i in reverse
    const int64_t first = p.reverse ? t1 - 1 - s : t0 + s;
    const int64_t step = p.reverse ? -1 : 1;
    __syncthreads();
    for (int e = threadIdx.x; e < m * XP; e += blockDim.x) {
      const int i = e / XP, x = e % XP;
      const int64_t t = first + step * i;
      sb[e] = x < p.X ? p.sk * load1<E>(p.b.p, ob + t * p.b.st + x) : 0.f;
      if (OUT) sa[e] = x < p.X ? load1<E>(p.a.p, oa + t * p.a.st + x) : 0.f;
    }
    for (int e = threadIdx.x; e < m * YB; e += blockDim.x) {
      const int i = e / YB, y = yb + e % YB;
      sc[e] = y < p.Y ? load1<E>(p.c.p, oc + (first + step * i) * p.c.st + y) : 0.f;
    }
    __syncthreads();
    for (int i = 0; i < m; ++i) {
      // reverse: the state handed in is not decayed before the first position
      const Decay f = p.reverse && s + i == 0 ? Decay{0.f, true} : lam;
      const float4 c = *reinterpret_cast<const float4 *>(sc + i * YB + yw);
      float y[4] = {0.f, 0.f, 0.f, 0.f};
      auto token = [&](auto decay1) {
#pragma unroll
        for (int r4 = 0; r4 < RX; r4 += 4) {
          const float4 bv = *reinterpret_cast<const float4 *>(sb + i * XP + x0 + r4);
          float4 av = make_float4(0.f, 0.f, 0.f, 0.f);
          if (OUT) av = *reinterpret_cast<const float4 *>(sa + i * XP + x0 + r4);
          const float br[4] = {bv.x, bv.y, bv.z, bv.w}, ar[4] = {av.x, av.y, av.z, av.w}, cr[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
          for (int q = 0; q < 4; ++q) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              float &R = S[r4 + q][e];
              R = fmaf(br[q], cr[e], decay1(R));
              if (OUT) y[e] = fmaf(ar[q], R, y[e]);
            }
          }
        }
      };
      if (f.near_one)  // one branch per position instead of a select per element
        token([&](float x) { return fmaf(x, f.m, x); });
      else
        token([&](float x) { return x * f.m; });
      if (OUT) {
        const float z = reduce_columns(y, lane);
        if (!(lane & 4)) so[i * YB + 16 * warp + reduced_column(lane)] = p.si * z;
      }
    }
    if (OUT) {
      __syncthreads();
      for (int e = threadIdx.x; e < m * YB; e += blockDim.x) {
        const int i = e / YB, y = yb + e % YB;
        if (y < p.Y) store1<E>(p.o.p, oo + (first + step * i) * p.o.st + y, so[e]);
      }
    }
  }
  if (p.reverse && count > 0) {
#pragma unroll
    for (int r = 0; r < RX; ++r)
#pragma unroll
      for (int q = 0; q < 4; ++q) S[r][q] = decayed(S[r][q], lam);
  }
  if (!OUT) {
    store_state<RX>(S, p.seg + blockIdx.x * XY, p.X, p.Y, x0, yb + yw);
  } else {
    if (p.nseg == 1 && p.s_out) store_state<RX>(S, p.s_out + bh * XY, p.X, p.Y, x0, yb + yw);
    for (int64_t t = t1; t < tz; ++t)  // padding
      for (int y = yb + threadIdx.x; y < min(p.Y, yb + YB); y += blockDim.x) store1<E>(p.o.p, oo + t * p.o.st + y, 0.f);
  }
}

// Joins the segments of every head in time order (or reverse): p.seg holds
// the segments' sums and receives the states at their starts; the state after
// the last one goes to s_out.  One thread per state element; eight segments'
// loads are in flight at a time, and the sum goes through them in order.
__global__ void __launch_bounds__(256) decay_scan_kernel(Pass p) {
  const int64_t XY = (int64_t)p.X * p.Y;
  const int64_t e = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  if (e >= p.B * p.H * XY) return;
  const int64_t bh = e / XY;
  const int f = (int)(e % XY);
  const int64_t n = row_len(p, bh / p.H);
  const float g = p.log_decay[bh % p.H];
  float run = 0.f;
  if (p.s_in) {
    const int x = f / p.Y, y = f % p.Y;
    run = p.s_in[bh * XY + (p.s_in_t ? y * p.X + x : f)];
  }
  float *base = p.seg + bh * p.nseg * XY + f;
  constexpr int kBatch = 8;
  for (int s0 = 0; s0 < p.nseg; s0 += kBatch) {
    float v[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int s = p.reverse ? p.nseg - 1 - (s0 + i) : s0 + i;
      v[i] = s0 + i < p.nseg ? base[s * XY] : 0.f;
    }
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      if (s0 + i < p.nseg) {
        const int s = p.reverse ? p.nseg - 1 - (s0 + i) : s0 + i;
        const int64_t len = max((int64_t)0, min(p.seg_len, n - s * p.seg_len));
        base[s * XY] = run;
        run = decayed(run, decay_of(g, len)) + v[i];
      }
    }
  }
  if (p.s_out) p.s_out[bh * XY + f] = run;
}

// One token: the state read once and written once, 8 N H D M bytes, which is
// all there is to it (a few FMAs per 8 bytes).  A block is one sequence and
// head, a warp 16 columns; each lane has its RX float4s of state in flight
// before anything else.
template <typename E, int RX>
__global__ void __launch_bounds__(32 * kRecWarps) decay_step_kernel(StepArgs s) {
  constexpr int XP = 8 * RX;
  __shared__ float sq[XP], sk[XP], sv[16 * kRecWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int x0 = (lane >> 2) * RX, y0 = 16 * warp + 4 * (lane & 3);
  const int64_t nh = blockIdx.x, n = nh / s.H, h = nh % s.H;
  const int64_t DM = (int64_t)s.D * s.M;
  float S[RX][4];
  load_state<RX>(S, s.s_in + nh * DM, s.D, s.M, x0, y0, false);
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
template <typename E, int RX>
cudaError_t rec_t(const Pass &p, bool sums_only, cudaStream_t st) {
  const int nw = std::min(kRecWarps, (p.Y + 15) / 16);
  const dim3 grid((unsigned)(p.B * p.H * p.nseg), (unsigned)((p.Y + 16 * nw - 1) / (16 * nw)));
  const size_t half = sizeof(float) * kTB * (8 * RX + 16 * nw);
  return sums_only ? launch_kernel(rec_kernel<E, RX, false>, grid, dim3(32 * nw), half, st, p)
                   : launch_kernel(rec_kernel<E, RX, true>, grid, dim3(32 * nw), 2 * half, st, p);
}
template <typename E>
cudaError_t rec_e(const Pass &p, bool sums_only, cudaStream_t st) {
  return p.X <= 32   ? rec_t<E, 4>(p, sums_only, st)
         : p.X <= 64 ? rec_t<E, 8>(p, sums_only, st)
                     : rec_t<E, 16>(p, sums_only, st);
}
template <typename E>
cudaError_t step_e(const StepArgs &s, cudaStream_t st) {
  const dim3 grid((unsigned)(s.N * s.H)), block(32 * ((s.M + 15) / 16));
  return s.D <= 32   ? launch_kernel(decay_step_kernel<E, 4>, grid, block, 0, st, s)
         : s.D <= 64 ? launch_kernel(decay_step_kernel<E, 8>, grid, block, 0, st, s)
                     : launch_kernel(decay_step_kernel<E, 16>, grid, block, 0, st, s);
}
}  // namespace

cudaError_t launch_rec(const Pass &p, int dtype, bool sums_only, cudaStream_t st) {
  return dtype == 0 ? rec_e<float>(p, sums_only, st) : rec_e<uint16_t>(p, sums_only, st);
}
cudaError_t launch_scan(const Pass &p, cudaStream_t st) {
  const int64_t n = p.B * p.H * p.X * p.Y;
  return launch_kernel(decay_scan_kernel, dim3((unsigned)((n + 255) / 256)), dim3(256), 0, st, p);
}
cudaError_t launch_step(const StepArgs &s, int dtype, cudaStream_t st) {
  return dtype == 0 ? step_e<float>(s, st) : step_e<uint16_t>(s, st);
}

}  // namespace decay
}  // namespace wkv
