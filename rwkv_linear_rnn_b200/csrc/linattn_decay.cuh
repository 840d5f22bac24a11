// linattn_decay.cuh -- linear attention with a decay for each head: what its
// kernels and its host code share (internal).
//
// Every output of the forward and of the backward is one pass of the same
// form over the positions of a head, with rows a_t, b_t of X elements and
// c_t of Y elements and a state R of X x Y:
//
//   forward in time   R_t = lam R_{t-1} + sk b_t c_t^T,   o_t = si a_t^T R_t
//   reverse in time   R_t = lam R_{t+1} + sk b_t c_t^T,   o_t = si a_t^T R_t
//                     (the state handed in is R_{n-1}'s, undecayed; the one
//                     handed out is lam R_0)
//
//   out     forward  a = q,        b = k,        c = v,        R = S
//   grad_q  forward  a = grad_out, b = v,        c = k,        R = S^T
//   grad_k  reverse  a = v,        b = grad_out, c = q,        R = W^T
//   grad_v  reverse  a = k,        b = q,        c = grad_out, R = W
//
// ("Transformers are RNNs" post, sections "인과 마스킹과 누적합" and "상수 메모리
// 기울기 계산": cumulative sums forward in time for the queries' gradient, in
// reverse for those of the keys and values.)
//
// Long sequences with few heads are cut into segments: one launch sums each
// segment's contribution to the state, a scan joins them in order, and the
// output launch starts every segment from its own state (the last one ends with
// the state that the pass hands out).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "wkv_internal.cuh"

namespace wkv {
namespace decay {

constexpr int kMaxHead = 128;

struct View {
  const void *p;
  int64_t sb, st, sh;
};

struct Pass {
  int64_t B, T, H;
  int X, Y;
  View a, b, c, o;
  const float *log_decay;  // [H]
  const int32_t *lengths;  // [B] or null
  const float *s_in;       // [B, H, X, Y], or [B, H, Y, X] if s_in_t; or null
  int s_in_t;
  float *s_out;            // [B, H, X, Y] or null
  float si, sk;            // factors of the output and of the products entering the state
  int reverse;
  int nseg;                // segments per head
  int64_t seg_len;         // positions per segment
  float *seg;              // [B * H][nseg][X][Y] float32: segment sums, then the states at the segments' starts
};

// Bounded waits inside a block: a role's wait gives up after `tries` (and a
// block that has to end with its loads or products under way after kTries).
struct Waits {
  int32_t *status;  // receives WKV_ERR_TIMEOUT; or null
  uint32_t tries;
  int hold;  // test: the first block's waits run out
};

// Passes of one call that are launched together (blockIdx.y): they have the
// same positions and segments, and sizes of one class.
struct Group {
  Pass p[3];
  int n;
  Waits w;
};

// Positions of row b.
__device__ __forceinline__ int64_t row_len(const Pass &p, int64_t b) {
  if (!p.lengths) return p.T;
  const int64_t n = p.lengths[b];
  return n < 0 ? 0 : n < p.T ? n : p.T;
}
// lam^n as a factor.  From 1/2 up it is kept as m = lam^n - 1 and applied as
// x + x m, exact to one rounding; a rounded lam^n near 1 would drift over many
// factors (2^-24 each time, 10^-5 after a memory of a few hundred positions).
// Below 1/2, m is lam^n itself: there x + x (lam^n - 1) would lose the result's
// low bits.  lam^0 is 1 whatever lam is.
struct Decay {
  float m;
  bool near_one;
};
__device__ __forceinline__ Decay decay_of(float g, int64_t n) {
  if (n == 0) return Decay{0.f, true};
  const float e = g * (float)n;
  return e > -0.69314718f ? Decay{expm1f(e), true} : Decay{expf(e), false};
}
__device__ __forceinline__ float decayed(float x, Decay d) { return fmaf(x, d.m, d.near_one ? x : 0.f); }

// ------------------------------------------------------ two-wide float32 ---
typedef unsigned long long f2;
__device__ __forceinline__ f2 fma2(f2 a, f2 b, f2 c) {
  f2 d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ f2 mul2(f2 a, f2 b) {
  f2 d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ f2 both(float x) {
  f2 d;
  asm("mov.b64 %0, {%1, %1};" : "=l"(d) : "f"(x));
  return d;
}
__device__ __forceinline__ f2 pair(float x, float y) {
  f2 d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(x), "f"(y));
  return d;
}
__device__ __forceinline__ float2 unpair(f2 a) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(a));
  return r;
}

// Launches.  Each returns the first launch's failure.  X of one rec_class may
// share a launch; rec_segments are the segments per head for `npass` passes.
int rec_class(int X);
int64_t rec_segments(int64_t BH, int64_t T, int X, int Y, int npass, int sms);
cudaError_t launch_rec(const Group &g, int dtype, bool sums_only, cudaStream_t st);
cudaError_t launch_scan(const Group &g, cudaStream_t st);
// The tensor-core passes (bfloat16): whether one can take the views, whether
// sizes share a launch, the segments per head and their length, the launches.
bool tc_fits(const Pass &p);
inline bool tc_one_class(int D, int M) { return (D <= 64) == (M <= 64); }
int64_t tc_segments(int64_t BH, int64_t T, int X, int Y, int npass, int sms);
int64_t tc_segment_len(int64_t T, int64_t nseg);
cudaError_t launch_tc(const Group &g, bool sums_only, int sms, cudaStream_t st);
// Tries that take about `us` microseconds when nothing arrives; the default for us <= 0.
uint32_t tc_tries(int64_t us);
struct StepArgs {
  int64_t N, H;
  int D, M;
  View q, k, v, o;
  const float *log_decay;
  float scale;
  const float *s_in;
  float *s_out;
};
cudaError_t launch_step(const StepArgs &s, int dtype, cudaStream_t st);

}  // namespace decay
}  // namespace wkv
