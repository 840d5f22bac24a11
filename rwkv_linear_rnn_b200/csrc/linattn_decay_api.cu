// linattn_decay_api.cu -- host side of linear attention with a decay for each
// head: argument checks, the choice of kernel and of segments, launches
// (C ABI in include/linattn.h).
#include <algorithm>
#include <utility>

#include "../../include/linattn.h"
#include "../../include/wkv.h"
#include "linattn_decay.cuh"

namespace {
using namespace wkv;
using namespace wkv::decay;

bool aligned(const void *p, size_t a) { return ((uintptr_t)p & (a - 1)) == 0; }
size_t elem(int dtype) { return dtype == WKV_F32 ? 4 : 2; }

int num_sms() {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return 148;
  return n;
}

struct Dims {
  int64_t B, T, H;
  int D, M, dtype;
};
int check_dims(const Dims &d) {
  if (d.B < 1 || d.H < 1 || d.T < 0 || d.T >= (int64_t(1) << 31) || d.B >= (int64_t(1) << 24) ||
      d.H >= (int64_t(1) << 24) || d.B * d.H >= (int64_t(1) << 24) || d.D < 1 || d.M < 1)
    return WKV_ERR_INVALID_ARG;
  if (d.dtype != WKV_F32 && d.dtype != WKV_BF16) return WKV_ERR_INVALID_ARG;
  return d.D > kMaxHead || d.M > kMaxHead ? WKV_ERR_UNSUPPORTED : WKV_OK;
}

// A view's pointer and strides; an output's positions must not overlap each
// other: sorted by stride, each dimension steps over the one below it.
int check_view(const linattn_view *v, int64_t n0, int64_t n1, int64_t n2, int width, int dtype, bool output) {
  if (!v || !v->ptr || v->stride_b < 0 || v->stride_t < 0 || v->stride_h < 0) return WKV_ERR_INVALID_ARG;
  if (!aligned(v->ptr, elem(dtype))) return WKV_ERR_UNSUPPORTED;
  constexpr int64_t kMost = int64_t(1) << 40;
  if ((n0 > 1 && v->stride_b > kMost) || (n1 > 1 && v->stride_t > kMost) || (n2 > 1 && v->stride_h > kMost))
    return WKV_ERR_INVALID_ARG;
  if (output) {
    std::pair<int64_t, int64_t> d[3] = {{v->stride_b, n0}, {v->stride_t, n1}, {v->stride_h, n2}};
    std::sort(d, d + 3);
    int64_t span = width;
    for (const auto &x : d) {
      if (x.second <= 1) continue;
      if (x.first < span) return WKV_ERR_INVALID_ARG;
      span += x.first * (x.second - 1);
    }
  }
  return WKV_OK;
}
// First failure among several checks.
int first_of(std::initializer_list<int> rcs) {
  for (int rc : rcs)
    if (rc != WKV_OK) return rc;
  return WKV_OK;
}
bool overlap(const void *a, const void *b, size_t bytes) {
  const uintptr_t x = (uintptr_t)a, y = (uintptr_t)b;
  return a && b && x < y + bytes && y < x + bytes;
}

View view(const linattn_view *v) { return View{v->ptr, v->stride_b, v->stride_t, v->stride_h}; }

size_t up256(size_t x) { return (x + 255) & ~size_t(255); }
size_t seg_bytes(const Dims &d, int64_t nseg) { return nseg > 1 ? up256(sizeof(float) * d.B * d.H * nseg * d.D * d.M) : 0; }

// Whether a call's passes run on the tensor cores, as far as its sizes say.
// Up to 32 positions a chunk of 128 is mostly padding, and the recurrence keeps
// float32's digits in what it multiplies.  Its time grows with the positions:
// forward of 256 x T x 12 heads of 64, 46 us for 8, 77 for 16 and 137 for 32,
// where a chunk takes 75 whatever it holds; 64 x T x 16 of 128, 49, 77 and 137
// against 52; gradients 121, 204 and 431 against 200; one sequence of 12 heads
// of 64, 12, 18 and 30 against 8.  So over many sequences it is the faster one
// as well up to about 8 positions (16 of heads up to 64), and from there to 32
// the digits cost up to two or three times the time (one sequence: almost four).
bool uses_tc(const Dims &d) { return d.dtype == WKV_BF16 && d.T > 32 && d.D % 8 == 0 && d.M % 8 == 0; }

// Bytes of the segments' states of `n` passes of X x Y launched together.
size_t group_bytes(const Dims &d, int X, int Y, int n) {
  const int64_t BH = d.B * d.H;
  const size_t rec = seg_bytes(d, rec_segments(BH, d.T, X, Y, n, num_sms()));
  return n * (uses_tc(d) ? std::max(rec, seg_bytes(d, tc_segments(BH, d.T, X, Y, n, num_sms()))) : rec);
}
// Groups run one after the other and share the workspace.  A backward's
// passes are one group or, with heads of two classes, {grad_q, grad_k} and
// {grad_v}.
size_t workspace(int op, const Dims &d) {
  if (op == LINATTN_OP_FORWARD) return group_bytes(d, d.D, d.M, 1);
  const int x = std::max(d.D, d.M);
  return std::max({group_bytes(d, x, x, 3), group_bytes(d, d.M, d.D, 2), group_bytes(d, d.D, d.M, 1)});
}
int check_ws(size_t need, const void *ws, size_t bytes) {
  if (need == 0) return WKV_OK;
  return !ws || !aligned(ws, 256) || bytes < need ? WKV_ERR_WORKSPACE : WKV_OK;
}

// The passes of a group: segment sums and their scan if the heads are split,
// then the outputs.
cudaError_t run_group(Group &g, const Dims &d, bool tc, void *ws, cudaStream_t st) {
  int X = 0, Y = 0;
  for (int i = 0; i < g.n; ++i) X = std::max(X, g.p[i].X), Y = std::max(Y, g.p[i].Y);
  const int64_t BH = d.B * d.H;
  const int64_t nseg = tc ? tc_segments(BH, d.T, X, Y, g.n, num_sms()) : rec_segments(BH, d.T, X, Y, g.n, num_sms());
  for (int i = 0; i < g.n; ++i) {
    Pass &p = g.p[i];
    p.nseg = (int)nseg;
    p.seg_len = tc ? tc_segment_len(d.T, nseg) : (d.T + nseg - 1) / nseg;
    p.seg = static_cast<float *>(ws) + i * (seg_bytes(d, nseg) / sizeof(float));
  }
  auto launch = [&](bool sums_only) { return tc ? launch_tc(g, sums_only, num_sms(), st) : launch_rec(g, d.dtype, sums_only, st); };
  cudaError_t e = cudaSuccess;
  if (nseg > 1) {
    e = launch(true);
    if (e == cudaSuccess) e = launch_scan(g, st);
  }
  return e == cudaSuccess ? launch(false) : e;
}
cudaError_t run_passes(const Pass *p, int n, const Dims &d, const Waits &w, void *ws, cudaStream_t st) {
  bool tc = uses_tc(d);
  for (int i = 0; i < n; ++i) tc = tc && tc_fits(p[i]);
  const bool one = tc ? tc_one_class(d.D, d.M) : rec_class(d.D) == rec_class(d.M);
  cudaError_t e = cudaSuccess;
  for (int i = 0; i < n && e == cudaSuccess;) {
    Group g{};
    g.w = w;
    const int X = p[i].X;
    while (i < n && (one || p[i].X == X)) g.p[g.n++] = p[i++];
    e = run_group(g, d, tc, ws, st);
  }
  return e;
}

// Options: AUTO is the only choice of kernel.
int check_options(const wkv_options *opt) {
  return opt && (opt->kernel != WKV_KERNEL_AUTO || opt->spin_limit < 0) ? WKV_ERR_INVALID_ARG : WKV_OK;
}
Waits waits(const wkv_options *opt, int32_t *status) {
  return Waits{status, tc_tries(opt ? opt->spin_limit : 0), opt ? opt->test_hold_first_chunk : 0};
}

// linattn_decay_status_word's, one on each device.
__device__ int32_t status_word;

// T = 0, or no work at all: the state goes through.
int pass_state_through(const Dims &d, const float *in, float *out, cudaStream_t st) {
  if (!out || in == out) return WKV_OK;
  const size_t bytes = sizeof(float) * d.B * d.H * d.D * d.M;
  return cuda_status(in ? cudaMemcpyAsync(out, in, bytes, cudaMemcpyDeviceToDevice, st) : cudaMemsetAsync(out, 0, bytes, st));
}
}  // namespace

extern "C" size_t linattn_decay_workspace_size(int op, int64_t B, int64_t T, int64_t H, int D, int M, int dtype) {
  const Dims d{B, T, H, D, M, dtype};
  if ((op != LINATTN_OP_FORWARD && op != LINATTN_OP_BACKWARD) || check_dims(d) != WKV_OK) return 0;
  return workspace(op, d);
}

extern "C" int linattn_decay_status_word(int32_t **word) {
  if (!word) return WKV_ERR_INVALID_ARG;
  // The first use of a module loads it, which a thread that captures may only do in the relaxed mode.
  cudaStreamCaptureMode mode = cudaStreamCaptureModeRelaxed;
  cudaError_t e = cudaThreadExchangeStreamCaptureMode(&mode);
  if (e != cudaSuccess) return cuda_status(e);
  void *p = nullptr;
  e = cudaGetSymbolAddress(&p, status_word);
  const cudaError_t back = cudaThreadExchangeStreamCaptureMode(&mode);
  *word = static_cast<int32_t *>(p);
  return cuda_status(e == cudaSuccess ? back : e);
}

extern "C" int linattn_decay_forward(int64_t B, int64_t T, int64_t H, int D, int M, int dtype, const linattn_view *q,
                                     const linattn_view *k, const linattn_view *v, const float *log_decay, float scale,
                                     const int32_t *lengths, const float *state_in, const linattn_view *out,
                                     float *state_out, void *ws, size_t ws_bytes, int32_t *status, void *stream) {
  return linattn_decay_forward_ex(B, T, H, D, M, dtype, q, k, v, log_decay, scale, lengths, state_in, out, state_out, ws,
                                  ws_bytes, status, stream, nullptr);
}

extern "C" int linattn_decay_forward_ex(int64_t B, int64_t T, int64_t H, int D, int M, int dtype,
                                        const linattn_view *q, const linattn_view *k, const linattn_view *v,
                                        const float *log_decay, float scale, const int32_t *lengths,
                                        const float *state_in, const linattn_view *out, float *state_out, void *ws,
                                        size_t ws_bytes, int32_t *status, void *stream, const wkv_options *opt) {
  const Dims d{B, T, H, D, M, dtype};
  int rc = first_of({check_dims(d), check_options(opt)});
  if (rc != WKV_OK) return rc;
  if (!log_decay) return WKV_ERR_INVALID_ARG;
  if (T > 0) {  // empty tensors may be null
    rc = first_of({check_view(q, B, T, H, D, dtype, false), check_view(k, B, T, H, D, dtype, false),
                   check_view(v, B, T, H, M, dtype, false), check_view(out, B, T, H, M, dtype, true)});
    if (rc != WKV_OK) return rc;
    if (out->ptr == q->ptr || out->ptr == k->ptr || out->ptr == v->ptr) return WKV_ERR_INVALID_ARG;
  }
  if (!aligned(log_decay, 4) || !aligned(lengths, 4) || !aligned(status, 4) || !aligned(state_in, 16) ||
      !aligned(state_out, 16))
    return WKV_ERR_UNSUPPORTED;
  if (state_in != state_out && overlap(state_in, state_out, sizeof(float) * B * H * D * M)) return WKV_ERR_UNSUPPORTED;
  rc = check_ws(workspace(LINATTN_OP_FORWARD, d), ws, ws_bytes);
  if (rc != WKV_OK) return rc;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (T == 0) return pass_state_through(d, state_in, state_out, st);
  Pass p{};
  p.B = B, p.T = T, p.H = H, p.X = D, p.Y = M;
  p.a = view(q), p.b = view(k), p.c = view(v), p.o = view(out);
  p.log_decay = log_decay, p.lengths = lengths, p.s_in = state_in, p.s_out = state_out;
  p.si = scale, p.sk = 1.f;
  return cuda_status(run_passes(&p, 1, d, waits(opt, status), ws, st));
}

extern "C" int linattn_decay_backward(int64_t B, int64_t T, int64_t H, int D, int M, int dtype, const linattn_view *q,
                                      const linattn_view *k, const linattn_view *v, const float *log_decay,
                                      float scale, const int32_t *lengths, const float *state_in,
                                      const linattn_view *grad_out, const float *grad_state_out,
                                      const linattn_view *grad_q, const linattn_view *grad_k,
                                      const linattn_view *grad_v, float *grad_state_in, void *ws, size_t ws_bytes,
                                      int32_t *status, void *stream) {
  return linattn_decay_backward_ex(B, T, H, D, M, dtype, q, k, v, log_decay, scale, lengths, state_in, grad_out,
                                   grad_state_out, grad_q, grad_k, grad_v, grad_state_in, ws, ws_bytes, status, stream,
                                   nullptr);
}

extern "C" int linattn_decay_backward_ex(int64_t B, int64_t T, int64_t H, int D, int M, int dtype,
                                         const linattn_view *q, const linattn_view *k, const linattn_view *v,
                                         const float *log_decay, float scale, const int32_t *lengths,
                                         const float *state_in, const linattn_view *grad_out,
                                         const float *grad_state_out, const linattn_view *grad_q,
                                         const linattn_view *grad_k, const linattn_view *grad_v, float *grad_state_in,
                                         void *ws, size_t ws_bytes, int32_t *status, void *stream,
                                         const wkv_options *opt) {
  const Dims d{B, T, H, D, M, dtype};
  int rc = first_of({check_dims(d), check_options(opt)});
  if (rc != WKV_OK) return rc;
  if (!log_decay) return WKV_ERR_INVALID_ARG;
  if (T > 0) {
    rc = first_of({check_view(q, B, T, H, D, dtype, false), check_view(k, B, T, H, D, dtype, false),
                   check_view(v, B, T, H, M, dtype, false), check_view(grad_out, B, T, H, M, dtype, false),
                   check_view(grad_q, B, T, H, D, dtype, true), check_view(grad_k, B, T, H, D, dtype, true),
                   check_view(grad_v, B, T, H, M, dtype, true)});
    if (rc != WKV_OK) return rc;
    const void *outs[3] = {grad_q->ptr, grad_k->ptr, grad_v->ptr};
    for (int i = 0; i < 3; ++i) {
      for (const linattn_view *in : {q, k, v, grad_out})
        if (outs[i] == in->ptr) return WKV_ERR_INVALID_ARG;
      if (outs[i] == outs[(i + 1) % 3]) return WKV_ERR_INVALID_ARG;
    }
  }
  if (!aligned(log_decay, 4) || !aligned(lengths, 4) || !aligned(status, 4) || !aligned(state_in, 16) ||
      !aligned(grad_state_out, 16) || !aligned(grad_state_in, 16))
    return WKV_ERR_UNSUPPORTED;
  const size_t sbytes = sizeof(float) * B * H * D * M;
  if (overlap(grad_state_in, state_in, sbytes) || overlap(grad_state_in, grad_state_out, sbytes))
    return WKV_ERR_UNSUPPORTED;
  rc = check_ws(workspace(LINATTN_OP_BACKWARD, d), ws, ws_bytes);
  if (rc != WKV_OK) return rc;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (T == 0) return pass_state_through(d, grad_state_out, grad_state_in, st);
  Pass p[3]{};
  for (Pass &x : p) {
    x.B = B, x.T = T, x.H = H;
    x.log_decay = log_decay, x.lengths = lengths;
  }
  // grad_q: forward in time, the state transposed
  p[0].X = M, p[0].Y = D;
  p[0].a = view(grad_out), p[0].b = view(v), p[0].c = view(k), p[0].o = view(grad_q);
  p[0].s_in = state_in, p[0].s_in_t = 1;
  p[0].si = scale, p[0].sk = 1.f;
  // grad_k: reverse, the state's adjoint transposed
  p[1].X = M, p[1].Y = D;
  p[1].a = view(v), p[1].b = view(grad_out), p[1].c = view(q), p[1].o = view(grad_k);
  p[1].s_in = grad_state_out, p[1].s_in_t = 1;
  p[1].si = 1.f, p[1].sk = scale, p[1].reverse = 1;
  // grad_v and the gradient of the state handed in
  p[2].X = D, p[2].Y = M;
  p[2].a = view(k), p[2].b = view(q), p[2].c = view(grad_out), p[2].o = view(grad_v);
  p[2].s_in = grad_state_out, p[2].s_out = grad_state_in;
  p[2].si = 1.f, p[2].sk = scale, p[2].reverse = 1;
  return cuda_status(run_passes(p, 3, d, waits(opt, status), ws, st));
}

extern "C" int linattn_decay_step(int64_t N, int64_t H, int D, int M, int dtype, const linattn_view *q,
                                  const linattn_view *k, const linattn_view *v, const float *log_decay, float scale,
                                  const float *state_in, const linattn_view *out, float *state_out, void *stream) {
  if (N < 1 || H < 1 || N >= (int64_t(1) << 31) || H >= (int64_t(1) << 31) || N * H >= (int64_t(1) << 31) || D < 1 ||
      M < 1 || (dtype != WKV_F32 && dtype != WKV_BF16) || !log_decay || !state_in || !state_out)
    return WKV_ERR_INVALID_ARG;
  if (D > kMaxHead || M > kMaxHead) return WKV_ERR_UNSUPPORTED;
  linattn_view w[4];
  const linattn_view *in[4] = {q, k, v, out};
  for (int i = 0; i < 4; ++i) {
    if (!in[i]) return WKV_ERR_INVALID_ARG;
    w[i] = *in[i];
    w[i].stride_t = 0;  // one position
    const int rc = check_view(&w[i], N, 1, H, i < 2 ? D : M, dtype, i == 3);
    if (rc != WKV_OK) return rc;
  }
  if (out->ptr == q->ptr || out->ptr == k->ptr || out->ptr == v->ptr) return WKV_ERR_INVALID_ARG;
  if (!aligned(log_decay, 4) || !aligned(state_in, 16) || !aligned(state_out, 16)) return WKV_ERR_UNSUPPORTED;
  if (state_in != state_out && overlap(state_in, state_out, sizeof(float) * N * H * D * M)) return WKV_ERR_UNSUPPORTED;
  const decay::StepArgs s{N, H, D, M, view(&w[0]), view(&w[1]), view(&w[2]), view(&w[3]), log_decay, scale, state_in, state_out};
  return cuda_status(launch_step(s, dtype, static_cast<cudaStream_t>(stream)));
}
