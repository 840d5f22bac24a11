// linattn_decay_tc.cu -- one pass of linear attention with a decay for each
// head on the sm_100a tensor cores (bfloat16 tensors; the passes are those of
// linattn_decay.cuh).
//
// Chunked form.  Positions are cut into chunks of L = 128; a, b, c are a
// chunk's rows, n of them valid, R the state at the chunk's start (in reverse
// time: at its end), i a row and j a column of the scores:
//
//   P   = (a b^T) o lam^{i-j} [j <= i]          reverse: lam^{j-i} [i <= j < n]
//   o   = si ( sk P c + lam^{i+1} a R )                  lam^{n-1-i}
//   R'  = lam^n R + sk (lam^{n-1-j} b)^T c               lam^{j+1}
//
// Every product is a chain of tcgen05.mma (kind::f16, bfloat16 operands,
// float32 accumulation in tensor memory): 128 x 128 x X for the scores,
// 128 x Y x 128, 128 x Y x X, and X x Y x 128 for the state, which stays in
// tensor memory for the whole segment.
//
// Roundings.  P and the copy of R that meets a are rounded to bfloat16 once
// (they are matrix operands); both errors are independent of the result's own
// rounding and as large.  Weights lam^n are never multiplied into a bfloat16
// operand with a single rounding: the scores are weighted in float32 before
// the rounding of P, the product with R is weighted in float32 afterwards, and
// the weighted keys enter the state as a sum of three bfloat16 terms (24 bits)
// in the passes that can hand it out (asked to or not, so that the outputs are
// the same bits), or two (16 bits, below the rounding of R's copy) elsewhere.
//
// One CTA runs one head's segment with specialised warps: a producer (TMA
// loads), an MMA issuer, two warpgroups for the state (weighted keys; state
// copy and decay), one for P, one for the outputs.  The floor is HBM: a chunk
// of 128 x (X + X + Y + Y) bfloat16 takes 2.9 us of an SM's share of the
// measured bandwidth at X = Y = 128 against about 1.7 us of MMAs.
#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "linattn_decay.cuh"
#include "wkv_tile.cuh"

namespace wkv {
namespace decay {

constexpr int kL = 128;                  // positions per chunk
constexpr uint32_t kHalf = kL * 128;     // bytes of 128 rows of 64 bfloat16
constexpr uint32_t kTmemCols = 512;
constexpr int64_t kBudgetNs = 1000000000;  // bound on any one wait

// ------------------------------------------------------------ tcgen05 ---
__device__ __forceinline__ void tmem_alloc(uint32_t dst, uint32_t ncols) {
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(dst), "r"(ncols) : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_dealloc(uint32_t taddr, uint32_t ncols) {
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}
__device__ __forceinline__ void tc_before_sync() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_after_sync() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
// D (tensor memory) = A B (+ D if `acc`): A from shared memory, or from tensor memory.
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool acc) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)acc)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool acc) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"((uint32_t)acc)
      : "memory");
}
// Arrive on `bar` once every MMA issued so far by this thread is complete.
__device__ __forceinline__ void mma_commit(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
// 32 columns of this warp's 32 lanes (lane = the thread's row).
__device__ __forceinline__ void tmem_ld32_nowait(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
      "%15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
        "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
        "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
// Uses of r stay behind the wait that stands before this.
__device__ __forceinline__ void pin(uint32_t (&r)[32]) {
#pragma unroll
  for (int k = 0; k < 32; ++k) asm volatile("" : "+r"(r[k]));
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
      "%15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
      "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
      "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
      "%15, %16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}

// Shared-memory matrix descriptors of tiles in the 128-byte swizzle: rows of
// 64 bfloat16 (128 bytes), wider tiles as consecutive halves of `rows` rows.
__device__ __forceinline__ uint64_t sdesc(uint32_t addr, uint32_t lbo, uint32_t sbo) {
  return (uint64_t)((addr >> 4) & 0x3FFFu) | ((uint64_t)((lbo >> 4) & 0x3FFFu) << 16) |
         ((uint64_t)((sbo >> 4) & 0x3FFFu) << 32) | (1ull << 46) | (2ull << 61);
}
// Contraction along the rows' 64-wide halves (128 rows), 16-wide step k16.
__device__ __forceinline__ uint64_t kmajor(uint32_t tile, int k16) {
  return sdesc(tile + kHalf * (k16 >> 2) + 32u * (k16 & 3), 16u, 1024u);
}
// Contraction down the rows; `half` bytes between 64-wide groups of columns.
__device__ __forceinline__ uint64_t mnmajor(uint32_t tile, int k16, uint32_t half) {
  return sdesc(tile + 2048u * k16, half, 1024u);
}
// Instruction descriptor: bf16 x bf16 -> f32, M x N, operand majors.
__host__ __device__ constexpr uint32_t idesc(int M, int N, bool a_mn, bool b_mn) {
  return (1u << 4) | (1u << 7) | (1u << 10) | ((a_mn ? 1u : 0u) << 15) | ((b_mn ? 1u : 0u) << 16) |
         ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}
// Byte offset of 16-byte unit u (0..7) of row r in the 128-byte swizzle.
__device__ __forceinline__ uint32_t sw128(int r, int u) { return (uint32_t)(r * 128 + ((u ^ (r & 7)) << 4)); }

__device__ __forceinline__ void tma_load_4d(uint32_t dst, const void *map, int x, int t, int h, int b, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(
          dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(t), "r"(h), "r"(b), "r"(bar)
      : "memory");
}

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}
__device__ __forceinline__ float lo16(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi16(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }
// lam^n for n >= 0 (1 for n = 0 whatever lam is); g2 = log_decay log2(e).
__device__ __forceinline__ float power(float g2, int64_t n) { return n == 0 ? 1.f : ex2(g2 * (float)n); }

// ------------------------------------------------------------- the pass ---
// Shared memory: NB stages of b, one tile for the weighted keys' second term
// (their first and third take the place of b), NC stages of c, NA of a, and
// the state's bfloat16 copy.  With X = 64 the state's products run with
// M = 128: their rows from 64 on are the bytes of the tile behind b's (there
// always is one) and their results are not read.
template <int XP, int YP>
struct Tiles {
  static constexpr uint32_t BT = XP / 64 * kHalf, CT = YP / 64 * kHalf, RT = YP / 64 * XP * 128;
  static constexpr int NB = XP == 128 ? 2 : YP == 128 ? 3 : 4;
  static constexpr int NA = XP == 128 ? (YP == 128 ? 1 : 2) : 3;
  static constexpr int NC = YP == 128 ? (XP == 128 ? 2 : 3) : XP == 128 ? 3 : 4;
  static constexpr uint32_t B = 0, W2 = B + NB * BT, C = W2 + BT, A = C + NC * CT, R = A + NA * BT, BYTES = R + RT;
};
static_assert(Tiles<128, 128>::BYTES == 224 * 1024 && Tiles<64, 128>::BYTES == 224 * 1024 &&
                  Tiles<128, 64>::BYTES == 224 * 1024 && Tiles<64, 64>::BYTES <= 224 * 1024,
              "the tiles, their alignment and the barriers fit 227 KB");

struct Bars {
  uint64_t b_full[4], c_full[4], a_full[4], b_empty[4], c_empty[4], a_empty[4];
  uint64_t scores;    // a b^T complete (MMA)
  uint64_t p_ready;   // P in tensor memory (P warpgroup)
  uint64_t w_ready;   // first two terms of the weighted keys in place, c's padding zeroed (state warpgroups)
  uint64_t w1_done;   // products with the first term complete: the third may overwrite it (MMA)
  uint64_t w3_ready;  // third term in place (state warpgroups)
  uint64_t state;     // all products into the state complete (MMA)
  uint64_t r_ready;   // the state's copy in shared memory, the state decayed in tensor memory (state warpgroups)
  uint64_t o_done;    // outputs complete in tensor memory (MMA)
  uint64_t o_free;    // outputs read (output warpgroup)
  uint64_t drain;     // every MMA complete
  uint32_t tmem;
  volatile int fail;  // some wait gave up
  alignas(16) float up[32];  // lam^r, lam^{31-r}; read four at a time
  alignas(16) float down[32];
};
constexpr int kStateThreads = 256;

// Bounded wait; a wait that gives up stores WKV_ERR_TIMEOUT and ends the CTA.
__device__ __forceinline__ bool wait(uint64_t &bar, uint32_t parity, Bars *s, int32_t *status) {
  const uint32_t addr = smem_addr(&bar);
  if (mbar_try_wait(addr, parity)) return true;
  if (mbar_wait(addr, parity, kBudgetNs, &s->fail)) return true;
  s->fail = 1;
  if (status) atomicCAS(status, 0, -5 /* WKV_ERR_TIMEOUT */);
  return false;
}
__device__ __forceinline__ bool wait_warp(uint64_t &bar, uint32_t parity, Bars *s, int32_t *status) {
  return __all_sync(~0u, wait(bar, parity, s, status));
}

// The chunks of this CTA's segment, in the pass's order.
struct Chunks {
  int64_t t0, t1;  // the segment's valid positions
  int64_t c0;      // first chunk
  int n;           // chunks with valid positions
  bool reverse;
  __device__ __forceinline__ int64_t start(int it) const { return (c0 + (reverse ? n - 1 - it : it)) * kL; }
  __device__ __forceinline__ int valid(int it) const { return (int)min((int64_t)kL, t1 - start(it)); }
};

// State warpgroups: R at the chunk's start -> its bfloat16 copy in shared
// memory and, decayed, tensor memory again; then the weighted keys.
// Whether the state after the segment goes anywhere; if not, its last chunk
// adds nothing to it.
template <bool OUT>
__device__ __forceinline__ bool wants_state(const Pass &p) {
  return !OUT || (p.nseg == 1 && p.s_out);
}
template <int XP, int YP, bool OUT>
__device__ __forceinline__ void state_role(const Pass &p, Bars *s, uint8_t *sm, const Chunks &ch, int64_t bh,
                                           int terms, float g, float g2) {
  using Ti = Tiles<XP, YP>;
  const int t = threadIdx.x, warp = t >> 5, lane = t & 31;
  const int x = 32 * (warp & 3) + lane;      // state row (tensor-memory lane)
  const int y0 = (warp >> 2) * (YP / 2);     // first of this thread's YP / 2 columns
  const uint32_t tm = s->tmem + 128 + 2 * YP + ((uint32_t)(32 * (warp & 3)) << 16) + y0;
  const bool rows = 32 * (warp & 3) < XP;    // this warp's lanes hold state rows
  const int64_t XY = (int64_t)p.X * p.Y;
  const float *init = !OUT ? nullptr : p.nseg > 1 ? p.seg + (bh * p.nseg + blockIdx.x % p.nseg) * XY
                                     : p.s_in ? p.s_in + bh * XY : nullptr;
  const bool init_t = p.nseg == 1 && p.s_in_t;
  float *result = !OUT ? p.seg + (bh * p.nseg + blockIdx.x % p.nseg) * XY
                       : wants_state<OUT>(p) ? p.s_out + bh * XY : nullptr;
  auto store_row = [&](int yb, const uint32_t(&v)[32]) {  // columns yb.. of row x
    if (x >= p.X) return;
    float *dst = result + (int64_t)x * p.Y + yb;
#pragma unroll
    for (int q = 0; q < 8; ++q)
      if (yb + 4 * q < p.Y) reinterpret_cast<uint4 *>(dst)[q] = make_uint4(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]);
  };
  auto load_row = [&](int yb, uint32_t(&v)[32]) {
#pragma unroll
    for (int q = 0; q < 32; ++q) {
      const int y = yb + q;
      v[q] = init && x < p.X && y < p.Y ? __float_as_uint(init[init_t ? (int64_t)y * p.X + x : (int64_t)x * p.Y + y]) : 0u;
    }
  };
  bool ok = true;
  for (int it = 0; it < ch.n && ok; ++it) {
    const int nv = ch.valid(it);
    const uint32_t ph = it & 1;
    if (it > 0 && !(ok = wait_warp(s->state, ph ^ 1u, s, p.status))) break;
    if (OUT) {
      if (rows) {
        const Decay d = decay_of(g, nv);
        tc_after_sync();
#pragma unroll
        for (int blk = 0; blk < YP / 64; ++blk) {
          const int yb = y0 + 32 * blk;
          uint32_t v[32];
          if (it == 0) {
            load_row(yb, v);
          } else {
            tmem_ld32_nowait(tm + 32 * blk, v);
            tmem_wait_ld();
            pin(v);
          }
          uint8_t *half = sm + Ti::R + (yb >> 6) * (XP * 128);
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            const float *f = reinterpret_cast<const float *>(v) + 8 * u;
            *reinterpret_cast<uint4 *>(half + sw128(x, ((yb & 63) >> 3) + u)) =
                make_uint4(pack2(f[0], f[1]), pack2(f[2], f[3]), pack2(f[4], f[5]), pack2(f[6], f[7]));
          }
#pragma unroll
          for (int q = 0; q < 32; ++q) v[q] = __float_as_uint(decayed(__uint_as_float(v[q]), d));
          tmem_st32(tm + 32 * blk, v);
        }
        tmem_wait_st();
        tc_before_sync();
        fence_proxy_async_smem();
      }
      mbar_arrive(smem_addr(&s->r_ready));
      if (!(ok = wait_warp(s->scores, ph, s, p.status))) break;  // b is no longer read as it came
    }
    // weighted keys: row j = t % 128, one half of its columns
    const int st = it % Ti::NB, cst = it % Ti::NC;
    if (!(ok = wait_warp(s->b_full[st], (it / Ti::NB) & 1, s, p.status))) break;
    const bool keys = wants_state<OUT>(p) || it + 1 < ch.n;
    const int j = t & 127;
    const int64_t n = p.reverse ? j + 1 + (OUT ? 0 : ch.start(it) - ch.t0)
                                : (OUT ? nv : ch.t1 - ch.start(it)) - 1 - j;
    const float w = j < nv ? p.sk * power(g2, n) : 0.f;
    constexpr int UN = XP / 16;  // 16-byte units per thread
    uint32_t third[4 * UN];
    uint8_t *tb = sm + Ti::B + st * Ti::BT, *t2 = sm + Ti::W2;
    const uint32_t hoff = XP == 128 ? (uint32_t)(t >> 7) * kHalf : 0u;
    const int u0 = XP == 128 ? 0 : (t >> 7) * UN;
#pragma unroll
    for (int u = 0; u < UN; ++u) {
      if (!keys) break;
      const uint32_t off = hoff + sw128(j, u0 + u);
      const uint4 in = *reinterpret_cast<const uint4 *>(tb + off);
      const uint32_t iw[4] = {in.x, in.y, in.z, in.w};
      uint32_t w1[4], w2[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        // rows behind the last position may hold anything: select, not multiply
        float x0 = j < nv ? lo16(iw[e]) * w : 0.f, x1 = j < nv ? hi16(iw[e]) * w : 0.f;
        w1[e] = pack2(x0, x1);
        x0 -= lo16(w1[e]), x1 -= hi16(w1[e]);
        w2[e] = pack2(x0, x1);
        x0 -= lo16(w2[e]), x1 -= hi16(w2[e]);
        third[4 * u + e] = pack2(x0, x1);
      }
      *reinterpret_cast<uint4 *>(tb + off) = make_uint4(w1[0], w1[1], w1[2], w1[3]);
      *reinterpret_cast<uint4 *>(t2 + off) = make_uint4(w2[0], w2[1], w2[2], w2[3]);
    }
    if (nv < kL) {  // c's rows behind the last position: 0 x anything has to be 0
      if (!(ok = wait_warp(s->c_full[cst], (it / Ti::NC) & 1, s, p.status))) break;
      uint8_t *tc = sm + Ti::C + cst * Ti::CT;
      for (int e = t; e < (int)(Ti::CT / 16); e += kStateThreads)
        if (((e >> 3) & 127) >= nv) reinterpret_cast<uint4 *>(tc)[e] = make_uint4(0u, 0u, 0u, 0u);
    }
    fence_proxy_async_smem();
    mbar_arrive(smem_addr(&s->w_ready));
    if (keys && terms == 3) {
      if (!(ok = wait_warp(s->w1_done, ph, s, p.status))) break;
#pragma unroll
      for (int u = 0; u < UN; ++u)
        *reinterpret_cast<uint4 *>(tb + hoff + sw128(j, u0 + u)) =
            make_uint4(third[4 * u], third[4 * u + 1], third[4 * u + 2], third[4 * u + 3]);
      fence_proxy_async_smem();
      mbar_arrive(smem_addr(&s->w3_ready));
    }
  }
  if (!ok || !result || !rows) return;
  if (ch.n > 0) {
    if (!wait_warp(s->state, (ch.n - 1) & 1, s, p.status)) return;
    tc_after_sync();
  }
#pragma unroll
  for (int blk = 0; blk < YP / 64; ++blk) {
    uint32_t v[32];
    if (ch.n > 0) {
      tmem_ld32_nowait(tm + 32 * blk, v);
      tmem_wait_ld();
      pin(v);
    } else {
      load_row(y0 + 32 * blk, v);  // no positions: the state goes through
    }
    store_row(y0 + 32 * blk, v);
  }
}

// P warpgroup: masked, weighted scores -> bfloat16 in tensor memory, over the
// scores' own columns (a thread reads 32 columns before it writes 16 of them).
__device__ __forceinline__ void scores_role(const Pass &p, Bars *s, const Chunks &ch, float g2) {
  const int i = threadIdx.x & 127, w = i >> 5, lane = i & 31;
  const uint32_t tm = s->tmem + ((uint32_t)(32 * w) << 16);
  const float f = p.si * p.sk;
  for (int it = 0; it < ch.n; ++it) {
    const int nv = ch.valid(it);
    if (!wait_warp(s->scores, it & 1, s, p.status)) return;
    tc_after_sync();
#pragma unroll 1
    for (int b = 0; b < 4; ++b) {
      uint32_t out[16];
      if (p.reverse ? b < w || 32 * b >= nv : b > w) {
#pragma unroll
        for (int r = 0; r < 16; ++r) out[r] = 0u;
      } else {
        uint32_t v[32];
        tmem_ld32_nowait(tm + 32 * b, v);
        tmem_wait_ld();
        pin(v);
        if (b == w) {  // the diagonal
          const int last = p.reverse ? nv - 32 * b : 32;
#pragma unroll
          for (int r = 0; r < 32; ++r) {
            const int n = p.reverse ? r - lane : lane - r;
            v[r] = __float_as_uint(n >= 0 && r < last ? __uint_as_float(v[r]) * (f * s->up[n & 31]) : 0.f);
          }
        } else {
          const float e = f * ex2(g2 * (float)(p.reverse ? 32 * b - i : i - 32 * b - 31));
          const float *tab = p.reverse ? s->up : s->down;
          const int last = p.reverse ? nv - 32 * b : 32;
#pragma unroll
          for (int q = 0; q < 8; ++q) {
            const float4 z = *reinterpret_cast<const float4 *>(tab + 4 * q);
            v[4 * q] = __float_as_uint(__uint_as_float(v[4 * q]) * (e * z.x));
            v[4 * q + 1] = __float_as_uint(__uint_as_float(v[4 * q + 1]) * (e * z.y));
            v[4 * q + 2] = __float_as_uint(__uint_as_float(v[4 * q + 2]) * (e * z.z));
            v[4 * q + 3] = __float_as_uint(__uint_as_float(v[4 * q + 3]) * (e * z.w));
          }
          if (last < 32) {
#pragma unroll
            for (int r = 0; r < 32; ++r) v[r] = r < last ? v[r] : 0u;
          }
        }
#pragma unroll
        for (int r = 0; r < 16; ++r) out[r] = pack2(__uint_as_float(v[2 * r]), __uint_as_float(v[2 * r + 1]));
      }
      tmem_st16(tm + 16 * b, out);
    }
    tmem_wait_st();
    tc_before_sync();
    mbar_arrive(smem_addr(&s->p_ready));
  }
}

// Output warpgroup: P c + weight x (a R), one row per thread, rounded and
// stored as 16- or 32-byte pieces of its row.
template <int YP>
__device__ __forceinline__ void output_role(const Pass &p, Bars *s, const Chunks &ch, int64_t b, int64_t h, float g2,
                                            bool wide) {
  const int i = threadIdx.x & 127;
  const uint32_t tm = s->tmem + 128 + ((uint32_t)(i & ~31) << 16);
  for (int it = 0; it < ch.n; ++it) {
    const int nv = ch.valid(it);
    if (!wait_warp(s->o_done, it & 1, s, p.status)) return;
    tc_after_sync();
    const float w = i < nv ? p.si * power(g2, p.reverse ? nv - 1 - i : i + 1) : 0.f;
    const int64_t t = ch.start(it) + i;
    uint16_t *dst = static_cast<uint16_t *>(const_cast<void *>(p.o.p)) + b * p.o.sb + h * p.o.sh + t * p.o.st;
#pragma unroll
    for (int blk = 0; blk < YP / 32; ++blk) {
      uint32_t o1[32], o2[32], out[16];
      tmem_ld32_nowait(tm + 32 * blk, o1);
      tmem_ld32_nowait(tm + YP + 32 * blk, o2);
      tmem_wait_ld();
      pin(o1);
      pin(o2);
      if (blk == YP / 32 - 1) {
        tc_before_sync();
        mbar_arrive(smem_addr(&s->o_free));
      }
#pragma unroll
      for (int r = 0; r < 16; ++r)
        out[r] = i < nv ? pack2(fmaf(w, __uint_as_float(o2[2 * r]), __uint_as_float(o1[2 * r])),
                                fmaf(w, __uint_as_float(o2[2 * r + 1]), __uint_as_float(o1[2 * r + 1])))
                        : 0u;
      if (t >= p.T) continue;
      if (wide) {
#pragma unroll
        for (int q = 0; q < 2; ++q)
          if (32 * blk + 16 * q < p.Y)
            asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst + 32 * blk + 16 * q),
                         "r"(out[8 * q]), "r"(out[8 * q + 1]), "r"(out[8 * q + 2]), "r"(out[8 * q + 3]),
                         "r"(out[8 * q + 4]), "r"(out[8 * q + 5]), "r"(out[8 * q + 6]), "r"(out[8 * q + 7])
                         : "memory");
      } else {
#pragma unroll
        for (int q = 0; q < 4; ++q)
          if (32 * blk + 8 * q < p.Y)
            *reinterpret_cast<uint4 *>(dst + 32 * blk + 8 * q) =
                make_uint4(out[4 * q], out[4 * q + 1], out[4 * q + 2], out[4 * q + 3]);
      }
    }
  }
}

// Loads: b and c of a chunk, then a, each as soon as its stage is free.
template <int XP, int YP, bool OUT>
__device__ __forceinline__ void load_role(const Pass &p, Bars *s, uint32_t sm, const Chunks &ch, int b, int h,
                                          const CUtensorMap *am, const CUtensorMap *bm, const CUtensorMap *cm) {
  using Ti = Tiles<XP, YP>;
  auto tile = [&](uint32_t dst, const CUtensorMap *m, uint64_t &full, uint32_t bytes, int64_t t) {
    const uint32_t bar = smem_addr(&full);
    mbar_expect_tx(bar, bytes);
    for (uint32_t o = 0; o < bytes; o += kHalf) tma_load_4d(dst + o, m, (int)(o / kHalf) * 64, (int)t, h, b, bar);
  };
  int nb = 0, nc = 0, na = 0;  // tiles whose loads were issued
  bool ok = true;
  for (int it = 0; it < ch.n && ok; ++it) {
    const int64_t t = ch.start(it);
    int st = it % Ti::NB;
    if (it >= Ti::NB && !(ok = wait(s->b_empty[st], (it / Ti::NB - 1) & 1, s, p.status))) break;
    tile(sm + Ti::B + st * Ti::BT, bm, s->b_full[st], Ti::BT, t);
    nb = it + 1;
    st = it % Ti::NC;
    if (it >= Ti::NC && !(ok = wait(s->c_empty[st], (it / Ti::NC - 1) & 1, s, p.status))) break;
    tile(sm + Ti::C + st * Ti::CT, cm, s->c_full[st], Ti::CT, t);
    nc = it + 1;
    if (OUT) {
      st = it % Ti::NA;
      if (it >= Ti::NA && !(ok = wait(s->a_empty[st], (it / Ti::NA - 1) & 1, s, p.status))) break;
      tile(sm + Ti::A + st * Ti::BT, am, s->a_full[st], Ti::BT, t);
      na = it + 1;
    }
  }
  // The loads in flight write shared memory that outlives this thread, not the
  // CTA: every one is waited for (in order to end; consumers wait for theirs).
  for (int it = max(0, nb - Ti::NB); it < nb; ++it)
    mbar_wait(smem_addr(&s->b_full[it % Ti::NB]), (it / Ti::NB) & 1, kBudgetNs, nullptr);
  for (int it = max(0, nc - Ti::NC); it < nc; ++it)
    mbar_wait(smem_addr(&s->c_full[it % Ti::NC]), (it / Ti::NC) & 1, kBudgetNs, nullptr);
  for (int it = max(0, na - Ti::NA); it < na; ++it)
    mbar_wait(smem_addr(&s->a_full[it % Ti::NA]), (it / Ti::NA) & 1, kBudgetNs, nullptr);
}

// MMAs, in an order that gives each warpgroup's step the products of another
// to hide behind: a R and P c, then the state's products, then the next
// chunk's scores while the state's copy is made.
template <int XP, int YP, bool OUT>
__device__ __forceinline__ void mma_role(const Pass &p, Bars *s, uint32_t sm, const Chunks &ch, int terms) {
  using Ti = Tiles<XP, YP>;
  constexpr uint32_t SCORES = 0, O1 = 128, O2 = 128 + YP, ST = 128 + 2 * YP;
  const uint32_t tm = s->tmem;
  auto scores = [&](int it) {
    if (!wait(s->b_full[it % Ti::NB], (it / Ti::NB) & 1, s, p.status)) return false;
    if (!wait(s->a_full[it % Ti::NA], (it / Ti::NA) & 1, s, p.status)) return false;
    const uint32_t ta = sm + Ti::A + (it % Ti::NA) * Ti::BT, tb = sm + Ti::B + (it % Ti::NB) * Ti::BT;
#pragma unroll
    for (int k = 0; k < XP / 16; ++k) mma_ss(tm + SCORES, kmajor(ta, k), kmajor(tb, k), idesc(128, 128, false, false), k > 0);
    mma_commit(smem_addr(&s->scores));
    return true;
  };
  bool ok = true;
  if (OUT && ch.n > 0) ok = scores(0);
  for (int it = 0; it < ch.n && ok; ++it) {
    const uint32_t ph = it & 1;
    const uint32_t ta = sm + Ti::A + (it % Ti::NA) * Ti::BT, tb = sm + Ti::B + (it % Ti::NB) * Ti::BT,
                   tc = sm + Ti::C + (it % Ti::NC) * Ti::CT;
    if (OUT) {
      if (!(ok = wait(s->r_ready, ph, s, p.status))) break;
      if (it > 0 && !(ok = wait(s->o_free, ph ^ 1u, s, p.status))) break;
      tc_after_sync();
#pragma unroll
      for (int k = 0; k < XP / 16; ++k)
        mma_ss(tm + O2, kmajor(ta, k), mnmajor(sm + Ti::R, k, XP * 128), idesc(128, YP, false, true), k > 0);
      mma_commit(smem_addr(&s->a_empty[it % Ti::NA]));
    }
    if (!(ok = wait(s->c_full[it % Ti::NC], (it / Ti::NC) & 1, s, p.status))) break;
    if (!(ok = wait(s->w_ready, ph, s, p.status))) break;
    if (OUT) {
      if (!(ok = wait(s->p_ready, ph, s, p.status))) break;
      tc_after_sync();
#pragma unroll
      for (int k = 0; k < kL / 16; ++k)
        mma_ts(tm + O1, tm + SCORES + 8 * k, mnmajor(tc, k, kHalf), idesc(128, YP, false, true), k > 0);
      mma_commit(smem_addr(&s->o_done));
    }
    tc_after_sync();
    const bool keys = wants_state<OUT>(p) || it + 1 < ch.n;
    for (int term = 0; keys && term < terms; ++term) {
      if (term == 2 && !(ok = wait(s->w3_ready, ph, s, p.status))) break;
      const uint32_t tw = term == 1 ? sm + Ti::W2 : tb;
#pragma unroll
      for (int k = 0; k < kL / 16; ++k)
        mma_ss(tm + ST, mnmajor(tw, k, kHalf), mnmajor(tc, k, kHalf), idesc(128, YP, true, true), OUT || it > 0 || term > 0 || k > 0);
      if (term == 0 && terms == 3) mma_commit(smem_addr(&s->w1_done));
    }
    if (!ok) break;
    mma_commit(smem_addr(&s->state));
    mma_commit(smem_addr(&s->b_empty[it % Ti::NB]));
    mma_commit(smem_addr(&s->c_empty[it % Ti::NC]));
    if (OUT && it + 1 < ch.n) ok = scores(it + 1);
  }
  // MMAs in flight read shared memory and write tensor memory: they end before the CTA does
  mma_commit(smem_addr(&s->drain));
  mbar_wait(smem_addr(&s->drain), 0, kBudgetNs, nullptr);
}

struct Maps {
  CUtensorMap a[3], b[3], c[3];
  int terms[3], wide[3];
};
template <int XP, int YP, bool OUT>
__global__ void __launch_bounds__(OUT ? 576 : 320, 1) decay_tc_kernel(const __grid_constant__ Maps maps,
                                                                      const __grid_constant__ Group group) {
  const Pass &p = group.p[blockIdx.y];
  const CUtensorMap &am = maps.a[blockIdx.y], &bm = maps.b[blockIdx.y], &cm = maps.c[blockIdx.y];
  const int terms = maps.terms[blockIdx.y], wide = maps.wide[blockIdx.y];
  if (!OUT && !p.scan_out && (int)blockIdx.x % p.nseg == (p.reverse ? 0 : p.nseg - 1)) return;  // no state starts from it
  extern __shared__ uint8_t smem_raw[];
  __shared__ Bars bars;
  uint8_t *sm = smem_raw + (((smem_addr(smem_raw) + 1023u) & ~1023u) - smem_addr(smem_raw));
  const int64_t bh = blockIdx.x / p.nseg, b = bh / p.H, h = bh % p.H;
  const int64_t n = row_len(p, b);
  Chunks ch;
  ch.t0 = (blockIdx.x % p.nseg) * p.seg_len;
  const int64_t tz = min(ch.t0 + p.seg_len, p.T);
  ch.t1 = max(ch.t0, min(tz, n));
  ch.c0 = ch.t0 / kL;
  ch.n = (int)((ch.t1 - ch.t0 + kL - 1) / kL);
  ch.reverse = p.reverse;
  const float g = p.log_decay[h], g2 = g * kLog2e;
  const int warp = threadIdx.x >> 5;
  constexpr int kLoadWarp = OUT ? 16 : 8;
  if (threadIdx.x == 0) {
    for (int i = 0; i < 4; ++i)
      for (uint64_t *f : {&bars.b_full[i], &bars.c_full[i], &bars.a_full[i], &bars.b_empty[i], &bars.c_empty[i], &bars.a_empty[i]})
        mbar_init(smem_addr(f), 1);
    for (uint64_t *f : {&bars.scores, &bars.w1_done, &bars.state, &bars.o_done, &bars.drain}) mbar_init(smem_addr(f), 1);
    for (uint64_t *f : {&bars.w_ready, &bars.w3_ready, &bars.r_ready}) mbar_init(smem_addr(f), kStateThreads);
    for (uint64_t *f : {&bars.p_ready, &bars.o_free}) mbar_init(smem_addr(f), 128);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    bars.fail = 0;
  }
  if (threadIdx.x >= 32 && threadIdx.x < 64) {
    const int r = threadIdx.x - 32;
    bars.up[r] = power(g2, r);
    bars.down[r] = power(g2, 31 - r);
  }
  if (warp == 0) tmem_alloc(smem_addr(&bars.tmem), kTmemCols);
  tc_before_sync();
  __syncthreads();
  tc_after_sync();
  if (warp < kStateThreads / 32) {
    state_role<XP, YP, OUT>(p, &bars, sm, ch, bh, terms, g, g2);
  } else if (OUT && warp < 12) {
    scores_role(p, &bars, ch, g2);
  } else if (OUT && warp < 16) {
    output_role<YP>(p, &bars, ch, b, h, g2, wide != 0);
  } else if (warp == kLoadWarp) {
    if ((threadIdx.x & 31) == 0) load_role<XP, YP, OUT>(p, &bars, smem_addr(sm), ch, (int)b, (int)h, &am, &bm, &cm);
  } else {
    if ((threadIdx.x & 31) == 0) mma_role<XP, YP, OUT>(p, &bars, smem_addr(sm), ch, terms);
  }
  __syncwarp();
  if (OUT) {  // chunks without valid positions
    const int units = p.Y / 8;
    const int64_t z0 = min((ch.c0 + ch.n) * (int64_t)kL, tz);
    for (int64_t e = threadIdx.x; e < (tz - z0) * units; e += blockDim.x) {
      uint16_t *dst = static_cast<uint16_t *>(const_cast<void *>(p.o.p)) + b * p.o.sb + h * p.o.sh;
      reinterpret_cast<uint4 *>(dst + (z0 + e / units) * p.o.st)[e % units] = make_uint4(0u, 0u, 0u, 0u);
    }
  }
  tc_before_sync();
  __syncthreads();
  if (warp == 0) {
    tc_after_sync();
    tmem_dealloc(bars.tmem, kTmemCols);
  }
}

// ---------------------------------------------------------------- host ---
namespace {
typedef CUresult (*EncodeFn)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                             const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                             CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
void *driver_entry(const char *name) {
  void *f = nullptr;
  cudaDriverEntryPointQueryResult q;
  return cudaGetDriverEntryPoint(name, &f, cudaEnableDefault, &q) == cudaSuccess && q == cudaDriverEntryPointSuccess
             ? f
             : nullptr;
}
EncodeFn encoder() {
  static const EncodeFn fn = reinterpret_cast<EncodeFn>(driver_entry("cuTensorMapEncodeTiled"));
  return fn;
}
// The encoder is a driver call and needs a current context; a thread whose
// first CUDA use is this call may have none.
bool ensure_context() {
  static const auto get = reinterpret_cast<CUresult (*)(CUcontext *)>(driver_entry("cuCtxGetCurrent"));
  CUcontext ctx = nullptr;
  if (get && get(&ctx) == CUDA_SUCCESS && ctx) return true;
  int dev = 0;
  return cudaGetDevice(&dev) == cudaSuccess && cudaSetDevice(dev) == cudaSuccess;
}
// A [B, T, H, width] view in boxes of 128 positions x 64 elements; what lies
// outside the tensor reads as zero.
bool encode(CUtensorMap *m, const View &v, const Pass &p, int width) {
  const cuuint64_t dims[4] = {(cuuint64_t)width, (cuuint64_t)p.T, (cuuint64_t)p.H, (cuuint64_t)p.B};
  auto bytes = [](int64_t stride, int64_t n) { return (cuuint64_t)(n > 1 ? 2 * stride : 16); };
  const cuuint64_t strides[3] = {bytes(v.st, p.T), bytes(v.sh, p.H), bytes(v.sb, p.B)};
  const cuuint32_t box[4] = {64, kL, 1, 1}, step[4] = {1, 1, 1, 1};
  return encoder()(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void *>(v.p), dims, strides, box, step,
                   CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                   CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
bool rows16(const View &v, const Pass &p, bool tma) {
  auto fits = [&](int64_t s, int64_t n) { return n <= 1 || (s % 8 == 0 && (!tma || s > 0)); };
  return ((uintptr_t)v.p & 15u) == 0 && fits(v.sb, p.B) && fits(v.st, p.T) && fits(v.sh, p.H);
}
template <int XP, int YP, bool OUT>
cudaError_t launch_t(const Group &g, cudaStream_t st) {
  Maps m{};
  if (!encoder() || !ensure_context()) return cudaErrorNotSupported;
  const auto kern = decay_tc_kernel<XP, YP, OUT>;
  constexpr int smem = (int)Tiles<XP, YP>::BYTES + 1024;
  int blocks = 0;
  const cudaError_t e = blocks_per_sm((const void *)kern, OUT ? 576 : 320, smem, &blocks);
  if (e != cudaSuccess) return e;
  if (blocks < 1) return cudaErrorInvalidConfiguration;
  auto even = [](int64_t s, int64_t n) { return n <= 1 || s % 16 == 0; };
  for (int i = 0; i < g.n; ++i) {
    const Pass &p = g.p[i];
    if ((OUT && !encode(&m.a[i], p.a, p, p.X)) || !encode(&m.b[i], p.b, p, p.X) || !encode(&m.c[i], p.c, p, p.Y))
      return cudaErrorInvalidValue;
    m.wide[i] = OUT && ((uintptr_t)p.o.p & 31u) == 0 && p.Y % 16 == 0 && even(p.o.sb, p.B) && even(p.o.st, p.T) &&
                even(p.o.sh, p.H);
    // states that a call may hand out are float32; those that only meet rows as bfloat16 copies need not be
    m.terms[i] = p.exact_state && (!OUT || p.nseg == 1) ? 3 : 2;
  }
  const Pass &p = g.p[0];
  return launch_kernel(kern, dim3((unsigned)(p.B * p.H * p.nseg), (unsigned)g.n), dim3(OUT ? 576 : 320), smem, st, m, g);
}
template <bool OUT>
cudaError_t launch_o(const Group &g, cudaStream_t st) {
  const int X = g.p[0].X, Y = g.p[0].Y;
  if (X <= 64) return Y <= 64 ? launch_t<64, 64, OUT>(g, st) : launch_t<64, 128, OUT>(g, st);
  return Y <= 64 ? launch_t<128, 64, OUT>(g, st) : launch_t<128, 128, OUT>(g, st);
}
}  // namespace

bool tc_fits(const Pass &p) {
  return p.X % 8 == 0 && p.Y % 8 == 0 && p.X <= 128 && p.Y <= 128 && rows16(p.a, p, true) && rows16(p.b, p, true) &&
         rows16(p.c, p, true) && rows16(p.o, p, false);
}
int64_t tc_segments(int64_t BH, int64_t T, int npass, int sms) {
  BH *= npass;
  // in units of one chunk's outputs: a segment costs its chunks and about 2 for
  // starting and ending its CTA; a head in several segments also its sums (b
  // and c are read twice) and the scan
  const int64_t nch = (T + kL - 1) / kL;
  int64_t best = 1;
  double least = 1e300;
  for (int64_t n = 1; n <= std::min<int64_t>(nch, std::max<int64_t>(1, 2 * sms / BH)); ++n) {
    const int64_t per = (nch + n - 1) / n;
    if ((nch + per - 1) / per != n) continue;
    const double waves = (double)((BH * n + sms - 1) / sms);
    const double t = waves * (per + 2.0) + (n > 1 ? waves * (0.6 * per + 2.0) + 2.0 : 0.0);
    if (t < least) least = t, best = n;
  }
  return best;
}
int64_t tc_segment_len(int64_t T, int64_t nseg) {
  const int64_t nch = (T + kL - 1) / kL;
  return (nch + nseg - 1) / nseg * kL;
}
cudaError_t launch_tc(const Group &g, bool sums_only, cudaStream_t st) {
  return sums_only ? launch_o<false>(g, st) : launch_o<true>(g, st);
}

}  // namespace decay
}  // namespace wkv
