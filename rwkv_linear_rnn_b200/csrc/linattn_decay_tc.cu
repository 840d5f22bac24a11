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
// rounding and as large.  Weights are applied in float32 before the rounding
// (P) or afterwards (a R).  The weighted keys lam^n b enter the state, which is
// float32, as a sum of two bfloat16 terms: 16 bits, below the rounding of R's
// copy, and an error of 4e-6 of a state that is handed out.  (A third term,
// 24 bits, leaves 1e-6 there, the accumulation's own, and costs 40 % of the
// time at X = Y = 128; a single one would be a rounding more in the outputs.)
//
// One CTA runs one head's segment with specialised warps: a producer (TMA
// loads), an MMA issuer, a warpgroup for the state (its bfloat16 copy and its
// decay), one for the outputs, two for P, one for the weighted keys (fewer where
// two CTAs share an SM).  The MMAs
// of a chunk are issued in the order scores, keys (first term), a R, keys
// (second term), P c, so that each step of a warpgroup has the products of
// others to hide behind: P behind keys and a R, the state's step behind P c and
// the next scores, the next chunk's keys behind all of them.
//
// The floor is HBM: a chunk of 128 x (X + X + Y + Y) bfloat16 takes 2.9 us of
// an SM's share of the measured bandwidth at X = Y = 128; its MMAs take 1.4 us.
// Measured: 3.3 us a chunk (8 x 4096 x 16 heads of 128: forward 105 to 112 us,
// 4.8 to 5.1 TB/s; backward 303 to 318 us), 2.2 us at X = Y = 64.  A chunk is
// the chain scores, P, P c, outputs read, next a R, with the state's step beside
// it, and the loads' latency under load is 1.9 us; the tensor pipe is busy 37 %
// of the time and the schedulers 40 %.  What it took, at X = Y = 128: the MMA
// warp whole under an election (an MMA in 64 cycles, not 130) and its operands
// known uniform; roles without spills (one word is left at X = 128) and in short
// loops (the GPC's instruction cache was 82 % busy); masks as bits; the state never waiting for
// the keys: 177 -> 108 us forward.
#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "../../include/wkv.h"
#include "linattn_decay.cuh"
#include "wkv_tile.cuh"

namespace wkv {
namespace decay {

constexpr int kL = 128;                  // positions per chunk
constexpr uint32_t kHalf = kL * 128;     // bytes of 128 rows of 64 bfloat16
constexpr int kMostSlots = 8;             // of the ring of tiles
// Bound on any one wait: the hardware suspends a try for about kTryUs
// microseconds when nothing arrives (measured: 3.9), so that kTries are about a second.
constexpr int64_t kTryUs = 4;
constexpr uint32_t kTries = 1000000 / kTryUs;

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
// Upper word of every shared-memory matrix descriptor here: 1024 bytes between
// groups of 8 rows, 128-byte swizzle.
constexpr uint32_t kDescHigh = (1024u >> 4) | (1u << 14) | (2u << 29);
// D (tensor memory) = A B (+ D if `acc`): A from shared memory, or from tensor
// memory.  a and b are descriptors' lower words (below).
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, bool acc) {
  asm volatile(
      "{\n .reg .pred p;\n .reg .b64 a, b;\n setp.ne.b32 p, %4, 0;\n mov.b64 a, {%1, %5};\n mov.b64 b, {%2, %5};\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, p;\n}\n" ::"r"(d),
      "r"(a), "r"(b), "r"(idesc), "r"((uint32_t)acc), "n"(kDescHigh)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, bool acc) {
  asm volatile(
      "{\n .reg .pred p;\n .reg .b64 b;\n setp.ne.b32 p, %4, 0;\n mov.b64 b, {%2, %5};\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %3, p;\n}\n" ::"r"(d),
      "r"(a), "r"(b), "r"(idesc), "r"((uint32_t)acc), "n"(kDescHigh)
      : "memory");
}
// One lane of a converged warp.  The MMA and load warps run their loops whole
// and issue under this election: with operands that the compiler knows to be
// the same in every lane a tcgen05.mma is one instruction (in a branch on the
// lane's index each costs about 130 cycles).
__device__ __forceinline__ bool elect_one() {
  uint32_t ok;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xFFFFFFFF;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(ok));
  return ok != 0;
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
__device__ __forceinline__ void tmem_ld16_nowait(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
      "%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
// Uses of r stay behind the wait that stands before this.
template <int N>
__device__ __forceinline__ void pin(uint32_t (&r)[N]) {
#pragma unroll
  for (int k = 0; k < N; ++k) asm volatile("" : "+r"(r[k]));
}
// f(c, v) for c = first, first + 1, .. end - 1 and the 16 columns v from tm + 16 c on.
template <typename F>
__device__ __forceinline__ void tmem_each16(uint32_t tm, int first, int end, F f) {
#pragma unroll 1
  for (int c = first; c < end; ++c) {
    uint32_t v[16];
    tmem_ld16_nowait(tm + 16 * c, v);
    tmem_wait_ld();
    pin(v);
    f(c, v);
  }
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
// The upper word is the same for all (1024 bytes between groups of 8 rows);
// the lower one holds the address and the distance between halves, and a step
// along the contraction adds to it (addresses below 256 KB do not carry out).
__device__ __forceinline__ uint32_t sdesc(uint32_t addr, uint32_t lbo) { return (addr >> 4) | ((lbo >> 4) << 16); }
// Contraction along the rows' 64-wide halves (128 rows); the step to the
// 16-wide slice k16.
__device__ __forceinline__ uint32_t kmajor(uint32_t tile) { return sdesc(tile, 16u); }
__device__ __forceinline__ constexpr uint32_t kstep(int k16) { return (kHalf * (k16 >> 2) + 32u * (k16 & 3)) >> 4; }
// Contraction down the rows; `half` bytes between 64-wide groups of columns.
__device__ __forceinline__ uint32_t mnmajor(uint32_t tile, uint32_t half) { return sdesc(tile, half); }
__device__ __forceinline__ constexpr uint32_t mnstep(int k16) { return 2048u * k16 >> 4; }
// Instruction descriptor: bf16 x bf16 -> f32, M x N, operand majors, A negated.
constexpr uint32_t kNegateA = 1u << 13;
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
// Pairs of bfloat16, each operation rounded once.
__device__ __forceinline__ uint32_t mulb(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ uint32_t fmab(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t d;
  asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
  return d;
}
__device__ __forceinline__ uint32_t pack2(f2 v) {
  const float2 f = unpair(v);
  return pack2(f.x, f.y);
}
__device__ __forceinline__ f2 pair_at(const uint32_t *r) { return pair(__uint_as_float(r[0]), __uint_as_float(r[1])); }
// lam^n for n >= 0 (1 for n = 0 whatever lam is); g2 = log_decay log2(e).
__device__ __forceinline__ float power(float g2, int n) { return n == 0 ? 1.f : ex2(g2 * (float)n); }

// ------------------------------------------------------------- the pass ---
// Shared memory: the state's bfloat16 copy, a buffer for the weighted keys (a
// second term takes b's place), and a ring of tiles that the chunks' a, b and c
// pass through in this order.  The order decides which tile waits for which
// slot: with five slots c waits for the a of the chunk before it, a and b for b
// and c of the one before that.  With X = 64 the state's products run with
// M = 128: their rows from 64 on are the bytes behind the keys (there always
// are some; TWO: the keys again) and their results are not read.
//
// TWO (X = Y = 64): two CTAs on an SM, each with half of its shared memory,
// tensor memory and registers, so that one's chain of steps fills the other's
// waits; the rule for it is at the launch.
template <int XP, int YP, bool OUT, bool TWO>
struct Tiles {
  static constexpr uint32_t BT = XP / 64 * kHalf, CT = YP / 64 * kHalf, RT = OUT ? YP / 64 * XP * 128 : 0;
  static constexpr uint32_t SLOT = BT > CT ? BT : CT;
  static constexpr uint32_t MOST = TWO ? 104 * 1024 : 224 * 1024;
  static constexpr int FIT = (int)((MOST - BT - RT) / SLOT), NS = FIT < kMostSlots ? FIT : kMostSlots;
  static constexpr int PER = OUT ? 3 : 2;  // tiles of a chunk: (a,) b, c
  static constexpr uint32_t R = 0, W = RT, RING = W + BT, BYTES = RING + NS * SLOT;
  static_assert(NS >= 5 && BYTES <= MOST, "the ring holds a chunk and more; the rows behind a b of the last slot exist");
  static_assert(XP == 128 || TWO || SLOT > BT || BYTES + BT <= MOST, "");
};

// Columns of tensor memory.  TWO: O1 (P c) lies between P's halves, where
// scores were, so that two CTAs' share is enough.
template <int YP, bool TWO>
struct Cols {
  static constexpr uint32_t SCORES = 0, O1 = TWO ? 32 : 128, O2 = TWO ? 128 : 128 + YP, ST = O2 + YP, ALL = TWO ? 256 : 512;
  static_assert(ST + YP <= ALL && (!TWO || YP == 64), "");
};

struct Bars {
  uint64_t full[kMostSlots], empty[kMostSlots];  // ring slots
  uint64_t scores;             // a b^T complete (MMA)
  uint64_t p_ready;            // P in tensor memory (P warpgroups)
  uint64_t w_full[2];          // first and second term of the weighted keys in place (key warpgroup)
  uint64_t w_free;             // the first term's products complete (MMA)
  uint64_t c_clean;            // c's rows behind the last position zeroed (key warpgroup; a segment has one such chunk)
  uint64_t state;              // a R and all products into the state complete (MMA)
  uint64_t r_ready;            // the state's copy in shared memory, the state decayed in tensor memory (state warpgroup)
  uint64_t o_done;             // outputs complete in tensor memory (MMA)
  uint64_t o_free;             // outputs read (output warpgroup)
  uint64_t drain;              // every MMA complete
  uint32_t tmem;
  alignas(16) float up[32];  // lam^r, lam^{31-r}; read four at a time
  alignas(16) float down[32];
};
constexpr int kKeyThreads = 128;
// Warps of a CTA: 4 state, (4 outputs, 8 P,) 4 keys, loads, MMAs; TWO: 2 state,
// loads, MMAs, 4 P and outputs, 4 keys.  Their hot
// loops are kept short: one that does not fit the instruction cache with the
// others waits for its instructions, chunk after chunk.  Nor may a register
// spill: shared memory takes L1's place and a reload is a trip to L2.
template <bool OUT, bool TWO>
struct Roles {
  static constexpr int STATE = TWO ? 2 : 4, SCORES = TWO ? 4 : 8, KEYS = TWO ? 8 : OUT ? 16 : 4;
  static constexpr int LOAD = TWO ? 2 : KEYS + 4, MMA = LOAD + 1, THREADS = TWO ? 384 : 32 * (MMA + 1);
};

// Waits for the phase of the barrier at `addr` with the given parity, in at
// most `tries` tries (each is suspended by the hardware for a while).
__device__ __forceinline__ bool spin(uint32_t addr, uint32_t parity, uint32_t tries) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p, q;\n .reg .u32 n;\n mov.u32 n, %3;\n"
      "TRY%=:\n"
      " mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n @p bra DONE%=;\n"
      " sub.u32 n, n, 1;\n setp.ne.u32 q, n, 0;\n @q bra TRY%=;\n"
      "DONE%=:\n selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(ok)
      : "r"(addr), "r"(parity), "r"(tries)
      : "memory");
  return ok != 0;
}
__device__ __forceinline__ void gave_up(const Waits &w) {
  if (w.status) *w.status = WKV_ERR_TIMEOUT;
}
// The same for a whole warp; a wait that gives up ends its role.
__device__ __forceinline__ bool wait_warp(uint64_t &bar, uint32_t parity, const Waits &w) {
  const bool ok = __all_sync(~0u, spin(smem_addr(&bar), parity, w.tries));
  if (!ok) gave_up(w);
  return ok;
}
// One arrival for a whole warp, behind what its lanes have done.
__device__ __forceinline__ void arrive_warp(uint64_t &bar) {
  __syncwarp();
  asm volatile(
      "{\n .reg .pred p;\n .reg .b64 s;\n setp.eq.u32 p, %1, 0;\n @p mbarrier.arrive.shared::cta.b64 s, [%0];\n}\n" ::"r"(
          smem_addr(&bar)),
      "r"(threadIdx.x & 31u)
      : "memory");
}

// A place in the ring of NS tiles.
template <int NS>
struct Place {
  int slot = 0;
  uint32_t phase = 0;
  __device__ __forceinline__ Place next() const { return slot == NS - 1 ? Place{0, phase ^ 1u} : Place{slot + 1, phase}; }
};

// The chunks of this CTA's segment, in the pass's order.
struct Chunks {
  int t0, t1;  // the segment's valid positions
  int n;       // chunks with valid positions
  bool reverse;
  __device__ __forceinline__ int start(int it) const { return t0 + (reverse ? n - 1 - it : it) * kL; }
  __device__ __forceinline__ int valid(int it) const { return min(kL, t1 - start(it)); }
};

// State warpgroup: R at the chunk's start -> its bfloat16 copy in shared memory
// and, decayed, tensor memory again.  A thread is a row of the state.
template <int XP, int YP, bool OUT, bool TWO>
__device__ __forceinline__ void state_role(const Pass &p, const Waits &lim, Bars *s, uint8_t *sm, const Chunks &ch,
                                           int64_t unit, float g, float *result) {
  using Ti = Tiles<XP, YP, OUT, TWO>;
  const int x = threadIdx.x, warp = x >> 5;
  const int64_t bh = unit / p.nseg;
  const uint32_t tm = s->tmem + Cols<YP, TWO>::ST + ((uint32_t)(32 * warp) << 16);
  const bool rows = 32 * warp < XP;  // this warp's lanes hold state rows
  const int64_t XY = (int64_t)p.X * p.Y;
  const float *init = !OUT ? nullptr : p.nseg > 1 ? p.seg + unit * XY : p.s_in ? p.s_in + bh * XY : nullptr;
  const bool init_t = p.nseg == 1 && p.s_in_t;
  auto load_row = [&](int yb, uint32_t(&v)[32]) {
    if (!init || x >= p.X) {
#pragma unroll
      for (int q = 0; q < 32; ++q) v[q] = 0u;
    } else if (init_t) {
#pragma unroll
      for (int q = 0; q < 32; ++q) v[q] = yb + q < p.Y ? __float_as_uint(init[(int64_t)(yb + q) * p.X + x]) : 0u;
    } else {
      const uint4 *src = reinterpret_cast<const uint4 *>(init + (int64_t)x * p.Y + yb);
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        const uint4 f = yb + 4 * q < p.Y ? src[q] : make_uint4(0u, 0u, 0u, 0u);
        v[4 * q] = f.x, v[4 * q + 1] = f.y, v[4 * q + 2] = f.z, v[4 * q + 3] = f.w;
      }
    }
  };
  if (OUT) {
    if (rows && ch.n > 0) {
#pragma unroll 1
      for (int yb = 0; yb < YP; yb += 32) {
        uint32_t v[32];
        load_row(yb, v);
        tmem_st32(tm + yb, v);
      }
      tmem_wait_st();
    }
#pragma unroll 1
    for (int it = 0; it < ch.n; ++it) {
      if (it > 0 && !wait_warp(s->state, (it - 1) & 1, lim)) return;
      if (rows) {
        const Decay d = decay_of(g, ch.valid(it));
        const f2 dm = both(d.m);
        tc_after_sync();
        tmem_each16(tm, 0, YP / 16, [&](int c, uint32_t(&v)[16]) {
              uint8_t *half = sm + Ti::R + (c >> 2) * (XP * 128);
#pragma unroll
              for (int u = 0; u < 2; ++u) {
                uint32_t *f = v + 8 * u;
                *reinterpret_cast<uint4 *>(half + sw128(x, 2 * (c & 3) + u)) =
                    make_uint4(pack2(pair_at(f)), pack2(pair_at(f + 2)), pack2(pair_at(f + 4)), pack2(pair_at(f + 6)));
#pragma unroll
                for (int q = 0; q < 8; q += 2) {  // decayed(), by pairs
                  const f2 z = pair_at(f + q);
                  const float2 r = unpair(fma2(z, dm, d.near_one ? z : 0ull));
                  f[q] = __float_as_uint(r.x), f[q + 1] = __float_as_uint(r.y);
                }
              }
              tmem_st16(tm + 16 * c, v);
            });
        tmem_wait_st();
        tc_before_sync();
        fence_proxy_async_smem();
      }
      arrive_warp(s->r_ready);
    }
  }
  if (!result || !rows) return;
  if (ch.n > 0) {
    if (!wait_warp(s->state, OUT ? (ch.n - 1) & 1 : 0, lim)) return;
    tc_after_sync();
  }
#pragma unroll 1
  for (int yb = 0; yb < YP; yb += 32) {
    uint32_t v[32];
    if (ch.n > 0) {
      tmem_ld32_nowait(tm + yb, v);
      tmem_wait_ld();
      pin(v);
    } else {
      load_row(yb, v);  // no positions: the state goes through
    }
    float *dst = result + (int64_t)x * p.Y + yb;
#pragma unroll
    for (int q = 0; q < 8; ++q)
      if (x < p.X && yb + 4 * q < p.Y) reinterpret_cast<uint4 *>(dst)[q] = make_uint4(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]);
    __syncwarp();
  }
}

// Key warpgroup: lam^n b as two bfloat16 terms, the second in b's place once
// its scores are formed; a thread has a row (position).
template <int XP, int YP, bool OUT, bool TWO>
__device__ __forceinline__ void keys_role(const Pass &p, const Waits &lim, Bars *s, uint8_t *sm, const Chunks &ch, float g2,
                                          bool more) {
  using Ti = Tiles<XP, YP, OUT, TWO>;
  const int j = threadIdx.x - 32 * Roles<OUT, TWO>::KEYS;
  Place<Ti::NS> place;
  // One term: f of every pair of the tile at src.
  auto convert = [&](const uint8_t *src, uint8_t *dst, uint64_t &full, auto f) {
#pragma unroll 1
    for (uint32_t o = 0; o < Ti::BT; o += kHalf) {
#pragma unroll
      for (int v = 0; v < 8; v += 4) {
        uint4 x[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) x[u] = *reinterpret_cast<const uint4 *>(src + o + sw128(j, v + u));
#pragma unroll
        for (int u = 0; u < 4; ++u)
          *reinterpret_cast<uint4 *>(dst + o + sw128(j, v + u)) = make_uint4(f(x[u].x), f(x[u].y), f(x[u].z), f(x[u].w));
      }
    }
    fence_proxy_async_smem();
    arrive_warp(full);
  };
#pragma unroll 1
  for (int it = 0; it < ch.n; ++it) {
    const int nv = ch.valid(it);
    const Place<Ti::NS> b = OUT ? place.next() : place, c = b.next();
    place = c.next();
    const bool wanted = more || it + 1 < ch.n;
    uint8_t *src = sm + Ti::RING + b.slot * Ti::SLOT, *dst = sm + Ti::W;
    if (wanted && !wait_warp(s->full[b.slot], b.phase, lim)) return;
    if (nv < kL) {  // rows behind the last position may hold anything: 0 x anything has to be 0
      if (!wait_warp(s->full[c.slot], c.phase, lim)) return;
      uint8_t *tc = sm + Ti::RING + c.slot * Ti::SLOT;
      if (j >= nv) {
#pragma unroll 1
        for (int u = 0; u < 8; ++u) {
          for (uint32_t o = 0; o < Ti::BT && wanted; o += kHalf) *reinterpret_cast<uint4 *>(src + o + sw128(j, u)) = make_uint4(0u, 0u, 0u, 0u);
          for (uint32_t o = 0; o < Ti::CT; o += kHalf) *reinterpret_cast<uint4 *>(tc + o + sw128(j, u)) = make_uint4(0u, 0u, 0u, 0u);
        }
      }
      fence_proxy_async_smem();
      arrive_warp(s->c_clean);
    }
    if (!wanted) return;
    const int n = p.reverse ? j + 1 + (OUT ? 0 : ch.start(it) - ch.t0) : (OUT ? nv : ch.t1 - ch.start(it)) - 1 - j;
    const float w = j < nv ? p.sk * power(g2, n) : 0.f;
    // the weight in two bfloat16 parts: the first term is w1 b rounded; the
    // second, negated (the products subtract it), what that leaves (exact in
    // bfloat16) plus w2 b, rounded once
    const uint32_t w1 = pack2(w, w), w2 = pack2(w - lo16(w1), w - lo16(w1)), m1 = w1 ^ 0x80008000u, m2 = w2 ^ 0x80008000u;
    if (it > 0 && !wait_warp(s->w_free, (it - 1) & 1, lim)) return;
    convert(src, dst, s->w_full[0], [&](uint32_t x) { return mulb(w1, x); });
    if (OUT && !wait_warp(s->scores, it & 1, lim)) return;
    convert(src, src, s->w_full[1], [&](uint32_t x) { return fmab(m2, x, fmab(m1, x, mulb(w1, x))); });
  }
}

// P warpgroups: the masked, weighted scores, rounded to bfloat16, in tensor
// memory over the scores' own columns; a thread has a row and half its columns
// (TWO: all of them), and the halves' P lies at columns 0 and 64 (TWO: 96).
template <bool TWO>
struct Scores {
  const Pass &p;
  const Waits &lim;
  float g2, f;
  int w, lane, half;
  uint32_t tm;
  __device__ __forceinline__ Scores(const Pass &p, const Waits &lim, const Bars *s, float g2)
      : p(p), lim(lim), g2(g2), f(p.si * p.sk) {
    const int t = threadIdx.x & 255;
    w = (t >> 5) & 3, lane = t & 31, half = TWO ? 0 : t >> 7;
    tm = s->tmem + ((uint32_t)(32 * w) << 16);
  }
  __device__ __forceinline__ bool chunk(Bars *s, const Chunks &ch, int it) const {
    const bool moderate = g2 * 31.f > -100.f && fabsf(f) < 0x1p27f;  // their product below 2^127
    const uint32_t causal = p.reverse ? ~0u << lane : (2u << lane) - 1u;  // columns of the diagonal block that count
    const float *tab = p.reverse ? s->up : s->down;
    const int nv = ch.valid(it);
    if (!wait_warp(s->scores, it & 1, lim)) return false;
    tc_after_sync();
    // blocks of 32 columns; the P of two, 16 columns each, lies where the first's
    // scores were, which are read by then (or not needed)
#pragma unroll 1
    for (int k = 0; k < (TWO ? 4 : 2); ++k) {
      const int cb = TWO ? k ^ (k >> 1) : 2 * half + k;  // TWO: 0, 1, 3, 2
      uint32_t out[16];
      if (p.reverse ? cb < w || 32 * cb >= nv : cb > w) {
#pragma unroll
        for (int r = 0; r < 16; ++r) out[r] = 0u;
      } else {
        uint32_t v[32];
        tmem_ld32_nowait(tm + 32 * cb, v);
        // lam^{|i-j|} as a factor of the row and one of the column; on the
        // diagonal the row's is up to f lam^{-31}, so strong decays and large
        // scales take the product from a table there
        const int i = 32 * (w - cb) + lane;
        const f2 e = both(f * ex2(g2 * (float)(p.reverse ? -i : i - 31)));
        tmem_wait_ld();
        pin(v);
        if (cb == w || 32 * cb + 32 > nv) {
          uint32_t keep = cb == w ? causal : ~0u;
          if (32 * cb + 32 > nv) keep &= nv > 32 * cb ? (1u << (nv - 32 * cb)) - 1u : 0u;  // what lies behind the last position may be anything
#pragma unroll
          for (int r = 0; r < 32; ++r) v[r] = (keep >> r) & 1u ? v[r] : 0u;
        }
        if (cb == w && !moderate) {
#pragma unroll
          for (int r = 0; r < 16; ++r) {
            const int n0 = p.reverse ? 2 * r - lane : lane - 2 * r, n1 = p.reverse ? n0 + 1 : n0 - 1;
            out[r] = pack2(__uint_as_float(v[2 * r]) * (f * s->up[max(n0, 0)]),
                           __uint_as_float(v[2 * r + 1]) * (f * s->up[max(n1, 0)]));
          }
        } else {
#pragma unroll
          for (int q = 0; q < 8; ++q) {
            const ulonglong2 z = *reinterpret_cast<const ulonglong2 *>(tab + 4 * q);
            out[2 * q] = pack2(mul2(pair_at(v + 4 * q), mul2(e, z.x)));
            out[2 * q + 1] = pack2(mul2(pair_at(v + 4 * q + 2), mul2(e, z.y)));
          }
        }
      }
      tmem_st16(tm + (TWO ? 16 * cb + (cb >> 1) * 64 : 64 * half + 16 * k), out);
    }
    tmem_wait_st();
    tc_before_sync();
    arrive_warp(s->p_ready);
    return true;
  }
};

// Output warpgroup, a thread per row: P c + weight x (a R), rounded and stored
// as 16- or 32-byte pieces of the row.
template <int YP, bool TWO>
struct Outputs {
  const Pass &p;
  const Waits &lim;
  float g2;
  bool wide;
  uint32_t tm;
  uint16_t *row;  // of position 0
  __device__ __forceinline__ Outputs(const Pass &p, const Waits &lim, const Bars *s, int64_t b, int64_t h, float g2,
                                     bool wide)
      : p(p), lim(lim), g2(g2), wide(wide), tm(s->tmem + ((threadIdx.x & 96u) << 16)),
        row(static_cast<uint16_t *>(const_cast<void *>(p.o.p)) + b * p.o.sb + h * p.o.sh) {}
  __device__ __forceinline__ bool chunk(Bars *s, const Chunks &ch, int it) const {
    constexpr uint32_t O1 = Cols<YP, TWO>::O1, O2 = Cols<YP, TWO>::O2;
    const int i = threadIdx.x & 127, nv = ch.valid(it);
    const f2 w = both(i < nv ? p.si * power(g2, p.reverse ? nv - 1 - i : i + 1) : 0.f);
    const int64_t t = (int64_t)ch.start(it) + i;
    uint16_t *dst = row + t * p.o.st;
    if (!wait_warp(s->o_done, it & 1, lim)) return false;
    tc_after_sync();
    uint32_t o1[16], o2[16], z[8];
    tmem_ld16_nowait(tm + O1, o1);
    tmem_ld16_nowait(tm + O2, o2);
#pragma unroll 1
    for (int y = 0; y < YP; y += 16) {
      tmem_wait_ld();
      pin(o1);
      pin(o2);
#pragma unroll
      for (int r = 0; r < 8; ++r) {
        z[r] = pack2(fma2(w, pair_at(o2 + 2 * r), pair_at(o1 + 2 * r)));
      }
      if (nv < kL) {
#pragma unroll
        for (int r = 0; r < 8; ++r) z[r] = i < nv ? z[r] : 0u;
      }
      if (y < YP - 16) {
        tmem_ld16_nowait(tm + O1 + y + 16, o1);
        tmem_ld16_nowait(tm + O2 + y + 16, o2);
      } else {
        tc_before_sync();
        arrive_warp(s->o_free);
      }
      if (t < p.T && wide) {
        if (y < p.Y)
          asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst + y), "r"(z[0]), "r"(z[1]),
                       "r"(z[2]), "r"(z[3]), "r"(z[4]), "r"(z[5]), "r"(z[6]), "r"(z[7])
                       : "memory");
      } else if (t < p.T) {
        if (y < p.Y) *reinterpret_cast<uint4 *>(dst + y) = make_uint4(z[0], z[1], z[2], z[3]);
        if (y + 8 < p.Y) *reinterpret_cast<uint4 *>(dst + y + 8) = make_uint4(z[4], z[5], z[6], z[7]);
      }
      __syncwarp();
    }
    return true;
  }
};

// Loads: the tiles of each chunk in the ring's order, each as soon as its slot
// is free; one whole warp.
template <int XP, int YP, bool OUT, bool TWO>
__device__ __forceinline__ void load_role(const Pass &p, const Waits &lim, Bars *s, uint32_t sm, const Chunks &ch, int b,
                                          int h, const CUtensorMap *am, const CUtensorMap *bm, const CUtensorMap *cm) {
  using Ti = Tiles<XP, YP, OUT, TWO>;
  Place<Ti::NS> place;
  int n = 0;  // tiles whose loads were issued
  bool ok = true;
#pragma unroll 1
  for (int it = 0; it < ch.n && ok; ++it) {
    const int t = ch.start(it);
#pragma unroll 1
    for (int k = 0; k < Ti::PER; ++k) {
      const int slot = place.slot;
      if (n >= Ti::NS && !(ok = wait_warp(s->empty[slot], place.phase ^ 1u, lim))) break;
      const bool is_c = k == Ti::PER - 1;
      const CUtensorMap *m = is_c ? cm : k == Ti::PER - 2 ? bm : am;
      const uint32_t bytes = is_c ? Ti::CT : Ti::BT, dst = sm + Ti::RING + slot * Ti::SLOT, bar = smem_addr(&s->full[slot]);
      if (elect_one()) {
        mbar_expect_tx(bar, bytes);
        for (uint32_t o = 0; o < bytes; o += kHalf) tma_load_4d(dst + o, m, (int)(o / kHalf) * 64, t, h, b, bar);
      }
      __syncwarp();
      ++n;
      place = place.next();
    }
  }
  // The loads in flight write shared memory that outlives this warp, not the
  // CTA: every one is waited for (in order to end; consumers wait for theirs).
  for (int k = max(0, n - Ti::NS); k < n; ++k)
    ok = spin(smem_addr(&s->full[k % Ti::NS]), (k / Ti::NS) & 1, kTries) && ok;
  if (!ok) gave_up(lim);
}

// MMAs, in the order that the head of this file explains; one whole warp.
template <int XP, int YP, bool OUT, bool TWO>
__device__ __forceinline__ void mma_role(const Pass &p, const Waits &lim, Bars *s, uint32_t sm, const Chunks &ch,
                                         bool more) {
  using Ti = Tiles<XP, YP, OUT, TWO>;
  using Co = Cols<YP, TWO>;
  constexpr uint32_t SCORES = Co::SCORES, O1 = Co::O1, O2 = Co::O2, ST = Co::ST;
  const uint32_t tm = __shfl_sync(~0u, s->tmem, 0);
  auto loaded = [&](const Place<Ti::NS> &t) { return wait_warp(s->full[t.slot], t.phase, lim); };
  auto tile = [&](const Place<Ti::NS> &t) { return sm + Ti::RING + t.slot * Ti::SLOT; };
  Place<Ti::NS> place;
  bool ok = true;
  struct {
    int scores, keys, states, outputs, tiles;
  } done = {};  // commits to each of the barriers; tiles are freed in the ring's order
#pragma unroll 1
  for (int it = 0; it < ch.n; ++it) {
    const uint32_t ph = it & 1;
    const Place<Ti::NS> na = place, nb = OUT ? na.next() : na, nc = nb.next();
    place = nc.next();
    const uint32_t ta = tile(na), tb = tile(nb), tc = tile(nc);
    const int n_terms = more || it + 1 < ch.n ? 2 : 0;
    if (OUT) {
      if (!(ok = loaded(na) && loaded(nb))) break;
      if (TWO && it > 0) {  // the scores' columns hold O1
        if (!(ok = wait_warp(s->o_free, ph ^ 1u, lim))) break;
        tc_after_sync();
      }
      if (elect_one()) {
        const uint32_t da = kmajor(ta), db = kmajor(tb);
#pragma unroll
        for (int k = 0; k < XP / 16; ++k) mma_ss(tm + SCORES, da + kstep(k), db + kstep(k), idesc(128, 128, false, false), k > 0);
        mma_commit(smem_addr(&s->scores));
      }
      __syncwarp();
      ++done.scores;
      if (!(ok = wait_warp(s->r_ready, ph, lim))) break;
    }
    if (!(ok = loaded(nc))) break;
    if (ch.valid(it) < kL && !(ok = wait_warp(s->c_clean, 0, lim))) break;
    // the keys' terms, and a R behind the first of them
#pragma unroll 1
    for (int k = 0; k < max(n_terms, 1); ++k) {
      if (n_terms > 0) {
        if (!(ok = wait_warp(s->w_full[k], ph, lim))) break;
        tc_after_sync();
        if (elect_one()) {
          const uint32_t dw = mnmajor(k == 0 ? sm + Ti::W : tb, TWO ? 0u : kHalf), dc = mnmajor(tc, kHalf);
          const bool acc = OUT || it > 0 || k > 0;
          const uint32_t id = idesc(128, YP, true, true) | (k > 0 ? kNegateA : 0u);
#pragma unroll
          for (int i = 0; i < kL / 16; ++i)
            mma_ss(tm + ST, dw + mnstep(i), dc + mnstep(i), id, acc || i > 0);
          if (k == 0) mma_commit(smem_addr(&s->w_free));
        }
        __syncwarp();
        if (k == 0) ++done.keys;
      }
      if (OUT && k == 0) {
        if (!TWO && it > 0 && !(ok = wait_warp(s->o_free, ph ^ 1u, lim))) break;
        tc_after_sync();
        if (elect_one()) {
          const uint32_t da = kmajor(ta), dr = mnmajor(sm + Ti::R, XP * 128);
#pragma unroll
          for (int i = 0; i < XP / 16; ++i)
            mma_ss(tm + O2, da + kstep(i), dr + mnstep(i), idesc(128, YP, false, true), i > 0);
          mma_commit(smem_addr(&s->empty[na.slot]));
        }
        __syncwarp();
        ++done.tiles;
      }
    }
    if (!ok) break;
    const bool state_done = n_terms > 0 && (OUT || it + 1 == ch.n);
    if (elect_one()) {
      // b is free once its scores are formed and its keys read, or multiplied
      mma_commit(smem_addr(&s->empty[nb.slot]));
      if (state_done) mma_commit(smem_addr(&s->state));
    }
    __syncwarp();
    ++done.tiles;
    done.states += state_done;
    if (OUT) {
      if (!(ok = wait_warp(s->p_ready, ph, lim))) break;
      tc_after_sync();
    }
    if (elect_one()) {
      if (OUT) {
        const uint32_t dc = mnmajor(tc, kHalf);
#pragma unroll
        for (int k = 0; k < kL / 16; ++k)
          mma_ts(tm + O1, tm + SCORES + 8 * k + (k >= 4 ? (TWO ? 64 : 32) : 0), dc + mnstep(k), idesc(128, YP, false, true), k > 0);
        mma_commit(smem_addr(&s->o_done));
      }
      mma_commit(smem_addr(&s->empty[nc.slot]));
    }
    __syncwarp();
    ++done.tiles;
    done.outputs += OUT;
  }
  // Nothing may be under way when the CTA ends.  MMAs in flight read shared
  // memory and write tensor memory, and a commit arrives on a barrier in shared
  // memory, which is the SM's next CTA's by then: an arrival too many there ends
  // a phase early.  So the last arrival of every barrier that MMAs complete is
  // waited for here, whether or not a role waits for it too.
  if (elect_one()) {
    mma_commit(smem_addr(&s->drain));
    bool ended = spin(smem_addr(&s->drain), 0, kTries);
    auto last_of = [&](uint64_t &bar, int n) {
      ended = (n == 0 || spin(smem_addr(&bar), (n - 1) & 1, kTries)) && ended;
    };
    last_of(s->scores, done.scores);
    last_of(s->w_free, done.keys);
    last_of(s->state, done.states);
    last_of(s->o_done, done.outputs);
    for (int k = max(0, done.tiles - Ti::NS); k < done.tiles; ++k)
      ended = spin(smem_addr(&s->empty[k % Ti::NS]), (k / Ti::NS) & 1, kTries) && ended;
    if (!ended) gave_up(lim);
  }
}

struct Maps {
  CUtensorMap a[3], b[3], c[3];
  int wide[3];
};
// Zeros in the chunks without valid positions.  (The block's place is read
// anew: nothing of this stays in registers while the roles run.)
__device__ __forceinline__ void zero_padding(const Group &group) {
  uint32_t block;
  asm volatile("mov.u32 %0, %%ctaid.x;" : "=r"(block));
  const Pass &p = group.p[block % (unsigned)group.n];
  const int64_t unit = block / (unsigned)group.n, bh = unit / p.nseg, t0 = unit % p.nseg * p.seg_len, b = bh / p.H;
  const int64_t tz = min(t0 + p.seg_len, p.T), t1 = max(t0, min(tz, row_len(p, b)));
  const int64_t z0 = min(t0 + (t1 - t0 + kL - 1) / kL * kL, tz);
  const int units = p.Y / 8;
  uint16_t *dst = static_cast<uint16_t *>(const_cast<void *>(p.o.p)) + b * p.o.sb + bh % p.H * p.o.sh;
#pragma unroll 1
  for (int64_t e = threadIdx.x; e < (tz - z0) * units; e += blockDim.x)
    reinterpret_cast<uint4 *>(dst + (z0 + e / units) * p.o.st)[e % units] = make_uint4(0u, 0u, 0u, 0u);
}

// A block is a segment of a head of one pass; the passes of a segment are
// neighbours, so that those that read the same tensors find them in L2.
template <int XP, int YP, bool OUT, bool TWO>
__global__ void __launch_bounds__(Roles<OUT, TWO>::THREADS, TWO ? 2 : 1) decay_tc_kernel(const __grid_constant__ Maps maps,
                                                                                         const __grid_constant__ Group group) {
  using Ro = Roles<OUT, TWO>;
  const int pass = (int)(blockIdx.x % (unsigned)group.n);
  const int64_t unit = blockIdx.x / (unsigned)group.n;
  const Pass &p = group.p[pass];
  const CUtensorMap &am = maps.a[pass], &bm = maps.b[pass], &cm = maps.c[pass];
  const int wide = maps.wide[pass];
  const int64_t bh = unit / p.nseg, sg = unit % p.nseg, b = bh / p.H, h = bh % p.H;
  const bool last = sg == (p.reverse ? 0 : p.nseg - 1);  // of the pass's segments
  if (!OUT && last) return;                              // no state starts from its sum
  // Where the state after the segment goes; if nowhere, the last chunk adds nothing to it.
  const int64_t XY = (int64_t)p.X * p.Y;
  float *result = !OUT ? p.seg + unit * XY : last && p.s_out ? p.s_out + bh * XY : nullptr;
  extern __shared__ uint8_t smem_raw[];
  __shared__ Bars bars;
  uint8_t *sm = smem_raw + (((smem_addr(smem_raw) + 1023u) & ~1023u) - smem_addr(smem_raw));
  const int64_t n = row_len(p, b);
  Chunks ch;
  const int64_t t0 = sg * p.seg_len, tz = min(t0 + p.seg_len, p.T);  // segments are whole chunks
  // (through a shuffle: the compiler then knows that the loops are the same in all lanes)
  ch.t0 = (int)t0;
  ch.t1 = __shfl_sync(~0u, (int)max(t0, min(tz, n)), 0);
  ch.n = (ch.t1 - ch.t0 + kL - 1) / kL;
  ch.reverse = p.reverse;
  const float g = p.log_decay[h], g2 = g * kLog2e;
  const int warp = __shfl_sync(~0u, (int)(threadIdx.x >> 5), 0);
  if (threadIdx.x == 0) {
    for (int i = 0; i < kMostSlots; ++i) mbar_init(smem_addr(&bars.full[i]), 1), mbar_init(smem_addr(&bars.empty[i]), 1);
    for (uint64_t *f : {&bars.scores, &bars.w_free, &bars.state, &bars.o_done, &bars.drain})
      mbar_init(smem_addr(f), 1);
    // (held: keys and P are waited for, and one arrival too few comes)
    const int held = blockIdx.x == 0 && group.w.hold ? 1 : 0;
    mbar_init(smem_addr(&bars.w_full[0]), kKeyThreads / 32 + held);
    mbar_init(smem_addr(&bars.w_full[1]), kKeyThreads / 32);
    mbar_init(smem_addr(&bars.c_clean), kKeyThreads / 32);
    mbar_init(smem_addr(&bars.p_ready), Ro::SCORES + held);
    mbar_init(smem_addr(&bars.o_free), 4);
    mbar_init(smem_addr(&bars.r_ready), Ro::STATE);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (threadIdx.x >= 32 && threadIdx.x < 64) {
    const int r = threadIdx.x - 32;
    bars.up[r] = power(g2, r);
    bars.down[r] = power(g2, 31 - r);
  }
  if (warp == 0) tmem_alloc(smem_addr(&bars.tmem), Cols<YP, TWO>::ALL);
  tc_before_sync();
  __syncthreads();
  tc_after_sync();
  if (warp < Ro::STATE) {
    state_role<XP, YP, OUT, TWO>(p, group.w, &bars, sm, ch, unit, g, result);
  } else if (warp == Ro::LOAD) {
    load_role<XP, YP, OUT, TWO>(p, group.w, &bars, smem_addr(sm), ch, (int)b, (int)h, &am, &bm, &cm);
  } else if (warp == Ro::MMA) {
    mma_role<XP, YP, OUT, TWO>(p, group.w, &bars, smem_addr(sm), ch, result != nullptr);
  } else if (warp >= Ro::KEYS) {
    keys_role<XP, YP, OUT, TWO>(p, group.w, &bars, sm, ch, g2, result != nullptr);
  } else if constexpr (TWO) {
    const Scores<TWO> scores(p, group.w, &bars, g2);
    const Outputs<YP, TWO> outputs(p, group.w, &bars, b, h, g2, wide != 0);
#pragma unroll 1
    for (int it = 0; it < ch.n; ++it)
      if (!scores.chunk(&bars, ch, it) || !outputs.chunk(&bars, ch, it)) break;
  } else if constexpr (OUT) {
    if (warp < 8) {
      const Outputs<YP, TWO> outputs(p, group.w, &bars, b, h, g2, wide != 0);
#pragma unroll 1
      for (int it = 0; it < ch.n; ++it)
        if (!outputs.chunk(&bars, ch, it)) break;
    } else {
      const Scores<TWO> scores(p, group.w, &bars, g2);
#pragma unroll 1
      for (int it = 0; it < ch.n; ++it)
        if (!scores.chunk(&bars, ch, it)) break;
    }
  }
  __syncwarp();
  if (OUT) zero_padding(group);
  tc_before_sync();
  __syncthreads();
  if (warp == 0) {
    tc_after_sync();
    tmem_dealloc(bars.tmem, Cols<YP, TWO>::ALL);
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
  auto fits = [&](int64_t s, int64_t n) { return n <= 1 || (s % 8 == 0 && (!tma || (s > 0 && s < (int64_t(1) << 39)))); };
  return ((uintptr_t)v.p & 15u) == 0 && fits(v.sb, p.B) && fits(v.st, p.T) && fits(v.sh, p.H);
}
template <int XP, int YP, bool OUT, bool TWO = false>
cudaError_t launch_t(const Group &g, cudaStream_t st) {
  Maps m{};
  if (!encoder() || !ensure_context()) return cudaErrorNotSupported;
  const auto kern = decay_tc_kernel<XP, YP, OUT, TWO>;
  constexpr int smem = (int)Tiles<XP, YP, OUT, TWO>::MOST + 1024;
  int blocks = 0;
  const cudaError_t e = blocks_per_sm((const void *)kern, Roles<OUT, TWO>::THREADS, smem, &blocks);
  if (e != cudaSuccess) return e;
  if (blocks < 1) return cudaErrorInvalidConfiguration;
  auto even = [](int64_t s, int64_t n) { return n <= 1 || s % 16 == 0; };
  for (int i = 0; i < g.n; ++i) {
    const Pass &p = g.p[i];
    if ((OUT && !encode(&m.a[i], p.a, p, p.X)) || !encode(&m.b[i], p.b, p, p.X) || !encode(&m.c[i], p.c, p, p.Y))
      return cudaErrorInvalidValue;
    m.wide[i] = OUT && ((uintptr_t)p.o.p & 31u) == 0 && p.Y % 16 == 0 && even(p.o.sb, p.B) && even(p.o.st, p.T) &&
                even(p.o.sh, p.H);
  }
  const Pass &p = g.p[0];
  return launch_kernel(kern, dim3((unsigned)(p.B * p.H * p.nseg * g.n)), dim3(Roles<OUT, TWO>::THREADS), smem, st, m, g);
}
// Time of the output launch when an SM has `units` CTAs of heads up to 64 to run,
// in chunks of a CTA alone on its SM (2.2 us each): one after the other with 22
// warps, or, with 12, two at a time (4.0 us for a chunk of each; 3.15 for the odd
// one's).  Forward, 4096 positions: 2 units 140 us and 128, 3 units 201 and 229;
// 2048 positions, 4 units: 151 and 130; 1024 positions, 6 units: 123 and 99.
double unit_time(int64_t units, bool two) { return two ? 1.82 * (double)(units / 2) + 1.43 * (double)(units % 2) : (double)units; }
bool pairs(int64_t units) { return unit_time(units, true) < unit_time(units, false); }
template <bool OUT>
cudaError_t launch_o(const Group &g, int sms, cudaStream_t st) {
  const int64_t units = (g.p[0].B * g.p[0].H * g.p[0].nseg * g.n + sms - 1) / sms;
  const int X = g.p[0].X, Y = g.p[0].Y;
  if constexpr (OUT)
    if (X <= 64 && Y <= 64 && pairs(units)) return launch_t<64, 64, OUT, true>(g, st);
  if (X <= 64) return Y <= 64 ? launch_t<64, 64, OUT>(g, st) : launch_t<64, 128, OUT>(g, st);
  return Y <= 64 ? launch_t<128, 64, OUT>(g, st) : launch_t<128, 128, OUT>(g, st);
}
}  // namespace

bool tc_fits(const Pass &p) {
  return p.X % 8 == 0 && p.Y % 8 == 0 && p.X <= 128 && p.Y <= 128 && rows16(p.a, p, true) && rows16(p.b, p, true) &&
         rows16(p.c, p, true) && rows16(p.o, p, false);
}
int64_t tc_segments(int64_t BH, int64_t T, int X, int Y, int npass, int sms) {
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
    const int64_t units = (BH * n + sms - 1) / sms;
    const double waves = (double)units, out = unit_time(units, X <= 64 && Y <= 64 && pairs(units));
    const double t = out * (per + 2.0) + (n > 1 ? waves * (0.6 * per + 2.0) + 2.0 : 0.0);
    if (t < least) least = t, best = n;
  }
  return best;
}
uint32_t tc_tries(int64_t us) { return us > 0 ? (uint32_t)std::min<int64_t>((us - 1) / kTryUs + 1, 1u << 30) : kTries; }
int64_t tc_segment_len(int64_t T, int64_t nseg) {
  const int64_t nch = (T + kL - 1) / kL;
  return (nch + nseg - 1) / nseg * kL;
}
cudaError_t launch_tc(const Group &g, bool sums_only, int sms, cudaStream_t st) {
  return sums_only ? launch_o<false>(g, sms, st) : launch_o<true>(g, sms, st);
}

}  // namespace decay
}  // namespace wkv
