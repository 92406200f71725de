// af_attn4_tc.cu -- attention of many query rows over the 4-bit key/value
// cache on the 5th-generation tensor cores (tcgen05, sm_100a).
//
// The query rows of all heads that share a key head are packed into one list,
// m = i * group + (head in group).  A CTA takes 256 of them (two groups of
// 128 rows) and one split of the sequence's keys, in tiles of 64.  With at
// most 128 packed rows both groups take the same rows and every other tile
// (PAIR), and their results are merged in shared memory at the end.
//
// The matrix products want bf16 operands, so keys and values are decoded once
// a CTA and tile, k = lo + n s in packed bf16 (one rounding), and used by both
// groups: 256 rows share the decoding.  Roles of the 32 warps (registers move
// from the others to the softmax warps, 4 x 80 + 2 x 56 + 2 x 40 = 8 x 64):
//   0-7, 8-15  softmax of group 0 / 1: two threads a query row, each with 32 of
//              a tile's 64 scores.  Q into shared memory at the start; per tile
//              the scores come from TMEM into registers and P = 2^(s - m) goes
//              back as bf16 over their columns.  m is not the running maximum:
//              the exponentials are taken with the m at hand and their sum is
//              looked at; only when it is above 2^9 (or m is not set) the two
//              warps of the rows take the maximum together, rescale O in TMEM
//              and do the tile again.  That bounds P as well as a maximum would
//              and needs neither its instructions nor an exchange between the
//              two threads, only a vote.  (One thread a row, with twice the
//              registers, had half as many warps to hide the latencies of TMEM,
//              exponentials and barriers behind.)
//   16-19, 20-23  decoding of K / of V: codes and parameters of a tile (bulk
//              copies, a ring of raw slots each) to swizzled bf16 operand tiles.
//   24         bulk copies of codes and parameters (contiguous in memory).
//   25, 26     MMA issue of group 0's / 1's S = Q K^T (M 128, N 64, K head_dim)
//   27, 28     and O += P V (M 128, N head_dim, K 64, P from TMEM).  A thread that
//              issues products is held until the tensor core takes them, so one
//              thread for both products left the tensor core idle.
// Scores have two buffers of 64 columns a group, so S of the next tile runs
// under this tile's exponentials.  (One buffer of 128 columns, whose next S has
// to wait for the P V of the P that lies in it, was slower although its S reads
// Q from shared memory half as often.)
//
// Keys at or past the last key that any row of the CTA attends are decoded as
// zeros (0 * NaN would reach every row through P V); scores that a row masks
// become -inf by selection, so what stands there does not matter.
// A barrier never completes a phase that someone has yet to wait for: S full,
// P ready and O done are kept per score buffer, whose next use needs all three.
// Measured, 16 heads of 128 channels: 8190 causal queries 302 us (910 TFLOP/s),
// 390 queries over 46800 keys 231 us (645; 122 of its two CTAs' 512 rows are no
// one's).  No pipe is full (tensor 39%, exponentials 41%, ALU 46%): what bounds it
// is issue, 63% of the cycles, of which about a quarter goes into waits, and the
// chain S -> P -> O of each group.  For the 8190 queries one score buffer of
// 128 columns and one thread a row took 516 us, two buffers of 64 took 438, issue
// by converged warps 428, two threads a row 299.
//
// Every wait is bounded; on expiry the CTA stops, waits for its copies and
// MMAs in flight, frees TMEM and reports ERR_ATTN_WAIT.
#include "af_cache4.cuh"
#include "af_kernels.h"

namespace af {

__device__ int g_ops_err;   // the error word of calls that have no model

namespace {

constexpr int BQ = 128, BKV = 64;
constexpr int kThreads = 1024;
constexpr uint64_t kDrainLimitNs = 2000000000ull;
constexpr float kMost = 512.f;    // largest sum of a tile's exponentials before the maximum is raised
constexpr int kMaxDevices = 64;

template <int HD> struct Cfg {
  static constexpr int G = HD / 32;
  static constexpr int KCH = HD / 64;                     // 64-column boxes of a row
  static constexpr uint32_t QBOX = BQ * 128, BOX = BKV * 128;   // rows of 64 bf16
  static constexpr uint32_t Q_BYTES = KCH * QBOX, KV_BYTES = KCH * BOX;
  static constexpr int ST = 4;                            // stages of the K and of the V operand ring
  static constexpr int NR = 3;                            // raw slots of K and of V: a tile's codes and parameters
  static constexpr uint32_t CODES = BKV * (HD / 2), PARS = BKV * (HD / 8);
  static constexpr uint32_t RAW = CODES + PARS + 128;     // parameter rows of 8 bytes may start 8 bytes in
  static constexpr uint32_t TILES = 2 * Q_BYTES + 2 * ST * KV_BYTES;
  // barriers: Q full [2], S full [2][2], P ready [2][2], O done [2][2], K / V full / empty, raw full / empty, drain [4]
  static constexpr int BARS = 2 + 4 + 4 + 4 + 4 * ST + 4 * NR + 4;
  static constexpr size_t SMEM = 1024 + TILES + 2 * NR * RAW + 8 * BARS;
  static constexpr uint32_t IDESC_S = (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(BKV >> 3) << 17) |
                                      ((uint32_t)(BQ >> 4) << 24);
  // A (P, in TMEM) K-major, B (V) MN-major
  static constexpr uint32_t IDESC_O = (1u << 4) | (1u << 7) | (1u << 10) | (1u << 16) | ((uint32_t)(HD >> 3) << 17) |
                                      ((uint32_t)(BQ >> 4) << 24);
};
static_assert(Cfg<64>::SMEM <= 232448 && Cfg<128>::SMEM <= 232448, "attention shared memory");

__device__ __forceinline__ uint32_t smem_u32(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }
// 32-bit shared addresses, so that accesses are not generic ones
__device__ __forceinline__ void sts128(uint32_t at, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}
__device__ __forceinline__ uint4 lds128(uint32_t at) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at) : "memory");
  return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t at) {
  uint2 v;
  asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(at) : "memory");
  return v;
}
__device__ __forceinline__ void mbar_init(uint32_t bar, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}
__device__ __forceinline__ void mbar_expect_tx(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}
__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ bool mbar_try(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n"
      " selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}
struct Abort {
  volatile int* flag;
  uint64_t limit_ns;
};
__device__ __forceinline__ bool mbar_wait_slow(uint32_t bar, uint32_t parity, volatile int* flag, uint64_t limit_ns) {
  const uint64_t t0 = globaltimer_ns();
  for (;;) {
    if (mbar_try(bar, parity)) return true;
    if (*flag) return false;
    if (globaltimer_ns() - t0 > limit_ns) {
      *flag = 1;
      return false;
    }
  }
}
__device__ __forceinline__ bool mbar_wait(uint32_t bar, uint32_t parity, const Abort& ab) {
  return mbar_try(bar, parity) || mbar_wait_slow(bar, parity, ab.flag, ab.limit_ns);
}
// the same for a whole warp, with one outcome
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, const Abort& ab) {
  return __all_sync(0xffffffffu, mbar_wait(bar, parity, ab));
}
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(src), "r"(bytes), "r"(bar)
               : "memory");
}
// K-major, 128-byte swizzle: rows of 64 bf16, 8-row groups 1024 B apart
__device__ __forceinline__ uint64_t desc_k(uint32_t saddr) {
  return (uint64_t)((saddr & 0x3FFFFu) >> 4) | ((uint64_t)1 << 16) | ((uint64_t)(1024 >> 4) << 32) |
         ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}
// MN-major, 128-byte swizzle: a row of 64 elements of N per K index, 64-wide N boxes `lbo` bytes apart
__device__ __forceinline__ uint64_t desc_mn(uint32_t saddr, uint32_t lbo) {
  return (uint64_t)((saddr & 0x3FFFFu) >> 4) | ((uint64_t)((lbo >> 4) & 0x3FFFu) << 16) |
         ((uint64_t)(1024 >> 4) << 32) | ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}
// Products and commits are issued by one elected thread of a converged warp:
// descriptors stay in uniform registers that way.  (A branch to one lane, whose
// operands the compiler has to move over one by one, took about 80 cycles a
// product, more than the tensor core's 32 to 64.)
__device__ __forceinline__ void umma_ss(uint32_t d_tmem, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accum) {
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.b32 p, %4, 0;\n elect.sync _|q, 0xffffffff;\n"
      " @q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d_tmem),
      "l"(a), "l"(b), "r"(idesc), "r"(accum));
}
__device__ __forceinline__ void umma_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b, uint32_t idesc, uint32_t accum) {
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.b32 p, %4, 0;\n elect.sync _|q, 0xffffffff;\n"
      " @q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b), "r"(idesc), "r"(accum));
}
__device__ __forceinline__ void umma_commit(uint32_t bar) {
  asm volatile(
      "{\n .reg .pred q;\n elect.sync _|q, 0xffffffff;\n"
      " @q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}\n" ::"r"(bar)
      : "memory");
}
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, float* v) {
  uint32_t r[32];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
        "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
        "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, float* v) {
  uint32_t r[16];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t* v) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
      "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
}
// The wait names the loaded registers, so that nothing that uses them moves before it.
__device__ __forceinline__ void tmem_wait_ld(float (&v)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]), "+f"(v[6]), "+f"(v[7]),
                 "+f"(v[8]), "+f"(v[9]), "+f"(v[10]), "+f"(v[11]), "+f"(v[12]), "+f"(v[13]), "+f"(v[14]), "+f"(v[15])
               :
               : "memory");
}
__device__ __forceinline__ void tmem_wait_ld(float (&v)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]), "+f"(v[6]), "+f"(v[7]),
                 "+f"(v[8]), "+f"(v[9]), "+f"(v[10]), "+f"(v[11]), "+f"(v[12]), "+f"(v[13]), "+f"(v[14]), "+f"(v[15]),
                 "+f"(v[16]), "+f"(v[17]), "+f"(v[18]), "+f"(v[19]), "+f"(v[20]), "+f"(v[21]), "+f"(v[22]), "+f"(v[23])
               :
               : "memory");
  asm volatile("" : "+f"(v[24]), "+f"(v[25]), "+f"(v[26]), "+f"(v[27]), "+f"(v[28]), "+f"(v[29]), "+f"(v[30]), "+f"(v[31]));
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t pack2(float lo, float hi) { return u32_of(__floats2bfloat162_rn(lo, hi)); }

// True in every thread of the two warps at barrier `id` if `v` is in any of them.
__device__ __forceinline__ bool pair_any(int id, bool v) {
  uint32_t r;
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n barrier.cta.red.or.pred q, %2, 64, p;\n selp.u32 %0, 1, 0, q;\n}\n"
      : "=r"(r)
      : "r"((uint32_t)v), "r"(id)
      : "memory");
  return r != 0;
}

template <int HD, bool PAIR>
__global__ void __launch_bounds__(kThreads, 1) k_attn4_tc(const Attn4Args a, int* err) {
  using C = Cfg<HD>;
  constexpr int G = C::G, ST = C::ST, NR = C::NR;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort;
  __shared__ float s_x[2][2][128];                          // exchange between the two threads of a row [group][half][row]
  __shared__ float s_m1[128];                               // PAIR: group 1's m of each row
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_trigger();

  uint8_t* sQ = smem;
  uint8_t* sK = sQ + 2 * C::Q_BYTES;
  uint8_t* sV = sK + ST * C::KV_BYTES;
  uint8_t* sR = sV + ST * C::KV_BYTES;
  const uint32_t QF = smem_u32(sR + 2 * NR * C::RAW), SF = QF + 16, PR = SF + 32, OD = PR + 32, KF = OD + 32,
                 KE = KF + 8 * ST, VF = KE + 8 * ST, VE = VF + 8 * ST, RF = VE + 8 * ST, RE = RF + 16 * NR,
                 DR = RE + 16 * NR;
  if (threadIdx.x == 0) {
    s_abort = 0;
    for (int g = 0; g < 2; ++g) {
      mbar_init(QF + 8 * g, 8);
      for (int i = 0; i < 2; ++i) {                         // of each score buffer
        mbar_init(SF + 16 * g + 8 * i, 1);
        mbar_init(PR + 16 * g + 8 * i, 8);
        mbar_init(OD + 16 * g + 8 * i, 1);
      }
    }
    for (int i = 0; i < 4; ++i) mbar_init(DR + 8 * i, 1);
    for (int i = 0; i < ST; ++i) {
      mbar_init(KF + 8 * i, 4);
      mbar_init(KE + 8 * i, 2);
      mbar_init(VF + 8 * i, 4);
      mbar_init(VE + 8 * i, 2);
    }
    for (int i = 0; i < 2 * NR; ++i) {
      mbar_init(RF + 8 * i, 1);
      mbar_init(RE + 8 * i, 4);
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 25) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&s_tmem)), "r"(512));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  pdl_wait();

  // ---- this CTA's rows and keys
  const int group = a.group;
  constexpr int RT = PAIR ? 128 : 256;
  const int mrows = a.rows * group;
  int u = blockIdx.x;
  const int split = u % a.nsplit;
  u /= a.nsplit;
  const int n_bh = a.c.batch * a.c.kv_heads;
  const int bh = u % n_bh;
  const int m0 = ((mrows + RT - 1) / RT - 1 - u / n_bh) * RT;   // the heaviest rows of a causal mask come first
  const int b = bh / a.c.kv_heads, hk = bh - b * a.c.kv_heads;
  const Seq4 sq = seq4_of(a, b);
  const int m_end = sq.nq * group;
  const int chunk = tc_chunk4(sq.len, a.nsplit, BKV);
  const int nsp = max(1, (sq.len + chunk - 1) / chunk);
  const bool live = m0 < m_end && split < nsp;
  const int kbeg = split * chunk;
  const int kmax = min(kbeg + chunk, sq.len);
  auto keys_of = [&](int last_row) { return min(key_end4(a, sq, last_row / group), kmax); };
  const int kend = live ? keys_of(min(m0 + RT, m_end) - 1) : 0;   // past the last key that any row attends
  const int T = kend > kbeg ? (kend - kbeg + BKV - 1) / BKV : 0;
  auto tiles_of = [&](int g) {                              // !PAIR: key tiles of group g, the first of the T
    const int r0 = m0 + 128 * g;
    if (r0 >= m_end) return 0;
    const int e = keys_of(min(r0 + 128, m_end) - 1);
    return e > kbeg ? (e - kbeg + BKV - 1) / BKV : 0;
  };
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s_tmem;
  const Abort ab{&s_abort, a.wait_ns};
  // an issuing warp's products are complete (or have had their time) before TMEM is freed
  auto drain = [&](uint32_t bar) {
    umma_commit(bar);
    const uint64_t t0 = globaltimer_ns();
    while (!__all_sync(0xffffffffu, mbar_try(bar, 0)))
      if (__any_sync(0xffffffffu, globaltimer_ns() - t0 > kDrainLimitNs)) {
        if (lane == 0) atomicOr(err ? err : &g_ops_err, ERR_DRAIN);
        break;
      }
  };

  if (!live) {
  } else if (warp < 16) {
    // ------------------------------------------------------------------ softmax of group g, half h of a tile's keys
    asm volatile("setmaxnreg.inc.sync.aligned.u32 80;");
    const int g = warp >> 3, h = (warp >> 2) & 1, q = warp & 3;
    const int row = q * 32 + lane;                          // = TMEM lane
    const int mg = m0 + (PAIR ? 0 : 128 * g);               // the group's first row
    const int m = mg + row;
    const bool on = m < m_end;
    const int qi = on ? m / group : 0;
    const int head = hk * group + (on ? m - qi * group : 0);
    if (!PAIR || g == 0) {
      // Q: 16 rows a warp, 16-byte unit x of a row at x ^ (row & 7) of its box; rows past the last as zeros
      constexpr int U = HD / 8, RPI = 32 / U;               // units of a row, rows of an instruction
      const int r0 = (warp & 7) * 16, mo = mg + r0 + (lane & 15);
      const int io = mo < m_end ? mo / group : 0;
      const long long own = mo < m_end ? (long long)io * a.q_rs + (long long)(hk * group + mo - io * group) * HD : -1;
      uint4 v[16 / RPI];
#pragma unroll
      for (int i = 0; i < 16 / RPI; ++i) {
        const long long off = __shfl_sync(0xffffffffu, own, i * RPI + lane / U);
        v[i] = off >= 0 ? *reinterpret_cast<const uint4*>(a.q + sq.q0 + off + (lane % U) * 8) : make_uint4(0u, 0u, 0u, 0u);
      }
#pragma unroll
      for (int i = 0; i < 16 / RPI; ++i) {
        const int r = r0 + i * RPI + lane / U, x = lane % U;
        *reinterpret_cast<uint4*>(sQ + g * C::Q_BYTES + (x >> 3) * C::QBOX + r * 128 + (((x & 7) ^ (r & 7)) << 4)) = v[i];
      }
      fence_async();
      __syncwarp();
      if (lane == 0) mbar_arrive(QF + 8 * g);
    }
    const uint32_t lane_off = (uint32_t)(q * 32) << 16;
    const uint32_t tS = tmem + 128 * g + lane_off, tO = tmem + 256 + HD * g + lane_off + (HD / 2) * h;
    const int id = 1 + 4 * g + q;                           // the barrier of this warp and the other of its rows
    const int lim = on ? min(key_end4(a, sq, qi), kmax) : 0;   // this row attends keys below lim
    // the fewest keys of the warp's rows (they grow with the row)
    const int w0 = m - lane;
    const int lim_lo = __shfl_sync(0xffffffffu, lim, 0);
    const float sl2 = a.scale_log2;
    float mx = on ? -INFINITY : 0.f;
    float2 l2 = make_float2(0.f, 0.f);
    const int nt = PAIR ? T : tiles_of(g);
    int t = 0;                                              // tiles this group has finished
    bool ok = true;
    for (int j = PAIR ? g : 0; j < nt; j += PAIR ? 2 : 1) {
      const int buf = 16 * g + 8 * (t & 1);
      if (!warp_wait(SF + buf, (uint32_t)((t >> 1) & 1), ab)) ok = false;
      if (w0 >= m_end) {                                    // no row of these two warps is anyone's: their P may be anything
        if (lane == 0) mbar_arrive(PR + buf);
        __syncwarp();
        ++t;
        continue;
      }
      tc_fence_after();
      const uint32_t tSb = tS + BKV * (t & 1);
      const int k0 = kbeg + j * BKV + 32 * h;
      float v[32];
      tmem_ld32(tSb + 32 * h, v);
      tmem_wait_ld(v);
      if (k0 + 32 > lim_lo) {                               // something is masked in this warp
#pragma unroll
        for (int i = 0; i < 32; ++i)
          if (k0 + i >= lim) v[i] = -INFINITY;              // 2^-inf = +0
      }
      uint32_t pk[16];
      float2 s2;
      auto exponentials = [&]() {
        const float2 nmb = splat(mx == -INFINITY ? 0.f : -mx);
        s2 = make_float2(0.f, 0.f);
#pragma unroll
        for (int i = 0; i < 32; i += 2) {
          const float2 x = ffma2(make_float2(v[i], v[i + 1]), splat(sl2), nmb);
          const float2 e = make_float2(ex2(x.x), ex2(x.y));
          s2 = fadd2(s2, e);
          pk[i >> 1] = pack2(e.x, e.y);
        }
      };
      exponentials();
      // (the vote also says that both warps have their scores, over which P is written)
      const bool raise = mx == -INFINITY || s2.x + s2.y > kMost;
      if (pair_any(id, raise)) {
        float r0 = v[0], r1 = v[1];
#pragma unroll
        for (int i = 2; i < 32; i += 2) {
          r0 = fmaxf(r0, v[i]);
          r1 = fmaxf(r1, v[i + 1]);
        }
        // a row is raised if either of its threads asks for it
        s_x[g][h][row] = raise ? INFINITY : fmaxf(r0, r1);
        asm volatile("bar.sync %0, 64;" ::"r"(id) : "memory");
        const float other = s_x[g][h ^ 1][row];
        const bool both = raise || other == INFINITY;
        asm volatile("bar.sync %0, 64;" ::"r"(id) : "memory");
        s_x[g][h][row] = fmaxf(r0, r1);
        asm volatile("bar.sync %0, 64;" ::"r"(id) : "memory");
        float corr = 1.f;
        if (both) {
          const float m_new = fmaxf(mx, fmaxf(fmaxf(r0, r1), s_x[g][h ^ 1][row]) * sl2);
          if (mx != -INFINITY) corr = ex2(mx - m_new);
          l2 = fmul2(l2, splat(corr));
          mx = m_new;
        }
        if (t > 0 && __any_sync(0xffffffffu, corr != 1.f)) {
          // O holds the group's earlier tiles once the P V of the last one is done; each warp has half of its columns
          if (!warp_wait(OD + 16 * g + 8 * ((t - 1) & 1), (uint32_t)(((t - 1) >> 1) & 1), ab)) ok = false;
          tc_fence_after();
#pragma unroll 1
          for (int x = 0; x < HD / 2; x += 16) {
            float o[16];
            tmem_ld16(tO + x, o);
            tmem_wait_ld(o);
            uint32_t w[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) w[i] = __float_as_uint(o[i] * corr);
            tmem_st16(tO + x, w);
          }
        }
        exponentials();
      }
      l2 = fadd2(l2, s2);
      tmem_st16(tSb + 16 * h, pk);
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(PR + buf);
      ++t;                                                  // (after an abort too: the pairs' barriers stay matched)
    }
    // ---- O of all tiles: normalise and store, or a partial
    // (a group without a tile has not waited for its Q, over which the rows of the output go)
    if (!(t > 0 ? warp_wait(OD + 16 * g + 8 * ((t - 1) & 1), (uint32_t)(((t - 1) >> 1) & 1), ab)
                : PAIR || warp_wait(QF + 8 * g, 0, ab)))
      ok = false;
    tc_fence_after();
    float l = l2.x + l2.y;
    s_x[g][h][row] = l;
    float* so = reinterpret_cast<float*>(sK);               // PAIR: group 1's O, column-major so that lanes are adjacent
    if (PAIR) {
      asm volatile("bar.sync 9, 512;" ::: "memory");        // both groups' products are done with the operand tiles
      if (g == 1) {
#pragma unroll 1
        for (int c = 0; c < HD / 2; c += 16) {
          float o[16];
          if (t > 0) {
            tmem_ld16(tO + c, o);
            tmem_wait_ld(o);
          }
#pragma unroll
          for (int i = 0; i < 16; ++i) so[(h * (HD / 2) + c + i) * 128 + row] = t > 0 ? o[i] : 0.f;
        }
        s_m1[row] = mx;
      }
      asm volatile("bar.sync 9, 512;" ::: "memory");
    } else {
      asm volatile("bar.sync %0, 64;" ::"r"(id) : "memory");
    }
    if (!PAIR || g == 0) {
      l = s_x[g][0][row] + s_x[g][1][row];
      float f0 = 1.f, f1 = 0.f;
      if (PAIR) {
        const float m1 = s_m1[row], l1 = s_x[1][0][row] + s_x[1][1][row];
        const float mm = fmaxf(mx, m1);
        f0 = mx == -INFINITY ? 0.f : ex2(mx - mm);
        f1 = m1 == -INFINITY ? 0.f : ex2(m1 - mm);
        l = f0 * l + f1 * l1;
        mx = mm;
      }
      const bool part = nsp > 1;
      const float inv = part ? 1.f : row_scale4(l, lim > 0);   // (without splits lim counts all its keys)
      // Rows go through the group's (now free) Q tile, HD bytes a row and warp at a time, so that the stores to
      // memory are contiguous: 16-byte unit x of row r at x ^ r.  All of the half row in bf16, or half of it in fp32.
      constexpr int U = HD / 16, RPI = 32 / U;
      uint8_t* stage = sQ + g * C::Q_BYTES + (warp & 7) * 32 * HD;
      const size_t at = ((size_t)split * n_bh + bh) * mrows + m;
      const long long dst = !on || !ok ? -1
                            : part     ? (long long)(at * HD + h * (HD / 2)) * 4
                                       : (long long)(sq.o0 + (size_t)qi * a.o_rs + (size_t)head * HD + h * (HD / 2)) * 2;
      uint8_t* base = part ? reinterpret_cast<uint8_t*>(a.opart) : reinterpret_cast<uint8_t*>(a.o);
#pragma unroll 1
      for (int c = 0; c < HD / 2; c += 16) {
        float o[16];
        if (t > 0) {
          tmem_ld16(tO + c, o);
          tmem_wait_ld(o);
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          o[i] = t > 0 ? o[i] : 0.f;
          if (PAIR) o[i] = f0 * o[i] + f1 * so[(h * (HD / 2) + c + i) * 128 + row];
        }
        uint8_t* rp = stage + lane * HD;
        const int x0 = part ? (c % (HD / 4)) / 4 : c / 8;
        if (part) {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            *reinterpret_cast<float4*>(rp + (((x0 + i) ^ (lane & (U - 1))) << 4)) =
                make_float4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
        } else {
#pragma unroll
          for (int i = 0; i < 2; ++i)
            *reinterpret_cast<uint4*>(rp + (((x0 + i) ^ (lane & (U - 1))) << 4)) =
                make_uint4(pack2(o[8 * i] * inv, o[8 * i + 1] * inv), pack2(o[8 * i + 2] * inv, o[8 * i + 3] * inv),
                           pack2(o[8 * i + 4] * inv, o[8 * i + 5] * inv), pack2(o[8 * i + 6] * inv, o[8 * i + 7] * inv));
        }
        if (c + 16 == HD / 2 || (part && c + 16 == HD / 4)) {
          __syncwarp();
#pragma unroll
          for (int i = 0; i < U; ++i) {
            const int r = i * RPI + lane / U, x = lane % U;
            const long long d = __shfl_sync(0xffffffffu, dst, r);
            if (d >= 0)
              *reinterpret_cast<uint4*>(base + d + (part && c + 16 == HD / 2 ? HD : 0) + x * 16) =
                  *reinterpret_cast<const uint4*>(stage + r * HD + ((x ^ (r & (U - 1))) << 4));
          }
          __syncwarp();
        }
      }
      if (h == 0 && ok && on && part) {
        a.ml[2 * at] = mx;
        a.ml[2 * at + 1] = l;
      }
    }
  } else if (warp < 24) {
    // ------------------------------------------------------------------ decoding of K (warps 16-19) or V
    // A lane takes one code vector (row r, t: the words of all groups) at a
    // time: its words are one 16-byte unit of the operand row each.  The 8 lanes
    // of a store phase hold rows r and r ^ 5 with all four t, which fall on
    // different banks both in the raw slot (row pitch 64 bytes) and under the
    // swizzle.
    asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
    const bool is_v = warp >= 20;
    const int dw = warp & 3;
    const int t = lane & 3, qp = lane >> 3, hi = (lane >> 2) & 1;
    const int r0 = (qp ^ (hi ? 5 : 0));                     // row within 8
    // lane addresses: its row (of each 32) and t in a raw slot, and its first unit in an operand tile
    const int r_lane = dw * 8 + r0;
    const uint32_t raw0 = smem_u32(sR) + r_lane * (HD / 2) + t * (HD / 8);
    const uint32_t par_at = C::CODES + r_lane * (HD / 8) - r_lane * (HD / 2) - t * (HD / 8) +
                            (HD == 64 ? (uint32_t)(((size_t)bh * a.c.cap + kbeg) & 1) * 8 : 0u);
    const uint32_t dst0 = smem_u32(is_v ? sV : sK) + r_lane * 128 + ((t ^ r0) << 4);
    const uint32_t full = is_v ? VF : KF, empty = is_v ? VE : KE;
    int slot = 0;
    uint32_t rph = 0;
    for (int j = 0; j < T; ++j) {
      const int st = j % ST, rs = slot + (is_v ? NR : 0);
      if (!warp_wait(empty + 8 * st, (uint32_t)((j / ST) & 1) ^ 1u, ab) || !warp_wait(RF + 8 * rs, rph, ab)) break;
      const int rows = min(BKV, kend - (kbeg + j * BKV));   // live rows of the tile
      const uint32_t raw = raw0 + rs * C::RAW, dst = dst0 + st * C::KV_BYTES;
#pragma unroll
      for (int s = 0; s < BKV / 32; ++s) {
        uint32_t w[G], p[G];
        if (G == 4) {
          const uint4 x = lds128(raw + s * 2048), y = lds128(raw + par_at + s * 512);
          w[0] = x.x; w[1] = x.y; w[G - 2] = x.z; w[G - 1] = x.w;
          p[0] = y.x; p[1] = y.y; p[G - 2] = y.z; p[G - 1] = y.w;
        } else {
          const uint2 x = lds64(raw + s * 1024), y = lds64(raw + par_at + s * 256);
          w[0] = x.x; w[1] = x.y;
          p[0] = y.x; p[1] = y.y;
        }
        if (rows < BKV && s * 32 + r_lane >= rows) {
#pragma unroll
          for (int g = 0; g < G; ++g) p[g] = 0u;
        }
#pragma unroll
        for (int g = 0; g < G; ++g) {
          const uint32_t s2 = __byte_perm(p[g], p[g], 0x1010), lo2 = __byte_perm(p[g], p[g], 0x3232);
          // 16-byte unit 4 g + t of the operand row: box g / 2, unit (4 (g & 1) + t) ^ (row & 7) of its row
          sts128((g & 1 ? dst ^ 64 : dst) + (g >> 1) * C::BOX + s * 4096, dequant2(lop_and_or(w[g], 0x000F000Fu, 0x43004300u), s2, lo2),
                 dequant2(lop_and_or(w[g] >> 4, 0x000F000Fu, 0x43004300u), s2, lo2),
                 dequant2(lop_and_or(w[g] >> 8, 0x000F000Fu, 0x43004300u), s2, lo2),
                 dequant2(lop_and_or(w[g] >> 12, 0x000F000Fu, 0x43004300u), s2, lo2));
        }
      }
      fence_async();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(full + 8 * st);
        mbar_arrive(RE + 8 * rs);
      }
      if (++slot == NR) { slot = 0; rph ^= 1u; }
    }
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 40;");
    if (warp == 24 && lane == 0) {
      // ---------------------------------------------------------------- copies of codes and parameters
      const size_t row0 = (size_t)bh * a.c.cap + kbeg;
      int n_copies[2] = {0, 0};                             // of K and of V
      for (int j = 0; j < T; ++j) {
        const size_t r = row0 + (size_t)j * BKV;
        const int rows = min(BKV, kend - (kbeg + j * BKV));
        const size_t p0 = (r * (HD / 8)) & ~(size_t)15;     // copies start and end on 16-byte boundaries
        const uint32_t pbytes = (uint32_t)((((r + rows) * (HD / 8) + 15) & ~(size_t)15) - p0);
        const uint32_t cbytes = (uint32_t)rows * (HD / 2);
        const uint32_t ph = (uint32_t)((j / NR) & 1) ^ 1u;
        auto fetch = [&](int rs, const uint8_t* codes, const uint8_t* pars) -> bool {
          if (!mbar_wait(RE + 8 * rs, ph, ab)) return false;
          const uint32_t dst = smem_u32(sR + rs * C::RAW);
          mbar_expect_tx(RF + 8 * rs, cbytes + pbytes);
          bulk_load(dst, codes + r * (HD / 2), cbytes, RF + 8 * rs);
          bulk_load(dst + C::CODES, pars + p0, pbytes, RF + 8 * rs);
          return true;
        };
        if (!fetch(j % NR, a.c.kc, a.c.kp)) break;
        ++n_copies[0];
        if (!fetch(NR + j % NR, a.c.vc, a.c.vp)) break;
        ++n_copies[1];
      }
      // each slot's last copy lands before the CTA ends, also when nothing consumes it after an abort
      const uint64_t t0 = globaltimer_ns();
      for (int v = 0; v < 2; ++v)
        for (int k = max(0, n_copies[v] - NR); k < n_copies[v]; ++k)
          while (!mbar_try(RF + 8 * (v * NR + k % NR), (uint32_t)((k / NR) & 1)))
            if (globaltimer_ns() - t0 > kDrainLimitNs) {
              atomicOr(err ? err : &g_ops_err, ERR_DRAIN);
              break;
            }
    } else if (warp == 25 || warp == 26) {
      // ---------------------------------------------------------------- S = Q K^T of group g
      const int g = warp - 25;
      const int nt = PAIR ? T : tiles_of(g);
      const uint64_t aq = desc_k(smem_u32(sQ + (PAIR ? 0 : g) * C::Q_BYTES)), dk = desc_k(smem_u32(sK));
      int ns = 0;                                           // scores issued
      bool ok = T == 0 || warp_wait(QF + 8 * (PAIR ? 0 : g), 0, ab);
      for (int j = 0; j < T && ok; ++j) {
        const int st = j % ST;
        if (!warp_wait(KF + 8 * st, (uint32_t)((j / ST) & 1), ab)) break;
        if (PAIR ? (j & 1) != g : j >= nt) {                // not this group's tile
          if (lane == 0) mbar_arrive(KE + 8 * st);
          __syncwarp();
          continue;
        }
        // S lies over the P of the group's tile before the last
        if (ns > 1 && !warp_wait(OD + 16 * g + 8 * (ns & 1), (uint32_t)(((ns - 2) >> 1) & 1), ab)) break;
        tc_fence_after();
        const uint64_t bk = dk + (uint64_t)(st * (C::KV_BYTES >> 4));
#pragma unroll
        for (int ks = 0; ks < HD / 16; ++ks)
          umma_ss(tmem + 128 * g + BKV * (ns & 1), aq + (uint64_t)((ks >> 2) * (C::QBOX >> 4) + (ks & 3) * 2),
                  bk + (uint64_t)((ks >> 2) * (C::BOX >> 4) + (ks & 3) * 2), C::IDESC_S, ks > 0 ? 1u : 0u);
        umma_commit(SF + 16 * g + 8 * (ns & 1));
        umma_commit(KE + 8 * st);
        ++ns;
      }
      drain(DR + 8 * g);
    } else if (warp == 27 || warp == 28) {
      // ---------------------------------------------------------------- O += P V of group g
      const int g = warp - 27;
      const int nt = PAIR ? T : tiles_of(g);
      const uint64_t dv = desc_mn(smem_u32(sV), C::BOX);
      const uint32_t tS = tmem + 128 * g, tO = tmem + 256 + HD * g;
      int np = 0;                                           // products issued
      for (int j = 0; j < T; ++j) {
        const int st = j % ST;
        if (!warp_wait(VF + 8 * st, (uint32_t)((j / ST) & 1), ab)) break;
        if (PAIR ? (j & 1) != g : j >= nt) {                // not this group's tile
          if (lane == 0) mbar_arrive(VE + 8 * st);
          __syncwarp();
          continue;
        }
        if (!warp_wait(PR + 16 * g + 8 * (np & 1), (uint32_t)((np >> 1) & 1), ab)) break;
        tc_fence_after();
        const uint64_t bv = dv + (uint64_t)(st * (C::KV_BYTES >> 4));
#pragma unroll
        for (int ks = 0; ks < BKV / 16; ++ks)
          umma_ts(tO, tS + BKV * (np & 1) + 8 * ks, bv + (uint64_t)(ks * (2048 >> 4)), C::IDESC_O,
                  (np > 0 || ks > 0) ? 1u : 0u);
        umma_commit(OD + 16 * g + 8 * (np & 1));
        umma_commit(VE + 8 * st);
        ++np;
      }
      drain(DR + 16 + 8 * g);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 25) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512));
  }
  if (threadIdx.x == 0 && s_abort) atomicOr(err ? err : &g_ops_err, ERR_ATTN_WAIT);
}

template <int HD, bool PAIR>
cudaError_t launch_hd(Attn4Args a, int* err, cudaStream_t st) {
  // the shared-memory opt-in is a per-device setting of the function
  static bool attr[kMaxDevices] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= kMaxDevices || !attr[dev]) {
    e = cudaFuncSetAttribute(k_attn4_tc<HD, PAIR>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)Cfg<HD>::SMEM);
    if (e != cudaSuccess) return e;
    if (dev < kMaxDevices) attr[dev] = true;
  }
  a.group = a.heads / a.c.kv_heads;
  const long long mrows = (long long)a.rows * a.group;
  constexpr int RT = PAIR ? 128 : 256;
  const long long items = (mrows + RT - 1) / RT * a.c.batch * a.c.kv_heads * a.nsplit;
  if (items > 0x7FFFFFFF) return cudaErrorInvalidConfiguration;
  e = launch_k(k_attn4_tc<HD, PAIR>, dim3((unsigned)items), dim3(kThreads), Cfg<HD>::SMEM, st, a, err);
  if (e != cudaSuccess || a.nsplit == 1) return e;
  return launch_attn4_combine(a, false, BKV, st);
}

}  // namespace

// Splits of the tensor-core kernel: a split costs its key tiles plus about
// eight tiles of set-up, write-out and merging.  The count with the least time
// for all CTAs, one an SM; beyond two waves they fill in behind one another.
int attn4_tc_splits(int batch, int kv_heads, int group, int rows, int cap, int num_sms) {
  const long long mrows = (long long)rows * group;
  const long long items = (mrows <= 128 ? 1 : (mrows + 255) / 256) * batch * kv_heads;
  const int tiles = (cap + BKV - 1) / BKV;
  int best = 1;
  double best_cost = 0;
  for (int n = 1; n <= 32 && n <= tiles; ++n) {
    const double full = (double)(items * n) / num_sms;
    const double waves = full > 2 ? full + 0.3 : (double)((items * n + num_sms - 1) / num_sms);
    const double cost = waves * ((tiles + n - 1) / n + 8);
    if (n == 1 || cost < best_cost) {
      best = n;
      best_cost = cost;
    }
  }
  return best;
}

cudaError_t launch_attn4_tc(const Attn4Args& a, int* err, cudaStream_t st) {
  const bool pair = (long long)a.rows * (a.heads / a.c.kv_heads) <= 128;
  if (a.c.D == 128) return pair ? launch_hd<128, true>(a, err, st) : launch_hd<128, false>(a, err, st);
  return pair ? launch_hd<64, true>(a, err, st) : launch_hd<64, false>(a, err, st);
}

// Reads and clears the error word of the current device.
cudaError_t ops_error(int* code) {
  cudaError_t e = cudaDeviceSynchronize();
  if (e == cudaSuccess) e = cudaMemcpyFromSymbol(code, g_ops_err, sizeof *code);
  const int zero = 0;
  if (e == cudaSuccess && *code) e = cudaMemcpyToSymbol(g_ops_err, &zero, sizeof zero);
  return e;
}

}  // namespace af
