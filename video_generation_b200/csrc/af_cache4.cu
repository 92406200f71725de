// af_cache4.cu -- the 4-bit key/value cache: writing rows, reading them back,
// and attention of few query rows over it (layout: af_cache4.cuh).
#include <type_traits>

#include "af_cache4.cuh"
#include "af_kernels.h"

namespace af {
namespace {

__device__ __forceinline__ uint32_t pack2(float lo, float hi) { return u32_of(__floats2bfloat162_rn(lo, hi)); }
__device__ __forceinline__ bool finite_bits(uint32_t bf16x2) {
  return (bf16x2 & 0x7F80u) != 0x7F80u && (bf16x2 & 0x7F800000u) != 0x7F800000u;
}

// The warp's head, rows and sequence: heads vary fastest, so that neighbouring
// warps read neighbouring slices of the same rows.
struct RowTile {
  int b, head, row0;
};
__device__ __forceinline__ RowTile row_tile(long long w, int rows, int kv_heads, int rows_per_warp) {
  const int tiles = (rows + rows_per_warp - 1) / rows_per_warp;
  const long long rest = w / kv_heads;
  return {(int)(rest / tiles), (int)(w % kv_heads), (int)(rest % tiles) * rows_per_warp};
}

// ------------------------------------------------------------------ write
// Codes of a group of 32 channels, in the operations that define them:
//   lo = min x, s = bf16((max x - lo) / 15), n = min(15, rint((x - lo) / s)),
// 0 where s is 0; differences and quotients are fp32 rounded to nearest, since
// a reciprocal alone would break the exact ties that bf16 rows often hit.  A
// lane holds a whole group of a key or of a value row (keys in the lower half
// of the warp, values in the upper), so minimum, step and reciprocal are made
// once for 32 channels and without shuffles; four shuffles bring the code words
// of a row's groups into the order of memory.
// Bound by DRAM (2 bytes read and 5/8 written a value) and, close to it, by
// issue: 99 us for 46800 tokens of 16 heads of 128 channels (5.1 TB/s), 105 with
// the quotients one by one instead of in pairs (13 instructions a value then, an
// issue in 68% of the cycles).  48 warps an SM hide the loads: with 40 it takes
// 104 us.  One row costs 2.8 us; a lane with a key's and a value's group one
// after the other took 4.9 us for it and as long for long runs.
constexpr int kWriteWarps = 4;

// x / s for s in the range where nothing under- or overflows: the product with
// the rounded reciprocal r, corrected once by its exact remainder (P. Markstein,
// IBM J. Res. Dev. 34, 1990), is the rounded quotient.
__device__ __forceinline__ float quotient(float x, float s, float r) {
  const float q = x * r;
  return fmaf(fmaf(-q, s, x), r, q);
}

// One group: its parameters (s low, lo high) and the words of its codes.
__device__ __forceinline__ void code_group(const uint4 (&x)[4], uint32_t (&word)[4], uint32_t& par, bool& fin) {
  uint32_t w[16];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    w[4 * i] = x[i].x;
    w[4 * i + 1] = x[i].y;
    w[4 * i + 2] = x[i].z;
    w[4 * i + 3] = x[i].w;
  }
  __nv_bfloat162 mn = bf2_of(w[0]), mx = mn, zero = bf2_of(0u);
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    mn = __hmin2(mn, bf2_of(w[i]));
    mx = __hmax2(mx, bf2_of(w[i]));
    zero = __hfma2(bf2_of(w[i]), bf2_of(0u), zero);           // 0 unless something is not finite
  }
  const float lo = fminf(__low2float(mn), __high2float(mn)), hi = fmaxf(__low2float(mx), __high2float(mx));
  const float range = hi - lo;
  const float s15 = range > 1e-30f && range < 1e38f ? quotient(range, 15.f, 1.f / 15.f) : __fdiv_rn(range, 15.f);
  const bf16 sb = __float2bfloat16_rn(s15);
  const float s = __bfloat162float(sb);
  fin = fin && __low2float(zero) == 0.f && __high2float(zero) == 0.f &&
        fmaf(15.f, s, fabsf(lo)) <= 3.3895313892515355e38f;   // bf16's largest: no value reads back infinite
  par = (uint32_t)__bfloat16_as_ushort(sb) | ((uint32_t)__bfloat16_as_ushort(__float2bfloat16_rn(lo)) << 16);
  constexpr float kRound = 12582912.f;                          // 1.5 * 2^23: adding it rounds to a whole number, half to even
  if (s > 1e-30f && s < 1e30f) {
    const float r = __frcp_rn(s);
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      // even channels into bits 0-15, odd ones into bits 16-31; the codes are the low bits of the rounded sums
      uint32_t even = 0, odd = 0;
#pragma unroll
      for (int i = 3; i >= 0; --i) {
        // two quotients at once, as in quotient()
        const float2 d = fadd2(make_float2(__uint_as_float(w[4 * t + i] << 16), __uint_as_float(w[4 * t + i] & 0xFFFF0000u)),
                               splat(-lo));
        const float2 q = fmul2(d, splat(r));
        const float2 n = fadd2(ffma2(ffma2(q, splat(-s), d), splat(r), q), splat(kRound));
        even = even * 16 + __float_as_uint(n.x);                // q <= 15 (1 + 2^-8): no code above 15
        odd = odd * 16 + __float_as_uint(n.y);
      }
      constexpr uint32_t kBits = 0x4B400000u * 0x1111u;         // what kRound's own bits add up to
      word[t] = ((even - kBits) & 0xFFFFu) | ((odd - kBits) << 16);
    }
  } else {
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      word[t] = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint32_t u = w[4 * t + (i >> 1)];
        const float f = __uint_as_float(i & 1 ? u & 0xFFFF0000u : u << 16);
        const uint32_t n = s > 0.f ? (uint32_t)fminf(15.f, rintf(__fdiv_rn(f - lo, s))) : 0u;
        word[t] |= n << (4 * (i >> 1) + 16 * (i & 1));
      }
    }
  }
}

template <int D>
__global__ void __launch_bounds__(32 * kWriteWarps, 48 / kWriteWarps) k_cache4_write(const Cache4W a) {
  constexpr int G = D / 32, RPW = 16 / G;         // lanes of a row, rows of a warp
  pdl_trigger();
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const RowTile tile = row_tile((long long)blockIdx.x * kWriteWarps + (threadIdx.x >> 5), a.rows, a.c.kv_heads, RPW);
  const bool v = lane >= 16;
  const int b = tile.b, g = lane % G, i = tile.row0 + (lane & 15) / G;
  if (b >= a.c.batch) return;
  int start, count;
  long long src_row0;
  if (a.ctl) {
    start = a.ctl->p0;
    count = min(a.ctl->R, a.rows);
    src_row0 = (long long)b * a.Lc + start;
  } else {
    start = a.start ? a.start[b] : 0;
    count = a.count ? max(0, min(a.count[b], a.rows)) : a.rows;
    src_row0 = 0;
  }
  const long long p = (long long)start + i;
  const bool on = i < count && p >= 0 && p < a.c.cap;
  uint4 x[4];
  const bf16* src = (v ? a.v : a.k) + b * (a.ctl ? 0 : (v ? a.v_bs : a.k_bs)) +
                    (src_row0 + i) * (v ? a.v_rs : a.k_rs) + tile.head * D + 32 * g;
#pragma unroll
  for (int j = 0; j < 4; ++j)
    x[j] = on ? reinterpret_cast<const uint4*>(src)[j] : make_uint4(0u, 0u, 0u, 0u);
  uint32_t w[4], par;
  bool fin = true;
  code_group(x, w, par, fin);
  uint32_t bad = __ballot_sync(0xffffffffu, !fin);
  bad |= bad >> 16;                                    // anywhere in the token's K or V row of this head
  const bool poisoned = (bad >> (lane & 15 & ~(G - 1)) & ((1u << G) - 1u)) != 0;
  const size_t r = ((size_t)b * a.c.kv_heads + tile.head) * a.c.cap + (on ? p : 0);
#pragma unroll
  for (int t = 0; t < 4; ++t) w[t] = poisoned ? 0u : w[t];
  if (G == 4) {
    // lane g holds words t = 0..3 of its group; afterwards those of all groups for t = g
    const bool odd = g & 1, high = g & 2;
    const uint32_t y0 = __shfl_xor_sync(0xffffffffu, odd ? w[0] : w[1], 1), y1 = __shfl_xor_sync(0xffffffffu, odd ? w[2] : w[3], 1);
    const uint32_t u0 = odd ? y0 : w[0], u1 = odd ? w[1] : y0, u2 = odd ? y1 : w[2], u3 = odd ? w[3] : y1;
    const uint32_t z0 = __shfl_xor_sync(0xffffffffu, high ? u0 : u2, 2), z1 = __shfl_xor_sync(0xffffffffu, high ? u1 : u3, 2);
    w[0] = high ? z0 : u0;
    w[1] = high ? z1 : u1;
    w[2] = high ? u2 : z0;
    w[3] = high ? u3 : z1;
  } else {
    // lane 0 takes t = 0, 1 of both groups, lane 1 t = 2, 3
    const uint32_t y0 = __shfl_xor_sync(0xffffffffu, g ? w[0] : w[2], 1), y1 = __shfl_xor_sync(0xffffffffu, g ? w[1] : w[3], 1);
    const uint32_t u0 = g ? y0 : w[0], u1 = g ? w[2] : y0, u2 = g ? y1 : w[1], u3 = g ? w[3] : y1;
    w[0] = u0; w[1] = u1; w[2] = u2; w[3] = u3;
  }
  if (!on) return;
  reinterpret_cast<uint4*>(const_cast<uint8_t*>(v ? a.c.vc : a.c.kc) + r * (D / 2))[g] = make_uint4(w[0], w[1], w[2], w[3]);
  reinterpret_cast<uint32_t*>(const_cast<uint8_t*>(v ? a.c.vp : a.c.kp) + r * (D / 8))[g] = poisoned ? (v ? 0u : 0x7FC07FC0u) : par;
}

// ------------------------------------------------------------------ read
// x = lo + n s, one fp32 rounding (and one to bf16); a poisoned token's K and
// V rows are NaN.  A lane takes 8 channels of each group of a row (the words t;
// 4 channels for fp32), 16 bytes of output each, so that a store writes whole
// sectors; a warp takes 8 (4) rows, keys or values, and an SM holds as many warps
// as it can.  Four times the rows a warp, with their loads in flight together, took
// 100 us, twice 84, once 79 for 46800 tokens of 16 heads of 128 channels to bf16
// (83 with 40 registers and three quarters of the warps).
// Bound by DRAM: 5/8 bytes read and 2 or 4 written a value (79 us are 6.4 TB/s;
// 8190 tokens to fp32 27 us, 5.7).
template <int D, typename T>
__global__ void __launch_bounds__(256, 8) k_cache4_read(const Cache4R a) {
  constexpr int G = D / 32;
  constexpr int N = 16 / sizeof(T), LPR = 32 / N, RPW = 32 / LPR;   // channels a lane and group, lanes of a row, rows of a warp
  pdl_trigger();
  pdl_wait();
  const int lane = threadIdx.x & 31, t = lane % LPR * N / 8, half = lane % LPR * N % 8;
  const long long w = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
  const bool is_v = w & 1;
  const RowTile tile = row_tile(w >> 1, a.rows, a.c.kv_heads, RPW);
  const int b = tile.b, i = tile.row0 + lane / LPR;
  if (b >= a.c.batch) return;
  const int start = a.start ? a.start[b] : 0;
  const int count = a.count ? max(0, min(a.count[b], a.rows)) : a.rows;
  const long long p = (long long)start + i;
  if (i >= count || p < 0 || p >= a.c.cap) return;
  const size_t r = ((size_t)b * a.c.kv_heads + tile.head) * a.c.cap + (size_t)p;
  const uint8_t* cp = (is_v ? a.c.vc : a.c.kc) + r * (D / 2);
  const uint8_t* pp = (is_v ? a.c.vp : a.c.kp) + r * (D / 8);
  uint32_t word[G], par[G];
  if (G == 4) {
    const uint4 x = reinterpret_cast<const uint4*>(cp)[t], y = *reinterpret_cast<const uint4*>(pp);
    word[0] = x.x; word[1] = x.y; word[G - 2] = x.z; word[G - 1] = x.w;
    par[0] = y.x; par[1] = y.y; par[G - 2] = y.z; par[G - 1] = y.w;
  } else {
    const uint2 x = reinterpret_cast<const uint2*>(cp)[t], y = *reinterpret_cast<const uint2*>(pp);
    word[0] = x.x; word[1] = x.y;
    par[0] = y.x; par[1] = y.y;
  }
  const float kstep = __uint_as_float((is_v ? *reinterpret_cast<const uint32_t*>(a.c.kp + r * (D / 8)) : par[0]) << 16);
  T* o = static_cast<T*>(is_v ? a.v : a.k) + b * a.bs + (long long)i * a.rs + tile.head * D + 8 * t + half;
#pragma unroll
  for (int g = 0; g < G; ++g) {
    const float s = __uint_as_float(par[g] << 16);
    const float lo = kstep != kstep ? kstep : __uint_as_float(par[g] & 0xFFFF0000u);
    const uint32_t codes = word[g] >> (2 * half);
    float f[N];
#pragma unroll
    for (int c = 0; c < N; ++c) {
      // 2^23 + n, exactly
      const float n = __uint_as_float(lop_and_or(codes >> (16 * (c & 1) + 4 * (c >> 1)), 15u, 0x4B000000u)) - 8388608.f;
      f[c] = fmaf(n, s, lo);
    }
    if (N == 4)
      store4(o + 32 * g, f[0], f[1], f[2], f[3]);
    else
      *reinterpret_cast<uint4*>(o + 32 * g) =
          make_uint4(pack2(f[0], f[1]), pack2(f[2], f[3]), pack2(f[N - 4], f[N - 3]), pack2(f[N - 2], f[N - 1]));
  }
}

// ------------------------------------------------------------------ attention of few rows
// The query rows of all heads that share a key head are packed into one list,
// m = i * group + (head in group); a CTA takes 8 or 16 of them and one split
// of the sequence's keys.  Its four warps walk 32-key blocks in turn, each with
// its own ring of asynchronous copies, its own running maximum and sum and its
// own output tile; the four are merged in shared memory at the end, the splits
// by k_attn4_combine.
//
// A single token's call has to read every live key and value once (5 bits
// each) and does 2 flops per code.  Turning 4-bit codes into operands costs
// more instructions than anything else: the kernel is bound by issue, DRAM is
// next.  Hence
//   scores: the products run on the codes themselves, as bytes (three
//     instructions for eight codes), in whole numbers: q = d (256 a + b), a and b
//     bytes in rows gr and gr + 8 of the 16-row operand, one product a group of 32
//     channels.  The group's step multiplies the exact sum:
//     S = d sum_g s_g I_g + sum_g lo_g sum(q_g).
//     The second sum is one more product with the parameters as operand and
//     the sums of q split into three bf16 parts (all 24 bits of them).
//     d is a power of two that puts the row's largest value just below 2^15, so
//     a bf16 value within 2^-7 of it is exact; with ordinary rows hardly any is
//     not.  A channel far above the others leaves them fewer bits: where the
//     rounding takes more than 2^-13 of a group's values (each counted up to
//     2^11 d, so that the large ones do not hide the small), the CTA adds a
//     third byte, q = d (256 a + b + c / 256), in one more product a group.
//   values: v = lo + n s in packed bf16 (one rounding, 2^-8 relative at most),
//     keys in pairs; they are the 16-row operand (channels) of O^T += V^T P^T, P
//     the 8-column one, which halves the products for 8 rows;
//   maximum: the exponentials are taken with the maximum at hand; only when a
//     lane's sum of them passes 2^9 are the block's maxima taken, O rescaled and
//     the block done again.
// Masked scores become -inf; keys at or past the last key that any row of the
// CTA attends are zero-filled on the way in, so nothing stored there is used.
// P is rounded to bf16 for the product (its sum l stays fp32).
//
// Measured: one row over 46800 keys of 16 heads of 128 channels 34 us (120 MB,
// 3.5 TB/s; the instructions issue in 62% of the cycles, the ALU pipe is half
// taken), 40 us with the third byte, one row in 32 sequences of up to 8192 keys
// with 32 query and 8 key heads 51 us, one row over 390 keys of 4 x 12 heads of
// 64 channels 4.4 us.
constexpr int kSmallWarps = 4;
constexpr int kSmallStages = 2;
constexpr int kBlock = 32;        // keys of a warp's step
constexpr float kMost = 512.f;    // largest sum of a lane's exponentials before the maximum is raised

__device__ __forceinline__ void mma16816(float* c, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
               : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// c = A B with 16 of K, whose second 8 rows of B are its first 8 again
__device__ __forceinline__ void mma16816_twice(float* c, const uint32_t* a, uint32_t b) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%8}, {%9,%9,%9,%9};"
               : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b), "f"(0.f));
}
// 8-bit whole numbers: A signed, B unsigned, 32 of K.  c = A B
__device__ __forceinline__ void imma16832(int* c, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                          uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k32.row.col.s32.s8.u8.s32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
               : "=r"(c[0]), "=r"(c[1]), "=r"(c[2]), "=r"(c[3])
               : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "r"(0));
}
template <int BYTES> __device__ __forceinline__ void cp_async(uint32_t dst, const void* src, bool on) {
  const int n = on ? BYTES : 0;                    // bytes past n are filled with zeros
  if (BYTES == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n));
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst), "l"(src), "r"(n));
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Keys of one split of a sequence of `len`: a multiple of 128 (a block for
// each warp), and up to kWhole keys one split.  `cap` > 0: the same for every
// sequence, by the capacity, so that sequences of different lengths are cut into
// pieces of one size, which the SMs take as they come free; else by the
// sequence's own.
constexpr int kWhole = 512;
__host__ __device__ __forceinline__ int small_chunk(int len, int cap, int nsplit) {
  const int n = cap > 0 ? cap : len;
  if (n <= kWhole) return kWhole;
  return ((n + nsplit - 1) / nsplit + 127) / 128 * 128;
}

template <int D> struct SmallCfg {
  static constexpr int G = D / 32;
  static constexpr int CODES = kBlock * (D / 2), PARS = kBlock * (D / 8);   // bytes of a block
  static constexpr int STAGE = 2 * (CODES + PARS);
  static constexpr int RING = kSmallWarps * kSmallStages * STAGE;
  static constexpr int MERGE = kSmallWarps * 16 * (D + 4) * 4 + kSmallWarps * 16 * 2 * 4;
  static constexpr int SMEM = RING > MERGE ? RING : MERGE;
};

template <int D, bool HALF>   // HALF: at most 8 rows
__global__ void __launch_bounds__(kSmallWarps * 32, HALF ? 4 : 3) k_attn4_small(const Attn4Args a) {
  using Cfg = SmallCfg<D>;
  constexpr int G = Cfg::G;
  constexpr int NQ = HALF ? 1 : 2;                 // sets of 8 rows
  extern __shared__ __align__(16) uint8_t sm[];
  pdl_trigger();
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int gr = lane >> 2, t = lane & 3;
  const int group = a.heads / a.c.kv_heads;
  const int tiles = (a.rows * group + 15) / 16;    // row tiles of a sequence and key head
  const int split = blockIdx.x % a.nsplit, u = blockIdx.x / a.nsplit;
  const int bh = u / tiles, m0 = (u - bh * tiles) * 16;
  const int b = bh / a.c.kv_heads, hk = bh - b * a.c.kv_heads;
  const Seq4 sq = seq4_of(a, b);
  const int m_end = sq.nq * group;                 // packed rows of this sequence
  if (m0 >= m_end) return;
  const int chunk = small_chunk(sq.len, a.even ? a.c.cap : 0, a.nsplit);
  const int nsp = max(1, (sq.len + chunk - 1) / chunk);
  if (split >= nsp) return;
  const int kend = min(key_end4(a, sq, min(m0 + 15, m_end - 1) / group), (split + 1) * chunk);
  const int kbeg = split * chunk;
  const int blocks = kend > kbeg ? (kend - kbeg + kBlock - 1) / kBlock : 0;   // of this CTA

  // This warp's ring.  Each lane copies the same 16-byte units of every block
  // and the parameters of one key.
  uint8_t* ring = sm + warp * kSmallStages * Cfg::STAGE;
  const uint32_t ring_s = (uint32_t)__cvta_generic_to_shared(ring);
  const size_t row0 = (size_t)bh * a.c.cap + kbeg + kBlock * warp;   // of this warp's first block
  const int my_blocks = blocks > warp ? (blocks - warp + kSmallWarps - 1) / kSmallWarps : 0;
  constexpr int UPR = D / 32, CPL = D / 32;        // 16-byte units of a code row; of a block's codes a lane
  constexpr size_t ADV = kBlock * kSmallWarps;     // keys from one block of the warp to the next
  const uint8_t* kc = a.c.kc + row0 * (D / 2) + lane * 16;
  const uint8_t* vc = a.c.vc + row0 * (D / 2) + lane * 16;
  const uint8_t* kp = a.c.kp + (row0 + lane) * (D / 8);
  const uint8_t* vp = a.c.vp + (row0 + lane) * (D / 8);
  // unit x of row r lies at x ^ (r / 2 or r / 4): rows 16 / UPR * 2 apart repeat it
  const int cr = lane / UPR, cx = lane % UPR;
  const uint32_t cdst = cr * (D / 2) + ((D == 128 ? cx ^ ((cr >> 1) & 3) : cx ^ ((cr >> 2) & 1)) << 4);
  int left = kend - kbeg - kBlock * warp;          // keys from the next block to fetch on
  uint32_t fst = ring_s;                           // its stage
  auto fetch = [&]() {
    if (left >= kBlock) {
#pragma unroll
      for (int i = 0; i < CPL; ++i) {
        cp_async<16>(fst + cdst + 512 * i, kc + 512 * i, true);
        cp_async<16>(fst + Cfg::CODES + Cfg::PARS + cdst + 512 * i, vc + 512 * i, true);
      }
      cp_async<D / 8>(fst + Cfg::CODES + lane * (D / 8), kp, true);
      cp_async<D / 8>(fst + 2 * Cfg::CODES + Cfg::PARS + lane * (D / 8), vp, true);
    } else if (left > 0) {                         // the last block: zeros past the last key
#pragma unroll
      for (int i = 0; i < CPL; ++i) {
        const bool in = cr + 32 / UPR * i < left;
        cp_async<16>(fst + cdst + 512 * i, kc + 512 * i, in);
        cp_async<16>(fst + Cfg::CODES + Cfg::PARS + cdst + 512 * i, vc + 512 * i, in);
      }
      cp_async<D / 8>(fst + Cfg::CODES + lane * (D / 8), kp, lane < left);
      cp_async<D / 8>(fst + 2 * Cfg::CODES + Cfg::PARS + lane * (D / 8), vp, lane < left);
    }
    cp_commit();
    kc += ADV * (D / 2);
    vc += ADV * (D / 2);
    kp += ADV * (D / 8);
    vp += ADV * (D / 8);
    left -= (int)ADV;
    fst ^= ring_s ^ (ring_s + Cfg::STAGE);
  };

  fetch();                                         // the first block travels while Q is made ready

  // Q, one group of channels a warp, handed round through shared memory: the
  // bytes of 256 a + b + c / 256 of the group's channels 8 t + {0,4,1,5} and
  // {2,6,3,7} for rows gr (and gr + 8), the row's factor d and the sums over each
  // group.
  __shared__ uint4 s_q[NQ][G][32];
  __shared__ uint32_t s_qc[G][32][4];              // the bytes c: rows gr in words 0 and 2, rows gr + 8 in 1 and 3
  __shared__ float s_big[G][16], s_sum[G][16];
  int lim[2];                                      // keys that rows gr and gr + 8 of the tile attend
  int low = 0x7FFFFFFF;                            // the fewest keys that a row in use attends
  float f[NQ][8];
#pragma unroll
  for (int x = 0; x < 2; ++x) {
    const int m = m0 + gr + 8 * x;
    const bool on = (x == 0 || !HALF) && m < m_end;
    const int i = on ? m / group : 0;
    lim[x] = on ? key_end4(a, sq, i) : 0;
    if (on) low = min(low, lim[x]);
    if (x < NQ && warp < G) {
      uint4 v = make_uint4(0u, 0u, 0u, 0u);
      if (on)
        v = *reinterpret_cast<const uint4*>(a.q + sq.q0 + (size_t)i * a.q_rs +
                                            (size_t)(hk * group + m - i * group) * D + 32 * warp + 8 * t);
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
      float sum = 0.f, big = 0.f;
      bool fin = true;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        f[x][2 * j] = __uint_as_float(w[j] << 16);
        f[x][2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
        fin = fin && finite_bits(w[j]);
        sum += f[x][2 * j] + f[x][2 * j + 1];
        big = fmaxf(big, fmaxf(fabsf(f[x][2 * j]), fabsf(f[x][2 * j + 1])));
      }
      if (!fin) big = INFINITY;
#pragma unroll
      for (int o = 1; o <= 2; o <<= 1) {
        sum += __shfl_xor_sync(0xffffffffu, sum, o);
        big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, o));
      }
      if (t == 0) {
        s_big[warp][gr + 8 * x] = big;
        s_sum[warp][gr + 8 * x] = sum;
      }
    }
  }
  __syncthreads();
  float qd[NQ];                                    // d
  uint32_t qs[4] = {0u, 0u, 0u, 0u};               // the sums of q as an A operand
  bool lossy = false;                              // two bytes are too few for a row's group
#pragma unroll
  for (int x = 0; x < NQ; ++x) {
    float big = 1e-31f;                            // (a row of zeros, or of almost nothing)
#pragma unroll
    for (int g = 0; g < G; ++g) big = fmaxf(big, s_big[g][gr + 8 * x]);
    const bool fin = big < INFINITY;
    // exponent of d: big / d < 2^15, and at most 2^15 - 2^8, whose high byte is 127
    const uint32_t bits = __float_as_uint(big) + 0x10000u, e = (bits >> 23) - 14;
    qd[x] = fin ? __uint_as_float(e << 23) : __int_as_float(0x7FC00000);   // a row that is not finite scores NaN
    if (warp < G) {
      const float per = __uint_as_float((254 - e) << 23) * 256.f;
      constexpr int order[8] = {0, 4, 1, 5, 2, 6, 3, 7};
      uint32_t w[4] = {0u, 0u, 0u, 0u}, wc[2] = {0u, 0u};   // a and b of four channels each, twice; c likewise
      int lost = 0, kept = 0;
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int n = fin ? (int)rintf(f[x][order[4 * j + k]] * per) : 0;
          const int m = (n + 128) >> 8, c = n - 256 * m, top = (m + 128) >> 8;
          w[2 * j] |= (uint32_t)(top & 255) << (8 * k);
          w[2 * j + 1] |= (uint32_t)((m - 256 * top) & 255) << (8 * k);
          wc[j] |= (uint32_t)(c & 255) << (8 * k);
          lost += abs(c);
          kept += min(abs(n), 1 << 19);
        }
#pragma unroll
      for (int o = 1; o <= 2; o <<= 1) {           // a row's group is in four lanes: at most 2^12 and 2^24
        lost += __shfl_xor_sync(0xffffffffu, lost, o);
        kept += __shfl_xor_sync(0xffffffffu, kept, o);
      }
      lossy = lossy || (lost << 13) > kept;
      s_q[x][warp][lane] = make_uint4(w[0], w[1], w[2], w[3]);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        s_qc[warp][lane][2 * j + x] = wc[j];
        if (HALF) s_qc[warp][lane][2 * j + 1] = 0u;
      }
    }
    // k index 0-3 high part, 4-7 middle part, 8-11 low part of the sum of group k & 3, 12-15 nothing; lane t holds
    // k = 2t, 2t + 1 and 2t + 8, 2t + 9
    float p[2] = {0.f, 0.f}, p2[2] = {0.f, 0.f};
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int g = 2 * (t & 1) + e;
      if (g < G) {
        const float sum = s_sum[g][gr + 8 * x], hi = __bfloat162float(__float2bfloat16_rn(sum)), rest = sum - hi;
        p[e] = t < 2 ? hi : rest;
        p2[e] = t < 2 ? rest - __bfloat162float(__float2bfloat16_rn(rest)) : 0.f;
      }
    }
    qs[x] = pack2(p[0], p[1]);
    qs[2 + x] = pack2(p2[0], p2[1]);
  }
  lossy = __syncthreads_or(lossy);
  uint32_t qa[NQ][G][4];
#pragma unroll
  for (int x = 0; x < NQ; ++x)
#pragma unroll
    for (int g = 0; g < G; ++g) {
      const uint4 v = s_q[x][g][lane];
      qa[x][g][0] = v.x; qa[x][g][1] = v.y; qa[x][g][2] = v.z; qa[x][g][3] = v.w;
    }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) low = min(low, __shfl_xor_sync(0xffffffffu, low, o));

  float o[NQ][G * 2][4];                           // O^T: channels 32 g + 8 (gr / 2) + 4 i + (gr & 1) and + 2, rows 2t, 2t + 1
#pragma unroll
  for (int x = 0; x < NQ; ++x)
#pragma unroll
    for (int n = 0; n < G * 2; ++n) o[x][n][0] = o[x][n][1] = o[x][n][2] = o[x][n][3] = 0.f;
  float mx[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
  // lane offsets within a stage
  const int un = gr >> 1;
  const int okc = D == 128 ? gr * 64 + ((t ^ ((gr >> 1) & 3)) << 4)
                           : gr * 32 + (((t >> 1) ^ ((gr >> 2) & 1)) << 4) + (t & 1) * 8;
  const int ovc = D == 128 ? 2 * t * 64 + ((un ^ t) << 4) : 2 * t * 32 + (((un >> 1) ^ ((t >> 1) & 1)) << 4) + (un & 1) * 8;
  const uint32_t sel = (gr & 1) ? 0x7632u : 0x5410u;

  int key0 = kbeg + kBlock * warp;
  constexpr int H = kBlock / 8;                    // tiles of 8 keys
  // With and without the bytes c: one loop with a branch for them took 35.2 instead of 33.4 us where they are not
  // needed (one row over 46800 keys of 16 heads of 128 channels; two loops with them 40).
  auto walk = [&](auto with_c) {
#pragma unroll 1
    for (int n = 0; n < my_blocks; ++n, key0 += (int)ADV) {
      fetch();
      cp_wait<1>();
      __syncwarp();
      const uint8_t* st = ring + (n & 1) * Cfg::STAGE;
      // ---- scores of the block: keys 8 h + .. in the columns of tile h
      float s[H][2 * NQ];
#pragma unroll
      for (int h = 0; h < H; ++h) {
        uint32_t w[G], pa[G], pb[G];                 // codes of key 8 h + gr; parameters of keys 8 h + 2 t, + 1
        const uint8_t* par = st + Cfg::CODES + (8 * h + 2 * t) * (D / 8);
        uint2 own;                                   // parameters of key 8 h + gr (operand of the offset product)
        if (D == 128) {
          const uint4 x = *reinterpret_cast<const uint4*>(st + h * 512 + okc);
          const uint4 y = *reinterpret_cast<const uint4*>(par), z = *reinterpret_cast<const uint4*>(par + 16);
          w[0] = x.x; w[1] = x.y; w[G - 2] = x.z; w[G - 1] = x.w;
          pa[0] = y.x; pa[1] = y.y; pa[G - 2] = y.z; pa[G - 1] = y.w;
          pb[0] = z.x; pb[1] = z.y; pb[G - 2] = z.z; pb[G - 1] = z.w;
          own = *reinterpret_cast<const uint2*>(st + Cfg::CODES + (8 * h + gr) * 16 + (t & 1) * 8);
        } else {
          const uint2 x = *reinterpret_cast<const uint2*>(st + h * 256 + okc);
          const uint4 y = *reinterpret_cast<const uint4*>(par);
          w[0] = x.x; w[1] = x.y;
          pa[0] = y.x; pa[1] = y.y;
          pb[0] = y.z; pb[1] = y.w;
          own = *reinterpret_cast<const uint2*>(st + Cfg::CODES + (8 * h + gr) * 8);
        }
        float off[4];                                // sum_g lo_g sum(q_g)
        mma16816_twice(off, qs, __byte_perm(own.x, own.y, 0x7632));
        float acc[2 * NQ];
#pragma unroll
        for (int x = 0; x < 2 * NQ; ++x) acc[x] = 0.f;
#pragma unroll
        for (int g = 0; g < G; ++g) {
          const uint32_t k0 = w[g] & 0x0F0F0F0Fu, k1 = (w[g] >> 4) & 0x0F0F0F0Fu;
          const float sa = __uint_as_float(pa[g] << 16), sb = __uint_as_float(pb[g] << 16);
#pragma unroll
          for (int x = 0; x < NQ; ++x) {
            int c[4];
            imma16832(c, qa[x][g][0], qa[x][g][1], qa[x][g][2], qa[x][g][3], k0, k1);
            acc[2 * x] = fmaf(sa, (float)(c[0] * 256 + c[2]), acc[2 * x]);   // below 2^24: exact
            acc[2 * x + 1] = fmaf(sb, (float)(c[1] * 256 + c[3]), acc[2 * x + 1]);
          }
        }
        if constexpr (decltype(with_c)::value) {     // the bytes c of both sets of rows in one product
#pragma unroll
          for (int g = 0; g < G; ++g) {
            const uint4 v = *reinterpret_cast<const uint4*>(s_qc[g][lane]);
            int c[4];
            imma16832(c, v.x, v.y, v.z, v.w, w[g] & 0x0F0F0F0Fu, (w[g] >> 4) & 0x0F0F0F0Fu);
            const float sa = __uint_as_float(pa[g] << 16) * (1.f / 256.f), sb = __uint_as_float(pb[g] << 16) * (1.f / 256.f);
#pragma unroll
            for (int x = 0; x < 2 * NQ; ++x) acc[x] = fmaf(x & 1 ? sb : sa, (float)c[x], acc[x]);
          }
        }
#pragma unroll
        for (int x = 0; x < 2 * NQ; ++x) s[h][x] = fmaf(qd[x >> 1], acc[x], off[x]);
      }
      // ---- softmax: this lane's keys key0 + 8 h + 2 t + {0, 1}
      if (key0 + kBlock > low) {
#pragma unroll
        for (int h = 0; h < H; ++h)
#pragma unroll
          for (int e = 0; e < 2 * NQ; ++e)
            if (key0 + 8 * h + 2 * t + (e & 1) >= lim[e >> 1]) s[h][e] = -INFINITY;
      }
      uint32_t p[NQ][H];
      float add[NQ];
      auto exponentials = [&]() {
#pragma unroll
        for (int x = 0; x < NQ; ++x) {
          const float nm = mx[x] == -INFINITY ? 0.f : -mx[x];
          add[x] = 0.f;
#pragma unroll
          for (int h = 0; h < H; ++h) {
            const float e0 = ex2(fmaf(s[h][2 * x], a.scale_log2, nm)), e1 = ex2(fmaf(s[h][2 * x + 1], a.scale_log2, nm));
            add[x] += e0 + e1;
            p[x][h] = pack2(e0, e1);
          }
        }
      };
      exponentials();
      bool raise = (mx[0] == -INFINITY && lim[0] > 0) || add[0] > kMost;
      if (!HALF) raise = raise || (mx[1] == -INFINITY && lim[1] > 0) || add[NQ - 1] > kMost;
      if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
        for (int x = 0; x < NQ; ++x) {
          float m = fmaxf(s[0][2 * x], s[0][2 * x + 1]), f = 1.f;
#pragma unroll
          for (int h = 1; h < H; ++h) m = fmaxf(m, fmaxf(s[h][2 * x], s[h][2 * x + 1]));
          m *= a.scale_log2;
#pragma unroll
          for (int d = 1; d <= 2; d <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
          m = fmaxf(m, mx[x]);
          if (mx[x] != -INFINITY) f = ex2(mx[x] - m);
          mx[x] = m;
          l[x] *= f;
          // the factors of this lane's columns of O^T
          const float fa = __shfl_sync(0xffffffffu, f, 8 * t), fb = __shfl_sync(0xffffffffu, f, 8 * t + 4);
#pragma unroll
          for (int i = 0; i < G * 2; ++i) {
            o[x][i][0] *= fa;
            o[x][i][1] *= fb;
            o[x][i][2] *= fa;
            o[x][i][3] *= fb;
          }
        }
        exponentials();
      }
#pragma unroll
      for (int x = 0; x < NQ; ++x) l[x] += add[x];
      // ---- O^T += V^T P^T, 16 keys at a time: keys 2t, 2t+1 and 2t+8, 2t+9 of this lane, channel parity gr & 1 of
      // unit gr / 2
      const uint8_t* sv = st + Cfg::CODES + Cfg::PARS;
#pragma unroll
      for (int j = 0; j < H / 2; ++j) {
        uint32_t vw[2][G], ps[2][G], pl[2][G];       // code pairs, (s, s) and (lo, lo) of the two keys
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int h = 2 * j + e;
          const uint8_t* vpar = sv + Cfg::CODES + (8 * h + 2 * t) * (D / 8);
          uint32_t xa[G], xb[G], ya[G], yb[G];       // codes and parameters of the two keys
          if (D == 128) {
            const uint4 c0 = *reinterpret_cast<const uint4*>(sv + h * 512 + ovc);
            const uint4 c1 = *reinterpret_cast<const uint4*>(sv + h * 512 + ovc + 64);
            const uint4 d0 = *reinterpret_cast<const uint4*>(vpar), d1 = *reinterpret_cast<const uint4*>(vpar + 16);
            xa[0] = c0.x; xa[1] = c0.y; xa[G - 2] = c0.z; xa[G - 1] = c0.w;
            xb[0] = c1.x; xb[1] = c1.y; xb[G - 2] = c1.z; xb[G - 1] = c1.w;
            ya[0] = d0.x; ya[1] = d0.y; ya[G - 2] = d0.z; ya[G - 1] = d0.w;
            yb[0] = d1.x; yb[1] = d1.y; yb[G - 2] = d1.z; yb[G - 1] = d1.w;
          } else {
            const uint2 c0 = *reinterpret_cast<const uint2*>(sv + h * 256 + ovc);
            const uint2 c1 = *reinterpret_cast<const uint2*>(sv + h * 256 + ovc + 32);
            const uint4 d = *reinterpret_cast<const uint4*>(vpar);
            xa[0] = c0.x; xa[1] = c0.y;
            xb[0] = c1.x; xb[1] = c1.y;
            ya[0] = d.x; ya[1] = d.y;
            yb[0] = d.z; yb[1] = d.w;
          }
#pragma unroll
          for (int g = 0; g < G; ++g) {
            vw[e][g] = __byte_perm(xa[g], xb[g], sel);
            ps[e][g] = __byte_perm(ya[g], yb[g], 0x5410);
            pl[e][g] = __byte_perm(ya[g], yb[g], 0x7632);
          }
        }
#pragma unroll
        for (int g = 0; g < G; ++g)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            uint32_t v[2][2];                        // [key half][channel row gr or gr + 8]
#pragma unroll
            for (int e = 0; e < 2; ++e)
#pragma unroll
              for (int k = 0; k < 2; ++k)
                v[e][k] = dequant2(lop_and_or(vw[e][g] >> (8 * i + 4 * k), 0x000F000Fu, 0x43004300u), ps[e][g], pl[e][g]);
#pragma unroll
            for (int x = 0; x < NQ; ++x)
              mma16816(o[x][2 * g + i], v[0][0], v[0][1], v[1][0], v[1][1], p[x][2 * j], p[x][2 * j + 1]);
          }
      }
      __syncwarp();                                  // the stage may be written again
    }
  };
  if (lossy)
    walk(std::true_type{});
  else
    walk(std::false_type{});
  cp_wait<0>();
#pragma unroll
  for (int x = 0; x < NQ; ++x)
#pragma unroll
    for (int d = 1; d <= 2; d <<= 1) l[x] += __shfl_xor_sync(0xffffffffu, l[x], d);
  // ---- merge the four warps: (max, sum) and the rows x D outputs through shared memory
  __syncthreads();                                 // every warp has left its ring
  constexpr int LD = D + 4;                        // row pitch in floats, rows on different banks
  float* so = reinterpret_cast<float*>(sm) + warp * 16 * LD;
  float* sml = reinterpret_cast<float*>(sm) + kSmallWarps * 16 * LD;
#pragma unroll
  for (int x = 0; x < NQ; ++x) {
    float* d = so + (8 * x + 2 * t) * LD + 8 * un + (gr & 1);
#pragma unroll
    for (int g = 0; g < G; ++g)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        d[32 * g + 4 * i] = o[x][2 * g + i][0];
        d[32 * g + 4 * i + LD] = o[x][2 * g + i][1];
        d[32 * g + 4 * i + 2] = o[x][2 * g + i][2];
        d[32 * g + 4 * i + 2 + LD] = o[x][2 * g + i][3];
      }
    if (t == 0) {
      sml[(warp * 16 + gr + 8 * x) * 2] = mx[x];
      sml[(warp * 16 + gr + 8 * x) * 2 + 1] = l[x];
    }
  }
  __syncthreads();
  const int rows_here = min(HALF ? 8 : 16, m_end - m0);
  const int mrows = a.rows * group;
  for (int e = threadIdx.x; e < rows_here * (D / 4); e += kSmallWarps * 32) {
    const int r = e / (D / 4), c = (e % (D / 4)) * 4;
    float m = -INFINITY;
#pragma unroll
    for (int w = 0; w < kSmallWarps; ++w) m = fmaxf(m, sml[(w * 16 + r) * 2]);
    float ls = 0.f, v0 = 0.f, v1 = 0.f, v2 = 0.f, v3 = 0.f;
#pragma unroll
    for (int w = 0; w < kSmallWarps; ++w) {
      const float mw = sml[(w * 16 + r) * 2];
      const float f = mw == -INFINITY ? 0.f : ex2(mw - m);
      const float4 x = *reinterpret_cast<const float4*>(reinterpret_cast<float*>(sm) + (w * 16 + r) * LD + c);
      ls = fmaf(f, sml[(w * 16 + r) * 2 + 1], ls);
      v0 = fmaf(f, x.x, v0); v1 = fmaf(f, x.y, v1); v2 = fmaf(f, x.z, v2); v3 = fmaf(f, x.w, v3);
    }
    const int mr = m0 + r, i = mr / group, h = hk * group + mr - i * group;
    if (nsp == 1) {
      const float inv = row_scale4(ls, key_end4(a, sq, i) > 0);
      store4(a.o + sq.o0 + (size_t)i * a.o_rs + (size_t)h * D + c, v0 * inv, v1 * inv, v2 * inv, v3 * inv);
    } else {
      const size_t at = ((size_t)split * a.c.batch * a.c.kv_heads + bh) * mrows + mr;
      store4(a.opart + at * D + c, v0, v1, v2, v3);
      if (c == 0) {
        a.ml[2 * at] = m;
        a.ml[2 * at + 1] = ls;
      }
    }
  }
}

// Merges a row's splits in split order: o = sum_i 2^(m_i - m) o_i / sum_i 2^(m_i - m) l_i.
// A warp a row; lane i holds the statistics of splits i and i + 32 (at most 64 splits).
template <int D, bool SMALL>
__global__ void __launch_bounds__(128) k_attn4_combine(const Attn4Args a, int bkv) {
  pdl_trigger();
  pdl_wait();
  const long long w = (long long)blockIdx.x * 4 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  const int group = a.heads / a.c.kv_heads;
  const long long mrows = (long long)a.rows * group;
  const int bh = (int)(w / mrows), mr = (int)(w - bh * mrows);
  if (bh >= a.c.batch * a.c.kv_heads) return;
  const int b = bh / a.c.kv_heads, hk = bh - b * a.c.kv_heads;
  const Seq4 sq = seq4_of(a, b);
  if (mr >= sq.nq * group) return;
  const int chunk = SMALL ? small_chunk(sq.len, a.even ? a.c.cap : 0, a.nsplit) : tc_chunk4(sq.len, a.nsplit, bkv);
  const int nsp = (sq.len + chunk - 1) / chunk;
  if (nsp <= 1) return;                            // the attention kernel wrote the row itself
  const size_t stride = (size_t)a.c.batch * a.c.kv_heads * mrows;
  const size_t at = (size_t)bh * mrows + mr;
  float m[2] = {-INFINITY, -INFINITY}, lp[2] = {0.f, 0.f}, f[2];
#pragma unroll
  for (int k = 0; k < 2; ++k)
    if (lane + 32 * k < nsp) {
      const float2 x = *reinterpret_cast<const float2*>(a.ml + 2 * (at + (lane + 32 * k) * stride));
      m[k] = x.x;
      lp[k] = x.y;
    }
  float mx = fmaxf(m[0], m[1]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
  float l = 0.f;
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    f[k] = m[k] == -INFINITY ? 0.f : ex2(m[k] - mx);
    l += f[k] * lp[k];                             // a NaN sum stays one
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
  constexpr int PER = D / 32;
  float acc[PER];
#pragma unroll
  for (int k = 0; k < PER; ++k) acc[k] = 0.f;
  const float* ob = a.opart + at * D + PER * lane;
  for (int s0 = 0; s0 < nsp; s0 += 8) {            // eight splits' loads in flight before their sums
    float v[8][PER];
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const bool on = s0 + u < nsp;
      if (PER == 4) {
        const float4 x = on ? *reinterpret_cast<const float4*>(ob + (s0 + u) * stride * D) : make_float4(0.f, 0.f, 0.f, 0.f);
        v[u][0] = x.x; v[u][1] = x.y; v[u][PER - 2] = x.z; v[u][PER - 1] = x.w;
      } else {
        const float2 x = on ? *reinterpret_cast<const float2*>(ob + (s0 + u) * stride * D) : make_float2(0.f, 0.f);
        v[u][0] = x.x; v[u][1] = x.y;
      }
    }
    const float fs = s0 < 32 ? f[0] : f[1];
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const float x = __shfl_sync(0xffffffffu, fs, (s0 + u) & 31);
#pragma unroll
      for (int k = 0; k < PER; ++k) acc[k] = s0 + u < nsp ? fmaf(x, v[u][k], acc[k]) : acc[k];
    }
  }
  const int i = mr / group, h = hk * group + mr - i * group;
  const float inv = row_scale4(l, key_end4(a, sq, i) > 0);
  bf16* dst = a.o + sq.o0 + (size_t)i * a.o_rs + (size_t)h * D + PER * lane;
  if (PER == 4)
    store4(dst, acc[0] * inv, acc[1] * inv, acc[PER - 2] * inv, acc[PER - 1] * inv);
  else
    *reinterpret_cast<uint32_t*>(dst) = pack2(acc[0] * inv, acc[1] * inv);
}

template <int D>
cudaError_t small_d(const Attn4Args& a, cudaStream_t st) {
  const int group = a.heads / a.c.kv_heads;
  const long long mrows = (long long)a.rows * group;
  const long long items = (mrows + 15) / 16 * a.c.batch * a.c.kv_heads * a.nsplit;
  if (items > 0x7FFFFFFF) return cudaErrorInvalidConfiguration;
  const dim3 grid((unsigned)items), block(kSmallWarps * 32);
  cudaError_t e = mrows <= 8 ? launch_k(k_attn4_small<D, true>, grid, block, SmallCfg<D>::SMEM, st, a)
                             : launch_k(k_attn4_small<D, false>, grid, block, SmallCfg<D>::SMEM, st, a);
  if (e != cudaSuccess || a.nsplit == 1) return e;
  return launch_attn4_combine(a, true, 0, st);
}

// Blocks of 8 warps for `per` rows of a sequence and head a warp; 0 when there are too many.
unsigned row_blocks(const Cache4& c, int rows, int per, int parts, int warps) {
  const long long blocks = ((long long)c.batch * ((rows + per - 1) / per) * c.kv_heads * parts + warps - 1) / warps;
  return blocks > 0x7FFFFFFF ? 0u : (unsigned)blocks;
}

}  // namespace

cudaError_t launch_cache4_write(const Cache4W& a, cudaStream_t st) {
  const dim3 grid(row_blocks(a.c, a.rows, 16 * 32 / a.c.D, 1, kWriteWarps)), block(32 * kWriteWarps);
  return a.c.D == 128 ? launch_k(k_cache4_write<128>, grid, block, 0, st, a)
                      : launch_k(k_cache4_write<64>, grid, block, 0, st, a);
}

cudaError_t launch_cache4_read(const Cache4R& a, bool f32, cudaStream_t st) {
  const dim3 grid(row_blocks(a.c, a.rows, f32 ? 4 : 8, 2, 8)), block(256);
  if (a.c.D == 128)
    return f32 ? launch_k(k_cache4_read<128, float>, grid, block, 0, st, a)
               : launch_k(k_cache4_read<128, bf16>, grid, block, 0, st, a);
  return f32 ? launch_k(k_cache4_read<64, float>, grid, block, 0, st, a)
             : launch_k(k_cache4_read<64, bf16>, grid, block, 0, st, a);
}

cudaError_t launch_attn4_combine(const Attn4Args& a, bool small, int bkv, cudaStream_t st) {
  const long long rows = (long long)a.c.batch * a.rows * a.heads;
  const dim3 grid((unsigned)((rows + 3) / 4)), block(128);
  if (a.c.D == 128)
    return small ? launch_k(k_attn4_combine<128, true>, grid, block, 0, st, a, bkv)
                 : launch_k(k_attn4_combine<128, false>, grid, block, 0, st, a, bkv);
  return small ? launch_k(k_attn4_combine<64, true>, grid, block, 0, st, a, bkv)
               : launch_k(k_attn4_combine<64, false>, grid, block, 0, st, a, bkv);
}

// Splits, each at least 512 keys.  Few sequences: so that the CTAs fill the SMs
// once (HALF: four fit an SM, else three), since a second wave would double the
// time of a call that is one long sequence.  Many: pieces of about 1024 keys,
// whatever a sequence's length, at most eight (*even).  Where that leaves SMs
// without a CTA, down to 128 keys a split until each has one (one row over 2000
// keys of 4 heads 7.3 us, over 1000 keys of 16 heads 6.8; with 512 keys a split 9.2
// both).  Up to 512 keys one split: 5.4 us for 390 keys of 48 heads, 7.1 in three.
int attn4_small_splits(int batch, int kv_heads, int group, int rows, int cap, int num_sms, int* even) {
  const long long tiles = ((long long)rows * group + 15) / 16 * batch * kv_heads;
  const long long fit = ((long long)rows * group <= 8 ? 4 : 3) * num_sms;
  *even = batch > 1 && tiles * 4 > fit;
  if (cap <= kWhole) return 1;
  long long n = *even ? (cap + 1023) / 1024 : fit / tiles;
  if (*even && n > 8) n = 8;
  if (n > (cap + 511) / 512) n = (cap + 511) / 512;
  const long long one = num_sms / tiles < (cap + 127) / 128 ? num_sms / tiles : (cap + 127) / 128;
  if (!*even && n < one) n = one;
  if (n > 64) n = 64;
  return n < 1 ? 1 : (int)n;
}

cudaError_t launch_attn4_small(const Attn4Args& a, cudaStream_t st) {
  return a.c.D == 128 ? small_d<128>(a, st) : small_d<64>(a, st);
}

}  // namespace af
