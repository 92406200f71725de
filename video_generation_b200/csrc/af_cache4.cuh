// af_cache4.cuh -- the 4-bit key/value cache: its layout in memory and what
// the kernels that write, read and attend it share.
//
// One layer's cache is one buffer of four parts, each starting on a 256-byte
// boundary and each laid out [batch][kv_heads][capacity][row]:
//   key codes (D/2 bytes a row), key parameters (D/8), value codes, value parameters.
// Channels form groups of 32.  A group's parameters are one 32-bit word: the
// step s (bf16, low half) and the lowest value lo (bf16, high half); channel c
// stands for lo + n_c * s, n_c in 0..15 (5 bits a value in all).
// The row's 4 * (D/32) code words are ordered [t][g] (t = 0..3, g the group):
// word (t, g) holds channels 32 g + 8 t + i, i = 0..7, even i in bits 4 (i/2),
// odd i in bits 16 + 4 (i/2).  The reasons:
//   - (w >> 4 j) & 0x000F000F is the pair of channels (2j, 2j+1), so one shift
//     and one logic operation give two adjacent codes as packed 16-bit lanes;
//   - an mma.sync lane t reads its words of all groups as one vector, and the
//     8 channels of a word are 16 adjacent bytes of a bf16 row, one swizzle
//     unit of a tcgen05 operand tile.
//
// A token whose key or value row of a head held a NaN or an infinity (or
// values whose range is not finite) is stored poisoned: its key parameters
// are NaN and its value parameters zero.  Every query that attends the token
// gets NaN through its score, and no query that masks it is touched, although
// whole key tiles go through the matrix products (0 * NaN would reach them).
#pragma once
#include "af_common.cuh"

namespace af {

struct Cache4 {
  const uint8_t *kc, *kp, *vc, *vp;   // the four parts
  int batch, kv_heads, D, cap;
};

__host__ __device__ inline size_t cache4_part(size_t rows, int row_bytes) {
  return (rows * (size_t)row_bytes + 255) & ~(size_t)255;
}
__host__ __device__ inline size_t cache4_bytes(int batch, int kv_heads, int D, int cap) {
  const size_t rows = (size_t)batch * kv_heads * cap;
  return 2 * (cache4_part(rows, D / 2) + cache4_part(rows, D / 8));
}
inline Cache4 cache4_at(const void* base, int batch, int kv_heads, int D, int cap) {
  const size_t rows = (size_t)batch * kv_heads * cap;
  const uint8_t* p = static_cast<const uint8_t*>(base);
  Cache4 c;
  c.kc = p;
  c.kp = c.kc + cache4_part(rows, D / 2);
  c.vc = c.kp + cache4_part(rows, D / 8);
  c.vp = c.vc + cache4_part(rows, D / 2);
  c.batch = batch;
  c.kv_heads = kv_heads;
  c.D = D;
  c.cap = cap;
  return c;
}

// Queries over the cache.  Sequence b has len[b] live positions; its nq[b]
// (<= rows) query rows are the last of them when `causal` (query i attends
// keys 0 .. len - nq + i) and attend all of them otherwise.  With ctl (a pass
// of an AF block) every sample has len = p0 + R, nq = R, and its query rows
// are R apart instead of q_bs.
struct Attn4Args {
  Cache4 c;
  const bf16* q;
  bf16* o;
  long long q_bs, q_rs, o_bs, o_rs;   // strides in elements
  int heads, rows, causal;
  int group;                          // heads of a key head (set by the launcher of the tensor-core kernel)
  const int *len, *nq;
  const Ctl* ctl;
  float scale_log2;                   // softmax scale * log2(e)
  int nsplit;                         // most key splits of a sequence
  int even;                           // small kernel: splits of one size for all sequences
  float* opart;                       // [nsplit][batch][kv_heads][rows * group][D], unnormalised
  float* ml;                          // [nsplit][batch][kv_heads][rows * group][2]: max (log2 units), sum
  uint64_t wait_ns;
};

// Rows to write into the cache: k and v [batch][rows][kv_heads * D]; row i of
// sequence b goes to position start[b] + i (start null: 0) for i < count[b]
// (count null: rows); positions outside 0 .. capacity-1 are dropped.  With ctl
// the rows are positions p0 .. p0 + R - 1 of [batch][Lc] rows.
struct Cache4W {
  Cache4 c;
  const bf16 *k, *v;
  long long k_bs, k_rs, v_bs, v_rs;
  int rows;
  const int *start, *count;
  const Ctl* ctl;
  int Lc;
};
struct Cache4R {
  Cache4 c;
  void *k, *v;
  long long bs, rs;
  int rows;
  const int *start, *count;
};
cudaError_t launch_cache4_write(const Cache4W& a, cudaStream_t st);
cudaError_t launch_cache4_read(const Cache4R& a, bool f32, cudaStream_t st);
// Attention over the cache.  The small kernel takes 16 packed query rows a
// CTA (any number of them); the partials of several splits are merged by the
// combine kernel (bkv: the tensor-core kernel's key tile).
int attn4_small_splits(int batch, int kv_heads, int group, int rows, int cap, int num_sms, int* even);
cudaError_t launch_attn4_small(const Attn4Args& a, cudaStream_t st);
// Which kernel takes a call of `rows * group` packed query rows a key head.
// Measured with 128 (64) channels: the small kernel needs 52 (30) us for each
// tile of 16 rows and 10^6 keys (of all sequences and key heads), the tensor-core
// kernel 105 (87) us for up to 128 rows and 160 (140) us for each 256, and 5 us
// more to start and finish.  With many CTAs their own starts add up: 5 us for each
// three CTAs an SM of the small kernel, 10 us for each one of the other.
// So with 128 channels 48 rows over 46800 keys of 16 heads go to the tensor cores
// (76 against 107 us) and 24 rows do not (74 against 80: the rule's error); 96 rows
// over 2000 keys of 8 heads do with four sequences (21 against 30 us), over 4
// heads with one they do not (18 against 13); 390 rows over 16 keys of 192 heads do
// (26 against 66 us).  Both kernels timed on 148 SMs, over 292 calls of 16 to 800
// keys and 48 to 4096 heads the rule loses 0.5% on average and 1.28 times at worst,
// over 198 calls of 17 to 390 rows and 2000 to 46800 keys 0.8% and 1.19 times.
inline bool attn4_use_tc(int batch, int kv_heads, int group, int rows, int cap, int head_dim, int num_sms) {
  const double m = (double)rows * group, heads = (double)batch * kv_heads;
  const double tiles = (double)(((long long)rows * group + 15) / 16), blocks = (double)(((long long)rows * group + 255) / 256);
  auto starts = [](double ctas, double fit, double us) { return ctas > 0.5 * fit ? us * (ctas / fit - 0.5) : 0.0; };
  const double small = (head_dim == 128 ? 52e-6 : 30e-6) * tiles * heads * cap + starts(tiles * heads, 3.0 * num_sms, 5);
  const double each = head_dim == 128 ? (m <= 128 ? 105e-6 : 160e-6 * blocks) : (m <= 128 ? 87e-6 : 140e-6 * blocks);
  return m > 16 && small - each * heads * cap - starts(blocks * heads, num_sms, 10) > 5;
}
// The tensor-core kernel (af_attn4_tc.cu) takes 128 or 256 packed rows a CTA;
// err: the error word of its bounded waits (null: that of calls without a model).
int attn4_tc_splits(int batch, int kv_heads, int group, int rows, int cap, int num_sms);
cudaError_t launch_attn4_tc(const Attn4Args& a, int* err, cudaStream_t st);
cudaError_t ops_error(int* code);
cudaError_t launch_attn4_combine(const Attn4Args& a, bool small, int bkv, cudaStream_t st);

struct Seq4 {
  int len, nq;
  size_t q0, o0;   // element offset of the sequence's first query and output row
};
__device__ __forceinline__ Seq4 seq4_of(const Attn4Args& a, int b) {
  Seq4 s;
  if (a.ctl) {
    s.len = min(a.ctl->p0 + a.ctl->R, a.c.cap);
    s.nq = min(a.ctl->R, a.rows);
    s.q0 = (size_t)b * a.ctl->R * a.q_rs;
    s.o0 = (size_t)b * a.ctl->R * a.o_rs;
  } else {
    s.len = max(0, min(a.len[b], a.c.cap));
    s.nq = a.nq ? max(0, min(a.nq[b], a.rows)) : a.rows;
    s.q0 = (size_t)b * a.q_bs;
    s.o0 = (size_t)b * a.o_bs;
  }
  return s;
}
// Keys that query i attends: 0 .. key_end - 1.
__device__ __forceinline__ int key_end4(const Attn4Args& a, const Seq4& s, int i) {
  return a.causal ? max(0, min(s.len, s.len - s.nq + i + 1)) : s.len;
}

// 1 / l of a row's finished sum; a row that attends nothing gives zeros.  A row
// with keys whose scores are all -inf (an infinite query channel against keys of
// one sign there, or sums beyond fp32) has the sum 0 too, and is 0 / 0: NaN.
__device__ __forceinline__ float row_scale4(float l, bool has_keys) {
  return l != 0.f ? 1.f / l : (has_keys ? __int_as_float(0x7FC00000) : 0.f);
}

// Keys of one split of the tensor-core attention: the sequence's key tiles of
// bkv keys in at most nsplit equal runs.
__host__ __device__ __forceinline__ int tc_chunk4(int len, int nsplit, int bkv) {
  const int tiles = (len + bkv - 1) / bkv;
  const int per = (tiles + nsplit - 1) / nsplit;
  return (per < 1 ? 1 : per) * bkv;
}

// (a & mask) | bits as one operation: written in C++ with two constants it became two
__device__ __forceinline__ uint32_t lop_and_or(uint32_t a, uint32_t mask, uint32_t bits) {
  uint32_t d;
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(d) : "r"(a), "r"(mask), "r"(bits));
  return d;
}
__device__ __forceinline__ __nv_bfloat162 bf2_of(uint32_t v) { return *reinterpret_cast<__nv_bfloat162*>(&v); }
__device__ __forceinline__ uint32_t u32_of(__nv_bfloat162 v) { return *reinterpret_cast<uint32_t*>(&v); }
// (128 + n) as bf16 pairs -> lo + n s, one rounding (128 + n - 128 is exact)
__device__ __forceinline__ uint32_t dequant2(uint32_t code128, uint32_t s2, uint32_t lo2) {
  return u32_of(__hfma2(__hsub2(bf2_of(code128), bf2_of(0x43004300u)), bf2_of(s2), bf2_of(lo2)));
}

}  // namespace af
