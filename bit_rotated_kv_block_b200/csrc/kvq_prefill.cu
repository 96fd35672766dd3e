// Attention of many query rows over the rotated paged cache: prompt chunks
// (kvq_paged_prefill_attn) and the shared prefix of a batch
// (kvq_shared_prefix_decode_attn), with scored options.
//
// Mathematics. A row is one (query token, query head) pair; the G heads of a
// KV head's group and the tokens of a sequence (or, over a shared prefix, the
// sequences of the batch) are the rows of one matrix product with that KV
// head's keys. With q^ = R q, codes c, row scale s and minimum m of a key,
//   z_j = sm_scale (s_j sum_i (64 + c_ji) q^_i + (m_j - 64 s_j) sum_i q^_i),
// then the cap, the distance bias and the interval mask [lo, hi) of the row,
// and out = R^-1 sum_j p_j v^_j with the online softmax in base 2.
//
// Work split. One CTA per (sequence, KV head, 128 rows, split of the key
// tiles); 17 of its warps have a role:
//  - 8 softmax warps of 16 rows each, which they read as fragments (two rows
//    per thread, a quarter of the columns), so that a row's maximum stays in
//    four lanes and a key's scale and offset are read once per two rows. (One
//    row per thread: the broadcast reads of scale and offset, 128 x 128 x 8
//    bytes into registers, took 1024 cycles of a tile. Rows shared by two
//    warps: their agreement on the maximum took 340.)
//  - 4 + 4 warps widen the packed keys and values of the next tiles to
//    binary16 operands in shared memory, one key per thread, with the codes of
//    two tiles ahead in registers.
//  - 1 warp issues every tcgen05.mma: S = Q K^T, and O += P V with P read from
//    tensor memory. S has two buffers, so one tile's softmax runs under the
//    products of its neighbours.
//
// What bounds it (d = 128, one B200): a key tile of 128 takes 1.40 us, 2700
// cycles at 1.92 GHz (2.7 us with a cap, 2.5 us with a bias alone), of which
// the softmax warps' own chain (read S, scale, maximum, exponentials, write P)
// is the whole: 24 products of 74 cycles take 1776 (2130 with their hand-overs
// and no softmax at all), the exponentials 1024 of the special-function pipe,
// all instructions 1290 issue slots per scheduler. A CTA's first S comes 6 us after its start and its end 3 us after
// the last product; at 4096 tokens that is a third of the time. Measured and
// not kept: one CTA per SM walking over items with the next query copied
// ahead (prompt 233 -> 234 us, few rows 25 -> 30 us), a tile per softmax
// warpgroup in turn (1.82 us), a part of the exponentials on the FMA pipe
// (0 to 2% slower), 16 softmax warps (1.66 us), binary16 scale and minimum
// (1.46 us).
//
// Precision. Key codes enter as 64 + c, exact in binary16 (the offset costs
// the binary32 sum three of its bits); the row's s and m are applied in
// binary32 after the product. The rotated query is scaled by a
// power of two per row and split into binary16 hi + lo (about 22 bits): rounded to
// one binary16 it would cost |z| 2^-12 in every exponent, which for outlier
// keys (|z| of 10 and more) is several times the output's own rounding. p and
// v^ are rounded to binary16 once each (2^-12 relative on average, like the
// binary16 output); where a CTA has 64 rows at most, p enters
// as hi + lo. All sums are binary32.

#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <climits>
#include <cstddef>
#include <type_traits>

#include "kvq_device.cuh"
#include "kvq_launch.h"
#include "kvq_rotate.cuh"
#include "kvq_tcgen05.cuh"

namespace kvq {

namespace {

constexpr int kPfNW = 2;                   // softmax warpgroups
constexpr int kPfSoft = kPfNW * 128;       // their threads
constexpr int kPfThreads = kPfSoft + 384;  // and keys, values, the issuing warp's group
constexpr int kPfIssue = kPfSoft / 32 + 8; // the issuing warp
constexpr int kPfRows = 128;      // rows of a CTA
constexpr uint32_t kPfTmemCols = 512;
// A row's reference maximum moves only when a score exceeds it by more than
// kPfSlack; weights are 2^(z - M + kPfLift), so they stay below 2^15 and the
// smallest normal binary16 weight lies 2^-21 below the reference.
constexpr float kPfSlack = 8.f;
constexpr float kPfLift = 7.f;

template <int D>
struct PfCfg {
  static constexpr int KT = D == 128 ? 128 : 64;  // keys per tile
  static constexpr int HC = D / kPfNW;                // channels of a row per softmax thread
  static constexpr int GRP = D * 16;              // bytes of 8 rows (D / 8 core matrices)
  // The query operand: in tensor memory at d = 128 (hi, then lo); in shared
  // memory at d = 256, where O leaves no columns for it. A product with A in
  // shared memory takes 107 cycles at N 128, from tensor memory 74 (measured,
  // M 128, K 16; 64 is the tensor core's own time).
  static constexpr bool QT = D == 128;
  static constexpr int Q_B = kPfRows * D * 2;     // one operand (hi or lo)
  static constexpr int NS = D == 128 ? 2 : 1;     // stages of the key and value tiles
  static constexpr int K_OFF = QT ? 0 : 2 * Q_B;
  static constexpr int K_B = KT * D * 2;
  static constexpr int V_OFF = K_OFF + NS * K_B;
  // 4 slots of (scale, scale, offset, offset) per pair of keys
  static constexpr int PAR_OFF = V_OFF + NS * K_B;
  // 4 slots of a bit per key (bad, or large) and a bit per large one
  static constexpr int BAD_OFF = PAR_OFF + 8 * KT * 4;
  static constexpr int BW = KT / 32;                    // words of a bit per key
  static constexpr int EX_OFF = BAD_OFF + 4 * 8 * BW;   // exchange: 2 slots x kPfNW x 128 floats
  // PfRowState of 128 rows. (At d = 256 it starts 64 bytes off a multiple of
  // 128; on one, the wide heads took 5% longer, 149.5 against 142.4 us.)
  static constexpr int ROW_OFF = EX_OFF + 2 * kPfNW * kPfRows * 4;
  // Rows of the query as copied in, and of the output on its way out. The
  // pitch lets eight threads on the same channels of consecutive rows meet
  // different banks. At d = 256 they lie where the query operand will be (its
  // rows are read before it is written) and was (at the end).
  static constexpr int QS_PITCH = 2 * D + 16;
  static constexpr int QS_OFF = QT ? ROW_OFF + 32 * kPfRows : 0;
  static constexpr int LPR = D / 8;  // 16-byte pieces of a row
  static constexpr int BAR_OFF = ROW_OFF + 32 * kPfRows + (QT ? kPfRows * QS_PITCH : 0);
  static constexpr int SMEM = BAR_OFF + 256;
  // tensor-memory columns: S0, S1, O, then Q (d = 128) or P (d = 256)
  static constexpr int O_COL = 2 * KT;
  static constexpr int Q_COL = O_COL + D;
  // weights P of tile j: over S j & 1 at d = 128, where no other columns are
  // left (the issuing warp lets O += P V complete before the next S is written
  // there: products are only ordered among themselves where they share the
  // accumulator); in columns of their own at d = 256
  static constexpr int P_COL = QT ? 0 : O_COL + D;
  static constexpr int P_STEP = QT ? KT : KT / 2;
  static_assert(O_COL + D + (QT ? D : KT) <= (int)kPfTmemCols, "tensor memory");
  static_assert(SMEM <= 227 * 1024, "shared memory");
};

// Barriers and small shared state at BAR_OFF.
struct PfShared {
  uint64_t kf[2], ke[2];  // key stage filled / consumed
  uint64_t vf[2], ve[2];  // value stage filled / consumed
  uint64_t sf[2];   // S of tile j (buffer j & 1), and the parameters of its keys
  uint64_t pv[4];   // O holds tile j's product (slot j & 3)
  uint64_t qf;      // query operands staged
  uint32_t tmem;
  int32_t lo[4], hi[4];          // positions some row sees, per 32 rows
  int32_t all_lo[4], all_hi[4];  // positions every row sees
  int32_t dead;                  // a wait ran out
};
static_assert(sizeof(PfShared) <= 256, "shared state");

}  // namespace

// Division of 0 <= n < 2^31 by a fixed d >= 1 without a divide: with
// 2^s >= d > 2^(s-1) and m = floor(2^32 (2^s - d) / d) + 1, n / d =
// (floor(m n / 2^32) + n) >> s (Granlund and Montgomery, "Division by
// invariant integers using multiplication", 1994).
struct FastDiv {
  uint32_t d, m, s;
  __device__ __forceinline__ int div(int n) const {
    return (int)((__umulhi(m, (uint32_t)n) + (uint32_t)n) >> s);
  }
};

struct PrefillArgs {
  FastDiv by_splits, by_heads, by_seqs, by_group;
  int S, T, Hq, H, G, lgP, NP, bt_stride, max_seq_len, max_q, mtiles, splits;
  int shared_len;  // < 0: prompt chunks; else the rows are the batch's sequences and the keys
                   // the first shared_len positions of block-table row 0
  int rot_kind, lgb;
  float hscale;    // the Hadamard scale 1 / sqrt(b)
  float scale2;    // sm_scale log2(e)
  float capk, cap2;  // 2 / cap and cap log2(e); 0: no cap
  int window;      // 0: none
  const __half* q;
  int64_t q_stride;
  const int32_t* q_start;
  const int32_t* seq_lens;
  const int32_t* block_table;
  const float* alibi;
  const int32_t* first_pos;
  const int32_t* prefix_lens;
  const float* quat;
  const float* rope;
  int rope_max_pos;
  const uint8_t* k_codes;
  const uint32_t* k_params;
  const uint8_t* v_codes;
  const uint32_t* v_params;
  __half* out;   // [T][Hq][D] (splits == 1)
  float* part;   // [T][Hq][splits][D + 4], or NULL: one split, out is written
  int32_t* err;
};

// Bounded wait. One that runs out (never expected) is the last of its CTA:
// `dead` makes every later one return at once, so that all barriers still see
// their arrivals and the CTA ends; the flag tells the caller to discard the
// launch's outputs.
__device__ __forceinline__ void pf_wait(uint32_t bar, uint32_t parity, volatile int32_t* dead) {
  for (uint32_t it = 0; it < kMbarSpinLimit; ++it) {
    uint32_t done;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(done)
        : "r"(bar), "r"(parity)
        : "memory");
    if (__all_sync(0xffffffffu, done)) return;
    if ((it & 1023u) == 1023u && *dead) return;
  }
  *dead = 1;
}

// cap tanh(u) (cap in base-2 units, cap2) for a pair with |u| <= kCapSeries:
// an odd polynomial on the FMA pipe (fitted to the relative error, 5.8e-8).
// Scores are far below the cap as a rule; the general form costs two
// special-function results per score beside the exponential's one (a capped
// chunk took 1.9 ms with it alone).
constexpr float kCapSeries = 0.8f;
__device__ __forceinline__ uint64_t pf_cap2(uint64_t u, uint64_t cap2) {
  auto c = [](float x) { return pk(x, x); };
  const uint64_t v = mul2(u, u);
  uint64_t p = fma2(v, c(-0.00435529462993145f), c(0.019093291833996773f));
  p = fma2(p, v, c(-0.053114309906959534f));
  p = fma2(p, v, c(0.13321048021316528f));
  p = fma2(p, v, c(-0.3333267569541931f));
  p = fma2(p, v, c(0.9999999403953552f));
  return mul2(mul2(u, cap2), p);
}

// Channels are visited in the order 0 4 1 5 2 6 3 7 inside each group of 8
// (the nibble pairs that one mask extracts) by every operand.
__device__ __forceinline__ constexpr int pf_perm(int i) { return (i >> 1) + 4 * (i & 1); }

// Barrier of the kPfNW warps that share 32 rows (named barrier 1 + quarter),
// with the ordering of their tensor-memory accesses.
__device__ __forceinline__ void pf_quarter_sync(int quarter) {
  tc_fence_before();
  asm volatile("bar.sync %0, %1;" ::"r"(1 + quarter), "n"(32 * kPfNW) : "memory");
  tc_fence_after();
}
// Barrier of a warpgroup: whether any of its threads holds p.
__device__ __forceinline__ bool pf_group_any(int bar, bool p) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %2, 0;\n\t"
      "barrier.cta.red.or.pred q, %1, 128, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(bar), "r"((uint32_t)p)
      : "memory");
  return r != 0u;
}
// One butterfly stage between columns [a, a + 16) and [b, b + 16) of a row.
__device__ __forceinline__ void pf_cross16(uint32_t scr, int a, int b) {
  uint32_t x[16], y[16];
  tmem_ld16(scr + a, x);
  tmem_ld16(scr + b, y);
  tmem_ld_wait();
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const float p = __uint_as_float(x[i]), q = __uint_as_float(y[i]);
    x[i] = __float_as_uint(p + q);
    y[i] = __float_as_uint(p - q);
  }
  tmem_st16(scr + a, x);
  tmem_st16(scr + b, y);
}

// The rotation of 32 channels [ch, ch + 32) as far as it stays inside them:
// sign flips, butterflies below 32 and the scale, or the quaternion blocks.
template <bool INV>
__device__ __forceinline__ void pf_rotate_in(float (&x)[32], int ch, int rot_kind, int lgb,
                                             float cb, const float* tbl) {
  if (rot_kind == KVQ_ROT_NONE) return;
  if (rot_kind == KVQ_ROT_HADAMARD || rot_kind == KVQ_ROT_HADAMARD_SIGNED) {
    const bool sgn = rot_kind == KVQ_ROT_HADAMARD_SIGNED;
    if (!INV && sgn) {
#pragma unroll
      for (int i = 0; i < 32; ++i) x[i] *= __ldg(tbl + ch + i);
    }
    if (lgb > 4) fwht_regs<32, 5>(x); else fwht_regs<32, 4>(x);
#pragma unroll
    for (int i = 0; i < 32; ++i) x[i] *= cb;
    return;
  }
  if (rot_kind == KVQ_ROT_QUAT) {
    if (INV) quat_inv_regs<32>(x, tbl, ch); else quat_regs<32>(x, tbl, ch);
  } else if (rot_kind == KVQ_ROT_QUAT_FAST) {
    if (INV) quat_fast_inv_regs<32>(x, tbl, ch); else quat_fast_regs<32>(x, tbl, ch);
  } else {
    quat_mat_fly_regs<32, INV>(x, tbl, ch);
  }
}
// The wider Hadamard stages of a row in D tensor-memory columns at `scr`, by
// the row's kPfNW threads (w = 0, 1); each stage's column pairs are dealt out
// evenly. Every thread has stored its own channels before.
template <int D>
__device__ __forceinline__ void pf_rotate_out(uint32_t scr, int w, int quarter, int rot_kind, int lgb) {
  if (rot_kind != KVQ_ROT_HADAMARD && rot_kind != KVQ_ROT_HADAMARD_SIGNED) return;
#pragma unroll 1
  for (int lg = 5; lg < lgb; ++lg) {
    tmem_st_wait();
    pf_quarter_sync(quarter);
    // the D / 2 column pairs of distance 2^lg, 16 at a time: pair group k
    // starts at column (k / g) 2^(lg + 1) + 16 (k % g), g = 2^lg / 16
#pragma unroll 1
    for (int k = w; k < D / 32; k += kPfNW) {
      const int g = (1 << lg) >> 4;
      const int a = (k / g) * (2 << lg) + 16 * (k % g);
      pf_cross16(scr, a, a + (1 << lg));
    }
  }
  tmem_st_wait();
  pf_quarter_sync(quarter);
}

// The power of two that brings a row's largest |q^| into [2^12, 2^13) (lo
// then keeps its bits above the binary16 subnormals) and its inverse; a zero
// query scores 0.
__device__ __forceinline__ void pf_query_scale(float amax, float& mul, float& rs) {
  int e = 12 - (((__float_as_int(amax) >> 23) & 0xFF) - 127);
  e = min(max(e, -126), 126);
  mul = amax > 0.f ? __int_as_float((e + 127) << 23) : 0.f;
  rs = amax > 0.f ? __int_as_float((127 - e) << 23) : 1.f;
}

// x0 mul, x1 mul as binary16 hi + lo pairs (hi + lo is off by 2^-22 of the
// value at most).
__device__ __forceinline__ void pf_split(float x0, float x1, float mul, uint32_t& hi, uint32_t& lo) {
  const __half2 hh = __floats2half2_rn(x0 * mul, x1 * mul);
  const float2 f = __half22float2(hh);
  hi = h2_as_u32(hh);
  lo = h2_as_u32(__floats2half2_rn(fmaf(x0, mul, -f.x), fmaf(x1, mul, -f.y)));
}

// What the softmax keeps per row in shared memory.
struct alignas(16) PfRowState {
  int lo, hi, p;    // interval and position
  float slope2;     // slope of the distance bias, base 2
  float rs, qsum;   // 2^-e of the scaled query, and its sum
  float M, l;       // at the end: reference exponent M - lift and weight sum
};
static_assert(sizeof(PfRowState) == 32, "row state");

// The row of a softmax thread in the first and last part.
struct PfRow {
  bool valid;     // the row exists
  int64_t row;    // token * Hq + head
  int tok, head;
  int p, lo, hi;  // position and the interval it sees
};

// A sequence's n tokens from q0 on are rows of the call (n wraps to a negative
// number or beyond max_q for ends that are not a range).
__device__ __forceinline__ bool pf_range_ok(int q0, int n, int max_q, int T) {
  return q0 >= 0 && n >= 0 && n <= max_q && q0 <= T - n;
}

// A value row is large if its largest dequantized value leaves the binary16 range though its scale and minimum are finite: a constant row of
// 20000 rotates to one channel of 226000. The values of a tile with such a
// row (1048000 at most) are staged times 2^-kPfLarge, and the tile's weights
// enter the product times 2^kPfLarge. (A factor per key, with its correction
// of the weights' sum, cost 2 to 6% of every call's time.)
constexpr int kPfLarge = 5;
enum PfValue { kPfPlain, kPfLargeRow, kPfNotFinite };
__device__ __forceinline__ PfValue pf_value_kind(uint32_t params) {
  const __half2 hp = u32_as_h2(params);
  // (linear in the code: the ends are the minimum and the largest code's value)
  const __half top = __hfma(__float2half(15.f), __low2half(hp), __high2half(hp));
  if (__habs(top) <= __float2half(65504.f)) return kPfPlain;
  const bool fin = (params & 0x7C00u) != 0x7C00u && (params & 0x7C000000u) != 0x7C000000u;
  return fin ? kPfLargeRow : kPfNotFinite;
}

// Four bytes of codes (8 channels) as binary16 pairs in the operands' channel
// order: 64 + c, exactly (the nibble OR-ed into bits 4-7 of the binary16 value
// 64, 0x5400; seven logic operations and no arithmetic).
__device__ __forceinline__ uint4 pf_codes_k(uint32_t x) {
  auto at = [](uint32_t w) {
    uint32_t t;
    asm("lop3.b32 %0, %1, %2, %3, 0xea;" : "=r"(t) : "r"(w), "r"(0x00F000F0u), "r"(0x54005400u));
    return t;
  };
  return make_uint4(at(x << 4), at(x), at(x >> 4), at(x >> 8));
}
// The dequantized values c s + m of 8 channels, rounded once.
__device__ __forceinline__ uint4 pf_codes_v(uint32_t x, __half2 s2, __half2 m2) {
  const uint32_t y = x >> 8;
  auto cv = [&](uint32_t c) { return h2_as_u32(__hfma2(u32_as_h2(c), s2, m2)); };
  return make_uint4(cv(nib_c0(x, 0x000F000Fu, 0)), cv(nib_c0(x, 0x00F000F0u, 1)),
                    cv(nib_c0(y, 0x000F000Fu, 0)), cv(nib_c0(y, 0x00F000F0u, 1)));
}

// OPT: the cap and the distance bias are evaluated (their presence is still a
// run-time, warp-uniform question).
// PAIR: at most 64 rows per (sequence, KV head). Row i is lane 32 (i / 16) +
// i % 16 of its CTA, and 16 lanes on enters what binary16 left of its weights.
template <int D, bool OPT, bool PAIR>
__global__ void __launch_bounds__(kPfThreads, 1) prefill_kernel(const PrefillArgs a) {
  using C = PfCfg<D>;
  constexpr int KT = C::KT, NS = C::NS, BW = C::BW;
  extern __shared__ __align__(1024) uint8_t smem[];
  PfShared& sh = *reinterpret_cast<PfShared*>(smem + C::BAR_OFF);
  PfRowState* const rst = reinterpret_cast<PfRowState*>(smem + C::ROW_OFF);
  const int tid = threadIdx.x, warp = tid / kWarp, lane = tid % kWarp;
  const int wg = tid / 128;

  // ---- which rows: splits fastest, then KV heads, then sequences, then row
  // tiles from the last (the longest under a causal mask) to the first
  const int b0 = blockIdx.x;
  const int b1 = a.by_splits.div(b0);
  const int b2 = a.by_heads.div(b1);
  const int b3 = a.by_seqs.div(b2);
  const int split = b0 - b1 * a.splits;
  const int h = b1 - b2 * a.H;
  const int s = b2 - b3 * (int)a.by_seqs.d;
  const int mt = a.mtiles - 1 - b3;

  pdl_wait();
  pdl_trigger();

  // ---- the sequence
  int q0, n, L;
  bool seq_ok = true;
  if (a.shared_len >= 0) {
    q0 = 0;
    n = a.S;
    L = a.shared_len;
    seq_ok = ((L + (1 << a.lgP) - 1) >> a.lgP) <= a.bt_stride;
  } else {
    q0 = a.q_start[s];
    n = a.q_start[s + 1] - q0;
    L = a.seq_lens[s];
    if (!pf_range_ok(q0, n, a.max_q, a.T)) {  // not a range of the T rows: untouched
      if (tid == 0 && h == 0 && mt == 0 && split == 0) raise_flag(a.err, KVQ_ERRF_SEQ);
      n = 0;
    }
    seq_ok = L >= n && L <= a.max_seq_len && ((L + (1 << a.lgP) - 1) >> a.lgP) <= a.bt_stride &&
             (a.rope == nullptr || L <= a.rope_max_pos);
  }
  const int64_t rows = (int64_t)n * a.G;
  const int64_t r0 = (int64_t)mt * kPfRows;
  if (r0 >= rows) return;  // (whole CTA; nothing allocated yet)
  if (!seq_ok && tid == 0 && h == 0 && mt == 0 && split == 0) raise_flag(a.err, KVQ_ERRF_LEN);

  if (tid == 0) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh.kf[i], 4);
      mbar_init(&sh.ke[i], 1);
      mbar_init(&sh.vf[i], 4);
      mbar_init(&sh.ve[i], 1);
      mbar_init(&sh.sf[i], 2);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      mbar_init(&sh.pv[i], 1);
    }
    mbar_init(&sh.qf, kPfSoft / 32);
    sh.dead = 0;
    mbar_fence_init();
  }
  if (warp == kPfIssue) {
    tmem_alloc(&sh.tmem, kPfTmemCols);
    tmem_relinquish();
  }
  // the row index of a lane of the tile (a number past every row: none)
  auto row_of = [&](int r) {
    if (!PAIR) return (int)r0 + r;
    return (r & 16) ? INT_MAX : 16 * (r >> 5) + (r & 15);
  };
  // ---- the query rows' copies (whole rows, coalesced, to shared memory)
  if (wg < kPfNW) {
#pragma unroll
    for (int k = 0; k < kPfRows * C::LPR / kPfSoft; ++k) {
      const int r = kPfSoft / C::LPR * k + tid / C::LPR, pc = tid % C::LPR;
      const int ri = row_of(r);
      const bool ok = ri < rows;
      const int i = ok ? a.by_group.div(ri) : 0;
      const int hd = ok ? h * a.G + ri - i * a.G : 0;
      cp_async16_zf(smem + C::QS_OFF + r * C::QS_PITCH + 16 * pc,
                    a.q + (int64_t)(ok ? q0 + i : 0) * a.q_stride + (int64_t)hd * D + 8 * pc,
                    ok ? 16u : 0u);
    }
    cp_async_commit();
  }

  // ---- each row's interval, and what the CTA sees
  PfRow R;
  R.valid = false;
  R.row = 0;
  R.tok = R.head = R.p = R.lo = R.hi = 0;
  if (wg < kPfNW) {
    const int ri = row_of(tid & 127);
    R.valid = ri < rows;
    if (R.valid) {
      const int i = a.by_group.div(ri);
      R.tok = q0 + i;
      R.head = h * a.G + ri - i * a.G;
      R.row = (int64_t)R.tok * a.Hq + R.head;
      bool ok = seq_ok;
      if (a.shared_len >= 0) {
        const int Ls = a.seq_lens[i];
        // length 0: an idle slot of a padded batch
        ok = ok && Ls >= a.shared_len && Ls <= a.max_seq_len && Ls > 0 &&
             ((Ls + (1 << a.lgP) - 1) >> a.lgP) <= a.bt_stride &&
             (a.rope == nullptr || Ls <= a.rope_max_pos);
        if (!ok && Ls != 0 && wg == 0) raise_flag(a.err, KVQ_ERRF_LEN);
        R.p = Ls - 1;
      } else {
        R.p = L - n + i;
      }
      R.hi = R.p + 1;
      if (a.shared_len < 0 && a.prefix_lens != nullptr) R.hi = max(R.hi, a.prefix_lens[s]);
      R.hi = min(R.hi, L);
      if (a.window > 0 && R.p >= a.window) R.lo = R.p - a.window + 1;
      if (a.first_pos != nullptr) R.lo = max(R.lo, a.first_pos[R.tok]);
      if (!ok || R.lo >= R.hi) R.lo = R.hi = 0;
    }
    if (wg == 0) {
      const int lo = __reduce_min_sync(0xffffffffu, R.hi > 0 ? R.lo : INT_MAX);
      const int hi = __reduce_max_sync(0xffffffffu, R.hi);
      const int alo = __reduce_max_sync(0xffffffffu, R.valid ? R.lo : 0);
      const int ahi = __reduce_min_sync(0xffffffffu, R.valid ? R.hi : INT_MAX);
      if (lane == 0) {
        sh.lo[warp] = lo;
        sh.hi[warp] = hi;
        sh.all_lo[warp] = alo;
        sh.all_hi[warp] = ahi;
      }
      PfRowState& w = rst[tid];
      w.lo = R.lo;
      w.hi = R.hi;
      w.p = R.p;
      w.slope2 = OPT && a.alibi != nullptr && R.valid ? a.alibi[R.head] * 1.4426950408889634f : 0.f;
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh.tmem;
  const int kv_lo = min(min(sh.lo[0], sh.lo[1]), min(sh.lo[2], sh.lo[3]));
  const int kv_hi = max(max(sh.hi[0], sh.hi[1]), max(sh.hi[2], sh.hi[3]));
  int t0 = 0, t1 = 0;  // key tiles of this split
  if (kv_hi > kv_lo) {
    const int ta = kv_lo / KT, tb = (kv_hi + KT - 1) / KT;
    t0 = ta + (int)((int64_t)(tb - ta) * split / a.splits);
    t1 = ta + (int)((int64_t)(tb - ta) * (split + 1) / a.splits);
  }
  const int ntile = t1 - t0;

  const uint32_t bars = smem_u32(&sh);
  auto wait = [&](const uint64_t* bar, uint32_t parity) {
    pf_wait(bars + (uint32_t)(reinterpret_cast<const uint8_t*>(bar) -
                              reinterpret_cast<const uint8_t*>(&sh)), parity, &sh.dead);
  };

  // One arrival per warp, after all its lanes: a barrier takes the arrivals of
  // a warp's 32 lanes one after the other (with an arrival per thread, 512 per
  // tile, a tile took twice its time).
  auto arrive = [&](uint64_t* bar) {
    __syncwarp();
    if (lane == 0) mbar_arrive(bar);
  };

  if (wg < kPfNW) {
    // =========================== softmax
    // (register shares: 256 x 144 + 256 x 72 + 128 x 40 of the 640 x 96 at launch)
    asm volatile("setmaxnreg.inc.sync.aligned.u32 144;");
    const int qd = warp & 3;                    // lane quarter of the warp
    const int row = tid & 127;
    const uint32_t lane_base = (uint32_t)(qd * 32) << 16;
    const uint32_t o_col = tmem + lane_base + C::O_COL;
    const int c0 = wg * C::HC;                  // the thread's channels of its row
    float* const ex = reinterpret_cast<float*>(smem + C::EX_OFF);
    cp_async_wait<0>();  // every query row is in shared memory
    asm volatile("bar.sync 7, %0;" ::"n"(kPfSoft) : "memory");
    if (ntile > 0) {
      // ---- the query row: RoPE, rotation (O's columns as scratch), then hi + lo
      const float* cs =
          a.rope != nullptr && R.valid && R.hi > 0 ? a.rope + (int64_t)R.p * D + c0 : nullptr;
      const uint4* src =
          reinterpret_cast<const uint4*>(smem + C::QS_OFF + row * C::QS_PITCH + 2 * c0);
#pragma unroll 1
      for (int c = 0; c < C::HC; c += 32) {
        float x[32];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const uint4 u = src[c / 8 + k];
          const uint32_t w4[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 f = __half22float2(u32_as_h2(w4[e]));
            x[8 * k + 2 * e] = f.x;
            x[8 * k + 2 * e + 1] = f.y;
          }
        }
        if (cs != nullptr) rope_regs<32>(x, cs + c);
        __syncwarp();
        pf_rotate_in<false>(x, c0 + c, a.rot_kind, a.lgb, a.hscale, a.quat);
        uint32_t r[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) r[i] = __float_as_uint(x[i]);
        tmem_st32(o_col + c0 + c, r);
      }
      tmem_st_wait();
      // (d = 256: the operand goes where the rows were read)
      if (!C::QT) asm volatile("bar.sync 7, %0;" ::"n"(kPfSoft) : "memory");
      pf_rotate_out<D>(o_col, wg, qd, a.rot_kind, a.lgb);
      float amax = 0.f;
#pragma unroll 1
      for (int c = 0; c < C::HC; c += 32) {
        uint32_t r[32];
        tmem_ld32(o_col + c0 + c, r);
        tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < 32; ++i) amax = fmaxf(amax, fabsf(__uint_as_float(r[i])));
      }
      ex[wg * kPfRows + row] = amax;
      asm volatile("bar.sync %0, %1;" ::"r"(1 + qd), "n"(32 * kPfNW) : "memory");
#pragma unroll
      for (int k = 0; k < kPfNW; ++k) amax = fmaxf(amax, ex[k * kPfRows + row]);
      float mul, rs, qsum = 0.f;
      pf_query_scale(amax, mul, rs);
#pragma unroll 1
      for (int c = 0; c < C::HC; c += 32) {
        uint32_t r[32], hw[16], lw[16];
        tmem_ld32(o_col + c0 + c, r);
        tmem_ld_wait();
#pragma unroll
        for (int k = 0; k < 16; ++k) {
          const int i = 8 * (k >> 2) + (k & 3);
          const float x0 = __uint_as_float(r[i]), x1 = __uint_as_float(r[i + 4]);
          qsum += x0 + x1;
          pf_split(x0, x1, mul, hw[k], lw[k]);
        }
        if (C::QT) {
          const uint32_t qc = tmem + lane_base + C::Q_COL + (c0 + c) / 2;
          tmem_st16(qc, hw);
          tmem_st16(qc + D / 2, lw);
        } else {
          uint8_t* const qh = smem + (row >> 3) * C::GRP + (row & 7) * 16 + ((c0 + c) >> 3) * 128;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            *reinterpret_cast<uint4*>(qh + 128 * k) =
                make_uint4(hw[4 * k], hw[4 * k + 1], hw[4 * k + 2], hw[4 * k + 3]);
            *reinterpret_cast<uint4*>(qh + 128 * k + C::Q_B) =
                make_uint4(lw[4 * k], lw[4 * k + 1], lw[4 * k + 2], lw[4 * k + 3]);
          }
        }
      }
      if (C::QT) tmem_st_wait(); else fence_async_smem();
      tc_fence_before();
      arrive(&sh.qf);
      ex[(kPfNW + wg) * kPfRows + row] = qsum * mul;
      pf_quarter_sync(qd);
      if (wg == 0) {
        rst[row].rs = rs;
        qsum *= mul;
#pragma unroll
        for (int k = 1; k < kPfNW; ++k) qsum += ex[(kPfNW + k) * kPfRows + row];
        rst[row].qsum = qsum;
      }
      pf_quarter_sync(qd);
    }

    // ---- two rows per thread: row rr at 32 qd + 16 wg + 8 rr + lane / 4,
    // columns 8 i + 2 (lane % 4) + {0, 1} of the key tile
    constexpr int NI = KT / 8;   // column groups
    constexpr int NB = NI / 8;   // of 8 groups: one fragment load each
    const int jl = lane & 3;
    const int row0 = 32 * qd + 16 * wg + (lane >> 2);
    const int all_lo = sh.all_lo[qd], all_hi = sh.all_hi[qd];
    const uint32_t lanes16 = lane_base + ((uint32_t)(16 * wg) << 16);  // the warp's 16 rows
    // per row: the reference maximum M, kept as M + slack and as the exponent's
    // offset (lift - M; 0 before any score)
    float thr[2], off[2], l[2], rs[2], qs[2];
#pragma unroll
    for (int rr = 0; rr < 2; ++rr) {
      thr[rr] = -INFINITY;
      off[rr] = 0.f;
      l[rr] = 0.f;
      rs[rr] = rst[row0 + 8 * rr].rs;
      qs[rr] = rst[row0 + 8 * rr].qsum;
    }
    const bool mine = row_of(32 * qd + 16 * wg) < rows;
    if (!mine) {  // a warp without rows only hands its (never read) weights on
      for (int j = 0; j < ntile; ++j) {
        wait(&sh.sf[j & 1], (j >> 1) & 1);
        asm volatile("bar.arrive %0, %1;" ::"r"(8 + (j & 1)), "n"(kPfSoft + 32) : "memory");
      }
    }
    for (int j = mine ? 0 : ntile; j < ntile; ++j) {
      wait(&sh.sf[j & 1], (j >> 1) & 1);
      tc_fence_after();
      // zr[i / 8][4 (i % 8) + 2 rr + e]: row rr, column 8 i + 2 jl + e
      uint32_t zr[NB][32];
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
        tmem_ld_frag<32>(tmem + lanes16 + (j & 1) * KT + 64 * nb, zr[nb]);
      const float4* ks = reinterpret_cast<const float4*>(smem + C::PAR_OFF) + (j & 3) * (KT / 2) + jl;
      const uint32_t* const bads = reinterpret_cast<const uint32_t*>(smem + C::BAD_OFF + (j & 3) * 8 * BW);
      const int base = (t0 + j) * KT;
      tmem_ld_wait();
      // z / rs = s'_j dot + m'_j qsum
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        const float4 pv = ks[4 * i];
#pragma unroll
        for (int rr = 0; rr < 2; ++rr) {
          uint32_t* z = &zr[i >> 3][4 * (i & 7) + 2 * rr];
          const float2 f = upk(fma2(pk(__uint_as_float(z[0]), __uint_as_float(z[1])), pk(pv.x, pv.y),
                                    mul2(pk(pv.z, pv.w), pk(qs[rr], qs[rr]))));
          z[0] = __float_as_uint(f.x);
          z[1] = __float_as_uint(f.y);
        }
      }
      if (OPT) {
        // the pair of column group i in row rr
        auto at = [&](int rr, int i) -> uint32_t* { return &zr[i >> 3][4 * (i & 7) + 2 * rr]; };
        auto get = [&](int rr, int i) {
          const uint32_t* z = at(rr, i);
          return pk(__uint_as_float(z[0]), __uint_as_float(z[1]));
        };
        auto put = [&](int rr, int i, uint64_t v) {
          const float2 f = upk(v);
          uint32_t* z = at(rr, i);
          z[0] = __float_as_uint(f.x);
          z[1] = __float_as_uint(f.y);
        };
        if (a.capk > 0.f) {
          // u = z / cap = z2 capk ln(2) / 2
          bool small = true;
#pragma unroll
          for (int rr = 0; rr < 2; ++rr) {
            const float ku = rs[rr] * a.capk * 0.34657359027997264f;
            float m0 = 0.f, m1 = 0.f;
#pragma unroll
            for (int i = 0; i < NI; ++i) {
              const uint32_t* z = at(rr, i);
              m0 = fmaxf(m0, fabsf(__uint_as_float(z[0])));
              m1 = fmaxf(m1, fabsf(__uint_as_float(z[1])));
            }
            small = small && fmaxf(m0, m1) * ku <= kCapSeries;
          }
          if (__all_sync(0xffffffffu, small)) {
            const uint64_t cp = pk(a.cap2, a.cap2);
#pragma unroll
            for (int rr = 0; rr < 2; ++rr) {
              const float ku = rs[rr] * a.capk * 0.34657359027997264f;
#pragma unroll
              for (int i = 0; i < NI; ++i)
                put(rr, i, pf_cap2(mul2(get(rr, i), pk(ku, ku)), cp));
            }
          } else {
            // cap tanh(z / cap) = cap (1 - 2 / (1 + e^(2 z / cap)))
#pragma unroll
            for (int rr = 0; rr < 2; ++rr) {
              const float k = rs[rr] * a.capk;
#pragma unroll
              for (int i = 0; i < NI; ++i) {
                uint32_t* z = at(rr, i);
#pragma unroll
                for (int e = 0; e < 2; ++e)
                  z[e] = __float_as_uint(
                      fmaf(fast_rcp(1.f + fast_exp2(__uint_as_float(z[e]) * k)), -2.f * a.cap2,
                           a.cap2));
              }
            }
          }
        } else {
#pragma unroll
          for (int rr = 0; rr < 2; ++rr)
#pragma unroll
            for (int i = 0; i < NI; ++i) put(rr, i, mul2(get(rr, i), pk(rs[rr], rs[rr])));
        }
        if (a.alibi != nullptr) {
#pragma unroll
          for (int rr = 0; rr < 2; ++rr) {
            const PfRowState& w = rst[row0 + 8 * rr];
            const float sl = w.slope2, d0 = (float)(base + 2 * jl - w.p);
            // (no later position than the query's, or none at all: no absolute value)
            if (__all_sync(0xffffffffu, base + KT - 1 <= w.p)) {
#pragma unroll
              for (int i = 0; i < NI; ++i)
                put(rr, i, fma2(pk(sl, sl), add2(pk(d0, d0), pk(8.f * i, 8.f * i + 1.f)), get(rr, i)));
            } else {
#pragma unroll
              for (int i = 0; i < NI; ++i) {
                uint32_t* z = at(rr, i);
#pragma unroll
                for (int e = 0; e < 2; ++e)
                  z[e] = __float_as_uint(
                      fmaf(-sl, fabsf(d0 + (float)(8 * i + e)), __uint_as_float(z[e])));
              }
            }
          }
        }
      }
      // positions outside the row's interval, and keys of a bad page
      if (base < all_lo || base + KT > all_hi) {
#pragma unroll
        for (int rr = 0; rr < 2; ++rr) {
          const PfRowState& w = rst[row0 + 8 * rr];
          const int lo = w.lo - base - 2 * jl;
          const uint32_t len = (uint32_t)(w.hi - w.lo);
#pragma unroll
          for (int i = 0; i < 2 * NI; ++i)
            if ((uint32_t)(8 * (i >> 1) + (i & 1) - lo) >= len)
              zr[i >> 4][4 * ((i >> 1) & 7) + 2 * rr + (i & 1)] = 0xff800000u;
        }
      }
      float up = 0.f;  // what the exponents of the tile's weights get on top
      if ((KT == 128 ? bads[0] | bads[1] | bads[2] | bads[3] : bads[0] | bads[1]) != 0u) {
        if ((KT == 128 ? bads[4] | bads[5] | bads[6] | bads[7] : bads[2] | bads[3]) != 0u) {
          up = (float)kPfLarge;
          thr[0] -= kPfSlack;  // (no slack in this tile, so that they stay below 2^12)
          thr[1] -= kPfSlack;
        }
#pragma unroll
        for (int i = 0; i < NI; ++i) {
          const uint32_t bw = (bads[i / 4] & ~bads[BW + i / 4]) >> (8 * (i & 3) + 2 * jl);
#pragma unroll
          for (int e = 0; e < 2; ++e)
            if ((bw >> e) & 1u)
              zr[i >> 3][4 * (i & 7) + e] = zr[i >> 3][4 * (i & 7) + 2 + e] = 0xff800000u;
        }
      }
      // row maxima: of the thread's columns, then of the row's four lanes
      float mx[2];
#pragma unroll
      for (int rr = 0; rr < 2; ++rr) {
        float m0 = -INFINITY, m1 = -INFINITY;
#pragma unroll
        for (int i = 0; i < NI; i += 2) {
          const uint32_t* const z = &zr[i >> 3][4 * (i & 7) + 2 * rr];
          m0 = max3(m0, __uint_as_float(z[0]), __uint_as_float(z[1]));
          m1 = max3(m1, __uint_as_float(z[4]), __uint_as_float(z[5]));
        }
        mx[rr] = fmaxf(m0, m1);
        if (!OPT) mx[rr] *= rs[rr];
      }
      // a score exceeds its row's reference by more than the slack: the rows
      // that do move theirs
      if (__any_sync(0xffffffffu, mx[0] > thr[0] || mx[1] > thr[1])) {
        float al[2];
#pragma unroll
        for (int rr = 0; rr < 2; ++rr) {
          mx[rr] = fmaxf(mx[rr], __shfl_xor_sync(0xffffffffu, mx[rr], 1));
          mx[rr] = fmaxf(mx[rr], __shfl_xor_sync(0xffffffffu, mx[rr], 2));
          const bool mv = mx[rr] > thr[rr];
          const float no = mv ? kPfLift - mx[rr] : off[rr];
          al[rr] = thr[rr] == -INFINITY ? 0.f : fast_exp2(no - off[rr]);
          off[rr] = no;
          if (mv) thr[rr] = mx[rr] + kPfSlack;
          l[rr] *= al[rr];
        }
        if (j > 0) {
          // (S of tile j implies the product of tile j - 2: the parity is not ambiguous)
          wait(&sh.pv[(j - 1) & 3], ((j - 1) >> 2) & 1);
          tc_fence_after();
#pragma unroll 1
          for (int c = 0; c < (PAIR ? 2 * D : D); c += 64) {
            // (the lower part's lanes follow the weights' own)
            const uint32_t at = tmem + lanes16 + C::O_COL + (c & (D - 1)) + (c >= D ? 16u << 16 : 0u);
            uint32_t o[32];
            tmem_ld_frag<32>(at, o);
            tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < 32; ++i)
              o[i] = __float_as_uint(__uint_as_float(o[i]) * al[(i >> 1) & 1]);
            tmem_st_frag<32>(at, o);
          }
        }
      }
      // the weights, rounded to binary16 once; their binary32 sum takes the
      // rounded ones, so that a weight's rounding cancels where it dominates its
      // row (the result's error against float64 3.2e-4 -> 3.0e-4, a percent of
      // time). With lanes to spare (PAIR) they enter as two binary16 parts.
      uint64_t l2[2] = {0ull, 0ull}, mu[2], of[2];
#pragma unroll
      for (int rr = 0; rr < 2; ++rr) {
        const float m1 = OPT ? 1.f : rs[rr];
        mu[rr] = pk(m1, m1);
        of[rr] = pk(off[rr] + up, off[rr] + up);
      }
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
        uint32_t pw[16], lw[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {  // column group i / 2, row i % 2
          const uint32_t* const z = &zr[nb][2 * i];
          const float2 x = upk(fma2(pk(__uint_as_float(z[0]), __uint_as_float(z[1])), mu[i & 1],
                                    of[i & 1]));
          const float p0 = fast_exp2(x.x), p1 = fast_exp2(x.y);
          const __half2 ph = __floats2half2_rn(p0, p1);
          if (PAIR) {
            l2[i & 1] = add2(l2[i & 1], pk(p0, p1));
            const float2 f = __half22float2(ph);
            lw[i] = h2_as_u32(__floats2half2_rn(p0 - f.x, p1 - f.y));
          } else {
            const float2 ls = upk(l2[i & 1]);
            l2[i & 1] = pk(add_h_f(__low2half(ph), ls.x), add_h_f(__high2half(ph), ls.y));
          }
          pw[i] = h2_as_u32(ph);
        }
        const uint32_t at = tmem + lanes16 + C::P_COL + (j & 1) * C::P_STEP + 32 * nb;
        tmem_st_half<16>(at, pw);
        if (PAIR) tmem_st_half<16>(at + (16u << 16), lw);
      }
#pragma unroll
      for (int rr = 0; rr < 2; ++rr) {
        const float2 f = upk(l2[rr]);
        l[rr] = fmaf(f.x + f.y, up != 0.f ? 1.f / (1 << kPfLarge) : 1.f, l[rr]);
        if (up != 0.f && thr[rr] != -INFINITY) thr[rr] = kPfLift - off[rr] + kPfSlack;
      }
      tmem_st_wait();
      tc_fence_before();
      // P is there: a named barrier that only the issuing warp waits at
      asm volatile("bar.arrive %0, %1;" ::"r"(8 + (j & 1)), "n"(kPfSoft + 32) : "memory");
    }
    float Mr = -INFINITY, lr = 0.f;  // of this thread's row in the last part
    if (ntile > 0) {
      wait(&sh.pv[(ntile - 1) & 3], ((ntile - 1) >> 2) & 1);
#pragma unroll
      for (int rr = 0; rr < 2; ++rr) {
        l[rr] += __shfl_xor_sync(0xffffffffu, l[rr], 1);
        l[rr] += __shfl_xor_sync(0xffffffffu, l[rr], 2);
        if (jl == 0) {
          rst[row0 + 8 * rr].l = l[rr];
          // (a row whose every score is NaN never moved its reference: off 0)
          rst[row0 + 8 * rr].M = thr[rr] == -INFINITY && l[rr] == l[rr] ? -INFINITY : -off[rr];
        }
      }
      pf_quarter_sync(qd);
      Mr = rst[row].M;
      lr = rst[row].l;
    }
    __syncwarp();
    // both parts of a row's result (the lower one 16 lanes on)
    auto join = [&](uint32_t (&o)[32]) {
      if (PAIR) {
#pragma unroll
        for (int i = 0; i < 32; ++i)
          o[i] = __float_as_uint(__uint_as_float(o[i]) +
                                 __shfl_down_sync(0xffffffffu, __uint_as_float(o[i]), 16));
      }
    };
    // ---- the thread's channels of its row's result
    if (a.part != nullptr) {
      float* dst = a.part + (R.row * a.splits + split) * (D + 4);
      const bool some = ntile > 0 && Mr != -INFINITY;
      if (ntile > 0) {
#pragma unroll 1
        for (int c = c0; c < c0 + C::HC; c += 32) {
          uint32_t o[32];
          tmem_ld32(o_col + c, o);
          tmem_ld_wait();
          join(o);
          if (R.valid && some) {
#pragma unroll
            for (int k = 0; k < 4; ++k)
#pragma unroll
              for (int q = 0; q < 2; ++q) {
                float4 f;
                f.x = __uint_as_float(o[8 * k + 0 + q]);
                f.y = __uint_as_float(o[8 * k + 2 + q]);
                f.z = __uint_as_float(o[8 * k + 4 + q]);
                f.w = __uint_as_float(o[8 * k + 6 + q]);
                *reinterpret_cast<float4*>(dst + c + 8 * k + 4 * q) = f;
              }
          }
          __syncwarp();
        }
      }
      if (R.valid && wg == 0)
        *reinterpret_cast<float2*>(dst + D) = make_float2(some ? Mr : -INFINITY, lr);
    } else {
      const float inv = lr > 0.f ? 1.f / lr : lr;  // (NaN stays)
      const bool zero = Mr == -INFINITY;
      if (ntile > 0) {
        // normalised, back in channel order, then R^-1
#pragma unroll 1
        for (int c = c0; c < c0 + C::HC; c += 32) {
          uint32_t o[32];
          float x[32];
          tmem_ld32(o_col + c, o);
          tmem_ld_wait();
          join(o);
#pragma unroll
          for (int i = 0; i < 32; ++i)
            x[(i & ~7) + pf_perm(i & 7)] = zero ? 0.f : __uint_as_float(o[i]) * inv;
          pf_rotate_in<true>(x, c, a.rot_kind, a.lgb, a.hscale, a.quat);
#pragma unroll
          for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(x[i]);
          tmem_st32(o_col + c, o);
        }
        tmem_st_wait();
        pf_rotate_out<D>(o_col, wg, qd, a.rot_kind, a.lgb);
      }
#pragma unroll 1
      for (int c = c0; c < c0 + C::HC; c += 32) {
        uint32_t o[32];
        if (ntile > 0) {
          tmem_ld32(o_col + c, o);
          tmem_ld_wait();
        } else {
#pragma unroll
          for (int i = 0; i < 32; ++i) o[i] = 0u;
        }
        if (a.rot_kind == KVQ_ROT_HADAMARD_SIGNED) {
#pragma unroll
          for (int i = 0; i < 32; ++i)
            o[i] = __float_as_uint(__uint_as_float(o[i]) * __ldg(a.quat + c + i));
        }
        // whole rows leave through shared memory, coalesced
        uint4* const st = reinterpret_cast<uint4*>(smem + C::QS_OFF + row * C::QS_PITCH + 2 * c);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          uint32_t w[4];
#pragma unroll
          for (int e = 0; e < 4; ++e)
            w[e] = h2_as_u32(__floats2half2_rn(__uint_as_float(o[8 * k + 2 * e]),
                                               __uint_as_float(o[8 * k + 2 * e + 1])));
          st[k] = make_uint4(w[0], w[1], w[2], w[3]);
        }
      }
      asm volatile("bar.sync %0, %1;" ::"r"(1 + qd), "n"(32 * kPfNW) : "memory");
      constexpr int RPI = 32 / C::LPR;  // rows per instruction
#pragma unroll
      for (int k = 0; k < 32 / kPfNW / RPI; ++k) {
        const int r = 32 / kPfNW * wg + RPI * k + lane / C::LPR;  // row of the quarter
        const int orow = __shfl_sync(0xffffffffu, (int)R.row, r);
        const bool ok = __shfl_sync(0xffffffffu, (int)R.valid, r) != 0;
        const uint4 u = *reinterpret_cast<const uint4*>(
            smem + C::QS_OFF + (32 * qd + r) * C::QS_PITCH + 16 * (lane % C::LPR));
        if (ok) *reinterpret_cast<uint4*>(a.out + (int64_t)orow * D + 8 * (lane % C::LPR)) = u;
      }
    }
    tc_fence_before();
  } else if (wg < kPfNW + 2) {
    // =========================== keys (warpgroup 2) and values (3) to binary16 operands
    asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
    const bool isv = wg == kPfNW + 1;
    const int dt = tid & 127;
    const int key = dt % KT, part = dt / KT;  // 128 channels of one key
    const int P1 = (1 << a.lgP) - 1;
    const int32_t* bt = a.block_table + (int64_t)(a.shared_len >= 0 ? 0 : s) * a.bt_stride;
    const uint8_t* const codes = (isv ? a.v_codes : a.k_codes) + part * 64;
    const uint32_t* const params = isv ? a.v_params : a.k_params;
    // (a tile is whole pages: the slot in its page is the key's own)
    const uint32_t span = (uint32_t)(kv_hi - kv_lo);
    const int tok0 = t0 * KT + key;
    const int32_t* const bt0 = bt + (tok0 >> a.lgP);
    const int pages = KT >> a.lgP;  // of a tile
    auto page_of = [&](int j) {
      return j < ntile && (uint32_t)(tok0 + j * KT - kv_lo) < span ? bt0[j * pages] : INT_MIN;  // not needed
    };
    const int64_t row0 = ((int64_t)h << a.lgP) + (key & P1);
    const uint8_t* const codes0 = codes + row0 * (D / 2);
    const uint32_t* const params0 = params + row0;
    const int64_t prows = (int64_t)a.H << a.lgP;  // rows of a page
    // A value that is no finite number would turn every row of the tile to NaN
    // (0 x NaN), also those that do not see it: it enters as zeros, and its key
    // with a NaN scale, which reaches the rows that see it and no other.
    const uint32_t* const vparams0 = a.v_params + row0;
    uint4 cr[2][4];         // codes of two tiles
    uint32_t pr[2], vr[2];  // parameters; key warps: the values' too
    uint32_t bad = 0;       // bit st: the page of registers st is bad
    auto load = [&](int page, int st) {
      const bool ok = (uint32_t)page < (uint32_t)a.NP;
      bad = (bad & ~(1u << st)) | ((uint32_t)(!ok && page != INT_MIN) << st);
      if (ok) {
        const int64_t row = page * prows;
        const uint4* src = reinterpret_cast<const uint4*>(codes0 + row * (D / 2));
#pragma unroll
        for (int i = 0; i < 4; ++i) cr[st][i] = __ldg(src + i);
        pr[st] = __ldg(params0 + row);
        vr[st] = isv ? 0u : __ldg(vparams0 + row);
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) cr[st][i] = make_uint4(0u, 0u, 0u, 0u);
        pr[st] = vr[st] = 0u;
      }
    };
    uint8_t* const dst0 = smem + (isv ? C::V_OFF : C::K_OFF) + (key >> 3) * C::GRP + part * 2048 +
                          (key & 7) * 16;
    uint64_t* const full = isv ? sh.vf : sh.kf;
    uint64_t* const empty = isv ? sh.ve : sh.ke;
    // tile j (registers st): stage, then load tile j + 2 with the page pg2
    auto step = [&](int j, int st, int pg2) {
      const int sl = NS == 2 ? (j & 1) : 0;
      const PfValue kind = pf_value_kind(isv ? pr[st] : vr[st]);
      // one warp polls for its warpgroup (polls of all eight took a tenth of
      // the issue slots beside the softmax)
      if (j >= NS && (warp & 3) == 0) wait(&empty[sl], NS == 2 ? ((j >> 1) - 1) & 1 : (j - 1) & 1);
      const bool large = pf_group_any(5 + (int)isv, kind == kPfLargeRow);
      uint8_t* const dst = dst0 + sl * C::K_B;
      const uint32_t w4[16] = {
          cr[st][0].x, cr[st][0].y, cr[st][0].z, cr[st][0].w, cr[st][1].x, cr[st][1].y,
          cr[st][1].z, cr[st][1].w, cr[st][2].x, cr[st][2].y, cr[st][2].z, cr[st][2].w,
          cr[st][3].x, cr[st][3].y, cr[st][3].z, cr[st][3].w};
      if (isv) {
        __half2 hp = u32_as_h2(pr[st]);
        if (large) hp = __hmul2(hp, __float2half2_rn(1.f / (1 << kPfLarge)));
        if (kind == kPfNotFinite) hp = __float2half2_rn(0.f);
        const __half2 s2 = __low2half2(hp), m2 = __high2half2(hp);
#pragma unroll
        for (int w = 0; w < 16; ++w)
          *reinterpret_cast<uint4*>(dst + w * 128) = pf_codes_v(w4[w], s2, m2);
      } else {
        float* ks = reinterpret_cast<float*>(smem + C::PAR_OFF) + (j & 3) * 2 * KT +
                    (key >> 1) * 4 + (key & 1);
        const bool bd = (bad >> st) & 1u;
        const uint32_t lm = __ballot_sync(0xffffffffu, kind == kPfLargeRow);
        const uint32_t bm = __ballot_sync(0xffffffffu, bd) | lm;
        if (part == 0) {
          const float2 sm = __half22float2(u32_as_h2(pr[st]));
          ks[0] = kind == kPfNotFinite ? __int_as_float(0x7FC00000) : sm.x * a.scale2;
          ks[2] = fmaf(-64.f, sm.x, sm.y) * a.scale2;  // (the operand holds 64 + c)
          if (lane == 0) {
            uint32_t* const bw = reinterpret_cast<uint32_t*>(smem + C::BAD_OFF + (j & 3) * 8 * BW);
            bw[key >> 5] = bm;
            bw[BW + (key >> 5)] = lm;
          }
          if (bd && h == 0 && ((key & P1) == 0 || tok0 + j * KT == kv_lo)) raise_flag(a.err, KVQ_ERRF_PAGE);
        }
#pragma unroll
        for (int w = 0; w < 16; ++w) *reinterpret_cast<uint4*>(dst + w * 128) = pf_codes_k(w4[w]);
      }
      fence_async_smem();
      arrive(&full[sl]);
      load(pg2, st);
    };
    if (ntile > 0) {
      int pga = page_of(0), pgb = page_of(1);
      load(pga, 0);
      load(pgb, 1);
      pga = page_of(2);
      pgb = page_of(3);
      for (int j = 0; j < ntile; j += 2) {
        step(j, 0, pga);
        pga = page_of(j + 4);
        if (j + 1 >= ntile) break;
        step(j + 1, 1, pgb);
        pgb = page_of(j + 5);
      }
    }
  } else {
    // =========================== the issuing warp
    asm volatile("setmaxnreg.dec.sync.aligned.u32 40;");
    if (warp == kPfIssue && ntile > 0) {
      constexpr uint32_t idS = umma_idesc_f16(kPfRows, KT, 0);
      constexpr uint32_t idO = umma_idesc_f16(kPfRows, D, 1);
      const bool one = elect_one();
      // keys: rows are keys, K-major; values: rows (the K dimension) are keys
      const uint64_t kd0 = umma_desc_kmajor(smem_u32(smem + C::K_OFF), 128, C::GRP);
      const uint64_t vd0 = umma_desc_kmajor(smem_u32(smem + C::V_OFF), C::GRP, 128);
      const uint64_t qd = umma_desc_kmajor(smem_u32(smem), 128, C::GRP);
      wait(&sh.qf, 0);
      // Round i: the products P V of tile i - 2, then Q K^T of tile i. With two
      // stages the operands of both are waited for before P, the last to come;
      // with one the keys of tile i are widened while P V runs. Where P lies
      // under the S that Q K^T writes, P V completes first.
      for (int i = 0; i < ntile + 2; ++i) {
        const int j = i - 2;
        const int sk = NS == 2 ? (i & 1) : 0, sv = NS == 2 ? (j & 1) : 0;
        if (NS == 2 && i < ntile) wait(&sh.kf[sk], (i >> 1) & 1);
        if (j >= 0) {
          wait(&sh.vf[sv], NS == 2 ? (j >> 1) & 1 : j & 1);
          asm volatile("bar.sync %0, %1;" ::"r"(8 + (j & 1)), "n"(kPfSoft + 32) : "memory");
        }
        tc_fence_after();
        if (one) {
          if (j >= 0) {
            const uint32_t p = tmem + C::P_COL + (j & 1) * C::P_STEP, d = tmem + C::O_COL;
            const uint64_t vd = vd0 + (uint64_t)(sv * (C::K_B >> 4));
#pragma unroll
            for (int k = 0; k < KT / 16; ++k)
              umma_f16_ts(d, p + 8 * k, vd + (uint64_t)(k * (2 * C::GRP >> 4)), idO, j > 0 || k > 0);
            umma_commit(&sh.pv[j & 3]);
            umma_commit(&sh.ve[sv]);
          }
        }
        __syncwarp();
        if (C::P_COL == 0 && j >= 0 && i < ntile) {
          wait(&sh.pv[j & 3], (j >> 2) & 1);
          tc_fence_after();
        }
        if (NS == 1 && i < ntile) {
          wait(&sh.kf[sk], i & 1);
          tc_fence_after();
        }
        if (one) {
          if (i < ntile) {
            const uint64_t kd = kd0 + (uint64_t)(sk * (C::K_B >> 4));
            const uint32_t d = tmem + (i & 1) * KT;
#pragma unroll
            for (int half = 0; half < 2; ++half)  // hi, then lo
#pragma unroll
              for (int k = 0; k < D / 16; ++k) {
                if (C::QT)
                  umma_f16_ts(d, tmem + C::Q_COL + half * (D / 2) + 8 * k, kd + (uint64_t)(16 * k),
                              idS, half + k > 0);
                else
                  umma_f16_ss(d, qd + (uint64_t)(half * (C::Q_B >> 4) + 16 * k),
                              kd + (uint64_t)(16 * k), idS, half + k > 0);
              }
            umma_commit(&sh.sf[i & 1]);
            umma_commit(&sh.ke[sk]);
            // (an ordinary arrival hands on what the wait for the keys saw: the parameters)
            mbar_arrive(&sh.sf[i & 1]);
          }
        }
        __syncwarp();
      }
      // nothing is in flight when tensor memory is given back
      wait(&sh.pv[(ntile - 1) & 3], ((ntile - 1) >> 2) & 1);
    }
    __syncwarp();
  }
  __syncthreads();
  if (tid == 0 && sh.dead) raise_flag(a.err, KVQ_ERRF_TIMEOUT);
  tc_fence_after();
  if (warp == kPfIssue) tmem_dealloc(tmem, kPfTmemCols);
}

// ---------------------------------------------------------------------------
// Merge of split partial results, one warp per (token, query head): the
// partials of up to two launches (the shared prefix's and the sequences' own)
// are combined by log-sum-exp, normalised, rotated back and rounded to
// binary16. A partial without weight (maximum -inf) is not read.
// ---------------------------------------------------------------------------
struct PfMergeArgs {
  int rows, G, rot_kind, lgb;
  int na;             // splits of part_a
  int nb, nhi;        // splits of part_b: nb for the first nhi KV-head pairs, nb - 1 after; 0: none
  const float* quat;
  const float* part_a;  // [rows][na][D + 4]
  const float* part_b;  // [rows][nb][D + 4]
  __half* out;
  // prompt chunks: the rows that no valid range of q_start holds have no
  // partials and are left as they are (NULL: every row has them)
  const int32_t* q_start;
  int S, T, Hq, max_q;
};

template <int D>
__global__ void __launch_bounds__(128) prefill_merge_kernel(const PfMergeArgs m) {
  constexpr int CPL = D / 32;
  const int lane = threadIdx.x % kWarp;
  const int64_t gw = (int64_t)blockIdx.x * 4 + threadIdx.x / kWarp;
  // (an input of the call: complete since the launch before this one passed
  // its own wait, which is before it let this one start)
  bool held = m.q_start == nullptr;
  if (!held) {
    const int tok = (int)(gw / m.Hq);
    for (int s = lane; s < m.S; s += kWarp) {
      const int b = __ldcg(m.q_start + s), n = __ldcg(m.q_start + s + 1) - b;
      held = held || (pf_range_ok(b, n, m.max_q, m.T) && tok >= b && tok - b < n);
    }
    held = __any_sync(0xffffffffu, held);
  }
  pdl_wait();
  pdl_trigger();
  if (gw >= m.rows || !held) return;
  float x[CPL];
#pragma unroll
  for (int c = 0; c < CPL; ++c) x[c] = 0.f;
  float Mr = -INFINITY, Ls = 0.f;
#pragma unroll 1
  for (int set = 0; set < 2; ++set) {
    const float* src = set == 0 ? m.part_a + gw * m.na * (D + 4) : m.part_b + gw * m.nb * (D + 4);
    const int np = set == 0 ? m.na : m.nb == 0 ? 0 : gw / m.G < m.nhi ? m.nb : m.nb - 1;
    for (int i0 = 0; i0 < np; i0 += kWarp) {
      // 32 splits at a time: lane i holds split i0 + i's (M, l)
      const int i = i0 + lane;
      float2 ml = make_float2(-INFINITY, 0.f);
      if (i < np) ml = __ldcg(reinterpret_cast<const float2*>(src + (int64_t)i * (D + 4) + D));
      float mx = ml.x;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
      const float Mn = fmaxf(Mr, mx);
      const float al = Mn == Mr ? 1.f : Mr == -INFINITY ? 0.f : fast_exp2(Mr - Mn);
      Mr = Mn;
      Ls *= al;
#pragma unroll
      for (int c = 0; c < CPL; ++c) x[c] *= al;
      const float w = ml.x == -INFINITY ? 0.f : fast_exp2(ml.x - Mn);
      float ls = w * ml.y;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) ls += __shfl_xor_sync(0xffffffffu, ls, o);
      Ls += ls;
      const uint32_t any = __ballot_sync(0xffffffffu, ml.x != -INFINITY);
      const int cnt = min(np - i0, kWarp);
      // 8 rows in flight at a time
      for (int k0 = 0; k0 < cnt; k0 += 8) {
        float4 f[8][CPL / 4];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const bool in = k0 + k < cnt && ((any >> (k0 + k)) & 1u);
          const float4* p =
              reinterpret_cast<const float4*>(src + (int64_t)(i0 + k0 + k) * (D + 4) + lane * CPL);
#pragma unroll
          for (int c = 0; c < CPL / 4; ++c)
            f[k][c] = in ? __ldcg(p + c) : make_float4(0.f, 0.f, 0.f, 0.f);
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const float wk = __shfl_sync(0xffffffffu, w, (k0 + k) & 31);
#pragma unroll
          for (int c = 0; c < CPL / 4; ++c) {
            x[4 * c] = fmaf(wk, f[k][c].x, x[4 * c]);
            x[4 * c + 1] = fmaf(wk, f[k][c].y, x[4 * c + 1]);
            x[4 * c + 2] = fmaf(wk, f[k][c].z, x[4 * c + 2]);
            x[4 * c + 3] = fmaf(wk, f[k][c].w, x[4 * c + 3]);
          }
        }
      }
    }
  }
  const float inv = Ls > 0.f ? 1.f / Ls : Ls;  // no weight: 0 (NaN stays)
#pragma unroll
  for (int c = 0; c < CPL; ++c) x[c] *= inv;
  row_unrotate<CPL>(x, lane, m.rot_kind, m.lgb, m.quat);
  uint32_t w[CPL / 2];
#pragma unroll
  for (int c = 0; c < CPL / 2; ++c) w[c] = h2_as_u32(__floats2half2_rn(x[2 * c], x[2 * c + 1]));
  __half* dst = m.out + gw * D + lane * CPL;
  if (CPL == 4)
    *reinterpret_cast<uint2*>(dst) = make_uint2(w[0], w[1]);
  else
    *reinterpret_cast<uint4*>(dst) = make_uint4(w[0], w[1], w[CPL / 2 - 2], w[CPL / 2 - 1]);
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------

static int log2i(int x) {
  int l = 0;
  while (l < 30 && (1 << l) < x) ++l;
  return l;
}

static FastDiv fast_div(uint32_t d) {
  FastDiv f;
  f.d = d;
  f.s = (uint32_t)log2i((int)d);
  f.m = (uint32_t)((((uint64_t)1 << 32) * (((uint64_t)1 << f.s) - d)) / d + 1);
  return f;
}

// Splits of the key tiles: enough CTAs for one per SM when the rows alone
// give fewer (each split holds at least two key tiles).
static PrefillPlan plan_rows(int D, int H, int64_t nseq, int64_t rows_per_seq, int64_t total_rows,
                             int64_t max_keys) {
  PrefillPlan pl{};
  const int rt = kPfRows;
  const int kt = D == 128 ? 128 : 64;
  pl.mtiles = (rows_per_seq + rt - 1) / rt;
  if (pl.mtiles < 1) pl.mtiles = 1;
  // at most half a tile's rows: the free lanes take the weights' lower parts and
  // the rows lie on all four schedulers. 8 sequences x 20 rows: 35.0 -> 34.2 us,
  // error 3.1e-4 -> 2.9e-4 (35.5 us since P V completes before the next S); a
  // 512-token prefix of 16 rows: 16.3 -> 17.1 us (two tiles per CTA, each with a
  // second store), 3.0e-4 -> 2.7e-4
  pl.pair = rows_per_seq <= rt / 2;
  const int64_t ctas = nseq * H * pl.mtiles;
  const int64_t tiles = (max_keys + kt - 1) / kt;
  const int sms = device_sm_count() > 0 ? device_sm_count() : 148;
  int64_t sp = sms / (ctas > 0 ? ctas : 1);
  if (sp > tiles / 2) sp = tiles / 2;
  if (sp < 1) sp = 1;
  pl.splits = (int)sp;
  pl.ctas = ctas * sp;
  pl.workspace = sp > 1 ? (size_t)total_rows * sp * (D + 4) * sizeof(float) : 0;
  return pl;
}

PrefillPlan prefill_plan(const kvq_cache_desc& d, int32_t S, int32_t Hq, int32_t T, int32_t max_q,
                         int32_t max_seq_len) {
  const int G = Hq / d.num_kv_heads;
  if (max_q > T) max_q = T > 0 ? T : 1;  // (an upper bound; no sequence has more tokens than all)
  return plan_rows(d.head_dim, d.num_kv_heads, S, (int64_t)max_q * G, (int64_t)T * Hq, max_seq_len);
}

template <int D, bool OPT, bool PAIR>
static cudaError_t launch_prefill(PrefillArgs a, int grid, cudaStream_t st) {
  a.by_splits = fast_div((uint32_t)a.splits);
  a.by_heads = fast_div((uint32_t)a.H);
  a.by_seqs = fast_div(a.shared_len >= 0 ? 1u : (uint32_t)a.S);
  a.by_group = fast_div((uint32_t)a.G);
  auto kern = prefill_kernel<D, OPT, PAIR>;
  cudaError_t e =
      cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, PfCfg<D>::SMEM);
  if (e != cudaSuccess) return e;
  e = launch_pdl(kern, grid, kPfThreads, PfCfg<D>::SMEM, st, a);
  return e != cudaSuccess ? e : cudaGetLastError();
}

static void fill_args(PrefillArgs& a, const kvq_cache_desc& d, int32_t S, int32_t Hq,
                      const void* q, const int32_t* seq_lens, int32_t max_seq_len,
                      const int32_t* block_table, int32_t bt_stride, float sm_scale,
                      const kvq_score_desc* sc, const uint8_t* k_codes, const void* k_params,
                      const uint8_t* v_codes, const void* v_params, int32_t* err) {
  a.S = S; a.Hq = Hq; a.H = d.num_kv_heads; a.G = Hq / d.num_kv_heads;
  a.lgP = log2i(d.page_size); a.NP = d.num_pages; a.bt_stride = bt_stride;
  a.max_seq_len = max_seq_len;
  a.rot_kind = d.rot_kind; a.lgb = log2i(d.rot_block);
  a.hscale = hadamard_scale(a.lgb);
  a.scale2 = (float)((double)sm_scale * 1.4426950408889634074);
  score_cap(sc, a.capk, a.cap2);
  a.window = sc ? sc->window : 0;
  a.alibi = sc ? sc->alibi : nullptr;
  a.first_pos = sc ? sc->first_pos : nullptr;
  a.prefix_lens = sc ? sc->prefix_lens : nullptr;
  a.q = static_cast<const __half*>(q);
  a.seq_lens = seq_lens; a.block_table = block_table;
  a.quat = d.quat; a.rope = d.rope; a.rope_max_pos = d.rope_max_pos;
  a.k_codes = k_codes; a.k_params = static_cast<const uint32_t*>(k_params);
  a.v_codes = v_codes; a.v_params = static_cast<const uint32_t*>(v_params);
  a.err = err;
}

template <int D, bool OPT>
static cudaError_t launch_pair(const PrefillArgs& a, bool pair, int grid, cudaStream_t st) {
  return pair ? launch_prefill<D, OPT, true>(a, grid, st) : launch_prefill<D, OPT, false>(a, grid, st);
}

static cudaError_t launch_any(const PrefillArgs& a, int D, const PrefillPlan& pl, cudaStream_t st) {
  const bool opt = a.capk > 0.f || a.alibi != nullptr;
  const int grid = (int)pl.ctas;
  if (D == 128)
    return opt ? launch_pair<128, true>(a, pl.pair, grid, st) : launch_pair<128, false>(a, pl.pair, grid, st);
  return opt ? launch_pair<256, true>(a, pl.pair, grid, st) : launch_pair<256, false>(a, pl.pair, grid, st);
}

static cudaError_t launch_merge(const kvq_cache_desc& d, int64_t rows, int G, int na, int nb,
                                int nhi, const float* pa, const float* pb, void* out,
                                const PrefillArgs* rows_of, cudaStream_t st) {
  PfMergeArgs m;
  m.rows = (int)rows; m.G = G; m.rot_kind = d.rot_kind; m.lgb = log2i(d.rot_block);
  m.na = na; m.nb = nb; m.nhi = nhi; m.quat = d.quat; m.part_a = pa; m.part_b = pb;
  m.out = static_cast<__half*>(out);
  m.q_start = rows_of ? rows_of->q_start : nullptr;
  m.S = rows_of ? rows_of->S : 0;
  m.T = rows_of ? rows_of->T : 0;
  m.Hq = rows_of ? rows_of->Hq : 1;
  m.max_q = rows_of ? rows_of->max_q : 0;
  const int grid = (int)((rows + 3) / 4);
  cudaError_t e = d.head_dim == 128 ? launch_pdl(prefill_merge_kernel<128>, grid, 128, 0, st, m)
                                    : launch_pdl(prefill_merge_kernel<256>, grid, 128, 0, st, m);
  return e != cudaSuccess ? e : cudaGetLastError();
}

int prefill_launch(const kvq_cache_desc& d, int32_t S, int32_t Hq, int32_t T, const void* q,
                   int64_t q_stride, const int32_t* q_start, int32_t max_q,
                   const int32_t* seq_lens, int32_t max_seq_len, const int32_t* block_table,
                   int32_t bt_stride, float sm_scale, const kvq_score_desc* sc,
                   const uint8_t* k_codes, const void* k_params, const uint8_t* v_codes,
                   const void* v_params, void* out, void* workspace, size_t workspace_bytes,
                   int32_t* err, cudaStream_t st) {
  if ((int64_t)T * Hq > INT_MAX - 256) return KVQ_ERR_UNSUPPORTED;  // (row numbers are 32-bit)
  const PrefillPlan pl = prefill_plan(d, S, Hq, T, max_q, max_seq_len);
  if (pl.workspace > 0 && (workspace == nullptr || workspace_bytes < pl.workspace))
    return KVQ_ERR_WORKSPACE;
  if (pl.ctas > INT_MAX) return KVQ_ERR_UNSUPPORTED;
  PrefillArgs a;
  fill_args(a, d, S, Hq, q, seq_lens, max_seq_len, block_table, bt_stride, sm_scale, sc, k_codes,
            k_params, v_codes, v_params, err);
  a.T = T; a.q_stride = q_stride; a.q_start = q_start; a.max_q = max_q;
  a.mtiles = (int)pl.mtiles; a.splits = pl.splits; a.shared_len = -1;
  a.out = static_cast<__half*>(out);
  a.part = pl.splits > 1 ? static_cast<float*>(workspace) : nullptr;
  if (launch_any(a, d.head_dim, pl, st) != cudaSuccess) return KVQ_ERR_CUDA;
  if (pl.splits > 1 &&
      launch_merge(d, (int64_t)T * Hq, a.G, pl.splits, 0, 0, a.part, nullptr, out, &a, st) !=
          cudaSuccess)
    return KVQ_ERR_CUDA;
  return KVQ_OK;
}

SharedPlan shared_plan(const kvq_cache_desc& d, int32_t S, int32_t Hq, int32_t prefix_len,
                       int32_t max_seq_len) {
  SharedPlan p{};
  if (prefix_len > 0) {
    p.prefix = plan_rows(d.head_dim, d.num_kv_heads, 1, (int64_t)S * (Hq / d.num_kv_heads),
                         (int64_t)S * Hq, prefix_len);
    p.prefix_bytes = (size_t)S * Hq * p.prefix.splits * (d.head_dim + 4) * sizeof(float);
  }
  p.own = decode_scored_plan(d, S, Hq, max_seq_len, prefix_len, nullptr);
  p.workspace = p.prefix_bytes + p.own.workspace;
  return p;
}

int shared_launch(const kvq_cache_desc& d, int32_t S, int32_t Hq, const void* q,
                  int32_t prefix_len, const int32_t* seq_lens, int32_t max_seq_len,
                  const int32_t* block_table, int32_t bt_stride, float sm_scale,
                  const kvq_score_desc* sc, const uint8_t* k_codes, const void* k_params,
                  const uint8_t* v_codes, const void* v_params, void* out, void* workspace,
                  size_t workspace_bytes, int32_t* err, cudaStream_t st) {
  if ((int64_t)S * Hq > INT_MAX - 256) return KVQ_ERR_UNSUPPORTED;
  const SharedPlan pl = shared_plan(d, S, Hq, prefix_len, max_seq_len);
  if (workspace == nullptr || workspace_bytes < pl.workspace) return KVQ_ERR_WORKSPACE;
  if (pl.prefix.ctas > INT_MAX) return KVQ_ERR_UNSUPPORTED;
  float* const pa = static_cast<float*>(workspace);
  float* const pb = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + pl.prefix_bytes);
  if (prefix_len > 0) {
    PrefillArgs a;
    fill_args(a, d, S, Hq, q, seq_lens, max_seq_len, block_table, bt_stride, sm_scale, sc, k_codes,
              k_params, v_codes, v_params, err);
    a.T = S; a.q_stride = (int64_t)Hq * d.head_dim; a.q_start = nullptr; a.max_q = S;
    a.mtiles = (int)pl.prefix.mtiles; a.splits = pl.prefix.splits; a.shared_len = prefix_len;
    a.out = nullptr;
    a.part = pa;
    if (launch_any(a, d.head_dim, pl.prefix, st) != cudaSuccess) return KVQ_ERR_CUDA;
  }
  const int r = decode_scored_split_launch(d, S, Hq, q, seq_lens, max_seq_len, block_table,
                                           bt_stride, sm_scale, sc, prefix_len, k_codes, k_params,
                                           v_codes, v_params, pb, err, st, prefix_len > 0);
  if (r != KVQ_OK) return r;
  // (a window shrinks the own part's plan: the launch's own counts)
  const DecodePlan own = decode_scored_plan(d, S, Hq, max_seq_len, prefix_len, sc);
  return launch_merge(d, (int64_t)S * Hq, Hq / d.num_kv_heads, pl.prefix.splits, own.splits,
                      own.nhi, pa, pb, out, nullptr, st) == cudaSuccess ? KVQ_OK : KVQ_ERR_CUDA;
}

}  // namespace kvq
