// Attention of many query rows over the rotated paged cache: prompt chunks
// (kvq_paged_prefill_attn) and the shared prefix of a batch
// (kvq_shared_prefix_decode_attn), with scored options.
//
// Mathematics. A row is one (query token, query head) pair; the G heads of a
// KV head's group and the tokens of a sequence (or, over a shared prefix, the
// sequences of the batch) are the rows of one matrix product with that KV
// head's keys. With q^ = R q, codes c, row scale s and minimum m of a key,
//   z_j = sm_scale (s_j sum_i (c_ji - 8) q^_i + (m_j + 8 s_j) sum_i q^_i),
// then the cap, the distance bias and the interval mask [lo, hi) of the row,
// and out = R^-1 sum_j p_j v^_j with the online softmax in base 2.
//
// Work split. One CTA per (sequence, KV head, 128 rows, split of the key
// tiles). Warpgroups 0 and 1 are the softmax: two threads per row, each with
// half of a key tile's scores (the row maximum is exchanged in shared memory,
// the weight sums are joined at the end). Warpgroups 2 and 3 widen the packed
// keys and values of the next tiles to binary16 operands in shared memory,
// one key per thread, with the codes of two tiles ahead in registers. One
// warp issues every tcgen05.mma: S = Q K^T and O += P V with P read from
// tensor memory. S has two buffers, so one tile's softmax runs under the
// products of its neighbours.
//
// Precision. Key codes enter as c - 8, exact in binary16; the row's s and m
// are applied in binary32 after the product. The rotated query is scaled by a
// power of two per row and split into binary16 hi + lo (about 22 bits): rounded to
// one binary16 it would cost |z| 2^-12 in every exponent, which for outlier
// keys (|z| of 10 and more) is several times the output's own rounding. p and
// v^ are rounded to binary16 once each (2^-12 relative on average, like the
// binary16 output). All sums are binary32.

#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <climits>
#include <type_traits>

#include "kvq_device.cuh"
#include "kvq_launch.h"
#include "kvq_rotate.cuh"
#include "kvq_tcgen05.cuh"

namespace kvq {

namespace {

constexpr int kPfThreads = 640;   // softmax 2 x 128, keys, values, and the issuing warp's group
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
  static constexpr int KC = KT / 2;               // keys per softmax thread
  static constexpr int HC = D / 2;                // channels per softmax thread
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
  static constexpr int PAR_OFF = V_OFF + NS * K_B;      // 4 slots x (scale, offset) x KT floats
  static constexpr int BAD_OFF = PAR_OFF + 8 * KT * 4;  // 4 slots x 4 words
  static constexpr int EX_OFF = BAD_OFF + 64;           // exchange: 2 slots x 2 halves x 128 floats
  static constexpr int BAR_OFF = EX_OFF + 2 * 2 * kPfRows * 4;
  static constexpr int SMEM = BAR_OFF + 256;
  // tensor-memory columns: S0, S1, O, then Q (d = 128) or P (d = 256)
  static constexpr int O_COL = 2 * KT;
  static constexpr int Q_COL = O_COL + D;
  // weights P of tile j: over S j & 1 where both products have one shape (M 128, N 128:
  // such products are executed in issue order, so the next S cannot overwrite
  // a P still being read); in columns of their own at d = 256, whose products
  // (N 64 and N 256) have no such order
  static constexpr int P_COL = QT ? 0 : O_COL + D;
  static constexpr int P_STEP = QT ? KT : KT / 2;
  static_assert(O_COL + D + (QT ? D : KT) <= (int)kPfTmemCols, "tensor memory");
  static_assert(SMEM <= 227 * 1024, "shared memory");
};

// Barriers and small shared state at BAR_OFF.
struct PfShared {
  uint64_t kf[2], ke[2];  // key stage filled / consumed
  uint64_t vf[2], ve[2];  // value stage filled / consumed
  // parameters of tile j (slot j & 3: the keys run up to three tiles ahead of
  // the softmax that reads them)
  uint64_t mf[4];
  uint64_t sf[2];   // S of tile j (buffer j & 1)
  uint64_t pf[2];   // P of tile j
  uint64_t pv;      // O holds tile j's product
  uint64_t qf;      // query operands staged
  uint32_t tmem;
  int32_t lo, hi;            // positions some row of the CTA sees
  int32_t all_lo, all_hi;    // positions every row sees
};
static_assert(sizeof(PfShared) <= 256, "shared state");

}  // namespace

struct PrefillArgs {
  int S, T, Hq, H, G, lgP, NP, bt_stride, max_seq_len, max_q, mtiles, splits;
  int shared_len;  // < 0: prompt chunks; else the rows are the batch's sequences and the keys
                   // the first shared_len positions of block-table row 0
  int rot_kind, lgb;
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

// Channels are visited in the order 0 4 1 5 2 6 3 7 inside each group of 8
// (the nibble pairs that one mask extracts) by every operand.
__device__ __forceinline__ constexpr int pf_perm(int i) { return (i >> 1) + 4 * (i & 1); }

// Barrier of the two warps that share 32 rows (named barrier 1 + quarter),
// with the ordering of their tensor-memory accesses.
__device__ __forceinline__ void pf_pair_sync(int quarter) {
  tc_fence_before();
  asm volatile("bar.sync %0, 64;" ::"r"(1 + quarter) : "memory");
  tc_fence_after();
}

// One butterfly stage between columns [a, a + 32 n) and [b, b + 32 n).
__device__ __forceinline__ void pf_cross(uint32_t scr, int a, int b, int n) {
#pragma unroll 1
  for (int c = 0; c < n; ++c) {
    uint32_t x[32], y[32];
    tmem_ld32(scr + a + 32 * c, x);
    tmem_ld32(scr + b + 32 * c, y);
    tmem_ld_wait();
#pragma unroll
    for (int i = 0; i < 32; ++i) {
      const float p = __uint_as_float(x[i]), q = __uint_as_float(y[i]);
      x[i] = __float_as_uint(p + q);
      y[i] = __float_as_uint(p - q);
    }
    tmem_st32(scr + a + 32 * c, x);
    tmem_st32(scr + b + 32 * c, y);
  }
  tmem_st_wait();
}

// The rotation (or its inverse with INV) of a row held as D binary32 columns
// of its tensor-memory lane at `scr`, by the row's two threads (w = 0, 1 own
// channels [w D/2, (w + 1) D/2)); warp-collective for both. Stages inside 64
// channels run in registers, wider ones between tensor-memory columns.
template <int D, bool INV>
__device__ __forceinline__ void pf_rotate(uint32_t scr, int w, int quarter, int rot_kind, int lgb,
                                          const float* tbl) {
  if (rot_kind == KVQ_ROT_NONE) return;
  const int c0 = w * (D / 2);
  if (rot_kind == KVQ_ROT_HADAMARD || rot_kind == KVQ_ROT_HADAMARD_SIGNED) {
    const bool sgn = rot_kind == KVQ_ROT_HADAMARD_SIGNED;
    const float cb = hadamard_scale(lgb);
#pragma unroll 1
    for (int h = 0; h < D / 128; ++h) {
      const int ch = c0 + 64 * h;
      uint32_t r[2][32];
      tmem_ld32(scr + ch, r[0]);
      tmem_ld32(scr + ch + 32, r[1]);
      tmem_ld_wait();
      float x[64];
#pragma unroll
      for (int i = 0; i < 64; ++i) x[i] = __uint_as_float(r[i >> 5][i & 31]);
      if (!INV && sgn) {
#pragma unroll
        for (int i = 0; i < 64; ++i) x[i] *= __ldg(tbl + ch + i);
      }
      fwht_regs<64, 4>(x);
#pragma unroll
      for (int st = 16; st < 64; st <<= 1) {
        if ((1 << lgb) <= st) break;
#pragma unroll
        for (int i = 0; i < 64; i += 2)
          if ((i & st) == 0) {
            const uint64_t a = pk(x[i], x[i + 1]), b = pk(x[i + st], x[i + st + 1]);
            const float2 s = upk(add2(a, b)), d = upk(sub2(a, b));
            x[i] = s.x; x[i + 1] = s.y; x[i + st] = d.x; x[i + st + 1] = d.y;
          }
      }
#pragma unroll
      for (int i = 0; i < 64; ++i) r[i >> 5][i & 31] = __float_as_uint(x[i] * cb);
      tmem_st32(scr + ch, r[0]);
      tmem_st32(scr + ch + 32, r[1]);
    }
    tmem_st_wait();
    if (lgb >= 7) {
      if (D == 128) {  // both threads' halves: 32 column pairs each
        pf_pair_sync(quarter);
        pf_cross(scr, 32 * w, 64 + 32 * w, 1);
        pf_pair_sync(quarter);
      } else {
        pf_cross(scr, c0, c0 + 64, 2);
      }
    }
    if (D == 256 && lgb == 8) {
      pf_pair_sync(quarter);
      pf_cross(scr, 64 * w, 128 + 64 * w, 2);
      pf_pair_sync(quarter);
    }
    if (INV && sgn) {
#pragma unroll 1
      for (int c = 0; c < D / 64; ++c) {
        uint32_t r[32];
        tmem_ld32(scr + c0 + 32 * c, r);
        tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < 32; ++i)
          r[i] = __float_as_uint(__uint_as_float(r[i]) * __ldg(tbl + c0 + 32 * c + i));
        tmem_st32(scr + c0 + 32 * c, r);
      }
      tmem_st_wait();
    }
    return;
  }
#pragma unroll 1
  for (int c = 0; c < D / 64; ++c) {
    uint32_t r[32];
    tmem_ld32(scr + c0 + 32 * c, r);
    tmem_ld_wait();
    float x[32];
#pragma unroll
    for (int i = 0; i < 32; ++i) x[i] = __uint_as_float(r[i]);
    if (rot_kind == KVQ_ROT_QUAT) {
      if (INV) quat_inv_regs<32>(x, tbl, c0 + 32 * c); else quat_regs<32>(x, tbl, c0 + 32 * c);
    } else if (rot_kind == KVQ_ROT_QUAT_FAST) {
      if (INV) quat_fast_inv_regs<32>(x, tbl, c0 + 32 * c);
      else quat_fast_regs<32>(x, tbl, c0 + 32 * c);
    } else {
      quat_mat_fly_regs<32, INV>(x, tbl, c0 + 32 * c);
    }
#pragma unroll
    for (int i = 0; i < 32; ++i) r[i] = __float_as_uint(x[i]);
    tmem_st32(scr + c0 + 32 * c, r);
  }
  tmem_st_wait();
}

// Row state of one softmax thread.
struct PfRow {
  bool valid;     // the row exists
  int64_t row;    // token * Hq + head
  int tok, head;
  int p, lo, hi;  // position and the interval it sees
};

// Four bytes of codes (8 channels) as binary16 pairs in the operands' channel
// order: c - 8, exactly.
__device__ __forceinline__ uint4 pf_codes_k(uint32_t x) {
  const uint32_t y = x >> 8;
  return make_uint4(nib_c8(x, 0x000F000Fu, 0), nib_c8(x, 0x00F000F0u, 1),
                    nib_c8(y, 0x000F000Fu, 0), nib_c8(y, 0x00F000F0u, 1));
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
template <int D, bool OPT>
__global__ void __launch_bounds__(kPfThreads, 1) prefill_kernel(const PrefillArgs a) {
  using C = PfCfg<D>;
  constexpr int KT = C::KT, KC = C::KC, NS = C::NS;
  extern __shared__ __align__(1024) uint8_t smem[];
  PfShared& sh = *reinterpret_cast<PfShared*>(smem + C::BAR_OFF);
  const int tid = threadIdx.x, warp = tid / kWarp, lane = tid % kWarp;
  const int wg = tid / 128;

  // ---- which rows: splits fastest, then KV heads, then sequences, then row
  // tiles from the last (the longest under a causal mask) to the first
  int b = blockIdx.x;
  const int split = b % a.splits;
  b /= a.splits;
  const int h = b % a.H;
  b /= a.H;
  const int nseq = a.shared_len >= 0 ? 1 : a.S;
  const int s = b % nseq;
  const int mt = a.mtiles - 1 - b / nseq;

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
    if (q0 < 0 || n < 0 || n > a.max_q || q0 > a.T - n) {  // not a range of the T rows: untouched
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
      mbar_init(&sh.kf[i], 128);
      mbar_init(&sh.ke[i], 1);
      mbar_init(&sh.vf[i], 128);
      mbar_init(&sh.ve[i], 1);
      mbar_init(&sh.sf[i], 1);
      mbar_init(&sh.pf[i], 256);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) mbar_init(&sh.mf[i], 128);
    mbar_init(&sh.pv, 1);
    mbar_init(&sh.qf, 256);
    sh.lo = INT_MAX;
    sh.hi = 0;
    sh.all_lo = 0;
    sh.all_hi = INT_MAX;
    mbar_fence_init();
  }
  if (warp == 16) {
    tmem_alloc(&sh.tmem, kPfTmemCols);
    tmem_relinquish();
  }
  __syncthreads();

  // ---- each row's interval, and what the CTA sees
  PfRow R;
  R.valid = false;
  R.row = 0;
  R.tok = R.head = R.p = R.lo = R.hi = 0;
  if (wg < 2) {
    const int64_t ri = r0 + (tid & 127);
    R.valid = ri < rows;
    if (R.valid) {
      const int i = (int)(ri / a.G);
      R.tok = q0 + i;
      R.head = h * a.G + (int)(ri - (int64_t)i * a.G);
      R.row = (int64_t)R.tok * a.Hq + R.head;
      bool ok = seq_ok;
      if (a.shared_len >= 0) {
        const int Ls = a.seq_lens[i];
        // length 0: an idle slot of a padded batch
        ok = ok && Ls >= a.shared_len && Ls <= a.max_seq_len && Ls > 0 &&
             ((Ls + (1 << a.lgP) - 1) >> a.lgP) <= a.bt_stride &&
             (a.rope == nullptr || Ls <= a.rope_max_pos);
        if (!ok && Ls != 0) raise_flag(a.err, KVQ_ERRF_LEN);
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
      if (wg == 0) {
        if (R.hi > 0) {
          atomicMin(&sh.lo, R.lo);
          atomicMax(&sh.hi, R.hi);
        }
        atomicMax(&sh.all_lo, R.lo);
        atomicMin(&sh.all_hi, R.hi);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh.tmem;
  const int kv_lo = sh.lo, kv_hi = sh.hi;
  int t0 = 0, t1 = 0;  // key tiles of this split
  if (kv_hi > kv_lo) {
    const int ta = kv_lo / KT, tb = (kv_hi + KT - 1) / KT;
    t0 = ta + (int)((int64_t)(tb - ta) * split / a.splits);
    t1 = ta + (int)((int64_t)(tb - ta) * (split + 1) / a.splits);
  }
  const int ntile = t1 - t0;

  auto wait = [&](uint64_t* bar, uint32_t parity) {
    if (!mbar_wait(bar, parity)) {
      raise_flag(a.err, KVQ_ERRF_TIMEOUT);
      return false;
    }
    return true;
  };

  if (wg < 2) {
    // =========================== softmax: two threads per row
    asm volatile("setmaxnreg.inc.sync.aligned.u32 144;");
    const int qd = warp & 3;                    // lane quarter of the warp
    const int row = tid & 127;
    const uint32_t lane_base = (uint32_t)(qd * 32) << 16;
    const uint32_t o_col = tmem + lane_base + C::O_COL;
    float* const ex = reinterpret_cast<float*>(smem + C::EX_OFF);
    float rs = 1.f, qsum = 0.f;  // 2^-e of the row's scaled query, and its sum
    if (ntile > 0) {
      // ---- the query row: RoPE, rotation (O's columns as scratch), then hi + lo
      const int c0 = wg * C::HC;
      const __half* src = a.q + (int64_t)R.tok * a.q_stride + (int64_t)R.head * D + c0;
      const float* cs =
          a.rope != nullptr && R.valid && R.hi > 0 ? a.rope + (int64_t)R.p * D + c0 : nullptr;
#pragma unroll 1
      for (int c = 0; c < C::HC / 32; ++c) {
        float x[32];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const uint4 u = R.valid ? __ldg(reinterpret_cast<const uint4*>(src + 32 * c) + k)
                                  : make_uint4(0u, 0u, 0u, 0u);
          const uint32_t w4[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 f = __half22float2(u32_as_h2(w4[e]));
            x[8 * k + 2 * e] = f.x;
            x[8 * k + 2 * e + 1] = f.y;
          }
        }
        if (cs != nullptr) rope_regs<32>(x, cs + 32 * c);
        __syncwarp();
        uint32_t r[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) r[i] = __float_as_uint(x[i]);
        tmem_st32(o_col + c0 + 32 * c, r);
      }
      tmem_st_wait();
      pf_rotate<D, false>(o_col, wg, qd, a.rot_kind, a.lgb, a.quat);
      float amax = 0.f;
#pragma unroll 1
      for (int c = 0; c < C::HC / 32; ++c) {
        uint32_t r[32];
        tmem_ld32(o_col + c0 + 32 * c, r);
        tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < 32; ++i) amax = fmaxf(amax, fabsf(__uint_as_float(r[i])));
      }
      ex[wg * kPfRows + row] = amax;
      pf_pair_sync(qd);
      amax = fmaxf(amax, ex[(wg ^ 1) * kPfRows + row]);
      // the power of two that brings the largest |q^| into [2^12, 2^13): lo
      // keeps its bits above the binary16 subnormals
      int e = 12 - (((__float_as_int(amax) >> 23) & 0xFF) - 127);
      e = min(max(e, -126), 126);
      const float mul = amax > 0.f ? __int_as_float((e + 127) << 23) : 0.f;
      rs = amax > 0.f ? __int_as_float((127 - e) << 23) : 1.f;  // (a zero query scores 0)
      uint8_t* const qh = smem + (row >> 3) * C::GRP + (row & 7) * 16;
#pragma unroll 1
      for (int c = 0; c < C::HC / 32; ++c) {
        uint32_t r[32], hw[16], lw[16];
        tmem_ld32(o_col + c0 + 32 * c, r);
        tmem_ld_wait();
#pragma unroll
        for (int k = 0; k < 16; ++k) {
          const int i = 8 * (k >> 2) + (k & 3);
          const float x0 = __uint_as_float(r[i]) * mul, x1 = __uint_as_float(r[i + 4]) * mul;
          const __half2 hh = __floats2half2_rn(x0, x1);
          const float2 f = __half22float2(hh);
          const __half2 ll = __floats2half2_rn(x0 - f.x, x1 - f.y);
          const float2 g = __half22float2(ll);
          qsum += (f.x + g.x) + (f.y + g.y);
          hw[k] = h2_as_u32(hh);
          lw[k] = h2_as_u32(ll);
        }
        if (C::QT) {
          const uint32_t qc = tmem + lane_base + C::Q_COL + (c0 + 32 * c) / 2;
          tmem_st16(qc, hw);
          tmem_st16(qc + D / 2, lw);
        } else {
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            uint8_t* dst = qh + ((c0 >> 3) + 4 * c + k) * 128;
            *reinterpret_cast<uint4*>(dst) =
                make_uint4(hw[4 * k], hw[4 * k + 1], hw[4 * k + 2], hw[4 * k + 3]);
            *reinterpret_cast<uint4*>(dst + C::Q_B) =
                make_uint4(lw[4 * k], lw[4 * k + 1], lw[4 * k + 2], lw[4 * k + 3]);
          }
        }
      }
      if (C::QT) tmem_st_wait(); else fence_async_smem();
      tc_fence_before();
      mbar_arrive(&sh.qf);
      ex[2 * kPfRows + wg * kPfRows + row] = qsum;
      pf_pair_sync(qd);
      qsum += ex[2 * kPfRows + (wg ^ 1) * kPfRows + row];
      pf_pair_sync(qd);
    }

    float M = -INFINITY, l = 0.f;
    const float slope2 = OPT && a.alibi != nullptr && R.valid
                             ? __ldg(a.alibi + R.head) * 1.4426950408889634f : 0.f;
    const int all_lo = sh.all_lo, all_hi = sh.all_hi;
    const int k0 = wg * KC;  // the thread's keys of a tile: [k0, k0 + KC)
    bool live = true;
    for (int j = 0; j < ntile; ++j) {
      const uint32_t s_col = tmem + lane_base + (j & 1) * KT + k0;
      live = wait(&sh.mf[j & 3], (j >> 2) & 1) && wait(&sh.sf[j & 1], (j >> 1) & 1);
      live = __all_sync(0xffffffffu, live);
      if (!live) break;
      tc_fence_after();
      uint32_t zr[KC / 32][32];
#pragma unroll
      for (int c = 0; c < KC / 32; ++c) tmem_ld32(s_col + 32 * c, zr[c]);
      tmem_ld_wait();
      const float* ks = reinterpret_cast<const float*>(smem + C::PAR_OFF) + (j & 3) * 2 * KT + k0;
      const int base = (t0 + j) * KT + k0;
      // z / rs = s'_j dot + m'_j qsum
      const uint64_t qs2 = pk(qsum, qsum);
#pragma unroll
      for (int c = 0; c < KC / 4; ++c) {
        const float4 sv = *reinterpret_cast<const float4*>(ks + 4 * c);
        const float4 mv = *reinterpret_cast<const float4*>(ks + KT + 4 * c);
        uint32_t* z = &zr[c >> 3][(4 * c) & 31];
        const float2 a0 = upk(fma2(pk(__uint_as_float(z[0]), __uint_as_float(z[1])),
                                   pk(sv.x, sv.y), mul2(pk(mv.x, mv.y), qs2)));
        const float2 a1 = upk(fma2(pk(__uint_as_float(z[2]), __uint_as_float(z[3])),
                                   pk(sv.z, sv.w), mul2(pk(mv.z, mv.w), qs2)));
        z[0] = __float_as_uint(a0.x);
        z[1] = __float_as_uint(a0.y);
        z[2] = __float_as_uint(a1.x);
        z[3] = __float_as_uint(a1.y);
      }
      float mul = rs;  // what is left to multiply z by
      if (OPT) {
        mul = 1.f;
        if (a.capk > 0.f) {
          // cap tanh(z / cap) = cap (1 - 2 / (1 + e^(2 z / cap)))
          const float k = rs * a.capk;
#pragma unroll
          for (int c = 0; c < KC; ++c) {
            const float e = fast_exp2(__uint_as_float(zr[c >> 5][c & 31]) * k);
            zr[c >> 5][c & 31] =
                __float_as_uint(fmaf(fast_rcp(1.f + e), -2.f * a.cap2, a.cap2));
          }
        } else {
#pragma unroll
          for (int c = 0; c < KC; ++c)
            zr[c >> 5][c & 31] = __float_as_uint(__uint_as_float(zr[c >> 5][c & 31]) * rs);
        }
        if (a.alibi != nullptr) {
          const float d0 = (float)(base - R.p);
#pragma unroll
          for (int c = 0; c < KC; ++c)
            zr[c >> 5][c & 31] = __float_as_uint(
                fmaf(-slope2, fabsf(d0 + (float)c), __uint_as_float(zr[c >> 5][c & 31])));
        }
      }
      // positions outside the row's interval, and keys of a bad page
      const uint4 bad = *reinterpret_cast<const uint4*>(smem + C::BAD_OFF + (j & 3) * 16);
      const bool anybad = (bad.x | bad.y | bad.z | bad.w) != 0u;
      if (anybad || base < all_lo || base + KC > all_hi) {
        const int lo = R.lo - base, hi = R.hi - base;
        // bad-page words of the thread's keys
        const uint32_t bw[2] = {KC == 64 ? (wg ? bad.z : bad.x) : (wg ? bad.y : bad.x),
                                KC == 64 ? (wg ? bad.w : bad.y) : 0u};
#pragma unroll
        for (int w = 0; w < KC / 32; ++w) {
          // bits [lo, hi) of this 32-key word, less the bad ones
          const int l0 = min(max(lo - 32 * w, 0), 32), h0 = min(max(hi - 32 * w, 0), 32);
          uint32_t m = h0 >= 32 ? 0xffffffffu : (1u << h0) - 1u;
          m &= l0 >= 32 ? 0u : 0xffffffffu << l0;
          m &= ~bw[w];
#pragma unroll
          for (int i = 0; i < 32; ++i)
            if (!((m >> i) & 1u)) zr[w][i] = 0xff800000u;
        }
      }
      float mx0 = -INFINITY, mx1 = -INFINITY;
#pragma unroll
      for (int c = 0; c < KC; c += 4) {
        const uint32_t* z = &zr[c >> 5][c & 31];
        mx0 = max3(mx0, __uint_as_float(z[0]), __uint_as_float(z[1]));
        mx1 = max3(mx1, __uint_as_float(z[2]), __uint_as_float(z[3]));
      }
      float mx = fmaxf(mx0, mx1) * mul;
      float* const exj = ex + (j & 1) * 2 * kPfRows;
      exj[wg * kPfRows + row] = mx;
      asm volatile("bar.sync %0, 64;" ::"r"(1 + qd) : "memory");
      mx = fmaxf(mx, exj[(wg ^ 1) * kPfRows + row]);
      const bool move = mx > M + kPfSlack;
      // every phase of pv is waited for once, before the arrival that lets the
      // next one complete (a parity names one of two phases only)
      bool waited = j == 0;
      if (__any_sync(0xffffffffu, move)) {
        const float Mn = move ? mx : M;
        const float alpha = !move ? 1.f : M == -INFINITY ? 0.f : fast_exp2(M - Mn);
        M = Mn;
        l *= alpha;
        if (j > 0) {
          waited = true;
          live = __all_sync(0xffffffffu, wait(&sh.pv, (j - 1) & 1));
          if (!live) break;
          tc_fence_after();
#pragma unroll 1
          for (int c = 0; c < C::HC / 16; ++c) {
            uint32_t o[16];
            tmem_ld16(o_col + wg * C::HC + 16 * c, o);
            tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
            tmem_st16(o_col + wg * C::HC + 16 * c, o);
          }
        }
      }
      const float off = M == -INFINITY ? 0.f : kPfLift - M;
      const uint64_t mul2v = pk(mul, mul), off2 = pk(off, off);
      // the weights, rounded to binary16; the sum takes the rounded ones, so a
      // weight's rounding cancels where it dominates its row
      float l0 = 0.f, l1 = 0.f;
      uint32_t pw[KC / 2];
#pragma unroll
      for (int i = 0; i < KC / 2; ++i) {
        const float2 x = upk(fma2(pk(__uint_as_float(zr[(2 * i) >> 5][(2 * i) & 31]),
                                     __uint_as_float(zr[(2 * i) >> 5][((2 * i) & 31) + 1])),
                                  mul2v, off2));
        const __half2 p = __floats2half2_rn(fast_exp2(x.x), fast_exp2(x.y));
        l0 = add_h_f(__low2half(p), l0);
        l1 = add_h_f(__high2half(p), l1);
        pw[i] = h2_as_u32(p);
      }
      const uint32_t p_col = tmem + lane_base + C::P_COL + (j & 1) * C::P_STEP + k0 / 2;
      if constexpr (KC == 64)
        tmem_st32(p_col, pw);
      else
        tmem_st16(p_col, pw);
      l += l0 + l1;
      tmem_st_wait();
      if (!waited) {
        live = __all_sync(0xffffffffu, wait(&sh.pv, (j - 1) & 1));
        if (!live) break;
      }
      tc_fence_before();
      mbar_arrive(&sh.pf[j & 1]);
    }
    if (ntile > 0) {
      wait(&sh.pv, (ntile - 1) & 1);
      tc_fence_after();
      // the two halves' weight sums (the slot that tile ntile - 1 did not use)
      float* const exj = ex + (ntile & 1) * 2 * kPfRows;
      exj[wg * kPfRows + row] = l;
      pf_pair_sync(qd);
      l += exj[(wg ^ 1) * kPfRows + row];
    }
    __syncwarp();
    // ---- the thread's half of the row's result (V entered halved)
    const int c0 = wg * C::HC;
    if (a.part != nullptr) {
      float* dst = a.part + (R.row * a.splits + split) * (D + 4);
      const bool some = ntile > 0 && M != -INFINITY;
      if (ntile > 0) {
#pragma unroll 1
        for (int c = c0; c < c0 + C::HC; c += 32) {
          uint32_t o[32];
          tmem_ld32(o_col + c, o);
          tmem_ld_wait();
          if (R.valid && some) {
#pragma unroll
            for (int k = 0; k < 4; ++k)
#pragma unroll
              for (int q = 0; q < 2; ++q) {
                float4 f;
                f.x = 2.f * __uint_as_float(o[8 * k + 0 + q]);
                f.y = 2.f * __uint_as_float(o[8 * k + 2 + q]);
                f.z = 2.f * __uint_as_float(o[8 * k + 4 + q]);
                f.w = 2.f * __uint_as_float(o[8 * k + 6 + q]);
                *reinterpret_cast<float4*>(dst + c + 8 * k + 4 * q) = f;
              }
          }
          __syncwarp();
        }
      }
      if (R.valid && wg == 0)
        *reinterpret_cast<float2*>(dst + D) = make_float2(some ? M - kPfLift : -INFINITY, l);
    } else {
      __half* dst = a.out + R.row * D;
      if (ntile > 0) {
        const float inv = l > 0.f ? 2.f / l : l;  // (NaN stays)
        const bool zero = M == -INFINITY;
        // normalised, back in channel order, then R^-1
#pragma unroll 1
        for (int c = c0; c < c0 + C::HC; c += 32) {
          uint32_t o[32], x[32];
          tmem_ld32(o_col + c, o);
          tmem_ld_wait();
#pragma unroll
          for (int i = 0; i < 32; ++i)
            x[(i & ~7) + pf_perm(i & 7)] =
                zero ? 0u : __float_as_uint(__uint_as_float(o[i]) * inv);
          tmem_st32(o_col + c, x);
        }
        tmem_st_wait();
        pf_rotate<D, true>(o_col, wg, qd, a.rot_kind, a.lgb, a.quat);
#pragma unroll 1
        for (int c = c0; c < c0 + C::HC; c += 32) {
          uint32_t o[32];
          tmem_ld32(o_col + c, o);
          tmem_ld_wait();
          if (R.valid) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              uint32_t w[4];
#pragma unroll
              for (int e = 0; e < 4; ++e)
                w[e] = h2_as_u32(__floats2half2_rn(__uint_as_float(o[8 * k + 2 * e]),
                                                   __uint_as_float(o[8 * k + 2 * e + 1])));
              *reinterpret_cast<uint4*>(dst + c + 8 * k) = make_uint4(w[0], w[1], w[2], w[3]);
            }
          }
          __syncwarp();
        }
      } else if (R.valid) {
#pragma unroll 1
        for (int c = c0; c < c0 + C::HC; c += 8)
          *reinterpret_cast<uint4*>(dst + c) = make_uint4(0u, 0u, 0u, 0u);
      }
    }
    tc_fence_before();
  } else if (wg < 4) {
    // =========================== keys (warpgroup 2) and values (3) to binary16 operands
    asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
    const bool isv = wg == 3;
    const int dt = tid & 127;
    const int key = dt % KT, part = dt / KT;  // 128 channels of one key
    const int P1 = (1 << a.lgP) - 1;
    const int32_t* bt = a.block_table + (int64_t)(a.shared_len >= 0 ? 0 : s) * a.bt_stride;
    const uint8_t* const codes = (isv ? a.v_codes : a.k_codes) + part * 64;
    const uint32_t* const params = isv ? a.v_params : a.k_params;
    auto page_of = [&](int j) {
      const int tok = (t0 + j) * KT + key;
      return j < ntile && tok >= kv_lo && tok < kv_hi ? bt[tok >> a.lgP] : INT_MIN;  // not needed
    };
    uint4 cr[2][4];         // codes of two tiles
    uint32_t pr[2];
    bool bad[2];
    auto load = [&](int page, int j, int st) {
      const bool ok = page >= 0 && page < a.NP;
      bad[st] = !ok && page != INT_MIN;
      if (ok) {
        const int tok = (t0 + j) * KT + key;
        const int64_t row = (((int64_t)page * a.H + h) << a.lgP) + (tok & P1);
        const uint4* src = reinterpret_cast<const uint4*>(codes + row * (D / 2));
#pragma unroll
        for (int i = 0; i < 4; ++i) cr[st][i] = __ldg(src + i);
        pr[st] = __ldg(params + row);
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) cr[st][i] = make_uint4(0u, 0u, 0u, 0u);
        pr[st] = 0u;
      }
    };
    uint8_t* const dst0 = smem + (isv ? C::V_OFF : C::K_OFF) + (key >> 3) * C::GRP + part * 2048 +
                          (key & 7) * 16;
    uint64_t* const full = isv ? sh.vf : sh.kf;
    uint64_t* const empty = isv ? sh.ve : sh.ke;
    // tile j (registers st): stage, then load tile j + 2 with the page pg2
    auto step = [&](int j, int st, int pg2) {
      const int sl = NS == 2 ? (j & 1) : 0;
      if (j >= NS && !wait(&empty[sl], NS == 2 ? ((j >> 1) - 1) & 1 : (j - 1) & 1)) return false;
      uint8_t* const dst = dst0 + sl * C::K_B;
      const uint32_t w4[16] = {
          cr[st][0].x, cr[st][0].y, cr[st][0].z, cr[st][0].w, cr[st][1].x, cr[st][1].y,
          cr[st][1].z, cr[st][1].w, cr[st][2].x, cr[st][2].y, cr[st][2].z, cr[st][2].w,
          cr[st][3].x, cr[st][3].y, cr[st][3].z, cr[st][3].w};
      if (isv) {
        // halved: the largest dequantized value (15 s + m, s rounded up) may
        // exceed the binary16 range by its rounding
        const __half2 hp = __hmul2(u32_as_h2(pr[st]), __float2half2_rn(0.5f));
        const __half2 s2 = __low2half2(hp), m2 = __high2half2(hp);
#pragma unroll
        for (int w = 0; w < 16; ++w)
          *reinterpret_cast<uint4*>(dst + w * 128) = pf_codes_v(w4[w], s2, m2);
      } else {
        float* ks = reinterpret_cast<float*>(smem + C::PAR_OFF) + (j & 3) * 2 * KT;
        const uint32_t bm = __ballot_sync(0xffffffffu, bad[st]);
        if (part == 0) {
          const float2 sm = __half22float2(u32_as_h2(pr[st]));
          ks[key] = sm.x * a.scale2;
          ks[KT + key] = fmaf(8.f, sm.x, sm.y) * a.scale2;
          if (lane == 0) {
            uint32_t* bw = reinterpret_cast<uint32_t*>(smem + C::BAD_OFF + (j & 3) * 16);
            bw[key >> 5] = bm;
            if (KT == 64) bw[2 + (key >> 5)] = 0u;
          }
          const int tok = (t0 + j) * KT + key;
          if (bad[st] && h == 0 && ((tok & P1) == 0 || tok == kv_lo)) raise_flag(a.err, KVQ_ERRF_PAGE);
        }
        mbar_arrive(&sh.mf[j & 3]);
#pragma unroll
        for (int w = 0; w < 16; ++w) *reinterpret_cast<uint4*>(dst + w * 128) = pf_codes_k(w4[w]);
      }
      fence_async_smem();
      mbar_arrive(&full[sl]);
      load(pg2, j + 2, st);
      return true;
    };
    if (ntile > 0) {
      int pga = page_of(0), pgb = page_of(1);
      load(pga, 0, 0);
      load(pgb, 1, 1);
      pga = page_of(2);
      pgb = page_of(3);
      for (int j = 0; j < ntile; j += 2) {
        if (!step(j, 0, pga)) break;
        pga = page_of(j + 4);
        if (j + 1 >= ntile || !step(j + 1, 1, pgb)) break;
        pgb = page_of(j + 5);
      }
    }
  } else {
    // =========================== the issuing warp
    asm volatile("setmaxnreg.dec.sync.aligned.u32 40;");
    if (warp == 16 && ntile > 0) {
    constexpr uint32_t idS = umma_idesc_f16(kPfRows, KT, 0);
    constexpr uint32_t idO = umma_idesc_f16(kPfRows, D, 1);
    const bool one = elect_one();
    // keys: rows are keys, K-major; values: rows (the K dimension) are keys
    const uint64_t kd0 = umma_desc_kmajor(smem_u32(smem + C::K_OFF), 128, C::GRP);
    const uint64_t vd0 = umma_desc_kmajor(smem_u32(smem + C::V_OFF), C::GRP, 128);
    const uint64_t qd = umma_desc_kmajor(smem_u32(smem), 128, C::GRP);
    auto qk = [&](int j) {
      const int sl = NS == 2 ? (j & 1) : 0;
      const bool ok = wait(&sh.kf[sl], NS == 2 ? (j >> 1) & 1 : j & 1);
      tc_fence_after();
      const uint64_t kd = kd0 + (uint64_t)(sl * (C::K_B >> 4));
      const uint32_t d = tmem + (j & 1) * KT;
      if (one) {
#pragma unroll
        for (int half = 0; half < 2; ++half)  // hi, then lo
#pragma unroll
          for (int k = 0; k < D / 16; ++k) {
            if (C::QT)
              umma_f16_ts(d, tmem + C::Q_COL + half * (D / 2) + 8 * k, kd + (uint64_t)(16 * k), idS,
                          half + k > 0);
            else
              umma_f16_ss(d, qd + (uint64_t)(half * (C::Q_B >> 4) + 16 * k),
                          kd + (uint64_t)(16 * k), idS, half + k > 0);
          }
        umma_commit(&sh.sf[j & 1]);
        umma_commit(&sh.ke[sl]);
      }
      __syncwarp();
      return ok;
    };
    bool ok = wait(&sh.qf, 0);
    ok = ok && qk(0);
    if (ntile > 1) ok = ok && qk(1);
    for (int j = 0; j < ntile && ok; ++j) {
      const int sl = NS == 2 ? (j & 1) : 0;
      ok = wait(&sh.pf[j & 1], (j >> 1) & 1) && wait(&sh.vf[sl], NS == 2 ? (j >> 1) & 1 : j & 1);
      if (!ok) break;
      tc_fence_after();
      const uint32_t p = tmem + C::P_COL + (j & 1) * C::P_STEP, d = tmem + C::O_COL;
      const uint64_t vd = vd0 + (uint64_t)(sl * (C::K_B >> 4));
      if (one) {
#pragma unroll
        for (int k = 0; k < KT / 16; ++k)
          umma_f16_ts(d, p + 8 * k, vd + (uint64_t)(k * (2 * C::GRP >> 4)), idO, j > 0 || k > 0);
        umma_commit(&sh.pv);
        umma_commit(&sh.ve[sl]);
      }
      __syncwarp();
      if (j + 2 < ntile) ok = qk(j + 2);
    }
    }
  }
  __syncthreads();
  tc_fence_after();
  if (warp == 16) tmem_dealloc(tmem, kPfTmemCols);
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
};

template <int D>
__global__ void __launch_bounds__(128) prefill_merge_kernel(const PfMergeArgs m) {
  constexpr int CPL = D / 32;
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x % kWarp;
  const int64_t gw = (int64_t)blockIdx.x * 4 + threadIdx.x / kWarp;
  if (gw >= m.rows) return;
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
#pragma unroll 4
      for (int k = 0; k < cnt; ++k) {
        const float wk = __shfl_sync(0xffffffffu, w, k);
        if (!((any >> k) & 1u)) continue;
        const float4* p = reinterpret_cast<const float4*>(src + (int64_t)(i0 + k) * (D + 4) + lane * CPL);
#pragma unroll
        for (int c = 0; c < CPL / 4; ++c) {
          const float4 f = __ldcg(p + c);
          x[4 * c] = fmaf(wk, f.x, x[4 * c]);
          x[4 * c + 1] = fmaf(wk, f.y, x[4 * c + 1]);
          x[4 * c + 2] = fmaf(wk, f.z, x[4 * c + 2]);
          x[4 * c + 3] = fmaf(wk, f.w, x[4 * c + 3]);
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
  while ((1 << l) < x) ++l;
  return l;
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
  return plan_rows(d.head_dim, d.num_kv_heads, S, (int64_t)max_q * G, (int64_t)T * Hq, max_seq_len);
}

template <int D, bool OPT>
static cudaError_t launch_prefill(const PrefillArgs& a, int grid, cudaStream_t st) {
  auto kern = prefill_kernel<D, OPT>;
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
  a.scale2 = (float)((double)sm_scale * 1.4426950408889634074);
  a.capk = sc && sc->softcap > 0.f ? 2.f / sc->softcap : 0.f;
  a.cap2 = sc ? (float)((double)sc->softcap * 1.4426950408889634074) : 0.f;
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

static cudaError_t launch_any(const PrefillArgs& a, int D, int grid, cudaStream_t st) {
  const bool opt = a.capk > 0.f || a.alibi != nullptr;
  if (D == 128) return opt ? launch_prefill<128, true>(a, grid, st) : launch_prefill<128, false>(a, grid, st);
  return opt ? launch_prefill<256, true>(a, grid, st) : launch_prefill<256, false>(a, grid, st);
}

static cudaError_t launch_merge(const kvq_cache_desc& d, int64_t rows, int G, int na, int nb,
                                int nhi, const float* pa, const float* pb, void* out,
                                cudaStream_t st) {
  PfMergeArgs m;
  m.rows = (int)rows; m.G = G; m.rot_kind = d.rot_kind; m.lgb = log2i(d.rot_block);
  m.na = na; m.nb = nb; m.nhi = nhi; m.quat = d.quat; m.part_a = pa; m.part_b = pb;
  m.out = static_cast<__half*>(out);
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
  const PrefillPlan pl = prefill_plan(d, S, Hq, T, max_q, max_seq_len);
  if (pl.workspace > 0 && (workspace == nullptr || workspace_bytes < pl.workspace))
    return KVQ_ERR_WORKSPACE;
  if (pl.ctas > INT_MAX || (int64_t)T * Hq > INT_MAX) return KVQ_ERR_UNSUPPORTED;
  PrefillArgs a;
  fill_args(a, d, S, Hq, q, seq_lens, max_seq_len, block_table, bt_stride, sm_scale, sc, k_codes,
            k_params, v_codes, v_params, err);
  a.T = T; a.q_stride = q_stride; a.q_start = q_start; a.max_q = max_q;
  a.mtiles = (int)pl.mtiles; a.splits = pl.splits; a.shared_len = -1;
  a.out = static_cast<__half*>(out);
  a.part = pl.splits > 1 ? static_cast<float*>(workspace) : nullptr;
  if (launch_any(a, d.head_dim, (int)pl.ctas, st) != cudaSuccess) return KVQ_ERR_CUDA;
  if (pl.splits > 1 &&
      launch_merge(d, (int64_t)T * Hq, a.G, pl.splits, 0, 0, a.part, nullptr, out, st) != cudaSuccess)
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
  const SharedPlan pl = shared_plan(d, S, Hq, prefix_len, max_seq_len);
  if (workspace == nullptr || workspace_bytes < pl.workspace) return KVQ_ERR_WORKSPACE;
  if (pl.prefix.ctas > INT_MAX || (int64_t)S * Hq > INT_MAX) return KVQ_ERR_UNSUPPORTED;
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
    if (launch_any(a, d.head_dim, (int)pl.prefix.ctas, st) != cudaSuccess) return KVQ_ERR_CUDA;
  }
  const int r = decode_scored_split_launch(d, S, Hq, q, seq_lens, max_seq_len, block_table,
                                           bt_stride, sm_scale, sc, prefix_len, k_codes, k_params,
                                           v_codes, v_params, pb, err, st);
  if (r != KVQ_OK) return r;
  // (a window shrinks the own part's plan: the launch's own counts)
  const DecodePlan own = decode_scored_plan(d, S, Hq, max_seq_len, prefix_len, sc);
  return launch_merge(d, (int64_t)S * Hq, Hq / d.num_kv_heads, pl.prefix.splits, own.splits,
                      own.nhi, pa, pb, out, st) == cudaSuccess ? KVQ_OK : KVQ_ERR_CUDA;
}

}  // namespace kvq
