// Attention over the 8-bit cache (pi_attend): softmax(scale q k^T) v with the
// softmax's running maximum and sum, one pass over the pages.
//
// Mathematics.  For a block of 32 tokens, S^T = K Q^T on the matrix cores
// (v_mfma_f32_16x16x32_f16; the codes minus 128 are exact in fp16), 16 query
// rows to a tile.  The block's key scale multiplies S, its value scale is an
// addend of the exponent: p = 2^(S ks c - m + log2(vs / vref)), so neither
// costs an instruction per element, and the sum of the weights takes
// vs / vref out again once per block (far below vref, its power of two goes to the
// codes instead, kNear).  O^T += V^T P^T with P in fp16.  A lane holds
// the weights of 8 tokens of one row, which is what the second product's
// operand takes from it: P never leaves the registers.  The reference
// exponent m moves only when the weights of a block outgrow fp16's range above it (a
// ballot sees their sum), so maxima are seldom taken and sums seldom rescaled.
//
// The pages' byte order gives each lane its 16 codes of an operand in one
// 16-byte load, 1 KB in a row for a wave.
//
// Two ways to cut the work, by size (attend_plan).  Few rows (k_attend): the
// pages' bytes bound the time; the eight waves of a workgroup share the rows
// and take every eighth block.  Many rows (k_attend_many): the weights'
// exponentials and the products do; each wave has rows of its own and all walk
// the blocks in step, whose codes are turned to fp16 once for the workgroup, in
// LDS (groups of waves take different blocks where the rows leave waves over).
// Both split the blocks over workgroups as well where the rows do not fill the
// CUs (few rows of unlike sequences by their lengths, Shares); partial means are
// joined in a fixed order (in LDS, then in k_attend_join).
//
// Measured (streaming read 6.45 TB/s, fp16 product 1160 TFLOP/s on the same
// card): one token of 64 heads over 131072 tokens of 8 kv heads, D = 128, 48.5 us with
// the join (269 MB, 5.5 TB/s); 32 sequences of 16384 tokens and less with
// scores 156 us (863 MB, 5.5 TB/s); fp32, 56 kv heads of their own, 34.2 us (180
// MB, 5.3 TB/s); 512 tokens of 128 heads over 8200 tokens, D = 64, 162 us (133
// GFLOP, 820 TFLOP/s): there the instructions around the products bind, 232 k
// cycles a SIMD beside the products' 144 k, of 367 k; 4096 tokens of 64 heads, 8 of
// kv, D = 128, whole, 312 us (275 GFLOP, 880 TFLOP/s).
#include "attn_device.h"

namespace pi {
namespace {

typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x4 __attribute__((ext_vector_type(4)));
typedef float f32x8 __attribute__((ext_vector_type(8)));

constexpr int kAtThreads = 256;              // k_attend_join
constexpr int kFewThreads = 512, kFewWaves = kFewThreads / kWave;
constexpr int kManyThreads = 512;
static_assert(kManyThreads == kFewThreads, "attend_plan counts the threads of either");
constexpr int kManyWaves = kManyThreads / kWave;
constexpr int kMaxSplits = 64;
constexpr int kSlots = 256;                  // workgroups that run at once
constexpr float kNoMax = -3e38f;     // reference before the first visible token
// Weights are held times 2^8, and a lane's eight of a block may sum to 2^15
// (fp16 holds 65504) before the reference moves: no maximum is taken but then.
// A block's value scale goes with its weights as far as 2^-kNear of the wave's
// largest; farther, its power of two is the factor of the block's codes instead
// (exact).  So what a weight loses below fp16's smallest step is at most 2^-31 of
// the row's largest weight, in the product and in the sum of rounded weights,
// and 10^5 such tokens beside one that takes the row are still counted.  (Less bias
// sends more blocks the second way, more moves the reference oftener: 2^7 and 1 320
// us, 2^8 and 2 306, 2^9 and 3 308 for 4096 tokens, 64 heads, D = 128.)
constexpr float kBias = 8.f;
constexpr float kMost = 0x1p15f;
constexpr int kNear = 2;
// k_attend_many has fp16 rows' weights as one fp16 part, which leaves half a step of
// fp16 of each weight in the output, unless the rows see 512 tokens or less (where one
// weight's rounding may be the row's: error against 64 bits 2.07e-4, the output's own
// rounding, and 2.6e-4 with one part; 3000 tokens 2.4e-4 with one) or a kv head has 32 rows
// or less, as k_attend's; by what the rows see and are, not by the call's bounds.  Two
// parts everywhere would take 287 us for 159 (512 tokens over 8200, 128 heads, D = 64).
constexpr int kTwoTokens = 512, kTwoRows = 32;
// Powers of two down to 2^-14 are a normal fp16 factor of the codes.  Farther, the
// sums are brought to the block's unit for its product and back, by up to 2^60; a
// block whose value scale lies farther than that counts as one of scale 0, which
// makes 0 of any code (its weights count).
constexpr int kFactor = 14, kUnit = 60;

__device__ __forceinline__ f32x4 mfma16(f16x8 a, f16x8 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
}

// 8 codes to fp16 values code - 128 (times factor, with off = -1152 factor): the
// bytes become 1024 + code by their place in the fraction of 0x6400, less 1152.
// Exact, with the factors of Blocks too.
__device__ __forceinline__ f16x8 codes_f16(unsigned lo, unsigned hi, f16x2 factor, f16x2 off) {
  const f16x2 h[4] = {as_h2(__builtin_amdgcn_perm(0x64646464u, lo, 0x04010400u)),
                      as_h2(__builtin_amdgcn_perm(0x64646464u, lo, 0x04030402u)),
                      as_h2(__builtin_amdgcn_perm(0x64646464u, hi, 0x04010400u)),
                      as_h2(__builtin_amdgcn_perm(0x64646464u, hi, 0x04030402u))};
  unsigned w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = __builtin_bit_cast(unsigned, __builtin_elementwise_fma(h[i], factor, off));
  return __builtin_bit_cast(f16x8, u32x4{w[0], w[1], w[2], w[3]});
}
__device__ __forceinline__ f16x8 codes_f16(unsigned lo, unsigned hi) {
  const f16x2 off = {(f16)-1152.f, (f16)-1152.f};
  const f16x2 h[4] = {as_h2(__builtin_amdgcn_perm(0x64646464u, lo, 0x04010400u)) + off,
                      as_h2(__builtin_amdgcn_perm(0x64646464u, lo, 0x04030402u)) + off,
                      as_h2(__builtin_amdgcn_perm(0x64646464u, hi, 0x04010400u)) + off,
                      as_h2(__builtin_amdgcn_perm(0x64646464u, hi, 0x04030402u)) + off};
  return __builtin_bit_cast(f16x8, u32x4{__builtin_bit_cast(unsigned, h[0]), __builtin_bit_cast(unsigned, h[1]),
                                         __builtin_bit_cast(unsigned, h[2]), __builtin_bit_cast(unsigned, h[3])});
}

__device__ __forceinline__ float lane_f(float v, int lane) {
  return as_f((unsigned)__builtin_amdgcn_readlane((int)__builtin_bit_cast(unsigned, v), lane));
}

// Sum and maximum over the four lanes that hold a row (lane % 16): a value's
// rows of 16 (32) lanes are swapped with a copy's, which leaves both partners in every lane.
template <typename F>
__device__ __forceinline__ float over_row(float v, F f) {
  const unsigned a = __builtin_bit_cast(unsigned, v);
  const auto x = __builtin_amdgcn_permlane16_swap(a, a, false, false);
  const unsigned b = __builtin_bit_cast(unsigned, f(as_f(x[0]), as_f(x[1])));
  const auto y = __builtin_amdgcn_permlane32_swap(b, b, false, false);
  return f(as_f(y[0]), as_f(y[1]));
}
__device__ __forceinline__ float row_sum(float v) {
  return over_row(v, [](float a, float b) { return a + b; });
}
__device__ __forceinline__ float row_max(float v) {
  return over_row(v, [](float a, float b) { return fmaxf(a, b); });
}

// 1 / a sum of weights; 0 where there are none.
__device__ __forceinline__ float inverse(float sum) { return sum == 0.f ? 0.f : 1.f / sum; }
// Of a whole row: where it sees tokens, a sum of 0 is that of logits that are all
// -infinity, whose softmax is NaN.
__device__ __forceinline__ bool no_softmax(float sum, int sees) { return sum == 0.f && sees > 0; }

__device__ __forceinline__ float exp2_hw(float x) { return __builtin_amdgcn_exp2f(x); }
__device__ __forceinline__ float log2_hw(float x) { return __builtin_amdgcn_logf(x); }

// Rows of a tile that an invalid sequence leaves NaN.
template <typename T>
__device__ void nan_rows(const AttendArgs& a, const Seq& q, int h, int d, int64_t first, int64_t step) {
  constexpr int V = Vec<T>::N;
  float f[V];
#pragma unroll
  for (int k = 0; k < V; ++k) f[k] = quiet_nan();
  const int ch = d / V;
  for (int64_t id = first; id < (int64_t)q.n * a.group * ch; id += step) {
    const int r = (int)(id / ch), e = (int)(id % ch) * V;
    T* p = static_cast<T*>(a.out) + (int64_t)(q.q0 + r / a.group) * a.o_ts + (int64_t)(h * a.group + r % a.group) * a.o_hs;
    *reinterpret_cast<u32x4*>(p + e) = Vec<T>::pack(f);
  }
}

// How sequences share a.slots workgroups by their lengths: the fewest blocks to
// a workgroup (of 64 counts between the bounds) that leave no more workgroups than
// there are.  Lane s has sequence s's.
struct Shares {
  Seq q;
  int n, first;          // workgroups of each of its kv heads; the first of them
  __device__ Shares(const AttendArgs& a) {
    const int s = lane_id();
    q = read_seq(a.lens, a.q_start, s < a.n_seqs ? s : 0, a.max_q, a.n_tok, a.max_len);
    // One for a sequence that is invalid or without tokens, for its NaN or zeros
    // (without rows it needs none, but splits_max counts it).
    int nb = q.n ? (q.len + kBlk - 1) / kBlk : 0;
    nb = s < a.n_seqs ? (nb > 1 ? nb : 1) : 0;
    const float sum = (float)__builtin_amdgcn_readlane((int)wave_scan((unsigned)nb), kWave - 1);
    const float most = (float)__builtin_amdgcn_readlane((int)wave_max((unsigned)nb), kWave - 1);
    // Between an even share (a block to each wave at least, kMaxSplits at most)
    // and what is always enough: the longest, and sum / per + n_seqs workgroups.
    const float lo = fmaxf(fmaxf(sum * a.share_even, most * (1.f / kMaxSplits)), (float)kFewWaves);
    const float hi = fmaxf(fminf(most, sum * a.share_safe), lo);
    const float per = s == kWave - 1 ? hi : lo + (hi - lo) * ((float)s * (1.f / (kWave - 1)));
    const float inv = __builtin_amdgcn_rcpf(per), x = (float)nb - 0.5f;
    int used = 0;
    for (int i = 0; i < a.n_seqs; ++i) used += count(lane_f(x, i), inv);
    const int at = __builtin_ctzll(__ballot(used <= a.slots / a.hk) | 1ull << (kWave - 1));
    n = s < a.n_seqs ? count(x, lane_f(inv, at)) : 0;
    first = ((int)wave_scan((unsigned)n) - n) * a.hk;
  }
  // ceil(nb / per) of nb - 0.5, which is exact (nb is under 2^20) and clear of whole numbers.
  __device__ static int count(float x, float inv) { return (int)(x * inv) + 1; }
};

// What a (sequence, kv head, split) walks, the same for its whole workgroup.
struct Walk {
  int pair, s, h, tile, split, splits;
  Seq q;                 // (without rows where the slot is nobody's)
  int rows, seen0;       // rows of the pair; tokens that its first row sees (may be < 1)
  __device__ __forceinline__ Walk(const AttendArgs& a, bool shared) {
    if (shared) {
      const Shares x(a);
      const int slot = blockIdx.x;
      s = __popcll(__ballot(x.first + x.n * a.hk <= slot));
      const bool used = s < a.n_seqs;
      s = used ? s : 0;
      auto of = [&](int v) { return __builtin_amdgcn_readlane(v, s); };
      q = {of(x.q.q0), used ? of(x.q.n) : 0, of(x.q.len), !used || of(x.q.ok)};
      splits = used ? of(x.n) : 1;
      const int k = slot - of(x.first);
      h = used ? (int)(((float)k + 0.5f) * __builtin_amdgcn_rcpf((float)splits)) : 0;      // k < 2^13
      split = k - h * splits, tile = 0;
      pair = s * a.hk + h;
      if (used && split == 0 && threadIdx.x == 0) a.count[pair] = splits;
    } else {
      const int pairs = a.n_seqs * a.hk;
      pair = blockIdx.x % pairs;
      tile = blockIdx.x / pairs % a.tiles;
      split = blockIdx.x / pairs / a.tiles, splits = a.splits;
      s = pair / a.hk, h = pair % a.hk;
      q = read_seq(a.lens, a.q_start, s, a.max_q, a.n_tok, a.max_len);
    }
    rows = q.n * a.group;
    seen0 = q.len - q.n + 1;
  }
  __device__ int64_t part_at(const AttendArgs& a, int r) const {
    return ((int64_t)split * a.n_seqs * a.hk + pair) * a.r_max + r;
  }
  // Tokens that row r sees.
  __device__ int sees(const AttendArgs& a, int r) const {
    const int v = seen0 + r / a.group;
    return v < 0 ? 0 : v;
  }
  __device__ int64_t out_at(const AttendArgs& a, int r) const {
    return (int64_t)(q.q0 + r / a.group) * a.o_ts + (int64_t)(h * a.group + r % a.group) * a.o_hs;
  }
};

// Pages and scales of up to 64 blocks, lane i those of the i-th.
struct Blocks {
  int page;
  float ks, lr, iv, unit;        // key scale; log2 of the weights' share (and kBias), 1 / share; the sums' unit
  f16 factor;                    // of the values' codes: value scale = share factor unit vref
  unsigned long long smalls;     // blocks whose unit is not 1
  unsigned long long odds;       // blocks whose factor is not 1

  __device__ void find(const AttendArgs& a, int pair, int first, int step, int cnt, bool& bad) {
    page = 0;
    if (lane_id() < cnt) {
      page = a.table[(int64_t)pair * a.max_blocks + first + lane_id() * step];
      const bool none = (unsigned)page >= (unsigned)a.n_pages;
      ks = none ? -1.f : 0.f;
      page = none ? 0 : page;
      bad |= none;
    }
  }
  // Returns the largest value scale.
  __device__ float read_scales(const AttendArgs& a, int cnt, float& vs) {
    vs = 0.f;
    float k = 0.f;
    if (lane_id() < cnt) {
      const float2 sc = reinterpret_cast<const float2*>(a.scales)[page];
      k = ks < 0.f ? -1.f : sc.x, vs = sc.y;
      // A scale that is no number: what sees the block is NaN, through its logits.
      if (!(k >= 0.f && k < __builtin_inff() && vs >= 0.f && vs < __builtin_inff())) k = quiet_nan(), vs = 0.f;
    }
    ks = k;
    float vmax = vs;
#pragma unroll
    for (int x = 32; x >= 1; x >>= 1) vmax = fmaxf(vmax, __shfl_xor(vmax, x, kWave));
    return vmax;
  }
  __device__ void set_units(float vs, float vref) {
    const bool some = vs > 0.f;
    const int ev = __builtin_amdgcn_frexp_expf(vs), e = some ? ev - __builtin_amdgcn_frexp_expf(vref) : 0;
    const bool near = e >= -kNear;
    const float share = some ? __builtin_amdgcn_ldexpf(vs, near ? e - ev + 1 : 1 - ev) : 1.f;
    const int fe = near ? 0 : (e > -kFactor ? e : -kFactor);
    const bool none = !some || e < -kFactor - kUnit;
    unit = near || none ? 1.f : __builtin_amdgcn_ldexpf(1.f, e - fe);
    factor = none ? (f16)0.f : (f16)__builtin_amdgcn_ldexpf(1.f, fe);
    lr = log2_hw(share) + kBias, iv = 1.f / share;
    smalls = __ballot(unit != 1.f);
    odds = __ballot(factor != (f16)1.f);
  }
  __device__ __forceinline__ f16 factor_of(int i) const {
    return __builtin_bit_cast(f16, (uint16_t)__builtin_amdgcn_readlane((int)__builtin_bit_cast(uint16_t, factor), i));
  }
};

// NB * 16 rows of a wave: queries, running reference and sums.  T: fp16, or fp32 as
// two fp16 parts; TWOP: the weights as two fp16 parts too.
template <typename T, int D, int NB, bool SCORE, bool TWOP>
struct Rows {
  static constexpr int KK = D / 64, DT = D / 16;
  static constexpr bool kTwo = sizeof(T) == 4;
  static constexpr bool kSum = TWOP || SCORE;      // sums of the unrounded weights
  int r0;
  f16x8 qf[NB][KK][2], ql[NB][kTwo ? KK : 1][2];   // lane (g, c): elements 64 kk + 16 g .. + 16 of row c
  float rs[NB];                                    // a row's power of two (fp32 rows)
  int sees[NB];
  f32x4 o[NB][DT];
  float m[NB], l[NB];                              // reference; sum of the weights, a lane's share until finish()
  float lr[NB];                                    // of the rounded weights, the row's
  float lt[NB];                                    // l of the blocks before the last fold() (fp32)
  float vref;                                      // o is in units of it

  __device__ __forceinline__ void load(const AttendArgs& a, const Walk& w, int first) {
    r0 = first;
    const int lane = lane_id(), g = lane / 16, c = lane % 16;
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      const int r = r0 + nb * 16 + c;
      const bool in = r < w.rows;
      const int t = in ? r / a.group : 0, head = w.h * a.group + (in ? r % a.group : 0);
      const T* p = static_cast<const T*>(a.q) + (int64_t)(w.q.q0 + t) * a.q_ts + (int64_t)head * a.q_hs + 16 * g;
      sees[nb] = in ? w.sees(a, r) : 0;
      rs[nb] = 1.f;
      if constexpr (!kTwo) {
#pragma unroll
        for (int kk = 0; kk < KK; ++kk)
#pragma unroll
          for (int f = 0; f < 2; ++f) {
            u32x4 v = {0, 0, 0, 0};
            if (in) v = ld16(p + 64 * kk + 8 * f);
            qf[nb][kk][f] = __builtin_bit_cast(f16x8, v);
          }
      } else {
        float x[KK][16];
        float top = 0.f;
#pragma unroll
        for (int kk = 0; kk < KK; ++kk)
#pragma unroll
          for (int f = 0; f < 4; ++f) {
            u32x4 v = {0, 0, 0, 0};
            if (in) v = ld16(p + 64 * kk + 4 * f);
            Vec<float>::unpack(v, &x[kk][4 * f]);
#pragma unroll
            for (int i = 0; i < 4; ++i) top = fmaxf(top, __builtin_fabsf(x[kk][4 * f + i]));
          }
        top = row_max(top);
        // The row times 2^-e lies below 2^14: both parts are normal fp16 numbers to 2^-38 of the largest.
        int e = 0;
        if (top > 0.f && top < __builtin_inff()) e = __builtin_amdgcn_frexp_expf(top) - 14;
        e = e < -126 ? -126 : e;
        rs[nb] = __builtin_amdgcn_ldexpf(1.f, e);
#pragma unroll
        for (int kk = 0; kk < KK; ++kk)
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const float v = __builtin_amdgcn_ldexpf(x[kk][i], -e);
            const f16 hi = (f16)v;
            qf[nb][kk][i / 8][i % 8] = hi;
            ql[nb][kk][i / 8][i % 8] = (f16)(v - (float)hi);
          }
      }
    }
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      m[nb] = kNoMax, l[nb] = lr[nb] = lt[nb] = 0.f;
#pragma unroll
      for (int t = 0; t < DT; ++t) o[nb][t] = f32x4{0.f, 0.f, 0.f, 0.f};
    }
    vref = 0x1p-126f;
  }

  __device__ __forceinline__ void rescale(float f) {
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
      for (int t = 0; t < DT; ++t) o[nb][t] *= f;
  }

  // The sums' unit follows the largest value scale, a power of two.
  __device__ __forceinline__ void raise_unit(float vmax) {
    const float top = as_f(__builtin_bit_cast(unsigned, fmaxf(vmax, 0x1p-126f)) & 0x7f800000u);
    if (top > vref) {
      rescale(vref / top);
      vref = top;
    }
  }

  // Block b, the i-th of x.  keys(mb, kk, f) and values(t) give the operands;
  // keys_done() is called when the last of the keys has been taken, scale_values()
  // before the values are where their factor is not 1.  All the rows see the first `whole` tokens.
  template <typename K, typename KD, typename VS, typename V>
  __device__ __forceinline__ void block(const AttendArgs& a, const Walk& w, const Blocks& x, int i, int b, int whole,
                                        K keys, KD keys_done, VS scale_values, V values) {
    const int lane = lane_id(), g = lane / 16, c = lane % 16;
    f32x4 st[NB][2];
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) st[nb][0] = st[nb][1] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int kk = 0; kk < KK; ++kk)
#pragma unroll
      for (int f = 0; f < 2; ++f)
#pragma unroll
        for (int mb = 0; mb < 2; ++mb) {
          const f16x8 kf = keys(mb, kk, f);
#pragma unroll
          for (int nb = 0; nb < NB; ++nb) {
            st[nb][mb] = mfma16(kf, qf[nb][kk][f], st[nb][mb]);
            if constexpr (kTwo) st[nb][mb] = mfma16(kf, ql[nb][kk][f], st[nb][mb]);
          }
        }
    keys_done();
    const float ksc = lane_f(x.ks, i) * a.scale;
    const float lrb = lane_f(x.lr, i), ivb = lane_f(x.iv, i);
    const bool edge = (b + 1) * kBlk > whole;      // some row does not see all of the block
    auto scale_of = [&](int nb) { return kTwo ? ksc * rs[nb] : ksc; };
    if (edge) {
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
        const float sc = scale_of(nb);
        const int left = sees[nb] - b * kBlk - 4 * g;
#pragma unroll
        for (int mb = 0; mb < 2; ++mb)
#pragma unroll
          for (int j = 0; j < 4; ++j) st[nb][mb][j] = mb * 16 + j < left ? st[nb][mb][j] * sc : -__builtin_inff();
      }
    }
    const float scv = edge ? 1.f : ksc;
    f16x8 pf[NB], pl[NB];
    float sum[NB], sumr[NB];
    auto weights = [&](int nb) {
      const float sc = kTwo ? (edge ? 1.f : ksc * rs[nb]) : scv, off = lrb - m[nb];
      float p[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) p[j] = exp2_hw(__builtin_fmaf(st[nb][j / 4][j % 4], sc, off));
      const f32x8 pv = {p[0], p[1], p[2], p[3], p[4], p[5], p[6], p[7]};
      pf[nb] = __builtin_convertvector(pv, f16x8);
      if constexpr (TWOP) pl[nb] = __builtin_convertvector(pv - __builtin_convertvector(pf[nb], f32x8), f16x8);
      if constexpr (kSum) sum[nb] = (p[0] + p[1] + (p[2] + p[3])) + (p[4] + p[5] + (p[6] + p[7]));
      if constexpr (!TWOP) {
        // The sum of the rounded weights over the row, by a product with ones: with it
        // the rounding of a weight that takes the row cancels.
        const f16x8 ones = {(f16)1.f, (f16)1.f, (f16)1.f, (f16)1.f, (f16)1.f, (f16)1.f, (f16)1.f, (f16)1.f};
        sumr[nb] = mfma16(ones, pf[nb], f32x4{0.f, 0.f, 0.f, 0.f})[0];
      }
      // Here and not behind the branch below: else the weights stay in fp32 until then
      // (D = 128, few rows 183 registers and 145 so; 335 and 308 us for fp32 prompts).
      if constexpr (kSum) asm volatile("" : "+v"(pf[nb]), "+v"(sum[nb]));
      else asm volatile("" : "+v"(pf[nb]));
    };
    bool over = false;
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      weights(nb);
      over |= !(kSum ? sum[nb] < kMost : sumr[nb] < 2.f * kMost);
    }
    if (__any(over)) {                             // a weight passes the reference by too much: move it
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
        const f32x4 s0 = st[nb][0], s1 = st[nb][1];
        const float top = fmaxf(fmaxf(fmaxf(s0[0], s0[1]), fmaxf(s0[2], s0[3])),
                                fmaxf(fmaxf(s1[0], s1[1]), fmaxf(s1[2], s1[3]))) * (edge ? 1.f : scale_of(nb));
        const float mn = fmaxf(m[nb], row_max(top));
        const float f = exp2_hw(m[nb] - mn);
        m[nb] = mn;
        l[nb] *= f, lr[nb] *= f;
        if constexpr (kTwo) lt[nb] *= f;
#pragma unroll
        for (int t = 0; t < DT; ++t) o[nb][t] *= f;
        weights(nb);
      }
    }
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      if constexpr (kSum) l[nb] = __builtin_fmaf(sum[nb], ivb, l[nb]);
      if constexpr (!TWOP) lr[nb] = __builtin_fmaf(sumr[nb], ivb, lr[nb]);
      if constexpr (SCORE) {
        const float bw = row_sum(sum[nb]) * ivb;
        const int r = r0 + nb * 16 + c;
        if (g == 0 && r < w.rows) a.lse[((int64_t)w.pair * a.max_nb + b) * a.r_max + r] = m[nb] + log2_hw(bw);
      }
    }
    const bool far = x.smalls >> i & 1;
    if (far) rescale(1.f / lane_f(x.unit, i));
    if (x.odds >> i & 1) scale_values(x.factor_of(i));
#pragma unroll
    for (int t = 0; t < DT; ++t) {
      const f16x8 v = values(t);
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
        o[nb][t] = mfma16(v, pf[nb], o[nb][t]);
        if constexpr (TWOP) o[nb][t] = mfma16(v, pl[nb], o[nb][t]);
      }
    }
    if (far) rescale(lane_f(x.unit, i));
  }

  // After every 64 blocks at most: fp32 rows' sums of weights stay short chains of
  // additions, whose roundings like terms do not add up (4096 blocks in one chain:
  // 1e-4 of the sum; fp16 rows' outputs are rounded to more).
  __device__ __forceinline__ void fold() {
    if constexpr (kTwo) {
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) lt[nb] += l[nb], l[nb] = 0.f;
    }
  }

  // o becomes the mean of the values by their weights, l the weights' sum: a mean is
  // no larger than the values, while a sum of them may pass fp32's range.
  __device__ __forceinline__ void finish() {
    if constexpr (kTwo) {
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) l[nb] = lt[nb];
    }
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      if constexpr (kSum) l[nb] = row_sum(l[nb]);
      else l[nb] = lr[nb];
      // (rows over the rounded sum, but the sum itself unrounded where there are scores: their blocks' are)
      const float inv = inverse(TWOP ? l[nb] : lr[nb]);
#pragma unroll
      for (int t = 0; t < DT; ++t) o[nb][t] = o[nb][t] * inv * vref;
    }
  }
};

// Four elements of a row, from fp32.
template <typename T>
__device__ __forceinline__ void store4(T* p, f32x4 v) {
  if constexpr (sizeof(T) == 4) *reinterpret_cast<f32x4*>(p) = v;
  else *reinterpret_cast<f16x4*>(p) = __builtin_convertvector(v, f16x4);
}

template <typename T, int D, int NB, bool SCORE>
__global__ __launch_bounds__(kFewThreads, 2) void k_attend(AttendArgs a) {
  constexpr int KK = D / 64, DT = D / 16, DB = D / 32;
  const Walk w(a, a.slots != 0);
  const int lane = lane_id(), wave = wave_id(), g = lane / 16, c = lane % 16;
  if (!w.q.ok) {
    if (w.split == 0) nan_rows<T>(a, w.q, w.h, D, (int64_t)w.tile * kFewThreads + threadIdx.x, (int64_t)a.tiles * kFewThreads);
    if (threadIdx.x == 0) raise_flag(a.flags, PI_FLAG_KV_RANGE);
    return;
  }
  const int r0 = w.tile * 16 * NB;
  if (r0 >= w.rows) return;
  const int r1 = r0 + 16 * NB < w.rows ? r0 + 16 * NB : w.rows;
  const int kmin = w.sees(a, r0), kmax = w.sees(a, r1 - 1);
  const int nbk = (kmax + kBlk - 1) / kBlk;
  const int per = (nbk + w.splits - 1) / w.splits;
  const int b0 = w.split * per, b1 = b0 + per < nbk ? b0 + per : nbk;
  const int start = b0 + wave;
  const int mine = start < b1 ? (b1 - start + kFewWaves - 1) / kFewWaves : 0;

  // The weights as two parts: the products have time while the pages come (D = 128,
  // fp16, 32 x 8 pairs of 4000 tokens, 24 rows 48.2 us for 46.4 with one).
  Rows<T, D, NB, SCORE, true> rows;
  rows.load(a, w, r0);
  u32x4 rk[2 * KK], rv[DB];                         // a block's codes, as they lie in the page
  bool bad = false;
  Blocks x;
  for (int base = 0; base < mine; base += kWave) {
    const int cnt = mine - base < kWave ? mine - base : kWave;
    x.find(a, w.pair, start + base * kFewWaves, kFewWaves, cnt, bad);
    auto page_at = [&](int i) {
      return a.pages + (int64_t)__builtin_amdgcn_readlane(x.page, i) * (2 * kBlk * D) + lane * 16;
    };
    auto load_k = [&](int i) {
      const uint8_t* p = page_at(i);
#pragma unroll
      for (int u = 0; u < 2 * KK; ++u) rk[u] = ld_nt(p + u * 1024);
    };
    auto load_v = [&](int i) {
      const uint8_t* p = page_at(i) + kBlk * D;
#pragma unroll
      for (int u = 0; u < DB; ++u) rv[u] = ld_nt(p + u * 1024);
    };
    // The first block's codes are on their way while the scales come.
    load_k(0);
    load_v(0);
    float vs;
    rows.raise_unit(x.read_scales(a, cnt, vs));
    x.set_units(vs, rows.vref);
    // One set of registers for the codes: the next block's keys are on their
    // way from the end of the first product on, its values from the second's.
    // (Past the last block they read page 0, which the caches hold: loads under a
    // condition would be waited for as if they had not been issued.)
    for (int i = 0; i < cnt; ++i) {
      const int n = i + 1 < kWave ? i + 1 : i;
      const f16 f = x.factor_of(i);
      const f16x2 vf = {f, f}, vo = vf * (f16)-1152.f;
      rows.block(
          a, w, x, i, start + (base + i) * kFewWaves, kmin,
          [&](int mb, int kk, int f) {
            const u32x4 v = rk[mb * KK + kk];
            return f ? codes_f16(v.z, v.w) : codes_f16(v.x, v.y);
          },
          [&] { load_k(n); }, [](f16) {},            // (the factor is in codes_f16's)
          [&](int t) {
            const u32x4 v = rv[t / 2];
            return t % 2 ? codes_f16(v.z, v.w, vf, vo) : codes_f16(v.x, v.y, vf, vo);
          });
      load_v(n);
    }
    rows.fold();
  }
  raise_flag_if_any(a.flags, bad, PI_FLAG_KV_RANGE);
  rows.finish();

  // The waves' means by their sums, added in wave order.
  __shared__ float so[kFewWaves][16][D + 4];
  __shared__ float sm[kFewWaves][16], sl[kFewWaves][16];
  __shared__ float rl[SCORE ? NB * 16 : 1];         // log2 of a row's weights, where this workgroup has all of them
  constexpr int E = D * 16 / kFewThreads > 4 ? D * 16 / kFewThreads : 4;     // elements of a thread
  const int row = threadIdx.x / (D / E), e0 = threadIdx.x % (D / E) * E;
#pragma unroll
  for (int nb = 0; nb < NB; ++nb) {
    if (nb) __syncthreads();
#pragma unroll
    for (int t = 0; t < DT; ++t) *reinterpret_cast<f32x4*>(&so[wave][c][16 * t + 4 * g]) = rows.o[nb][t];
    if (g == 0) sm[wave][c] = rows.m[nb], sl[wave][c] = rows.l[nb];
    __syncthreads();
    const int r = r0 + nb * 16 + row;
    if (row >= 16 || r >= w.rows) continue;
    float top = sm[0][row];
#pragma unroll
    for (int y = 1; y < kFewWaves; ++y) top = fmaxf(top, sm[y][row]);
    float sum = 0.f, f[kFewWaves], v[E];
#pragma unroll
    for (int y = 0; y < kFewWaves; ++y) sum += f[y] = exp2_hw(sm[y][row] - top) * sl[y][row];
    const float inv = inverse(sum);
#pragma unroll
    for (int k = 0; k < E; ++k) v[k] = 0.f;
#pragma unroll
    for (int y = 0; y < kFewWaves; ++y) {
#pragma unroll
      for (int k = 0; k < E; ++k) v[k] = __builtin_fmaf(f[y] * inv, so[y][row][e0 + k], v[k]);
    }
    const int64_t at = w.part_at(a, r);
    const bool whole = w.splits == 1;
    T* p = static_cast<T*>(a.out) + w.out_at(a, r) + e0;
    if (whole && no_softmax(sum, w.sees(a, r))) {
#pragma unroll
      for (int k = 0; k < E; ++k) v[k] = quiet_nan();
    }
#pragma unroll
    for (int k = 0; k < E; k += 4) {
      const f32x4 y = {v[k], v[k + 1], v[k + 2], v[k + 3]};
      if (whole) store4(p + k, y);
      else *reinterpret_cast<f32x4*>(a.part + at * D + e0 + k) = y;
    }
    if (!whole && e0 == 0) a.ml[at] = float2{top, sum};
    if (SCORE && e0 == 0) {
      if (a.tiles > 1) a.ml[at] = float2{top, sum};
      rl[nb * 16 + row] = top + log2_hw(sum);
    }
  }
  if constexpr (SCORE) {
    // The blocks' weights are in the workspace, from this workgroup's waves.
    if (w.splits > 1 || a.tiles > 1) return;
    __threadfence_block();
    __syncthreads();
    constexpr int Q = 4;                            // lanes that share a block's rows
    const int sub = threadIdx.x % Q;
    for (int b = threadIdx.x / Q; b < nbk; b += kFewThreads / Q) {
      const float* from = a.lse + ((int64_t)w.pair * a.max_nb + b) * a.r_max;
      float sum = 0.f;
      for (int r = sub; r < w.rows; r += Q)
        if (b * kBlk < w.sees(a, r)) sum += exp2_hw(from[r] - rl[r]);
      sum += __shfl_xor(sum, 1, kWave);
      sum += __shfl_xor(sum, 2, kWave);
      if (sub == 0) a.score[(int64_t)w.pair * a.max_blocks + b] += sum;
    }
  }
}

// NB * 16 rows to a wave, W waves to a group; the G groups share the rows and
// take blocks of their own in each step.  The codes of a step's blocks become
// fp16 operands in LDS once for all of them: a wave turns U units (1 KB of a page)
// per step, and the next step's units are on their way meanwhile.
// Waves to a SIMD: those of a workgroup, or two workgroups' where the registers last for them.
template <typename T, int D, bool SCORE>
constexpr int many_waves(int waves) { return D == 64 && sizeof(T) == 2 && !SCORE && waves == 8 ? 4 : waves / 4; }
template <int D, int NB, int W, int G>
struct ManyLds {
  static constexpr int kUnits = D / 16, kPart = W > kUnits ? W / kUnits : 1, kStep = G * kPart;
  u32x4 ops[2][kStep][kUnits][2][kWave];
  float2 sml[G > 1 ? W : 1][NB][kWave];
};

// The rows from g0 on, as many as the workgroup's waves hold; the weights as two parts (TWO) or one.
template <typename T, int D, int NB, bool SCORE, int W, int G, bool TWO, typename L>
__device__ __forceinline__ void many_rows(const AttendArgs& a, const Walk& w, L& lds, int g0) {
  constexpr int KK = D / 64, DT = D / 16, kUnits = L::kUnits, kPart = L::kPart, kStep = L::kStep;
  constexpr int U = kStep * kUnits / (W * G);       // units that a wave turns
  constexpr int kRows = 16 * NB * W;
  const int lane = lane_id(), g = lane / 16, c = lane % 16;
  const int wave = wave_id() % W, group = wave_id() / W;
  const int g1 = g0 + kRows < w.rows ? g0 + kRows : w.rows;
  const int nbk = (w.sees(a, g1 - 1) + kBlk - 1) / kBlk;
  const int per = (nbk + a.splits - 1) / a.splits;
  const int b0 = w.split * per, b1 = b0 + per < nbk ? b0 + per : nbk;
  const int r0 = g0 + wave * 16 * NB;
  const int r1 = r0 + 16 * NB < w.rows ? r0 + 16 * NB : w.rows;
  const int kmin = r0 < w.rows ? w.sees(a, r0) : 0, kmax = r0 < w.rows ? w.sees(a, r1 - 1) : 0;

  Rows<T, D, NB, SCORE, TWO> rows;
  f16x8 vals[DT];                                   // a block's values, on their way while its weights are taken
  rows.load(a, w, r0);
  bool bad = false;
  Blocks x;
  for (int base = b0; base < b1; base += kWave) {
    const int cnt = b1 - base < kWave ? b1 - base : kWave;
    x.find(a, w.pair, base, 1, cnt, bad);
    u32x4 next[U];
    auto fetch = [&](int i) {                        // of the step that begins with block i (past cnt: any page, not used)
#pragma unroll
      for (int k = 0; k < U; ++k) {
        const int u = wave_id() * U + k;
        const int64_t page = __builtin_amdgcn_readlane(x.page, (i + u / kUnits) % kWave);
        next[k] = ld16(a.pages + page * (2 * kBlk * D) + u % kUnits * 1024 + lane * 16);
      }
    };
    auto turn = [&](int buf) {
#pragma unroll
      for (int k = 0; k < U; ++k) {
        const int u = wave_id() * U + k;
        const u32x4 v = next[k];
        lds.ops[buf][u / kUnits][u % kUnits][0][lane] = __builtin_bit_cast(u32x4, codes_f16(v.x, v.y));
        lds.ops[buf][u / kUnits][u % kUnits][1][lane] = __builtin_bit_cast(u32x4, codes_f16(v.z, v.w));
      }
    };
    fetch(0);
    float vs;
    rows.raise_unit(x.read_scales(a, cnt, vs));
    x.set_units(vs, rows.vref);
    turn(0);
    __syncthreads();
    int buf = 0;
    for (int i = 0; i < cnt; i += kStep) {
      // (past cnt too: a condition costs more than the last one's load, 158 us for 156 of a 512-token chunk)
      fetch(i + kStep);
#pragma unroll
      for (int y = 0; y < kPart; ++y) {
        const int j = group * kPart + y, b = base + i + j;
        if (i + j < cnt && b * kBlk < kmax)
          rows.block(
              a, w, x, i + j, b, kmin,
              [&](int mb, int kk, int f) { return __builtin_bit_cast(f16x8, lds.ops[buf][j][mb * KK + kk][f][lane]); },
              [&] {
#pragma unroll
                for (int t = 0; t < DT; ++t) vals[t] = __builtin_bit_cast(f16x8, lds.ops[buf][j][2 * KK + t / 2][t % 2][lane]);
              },
              [&](f16 f) {
#pragma unroll
                for (int t = 0; t < DT; ++t) vals[t] *= f;
              },
              [&](int t) { return vals[t]; });
      }
      buf ^= 1;
      turn(buf);
      __syncthreads();                               // this step's operands are free, the next one's there
    }
    rows.fold();
  }
  raise_flag_if_any(a.flags, bad, PI_FLAG_KV_RANGE);
  rows.finish();
  if constexpr (G > 1) {
    // The groups' means by their sums, in the order of the groups; a lane's elements are the same in each.
    static_assert(sizeof(lds.ops) >= sizeof(f32x4) * W * NB * DT * kWave, "a group's means fit the operands' place");
    f32x4* so = &reinterpret_cast<f32x4*>(lds.ops)[(wave * NB * DT) * kWave + lane];
    for (int y = 1; y < G; ++y) {
      if (group == y) {
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
          lds.sml[wave][nb][lane] = float2{rows.m[nb], rows.l[nb]};
#pragma unroll
          for (int t = 0; t < DT; ++t) so[(nb * DT + t) * kWave] = rows.o[nb][t];
        }
      }
      __syncthreads();
      if (group == 0) {
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
          const float2 v = lds.sml[wave][nb][lane];
          const float top = fmaxf(rows.m[nb], v.x);
          const float l0 = rows.l[nb] * exp2_hw(rows.m[nb] - top), l1 = v.y * exp2_hw(v.x - top);
          const float inv = inverse(l0 + l1), f0 = l0 * inv, f1 = l1 * inv;
          rows.m[nb] = top;
          rows.l[nb] = l0 + l1;
#pragma unroll
          for (int t = 0; t < DT; ++t) rows.o[nb][t] = rows.o[nb][t] * f0 + so[(nb * DT + t) * kWave] * f1;
        }
      }
      if (y + 1 < G) __syncthreads();
    }
    if (group) return;
  }
#pragma unroll
  for (int nb = 0; nb < NB; ++nb) {
    const int r = r0 + nb * 16 + c;
    if (r >= w.rows) continue;
    const bool whole = a.splits == 1;
    const int64_t at = w.part_at(a, r);
    T* p = static_cast<T*>(a.out) + w.out_at(a, r) + 4 * g;
    const bool none = whole && no_softmax(rows.l[nb], rows.sees[nb]);
#pragma unroll
    for (int t = 0; t < DT; ++t) {
      if (whole) store4(p + 16 * t, none ? f32x4{quiet_nan(), quiet_nan(), quiet_nan(), quiet_nan()} : rows.o[nb][t]);
      else *reinterpret_cast<f32x4*>(a.part + at * D + 16 * t + 4 * g) = rows.o[nb][t];
    }
    if ((!whole || SCORE) && g == 0) a.ml[at] = float2{rows.m[nb], rows.l[nb]};
  }
}

template <typename T, int D, int NB, bool SCORE, int W, int G, bool TWO>
__global__ __launch_bounds__(W * G * kWave, (many_waves<T, D, SCORE>(W * G))) void k_attend_many(AttendArgs a) {
  constexpr int kThreads = W * G * kWave, kRows = 16 * NB * W;
  const Walk w(a, false);
  if (!w.q.ok) {
    if (w.split == 0) nan_rows<T>(a, w.q, w.h, D, (int64_t)w.tile * kThreads + threadIdx.x, (int64_t)a.tiles * kThreads);
    if (threadIdx.x == 0) raise_flag(a.flags, PI_FLAG_KV_RANGE);
    return;
  }
  // The last rows see the most: they begin first.
  const int g0 = (a.tiles - 1 - w.tile) * kRows;
  if (g0 >= w.rows) return;
  __shared__ ManyLds<D, NB, W, G> lds;
  if constexpr (TWO || sizeof(T) == 4) {
    many_rows<T, D, NB, SCORE, W, G, true>(a, w, lds, g0);
  } else if (w.sees(a, g0) <= kTwoTokens || w.rows <= kTwoRows) {
    // D = 64: a tile of each wave at a time, as two tiles' registers would be spilled in
    // the other branch too (512 tokens over 8200, 128 heads 207 us for 162).  D = 128: at
    // once (4096 tokens, 64 heads 311 us for 319).
    constexpr int B = D == 64 ? 1 : NB;
#pragma unroll 1
    for (int at = g0; at < g0 + kRows && at < w.rows; at += 16 * B * W) {
      if (at > g0) __syncthreads();
      many_rows<T, D, B, SCORE, W, G, true>(a, w, lds, at);
    }
  } else {
    many_rows<T, D, NB, SCORE, W, G, false>(a, w, lds, g0);
  }
}

// Reference exponent and sum of a row over its n splits.
__device__ __forceinline__ float2 row_ml(const AttendArgs& a, int pairs, int pair, int n, int r) {
  float2 v = a.ml[(int64_t)pair * a.r_max + r];
  for (int i = 1; i < n; ++i) {
    const float2 w = a.ml[((int64_t)i * pairs + pair) * a.r_max + r];
    const float top = fmaxf(v.x, w.x);
    v.y = v.y * exp2_hw(v.x - top) + w.y * exp2_hw(w.x - top);
    v.x = top;
  }
  return v;
}

// Joins the splits' means into rows (workgroups below row_groups: kFewSplits
// splits or less, a thread adds them and a workgroup takes as many rows as it
// has threads for; more, a workgroup takes one row and shares the splits), and
// adds the blocks' weights to the score (the others, kAtThreads / score_lanes()
// blocks of a (sequence, kv head) each).
//
// Lanes that share a block's rows: few where the rows are few, a wave where the
// rows' sums over the splits are worth sharing among blocks, else the workgroup
// (2000 rows x 8 pairs, 63 blocks: 1006 us with four lanes, 100 with a wave, 14 so).
__host__ __device__ constexpr int score_lanes(int r_max, int splits) {
  return r_max <= 32 ? 4 : (splits > 1 ? kWave : kAtThreads);
}
constexpr int kFewSplits = 8;
template <typename T, int D>
__global__ __launch_bounds__(kAtThreads) void k_attend_join(AttendArgs a, int row_groups) {
  const int pairs = a.n_seqs * a.hk;
  if ((int)blockIdx.x < row_groups) {
    constexpr int L = D / 4, G = kAtThreads / L;    // lanes of a row, splits (or rows) at a time
    if (a.splits <= kFewSplits) {
      const int64_t id = (int64_t)blockIdx.x * G + threadIdx.x / L;
      const int pair = (int)(id / a.r_max), r = (int)(id % a.r_max), e = threadIdx.x % L * 4;
      if (pair >= pairs) return;
      const Seq q = read_seq(a.lens, a.q_start, pair / a.hk, a.max_q, a.n_tok, a.max_len);
      f32x4 x[kFewSplits], o = {0.f, 0.f, 0.f, 0.f};
      float2 v[kFewSplits];
      float top = kNoMax, sum = 0.f;
      int n = kFewSplits;
      if (a.slots > kSlots) {
        n = a.count[pair];
        if (n == 1) return;
      }
      for (int i = 0; i < n; i += kFewSplits) {
        // (mostly the first ones are on their way before their number is known)
#pragma unroll
        for (int k = 0; k < kFewSplits; ++k) {
          const int64_t at = ((int64_t)(i + k < a.splits_max ? i + k : 0) * pairs + pair) * a.r_max + r;
          v[k] = a.ml[at];
          x[k] = *reinterpret_cast<const f32x4*>(a.part + at * D + e);
        }
        if (i == 0) {
          n = a.slots ? a.count[pair] : a.splits;
          if (!q.ok || r >= q.n * a.group || n == 1) return;
        }
        float to = top;
#pragma unroll
        for (int k = 0; k < kFewSplits; ++k) to = i + k < n ? fmaxf(to, v[k].x) : to;
        const float before = sum * exp2_hw(top - to);
        float f[kFewSplits];
        top = to, sum = before;
#pragma unroll
        for (int k = 0; k < kFewSplits; ++k) sum += f[k] = i + k < n ? exp2_hw(v[k].x - top) * v[k].y : 0.f;
        const float inv = inverse(sum);
        o *= before * inv;
#pragma unroll
        for (int k = 0; k < kFewSplits; ++k) o += i + k < n ? f[k] * inv * x[k] : f32x4{0.f, 0.f, 0.f, 0.f};
      }
      const int h = pair % a.hk;
      T* p = static_cast<T*>(a.out) + (int64_t)(q.q0 + r / a.group) * a.o_ts + (int64_t)(h * a.group + r % a.group) * a.o_hs;
      if (no_softmax(sum, q.len - q.n + 1 + r / a.group)) o = f32x4{quiet_nan(), quiet_nan(), quiet_nan(), quiet_nan()};
      store4(p + e, o);
      return;
    }
    __shared__ f32x4 acc[G][L];
    const int pair = blockIdx.x / a.r_max, r = blockIdx.x % a.r_max;
    const Seq q = read_seq(a.lens, a.q_start, pair / a.hk, a.max_q, a.n_tok, a.max_len);
    const int n = a.slots ? a.count[pair] : a.splits;
    if (!a.slots && (!q.ok || r >= q.n * a.group)) return;
    // Every split's part of this thread's elements, in flight while the weights are found.
    const int lane = lane_id(), part = threadIdx.x / L, e = threadIdx.x % L * 4;
    constexpr int N = kMaxSplits / G;
    f32x4 x[N];
#pragma unroll
    for (int k = 0; k < N; ++k) {
      const int i = k * G + part < a.splits_max ? k * G + part : 0;
      x[k] = *reinterpret_cast<const f32x4*>(a.part + (((int64_t)i * pairs + pair) * a.r_max + r) * D + e);
    }
    float2 v = a.ml[((int64_t)(lane < a.splits_max ? lane : 0) * pairs + pair) * a.r_max + r];
    if (a.slots && (!q.ok || r >= q.n * a.group || n == 1)) return;
    if (lane >= n) v = {kNoMax, 0.f};
    float top = v.x;
#pragma unroll
    for (int y = 32; y >= 1; y >>= 1) top = fmaxf(top, __shfl_xor(top, y, kWave));
    float f = exp2_hw(v.x - top) * v.y;
    const float sum = wave_sum(f);
    f *= inverse(sum);
    f32x4 o = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int k = 0; k < N; ++k) {
      const int i = k * G + part;
      const float w = __shfl(f, i, kWave);
      o += i < n ? w * x[k] : f32x4{0.f, 0.f, 0.f, 0.f};
    }
    acc[part][e / 4] = o;
    __syncthreads();
    if (part) return;
#pragma unroll
    for (int i = 1; i < G; ++i) o += acc[i][e / 4];
    if (no_softmax(sum, q.len - q.n + 1 + r / a.group)) o = f32x4{quiet_nan(), quiet_nan(), quiet_nan(), quiet_nan()};
    const int h = pair % a.hk;
    T* p = static_cast<T*>(a.out) + (int64_t)(q.q0 + r / a.group) * a.o_ts + (int64_t)(h * a.group + r % a.group) * a.o_hs + e;
    store4(p, o);
    return;
  }
  const int lanes = score_lanes(a.r_max, a.splits), each = kAtThreads / lanes;
  const int per = (a.max_nb + each - 1) / each;
  const int pair = (blockIdx.x - row_groups) / per, first = (blockIdx.x - row_groups) % per * each;
  const Seq q = read_seq(a.lens, a.q_start, pair / a.hk, a.max_q, a.n_tok, a.max_len);
  if (!q.ok || first * kBlk >= q.len) return;
  const int rows = q.n * a.group, seen0 = q.len - q.n + 1;
  if (rows == 0) return;
  const int splits = a.slots ? a.count[pair] : a.splits;
  if (a.slots && splits == 1) return;               // k_attend has them whole
  const int b = first + threadIdx.x / lanes, sub = threadIdx.x % lanes;
  const bool held = b * kBlk < q.len;
  // The first row that sees a token of block b (the rows after it do too).
  const int64_t t = (int64_t)b * kBlk + 1 - seen0, r0 = t > 0 ? t * a.group : 0;
  const float* from = a.lse + ((int64_t)pair * a.max_nb + (held ? b : 0)) * a.r_max;
  float w = 0.f;
  if (lanes == kAtThreads) {
    if (held && r0 < rows) {
#pragma unroll 4
      for (int r = (int)r0 + sub; r < rows; r += kAtThreads) {
        const float2 v = row_ml(a, pairs, pair, splits, r);
        w += exp2_hw(from[r] - v.x - log2_hw(v.y));
      }
    }
  } else {
    __shared__ float lse[kAtThreads];               // of a chunk of the rows, for all the workgroup's blocks
    const int64_t t0 = (int64_t)first * kBlk + 1 - seen0, low = t0 > 0 ? t0 * a.group : 0;
    for (int64_t c0 = low / kAtThreads * kAtThreads; c0 < rows; c0 += kAtThreads) {
      __syncthreads();
      const int r = (int)c0 + threadIdx.x;
      if (r < rows) {
        const float2 v = row_ml(a, pairs, pair, splits, r);
        lse[threadIdx.x] = v.x + log2_hw(v.y);
      }
      __syncthreads();
      const int end = rows - c0 < kAtThreads ? (int)(rows - c0) : kAtThreads;
      if (held)
        for (int k = sub; k < end; k += lanes)
          if (c0 + k >= r0) w += exp2_hw(from[c0 + k] - lse[k]);
    }
  }
  for (int x = 1; x < lanes && x < kWave; x <<= 1) w += __shfl_xor(w, x, kWave);
  if (lanes > kWave) {
    __shared__ float part[kAtThreads / kWave];
    if (lane_id() == 0) part[wave_id()] = w;
    __syncthreads();
    w = 0.f;
#pragma unroll
    for (int i = 0; i < kAtThreads / kWave; ++i) w += part[i];
  }
  if (sub == 0 && held) a.score[(int64_t)pair * a.max_blocks + b] += w;
}

// 16-row tiles of a wave: what its registers hold, beside the pages' codes in k_attend.
constexpr int few_tiles(int d, bool f32) { return d == 64 || !f32 ? 2 : 1; }
constexpr int many_tiles(int d, bool f32) { return d == 128 && f32 ? 1 : 2; }

// Launches one of the two kernels and the join.
template <typename T, int D, int NB, bool MANY, int W = kManyWaves, bool TWO = false>
hipError_t attend_run(const AttendArgs& a, const AttendPlan& p, hipStream_t s) {
  const int pairs = a.n_seqs * a.hk;
  const dim3 grid((unsigned)(a.slots ? a.slots : pairs * a.tiles * a.splits));
  if constexpr (MANY) {
    // Two groups where the rows' registers leave room for four waves a SIMD, unless
    // there are workgroups for two to a CU (64 heads, 8 of kv, 4096 tokens 169 us
    // and 189; 8 x 1024 tokens, 32 heads 62 and 86; but whole prompts whose 512 workgroups
    // end apart, 4096 tokens, 32 heads, 108 and 96).
    constexpr int G = D == 64 && sizeof(T) == 2 ? 2 : 1;
    const bool two = grid.x > 2 * kSlots || (grid.x == 2 * kSlots && a.max_nb <= 32);
    if constexpr (W < kManyWaves) {
      if (a.score) k_attend_many<T, D, NB, true, W, kManyWaves / W, TWO><<<grid, kManyThreads, 0, s>>>(a);
      else k_attend_many<T, D, NB, false, W, kManyWaves / W, TWO><<<grid, kManyThreads, 0, s>>>(a);
    } else {
      if (a.score) k_attend_many<T, D, NB, true, W, 1, TWO><<<grid, kManyThreads, 0, s>>>(a);
      else if (two) k_attend_many<T, D, NB, false, W, 1, TWO><<<grid, kManyThreads, 0, s>>>(a);
      else k_attend_many<T, D, NB, false, W, G, TWO><<<grid, G * kManyThreads, 0, s>>>(a);
    }
  } else {
    if (a.score) k_attend<T, D, NB, true><<<grid, kFewThreads, 0, s>>>(a);
    else k_attend<T, D, NB, false><<<grid, kFewThreads, 0, s>>>(a);
  }
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || p.row_groups + p.score_groups == 0) return e;
  k_attend_join<T, D><<<dim3((unsigned)(p.row_groups + p.score_groups)), kAtThreads, 0, s>>>(a, (int)p.row_groups);
  return hipGetLastError();
}

template <typename T, int D>
hipError_t attend_nb(const AttendArgs& a, const AttendPlan& p, hipStream_t s) {
  constexpr bool f32 = sizeof(T) == 4;
  if (p.many) {
    if constexpr (!f32)
      if (p.two) return attend_run<T, D, 1, true, kManyWaves, true>(a, p, s);
    if constexpr (f32 || D == 128) {
      if (p.waves == 2) return attend_run<T, D, many_tiles(D, f32), true, 2>(a, p, s);
      if (p.waves == 4) return attend_run<T, D, many_tiles(D, f32), true, 4>(a, p, s);
    }
    if constexpr (many_tiles(D, f32) == 2)
      if (p.nb == 1) return attend_run<T, D, 1, true>(a, p, s);
    return attend_run<T, D, many_tiles(D, f32), true>(a, p, s);
  }
  if constexpr (few_tiles(D, f32) == 2)
    if (p.nb == 2) return attend_run<T, D, 2, false>(a, p, s);
  return attend_run<T, D, 1, false>(a, p, s);
}

}  // namespace

AttendPlan attend_plan(int n_seqs, int hk, int group, int d, int dtype, int max_q, int max_len, bool score) {
  AttendPlan p;
  const int64_t pairs = (int64_t)n_seqs * hk;
  p.r_max = max_q * group;
  p.max_nb = (max_len + kBlk - 1) / kBlk;
  const bool f32 = dtype == PI_F32;
  // k_attend for the rows of one workgroup: fp16, D = 128, 32 x 8 pairs of 4000
  // tokens, 24 rows 46.5 us and 58 in k_attend_many; D = 64, 32 rows over 8000
  // tokens 12.2 and 15.7 us, 64 rows 25.9 and 14.7.  In fp32, whose products are
  // twice as many, also for a few workgroups that read the same pages: 8 pairs of
  // 30000 tokens, D = 128, 64 rows 30.7 and 38.2, 256 rows 85 and 77 (of 1500
  // tokens 15.1 and 21.4); but 32 x 8 pairs of 4000, 64 rows 177 and 88.
  const int few_rows = 16 * few_tiles(d, f32);
  p.many = p.r_max > few_rows && (!f32 || p.r_max > 256 || pairs * ((p.r_max + few_rows - 1) / few_rows) > 128);
  const int64_t shares = pairs * ((p.max_nb + 7) / 8);
  // Few enough rows for two or four waves leave the others for other blocks, and
  // fewer waves read a block's operands (32 x 8 pairs of 4000 tokens: fp16, D = 128,
  // 40 rows 64 us, 72 with one tile and twice the waves, 104 with eight waves at the
  // same block; 72 rows 80, 107; fp32, D = 128, 24 rows 63.5, 108, D = 64, 64 rows 54.7,
  // 72.5).  Not in small calls (fp16, 8 pairs of 1500, 40 rows: 15.1 and 13.6) nor for
  // fp16 of D = 64 (72 rows: 59 and 52).
  // All rows see kTwoTokens at most: no other kernel is needed, and one tile a wave (16
  // prompts of 512 tokens, 32 heads, D = 64 57 us, with one part 51; 8 of D = 128 58 and 43).
  p.two = p.many && !f32 && p.max_nb * kBlk <= kTwoTokens;
  p.waves = !p.many ? 1 : kManyWaves;
  const int two = 32 * many_tiles(d, f32);             // rows of two waves
  if (p.many && !p.two && (f32 || d == 128) && shares > 256) p.waves = p.r_max <= two ? 2 : p.r_max <= 2 * two ? 4 : kManyWaves;
  // Else one tile a wave while that is enough, and in small calls (counted in
  // shares of eight blocks): 100 of 1000 tokens, 32 heads, 8 of kv, D = 128 17.7 us
  // and 22.3 with two; 200 of 3000, 32 and 8, D = 64 20.8 and 24.9; 200 of 8000, 64
  // and 8, D = 64 57.2 and 52.1.
  const int narrow = 16 * p.waves, most_tiles = p.many ? many_tiles(d, f32) : few_tiles(d, f32);
  // Nor two for whole prompts whose workgroups would all run at once: their last rows
  // see the most, and twice as many that begin with those end together (2048
  // tokens, 32 heads, 8 of kv, D = 128 63 us and 72, D = 64 37 and 46).
  auto tiles_of = [&](int nb) { return (p.r_max + narrow * nb - 1) / (narrow * nb); };
  const bool small = shares * tiles_of(1) <= 1024 || (pairs * tiles_of(2) <= kSlots && max_q >= max_len - max_q);
  p.nb = p.r_max <= narrow && (!p.many || p.waves == kManyWaves) ? 1 : most_tiles;
  if (p.many && p.waves == kManyWaves && (small || p.two)) p.nb = 1;
  const int wg_rows = narrow * p.nb;
  p.tiles = (p.r_max + wg_rows - 1) / wg_rows;
  const int64_t wgs = pairs * p.tiles;
  // Splits as long as all workgroups run at once, one a CU: 8 x 32 pairs of
  // 8192 tokens, D = 128, 91.9 us without and 96.3 with two; 56 x 4 pairs of
  // 4001 tokens in fp32 38.9 us without and 45.2 with two.
  int64_t splits = 256 / wgs;
  // Up to four blocks a wave one launch beats the split and its join: 8 pairs, D =
  // 128, 400 / 800 / 1000 / 1500 tokens 7.1 / 8.9 / 10.0 / 12.3 us whole and 9.1 /
  // 9.9 / 10.0 / 10.1 split; with scores and several tiles the join runs anyway
  // (fp32, 40 rows, 1000 tokens 15.5 and 13.9).
  const bool whole = !p.many && p.max_nb <= 4 * kFewWaves && (!score || p.tiles == 1);
  const int64_t most = whole ? 1 : (p.max_nb + 7) / 8;
  splits = splits < most ? splits : most;
  splits = splits < kMaxSplits ? splits : kMaxSplits;
  p.splits = (int)(splits > 1 ? splits : 1);
  p.slots = 0, p.splits_max = p.splits, p.share_even = p.share_safe = 0.f;
  // Sequences share the workgroups by their lengths where the longest may have 32
  // blocks and more to a split: 8 sequences x 8 heads, D = 128, 16000 tokens each 47.5 us
  // and 46.0 without; 16000 down to 2700 31.9 and 34.2; one of 16000 beside seven of 300
  // 18.8 and 27.4; under 32 blocks (4 x 8, 2000 tokens and less) 11.1 and 10.2.
  // Beyond 128 pairs only those are split that have twice the mean of 256 pairs: 32 x
  // 8 of 16384 168 us and 163 (the join's launch), lengths between 100 and 16384,
  // the mean a fifth of the longest, 53 and 85; one of 16384 beside 31 of 200 21 and 79.
  // (Half as much more than the mean: 20 x 8 of 8192 72 us and 58.)
  const bool spare = p.splits == 1;
  if (!p.many && p.tiles == 1 && n_seqs > 1 && n_seqs <= kWave && hk <= kWave && p.max_nb < 1 << 20 &&
      (spare ? p.max_nb >= 8 * 32 : p.max_nb / p.splits >= 32)) {
    p.slots = kSlots + (spare ? (int)pairs : 0);
    const float each = (float)(p.slots / hk);
    p.share_even = (spare ? 2.f : 1.f) / (float)(kSlots / hk);
    p.share_safe = each > n_seqs ? (1.f + 0x1p-16f) / (each - (float)n_seqs) : 1e30f;
    if (spare) p.splits = 2;
    // one sequence has what the others leave
    p.splits_max = p.slots / hk - (n_seqs - 1);
    p.splits_max = p.splits_max < kMaxSplits ? p.splits_max : kMaxSplits;
  }
  // (k_attend adds up the scores of rows that one workgroup has whole)
  const bool join = p.splits > 1 || (score && (p.many || p.tiles > 1));
  const int each = p.splits <= kFewSplits ? kAtThreads / (d / 4) : 1;         // rows of a workgroup
  const int blocks = kAtThreads / score_lanes(p.r_max, p.splits);             // blocks of a workgroup
  p.row_groups = p.splits > 1 ? (pairs * p.r_max + each - 1) / each : 0;
  p.score_groups = join && score ? pairs * ((p.max_nb + blocks - 1) / blocks) : 0;
  p.threads = (p.slots ? p.slots : wgs * p.splits) * kFewThreads;             // (k_attend_many: twice, in small grids alone)
  const int64_t joins = (p.row_groups + p.score_groups) * kAtThreads;
  p.threads = p.threads > joins ? p.threads : joins;
  const size_t parts = (size_t)p.splits_max * pairs;
  auto up256 = [](size_t v) { return (v + 255) & ~size_t(255); };
  size_t off = PI_WS_HEADER_BYTES;
  p.part = off;
  off += up256(p.splits > 1 ? parts * p.r_max * d * sizeof(float) : 0);
  p.ml = off;
  off += up256(p.splits > 1 || score ? parts * p.r_max * sizeof(float2) : 0);
  p.lse = off;
  off += up256(score ? (size_t)pairs * p.max_nb * p.r_max * sizeof(float) : 0);
  p.count = off;
  off += up256(p.slots ? (size_t)pairs * sizeof(int) : 0);
  p.total = off;
  return p;
}

hipError_t launch_attend(const AttendArgs& a, const AttendPlan& p, int d, int dtype, hipStream_t s) {
  if (dtype == PI_F16) return d == 64 ? attend_nb<f16, 64>(a, p, s) : attend_nb<f16, 128>(a, p, s);
  return d == 64 ? attend_nb<float, 64>(a, p, s) : attend_nb<float, 128>(a, p, s);
}

}  // namespace pi
