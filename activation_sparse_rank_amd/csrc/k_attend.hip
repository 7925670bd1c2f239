// Attention over the 8-bit cache (pi_attend): softmax(scale q k^T) v with the
// softmax's running maximum and sum, one pass over the pages.
//
// Mathematics.  For a block of 32 tokens, S^T = K Q^T on the matrix cores
// (v_mfma_f32_16x16x32_f16; the codes minus 128 are exact in fp16), 16 query
// rows to a tile.  The block's key scale multiplies S, its value scale is an
// addend of the exponent: p = 2^(S ks c - m + log2(vs / vref)), so neither
// costs an instruction per element, and the sum of the weights takes
// vs / vref out again once per block.  O^T += V^T P^T with P in fp16.  A lane holds
// the weights of 8 tokens of one row, which is what the second product's
// operand takes from it: P never leaves the registers.  The reference
// exponent m moves only when the weights of a block outgrow fp16's range above it (a
// ballot sees their sum), so maxima are seldom taken and sums seldom rescaled.
//
// The pages' byte order gives each lane its 16 codes of an operand in one
// 16-byte load, 1 KB in a row for a wave.
//
// Two ways to cut the work, by size (attend_plan): with few rows the four
// waves of a workgroup share the rows and take every fourth block, the blocks
// are split over workgroups as well, and partial sums are joined in a fixed
// order (in LDS, then in k_attend_join); with many rows each wave has rows
// of its own and walks all the blocks they see.
#include "attn_device.h"

namespace pi {
namespace {

typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x4 __attribute__((ext_vector_type(4)));
typedef float f32x8 __attribute__((ext_vector_type(8)));

constexpr int kAtThreads = 256;
constexpr int kAtWaves = kAtThreads / kWave;
constexpr int kMaxSplits = 64;
constexpr float kNoMax = -1e30f;     // reference before the first visible token
// Weights are held times 2^6, and a lane's eight of a block may sum to 2^15
// (fp16 holds 65504) before the reference moves: no maximum is taken but
// then.  What a weight loses below fp16's smallest step is at most 2^-31 of the
// row's largest weight, so that 10^5 such tokens beside one that takes the
// row are still counted.
constexpr float kBias = 6.f;
constexpr float kMost = 0x1p15f;
// Under this share of the wave's largest value scale a block's weights would
// leave fp16's range: the sums are brought to the block's scale (a power of
// two, exact, 2^-60 at least) for its product and back.
constexpr float kSmall = 0x1p-10f, kSmallest = 0x1p-60f;

__device__ __forceinline__ f32x4 mfma16(f16x8 a, f16x8 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
}

// 8 codes to fp16 values code - 128: the bytes become 1024 + code by their
// place in the fraction of 0x6400, less 1152.  Exact.
__device__ __forceinline__ f16x8 codes_f16(unsigned lo, unsigned hi) {
  const f16x2 off = {(f16)-1152.f, (f16)-1152.f};
  f16x2 h[4];
  h[0] = as_h2(__builtin_amdgcn_perm(0x64646464u, lo, 0x04010400u)) + off;
  h[1] = as_h2(__builtin_amdgcn_perm(0x64646464u, lo, 0x04030402u)) + off;
  h[2] = as_h2(__builtin_amdgcn_perm(0x64646464u, hi, 0x04010400u)) + off;
  h[3] = as_h2(__builtin_amdgcn_perm(0x64646464u, hi, 0x04030402u)) + off;
  return __builtin_bit_cast(f16x8, u32x4{__builtin_bit_cast(unsigned, h[0]), __builtin_bit_cast(unsigned, h[1]),
                                         __builtin_bit_cast(unsigned, h[2]), __builtin_bit_cast(unsigned, h[3])});
}

__device__ __forceinline__ float lane_f(float v, int lane) {
  return as_f((unsigned)__builtin_amdgcn_readlane((int)__builtin_bit_cast(unsigned, v), lane));
}

// Sum and maximum over the four lanes that hold a row (lane % 16).
__device__ __forceinline__ float row_sum(float v) {
  v += __shfl_xor(v, 16, kWave);
  return v + __shfl_xor(v, 32, kWave);
}
__device__ __forceinline__ float row_max(float v) {
  v = fmaxf(v, __shfl_xor(v, 16, kWave));
  return fmaxf(v, __shfl_xor(v, 32, kWave));
}

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

// Waves that a SIMD holds: what the registers of a wave's rows leave.
constexpr int waves_per_simd(int d, int nb, bool f32) {
  return d * nb * (f32 ? 2 : 1) <= 64 ? 4 : (d * nb * (f32 ? 2 : 1) <= 128 ? 3 : 2);
}

// T: rows (fp16; fp32 as two fp16 parts).  NB: 16-row tiles of a wave.
// SCORE: the weights of each block are wanted.  ROWS: see above.
template <typename T, int D, int NB, bool SCORE, bool ROWS>
__global__ __launch_bounds__(kAtThreads, waves_per_simd(D, NB, sizeof(T) == 4)) void k_attend(AttendArgs a) {
  constexpr int KK = D / 64, DT = D / 16, DB = D / 32;
  constexpr bool kTwo = sizeof(T) == 4;             // two fp16 parts of q
  constexpr bool kTwoP = kTwo || !ROWS;             // and of p: always where the pages' bytes bound the time
  const int pairs = a.n_seqs * a.hk;
  const int pair = blockIdx.x % pairs;
  const int tile = blockIdx.x / pairs % a.tiles;
  const int split = blockIdx.x / pairs / a.tiles;
  const int s = pair / a.hk, h = pair % a.hk;
  const int lane = lane_id(), wave = wave_id(), g = lane / 16, c = lane % 16;
  const Seq q = read_seq(a.lens, a.q_start, s, a.max_q, a.n_tok, a.max_len);
  if (!q.ok) {
    if (split == 0) nan_rows<T>(a, q, h, D, (int64_t)tile * kAtThreads + threadIdx.x, (int64_t)a.tiles * kAtThreads);
    if (threadIdx.x == 0) raise_flag(a.flags, PI_FLAG_KV_RANGE);
    return;
  }
  const int rows = q.n * a.group;
  const int r0 = tile * 16 * NB;
  if (r0 >= rows) return;
  const int seen0 = q.len - q.n + 1;                // tokens that the sequence's first row sees (may be < 1)
  const int r1 = r0 + 16 * NB < rows ? r0 + 16 * NB : rows;
  auto clamp_len = [&](int v) { return v < 0 ? 0 : v; };
  const int kmin = clamp_len(seen0 + r0 / a.group), kmax = clamp_len(seen0 + (r1 - 1) / a.group);
  const int nbk = (kmax + kBlk - 1) / kBlk;
  const int per = (nbk + a.splits - 1) / a.splits;
  const int b0 = split * per, b1 = b0 + per < nbk ? b0 + per : nbk;
  constexpr int kStep = kAtWaves;
  const int start = b0 + wave;
  const int mine = start < b1 ? (b1 - start + kStep - 1) / kStep : 0;

  // Queries: lane (g, c) has elements 64 kk + 16 g .. + 16 of row c.
  f16x8 qf[NB][KK][2], ql[NB][kTwo ? KK : 1][2];
  float rs[NB];                                     // a row's power of two (fp32 rows)
  int sees[NB];
#pragma unroll
  for (int nb = 0; nb < NB; ++nb) {
    const int r = r0 + nb * 16 + c;
    const bool in = r < rows;
    const int t = in ? r / a.group : 0, head = h * a.group + (in ? r % a.group : 0);
    const T* p = static_cast<const T*>(a.q) + (int64_t)(q.q0 + t) * a.q_ts + (int64_t)head * a.q_hs + 16 * g;
    sees[nb] = in ? clamp_len(seen0 + t) : 0;
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
      rs[nb] = __builtin_amdgcn_ldexpf(1.f, e < -126 ? -126 : e);
#pragma unroll
      for (int kk = 0; kk < KK; ++kk)
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const float v = __builtin_amdgcn_ldexpf(x[kk][i], -(e < -126 ? -126 : e));
          const f16 hi = (f16)v;
          qf[nb][kk][i / 8][i % 8] = hi;
          ql[nb][kk][i / 8][i % 8] = (f16)(v - (float)hi);
        }
    }
  }

  f32x4 o[NB][DT];
  float m[NB], l[NB];
#pragma unroll
  for (int nb = 0; nb < NB; ++nb) {
    m[nb] = kNoMax, l[nb] = 0.f;
#pragma unroll
    for (int t = 0; t < DT; ++t) o[nb][t] = f32x4{0.f, 0.f, 0.f, 0.f};
  }
  float vref = 0x1p-126f;                           // o is in units of it

  u32x4 rk[2 * KK], rv[DB];                         // a block's codes, as they lie in the page
  bool bad = false;
  for (int base = 0; base < mine; base += kWave) {
    const int cnt = mine - base < kWave ? mine - base : kWave;
    // Lane i: page and scales of the i-th block.
    int page = 0;
    float ks = 0.f, vs = 0.f;
    bool no_page = false;
    if (lane < cnt) {
      page = a.table[(int64_t)pair * a.max_blocks + start + (base + lane) * kStep];
      no_page = (unsigned)page >= (unsigned)a.n_pages;
      page = no_page ? 0 : page;
      bad |= no_page;
    }
    auto page_at = [&](int i) {
      return a.pages + (int64_t)__builtin_amdgcn_readlane(page, i) * (2 * kBlk * D) + lane * 16;
    };
    auto load_k = [&](int i) {
      const uint8_t* p = page_at(i);
#pragma unroll
      for (int u = 0; u < 2 * KK; ++u) rk[u] = ROWS ? ld16(p + u * 1024) : ld_nt(p + u * 1024);
    };
    auto load_v = [&](int i) {
      const uint8_t* p = page_at(i) + kBlk * D;
#pragma unroll
      for (int u = 0; u < DB; ++u) rv[u] = ROWS ? ld16(p + u * 1024) : ld_nt(p + u * 1024);
    };
    // The first block's codes are on their way while the scales come.
    load_k(0);
    load_v(0);
    if (lane < cnt) {
      const float2 sc = reinterpret_cast<const float2*>(a.scales)[page];
      ks = no_page ? -1.f : sc.x, vs = sc.y;
      // A scale that is no number: what sees the block is NaN, through its logits.
      if (!(ks >= 0.f && ks < __builtin_inff() && vs >= 0.f && vs < __builtin_inff())) ks = quiet_nan(), vs = 0.f;
    }
    float vmax = vs;
#pragma unroll
    for (int x = 32; x >= 1; x >>= 1) vmax = fmaxf(vmax, __shfl_xor(vmax, x, kWave));
    const float vtop = as_f(__builtin_bit_cast(unsigned, fmaxf(vmax, 0x1p-126f)) & 0x7f800000u);
    if (vtop > vref) {
      const float f = vref / vtop;
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int t = 0; t < DT; ++t) o[nb][t] *= f;
      vref = vtop;
    }
    const float ratio = vs > 0.f ? vs / vref : 1.f;
    const unsigned long long smalls = __ballot(ratio < kSmall);
    const float unit = ratio < kSmall ? as_f(__builtin_bit_cast(unsigned, fmaxf(ratio, kSmallest)) & 0x7f800000u) : 1.f;
    const float share = fmaxf(ratio / unit, 0x1p-60f);
    const float lr = log2_hw(share) + kBias, iv = 1.f / share;

    // One set of registers for the codes: the next block's keys are on their
    // way from the end of the first product on, its values from the second's.
    for (int i = 0; i < cnt; ++i) {
      const int b = start + (base + i) * kStep;
      const float ksc = lane_f(ks, i) * a.scale;
      const float lrb = lane_f(lr, i), ivb = lane_f(iv, i);
      f32x4 st[NB][2];
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) st[nb][0] = st[nb][1] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int kk = 0; kk < KK; ++kk)
#pragma unroll
        for (int f = 0; f < 2; ++f)
#pragma unroll
          for (int mb = 0; mb < 2; ++mb) {
            const u32x4 w = rk[mb * KK + kk];
            const f16x8 kf = f ? codes_f16(w.z, w.w) : codes_f16(w.x, w.y);
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) {
              st[nb][mb] = mfma16(kf, qf[nb][kk][f], st[nb][mb]);
              if constexpr (kTwo) st[nb][mb] = mfma16(kf, ql[nb][kk][f], st[nb][mb]);
            }
          }
      if (i + 1 < cnt) load_k(i + 1);
      const bool edge = (b + 1) * kBlk > kmin;      // some row does not see all of the block
      auto scale_of = [&](int nb) { return kTwo ? ksc * rs[nb] : ksc; };
      if (edge) {
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
          const float sc = scale_of(nb);
#pragma unroll
          for (int mb = 0; mb < 2; ++mb)
#pragma unroll
            for (int j = 0; j < 4; ++j)
              st[nb][mb][j] = b * kBlk + mb * 16 + 4 * g + j < sees[nb] ? st[nb][mb][j] * sc : -__builtin_inff();
        }
      }
      f16x8 pf[NB], pl[NB];
      float sum[NB];
      auto weights = [&](int nb) {
        const float sc = edge ? 1.f : scale_of(nb), off = lrb - m[nb];
        float p[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) p[j] = exp2_hw(__builtin_fmaf(st[nb][j / 4][j % 4], sc, off));
        const f32x8 pv = {p[0], p[1], p[2], p[3], p[4], p[5], p[6], p[7]};
        pf[nb] = __builtin_convertvector(pv, f16x8);
        if constexpr (kTwoP) pl[nb] = __builtin_convertvector(pv - __builtin_convertvector(pf[nb], f32x8), f16x8);
        if constexpr (kTwoP || SCORE) {
          sum[nb] = (p[0] + p[1] + (p[2] + p[3])) + (p[4] + p[5] + (p[6] + p[7]));
        } else {
          // the sum of the rounded weights, which the second product multiplies
          const u32x4 w = __builtin_bit_cast(u32x4, pf[nb]);
          const f16x2 one = {(f16)1.f, (f16)1.f};
          float x = __builtin_amdgcn_fdot2(as_h2(w.x), one, 0.f, false);
          x = __builtin_amdgcn_fdot2(as_h2(w.y), one, x, false);
          x = __builtin_amdgcn_fdot2(as_h2(w.z), one, x, false);
          sum[nb] = __builtin_amdgcn_fdot2(as_h2(w.w), one, x, false);
        }
      };
      bool over = false;
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
        weights(nb);
        over |= !(sum[nb] < kMost);
      }
      if (__any(over)) {                            // a weight passes the reference by too much: move it
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
          const f32x4 s0 = st[nb][0], s1 = st[nb][1];
          const float top = fmaxf(fmaxf(fmaxf(s0[0], s0[1]), fmaxf(s0[2], s0[3])),
                                  fmaxf(fmaxf(s1[0], s1[1]), fmaxf(s1[2], s1[3]))) * (edge ? 1.f : scale_of(nb));
          const float mn = fmaxf(m[nb], row_max(top));
          const float f = exp2_hw(m[nb] - mn);
          m[nb] = mn;
          l[nb] *= f;
#pragma unroll
          for (int t = 0; t < DT; ++t) o[nb][t] *= f;
          weights(nb);
        }
      }
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
        l[nb] = __builtin_fmaf(sum[nb], ivb, l[nb]);
        if constexpr (SCORE) {
          const float w = row_sum(sum[nb]) * ivb;
          const int r = r0 + nb * 16 + c;
          if (g == 0 && r < rows) a.lse[((int64_t)pair * a.max_nb + b) * a.r_max + r] = m[nb] + log2_hw(w);
        }
      }
      auto rescale = [&](float f) {
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int t = 0; t < DT; ++t) o[nb][t] *= f;
      };
      const bool far = smalls >> i & 1;
      if (far) rescale(1.f / lane_f(unit, i));
#pragma unroll
      for (int t = 0; t < DT; ++t) {
        const u32x4 w = rv[t / 2];
        const f16x8 v = t % 2 ? codes_f16(w.z, w.w) : codes_f16(w.x, w.y);
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
          o[nb][t] = mfma16(v, pf[nb], o[nb][t]);
          if constexpr (kTwoP) o[nb][t] = mfma16(v, pl[nb], o[nb][t]);
        }
      }
      if (far) rescale(lane_f(unit, i));
      if (i + 1 < cnt) load_v(i + 1);
    }
  }
  raise_flag_if_any(a.flags, bad, PI_FLAG_KV_RANGE);

#pragma unroll
  for (int nb = 0; nb < NB; ++nb) {
    l[nb] = row_sum(l[nb]);
#pragma unroll
    for (int t = 0; t < DT; ++t) o[nb][t] *= vref;
  }
  auto out_row = [&](int r) {
    return static_cast<T*>(a.out) + (int64_t)(q.q0 + r / a.group) * a.o_ts + (int64_t)(h * a.group + r % a.group) * a.o_hs;
  };
  {
    // The four waves' sums, added in wave order.
    __shared__ float so[kAtWaves][16][D + 4];
    __shared__ float sm[kAtWaves][16], sl[kAtWaves][16];
    constexpr int E = D / 16;                       // elements of a thread
    const int row = threadIdx.x / 16, e0 = threadIdx.x % 16 * E;
    for (int nb = 0; nb < NB; ++nb) {
      if (nb) __syncthreads();
#pragma unroll
      for (int x = 0; x < NB; ++x) {
        if (x != nb) continue;
#pragma unroll
        for (int t = 0; t < DT; ++t) *reinterpret_cast<f32x4*>(&so[wave][c][16 * t + 4 * g]) = o[x][t];
        if (g == 0) sm[wave][c] = m[x], sl[wave][c] = l[x];
      }
      __syncthreads();
      const int r = r0 + nb * 16 + row;
      if (r >= rows) continue;
      float top = sm[0][row];
#pragma unroll
      for (int w = 1; w < kAtWaves; ++w) top = fmaxf(top, sm[w][row]);
      float sum = 0.f, v[E];
#pragma unroll
      for (int k = 0; k < E; ++k) v[k] = 0.f;
#pragma unroll
      for (int w = 0; w < kAtWaves; ++w) {
        const float f = exp2_hw(sm[w][row] - top);
        sum = __builtin_fmaf(f, sl[w][row], sum);
#pragma unroll
        for (int k = 0; k < E; ++k) v[k] = __builtin_fmaf(f, so[w][row][e0 + k], v[k]);
      }
      const int64_t at = ((int64_t)split * pairs + pair) * a.r_max + r;
      if (a.splits > 1) {
#pragma unroll
        for (int k = 0; k < E; k += 4)
          *reinterpret_cast<f32x4*>(a.part + at * D + e0 + k) = f32x4{v[k], v[k + 1], v[k + 2], v[k + 3]};
      } else {
        const float inv = sum == 0.f ? 0.f : 1.f / sum;
        T* p = out_row(r) + e0;
#pragma unroll
        for (int k = 0; k < E; k += 4) {
          const f32x4 x = f32x4{v[k], v[k + 1], v[k + 2], v[k + 3]} * inv;
          if constexpr (kTwo) *reinterpret_cast<f32x4*>(p + k) = x;
          else *reinterpret_cast<f16x4*>(p + k) = __builtin_convertvector(x, f16x4);
        }
      }
      if ((a.splits > 1 || SCORE) && e0 == 0) a.ml[at] = float2{top, sum};
    }
  }
}

// Reference exponent and sum of a row over its splits.
__device__ __forceinline__ float2 row_ml(const AttendArgs& a, int pairs, int pair, int r) {
  float2 v = a.ml[(int64_t)pair * a.r_max + r];
  for (int i = 1; i < a.splits; ++i) {
    const float2 w = a.ml[((int64_t)i * pairs + pair) * a.r_max + r];
    const float top = fmaxf(v.x, w.x);
    v.y = v.y * exp2_hw(v.x - top) + w.y * exp2_hw(w.x - top);
    v.x = top;
  }
  return v;
}

// Joins the splits' sums into rows (workgroups below row_groups, one a row)
// and adds the blocks' weights to the score (the others, kScoreBlocks blocks
// of a (sequence, kv head) each).
constexpr int kScoreBlocks = 64;
template <typename T, int D>
__global__ __launch_bounds__(kAtThreads) void k_attend_join(AttendArgs a, int row_groups) {
  const int pairs = a.n_seqs * a.hk;
  if ((int)blockIdx.x < row_groups) {
    constexpr int L = D / 4, G = kAtThreads / L;    // lanes of a row, splits at a time
    __shared__ f32x4 acc[G][L];
    const int pair = blockIdx.x / a.r_max, r = blockIdx.x % a.r_max;
    const Seq q = read_seq(a.lens, a.q_start, pair / a.hk, a.max_q, a.n_tok, a.max_len);
    if (!q.ok || r >= q.n * a.group) return;
    // Every split's part of this thread's elements, in flight while the weights are found.
    const int lane = lane_id(), part = threadIdx.x / L, e = threadIdx.x % L * 4;
    constexpr int N = kMaxSplits / G;
    f32x4 x[N];
#pragma unroll
    for (int k = 0; k < N; ++k) {
      const int i = k * G + part < a.splits ? k * G + part : 0;
      x[k] = *reinterpret_cast<const f32x4*>(a.part + (((int64_t)i * pairs + pair) * a.r_max + r) * D + e);
    }
    float2 v = {kNoMax, 0.f};
    if (lane < a.splits) v = a.ml[((int64_t)lane * pairs + pair) * a.r_max + r];
    float top = v.x;
#pragma unroll
    for (int y = 32; y >= 1; y >>= 1) top = fmaxf(top, __shfl_xor(top, y, kWave));
    const float f = exp2_hw(v.x - top);
    const float sum = wave_sum(f * v.y);
    f32x4 o = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int k = 0; k < N; ++k) {
      const int i = k * G + part;
      const float w = __shfl(f, i, kWave);
      o += i < a.splits ? w * x[k] : f32x4{0.f, 0.f, 0.f, 0.f};
    }
    acc[part][e / 4] = o;
    __syncthreads();
    if (part) return;
#pragma unroll
    for (int i = 1; i < G; ++i) o += acc[i][e / 4];
    o *= sum == 0.f ? 0.f : 1.f / sum;
    const int h = pair % a.hk;
    T* p = static_cast<T*>(a.out) + (int64_t)(q.q0 + r / a.group) * a.o_ts + (int64_t)(h * a.group + r % a.group) * a.o_hs + e;
    if constexpr (sizeof(T) == 4) *reinterpret_cast<f32x4*>(p) = o;
    else *reinterpret_cast<f16x4*>(p) = __builtin_convertvector(o, f16x4);
    return;
  }
  const int per = (a.max_nb + kScoreBlocks - 1) / kScoreBlocks;
  const int pair = (blockIdx.x - row_groups) / per, first = (blockIdx.x - row_groups) % per * kScoreBlocks;
  const Seq q = read_seq(a.lens, a.q_start, pair / a.hk, a.max_q, a.n_tok, a.max_len);
  if (!q.ok || first * kBlk >= q.len) return;
  constexpr int kChunk = 256, Q = kAtThreads / kScoreBlocks;
  __shared__ float lse[kChunk];
  const int rows = q.n * a.group, seen0 = q.len - q.n + 1;
  const int b = first + threadIdx.x / Q, sub = threadIdx.x % Q;
  float w = 0.f;
  for (int c0 = 0; c0 < rows; c0 += kChunk) {
    __syncthreads();
    const int r = c0 + threadIdx.x;
    if (r < rows) {
      const float2 v = row_ml(a, pairs, pair, r);
      lse[threadIdx.x] = v.x + log2_hw(v.y);
    }
    __syncthreads();
    if (b * kBlk < q.len) {
      const float* from = a.lse + ((int64_t)pair * a.max_nb + b) * a.r_max;
      for (int k = sub; k < kChunk && c0 + k < rows; k += Q)
        if (b * kBlk < seen0 + (c0 + k) / a.group) w += exp2_hw(from[c0 + k] - lse[k]);
    }
  }
#pragma unroll
  for (int x = 1; x < Q; x <<= 1) w += __shfl_xor(w, x, kWave);
  if (sub == 0 && b * kBlk < q.len) a.score[(int64_t)pair * a.max_blocks + b] += w;
}

template <typename T, int D, int NB, bool ROWS>
hipError_t attend_run(const AttendArgs& a, hipStream_t s) {
  const int pairs = a.n_seqs * a.hk;
  const dim3 grid((unsigned)pairs * a.tiles * a.splits);
  if (a.score) k_attend<T, D, NB, true, ROWS><<<grid, kAtThreads, 0, s>>>(a);
  else k_attend<T, D, NB, false, ROWS><<<grid, kAtThreads, 0, s>>>(a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || (a.splits == 1 && !a.score)) return e;
  const int row_groups = a.splits > 1 ? pairs * a.r_max : 0;
  const int score_groups = a.score ? pairs * ((a.max_nb + kScoreBlocks - 1) / kScoreBlocks) : 0;
  k_attend_join<T, D><<<dim3((unsigned)row_groups + score_groups), kAtThreads, 0, s>>>(a, row_groups);
  return hipGetLastError();
}

// 16-row tiles that a wave's registers hold.
constexpr int max_tiles(int d, bool f32) { return (d == 64 ? 4 : 2) / (f32 ? 2 : 1); }

template <typename T, int D>
hipError_t attend_nb(const AttendArgs& a, const AttendPlan& p, hipStream_t s) {
  constexpr int kMax = max_tiles(D, sizeof(T) == 4);
  if (p.rows) return attend_run<T, D, kMax, true>(a, s);
  if constexpr (kMax >= 4)
    if (p.nb == 4) return attend_run<T, D, 4, false>(a, s);
  if constexpr (kMax >= 2)
    if (p.nb == 2) return attend_run<T, D, 2, false>(a, s);
  return attend_run<T, D, 1, false>(a, s);
}

}  // namespace

AttendPlan attend_plan(int n_seqs, int hk, int group, int d, int dtype, int max_q, int max_len, bool score) {
  AttendPlan p;
  const int64_t pairs = (int64_t)n_seqs * hk;
  p.r_max = max_q * group;
  p.max_nb = (max_len + kBlk - 1) / kBlk;
  const int cap = max_tiles(d, dtype == PI_F32);
  p.nb = 1;
  while (p.nb < cap && p.nb * 16 < p.r_max) p.nb *= 2;
  // Waves with rows of their own where that fills the waves and the CUs.
  const int own = (p.r_max + 16 * cap - 1) / (16 * cap);
  p.rows = p.r_max >= 16 * cap * kAtWaves && pairs * own >= 256;
  p.tiles = p.rows ? own : (p.r_max + 16 * p.nb - 1) / (16 * p.nb);
  int64_t splits = 1;
  if (!p.rows) {
    const int64_t want = (1024 + pairs * p.tiles - 1) / (pairs * p.tiles), most = (p.max_nb + 7) / 8;
    splits = want < most ? want : most;
    splits = splits < kMaxSplits ? splits : kMaxSplits;
  }
  p.splits = (int)splits;
  auto up256 = [](size_t v) { return (v + 255) & ~size_t(255); };
  size_t off = PI_WS_HEADER_BYTES;
  p.part = off;
  off += up256(p.splits > 1 ? (size_t)p.splits * pairs * p.r_max * d * sizeof(float) : 0);
  p.ml = off;
  off += up256(p.splits > 1 || score ? (size_t)p.splits * pairs * p.r_max * sizeof(float2) : 0);
  p.lse = off;
  off += up256(score ? (size_t)pairs * p.max_nb * p.r_max * sizeof(float) : 0);
  p.total = off;
  return p;
}

hipError_t launch_attend(const AttendArgs& a, const AttendPlan& p, int d, int dtype, hipStream_t s) {
  if (dtype == PI_F16) return d == 64 ? attend_nb<f16, 64>(a, p, s) : attend_nb<f16, 128>(a, p, s);
  return d == 64 ? attend_nb<float, 64>(a, p, s) : attend_nb<float, 128>(a, p, s);
}

}  // namespace pi
