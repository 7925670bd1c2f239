// Device helpers that the attention-side kernels share: elements of 16 bytes
// as floats, and the checks of values that live in device memory.
#pragma once

#include "attn_internal.h"

namespace pi {

constexpr int kBlk = PI_KV_BLOCK;

// 16 bytes of T as floats and back (one rounding, to nearest even).
template <typename T>
struct Vec;
template <>
struct Vec<float> {
  static constexpr int N = 4;
  __device__ static void unpack(u32x4 v, float* f) {
    f[0] = as_f(v.x), f[1] = as_f(v.y), f[2] = as_f(v.z), f[3] = as_f(v.w);
  }
  __device__ static u32x4 pack(const float* f) {
    u32x4 v;
    v.x = __builtin_bit_cast(unsigned, f[0]), v.y = __builtin_bit_cast(unsigned, f[1]);
    v.z = __builtin_bit_cast(unsigned, f[2]), v.w = __builtin_bit_cast(unsigned, f[3]);
    return v;
  }
};
template <>
struct Vec<f16> {
  static constexpr int N = 8;
  __device__ static void unpack(u32x4 v, float* f) {
    const unsigned w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const f16x2 h = as_h2(w[i]);
      f[2 * i] = (float)h.x, f[2 * i + 1] = (float)h.y;
    }
  }
  __device__ static u32x4 pack(const float* f) {
    unsigned w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f16x2 h;
      h.x = (f16)f[2 * i], h.y = (f16)f[2 * i + 1];
      w[i] = __builtin_bit_cast(unsigned, h);
    }
    return u32x4{w[0], w[1], w[2], w[3]};
  }
};

__device__ __forceinline__ float quiet_nan() { return __builtin_bit_cast(float, 0x7fc00000u); }

// Inclusive sums over the lanes of a wave, lane 0 first: shifts inside rows of
// 16 lanes, then the rows' ends handed on.
__device__ __forceinline__ unsigned wave_scan(unsigned x) {
  int v = (int)x;
  v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xf, 0xf, false);   // row_shr:1
  v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xf, 0xf, false);   // row_shr:2
  v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xf, 0xf, false);   // row_shr:4
  v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xf, 0xf, false);   // row_shr:8
  v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xa, 0xf, false);   // row_bcast:15 into rows 1 and 3
  v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xc, 0xf, false);   // row_bcast:31 into rows 2 and 3
  return (unsigned)v;
}

// The largest of the lanes' values, in lane 63 (the same steps).
__device__ __forceinline__ unsigned wave_max(unsigned v) {
  auto step = [&](unsigned x) { v = v > x ? v : x; };
  step((unsigned)__builtin_amdgcn_update_dpp(0, (int)v, 0x111, 0xf, 0xf, false));
  step((unsigned)__builtin_amdgcn_update_dpp(0, (int)v, 0x112, 0xf, 0xf, false));
  step((unsigned)__builtin_amdgcn_update_dpp(0, (int)v, 0x114, 0xf, 0xf, false));
  step((unsigned)__builtin_amdgcn_update_dpp(0, (int)v, 0x118, 0xf, 0xf, false));
  step((unsigned)__builtin_amdgcn_update_dpp(0, (int)v, 0x142, 0xa, 0xf, false));
  step((unsigned)__builtin_amdgcn_update_dpp(0, (int)v, 0x143, 0xc, 0xf, false));
  return v;
}

// The rows and the length of sequence s as device memory has them, checked.
struct Seq {
  int q0;      // its first row
  int n;       // its rows (of an invalid sequence: those inside [0, n_tok], to be marked)
  int len;     // tokens held, 0 where invalid
  bool ok;
};
__device__ __forceinline__ Seq read_seq(const int32_t* lens, const int32_t* q_start, int s, int max_new, int n_tok,
                                        int max_len) {
  const long long q0 = q_start ? q_start[s] : (long long)s * max_new;
  const long long q1 = q_start ? q_start[s + 1] : q0 + max_new;
  const int len = lens[s];
  Seq r;
  r.ok = q0 >= 0 && q1 >= q0 && q1 <= n_tok && q1 - q0 <= max_new && len >= 0 && len <= max_len;
  const long long a = q0 < 0 ? 0 : (q0 > n_tok ? n_tok : q0);
  const long long b = q1 < a ? a : (q1 > n_tok ? n_tok : q1);
  r.q0 = (int)a;
  r.n = (int)(b - a);
  r.len = r.ok ? len : 0;
  return r;
}

}  // namespace pi
