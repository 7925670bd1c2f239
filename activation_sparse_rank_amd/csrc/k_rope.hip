// Rotary positions of queries and keys with an optional RMS norm of each
// head, in one pass (pi_qk_rope).
//
// y = x * w / sqrt(mean(x^2) + eps); pair (a, b) -> scale * (a cos - b sin,
// b cos + a sin).  Memory bound: every element is read and written once, and
// what a token's heads share, its cosines and sines, is computed once per
// workgroup into LDS (rot / 2 angles, reduced in 64 bits), while the first
// heads' loads are in flight.  A workgroup owns one token; D / (16 bytes)
// lanes hold a head, so a norm's sum is a butterfly inside a wave and a
// half-layout element finds its partner by a second 16-byte load that the
// first level cache answers.
#include "attn_device.h"

namespace pi {
namespace {

constexpr int kRopeThreads = 256;
constexpr int kRopeMaxD = 256;

// Workgroups of a call with few tokens split the heads, so that one token is
// not one CU's work alone.
constexpr int kRopeMinGroups = 512;

// PART: 0 interleaved; 1 half layout, rot / 2 a multiple of the 16-byte
// chunk; 2 half layout, partners at any offset (loaded one by one).
template <typename T, int PART, bool NORM>
__global__ __launch_bounds__(kRopeThreads) void k_qk_rope(RopeArgs a, int group, int hsplit) {
  constexpr int V = Vec<T>::N;
  __shared__ float2 cs[kRopeMaxD / 2];
  __shared__ float wn[NORM ? 2 * kRopeMaxD : 1];
  const int tok = blockIdx.x / hsplit, part = blockIdx.x % hsplit;
  const int half = a.rot / 2;
  const int per = kRopeThreads / group;
  const int lane = threadIdx.x % group;
  const int e0 = lane * V;
  const bool in_head = e0 < a.d;
  const int n_heads = a.in[0].n + a.in[1].n;
  const int step = per * hsplit;

  auto row = [&](const HeadRows* r, int h) {
    const int i = h >= a.in[0].n;
    const HeadRows& x = i ? r[1] : r[0];
    return static_cast<T*>(x.p) + (int64_t)tok * x.ts + (int64_t)(i ? h - a.in[0].n : h) * x.hs;
  };
  // A chunk of the head and, in the half layout, its partners.
  u32x4 x = {0, 0, 0, 0}, xp = {0, 0, 0, 0};
  auto load = [&](int h) {
    if (h >= n_heads || !in_head) return;
    const T* p = row(a.in, h);
    x = ld16(p + e0);
    if constexpr (PART == 1) {
      if (e0 < a.rot) xp = ld16(p + (e0 < half ? e0 + half : e0 - half));
    } else if constexpr (PART == 2) {
      if (e0 < a.rot) {
        float f[V];
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const int e = e0 + i;
          f[i] = e < a.rot ? (float)p[e < half ? e + half : e - half] : 0.f;
        }
        xp = Vec<T>::pack(f);      // the same values back: no rounding
      }
    }
  };

  int h = part * per + threadIdx.x / group;
  load(h);
  for (int i = threadIdx.x; i < half; i += kRopeThreads) {
    double t = (double)a.pos[tok] * a.freqs[i];
    t -= rint(t);
    float s, c;
    sincospif(2.f * (float)t, &s, &c);
    cs[i] = float2{a.scale * c, a.scale * s};
  }
  if constexpr (NORM) {
    for (int i = threadIdx.x; i < a.d; i += kRopeThreads) {
      wn[i] = a.w[0] ? a.w[0][i] : 1.f;
      wn[kRopeMaxD + i] = a.w[1] ? a.w[1][i] : 1.f;
    }
  }
  __syncthreads();

  for (; h - (int)(threadIdx.x / group) < n_heads; h += step) {
    const bool mine = h < n_heads && in_head;
    float y[V], yp[V];
    Vec<T>::unpack(x, y);
    Vec<T>::unpack(xp, yp);
    if constexpr (NORM) {
      float ss = 0.f;
      if (mine) {
#pragma unroll
        for (int i = 0; i < V; ++i) ss = __builtin_fmaf(y[i], y[i], ss);
      }
      for (int m = group / 2; m >= 1; m >>= 1) ss += __shfl_xor(ss, m, kWave);
      const int k = h >= a.in[0].n;
      if (mine && a.w[k]) {
        const float r = 1.f / sqrtf(ss / (float)a.d + a.eps);
        const float* w = wn + k * kRopeMaxD;
#pragma unroll
        for (int i = 0; i < V; ++i) {
          y[i] = y[i] * r * w[e0 + i];
          if constexpr (PART > 0) {
            const int e = e0 + i;
            if (e < a.rot) yp[i] = yp[i] * r * w[e < half ? e + half : e - half];
          }
        }
      }
    }
    if (mine) {
      float o[V];
      if constexpr (PART == 0) {
#pragma unroll
        for (int i = 0; i < V; i += 2) {
          o[i] = y[i], o[i + 1] = y[i + 1];
          if (e0 + i < a.rot) {
            const float2 t = cs[(e0 + i) / 2];
            o[i] = __builtin_fmaf(y[i], t.x, -(y[i + 1] * t.y));
            o[i + 1] = __builtin_fmaf(y[i + 1], t.x, y[i] * t.y);
          }
        }
      } else {
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const int e = e0 + i;
          o[i] = y[i];
          if (e < a.rot) {
            const float2 t = cs[e < half ? e : e - half];
            o[i] = __builtin_fmaf(y[i], t.x, e < half ? -(yp[i] * t.y) : yp[i] * t.y);
          }
        }
      }
      *reinterpret_cast<u32x4*>(row(a.out, h) + e0) = Vec<T>::pack(o);
    }
    load(h + step);
  }
}

template <typename T, int PART>
hipError_t rope_part(const RopeArgs& a, int group, int hsplit, hipStream_t s) {
  const dim3 grid((unsigned)a.n_tok * hsplit);
  if (a.w[0] || a.w[1])
    k_qk_rope<T, PART, true><<<grid, kRopeThreads, 0, s>>>(a, group, hsplit);
  else
    k_qk_rope<T, PART, false><<<grid, kRopeThreads, 0, s>>>(a, group, hsplit);
  return hipGetLastError();
}

template <typename T>
hipError_t rope_type(const RopeArgs& a, hipStream_t s) {
  constexpr int V = Vec<T>::N;
  int group = 1;
  while (group * V < a.d) group *= 2;
  const int per = kRopeThreads / group;
  const int passes = (a.in[0].n + a.in[1].n + per - 1) / per;
  int hsplit = (kRopeMinGroups + a.n_tok - 1) / a.n_tok;
  hsplit = hsplit < passes ? hsplit : passes;
  if (a.layout == PI_ROPE_INTERLEAVED) return rope_part<T, 0>(a, group, hsplit, s);
  return (a.rot / 2) % V ? rope_part<T, 2>(a, group, hsplit, s) : rope_part<T, 1>(a, group, hsplit, s);
}

}  // namespace

hipError_t launch_qk_rope(const RopeArgs& a, hipStream_t s) {
  return a.dtype == PI_F16 ? rope_type<f16>(a, s) : rope_type<float>(a, s);
}

}  // namespace pi
