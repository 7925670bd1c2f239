// Rotary positions of queries and keys with an optional RMS norm of each
// head, in one pass (pi_qk_rope).
//
// y = x * w / sqrt(mean(x^2) + eps); pair (a, b) -> scale * (a cos - b sin,
// b cos + a sin).  Memory bound: every element is read and written once, and
// what a token's heads share, its cosines and sines, is computed once per
// workgroup into LDS (rot / 2 angles, reduced in 64 bits) while the first heads'
// loads are in flight.  A workgroup owns one token; a few lanes hold a head, so a norm's
// sum is a butterfly inside a wave.  In the half layout a lane takes 16 bytes
// of the first half and the 16 bytes that they are paired with, so nothing is
// read twice and nothing changes lanes.
//
// Measured: 4096 tokens of 72 fp16 heads with norms 31.0 us (151 MB, 4.9 TB/s, a
// copy's rate), 777 tokens of 112 fp32 heads 18.4 us (89 MB, 4.8 TB/s), one token 2.8
// us.  Partners at any offset are loaded one by one: 4096 tokens, 20 of 128 elements, 43 us.
#include "attn_device.h"

namespace pi {
namespace {

constexpr int kRopeThreads = 1024;
constexpr int kRopeMaxD = 256;

// Workgroups of a call with few tokens split the heads, so that one token is
// not one CU's work alone.
constexpr int kRopeMinGroups = 512;
constexpr int64_t kRopeFill = 256 * 2048;      // threads that the CUs hold

// How a head is laid over lanes.
enum : int {
  kRopeInter,    // interleaved: a chunk of 16 bytes holds whole pairs
  kRopePairs,    // half layout, rot / 2 a multiple of the chunk: a lane has both chunks of its pairs
  kRopeAny       // half layout, partners at any offset: loaded one by one
};

template <typename T, int KIND, bool NORM>
__global__ __launch_bounds__(kRopeThreads) void k_qk_rope(RopeArgs a, int group, int hsplit) {
  constexpr int V = Vec<T>::N;
  constexpr bool kTwo = KIND == kRopePairs;
  __shared__ float2 cs[kRopeMaxD / 2];
  __shared__ float wn[NORM ? 2 * kRopeMaxD : 1];
  const int tok = blockIdx.x / hsplit, part = blockIdx.x % hsplit;
  const int half = a.rot / 2;
  const int per = blockDim.x / group;
  const int lane = threadIdx.x % group;
  // This lane's chunk of each head; rotated pairs' second chunk is half later.
  const int pairs = half / V;
  const int e0 = kTwo && lane >= pairs ? a.rot + (lane - pairs) * V : lane * V;
  const bool in_head = e0 < a.d;
  const bool two = kTwo && lane < pairs;
  const int n_heads = a.in[0].n + a.in[1].n;
  const int step = per * hsplit;

  auto row = [&](const HeadRows* r, int h) {
    const int i = h >= a.in[0].n;
    const HeadRows& x = i ? r[1] : r[0];
    return static_cast<T*>(x.p) + (int64_t)tok * x.ts + (int64_t)(i ? h - a.in[0].n : h) * x.hs;
  };
  // A chunk of the head and, in the half layout, its partners.
  auto load = [&](int h, u32x4& x, u32x4& xp) {
    if (h >= n_heads || !in_head) return;
    const T* p = row(a.in, h);
    x = ld_nt(p + e0);
    if constexpr (KIND == kRopePairs) {
      if (two) xp = ld_nt(p + e0 + half);
    } else if constexpr (KIND == kRopeAny) {
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
  u32x4 x = {0, 0, 0, 0}, xp = {0, 0, 0, 0};
  load(h, x, xp);
  for (int i = threadIdx.x; i < half; i += blockDim.x) {
    double t = (double)a.pos[tok] * a.freqs[i];
    t -= rint(t);
    const float f = (float)t;
    float s, c;
    sincospif(2.f * f, &s, &c);
    // What fp32 leaves of the angle (2^-26 of a turn at most: its square is nothing).
    const float r = (float)((t - (double)f) * 6.283185307179586);
    cs[i] = float2{a.scale * __builtin_fmaf(-s, r, c), a.scale * __builtin_fmaf(c, r, s)};
  }
  if constexpr (NORM) {
    for (int i = threadIdx.x; i < a.d; i += blockDim.x) {
      wn[i] = a.w[0] ? a.w[0][i] : 1.f;
      wn[kRopeMaxD + i] = a.w[1] ? a.w[1][i] : 1.f;
    }
  }
  __syncthreads();
  // The same for every head of this lane.
  float2 t[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int e = e0 + i;
    t[i] = float2{1.f, 0.f};
    if (e < a.rot) t[i] = cs[KIND == kRopeInter ? e / 2 : (e < half ? e : e - half)];
  }

  for (; h - (int)(threadIdx.x / group) < n_heads; h += step) {
    const bool mine = h < n_heads && in_head;
    u32x4 nx = {0, 0, 0, 0}, nxp = {0, 0, 0, 0};
    load(h + step, nx, nxp);
    float y[V], yp[V];
    Vec<T>::unpack(x, y);
    Vec<T>::unpack(xp, yp);
    if constexpr (NORM) {
      float ss = 0.f;
      if (mine) {
#pragma unroll
        for (int i = 0; i < V; ++i) ss = __builtin_fmaf(y[i], y[i], ss);
        if (two) {
#pragma unroll
          for (int i = 0; i < V; ++i) ss = __builtin_fmaf(yp[i], yp[i], ss);
        }
      }
      for (int m = group / 2; m >= 1; m >>= 1) ss += __shfl_xor(ss, m, kWave);
      const int k = h >= a.in[0].n;
      if (mine && a.w[k]) {
        const float r = 1.f / sqrtf(ss / (float)a.d + a.eps);
        const float* w = wn + k * kRopeMaxD;
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const int e = e0 + i;
          y[i] = y[i] * r * w[e];
          if constexpr (KIND != kRopeInter)
            if (e < a.rot) yp[i] = yp[i] * r * w[e < half ? e + half : e - half];
        }
      }
    }
    if (mine) {
      T* p = row(a.out, h) + e0;
      float o[V];
      if constexpr (KIND == kRopeInter) {
#pragma unroll
        for (int i = 0; i < V; i += 2) {
          // (1, 0) past the rotated elements: y * 1 - z * 0 must not make a NaN of an infinite z
          const bool in = e0 + i < a.rot;
          o[i] = in ? __builtin_fmaf(y[i], t[i].x, -(y[i + 1] * t[i].y)) : y[i];
          o[i + 1] = in ? __builtin_fmaf(y[i + 1], t[i].x, y[i] * t[i].y) : y[i + 1];
        }
        *reinterpret_cast<u32x4*>(p) = Vec<T>::pack(o);
      } else if constexpr (KIND == kRopePairs) {
        if (two) {
          float q[V];
#pragma unroll
          for (int i = 0; i < V; ++i) {
            o[i] = __builtin_fmaf(y[i], t[i].x, -(yp[i] * t[i].y));
            q[i] = __builtin_fmaf(yp[i], t[i].x, y[i] * t[i].y);
          }
          *reinterpret_cast<u32x4*>(p) = Vec<T>::pack(o);
          *reinterpret_cast<u32x4*>(p + half) = Vec<T>::pack(q);
        } else {
          *reinterpret_cast<u32x4*>(p) = Vec<T>::pack(y);
        }
      } else {
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const int e = e0 + i;
          const float s = e < half ? -(yp[i] * t[i].y) : yp[i] * t[i].y;
          o[i] = e < a.rot ? __builtin_fmaf(y[i], t[i].x, s) : y[i];
        }
        *reinterpret_cast<u32x4*>(p) = Vec<T>::pack(o);
      }
    }
    x = nx, xp = nxp;
  }
}

int rope_kind(const RopeArgs& a) {
  if (a.layout == PI_ROPE_INTERLEAVED) return kRopeInter;
  return (a.rot / 2) % (a.dtype == PI_F16 ? Vec<f16>::N : Vec<float>::N) ? kRopeAny : kRopePairs;
}

struct RopeGrid {
  int group, threads, hsplit;      // lanes of a head; of a workgroup; workgroups of a token
};
RopeGrid rope_grid(const RopeArgs& a) {
  const int V = a.dtype == PI_F16 ? Vec<f16>::N : Vec<float>::N;
  const int lanes = rope_kind(a) == kRopePairs ? a.rot / 2 / V + (a.d - a.rot) / V : a.d / V;
  RopeGrid g;
  g.group = 1;                                        // a power of two, so that a head stays in a wave
  while (g.group < lanes) g.group *= 2;
  const int n_heads = a.in[0].n + a.in[1].n;
  // A token's heads in passes of one size.  Threads by what fills the card, at
  // least 256: 4096 tokens of 72 fp16 heads 31.9 us with 256 (three passes) and 46.7
  // with 1024 (one); 777 tokens of 112 fp32 heads 23.1 and 18.9.  Very few
  // tokens: a pass to a workgroup of few threads.
  int most = 256;
  while (most < kRopeThreads && (int64_t)a.n_tok * most < kRopeFill) most *= 2;
  while (most > 256 && (int64_t)a.n_tok * (((int64_t)n_heads * g.group + most - 1) / most) < kRopeMinGroups) most /= 2;
  const int passes = (int)(((int64_t)n_heads * g.group + most - 1) / most);
  g.threads = (int)(((int64_t)n_heads * g.group + passes - 1) / passes + kWave - 1) / kWave * kWave;
  const int64_t hsplit = ((int64_t)kRopeMinGroups + a.n_tok - 1) / a.n_tok;
  g.hsplit = (int)(hsplit < passes ? hsplit : passes);
  return g;
}

template <typename T, int KIND>
hipError_t rope_run(const RopeArgs& a, hipStream_t s) {
  const RopeGrid g = rope_grid(a);
  const dim3 grid((unsigned)a.n_tok * g.hsplit);
  if (a.w[0] || a.w[1])
    k_qk_rope<T, KIND, true><<<grid, g.threads, 0, s>>>(a, g.group, g.hsplit);
  else
    k_qk_rope<T, KIND, false><<<grid, g.threads, 0, s>>>(a, g.group, g.hsplit);
  return hipGetLastError();
}

template <typename T>
hipError_t rope_type(const RopeArgs& a, hipStream_t s) {
  switch (rope_kind(a)) {
    case kRopeInter: return rope_run<T, kRopeInter>(a, s);
    case kRopePairs: return rope_run<T, kRopePairs>(a, s);
    default: return rope_run<T, kRopeAny>(a, s);
  }
}

}  // namespace

int64_t qk_rope_threads(const RopeArgs& a) {
  const RopeGrid g = rope_grid(a);
  return (int64_t)a.n_tok * g.hsplit * g.threads;
}

hipError_t launch_qk_rope(const RopeArgs& a, hipStream_t s) {
  return a.dtype == PI_F16 ? rope_type<f16>(a, s) : rope_type<float>(a, s);
}

}  // namespace pi
