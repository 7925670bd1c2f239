// The 8-bit key/value cache: appending rows (pi_kv_append) and reading them
// back (pi_kv_read).
//
// code = 128 + rint(127 x / amax), scale = amax / 127, amax over a block of
// 32 tokens of one head.  Memory bound: a workgroup owns one half (keys or
// values) of one block, holds its rows in registers between the amax and the
// codes, and turns the codes into the page's byte order through LDS, so rows
// are read and pages written in whole 16-byte pieces.
//
// Measured: a token each of 8 sequences 4.9 us and 3.3 to read back (two
// dependent trips to memory: the lengths, then rows or table and page), 2 x
// 2047 tokens of D = 64 7.2 and 5.9 us (12.6 MB each: the trips, then one burst),
// of D = 128 in fp32 11.9 and 9.4 us (42 MB each).
#include "attn_device.h"

namespace pi {
namespace {

// Threads of a workgroup: one for each 16 bytes of a page's half.  (128 for D =
// 64: a prompt's 2080 workgroups run in one round, where 256 threads each left a second one.)
constexpr int kv_threads(int d) { return 2 * d; }

// Blocks that a call of max_new rows can touch in one sequence.
int touched_blocks(int max_new) { return (int)(((long long)max_new + 2 * kBlk - 2) / kBlk); }

// The place of unit u's bytes (16 of a page's half): the token and element of
// byte k.  Keys: 16 elements of one token.  Values: two elements of 8 tokens.
template <int D>
struct Unit {
  __device__ static void key(int u, int& t, int& e) {
    const int rest = u / 64;
    t = rest / (D / 64) * 16 + u % 16;
    e = rest % (D / 64) * 64 + u / 16 % 4 * 16;
  }
  __device__ static void value(int u, int k, int& t, int& e) {
    t = k % 8 / 4 * 16 + u / 16 % 4 * 4 + k % 4;
    e = u / 64 * 32 + k / 8 * 16 + u % 16;
  }
};

// code - 128 = rint(127 x / amax) as a float, by the fp32 quotient; close: it
// lies within 1e-3 of the middle of two codes, where exact_code decides.  x and
// amax are finite, amax > 0; inv = 127 / amax.
__device__ __forceinline__ float quick_code(float x, float inv, bool& close) {
  const float r = x * inv, q = rintf(r);
  close |= __builtin_fabsf(r - q) > 0.499f;
  return q;
}

// 254 |x| against the middle (2 k + 1) amax, both exact in 64 bits; a tie goes to the even code.
__device__ __forceinline__ float exact_code(float x, float amax, float inv) {
  const float r = __builtin_fabsf(x) * inv;
  float q = rintf(r);
  if (__builtin_fabsf(r - q) > 0.499f) {
    const float k = floorf(r);
    const double n = 254.0 * (double)__builtin_fabsf(x), mid = (2.0 * (double)k + 1.0) * (double)amax;
    const bool odd = ((int)k & 1) != 0;
    q = n > mid || (n == mid && odd) ? k + 1.f : k;
  }
  return x < 0.f ? -q : q;
}

template <typename T, int D>
__global__ __launch_bounds__(kv_threads(D)) void k_kv_append(CacheArgs a, int count) {
  constexpr int kKvThreads = kv_threads(D), V = Vec<T>::N, CH = D / V, N = kBlk * CH / kKvThreads;
  constexpr int kRow = D + 16;                      // bytes of an LDS row (16 more: no bank conflicts down a column)
  __shared__ alignas(16) uint8_t codes[kBlk * kRow];
  __shared__ unsigned red[kKvThreads / kWave];
  const int j = blockIdx.x % count;
  const int half = blockIdx.x / count % 2;
  const int pair = blockIdx.x / count / 2;
  const int s = pair / a.hk, h = pair % a.hk;
  const Seq q = read_seq(a.lens, a.q_start, s, a.max_new, a.n_tok, a.max_blocks * kBlk);
  const int before = q.len - q.n;
  if (!q.ok || before < 0 || q.n == 0) return;
  const int first = before / kBlk, blk = first + j, last = (q.len + kBlk - 1) / kBlk;
  if (blk >= last) return;
  const HeadRows& in = half ? a.kv[1] : a.kv[0];
  const T* rows = static_cast<const T*>(in.p) + (int64_t)q.q0 * in.ts + (int64_t)h * in.hs;
  T* open = static_cast<T*>(a.open) + ((int64_t)pair * 2 + half) * (kBlk * D);
  const int page = a.table[(int64_t)pair * a.max_blocks + blk];

  float x[N][V];
  unsigned top = 0;                                 // the largest magnitude's bits; above infinity's: a NaN
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int id = i * kKvThreads + threadIdx.x, t = id / CH, e = id % CH * V, tok = blk * kBlk + t;
    u32x4 v = {0, 0, 0, 0};
    if (tok < before) v = ld16(open + t * D + e);
    else if (tok < q.len) v = ld16(rows + (int64_t)(tok - before) * in.ts + e);
    Vec<T>::unpack(v, x[i]);
#pragma unroll
    for (int k = 0; k < V; ++k) {
      const unsigned b = __builtin_bit_cast(unsigned, x[i][k]) & 0x7fffffffu;
      top = top > b ? top : b;
    }
  }
#pragma unroll
  for (int m = 32; m >= 1; m >>= 1) {
    const unsigned o = (unsigned)__shfl_xor((int)top, m, kWave);
    top = top > o ? top : o;
  }
  if (lane_id() == 0) red[wave_id()] = top;
  __syncthreads();
  // Every read of the open rows is done (their values are in registers).
#pragma unroll
  for (int w = 0; w < kKvThreads / kWave; ++w) top = top > red[w] ? top : red[w];
  const bool finite = top < 0x7f800000u;
  const float amax = as_f(top);
  // Below 2^-90 the quotient's inverse would not fit: both are scaled up.
  const float up = amax < 0x1p-90f ? 0x1p100f : 1.f;
  const float inv = 127.f / (amax * up);
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int id = i * kKvThreads + threadIdx.x, t = id / CH, e = id % CH * V;
    float q[V];
    bool close = false;
#pragma unroll
    for (int k = 0; k < V; ++k) q[k] = quick_code(x[i][k] * up, inv, close);
    // (one branch for all the elements: some lane's is close in one chunk of ten)
    if (close) {
#pragma unroll
      for (int k = 0; k < V; ++k) q[k] = exact_code(x[i][k] * up, amax * up, inv);
    }
    unsigned w[V / 4];
#pragma unroll
    for (int k = 0; k < V; ++k) {
      const unsigned c = finite && top != 0 ? (unsigned)(128 + (int)q[k]) : 128u;
      w[k / 4] = k % 4 ? w[k / 4] | c << 8 * (k % 4) : c;
    }
#pragma unroll
    for (int k = 0; k < V / 4; ++k) *reinterpret_cast<unsigned*>(codes + t * kRow + e + 4 * k) = w[k];
  }
  __syncthreads();
  if ((unsigned)page < (unsigned)a.n_pages) {
    const int u = threadIdx.x;
    u32x4 out;
    int t, e;
    if (half == 0) {
      Unit<D>::key(u, t, e);
      out = *reinterpret_cast<const u32x4*>(codes + t * kRow + e);
    } else {
      unsigned w[4] = {0, 0, 0, 0};
#pragma unroll
      for (int k = 0; k < 16; ++k) {
        Unit<D>::value(u, k, t, e);
        w[k / 4] |= (unsigned)codes[t * kRow + e] << 8 * (k % 4);
      }
      out = u32x4{w[0], w[1], w[2], w[3]};
    }
    *reinterpret_cast<u32x4*>(a.pages + ((int64_t)page * 2 + half) * (kBlk * D) + 16 * u) = out;
    if (u == 0) a.scales[(int64_t)page * 2 + half] = finite ? (float)((double)amax / 127.0) : quiet_nan();
  }
  // The new rows of the block that stays open.  The workgroup of the first
  // block writes them: it alone has read the open rows.
  if (j == 0) {
    const int filled = q.len % kBlk, from = q.len - filled > before ? q.len - filled : before;
    for (int id = threadIdx.x; id < (q.len - from) * CH; id += kKvThreads) {
      const int tok = from + id / CH, e = id % CH * V;
      *reinterpret_cast<u32x4*>(open + tok % kBlk * D + e) = ld16(rows + (int64_t)(tok - before) * in.ts + e);
    }
  }
}

template <typename T, int D>
__global__ __launch_bounds__(kv_threads(D)) void k_kv_read(CacheArgs a, int count) {
  constexpr int kKvThreads = kv_threads(D), V = Vec<T>::N, CH = D / V;
  constexpr int kRow = D + 16;
  __shared__ alignas(16) uint8_t codes[kBlk * kRow];
  const int j = blockIdx.x % count;
  const int half = blockIdx.x / count % 2;
  const int pair = blockIdx.x / count / 2;
  const int s = pair / a.hk, h = pair % a.hk;
  const Seq q = read_seq(a.lens, a.q_start, s, a.max_new, a.n_tok, a.max_blocks * kBlk);
  const HeadRows& to = half ? a.kv[1] : a.kv[0];
  T* rows = static_cast<T*>(to.p) + (int64_t)q.q0 * to.ts + (int64_t)h * to.hs;
  const int before = q.len - q.n;
  if (!q.ok || before < 0) {
    float f[V];
#pragma unroll
    for (int k = 0; k < V; ++k) f[k] = quiet_nan();
    for (int64_t id = (int64_t)j * kKvThreads + threadIdx.x; id < (int64_t)q.n * CH; id += (int64_t)count * kKvThreads)
      *reinterpret_cast<u32x4*>(rows + id / CH * to.ts + id % CH * V) = Vec<T>::pack(f);
    return;
  }
  const int blk = before / kBlk + j;
  if (q.n == 0 || blk * kBlk >= q.len) return;
  const int page = a.table[(int64_t)pair * a.max_blocks + blk];
  const bool good = (unsigned)page < (unsigned)a.n_pages;
  const int u = threadIdx.x;
  float scale = quiet_nan();
  if (good) {
    scale = a.scales[(int64_t)page * 2 + half];
    scale = scale >= 0.f ? scale : quiet_nan();
    const u32x4 v = ld16(a.pages + ((int64_t)page * 2 + half) * (kBlk * D) + 16 * u);
    int t, e;
    if (half == 0) {
      Unit<D>::key(u, t, e);
      *reinterpret_cast<u32x4*>(codes + t * kRow + e) = v;
    } else {
      const unsigned w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int k = 0; k < 16; ++k) {
        Unit<D>::value(u, k, t, e);
        codes[t * kRow + e] = (uint8_t)(w[k / 4] >> 8 * (k % 4));
      }
    }
  }
  __syncthreads();
  for (int id = threadIdx.x; id < kBlk * CH; id += kKvThreads) {
    const int t = id / CH, e = id % CH * V, tok = blk * kBlk + t;
    if (tok < before || tok >= q.len) continue;
    float f[V];
#pragma unroll
    for (int k = 0; k < V; ++k) f[k] = good ? scale * (float)((int)codes[t * kRow + e + k] - 128) : quiet_nan();
    *reinterpret_cast<u32x4*>(rows + (int64_t)(tok - before) * to.ts + e) = Vec<T>::pack(f);
  }
}

template <typename F>
hipError_t by_type(const CacheArgs& a, F f) {
  if (a.dtype == PI_F16) {
    if (a.d == 64) f(f16(), std::integral_constant<int, 64>());
    else f(f16(), std::integral_constant<int, 128>());
  } else {
    if (a.d == 64) f(float(), std::integral_constant<int, 64>());
    else f(float(), std::integral_constant<int, 128>());
  }
  return hipGetLastError();
}

}  // namespace

int64_t kv_cache_threads(const CacheArgs& a) {
  return (int64_t)a.n_seqs * a.hk * 2 * touched_blocks(a.max_new) * kv_threads(a.d);
}

hipError_t launch_kv_append(const CacheArgs& a, hipStream_t s) {
  const int count = touched_blocks(a.max_new);
  const dim3 grid((unsigned)a.n_seqs * a.hk * 2 * count);
  return by_type(a, [&](auto t, auto d) {
    k_kv_append<decltype(t), decltype(d)::value><<<grid, kv_threads(decltype(d)::value), 0, s>>>(a, count);
  });
}

hipError_t launch_kv_read(const CacheArgs& a, hipStream_t s) {
  const int count = touched_blocks(a.max_new);
  const dim3 grid((unsigned)a.n_seqs * a.hk * 2 * count);
  return by_type(a, [&](auto t, auto d) {
    k_kv_read<decltype(t), decltype(d)::value><<<grid, kv_threads(decltype(d)::value), 0, s>>>(a, count);
  });
}

}  // namespace pi
