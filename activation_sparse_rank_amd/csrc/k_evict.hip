// Eviction from the cache's table by accumulated attention weight
// (pi_kv_evict).
//
// One workgroup per (sequence, kv head).  The keep - recent heaviest of the
// older blocks are found by a radix selection of the weights' order-keeping
// integers (11, 11 and 10 bits: the first digit is sign, exponent and two
// bits of the fraction, so weights with a heavy tail spread over many bins
// and the counters' atomics seldom meet; they count whole numbers, whose sum
// has no order).  Ballots give every block its place.  Latency bound: a table row
// (8 bytes a block in, 8 out) is far less than a CU moves in the time of the
// barriers.
#include "attn_device.h"

namespace pi {
namespace {

constexpr int kEvThreads = 1024;
constexpr int kEvWaves = kEvThreads / kWave;
constexpr int kBins = 2048;

// Larger weight, larger integer; -0 and 0 alike, NaN above all.
__device__ __forceinline__ unsigned order_key(float f) {
  if (f != f) return 0xffffffffu;
  const unsigned b = f == 0.f ? 0u : __builtin_bit_cast(unsigned, f);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}

// VPT > 0: the row's max_blocks <= VPT * kEvThreads slots stay in registers
// from their one read to the writes, so the outputs may be the inputs.
// VPT == 0: longer rows, read again where needed.
template <int VPT>
__global__ __launch_bounds__(kEvThreads) void k_kv_evict(EvictArgs a) {
  constexpr int R = VPT ? VPT : 1;
  __shared__ unsigned hist[kBins];
  __shared__ unsigned wsum[kEvWaves];
  __shared__ unsigned pick[2];
  __shared__ int2 cnt[R * kEvWaves];
  const int s = blockIdx.x / a.hk;
  const int64_t at = (int64_t)blockIdx.x * a.max_blocks;
  const int tid = threadIdx.x, n = a.max_blocks;
  const int chunks = VPT ? VPT : (n + kEvThreads - 1) / kEvThreads;
  const int len = a.lens[s] < 0 ? 0 : a.lens[s];
  const int blocks = (int)(((long long)len + kBlk - 1) / kBlk);
  const int nb = blocks < n ? blocks : n;
  const int gone = nb > a.keep ? nb - a.keep : 0;
  const int old = gone ? nb - a.recent : 0;           // candidates: slots [0, old)
  const int32_t* table = a.table + at;
  const float* score = a.score + at;

  float sc[R];
  int32_t pg[R];
  if constexpr (VPT > 0) {
#pragma unroll
    for (int c = 0; c < R; ++c) {
      const int i = c * kEvThreads + tid;
      if (i < n) sc[c] = score[i], pg[c] = table[i];
    }
  }
  auto score_at = [&](int c, int i) { return VPT ? sc[VPT ? c : 0] : score[i]; };

  // The threshold: the weight of the last block that stays, and how many of
  // the blocks with just this weight stay.
  unsigned bound = 0, left = (unsigned)(old ? a.keep - a.recent : 0);
  if (left) {
    unsigned mask = 0;
#pragma unroll
    for (int d = 0; d < 3; ++d) {
      const int shift = d == 0 ? 21 : (d == 1 ? 10 : 0), bits = d == 2 ? 10 : 11;
      for (int i = tid; i < kBins; i += kEvThreads) hist[i] = 0;
      __syncthreads();
#pragma unroll R
      for (int c = 0; c < chunks; ++c) {
        const int i = c * kEvThreads + tid;
        if (i < old) {
          const unsigned k = order_key(score_at(c, i));
          if ((k & mask) == bound) atomicAdd(&hist[k >> shift & ((1u << bits) - 1)], 1u);
        }
      }
      __syncthreads();
      // Thread t holds the bins 2 t and 2 t + 1 counted from the top.
      const unsigned h0 = hist[kBins - 1 - 2 * tid], h1 = hist[kBins - 2 - 2 * tid];
      unsigned run = h0 + h1;
#pragma unroll
      for (int m = 1; m < kWave; m <<= 1) {
        const unsigned o = (unsigned)__shfl_up((int)run, m, kWave);
        if (lane_id() >= m) run += o;
      }
      if (lane_id() == kWave - 1) wsum[wave_id()] = run;
      __syncthreads();
      unsigned above = run - h0 - h1;
      for (int w = 0; w < wave_id(); ++w) above += wsum[w];
      if (above < left && left <= above + h0 + h1) {
        const bool second = left > above + h0;
        pick[0] = (unsigned)(kBins - 1 - 2 * tid - (second ? 1 : 0));
        pick[1] = left - above - (second ? h0 : 0);
      }
      __syncthreads();
      bound |= pick[0] << shift;
      left = pick[1];
      mask |= ((1u << bits) - 1) << shift;
    }
  }
  const bool none = old && a.keep == a.recent;        // no older block stays

  auto place = [&](int i, float f, int32_t p, bool out, int out_before) {
    const int to = out ? nb - gone + out_before : (i < nb ? i - out_before : i);
    a.table_out[at + to] = p;
    a.score_out[at + to] = out ? 0.f : f;
  };
  const unsigned long long below = (1ull << lane_id()) - 1;
  int more = 0, same = 0;                             // blocks above the threshold, at it, before this chunk
  if constexpr (VPT > 0) {
    unsigned long long bg[R], be[R];
#pragma unroll
    for (int c = 0; c < R; ++c) {
      const int i = c * kEvThreads + tid;
      const unsigned k = i < old && !none ? order_key(sc[c]) : 0;
      bg[c] = __ballot(i < old && !none && k > bound);
      be[c] = __ballot(i < old && !none && k == bound);
      if (lane_id() == 0) cnt[c * kEvWaves + wave_id()] = int2{__popcll(bg[c]), __popcll(be[c])};
    }
    __syncthreads();                                  // also: every slot has been read
    if (wave_id() == 0) {
      // exclusive sums over (chunk, wave), R * 16 entries
      constexpr int E = R * kEvWaves, PER = (E + kWave - 1) / kWave;
      int2 v[PER];
      int2 sum = {0, 0};
#pragma unroll
      for (int k = 0; k < PER; ++k) {
        const int e = lane_id() * PER + k;
        v[k] = e < E ? cnt[e] : int2{0, 0};
        sum.x += v[k].x, sum.y += v[k].y;
      }
      int2 run = sum;
#pragma unroll
      for (int m = 1; m < kWave; m <<= 1) {
        const int ox = __shfl_up(run.x, m, kWave), oy = __shfl_up(run.y, m, kWave);
        if (lane_id() >= m) run.x += ox, run.y += oy;
      }
      int2 pre = {run.x - sum.x, run.y - sum.y};
#pragma unroll
      for (int k = 0; k < PER; ++k) {
        const int e = lane_id() * PER + k;
        if (e < E) cnt[e] = pre;
        pre.x += v[k].x, pre.y += v[k].y;
      }
    }
    __syncthreads();
#pragma unroll
    for (int c = 0; c < R; ++c) {
      const int i = c * kEvThreads + tid;
      if (i >= n) continue;
      const int2 pre = cnt[c * kEvWaves + wave_id()];
      const int eq = pre.y + __popcll(be[c] & below);
      const int stay = pre.x + __popcll(bg[c] & below) + (eq < (int)left ? eq : (int)left);
      const bool kept = (bg[c] >> lane_id() & 1) || ((be[c] >> lane_id() & 1) && eq < (int)left);
      const bool older = i < old;
      place(i, sc[c], pg[c], older && !kept, older ? i - stay : gone);
    }
  } else {
    for (int c = 0; c < chunks; ++c) {
      const int i = c * kEvThreads + tid;
      const bool in = i < n;
      const float f = in ? score[i] : 0.f;
      const int32_t p = in ? table[i] : 0;
      const unsigned k = i < old && !none ? order_key(f) : 0;
      const unsigned long long bg = __ballot(i < old && !none && k > bound);
      const unsigned long long be = __ballot(i < old && !none && k == bound);
      if (lane_id() == 0) cnt[wave_id() % (R * kEvWaves)] = int2{__popcll(bg), __popcll(be)};
      __syncthreads();
      int g = more, e = same;
      for (int w = 0; w < kEvWaves; ++w) {
        const int2 v = cnt[w];
        if (w < wave_id()) g += v.x, e += v.y;
        more += v.x, same += v.y;
      }
      __syncthreads();
      if (in) {
        const int eq = e + __popcll(be & below);
        const int stay = g + __popcll(bg & below) + (eq < (int)left ? eq : (int)left);
        const bool kept = (bg >> lane_id() & 1) || ((be >> lane_id() & 1) && eq < (int)left);
        const bool older = i < old;
        place(i, f, p, older && !kept, older ? i - stay : gone);
      }
    }
  }
  if (blockIdx.x % a.hk == 0 && tid == 0) a.lens_out[s] = len < (long long)n * kBlk ? len - gone * kBlk : (n - gone) * kBlk;
}

}  // namespace

hipError_t launch_kv_evict(const EvictArgs& a, hipStream_t s) {
  const dim3 grid((unsigned)a.n_seqs * a.hk);
  const int v = (a.max_blocks + kEvThreads - 1) / kEvThreads;
  if (v <= 1) k_kv_evict<1><<<grid, kEvThreads, 0, s>>>(a);
  else if (v <= 4) k_kv_evict<4><<<grid, kEvThreads, 0, s>>>(a);
  else if (v <= 8) k_kv_evict<8><<<grid, kEvThreads, 0, s>>>(a);
  else if (v <= PI_KV_EVICT_IN_PLACE / kEvThreads) k_kv_evict<16><<<grid, kEvThreads, 0, s>>>(a);
  else k_kv_evict<0><<<grid, kEvThreads, 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace pi
