// Eviction from the cache's table by accumulated attention weight
// (pi_kv_evict).
//
// One workgroup per (sequence, kv head).  Latency bound: a table row (8 bytes
// a block in, 8 out) is far less than a CU moves in the time of the barriers,
// so the rows take as few of those as they can.
//  - Up to kRankMax blocks (k_kv_evict_short): every block counts the older
//    blocks that go before it, from LDS.
//  - Longer rows (k_kv_evict): the weights' order-keeping integers, from the
//    least to the largest of them, are counted in 2048 bins (whole numbers,
//    whose sum has no order; weights with a heavy tail are even in their
//    exponents, so the counters' atomics seldom meet).  The blocks of the bin
//    that the threshold falls into, seldom many, are ranked among themselves by
//    counting; where they are many, the bin is cut into 2048 again.
// Ballots then give every block its place.
// Measured: 130 blocks 4.2 us a call, 32 x 8 rows of 4099 blocks 10.4 us (waves wait 60% of
// their time), 8 rows of 9003 blocks 16, of 20003 43 us.
#include "attn_device.h"

namespace pi {
namespace {

constexpr int kEvThreads = 1024;
constexpr int kEvWaves = kEvThreads / kWave;
constexpr int kBins = 2048;
constexpr int kRankMax = 512;         // blocks of a row, and candidates of a bin, that are ranked by counting

// Larger weight, larger integer; -0 and 0 alike, NaN above all.
__device__ __forceinline__ unsigned order_key(float f) {
  if (f != f) return 0xffffffffu;
  const unsigned b = f == 0.f ? 0u : __builtin_bit_cast(unsigned, f);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}

// How many of keys[0 .. n) go before the key k of number i: larger, or equal
// with a lower number.  The wave's lanes have the numbers base .. base + 63 and
// their keys (0 past n); n is a multiple of 4.
__device__ __forceinline__ int rank_of(const unsigned* keys, int n, unsigned k, int i, int base) {
  int r = 0;
  const int hi = base + kWave < n ? base + kWave : n;
#pragma unroll 8
  for (int j = 0; j < base; j += 4) {
    const u32x4 v = *reinterpret_cast<const u32x4*>(keys + j);
    r += (v.x >= k) + (v.y >= k) + (v.z >= k) + (v.w >= k);
  }
#pragma unroll
  for (int j = 0; j < kWave; ++j) {
    const unsigned o = (unsigned)__builtin_amdgcn_readlane((int)k, j);
    r += o > k || (o == k && j < i - base);
  }
#pragma unroll 8
  for (int j = hi; j < n; j += 4) {
    const u32x4 v = *reinterpret_cast<const u32x4*>(keys + j);
    r += (v.x > k) + (v.y > k) + (v.z > k) + (v.w > k);
  }
  return r;
}

// A row's lengths: blocks held, blocks that leave, and the older ones (0 when none leaves).
struct Row {
  int len, nb, gone, old;
};
__device__ __forceinline__ Row read_row(const EvictArgs& a, int s) {
  Row r;
  r.len = a.lens[s] < 0 ? 0 : a.lens[s];
  const int blocks = (int)(((long long)r.len + kBlk - 1) / kBlk);
  r.nb = blocks < a.max_blocks ? blocks : a.max_blocks;
  r.gone = r.nb > a.keep ? r.nb - a.keep : 0;
  r.old = r.gone ? r.nb - a.recent : 0;
  return r;
}
__device__ __forceinline__ void write_len(const EvictArgs& a, int s, const Row& r) {
  const long long most = (long long)a.max_blocks * kBlk;
  a.lens_out[s] = (int)(r.len < most ? r.len : most) - r.gone * kBlk;
}

// Moves slot i: out_before older blocks below it leave (all that leave, past the older ones).
__device__ __forceinline__ void place(const EvictArgs& a, int64_t at, const Row& r, int i, float f, int32_t p, bool out,
                                      int out_before) {
  const int to = out ? r.nb - r.gone + out_before : (i < r.nb ? i - out_before : i);
  a.table_out[at + to] = p;
  a.score_out[at + to] = out ? 0.f : f;
}

__global__ __launch_bounds__(kRankMax) void k_kv_evict_short(EvictArgs a) {
  __shared__ alignas(16) unsigned keys[kRankMax];
  __shared__ int kept[kRankMax / kWave];
  const int64_t at = (int64_t)blockIdx.x * a.max_blocks;
  const int s = blockIdx.x / a.hk, i = threadIdx.x;
  float f = 0.f;
  int32_t p = 0;
  if (i < a.max_blocks) f = a.score[at + i], p = a.table[at + i];
  const Row r = read_row(a, s);
  const bool older = i < r.old;
  const unsigned k = older ? order_key(f) : 0;
  keys[i] = k;                                        // past the older blocks: before none of them
  __syncthreads();                                    // also: every slot has been read
  bool stay = false;
  if (wave_id() * kWave < r.old) {
    // keys past the older blocks are 0 and their numbers higher, so they count for none
    stay = older && rank_of(keys, (r.old + 3) & ~3, k, i, wave_id() * kWave) < a.keep - a.recent;
  }
  const unsigned long long b = __ballot(stay);
  if (lane_id() == 0) kept[wave_id()] = __popcll(b);
  __syncthreads();
  int before = __popcll(b & ((1ull << lane_id()) - 1));
#pragma unroll
  for (int w = 0; w < kRankMax / kWave; ++w) before += w < wave_id() ? kept[w] : 0;
  if (i < a.max_blocks) place(a, at, r, i, f, p, older && !stay, older ? i - before : r.gone);
  if (blockIdx.x % a.hk == 0 && i == 0) write_len(a, s, r);
}

// VPT > 0: the row's max_blocks <= VPT * kEvThreads slots stay in registers
// from their one read to the writes, so the outputs may be the inputs.
// VPT == 0: longer rows, read again where needed.
template <int VPT>
__global__ __launch_bounds__(kEvThreads) void k_kv_evict(EvictArgs a) {
  constexpr int R = VPT ? VPT : 1;
  __shared__ unsigned hist[kBins];
  __shared__ unsigned wsum[kEvWaves];
  __shared__ unsigned pick[3];
  __shared__ int kept[R * kEvWaves];
  __shared__ alignas(16) unsigned ckey[kRankMax];
  __shared__ int cslot[kRankMax];
  __shared__ unsigned found;
  __shared__ uint2 ends[kEvWaves];
  const int s = blockIdx.x / a.hk;
  const int64_t at = (int64_t)blockIdx.x * a.max_blocks;
  const int tid = threadIdx.x, n = a.max_blocks;
  const int chunks = VPT ? VPT : (n + kEvThreads - 1) / kEvThreads;
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
  const Row row = read_row(a, s);
  const int old = row.old;
  auto key_at = [&](int c, int i) { return order_key(VPT ? sc[VPT ? c : 0] : score[i]); };

  // The threshold: a block stays when its (key, number) does not go after the
  // bound's, i.e. key > bound, or key == bound and number <= last.
  unsigned bound = 0;
  int last = -1;
  unsigned left = (unsigned)(old ? a.keep - a.recent : 0);
  const bool none = left == 0;                        // no older block stays (or none leaves)
  if (!none) {
    unsigned least = 0xffffffffu, most = 0;
#pragma unroll R
    for (int c = 0; c < chunks; ++c) {
      const int i = c * kEvThreads + tid;
      if (c * kEvThreads >= old) break;
      if (i < old) {
        const unsigned k = key_at(c, i);
        least = least < k ? least : k, most = most > k ? most : k;
      }
    }
    // least as the complement of the largest complement
    const uint2 e = {~wave_max(~least), wave_max(most)};
    if (lane_id() == kWave - 1) ends[wave_id()] = e;
    for (int i = tid; i < kBins; i += kEvThreads) hist[i] = 0;
    if (tid < kRankMax) ckey[tid] = 0;
    if (tid == 0) found = 0;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kEvWaves; ++w) {
      const uint2 e = ends[w];
      least = least < e.x ? least : e.x, most = most > e.y ? most : e.y;
    }
    // Keys base + [0, 2^bits) are in question, bits - shift <= 11 of them the bin.
    unsigned base = least;
    int bits = most > least ? 32 - __builtin_clz(most - least) : 0;
    for (;;) {
      const int shift = bits > 11 ? bits - 11 : 0;
      auto inside = [&](unsigned k) { return k >= base && (unsigned long long)(k - base) >> bits == 0; };
#pragma unroll R
      for (int c = 0; c < chunks; ++c) {
        const int i = c * kEvThreads + tid;
        if (c * kEvThreads >= old) break;
        if (i < old) {
          const unsigned k = key_at(c, i);
          if (inside(k)) atomicAdd(&hist[(k - base) >> shift], 1u);
        }
      }
      __syncthreads();
      // Thread t holds the bins 2 t and 2 t + 1 counted from the top.
      const unsigned h0 = hist[kBins - 1 - 2 * tid], h1 = hist[kBins - 2 - 2 * tid];
      const unsigned run = wave_scan(h0 + h1);
      if (lane_id() == kWave - 1) wsum[wave_id()] = run;
      __syncthreads();
      unsigned above = run - h0 - h1;
#pragma unroll
      for (int w = 0; w < kEvWaves; ++w) above += w < wave_id() ? wsum[w] : 0;
      if (above < left && left <= above + h0 + h1) {
        const bool second = left > above + h0;
        pick[0] = (unsigned)(kBins - 1 - 2 * tid - (second ? 1 : 0));
        pick[1] = left - above - (second ? h0 : 0);
        pick[2] = second ? h1 : h0;
      }
      __syncthreads();
      base += pick[0] << shift;
      left = pick[1];
      bits = shift;
      const int many = (int)pick[2];
      if (many <= kRankMax) {
        // Rank the bin's blocks: left of them stay.
#pragma unroll R
        for (int c = 0; c < chunks; ++c) {
          const int i = c * kEvThreads + tid;
          if (c * kEvThreads >= old) break;
          if (i < old) {
            const unsigned k = key_at(c, i);
            if (inside(k)) {
              const unsigned x = atomicAdd(&found, 1u);      // any order: the ranks go by key and number
              ckey[x] = k, cslot[x] = i;
            }
          }
        }
        __syncthreads();
        if (tid < many) {
          const unsigned k = ckey[tid];
          const int i = cslot[tid];
          int over = 0, same = 0;
#pragma unroll 4
          for (int x = 0; x < many; x += 4) {                // keys past the candidates are 0, less than any
            const u32x4 v = *reinterpret_cast<const u32x4*>(ckey + x);
            over += (v.x > k) + (v.y > k) + (v.z > k) + (v.w > k);
            same += (v.x == k) + (v.y == k) + (v.z == k) + (v.w == k);
          }
          int r = over;
          if (same > 1)
            for (int x = 0; x < many; ++x) r += ckey[x] == k && cslot[x] < i;
          if (r == (int)left - 1) pick[0] = k, pick[1] = (unsigned)i;
        }
        __syncthreads();
        bound = pick[0];
        last = (int)pick[1];
        break;
      }
      if (bits == 0) {
        // More than kRankMax blocks with the bound's very key: the left-th of
        // them by number.  Counted chunk after chunk.
        bound = base;
        unsigned before = 0;
        for (int c = 0; c < chunks; ++c) {
          const int i = c * kEvThreads + tid;
          bool eq = false;
          if constexpr (VPT > 0) {
#pragma unroll
            for (int x = 0; x < R; ++x)
              if (x == c) eq = i < old && order_key(sc[x]) == bound;
          } else {
            eq = i < old && order_key(score[i]) == bound;
          }
          const unsigned long long b = __ballot(eq);
          if (lane_id() == 0) wsum[wave_id()] = (unsigned)__popcll(b);
          __syncthreads();
          unsigned mine = before + (unsigned)__popcll(b & ((1ull << lane_id()) - 1));
          for (int w = 0; w < kEvWaves; ++w) {
            if (w < wave_id()) mine += wsum[w];
            before += wsum[w];
          }
          if (eq && mine == left - 1) pick[1] = (unsigned)i;
          __syncthreads();
        }
        last = (int)pick[1];
        break;
      }
      for (int i = tid; i < kBins; i += kEvThreads) hist[i] = 0;
      __syncthreads();
    }
  }
  auto stays = [&](int i, float f) {
    const unsigned k = order_key(f);
    return !none && (k > bound || (k == bound && i <= last));
  };
  const unsigned long long below = (1ull << lane_id()) - 1;
  if constexpr (VPT > 0) {
    unsigned long long b[R];
#pragma unroll
    for (int c = 0; c < R; ++c) {
      const int i = c * kEvThreads + tid;
      b[c] = c * kEvThreads < old ? __ballot(i < old && stays(i, sc[c])) : 0;
      if (lane_id() == 0) kept[c * kEvWaves + wave_id()] = __popcll(b[c]);
    }
    __syncthreads();                                  // also: every slot has been read
    // Every wave sums the counts before each of its chunks: R * 16 entries, lane e has e * PER ...
    constexpr int E = R * kEvWaves, PER = (E + kWave - 1) / kWave;
    int v[PER], sum = 0;
#pragma unroll
    for (int k = 0; k < PER; ++k) {
      const int e = lane_id() * PER + k;
      v[k] = sum;
      sum += e < E ? kept[e] : 0;
    }
    const int run = (int)wave_scan((unsigned)sum) - sum;      // before this lane's entries
#pragma unroll
    for (int c = 0; c < R; ++c) {
      const int i = c * kEvThreads + tid, e = c * kEvWaves + wave_id();
      if (c * kEvThreads >= n) break;
      int pre = 0;
#pragma unroll
      for (int k = 0; k < PER; ++k)
        if (e % PER == k) pre = __builtin_amdgcn_readlane(run + v[k], e / PER);
      if (i >= n) continue;
      const bool older = i < old;
      const int before = pre + __popcll(b[c] & below);
      place(a, at, row, i, sc[c], pg[c], older && !(b[c] >> lane_id() & 1), older ? i - before : row.gone);
    }
  } else {
    int total = 0;                                    // blocks that stay before this chunk
    for (int c = 0; c < chunks; ++c) {
      const int i = c * kEvThreads + tid;
      const float f = i < n ? score[i] : 0.f;
      const unsigned long long b = __ballot(i < old && stays(i, f));
      if (lane_id() == 0) wsum[wave_id()] = (unsigned)__popcll(b);
      __syncthreads();
      int before = total + __popcll(b & below);
      for (int w = 0; w < kEvWaves; ++w) {
        if (w < wave_id()) before += (int)wsum[w];
        total += (int)wsum[w];
      }
      __syncthreads();
      if (i < n) {
        const bool older = i < old;
        place(a, at, row, i, f, table[i], older && !(b >> lane_id() & 1), older ? i - before : row.gone);
      }
    }
  }
  if (blockIdx.x % a.hk == 0 && tid == 0) write_len(a, s, row);
}

}  // namespace

int64_t kv_evict_threads(const EvictArgs& a) {
  return (int64_t)a.n_seqs * a.hk * (a.max_blocks <= kRankMax ? (a.max_blocks + kWave - 1) / kWave * kWave : kEvThreads);
}

hipError_t launch_kv_evict(const EvictArgs& a, hipStream_t s) {
  const dim3 grid((unsigned)a.n_seqs * a.hk);
  const int v = (a.max_blocks + kEvThreads - 1) / kEvThreads;
  if (a.max_blocks <= kRankMax) {
    const int threads = (a.max_blocks + kWave - 1) / kWave * kWave;
    k_kv_evict_short<<<grid, threads, 0, s>>>(a);
  } else if (v <= 4) {
    k_kv_evict<4><<<grid, kEvThreads, 0, s>>>(a);
  } else if (v <= 8) {
    k_kv_evict<8><<<grid, kEvThreads, 0, s>>>(a);
  } else if (v <= PI_KV_EVICT_IN_PLACE / kEvThreads) {
    k_kv_evict<16><<<grid, kEvThreads, 0, s>>>(a);
  } else {
    k_kv_evict<0><<<grid, kEvThreads, 0, s>>>(a);
  }
  return hipGetLastError();
}

}  // namespace pi
