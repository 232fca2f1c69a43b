// Mean keys of key blocks (svg_block_mean) and, for every query, the blocks
// with the largest score (svg_block_select).
//
//   mean[j] = sum of the block's keys / their number      (fp64 sum, one rounding)
//   score(n, j) = (sum over the group's heads of q[n]) . mean[j]
//
// The selection is an integer result, so it is the one that exact scores give,
// ties going to the lower block: scores are formed in fp32 with a known error
// bound e, and the candidates within 2e of the last place are compared again
// in fp64 (products of bf16 sums and fp32 means are exact there).  With t the
// approximate score in the last place, the exact one v satisfies |v - t| <= e,
// so a candidate above t + 2e is in, one below t - 2e is out.
#pragma once

#include "common.cuh"
#include "mma.cuh"
#include "rope.cuh"

namespace svg {

constexpr int kMaxBlocks = 4096;       // blocks of one sequence
constexpr int kMaxBlockTopk = 1024;

// Keys of a sequence: its entry of kv_len, kept inside the buffer.
__device__ __forceinline__ int seq_len(const int32_t *kv_len, int b, int Nk) {
  return kv_len ? min(max(kv_len[b], 0), Nk) : Nk;
}

// bf16 to fp64 at the two halves of a word.  The low one goes through the
// conversion unit, which would take as long as the memory for all; the high one
// is put together by integer operations: its bits, moved to a double's sign,
// exponent and mantissa, are the value times 2^-896 (subnormals included, but
// not infinities and NaN).
__device__ __forceinline__ double low_bf16(uint32_t x) { return static_cast<double>(__uint_as_float(x << 16)); }
__device__ __forceinline__ double high_bf16_scaled(uint32_t x) {
  return __hiloint2double(static_cast<int>(((x & 0x7FFF0000u) >> 3) | (x & 0x80000000u)), 0);
}

// One warp per block: D/8 lanes hold the 16-byte columns of a row, the warp 2
// (D = 64: 4) rows at a time with 8 loads in flight, so that neither shared
// memory nor a barrier is needed.  HBM bound: reads the keys once (40 heads x
// 32,760 keys x D = 128: 64 us, 5.4 TB/s).
constexpr int kMeanThreads = 128;

template <int D>
__global__ void __launch_bounds__(kMeanThreads) block_mean_kernel(const __nv_bfloat16 *k, int Nk, int block, int nblk,
                                                                  const int32_t *kv_len, int heads_per_seq, int fresh,
                                                                  int per_head, int blocks, float *mean) {
  constexpr int COLS = D / 8, SLOTS = 32 / COLS, U = 8;
  const int i = blockIdx.x * (kMeanThreads / 32) + warp_id();
  if (i >= blocks) return;
  const int head = i / per_head;
  const int len = seq_len(kv_len, head / heads_per_seq, Nk);
  const int blk = i % per_head + (fresh > 0 ? max(0, len - fresh) / block : 0);
  if (blk >= nblk) return;
  const int rows = min(max(len - blk * block, 0), block);
  if (fresh > 0 && rows == 0) return;
  const int col = lane_id() % COLS, slot = lane_id() / COLS;
  const __nv_bfloat16 *src = k + (static_cast<int64_t>(head) * Nk + static_cast<int64_t>(blk) * block) * D + 8 * col;
  double acc[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) acc[e] = 0.0;
  uint32_t big = 0;
  for (int r0 = 0; r0 < rows; r0 += U * SLOTS) {
    uint4 v[U];
#pragma unroll
    for (int u = 0; u < U; ++u)        // without conditions, so that all are in flight
      v[u] = __ldg(reinterpret_cast<const uint4 *>(src + static_cast<int64_t>(min(r0 + u * SLOTS + slot, rows - 1)) * D));
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const bool in = r0 + u * SLOTS + slot < rows;
      const uint32_t w[4] = {in ? v[u].x : 0u, in ? v[u].y : 0u, in ? v[u].z : 0u, in ? v[u].w : 0u};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        acc[2 * e] += low_bf16(w[e]);
        acc[2 * e + 1] += high_bf16_scaled(w[e]);
        big = max(big, w[e] & 0x7FFFFFFFu);
      }
    }
  }
  if (__any_sync(0xffffffffu, big >= 0x7F800000u)) {       // infinities or NaN: the high halves again
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[2 * e + 1] = 0.0;
    for (int r = slot; r < rows; r += SLOTS) {
      const uint4 x = __ldg(reinterpret_cast<const uint4 *>(src + static_cast<int64_t>(r) * D));
      const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[2 * e + 1] += static_cast<double>(__uint_as_float(w[e] & 0xFFFF0000u));
    }
  } else {
    const double unscale = __hiloint2double((1023 + 896) << 20, 0);
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[2 * e + 1] *= unscale;
  }
#pragma unroll
  for (int o = COLS; o < 32; o <<= 1)
#pragma unroll
    for (int e = 0; e < 8; ++e) acc[e] += __shfl_xor_sync(0xffffffffu, acc[e], o);
  if (slot == 0) {
    float f[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] = rows > 0 ? static_cast<float>(acc[e] / static_cast<double>(rows)) : 0.f;
    float4 *dst = reinterpret_cast<float4 *>(mean + (static_cast<int64_t>(head) * nblk + blk) * D + 8 * col);
    dst[0] = make_float4(f[0], f[1], f[2], f[3]);
    dst[1] = make_float4(f[4], f[5], f[6], f[7]);
  }
}

struct SelectArgs {
  const __nv_bfloat16 *q;              // [BHk * G, Nq, D]
  const float *mean;                   // [BHk, nblk, D]
  const int32_t *kv_len;
  int32_t *sel;                        // [BHk, Nq, topk]
  // many queries only (workspace):
  __nv_bfloat16 *mean_hi, *mean_lo;    // [BHk, nblk up to whole tiles, D]: the means' bf16 parts
  float *tile_norm;                    // [BHk, tiles] largest |mean|^2 of a tile
  float *scores;                       // [items of a part][64][nblk up to whole tiles]
  float *bounds;                       // [items of a part][64] error bound of a row's scores
  double *exact;                       // per warp of the picking kernel [nblk]
  int item0, items;                    // the part's first item, and how many
  int BHk, G, heads_per_seq, Nq, Nk, nblk, block, topk, sink, local, causal;
};

// Order-preserving integers: larger value, larger key; NaN counts as -inf.
__device__ __forceinline__ uint32_t key32(float f) {
  if (f != f) f = -INFINITY;
  const uint32_t u = __float_as_uint(f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ float unkey32(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? (k & 0x7FFFFFFFu) : ~k);
}
__device__ __forceinline__ uint64_t key64(double d) {
  if (d != d) d = -INFINITY;
  if (d == 0.0) d = 0.0;               // -0 and +0 are a tie
  const uint64_t u = static_cast<uint64_t>(__double_as_longlong(d));
  return (u >> 63) ? ~u : (u | (1ull << 63));
}

// What a query may select: blocks [0, may), of which [0, s1) and [l0, l1) are forced.
struct SelectRange {
  int may, s1, l0, l1;
  __device__ __forceinline__ bool forced(int j) const { return j < s1 || (j >= l0 && j < l1); }
  __device__ __forceinline__ int num_forced() const { return s1 + max(0, l1 - max(l0, s1)); }
};
__device__ __forceinline__ SelectRange select_range(const SelectArgs &a, int len, int n) {
  const int pos = len - a.Nq + n;
  const int seen = a.causal ? min(pos + 1, len) : len;
  SelectRange r;
  r.may = seen <= 0 ? 0 : (seen - 1) / a.block + 1;
  r.s1 = min(a.sink, r.may);
  r.l1 = pos < 0 ? 0 : min(pos / a.block + 1, r.may);
  r.l0 = max(0, r.l1 - a.local);
  return r;
}

// Exact score of block j: the lane's share, from its channels of the summed
// query, and the whole (every lane returns it).
template <int D>
__device__ __forceinline__ double exact_part(const SelectArgs &a, const double (&qs)[D / 32], int head, int j) {
  const float2 *m = reinterpret_cast<const float2 *>(a.mean + (static_cast<int64_t>(head) * a.nblk + j) * D +
                                                     lane_id() * (D / 32));
  double s = 0.0;
#pragma unroll
  for (int i = 0; i < D / 64; ++i) {
    const float2 v = __ldg(m + i);
    s += qs[2 * i] * static_cast<double>(v.x) + qs[2 * i + 1] * static_cast<double>(v.y);
  }
  return s;
}
template <int D>
__device__ __forceinline__ double exact_score(const SelectArgs &a, const double (&qs)[D / 32], int head, int j) {
  double s = exact_part<D>(a, qs, head, j);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  return s;
}
template <int D>
__device__ __forceinline__ void exact_query(const SelectArgs &a, double (&qs)[D / 32], int head, int n) {
  const __nv_bfloat16 *src = a.q + (static_cast<int64_t>(head) * a.G * a.Nq + n) * D + lane_id() * (D / 32);
#pragma unroll
  for (int i = 0; i < D / 32; ++i) qs[i] = 0.0;
  for (int g0 = 0; g0 < a.G; g0 += 4) {             // 4 loads in flight
    uint32_t x[4][D / 64];
#pragma unroll
    for (int g = 0; g < 4; ++g)
#pragma unroll
      for (int i = 0; i < D / 64; ++i) {
        x[g][i] = 0;
        if (g0 + g < a.G) x[g][i] = *reinterpret_cast<const uint32_t *>(src + static_cast<int64_t>(g0 + g) * a.Nq * D + 2 * i);
      }
#pragma unroll
    for (int g = 0; g < 4; ++g)
#pragma unroll
      for (int i = 0; i < D / 64; ++i) {
        qs[2 * i] += static_cast<double>(__uint_as_float(x[g][i] << 16));
        qs[2 * i + 1] += static_cast<double>(__uint_as_float(x[g][i] & 0xFFFF0000u));
      }
  }
}

// A thread's share of a squared norm: not below a floor where any value is not
// zero, so that squares which underflow cannot make the error bound too small
// (and a bound of zero means that every score is zero).  NaN stays.
constexpr float kNormFloor = 1e-28f;
template <int E>
__device__ __forceinline__ float norm_part(float sum, const float (&v)[E]) {
  bool none = true;
#pragma unroll
  for (int e = 0; e < E; ++e) none = none && v[e] == 0.f;
  return none ? 0.f : sum < kNormFloor ? kNormFloor : sum;
}

// Largest error of approximate scores, `rel` times the norms' product.  Where
// that product nears fp32's range (or is not a number), scores or their partial
// sums may be infinite or NaN: the bound is infinite, and all are compared
// exactly.
__device__ __forceinline__ float score_bound(float rel, float q_norm, float mean_norm) {
  const float size = q_norm * mean_norm;
  return size <= 3.0e38f ? rel * size : INFINITY;
}

// Where an approximate score stands against the last place's, t: above (in),
// near (to be compared exactly), else out.  Written so that an infinite bound
// or a NaN makes everything near.
__device__ __forceinline__ bool score_above(float f, float t, float bound) { return f > t + 2.f * bound; }
__device__ __forceinline__ bool score_near(float f, float t, float bound) {
  return !score_above(f, t, bound) && !(f < t - 2.f * bound);
}

// Exact scores of the `count` <= 32 near blocks at `near`: bit c of the result
// says that the c-th is among the `need` best (better score, or lower block).
template <int D>
__device__ __noinline__ uint32_t rank_near(const SelectArgs &a, const int *near, int count, int need, int head, int n) {
  const int lane = lane_id();
  double qs[D / 32], v = 0.0;
  exact_query<D>(a, qs, head, n);
  for (int c0 = 0; c0 < count; c0 += 4) {           // 4 at a time, for their latency
    double x[4];
#pragma unroll
    for (int c = 0; c < 4; ++c) x[c] = exact_part<D>(a, qs, head, near[min(c0 + c, count - 1)]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
#pragma unroll
      for (int c = 0; c < 4; ++c) x[c] += __shfl_xor_sync(0xffffffffu, x[c], o);
#pragma unroll
    for (int c = 0; c < 4; ++c)
      if (lane == c0 + c) v = x[c] != x[c] ? -INFINITY : x[c];
  }
  int better = 0;
  for (int c = 0; c < count; ++c) {
    const double x = __shfl_sync(0xffffffffu, v, c);
    better += x > v || (x == v && c < lane);
  }
  return __ballot_sync(0xffffffffu, lane < count && better < need);
}

// One warp writes one query's list, in two ways.  s: approximate scores of the
// blocks [0, r.may); bound: their largest error.  Block j belongs to lane
// j % 32, place j / 32.
//
// The ordinary one keeps the row in registers (VPL places; forced blocks and
// places without one are NaN, which no comparison takes) and finds the last
// place's score from the lanes' largest ones (few places), or by bisection.
// Returns false, with nothing written, for rows that are flat (more than 32
// near the border) or whose scores have no finite bound.
template <int D, int VPL>
__device__ __forceinline__ bool select_row(const SelectArgs &a, const float *s, int *near_list, float bound, int head,
                                           int n, const SelectRange &r) {
  const uint32_t all = 0xffffffffu;
  const int lane = lane_id();
  const uint32_t below = (1u << lane) - 1;
  int32_t *out = a.sel + (static_cast<int64_t>(head) * a.Nq + n) * a.topk;
  if (r.may <= a.topk) {                            // every block
    for (int i = lane; i < a.topk; i += 32) out[i] = i < r.may ? i : -1;
    return true;
  }
  const int need = a.topk - r.num_forced();
  // (with an infinite bound the borders t +- 2 bound could be NaN below)
  if (need == 0 || !(bound < INFINITY)) return false;
  const float none = __int_as_float(0x7FFFFFFF);
  float f[VPL], mine = -INFINITY;
#pragma unroll
  for (int i = 0; i < VPL; ++i) {                   // no branch between them: all loads in flight
    f[i] = none;
    if (i * 32 + lane < r.may) f[i] = s[i * 32 + lane];
  }
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    const int j = i * 32 + lane;
    // NaN counts as -inf
    f[i] = j < r.s1 || (j >= r.l0 && j < r.l1) || j >= r.may ? none : fmaxf(f[i], -INFINITY);
    mine = fmaxf(mine, f[i]);
  }
  // the lanes' largest scores in descending order
  float best = mine;
#pragma unroll
  for (int k = 2; k <= 32; k <<= 1)
#pragma unroll
    for (int o = k >> 1; o > 0; o >>= 1) {
      const float x = __shfl_xor_sync(all, best, o);
      best = ((lane & k) == 0) == ((lane & o) == 0) ? fmaxf(best, x) : fminf(best, x);
    }
  const float top = __shfl_sync(all, best, 0);
  // The need-th of them is a lower bound of the last place's score, and close
  // while places are few beside lanes: a few steps up, from one score to the
  // next, reach it.  Steps / bisection, us for 16,384 queries, 5 / 1, 8 key heads:
  // 512 blocks: 5 places 373 / 416, 13 457 / 463, 17 526 / 481, 29 623 / 508; 1,500
  // blocks: 5 places 1,259 / 1,449, 11 1,560 / 1,575, 13 1,740 / 1,611, 29 2,315 / 1,837.
  constexpr int FEW = VPL <= 16 ? 13 : 11;
  float t = __shfl_sync(all, best, min(need, 32) - 1);
  bool found = false;
  if (need <= FEW && t > -INFINITY)
    for (int round = 0; round < 8; ++round) {
      float c0 = 0.f, c1 = 0.f, next = INFINITY;
#pragma unroll
      for (int i = 0; i < VPL; i += 2) {
        if (VPL > 16 && i % 16 == 0 && i * 32 >= r.may) break;
        c0 += f[i] > t ? 1.f : 0.f;                 // a comparison yields 1.0f in one instruction
        c1 += f[i + 1] > t ? 1.f : 0.f;
        next = fminf(next, fminf(f[i] > t ? f[i] : INFINITY, f[i + 1] > t ? f[i + 1] : INFINITY));
      }
      found = __reduce_add_sync(all, static_cast<int>(c0 + c1)) < need;
      if (found) break;
      t = unkey32(__reduce_min_sync(all, key32(next)));
    }
  if (!found) {
    // bisection between lo (at least `need` are not below it) and hi (one is not, unless equal)
    float lo = INFINITY, hi = top;
#pragma unroll
    for (int i = 0; i < VPL; ++i) lo = fminf(lo, f[i]);
    lo = unkey32(__reduce_min_sync(all, key32(lo)));
    if (!(hi - lo < 3.0e38f)) return false;
    float mid = hi;
    while (true) {
      float c0 = 0.f, c1 = 0.f;
#pragma unroll
      for (int i = 0; i < VPL; i += 2) {
        if (VPL > 16 && i % 16 == 0 && i * 32 >= r.may) break;
        c0 += f[i] >= mid ? 1.f : 0.f;
        c1 += f[i + 1] >= mid ? 1.f : 0.f;
      }
      const int c = __reduce_add_sync(all, static_cast<int>(c0 + c1));
      if (c >= need) lo = mid;
      else hi = mid;
      if (c == need) break;
      mid = lo + 0.5f * (hi - lo);
      if (!(mid > lo && mid < hi)) break;           // equal, or neighbours: equal scores
    }
    float least = INFINITY;
#pragma unroll
    for (int i = 0; i < VPL; ++i)
      if (f[i] >= lo) least = fminf(least, f[i]);
    t = unkey32(__reduce_min_sync(all, key32(least)));
  }
  // who is near the last place's score, t, or above: bit i of a lane's words
  const float over = t + 2.f * bound, under = t - 2.f * bound;
  constexpr int WORDS = (VPL + 31) / 32;
  uint32_t cand[WORDS], sure_bits[WORDS];
  int both = 0;                                     // near ones above 2^16, above ones below
#pragma unroll
  for (int w = 0; w < WORDS; ++w) {
    cand[w] = sure_bits[w] = 0;
#pragma unroll
    for (int i = 32 * w; i < min(VPL, 32 * w + 32); ++i) {
      cand[w] |= f[i] >= under ? 1u << (i & 31) : 0u;
      sure_bits[w] |= f[i] > over ? 1u << (i & 31) : 0u;
    }
    both += __popc(sure_bits[w]) + (__popc(cand[w] & ~sure_bits[w]) << 16);
  }
  both = __reduce_add_sync(all, both);
  const int sure = both & 0xFFFF, nears = both >> 16;
  uint32_t stay = all;
  if (nears > need - sure) {
    if (nears > 32) return false;
    int at = 0;
#pragma unroll
    for (int w = 0; w < WORDS; ++w) {
      const uint32_t near = cand[w] & ~sure_bits[w];
      for (uint32_t places = __reduce_or_sync(all, near); places; places &= places - 1) {
        const int i = __ffs(places) - 1;
        const uint32_t m = __ballot_sync(all, (near >> i) & 1u);
        if ((near >> i) & 1u) near_list[at + __popc(m & below)] = (32 * w + i) * 32 + lane;
        at += __popc(m);
      }
    }
    __syncwarp();
    stay = rank_near<D>(a, near_list, nears, need - sure, head, n);
  }
  int seen = 0, at = 0, low = 0;
  const int l0 = max(r.l0, r.s1);
#pragma unroll
  for (int w = 0; w < WORDS; ++w)
    for (uint32_t places = __reduce_or_sync(all, cand[w]); places; places &= places - 1) {
      const int i = __ffs(places) - 1, j = (32 * w + i) * 32 + lane;
      const bool is = (cand[w] >> i) & 1u, near = is && !((sure_bits[w] >> i) & 1u);
      const uint32_t nm = __ballot_sync(all, near);
      const bool in = is && (!near || ((stay >> ((seen + __popc(nm & below)) & 31)) & 1u));
      const uint32_t m = __ballot_sync(all, in);
      seen += __popc(nm);
      // before it: forced blocks below it and kept ones
      if (in) out[at + __popc(m & below) + r.s1 + max(0, min(j, r.l1) - l0)] = j;
      at += __popc(m);
      if ((32 * w + i) * 32 < l0) low += __popc(__ballot_sync(all, in && j < l0));
    }
  for (int i = lane; i < r.s1; i += 32) out[i] = i;
  for (int i = l0 + lane; i < r.l1; i += 32) out[low + r.s1 + i - l0] = i;
  return true;
}

// The general one reads the scores again for every step; exact: scratch of
// nblk doubles.
template <int D>
__device__ __noinline__ void select_row_any(const SelectArgs &a, const float *s, double *exact, float bound, int head,
                                            int n, const SelectRange r) {
  const int lane = lane_id();
  int32_t *out = a.sel + (static_cast<int64_t>(head) * a.Nq + n) * a.topk;
  const int places = (r.may + 31) / 32;
  int need = a.topk - r.num_forced();               // fewer than the others: see select_row
  auto key = [&](int i) {
    const int j = i * 32 + lane;
    return j < r.may && !r.forced(j) ? key32(s[j]) : 0u;
  };
  uint32_t cut = 0;
  for (int bit = 31; bit >= 0 && need > 0; --bit) {
    const uint32_t trial = cut | (1u << bit);
    int c = 0;
    for (int i = 0; i < places; ++i) c += key(i) >= trial;
    c = __reduce_add_sync(0xffffffffu, c);
    if (c >= need) cut = trial;
    if (c == need) break;
  }
  uint32_t least = 0xFFFFFFFFu;
  for (int i = 0; i < places; ++i) {
    const uint32_t k = key(i);
    if (k >= cut && k != 0) least = min(least, k);
  }
  least = __reduce_min_sync(0xffffffffu, least);
  const float t = unkey32(least);
  int sure = 0, near = 0;
  for (int i = 0; i < places && need > 0; ++i) {
    const uint32_t k = key(i);
    if (k != 0) {
      sure += score_above(unkey32(k), t, bound);
      near += score_near(unkey32(k), t, bound);
    }
  }
  sure = __reduce_add_sync(0xffffffffu, sure);
  near = __reduce_add_sync(0xffffffffu, near);
  need -= sure;
  // exact values where there are more near ones than places; a bound of zero
  // means scores of zero: all tie
  uint64_t cut64 = 0;
  int ties = need;
  const bool rank = near > need && bound > 0.f;
  if (rank) {
    double qs[D / 32];
    exact_query<D>(a, qs, head, n);
    for (int i = 0; i < places; ++i) {
      const uint32_t k = key(i);
      for (uint32_t m = __ballot_sync(0xffffffffu, k != 0 && score_near(unkey32(k), t, bound)); m; m &= m - 1) {
        const int l = __ffs(m) - 1;
        const double x = exact_score<D>(a, qs, head, i * 32 + l);
        if (lane == l) exact[i * 32 + l] = x;       // each lane reads only its own
      }
    }
    auto exact_key = [&](int i) {
      const uint32_t k = key(i);
      return k != 0 && score_near(unkey32(k), t, bound) ? key64(exact[i * 32 + lane]) : 0ull;
    };
    for (int b = 63; b >= 0; --b) {
      const uint64_t trial = cut64 | (1ull << b);
      int c = 0;
      for (int i = 0; i < places; ++i) c += exact_key(i) >= trial;
      if (__reduce_add_sync(0xffffffffu, c) >= need) cut64 = trial;
    }
    int better = 0;
    for (int i = 0; i < places; ++i) better += exact_key(i) > cut64;
    ties = need - __reduce_add_sync(0xffffffffu, better);
  }
  int at = 0;
  for (int i = 0; i < places; ++i) {
    const int j = i * 32 + lane;
    const uint32_t k = key(i);
    const float f = unkey32(k);
    bool keep = j < r.may && r.forced(j), tie = false;
    if (k != 0 && a.topk > r.num_forced()) {
      keep = score_above(f, t, bound);
      if (!keep && score_near(f, t, bound)) {
        const uint64_t x = rank ? key64(exact[j]) : 0ull;
        keep = rank && x > cut64;
        tie = !rank || x == cut64;
      }
    }
    const uint32_t tied = __ballot_sync(0xffffffffu, tie);
    if (tie) keep = __popc(tied & ((1u << lane) - 1)) < ties;
    ties -= min(ties, __popc(tied));
    const uint32_t m = __ballot_sync(0xffffffffu, keep);
    if (keep) out[at + __popc(m & ((1u << lane) - 1))] = j;
    at += __popc(m);
  }
  for (int i = at + lane; i < a.topk; i += 32) out[i] = -1;
}

// Many queries: one CTA takes 64 queries of a key head and all their blocks.
// Scores run on the tensor cores with the summed queries and the means split
// into bf16 high and low parts: each low part's rounding and the omitted lo lo
// are at most 2^-16 of a product, the roundings of the fp32 sums (24 matrix
// steps) less than 2^-17, so the error is below 2^-14 |q| |mean| (norms of the
// head-wise absolute sum and of the block's mean).  The queries' parts stay in
// registers, the means' stream through two buffers, and the scores go to
// scratch rows.  A second kernel with a warp per row picks; it needs few
// registers, so more warps hide its latencies (one kernel for both took
// 1.17 times as long).  Both run over parts of the queries that bound the scratch.
// 32,760 queries, 5 heads to a key head, 8 x 512 blocks: scores 330 us, picking
// 400 us.  tcgen05 has twice the rate for these products; a kernel that formed
// the head sums of 128 rows in each CTA, as this one does of 64, took 174 us a
// part where this takes 143 (sums formed once beforehand were not tried).
constexpr int kSelTile = 64, kSelThreads = 128;
constexpr float kSelSplitError = 1.f / 16384.f;

template <int D>
constexpr int select_smem() {
  return 4 * kSelTile * D * 2 + kSelTile * 4;
}

__device__ __forceinline__ void split8(const float (&f)[8], uint4 &hi, uint4 &lo) {
  hi = pack8(f);
  float h[8], l[8];
  unpack8(hi, h);
#pragma unroll
  for (int i = 0; i < 8; ++i) l[i] = f[i] - h[i];
  lo = pack8(l);
}

// The means' two parts, zeros behind the last block, and each tile's largest
// norm: one CTA per tile of 64 blocks.
template <int D>
__global__ void __launch_bounds__(256) block_select_split_kernel(const SelectArgs a, int tiles) {
  __shared__ uint32_t mn;
  const int head = blockIdx.x / tiles, tile = blockIdx.x % tiles;
  if (threadIdx.x == 0) mn = 0;
  __syncthreads();
  constexpr int COLS = D / 8;
  for (int i = threadIdx.x; i < kSelTile * COLS; i += 256) {
    const int r = i / COLS, c = i % COLS, j = tile * kSelTile + r;
    float f[8], nn = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] = 0.f;
    if (j < a.nblk) {
      const float4 *src = reinterpret_cast<const float4 *>(a.mean + (static_cast<int64_t>(head) * a.nblk + j) * D + 8 * c);
      const float4 x = __ldg(src), y = __ldg(src + 1);
      f[0] = x.x; f[1] = x.y; f[2] = x.z; f[3] = x.w;
      f[4] = y.x; f[5] = y.y; f[6] = y.z; f[7] = y.w;
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) nn += f[e] * f[e];
    nn = norm_part(nn, f);
    uint4 hi, lo;
    split8(f, hi, lo);
    const int64_t at = (static_cast<int64_t>(head) * tiles * kSelTile + j) * D + 8 * c;
    *reinterpret_cast<uint4 *>(a.mean_hi + at) = hi;
    *reinterpret_cast<uint4 *>(a.mean_lo + at) = lo;
#pragma unroll
    for (int o = COLS / 2; o > 0; o >>= 1) nn += __shfl_xor_sync(0xffffffffu, nn, o);
    // a NaN or infinite mean makes every comparison an exact one; values >= 0 order like integers
    if (c == 0) atomicMax(&mn, nn <= 3.4e38f ? __float_as_uint(nn) : 0x7F800000u);
  }
  __syncthreads();
  if (threadIdx.x == 0) a.tile_norm[blockIdx.x] = __uint_as_float(mn);
}

// An item is a tile of 64 queries of a key head; the last ones come first (long
// causal rows).
struct SelectItem {
  int head, n0, len;
};
__device__ __forceinline__ SelectItem select_item(const SelectArgs &a, int item) {
  const int qtiles = (a.Nq + kSelTile - 1) / kSelTile;
  SelectItem x;
  x.head = item % a.BHk;
  x.n0 = (qtiles - 1 - item / a.BHk) * kSelTile;
  x.len = seq_len(a.kv_len, x.head / a.heads_per_seq, a.Nk);
  return x;
}

template <int D>
__global__ void __launch_bounds__(kSelThreads, 3) block_select_score_kernel(const SelectArgs a) {
  extern __shared__ __align__(1024) uint8_t smem[];
  constexpr int TILE = kSelTile * D * 2, COLS = D / 8;
  float *qn = reinterpret_cast<float *>(smem + 4 * TILE);      // |q| of every row
  const uint32_t base = smem_u32(smem);
  const int warp = warp_id();
  const int tiles = (a.nblk + kSelTile - 1) / kSelTile;
  const int wide = tiles * kSelTile;   // a scratch row
  float *scores = a.scores + static_cast<int64_t>(blockIdx.x) * kSelTile * wide;
  const SelectItem item = select_item(a, a.item0 + blockIdx.x);
  const int head = item.head, n0 = item.n0, len = item.len;
  {
    const int most = select_range(a, len, min(n0 + kSelTile, a.Nq) - 1).may;
    const __nv_bfloat16 *hi = a.mean_hi + static_cast<int64_t>(head) * tiles * kSelTile * D;
    const __nv_bfloat16 *lo = a.mean_lo + static_cast<int64_t>(head) * tiles * kSelTile * D;
    auto fetch = [&](int t) {          // tile t of the means' parts
      if (t * kSelTile < most) {
        const uint32_t dst = base + static_cast<uint32_t>(t & 1) * 2 * TILE;
        for (int i = threadIdx.x; i < kSelTile * COLS; i += kSelThreads) {
          const int r = i / COLS, c = i % COLS;
          const int64_t at = (static_cast<int64_t>(t) * kSelTile + r) * D + 8 * c;
          cp_async16(dst + tile_at<D>(r, c), hi + at, 16);
          cp_async16(dst + TILE + tile_at<D>(r, c), lo + at, 16);
        }
      }
      cp_async_commit();
    };
    fetch(0);
    // queries: sum over heads, split, by way of the second buffer into registers
    for (int i = threadIdx.x; i < kSelTile * COLS; i += kSelThreads) {
      const int r = i / COLS, c = i % COLS;
      float f[8], ab = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] = 0.f;
      if (n0 + r < a.Nq) {
        float w[8], z[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) z[e] = 0.f;
        const __nv_bfloat16 *src = a.q + (static_cast<int64_t>(head) * a.G * a.Nq + n0 + r) * D + 8 * c;
        for (int g0 = 0; g0 < a.G; g0 += 8) {       // 8 loads in flight
          uint4 x[8];
#pragma unroll
          for (int g = 0; g < 8; ++g)
            x[g] = g0 + g < a.G ? __ldg(reinterpret_cast<const uint4 *>(src + static_cast<int64_t>(g0 + g) * a.Nq * D))
                                : make_uint4(0, 0, 0, 0);
#pragma unroll
          for (int g = 0; g < 8; ++g) {
            if (g0 + g >= a.G) break;
            unpack8(x[g], w);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              f[e] += w[e];
              z[e] += fabsf(w[e]);
            }
          }
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) ab += z[e] * z[e];
        ab = norm_part(ab, z);
      }
      uint4 h, l;
      split8(f, h, l);
      *reinterpret_cast<uint4 *>(smem + 2 * TILE + tile_at<D>(r, c)) = h;
      *reinterpret_cast<uint4 *>(smem + 3 * TILE + tile_at<D>(r, c)) = l;
#pragma unroll
      for (int o = COLS / 2; o > 0; o >>= 1) ab += __shfl_xor_sync(0xffffffffu, ab, o);
      if (c == 0) qn[r] = sqrtf(ab);
    }
    __syncthreads();
    uint32_t ah[D / 16][4], al[D / 16][4];
#pragma unroll
    for (int ks = 0; ks < D / 16; ++ks) {
      ldsm_x4(piece<D>(lane_a<D>(base + 2 * TILE), 16 * warp, ks), ah[ks]);
      ldsm_x4(piece<D>(lane_a<D>(base + 3 * TILE), 16 * warp, ks), al[ks]);
    }
    __syncthreads();
    float norm = 0.f;
    for (int tile = 0; tile * kSelTile < most; ++tile) {
      const int j0 = tile * kSelTile;
      norm = fmaxf(norm, a.tile_norm[head * tiles + tile]);
      fetch(tile + 1);
      cp_async_wait<1>();
      __syncthreads();
      const uint32_t m_hi = lane_b<D>(base + static_cast<uint32_t>(tile & 1) * 2 * TILE), m_lo = m_hi + TILE;
      float acc[8][4];
#pragma unroll
      for (int t = 0; t < 8; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[t][e] = 0.f;
#pragma unroll
      for (int ks = 0; ks < D / 16; ++ks) {
        // eight independent sums between two steps of one
        uint32_t bh[4][4], bl[4][4];
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          ldsm_x4(piece<D>(m_hi, 16 * t, ks), bh[t]);
          ldsm_x4(piece<D>(m_lo, 16 * t, ks), bl[t]);
        }
#pragma unroll
        for (int t = 0; t < 8; ++t) mma_bf16(acc[t], al[ks], bh[t / 2][2 * (t & 1)], bh[t / 2][2 * (t & 1) + 1]);
#pragma unroll
        for (int t = 0; t < 8; ++t) mma_bf16(acc[t], ah[ks], bl[t / 2][2 * (t & 1)], bl[t / 2][2 * (t & 1) + 1]);
#pragma unroll
        for (int t = 0; t < 8; ++t) mma_bf16(acc[t], ah[ks], bh[t / 2][2 * (t & 1)], bh[t / 2][2 * (t & 1) + 1]);
      }
      float *row = scores + static_cast<int64_t>(16 * warp + frag_row()) * wide + j0 + frag_col();
#pragma unroll
      for (int t = 0; t < 8; ++t) {
        *reinterpret_cast<float2 *>(row + 8 * t) = make_float2(acc[t][0], acc[t][1]);
        *reinterpret_cast<float2 *>(row + 8 * wide + 8 * t) = make_float2(acc[t][2], acc[t][3]);
      }
      __syncthreads();
    }
    if (threadIdx.x < kSelTile) {
      a.bounds[blockIdx.x * kSelTile + threadIdx.x] = score_bound(kSelSplitError, qn[threadIdx.x], sqrtf(norm));
    }
  }
}

// Picks: a warp per row, `gridDim.x` CTAs in turn over the part's rows.
template <int D, int VPL>
__global__ void __launch_bounds__(kSelThreads, VPL <= 16 ? 6 : VPL <= 32 ? 5 : 3) block_select_pick_kernel(const SelectArgs a) {
  constexpr int WARPS = kSelThreads / 32;
  __shared__ int near[WARPS][32];
  const int wide = (a.nblk + kSelTile - 1) / kSelTile * kSelTile, warp = warp_id();
  double *exact = a.exact + (static_cast<int64_t>(blockIdx.x) * WARPS + warp) * a.nblk;
  const int rows = a.items * kSelTile;
  for (int row = blockIdx.x * WARPS + warp; row < rows; row += gridDim.x * WARPS) {
    const SelectItem item = select_item(a, a.item0 + row / kSelTile);
    const int n = item.n0 + row % kSelTile;
    if (n >= a.Nq) continue;
    const SelectRange range = select_range(a, item.len, n);
    const float *s = a.scores + static_cast<int64_t>(row) * wide;
    const float bound = a.bounds[row];
    if (!select_row<D, VPL>(a, s, near[warp], bound, item.head, n, range))
      select_row_any<D>(a, s, exact, bound, item.head, n, range);
    __syncwarp();
  }
}

// Few queries: one CTA per (key head, query).  8 lanes (D = 64: 4) form one
// score in fp32; 16 products, two levels of sums: error below 2^-18 |q| |mean|.
// HBM bound: reads the means once.  All threads search the border together.
// 16 sequences x 8 heads, up to 2,048 blocks: 26 us, of which the search takes 6.
constexpr int kSelDecodeThreads = 512;
constexpr float kSelDotError = 1.f / 262144.f;
constexpr int kSelDecodePlaces = kMaxBlocks / kSelDecodeThreads;

// Shared memory: exact scores, their blocks, approximate scores, kept blocks.
__host__ __device__ inline size_t select_decode_smem(int nblk) {
  return static_cast<size_t>(nblk) * 16 + (nblk + 31) / 32 * 4 + 4;
}

// Sum over the CTA; `turn` alternates between two rows of warp sums.
__device__ __forceinline__ int cta_sum(int v, int (&part)[2][kSelDecodeThreads / 32], int turn) {
  v = __reduce_add_sync(0xffffffffu, v);
  if (lane_id() == 0) part[turn & 1][warp_id()] = v;
  __syncthreads();
  const int x = lane_id() < kSelDecodeThreads / 32 ? part[turn & 1][lane_id()] : 0;
  return __reduce_add_sync(0xffffffffu, x);
}

template <int D>
__global__ void __launch_bounds__(kSelDecodeThreads, 1) block_select_decode_kernel(const SelectArgs a) {
  extern __shared__ __align__(1024) uint8_t smem[];
  double *exact = reinterpret_cast<double *>(smem);               // [nblk]
  float *scores = reinterpret_cast<float *>(exact + a.nblk);      // [nblk]
  int *who = reinterpret_cast<int *>(scores + a.nblk);            // [nblk]
  uint32_t *kept = reinterpret_cast<uint32_t *>(who + a.nblk);    // bit set of the list
  __shared__ uint32_t mn, top, least;
  __shared__ int part[2][kSelDecodeThreads / 32], nears;
  constexpr int GT = D / 16, WARPS = kSelDecodeThreads / 32;
  const int head = blockIdx.x / a.Nq, n = blockIdx.x % a.Nq;
  const int len = seq_len(a.kv_len, head / a.heads_per_seq, a.Nk);
  const SelectRange r = select_range(a, len, n);
  const int c = threadIdx.x % GT;
  if (threadIdx.x == 0) {
    mn = top = 0;
    least = 0xFFFFFFFFu;
    nears = 0;
  }
  for (int i = threadIdx.x; i < (a.nblk + 31) / 32; i += kSelDecodeThreads) kept[i] = 0;
  float qs[16], qa = 0.f;
  {
    float z[16];
#pragma unroll
    for (int e = 0; e < 16; ++e) qs[e] = z[e] = 0.f;
    for (int g = 0; g < a.G; ++g) {
      const uint4 *src = reinterpret_cast<const uint4 *>(
          a.q + ((static_cast<int64_t>(head) * a.G + g) * a.Nq + n) * D);
      float x[8], y[8];
      unpack8(__ldg(src + c), x);
      unpack8(__ldg(src + GT + c), y);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        qs[e] += x[e];
        qs[8 + e] += y[e];
        z[e] += fabsf(x[e]);
        z[8 + e] += fabsf(y[e]);
      }
    }
#pragma unroll
    for (int e = 0; e < 16; ++e) qa += z[e] * z[e];
    qa = row_sum<D>(norm_part(qa, z));
  }
  __syncthreads();
  // A group of GT lanes takes U = GT/2 blocks at a time, which makes GT sums (U
  // scores, U squared norms): they are added over the lanes by halving, so that
  // lane c ends with the c-th sum.
  uint32_t biggest = 0;
  constexpr int PER = kSelDecodeThreads / GT, U = GT / 2;
#pragma unroll 2
  for (int j0 = 0; j0 < r.may; j0 += PER * U) {
    float4 v[U][4];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int j = j0 + u * PER + threadIdx.x / GT;
      const float4 *src = reinterpret_cast<const float4 *>(a.mean + (static_cast<int64_t>(head) * a.nblk + j) * D);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        v[u][e] = make_float4(0, 0, 0, 0);
        if (j < r.may) v[u][e] = __ldg(src + (e < 2 ? 2 * c + e : 2 * GT + 2 * c + e - 2));
      }
    }
    float sum[GT];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      float2 s = make_float2(0.f, 0.f), nn = s;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 lo = make_float2(v[u][e].x, v[u][e].y), hi = make_float2(v[u][e].z, v[u][e].w);
        s = fma_f32x2(lo, make_float2(qs[4 * e], qs[4 * e + 1]), s);
        s = fma_f32x2(hi, make_float2(qs[4 * e + 2], qs[4 * e + 3]), s);
        nn = fma_f32x2(lo, lo, nn);
        nn = fma_f32x2(hi, hi, nn);
      }
      sum[u] = s.x + s.y;
      sum[U + u] = nn.x + nn.y;
    }
#pragma unroll
    for (int half = GT / 2; half > 0; half >>= 1) {
      const bool upper = (c & half) != 0;
#pragma unroll
      for (int i = 0; i < half; ++i) {
        const float give = upper ? sum[i] : sum[half + i], keep = upper ? sum[half + i] : sum[i];
        sum[i] = keep + __shfl_xor_sync(0xffffffffu, give, half);
      }
    }
    const int j = j0 + (c % U) * PER + threadIdx.x / GT;
    if (c < U) {
      if (j < r.may) scores[j] = sum[0];
    } else {
      // not below the floor (see norm_part), and NaN or infinity: all exact
      biggest = max(biggest, sum[0] <= 3.4e38f ? __float_as_uint(fmaxf(sum[0], kNormFloor)) : 0x7F800000u);
    }
  }
  biggest = __reduce_max_sync(0xffffffffu, biggest);
  if (lane_id() == 0) atomicMax(&mn, biggest);
  __syncthreads();
  const float bound = score_bound(kSelDotError, sqrtf(qa), sqrtf(__uint_as_float(mn)));

  // block i * 512 + thread, place i
  const int forced = r.num_forced();
  int need = a.topk - forced;
  uint32_t key[kSelDecodePlaces], mine = 0;
#pragma unroll
  for (int i = 0; i < kSelDecodePlaces; ++i) {
    const int j = i * kSelDecodeThreads + threadIdx.x;
    key[i] = (j < r.may && !r.forced(j)) ? key32(scores[j]) : 0u;
    mine = max(mine, key[i]);
    if (j < r.may && r.forced(j)) atomicOr(&kept[j >> 5], 1u << (j & 31));
  }
  if (r.may - forced <= need) {
#pragma unroll
    for (int i = 0; i < kSelDecodePlaces; ++i) {
      const int j = i * kSelDecodeThreads + threadIdx.x;
      if (key[i] != 0) atomicOr(&kept[j >> 5], 1u << (j & 31));
    }
  } else if (need > 0) {
    mine = __reduce_max_sync(0xffffffffu, mine);
    if (lane_id() == 0) atomicMax(&top, mine);
    __syncthreads();
    int turn = 0;
    uint32_t cut = 0;
    for (int bit = 31 - __clz(top); bit >= 0; --bit) {
      const uint32_t trial = cut | (1u << bit);
      int x = 0;
#pragma unroll
      for (int i = 0; i < kSelDecodePlaces; ++i) x += key[i] >= trial;
      x = cta_sum(x, part, turn++);
      if (x >= need) cut = trial;
      if (x == need) break;
    }
    uint32_t l = 0xFFFFFFFFu;
#pragma unroll
    for (int i = 0; i < kSelDecodePlaces; ++i)
      if (key[i] >= cut && key[i] != 0) l = min(l, key[i]);
    l = __reduce_min_sync(0xffffffffu, l);
    if (lane_id() == 0) atomicMin(&least, l);
    __syncthreads();
    const float t = unkey32(least);
    int sure = 0;
#pragma unroll
    for (int i = 0; i < kSelDecodePlaces; ++i) {
      const int j = i * kSelDecodeThreads + threadIdx.x;
      if (key[i] == 0) continue;
      const float f = unkey32(key[i]);
      if (score_above(f, t, bound)) {
        ++sure;
        atomicOr(&kept[j >> 5], 1u << (j & 31));
      } else if (score_near(f, t, bound)) {
        who[atomicAdd(&nears, 1)] = j;
      }
    }
    need -= cta_sum(sure, part, turn);
    const int near = nears;
    if (near > need) {
      // exact scores, then each one's rank (better score, or lower block)
      double q64[D / 32];
      exact_query<D>(a, q64, head, n);
      for (int i = warp_id(); i < near; i += WARPS) {
        double x = exact_score<D>(a, q64, head, who[i]);
        if (x != x) x = -INFINITY;
        if (lane_id() == 0) exact[i] = x;
      }
      __syncthreads();
    }
    for (int i = threadIdx.x; i < near; i += kSelDecodeThreads) {
      const int j = who[i];
      int better = 0;
      if (near > need)
        for (int o = 0; o < near; ++o) better += exact[o] > exact[i] || (exact[o] == exact[i] && who[o] < j);
      if (near <= need || better < need) atomicOr(&kept[j >> 5], 1u << (j & 31));
    }
  }
  __syncthreads();
  if (warp_id() == 0) {
    int32_t *out = a.sel + (static_cast<int64_t>(head) * a.Nq + n) * a.topk;
    const int words = (a.nblk + 31) / 32;
    int at = 0;
    for (int w0 = 0; w0 < words; w0 += 32) {
      const int w = w0 + lane_id();
      uint32_t u = w < words ? kept[w] : 0u;
      int pre = __popc(u);
      const int own = pre;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, pre, o);
        if (static_cast<int>(lane_id()) >= o) pre += x;
      }
      int p = at + pre - own;
      for (; u; u &= u - 1) out[p++] = w * 32 + __ffs(u) - 1;
      at += __shfl_sync(0xffffffffu, pre, 31);
    }
    for (int i = at + lane_id(); i < a.topk; i += 32) out[i] = -1;
  }
}

}  // namespace svg
